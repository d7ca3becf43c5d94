"""Paged cache and rotary entry points without a GPU: frequencies against the oracle's, and every
host-side refusal (no call here reaches the device: pointers are never dereferenced)."""
import ctypes
import math

import pytest
import torch

import learned_kv_cache_dckv_b200 as D
import oracle.cache as OC
from learned_kv_cache_dckv_b200 import build as B

FAKE = 0x10000  # 16- and 256-byte aligned


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return D.lib()


@pytest.mark.parametrize("rotary", [2, 16, 96, 256])
@pytest.mark.parametrize("kind", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                  dict(scaling="parts", factor=8.0, original_len=8192, low=1.0, high=32.0)])
def test_rope_frequencies(rotary, kind):
    if kind.get("scaling") == "ntk" and rotary == 2:
        with pytest.raises(D.DckvError):
            D.rope_spec(rotary, **kind)
        return
    s = D.rope_spec(rotary, base=5e5, magnitude=1.25, **kind)
    want = OC.rope_freq(rotary, base=5e5, **kind)
    assert s.rotary_dim == rotary and s.magnitude == 1.25
    # a few fp64 roundings of numbers below 1 (pow, products) on either side
    assert max(abs(a - b) / b for a, b in zip(s.freq, want)) < 64 * 2.0 ** -53
    assert all(f == 0.0 for f in s.freq[rotary // 2:])


@pytest.mark.parametrize("bad", [dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=258), dict(layout="other"),
                                 dict(scaling="other"), dict(base=1.0), dict(base=math.inf), dict(magnitude=0.0),
                                 dict(magnitude=math.nan), dict(scaling="linear", factor=0.0),
                                 dict(scaling="parts", factor=2.0), dict(scaling="parts", factor=2.0, original_len=4096,
                                                                         low=2.0, high=2.0)])
def test_rope_spec_refusals(bad):
    args = dict(rotary_dim=64)
    args.update(bad)
    with pytest.raises(D.DckvError) as e:
        D.rope_spec(**args)
    assert e.value.code == D.DCKV_EINVAL


def _rope(**kw):
    a = dict(spec=D.rope_spec(64), mode=0, device=0, dtype=0, x=FAKE, xt=512, xh=256, out=2 * FAKE, ot=512, oh=256, n=4,
             heads=2, dim=256, pos=FAKE)
    a.update(kw)
    spec = None if a["spec"] is None else ctypes.byref(a["spec"])
    args = D._RopeArgs(a["x"], a["out"], a["xt"], a["xh"], a["ot"], a["oh"], a["n"], a["heads"], a["dim"], a["pos"],
                       a["dtype"], a["device"])
    return D.lib().dckv_rope(spec, a["mode"], ctypes.byref(args), None)


@pytest.mark.parametrize("bad", [dict(spec=None), dict(x=None), dict(out=None), dict(pos=None), dict(mode=3),
                                 dict(device=-1), dict(dtype=3), dict(x=FAKE + 1), dict(pos=FAKE + 2), dict(n=-1),
                                 dict(heads=0), dict(dim=62), dict(xt=-512), dict(ot=0), dict(out=FAKE + 64),
                                 dict(out=FAKE, ot=1024), dict(xt=1 << 40)])
def test_rope_refusals(bad):
    assert _rope(**bad) == D.DCKV_EINVAL


def test_rope_spec_by_hand_is_checked():
    s = D.rope_spec(64)
    s.freq[3] = math.nan
    assert _rope(spec=s) == D.DCKV_EINVAL
    s = D.rope_spec(64)
    s.rotary_dim = 1000
    assert _rope(spec=s) == D.DCKV_EINVAL


def test_nothing_to_do_needs_no_device():
    assert _rope(n=0) == D.DCKV_OK
    assert _append(dict(n_tokens=0)) == D.DCKV_OK
    assert _attend(dict(n_tokens=0)) == D.DCKV_OK


def _pool(**kw):
    a = dict(k=FAKE, v=FAKE, device=0, dtype=0, n_layers=6, n_kv_heads=2, head_dim=256, page_size=64, n_pages=10,
             k_layer_stride=10 * 64 * 512, k_page_stride=64 * 512, k_row_stride=512, k_head_stride=256,
             v_layer_stride=10 * 64 * 512, v_page_stride=64 * 512, v_row_stride=512, v_head_stride=256)
    a.update(kw)
    return D.KvPool(*[a[n] for n, _ in D.KvPool._fields_])


def _batch(**kw):
    a = dict(batch=2, max_new=4, max_pages=5, reserved=0, offsets=FAKE, kv_lens=FAKE, page_table=FAKE, table_stride=5)
    a.update(kw)
    return D.CacheBatch(*[a[n] for n, _ in D.CacheBatch._fields_])


def _append(args=(), pool=(), batch=(), rope=True, status=FAKE):
    a = dict(k=FAKE, v=FAKE, k_layer_stride=4096, k_token_stride=512, k_head_stride=256, v_layer_stride=4096,
             v_token_stride=512, v_head_stride=256, q=FAKE, q_out=2 * FAKE, q_token_stride=2048, q_head_stride=256,
             q_out_token_stride=2048, q_out_head_stride=256, n_tokens=8, n_q_heads=8, reserved=0, positions=None)
    a.update(dict(args))
    s = D._AppendArgs(*[a[n] for n, _ in D._AppendArgs._fields_])
    spec = ctypes.byref(D.rope_spec(256)) if rope else None
    return D.lib().dckv_cache_append(ctypes.byref(_pool(**dict(pool))), ctypes.byref(_batch(**dict(batch))), spec,
                                     ctypes.byref(s), status, None)


def _attend(args=(), pool=(), batch=(), ws=FAKE, ws_bytes=1 << 40, status=FAKE):
    a = dict(q=FAKE, out=2 * FAKE, lse=None, q_token_stride=2048, q_head_stride=256, out_token_stride=2048,
             out_head_stride=256, n_tokens=8, n_q_heads=8, layer=0, causal=1, scale=0.0625)
    a.update(dict(args))
    s = D._AttentionArgs(*[a[n] for n, _ in D._AttentionArgs._fields_])
    return D.lib().dckv_attention(ctypes.byref(_pool(**dict(pool))), ctypes.byref(_batch(**dict(batch))),
                                  ctypes.byref(s), status, ws, ws_bytes, None)


BAD_POOL = [dict(k=None), dict(v=FAKE + 8), dict(device=64), dict(dtype=2), dict(head_dim=96), dict(page_size=8),
            dict(page_size=24), dict(page_size=1 << 17), dict(n_layers=0), dict(n_kv_heads=0), dict(n_pages=0),
            dict(n_pages=1 << 31), dict(k_row_stride=516), dict(v_page_stride=0), dict(k_head_stride=-256)]
BAD_BATCH = [dict(batch=0), dict(batch=65537), dict(max_new=0), dict(max_pages=0), dict(reserved=1), dict(offsets=None),
             dict(kv_lens=FAKE + 2), dict(page_table=None), dict(table_stride=4)]


@pytest.mark.parametrize("bad", BAD_POOL)
def test_pool_refusals(bad):
    assert _append(pool=bad) == D.DCKV_EINVAL
    assert _attend(pool=bad) == D.DCKV_EINVAL
    p, b = _pool(**bad), _batch()
    assert D.lib().dckv_cache_rows(ctypes.byref(p), ctypes.byref(b), None, FAKE, 6144, 4, None, FAKE, None) == D.DCKV_EINVAL
    assert D.lib().dckv_attention_workspace_bytes(ctypes.byref(p), ctypes.byref(b), 8) == 0


@pytest.mark.parametrize("bad", BAD_BATCH)
def test_batch_refusals(bad):
    assert _append(batch=bad) == D.DCKV_EINVAL
    assert _attend(batch=bad) == D.DCKV_EINVAL
    p, b = _pool(), _batch(**bad)
    assert D.lib().dckv_cache_rows(ctypes.byref(p), ctypes.byref(b), None, FAKE, 6144, 4, None, FAKE, None) == D.DCKV_EINVAL
    assert D.lib().dckv_attention_workspace_bytes(ctypes.byref(p), ctypes.byref(b), 8) == 0


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=FAKE + 2), dict(n_tokens=-1), dict(n_tokens=1 << 31),
                                 dict(k_token_stride=500), dict(v_layer_stride=0), dict(positions=FAKE + 1),
                                 dict(q_out=None), dict(q=FAKE + 8), dict(n_q_heads=0), dict(q_head_stride=4),
                                 dict(q_out=FAKE + 512), dict(reserved=1)])
def test_append_refusals(bad):
    assert _append(bad) == D.DCKV_EINVAL


def test_append_needs_a_rotation_for_q_and_a_status():
    assert _append(rope=False) == D.DCKV_EINVAL
    assert _append(status=None) == D.DCKV_EINVAL
    assert _append(pool=dict(head_dim=128)) == D.DCKV_EINVAL  # rotary_dim 256


@pytest.mark.parametrize("bad", [dict(q=None), dict(out=FAKE + 4), dict(lse=FAKE + 2), dict(n_tokens=-1),
                                 dict(n_q_heads=7), dict(n_q_heads=0), dict(layer=6), dict(layer=-1), dict(causal=2),
                                 dict(scale=0.0), dict(scale=math.nan), dict(scale=-1.0), dict(q_token_stride=4),
                                 dict(out_head_stride=0), dict(out=FAKE), dict(out=FAKE + 1024)])
def test_attention_refusals(bad):
    assert _attend(bad) == D.DCKV_EINVAL


def test_attention_workspace_refusals():
    need = D.lib().dckv_attention_workspace_bytes(ctypes.byref(_pool()), ctypes.byref(_batch()), 8)
    assert need > 0
    assert _attend(ws=None) == D.DCKV_EINVAL
    assert _attend(ws=FAKE + 16) == D.DCKV_EINVAL
    assert _attend(status=None) == D.DCKV_EINVAL
    assert _attend(ws_bytes=need - 1) == D.DCKV_ECAPACITY
    assert D.lib().dckv_attention_workspace_bytes(ctypes.byref(_pool()), ctypes.byref(_batch()), 7) == 0


def test_rows_refusals():
    p, b, L = ctypes.byref(_pool()), ctypes.byref(_batch()), D.lib()
    assert L.dckv_cache_rows(p, b, None, None, 6144, 4, None, FAKE, None) == D.DCKV_EINVAL
    assert L.dckv_cache_rows(p, b, None, FAKE + 8, 6144, 4, None, FAKE, None) == D.DCKV_EINVAL
    assert L.dckv_cache_rows(p, b, None, FAKE, 6136, 4, None, FAKE, None) == D.DCKV_EINVAL
    assert L.dckv_cache_rows(p, b, None, FAKE, 6144, -1, None, FAKE, None) == D.DCKV_EINVAL
    assert L.dckv_cache_rows(p, b, None, FAKE, 6144, 4, None, None, None) == D.DCKV_EINVAL
    assert L.dckv_cache_rows(p, b, None, FAKE, 6144, 0, None, FAKE, None) == D.DCKV_OK


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 2, 64)
    with pytest.raises(D.DckvError):
        D.dckv_rope(D.rope_spec(64), x, torch.zeros(4, dtype=torch.int32), x)
    with pytest.raises(D.DckvError):
        D.kv_pool(torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16))
    with pytest.raises(D.DckvError):
        D.cache_batch(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                      torch.zeros(2, 4, dtype=torch.int32), 1)


@pytest.mark.parametrize("magnitude", [1e39, 1e-39, 1e300, 1e-300, 2.0 ** 127, 2.0 ** -127])
def test_rope_magnitude_that_fp32_does_not_hold(magnitude):
    """The kernels multiply by m and 1 / m in fp32: infinity would make NaN of a 0, and 0 everything 0."""
    with pytest.raises(D.DckvError) as e:
        D.rope_spec(64, magnitude=magnitude)
    assert e.value.code == D.DCKV_EINVAL
    spec = D.rope_spec(64)
    spec.magnitude = magnitude
    assert all(_rope(spec=spec, mode=m) == D.DCKV_EINVAL for m in D.ROPE_MODES.values())


@pytest.mark.parametrize("magnitude", [2.0 ** 126, 2.0 ** -126, 1.0, 0.8])
def test_rope_magnitude_that_fp32_holds(magnitude):
    assert D.rope_spec(64, magnitude=magnitude).magnitude == magnitude
