"""PagedCache without a GPU: its tensors sit on the host and the library's calls are recorded, so
nothing here reaches a device.  What the class refuses, and what it keeps when it refuses."""
import ctypes
import gc
import weakref

import numpy as np
import pytest
import torch

import learned_kv_cache_dckv_b200 as D
from learned_kv_cache_dckv_b200 import build as B

HOST = torch.device("cpu")


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return D.lib()


class Codec:
    """Stands in for D.Codec: counts the calls, gives decoded prompts of zeros."""

    def __init__(self, device=HOST):
        self.device, self.calls = device, []

    def decode(self, blob, blob_bytes, token_ids, seq_offsets, k_out=None, v_out=None, stream=None):
        self.calls.append("decode")
        n = int(np.asarray(seq_offsets)[-1])
        return [torch.zeros(6, n, 2, 256, dtype=torch.bfloat16) for _ in range(2)]

    def encode(self, rows, token_ids, seq_offsets, blob=None, stream=None):
        self.calls.append(("encode", tuple(rows.shape), rows.dtype))
        return torch.zeros(16, dtype=torch.uint8)


@pytest.fixture
def host(monkeypatch):
    """PagedCache(...) on the host; .calls has the library's calls: (name, arguments, keywords)."""
    calls = []
    real = torch.device
    monkeypatch.setattr(D, "_on", lambda device, name, t: t.stride())
    monkeypatch.setattr(D, "_int32_on", lambda device, name, t: t.data_ptr())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    for name in ("dckv_cache_append", "dckv_cache_rows", "dckv_attention"):
        monkeypatch.setattr(D, name, lambda *a, _n=name, **kw: calls.append((_n, a, kw)))

    def make(n_pages=8, page_size=16, **kw):
        with monkeypatch.context() as m:
            m.setattr(torch, "device", lambda *a: HOST if a[0] == "cuda" else real(*a))
            c = D.PagedCache(n_pages, page_size, **kw)
        c.calls = calls
        return c

    return make


def offsets(*lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)


def tokens(n):
    return torch.zeros(n, dtype=torch.int32)


def keys(cache, n, heads=None):
    return torch.zeros(cache.pool.n_layers, n, heads or cache.pool.n_kv_heads, cache.pool.head_dim, dtype=cache.k.dtype)


def extended(cache, *counts):
    seqs = [cache.add() for _ in counts]
    return seqs, cache.extend(seqs, counts)


# ------------------------------------------------------------------ the codec's shape and type
OTHER = [dict(n_layers=1), dict(n_kv_heads=4), dict(head_dim=128), dict(dtype=torch.float16)]


@pytest.mark.parametrize("kw", OTHER)
def test_store_refuses_a_cache_that_is_not_the_codecs(host, kw):
    """The encoder reads 12,288 bytes per row whatever tensor it is given: rows of another cache
    would be read out of their bounds."""
    cache, codec = host(**kw), Codec()
    seqs, _ = extended(cache, 20)
    with pytest.raises(D.DckvError) as e:
        cache.store(codec, seqs, tokens(20))
    assert e.value.code == D.DCKV_EINVAL and codec.calls == []


@pytest.mark.parametrize("kw", OTHER)
def test_restore_refuses_a_cache_that_is_not_the_codecs(host, kw):
    cache, codec = host(**kw), Codec()
    with pytest.raises(D.DckvError) as e:
        cache.restore(codec, None, 0, tokens(20), offsets(20))
    assert e.value.code == D.DCKV_EINVAL and codec.calls == []
    assert len(cache._free) == 8 and cache._len == {}


def test_store_and_restore_refuse_another_device(host):
    cache, codec = host(), Codec(torch.device("meta"))
    seqs, _ = extended(cache, 20)
    with pytest.raises(D.DckvError):
        cache.store(codec, seqs, tokens(20))
    with pytest.raises(D.DckvError):
        cache.restore(codec, None, 0, tokens(20), offsets(20))
    assert codec.calls == []


def test_restore_and_store_pass_the_codecs_shape(host):
    cache, codec = host(), Codec()
    seqs = cache.restore(codec, None, 0, tokens(53), offsets(20, 33))
    assert [cache.length(s) for s in seqs] == [20, 33] and len(cache._free) == 8 - 2 - 3
    _, offs = cache.store(codec, seqs, tokens(53))
    assert codec.calls == ["decode", ("encode", (53, 6144), torch.bfloat16)] and offs.tolist() == [0, 20, 53]


# ------------------------------------------------------------------ token ids
BAD_TOKENS = [tokens(19), tokens(20).long(), tokens(40)[::2], torch.zeros(20, dtype=torch.int32, device="meta")]


@pytest.mark.parametrize("ids", BAD_TOKENS, ids=["short", "int64", "strided", "elsewhere"])
def test_restore_and_store_refuse_token_ids_that_do_not_fit(host, ids):
    """The codec reads one int32 per token from the address that it is given."""
    cache, codec = host(), Codec()
    seqs, _ = extended(cache, 20)
    with pytest.raises(D.DckvError):
        cache.store(codec, seqs, ids)
    with pytest.raises(D.DckvError):
        cache.restore(codec, None, 0, ids, offsets(20))
    assert codec.calls == [] and len(cache._len) == 1


def test_store_counts_every_token_of_a_sequence(host):
    """Tokens appended behind the prompt count by default: the prompt's ids alone are too few."""
    cache, codec = host(), Codec()
    seqs = cache.restore(codec, None, 0, tokens(20), offsets(20))
    cache.append(cache.extend(seqs, [1]), keys(cache, 1), keys(cache, 1))
    with pytest.raises(D.DckvError):
        cache.store(codec, seqs, tokens(20))
    cache.store(codec, seqs, tokens(20), [20])
    cache.store(codec, seqs, tokens(21))
    cache.store(codec, seqs, None)  # a codec without mean models takes none


# ------------------------------------------------------------------ keys that are not rotated at their slots
def test_rows_refuses_keys_appended_with_positions_of_their_own(host):
    cache, codec = host(), Codec()
    a, b = seqs = cache.restore(codec, None, 0, tokens(30), offsets(20, 10))
    cache.append(cache.extend([a], [3]), keys(cache, 3), keys(cache, 3), positions=tokens(3))
    cache.append(cache.extend([b], [3]), keys(cache, 3), keys(cache, 3))
    for call in (lambda: cache.rows(seqs), lambda: cache.rows([a], [21]), lambda: cache.store(codec, [a], tokens(23))):
        with pytest.raises(D.DckvError) as e:
            call()
        assert e.value.code == D.DCKV_EINVAL
    assert codec.calls == ["decode"]
    cache.rows(seqs, [20, 13])  # the slots before them are as they were
    where = torch.arange(36, dtype=torch.int32)
    cache.rows(seqs, positions=where)  # told where, it passes that on
    assert cache.calls[-1][0] == "dckv_cache_rows" and cache.calls[-1][2]["positions"] is where
    cache.store(codec, seqs, tokens(36), positions=where)
    assert cache.calls[-1][2]["positions"] is where and codec.calls[-1][1] == (36, 6144)


def test_rows_refuses_keys_appended_as_they_come(host):
    cache = host()
    (a, b), batch = extended(cache, 5, 0)
    cache.append(batch, keys(cache, 5), keys(cache, 5), rotate=False)
    with pytest.raises(D.DckvError):
        cache.rows([a])
    cache.append(cache.extend([a, b], [2, 2]), keys(cache, 4), keys(cache, 4))
    with pytest.raises(D.DckvError):
        cache.rows([a, b])
    cache.rows([b])
    cache.drop(a)
    c, batch = extended(cache, 4)
    cache.append(batch, keys(cache, 4), keys(cache, 4))
    cache.rows(c)


def test_an_append_that_is_refused_marks_nothing(host, monkeypatch):
    cache = host()
    (a,), batch = extended(cache, 5)
    with monkeypatch.context() as m:
        m.setattr(D, "dckv_cache_append", lambda *_, **__: D._bad("refused"))
        with pytest.raises(D.DckvError):
            cache.append(batch, keys(cache, 5), keys(cache, 5), rotate=False)
    cache.append(batch, keys(cache, 5), keys(cache, 5))
    cache.rows([a])


def test_a_batch_from_elsewhere_marks_every_sequence(host):
    """cache_batch's own batches name pages, not sequences."""
    cache = host()
    (a,), batch = extended(cache, 5)
    cache.append(D.cache_batch(*batch.tensors, 5), keys(cache, 5), keys(cache, 5), positions=tokens(5))
    with pytest.raises(D.DckvError):
        cache.rows([a])


# ------------------------------------------------------------------ restore takes all or nothing
@pytest.mark.parametrize("rope", [dict(rotary_dim=64), dict(rotary_dim=256, base=1e6),
                                  dict(rotary_dim=256, layout="interleaved"), dict(rotary_dim=256, magnitude=1.5),
                                  dict(rotary_dim=256, scaling="linear", factor=2.0)])
def test_restore_refuses_a_cache_with_another_rotation(host, rope):
    """The decoder rotates by the codec's own rotation; the cache would append, attend and rotate
    back by another."""
    cache, codec = host(rope=D.rope_spec(**rope)), Codec()
    with pytest.raises(D.DckvError) as e:
        cache.restore(codec, None, 0, tokens(20), offsets(20))
    assert e.value.code == D.DCKV_EINVAL and codec.calls == [] and cache._len == {}


def test_restore_takes_the_codecs_rotation_however_it_was_made(host):
    spec = D.rope_spec(256)
    same = D.RopeSpec(256, 0, 1.0, (ctypes.c_double * 128)(*spec.freq))
    for rope in (None, spec, same):
        cache = host(rope=rope)
        assert [cache.length(s) for s in cache.restore(Codec(), None, 0, tokens(20), offsets(20))] == [20]


@pytest.mark.parametrize("error", [D.DckvError(D.DCKV_ECUDA, "launch"), RuntimeError("out of memory")])
@pytest.mark.parametrize("where", ["dckv_cache_append", "cache_batch"])
def test_restore_gives_its_pages_back_when_a_call_fails(host, monkeypatch, where, error):
    cache = host()

    def fail(*a, **kw):
        raise error

    with monkeypatch.context() as m:
        m.setattr(D, where, fail)
        with pytest.raises(type(error)):
            cache.restore(Codec(), None, 0, tokens(53), offsets(20, 33))
    assert cache._len == {} and cache._pages == {} and sorted(cache._free) == list(range(8))
    assert [cache.length(s) for s in cache.restore(Codec(), None, 0, tokens(53), offsets(20, 33))] == [20, 33]


def test_restore_without_room_takes_nothing(host):
    cache, codec = host(n_pages=4), Codec()
    with pytest.raises(D.DckvError) as e:
        cache.restore(codec, None, 0, tokens(53), offsets(20, 33))
    assert e.value.code == D.DCKV_ECAPACITY and cache._len == {} and sorted(cache._free) == list(range(4))


def test_extend_takes_nothing_when_its_batch_fails(host, monkeypatch):
    cache = host()
    a, b = cache.add(), cache.add()
    cache.extend([a], [20])
    before = {s: list(p) for s, p in cache._pages.items()}, dict(cache._len), list(cache._free)

    def fail(*args):
        raise RuntimeError("out of memory")

    with monkeypatch.context() as m:
        m.setattr(D, "cache_batch", fail)
        with pytest.raises(RuntimeError):
            cache.extend([a, b], [20, 17])
    assert (cache._pages, cache._len, cache._free) == before


# ------------------------------------------------------------------ counts that the host can check
@pytest.mark.parametrize("counts", [[21, 5], [20, -1], [20], [20, 5, 1]])
def test_rows_and_store_refuse_counts_that_the_sequences_do_not_have(host, counts):
    """Rows past a sequence's length would be left as the allocation had them."""
    cache, codec = host(), Codec()
    seqs, _ = extended(cache, 20, 5)
    for call in (lambda: cache.rows(seqs, counts), lambda: cache.store(codec, seqs, tokens(64), counts)):
        with pytest.raises(D.DckvError) as e:
            call()
        assert e.value.code == D.DCKV_EINVAL
    assert codec.calls == [] and cache.calls == []


def test_rows_store_and_restore_refuse_no_sequences(host):
    cache, codec = host(), Codec()
    for call in (lambda: cache.rows([]), lambda: cache.store(codec, [], tokens(0)),
                 lambda: cache.restore(codec, None, 0, tokens(0), offsets())):
        with pytest.raises(D.DckvError):
            call()
    assert codec.calls == []


def test_rows_takes_parts_of_sequences(host):
    cache = host()
    seqs, _ = extended(cache, 20, 5, 0)
    for counts, want in ((None, [0, 20, 25, 25]), ([0, 5, 0], [0, 0, 5, 5]), ([20, 1, 0], [0, 20, 21, 21])):
        rows, offs = cache.rows(seqs, counts)
        assert offs.tolist() == want and rows.shape == (want[-1], 6144)


# ------------------------------------------------------------------ lifetimes
def test_descriptors_do_not_outlive_their_last_reference(host):
    """A pool's pages and a batch's arrays go with it, not with a later collection of cycles."""
    cache = host()
    seqs, batch = extended(cache, 5)
    gone = [weakref.ref(t) for t in (cache.k, cache.v, *batch.tensors)]
    assert all(r() is not None for r in gone)
    gc.collect()
    gc.disable()
    try:
        del batch
        assert all(r() is None for r in gone[2:])
        del cache
        assert all(r() is None for r in gone)
    finally:
        gc.enable()


def test_a_larger_call_leaves_the_workspace_of_captured_ones(host, monkeypatch):
    """A captured graph writes the workspace of its capture on every replay, so that memory must stay
    the cache's when another call needs more."""
    cache = host()
    (a,), batch = extended(cache, 5)
    q = torch.zeros(5, 8, 256, dtype=torch.bfloat16)
    used = []
    monkeypatch.setattr(D, "dckv_attention", lambda *args, **kw: used.append(args[6]))
    for need in (1000, 5000, 1000, 9000, 5000):
        monkeypatch.setattr(D, "dckv_attention_workspace_bytes", lambda *args, n=need: n)
        cache.attend(0, batch, q)
        assert used[-1].numel() >= need
    at = [t.data_ptr() for t in used]
    alive = {i: weakref.ref(t) for i, t in enumerate(used)}
    used.clear()
    gc.collect()
    assert all(r() is not None and r().data_ptr() == at[i] for i, r in alive.items())


# ------------------------------------------------------------------ layer by layer
def test_append_takes_one_layer(host):
    cache = host(n_layers=3)
    _, batch = extended(cache, 5)
    k = torch.zeros(5, 2, 256, dtype=torch.bfloat16)
    for layer in (0, 2):
        cache.append(batch, k, k, layer=layer)
        pool = cache.calls[-1][1][0]
        assert pool.kv_shape == (1, 2, 256) and pool.n_pages == 8
        assert pool.k == cache.k[layer].data_ptr() and pool.v == cache.v[layer].data_ptr()
    cache.append(batch, keys(cache, 5), keys(cache, 5))
    assert cache.calls[-1][1][0] is cache.pool


@pytest.mark.parametrize("layer", [-1, 3])
def test_append_refuses_a_layer_that_is_not_there(host, layer):
    cache = host(n_layers=3)
    _, batch = extended(cache, 5)
    k = torch.zeros(5, 2, 256, dtype=torch.bfloat16)
    with pytest.raises(D.DckvError) as e:
        cache.append(batch, k, k, layer=layer)
    assert e.value.code == D.DCKV_EINVAL and cache.calls == []
