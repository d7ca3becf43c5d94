"""Rotary positions, the paged cache and attention over it against plain fp64 definitions
(oracle/cache.py), on a GPU.

Tolerances, from arithmetic (u(t) = finfo(t).eps / 2, half a step relative):
  rotation   |out| u(t) for the one rounding, plus (|a| + |b|) m 8e-7 for fp32 arithmetic: the
             reduced angle's rounding to fp32 (pi 2^-24 = 1.9e-7), its fp64 product and reduction
             (|angle| 2^-52, 4.8e-7 at 2^31 radians, below 1e-9 under 10^6), cos and sin (2 ulp,
             1.2e-7) and the two products and their sum and the magnitude's product (4 roundings,
             2.4e-7 of |a| + |b|); the sums stay below 8e-7 for positions up to 2^28.
  attention  a score's error ds: dim products summed in fp32, each partial sum at most reach =
             scale sum |q||k|, truncated or rounded by 2^-23 of it, and a few products and
             subtractions of numbers up to 2 reach: ds = reach (dim + 8) 2^-23.  A weight is off by
             the factor exp(2 ds) (its own score and the normaliser's), by the exponential's own
             error and by its rounding u(t); n weighted values are summed in fp32 (truncated: n
             2^-23), with a few joins.  So |out| u(t) + mass (u(t) + 2.2 ds + (n + 64) 2^-23 + exp
             error), mass = sum w |v|; EXP_ERR bounds the exponential's relative error.  lse: ds +
             EXP_ERR + n 2^-23, plus |lse| 2^-22 for its logarithm, scaling and roundings.
"""
import numpy as np
import pytest
import torch

import dckv_synth as S
import learned_kv_cache_dckv_b200 as D
import oracle.cache as OC

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
EXP_ERR = 2.0 ** -18


def u(t):
    return torch.finfo(t).eps / 2


def normal(seed, *shape, dtype=BF16, gain=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * gain).to(dtype)


def ints(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def within(got, want, tol, what=""):
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    excess = (got.double() - want).abs() - tol
    assert float(excess.max()) <= 0.0, f"{what}: over the tolerance by {float(excess.max()):.3g}"


def rope_tol(out, size, dtype):
    return out.abs() * u(dtype) + size * 8e-7


# ------------------------------------------------------------------ rotation
KINDS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
         dict(scaling="parts", factor=8.0, original_len=8192)]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("mode", ["forward", "gradient", "inverse"])
@pytest.mark.parametrize("n,heads,dim,rotary", [(1, 1, 64, 64), (3, 10, 256, 64), (37, 2, 128, 96), (5, 3, 80, 20),
                                                (4, 2, 7, 6), (129, 1, 256, 256), (6, 2, 66, 2)])
def test_rope(dtype, layout, mode, n, heads, dim, rotary):
    kind = KINDS[(n + heads) % 4] if rotary > 2 else KINDS[0]
    spec = D.rope_spec(rotary, layout=layout, base=5e5, magnitude=1.3, **kind)
    x = normal(n, n, heads, dim, dtype=dtype)
    pos = torch.randint(0, 1 << 20, (n,), generator=torch.Generator().manual_seed(dim)).int().cuda()
    pos[0] = -7  # any int32
    out = torch.full_like(x, float("nan"))
    D.dckv_rope(spec, x, pos, out, mode=mode)
    want, size = OC.rope(x, pos, OC.rope_freq(rotary, base=5e5, **kind), layout, mode, 1.3)
    within(out, want, rope_tol(want, size, dtype))
    assert torch.equal(out[..., rotary:], x[..., rotary:])
    y = x.clone()
    D.dckv_rope(spec, y, pos, y, mode=mode)
    assert torch.equal(out, y)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_rope_strided_and_unaligned(dtype):
    spec = D.rope_spec(32)
    pos = ints(*range(9))
    base = normal(1, 9, 6 * 48 + 1, dtype=dtype)
    x = base[:, 1:].view(9, 6, 48)[:, 1:5]  # an odd first element: no 16-byte vectors
    out = torch.zeros(4, 9, 48, device="cuda", dtype=dtype).transpose(0, 1)
    D.dckv_rope(spec, x, pos, out)
    want, size = OC.rope(x, pos, OC.rope_freq(32))
    within(out, want, rope_tol(want, size, dtype))


def test_rope_gradient_is_the_transpose():
    """<forward(x), y> = <x, gradient(y)>, and the gradient against central differences of the
    forward pass (fp32: differences of a linear map with step h are exact up to its rounding)."""
    spec = D.rope_spec(96, layout="interleaved", base=1e4, magnitude=1.7)
    x, y = normal(2, 11, 3, 128, dtype=FP32), normal(3, 11, 3, 128, dtype=FP32)
    pos = ints(*range(0, 1100, 100))
    fx, gy = torch.empty_like(x), torch.empty_like(y)
    D.dckv_rope(spec, x, pos, fx)
    D.dckv_rope(spec, y, pos, gy, mode="gradient")
    a, b = (fx.double() * y.double()).sum((1, 2)), (x.double() * gy.double()).sum((1, 2))
    size = 2 * 1.7 * (x.double().abs().flatten(1).norm(dim=1) * y.double().abs().flatten(1).norm(dim=1))
    assert ((a - b).abs() <= 2 * size * 1e-6).all()
    d = torch.zeros_like(x)
    d[:, :, 5] = 0.5
    up, down = torch.empty_like(x), torch.empty_like(x)
    D.dckv_rope(spec, x + d, pos, up)
    D.dckv_rope(spec, x - d, pos, down)
    slope = ((up.double() - down.double()) * y.double()).sum(2)
    # x +- d round to fp32 (2^-24 of at most 6), the two passes are off by 8e-7 m (|a| + |b|) each
    assert ((slope - gy[:, :, 5].double()).abs() <= 1.7 * 2 * 12 * 2e-6 * y.double().abs().amax(2)).all()


def test_rope_inverse_returns():
    spec = D.rope_spec(256, magnitude=0.8)
    x, pos = normal(4, 33, 4, 256, dtype=FP32), torch.arange(33, device="cuda", dtype=torch.int32) * 40000
    y, z = torch.empty_like(x), torch.empty_like(x)
    D.dckv_rope(spec, x, pos, y)
    D.dckv_rope(spec, y, pos, z, mode="inverse")
    pair = x.double()[..., :128].abs() + x.double()[..., 128:].abs()
    # both passes' errors, the first one's turned and scaled back by 1 / m
    within(z, x.double(), 2 * 2 * 2 * torch.cat([pair, pair], -1) * 8e-7)


# ------------------------------------------------------------------ the paged cache
class Paged:
    """Pools with every unused slot NaN, pages in scattered order, garbage behind the tables."""

    def __init__(self, seed, lens, layers=1, heads=2, dim=256, page=16, order="token", dtype=BF16, gain=1.0, extra=3):
        self.lens, self.page, self.layers, self.heads, self.dim, self.dtype = lens, page, layers, heads, dim, dtype
        need = [-(-n // page) for n in lens]
        count = sum(need) + extra
        perm = np.random.RandomState(seed).permutation(count).tolist()
        self.tables = []
        for n in need:
            self.tables.append([perm.pop() for _ in range(n)])
        shape = (layers, count, heads, page, dim) if order == "head" else (layers, count, page, heads, dim)
        self.k, self.v = [torch.full(shape, float("nan"), device="cuda", dtype=dtype) for _ in range(2)]
        if order == "head":
            self.k, self.v = self.k.transpose(2, 3), self.v.transpose(2, 3)
        self.pool = D.kv_pool(self.k, self.v)
        for b, n in enumerate(lens):
            pages, rows = [t.cuda() for t in OC.slots(self.tables[b], n, page)]
            for l in range(layers):
                self.k[l, pages, rows] = normal(seed + 7 * b + l, n, heads, dim, dtype=dtype, gain=gain)
                self.v[l, pages, rows] = normal(seed + 7 * b + l + 1000, n, heads, dim, dtype=dtype)

    def batch(self, news, max_new=None, lens=None, pad_columns=2):
        lens = self.lens if lens is None else lens
        width = max(len(t) for t in self.tables) + pad_columns
        table = torch.full((len(lens), width), 0x7fffffff, dtype=torch.int32)  # never a page
        for b, t in enumerate(self.tables):
            table[b, : len(t)] = torch.tensor(t, dtype=torch.int32)
        offs = np.concatenate([[0], np.cumsum(news)])
        return D.cache_batch(ints(*offs.tolist()), ints(*lens), table.cuda(), max_new or max(1, max(news)))


@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("dtype,layers,heads,dim,page,rotary,layout", [
    (BF16, 6, 2, 256, 64, 256, "half"), (FP16, 1, 3, 64, 16, 48, "interleaved"), (BF16, 2, 1, 128, 48, 20, "half")])
def test_append(order, dtype, layers, heads, dim, page, rotary, layout):
    lens, news = [70, 1, 16, 0, 33], [7, 1, 16, 0, 2]
    c = Paged(5, lens, layers, heads, dim, page, order, dtype)
    before_k, before_v = c.k.clone(), c.v.clone()
    n, pad, hq = sum(news), 3, 5
    qkv = normal(9, n + pad, layers * 2 * heads + hq, dim, dtype=dtype)
    k = qkv[:, : layers * heads].unflatten(1, (layers, heads)).transpose(0, 1)
    v = qkv[:, layers * heads: 2 * layers * heads].unflatten(1, (layers, heads)).transpose(0, 1)
    q = qkv[:, 2 * layers * heads:]
    q_out = torch.full((n + pad, hq, dim), 7.0, device="cuda", dtype=dtype)
    spec, st = D.rope_spec(rotary, layout=layout, magnitude=1.1), status()
    D.dckv_cache_append(c.pool, c.batch(news), k, v, st, rope=spec, q=q, q_out=q_out)
    assert int(st) == 0
    freq = OC.rope_freq(rotary)
    want_k, want_v, at = before_k.clone(), before_v.clone(), 0
    touched = torch.zeros(c.k.shape[1:3], dtype=torch.bool, device="cuda")
    for b, (length, new) in enumerate(zip(lens, news)):
        pages, rows = [t.cuda()[length - new:] for t in OC.slots(c.tables[b], length, page)]
        pos = torch.arange(length - new, length, device="cuda")
        touched[pages, rows] = True
        for l in range(layers):
            r, size = OC.rope(k[l, at: at + new], pos, freq, layout, "forward", 1.1)
            if new:
                within(c.k[l, pages, rows], r, rope_tol(r, size, dtype), f"keys {b}")
                assert torch.equal(c.v[l, pages, rows], v[l, at: at + new])
        r, size = OC.rope(q[at: at + new], pos, freq, layout, "forward", 1.1)
        if new:
            within(q_out[at: at + new], r, rope_tol(r, size, dtype), f"queries {b}")
        at += new
    bits = lambda t: t.contiguous().view(torch.int16)
    assert torch.equal(bits(c.k[:, ~touched]), bits(before_k[:, ~touched]))
    assert torch.equal(bits(c.v[:, ~touched]), bits(before_v[:, ~touched]))
    assert bool((q_out[n:] == 7.0).all())  # rows behind the last sequence


def test_append_positions_copy_and_many_sequences():
    """More sequences than one scan of the offsets takes (bisection), own positions, no rotation."""
    B = 700
    lens, news = [1 + b % 3 for b in range(B)], [b % 2 for b in range(B)]
    c = Paged(11, lens, 1, 1, 64, 16)
    n = sum(news)
    k, v, st = normal(1, 1, n, 1, 64), normal(2, 1, n, 1, 64), status()
    pos = torch.arange(n, device="cuda", dtype=torch.int32) * 1000 + 5
    for rope in (None, D.rope_spec(64)):
        D.dckv_cache_append(c.pool, c.batch(news), k, v, st, rope=rope, positions=pos)
        assert int(st) == 0
        pages = torch.tensor([t[0] for t, m in zip(c.tables, news) if m], device="cuda")
        rows = torch.tensor([l - 1 for l, m in zip(lens, news) if m], device="cuda")
        got_k, got_v = c.k[0, pages, rows], c.v[0, pages, rows]
        assert torch.equal(got_v, v[0])
        if rope is None:
            assert torch.equal(got_k, k[0])
        else:
            r, size = OC.rope(k[0], pos, OC.rope_freq(64))
            within(got_k, r, rope_tol(r, size, BF16))


def test_append_flags_what_it_leaves_out():
    c = Paged(3, [20, 20, 20], 1, 2, 64, 16)
    k = normal(1, 1, 6, 2, 64)
    before = c.k.clone()
    ok = c.batch([2, 2, 2])
    cases = []
    for b, col, val in ((0, 1, -1), (1, 1, c.k.shape[1])):  # a page before and behind the pool
        bt = c.batch([2, 2, 2])
        bt.tensors[2][b, col] = val
        cases.append((bt, b))
    bt = c.batch([2, 2, 2], lens=[20, 20, 1])  # more new tokens than slots in use
    cases.append((bt, 2))
    for bt, bad in cases:
        st = status()
        c.k.copy_(before)
        D.dckv_cache_append(c.pool, bt, k, k, st)
        assert int(st) == D.DCKV_ERANGE
        for b in range(3):
            pages, rows = [t.cuda()[18:] for t in OC.slots(c.tables[b], 20, 16)]
            same = torch.equal(c.k[0, pages, rows], k[0, 2 * b: 2 * b + 2])
            assert same == (b != bad)
    st = status()
    D.dckv_cache_append(c.pool, c.batch([2, 2, 2], max_new=1), k, k, st)
    assert int(st) == D.DCKV_ERANGE
    st = status()
    D.dckv_cache_append(c.pool, ok, k, k, st)
    assert int(st) == 0


@pytest.mark.parametrize("dtype,layers,heads,dim,rotary,layout", [(BF16, 6, 2, 256, 256, "half"),
                                                                  (FP16, 2, 3, 64, 20, "interleaved")])
def test_rows(dtype, layers, heads, dim, rotary, layout):
    lens, news = [70, 16, 5, 0, 33], [70, 10, 0, 0, 33]
    c = Paged(21, lens, layers, heads, dim, 48, "head", dtype)
    n, width, st = sum(news), layers * 2 * heads * dim, status()
    wide = torch.full((n + 2, width + 8), 3.0, device="cuda", dtype=dtype)
    rows = wide[:, :width]
    D.dckv_cache_rows(c.pool, c.batch(news), rows, st, rope=D.rope_spec(rotary, layout=layout, magnitude=1.5))
    assert int(st) == 0
    at = 0
    for b, new in enumerate(news):
        pages, r = [t.cuda() for t in OC.slots(c.tables[b], new, 48)]
        got = rows[at: at + new].reshape(new, layers, 2, heads, dim)
        for l in range(layers if new else 0):
            want, size = OC.rope(c.k[l, pages, r], torch.arange(new, device="cuda"), OC.rope_freq(rotary), layout,
                                 "inverse", 1.5)
            within(got[:, l, 0], want, rope_tol(want, size, dtype))
            assert torch.equal(got[:, l, 1], c.v[l, pages, r])
        at += new
    assert bool((wide[n:] == 3.0).all()) and bool((wide[:, width:] == 3.0).all())
    plain = torch.empty(n, width, device="cuda", dtype=dtype)
    D.dckv_cache_rows(c.pool, c.batch(news), plain, st)
    pages, r = [t.cuda() for t in OC.slots(c.tables[0], 70, 48)]
    assert torch.equal(plain[:70].view(70, layers, 2, heads, dim)[:, 0, 0], c.k[0, pages, r])
    D.dckv_cache_rows(c.pool, c.batch([70, 17, 0, 0, 33]), torch.empty(120, width, device="cuda", dtype=dtype), st)
    assert int(st) == D.DCKV_ERANGE  # a slot that is not in use


# ------------------------------------------------------------------ attention
def attend(c, news, hq, causal=True, scale=None, layer=0, pad=0, max_new=None, q=None, lse=True, lens=None, gain=1.0):
    n = sum(news)
    if q is None:
        q = normal(77, n + pad, hq, c.dim, dtype=c.dtype, gain=gain)
    out = torch.full((n + pad, hq, c.dim), 7.0, device="cuda", dtype=c.dtype)
    ls = torch.full((n + pad, hq), 7.0, device="cuda") if lse else None
    bt, st = c.batch(news, max_new, lens), status()
    size = D.dckv_attention_workspace_bytes(c.pool, bt, hq)
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten
    D.dckv_attention(c.pool, layer, bt, q, out, st, ws, scale=scale, causal=causal, lse=ls)
    assert int(st) == 0
    return q, out, ls


def check_attention(c, news, hq, causal=True, scale=None, layer=0, pad=0, max_new=None, gain=1.0):
    q, out, lse = attend(c, news, hq, causal, scale, layer, pad, max_new, gain=gain)
    n = sum(news)
    want, want_lse, mass, reach = OC.attention(q[:n], c.k[layer], c.v[layer], news, c.lens, c.tables,
                                               c.dim ** -0.5 if scale is None else scale, causal)
    ds = reach * (c.dim + 8) * 2.0 ** -23
    m = max(c.lens) + 64
    tol = want.abs() * u(c.dtype) + mass * (u(c.dtype) + 2.2 * ds + m * 2.0 ** -23 + EXP_ERR)[..., None]
    empty = torch.isinf(want_lse)
    if n:
        within(out[:n], want, tol, "out")
        assert bool((out[:n][empty] == 0).all()) and bool((lse[:n][empty] == -float("inf")).all())
        if bool((~empty).any()):
            within(lse[:n][~empty], want_lse[~empty],
                   (ds + EXP_ERR + m * 2.0 ** -23 + want_lse.abs() * 2.0 ** -22)[~empty], "lse")
    assert bool((out[n:] == 7.0).all()) and bool((lse[n:] == 7.0).all())  # rows behind the last sequence
    return q, out, lse


LENS = [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype,order,page", [(BF16, "token", 64), (FP16, "head", 16), (BF16, "head", 48)])
@pytest.mark.parametrize("heads,group", [(2, 4), (1, 16), (3, 1)])
def test_attention_single_tokens(dim, dtype, order, page, heads, group):
    c = Paged(31, LENS, 1, heads, dim, page, order, dtype)
    check_attention(c, [1] * len(LENS), heads * group)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype,order,page", [(BF16, "token", 64), (FP16, "head", 16), (FP16, "token", 80)])
@pytest.mark.parametrize("group,causal", [(1, True), (3, True), (8, False), (17, True)])
def test_attention_chunks(dim, dtype, order, page, group, causal):
    """Ragged chunks: a whole prompt, a chunk after cached tokens, one token, none, an empty cache,
    and more new tokens than cached slots (the first ones see nothing)."""
    lens, news = [90, 300, 129, 64, 0, 20, 140], [90, 37, 1, 0, 3, 33, 128]
    c = Paged(41, lens, 1, 2, dim, page, order, dtype)
    check_attention(c, news, 2 * group, causal, pad=2)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("length,new", [(1500, 2), (1500, 130), (2049, 1), (700, 513)])
def test_attention_long_axis(dim, length, new):
    """Few rows over long caches: the slots are split and the parts joined."""
    c = Paged(51, [length], 1, 1, dim, 32)
    check_attention(c, [new], 2, max_new=new)
    check_attention(c, [new], 2, causal=False)


@pytest.mark.parametrize("dim,dtype,group,page", [(256, BF16, 4, 64), (128, FP16, 3, 16), (64, BF16, 5, 48)])
def test_attention_many_tiles_per_block(dim, dtype, group, page):
    """Enough slots that a block walks several key tiles and several sequences; row counts that
    leave one row, or none, in a block's warps."""
    lens, news = [1577, 1416, 926, 2099, 1820, 700, 1501], [77, 33, 43, 31, 21, 129 // group, 0]
    c = Paged(57, lens, 1, 4, dim, page, "token", dtype)
    check_attention(c, news, 4 * group)
    check_attention(c, [1] * 7, 4 * group)


@pytest.mark.parametrize("count", [33, 400])
@pytest.mark.parametrize("dim,group,new", [(64, 4, 1), (128, 3, 9), (64, 40, 1)])
def test_attention_many_sequences(count, dim, group, new):
    """More units than a warp or a block has lanes to count them; sequences without new tokens or
    slots among them."""
    r = np.random.RandomState(count)
    lens = r.randint(0, 90, count).tolist()
    news = [int(r.randint(0, new + 1)) for _ in range(count)]
    c = Paged(58, lens, 1, 1, dim, 16)
    check_attention(c, news, group, max_new=new, pad=1)


@pytest.mark.parametrize("new", [1, 3])
def test_attention_more_heads_than_rows(new):
    """200 query heads on one KV head: more than a row tile holds."""
    c = Paged(59, [300, 40], 1, 1, 128, 32)
    check_attention(c, [new, new], 200)


def test_cache_beyond_32_bits():
    """Pages whose offsets pass 2^32 bytes and 2^31 elements: append, attention and rows."""
    pages, rows, dim = 300_000, 16, 256
    k = torch.empty(1, pages, rows, 2, dim, dtype=BF16, device="cuda")
    v = torch.empty_like(k)
    c = Paged.__new__(Paged)
    c.__dict__.update(lens=[40, 70], page=rows, layers=1, heads=2, dim=dim, dtype=BF16, k=k, v=v, pool=D.kv_pool(k, v),
                      tables=[[pages - 1, 3, pages - 7], [pages - 2, pages // 2, pages - 3, 0, pages - 4]])
    new_k, new_v, st = normal(1, 1, 110, 2, dim), normal(2, 1, 110, 2, dim), status()
    D.dckv_cache_append(c.pool, c.batch([40, 70]), new_k, new_v, st)
    at = 0
    for table, n in zip(c.tables, c.lens):
        p, r = [t.cuda() for t in OC.slots(table, n, rows)]
        assert torch.equal(k[0, p, r], new_k[0, at: at + n]) and torch.equal(v[0, p, r], new_v[0, at: at + n])
        at += n
    check_attention(c, [1, 1], 8)
    check_attention(c, [40, 33], 8)
    out = torch.empty(110, 2 * 2 * dim, dtype=BF16, device="cuda")
    D.dckv_cache_rows(c.pool, c.batch([40, 70]), out, st)
    assert int(st) == 0
    assert torch.equal(out.view(110, 2, 2, dim), torch.stack([new_k[0], new_v[0]], 1))


@pytest.mark.parametrize("dim,new", [(256, 1), (128, 40), (256, 200)])
def test_attention_large_scores(dim, new):
    """Scores far beyond exp's range (the running maximum moves, weights underflow)."""
    c = Paged(61, [500, 77], 1, 2, dim, 16, gain=12.0)
    check_attention(c, [new, min(new, 77)], 8, gain=6.0)


@pytest.mark.parametrize("dim,new", [(256, 1), (128, 1), (256, 90), (64, 70)])
def test_attention_rising_scores(dim, new):
    """Keys whose scores rise along the cache: every tile moves the running maximum."""
    c = Paged(63, [600], 1, 1, dim, 32)
    q = normal(5, new, 4, dim)
    pages, rows = [t.cuda() for t in OC.slots(c.tables[0], 600, 32)]
    ramp = torch.linspace(-3, 3, 600, device="cuda")[:, None, None]
    c.k[0, pages, rows] = (q.float().mean((0, 1)) * ramp * 20 + c.k[0, pages, rows].float()).to(BF16)
    check_attention_with(c, [new], q)


def check_attention_with(c, news, q, causal=True):
    _, out, lse = attend(c, news, q.shape[1], causal, q=q)
    want, want_lse, mass, reach = OC.attention(q, c.k[0], c.v[0], news, c.lens, c.tables, c.dim ** -0.5, causal)
    ds = reach * (c.dim + 8) * 2.0 ** -23
    m = max(c.lens) + 64
    within(out, want, want.abs() * u(c.dtype) + mass * (u(c.dtype) + 2.2 * ds + m * 2.0 ** -23 + EXP_ERR)[..., None])
    within(lse, want_lse, ds + EXP_ERR + m * 2.0 ** -23 + want_lse.abs() * 2.0 ** -22)


@pytest.mark.parametrize("new", [1, 50])
def test_attention_layers_strides_scale(new):
    """Third of four layers, q and out as slices of wider tensors, an own scale, no lse."""
    c = Paged(71, [200, 50], 4, 2, 128, 16, "head")
    n = 2 * new
    wide = normal(8, n, 11, 128)
    q = wide[:, 2:8]
    out = torch.zeros(6, n, 128, device="cuda", dtype=BF16).transpose(0, 1)
    bt, st = c.batch([new, new]), status()
    ws = torch.empty(D.dckv_attention_workspace_bytes(c.pool, bt, 6), dtype=torch.uint8, device="cuda")
    D.dckv_attention(c.pool, 2, bt, q, out, st, ws, scale=0.3)
    want, _, mass, reach = OC.attention(q, c.k[2], c.v[2], [new, new], c.lens, c.tables, 0.3, True)
    ds = reach * (128 + 8) * 2.0 ** -23
    assert int(st) == 0
    within(out, want, want.abs() * u(BF16) + mass * (u(BF16) + 2.2 * ds + 300 * 2.0 ** -23 + EXP_ERR)[..., None])


@pytest.mark.parametrize("new", [1, 40])
def test_attention_repeats_bit_for_bit(new):
    c = Paged(81, [1000, 333, 64, 2000], 1, 2, 256, 64)
    news = [new] * 4
    q, out, lse = attend(c, news, 8)
    for _ in range(3):
        _, o2, l2 = attend(c, news, 8, q=q)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("dim,new,other", [(64, 40, 64), (64, 40, 1), (256, 20, 30)])
def test_attention_overlapping_calls(dim, new, other):
    """Two calls in flight on two streams over and over: each gives what it gives alone."""
    c = Paged(83, [700, 900, 333], 1, 2, dim, 32)
    jobs = []
    for n, seed in ((new, 1), (other, 2)):
        q = normal(seed, 3 * n, 8, dim)
        bt = c.batch([n] * 3)
        _, want, _ = attend(c, [n] * 3, 8, q=q)
        ws = torch.empty(D.dckv_attention_workspace_bytes(c.pool, bt, 8), dtype=torch.uint8, device="cuda")
        jobs.append((bt, q, want, torch.empty_like(want), status(), ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(50):
        for bt, q, _, got, st, ws, s in jobs:
            D.dckv_attention(c.pool, 0, bt, q, got, st, ws, stream=s)
    torch.cuda.synchronize()
    for _, _, want, got, st, _, _ in jobs:
        assert torch.equal(want, got) and int(st) == 0


@pytest.mark.parametrize("new", [1, 40])
def test_attention_parts_join_by_lse(new):
    """Outputs over two disjoint sets of slots, joined by their lse, give the whole's output."""
    c = Paged(91, [320], 1, 2, 128, 32)
    q, out, lse = attend(c, [new], 8, causal=False)
    parts = []
    for pages in (c.tables[0][:4], c.tables[0][4:]):
        part = Paged.__new__(Paged)
        part.__dict__.update(c.__dict__, lens=[32 * len(pages)], tables=[pages])
        parts.append(attend(part, [new], 8, causal=False, q=q)[1:])
    w = [torch.exp(l.double() - lse.double())[..., None] for _, l in parts]
    joined = sum(o.double() * x for (o, _), x in zip(parts, w))
    mass = c.v[0, torch.tensor(c.tables[0], device="cuda")].abs().amax().double()
    # every |out| <= max |v|; each part is rounded once (u), the weights of P too (u), both sides
    assert float((joined - out.double()).abs().max()) <= float(mass) * (4 * u(BF16) + 1e-3)


def test_attention_flags_ranges():
    c = Paged(101, [100, 100], 1, 2, 64, 16)
    q = normal(1, 4, 4, 64)
    out = torch.empty_like(q)

    def call(bt):
        st = status()
        ws = torch.empty(D.dckv_attention_workspace_bytes(c.pool, bt, 4), dtype=torch.uint8, device="cuda")
        D.dckv_attention(c.pool, 0, bt, q, out, st, ws)
        return int(st)

    assert call(c.batch([2, 2])) == 0
    for value in (-1, c.k.shape[1]):
        bt = c.batch([2, 2])
        bt.tensors[2][1, 3] = value
        assert call(bt) == D.DCKV_ERANGE
    assert call(c.batch([2, 2], lens=[100, 5000])) == D.DCKV_ERANGE  # more slots than the table has
    assert call(c.batch([2, 2], lens=[-1, 100])) == D.DCKV_ERANGE
    assert call(c.batch([2, 2], max_new=1)) == D.DCKV_ERANGE
    assert call(c.batch([2, 2000])) == D.DCKV_ERANGE  # offsets behind q's rows
    bt = c.batch([2, 2])
    bt.tensors[0].copy_(ints(0, -5, 4))
    assert call(bt) == D.DCKV_ERANGE


def test_status_collects():
    """The status word is not cleared by a later call without errors."""
    c = Paged(103, [40], 1, 2, 64, 16)
    st, k = status(), normal(1, 1, 2, 2, 64)
    bad = c.batch([2], lens=[1])
    D.dckv_cache_append(c.pool, bad, k, k, st)
    D.dckv_cache_append(c.pool, c.batch([2]), k, k, st)
    assert int(st) == D.DCKV_ERANGE


# ------------------------------------------------------------------ as they are used together
@pytest.mark.parametrize("new", [1, 20])
def test_step_in_a_graph(new):
    """Append and attention of a step, captured once and replayed with other tokens and lengths,
    beside a second graph with its own workspace; then the same on a side stream."""
    lens = [200, 90]
    c = Paged(111, lens, 1, 2, 256, 64)
    spec, hq, n = D.rope_spec(256), 8, 2 * new
    bt = c.batch([new, new])
    x = [normal(i, n, hq + 4, 256) for i in range(3)]
    steps = []
    for _ in range(2):
        s = dict(x=x[0].clone(), q=torch.empty(n, hq, 256, device="cuda", dtype=BF16), st=status(),
                 ws=torch.empty(D.dckv_attention_workspace_bytes(c.pool, bt, hq), dtype=torch.uint8, device="cuda"))
        s["out"] = torch.empty_like(s["q"])
        steps.append(s)

    def step(s):
        D.dckv_cache_append(c.pool, bt, s["x"][:, hq: hq + 2], s["x"][:, hq + 2:], s["st"], rope=spec,
                            q=s["x"][:, :hq], q_out=s["q"])
        D.dckv_attention(c.pool, 0, bt, s["q"], s["out"], s["st"], s["ws"])

    def expect(s, now):
        _, out, _ = attend(c, [new, new], hq, q=s["q"], lens=now)
        assert torch.equal(out, s["out"]) and int(s["st"]) == 0

    step(steps[0])
    torch.cuda.synchronize()
    graphs = []
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(s)
        graphs.append(g)
    for i, now in enumerate(([200, 90], [150, 33], [180, 64])):
        bt.tensors[1].copy_(ints(*now))
        for s, g in zip(steps, graphs):
            s["x"].copy_(x[i])
            g.replay()
            torch.cuda.synchronize()
            expect(s, now)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        steps[0]["out"].zero_()
        step(steps[0])
    torch.cuda.current_stream().wait_stream(side)
    expect(steps[0], now)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("new", [1, 40])
def test_inputs_from_another_stream(new, captured):
    """Queries, keys and values come late from another stream, by events, and the outputs go back to
    it; eager and in a captured graph that forks and joins.  The calls' chained launches must wait."""
    c = Paged(117, [900, 300], 1, 2, 128, 32)
    spec, n, hq = D.rope_spec(128), 2 * new, 8
    bt, st = c.batch([new, new]), status()
    ws = torch.empty(D.dckv_attention_workspace_bytes(c.pool, bt, hq), dtype=torch.uint8, device="cuda")
    fresh = normal(5, n, hq + 4, 128)
    x, q = torch.zeros_like(fresh), torch.zeros(n, hq, 128, device="cuda", dtype=BF16)
    out, copy = torch.zeros_like(q), torch.zeros_like(q)
    where = torch.cat([torch.arange(900 - new, 900), torch.arange(300 - new, 300)]).int().cuda()
    load = torch.randn(2048, 2048, device="cuda")
    side = torch.cuda.Stream()

    def work():
        y = load
        for _ in range(20):  # some milliseconds before the inputs are there
            y = (y @ load).clamp_(-1, 1)
        x.copy_(fresh + 0 * y[0, 0].to(BF16))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            D.dckv_cache_append(c.pool, bt, x[:, hq: hq + 2], x[:, hq + 2:], st, rope=spec, q=x[:, :hq], q_out=q)
            D.dckv_attention(c.pool, 0, bt, q, out, st, ws)
        torch.cuda.current_stream().wait_stream(side)
        copy.copy_(out)

    work()
    torch.cuda.synchronize()
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            work()
    for i in range(3):
        fresh.copy_(normal(20 + i, n, hq + 4, 128))
        x.fill_(float("nan"))
        out.fill_(float("nan"))
        g.replay() if captured else work()
        torch.cuda.synchronize()
        q2 = torch.empty_like(q)
        D.dckv_rope(spec, fresh[:, :hq], where, q2)
        assert torch.equal(q, q2)
        _, out2, _ = attend(c, [new, new], hq, q=q2)
        assert torch.equal(copy, out2) and int(st) == 0


def test_two_streams_at_once():
    """Two calls in flight on two streams, each with its own workspace."""
    c = Paged(113, [3000, 2500], 1, 2, 256, 64)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    jobs = []
    for new in (1, 64):
        q, out, lse = attend(c, [new, new], 8)
        bt = c.batch([new, new])
        ws = torch.empty(D.dckv_attention_workspace_bytes(c.pool, bt, 8), dtype=torch.uint8, device="cuda")
        jobs.append((bt, q, out, torch.empty_like(out), status(), ws))
    torch.cuda.synchronize()
    for _ in range(20):
        for (bt, q, _, got, st, ws), s in zip(jobs, streams):
            D.dckv_attention(c.pool, 0, bt, q, got, st, ws, stream=s)
    torch.cuda.synchronize()
    for _, _, want, got, st, _ in jobs:
        assert torch.equal(want, got) and int(st) == 0


def test_codec_and_cache_together(src, codec_literal):
    """A prompt's way: rows -> encode -> blob -> restore into pages -> steps of new tokens with
    attention -> the prompt's rows from the pages -> encode again."""
    gc = D.Codec(D.upload_params(codec_literal), 0)
    x, tok, offs = S.batch(src, [200, 141], seeds=[0, 1], device="cuda")
    blob = gc.encode(x, tok, offs)
    torch.cuda.synchronize()
    size = int(gc.blob_size.item())
    cache = D.PagedCache(16, page_size=48)
    seqs = cache.restore(gc, blob, size, tok, offs)
    k, v = gc.decode(blob, size, tok, offs)
    assert int(gc.status.item()) == D.DCKV_OK and [cache.length(s) for s in seqs] == [200, 141]
    for counts in ([1, 1], [7, 0], [1, 1]):
        n = sum(counts)
        bt = cache.extend(seqs, counts)
        new_k, new_v, q = normal(1, 6, n, 2, 256), normal(2, 6, n, 2, 256), normal(3, n, 8, 256)
        q_rot = torch.empty_like(q)
        cache.append(bt, new_k, new_v, q=q, q_out=q_rot)
        for layer in (0, 5):
            lse = torch.empty(n, 8, device="cuda")
            out = cache.attend(layer, bt, q_rot, lse=lse)
            lens = [cache.length(s) for s in seqs]
            tables = [cache._pages[s] for s in seqs]
            want, want_lse, mass, reach = OC.attention(q_rot, cache.k[layer], cache.v[layer], counts, lens, tables,
                                                       1 / 16, True)
            ds = reach * 264 * 2.0 ** -23
            within(out, want, want.abs() * u(BF16) + mass * (u(BF16) + 2.2 * ds + 300 * 2.0 ** -23 + EXP_ERR)[..., None])
    assert int(cache.status.item()) == 0
    rows, offsets = cache.rows(seqs, [200, 141])
    assert offsets.tolist() == list(offs)
    r = rows.view(-1, 6, 2, 2, 256)
    pos = torch.cat([torch.arange(200), torch.arange(141)]).cuda()
    for l in range(6):
        assert torch.equal(r[:, l, 1], v[l])
        want, pair = OC.rope(k[l], pos, OC.rope_freq(256), "half", "inverse")
        within(r[:, l, 0], want, rope_tol(want, pair, BF16))
    blob2, offsets = cache.store(gc, seqs, tok, [200, 141])
    torch.cuda.synchronize()
    assert int(gc.status.item()) == D.DCKV_OK and int(gc.blob_size.item()) > 0
    k2, v2 = gc.decode(blob2, int(gc.blob_size.item()), tok, offsets)
    torch.cuda.synchronize()
    assert int(gc.status.item()) == D.DCKV_OK
    free = len(cache._free)
    with pytest.raises(D.DckvError) as e:
        cache.extend(seqs, [48 * 16, 0])
    assert e.value.code == D.DCKV_ECAPACITY and len(cache._free) == free
    cache.drop(seqs[0])
    cache.drop(seqs[1])
    assert len(cache._free) == 16
    gc.close()


def test_append_matches_the_decoders_rotation(src, codec_literal):
    """Pre-RoPE keys appended with the codec's rotation are the decoder's on kept rows: each lies
    within rope_tol of the exact rotation, so they are within twice that of one another."""
    gc = D.Codec(D.upload_params(codec_literal), 0)
    x, tok, offs = S.batch(src, [120], seeds=[3], device="cuda")  # shorter than 132: every row kept
    blob = gc.encode(x, tok, offs)
    torch.cuda.synchronize()
    k, v = gc.decode(blob, int(gc.blob_size.item()), tok, offs)
    cache = D.PagedCache(4, page_size=32)
    s = cache.add()
    bt = cache.extend([s], [120])
    r = x.view(120, 6, 2, 2, 256).permute(1, 2, 0, 3, 4)
    cache.append(bt, r[:, 0], r[:, 1])
    pages, rows = [t.cuda() for t in OC.slots(cache._pages[s], 120, 32)]
    assert torch.equal(cache.v[:, pages, rows], v)
    for l in range(6):
        want, size = OC.rope(r[l, 0], torch.arange(120, device="cuda"), OC.rope_freq(256))
        within(cache.k[l, pages, rows], want, rope_tol(want, size, BF16))
        within(cache.k[l, pages, rows], k[l].double(), 2 * rope_tol(want, size, BF16))
    gc.close()
