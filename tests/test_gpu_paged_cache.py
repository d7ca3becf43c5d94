"""PagedCache and the calls behind it on a GPU, against oracle/cache.py (fp64).  Tolerances as in
test_gpu_cache.py; a row that was rotated on its way in and back on its way out has both passes'
errors, the first one's turned (a pair's |a| + |b| grows by at most 2 in the turn)."""
import pytest
import torch

import learned_kv_cache_dckv_b200 as D
import oracle.cache as OC
from test_gpu_cache import BF16, FP16, Paged, ints, normal, rope_tol, status, u, within

pytestmark = pytest.mark.gpu


def back_and_forth(x, dtype=BF16):
    """Tolerance of keys x [n, heads, dim] rotated (half layout, whole head, magnitude 1) into
    `dtype` and back: the forward pass rounds |y| <= |a| + |b| and errs by 8e-7 (|a| + |b|); the
    inverse turns those errors of a pair into at most their sum, and adds its own, on inputs of
    |y_a| + |y_b| <= 2 (|a| + |b|)."""
    half = x.shape[-1] // 2
    pair = (x[..., :half].double().abs() + x[..., half:].double().abs()).repeat(1, 1, 2)
    first = 2 * pair * (u(dtype) + 8e-7)
    return first + (x.double().abs() + first) * u(dtype) + 2 * pair * 8e-7


# ------------------------------------------------------------------ rows of keys at positions of their own
@pytest.mark.parametrize("dtype,layers,heads,dim,layout", [(BF16, 6, 2, 256, "half"), (FP16, 1, 3, 64, "interleaved")])
def test_rows_at_given_positions(dtype, layers, heads, dim, layout):
    lens, news = [40, 3, 20], [33, 0, 20]
    c = Paged(201, lens, layers, heads, dim, 16, "token", dtype)
    n, st = sum(news), status()
    pos = torch.randint(0, 1 << 20, (n,), generator=torch.Generator().manual_seed(1)).int().cuda()
    rows = torch.empty(n, layers * 2 * heads * dim, device="cuda", dtype=dtype)
    D.dckv_cache_rows(c.pool, c.batch(news), rows, st, rope=D.rope_spec(dim, layout=layout, magnitude=1.5), positions=pos)
    assert int(st) == 0
    got, at = rows.view(n, layers, 2, heads, dim), 0
    for b, new in enumerate(news):
        pages, r = [t.cuda() for t in OC.slots(c.tables[b], new, 16)]
        for l in range(layers if new else 0):
            want, size = OC.rope(c.k[l, pages, r], pos[at: at + new], OC.rope_freq(dim), layout, "inverse", 1.5)
            within(got[at: at + new, l, 0], want, rope_tol(want, size, dtype))
            assert torch.equal(got[at: at + new, l, 1], c.v[l, pages, r])
        at += new


def test_paged_cache_gives_back_rows_at_their_positions():
    """Tokens at their slots, then tokens at positions of their own: rows come back pre-RoPE when it
    is told the positions, and not otherwise."""
    cache = D.PagedCache(8, page_size=32)
    a, b = cache.add(), cache.add()
    k, v = normal(1, 6, 50, 2, 256), normal(2, 6, 50, 2, 256)
    cache.append(cache.extend([a, b], [30, 20]), k, v)
    k2, v2 = normal(3, 6, 7, 2, 256), normal(4, 6, 7, 2, 256)
    own = ints(*range(1000, 7000, 1000), 5)
    cache.append(cache.extend([a], [7]), k2, v2, positions=own)
    with pytest.raises(D.DckvError):
        cache.rows([a, b])
    slots = lambda n: torch.arange(n, device="cuda", dtype=torch.int32)
    for rows, offsets in (cache.rows([a, b], positions=torch.cat([slots(30), own, slots(20)])), cache.rows([a, b], [30, 20])):
        r = rows.view(-1, 6, 2, 2, 256)
        at = int(offsets[1])
        for l in range(6):
            want_k = torch.cat([k[l, :30], k2[l], k[l, 30:]]) if at == 37 else k[l]
            want_v = torch.cat([v[l, :30], v2[l], v[l, 30:]]) if at == 37 else v[l]
            within(r[:, l, 0], want_k.double(), back_and_forth(want_k))
            assert torch.equal(r[:, l, 1], want_v)
    assert int(cache.status) == 0


# ------------------------------------------------------------------ a model's step
@pytest.mark.parametrize("dtype,heads,dim", [(BF16, 2, 256), (FP16, 1, 64)])
def test_append_layer_by_layer(dtype, heads, dim):
    """Layer l + 1's keys come out of layer l's attention: append and attend in turn.  The pages and
    outputs are those of keys appended at once."""
    L, group = 4, 4
    caches = [D.PagedCache(12, 32, L, heads, dim, dtype) for _ in range(2)]
    seqs = [[c.add(), c.add()] for c in caches]
    mix = normal(1, L, heads * group * dim, (group + 2) * heads * dim, dtype=dtype, gain=(heads * group * dim) ** -0.5)
    x = normal(2, 45, heads * group * dim, dtype=dtype)
    at = 0
    for counts in ([40, 3], [1, 1]):
        n = sum(counts)
        batches = [c.extend(s, counts) for c, s in zip(caches, seqs)]
        h, kept = x[at: at + n], []
        for l in range(L):
            q, k, v = (h @ mix[l]).view(n, -1, dim).split([group * heads, heads, heads], 1)
            turned = torch.empty_like(q.contiguous())
            caches[0].append(batches[0], k, v, q=q, q_out=turned, layer=l)
            out = caches[0].attend(l, batches[0], turned)
            kept.append((k, v, turned, out))
            h = out.flatten(1)
        caches[1].append(batches[1], *[torch.stack([s[i] for s in kept]) for i in (0, 1)])
        for l, (_, _, turned, out) in enumerate(kept):
            assert torch.equal(caches[1].attend(l, batches[1], turned), out)
        at += n
    for a, b in zip(*seqs):
        pages, rows = [t.cuda() for t in OC.slots(caches[0]._pages[a], caches[0].length(a), 32)]
        assert caches[0]._pages[a] == caches[1]._pages[b]
        assert torch.equal(caches[0].k[:, pages, rows], caches[1].k[:, pages, rows])
        assert torch.equal(caches[0].v[:, pages, rows], caches[1].v[:, pages, rows])
    assert int(caches[0].status) == 0 and int(caches[1].status) == 0


def test_a_captured_step_outlives_larger_calls():
    """A graph of a single token's step is replayed after a chunk has needed a larger workspace and
    other tensors have taken what memory was free."""
    cache = D.PagedCache(200, page_size=32, n_layers=1)
    a, b = cache.add(), cache.add()
    k, v = normal(1, 1, 5000, 2, 256), normal(2, 1, 5000, 2, 256)
    cache.append(cache.extend([a, b], [4000, 1000]), k, v)
    step = cache.extend([a, b], [1, 1])
    cache.append(step, k[:, :2], v[:, :2])
    q, out = normal(3, 2, 8, 256), torch.empty(2, 8, 256, dtype=BF16, device="cuda")
    want = cache.attend(0, step, q).clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.attend(0, step, q, out=out)
    chunk = cache.extend([b], [64])
    cache.append(chunk, k[:, :64], v[:, :64])
    q2 = normal(4, 64, 8, 256)
    want2 = cache.attend(0, chunk, q2).clone()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    others = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    assert torch.equal(cache.attend(0, chunk, q2), want2)
    assert all(bool((t == 7).all()) for t in others) and int(cache.status) == 0
