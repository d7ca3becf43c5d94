"""Attention over the pages where its kernels treat rows apart: queries that hold NaN, fp16 weights
far below a row's largest, and pages that a whole key tile fits in.  Against oracle/cache.py (fp64);
tolerances as in test_gpu_cache.py."""
import pytest
import torch

import oracle.cache as OC
from test_gpu_cache import BF16, EXP_ERR, FP16, Paged, attend, check_attention, normal, u, within

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ NaN in queries
@pytest.mark.parametrize("dim,new,length", [(64, 1, 70), (128, 1, 2500), (256, 1, 40), (256, 1, 9000), (64, 40, 90),
                                            (128, 40, 3500), (256, 70, 200), (256, 40, 6000), (64, 150, 20000)])
def test_attention_keeps_nan(dim, new, length):
    """A row whose query holds NaN gives NaN, in out and in lse (-infinity there means that it saw no
    slot), whether its slots are split or not; every other row is as without it."""
    c = Paged(301, [length, 33], 1, 2, dim, 32)
    q = normal(7, new + 1, 8, dim)
    _, out, lse = attend(c, [new, 1], 8, q=q)
    bad = q.clone()
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    for t, h, d in ((0, 1, 3), (new - 1, 6, dim - 1), (new // 2, 2, slice(None)), (new, 7, 0)):
        bad[t, h, d] = float("nan")
        hit[t, h] = True
    _, out2, lse2 = attend(c, [new, 1], 8, q=bad)
    assert bool(out2[hit].isnan().all()) and bool(lse2[hit].isnan().all())
    assert torch.equal(out2[~hit], out[~hit]) and torch.equal(lse2[~hit], lse[~hit])


@pytest.mark.parametrize("dim,new", [(256, 3), (64, 40)])
def test_attention_nan_that_sees_nothing(dim, new):
    c = Paged(303, [1], 1, 1, dim, 16)  # only the last of the new tokens sees a slot
    q = normal(8, new, 2, dim)
    q[0] = float("nan")
    _, out, lse = attend(c, [new], 2, q=q)
    assert bool((out[:-1] == 0).all()) and bool((lse[:-1] == -float("inf")).all())
    assert bool(out[-1].isfinite().all()) and bool(lse[-1].isfinite().all())


# ------------------------------------------------------------------ fp16 weights below its normal range
@pytest.mark.parametrize("dim,group", [(64, 2), (128, 12), (256, 8), (64, 20), (128, 20), (256, 20)])
def test_attention_fp16_small_weights(dim, group):
    """One key of each sequence scores 17 above all others (weights of e^-17 = 2^-24.5), and only the
    others' values are not 0.  A weight w of the row's largest is held as fp16(w 2^h) with h >= 7: off
    by u(fp16) relative where that is a normal number, by 2^-25 - h <= 2^-32 absolute below; the second
    adds sum |v| 2^-32 at most.  (In a step of 2^-24 each of these weights would be off by 44%.)"""
    count, length = 150, 1200
    c = Paged(305, [length] * count, 1, 1, dim, 16, dtype=FP16)
    c.k[:] = 0
    c.v.uniform_(2.0, 6.0)
    first = torch.tensor([t[0] for t in c.tables], device="cuda")
    c.k[0, first, 0, 0, 0] = 17.0
    c.v[0, first, 0] = 0.0
    q = torch.zeros(count, group, dim, device="cuda", dtype=FP16)
    q[..., 0] = 1.0
    news = [1] * count
    _, out, lse = attend(c, news, group, q=q, scale=1.0)
    some = 8  # sequences that the definition is worked out for; they are alike but for their values
    want, want_lse, mass, reach = OC.attention(q[:some], c.k[0], c.v[0], news[:some], c.lens[:some], c.tables[:some], 1.0,
                                               True)
    ds = reach * (dim + 8) * 2.0 ** -23
    rel = (u(FP16) + 2.2 * ds + (length + 64) * 2.0 ** -23 + EXP_ERR)[..., None]
    within(out[:some], want, want.abs() * u(FP16) + mass * rel + length * 6.0 * 2.0 ** -32, "out")
    within(lse[:some], want_lse, ds + EXP_ERR + (length + 64) * 2.0 ** -23 + want_lse.abs() * 2.0 ** -22, "lse")


# ------------------------------------------------------------------ pages of a key tile and more
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype,order,page", [(BF16, "token", 128), (FP16, "head", 128), (BF16, "head", 256),
                                              (FP16, "token", 384)])
@pytest.mark.parametrize("group,causal", [(3, True), (8, False)])
def test_attention_large_pages(dim, dtype, order, page, group, causal):
    """Lengths of 1, 127, 128, 129 and 255 beyond whole pages: one box holds a tile's values, and up to
    127 of its rows behind the last slot hold NaN."""
    lens = [1, 127, 128, 129, 255, page + 1, page + 127, 2 * page + 128, 2 * page + 129, page + 255]
    news = [1, 127, 40, 129, 0, 33, 1, 64, 9, 100]
    c = Paged(307, lens, 1, 2, dim, page, order, dtype)
    check_attention(c, news, 2 * group, causal, pad=1)
    check_attention(c, [1] * len(lens), 2 * group, causal)  # single tokens


@pytest.mark.parametrize("dim,group", [(64, 5), (128, 3), (256, 4)])
@pytest.mark.parametrize("page", [128, 256])
def test_attention_large_pages_many_tiles_per_block(dim, group, page):
    lens, news = [1577, 1416, 926, 2099, 1820, 700, 1501], [77, 33, 43, 31, 21, 129 // group, 0]
    c = Paged(309, lens, 1, 4, dim, page)
    check_attention(c, news, 4 * group)
