"""Attention over the pages where its kernels treat rows apart: queries that hold NaN."""
import pytest
import torch

from test_gpu_cache import Paged, attend, normal

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
