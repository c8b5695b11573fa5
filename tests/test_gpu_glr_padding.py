"""Padded batches whose outputs the calls allocate: the rows behind lens are 0,
whatever the memory held before."""
import pytest
import torch

from helpers import need_gpu
from test_gpu_glr import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_new_outputs_are_zero_behind_the_lengths(T, dt):
    sdm = need_gpu()
    c = Case(4, T, 130, dt, seed=61, lens=[0, T, 1, T - 2])
    behind = (torch.arange(T, device="cuda")[None] >= c.lens[:, None])[..., None].expand(4, T, 130)

    def used_memory():      # what the allocator hands out next held NaN
        torch.cuda.empty_cache()
        held = [torch.full_like(c.x, float("nan")) for _ in range(6)]
        del held

    used_memory()
    y = sdm.glr_scan(c.h0.clone(), *c.args(), **c.kw())
    assert torch.all(y[behind] == 0)
    used_memory()
    y2, carry, ckpt = sdm.glr_scan_train(c.h0.clone(), *c.args(), **c.kw(), keep8=True)
    assert torch.equal(y2, y)
    for saved, kept in (((c.x, c.r, c.g), None), ((None, None, None), ckpt)):
        used_memory()
        *grads, drate = sdm.glr_scan_backward(c.dhT.clone(), *saved, c.rate, carry, c.dy, **c.kw(), ckpt=kept)
        assert all(torch.all(d[behind] == 0) for d in grads) and torch.isfinite(drate).all()
    given = torch.full_like(c.x, 5.0)       # a buffer that is given keeps its rows
    sdm.glr_scan(c.h0.clone(), *c.args(), **c.kw(), y=given)
    assert torch.all(given[behind] == 5.0)
