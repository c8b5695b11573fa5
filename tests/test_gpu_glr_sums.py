"""drate of a long sequence whose terms cancel to one run in 16,385."""
import numpy as np
import pytest
import torch

import glr_sums as sums
from helpers import host, need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B", [1, 3])
def test_a_sum_that_cancels(B, dt):
    sdm = need_gpu()
    T, D = sums.TOKENS, sums.CHANNELS
    x, r, g, rate = sums.constants()
    x, r, g = (torch.from_numpy(v).to(dt).cuda().expand(1, T, D).contiguous() for v in (x, r, g))
    dy = torch.ones((1, T, D), dtype=dt, device="cuda")
    dy[:, sums.PLUS:] = -1
    x, r, g, dy = (v.expand(B, T, D).contiguous() for v in (x, r, g, dy))
    rate = torch.from_numpy(rate).float().cuda()
    reset, zero = torch.ones((B, T), dtype=torch.uint8, device="cuda"), torch.zeros((B, D), device="cuda")
    carry = torch.zeros((B, -(-T // 8), D), device="cuda")      # not used: every token resets
    drate = sdm.glr_scan_backward(zero, x, r, g, rate, carry, dy, reset=reset)[3]
    value, bound = sums.want()
    # B sequences: B times it, each within its bound, and the additions of the second launch
    off = np.abs(host(drate).astype(np.float64) - B * value)
    assert np.all(off <= B * bound + (B - 1) * sums.E * B * value), np.max(off / (B * bound))
