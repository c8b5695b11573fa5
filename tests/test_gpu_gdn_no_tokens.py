"""Sequences without a token hand their state, and its gradient, on bit for bit."""
import pytest
import torch

from helpers import need_gpu
from test_gpu_gdn_train import Case

pytestmark = pytest.mark.gpu

ODD = [float("inf"), -float("inf"), float("nan"), 3.4028234e38, -3.4e38, 1e-45, -1.17549435e-38, 0.0, -0.0, 1.0 / 3]


@pytest.mark.parametrize("dims,lens", [((2, 0, 1, 2, 24, 40), None), ((3, 70, 1, 2, 128, 48), [0, 70, 0]), ((2, 70, 20, 20, 32, 128), [0, 3]),
                                       ((2, 70, 40, 40, 36, 116), [0, 64])], ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_bits(dims, lens, in_place):
    sdm = need_gpu()
    c = Case(*dims, seed=3, lens=lens)
    still = [b for b in range(dims[0]) if lens is None or lens[b] == 0]
    for t in (c.S0, c.dS):
        for i, v in enumerate(ODD):
            t[still, :, i, ::i + 1] = v
    x, m = [*c.layout(c.q, c.k, c.v), *c.gates()], c.masks()
    S, dS = c.S0.cuda(), c.dS.cuda()
    ST, d0 = (S, dS) if in_place else (torch.empty_like(S), torch.empty_like(dS))
    _, saved = sdm.gdn_train(S, *x, **m, state_out=None if in_place else ST)
    sdm.gdn_backward(dS, *x, saved, c.dy.cuda(), **m, dstate_out=None if in_place else d0)
    for got, want in ((ST, c.S0), (d0, c.dS)):
        assert torch.equal(got[still].view(torch.int32).cpu(), want[still].view(torch.int32))
