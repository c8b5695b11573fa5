"""The gradient of the decay's logarithm, head by head, at weak and strong decays.

Tolerance.  Every term of the sum carries the token's decay.  A term is a product
of at most six factors, each exact to 2^-24 an operation, with a chunk's chain of
at most 2^7 roundings that the decays do not shrink behind it (2^-17, as for the
states); sums have terms of like size and either sign, so the same 2^-17 of the
norm holds for a head's own gradient, whatever the decays of the others are."""
import pytest
import torch

import gdn_reference as ref
from helpers import need_gpu
from test_gpu_gdn_train import Case, check, close32

pytestmark = pytest.mark.gpu


def with_levels(c, levels, seed):
    g = torch.Generator().manual_seed(seed)
    B, T, _, H = c.dims[:4]
    c.la = torch.tensor(levels)[None, None] * (0.75 + 0.5 * torch.rand((B, T, H), generator=g))
    return c


def by_head(sdm, c):
    out = c.run(sdm)
    f, b = c.reference()
    check(c, out, f, b)
    for h in range(c.dims[3]):
        close32(out[1][4][..., h], b[4][..., h], f"dlog_alpha of head {h}", 2.0 ** -17)
    return out


@pytest.mark.parametrize("dims", [(1, 192, 8, 8, 128, 128), (2, 150, 2, 8, 64, 48), (1, 333, 8, 8, 100, 33), (3, 64, 4, 8, 16, 80)], ids=str)
@pytest.mark.parametrize("reset", [0.0, 0.04])
def test_levels(dims, reset):
    sdm = need_gpu()
    by_head(sdm, with_levels(Case(*dims, seed=sum(dims), reset=reset), [-0.01, -0.7, -3.0, -5.0, -8.0, -12.0, -16.0, -20.0], 1))


def test_lengths_and_groups():
    sdm = need_gpu()
    by_head(sdm, with_levels(Case(3, 130, 1, 4, 72, 40, seed=5, lens=[130, 67, 3], reset=0.02), [-1.0, -8.0, -16.0, -30.0], 2))


def test_heads_that_forget_everything():
    """A decay of 0, and ones whose exponential is 0 in 32 bits, have no gradient; the other heads keep theirs."""
    sdm = need_gpu()
    c = with_levels(Case(1, 140, 4, 4, 64, 32, seed=6), [-0.5, 0.0, -300.0, -8.0], 3)
    c.la[..., 1] = float("-inf")
    out = by_head(sdm, c)
    assert bool((out[1][4][..., 1:3] == 0).all())


@pytest.mark.parametrize("at", [1, 31, 32, 33, 63, 64, 100])
def test_one_strong_decay_among_weak_ones(at):
    """The one token's gradient is right by itself: nothing of its neighbours', e^14 times as large, is in it."""
    sdm = need_gpu()
    c = Case(1, 128, 1, 1, 64, 64, seed=7, decay=0.05)
    c.la[:, at] = -14.0
    out = c.run(sdm)
    want = c.reference()[1][4]
    got = out[1][4].cpu().double()
    # the token's terms alone, of either sign: their sizes are those of the reference at a decay of 1 there
    c.la[:, at] = 0.0
    size = float(ref.backward(ref.forward(c.S0, c.q, c.k, c.v, c.la, c.beta), c.dS, c.q, c.k, c.v, c.la, c.beta, c.dy)[4][0].abs().max())
    assert abs(float(got[0, at, 0] - want[0, at, 0])) <= 2.0 ** -14 * size * 2.718281828 ** -14.0
