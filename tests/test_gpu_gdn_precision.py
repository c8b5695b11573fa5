"""gdn_train and gdn_backward as exact as 32-bit sums make them, over more chunks
than the chains have stages, at each number of column tiles a CTA.

Tolerances.  What is not exact in bf16 enters the tensor cores in three parts, all
24 bits of it.  A product cuts its sum off by at most 2^-24 of the largest partial
sum, so a result with n leading products behind it is at most n 2^-24 off:
- the states: 8 products with the keys, 4 with the triangle, 4 of the update, and
  what the chunks before left, which the decays (at most e^-0.6 a chunk) shrink:
  below 16 * 2.3 * 2^-24 < 2^-18; terms of either sign stay below half of it: 2^-19
  in the 2-norm.
- dbeta: a sum over the columns of products of two such: 2^-18.
- dlog_alpha: sums with up to 48 products behind them, times another: 2^-17.
- y, dq, dk, dv: half a step of bf16 at the value, and at most 84 products on
  partial sums of up to four times the sums' root mean square: 84 * 4 * 2^-24 < 2^-15.
A decay's exponential is 2^-22 of itself off, twice in a product of two: below these."""
import pytest
import torch

import gdn_reference as ref
from helpers import need_gpu
from test_gpu_gdn_train import Case, close32

pytestmark = pytest.mark.gpu


def half_step(x):
    """Half of the distance between neighbouring bf16 at |x|: 8 bits of significand."""
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=1e-30))) - 8)


def rounded(got, want, what):
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape and bool(torch.isfinite(got).all()), what
    for h in range(want.shape[2]):
        w = want[:, :, h]
        # want may lie just below a power of two that got was rounded up to: the step above it then
        step = torch.maximum(half_step(w), half_step(got[:, :, h]))
        off = (got[:, :, h] - w).abs() - step - 2.0 ** -15 * w.square().mean().sqrt()
        assert bool((off <= 1e-30).all()), f"{what} of head {h}: {float(off.max()):.3e} over"


def compare(sdm, c):
    (y, ST), (d0, dq, dk, dv, dla, dbeta) = c.run(sdm)
    f, b = c.reference()
    for h in range(c.dims[3]):
        close32(ST[:, h], f[1][:, h], f"state of head {h}", 2.0 ** -19)
        close32(d0[:, h], b[0][:, h], f"dstate of head {h}", 2.0 ** -19)
        close32(dbeta[..., h], b[5][..., h], f"dbeta of head {h}", 2.0 ** -18)
        close32(dla[..., h], b[4][..., h], f"dlog_alpha of head {h}", 2.0 ** -17)
    for got, want, what in ((y, f[0], "y"), (dq, b[1], "dq"), (dk, b[2], "dk"), (dv, b[3], "dv")):
        rounded(got, want, what)
    sdm.sdm_check()


# one, two and four tiles of 16 columns a CTA; rows by tensor copies and by the helping warps
@pytest.mark.parametrize("dims", [(1, 700, 2, 4, 128, 128), (2, 450, 1, 1, 100, 72), (1, 330, 20, 20, 32, 128),
                                  (1, 330, 4, 40, 32, 128), (1, 330, 40, 40, 36, 116)], ids=str)
@pytest.mark.parametrize("reset", [0.0, 0.01])
def test_many_chunks(dims, reset):
    compare(need_gpu(), Case(*dims, seed=sum(dims), reset=reset, decay=0.5))


@pytest.mark.parametrize("decay", [0.01, 3.0])
def test_heads_that_remember_and_forget(decay):
    compare(need_gpu(), Case(2, 400, 2, 2, 64, 48, seed=3, decay=decay))


def test_lengths_over_many_chunks():
    compare(need_gpu(), Case(4, 390, 2, 4, 128, 64, seed=4, lens=[390, 321, 0, 257], reset=0.01, decay=0.5))


def test_y_of_a_state_that_cancels():
    """Queries at right angles to what the state holds most of: y is far smaller than the products it is summed from."""
    sdm = need_gpu()
    c = Case(1, 64, 1, 1, 64, 32, seed=5, decay=0.01)
    c.beta[:] = 0.0
    c.la[:] = 0.0
    c.q[:] = 0.0
    c.q[..., 0], c.q[..., 1] = 1.0, -1.0
    c.S0[:, :, 1] = c.S0[:, :, 0] * (1 + 2.0 ** -12)
    y, _ = sdm.gdn_train(c.S0.cuda(), *c.layout(c.q, c.k, c.v), *c.gates())
    want = ref.forward(c.S0, c.q, c.k, c.v, c.la, c.beta)[0]
    # the state's rounding aside (it is an input), 24 bits of each product: 2 * 2^-24 of the larger one
    off = (y.cpu().double() - want).abs() - half_step(want) - 2.0 ** -22 * c.S0.abs().amax().double()
    assert bool((off <= 0).all()), float(off.max())


@pytest.mark.parametrize("total", [-1.0, -20.0, -80.0])
def test_a_chunks_decay_alone(total):
    """Nothing written: the state at the end is the decays' product times the one at the start.  The exponential is 2^-22
    of itself off and the product rounded once, 2^-24, whatever the decays sum up to; so is the gradient that comes back."""
    sdm = need_gpu()
    c = Case(1, 64, 64, 64, 16, 16, seed=6)
    g = torch.Generator().manual_seed(7)
    c.k[:] = 0.0
    c.q[:] = 0.0
    c.la = total / 64 * (0.5 + torch.rand((1, 64, 64), generator=g))
    (_, ST), (d0, *_) = c.run(sdm)
    keep = torch.exp(c.la.double().sum(1))[0, :, None, None]
    # at e^-80 = 2^-115 small entries pass the end of the normal numbers, where steps are absolute: 2^-149 in fp32, so a
    # rounding is up to 2^-150 off; the gradient is held as bf16 parts, whose steps end at 2^-133, so up to 2^-134
    for got, start, least in ((ST, c.S0, 2.0 ** -150), (d0, c.dS, 2.0 ** -134)):
        want = keep * start[0].double()
        assert bool(((got[0].cpu().double() - want).abs() <= (2.0 ** -22 + 2.0 ** -24) * want.abs() + least).all())
