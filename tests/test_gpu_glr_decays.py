"""The gated linear recurrence where its factors are small: decays far below 1
and gates that are nearly closed, within fp32's error relative to each factor
itself.

Where y = rate sigmoid(r) is above 0.15 the decay is the exponential unit's
own result: relative error 2^-22 for the unit, 2 E y for the two roundings
of its argument, y d_y for y's own error (d_y as in glr_reference.gates).
glr_reference allows an absolute 2^-24 there, which says nothing about a
decay of 1e-6, nor about dr and drate, which are proportional to it."""
import numpy as np
import pytest
import torch

import glr_reference as ref
from helpers import need_gpu
from test_gpu_glr import Case, assert_within

pytestmark = pytest.mark.gpu

E = ref.E
loose = ref.gates


def gates(x, r, g, rate):
    """glr_reference.gates with the decay's bound relative to the decay beyond y = 0.15."""
    sr, sg, a, m, e_a, d_m = loose(x, r, g, rate)
    y = rate * sr
    far = a * (y * (ref.rel_sig(r) + 3 * E) + 2.0 ** -22)
    return sr, sg, a, m, np.where(y > 0.151, far, e_a), d_m


@pytest.fixture(autouse=True)
def relative(monkeypatch):
    monkeypatch.setattr(ref, "gates", gates)


def gradients(c, f):
    """The reference's gradients, drate's bound with the kernel's own depth of
    additions in place of the n that glr_reference counts: 8 tokens of a run, the
    join of the runs and what it lost, 3 more warps, 15 more CTAs, and over
    B sequences a second launch's ceil(B / 32) + 31."""
    b = ref.backward(f, *c.np("dhT", "x", "r", "g", "rate", "dy", "reset", "lens"))
    r, rate = c.np("r", "rate")
    n = max(1, min(c.B * c.T, 4096))
    depth = 8 + 2 + 3 + 15 + (-(-c.B // 32) + 31 if c.B > 1 else 0)
    past = rate * (1 - ref.sig(r))      # dr = past times drate's term of the token
    terms = np.where(past > 0, np.abs(b["dr"]) / np.where(past > 0, past, 1), 0) * c.live()
    b["e_drate"] = b["e_drate"] - (n - depth) * E * (1 - 1e-9) * terms.sum((0, 1))
    return b


def check(sdm, c):
    f = c.forward()
    s = c.h0.clone()
    y, carry = sdm.glr_scan_train(s, *c.args(), **c.kw())
    assert_within(y, f["y"], f["e_y"], c.dt, "y")
    assert_within(s, f["hT"], f["e_hT"], torch.float32, "h_T")
    assert_within(carry, f["before"][:, ::8], f["e_before"][:, ::8], torch.float32, "carry")
    s2 = c.h0.clone()
    assert torch.equal(sdm.glr_scan(s2, *c.args(), **c.kw()), y) and torch.equal(s2, s)
    b = gradients(c, f)
    ds = c.dhT.clone()
    out = sdm.glr_scan_backward(ds, *c.args(), carry, c.dy, **c.kw())
    for k, got in zip(("dx", "dr", "dg"), out):
        assert_within(got, b[k], b["e_" + k], c.dt, k)
    assert_within(out[3], b["drate"], b["e_drate"], torch.float32, "drate")
    assert_within(ds, b["dh0"], b["e_dh0"], torch.float32, "dh_0")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rate", [(0.1, 4.0), (4.0, 20.0), (20.0, 60.0)], ids=["to4", "to20", "to60"])
@pytest.mark.parametrize("B,T,D", [(1, 1, 66), (2, 5, 40), (2, 150, 66), (1, 700, 64)])
def test_strong_decays(B, T, D, rate, dt):
    sdm = need_gpu()
    check(sdm, Case(B, T, D, dt, seed=31, rate=rate))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rate", [(0.1, 4.0), (4.0, 20.0)], ids=["to4", "to20"])
@pytest.mark.parametrize("T", [4, 90])
def test_strong_decays_without_input(T, rate, dt):
    """x = 0 (dropout, padding): y_t is a_t h_{t-1} and nothing else."""
    sdm = need_gpu()
    c = Case(2, T, 66, dt, seed=32, rate=rate)
    c.x.mul_((torch.arange(66, device="cuda") % 3 == 0) & (torch.arange(T, device="cuda")[:, None] % 4 == 3))
    check(sdm, c)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("size", [1.0, 1e30])
@pytest.mark.parametrize("T", [5, 100])
def test_gates_that_are_nearly_closed(T, size, dt):
    """Input gates of e^-44 to e^-86 into an empty state: the input term is all there is."""
    sdm = need_gpu()
    c = Case(2, T, 66, dt, seed=33)
    c.h0.zero_()
    c.g.copy_(-44 - 42 * torch.rand(c.g.shape, generator=torch.Generator().manual_seed(1)))
    c.x.mul_(size)
    f = c.forward()
    s = c.h0.clone()
    y = sdm.glr_scan(s, *c.args())
    assert torch.all(y[c.x != 0].abs() > 0)
    assert_within(y, f["y"], f["e_y"], c.dt, "y")
    assert_within(s, f["hT"], f["e_hT"], torch.float32, "h_T")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_an_infinite_input_at_a_nearly_closed_gate(dt):
    """m sigmoid(-60) is not 0, so an infinite x stays an infinity of its sign."""
    sdm = need_gpu()
    c = Case(1, 40, 64, dt, seed=34)
    c.g[0, 20] = -60.0
    c.x[0, 20, :32], c.x[0, 20, 32:] = float("inf"), -float("inf")
    y = sdm.glr_scan(c.h0.clone(), *c.args())
    assert torch.all(y[0, 20:, :32] == float("inf")) and torch.all(y[0, 20:, 32:] == -float("inf"))
    assert torch.isfinite(y[0, :20]).all()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_recurrence_gates_that_are_nearly_closed(dt):
    """sigmoid(r) down to fp32's smallest normal numbers: m, its root, keeps its digits."""
    sdm = need_gpu()
    c = Case(2, 100, 66, dt, seed=35, rate=(0.5, 0.8))
    c.h0.zero_()
    c.r.copy_(-60 - 26 * torch.rand(c.r.shape, generator=torch.Generator().manual_seed(2)))
    f = c.forward()
    y = sdm.glr_scan(c.h0.clone(), *c.args())
    assert_within(y, f["y"], f["e_y"], c.dt, "y")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_all_gradients_at_extreme_gates(dt):
    """Logits of -1e30 to 1e30 on both gates, in every combination."""
    sdm = need_gpu()
    c = Case(1, 80, 64, dt, seed=10)
    big = torch.tensor([-1e30, -200.0, -60.0, -20.0, 20.0, 60.0, 200.0, 1e30], dtype=c.dt, device="cuda")
    c.r[0, :64] = big.repeat(8)[None].expand(64, 64)
    c.g[0, 8:72] = big.repeat_interleave(8)[None].expand(64, 64)
    check(sdm, c)
