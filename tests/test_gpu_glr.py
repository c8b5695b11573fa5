"""GPU parity of the gated linear recurrence (glr_scan, glr_scan_train,
glr_scan_backward) against the fp64 token-by-token reference, element by
element within its running bound of fp32's error, plus half a step of the
output's type."""
import numpy as np
import pytest
import torch

import glr_reference as ref
from helpers import host, need_gpu

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def assert_within(got, want, bound, dtype, what):
    """|got - want| <= bound + half a step of dtype relative to the value
    (which itself may be off by the bound), and an absolute floor where fp32
    flushes to zero."""
    got = got.detach().float().cpu().numpy().astype(np.float64)
    half = torch.finfo(dtype).eps / 2
    tol = bound + half * (np.abs(want) + bound) + 1e-36
    off = np.abs(got - want)
    assert got.shape == want.shape, what
    assert np.all(off <= tol), f"{what}: {np.max(off / tol):.3f} of the tolerance at {np.unravel_index(np.argmax(off / tol), off.shape)}"


class Case:
    def __init__(self, B, T, D, dt="bf16", seed=0, fused=False, reset=0.0, lens=None, spread=1.0, rate=(0.005, 0.8)):
        gen = torch.Generator().manual_seed(seed)
        self.dt, self.B, self.T, self.D = DTYPES[dt], B, T, D
        n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
        if fused:
            p = (spread * n(B, T, 3 * D + 1)).to(self.dt).cuda()
            self.x, self.r, self.g = p[..., 1:D + 1], p[..., D + 1:2 * D + 1], p[..., 2 * D + 1:]
        else:
            self.x, self.r, self.g = ((spread * n(B, T, D)).to(self.dt).cuda() for _ in range(3))
        self.rate = (rate[0] + (rate[1] - rate[0]) * torch.rand(D, generator=gen)).cuda()
        self.h0 = n(B, D).cuda()
        self.reset = (torch.rand((B, T), generator=gen) < reset).to(torch.uint8).cuda() if reset else None
        self.lens = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.dy, self.dhT = n(B, T, D).to(self.dt).cuda(), n(B, D).cuda()

    def np(self, *names):
        out = []
        for k in names:
            v = getattr(self, k)
            out.append(None if v is None else v.float().cpu().numpy().astype(np.float64) if v.is_floating_point()
                       else v.cpu().numpy())
        return out

    def forward(self):
        return ref.forward(*self.np("h0", "x", "r", "g", "rate", "reset", "lens"))

    def live(self):
        lens = np.full(self.B, self.T) if self.lens is None else np.clip(host(self.lens), 0, self.T)
        return (np.arange(self.T)[None] < lens[:, None])[..., None]

    def args(self):
        return self.x, self.r, self.g, self.rate

    def kw(self):
        return dict(reset=self.reset, lens=self.lens)


# one run and less, a run and one, one CTA, several, clusters; a channel to several blocks; steps of up to 8 tokens
SHAPES = [(1, 1, 1), (2, 1, 64), (3, 2, 66), (1, 7, 3), (2, 8, 65), (2, 9, 130), (1, 63, 64), (1, 64, 32), (2, 65, 67),
          (1, 513, 129), (2, 1100, 192), (5, 300, 63), (1, 4099, 64), (70, 3, 256), (1, 2048, 1920)]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_forward(B, T, D, dt):
    sdm = need_gpu()
    c = Case(B, T, D, dt, seed=B * 1000 + T)
    f = c.forward()
    y0, hT = torch.full_like(c.x, 7.0), torch.empty_like(c.h0)
    y = sdm.glr_scan(c.h0, *c.args(), y=y0, state_out=hT)
    assert y is y0
    assert_within(y, f["y"], f["e_y"], c.dt, "y")
    assert_within(hT, f["hT"], f["e_hT"], torch.float32, "h_T")
    # in place, and the training forward: the same bits
    s = c.h0.clone()
    y2 = sdm.glr_scan(s, *c.args())
    assert torch.equal(s, hT) and torch.equal(y2, y)
    s = c.h0.clone()
    y3, carry = sdm.glr_scan_train(s, *c.args())
    assert torch.equal(s, hT) and torch.equal(y3, y)
    assert_within(carry, f["before"][:, ::8], f["e_before"][:, ::8], torch.float32, "carry")


MASKED = [dict(B=3, T=70, D=65, lens=[0, 70, 1]), dict(B=4, T=200, D=64, lens=[64, 63, 65, 128], reset=0.05),
          dict(B=2, T=515, D=130, lens=[512, 8], reset=0.02), dict(B=2, T=90, D=31, reset=1.0),
          dict(B=2, T=1300, D=96, reset=0.003), dict(B=3, T=1, D=40, lens=[1, 0, 1], reset=0.5),
          dict(B=1, T=2600, D=72, lens=[1031], reset=0.01)]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("kw", MASKED, ids=lambda k: f"B{k['B']}T{k['T']}D{k['D']}")
def test_lengths_resets_and_slices(kw, fused, dt):
    """Padded and packed batches, contiguous and as column slices (at an odd
    offset: elements aligned to themselves only); rows behind lens untouched
    in y, the carries, the checkpoints and the gradients."""
    sdm = need_gpu()
    c = Case(**kw, dt=dt, fused=fused, seed=5)
    f = c.forward()
    live = c.live()
    y, s = torch.full((c.B, c.T, c.D), -3.0, dtype=c.dt, device="cuda"), c.h0.clone()
    sdm.glr_scan(s, *c.args(), **c.kw(), y=y)
    assert_within(y, np.where(live, f["y"], -3.0), f["e_y"] * live, c.dt, "y")
    assert_within(s, f["hT"], f["e_hT"], torch.float32, "h_T")
    S = -(-c.T // 8)
    carry = torch.full((c.B, S, c.D), 9.0, device="cuda")
    codes = torch.full((3, c.B, c.T, c.D), 99, dtype=torch.int8, device="cuda")
    exps = torch.full((3, c.B, c.T, -(-c.D // 64)), 77, dtype=torch.uint8, device="cuda")
    y2 = torch.full_like(y, -3.0)
    sdm.glr_scan_train(c.h0.clone(), *c.args(), **c.kw(), y=y2, carry=carry, ckpt=(codes, exps))
    assert torch.equal(y2, y)
    first = live[:, ::8]
    assert_within(carry, np.where(first, f["before"][:, ::8], 9.0), f["e_before"][:, ::8] * first, torch.float32, "carry")
    for i, v in enumerate(c.np("x", "r", "g")):
        q, e = ref.pack8(v)
        assert np.array_equal(host(codes[i]), np.where(live, q, 99))
        assert np.array_equal(host(exps[i]), np.where(live, e, 77))
    # gradients, from the inputs and from the checkpoints
    check_backward(sdm, c, f, carry, None)
    check_backward(sdm, c, f, carry, (codes, exps))


def check_backward(sdm, c, f, carry, ckpt):
    x, r, g = c.np("x", "r", "g")
    if ckpt is not None:
        x, r, g = (ref.unpack8(*ref.pack8(v)) for v in (x, r, g))
    rate, dy, dhT, reset, lens = c.np("rate", "dy", "dhT", "reset", "lens")
    b = ref.backward(f, dhT, x, r, g, rate, dy, reset, lens, seg=8 if ckpt is not None else None)
    live = c.live()
    ds = c.dhT.clone()
    wide = torch.full((c.B, c.T, 3 * c.D + 2), -5.0, dtype=c.dt, device="cuda")     # slices of one buffer
    grads = tuple(wide[..., 1 + i * c.D:1 + (i + 1) * c.D] for i in range(3))
    saved = (None, None, None) if ckpt is not None else (c.x, c.r, c.g)
    out = sdm.glr_scan_backward(ds, *saved, c.rate, carry, c.dy, **c.kw(), ckpt=ckpt, grads=grads)
    for k, got in zip(("dx", "dr", "dg"), out):
        assert_within(got, np.where(live, b[k], -5.0), b["e_" + k] * live, c.dt, k)
    assert torch.all(wide[..., 0] == -5.0) and torch.all(wide[..., -1] == -5.0)
    assert_within(out[3], b["drate"], b["e_drate"], torch.float32, "drate")
    assert_within(ds, b["dh0"], b["e_dh0"], torch.float32, "dh_0")
    # again, into new buffers: the same bits
    ds2 = torch.empty_like(ds)
    out2 = sdm.glr_scan_backward(c.dhT, *saved, c.rate, carry, c.dy, **c.kw(), ckpt=ckpt, dstate_out=ds2)
    mask = torch.from_numpy(live).cuda()
    for p, q in zip(out[:3], out2[:3]):
        assert torch.equal(torch.where(mask, p, 0), torch.where(mask, q, 0))
    assert torch.equal(out[3], out2[3]) and torch.equal(ds, ds2)


@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_backward(B, T, D, dt, keep8):
    sdm = need_gpu()
    c = Case(B, T, D, dt, seed=B * 1000 + T + 1)
    f = c.forward()
    kept = sdm.glr_scan_train(c.h0.clone(), *c.args(), keep8=keep8)
    check_backward(sdm, c, f, kept[1], kept[2] if keep8 else None)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("rate", [(0.0, 0.0), (1e-7, 1e-6), (20.0, 60.0)], ids=["zero", "tiny", "large"])
def test_extreme_decays(rate, dt):
    """No decay at all (the state holds still, and the term with a / m is left
    out), decays next to 1, decays next to 0."""
    sdm = need_gpu()
    c = Case(2, 150, 66, dt, seed=9, rate=rate)
    f = c.forward()
    s = c.h0.clone()
    y, carry = sdm.glr_scan_train(s, *c.args())
    assert_within(y, f["y"], f["e_y"], c.dt, "y")
    assert_within(s, f["hT"], f["e_hT"], torch.float32, "h_T")
    check_backward(sdm, c, f, carry, None)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_extreme_gates(dt):
    """Gate logits far out: sigmoids of 0 and 1 without an infinity or a NaN."""
    sdm = need_gpu()
    c = Case(1, 80, 64, dt, seed=10)
    big = torch.tensor([-1e30, -200.0, -60.0, -20.0, 20.0, 60.0, 200.0, 1e30], dtype=c.dt, device="cuda")
    c.r[0, :64] = big.repeat(8)[None].expand(64, 64)
    c.g[0, 8:72] = big.repeat_interleave(8)[None].expand(64, 64)
    f = c.forward()
    s = c.h0.clone()
    y, carry = sdm.glr_scan_train(s, *c.args())
    assert_within(y, f["y"], f["e_y"] + 1e-17 * np.abs(f["y"]).max(), c.dt, "y")
    out = sdm.glr_scan_backward(c.dhT.clone(), c.x, c.r, c.g, c.rate, carry, c.dy)
    assert all(torch.isfinite(t.float()).all() for t in out)
    b = ref.backward(f, *c.np("dhT", "x", "r", "g", "rate", "dy"))
    for k, got in zip(("dx", "dg"), (out[0], out[2])):
        assert_within(got, b[k], b["e_" + k] + 1e-17 * np.abs(b[k]).max(), c.dt, k)


@pytest.mark.parametrize("B,T,D", [(1, 700, 64), (2, 96, 130)])
def test_bad_values_stay_in_their_channel(B, T, D):
    sdm = need_gpu()
    c = Case(B, T, D, "fp32", seed=11)
    y0, s0 = sdm.glr_scan(c.h0.clone(), *c.args()), c.h0.clone()
    sdm.glr_scan(s0, *c.args())
    for name, bad in (("x", float("nan")), ("r", float("nan")), ("g", float("nan")), ("x", float("inf"))):
        t = getattr(c, name)
        old = t[0, 20, 5].clone()
        t[0, 20, 5] = bad
        s = c.h0.clone()
        y = sdm.glr_scan(s, *c.args())
        t[0, 20, 5] = old
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[0, 20:, 5] = True
        assert not torch.isfinite(y[hit]).any() and not torch.isfinite(s[0, 5])
        assert torch.equal(y[~hit], y0[~hit])
    # a reset ends it
    c.reset = torch.zeros((B, T), dtype=torch.uint8, device="cuda")
    c.reset[0, 40] = 1
    c.x[0, 20, 5] = float("nan")
    s = c.h0.clone()
    y = sdm.glr_scan(s, *c.args(), **c.kw())
    assert torch.isnan(y[0, 20:40, 5]).all() and torch.isfinite(y[0, 40:]).all() and torch.isfinite(s).all()


def test_device_errors():
    sdm = need_gpu()
    c = Case(3, 20, 70, "fp32", seed=12)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sdm.glr_scan(c.h0.clone(), *c.args(), dev_err=err)
    sdm.sdm_check(err)
    # rates outside [0, inf) count as 0
    for bad in (-0.5, float("nan"), float("inf")):
        rate, zero = c.rate.clone(), c.rate.clone()
        rate[33], zero[33] = bad, 0.0
        err.zero_()
        s1, s2 = c.h0.clone(), c.h0.clone()
        y1, k1 = sdm.glr_scan_train(s1, c.x, c.r, c.g, rate, dev_err=err)
        y2, k2 = sdm.glr_scan_train(s2, c.x, c.r, c.g, zero)
        assert int(err.item()) == sdm.SDM_DEVERR_RATE
        assert torch.equal(y1, y2) and torch.equal(s1, s2) and torch.equal(k1, k2)
        with pytest.raises(sdm.SdmError, match="rate") as e:
            sdm.sdm_check(err)
        assert e.value.code == sdm.SDM_ERR_DEVICE
        err.zero_()
        g1 = sdm.glr_scan_backward(c.dhT.clone(), c.x, c.r, c.g, rate, k1, c.dy, dev_err=err)
        g2 = sdm.glr_scan_backward(c.dhT.clone(), c.x, c.r, c.g, zero, k1, c.dy)
        assert int(err.item()) == sdm.SDM_DEVERR_RATE
        assert all(torch.equal(p, q) for p, q in zip(g1, g2))
    # lengths outside [0, T] are clamped
    err.zero_()
    y1, y2 = torch.zeros_like(c.x), torch.zeros_like(c.x)
    bad, good = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([-4, 21, 7], [0, 20, 7]))
    sdm.glr_scan(c.h0.clone(), *c.args(), lens=bad, y=y1, dev_err=err)
    sdm.glr_scan(c.h0.clone(), *c.args(), lens=good, y=y2)
    assert int(err.item()) == sdm.SDM_DEVERR_INDEX_RANGE and torch.equal(y1, y2)
    # a checkpoint group with an infinity unpacks to NaN, and only that group
    err.zero_()
    c.x[1, 3, 2] = float("inf")
    _, _, (codes, exps) = sdm.glr_scan_train(c.h0.clone(), *c.args(), keep8=True, dev_err=err)
    assert int(err.item()) == sdm.SDM_DEVERR_NONFINITE
    v = sdm.ckpt8_unpack(codes, exps, torch.float32)
    bad = torch.zeros_like(v, dtype=torch.bool)
    bad[0, 1, 3, :64] = True
    assert torch.isnan(v[bad]).all() and torch.isfinite(v[~bad]).all()


def test_a_split_sequence_continues():
    """[0, T1) and then [T1, T) against the whole: each within the bound."""
    sdm = need_gpu()
    for T1 in (1, 8, 130, 299):
        c = Case(2, 300, 96, "fp32", seed=13)
        f = c.forward()
        s = c.h0.clone()
        part = lambda a, b: (t[:, a:b].contiguous() for t in (c.x, c.r, c.g))  # noqa: E731
        y = torch.cat([sdm.glr_scan(s, *part(0, T1), c.rate), sdm.glr_scan(s, *part(T1, 300), c.rate)], 1)
        assert_within(y, f["y"], f["e_y"], c.dt, "y")
        assert_within(s, f["hT"], f["e_hT"], torch.float32, "h_T")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_many_short_sequences(dt):
    """A batch at the limit of the grid, by the step kernel and by the training forward."""
    sdm = need_gpu()
    c = Case(65535, 2, 3, dt, seed=19)
    f = c.forward()
    s, s2 = c.h0.clone(), c.h0.clone()
    y = sdm.glr_scan(s, *c.args())
    y2, carry = sdm.glr_scan_train(s2, *c.args())
    assert torch.equal(y, y2) and torch.equal(s, s2)
    assert_within(y, f["y"], f["e_y"], c.dt, "y")
    check_backward(sdm, c, f, carry, None)


def _apart(t, shift, ld):
    """t's rows at `ld` elements, the first `shift` elements into a buffer of NaN."""
    B, T, D = t.shape
    buf = torch.full((shift + B * T * ld + 1,), float("nan"), dtype=t.dtype, device="cuda")
    v = torch.as_strided(buf, (B, T, D), (T * ld, ld, 1), shift)
    v.copy_(t)
    return v


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 70, 131])
def test_rows_at_every_boundary(D, dt):
    """Inputs and gradients that begin anywhere among 16 bytes, at odd and even
    distances, between NaNs: the bits of the contiguous call."""
    sdm = need_gpu()
    c = Case(2, 75, D, dt, seed=23)
    s0 = c.h0.clone()
    y0, carry0, ckpt0 = sdm.glr_scan_train(s0, *c.args(), keep8=True)
    ds0 = c.dhT.clone()
    want = sdm.glr_scan_backward(ds0, *c.args(), carry0, c.dy)
    for shift, more in [(0, 1), (1, 2), (2, 3), (3, 5), (4, 8), (5, 16 - D % 16), (6, 6), (7, 9), (8, 24 - D % 8)]:
        x, r, g = _apart(c.x, shift, D + more), _apart(c.r, shift + 1, D + more + 1), _apart(c.g, 2 * shift, D + 2 * more)
        s = c.h0.clone()
        assert torch.equal(sdm.glr_scan(s, x, r, g, c.rate), y0) and torch.equal(s, s0)
        y, carry, ckpt = sdm.glr_scan_train(c.h0.clone(), x, r, g, c.rate, keep8=True)
        assert torch.equal(y, y0) and torch.equal(carry, carry0)
        assert torch.equal(ckpt[0], ckpt0[0]) and torch.equal(ckpt[1], ckpt0[1])
        ds, grads = c.dhT.clone(), [_apart(torch.zeros_like(c.x), shift + i, D + more) for i in range(3)]
        out = sdm.glr_scan_backward(ds, x, r, g, c.rate, carry, c.dy, grads=grads)
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(ds, ds0)


def test_one_tensor_as_several_inputs_and_a_state_that_is_kept():
    sdm = need_gpu()
    c = Case(2, 40, 64, "bf16", seed=20)
    y = sdm.glr_scan(c.h0.clone(), c.x, c.x, c.x, c.rate)
    assert torch.equal(y, sdm.glr_scan(c.h0.clone(), c.x, c.x.clone(), c.x.clone(), c.rate))
    before = c.h0.clone()
    out = torch.empty_like(c.h0)
    sdm.glr_scan(c.h0, c.x, c.r, c.g, c.rate, state_out=out)
    assert torch.equal(c.h0, before) and not torch.equal(out, before)


def test_empty_calls():
    sdm = need_gpu()
    c = Case(2, 5, 8, "bf16", seed=14)
    e = torch.empty((2, 0, 8), dtype=c.dt, device="cuda")
    out = torch.empty_like(c.h0)
    y = sdm.glr_scan(c.h0, e, e, e, c.rate, state_out=out)      # T = 0: the state as it was
    assert y.shape == (2, 0, 8) and torch.equal(out, c.h0)
    y, carry, _ = sdm.glr_scan_train(c.h0, e, e, e, c.rate, keep8=True, state_out=out)
    assert carry.shape == (2, 0, 8)
    ds = torch.empty_like(c.h0)
    *_, drate = sdm.glr_scan_backward(c.dhT, e, e, e, c.rate, carry, e, dstate_out=ds)
    assert torch.equal(ds, c.dhT) and torch.all(drate == 0)
    e = torch.empty((0, 5, 8), dtype=c.dt, device="cuda")
    s = torch.empty((0, 8), device="cuda")
    _, carry = sdm.glr_scan_train(s, e, e, e, c.rate)
    *_, drate = sdm.glr_scan_backward(s, e, e, e, c.rate, carry, e)
    assert torch.all(drate == 0)


def test_binding_refusals():
    sdm = need_gpu()
    c = Case(2, 6, 16, "bf16", seed=15)
    x, r, g, rate = c.args()
    for a, err in [((c.h0[:1], x, r, g, rate), ValueError), ((c.h0.double(), x, r, g, rate), TypeError),
                   ((c.h0, x.half(), r, g, rate), TypeError), ((c.h0, x, r.float(), g, rate), TypeError),
                   ((c.h0, x, r[:, :5], g, rate), ValueError), ((c.h0, x, r, g, rate[:8]), ValueError),
                   ((c.h0, x[0], r, g, rate), ValueError),
                   ((c.h0, x.transpose(1, 2).contiguous().transpose(1, 2), r, g, rate), ValueError),
                   ((c.h0, x[:, :1].expand(2, 6, 16), r, g, rate), ValueError),
                   ((c.h0, torch.cat([x, x], 1)[:, :6], r, g, rate), ValueError), ((None, x, r, g, rate), TypeError)]:
        with pytest.raises(err):
            sdm.glr_scan(*a)
        with pytest.raises(err):
            sdm.glr_scan_train(*a)
    for kw, err in [(dict(lens=torch.zeros(2, dtype=torch.int64, device="cuda")), TypeError),
                    (dict(lens=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError),
                    (dict(reset=torch.zeros((2, 5), dtype=torch.uint8, device="cuda")), ValueError),
                    (dict(reset=torch.zeros((2, 6), device="cuda")), TypeError), (dict(y=x.float()), TypeError),
                    (dict(state_out=c.h0[0]), ValueError)]:
        with pytest.raises(err):
            sdm.glr_scan(c.h0, x, r, g, rate, **kw)
    _, carry = sdm.glr_scan_train(c.h0.clone(), x, r, g, rate)
    for a, kw, err in [((x, r, g, rate, carry[:, :0], c.dy), {}, ValueError), ((x, r, g, rate, carry, c.dy.float()), {}, TypeError),
                       ((x, r, g, rate, carry, c.dy), dict(grads=(x, r, torch.empty((2, 6, 32), dtype=c.dt, device="cuda")[..., :16])), ValueError),
                       ((x, None, g, rate, carry, c.dy), {}, TypeError),
                       ((None, None, None, rate, carry, c.dy), dict(ckpt=(x, r)), TypeError)]:
        with pytest.raises(err):
            sdm.glr_scan_backward(c.dhT, *a, **kw)
    # a bool reset is taken as it is
    flags = torch.rand((2, 6), device="cuda") < 0.5
    assert torch.equal(sdm.glr_scan(c.h0.clone(), x, r, g, rate, reset=flags),
                       sdm.glr_scan(c.h0.clone(), x, r, g, rate, reset=flags.to(torch.uint8)))


@pytest.mark.parametrize("B,T,D", [(2, 1, 128), (1, 700, 192), (4, 130, 66)])
def test_streams_and_graphs(B, T, D):
    """On another stream, two calls at once, and captured with its training
    step into a graph that is replayed on new inputs."""
    sdm = need_gpu()
    c, c2 = Case(B, T, D, "bf16", seed=16), Case(B, T, D, "bf16", seed=17)

    def step(k, **kw):
        s, ds = k.h0.clone(), k.dhT.clone()
        y, carry, ck = sdm.glr_scan_train(s, *k.args(), keep8=True, **kw)
        out = sdm.glr_scan_backward(ds, None, None, None, k.rate, carry, k.dy, ckpt=ck, **kw)
        return (y, s, ds, *out)

    want, want2 = step(c), step(c2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        s1.wait_stream(torch.cuda.current_stream())
        s2.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s1):
            got = step(c)
        with torch.cuda.stream(s2):
            got2 = step(c2)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert all(torch.equal(p, q) for p, q in zip(got2, want2))
    a, b = c.h0.clone(), c.h0.clone()
    torch.cuda.synchronize()
    y = sdm.glr_scan(a, *c.args(), stream=s1)       # the stream as an argument
    yi = sdm.glr_scan(b, *c.args(), stream=s2.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(yi, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(c)
    for k in ("x", "r", "g", "dy", "dhT", "h0", "rate"):
        getattr(c, k).copy_(getattr(c2, k))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(held, want2))


def test_a_wait_that_runs_out_is_reported(monkeypatch):
    """SDM_TEST_DROP_SIGNAL=1: a CTA of each cluster keeps its runs to itself, the
    others' bounded waits give up, the call reports it, and the next is exact."""
    sdm = need_gpu()
    c = Case(1, 600, 64, "bf16", seed=18)      # one channel block: split over a cluster
    f = c.forward()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    s = c.h0.clone()
    y, carry = sdm.glr_scan_train(s, *c.args(), dev_err=err)
    sdm.sdm_check(err)
    monkeypatch.setenv("SDM_TEST_DROP_SIGNAL", "1")
    for call in (lambda e: sdm.glr_scan(c.h0.clone(), *c.args(), dev_err=e),
                 lambda e: sdm.glr_scan_backward(c.dhT.clone(), c.x, c.r, c.g, c.rate, carry, c.dy, dev_err=e)):
        call(err)
        assert int(err.item()) == sdm.SDM_DEVERR_TIMEOUT
        err.zero_()
        with pytest.raises(sdm.SdmError, match="gave up"):
            sdm.sdm_check()                     # the library's own record, without an error word
        sdm.sdm_check()
    monkeypatch.delenv("SDM_TEST_DROP_SIGNAL")
    s2 = c.h0.clone()
    assert torch.equal(sdm.glr_scan(s2, *c.args(), dev_err=err), y) and torch.equal(s, s2)
    assert_within(y, f["y"], f["e_y"], c.dt, "y")
    check_backward(sdm, c, f, carry, None)
    sdm.sdm_check(err)


def test_offsets_beyond_32_bits():
    """2.3e9 elements: the last tokens against a call on them alone that
    continues from the state before them."""
    sdm = need_gpu()
    T, D, cut = 36000, 65536, 35968
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(1)
    one = torch.randn((1, 64, D), generator=gen, device="cuda").to(torch.bfloat16)
    x = one.repeat(1, T // 64 + 1, 1)[:, :T].contiguous()
    rate = torch.rand(D, generator=gen, device="cuda") * 0.5 + 0.1
    h0 = torch.randn((1, D), generator=gen, device="cuda")
    s = h0.clone()
    y, carry = sdm.glr_scan_train(s, x, x, x, rate)
    last = x[:, cut:].contiguous()
    s2 = carry[:, cut // 8].clone()
    y2, carry2 = sdm.glr_scan_train(s2, last, last, last, rate)
    # fp32 roundings of two splits of the same sums: the bound of 32 tokens at these decays is below 1e-4
    assert torch.allclose(s, s2, rtol=1e-4, atol=1e-4)
    assert torch.allclose(y[:, cut:].float(), y2.float(), rtol=2 ** -7, atol=1e-4)
    ds, ds2 = h0.clone(), h0.clone()
    dx, dr, dg, _ = sdm.glr_scan_backward(ds, x, x, x, rate, carry, y)
    dx2, dr2, dg2, _ = sdm.glr_scan_backward(ds2, last, last, last, rate, carry2, y[:, cut:].contiguous())
    for p, q in ((dx, dx2), (dr, dr2), (dg, dg2)):
        assert torch.allclose(p[:, cut:].float(), q.float(), rtol=2 ** -7, atol=2e-3)
    del dx, dr, dg, y
    codes, exps = sdm.ckpt8_pack(x)
    c2, e2 = sdm.ckpt8_pack(last)
    assert torch.equal(codes[:, cut:], c2) and torch.equal(exps[:, cut:], e2)
    v = sdm.ckpt8_unpack(codes, exps, torch.bfloat16)
    assert torch.equal(v[:, cut:], sdm.ckpt8_unpack(c2, e2, torch.bfloat16))


def test_a_layer_of_the_scan_family_together():
    """A step of two layers as they are used: the recurrence over one
    projection's slices, its output as the values of the sparse scan's
    training step, and the recurrence's backward from the scan's dL/dv through
    8-bit checkpoints."""
    sdm = need_gpu()
    import oracle
    import synth
    sh = synth.SDM_TINY
    inp = synth.sdm_inputs(sh, 21)
    D = sh.H * sh.d_v
    c = Case(sh.B, sh.T, D, "fp32", seed=22, fused=True)
    f = c.forward()
    s = c.h0.clone()
    y, carry, ck = sdm.glr_scan_train(s, *c.args(), keep8=True)
    from helpers import assert_y_close, dev
    iw, ww = sdm.sdm_address(dev(inp["s1w"]), dev(inp["s2w"]), sh.k, sh.W)
    ir, wr = sdm.sdm_address(dev(inp["s1r"]), dev(inp["s2r"]), sh.k, sh.R)
    table = torch.zeros((sh.B, sh.H, sh.N, sh.d_v), device="cuda")
    v = y.view(sh.B, sh.T, sh.H, sh.d_v)
    al, be = dev(inp["alpha"]), dev(inp["beta"])
    out, undo = sdm.sdm_scan_train(table, v, al, be, iw, ww, ir, wr)
    dout = torch.randn(out.shape, generator=torch.Generator().manual_seed(3)).cuda()
    dv = sdm.sdm_scan_backward(table, torch.zeros_like(table), v, al, be, iw, ww, ir, wr, undo, dout)[0]
    ds = torch.zeros_like(c.h0)
    dx, dr, dg, drate = sdm.glr_scan_backward(ds, None, None, None, c.rate, carry, dv.view(sh.B, sh.T, D), ckpt=ck)
    yr, _, _ = oracle.sdm_forward(dict(inp, v=f["y"].reshape(v.shape).astype(np.float32)), sh.k, sh.W, sh.R)["y"], None, None
    assert_y_close(host(out), yr)
    x8, r8, g8 = (ref.unpack8(*ref.pack8(t)) for t in c.np("x", "r", "g"))
    b = ref.backward(f, np.zeros((sh.B, D)), x8, r8, g8, *c.np("rate"), host(dv).reshape(sh.B, sh.T, D).astype(np.float64),
                     seg=8)
    for k, got in zip(("dx", "dr", "dg"), (dx, dr, dg)):
        assert_within(got, b[k], b["e_" + k], torch.float32, k)
    assert_within(drate, b["drate"], b["e_drate"], torch.float32, "drate")
