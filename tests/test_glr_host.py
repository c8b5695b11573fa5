"""Gated linear recurrence and 8-bit checkpoints without a GPU: the formulas'
gradients against differences, the checkpoint format's properties, and the
calls' refusals before anything reaches the device."""
import numpy as np
import pytest

import glr_reference as ref
from synth import bf16_bits_to_f32, to_bf16_bits

A = 1 << 20     # a fake, aligned "device" address


@pytest.fixture(scope="module")
def sdm():
    from delta_rule_memory_gb300 import build as b
    b.build()
    import delta_rule_memory_gb300 as m
    return m


@pytest.mark.parametrize("with_reset,with_lens", [(False, False), (True, False), (False, True), (True, True)])
def test_formulas_gradients_match_differences(with_reset, with_lens):
    rng = np.random.default_rng(3)
    B, T, D = 2, 9, 3
    x, r, g = (rng.normal(size=(B, T, D)) for _ in range(3))
    rate, h0 = rng.uniform(0.05, 1.5, D), rng.normal(size=(B, D))
    dy, dhT = rng.normal(size=(B, T, D)), rng.normal(size=(B, D))
    reset = (rng.random((B, T)) < 0.3).astype(np.uint8) if with_reset else None
    lens = np.array([6, 9]) if with_lens else None
    live = 1.0 if lens is None else (np.arange(T)[None] < lens[:, None])[..., None]

    def loss(h0, x, r, g, rate):
        f = ref.forward(h0, x, r, g, rate, reset, lens)
        return float((f["y"] * dy * live).sum() + (f["hT"] * dhT).sum())

    f = ref.forward(h0, x, r, g, rate, reset, lens)
    b = ref.backward(f, dhT, x, r, g, rate, dy, reset, lens)
    args = [h0, x, r, g, rate]
    for i, name in enumerate(("dh0", "dx", "dr", "dg", "drate")):
        got = b[name] * live if name in ("dx", "dr", "dg") else b[name]
        for _ in range(4):
            v, h = rng.normal(size=args[i].shape), 1e-5
            up, down = (loss(*(a + s * h * v if j == i else a for j, a in enumerate(args))) for s in (1, -1))
            # central difference: error O(h^2) = 1e-10 times third derivatives, cancellation 1e-16 / 1e-5
            np.testing.assert_allclose((got * v).sum(), (up - down) / (2 * h), rtol=1e-6, atol=1e-7)


def test_recomputed_segments_are_the_states_when_the_values_are_the_same():
    rng = np.random.default_rng(4)
    x, r, g = (rng.normal(size=(2, 21, 5)) for _ in range(3))
    rate, h0 = rng.uniform(0, 1, 5), rng.normal(size=(2, 5))
    reset = (rng.random((2, 21)) < 0.2).astype(np.uint8)
    f = ref.forward(h0, x, r, g, rate, reset)
    dy, dhT = rng.normal(size=(2, 21, 5)), rng.normal(size=(2, 5))
    b1 = ref.backward(f, dhT, x, r, g, rate, dy, reset)
    b2 = ref.backward(f, dhT, x, r, g, rate, dy, reset, seg=8)
    for k in ("dx", "dr", "dg", "drate", "dh0"):
        np.testing.assert_allclose(b1[k], b2[k], rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("D", [1, 63, 64, 65, 200])
def test_checkpoint_format(D):
    rng = np.random.default_rng(D)
    x = (rng.normal(size=(7, D)) * np.exp(3 * rng.normal(size=(7, 1)))).astype(np.float32)
    x[0] = 0
    x[1, 0] = 127.0         # exactly 127 steps
    codes, exps = ref.pack8(x)
    assert codes.min() >= -127 and exps.shape == (7, -(-D // 64))
    v = ref.unpack8(codes, exps)
    step = np.repeat(2.0 ** (exps.astype(float) - 127), 64, axis=-1)[:, :D]
    assert np.all(np.abs(v - x) <= step / 2)
    # exact in bf16
    import torch
    assert np.array_equal(bf16_bits_to_f32(to_bf16_bits(torch.from_numpy(v.astype(np.float32)))), v)
    # packing what was unpacked changes nothing more
    assert np.array_equal(ref.unpack8(*ref.pack8(v)), v)
    # a group uses at least half of the range, or the smallest exponent
    for gcol in range(exps.shape[1]):
        top = np.abs(codes[:, gcol * 64:(gcol + 1) * 64].astype(int)).max(1)
        assert np.all((top >= 63) | (exps[:, gcol] == 1))


def _scan(L, train=False, **kw):
    a = dict(state=A, out=A, x=A, ldx=8, r=A, ldr=8, g=A, ldg=8, dt=1, rate=A, reset=None, lens=None, B=2, T=4, D=8, y=A,
             carry=A, codes=None, exps=None, err=None)
    a.update(kw)
    head = (a["state"], a["out"], a["x"], a["ldx"], a["r"], a["ldr"], a["g"], a["ldg"], a["dt"], a["rate"], a["reset"],
            a["lens"], a["B"], a["T"], a["D"], a["y"])
    if train:
        return L.glr_scan_train(*head, a["carry"], a["codes"], a["exps"], a["err"], None)
    return L.glr_scan(*head, a["err"], None)


@pytest.mark.parametrize("train", [False, True])
def test_scan_refusals(sdm, train):
    L = sdm.lib()
    for kw, code in [(dict(state=None), 1), (dict(out=None), 1), (dict(x=None), 1), (dict(r=None), 1),
                     (dict(g=None), 1), (dict(y=None), 1), (dict(rate=None), 1), (dict(B=-1), 1), (dict(T=-1), 1),
                     (dict(D=-8), 1), (dict(dt=2), 4), (dict(B=65536), 2), (dict(T=1 << 30), 2),
                     (dict(D=1 << 24, ldx=1 << 24, ldr=1 << 24, ldg=1 << 24), 2), (dict(ldx=7), 2), (dict(ldr=0), 2),
                     (dict(ldg=-8), 2), (dict(ldx=1 << 31), 2), (dict(x=A + 1), 3), (dict(y=A + 1), 3),
                     (dict(dt=0, r=A + 2), 3), (dict(state=A + 2), 3), (dict(out=A + 1), 3), (dict(rate=A + 2), 3),
                     (dict(lens=A + 2), 3), (dict(err=A + 2), 3)]:
        assert _scan(L, train, **kw) == code, kw
        assert (b"glr_scan_train" if train else b"glr_scan") in L.sdm_last_error()
    assert _scan(L, train, B=0) == 0 and _scan(L, train, D=0) == 0      # nothing to do: nothing launched


def test_train_refusals(sdm):
    L = sdm.lib()
    assert _scan(L, True, carry=None) == sdm.SDM_ERR_INVALID_ARG
    assert _scan(L, True, carry=A + 2) == sdm.SDM_ERR_ALIGN
    assert _scan(L, True, codes=A) == sdm.SDM_ERR_INVALID_ARG
    assert _scan(L, True, exps=A) == sdm.SDM_ERR_INVALID_ARG


def test_backward_refusals(sdm):
    L = sdm.lib()

    def call(**kw):
        a = dict(ds=A, out=A, x=A, ldx=8, r=A, ldr=8, g=A, ldg=8, codes=None, exps=None, dt=1, rate=A, reset=None,
                 lens=None, carry=A, dy=A, B=2, T=4, D=8, dx=A, dr=A, dg=A, ldd=8, drate=A, ws=A, wsb=1 << 20, err=None)
        a.update(kw)
        return L.glr_scan_backward(a["ds"], a["out"], a["x"], a["ldx"], a["r"], a["ldr"], a["g"], a["ldg"], a["codes"],
                                   a["exps"], a["dt"], a["rate"], a["reset"], a["lens"], a["carry"], a["dy"], a["B"],
                                   a["T"], a["D"], a["dx"], a["dr"], a["dg"], a["ldd"], a["drate"], a["ws"], a["wsb"],
                                   a["err"], None)

    none = dict(x=None, r=None, g=None)
    for kw, code in [(dict(out=None), 1), (dict(x=None), 1), (none, 1), (dict(codes=A, exps=A), 1),
                     (dict(none, codes=A), 1), (dict(none, exps=A), 1), (dict(codes=A, exps=A, x=None, r=None), 1),
                     (dict(carry=None), 1), (dict(dy=None), 1), (dict(dx=None), 1), (dict(dr=None), 1),
                     (dict(dg=None), 1), (dict(drate=None), 1), (dict(rate=None), 1), (dict(ws=None), 1),
                     (dict(wsb=sdm.glr_scan_backward_workspace_size(2, 4, 8) - 1), 1), (dict(ws=A + 8), 3),
                     (dict(ldd=7), 2), (dict(dt=3), 4), (dict(B=-2), 1), (dict(dy=A + 1), 3), (dict(dx=A + 1), 3),
                     (dict(ds=A + 2), 3), (dict(drate=A + 2), 3), (dict(carry=A + 1), 3)]:
        assert call(**kw) == code, kw
    assert call(D=0) == 0


def test_checkpoint_refusals(sdm):
    L = sdm.lib()
    for kw, code in [(dict(x=None), 1), (dict(codes=None), 1), (dict(exps=None), 1), (dict(rows=-1), 1),
                     (dict(D=-1), 1), (dict(D=1 << 24), 2), (dict(ld=7), 2), (dict(dt=5), 4), (dict(x=A + 1), 3),
                     (dict(rows=1 << 60), 2)]:
        a = dict(x=A, ld=8, dt=1, rows=3, D=8, codes=A, exps=A)
        a.update(kw)
        assert L.ckpt8_pack(a["x"], a["ld"], a["dt"], a["rows"], a["D"], a["codes"], a["exps"], None, None) == code, kw
        assert L.ckpt8_unpack(a["codes"], a["exps"], a["rows"], a["D"], a["x"], a["ld"], a["dt"], None) == code, kw
    assert L.ckpt8_pack(A, 8, 1, 3, 8, A, A, A + 2, None) == sdm.SDM_ERR_ALIGN
    assert L.ckpt8_pack(None, 0, 1, 0, 8, None, None, None, None) == 0
    assert L.ckpt8_unpack(None, None, 5, 0, None, 0, 0, None) == 0


def test_sizes(sdm):
    assert sdm.glr_scan_carry_size(2, 17, 5) == 4 * 2 * 3 * 5
    assert sdm.glr_scan_carry_size(2, 0, 5) == 0
    assert sdm.glr_scan_carry_size(-1, 17, 5) == 0
    assert sdm.glr_scan_carry_size(4, 1 << 29, 1 << 20) == 4 * 4 * (1 << 26) * (1 << 20)      # beyond 32 bits
    assert sdm.glr_scan_backward_workspace_size(3, 100, 65) >= 4 * 65
    assert sdm.glr_scan_backward_workspace_size(3, 100, -1) == 0


def test_the_binding_refuses_host_tensors(sdm):
    import torch
    x = torch.zeros(1, 2, 8)
    s = torch.zeros(1, 8)
    with pytest.raises(TypeError, match="CUDA"):
        sdm.glr_scan(s, x, x, x, torch.zeros(8))
    with pytest.raises(TypeError, match="CUDA"):
        sdm.glr_scan_train(s, x, x, x, torch.zeros(8))
    with pytest.raises(TypeError, match="CUDA"):
        sdm.glr_scan_backward(s, x, x, x, torch.zeros(8), torch.zeros(1, 1, 8), x)
    with pytest.raises(ValueError, match="not both"):
        sdm.glr_scan_backward(s, x, x, x, torch.zeros(8), torch.zeros(1, 1, 8), x, ckpt=(x, x))
    with pytest.raises(ValueError, match="needed"):
        sdm.glr_scan_backward(s, None, None, None, torch.zeros(8), torch.zeros(1, 1, 8), x)
    with pytest.raises(TypeError, match="CUDA"):
        sdm.ckpt8_pack(x)
    with pytest.raises(TypeError, match="CUDA"):
        sdm.ckpt8_unpack(torch.zeros(2, 8, dtype=torch.int8), torch.zeros(2, 1, dtype=torch.uint8))
