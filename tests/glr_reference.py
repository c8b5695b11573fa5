"""The gated linear recurrence, its gradients and the 8-bit checkpoint format
in fp64 numpy, token by token, with a running bound of the error that fp32
arithmetic may make.

Bounds.  E = 2^-24 is fp32's half step.  The kernels' exponential and
reciprocal are good to 2^-22 and 2^-23 (relative).
  sigmoid(z): the exponent z log2(e) is rounded twice (|z| 2 E), so
      rel <= (1 - sigmoid) (2 |z| E + 2^-22) + 2^-23 + 2 E.
  a = 2^l: l = rate2 sigmoid(r) has three roundings and sigmoid's error,
      rel <= |L| (rel_sigmoid + 3 E) + 2^-22.
  m = sqrt(1 - a^2), the larger of two forms, neither above it but by rounding.
      The polynomial in w = -2 L has w's error (rel_sigmoid + 5 E), eight roundings,
      and falls short by 8e-7 of m^2 up to w = 0.28, by more behind that.  The
      difference 1 - 6e-7 - a^2 has a^2's error, 2 a^2 d_a, and 6e-7 and a
      rounding.  The larger falls short by the smaller of the two, and is above
      m^2 by what a^2's error is over 6e-7 (0.9 of it: the constant is rounded);
      half of it, and the root's own 2^-22.
Along the recurrence every token adds a's error and a product's and a sum's
rounding on top of the decayed one; a split over time multiplies decays with
one another first, one more rounding a token: 4 E a token covers each order.
What those are relative to: a split forms what the tokens of a run leave and
what the state before the run leaves as two numbers and adds them at the end,
a (h + u') as a h + a u', so each rounds by itself and their sum may cancel:
with h = -u' (1 + d) the exact result is a d u', while the two products are off
by E |a u'| each, however small d is.  The roundings are therefore relative to
the same recurrence over absolute values, G_t = a_t G_{t-1} + |u_t|, which
bounds every partial sum of every split, and not to |h_t|.
"""
import numpy as np

E = 2.0 ** -24


def sig(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def rel_sig(z):
    az = np.minimum(np.abs(z), 90.0)
    return (1 - sig(z)) * (2 * az * E + 2.0 ** -22) + 2.0 ** -23 + 2 * E


def gates(x, r, g, rate):
    sr, sg = sig(r), sig(g)
    L = -rate * sr
    a, m2 = np.exp(L), -np.expm1(2 * L)
    m = np.sqrt(m2)
    d_a = -L * (rel_sig(r) + 3 * E) + 2.0 ** -22                     # rel error of a
    w, a2 = -2 * L, 2 * a * a * d_a
    with np.errstate(divide="ignore", invalid="ignore"):
        short = np.where(m2 > 0, np.minimum(np.where(w <= 0.28, 8e-7, np.inf), (a2 + 6.6e-7) / m2), 0)
        over = np.where(m2 > 0, np.maximum(0, a2 - 5.4e-7) / m2, 0)
    d_m = 0.5 * (rel_sig(r) + 13 * E + short + over) + 2.0 ** -22
    return sr, sg, a, m, d_a, d_m


def forward(h0, x, r, g, rate, reset=None, lens=None):
    """y, h_T, all states before each token, and the bounds of y and h_T."""
    B, T, D = x.shape
    _, sg, a, m, d_a, d_m = gates(x, r, g, rate)
    u = m * sg * x
    e_u = np.abs(u) * (d_m + rel_sig(g) + 3 * E)
    y, before = np.zeros((B, T, D)), np.zeros((B, T, D))
    e_y, e_b = np.zeros((B, T, D)), np.zeros((B, T, D))
    h, e = h0.astype(np.float64).copy(), np.zeros((B, D))
    G = np.abs(h)
    for t in range(T):
        live = np.ones(B, bool) if lens is None else t < lens
        keep = np.ones((B, 1)) if reset is None else (reset[:, t] == 0)[:, None].astype(float)
        before[:, t], e_b[:, t] = h, e
        hn = a[:, t] * h * keep + u[:, t]
        Gn = a[:, t] * G * keep + np.abs(u[:, t])
        en = keep * a[:, t] * (e + G * (d_a[:, t] + 4 * E)) + e_u[:, t] + 2 * E * Gn
        G = np.where(live[:, None], Gn, G)
        h, e = np.where(live[:, None], hn, h), np.where(live[:, None], en, e)
        y[:, t], e_y[:, t] = h, e
    return dict(y=y, hT=h, before=before, e_y=e_y, e_hT=e, e_before=e_b)


def backward(f, dhT, x, r, g, rate, dy, reset=None, lens=None, seg=None):
    """Gradients by the formulas and their bounds; f: what forward returned on
    the true inputs.  seg: states inside a segment of that many tokens are
    recomputed from x, r, g (an 8-bit checkpoint's values) and its first one."""
    B, T, D = x.shape
    sr, sg, a, m, d_a, d_m = gates(x, r, g, rate)
    u = m * sg * x
    e_u = np.abs(u) * (d_m + rel_sig(g) + 3 * E)
    before, e_b = f["before"].copy(), f["e_before"].copy()
    keep = np.ones((B, T, 1)) if reset is None else (reset == 0)[:, :, None].astype(float)
    live = np.ones((B, T, 1)) if lens is None else (np.arange(T)[None] < lens[:, None])[:, :, None].astype(float)
    if seg:
        for t in range(T):
            if t % seg:
                before[:, t] = a[:, t - 1] * before[:, t - 1] * keep[:, t - 1] + u[:, t - 1]
                e_b[:, t] = (keep[:, t - 1] * a[:, t - 1] * (e_b[:, t - 1] + np.abs(before[:, t - 1]) *
                             (d_a[:, t - 1] + 4 * E)) + e_u[:, t - 1] + 2 * E * np.abs(before[:, t]))
    before, e_b = before * keep, e_b * keep
    dh, e_dh = np.zeros((B, T, D)), np.zeros((B, T, D))
    c, e = dhT.astype(np.float64).copy(), np.zeros((B, D))
    G = np.abs(c)
    for t in range(T - 1, -1, -1):
        lv = live[:, t] > 0
        dh[:, t] = dy[:, t] + c
        H = G + np.abs(dy[:, t])
        e_dh[:, t] = e + 2 * E * H
        e = np.where(lv, keep[:, t] * a[:, t] * (e_dh[:, t] + H * (d_a[:, t] + 4 * E)), e)
        G = np.where(lv, keep[:, t] * a[:, t] * H, G)
        c = np.where(lv, keep[:, t] * a[:, t] * dh[:, t], c)
    with np.errstate(divide="ignore", invalid="ignore"):
        am = np.where(m > 0, a / m, 0.0)
    dx, dg = dh * m * sg, dh * m * sg * (1 - sg) * x
    rel = d_m + rel_sig(g) + 4 * E
    e_dx = np.abs(dx) * rel + m * sg * e_dh
    # 1 - sigmoid: absolute error of sigmoid and one rounding
    e_dg = (np.abs(dg) * rel + np.abs(m * sg * (1 - sg) * x) * e_dh +
            np.abs(dh * m * sg * x) * (sg * rel_sig(g) + E))
    k = am * sg * x
    inner = before - k
    e_in = e_b + np.abs(k) * (d_a + d_m + rel_sig(g) + 4 * E) + E * np.abs(inner)
    dL = a * dh * inner
    e_dL = np.abs(dL) * (d_a + 4 * E) + a * np.abs(inner) * e_dh + a * np.abs(dh) * e_in
    dr = -rate * sr * (1 - sr) * dL
    e_dr = (rate * sr * (1 - sr) * e_dL + np.abs(dr) * (rel_sig(r) + 4 * E) +
            rate * sr * np.abs(dL) * (sr * rel_sig(r) + E))
    term = -sr * dL * live
    e_term = (sr * e_dL + np.abs(term) * (rel_sig(r) + E)) * live
    n = max(1, min(B * T, 4096))          # additions in a row, at most
    out = dict(dx=dx, dr=dr, dg=dg, drate=term.sum((0, 1)), dh0=c)
    out.update(e_dx=e_dx, e_dr=e_dr, e_dg=e_dg, e_drate=e_term.sum((0, 1)) + n * E * np.abs(term).sum((0, 1)), e_dh0=e)
    return out


def pack8(x):
    """codes int8, exponent bytes uint8 of fp32 or fp64 x [..., D] (D > 0)."""
    x = np.asarray(x, np.float64)
    D = x.shape[-1]
    G = -(-D // 64)
    v = np.zeros((*x.shape[:-1], G * 64))
    v[..., :D] = x
    v = v.reshape(*x.shape[:-1], G, 64)
    fine = (np.abs(v) <= 127 * 2.0 ** 121).all(-1)      # NaN compares false
    top = np.abs(np.where(fine[..., None], v, 0)).max(-1)
    e = np.full(top.shape, -126)
    while True:
        up = top > 127 * 2.0 ** e
        if not up.any():
            break
        e = e + up
    codes = np.where(fine[..., None], np.rint(np.where(fine[..., None], v, 0) / 2.0 ** e[..., None]), 0)
    exps = np.where(fine, e + 127, 255).astype(np.uint8)
    return codes.reshape(*x.shape[:-1], G * 64)[..., :D].astype(np.int8), exps


def unpack8(codes, exps):
    D = codes.shape[-1]
    step = np.where(exps == 255, np.nan, 2.0 ** (exps.astype(np.float64) - 127))
    return codes.astype(np.float64) * np.repeat(step, 64, axis=-1)[..., :D]
