"""The gated linear recurrence, its gradients and the 8-bit checkpoint format
in fp64 numpy, token by token, with a running bound of the error that fp32
arithmetic may make.

Bounds.  E = 2^-24 is fp32's half step.  The kernels' exponential and
reciprocal are good to 2^-22 and 2^-23 (relative).
  sigmoid(z): the exponent z log2(e) is rounded twice (|z| 2 E), so
      rel <= (1 - sigmoid) (2 |z| E + 2^-22) + 2^-23 + 2 E.
  y = rate sigmoid(r): sigmoid's error and a rounding, d_y.
  1 - a = 1 - e^-y, two forms that meet at y = 0.15.  Below: a cubic times y, good
      to 6e-8, with four roundings, so d_y y a / (1 - a) <= d_y, and 6e-8 + 5 E,
      relative.  Above: the exponential's 2^-22 and two roundings of its argument
      (2 E y), relative to a, and a rounding of the difference.
  a itself: 1 less that, an absolute error e_a (E for the last rounding).
  m = sqrt((1 - a) (1 + a)): half of 1 - a's relative error (and of 1 + a's, whose
      absolute error is the same and whose size is between 1 and 2), three
      roundings, and the root's own 2^-22.
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
    """sigmoids, decay, m, and the bounds: of a (absolute), of m (relative)."""
    sr, sg = sig(r), sig(g)
    y = rate * sr
    a, c = np.exp(-y), -np.expm1(-y)                # the decay and 1 - a
    m = np.sqrt(c * (1 + a))
    d_y = rel_sig(r) + E
    near = c * (d_y + 6e-8 + 5 * E)
    far = a * (y * (d_y + 2 * E) + 2.0 ** -22) + E
    e_c = np.where(y < 0.149, near, np.where(y > 0.151, far, np.maximum(near, far)))
    e_a = e_c + E
    with np.errstate(divide="ignore", invalid="ignore"):
        d_m = 0.5 * (np.where(c > 0, e_c / c, 0) + e_c) + 1.5 * E + 2.0 ** -22
    return sr, sg, a, m, e_a, d_m


def forward(h0, x, r, g, rate, reset=None, lens=None):
    """y, h_T, all states before each token, and the bounds of y and h_T."""
    B, T, D = x.shape
    _, sg, a, m, e_a, d_m = gates(x, r, g, rate)
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
        en = keep * (a[:, t] * (e + 4 * E * G) + e_a[:, t] * G) + e_u[:, t] + 2 * E * Gn
        G = np.where(live[:, None], Gn, G)
        h, e = np.where(live[:, None], hn, h), np.where(live[:, None], en, e)
        y[:, t], e_y[:, t] = h, e
    return dict(y=y, hT=h, before=before, e_y=e_y, e_hT=e, e_before=e_b)


def backward(f, dhT, x, r, g, rate, dy, reset=None, lens=None, seg=None):
    """Gradients by the formulas and their bounds; f: what forward returned on
    the true inputs.  seg: states inside a segment of that many tokens are
    recomputed from x, r, g (an 8-bit checkpoint's values) and its first one."""
    B, T, D = x.shape
    sr, sg, a, m, e_a, d_m = gates(x, r, g, rate)
    u = m * sg * x
    e_u = np.abs(u) * (d_m + rel_sig(g) + 3 * E)
    before, e_b = f["before"].copy(), f["e_before"].copy()
    keep = np.ones((B, T, 1)) if reset is None else (reset == 0)[:, :, None].astype(float)
    live = np.ones((B, T, 1)) if lens is None else (np.arange(T)[None] < lens[:, None])[:, :, None].astype(float)
    if seg:
        for t in range(T):
            if t % seg:
                before[:, t] = a[:, t - 1] * before[:, t - 1] * keep[:, t - 1] + u[:, t - 1]
                e_b[:, t] = (keep[:, t - 1] * (a[:, t - 1] * (e_b[:, t - 1] + 4 * E * np.abs(before[:, t - 1])) +
                                            e_a[:, t - 1] * np.abs(before[:, t - 1])) + e_u[:, t - 1] + 2 * E * np.abs(before[:, t]))
    before, e_b = before * keep, e_b * keep
    dh, e_dh = np.zeros((B, T, D)), np.zeros((B, T, D))
    c, e = dhT.astype(np.float64).copy(), np.zeros((B, D))
    G = np.abs(c)
    for t in range(T - 1, -1, -1):
        lv = live[:, t] > 0
        dh[:, t] = dy[:, t] + c
        H = G + np.abs(dy[:, t])
        e_dh[:, t] = e + 2 * E * H
        e = np.where(lv, keep[:, t] * (a[:, t] * (e_dh[:, t] + 4 * E * H) + e_a[:, t] * H), e)
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
    with np.errstate(divide="ignore", invalid="ignore"):
        e_k = np.where(m > 0, np.abs(sg * x) * e_a / m, 0.0) + np.abs(k) * (d_m + rel_sig(g) + 4 * E)
    e_in = e_b + e_k + E * np.abs(inner)
    dL = a * dh * inner
    e_dL = np.abs(dh * inner) * (e_a + 4 * E * a) + (a + e_a) * (np.abs(inner) * e_dh + np.abs(dh) * e_in)
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
