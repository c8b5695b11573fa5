"""The gradient of the decay's logarithm as gdn_backward forms it, on the CPU: from
terms that each pass the token's decay, so that the sum is as exact, relative to
itself, at a decay of e^-16 as at one near 1."""
import pytest
import torch

import gdn_reference as ref

C = 64


def chunked(S0, q, k, v, la, beta, dS, dy, reset, dtype):
    """dlog_alpha of one head, chunk by chunk, what enters the sums rounded to `dtype` and summed in it:
    gam_C <S, G> + sum_{i >= t} gam_i (q_i . S dy_i - k_i . S dz_i) + sum_{j < t} tail_j u_j . G^T k_j
    + sum_{i >= t > j} (X_ij q_i . k_j + N_ij k_i . k_j)."""
    T = la.shape[1]
    parts = [slice(a, min(a + C, T)) for a in range(0, T, C)]
    fwd, S = [], S0
    for p in parts:
        fwd.append(ref.forward(S, q[:, p], k[:, p], v[:, p], la[:, p], beta[:, p], None if reset is None else reset[:, p]))
        S = fwd[-1][1]
    out, G = torch.zeros(T, dtype=dtype), dS.double()
    for c in range(len(parts) - 1, -1, -1):
        p, f = parts[c], fwd[c]
        Sc = (S0.double() if c == 0 else fwd[c - 1][1])[0, 0].to(dtype)
        b = ref.backward(f, G, q[:, p], k[:, p], v[:, p], la[:, p], beta[:, p], dy[:, p], None if reset is None else reset[:, p])
        g = G[0, 0].to(dtype)
        n = la[:, p].shape[1]
        l = la[0, p, 0].double().cumsum(0)
        seg = torch.zeros(n) if reset is None else (reset[0, p] != 0).double().cumsum(0)
        at = torch.arange(n)
        D = torch.where((seg[:, None] == seg[None]) & (at[:, None] >= at[None]), (l[:, None] - l[None]).clamp(max=0).exp(), 0.0).to(dtype)
        gam = torch.where(seg == 0, l.exp(), 0.0).to(dtype)
        tail = torch.where(seg == seg[-1], (l[-1] - l).exp(), 0.0).to(dtype)
        E, dz = torch.stack([e[0, 0] for e in f[3]]).to(dtype), b[3][0, :, 0].to(dtype)
        u = E * beta[0, p, 0, None].to(dtype)
        qc, kc, yc = q[0, p, 0].to(dtype), k[0, p, 0].to(dtype), dy[0, p, 0].to(dtype)
        A = gam * ((qc * (yc @ Sc.T)).sum(1) - (kc * (dz @ Sc.T)).sum(1))
        B = tail * (kc * (u @ g.T)).sum(1)
        P = D * (yc @ u.T) * (qc @ kc.T) - D * (at[:, None] > at[None]) * (dz @ u.T) * (kc @ kc.T)
        for t in range(n):
            out[p.start + t] = gam[-1] * (Sc * g).sum() + A[t:].sum() + B[:t].sum() + P[t:, :t].sum()
        G = b[0]
    return out


def inputs(level, T=192, d=32, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    q, k, v = n(1, T, 1, d), n(1, T, 1, d), n(1, T, 1, d)
    q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
    la = level * (0.75 + 0.5 * torch.rand((1, T, 1), generator=g))
    return 0.3 * n(1, 1, d, d), q, k, v, la, torch.sigmoid(n(1, T, 1)), 0.3 * n(1, 1, d, d), n(1, T, 1, d)


@pytest.mark.parametrize("level", [-0.7, -8.0, -16.0])
@pytest.mark.parametrize("resets", [False, True])
def test_formula(level, resets):
    S0, q, k, v, la, beta, dS, dy = inputs(level)
    reset = None
    if resets:
        reset = torch.zeros((1, 192), dtype=torch.uint8)
        reset[0, [0, 5, 64, 100, 101, 191]] = 1
    f = ref.forward(S0, q, k, v, la, beta, reset)
    want = ref.backward(f, dS, q, k, v, la, beta, dy, reset)[4][0, :, 0]
    # 64 bits: sums of at most 2^12 terms of like size, 2^-53 each
    assert float((chunked(S0, q, k, v, la, beta, dS, dy, reset, torch.float64) - want).norm()) <= 1e-12 * float(want.norm())
    # 32 bits: what enters rounded once, at most 2^5 roundings to a term, terms of either sign: 2^5 2^-24 and twice that in hand
    assert float((chunked(S0, q, k, v, la, beta, dS, dy, reset, torch.float32) - want).norm()) <= 2.0 ** -18 * float(want.norm())
