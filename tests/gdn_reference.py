"""The gated delta rule in 64 bits, token by token, with its gradients written
out; and visits sorted by partition with plain loops.  CPU torch tensors."""
import torch


def forward(S0, q, k, v, la, beta, reset=None, lens=None):
    """q, k [B,T,Hk,dk], v [B,T,H,dv], la, beta [B,T,H], S0 [B,H,dk,dv]: (y, S_T, the states
    after the decay, the residuals), zeros for tokens behind lens."""
    S = S0.double().clone()
    B, T, Hk = q.shape[:3]
    H = v.shape[2]
    q, k = (x.double().repeat_interleave(H // Hk, 2) for x in (q, k))
    v, la, beta = v.double(), la.double(), beta.double()
    y, decayed, resid, states = torch.zeros_like(v), [], [], [S]
    for t in range(T):
        keep = torch.exp(la[:, t])
        if reset is not None:
            keep = torch.where(reset[:, t, None] != 0, 0.0, keep)
        Sd = S * keep[..., None, None]
        Sd = torch.where(keep[..., None, None] == 0, 0.0, Sd)       # 0 whatever the state holds
        e = v[:, t] - (Sd * k[:, t, :, :, None]).sum(2)
        new = Sd + k[:, t, :, :, None] * (beta[:, t, :, None] * e)[:, :, None]
        live = torch.ones(B, dtype=torch.bool) if lens is None else t < lens
        S = torch.where(live[:, None, None, None], new, S)
        y[:, t] = torch.where(live[:, None, None], (S * q[:, t, :, :, None]).sum(2), 0.0)
        decayed.append(Sd)
        resid.append(e)
        states.append(S)
    return y, S, decayed, resid, states


def backward(saved, dS, q, k, v, la, beta, dy, reset=None, lens=None):
    """(dS_0, dq, dk, dv, dla, dbeta) of forward's (y, S_T)."""
    _, _, decayed, resid, states = saved
    B, T, Hk, dk = q.shape
    H = v.shape[2]
    q, k = (x.double().repeat_interleave(H // Hk, 2) for x in (q, k))
    la, beta, dy = la.double(), beta.double(), dy.double()
    dS = dS.double().clone()
    dq, dkk = torch.zeros_like(q), torch.zeros_like(k)
    dv, dla, dbeta = torch.zeros_like(dy), torch.zeros_like(la), torch.zeros_like(beta)
    for t in range(T - 1, -1, -1):
        live = torch.ones(B, dtype=torch.bool) if lens is None else t < lens
        m = live[:, None, None]
        keep = torch.exp(la[:, t])
        if reset is not None:
            keep = torch.where(reset[:, t, None] != 0, 0.0, keep)
        Sd, e, S = decayed[t], resid[t], states[t + 1]
        dq[:, t] = torch.where(m, (S * dy[:, t, :, None]).sum(3), 0.0)
        D = dS + q[:, t, :, :, None] * dy[:, t, :, None]
        du = (D * k[:, t, :, :, None]).sum(2)
        de = beta[:, t, :, None] * du
        dbeta[:, t] = torch.where(m[..., 0], (du * e).sum(-1), 0.0)
        dkk[:, t] = torch.where(m, (D * (beta[:, t, :, None] * e)[:, :, None]).sum(3) - (Sd * de[:, :, None]).sum(3), 0.0)
        dv[:, t] = torch.where(m, de, 0.0)
        dSd = D - k[:, t, :, :, None] * de[:, :, None]
        dla[:, t] = torch.where(m[..., 0], (dSd * Sd).sum((-1, -2)), 0.0)
        dS = torch.where(m[..., None], dSd * keep[..., None, None], dS)
    group = H // Hk
    dq, dkk = (x.reshape(B, T, Hk, group, dk).sum(3) for x in (dq, dkk))
    return dS, dq, dkk, dv, dla, dbeta


def sort_visits(sel, N):
    """(order, place, offsets) as lists."""
    flat = [int(x) for x in sel.flatten()]
    order = [i for p in range(N) for i, e in enumerate(flat) if e == p]
    place = [-1] * len(flat)
    for j, i in enumerate(order):
        place[i] = j
    offsets = [sum(0 <= e < p for e in flat) for p in range(N + 1)]
    return order + [-1] * (len(flat) - len(order)), place, offsets
