"""The measured calls of the gated delta rule's training and decoding forms and
of the visits sorted by partition: cases, inputs, the plain form of each
operator, its definition in 64 bits, and the library's own calls (``own``).

The gated delta rule, per sequence and value head h (key head h // (H / Hk)),
on a state S [dk, dv]:

    S~ = exp(log_alpha_t) S_{t-1}      (0 where token t resets)
    E_t = v_t - S~^T k_t,   S_t = S~ + beta_t k_t E_t^T,   y_t = S_t^T q_t

with only the first lens[b] tokens of sequence b read or written.  Training
returns y, S_T and the gradients of all inputs and of S_0; a decoding step
advances the states that `slots` names in a pool by T tokens.

Visits: token m has k of them, visit (m, r) to partition sel[m, r].  Sorted by
partition, equal ones by (m, r); a visit with sel -1 is dropped.  `gather`
copies each token's row to its visits' places, `combine` sums the rows at a
token's places times its weights.
"""
from __future__ import annotations

import math

import torch

own = False

C = 64          # tokens of a chunk in the plain form


def listed():
    gdn = dict(op="gdn", fused=False, reset=False, lens=False)
    return [
        # training steps of a gated delta layer.  A short one with two value heads to a key head: latency
        dict(gdn, name="gdn_short", B=1, T=200, Hk=2, H=4, dk=64, dv=64),
        # the dense benchmark's layer
        dict(gdn, name="gdn_layer", B=4, T=4096, Hk=16, H=16, dk=128, dv=128),
        # packed documents; q, k, v are slices of one projection, four value heads share a key head
        dict(gdn, name="gdn_packed_grouped", B=2, T=4093, Hk=4, H=16, dk=128, dv=128, fused=True, reset=True),
        # a padded batch at odd widths
        dict(gdn, name="gdn_padded_odd", B=3, T=1021, Hk=6, H=6, dk=100, dv=72, lens=True),
        # one long document: few sequences, many chunks in a row
        dict(gdn, name="gdn_long", B=1, T=16384, Hk=8, H=8, dk=128, dv=128),
        # decoding: one sequence; a large batch out of a pool of states; a few drafted tokens at odd widths
        dict(name="step_single", op="step", B=1, T=1, Hk=16, H=16, dk=128, dv=128, P=1, fused=False),
        dict(name="step_batch", op="step", B=256, T=1, Hk=4, H=16, dk=128, dv=128, P=300, fused=True),
        dict(name="step_draft_odd", op="step", B=24, T=5, Hk=6, H=6, dk=100, dv=72, P=40, fused=False),
        # routing: a decoding batch, a prefill with two visits a token, a training step with four visits to 64
        # partitions at the 8B layer's width, a small fp32 one at an odd width where a tenth of the visits is dropped
        dict(name="route_decode", op="route", M=64, k=2, N=8, D=1920, dtype="bf16", train=False, drop=False),
        dict(name="route_prefill", op="route", M=16384, k=2, N=8, D=1920, dtype="bf16", train=False, drop=False),
        dict(name="route_train", op="route", M=16384, k=4, N=64, D=3840, dtype="bf16", train=True, drop=False),
        dict(name="route_train_fp32_odd", op="route", M=4099, k=3, N=13, D=963, dtype="fp32", train=True, drop=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gdn", "gdn", "gdn", "step", "route", "route"])
    if op == "route":
        D, k = _log(rng, 48, 3840), rng.choice([1, 2, 2, 3, 4, 8])
        if rng.random() < 0.6:
            D = (D + 7) // 8 * 8
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        M = max(1, min(_log(rng, 1, 32768), (100_000_000 if dtype == "fp32" else 200_000_000) // (k * D)))
        return dict(op=op, M=M, k=k, N=_log(rng, 2, 128), D=D, dtype=dtype, train=rng.random() < 0.5,
                    drop=rng.random() < 0.3)
    Hk, group = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 4])
    H = min(Hk * group, 16)
    Hk = H // group if H % group == 0 else H
    if rng.random() < 0.5:
        dk = dv = 128
    else:
        dk, dv = rng.randint(16, 128), rng.randint(16, 192)
        if rng.random() < 0.5:
            dk, dv = dk // 8 * 8, dv // 8 * 8
    case = dict(op=op, Hk=Hk, H=H, dk=dk, dv=dv, fused=rng.random() < 0.4)
    if op == "step":
        B = _log(rng, 1, 256)
        return dict(case, B=B, T=rng.choice([1, 1, 1, 2, 4, 7]), P=B + rng.randint(0, 40))
    B = _log(rng, 1, 8)
    T = max(1, min(_log(rng, 16, 8192), 3_000_000_000 // (B * H * dk * dv)))
    return dict(case, B=B, T=T, reset=rng.random() < 0.4, lens=rng.random() < 0.4)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    s = {"case": case}
    if case["op"] == "route":
        M, k, N, D = (case[n] for n in ("M", "k", "N", "D"))
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        # a router's choices: its top k of N logits with a preference of its own (distinct where k <= N)
        logits = normal(M, N) + normal(N)
        e, sel = torch.sort(logits, dim=1, descending=True)
        s["sel"] = sel[:, torch.arange(k, device="cuda") % N].to(torch.int32).contiguous()
        s["w"] = torch.softmax(e, 1)[:, torch.arange(k, device="cuda") % N].contiguous()
        if case["drop"]:
            s["sel"] = torch.where(torch.rand((M, k), generator=gen, device="cuda") < 0.1, -1, s["sel"])
        s["x"] = normal(M, D).to(dt)
        s["out"] = normal(M * k, D).to(dt)                  # what the partitions' products answer
        if case["train"]:
            s["dy"] = normal(M, D).to(dt)
            s["dp"] = normal(M * k, D).to(dt)               # the gradient of the partitions' inputs
        return s
    B, T, Hk, H, dk, dv = (case[n] for n in ("B", "T", "Hk", "H", "dk", "dv"))

    def unit(v):        # keys and queries of length 1
        return v / v.square().sum(-1, keepdim=True).sqrt()

    q, k, v = unit(normal(B, T, Hk, dk)), unit(normal(B, T, Hk, dk)), normal(B, T, H, dv)
    if case["fused"]:       # one projection's output: q | k | v
        p = torch.cat([x.flatten(2) for x in (q, k, v)], -1).to(torch.bfloat16)
        q, k, v = p.split([Hk * dk, Hk * dk, H * dv], -1)
        s["q"], s["k"], s["v"] = q.unflatten(-1, (Hk, dk)), k.unflatten(-1, (Hk, dk)), v.unflatten(-1, (H, dv))
    else:
        s["q"], s["k"], s["v"] = (x.to(torch.bfloat16) for x in (q, k, v))
    # heads that forget within a few tokens up to heads that remember for hundreds
    rate = torch.exp(torch.linspace(math.log(0.01), 0.0, H, device="cuda"))
    s["la"] = -rate * torch.nn.functional.softplus(normal(B, T, H))
    s["beta"] = torch.sigmoid(normal(B, T, H))
    if case["op"] == "step":
        P = case["P"]
        s["pool"] = 0.3 * normal(P, H, dk, dv)
        s["slots"] = torch.randperm(P, generator=gen, device="cuda")[:B].to(torch.int32)
        s["y"] = torch.empty((B, T, H, dv), dtype=torch.bfloat16, device="cuda")
        return s
    s["h0"] = 0.3 * normal(B, H, dk, dv)
    s["hT"] = torch.empty_like(s["h0"])
    s["reset"] = s["lens"] = None
    if case["reset"]:       # documents of about 600 tokens, back to back
        s["reset"] = (torch.rand((B, T), generator=gen, device="cuda") < 1 / 600).to(torch.uint8)
    if case["lens"]:
        s["lens"] = torch.randint(max(1, T // 3), T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    s["dy"] = normal(B, T, H, dv).to(torch.bfloat16)
    s["dhT"] = 0.3 * normal(B, H, dk, dv)
    return s


# ---- the plain form: elementary torch operations in 32 bits (decays' sums in 64) ----

def _inverse(L):
    """Inverse of unit lower triangular [..., C, C]: the diagonal blocks' inverses joined two by two."""
    n = L.shape[-1]
    at = torch.arange(n, device=L.device)
    X, size = torch.eye(n, device=L.device, dtype=L.dtype).expand_as(L), 1
    while size < n:     # the block below the diagonal between the two halves of each block of 2 * size
        low = (at[:, None] // size % 2 == 1) & (at[None] // size == at[:, None] // size - 1)
        X = X - X @ (L * low) @ X
        size *= 2
    return X


def _plain_gdn(s):
    case = s["case"]
    B, T, Hk, H, dk, dv = (case[n] for n in ("B", "T", "Hk", "H", "dk", "dv"))
    n = (T + C - 1) // C
    live = torch.ones(B, T, dtype=torch.bool, device="cuda")
    if s["lens"] is not None:
        live = torch.arange(T, device="cuda")[None] < s["lens"][:, None]

    def rows(x, head):      # [B, T, heads, d] -> [B, H, n, C, d], zeros where there is no token
        x = torch.where(live[:, :, None, None], x.float(), 0.0)
        if x.shape[2] != head:
            x = x.repeat_interleave(head // x.shape[2], 2)
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, n * C - T))
        return x.reshape(B, n, C, head, -1).permute(0, 3, 1, 2, 4)

    q, k, v, dy = rows(s["q"], H), rows(s["k"], H), rows(s["v"], H), rows(s["dy"], H)
    beta = rows(s["beta"][..., None], H)                                        # [B,H,n,C,1]
    lam = rows(s["la"][..., None], H)[..., 0].double().cumsum(-1)               # [B,H,n,C]
    seg = torch.zeros(B, n, C, device="cuda")
    if s["reset"] is not None:
        seg = torch.nn.functional.pad((s["reset"] != 0).float() * live, (0, n * C - T)).reshape(B, n, C).cumsum(-1)
    seg = seg[:, None]                                                          # [B,1,n,C]
    same = seg[..., :, None] == seg[..., None, :]
    at = torch.arange(C, device="cuda")
    D = torch.exp((lam[..., :, None] - lam[..., None, :]).clamp(max=0).float())     # decay from token j to token i
    D = torch.where(same & (at[:, None] >= at[None]), D, 0.0)
    strict = D * (at[:, None] > at[None])
    gam = torch.where(seg == 0, torch.exp(lam.float()), 0.0)[..., None]         # decay since the chunk's start
    tail = torch.where(seg == seg[..., -1:], torch.exp((lam[..., -1:] - lam).float()), 0.0)[..., None]
    end = gam[..., -1:, :]                                                      # [B,H,n,1,1]
    kt, qt = k.transpose(-1, -2), q.transpose(-1, -2)
    inv = _inverse(torch.eye(C, device="cuda") + strict * (k @ kt) * beta.transpose(-1, -2))
    mq = D * (q @ kt)
    W, E = inv @ (gam * k), inv @ v                                             # E_t = E - W S
    S, states, Es = s["h0"], [], []
    for c in range(n):
        e = E[:, :, c] - W[:, :, c] @ S
        states.append(S)
        Es.append(e)
        S = end[:, :, c] * S + kt[:, :, c] @ (tail[:, :, c] * beta[:, :, c] * e)
    s["hT"].copy_(S)
    S0, E = torch.stack(states, 2), torch.stack(Es, 2)
    U = beta * E
    y = gam * (q @ S0) + mq @ U
    # backward
    dU0, Qd = mq.transpose(-1, -2) @ dy, qt @ (gam * dy)
    dS, ends, dZs = s["dhT"], [None] * n, [None] * n
    for c in range(n - 1, -1, -1):
        ends[c] = dS
        du = dU0[:, :, c] + tail[:, :, c] * (k[:, :, c] @ dS)
        dZs[c] = inv[:, :, c].transpose(-1, -2) @ (beta[:, :, c] * du)
        dS = end[:, :, c] * dS + Qd[:, :, c] - kt[:, :, c] @ (gam[:, :, c] * dZs[c])
    dSe, dZ = torch.stack(ends, 2), torch.stack(dZs, 2)
    dSet = dSe.transpose(-1, -2)
    dU = dU0 + tail * (k @ dSe)
    x = D * (dy @ U.transpose(-1, -2))
    z = -strict * (dZ @ U.transpose(-1, -2))
    S0t = S0.transpose(-1, -2)
    dq = gam * (dy @ S0t) + x @ k
    dk = tail * (U @ dSet) - gam * (dZ @ S0t) + x.transpose(-1, -2) @ q + (z + z.transpose(-1, -2)) @ k
    # dbeta_t = E_t . (dU - strict^T dZ) with (k k^T): the gradient that reaches U_t from its chunk and from behind it
    dbeta = ((dU - (strict * (k @ kt)).transpose(-1, -2) @ dZ) * E).sum(-1)
    # every output is linear in (S_0, v): what a decay scales is what the later outputs get through it
    flow = ((q * dq).sum(-1) - (v * dZ).sum(-1)).double()
    behind = flow.flip(-1).cumsum(-1).flip(-1)                                  # sum over t.. to the chunk's end
    nxt = torch.where(seg[..., None, :] == seg[..., :, None] + 1, at, C).amin(-1)   # the next segment's start
    cut = torch.where(nxt < C, torch.gather(behind, -1, nxt.clamp(max=C - 1).expand_as(behind)), 0.0)
    SC = torch.cat([S0[:, :, 1:], S[:, :, None]], 2)
    whole = (SC * dSe).sum((-1, -2)).double()[..., None]
    dla = behind - cut + torch.where(seg == seg[..., -1:], whole, 0.0)
    starts = (seg != torch.nn.functional.pad(seg, (1, 0))[..., :-1])
    dla = torch.where(starts, 0.0, dla)

    def back(x, group=1):   # [B,H,n,C,d] -> [B,T,H / group,d]
        x = x.permute(0, 2, 3, 1, 4).reshape(B, n * C, H // group, group, -1).sum(3)[:, :T]
        return torch.where(live[:, :, None, None], x, 0.0)

    bf = torch.bfloat16
    return {"y": back(y).to(bf), "hT": s["hT"], "dh0": dS, "dq": back(dq, H // Hk).to(bf),
            "dk": back(dk, H // Hk).to(bf), "dv": back(dZ).to(bf), "dla": back(dla.float()[..., None])[..., 0],
            "dbeta": back(dbeta[..., None])[..., 0]}


def _plain_step(s):
    case = s["case"]
    group = case["H"] // case["Hk"]
    at = s["slots"].long()
    S = s["pool"][at]
    y = []
    for t in range(case["T"]):
        q, k = (s[n][:, t].float().repeat_interleave(group, 1)[..., None] for n in ("q", "k"))     # [B,H,dk,1]
        S = torch.exp(s["la"][:, t])[..., None, None] * S
        e = s["v"][:, t].float() - (S * k).sum(-2)
        S = S + k * (s["beta"][:, t, :, None] * e)[..., None, :]
        y.append((S * q).sum(-2))
    s["pool"][at] = S
    return {"y": s["y"].copy_(torch.stack(y, 1)), "pool": s["pool"]}


def _plain_route(s):
    case = s["case"]
    M, k, N, D = (case[n] for n in ("M", "k", "N", "D"))
    key = s["sel"].flatten().long()
    key = torch.where(key < 0, N, key)
    mine = key[:, None] == torch.arange(N + 1, device="cuda")                   # [M k, N + 1]
    rank = torch.where(mine, mine.long().cumsum(0) - 1, 0).sum(1)
    ends = mine.sum(0).cumsum(0)
    starts = torch.cat([ends.new_zeros(1), ends])
    row = starts[key] + rank
    kept = key < N
    visit = torch.arange(M * k, device="cuda")
    order = torch.empty_like(visit)
    order[row] = torch.where(kept, visit, -1)
    place = torch.where(kept, row, -1).reshape(M, k)
    dt = s["x"].dtype
    rows = torch.where((order >= 0)[:, None], s["x"][(order // k).clamp(min=0)], 0)
    i32 = torch.int32
    out = {"order": order.to(i32), "place": place.to(i32), "offsets": starts[:N + 1].to(i32), "rows": rows}
    w, have = s["w"][..., None], (place >= 0)[..., None]

    def at(rows):           # [M, k, D] of the rows at each token's places
        return torch.where(have, rows[place.clamp(min=0)].float(), 0.0)

    o = at(s["out"])
    out["y"] = (w * o).sum(1).to(dt)
    if case["train"]:
        dy = s["dy"].float()[:, None]
        do = torch.zeros(M * k, D, dtype=dt, device="cuda")
        do[row] = torch.where(have, w * dy, 0.0).to(dt).flatten(0, 1)
        out["dout"], out["dw"] = do, (o * dy).sum(-1)
        out["dx"] = at(s["dp"]).sum(1).to(dt)
    return out


def run(state):
    s, case = state, state["case"]
    if not own:
        return {"gdn": _plain_gdn, "step": _plain_step, "route": _plain_route}[case["op"]](s)
    import delta_rule_memory_gb300 as sdm
    if case["op"] == "step":
        y = sdm.gdn_step(s["pool"], s["q"], s["k"], s["v"], s["la"], s["beta"], slots=s["slots"], y=s["y"])
        return {"y": y, "pool": s["pool"]}
    if case["op"] == "gdn":
        y, saved = sdm.gdn_train(s["h0"], s["q"], s["k"], s["v"], s["la"], s["beta"], reset=s["reset"], lens=s["lens"],
                                 state_out=s["hT"])
        dh0 = torch.empty_like(s["h0"])
        dq, dk, dv, dla, dbeta = sdm.gdn_backward(s["dhT"], s["q"], s["k"], s["v"], s["la"], s["beta"], saved, s["dy"],
                                                  reset=s["reset"], lens=s["lens"], dstate_out=dh0)
        return {"y": y, "hT": s["hT"], "dh0": dh0, "dq": dq, "dk": dk, "dv": dv, "dla": dla, "dbeta": dbeta}
    order, place, offsets = sdm.route_sort(s["sel"], case["N"])
    out = {"order": order, "place": place, "offsets": offsets, "rows": sdm.route_gather(s["x"], place, offsets),
           "y": sdm.route_combine(s["out"], place, s["w"])}
    if case["train"]:
        out["dout"], out["dw"] = sdm.route_combine_backward(s["dy"], s["out"], place, s["w"], offsets)
        out["dx"] = sdm.route_combine(s["dp"], place)
    return out


def work(case):
    """Inputs once, outputs once.  The recurrence: 8 dk dv operations a token and head forward, 20 more backward."""
    if case["op"] == "route":
        es, n = 2 if case["dtype"] == "bf16" else 4, case["M"] * case["D"]
        nbytes = 16 * case["M"] * case["k"] + es * n * (2 + 2 * case["k"])
        if case["train"]:       # dy and the places' rows in, a row for each place, dw and dx out
            nbytes += es * n * (2 + 2 * case["k"]) + 4 * case["M"] * case["k"]
        return {"bytes": nbytes, "flops": n * case["k"] * (6 if case["train"] else 2)}
    B, T, Hk, H, dk, dv = (case[n] for n in ("B", "T", "Hk", "H", "dk", "dv"))
    token = 2 * 2 * Hk * dk + 2 * 2 * H * dv + 8 * H        # q, k, v, y, the two gates
    if case["op"] == "step":
        return {"bytes": B * (8 * H * dk * dv + T * token), "flops": 8 * B * T * H * dk * dv}
    n = B * T * 2 // 3 if case["lens"] else B * T           # lengths between a third of T and T
    grads = 2 * 2 * Hk * dk + 2 * H * dv + 8 * H            # dq, dk, dv, the gates'
    return {"bytes": n * (token + grads + 2 * H * dv) + 16 * B * H * dk * dv, "flops": 28 * n * H * dk * dv}


# ---- the definition in 64 bits, token by token ----

def _exact_route(s, case):
    M, k, N, D = (case[n] for n in ("M", "k", "N", "D"))
    sel = s["sel"].flatten().tolist()
    order = [i for _, i in sorted((e, i) for i, e in enumerate(sel) if e >= 0)]
    counts = [0] * (N + 1)
    for e in sel:
        if e >= 0:
            counts[e + 1] += 1
    for p in range(N):
        counts[p + 1] += counts[p]
    place = [-1] * (M * k)
    for j, i in enumerate(order):
        place[i] = j
    dev = dict(device="cuda")
    idx = torch.tensor(order, dtype=torch.long, **dev)
    out = {"order": torch.tensor(order + [-1] * (M * k - len(order)), dtype=torch.int32, **dev),
           "place": torch.tensor(place, dtype=torch.int32, **dev).reshape(M, k),
           "offsets": torch.tensor(counts, dtype=torch.int32, **dev)}
    rows = torch.zeros(M * k, D, dtype=torch.float64, **dev)
    rows[:len(order)] = s["x"].double()[idx // k]
    out["rows"] = rows
    y = torch.zeros(M, D, dtype=torch.float64, **dev)
    y.index_add_(0, idx // k, s["out"][:len(order)].double() * s["w"].flatten().double()[idx][:, None])
    out["y"] = y
    if case["train"]:
        dy, wv = s["dy"].double()[idx // k], s["w"].flatten().double()[idx]
        dout = torch.zeros_like(rows)
        dout[:len(order)] = dy * wv[:, None]
        dw = torch.zeros(M * k, dtype=torch.float64, **dev)
        dw[idx] = (dy * s["out"][:len(order)].double()).sum(1)
        dx = torch.zeros_like(y)
        dx.index_add_(0, idx // k, s["dp"][:len(order)].double())
        out.update(dout=dout, dw=dw.reshape(M, k), dx=dx)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s, case)
    B, T, Hk, H, dk, dv = (case[n] for n in ("B", "T", "Hk", "H", "dk", "dv"))
    heads = torch.arange(H, device="cuda") // (H // Hk)
    q, k = s["q"].double()[:, :, heads].transpose(0, 1), s["k"].double()[:, :, heads].transpose(0, 1)    # [T,B,H,dk]
    v, beta = s["v"].double().transpose(0, 1), s["beta"].double().transpose(0, 1)
    decay = torch.exp(s["la"].double()).transpose(0, 1)                                                  # [T,B,H]
    if case["op"] == "step":
        S = s["pool"].double()[s["slots"].long()]
        y = torch.empty(T, B, H, dv, dtype=torch.float64, device="cuda")
        for t in range(T):
            S = S * decay[t][..., None, None]
            e = v[t] - torch.einsum("bhij,bhi->bhj", S, k[t])
            S = S + torch.einsum("bhi,bhj->bhij", k[t], beta[t][..., None] * e)
            y[t] = torch.einsum("bhij,bhi->bhj", S, q[t])
        pool = s["pool"].double()
        pool[s["slots"].long()] = S
        return {"y": y.transpose(0, 1), "pool": pool}
    live = torch.ones(T, B, dtype=torch.bool, device="cuda")
    if s["lens"] is not None:
        live = torch.arange(T, device="cuda")[:, None] < s["lens"][None]
    keep = decay
    if s["reset"] is not None:
        keep = torch.where((s["reset"] != 0).t()[..., None], 0.0, keep)
    zero = lambda x: torch.where(live.reshape(T, B, *[1] * (x.dim() - 2)), x, 0.0)  # noqa: E731
    q, k, v, beta, dy = zero(q), zero(k), zero(v), zero(beta), zero(s["dy"].double().transpose(0, 1))
    keep = torch.where(live[..., None], keep, 1.0).contiguous()

    def advance(S, t):      # (S~, E, S after token t)
        Sd = S * keep[t][..., None, None]
        e = v[t] - (k[t][..., None, :] @ Sd)[..., 0, :]
        return Sd, e, Sd + k[t][..., None] * (beta[t][..., None] * e)[..., None, :]

    S, marks = s["h0"].double(), []
    y = torch.empty(T, B, H, dv, dtype=torch.float64, device="cuda")
    for t in range(T):
        if t % 64 == 0:
            marks.append(S)
        S = advance(S, t)[2]
        y[t] = (q[t][..., None, :] @ S)[..., 0, :]
    out = {"y": y.transpose(0, 1), "hT": S}
    dq, dkk = torch.zeros_like(q), torch.zeros_like(k)
    dvv, dla, dbeta = torch.zeros_like(v), torch.zeros_like(beta), torch.zeros_like(beta)
    dS = s["dhT"].double()
    for m in range(len(marks) - 1, -1, -1):
        S, kept = marks[m], []
        for t in range(64 * m, min(64 * m + 64, T)):
            kept.append(advance(S, t))
            S = kept[-1][2]
        for t in range(min(64 * m + 64, T) - 1, 64 * m - 1, -1):
            Sd, e, S = kept[t - 64 * m]
            dq[t] = (S @ dy[t][..., None])[..., 0]
            dS = dS + q[t][..., None] * dy[t][..., None, :]
            du = (k[t][..., None, :] @ dS)[..., 0, :]
            dbeta[t] = (du * e).sum(-1)
            de = beta[t][..., None] * du
            dkk[t] = (dS @ (beta[t][..., None] * e)[..., None])[..., 0] - (Sd @ de[..., None])[..., 0]
            dvv[t] = de
            dSd = dS - k[t][..., None] * de[..., None, :]
            dla[t] = (dSd * Sd).sum((-1, -2))
            dS = dSd * keep[t][..., None, None]
    bt = lambda x: zero(x).transpose(0, 1).contiguous()  # noqa: E731
    shared = lambda x: bt(x).reshape(B, T, Hk, H // Hk, dk).sum(3)  # noqa: E731
    out.update(dh0=dS, dq=shared(dq), dk=shared(dkk), dv=bt(dvv), dla=bt(dla), dbeta=bt(dbeta))
    return out
