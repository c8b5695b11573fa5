"""The measured calls of the gated linear recurrence and of the 8-bit
activation checkpoints: cases, inputs, the plain form of each operator, its
definition in 64 bits, and the library's own calls (``own``).

The recurrence, for every channel (inputs x, r, g per token, rate per channel):

    L_t = -rate sigmoid(r_t),  a_t = exp(L_t),  m_t = sqrt(1 - a_t^2)
    h_t = a_t h_{t-1} + m_t sigmoid(g_t) x_t,   y_t = h_t

with h_{t-1} taken as 0 at a token whose reset flag is set, and only the first
lens[b] tokens of sequence b read or written.

An 8-bit checkpoint holds groups of 64 channels of one token as whole numbers
in [-127, 127] times a power of two, the smallest that fits the group.
"""
from __future__ import annotations

import math

import torch

own = False

GROUP = 64      # channels that share a step in an 8-bit checkpoint
SEGMENT = 8     # tokens between the states that a training forward keeps


def listed():
    return [
        # one new token of one sequence, the 1.4B layer's width: launch latency
        dict(name="step_single", op="scan", B=1, T=1, D=1920, dtype="bf16", fused=False, reset=False, lens=False),
        # one new token of a large serving batch, the 8B layer's width
        dict(name="step_batch", op="scan", B=256, T=1, D=3840, dtype="bf16", fused=True, reset=False, lens=False),
        # a padded batch of prompts; x, r, g are column slices of one projection
        dict(name="prefill_padded", op="scan", B=6, T=1531, D=1920, dtype="bf16", fused=True, reset=False, lens=True),
        # one long document: few channels, so the work has to be split over time
        dict(name="prefill_long", op="scan", B=1, T=32768, D=3840, dtype="bf16", fused=False, reset=False, lens=False),
        # fp32 activations at an odd width
        dict(name="prefill_fp32_odd", op="scan", B=3, T=2049, D=963, dtype="fp32", fused=False, reset=False,
             lens=False),
        # training steps: forward and backward.  A short one, the ordinary one (the 1.4B layer at the benchmark's
        # length), a packed one with 8-bit checkpoints (documents of any length in one row), a padded fp32 one
        dict(name="train_short", op="train", B=1, T=512, D=1920, dtype="bf16", fused=False, reset=False, lens=False,
             keep8=False),
        dict(name="train_layer", op="train", B=8, T=4096, D=1920, dtype="bf16", fused=False, reset=False, lens=False,
             keep8=False),
        dict(name="train_packed_keep8", op="train", B=2, T=8192, D=3840, dtype="bf16", fused=True, reset=True,
             lens=False, keep8=True),
        dict(name="train_fp32_keep8", op="train", B=3, T=1021, D=1285, dtype="fp32", fused=False, reset=False,
             lens=True, keep8=True),
        # checkpoints of other activations: one layer's short step, a whole batch's, fp32 scan outputs at an odd width
        dict(name="ckpt_short", op="ckpt", rows=512, D=1920, dtype="bf16", fused=False),
        dict(name="ckpt_large", op="ckpt", rows=32768, D=3840, dtype="bf16", fused=False),
        dict(name="ckpt_fp32_odd", op="ckpt", rows=8193, D=1955, dtype="fp32", fused=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "train", "train", "ckpt"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    D = _log(rng, 48, 3840)
    if rng.random() < 0.6:
        D = (D + 7) // 8 * 8
    if op == "ckpt":
        return dict(op=op, rows=min(_log(rng, 16, 32768), 60_000_000 // D), D=D, dtype=dtype,
                    fused=rng.random() < 0.3)
    if op == "scan" and rng.random() < 0.3:
        B, T = _log(rng, 1, 256), rng.choice([1, 1, 2, 5])
    else:
        B = _log(rng, 1, 16)
        most = 30_000_000 if dtype == "fp32" and op == "train" else 60_000_000      # elements
        T = max(1, min(_log(rng, 16, 32768), most // (B * D)))
    case = dict(op=op, B=B, T=T, D=D, dtype=dtype, fused=rng.random() < 0.4, reset=rng.random() < 0.4,
                lens=T > 1 and rng.random() < 0.4)
    if op == "train":
        case["keep8"] = rng.random() < 0.5
    return case


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    dt = _dtype(case)
    if case["op"] == "ckpt":
        rows, D = case["rows"], case["D"]
        # activations: a few channels much larger than the rest
        x = normal(rows, D + (D if case["fused"] else 0)) * torch.exp(0.7 * normal(D + (D if case["fused"] else 0)))
        x = x.to(dt)
        return {"case": case, "x": x[:, D:] if case["fused"] else x}
    B, T, D = case["B"], case["T"], case["D"]
    s = {"case": case}
    if case["fused"]:       # one projection's output: x | r | g
        p = normal(B, T, 3 * D).to(dt)
        s["x"], s["r"], s["g"] = p[..., :D], p[..., D:2 * D], p[..., 2 * D:]
    else:
        s["x"], s["r"], s["g"] = (normal(B, T, D).to(dt) for _ in range(3))
    # rate = -8 log of a base decay between 0.9 and 0.999, as such layers are started
    base = 0.9 + 0.099 * torch.rand(D, generator=gen, device="cuda", dtype=torch.float32)
    s["rate"] = -8.0 * torch.log(base)
    s["h0"] = normal(B, D)
    s["reset"] = s["lens"] = None
    if case["reset"]:       # documents of about 600 tokens, back to back
        s["reset"] = (torch.rand((B, T), generator=gen, device="cuda") < 1 / 600).to(torch.uint8)
    if case["lens"]:
        s["lens"] = torch.randint(max(1, T // 3), T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    s["y"] = torch.zeros((B, T, D), dtype=dt, device="cuda")
    s["hT"] = torch.empty((B, D), dtype=torch.float32, device="cuda")
    if case["op"] == "train":
        s["dy"] = normal(B, T, D).to(dt)
        s["dhT"] = normal(B, D)
        s["dx"], s["dr"], s["dg"] = (torch.zeros((B, T, D), dtype=dt, device="cuda") for _ in range(3))
        s["dh0"] = torch.empty((B, D), dtype=torch.float32, device="cuda")
    return s


# ---- the plain form: elementary torch operations in 32 bits ----

def _shares(x):
    """x [..., D] as groups [..., G, 64], zeros behind the last channel."""
    D = x.shape[-1]
    G = (D + GROUP - 1) // GROUP
    return torch.nn.functional.pad(x.float(), (0, G * GROUP - D)).reshape(*x.shape[:-1], G, GROUP)


def _through8(x):
    """The values that x's 8-bit checkpoint stands for, in 32 bits."""
    v = _shares(x)
    top = v.abs().amax(-1, keepdim=True)
    mant, e = torch.frexp(top)                      # top = mant 2^e, mant in [0.5, 1)
    e = torch.where(mant > 127 / 128, e + 1, e) - 7
    step = torch.ldexp(torch.ones_like(top), e.clamp(min=-126))
    return (torch.round(v / step) * step).flatten(-2)[..., :x.shape[-1]]


def _doubling(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 1 (h before the first is 0), by doubling the reach of each term."""
    k = 1
    while k < a.shape[1]:
        u = torch.cat([u[:, :k], u[:, k:] + a[:, k:] * u[:, :-k]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return u


def _gates(x, r, g, rate):
    sr, sg = torch.sigmoid(r), torch.sigmoid(g)
    L = -rate * sr
    m = torch.sqrt(-torch.expm1(2 * L))
    return sr, sg, torch.exp(L), m, m * sg * x


def _valid(s):
    T = s["x"].shape[1]
    if s["lens"] is None:
        return None
    return (torch.arange(T, device="cuda")[None] < s["lens"][:, None])[..., None]


def _states(s, a, u):
    """(a with resets and padding in place, all states h_1..h_T) in 32 bits."""
    valid = _valid(s)
    if s["reset"] is not None:
        a = a * (s["reset"] == 0).float()[..., None]
    if valid is not None:
        a, u = torch.where(valid, a, 1.0), torch.where(valid, u, 0.0)
    u = torch.cat([u[:, :1] + a[:, :1] * s["h0"][:, None], u[:, 1:]], 1)
    return a, _doubling(a, u)


def _put(buf, v, valid):
    v = v.to(buf.dtype)
    buf.copy_(v if valid is None else torch.where(valid, v, buf))
    return buf


def _plain_scan(s):
    *_, a, _, u = _gates(s["x"].float(), s["r"].float(), s["g"].float(), s["rate"])
    _, h = _states(s, a, u)
    return {"y": _put(s["y"], h, _valid(s)), "hT": h[:, -1].contiguous()}


def _plain_train(s):
    x, r, g = s["x"].float(), s["r"].float(), s["g"].float()
    rate, valid = s["rate"], _valid(s)
    sr, sg, a, m, u = _gates(x, r, g, rate)
    ar, h = _states(s, a, u)
    out = {"y": _put(s["y"], h, valid), "hT": h[:, -1].contiguous()}
    before = torch.cat([s["h0"][:, None], h[:, :-1]], 1)
    if s["case"]["keep8"]:
        x, r, g = _through8(s["x"]), _through8(s["r"]), _through8(s["g"])
        sr, sg, a, m, u = _gates(x, r, g, rate)
        ar = a if s["reset"] is None else a * (s["reset"] == 0).float()[..., None]
        if valid is not None:
            ar, u = torch.where(valid, ar, 1.0), torch.where(valid, u, 0.0)
        # the states inside each segment, from its kept first one and the checkpoint's values
        B, T, D = x.shape
        S = (T + SEGMENT - 1) // SEGMENT
        a8 = torch.nn.functional.pad(ar, (0, 0, 0, S * SEGMENT - T), value=1.0).reshape(B * S, SEGMENT, D)
        u8 = torch.nn.functional.pad(u, (0, 0, 0, S * SEGMENT - T)).reshape(B * S, SEGMENT, D)
        first = before[:, ::SEGMENT].reshape(B * S, 1, D)
        u8 = torch.cat([u8[:, :1] + a8[:, :1] * first, u8[:, 1:]], 1)
        h8 = _doubling(a8, u8)
        before = torch.cat([first, h8[:, :-1]], 1).reshape(B, S * SEGMENT, D)[:, :T]
    if s["reset"] is not None:
        before = before * (s["reset"] == 0).float()[..., None]
    dy = s["dy"].float()
    if valid is not None:
        dy = torch.where(valid, dy, 0.0)
    dy = torch.cat([dy[:, :-1], dy[:, -1:] + s["dhT"][:, None]], 1)
    after = torch.cat([ar[:, 1:], torch.ones_like(ar[:, :1])], 1)
    dh = _doubling(after.flip(1), dy.flip(1)).flip(1)
    out["dh0"] = (ar[:, 0] * dh[:, 0]).contiguous()
    dL = a * dh * (before - a / m * sg * x)
    if valid is not None:
        dL = torch.where(valid, dL, 0.0)
    out["dx"] = _put(s["dx"], dh * m * sg, valid)
    out["dr"] = _put(s["dr"], -rate * sr * (1 - sr) * dL, valid)
    out["dg"] = _put(s["dg"], dh * m * sg * (1 - sg) * x, valid)
    out["drate"] = (-sr * dL).sum((0, 1))
    return out


def run(state):
    s, case = state, state["case"]
    if not own:
        if case["op"] == "ckpt":
            return _through8(s["x"]).to(s["x"].dtype)
        return _plain_scan(s) if case["op"] == "scan" else _plain_train(s)
    import delta_rule_memory_gb300 as sdm
    if case["op"] == "ckpt":
        codes, exps = sdm.ckpt8_pack(s["x"])
        return sdm.ckpt8_unpack(codes, exps, s["x"].dtype)
    if case["op"] == "scan":
        y = sdm.glr_scan(s["h0"], s["x"], s["r"], s["g"], s["rate"], reset=s["reset"], lens=s["lens"], y=s["y"],
                         state_out=s["hT"])
        return {"y": y, "hT": s["hT"]}
    kept = sdm.glr_scan_train(s["h0"], s["x"], s["r"], s["g"], s["rate"], reset=s["reset"], lens=s["lens"],
                              keep8=case["keep8"], y=s["y"], state_out=s["hT"])
    saved = (None, None, None) if case["keep8"] else (s["x"], s["r"], s["g"])
    dx, dr, dg, drate = sdm.glr_scan_backward(s["dhT"], *saved, s["rate"], kept[1], s["dy"], reset=s["reset"],
                                              lens=s["lens"], ckpt=kept[2] if case["keep8"] else None,
                                              grads=(s["dx"], s["dr"], s["dg"]), dstate_out=s["dh0"])
    return {"y": kept[0], "hT": s["hT"], "dh0": s["dh0"], "dx": dx, "dr": dr, "dg": dg, "drate": drate}


def work(case):
    """Inputs once, outputs once; about 20 operations an element forward, 30 more backward."""
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "ckpt":        # packed and unpacked: the codes are written and read in between
        n = case["rows"] * case["D"]
        return {"bytes": n * (2 * es + 2) + 2 * case["rows"] * ((case["D"] + GROUP - 1) // GROUP), "flops": 4 * n}
    B, T, D = case["B"], case["T"], case["D"]
    n = B * T * D
    if case["lens"]:                # lengths between a third of T and T
        n = n * 2 // 3
    if case["op"] == "scan":
        return {"bytes": 4 * es * n + 8 * B * D + 4 * D, "flops": 20 * n}
    return {"bytes": 8 * es * n + 16 * B * D + 8 * D, "flops": 50 * n}


# ---- the definition in 64 bits, token by token ----

def _decoded64(x):
    """The checkpoint's values by its definition: the smallest power of two with max|x| <= 127 steps."""
    x = x.double()
    D = x.shape[-1]
    out = torch.empty_like(x)
    for c in range(0, D, GROUP):
        v = x[..., c:c + GROUP]
        e = torch.ceil(torch.log2(v.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -140) / 127)).clamp(min=-126)
        # log2 may be off by its last bit next to a power of two: settle it by the definition
        e = torch.where(v.abs().amax(-1, keepdim=True) > 127 * torch.exp2(e), e + 1, e)
        low = v.abs().amax(-1, keepdim=True) <= 127 * torch.exp2(e - 1)
        step = torch.exp2(torch.where(low & (e > -126), e - 1, e))
        out[..., c:c + GROUP] = torch.round(v / step) * step
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ckpt":
        return _decoded64(s["x"])
    B, T, D = s["x"].shape
    rate, h = s["rate"].double(), s["h0"].double()
    lens = s["lens"] if s["lens"] is not None else torch.full((B,), T, device="cuda", dtype=torch.int32)
    live = torch.arange(T, device="cuda")[:, None] < lens[None]                     # [T, B]
    keep = live.double()[..., None]
    past = torch.ones(T, B, 1, device="cuda", dtype=torch.float64)
    if s["reset"] is not None:
        past = (s["reset"] == 0).t().double()[..., None].contiguous()

    def terms(x, r, g):     # [T, B, D]: decay, sigmoid(r), sigmoid(g), m, x
        x, r, g = (v.double().transpose(0, 1).contiguous() for v in (x, r, g))
        sr, sg = 1 / (1 + torch.exp(-r)), 1 / (1 + torch.exp(-g))
        L = -rate * sr
        return torch.exp(L), sr, sg, torch.sqrt(-torch.expm1(2 * L)), x

    a, sr, sg, m, x = terms(s["x"], s["r"], s["g"])
    f = torch.where(keep > 0, a * past, 1.0)
    u = m * sg * x * keep
    hs = torch.empty(T + 1, B, D, device="cuda", dtype=torch.float64)
    hs[0] = h
    for t in range(T):
        torch.addcmul(u[t], f[t], hs[t], out=hs[t + 1])
    bt = lambda v, dead: torch.where(keep > 0, v, dead).transpose(0, 1).contiguous()  # noqa: E731
    out = {"y": bt(hs[1:], 0.0), "hT": hs[T].clone()}
    if case["op"] == "scan":
        return out
    before = hs[:T]
    if case["keep8"]:
        a, sr, sg, m, x = terms(_decoded64(s["x"]), _decoded64(s["r"]), _decoded64(s["g"]))
        f = torch.where(keep > 0, a * past, 1.0)
        u = m * sg * x * keep
        before = before.clone()
        for i in range(1, SEGMENT):     # token i of every segment, from token i - 1
            n = len(range(i, T, SEGMENT))
            before[i::SEGMENT] = f[i - 1::SEGMENT][:n] * before[i - 1::SEGMENT][:n] + u[i - 1::SEGMENT][:n]
    dh = torch.empty_like(u)
    at = s["dhT"].double()
    dy = s["dy"].double().transpose(0, 1).contiguous() * keep
    for t in range(T - 1, -1, -1):
        torch.add(dy[t], at, out=dh[t])
        at = f[t] * dh[t]
    dL = a * dh * (before * past - a / m * sg * x)
    out["dh0"] = at
    out["dx"] = bt(dh * m * sg, 0.0)
    out["dr"] = bt(-rate * sr * (1 - sr) * dL, 0.0)
    out["dg"] = bt(dh * m * sg * (1 - sg) * x, 0.0)
    out["drate"] = (-sr * dL * keep).sum((0, 1))
    return out
