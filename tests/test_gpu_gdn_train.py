"""gdn_train, gdn_backward and gdn_step against the 64-bit token-by-token
formulas.

Tolerances.  y, dq, dk and dv are rounded once to bf16: at most 2^-8 of the
value off.  Inside, what reaches only them is held in two bf16 parts, 16 bits:
each product is at most 2 * 2^-17 off relative to itself, and a sum of n <= 320
such terms at most sqrt(n) 2^-16 < 2^-11 relative to the root mean square of
the sums (terms of like size and either sign).  Everything else is fp32-exact
(2^-24 an operation): the states' and gates' gradients pass at most 2^7
roundings a chunk that the decays do not shrink: 2^-17 in the 2-norm; the
decay's gradient, a sum of up to 64 cancelling terms, 8 times that."""
import itertools

import pytest
import torch

import gdn_reference as ref
from helpers import need_gpu

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, B, T, Hk, H, dk, dv, seed=0, reset=0.0, lens=None, fused=False, decay=1.0, offset=0):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.dims = B, T, Hk, H, dk, dv
        q, k, v = n(B, T, Hk, dk), n(B, T, Hk, dk), n(B, T, H, dv)
        q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
        self.q, self.k, self.v = (x.to(torch.bfloat16) for x in (q, k, v))
        self.la = -decay * torch.nn.functional.softplus(n(B, T, H))
        self.beta = torch.sigmoid(n(B, T, H))
        self.S0, self.dS, self.dy = 0.3 * n(B, H, dk, dv), 0.3 * n(B, H, dk, dv), n(B, T, H, dv).to(torch.bfloat16)
        self.reset = (torch.rand((B, T), generator=g) < reset).to(torch.uint8) if reset else None
        self.lens = None if lens is None else torch.tensor(lens, dtype=torch.int32)
        self.fused, self.offset = fused, offset

    def layout(self, q, k, v):
        """On the device: contiguous, or as slices of one projection `offset` elements off its start."""
        if not self.fused:
            return [x.cuda() for x in (q, k, v)]
        B, T, Hk, H, dk, dv = self.dims
        W = 2 * Hk * dk + H * dv
        buf = torch.full((B * T * (W + 3) + 64,), float("nan"), dtype=torch.bfloat16, device="cuda")[self.offset:]
        p = buf[:B * T * (W + 3)].view(B, T, W + 3)
        out = []
        for x, at in ((q, 0), (k, Hk * dk), (v, 2 * Hk * dk)):
            s = p[..., at:at + x.shape[2] * x.shape[3]].unflatten(-1, tuple(x.shape[2:]))
            s.copy_(x)
            out.append(s)
        return out

    def gates(self):
        return self.la.cuda(), self.beta.cuda()

    def masks(self):
        return dict(reset=None if self.reset is None else self.reset.cuda(), lens=None if self.lens is None else self.lens.cuda())

    def reference(self):
        a = (self.q, self.k, self.v, self.la, self.beta)
        f = ref.forward(self.S0, *a, self.reset, self.lens)
        return f, ref.backward(f, self.dS, *a, self.dy, self.reset, self.lens)

    def run(self, sdm, **kw):
        x, m = [*self.layout(self.q, self.k, self.v), *self.gates()], self.masks()
        ST, d0 = torch.empty_like(self.S0, device="cuda"), torch.empty_like(self.S0, device="cuda")
        y, saved = sdm.gdn_train(self.S0.cuda(), *x, **m, state_out=ST, **kw)
        g = sdm.gdn_backward(self.dS.cuda(), *x, saved, self.dy.cuda(), **m, dstate_out=d0, **kw)
        return (y, ST), (d0, *g)


def close16(got, want, what):
    """bf16 outputs: the rounding, and the 16 bits of what went into them."""
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape
    rms = float(want.square().mean().sqrt()) if want.numel() else 0.0
    off = (got - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -11 * rms + 1e-30)
    assert bool((off <= 0).all()), f"{what}: {float(off.max()):.3e} over the bound, rms {rms:.3e}"


def close32(got, want, what, bound=2.0 ** -17):
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape and bool(torch.isfinite(got).all()), what
    err, size = float((got - want).norm()), float(want.norm())
    assert err <= bound * size + 1e-30, f"{what}: {err / max(size, 1e-30):.3e} of the norm"


def check(case, out, f, b):
    (y, ST), (d0, dq, dk, dv, dla, dbeta) = out
    close16(y, f[0], "y")
    close32(ST, f[1], "state")
    for got, want, n in ((dq, b[1], "dq"), (dk, b[2], "dk"), (dv, b[3], "dv")):
        close16(got, want, n)
    close32(d0, b[0], "dstate")
    close32(dbeta, b[5], "dbeta")
    close32(dla, b[4], "dlog_alpha", 2.0 ** -14)


SHAPES = [(1, 1, 1, 1, 1, 1), (2, 5, 1, 2, 7, 3), (1, 63, 2, 2, 16, 16), (2, 64, 1, 1, 64, 64), (1, 65, 2, 4, 100, 72),
          (2, 130, 3, 3, 128, 128), (1, 129, 1, 2, 65, 33), (1, 200, 1, 4, 128, 130), (1, 70, 2, 2, 33, 257), (3, 192, 2, 6, 96, 48)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("reset,fused", [(0.0, False), (0.05, True)])
def test_parity(shape, reset, fused):
    sdm = need_gpu()
    c = Case(*shape, seed=sum(shape), reset=reset, fused=fused)
    check(c, c.run(sdm), *c.reference())
    sdm.sdm_check()


@pytest.mark.parametrize("lens", [[0, 130, 64, 1], [65, 0, 0, 127]])
def test_padded_batch(lens):
    """Tokens behind lens: NaN there reaches nothing, and rows of given buffers keep their bits."""
    sdm = need_gpu()
    c = Case(4, 130, 1, 2, 128, 48, seed=9, lens=lens, reset=0.03)
    f, b = c.reference()
    dead = torch.arange(130)[None] >= c.lens[:, None]
    for x in (c.q, c.k, c.v, c.la, c.beta, c.dy):
        x[dead] = float("nan")
    check(c, c.run(sdm), f, b)
    x, m = [*c.layout(c.q, c.k, c.v), *c.gates()], c.masks()
    y = torch.full((4, 130, 2, 48), 7.0, dtype=torch.bfloat16, device="cuda")
    grads = [torch.full_like(t, 7.0) for t in x[:3]]
    _, saved = sdm.gdn_train(c.S0.cuda(), *x, **m, y=y)
    sdm.gdn_backward(c.dS.cuda(), *x, saved, c.dy.cuda(), **m, grads=grads)
    for t in (y, *grads):
        assert bool((t[dead.cuda()] == 7.0).all())
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    m["lens"] = torch.tensor([131, -1, 5, 64], dtype=torch.int32, device="cuda")
    sdm.gdn_train(c.S0.cuda(), *x, **m, dev_err=err)
    assert int(err) == sdm.SDM_DEVERR_INDEX_RANGE


@pytest.mark.parametrize("at", [[0], [63], [64], [1, 2, 3], [0, 64, 127], list(range(130))], ids=str)
def test_resets(at):
    sdm = need_gpu()
    c = Case(1, 130, 1, 1, 32, 16, seed=3)
    c.reset = torch.zeros((1, 130), dtype=torch.uint8)
    c.reset[0, at] = 1
    out = c.run(sdm)
    check(c, out, *c.reference())
    assert bool((out[1][4][0, at] == 0).all())      # the decay of a token that resets has no effect


def test_gates_at_their_ends():
    """Decays of 0 (log -inf, -300) and 1, write strengths of 0, tiny, 1 and 2."""
    sdm = need_gpu()
    c = Case(2, 140, 1, 2, 64, 32, seed=4)
    for i, v in enumerate((float("-inf"), -300.0, 0.0, -90.0, -1e-6)):
        c.la[:, i::11] = v
    for i, v in enumerate((0.0, 1e-30, 1.0, 2.0)):
        c.beta[:, i::7] = v
    check(c, c.run(sdm), *c.reference())


def test_strong_decay_then_weak_ones():
    """One decay of e^-150 early in a chunk leaves the later, weak ones their precision."""
    sdm = need_gpu()
    c = Case(1, 64, 1, 1, 32, 32, seed=5, decay=0.01)
    c.la[:, 3] = -150.0
    check(c, c.run(sdm), *c.reference())


def test_equal_keys():
    """The least favourable triangle: every key the same, full write strength, no decay."""
    sdm = need_gpu()
    c = Case(1, 128, 1, 1, 64, 16, seed=6)
    c.k[:] = c.k[:, :1]
    c.beta[:] = 1.0
    c.la[:] = 0.0
    check(c, c.run(sdm), *c.reference())


@pytest.mark.parametrize("scale", [1e-12, 1e12])
def test_scale_of_the_values(scale):
    sdm = need_gpu()
    c = Case(1, 100, 1, 1, 64, 32, seed=7)
    c.v, c.S0 = (c.v.float() * scale).to(torch.bfloat16), c.S0 * scale
    check(c, c.run(sdm), *c.reference())


@pytest.mark.parametrize("offset", [0, 1, 2, 4])
def test_rows_at_every_boundary(offset):
    """Slices of a projection whose rows lie off 16 bytes give the contiguous call's bits."""
    sdm = need_gpu()
    a = Case(1, 90, 2, 2, 64, 32, seed=8)
    b = Case(1, 90, 2, 2, 64, 32, seed=8, fused=True, offset=offset)
    for x, y in zip(itertools.chain(*a.run(sdm)), itertools.chain(*b.run(sdm))):
        assert torch.equal(x, y)


def test_gradients_into_slices_of_one_buffer():
    sdm = need_gpu()
    c = Case(2, 70, 2, 4, 48, 24, seed=10)
    x = [*c.layout(c.q, c.k, c.v), *c.gates()]
    _, saved = sdm.gdn_train(c.S0.cuda(), *x)
    want = sdm.gdn_backward(c.dS.cuda(), *x, saved, c.dy.cuda())
    buf = torch.full((2, 70, 2 * 96 + 96 + 5), 3.0, dtype=torch.bfloat16, device="cuda")
    grads = [buf[..., a:b].unflatten(-1, s) for a, b, s in ((0, 96, (2, 48)), (96, 192, (2, 48)), (192, 288, (4, 24)))]
    got = sdm.gdn_backward(c.dS.cuda(), *x, saved, c.dy.cuda(), grads=grads)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool((buf[..., 288:] == 3.0).all())


def test_no_tokens():
    sdm = need_gpu()
    c = Case(2, 0, 1, 1, 8, 8)
    (y, ST), (d0, *g) = c.run(sdm)
    assert torch.equal(ST.cpu(), c.S0) and torch.equal(d0.cpu(), c.dS) and y.shape == (2, 0, 1, 8)
    assert all(t.numel() == 0 for t in g)


def test_in_place_and_repeated():
    """The state in place; the same bits every time; two halves are the whole."""
    sdm = need_gpu()
    c = Case(2, 256, 2, 2, 128, 64, seed=11)
    x = [*c.layout(c.q, c.k, c.v), *c.gates()]
    one, two = c.run(sdm), c.run(sdm)
    assert all(torch.equal(a, b) for a, b in zip(itertools.chain(*one), itertools.chain(*two)))
    S = c.S0.cuda()
    parts = [[t[:, a:b].contiguous() for t in x] for a, b in ((0, 128), (128, 256))]
    ys, saved = zip(*(sdm.gdn_train(S, *p) for p in parts))
    assert torch.equal(S, one[0][1]) and torch.equal(torch.cat(ys, 1), one[0][0])
    d = c.dS.cuda()
    dy = c.dy.cuda()
    back = [sdm.gdn_backward(d, *parts[i], saved[i], dy[:, 128 * i:128 * i + 128].contiguous()) for i in (1, 0)][::-1]
    assert torch.equal(d, one[1][0])
    for i, whole in enumerate(one[1][1:4]):
        assert torch.equal(torch.cat([b[i] for b in back], 1), whole)


def test_streams_and_graphs():
    """On another stream than the inputs' own, and captured into a graph that is replayed with new inputs."""
    sdm = need_gpu()
    c, e = Case(1, 150, 1, 2, 64, 64, seed=12), Case(1, 150, 1, 2, 64, 64, seed=13)
    want = [x.clone() for x in itertools.chain(*c.run(sdm))]
    new = [x.clone() for x in itertools.chain(*e.run(sdm))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = list(itertools.chain(*c.run(sdm, stream=side)))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = [*c.layout(c.q, c.k, c.v), *c.gates()]
    S, dS, dy = c.S0.cuda(), c.dS.cuda(), c.dy.cuda()
    ST, d0 = torch.empty_like(S), torch.empty_like(S)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y, saved = sdm.gdn_train(S, *x, state_out=ST)
        g = sdm.gdn_backward(dS, *x, saved, dy, dstate_out=d0)
    for case, ref_ in ((c, want), (e, new), (c, want)):
        for t, n in zip((*x, S, dS, dy), (case.q, case.k, case.v, case.la, case.beta, case.S0, case.dS, case.dy)):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, ST, d0, *g), ref_))


def test_many_heads():
    """More tiles of columns than an SM's worth, and than two and four a CTA."""
    sdm = need_gpu()
    for H in (1, 20, 40, 81):
        c = Case(1, 70, 1, H, 32, 128, seed=H)
        check(c, c.run(sdm), *c.reference())


def test_capture_behind_other_streams():
    """Captured where the call follows copies and a join with another stream, and others follow it."""
    sdm = need_gpu()
    c, e = Case(2, 140, 1, 2, 64, 64, seed=14), Case(2, 140, 1, 2, 64, 64, seed=15)
    new = [x.clone() for x in itertools.chain(*e.run(sdm))]
    x = [*c.layout(c.q, c.k, c.v), *c.gates()]
    S, dS, dy = c.S0.cuda(), c.dS.cuda(), c.dy.cuda()
    inputs = (*x, S, dS, dy)
    stage = [t.cuda() for t in (e.q, e.k, e.v, e.la, e.beta, e.S0, e.dS, e.dy)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for t, n in zip(inputs[:4], stage[:4]):
                t.copy_(n)
        for t, n in zip(inputs[4:], stage[4:]):
            t.copy_(n)
        torch.cuda.current_stream().wait_stream(side)
        ST, d0 = torch.empty_like(S), torch.empty_like(S)
        y, saved = sdm.gdn_train(S, *x, state_out=ST)
        g = sdm.gdn_backward(dS, *x, saved, dy, dstate_out=d0)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            copies = [t.clone() for t in (y, ST, d0, *g)]
            for t in inputs:
                t.zero_()           # the next replay's copies bring them back
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(copies, new))


def test_two_streams_at_once():
    """Calls that share their inputs, on two streams that run beside one another."""
    sdm = need_gpu()
    c = Case(2, 700, 2, 4, 128, 128, seed=16)
    x, want = [*c.layout(c.q, c.k, c.v), *c.gates()], None
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    S, dS, dy = c.S0.cuda(), c.dS.cuda(), c.dy.cuda()
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for st in streams:
            ST, d0 = torch.empty_like(S), torch.empty_like(S)
            st.wait_stream(torch.cuda.current_stream())
            y, saved = sdm.gdn_train(S, *x, state_out=ST, stream=st)
            outs.append((y, ST, d0, *sdm.gdn_backward(dS, *x, saved, dy, dstate_out=d0, stream=st)))
    torch.cuda.synchronize()
    want = list(itertools.chain(*c.run(sdm)))
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))


@pytest.mark.parametrize("dims", [(3, 130, 3, 3, 48, 48), (3, 130, 3, 3, 128, 72)], ids=str)
def test_nan_stays_in_its_sequence_and_head(dims):
    """What one sequence or one head holds does not reach the others, whose tokens share its tiles' copies."""
    sdm = need_gpu()
    c = Case(*dims, seed=17)
    want = c.run(sdm)
    for t in (c.q, c.k, c.v, c.la, c.beta, c.dy):
        t[1] = float("nan")
        t[2, :, 1] = float("nan")
    got = c.run(sdm)
    for a, b in zip(itertools.chain(*got), itertools.chain(*want)):
        heads = 1 if a.shape[1] == dims[3] and a.dim() == 4 and a.dtype == torch.float32 else 2
        assert torch.equal(a[0], b[0])
        rows = (a[2], b[2]) if heads == 1 else (a[2].transpose(0, 1), b[2].transpose(0, 1))
        assert all(torch.equal(rows[0][h], rows[1][h]) for h in (0, 2))


def test_no_value_heads():
    """No value head reads the key heads: their gradients are 0."""
    sdm = need_gpu()
    bf = dict(dtype=torch.bfloat16, device="cuda")
    q, v, gate = torch.randn(2, 70, 2, 24, **bf), torch.zeros(2, 70, 0, 16, **bf), torch.zeros(2, 70, 0, device="cuda")
    state = torch.zeros(2, 0, 24, 16, device="cuda")
    y, saved = sdm.gdn_train(state, q, q, v, gate, gate)
    grads = [torch.full_like(q, 3.0), torch.full_like(q, 3.0), torch.zeros_like(v)]
    lens = torch.tensor([70, 5], dtype=torch.int32, device="cuda")
    sdm.gdn_backward(state, q, q, v, gate, gate, saved, y, grads=grads, lens=lens)
    for g in grads[:2]:
        assert bool((g[0] == 0).all()) and bool((g[1, :5] == 0).all()) and bool((g[1, 5:] == 3.0).all())


def test_offsets_past_32_bits():
    """Tokens 2^20 elements apart, 2^32 elements in all; a pool of more than 2^31 elements."""
    sdm = need_gpu()
    c = Case(1, 4097, 1, 1, 64, 64, seed=18)
    want = list(itertools.chain(*c.run(sdm)))
    p = torch.empty(4097, 1 << 20, dtype=torch.bfloat16, device="cuda")
    x = []
    for i, t in enumerate((c.q, c.k, c.v)):
        s = p[:, 64 * i:64 * i + 64].view(1, 4097, 1, 64)
        s.copy_(t)
        x.append(s)
    grads = [p[:, 64 * i:64 * i + 64].view(1, 4097, 1, 64) for i in (3, 4, 5)]
    S, d = c.S0.cuda(), c.dS.cuda()
    y, saved = sdm.gdn_train(S, *x, *c.gates())
    got = (y, S, d, *sdm.gdn_backward(d, *x, *c.gates(), saved, c.dy.cuda(), grads=grads))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del p, x, grads
    c = Case(2, 1, 1, 1, 128, 128, seed=19)
    pool = torch.empty((1 << 17) + 2, 1, 128, 128, device="cuda")
    slots = torch.tensor([(1 << 17) + 1, 0], dtype=torch.int32, device="cuda")
    pool[slots.long()] = c.S0.cuda()
    y = sdm.gdn_step(pool, *c.layout(c.q, c.k, c.v), *c.gates(), slots=slots)
    f = ref.forward(c.S0, c.q, c.k, c.v, c.la, c.beta)
    close16(y, f[0], "y")
    close32(pool[slots.long()], f[1], "state")


@pytest.mark.parametrize("B", [1, 2, 4])
def test_odd_rows_of_many_heads(B):
    """Rows that no tensor copy takes, one, two and four tiles of columns a CTA, tiles behind the last column."""
    sdm = need_gpu()
    c = Case(B, 200, 15, 15, 36, 129, seed=50 + B, reset=0.02, lens=[200, 150, 1, 128][:B], fused=True, offset=1)
    check(c, c.run(sdm), *c.reference())
    aligned = Case(B, 200, 15, 15, 40, 136, seed=60 + B, reset=0.02, lens=[193, 192, 0, 65][:B])
    check(aligned, aligned.run(sdm), *aligned.reference())


@pytest.mark.parametrize("shape", [(1, 200, 1, 1, 128, 128), (3, 130, 1, 20, 64, 64), (4, 130, 1, 20, 64, 64)], ids=str)
def test_a_wait_that_runs_out_is_reported(shape, monkeypatch):
    """A copy that is never asked for: both calls end, report it, and the next ones are right."""
    sdm = need_gpu()
    c = Case(*shape, seed=40)
    x = [*c.layout(c.q, c.k, c.v), *c.gates()]
    _, saved = sdm.gdn_train(c.S0.cuda(), *x)
    monkeypatch.setenv("SDM_TEST_DROP_SIGNAL", "1")
    for call in (lambda e: sdm.gdn_train(c.S0.cuda(), *x, dev_err=e), lambda e: sdm.gdn_backward(c.dS.cuda(), *x, saved, c.dy.cuda(), dev_err=e)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(err)
        assert int(err) == sdm.SDM_DEVERR_TIMEOUT
        with pytest.raises(sdm.SdmError):
            sdm.sdm_check()
    monkeypatch.delenv("SDM_TEST_DROP_SIGNAL")
    check(c, c.run(sdm), *c.reference())
    sdm.sdm_check()


# ---- decoding ----

@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1, 1), (3, 1, 2, 4, 128, 128), (2, 5, 2, 2, 100, 72), (4, 2, 1, 3, 64, 33),
                                   (2, 3, 1, 1, 65, 130)], ids=str)
@pytest.mark.parametrize("fused", [False, True])
def test_step(shape, fused):
    sdm = need_gpu()
    c = Case(*shape, seed=sum(shape) + 1, fused=fused)
    B, H, dk, dv = shape[0], *shape[3:]
    f = ref.forward(c.S0, c.q, c.k, c.v, c.la, c.beta)
    pool = torch.randn(B + 3, H, dk, dv).cuda()
    slots = torch.randperm(B + 3)[:B].to(torch.int32).cuda()
    pool[slots.long()] = c.S0.cuda()
    before = pool.clone()
    y = sdm.gdn_step(pool, *c.layout(c.q, c.k, c.v), *c.gates(), slots=slots)
    close16(y, f[0], "y")
    close32(pool[slots.long()], f[1], "state")
    rest = torch.ones(B + 3, dtype=torch.bool)
    rest[slots.long().cpu()] = False
    assert torch.equal(pool[rest.cuda()], before[rest.cuda()])
    own = c.S0.cuda()       # without slots
    assert torch.equal(sdm.gdn_step(own, *c.layout(c.q, c.k, c.v), *c.gates()), y) and torch.equal(own, pool[slots.long()])


def test_step_slots():
    """Sequences that do not exist, slots outside the pool and repeated ones: nothing of them is touched."""
    sdm = need_gpu()
    c = Case(6, 2, 1, 1, 32, 32, seed=20)
    pool = torch.randn(4, 1, 32, 32).cuda()
    start = pool.clone()
    slots = torch.tensor([2, -1, 4, 0, 2, -7], dtype=torch.int32, device="cuda")
    lens = torch.tensor([2, 2, 2, 1, 2, 2], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = [*c.layout(c.q, c.k, c.v), *c.gates()]
    y = torch.full((6, 2, 1, 32), 5.0, dtype=torch.bfloat16, device="cuda")
    sdm.gdn_step(pool, *x, slots=slots, lens=lens, y=y, dev_err=err)
    assert int(err) == sdm.SDM_DEVERR_INDEX_RANGE | sdm.SDM_DEVERR_INDEX_REPEAT
    assert bool((y[[1, 2, 4, 5]] == 5.0).all()) and bool((y[3, 1] == 5.0).all())
    assert torch.equal(pool[[1, 3]], start[[1, 3]])
    f = ref.forward(start[[2, 0]].cpu(), *(t[[0, 3]] for t in (c.q, c.k, c.v, c.la, c.beta)), lens=torch.tensor([2, 1]))
    close32(pool[[2, 0]], f[1], "state")
    close16(y[0], f[0][0], "y")
    assert bool((sdm.gdn_step(pool, *x, slots=slots)[1] == 0).all())        # a new y is 0 there


def test_steps_continue_a_training_forward():
    sdm = need_gpu()
    c = Case(2, 100, 1, 2, 64, 64, seed=21)
    x = [*c.layout(c.q, c.k, c.v), *c.gates()]
    S = c.S0.cuda()
    first = [t[:, :97].contiguous() for t in x]
    y0, _ = sdm.gdn_train(S, *first)
    ys = [sdm.gdn_step(S, *(t[:, i:i + 1].contiguous() for t in x)) for i in range(97, 100)]
    f = ref.forward(c.S0, c.q, c.k, c.v, c.la, c.beta)
    close16(torch.cat([y0, *ys], 1), f[0], "y")
    close32(S, f[1], "state")


def test_step_in_a_graph():
    sdm = need_gpu()
    c = Case(3, 1, 1, 2, 128, 128, seed=22)
    x = [*c.layout(c.q, c.k, c.v), *c.gates()]
    slots = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    pool, y = torch.zeros(5, 2, 128, 128, device="cuda"), torch.zeros(3, 1, 2, 128, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        sdm.gdn_step(pool, *x, slots=slots, y=y)
    pool.copy_(torch.randn(5, 2, 128, 128))
    S = pool.clone()
    for order in ([0, 1, 2], [4, -1, 0]):
        slots.copy_(torch.tensor(order, dtype=torch.int32))
        graph.replay()
        sdm.gdn_step(S, *x, slots=slots)
        assert torch.equal(pool, S)
