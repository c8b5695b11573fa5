"""Visits sorted by partition and back, against plain loops; and a routed
layer of the gated delta rule made of them.

Tolerances: indices and copies are exact.  A sum of k <= 32 products in fp32 is
at most (k + 1) 2^-24 of the sum of their magnitudes off, a dot product of D terms,
in a tree of at most D / 32 + 5 additions a lane, (D / 32 + 6) 2^-24; bf16 outputs
another 2^-8 of the value."""
import pytest
import torch

import gdn_reference as ref
from helpers import need_gpu

pytestmark = pytest.mark.gpu


def visits(M, k, N, seed, drop=0.0):
    g = torch.Generator().manual_seed(seed)
    sel = torch.randint(0, max(N, 1), (M, k), generator=g, dtype=torch.int32)
    if drop:
        sel[torch.rand((M, k), generator=g) < drop] = -1
    return sel


@pytest.mark.parametrize("M,k,N,drop", [(0, 2, 4, 0.0), (1, 1, 1, 0.0), (1, 32, 3, 0.3), (5, 3, 1024, 0.1), (1000, 2, 7, 0.1),
                                        (1024, 2, 8, 0.0), (1025, 2, 8, 0.0), (3000, 5, 64, 0.05), (7, 4, 5, 1.0),
                                        (9000, 4, 1024, 0.02), (40000, 1, 300, 0.0), (3, 0, 4, 0.0)])
def test_sort(M, k, N, drop):
    sdm = need_gpu()
    sel = visits(M, k, N, M + k + N, drop)
    got = [x.cpu() for x in sdm.route_sort(sel.cuda(), N)]
    flat = sel.flatten().long()
    key = torch.where(flat < 0, N, flat)
    order = torch.argsort(key, stable=True)
    kept = int((flat >= 0).sum())
    place = torch.empty_like(order)
    place[order] = torch.arange(M * k)
    place[flat < 0] = -1
    order[kept:] = -1
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), torch.bincount(flat[flat >= 0], minlength=N).cumsum(0)])
    for x, want in zip(got, (order, place.reshape(M, k), offsets)):
        assert torch.equal(x.long(), want)
    if M * k <= 200:
        for x, want in zip(got, ref.sort_visits(sel, N)):
            assert x.flatten().tolist() == want


def test_sort_out_of_range_and_repeats():
    sdm = need_gpu()
    sel = torch.tensor([[0, 0], [3, 1], [2 ** 31 - 1, -2 ** 31], [1, 1]], dtype=torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    order, place, offsets = sdm.route_sort(sel.cuda(), 3, dev_err=err)
    assert int(err) == sdm.SDM_DEVERR_INDEX_RANGE
    assert order.tolist() == [0, 1, 3, 6, 7, -1, -1, -1] and offsets.tolist() == [0, 2, 5, 5]
    assert place.tolist() == [[0, 1], [-1, 2], [-1, -1], [3, 4]]
    order, place, offsets = sdm.route_sort(sel.cuda(), 0)
    assert offsets.tolist() == [0] and bool((place == -1).all()) and bool((order == -1).all())


def bound(dtype, value, magnitude, ops):
    return (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) * value.abs() + ops * 2.0 ** -24 * magnitude + 1e-30


@pytest.mark.parametrize("M,k,N,D", [(1, 1, 1, 1), (64, 2, 8, 1920), (37, 3, 5, 963), (50, 4, 9, 130), (20, 32, 6, 40), (33, 5, 4, 4100),
                                     (700, 2, 3, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("drop,strided", [(0.0, False), (0.3, True)])
def test_rows(M, k, N, D, dtype, drop, strided):
    sdm = need_gpu()
    g = torch.Generator().manual_seed(M + D)
    n = lambda *s: torch.randn(s, generator=g).to(dtype)  # noqa: E731
    sel = visits(M, k, N, D, drop)
    order, place, offsets = sdm.route_sort(sel.cuda(), N)
    x, out, dy, w = n(M, D), n(M * k, D), n(M, D), torch.rand((M, k), generator=g)
    wide = lambda t: torch.cat([t, torch.full((M, 3), float("nan"), dtype=dtype)], 1).cuda()[:, :D] if strided else t.cuda()  # noqa: E731
    rows = sdm.route_gather(wide(x), place, offsets).cpu()
    pl, kept = place.cpu().long(), int(offsets[-1])
    want = torch.zeros(M * k, D, dtype=dtype)
    want[pl[pl >= 0]] = x[:, None].expand(M, k, D)[pl >= 0]
    assert torch.equal(rows, want) and bool((rows[kept:] == 0).all())
    o = torch.where((pl >= 0)[..., None], out[pl.clamp(min=0)], 0).double()
    for weights in (w, None):
        y = sdm.route_combine(out.cuda(), place, None if weights is None else weights.cuda()).cpu().double()
        ww = torch.ones_like(w) if weights is None else weights
        terms = ww.double()[..., None] * o
        assert bool(((y - terms.sum(1)).abs() <= bound(dtype, terms.sum(1), terms.abs().sum(1), k + 1)).all())
    drows, dw = (t.cpu() for t in sdm.route_combine_backward(wide(dy), out.cuda(), place, w.cuda(), offsets))
    want = torch.zeros(M * k, D, dtype=torch.float64)
    want[pl[pl >= 0]] = (w.double()[..., None] * dy.double()[:, None])[pl >= 0]
    assert bool(((drows.double() - want).abs() <= bound(dtype, want, want.abs(), 1)).all()) and bool((drows[kept:] == 0).all())
    terms = o * dy.double()[:, None]
    assert bool(((dw.double() - terms.sum(-1)).abs() <= (D / 32 + 6) * 2.0 ** -24 * terms.abs().sum(-1) + 1e-30).all())
    assert bool((dw[pl < 0] == 0).all())


def test_gather_is_the_transpose_of_combine():
    sdm = need_gpu()
    sel = visits(200, 3, 6, 1, 0.1)
    _, place, offsets = sdm.route_sort(sel.cuda(), 6)
    # small whole numbers: every sum exact
    x, r = torch.randint(-8, 9, (200, 64)).float().cuda(), torch.randint(-8, 9, (600, 64)).float().cuda()
    r[int(offsets[-1]):] = 0
    assert float((sdm.route_gather(x, place, offsets) * r).sum()) == float((x * sdm.route_combine(r, place)).sum())


def test_places_outside_the_rows_are_dropped():
    sdm = need_gpu()
    place = torch.tensor([[0, 9], [-5, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    x = torch.ones(2, 16, device="cuda")
    rows = sdm.route_gather(x, place, offsets)
    assert bool((rows[0] == 1).all()) and bool((rows[1:] == 0).all())
    assert bool((sdm.route_combine(rows, place)[1] == 0).all())


def test_offsets_past_32_bits():
    """Rows of more than 2^32 elements in all, and tokens 2^26 elements apart."""
    sdm = need_gpu()
    M, k, D = 33000, 2, 1 << 16
    sel = torch.zeros(M, k, dtype=torch.int32, device="cuda")
    sel[:, 1] = 1
    _, place, offsets = sdm.route_sort(sel, 2)
    x = torch.empty(M, D, dtype=torch.bfloat16, device="cuda")
    x[:] = (torch.arange(M, device="cuda") % 16)[:, None]
    rows = sdm.route_gather(x, place, offsets)
    assert bool((rows[:M, ::4095] == x[:, ::4095]).all()) and bool((rows[M:, ::4095] == x[:, ::4095]).all())
    y = sdm.route_combine(rows, place)
    assert bool((y[:, ::4095] == 2 * x[:, ::4095]).all())
    del y
    w = torch.full((M, k), 0.5, device="cuda")
    drows, dw = sdm.route_combine_backward(x, rows, place, w, offsets)
    assert bool((drows[:, ::4095] == 0.5 * rows[:, ::4095]).all())
    assert torch.equal(dw, (x[:, :1].float() ** 2 * D).expand(M, k))       # whole numbers below 2^24
    del drows, rows
    far = torch.empty(70, 1 << 26, dtype=torch.bfloat16, device="cuda")[:, :40]
    far.copy_(x[:70, :40])
    p = torch.arange(70, dtype=torch.int32, device="cuda")[:, None].contiguous()
    assert torch.equal(sdm.route_gather(far, p, torch.tensor([0, 70], dtype=torch.int32, device="cuda")), x[:70, :40])


def test_graph_and_stream():
    sdm = need_gpu()
    sel = [visits(300, 2, 5, s).cuda() for s in (1, 2)]
    x, w = torch.randn(300, 96, device="cuda"), torch.rand(300, 2, device="cuda")

    def layer(s, **kw):
        _, p, o = sdm.route_sort(s, 5, **kw)
        return sdm.route_combine(sdm.route_gather(x, p, o, **kw), p, w, **kw)

    want = [layer(s) for s in sel]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = layer(sel[0], stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])
    buf, graph = sel[0].clone(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = layer(buf)
    for s, v in zip(sel[::-1], want[::-1]):
        buf.copy_(s)
        graph.replay()
        assert torch.equal(y, v)


def test_routed_layer():
    """The operators together: each token's row q | k | v goes to its partitions, the gated delta rule
    runs over every partition's tokens in order (a reset where a partition begins), the outputs come back weighted;
    and the gradient of it all, against 64 bits run partition by partition."""
    sdm = need_gpu()
    M, k, N, Hk, H, dk, dv = 90, 2, 4, 1, 2, 32, 16
    W = 2 * Hk * dk + H * dv
    g = torch.Generator().manual_seed(30)
    x = torch.randn((M, W), generator=g)
    x[:, :2 * dk] /= 5.0
    x = x.to(torch.bfloat16)
    sel = torch.stack([torch.randperm(N, generator=g)[:k] for _ in range(M)]).to(torch.int32)
    sel[5, 1] = -1
    w = torch.rand((M, k), generator=g)
    gate = torch.stack([-torch.rand((M, H), generator=g), torch.rand((M, H), generator=g)], 1)      # log_alpha | beta
    dy = torch.randn((M, H * dv), generator=g).to(torch.bfloat16)

    order, place, offsets = sdm.route_sort(sel.cuda(), N)
    kept = offsets[-1:]                         # stays on the device: the rows behind it are a sequence's padding
    rows = sdm.route_gather(x.cuda(), place, offsets)[None]
    gates = sdm.route_gather(gate.reshape(M, 2 * H).cuda(), place, offsets).view(1, M * k, 2, H)
    la, beta = gates[:, :, 0].contiguous(), gates[:, :, 1].contiguous()
    reset = torch.zeros((1, M * k + 1), dtype=torch.uint8, device="cuda")
    reset[0, offsets.long()] = 1
    reset = reset[:, :-1].contiguous()
    split = lambda t: (t[..., :Hk * dk].unflatten(-1, (Hk, dk)), t[..., Hk * dk:2 * Hk * dk].unflatten(-1, (Hk, dk)),  # noqa: E731
                       t[..., 2 * Hk * dk:].unflatten(-1, (H, dv)))
    S = torch.zeros(1, H, dk, dv, device="cuda")
    out, saved = sdm.gdn_train(S.clone(), *split(rows), la, beta, reset=reset, lens=kept)
    y = sdm.route_combine(out.view(M * k, H * dv), place, w.cuda())
    dout, dw = sdm.route_combine_backward(dy.cuda(), out.view(M * k, H * dv), place, w.cuda(), offsets)
    buf = torch.zeros_like(rows)
    *_, dla, dbeta = sdm.gdn_backward(S.clone(), *split(rows), la, beta, saved, dout.view(1, M * k, H, dv), reset=reset, lens=kept,
                                      grads=split(buf))
    dx = sdm.route_combine(buf[0], place)

    places, n = ref.sort_visits(sel, N)[1], sum(int(s) >= 0 for s in sel.flatten())
    tokens = [i // k for i in ref.sort_visits(sel, N)[0][:n]]
    r = x[tokens][None]
    la_, beta_ = gate[tokens, 0][None], gate[tokens, 1][None]
    rs = torch.zeros((1, n), dtype=torch.uint8)
    rs[0, [o for o in ref.sort_visits(sel, N)[2] if o < n]] = 1
    S0 = torch.zeros(1, H, dk, dv)
    f = ref.forward(S0, *split(r), la_, beta_, rs)
    o = out[0, :n].cpu().double().flatten(1)                # what combine was given
    y_ = torch.zeros(M, H * dv, dtype=torch.float64)
    do = torch.zeros(n, H * dv, dtype=torch.float64)
    for m in range(M):
        for j in range(k):
            p = places[m * k + j]
            if p >= 0:
                y_[m] += w[m, j].double() * o[p]
                do[p] = w[m, j].double() * dy[m].double()
    # out: a bf16 rounding and 16 bits inside; y: one more rounding of sums of two
    assert bool(((o - f[0][0].flatten(1)).abs() <= 2.0 ** -8 * f[0][0].flatten(1).abs() + 2.0 ** -11 * f[0].square().mean().sqrt()).all())
    assert bool(((y.cpu().double() - y_).abs() <= 2.0 ** -8 * y_.abs() + 1e-6).all())
    b = ref.backward(f, S0, *split(r), la_, beta_, dout[:n].cpu().view(1, n, H, dv), rs)
    dr = torch.cat([t.flatten(2) for t in b[1:4]], -1)[0]
    dx_ = torch.zeros(M, W, dtype=torch.float64)
    dx_.index_add_(0, torch.tensor(tokens), dr)
    # rows rounded once, then sums of two rounded again
    assert bool(((dx.cpu().double() - dx_).abs() <= 2.0 ** -7 * dx_.abs() + 2.0 ** -6 * dr.abs().amax(0) + 2.0 ** -11).all())
    assert float((dla[0, :n].cpu().double() - b[4][0]).norm()) <= 2.0 ** -14 * float(b[4].norm())
    assert float((dbeta[0, :n].cpu().double() - b[5][0]).norm()) <= 2.0 ** -17 * float(b[5].norm())
    assert float((dout[:n].cpu().double() - do).norm()) <= 2.0 ** -8 * float(do.norm())
