"""A routed layer of the gated delta rule, forward and gradient, element by element.

Tolerance of dx.  A token's gradient is the sum of its visits' rows: each row
rounded once to bf16 (half a step, at most 2^-8 of it), the sum formed in fp32 and
rounded once (2^-8 of it, and of the rows' own errors), and inside each row 32-bit
sums: 2^-15 of a row's root mean square, as for the rows alone."""
import pytest
import torch

import gdn_reference as ref
from helpers import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k,decay,seed", [(1, 0.5, 1), (2, 0.5, 2), (3, 2.0, 3), (2, 8.0, 4)])
def test_gradient_of_the_inputs(k, decay, seed):
    sdm = need_gpu()
    M, N, Hk, H, dk, dv = 170, 4, 2, 4, 32, 24
    W = 2 * Hk * dk + H * dv
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, W), generator=g)
    x[:, :2 * Hk * dk] /= dk ** 0.5
    x = x.to(torch.bfloat16)
    sel = torch.stack([torch.randperm(N, generator=g)[:k] for _ in range(M)]).to(torch.int32)
    sel[torch.rand((M, k), generator=g) < 0.1] = -1
    w = torch.rand((M, k), generator=g)
    la, beta = -decay * torch.rand((M, H), generator=g), torch.rand((M, H), generator=g)
    dy = torch.randn((M, H * dv), generator=g).to(torch.bfloat16)
    split = lambda t: (t[..., :Hk * dk].unflatten(-1, (Hk, dk)), t[..., Hk * dk:2 * Hk * dk].unflatten(-1, (Hk, dk)),  # noqa: E731
                       t[..., 2 * Hk * dk:].unflatten(-1, (H, dv)))

    order, place, offsets = sdm.route_sort(sel.cuda(), N)
    kept = offsets[-1:]
    rows = sdm.route_gather(x.cuda(), place, offsets)[None]
    gates = [sdm.route_gather(t.cuda(), place, offsets)[None] for t in (la, beta)]
    reset = torch.zeros((1, M * k + 1), dtype=torch.uint8, device="cuda")
    reset[0, offsets.long()] = 1
    reset = reset[:, :-1].contiguous()
    S = torch.full((1, H, dk, dv), float("nan"), device="cuda")     # the first row resets: never read
    out, saved = sdm.gdn_train(S, *split(rows), *gates, reset=reset, lens=kept, state_out=torch.empty_like(S))
    dout, _ = sdm.route_combine_backward(dy.cuda(), out.view(M * k, H * dv), place, w.cuda(), offsets)
    buf = torch.zeros_like(rows)
    dS = torch.zeros_like(S)
    *_, dla, dbeta = sdm.gdn_backward(dS, *split(rows), *gates, saved, dout.view(1, M * k, H, dv), reset=reset, lens=kept,
                                      grads=split(buf))
    dx = sdm.route_combine(buf[0], place).cpu().double()
    dgates = [sdm.route_combine(t[0], place).cpu().double() for t in (dla, dbeta)]

    n = int(kept)
    tokens = (order[:n].cpu().long() // k)
    rs = reset[:, :n].cpu()
    r = x[tokens][None]
    la_, beta_, S0 = la[tokens][None], beta[tokens][None], torch.zeros(1, H, dk, dv)
    f = ref.forward(S0, *split(r), la_, beta_, rs)
    b = ref.backward(f, S0, *split(r), la_, beta_, dout[:n].cpu().view(1, n, H, dv), rs)
    dr = torch.cat([t.flatten(2) for t in b[1:4]], -1)[0]
    want = torch.zeros(M, W, dtype=torch.float64).index_add_(0, tokens, dr)
    size = torch.zeros(M, W, dtype=torch.float64).index_add_(0, tokens, dr.abs())
    rms = torch.cat([t.flatten(2)[0].square().mean().sqrt().expand(t.shape[2] * t.shape[3]) for t in b[1:4]])
    bound = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -16) * size + k * 2.0 ** -15 * rms
    assert bool(((dx - want).abs() <= bound).all()), float(((dx - want).abs() / bound).max())
    assert bool((dx[(sel < 0).all(1)] == 0).all())
    for got, part, tol in ((dgates[0], b[4], 2.0 ** -17), (dgates[1], b[5], 2.0 ** -18)):
        exact = torch.zeros(M, H, dtype=torch.float64).index_add_(0, tokens, part[0])
        # sums of k rows, terms of either sign: the rows' bound and k roundings
        assert float((got - exact).norm()) <= (tol + k * 2.0 ** -24) * float(part.norm())
