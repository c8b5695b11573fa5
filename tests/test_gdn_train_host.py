"""The gated delta rule's training and decoding calls and the sorted visits
without a GPU: the formulas' gradients against differences, and the calls'
refusals before anything reaches the device."""
import pytest
import torch

import gdn_reference as ref

A = 1 << 20     # a fake, aligned "device" address


@pytest.fixture(scope="module")
def sdm():
    from delta_rule_memory_gb300 import build as b
    b.build()
    import delta_rule_memory_gb300 as m
    return m


@pytest.mark.parametrize("with_reset,with_lens", [(False, False), (True, False), (False, True), (True, True)])
def test_formulas_gradients_match_differences(with_reset, with_lens):
    g = torch.Generator().manual_seed(5)
    B, T, Hk, H, dk, dv = 2, 7, 2, 4, 3, 5
    n = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    args = [n(B, H, dk, dv), n(B, T, Hk, dk), n(B, T, Hk, dk), n(B, T, H, dv), -n(B, T, H).abs(), torch.sigmoid(n(B, T, H))]
    dy, dS = n(B, T, H, dv), n(B, H, dk, dv)
    reset = (torch.rand((B, T), generator=g) < 0.3).to(torch.uint8) if with_reset else None
    lens = torch.tensor([4, 7]) if with_lens else None

    def loss(*a):
        y, S = ref.forward(*a, reset, lens)[:2]
        return float((y * dy).sum() + (S * dS).sum())

    grads = ref.backward(ref.forward(*args, reset, lens), dS, *args[1:], dy, reset, lens)
    for i, got in enumerate(grads):
        for _ in range(4):
            d, h = n(*args[i].shape), 1e-5
            up, down = (loss(*(a + s * h * d if j == i else a for j, a in enumerate(args))) for s in (1, -1))
            # central difference: error O(h^2) = 1e-10 times third derivatives, cancellation 1e-16 / 1e-5
            assert abs(float((got * d).sum()) - (up - down) / (2 * h)) <= 1e-6 * abs(up - down) / (2 * h) + 1e-7


def _train(L, **kw):
    a = dict(s=A, so=A, q=A, lq=32, k=A, lk=32, v=A, lv=64, la=A, be=A, rs=None, ln=None, B=2, T=65, Hk=2, H=4, dk=16, dv=16,
             y=A, sv=A, sb=1 << 40, err=None)
    a.update(kw)
    return L.gdn_train(*(a[n] for n in ("s", "so", "q", "lq", "k", "lk", "v", "lv", "la", "be", "rs", "ln", "B", "T", "Hk", "H",
                                        "dk", "dv", "y", "sv", "sb", "err")), None)


def _backward(L, **kw):
    a = dict(s=A, so=A, q=A, lq=32, k=A, lk=32, v=A, lv=64, la=A, be=A, rs=None, ln=None, sv=A, sb=1 << 40, dy=A, B=2, T=65, Hk=2,
             H=4, dk=16, dv=16, dq=A, ldq=32, dko=A, ldk=32, dvo=A, ldv=64, dla=A, dbe=A, ws=A, wb=1 << 40, err=None)
    a.update(kw)
    return L.gdn_backward(*(a[n] for n in ("s", "so", "q", "lq", "k", "lk", "v", "lv", "la", "be", "rs", "ln", "sv", "sb", "dy", "B",
                                           "T", "Hk", "H", "dk", "dv", "dq", "ldq", "dko", "ldk", "dvo", "ldv", "dla", "dbe", "ws",
                                           "wb", "err")), None)


def _step(L, **kw):
    a = dict(s=A, q=A, lq=32, k=A, lk=32, v=A, lv=64, la=A, be=A, sl=A, ln=None, P=4, B=2, T=1, Hk=2, H=4, dk=16, dv=16, y=A, err=None)
    a.update(kw)
    return L.gdn_step(*(a[n] for n in ("s", "q", "lq", "k", "lk", "v", "lv", "la", "be", "sl", "ln", "P", "B", "T", "Hk", "H", "dk",
                                       "dv", "y", "err")), None)


SIZES = [(dict(B=-1), 1), (dict(T=-1), 1), (dict(H=-4), 1), (dict(Hk=-1), 1), (dict(B=65536), 2), (dict(T=1 << 30), 2),
         (dict(dk=0), 2), (dict(dk=129, lq=1000, lk=1000), 2), (dict(dv=0), 2), (dict(dv=1025, lv=9000), 2), (dict(Hk=3), 2),
         (dict(Hk=0), 2), (dict(lq=31), 2), (dict(lk=0), 2), (dict(lv=63), 2), (dict(lq=1 << 27), 2), (dict(q=None), 1),
         (dict(k=None), 1), (dict(v=None), 1), (dict(la=None), 1), (dict(be=None), 1), (dict(q=A + 1), 3), (dict(k=A + 1), 3),
         (dict(v=A + 1), 3), (dict(la=A + 2), 3), (dict(be=A + 1), 3), (dict(ln=A + 2), 3), (dict(err=A + 1), 3), (dict(s=A + 2), 3)]


@pytest.mark.parametrize("fn,more", [
    (_train, [(dict(so=None), 1), (dict(y=None), 1), (dict(sv=None), 1), (dict(sb=1000), 1), (dict(y=A + 1), 3), (dict(sv=A + 8), 3),
              (dict(so=A + 1), 3)]),
    (_backward, [(dict(so=None), 1), (dict(dy=None), 1), (dict(dq=None), 1), (dict(dko=None), 1), (dict(dvo=None), 1),
                 (dict(dla=None), 1), (dict(dbe=None), 1), (dict(ws=None), 1), (dict(wb=100), 1), (dict(sb=100), 1), (dict(sv=None), 1),
                 (dict(ldq=31), 2), (dict(ldk=1), 2), (dict(ldv=63), 2), (dict(ldv=1 << 27), 2), (dict(dq=A + 1), 3),
                 (dict(dla=A + 2), 3), (dict(ws=A + 4), 3)]),
    (_step, [(dict(y=None), 1), (dict(s=None), 1), (dict(P=-1), 1), (dict(sl=None, P=1), 2), (dict(sl=A + 2), 3), (dict(y=A + 1), 3)]),
])
def test_refusals(sdm, fn, more):
    L = sdm.lib()
    name = {_train: b"gdn_train", _backward: b"gdn_backward", _step: b"gdn_step"}[fn]
    for kw, code in SIZES + more:
        assert fn(L, **kw) == code, kw
        assert name in L.sdm_last_error()
    assert fn(L, B=0) == 0 and fn(L, H=0, Hk=0) == 0        # nothing to do: nothing launched


def test_sizes(sdm):
    # per chunk of 64 tokens: 384 floats, two triangles of 3 x 5120 bytes, the state and the residuals
    units = 2 * 4 * 2
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    want = up(units * 1536) + 2 * up(units * 15360) + up(units * 1 * 16 * 64 * 4) + up(units * 16 * 64 * 4)
    assert sdm.gdn_train_saved_size(2, 65, 2, 4, 16, 16) == want
    assert sdm.gdn_train_saved_size(2, 0, 2, 4, 16, 16) == 0
    assert sdm.gdn_train_saved_size(2, 65, 3, 4, 16, 16) == 0           # invalid
    assert sdm.gdn_backward_workspace_size(1, 64, 1, 1, 128, 128) == 2 * 128 * 128 * 4 + 128 * 64 * 4


def test_route_refusals(sdm):
    L = sdm.lib()

    def sort(**kw):
        a = dict(sel=A, M=10, k=2, N=4, o=A, p=A, f=A, ws=None, wb=0, err=None)
        a.update(kw)
        return L.route_sort(*(a[n] for n in ("sel", "M", "k", "N", "o", "p", "f", "ws", "wb", "err")), None)

    for kw, code in [(dict(M=-1), 1), (dict(k=-1), 1), (dict(N=-1), 1), (dict(k=33), 2), (dict(N=1025), 2), (dict(M=1 << 31), 2),
                     (dict(M=1 << 30), 2), (dict(sel=None), 1), (dict(o=None), 1), (dict(p=None), 1), (dict(f=None), 1),
                     (dict(M=5000), 1), (dict(sel=A + 2), 3), (dict(f=A + 1), 3), (dict(err=A + 3), 3)]:
        assert sort(**kw) == code, kw
        assert b"route_sort" in L.sdm_last_error()

    def gather(**kw):
        a = dict(x=A, ld=8, dt=1, p=A, f=A, M=10, k=2, N=4, D=8, o=A)
        a.update(kw)
        return L.route_gather(*(a[n] for n in ("x", "ld", "dt", "p", "f", "M", "k", "N", "D", "o")), None)

    for kw, code in [(dict(dt=2), 4), (dict(ld=7), 2), (dict(ld=1 << 27), 2), (dict(D=1 << 24, ld=1 << 24), 2), (dict(x=None), 1),
                     (dict(p=None), 1), (dict(f=None), 1), (dict(o=None), 1), (dict(x=A + 1), 3), (dict(o=A + 1), 3), (dict(M=-2), 1)]:
        assert gather(**kw) == code, kw
    assert gather(M=0) == 0 and gather(k=0) == 0 and gather(D=0, ld=0) == 0

    def combine(**kw):
        a = dict(r=A, dt=0, p=A, w=A, M=10, k=2, D=8, y=A)
        a.update(kw)
        return L.route_combine(*(a[n] for n in ("r", "dt", "p", "w", "M", "k", "D", "y")), None)

    for kw, code in [(dict(dt=-1), 4), (dict(k=40), 2), (dict(r=None), 1), (dict(p=None), 1), (dict(y=None), 1), (dict(r=A + 2), 3),
                     (dict(w=A + 2), 3), (dict(D=-1), 1)]:
        assert combine(**kw) == code, kw

    def back(**kw):
        a = dict(dy=A, ld=8, dt=0, r=A, p=A, w=A, f=A, M=10, k=2, N=4, D=8, dr=A, dw=A)
        a.update(kw)
        return L.route_combine_backward(*(a[n] for n in ("dy", "ld", "dt", "r", "p", "w", "f", "M", "k", "N", "D", "dr", "dw")), None)

    for kw, code in [(dict(dt=3), 4), (dict(ld=4), 2), (dict(w=None), 1), (dict(dw=None), 1), (dict(dr=None), 1), (dict(dy=None), 1),
                     (dict(f=None), 1), (dict(dw=A + 1), 3), (dict(dy=A + 2), 3)]:
        assert back(**kw) == code, kw


def test_workspace_of_the_sort(sdm):
    assert sdm.route_sort_workspace_size(1024, 2, 8) == 0               # one block
    assert sdm.route_sort_workspace_size(1025, 2, 8) == 3 * 8 * 4       # two blocks' counts and the totals
    assert sdm.route_sort_workspace_size(10, 33, 8) == 0


def test_cpu_tensors_are_refused(sdm):
    x, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: sdm.route_sort(i, 4), lambda: sdm.route_gather(x, i, i[0]), lambda: sdm.route_combine(x, i),
                 lambda: sdm.route_combine_backward(x, x, i, x, i[0]),
                 lambda: sdm.gdn_train(torch.zeros(1, 1, 2, 2), *[torch.zeros(1, 1, 1, 2)] * 3, x, x),
                 lambda: sdm.gdn_step(torch.zeros(1, 1, 2, 2), *[torch.zeros(1, 1, 1, 2)] * 3, x, x)):
        with pytest.raises(TypeError):
            call()


def test_reference_sort():
    order, place, offsets = ref.sort_visits(torch.tensor([[1, 0], [-1, 1], [0, 2]]), 3)
    assert order == [1, 4, 0, 3, 5, -1] and place == [2, 0, -1, 3, 1, 4] and offsets == [0, 2, 4, 5]
