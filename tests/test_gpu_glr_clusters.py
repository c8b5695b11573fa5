"""The gated linear recurrence on clusters of more than eight thread blocks: few
channels and more than 8,192 tokens forward, 4,096 backward (15 and 16 blocks
at these sizes), against the fp64 reference."""
import numpy as np
import pytest
import torch

import glr_reference as ref
from helpers import host, need_gpu
from test_gpu_glr import Case, assert_within, check_backward
from test_gpu_glr_decays import gradients

pytestmark = pytest.mark.gpu

CASES = [dict(B=1, T=8193, D=64), dict(B=1, T=9001, D=70), dict(B=2, T=9001, D=33, reset=0.002, lens=[9001, 8400]),
         dict(B=1, T=8500, D=64, reset=0.001, fused=True)]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("kw", CASES, ids=lambda k: f"B{k['B']}T{k['T']}D{k['D']}")
def test_large_clusters(kw, dt):
    sdm = need_gpu()
    c = Case(**kw, dt=dt, seed=41)
    f, live = c.forward(), c.live()
    s = c.h0.clone()
    y = sdm.glr_scan(s, *c.args(), **c.kw(), y=torch.full((c.B, c.T, c.D), -3.0, dtype=c.dt, device="cuda"))
    assert_within(y, np.where(live, f["y"], -3.0), f["e_y"] * live, c.dt, "y")
    assert_within(s, f["hT"], f["e_hT"], torch.float32, "h_T")
    carry = torch.full((c.B, -(-c.T // 8), c.D), 9.0, device="cuda")
    codes = torch.full((3, c.B, c.T, c.D), 99, dtype=torch.int8, device="cuda")
    exps = torch.full((3, c.B, c.T, -(-c.D // 64)), 77, dtype=torch.uint8, device="cuda")
    s2, y2 = c.h0.clone(), torch.full_like(y, -3.0)
    sdm.glr_scan_train(s2, *c.args(), **c.kw(), y=y2, carry=carry, ckpt=(codes, exps))
    assert torch.equal(y2, y) and torch.equal(s2, s)
    first = live[:, ::8]
    assert_within(carry, np.where(first, f["before"][:, ::8], 9.0), f["e_before"][:, ::8] * first, torch.float32, "carry")
    for i, v in enumerate(c.np("x", "r", "g")):
        q, e = ref.pack8(v)
        assert np.array_equal(host(codes[i]), np.where(live, q, 99))
        assert np.array_equal(host(exps[i]), np.where(live, e, 77))
    check_backward(sdm, c, f, carry, None)
    check_backward(sdm, c, f, carry, (codes, exps))
    b = gradients(c, f)
    drate = sdm.glr_scan_backward(c.dhT.clone(), *c.args(), carry, c.dy, **c.kw())[3]
    assert_within(drate, b["drate"], b["e_drate"], torch.float32, "drate")
