"""The default stream's handle as a call's `stream`: in order with the default stream's work."""
import pytest
import torch

from helpers import need_gpu
from test_gpu_glr import Case

pytestmark = pytest.mark.gpu


def test_the_null_handle_is_the_default_stream():
    sdm = need_gpu()
    c = Case(2, 40, 64, "bf16", seed=51)
    want = sdm.glr_scan(c.h0.clone(), *c.args())
    q, e = sdm.ckpt8_pack(c.x)
    late = c.x.clone()
    torch.cuda.synchronize()
    for handle in (0, torch.cuda.default_stream().cuda_stream):
        c.x.zero_()
        torch.cuda._sleep(20_000_000)       # the inputs come 10 ms later, on the default stream
        c.x.copy_(late)
        y = sdm.glr_scan(c.h0.clone(), *c.args(), stream=handle)
        codes, exps = sdm.ckpt8_pack(c.x, stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(codes, q) and torch.equal(exps, e)
