"""ckpt8_unpack into a buffer takes the buffer's type."""
import pytest
import torch

from helpers import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_the_buffer_s_type(dt):
    sdm = need_gpu()
    codes, exps = sdm.ckpt8_pack(torch.randn((5, 130), device="cuda"))
    want = sdm.ckpt8_unpack(codes, exps, dt)
    out = torch.empty((5, 130), dtype=dt, device="cuda")
    assert sdm.ckpt8_unpack(codes, exps, x=out) is out and torch.equal(out, want)
    assert sdm.ckpt8_unpack(codes, exps).dtype == torch.bfloat16
    other = torch.float32 if dt is torch.bfloat16 else torch.bfloat16
    with pytest.raises(TypeError):      # both given, and not the same
        sdm.ckpt8_unpack(codes, exps, other, x=out)
    with pytest.raises(TypeError):
        sdm.ckpt8_unpack(codes, exps, x=out.double())
