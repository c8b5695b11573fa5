"""Sizes beyond 32 bits are refused by the binding, not cut off."""
import pytest
import torch

from helpers import need_gpu

pytestmark = pytest.mark.gpu


def test_sizes_beyond_32_bits_are_refused():
    sdm = need_gpu()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    x = torch.zeros((1, (1 << 32) + 9, 1), dtype=torch.bfloat16, device="cuda")      # 9 in an int of 32 bits
    s, rate = torch.zeros((1, 1), device="cuda"), torch.ones(1, device="cuda")
    carry = torch.zeros((1, 2, 1), device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        sdm.glr_scan(s, x, x, x, rate, y=x)
    with pytest.raises(ValueError, match="2\\^31"):
        sdm.glr_scan_train(s, x, x, x, rate, y=x, carry=carry)
    with pytest.raises(ValueError, match="2\\^31"):
        sdm.glr_scan_backward(s, x, x, x, rate, carry, x)
    with pytest.raises(ValueError, match="2\\^31"):
        sdm.ckpt8_pack(x.view(-1))
    codes = torch.zeros((1 << 32) + 64, dtype=torch.int8, device="cuda")
    with pytest.raises(ValueError, match="2\\^31"):
        sdm.ckpt8_unpack(codes, torch.zeros((1 << 26) + 1, dtype=torch.uint8, device="cuda"), x=x.view(-1)[:codes.numel()])
    with pytest.raises(sdm.SdmError):       # a flat tensor of 2^24 and more is the library's to refuse
        sdm.ckpt8_pack(x.view(-1)[:1 << 24])
