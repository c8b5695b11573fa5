"""The 8-bit activation checkpoints on the GPU: every code and exponent equal
to the reference's, every unpacked value equal to what it stands for."""
import numpy as np
import pytest
import torch

import glr_reference as ref
from helpers import host, need_gpu

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (3, 2), (1, 63), (5, 64), (2, 65), (7, 127), (4, 128), (33, 200), (2, 1920), (300, 963), (1, 100000)]


def _values(rows, D, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, D)) * np.exp(rng.normal(size=(rows, 1)) * 4)
    x[rng.random((rows, D)) < 0.02] *= 300
    return torch.from_numpy(x.astype(np.float32)).cuda()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["plain", "wide", "odd"])
@pytest.mark.parametrize("rows,D", SHAPES)
def test_pack_and_unpack(rows, D, layout, dt):
    sdm = need_gpu()
    x = _values(rows, D, rows + D).to(dt)
    if layout != "plain":
        off, more = (64, 64) if layout == "wide" else (1, 2)
        wide = torch.full((rows, D + off + more), 5.0, dtype=dt, device="cuda")
        wide[:, off:off + D] = x
        x = wide[:, off:off + D]
    codes, exps = sdm.ckpt8_pack(x)
    q, e = ref.pack8(x.double().cpu().numpy())
    assert np.array_equal(host(codes), q) and np.array_equal(host(exps), e)
    want = ref.unpack8(q, e)
    for to in (torch.bfloat16, torch.float32):
        assert np.array_equal(sdm.ckpt8_unpack(codes, exps, to).double().cpu().numpy(), want)
    if layout != "plain":
        out = torch.full_like(wide, 3.0)
        sdm.ckpt8_unpack(codes, exps, dt, x=out[:, off:off + D])
        assert np.array_equal(out[:, off:off + D].double().cpu().numpy(), want)
        assert torch.all(out[:, :off] == 3.0) and torch.all(out[:, off + D:] == 3.0)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_edges_of_the_format(dt):
    """Zeros, denormals, the largest values (above 127 * 2^121: NaN), exact powers and 127 times one,
    halves between two codes, and one value of each kind alone in its group."""
    sdm = need_gpu()
    top = torch.finfo(dt).max
    vals = [0.0, -0.0, 1.0, -1.0, 127.0, 127.5, 128.0, 0.5, 63.5, 2.0 ** -126, 2.0 ** -130, 2.0 ** -149, top, -top, top / 2,
            1e-30, 254.0, 2.0 ** 120 * 127, 2.0 ** 121 * 127, 2.0 ** 121 * 127.5, 2.0 ** -126 * 127, 2.0 ** -126 * 128]
    x = torch.zeros((len(vals), 130), dtype=dt)
    for i, v in enumerate(vals):
        x[i, (7 * i) % 130] = v
    ties = torch.arange(64, dtype=torch.float32) * 2 + 0.5
    ties[63] = 127.0
    x = torch.cat([x, torch.cat([ties, -ties, torch.zeros(2)])[None].to(dt)]).cuda()
    codes, exps = sdm.ckpt8_pack(x)
    q, e = ref.pack8(x.double().cpu().numpy())
    assert np.array_equal(host(codes), q) and np.array_equal(host(exps), e)
    assert np.array_equal(sdm.ckpt8_unpack(codes, exps, torch.float32).double().cpu().numpy(), ref.unpack8(q, e), equal_nan=True)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite(bad, dt):
    sdm = need_gpu()
    x = _values(6, 200, 1).to(dt)
    x[2, 70] = bad
    x[4, 199] = bad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    codes, exps = sdm.ckpt8_pack(x, dev_err=err)
    q, e = ref.pack8(x.double().cpu().numpy())
    assert int(err.item()) == sdm.SDM_DEVERR_NONFINITE
    assert np.array_equal(host(codes), q) and np.array_equal(host(exps), e)
    for to in (torch.bfloat16, torch.float32):
        assert np.array_equal(sdm.ckpt8_unpack(codes, exps, to).double().cpu().numpy(), ref.unpack8(q, e), equal_nan=True)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rows_at_every_boundary(dt):
    """Rows that begin anywhere among 32 bytes: what lies between them stays out and is left alone."""
    sdm = need_gpu()
    rows, D = 9, 72
    v = _values(rows, D, 3).to(dt)
    q, e = ref.pack8(v.double().cpu().numpy())
    want = ref.unpack8(q, e)
    for shift in range(17):
        for ld in (72, 73, 76, 80, 88):
            buf = torch.full((shift + rows * ld + 1,), float("nan"), dtype=dt, device="cuda")
            x = torch.as_strided(buf, (rows, D), (ld, 1), shift)
            x.copy_(v)
            codes, exps = sdm.ckpt8_pack(x)
            assert np.array_equal(host(codes), q) and np.array_equal(host(exps), e)
            buf.fill_(3.0)
            sdm.ckpt8_unpack(codes, exps, dt, x=x)
            assert np.array_equal(x.double().cpu().numpy(), want)
            x.fill_(3.0)
            assert torch.all(buf == 3.0)


def test_shapes_and_refusals():
    sdm = need_gpu()
    x = torch.randn((2, 3, 5, 70), device="cuda")
    codes, exps = sdm.ckpt8_pack(x)
    assert codes.shape == x.shape and exps.shape == (2, 3, 5, 2)
    flat, _ = sdm.ckpt8_pack(x.view(-1, 70))
    assert torch.equal(flat.view_as(codes), codes)
    row, _ = sdm.ckpt8_pack(x[0, 0, 0])                      # one row, no leading dimension
    assert torch.equal(row, codes[0, 0, 0])
    for shape in ((0, 70), (4, 0)):
        c, e = sdm.ckpt8_pack(torch.empty(shape, device="cuda"))
        assert c.shape == shape and sdm.ckpt8_unpack(c, e, torch.float32).shape == shape
    for bad, err in ((x.half(), TypeError), (x.transpose(2, 3), ValueError), (x[:, :, ::2], ValueError), (x.cpu(), TypeError),
                     (x[:, :, :1].expand(2, 3, 5, 70), ValueError)):
        with pytest.raises(err):
            sdm.ckpt8_pack(bad)
    with pytest.raises(ValueError):
        sdm.ckpt8_unpack(codes, exps[..., :1].contiguous())
    with pytest.raises(TypeError):
        sdm.ckpt8_unpack(codes, exps, torch.float16)
    with pytest.raises(TypeError):
        sdm.ckpt8_unpack(codes.to(torch.uint8), exps)
