"""GPU parity of the 8-bit activations against the oracle: codes, scale bytes and values are equal."""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import assert_bitexact

pytestmark = pytest.mark.gpu
DEV = "cuda"
X8 = O.mx8


def qlib():
    import bit_quantized_lora_blockwise_amd as q
    return q


def wild(rng, rows, cols):
    """Blocks that differ in size by many powers of two, zeros of both signs, ties, single spikes."""
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-30, 30, (rows, 1)))
    x *= np.where(rng.random((rows, cols)) < 0.02, 1000.0, 1.0)
    x[rng.random((rows, cols)) < 0.1] = 0.0
    x[rng.random((rows, cols)) < 0.05] *= -0.0
    if rows > 2:
        x[1] = 0.0
        x[2] = np.resize([448.0, -17.0, 19.0, 21.0, 2.0**-10, -3 * 2.0**-10, 5 * 2.0**-10, 2.0**-7, 440.0, 15.5], cols)
    return x.astype(np.float32)


SHAPES = [(1, 1), (1, 4096), (3, 31), (5, 32), (2, 33), (17, 127), (16, 128), (33, 129), (333, 1000), (64, 1096),
          (130, 8), (1000, 3), (7, 22016)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_pack_and_values(rows, cols, dtype):
    q = qlib()
    x = torch.from_numpy(wild(np.random.default_rng(rows * 7919 + cols), rows, cols)).to(dtype)
    codes, scales = q.mx8_quantize(x.to(DEV))
    rc, rs = X8.quantize(x.float().numpy())
    assert_bitexact(scales.cpu().numpy(), rs, "scales")
    assert_bitexact(codes.cpu().numpy(), rc, "codes")
    out = q.mx8_dequantize(codes, scales, rows, cols)
    assert_bitexact(out.float().cpu().numpy(), X8.values(rc, rs, cols).astype(np.float32), "values")


def test_every_value_and_every_border():
    """All 254 codes at a scale of 1, the midpoints between them and the fp32 neighbours of these."""
    q = qlib()
    mags = X8.E4M3.astype(np.float32)
    mid = ((X8.E4M3[1:] + X8.E4M3[:-1]) / 2).astype(np.float32)
    v = np.concatenate([mags, mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9))])
    v = np.concatenate([v, -v])
    v = np.pad(v, (0, -v.size % 31)).reshape(-1, 31)
    x = np.concatenate([np.full((v.shape[0], 1), 448, np.float32), v], 1)            # a 448 in each block: scale 1
    codes, scales = q.mx8_quantize(torch.from_numpy(x).to(DEV))
    rc, rs = X8.quantize(x)
    assert (rs == 127).all()
    assert_bitexact(scales.cpu().numpy(), rs, "scales")
    assert_bitexact(codes.cpu().numpy(), rc, "codes")


@pytest.mark.parametrize("k", [-149, -140, -126, -125, -118, -117, -109, -108, -1, 0, 8, 9, 100, 120, 127])
def test_block_maxima_of_every_size(k):
    q = qlib()
    with np.errstate(over="ignore"):
        x = np.ldexp(np.float32([[1.0, 1.75, np.nextafter(np.float32(1.75), np.float32(2)), 1.99]]).T, k) * np.float32(
            [[1.0] + [0.3, -0.01, 0.0] * 10 + [-0.5]])
    x = x.astype(np.float32)
    codes, scales = q.mx8_quantize(torch.from_numpy(x).to(DEV))
    rc, rs = X8.quantize(x)
    assert_bitexact(scales.cpu().numpy(), rs, "scales")
    assert_bitexact(codes.cpu().numpy(), rc, "codes")


def test_blocks_that_are_not_finite():
    q = qlib()
    x = torch.randn(4, 100, generator=torch.Generator().manual_seed(1))
    x[0, 5], x[1, 40], x[2, 99], x[3, 64] = float("inf"), float("nan"), -float("inf"), float("nan")
    for dtype in (torch.float32, torch.bfloat16):
        xx = x.to(dtype)
        codes, scales = q.mx8_quantize(xx.to(DEV))
        rc, rs = X8.quantize(xx.float().numpy())
        assert_bitexact(scales.cpu().numpy(), rs, "scales")
        assert_bitexact(codes.cpu().numpy(), rc, "codes")
        out = q.mx8_dequantize(codes, scales, 4, 100).float().cpu().numpy()
        assert np.array_equal(np.isnan(out), np.repeat(rs == 255, 32, 1)[:, :100])


def test_rows_apart_and_given_outputs():
    q = qlib()
    big = torch.randn(9, 200, device=DEV).to(torch.bfloat16)
    x = big[:, 8:108]
    codes = torch.full((9, 128), 77, dtype=torch.uint8, device=DEV)
    scales = torch.full((9, 4), 77, dtype=torch.uint8, device=DEV)
    got = q.mx8_quantize(x, codes=codes, scales=scales)
    rc, rs = X8.quantize(x.float().cpu().numpy())
    assert got[0] is codes and got[1] is scales
    assert_bitexact(codes.cpu().numpy(), rc, "codes")
    assert_bitexact(scales.cpu().numpy(), rs, "scales")


@pytest.mark.parametrize("rows,cols", [(70000, 40), (2, 70001)])
def test_many_rows_and_long_rows(rows, cols):
    q = qlib()
    x = torch.randn(rows, cols, device=DEV, generator=torch.Generator(DEV).manual_seed(3)).to(torch.bfloat16)
    codes, scales = q.mx8_quantize(x)
    pick = np.unique(np.linspace(0, rows - 1, 500).astype(int))
    rc, rs = X8.quantize(x[torch.from_numpy(pick).to(DEV)].float().cpu().numpy())
    assert_bitexact(codes.cpu().numpy()[pick], rc, "codes")
    assert_bitexact(scales.cpu().numpy()[pick], rs, "scales")
    out = q.mx8_dequantize(codes, scales, rows, cols)
    assert_bitexact(out.float().cpu().numpy()[pick], X8.values(rc, rs, cols).astype(np.float32), "values")
