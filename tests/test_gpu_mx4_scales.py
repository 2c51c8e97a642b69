"""Packed matrices of any producer: every scale byte of the format, not only those that mx4_quantize writes."""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
X4 = O.mx4


def qlib():
    import bit_quantized_lora_blockwise_amd as q
    return q


def packed(scales):
    """A matrix [len(scales), 32]: every code twice a row, one scale byte a row."""
    codes = np.tile(np.arange(16, dtype=np.uint8), (len(scales), 8))
    codes[:, 32:] = 0
    by = np.full((len(scales), 4), 127, np.uint8)
    by[:, 0] = scales
    return codes, by


def test_dequantize_every_scale_byte():
    """The nearest bf16 of every value: exact, subnormals among them, infinite past bf16's range, NaN for byte 255."""
    q = qlib()
    codes, by = packed(np.arange(256))
    c, s = (torch.from_numpy(a).to(DEV) for a in X4.pack(codes, by))
    got = q.mx4_dequantize(c, s, 256, 32).float().cpu().numpy().astype(np.float64)
    ref = X4.values(codes, by, 32)
    top = float(torch.finfo(torch.bfloat16).max)
    ref = np.where(np.abs(ref) > top, np.copysign(np.inf, ref), ref)
    bad = np.nonzero(~((got == ref) | (np.isnan(got) & np.isnan(ref))))
    assert bad[0].size == 0, (sorted(set(bad[0])), got[bad][:8], ref[bad][:8])
    assert np.array_equal(np.signbit(got[:255]), np.signbit(ref[:255]))


@pytest.mark.parametrize("rows", [255, 300])
def test_matmul_every_scale_byte(rows):
    """Rows of A with every scale byte against columns of B whose scale brings the product back near 1: exact."""
    q = qlib()
    a_codes, a_by = packed(np.arange(255))
    b_codes, b_by = packed(254 - np.arange(255))
    b_codes[:, 1:] = 0
    b_codes[:, 0] = 2                                        # 1.0, at the first element alone
    a_codes = np.roll(a_codes[:, :32], -5, axis=1)           # whose code in A is 5: 3.0
    a_codes = np.concatenate([a_codes, np.zeros((255, 96), np.uint8)], 1)
    a_codes, a_by = np.tile(a_codes, (2, 1))[:rows], np.tile(a_by, (2, 1))[:rows]
    ac, asc = (torch.from_numpy(x).to(DEV) for x in X4.pack(a_codes, a_by))
    bc, bsc = (torch.from_numpy(x).to(DEV) for x in X4.pack(b_codes, b_by))
    got = q.mx4_matmul(ac, asc, rows, bc, bsc, 255, 32).float().cpu().numpy()
    i = np.arange(rows)
    assert np.array_equal(got[i, a_by[:, 0]], np.full(rows, 3.0))
