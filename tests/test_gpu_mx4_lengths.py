"""Packing of the longest rows and columns that the calls accept, 2^31 - 1 elements."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols,transpose", [(2**31 - 1, 1, True), (1, 2**31 - 1, True), (1, 2**31 - 1, False),
                                                 (2**31 - 1, 1, False)])
def test_longest(rows, cols, transpose):
    import bit_quantized_lora_blockwise_amd as q
    n = 2**31 - 1
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    places = [0, 1, 2**29 + 3, 2**30 - 1, 2**30, 2**31 - 130, n - 2, n - 1]
    values = [0.5, 3.0, -1.5, 4.0, -6.0, 2.0, -0.5, 1.5]
    x[torch.tensor(places, device="cuda")] = torch.tensor(values, dtype=torch.bfloat16, device="cuda")
    codes, scales = q.mx4_quantize(x.view(rows, cols), transpose=transpose)
    v = q.mx4_dequantize(codes, scales, *((cols, rows) if transpose else (rows, cols))).view(-1)
    del codes, scales
    assert int((v != x).sum()) == 0
