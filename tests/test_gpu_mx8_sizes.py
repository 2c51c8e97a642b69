"""Packing of matrices past 2^31 elements and 2^32 bytes of codes: every value is one that packs exactly."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(66000, 32768), (3, 2**30 + 37), (1, 2**31 - 1), (2**27 + 5, 1)])
def test_many_elements(rows, cols):
    import bit_quantized_lora_blockwise_amd as q
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    flat, n = x.view(-1), rows * cols
    places = sorted({p for p in (0, 1, 2**27 - 1, 2**30 - 1, 2**30, 2**31 - 130, 2**31 - 2, 2**31, 2**31 + 65, n - 2, n - 1)
                     if p < n})
    values = ([0.5, 3.0, -1.5, 4.0, -6.0, 2.0, -0.5, 1.5, 7.0, -3.5, 0.25])[:len(places)]
    flat[torch.tensor(places, device="cuda")] = torch.tensor(values, dtype=torch.bfloat16, device="cuda")
    codes, scales = q.mx8_quantize(x)
    v = q.mx8_dequantize(codes, scales, rows, cols)
    del codes, scales
    assert int((v != x).sum()) == 0
    got = v.view(-1)[torch.tensor(places, device="cuda")].float().cpu().tolist()
    assert got == values
