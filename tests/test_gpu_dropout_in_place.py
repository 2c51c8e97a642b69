"""lora_dropout into its own input: rows whose last piece is not whole are the ones where threads' pieces meet."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 8), (4096, 9), (3000, 15), (2000, 513), (777, 4097), (4093, 11007)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("p", [0.0, 0.4])
def test_in_place(rows, cols, dtype, p):
    import bit_quantized_lora_blockwise_amd as q
    x = torch.randn(rows, cols, device=DEV).to(dtype)
    want = q.lora_dropout(x, p, 3, 5)
    for _ in range(5):                               # the order of the threads varies
        y = x.clone()
        assert q.lora_dropout(y, p, 3, 5, out=y) is y
        assert torch.equal(y, want)
