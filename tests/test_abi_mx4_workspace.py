"""Workspace queries of the microscaled layer: scratch for the kernels that a size takes, not for the others."""
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(
    not os.path.exists(os.path.join(ROOT, "bit_quantized_lora_blockwise_amd", "libqlora.so")),
    reason="libqlora.so not built (run __graft_entry__.build())")


@pytest.mark.parametrize("M,K,N,r", [(65536, 4096, 4096, 64), (65536, 4096, 11008, 64), (32768, 11008, 4096, 16)])
def test_many_rows_keep_few_slices(M, K, N, r):
    """Tiles of 64 rows times slices make about 768 work groups: packed activations, T (G's planes) and as many fp32
    sums of it as that is slices, or the gradients' partial sums."""
    import bit_quantized_lora_blockwise_amd as q
    L = q.lib()
    rest = 8 * 256                                           # each part is rounded up
    sums = -(-768 * 64 // M) * 4 * M * r
    packed = L.mx4_codes_bytes(M, K) + L.mx4_scales_bytes(M, K)
    assert L.mx4_linear_fwd_workspace(M, K, N, r) <= packed + 2 * M * r + sums + rest
    packed = L.mx4_codes_bytes(M, N) + L.mx4_scales_bytes(M, N)
    slices = L.qlora_linear_bwd_workspace(M, K, N, r)        # a bf16 G in place of the planes, otherwise as many
    assert L.mx4_linear_bwd_workspace(M, K, N, r) <= packed + 8 * M * r + max(slices, sums) + rest


@pytest.mark.parametrize("M", [1, 17, 64])
def test_few_rows_keep_eight_slices(M):
    import bit_quantized_lora_blockwise_amd as q
    L = q.lib()
    for K, N, r in ((4096, 11008, 64), (1000, 777, 12)):
        packed = L.mx4_codes_bytes(M, K) + L.mx4_scales_bytes(M, K)
        assert L.mx4_linear_fwd_workspace(M, K, N, r) >= packed + 2 * M * r + 8 * 4 * M * r
        packed = L.mx4_codes_bytes(M, N) + L.mx4_scales_bytes(M, N)
        assert L.mx4_linear_bwd_workspace(M, K, N, r) >= packed + 8 * M * r + 8 * 4 * M * r
