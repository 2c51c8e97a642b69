"""Adapters of rank below 8: their rows are shorter than a 16-byte piece, the activations' are not."""
import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_mx4 import check_backward, check_forward, f64, layer_data

pytestmark = pytest.mark.gpu
DEV = "cuda"
X4 = O.mx4


def qlib():
    import bit_quantized_lora_blockwise_amd as q
    return q


# K and N multiples of 8 or not, past the sizes of the few-rows kernels; M on both sides of a tile of 64
SHAPES = [(2100, 1024, 8200, 3), (2093, 8200, 701, 7), (2100, 701, 8200, 1), (700, 1027, 1025, 6), (600, 2048, 2000, 4)]


@pytest.mark.parametrize("M,K,N,r", SHAPES)
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_mx4_layer(M, K, N, r, p):
    q = qlib()
    s, kw = 2.0, dict(p=p, seed=12345, offset=2**32 + 3)
    print(f"[mx4 layer] M={M} K={K} N={N} r={r} p={p}", flush=True)
    d = layer_data(M, K, N, r)
    w, wt = q.mx4_quantize(d["W"]), q.mx4_quantize(d["W"], transpose=True)
    Y, T = q.mx4_linear_fwd(d["X"], *w, N, d["L1"], d["L2"], s, T_out=True, **kw)
    check_forward(Y, T, d, X4.rounded(f64(d["X"])), X4.rounded(f64(d["W"])), s, p, kw["seed"], kw["offset"])
    dX, dL1, dL2 = q.mx4_linear_bwd(d["X"], d["dY"], *wt, d["L1"], d["L2"], s, T=T, **kw)
    check_backward(dX, dL1, dL2, T, d, X4.rounded(f64(d["dY"])), X4.rounded(f64(d["W"]).T), s, p, kw["seed"], kw["offset"])


@pytest.mark.parametrize("M,K,N,r", [(2100, 1024, 2000, 3), (2093, 1088, 701, 7), (600, 2048, 333, 1)])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_nf4_layer(M, K, N, r, p):
    q = qlib()
    s, kw = 1.5, dict(p=p, seed=77, offset=2**45 + 1)
    print(f"[nf4 layer] M={M} K={K} N={N} r={r} p={p}", flush=True)
    d = layer_data(M, K, N, r)
    codes, absmax = q.nf4_quantize(d["W"])
    base = (codes, *q.nf4_double_quant(absmax))
    Wv = f64(q.nf4_dequantize(*base, N, K))
    Y, T = q.qlora_linear_fwd_dropout(d["X"], *base, N, d["L1"], d["L2"], s, T_out=True, **kw)
    check_forward(Y, T, d, f64(d["X"]), Wv, s, p, kw["seed"], kw["offset"])
    dX, dL1, dL2 = q.qlora_linear_bwd_dropout(d["X"], d["dY"], *base, d["L1"], d["L2"], s, T=T, **kw)
    check_backward(dX, dL1, dL2, T, d, f64(d["dY"]), Wv.T.copy(), s, p, kw["seed"], kw["offset"])


def fastest(call, rounds=7, calls=20):
    """Microseconds of the fastest of a few rounds of queued calls."""
    best = float("inf")
    for _ in range(rounds):
        ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        ends[0].record()
        for _ in range(calls):
            call()
        ends[1].record()
        ends[1].synchronize()
        best = min(best, ends[0].elapsed_time(ends[1]) * 1e3 / calls)
    return best


def test_a_small_rank_costs_no_more_than_a_larger_one():
    """T and both gradients at rank 1 read what they read at rank 9, and have less to do.  Half as much again is allowed:
    with the activations read element by element they took twice the time and more."""
    q = qlib()
    M, K, N = 4096, 11008, 4096
    X = torch.randn(M, K, device=DEV).to(torch.bfloat16)
    dY = torch.randn(M, N, device=DEV).to(torch.bfloat16)
    base = (torch.zeros(N, K // 2, dtype=torch.uint8, device=DEV), torch.zeros(N * K // 64, dtype=torch.uint8, device=DEV),
            torch.zeros(N * K // 16384, device=DEV))
    took = {}
    for r in (1, 9):
        L1 = torch.randn(K, r, device=DEV).to(torch.bfloat16)
        L2 = torch.randn(r, N, device=DEV).to(torch.bfloat16)
        T = q.qlora_lora_down(X, L1)
        ws = torch.empty(1 << 27, dtype=torch.uint8, device=DEV)
        kw = dict(T=T, dX=False, workspace=ws)
        took[r] = (fastest(lambda: q.qlora_lora_down(X, L1, T=T, workspace=ws)),
                   fastest(lambda: q.qlora_linear_bwd(X, dY, *base, L1, L2, **kw)),
                   fastest(lambda: q.qlora_linear_bwd_dropout(X, dY, *base, L1, L2, p=0.1, **kw)))
    print(f"rank 1: {took[1]}\nrank 9: {took[9]}", flush=True)
    for a, b in zip(took[1], took[9]):
        assert a <= 1.5 * b
