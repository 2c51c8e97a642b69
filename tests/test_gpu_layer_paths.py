"""Paths of the dropout layers that only larger or odd sizes take, against the float64 oracle."""
import pytest
import torch

import oracle as O
from test_gpu_mx4 import LAYER, check_backward, check_forward, f64, layer_data

pytestmark = pytest.mark.gpu
X4 = O.mx4


def qlib():
    import bit_quantized_lora_blockwise_amd as q
    return q


# rows of W that are no 16-byte pieces (dX in tiles of 128 x 128); more tiles of 256 x 256 than CUs, the last round partly
# empty, so that a work group draws the masks of several tiles and the gradients run beside it: whole and ragged steps
NF4 = [(2093, 1024, 333, 5), (1000, 2048, 77, 64), (2100, 8256, 320, 16), (2093, 8256, 328, 12), (4352, 4160, 128, 64)]


@pytest.mark.parametrize("M,K,N,r", NF4)
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_nf4_layer(M, K, N, r, p):
    q = qlib()
    s, kw = 1.5, dict(p=p, seed=2**63 + 5, offset=2**45 + 1)
    print(f"[nf4 dropout] M={M} K={K} N={N} r={r} p={p}", flush=True)
    d = layer_data(M, K, N, r)
    codes, absmax = q.nf4_quantize(d["W"])
    base = (codes, *q.nf4_double_quant(absmax))
    Wv = f64(q.nf4_dequantize(*base, N, K))
    Y, T = q.qlora_linear_fwd_dropout(d["X"], *base, N, d["L1"], d["L2"], s, T_out=True, **kw)
    check_forward(Y, T, d, f64(d["X"]), Wv, s, p, kw["seed"], kw["offset"])
    dX, dL1, dL2 = q.qlora_linear_bwd_dropout(d["X"], d["dY"], *base, d["L1"], d["L2"], s, T=T, **kw)
    check_backward(dX, dL1, dL2, T, d, f64(d["dY"]), Wv.T.copy(), s, p, kw["seed"], kw["offset"])


@pytest.mark.parametrize("M,K,N,r", LAYER + [(2100, 700, 8200, 16), (700, 1100, 60, 20), (600, 1027, 1025, 6)])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_mx4_gradients_without_t(M, K, N, r, p):
    """T formed again is the forward's, at every size: both gradients have the same bits."""
    q = qlib()
    d = layer_data(M, K, N, r)
    w, wt = q.mx4_quantize(d["W"]), q.mx4_quantize(d["W"], transpose=True)
    kw = dict(p=p, seed=9, offset=10)
    T = q.mx4_linear_fwd(d["X"], *w, N, d["L1"], d["L2"], 2.0, T_out=True, **kw)[1]
    for dX in (True, False):
        _, a1, a2 = q.mx4_linear_bwd(d["X"], d["dY"], *wt, d["L1"], d["L2"], 2.0, T=T, dX=dX, **kw)
        _, b1, b2 = q.mx4_linear_bwd(d["X"], d["dY"], *wt, d["L1"], d["L2"], 2.0, dX=dX, **kw)
        assert torch.equal(a1, b1) and torch.equal(a2, b2)
