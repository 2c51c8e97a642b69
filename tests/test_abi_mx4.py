"""Host-only checks of the microscaled and dropout entry points: refusals with
the documented status before anything reaches the GPU, workspace and size
queries, and the binding's own checks."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(
    not os.path.exists(os.path.join(ROOT, "bit_quantized_lora_blockwise_amd", "libqlora.so")),
    reason="libqlora.so not built (run __graft_entry__.build())")

P = ctypes.c_void_p
A, MIS = P(4096), P(4104)      # stand-in pointers (never dereferenced); MIS is 8-byte aligned only


def _lib():
    import bit_quantized_lora_blockwise_amd as q
    return q, q.lib()


def test_packed_sizes():
    _, L = _lib()
    assert L.mx4_codes_bytes(1, 1) == 64 and L.mx4_scales_bytes(1, 1) == 4
    assert L.mx4_codes_bytes(333, 1000) == 333 * 512 and L.mx4_scales_bytes(333, 1000) == 333 * 32
    for rows, cols in ((0, 4), (4, 0), (-1, 4), (2**31, 1), (4, 2**31)):
        assert L.mx4_codes_bytes(rows, cols) == 0 and L.mx4_scales_bytes(rows, cols) == 0


def test_quantize_refusals():
    _, L = _lib()
    f = lambda X=A, dt=1, rows=4, cols=40, ld=40, codes=A, scales=A: L.mx4_quantize(  # noqa: E731
        X, dt, rows, cols, ld, 0, codes, scales, None)
    assert f(X=None) == -1 and f(codes=None) == -1 and f(scales=None) == -1
    assert f(dt=2) == -3
    assert f(rows=0) == -2 and f(cols=-1) == -2 and f(ld=39) == -2 and f(rows=2**30, ld=2**30) == -2
    assert f(X=MIS) == -4 and f(codes=MIS) == -4 and f(scales=MIS) == -4
    assert L.mx4_dequantize(A, None, 4, 40, A, None) == -1
    assert L.mx4_dequantize(A, A, 4, 0, A, None) == -2
    assert L.mx4_dequantize(A, A, 4, 40, MIS, None) == -4
    assert L.mx4_matmul(A, A, 4, A, A, 4, 40, None, None) == -1
    assert L.mx4_matmul(A, A, 0, A, A, 4, 40, A, None) == -2
    assert L.mx4_matmul(A, A, 2**16, A, A, 2**15, 40, A, None) == -2          # C reaches 2^31 bytes
    assert L.mx4_matmul(A, A, 4, A, A, 2**25, 128, A, None) == -2             # B's codes reach 2^31 bytes
    assert L.mx4_matmul(A, A, 4, A, MIS, 4, 40, A, None) == -4


def test_dropout_refusals():
    _, L = _lib()
    f = lambda X=A, dt=0, rows=4, cols=40, ld=40, p=0.1, Y=A: L.lora_dropout(  # noqa: E731
        X, dt, rows, cols, ld, p, 1, 2, Y, None)
    assert f(X=None) == -1 and f(Y=None) == -1 and f(dt=7) == -3 and f(cols=0) == -2 and f(ld=1) == -2
    assert f(p=1.0) == -7 and f(p=-0.01) == -7 and f(p=float("nan")) == -7
    assert f(Y=MIS) == -4


@pytest.mark.parametrize("fn", ["mx4", "qlora"])
def test_layer_refusals(fn):
    _, L = _lib()
    M, K, N, r = 32, 512, 512, 8
    fws = getattr(L, "mx4_linear_fwd_workspace" if fn == "mx4" else "qlora_linear_fwd_dropout_workspace")
    bws = getattr(L, "mx4_linear_bwd_workspace" if fn == "mx4" else "qlora_linear_bwd_dropout_workspace")
    base = 2 if fn == "mx4" else 3
    need, needb = fws(M, K, N, r), bws(M, K, N, r)
    assert need > 0 and needb > 0
    for bad in ((0, K, N, r), (M, 0, N, r), (M, K, -1, r), (M, K, N, 0), (M, K, N, 65), (2**30, K, N, r)):
        assert fws(*bad) == 0 and bws(*bad) == 0

    def fwd(X=A, M=M, K=K, r=r, p=0.1, Y=A, T=None, ws=A, wsb=need, w=A):
        f = L.mx4_linear_fwd if fn == "mx4" else L.qlora_linear_fwd_dropout
        return f(X, M, K, N, *[w] * base, A, A, r, 1.0, p, 5, 6, Y, T, ws, wsb, None)

    assert fwd(X=None) == -1 and fwd(w=None) == -1 and fwd(Y=None) == -1
    assert fwd(M=0) == -2 and fwd(r=65) == -2 and fwd(M=2**30) == -2
    assert fwd(p=1.0) == -7 and fwd(p=-1.0) == -7 and fwd(p=float("nan")) == -7
    assert fwd(X=MIS) == -4 and fwd(T=MIS) == -4 and fwd(ws=MIS) == -4
    assert fwd(ws=None) == -5 and fwd(wsb=need - 1) == -5

    def bwd(X=A, dY=A, M=M, r=r, p=0.1, T=A, dX=A, dL1=A, ws=A, wsb=needb, w=A):
        f = L.mx4_linear_bwd if fn == "mx4" else L.qlora_linear_bwd_dropout
        return f(X, dY, M, K, N, *[w] * base, A, A, r, 1.0, p, 5, 6, T, dX, dL1, A, ws, wsb, None)

    assert bwd(dY=None) == -1 and bwd(dL1=None) == -1 and bwd(w=None) == -1
    assert bwd(M=-4) == -2 and bwd(r=0) == -2
    assert bwd(p=1.5) == -7
    assert bwd(dX=MIS) == -4 and bwd(T=MIS) == -4 and bwd(dL1=MIS) == -4
    assert bwd(ws=None) == -5 and bwd(wsb=needb - 1) == -5


def test_qlora_dropout_needs_whole_blocks():
    _, L = _lib()
    assert L.qlora_linear_fwd_dropout(A, 4, 100, 8, A, A, A, A, A, 4, 1.0, 0.1, 0, 0, A, None, A, 1 << 20, None) == -2


def test_binding_checks():
    q, _ = _lib()
    x = torch.zeros(4, 40, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        q.mx4_quantize(x.half())
    with pytest.raises(ValueError):
        q.mx4_quantize(x.t())
    with pytest.raises(ValueError):
        q.mx4_quantize(x.view(2, 2, 40))
    with pytest.raises(ValueError):
        q.mx4_quantize(x[:1].expand(4, 40))                  # rows that overlap
    with pytest.raises(ValueError):
        q.mx4_quantize(x[:0])
    with pytest.raises(ValueError, match="on the GPU"):
        q.mx4_quantize(x)
    c, s = torch.zeros(4, 4, 16, dtype=torch.uint8), torch.zeros(1, 4, 4, dtype=torch.uint8)
    with pytest.raises(ValueError):
        q.mx4_dequantize(c, s, 4, 129)
    with pytest.raises(ValueError):
        q.mx4_dequantize(c, s, 5, 40)
    with pytest.raises(ValueError):
        q.mx4_matmul(c, s, 4, c, s, 3, 40)
    with pytest.raises(ValueError):
        q.lora_dropout(x, 0.1, -1)
    with pytest.raises(ValueError):
        q.lora_dropout(x, 0.1, 1, 2**64)
    with pytest.raises(ValueError):
        q.lora_dropout(x, 0.1, 0.5)
    l1, l2 = torch.zeros(40, 3, dtype=torch.bfloat16), torch.zeros(3, 4, dtype=torch.bfloat16)
    for bad in (dict(L1=l1[:39]), dict(L2=l2[:2]), dict(N=5), dict(scales=s[:, :3])):
        a = dict(X=x, codes=c, scales=s, N=4, L1=l1, L2=l2)
        a.update(bad)
        with pytest.raises(ValueError):
            q.mx4_linear_fwd(**a)
    with pytest.raises(ValueError):
        q.mx4_linear_bwd(x, x, c, s, l1, l2)                 # dY has 40 columns, L2 has 4
