"""Host-only checks of the 8-bit activations', the norm's and the gated product's entry points: refusals with
the documented status before anything reaches the GPU, size and workspace queries, and the binding's own checks."""
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
    assert L.mx8_codes_bytes(1, 1) == 32 and L.mx8_scales_bytes(1, 1) == 1
    assert L.mx8_codes_bytes(333, 1000) == 333 * 1024 and L.mx8_scales_bytes(333, 1000) == 333 * 32
    for rows, cols in ((0, 4), (4, 0), (-1, 4), (2**31, 1), (4, 2**31), (2**30, 2**20)):
        assert L.mx8_codes_bytes(rows, cols) == 0 and L.mx8_scales_bytes(rows, cols) == 0


def test_quantize_refusals():
    _, L = _lib()
    f = lambda X=A, dt=1, rows=4, cols=40, ld=40, codes=A, scales=A: L.mx8_quantize(  # noqa: E731
        X, dt, rows, cols, ld, codes, scales, None)
    assert f(X=None) == -1 and f(codes=None) == -1 and f(scales=None) == -1
    assert f(dt=2) == -3
    assert f(rows=0) == -2 and f(cols=-1) == -2 and f(ld=39) == -2 and f(rows=2**30, ld=2**30) == -2
    assert f(X=MIS) == -4 and f(codes=MIS) == -4 and f(scales=MIS) == -4
    assert L.mx8_dequantize(A, None, 4, 40, A, None) == -1
    assert L.mx8_dequantize(A, A, 4, 0, A, None) == -2
    assert L.mx8_dequantize(A, A, 4, 40, MIS, None) == -4


def test_norm_refusals():
    _, L = _lib()
    f = lambda X=A, R=None, dt=1, rows=4, cols=40, w=A, wdt=1, eps=1e-5, S=None, Y=A, c=None, s=None: L.rms_norm_fwd(  # noqa: E731
        X, R, dt, rows, cols, w, wdt, eps, S, Y, c, s, None)
    assert f(X=None) == -1 and f(w=None) == -1 and f(R=A) == -1 and f(Y=None) == -1 and f(c=A) == -1 and f(s=A) == -1
    assert f(dt=2) == -3 and f(wdt=-1) == -3
    assert f(rows=0) == -2 and f(cols=0) == -2 and f(cols=32769) == -2 and f(rows=2**31) == -2
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert f(eps=eps) == -7
    for k in ("X", "w", "Y"):
        assert f(**{k: MIS}) == -4
    assert f(R=MIS, S=A) == -4 and f(R=A, S=MIS) == -4 and f(c=MIS, s=A) == -4 and f(c=A, s=MIS) == -4
    g = lambda dY=A, S=A, dS=None, dt=1, rows=4, cols=40, w=A, wdt=1, eps=1e-5, dX=A, dW=A, ws=A, n=1 << 30: L.rms_norm_bwd(  # noqa: E731
        dY, S, dS, dt, rows, cols, w, wdt, eps, dX, dW, ws, n, None)
    assert g(dY=None) == -1 and g(S=None) == -1 and g(w=None) == -1 and g(dX=None, dW=None) == -1
    assert g(dt=5) == -3 and g(wdt=5) == -3 and g(cols=32769) == -2 and g(eps=0.0) == -7
    assert g(ws=None) == -5 and g(n=L.rms_norm_bwd_workspace(4, 40) - 1) == -5 and g(ws=MIS) == -4
    for k in ("dY", "S", "dS", "w", "dX", "dW"):
        assert g(**{k: MIS}) == -4
    assert L.rms_norm_bwd_workspace(4, 32769) == 0 and L.rms_norm_bwd_workspace(0, 40) == 0


def _fwd(L):
    return lambda X=A, M=4, K=64, F=10, codes=A, c2=A, c1=A, L1=A, L2=A, r=8, H=A, T=None, gc=None, gs=None, ws=A, n=1 << 40: (  # noqa: E731
        L.qlora_swiglu_fwd(X, M, K, F, codes, c2, c1, L1, L2, r, 1.0, H, T, gc, gs, ws, n, None))


def _bwd(L):
    return lambda xc=A, xs=A, d=A, M=4, K=64, F=10, codes=A, c2=A, c1=A, L1=A, L2=A, r=8, gc=A, gs=A, T=A, dX=A, dL1=A, dL2=A, ws=A, n=1 << 40: (  # noqa: E731
        L.qlora_swiglu_bwd(xc, xs, d, M, K, F, codes, c2, c1, L1, L2, r, 1.0, gc, gs, T, dX, dL1, dL2, ws, n, None))


def _lin(L):
    return lambda xc=A, xs=A, d=A, M=4, K=64, F=10, codes=A, c2=A, c1=A, L1=A, L2=A, r=8, T=A, dX=A, dL1=A, dL2=A, ws=A, n=1 << 40: (  # noqa: E731
        L.qlora_linear_bwd_mx8(xc, xs, d, M, K, F, codes, c2, c1, L1, L2, r, 1.0, T, dX, dL1, dL2, ws, n, None))


BASE = ("codes", "c2", "c1", "L1", "L2")


@pytest.mark.parametrize("make,need,may,query", [
    (_fwd, ("X", "H") + BASE, ("T",), "qlora_swiglu_fwd_workspace"),
    (_bwd, ("xc", "xs", "d", "gc", "gs", "T", "dL1", "dL2") + BASE, ("dX",), "qlora_swiglu_bwd_workspace"),
    (_lin, ("xc", "xs", "d", "T", "dL1", "dL2") + BASE, ("dX",), "qlora_linear_bwd_mx8_workspace")])
def test_layer_refusals(make, need, may, query):
    _, L = _lib()
    f, q = make(L), getattr(L, query)
    for k in need:
        assert f(**{k: None}) == -1, k
        assert f(**{k: MIS}) == -4, k
    for k in may:
        assert f(**{k: MIS}) == -4, k
    assert f(ws=None) == -5 and f(ws=MIS) == -4 and f(n=q(4, 64, 10, 8) - 1) == -5
    bad = [dict(M=0), dict(K=0), dict(F=0), dict(F=-3), dict(K=63), dict(K=96), dict(r=0), dict(r=65), dict(M=2**31),
           dict(M=2**24, K=64), dict(M=2**20, F=2**20), dict(M=17, K=2**26), dict(K=2**16, F=2**16), dict(F=2**40),
           dict(M=2**62, K=64)]
    for b in bad:
        assert f(**b) == -2, b
        a = {**dict(M=4, K=64, F=10, r=8), **b}
        assert q(a["M"], a["K"], a["F"], a["r"]) == 0, b
    assert q(4, 64, 10, 8) > 0 and q(1, 64, 1, 1) > 0 and q(4093, 4096, 11007, 37) > 0


def test_forward_copies_go_together():
    _, L = _lib()
    f = _fwd(L)
    assert f(gc=A) == -1 and f(gs=A) == -1 and f(gc=MIS, gs=A) == -4 and f(gc=A, gs=MIS) == -4


def test_workspaces_cover_the_saved_sums():
    """T's planes and at least one slice of both halves; dZ, B's planes turned, and the gradients' slices."""
    _, L = _lib()
    for M, K, F, r in ((1, 64, 1, 1), (17, 4096, 777, 5), (4096, 4096, 11008, 64)):
        assert L.qlora_swiglu_fwd_workspace(M, K, F, r) >= 8 * M * r + 8 * M * r
        turned = 4 * 2 * 2 * r * M
        assert L.qlora_swiglu_bwd_workspace(M, K, F, r) >= 4 * M * F + turned + 8 * r * (K + F)


BF = torch.bfloat16


def test_binding_checks():
    q, _ = _lib()
    z = lambda *s, t=BF: torch.zeros(*s, dtype=t)  # noqa: E731
    u8 = torch.uint8
    with pytest.raises(TypeError):
        q.mx8_quantize(z(4, 40, t=torch.float16))
    with pytest.raises(ValueError):
        q.mx8_quantize(z(40))
    with pytest.raises(ValueError):
        q.mx8_quantize(z(40, 4).t())
    with pytest.raises(ValueError):
        q.mx8_quantize(z(4, 40), codes=z(4, 40, t=u8))
    with pytest.raises(ValueError):
        q.mx8_dequantize(z(4, 40, t=u8), z(4, 2, t=u8), 4, 40)
    with pytest.raises(ValueError):
        q.rms_norm_fwd(z(4, 40), z(41), 1e-5)
    with pytest.raises(ValueError):
        q.rms_norm_fwd(z(4, 40), z(40), 1e-5, residual=z(4, 41))
    with pytest.raises(TypeError):
        q.rms_norm_fwd(z(4, 40), z(40), 1e-5, residual=z(4, 40, t=torch.float32))
    with pytest.raises(ValueError):
        q.rms_norm_fwd(z(4, 40), z(40), 1e-5, S=z(4, 40))
    with pytest.raises(TypeError):
        q.rms_norm_fwd(z(4, 40), z(40), 1e-5, mx8=z(4, 64, t=u8))
    with pytest.raises(ValueError):
        q.rms_norm_fwd(z(40, 4).t(), z(40), 1e-5)
    with pytest.raises(ValueError):
        q.rms_norm_bwd(z(4, 41), z(4, 40), z(40), 1e-5)
    with pytest.raises(TypeError):
        q.rms_norm_bwd(z(4, 40, t=torch.float32), z(4, 40), z(40), 1e-5)
    base = (z(20 * 32, t=u8), z(20, t=u8), z(1, t=torch.float32))
    L1, L2 = z(2, 64, 8), z(2, 8, 10)
    with pytest.raises(ValueError):
        q.qlora_swiglu_fwd(z(4, 64), *base, 11, L1, L2)
    with pytest.raises(ValueError):
        q.qlora_swiglu_fwd(z(4, 64), *base, 10, L1[0], L2)
    with pytest.raises(ValueError):
        q.qlora_swiglu_fwd(z(4, 64), *base, 10, L1, z(2, 7, 10))
    x8, gu8 = (z(4, 64, t=u8), z(4, 2, t=u8)), (z(8, 32, t=u8), z(8, 1, t=u8))
    with pytest.raises(ValueError):
        q.qlora_swiglu_bwd(x8, z(4, 10), *base, L1, L2, x8, z(2, 4, 8))
    with pytest.raises(ValueError):
        q.qlora_swiglu_bwd(x8, z(4, 10), *base, L1, L2, gu8, z(4, 8))
    with pytest.raises(ValueError):                          # everything fits but lies in host memory
        q.qlora_swiglu_bwd(x8, z(4, 10), *base, L1, L2, gu8, z(2, 4, 8))
    with pytest.raises(ValueError):
        q.qlora_linear_bwd_mx8(gu8, z(4, 20), *base, L1[0], z(8, 20), z(4, 8))
    with pytest.raises(ValueError):
        q.qlora_linear_bwd_mx8(x8, z(4, 20), *base, L1[0], z(8, 20), z(4, 8))


def test_binding_wants_one_device():
    """Tensors are refused on another device than the call's stream, and off the GPU, before anything is launched."""
    from bit_quantized_lora_blockwise_amd._lib import _ptrs

    class On:
        shape = (1,)

        def __init__(self, at):
            self.at, self.is_cuda, self.device = at, at >= 0, f"cuda:{at}" if at >= 0 else "cpu"

        def get_device(self):
            return self.at

        def data_ptr(self):
            return 4096 + self.at

    class Stream:
        device_index = 1

    class Handle:
        cuda_stream = 0

    assert _ptrs(Stream, On(1), None, On(1)) == [4097, None, 4097]
    assert _ptrs(Handle, None, On(1), On(1)) == [None, 4097, 4097]
    with pytest.raises(ValueError):
        _ptrs(Handle, On(1), On(0))
    for bad in ((On(0),), (On(1), On(0)), (On(1), None, On(-1)), (On(-1),)):
        with pytest.raises(ValueError):
            _ptrs(Stream, *bad)
