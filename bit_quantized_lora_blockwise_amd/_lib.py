"""ctypes binding of libqlora.so: argument marshalling only.

Every function here has the name of the C entry point it calls (see
include/qlora.h for the contract).  Tensors are torch tensors on the GPU; the
binding checks dtype, shape or element count, contiguity and device of every
tensor (inputs and caller-supplied outputs), allocates missing outputs with torch,
passes raw pointers and the current HIP stream, and raises QloraError on a
non-zero status.  All computation happens in the HIP kernels.
"""
from __future__ import annotations

import ctypes
import os

import torch

# QLORA_LIBRARY selects another build of the same library (the host-sanitized
# one that the sanitizer test runs the ABI checks against); default: in-tree.
_LIB_PATH = os.environ.get("QLORA_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqlora.so")
_lib = None

QL_F32, QL_BF16 = 0, 1
CODEBOOKS = {"nf4": 0, "fp4": 1, "int4": 2}
SCALE_CODES = {"groupmax": 0, "fullrange": 1, "mean": 2, "absmax": 3}
STATUS = {0: "QL_OK", -1: "QL_ERR_NULL", -2: "QL_ERR_SHAPE", -3: "QL_ERR_DTYPE", -4: "QL_ERR_ALIGN",
          -5: "QL_ERR_WORKSPACE", -6: "QL_ERR_HIP", -7: "QL_ERR_VALUE"}
EXPORTS = ("nf4_quantize", "nf4_quantize_dq", "nf4_double_quant", "nf4_dequantize", "qlora_linear_fwd_workspace",
           "qlora_linear_fwd", "qlora_linear_bwd_workspace", "qlora_linear_bwd", "qlora_nf4_levels",
           "ql_status_string", "qlora_lora_down_workspace", "qlora_lora_down", "qlora_linear_fwd_t",
           "qlora_lora_grad_in_workspace", "qlora_lora_grad_in", "qlora_linear_dx", "qlora_merge",
           "q4_quantize", "q4_double_quant", "q4_dequantize", "q4_levels",
           "qlora_group_fwd_workspace", "qlora_group_fwd", "qlora_group_bwd_workspace", "qlora_group_bwd",
           "qlora_adamw_step", "qlora_linear_fwd_noalloc",
           "lora_linear_fwd", "lora_linear_bwd", "lora_linear_fwd_t", "lora_linear_dx",
           "lora_dropout", "qlora_linear_fwd_dropout_workspace", "qlora_linear_fwd_dropout",
           "qlora_linear_bwd_dropout_workspace", "qlora_linear_bwd_dropout",
           "mx4_codes_bytes", "mx4_scales_bytes", "mx4_quantize", "mx4_dequantize", "mx4_matmul",
           "mx4_linear_fwd_workspace", "mx4_linear_fwd", "mx4_linear_bwd_workspace", "mx4_linear_bwd",
           "mx8_codes_bytes", "mx8_scales_bytes", "mx8_quantize", "mx8_dequantize",
           "rms_norm_fwd", "rms_norm_bwd_workspace", "rms_norm_bwd",
           "qlora_swiglu_fwd_workspace", "qlora_swiglu_fwd", "qlora_swiglu_bwd_workspace", "qlora_swiglu_bwd",
           "qlora_linear_bwd_mx8_workspace", "qlora_linear_bwd_mx8")


class QloraError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({lib().ql_status_string(status).decode()})")


def lib():
    """The loaded library; raises if it has not been built (no fallback path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                               "`python -m bit_quantized_lora_blockwise_amd.build`")
        L = ctypes.CDLL(_LIB_PATH)
        P, I64, I32, F32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        F64, U64 = ctypes.c_double, ctypes.c_uint64
        sig = {
            "nf4_quantize": ([P, I32, I64, I64, P, P, P], I32),
            "nf4_double_quant": ([P, I64, P, P, P], I32),
            "nf4_dequantize": ([P, P, P, I64, I64, P, P], I32),
            "nf4_quantize_dq": ([P, I32, I64, I64, P, P, P, P, P], I32),
            "qlora_linear_fwd_workspace": ([I64, I64, I64, I32], SZ),
            "qlora_linear_fwd": ([P, I64, I64, I64, P, P, P, P, P, I32, F32, P, P, P, SZ, P], I32),
            "qlora_linear_bwd_workspace": ([I64, I64, I64, I32], SZ),
            "qlora_linear_bwd": ([P, P, I64, I64, I64, P, P, P, P, P, I32, F32, P, P, P, P, P, SZ, P], I32),
            "qlora_nf4_levels": ([P], I32),
            "ql_status_string": ([I32], ctypes.c_char_p),
            "qlora_lora_down_workspace": ([I64, I64, I32], SZ),
            "qlora_lora_down": ([P, I64, I64, P, I32, P, P, SZ, P], I32),
            "qlora_linear_fwd_t": ([P, I64, I64, I64, P, P, P, P, P, I32, F32, P, P], I32),
            "qlora_lora_grad_in_workspace": ([I64, I64, I32], SZ),
            "qlora_lora_grad_in": ([P, I64, I64, P, I32, F32, P, P, SZ, P], I32),
            "qlora_linear_dx": ([P, I64, I64, I64, P, P, P, P, P, I32, P, P], I32),
            "qlora_merge": ([P, P, P, I64, I64, P, P, I32, F32, P, P], I32),
            "q4_quantize": ([P, I32, I64, I64, I32, P, P, P], I32),
            "q4_double_quant": ([P, I64, I32, P, P, P, P], I32),
            "q4_dequantize": ([P, I64, I64, I32, I32, P, P, P, P, P, P], I32),
            "q4_levels": ([I32, P], I32),
            "qlora_group_fwd_workspace": ([I64, I64, I64, I32, I32], SZ),
            "qlora_group_fwd": ([P, I64, I64, I64, I32, P, P, P, P, P, I32, F32, P, P, P, SZ, P], I32),
            "qlora_group_bwd_workspace": ([I64, I64, I64, I32, I32], SZ),
            "qlora_group_bwd": ([P, P, I64, I64, I64, I32, P, P, P, P, P, I32, F32, P, P, P, P, P, SZ, P], I32),
            "qlora_adamw_step": ([P, P, P, P, P, I64, F32, F32, F32, F32, F32, I64, P], I32),
            "qlora_linear_fwd_noalloc": ([P, I64, I64, I64, P, P, P, P, P, I32, F32, P, P, P], I32),
            "lora_linear_fwd": ([P, I64, I64, I64, P, P, P, I32, F32, P, P, P, SZ, P], I32),
            "lora_linear_bwd": ([P, P, I64, I64, I64, P, P, P, I32, F32, P, P, P, P, P, SZ, P], I32),
            "lora_linear_fwd_t": ([P, I64, I64, I64, P, P, P, I32, F32, P, P], I32),
            "lora_linear_dx": ([P, I64, I64, I64, P, P, P, I32, P, P], I32),
            "lora_dropout": ([P, I32, I64, I64, I64, F64, U64, U64, P, P], I32),
            "qlora_linear_fwd_dropout_workspace": ([I64, I64, I64, I32], SZ),
            "qlora_linear_fwd_dropout": ([P, I64, I64, I64, P, P, P, P, P, I32, F32, F64, U64, U64, P, P, P, SZ, P],
                                         I32),
            "qlora_linear_bwd_dropout_workspace": ([I64, I64, I64, I32], SZ),
            "qlora_linear_bwd_dropout": ([P, P, I64, I64, I64, P, P, P, P, P, I32, F32, F64, U64, U64, P, P, P, P, P,
                                          SZ, P], I32),
            "mx4_codes_bytes": ([I64, I64], SZ),
            "mx4_scales_bytes": ([I64, I64], SZ),
            "mx4_quantize": ([P, I32, I64, I64, I64, I32, P, P, P], I32),
            "mx4_dequantize": ([P, P, I64, I64, P, P], I32),
            "mx4_matmul": ([P, P, I64, P, P, I64, I64, P, P], I32),
            "mx4_linear_fwd_workspace": ([I64, I64, I64, I32], SZ),
            "mx4_linear_fwd": ([P, I64, I64, I64, P, P, P, P, I32, F32, F64, U64, U64, P, P, P, SZ, P], I32),
            "mx4_linear_bwd_workspace": ([I64, I64, I64, I32], SZ),
            "mx4_linear_bwd": ([P, P, I64, I64, I64, P, P, P, P, I32, F32, F64, U64, U64, P, P, P, P, P, SZ, P], I32),
            "mx8_codes_bytes": ([I64, I64], SZ),
            "mx8_scales_bytes": ([I64, I64], SZ),
            "mx8_quantize": ([P, I32, I64, I64, I64, P, P, P], I32),
            "mx8_dequantize": ([P, P, I64, I64, P, P], I32),
            "rms_norm_fwd": ([P, P, I32, I64, I64, P, I32, F32, P, P, P, P, P], I32),
            "rms_norm_bwd_workspace": ([I64, I64], SZ),
            "rms_norm_bwd": ([P, P, P, I32, I64, I64, P, I32, F32, P, P, P, SZ, P], I32),
            "qlora_swiglu_fwd_workspace": ([I64, I64, I64, I32], SZ),
            "qlora_swiglu_fwd": ([P, I64, I64, I64, P, P, P, P, P, I32, F32, P, P, P, P, P, SZ, P], I32),
            "qlora_swiglu_bwd_workspace": ([I64, I64, I64, I32], SZ),
            "qlora_swiglu_bwd": ([P, P, P, I64, I64, I64, P, P, P, P, P, I32, F32, P, P, P, P, P, P, P, SZ, P], I32),
            "qlora_linear_bwd_mx8_workspace": ([I64, I64, I64, I32], SZ),
            "qlora_linear_bwd_mx8": ([P, P, P, I64, I64, I64, P, P, P, P, P, I32, F32, P, P, P, P, P, SZ, P], I32),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, res
        _lib = L
    return _lib


def _ptr(t):
    """Device address of a tensor argument (None -> NULL).  Every tensor reaches
    the library through here, after all size checks: this is the device check."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"every tensor argument must be on the GPU (got a {t.device} tensor of shape "
                         f"{tuple(t.shape)})")
    return t.data_ptr()


def _stream(stream=None):
    """The HIP stream of a call.  Without one given, the current device's current
    stream, asked for as a number: building a torch.cuda.Stream for it takes 3 us,
    as long as a kernel launch."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _ptrs(stream, *tensors):
    """Device addresses of a call's tensor arguments (None -> NULL), which all have to be on the device of
    its stream (of one another, where only the stream's handle is known): a kernel runs there, and memory of
    another device may not be mapped on it."""
    dev, out = None, []
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        at = t.get_device()
        if at != dev:
            out.append(_ptr(t))            # refuses what is not on a GPU
            if dev is None:
                dev = torch._C._cuda_getDevice() if stream is None else getattr(stream, "device_index", at)
            if at != dev:
                raise ValueError(f"every tensor argument must be on the device of the call's stream, cuda:{dev} (got a "
                                 f"{t.device} tensor of shape {tuple(t.shape)})")
        else:
            out.append(t.data_ptr())
    return out


def _need(t, name, dtype, ndim=None, shape=None, numel=None):
    """Check a tensor argument: type, dtype, rank, shape or element count and
    contiguity (the device is checked when its pointer is taken, after every
    size check of the call)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if shape is not None and t.shape != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} elements, got {t.numel()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _packed(codes, c2, c1, rows, cols):
    """The packed base of a [rows, cols] weight: codes rows*cols/2 bytes, c2 one
    byte per block of 64, c1 one fp32 per group of 256 blocks."""
    if rows <= 0 or cols <= 0 or cols % 64:
        raise ValueError(f"weight shape [{rows}, {cols}]: sizes must be > 0 and cols a multiple of 64")
    nb = rows * cols // 64
    _need(codes, "codes", torch.uint8, numel=rows * cols // 2)
    _need(c2, "c2", torch.uint8, numel=nb)
    _need(c1, "c1", torch.float32, numel=(nb + 255) // 256)


def _out(t, name, dtype, shape, like, stream):
    """An output: allocated here when None, else checked to have exactly the
    element count of `shape` (any contiguous layout of that many elements)."""
    if t is None:
        return _empty(shape, dtype, like) if stream is None else _new_on(stream, shape, dtype, like)
    n = 1
    for d in shape:
        n *= d
    return _need(t, name, dtype, numel=n)


def _check(fn, status):
    if status != 0:
        raise QloraError(fn, status)


def _empty(shape, dtype, like):
    """torch.empty on like's device; with the strides given it takes 1.3 us in place of 1.7."""
    if len(shape) == 2:
        strides = (shape[1], 1)
    elif len(shape) == 1:
        strides = (1,)
    else:
        strides = (shape[1] * shape[2], shape[2], 1)
    return torch.empty_strided(shape, strides, dtype=dtype, device=like.device)


def _empty_on(stream, shape, dtype, like):
    """_empty for a call on `stream`: from that stream's own memory where it is not the current one.
    What the current stream may still be using is not handed to it, nor the reverse."""
    if not like.is_cuda or stream.cuda_stream == _stream():
        return _empty(shape, dtype, like)
    if not isinstance(stream, torch.cuda.Stream):             # anything that holds a stream's handle
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=like.device)
    with torch.cuda.stream(stream):
        return _empty(shape, dtype, like)


def _new_on(stream, shape, dtype, like):
    """An output so allocated; the current stream, which reads it next, has it until it lets go of it."""
    t = _empty_on(stream, shape, dtype, like)
    if t.is_cuda:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _wdtype(W):
    if not isinstance(W, torch.Tensor) or W.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("W must be a float32 or bfloat16 torch.Tensor")
    return QL_BF16 if W.dtype == torch.bfloat16 else QL_F32


def nf4_quantize(W, codes=None, absmax=None, stream=None):
    """Packed NF4 codes [rows, cols/2] (uint8) and fp32 absmax [rows*cols/64] of W [rows, cols]."""
    dt = _wdtype(W)
    _need(W, "W", W.dtype, ndim=2)
    rows, cols = W.shape
    codes = _out(codes, "codes", torch.uint8, (rows, cols // 2), W, stream)
    absmax = _out(absmax, "absmax", torch.float32, (rows * cols // 64,), W, stream)
    _check("nf4_quantize", lib().nf4_quantize(_ptr(W), dt, rows, cols, _ptr(codes), _ptr(absmax), _stream(stream)))
    return codes, absmax


def nf4_quantize_dq(W, codes=None, c2=None, c1=None, absmax=None, stream=None):
    """Codes, c2 and c1 of W [rows, cols] in one pass (absmax written too when given a buffer or True)."""
    dt = _wdtype(W)
    _need(W, "W", W.dtype, ndim=2)
    rows, cols = W.shape
    nb = rows * cols // 64
    codes = _out(codes, "codes", torch.uint8, (rows, cols // 2), W, stream)
    c2 = _out(c2, "c2", torch.uint8, (nb,), W, stream)
    c1 = _out(c1, "c1", torch.float32, ((nb + 255) // 256,), W, stream)
    if absmax is True:
        absmax = _opt_out(True, "absmax", torch.float32, (nb,), W, stream)
    elif absmax is not None:
        _out(absmax, "absmax", torch.float32, (nb,), W, stream)
    _check("nf4_quantize_dq", lib().nf4_quantize_dq(_ptr(W), dt, rows, cols, _ptr(codes), _ptr(absmax), _ptr(c2),
                                                    _ptr(c1), _stream(stream)))
    return codes, c2, c1, absmax


def nf4_double_quant(absmax, c2=None, c1=None, stream=None):
    """E4M3FN codes c2 [n_blocks] (uint8) and fp32 group scales c1 [ceil(n_blocks/256)]."""
    _need(absmax, "absmax", torch.float32)
    nb = absmax.numel()
    c2 = _out(c2, "c2", torch.uint8, (nb,), absmax, stream)
    c1 = _out(c1, "c1", torch.float32, ((nb + 255) // 256,), absmax, stream)
    _check("nf4_double_quant", lib().nf4_double_quant(_ptr(absmax), nb, _ptr(c2), _ptr(c1), _stream(stream)))
    return c2, c1


def nf4_dequantize(codes, c2, c1, rows, cols, out=None, stream=None):
    """Bit-exact bf16 doubleDequant(c1, c2, W_NF4) [rows, cols]."""
    _packed(codes, c2, c1, rows, cols)
    out = _out(out, "out", torch.bfloat16, (rows, cols), codes, stream)
    _check("nf4_dequantize", lib().nf4_dequantize(_ptr(codes), _ptr(c2), _ptr(c1), rows, cols, _ptr(out),
                                                  _stream(stream)))
    return out


def _codebook(name):
    if name not in CODEBOOKS:
        raise ValueError(f"unknown code book {name!r} (one of {sorted(CODEBOOKS)})")
    return CODEBOOKS[name]


def _scale_code(name):
    if name not in SCALE_CODES:
        raise ValueError(f"unknown scale code {name!r} (one of {sorted(SCALE_CODES)})")
    return SCALE_CODES[name]


def q4_quantize(W, codebook="nf4", codes=None, absmax=None, stream=None):
    """Packed 4-bit codes [rows, cols/2] and fp32 absmax [rows*cols/64] with the given code book."""
    dt = _wdtype(W)
    _need(W, "W", W.dtype, ndim=2)
    rows, cols = W.shape
    codes = _out(codes, "codes", torch.uint8, (rows, cols // 2), W, stream)
    absmax = _out(absmax, "absmax", torch.float32, (rows * cols // 64,), W, stream)
    _check("q4_quantize", lib().q4_quantize(_ptr(W), dt, rows, cols, _codebook(codebook), _ptr(codes), _ptr(absmax),
                                            _stream(stream)))
    return codes, absmax


def q4_double_quant(absmax, scale_code="groupmax", stream=None):
    """(c2 [n_blocks] uint8, c1 [groups] fp32, mu [groups] fp32 or None) for a scale code."""
    _need(absmax, "absmax", torch.float32)
    sc = _scale_code(scale_code)
    if sc == SCALE_CODES["absmax"]:
        raise ValueError("absmax scales need no second level")
    nb = absmax.numel()
    ng = (nb + 255) // 256
    c2 = _out(None, "c2", torch.uint8, (nb,), absmax, stream)
    c1 = _out(None, "c1", torch.float32, (ng,), absmax, stream)
    mu = _opt_out(scale_code == "mean", "mu", torch.float32, (ng,), absmax, stream)
    _check("q4_double_quant", lib().q4_double_quant(_ptr(absmax), nb, sc, _ptr(c2), _ptr(c1),
                                                    _ptr(mu) if mu is not None else None, _stream(stream)))
    return c2, c1, mu


def q4_dequantize(codes, rows, cols, codebook="nf4", scale_code="groupmax", absmax=None, c2=None, c1=None, mu=None,
                  out=None, stream=None):
    """bf16 W' [rows, cols] from codes and the block scales of `scale_code`."""
    if rows <= 0 or cols <= 0 or cols % 64:
        raise ValueError(f"weight shape [{rows}, {cols}]: sizes must be > 0 and cols a multiple of 64")
    nb = rows * cols // 64
    ng = (nb + 255) // 256
    _need(codes, "codes", torch.uint8, numel=rows * cols // 2)
    for t, n, d, cnt in ((absmax, "absmax", torch.float32, nb), (c2, "c2", torch.uint8, nb),
                         (c1, "c1", torch.float32, ng), (mu, "mu", torch.float32, ng)):
        if t is not None:
            _need(t, n, d, numel=cnt)
    out = _out(out, "out", torch.bfloat16, (rows, cols), codes, stream)
    p = lambda t: _ptr(t) if t is not None else None
    _check("q4_dequantize", lib().q4_dequantize(_ptr(codes), rows, cols, _codebook(codebook), _scale_code(scale_code),
                                                p(absmax), p(c2), p(c1), p(mu), _ptr(out), _stream(stream)))
    return out


def q4_levels(codebook="nf4"):
    """The 16 fp32 levels of a code book compiled into the library (host call)."""
    buf = (ctypes.c_float * 16)()
    _check("q4_levels", lib().q4_levels(_codebook(codebook), ctypes.cast(buf, ctypes.c_void_p)))
    return list(buf)


def _rank(L1, K):
    """Rank r of the adapter from L1 [K, r]."""
    _need(L1, "L1", torch.bfloat16, ndim=2)
    if L1.shape[0] != K:
        raise ValueError(f"L1 must have {K} rows, got {tuple(L1.shape)}")
    return L1.shape[1]


def qlora_merge(codes, c2, c1, N, K, L1, L2, lora_scale=1.0, out=None, stream=None):
    """Merged bf16 weight W' + lora_scale (L1 L2)^T [N, K], rounded once."""
    _packed(codes, c2, c1, N, K)
    r = _rank(L1, K)
    _need(L2, "L2", torch.bfloat16, shape=(r, N))
    out = _out(out, "out", torch.bfloat16, (N, K), codes, stream)
    _check("qlora_merge", lib().qlora_merge(_ptr(codes), _ptr(c2), _ptr(c1), N, K, _ptr(L1), _ptr(L2), r,
                                            float(lora_scale), _ptr(out), _stream(stream)))
    return out


def qlora_linear_fwd_workspace(M, K, N, r):
    return int(lib().qlora_linear_fwd_workspace(M, K, N, r))


def qlora_linear_bwd_workspace(M, K, N, r):
    return int(lib().qlora_linear_bwd_workspace(M, K, N, r))


def _workspace(nbytes, like, workspace, stream):
    """The call's scratch."""
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8)
        if workspace.numel() < nbytes:
            raise ValueError(f"workspace must hold at least {nbytes} bytes, got {workspace.numel()}")
        return workspace
    shape = (max(nbytes, 16),)
    return _empty(shape, torch.uint8, like) if stream is None else _empty_on(stream, shape, torch.uint8, like)


def _opt_out(t, name, dtype, shape, like, stream):
    """Optional output: True -> allocated here, None/False -> absent, else checked."""
    if t is True:
        return _empty(shape, dtype, like) if stream is None else _new_on(stream, shape, dtype, like)
    if t is None or t is False:
        return None
    return _out(t, name, dtype, shape, like, stream)


def qlora_linear_fwd(X, codes, c2, c1, N, L1, L2, lora_scale=1.0, Y=None, T_out=None, workspace=None,
                     stream=None):
    """Y = bf16(X W'^T + s T L2), T = bf16(X L1).  Returns (Y, T_out or None).

    T_out: None (not returned), True (allocated here) or a bf16 [M, r] tensor."""
    _need(X, "X", torch.bfloat16, ndim=2)
    M, K = X.shape
    _packed(codes, c2, c1, N, K)
    r = _rank(L1, K)
    _need(L2, "L2", torch.bfloat16, shape=(r, N))
    Y = _out(Y, "Y", torch.bfloat16, (M, N), X, stream)
    T_out = _opt_out(T_out, "T_out", torch.bfloat16, (M, r), X, stream)
    ws = _workspace(qlora_linear_fwd_workspace(M, K, N, r), X, workspace, stream)
    _check("qlora_linear_fwd", lib().qlora_linear_fwd(
        _ptr(X), M, K, N, _ptr(codes), _ptr(c2), _ptr(c1), _ptr(L1), _ptr(L2), r, float(lora_scale),
        _ptr(Y), _ptr(T_out), _ptr(ws), ws.numel(), _stream(stream)))
    return Y, T_out


NOALLOC_SCRATCH_BYTES = 16777216      # QL_NOALLOC_SCRATCH_BYTES of include/qlora.h


def qlora_linear_fwd_noalloc(X, codes, c2, c1, N, L1, L2, lora_scale=1.0, Y=None, T_out=None, stream=None):
    """qlora_linear_fwd with its scratch in the library's per-GPU static array
    (for callers that cannot allocate; calls that overlap on one GPU race).
    Returns (Y, T_out or None); Y and T_out must be supplied to allocate nothing."""
    _need(X, "X", torch.bfloat16, ndim=2)
    M, K = X.shape
    _packed(codes, c2, c1, N, K)
    r = _rank(L1, K)
    _need(L2, "L2", torch.bfloat16, shape=(r, N))
    Y = _out(Y, "Y", torch.bfloat16, (M, N), X, stream)
    T_out = _opt_out(T_out, "T_out", torch.bfloat16, (M, r), X, stream)
    _check("qlora_linear_fwd_noalloc", lib().qlora_linear_fwd_noalloc(
        _ptr(X), M, K, N, _ptr(codes), _ptr(c2), _ptr(c1), _ptr(L1), _ptr(L2), r, float(lora_scale),
        _ptr(Y), _ptr(T_out), _stream(stream)))
    return Y, T_out


def qlora_linear_bwd(X, dY, codes, c2, c1, L1, L2, lora_scale=1.0, T=None, dX=True, dL1=None, dL2=None,
                     workspace=None, stream=None):
    """(dX or None, dL1 fp32 [K, r], dL2 fp32 [r, N]); the frozen base gets no gradient.

    dX: True (allocated here), False/None (skipped) or a bf16 [M, K] tensor."""
    _need(X, "X", torch.bfloat16, ndim=2)
    M, K = X.shape
    _need(dY, "dY", torch.bfloat16, ndim=2)
    if dY.shape[0] != M:
        raise ValueError(f"dY must have {M} rows, got {tuple(dY.shape)}")
    N = dY.shape[1]
    _packed(codes, c2, c1, N, K)
    r = _rank(L1, K)
    _need(L2, "L2", torch.bfloat16, shape=(r, N))
    if T is not None:
        _need(T, "T", torch.bfloat16, numel=M * r)
    dX = _opt_out(dX, "dX", torch.bfloat16, (M, K), X, stream)
    dL1 = _out(dL1, "dL1", torch.float32, (K, r), X, stream)
    dL2 = _out(dL2, "dL2", torch.float32, (r, N), X, stream)
    ws = _workspace(qlora_linear_bwd_workspace(M, K, N, r), X, workspace, stream)
    _check("qlora_linear_bwd", lib().qlora_linear_bwd(
        _ptr(X), _ptr(dY), M, K, N, _ptr(codes), _ptr(c2), _ptr(c1), _ptr(L1), _ptr(L2), r, float(lora_scale),
        _ptr(T), _ptr(dX), _ptr(dL1), _ptr(dL2), _ptr(ws), ws.numel(), _stream(stream)))
    return dX, dL1, dL2


def _group_adapters(L1, L2, G, K, N):
    _need(L1, "L1", torch.bfloat16, ndim=3)
    if L1.shape[0] != G or L1.shape[1] != K:
        raise ValueError(f"L1 must have shape ({G}, {K}, r), got {tuple(L1.shape)}")
    r = L1.shape[2]
    _need(L2, "L2", torch.bfloat16, shape=(G, r, N))
    return r


def qlora_group_fwd(X, codes, c2, c1, N, G, L1, L2, lora_scale=1.0, Y=None, T_out=None, workspace=None,
                    stream=None):
    """G stacked linears sharing X (W [G N, K] quantized as one; L1 [G, K, r], L2 [G, r, N]):
    Y [M, G N] = [Y_0 | ... | Y_{G-1}].  Returns (Y, T_out [G, M, r] or None)."""
    _need(X, "X", torch.bfloat16, ndim=2)
    M, K = X.shape
    _packed(codes, c2, c1, G * N, K)
    r = _group_adapters(L1, L2, G, K, N)
    Y = _out(Y, "Y", torch.bfloat16, (M, G * N), X, stream)
    T_out = _opt_out(T_out, "T_out", torch.bfloat16, (G, M, r), X, stream)
    ws = _workspace(int(lib().qlora_group_fwd_workspace(M, K, N, G, r)), X, workspace, stream)
    _check("qlora_group_fwd", lib().qlora_group_fwd(
        _ptr(X), M, K, N, G, _ptr(codes), _ptr(c2), _ptr(c1), _ptr(L1), _ptr(L2), r, float(lora_scale),
        _ptr(Y), _ptr(T_out), _ptr(ws), ws.numel(), _stream(stream)))
    return Y, T_out


def qlora_group_bwd(X, dY, codes, c2, c1, G, L1, L2, lora_scale=1.0, T=None, dX=True, dL1=None, dL2=None,
                    workspace=None, stream=None):
    """(dX or None, dL1 [G, K, r], dL2 [G, r, N]) of G stacked linears; dX sums the segments, rounded once."""
    _need(X, "X", torch.bfloat16, ndim=2)
    M, K = X.shape
    _need(dY, "dY", torch.bfloat16, ndim=2)
    if dY.shape[0] != M or dY.shape[1] % G:
        raise ValueError(f"dY must have {M} rows and a multiple of G={G} columns, got {tuple(dY.shape)}")
    N = dY.shape[1] // G
    _packed(codes, c2, c1, G * N, K)
    r = _group_adapters(L1, L2, G, K, N)
    if T is not None:
        _need(T, "T", torch.bfloat16, numel=G * M * r)
    dX = _opt_out(dX, "dX", torch.bfloat16, (M, K), X, stream)
    dL1 = _out(dL1, "dL1", torch.float32, (G, K, r), X, stream)
    dL2 = _out(dL2, "dL2", torch.float32, (G, r, N), X, stream)
    ws = _workspace(int(lib().qlora_group_bwd_workspace(M, K, N, G, r)), X, workspace, stream)
    _check("qlora_group_bwd", lib().qlora_group_bwd(
        _ptr(X), _ptr(dY), M, K, N, G, _ptr(codes), _ptr(c2), _ptr(c1), _ptr(L1), _ptr(L2), r, float(lora_scale),
        _ptr(T), _ptr(dX), _ptr(dL1), _ptr(dL2), _ptr(ws), ws.numel(), _stream(stream)))
    return dX, dL1, dL2


def qlora_adamw_step(param, exp_avg, exp_avg_sq, grad, step, lr, beta1=0.9, beta2=0.999, eps=1e-8,
                     weight_decay=0.0, param_bf16=None, stream=None):
    """One AdamW step over flat fp32 tensors (in place); param_bf16 (optional) gets bf16(param)."""
    _need(param, "param", torch.float32)
    n = param.numel()
    for t, name in ((exp_avg, "exp_avg"), (exp_avg_sq, "exp_avg_sq"), (grad, "grad")):
        _need(t, name, torch.float32, numel=n)
    if param_bf16 is not None:
        _need(param_bf16, "param_bf16", torch.bfloat16, numel=n)
    _check("qlora_adamw_step", lib().qlora_adamw_step(
        _ptr(param), _ptr(exp_avg), _ptr(exp_avg_sq), _ptr(grad), _ptr(param_bf16), n, float(lr), float(beta1),
        float(beta2), float(eps), float(weight_decay), int(step), _stream(stream)))


def qlora_nf4_levels():
    """The 16 fp32 NF4 levels compiled into the library (host call, no GPU)."""
    buf = (ctypes.c_float * 16)()
    _check("qlora_nf4_levels", lib().qlora_nf4_levels(ctypes.cast(buf, ctypes.c_void_p)))
    return [float(v) for v in buf]


def ql_status_string(status):
    return lib().ql_status_string(int(status)).decode()


# --- stage entry points -------------------------------------------------------

def qlora_lora_down(X, L1, T=None, workspace=None, stream=None):
    """T = bf16(X L1) [M, r]."""
    _need(X, "X", torch.bfloat16, ndim=2)
    M, K = X.shape
    r = _rank(L1, K)
    T = _out(T, "T", torch.bfloat16, (M, r), X, stream)
    ws = _workspace(int(lib().qlora_lora_down_workspace(M, K, r)), X, workspace, stream)
    _check("qlora_lora_down", lib().qlora_lora_down(_ptr(X), M, K, _ptr(L1), r, _ptr(T), _ptr(ws), ws.numel(),
                                                    _stream(stream)))
    return T


def qlora_linear_fwd_t(X, codes, c2, c1, N, T, L2, lora_scale=1.0, Y=None, stream=None):
    """Y = bf16(X W'^T + s T L2) given T (one kernel)."""
    _need(X, "X", torch.bfloat16, ndim=2)
    M, K = X.shape
    _packed(codes, c2, c1, N, K)
    _need(T, "T", torch.bfloat16, ndim=2)
    if T.shape[0] != M:
        raise ValueError(f"T must have {M} rows, got {tuple(T.shape)}")
    r = T.shape[1]
    _need(L2, "L2", torch.bfloat16, shape=(r, N))
    Y = _out(Y, "Y", torch.bfloat16, (M, N), X, stream)
    _check("qlora_linear_fwd_t", lib().qlora_linear_fwd_t(
        _ptr(X), M, K, N, _ptr(codes), _ptr(c2), _ptr(c1), _ptr(T), _ptr(L2), r, float(lora_scale), _ptr(Y),
        _stream(stream)))
    return Y


def qlora_lora_grad_in(dY, L2, lora_scale=1.0, G=None, workspace=None, stream=None):
    """G = bf16(s dY L2^T) [M, r]."""
    _need(dY, "dY", torch.bfloat16, ndim=2)
    M, N = dY.shape
    _need(L2, "L2", torch.bfloat16, ndim=2)
    if L2.shape[1] != N:
        raise ValueError(f"L2 must have {N} columns, got {tuple(L2.shape)}")
    r = L2.shape[0]
    G = _out(G, "G", torch.bfloat16, (M, r), dY, stream)
    ws = _workspace(int(lib().qlora_lora_grad_in_workspace(M, N, r)), dY, workspace, stream)
    _check("qlora_lora_grad_in", lib().qlora_lora_grad_in(_ptr(dY), M, N, _ptr(L2), r, float(lora_scale), _ptr(G),
                                                          _ptr(ws), ws.numel(), _stream(stream)))
    return G


def qlora_linear_dx(dY, codes, c2, c1, K, G, L1, dX=None, stream=None):
    """dX = bf16(dY W' + G L1^T) given G (one kernel)."""
    _need(dY, "dY", torch.bfloat16, ndim=2)
    M, N = dY.shape
    _packed(codes, c2, c1, N, K)
    _need(G, "G", torch.bfloat16, ndim=2)
    if G.shape[0] != M:
        raise ValueError(f"G must have {M} rows, got {tuple(G.shape)}")
    r = G.shape[1]
    _need(L1, "L1", torch.bfloat16, shape=(K, r))
    dX = _out(dX, "dX", torch.bfloat16, (M, K), dY, stream)
    _check("qlora_linear_dx", lib().qlora_linear_dx(
        _ptr(dY), M, K, N, _ptr(codes), _ptr(c2), _ptr(c1), _ptr(G), _ptr(L1), r, _ptr(dX), _stream(stream)))
    return dX


# --- LoRA over a bf16 base (same GEMM kernels, bf16 weight) --------------------

def _bf16_weight(W, N, K):
    return _need(W, "W", torch.bfloat16, shape=(N, K))


def lora_linear_fwd(X, W, L1, L2, lora_scale=1.0, Y=None, T_out=None, workspace=None, stream=None):
    """Y = bf16(X W^T + s T L2), T = bf16(X L1) with a bf16 base W [N, K]."""
    _need(X, "X", torch.bfloat16, ndim=2)
    M, K = X.shape
    _need(W, "W", torch.bfloat16, ndim=2)
    N = W.shape[0]
    _bf16_weight(W, N, K)
    r = _rank(L1, K)
    _need(L2, "L2", torch.bfloat16, shape=(r, N))
    Y = _out(Y, "Y", torch.bfloat16, (M, N), X, stream)
    T_out = _opt_out(T_out, "T_out", torch.bfloat16, (M, r), X, stream)
    ws = _workspace(qlora_linear_fwd_workspace(M, K, N, r), X, workspace, stream)
    _check("lora_linear_fwd", lib().lora_linear_fwd(
        _ptr(X), M, K, N, _ptr(W), _ptr(L1), _ptr(L2), r, float(lora_scale), _ptr(Y), _ptr(T_out), _ptr(ws),
        ws.numel(), _stream(stream)))
    return Y, T_out


def lora_linear_bwd(X, dY, W, L1, L2, lora_scale=1.0, T=None, dX=True, dL1=None, dL2=None, workspace=None,
                    stream=None):
    """(dX or None, dL1 fp32 [K, r], dL2 fp32 [r, N]) with a bf16 base W [N, K] (no gradient for W)."""
    _need(X, "X", torch.bfloat16, ndim=2)
    M, K = X.shape
    _need(dY, "dY", torch.bfloat16, ndim=2)
    if dY.shape[0] != M:
        raise ValueError(f"dY must have {M} rows, got {tuple(dY.shape)}")
    N = dY.shape[1]
    _bf16_weight(W, N, K)
    r = _rank(L1, K)
    _need(L2, "L2", torch.bfloat16, shape=(r, N))
    if T is not None:
        _need(T, "T", torch.bfloat16, numel=M * r)
    dX = _opt_out(dX, "dX", torch.bfloat16, (M, K), X, stream)
    dL1 = _out(dL1, "dL1", torch.float32, (K, r), X, stream)
    dL2 = _out(dL2, "dL2", torch.float32, (r, N), X, stream)
    ws = _workspace(qlora_linear_bwd_workspace(M, K, N, r), X, workspace, stream)
    _check("lora_linear_bwd", lib().lora_linear_bwd(
        _ptr(X), _ptr(dY), M, K, N, _ptr(W), _ptr(L1), _ptr(L2), r, float(lora_scale), _ptr(T), _ptr(dX),
        _ptr(dL1), _ptr(dL2), _ptr(ws), ws.numel(), _stream(stream)))
    return dX, dL1, dL2


def lora_linear_fwd_t(X, W, T, L2, lora_scale=1.0, Y=None, stream=None):
    """Y = bf16(X W^T + s T L2) given T, bf16 base W [N, K] (one kernel)."""
    _need(X, "X", torch.bfloat16, ndim=2)
    M, K = X.shape
    _need(W, "W", torch.bfloat16, ndim=2)
    N = W.shape[0]
    _bf16_weight(W, N, K)
    _need(T, "T", torch.bfloat16, ndim=2)
    if T.shape[0] != M:
        raise ValueError(f"T must have {M} rows, got {tuple(T.shape)}")
    r = T.shape[1]
    _need(L2, "L2", torch.bfloat16, shape=(r, N))
    Y = _out(Y, "Y", torch.bfloat16, (M, N), X, stream)
    _check("lora_linear_fwd_t", lib().lora_linear_fwd_t(
        _ptr(X), M, K, N, _ptr(W), _ptr(T), _ptr(L2), r, float(lora_scale), _ptr(Y), _stream(stream)))
    return Y


def lora_linear_dx(dY, W, G, L1, dX=None, stream=None):
    """dX = bf16(dY W + G L1^T) given G, bf16 base W [N, K] (one kernel)."""
    _need(dY, "dY", torch.bfloat16, ndim=2)
    M, N = dY.shape
    _need(W, "W", torch.bfloat16, ndim=2)
    K = W.shape[1]
    _bf16_weight(W, N, K)
    _need(G, "G", torch.bfloat16, ndim=2)
    if G.shape[0] != M:
        raise ValueError(f"G must have {M} rows, got {tuple(G.shape)}")
    r = G.shape[1]
    _need(L1, "L1", torch.bfloat16, shape=(K, r))
    dX = _out(dX, "dX", torch.bfloat16, (M, K), dY, stream)
    _check("lora_linear_dx", lib().lora_linear_dx(
        _ptr(dY), M, K, N, _ptr(W), _ptr(G), _ptr(L1), r, _ptr(dX), _stream(stream)))
    return dX


# --- dropout on the adapter's input --------------------------------------------

def _rows(X, name):
    """(dtype code, rows, cols, ld) of a 2-D fp32 or bf16 matrix whose rows are contiguous (and may be apart)."""
    if not isinstance(X, torch.Tensor) or X.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{name} must be a float32 or bfloat16 torch.Tensor")
    if X.dim() != 2:
        raise ValueError(f"{name} must have 2 dims, got {X.dim()}")
    rows, cols = X.shape
    ld = X.stride(0) if rows > 1 else cols
    if (cols > 1 and X.stride(1) != 1) or ld < cols:
        raise ValueError(f"{name} must have contiguous rows that do not overlap, got strides {X.stride()}")
    return QL_BF16 if X.dtype == torch.bfloat16 else QL_F32, rows, cols, ld


def _u64(v, name):
    if int(v) != v or not 0 <= v < 1 << 64:
        raise ValueError(f"{name} must be a whole number in [0, 2^64), got {v}")
    return int(v)


def _draw(p, seed, offset):
    return float(p), _u64(seed, "seed"), _u64(offset, "offset")


def lora_dropout(X, p, seed, offset=0, out=None, stream=None):
    """D o X for X [rows, cols] (fp32 or bf16, rows may be apart): kept elements over 1 - p, the others 0.
    The mask is a function of (p, seed, offset) and is never stored; the same call is the backward."""
    dt, rows, cols, ld = _rows(X, "X")
    out = _out(out, "out", X.dtype, (rows, cols), X, stream)
    _check("lora_dropout", lib().lora_dropout(_ptr(X), dt, rows, cols, ld, *_draw(p, seed, offset), _ptr(out),
                                              _stream(stream)))
    return out


def qlora_linear_fwd_dropout(X, codes, c2, c1, N, L1, L2, lora_scale=1.0, p=0.0, seed=0, offset=0, Y=None, T_out=None,
                             workspace=None, stream=None):
    """qlora_linear_fwd with T = bf16((D o X) L1).  Returns (Y, T_out or None)."""
    _need(X, "X", torch.bfloat16, ndim=2)
    M, K = X.shape
    _packed(codes, c2, c1, N, K)
    r = _rank(L1, K)
    _need(L2, "L2", torch.bfloat16, shape=(r, N))
    Y = _out(Y, "Y", torch.bfloat16, (M, N), X, stream)
    T_out = _opt_out(T_out, "T_out", torch.bfloat16, (M, r), X, stream)
    ws = _workspace(int(lib().qlora_linear_fwd_dropout_workspace(M, K, N, r)), X, workspace, stream)
    _check("qlora_linear_fwd_dropout", lib().qlora_linear_fwd_dropout(
        _ptr(X), M, K, N, _ptr(codes), _ptr(c2), _ptr(c1), _ptr(L1), _ptr(L2), r, float(lora_scale),
        *_draw(p, seed, offset), _ptr(Y), _ptr(T_out), _ptr(ws), ws.numel(), _stream(stream)))
    return Y, T_out


def qlora_linear_bwd_dropout(X, dY, codes, c2, c1, L1, L2, lora_scale=1.0, p=0.0, seed=0, offset=0, T=None, dX=True,
                             dL1=None, dL2=None, workspace=None, stream=None):
    """(dX or None, dL1 fp32 [K, r], dL2 fp32 [r, N]) of qlora_linear_fwd_dropout; dX as in qlora_linear_bwd."""
    _need(X, "X", torch.bfloat16, ndim=2)
    M, K = X.shape
    _need(dY, "dY", torch.bfloat16, ndim=2)
    if dY.shape[0] != M:
        raise ValueError(f"dY must have {M} rows, got {tuple(dY.shape)}")
    N = dY.shape[1]
    _packed(codes, c2, c1, N, K)
    r = _rank(L1, K)
    _need(L2, "L2", torch.bfloat16, shape=(r, N))
    if T is not None:
        _need(T, "T", torch.bfloat16, numel=M * r)
    dX = _opt_out(dX, "dX", torch.bfloat16, (M, K), X, stream)
    dL1 = _out(dL1, "dL1", torch.float32, (K, r), X, stream)
    dL2 = _out(dL2, "dL2", torch.float32, (r, N), X, stream)
    ws = _workspace(int(lib().qlora_linear_bwd_dropout_workspace(M, K, N, r)), X, workspace, stream)
    _check("qlora_linear_bwd_dropout", lib().qlora_linear_bwd_dropout(
        _ptr(X), _ptr(dY), M, K, N, _ptr(codes), _ptr(c2), _ptr(c1), _ptr(L1), _ptr(L2), r, float(lora_scale),
        *_draw(p, seed, offset), _ptr(T), _ptr(dX), _ptr(dL1), _ptr(dL2), _ptr(ws), ws.numel(), _stream(stream)))
    return dX, dL1, dL2


# --- microscaled 4-bit (MXFP4) --------------------------------------------------

def _mx4_shapes(rows, cols):
    if rows <= 0 or cols <= 0:
        raise ValueError(f"matrix [{rows}, {cols}]: sizes must be > 0")
    kp = -(-cols // 128) * 128
    return (kp // 32, rows, 16), (kp // 128, rows, 4)


def _mx4_packed(codes, scales, rows, cols, what=""):
    """The packed form of a [rows, cols] matrix: codes [Kp/32, rows, 16], scales [Kp/128, rows, 4]."""
    sc, ss = _mx4_shapes(rows, cols)
    if (isinstance(codes, torch.Tensor) and codes.shape == sc and codes.dtype == torch.uint8 and codes.is_contiguous()
            and isinstance(scales, torch.Tensor) and scales.shape == ss and scales.dtype == torch.uint8
            and scales.is_contiguous()):
        return
    _need(codes, what + "codes", torch.uint8, shape=sc)
    _need(scales, what + "scales", torch.uint8, shape=ss)


def mx4_quantize(X, transpose=False, codes=None, scales=None, stream=None):
    """(codes [Kp/32, R, 16], scales [Kp/128, R, 4]) of X (fp32 or bf16, rows may be apart) in blocks of 32 along
    its rows (R = rows), or with transpose down its columns (the packed matrix is X^T, R = cols)."""
    dt, rows, cols, ld = _rows(X, "X")
    sc, ss = _mx4_shapes(*((cols, rows) if transpose else (rows, cols)))
    codes = _out(codes, "codes", torch.uint8, sc, X, stream)
    scales = _out(scales, "scales", torch.uint8, ss, X, stream)
    _check("mx4_quantize", lib().mx4_quantize(_ptr(X), dt, rows, cols, ld, int(bool(transpose)), _ptr(codes),
                                              _ptr(scales), _stream(stream)))
    return codes, scales


def mx4_dequantize(codes, scales, rows, cols, out=None, stream=None):
    """bf16 values [rows, cols] of a packed matrix (exact)."""
    _mx4_packed(codes, scales, rows, cols)
    out = _out(out, "out", torch.bfloat16, (rows, cols), codes, stream)
    _check("mx4_dequantize", lib().mx4_dequantize(_ptr(codes), _ptr(scales), rows, cols, _ptr(out), _stream(stream)))
    return out


def mx4_matmul(a_codes, a_scales, M, b_codes, b_scales, N, K, out=None, stream=None):
    """bf16 [M, N] = A B^T of packed A [M, K] and B [N, K]."""
    _mx4_packed(a_codes, a_scales, M, K, "a_")
    _mx4_packed(b_codes, b_scales, N, K, "b_")
    out = _out(out, "out", torch.bfloat16, (M, N), a_codes, stream)
    _check("mx4_matmul", lib().mx4_matmul(_ptr(a_codes), _ptr(a_scales), M, _ptr(b_codes), _ptr(b_scales), N, K,
                                          _ptr(out), _stream(stream)))
    return out


def mx4_linear_fwd(X, codes, scales, N, L1, L2, lora_scale=1.0, p=0.0, seed=0, offset=0, Y=None, T_out=None,
                   workspace=None, stream=None):
    """Y = bf16(q(X) W'^T + s T L2), T = bf16((D o X) L1), with W [N, K] packed by mx4_quantize.
    Returns (Y, T_out or None); T_out as in qlora_linear_fwd."""
    _need(X, "X", torch.bfloat16, ndim=2)
    M, K = X.shape
    _mx4_packed(codes, scales, N, K)
    r = _rank(L1, K)
    _need(L2, "L2", torch.bfloat16, shape=(r, N))
    Y = _out(Y, "Y", torch.bfloat16, (M, N), X, stream)
    T_out = _opt_out(T_out, "T_out", torch.bfloat16, (M, r), X, stream)
    ws = _workspace(int(lib().mx4_linear_fwd_workspace(M, K, N, r)), X, workspace, stream)
    _check("mx4_linear_fwd", lib().mx4_linear_fwd(
        _ptr(X), M, K, N, _ptr(codes), _ptr(scales), _ptr(L1), _ptr(L2), r, float(lora_scale),
        *_draw(p, seed, offset), _ptr(Y), _ptr(T_out), _ptr(ws), ws.numel(), _stream(stream)))
    return Y, T_out


def mx4_linear_bwd(X, dY, codes_t, scales_t, L1, L2, lora_scale=1.0, p=0.0, seed=0, offset=0, T=None, dX=True,
                   dL1=None, dL2=None, workspace=None, stream=None):
    """(dX or None, dL1 fp32 [K, r], dL2 fp32 [r, N]); codes_t and scales_t pack W [N, K] with transpose=True.

    dX: True (allocated here), False/None (skipped) or a bf16 [M, K] tensor."""
    _need(X, "X", torch.bfloat16, ndim=2)
    M, K = X.shape
    _need(dY, "dY", torch.bfloat16, ndim=2)
    if dY.shape[0] != M:
        raise ValueError(f"dY must have {M} rows, got {tuple(dY.shape)}")
    N = dY.shape[1]
    _mx4_packed(codes_t, scales_t, K, N)
    r = _rank(L1, K)
    _need(L2, "L2", torch.bfloat16, shape=(r, N))
    if T is not None:
        _need(T, "T", torch.bfloat16, numel=M * r)
    dX = _opt_out(dX, "dX", torch.bfloat16, (M, K), X, stream)
    dL1 = _out(dL1, "dL1", torch.float32, (K, r), X, stream)
    dL2 = _out(dL2, "dL2", torch.float32, (r, N), X, stream)
    ws = _workspace(int(lib().mx4_linear_bwd_workspace(M, K, N, r)), X, workspace, stream)
    _check("mx4_linear_bwd", lib().mx4_linear_bwd(
        _ptr(X), _ptr(dY), M, K, N, _ptr(codes_t), _ptr(scales_t), _ptr(L1), _ptr(L2), r, float(lora_scale),
        *_draw(p, seed, offset), _ptr(T), _ptr(dX), _ptr(dL1), _ptr(dL2), _ptr(ws), ws.numel(), _stream(stream)))
    return dX, dL1, dL2


# --- microscaled 8-bit activations (MXFP8) ---------------------------------------

def _mx8_shapes(rows, cols):
    if rows <= 0 or cols <= 0:
        raise ValueError(f"matrix [{rows}, {cols}]: sizes must be > 0")
    kb = -(-cols // 32)
    return (rows, 32 * kb), (rows, kb)


def _mx8_packed(packed, name, rows, cols):
    """(codes [rows, Kp], scales [rows, Kp/32]) of a packed [rows, cols] matrix."""
    if not isinstance(packed, (tuple, list)) or len(packed) != 2:
        raise TypeError(f"{name} must be the pair (codes, scales) of a packed matrix")
    sc, ss = _mx8_shapes(rows, cols)
    codes, scales = packed
    if (isinstance(codes, torch.Tensor) and codes.shape == sc and codes.dtype == torch.uint8 and codes.is_contiguous()
            and isinstance(scales, torch.Tensor) and scales.shape == ss and scales.dtype == torch.uint8
            and scales.is_contiguous()):
        return packed
    _need(packed[0], f"{name} codes", torch.uint8, shape=sc)
    _need(packed[1], f"{name} scales", torch.uint8, shape=ss)
    return packed


def _mx8_out(packed, name, rows, cols, like, stream):
    """A packed output: None or False -> absent, True -> allocated here, else checked."""
    if packed is None or packed is False:
        return None
    if packed is not True:
        return tuple(_mx8_packed(packed, name, rows, cols))
    sc, ss = _mx8_shapes(rows, cols)
    return (_out(None, name, torch.uint8, sc, like, stream), _out(None, name, torch.uint8, ss, like, stream))


def mx8_quantize(X, codes=None, scales=None, stream=None):
    """(codes [rows, Kp], scales [rows, Kp/32]) of X (fp32 or bf16, rows may be apart) in blocks of 32 along its rows."""
    dt, rows, cols, ld = _rows(X, "X")
    sc, ss = _mx8_shapes(rows, cols)
    codes = _out(codes, "codes", torch.uint8, sc, X, stream)
    scales = _out(scales, "scales", torch.uint8, ss, X, stream)
    px, pc, ps = _ptrs(stream, X, codes, scales)
    _check("mx8_quantize", lib().mx8_quantize(px, dt, rows, cols, ld, pc, ps, _stream(stream)))
    return codes, scales


def mx8_dequantize(codes, scales, rows, cols, out=None, stream=None):
    """bf16 values [rows, cols] of a packed matrix (exact)."""
    _mx8_packed((codes, scales), "packed", rows, cols)
    out = _out(out, "out", torch.bfloat16, (rows, cols), codes, stream)
    pc, ps, po = _ptrs(stream, codes, scales, out)
    _check("mx8_dequantize", lib().mx8_dequantize(pc, ps, rows, cols, po, _stream(stream)))
    return out


# --- root-mean-square norm --------------------------------------------------------

_NORM_DTYPES = {torch.float32: QL_F32, torch.bfloat16: QL_BF16}


def _norm_args(X, weight, name):
    if (isinstance(X, torch.Tensor) and isinstance(weight, torch.Tensor) and X.dim() == 2 and X.dtype in _NORM_DTYPES
            and weight.dtype in _NORM_DTYPES and weight.shape == X.shape[1:] and X.is_contiguous()
            and weight.is_contiguous()):
        rows, cols = X.shape
        return rows, cols, _NORM_DTYPES[X.dtype], _NORM_DTYPES[weight.dtype]
    if not isinstance(X, torch.Tensor) or X.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{name} must be a float32 or bfloat16 torch.Tensor")
    _need(X, name, X.dtype, ndim=2)
    rows, cols = X.shape
    if not isinstance(weight, torch.Tensor) or weight.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("weight must be a float32 or bfloat16 torch.Tensor")
    _need(weight, "weight", weight.dtype, shape=(cols,))
    return rows, cols, _NORM_DTYPES[X.dtype], _NORM_DTYPES[weight.dtype]


def rms_norm_fwd(X, weight, eps, residual=None, Y=None, S=None, mx8=None, stream=None):
    """Y = bf16(S w / sqrt(mean(S^2) + eps)) [rows, cols] with S = X + residual in X's type.
    Returns (Y or None, S or None, packed or None).

    Y: None (allocated here), False (skipped; then mx8 is wanted) or a bf16 [rows, cols] tensor.
    S: the sum, None without a residual; given, it may be X or residual itself.
    mx8: None or False (not written), True (allocated here) or the pair (codes, scales): Y in 8 bits."""
    rows, cols, dt, wdt = _norm_args(X, weight, "X")
    Y = _out(Y, "Y", torch.bfloat16, (rows, cols), X, stream) if Y is not False else None
    if residual is not None:
        _need(residual, "residual", X.dtype, shape=(rows, cols))
        S = _out(S, "S", X.dtype, (rows, cols), X, stream)
    elif S is not None:
        raise ValueError("S is the sum with a residual: without one it is X")
    packed = _mx8_out(mx8, "mx8", rows, cols, X, stream)
    px, pr, pw, ps, py, pc, pk = _ptrs(stream, X, residual, weight, S, Y, *(packed or (None, None)))
    _check("rms_norm_fwd", lib().rms_norm_fwd(px, pr, dt, rows, cols, pw, wdt, float(eps), ps, py, pc, pk,
                                              _stream(stream)))
    return Y, S, packed


def rms_norm_bwd(dY, S, weight, eps, dS=None, dX=True, dW=True, workspace=None, stream=None):
    """(dX in S's type or None, dW fp32 [cols] or None) of rms_norm_fwd; dS is added to dX.

    dX, dW: True (allocated here), False/None (skipped) or a tensor; dX may be S or dS itself."""
    rows, cols, dt, wdt = _norm_args(S, weight, "S")
    _need(dY, "dY", torch.bfloat16, shape=(rows, cols))
    if dS is not None:
        _need(dS, "dS", S.dtype, shape=(rows, cols))
    dX = _opt_out(dX, "dX", S.dtype, (rows, cols), S, stream)
    dW = _opt_out(dW, "dW", torch.float32, (cols,), S, stream)
    ws = _workspace(int(lib().rms_norm_bwd_workspace(rows, cols)) if dW is not None else 0, S, workspace, stream)
    py, ps, pd, pw, px, pg, pk = _ptrs(stream, dY, S, dS, weight, dX, dW, ws)
    _check("rms_norm_bwd", lib().rms_norm_bwd(py, ps, pd, dt, rows, cols, pw, wdt, float(eps), px, pg, pk, ws.numel(),
                                              _stream(stream)))
    return dX, dW


# --- gated feed-forward product, backward passes from 8-bit activations ------------

def qlora_swiglu_fwd(X, codes, c2, c1, F, L1, L2, lora_scale=1.0, H=None, T_out=None, mx8=None, workspace=None,
                     stream=None):
    """H = bf16(silu(G) U) [M, F], [G | U] = X W'^T + s T L2 of a stacked gate|up weight W [2 F, K] (quantized as one;
    L1 [2, K, r], L2 [2, r, F]).  Returns (H, T_out [2, M, r] or None, packed or None).

    mx8: None or False (not written), True (allocated here) or the pair (codes, scales): G over U in 8 bits, 2 M rows."""
    _need(X, "X", torch.bfloat16, ndim=2)
    M, K = X.shape
    _packed(codes, c2, c1, 2 * F, K)
    r = _group_adapters(L1, L2, 2, K, F)
    H = _out(H, "H", torch.bfloat16, (M, F), X, stream)
    T_out = _opt_out(T_out, "T_out", torch.bfloat16, (2, M, r), X, stream)
    packed = _mx8_out(mx8, "mx8", 2 * M, F, X, stream)
    ws = _workspace(int(lib().qlora_swiglu_fwd_workspace(M, K, F, r)), X, workspace, stream)
    p = _ptrs(stream, X, codes, c2, c1, L1, L2, H, T_out, *(packed or (None, None)), ws)
    _check("qlora_swiglu_fwd", lib().qlora_swiglu_fwd(
        p[0], M, K, F, *p[1:6], r, float(lora_scale), *p[6:], ws.numel(), _stream(stream)))
    return H, T_out, packed


def qlora_swiglu_bwd(x8, dH, codes, c2, c1, L1, L2, gu8, T, lora_scale=1.0, dX=True, dL1=None, dL2=None,
                     workspace=None, stream=None):
    """(dX or None, dL1 [2, K, r], dL2 [2, r, F]) of qlora_swiglu_fwd from dH and what it left: x8, the packed
    (codes, scales) of X; gu8, those of G over U; T.  dX as in qlora_linear_bwd."""
    _need(dH, "dH", torch.bfloat16, ndim=2)
    M, F = dH.shape
    _need(L1, "L1", torch.bfloat16, ndim=3)
    K = L1.shape[1]
    _packed(codes, c2, c1, 2 * F, K)
    r = _group_adapters(L1, L2, 2, K, F)
    _mx8_packed(x8, "x8", M, K)
    _mx8_packed(gu8, "gu8", 2 * M, F)
    _need(T, "T", torch.bfloat16, numel=2 * M * r)
    dX = _opt_out(dX, "dX", torch.bfloat16, (M, K), dH, stream)
    dL1 = _out(dL1, "dL1", torch.float32, (2, K, r), dH, stream)
    dL2 = _out(dL2, "dL2", torch.float32, (2, r, F), dH, stream)
    ws = _workspace(int(lib().qlora_swiglu_bwd_workspace(M, K, F, r)), dH, workspace, stream)
    p = _ptrs(stream, *x8, dH, codes, c2, c1, L1, L2, *gu8, T, dX, dL1, dL2, ws)
    _check("qlora_swiglu_bwd", lib().qlora_swiglu_bwd(
        *p[:3], M, K, F, *p[3:8], r, float(lora_scale), *p[8:], ws.numel(), _stream(stream)))
    return dX, dL1, dL2


def qlora_linear_bwd_mx8(x8, dY, codes, c2, c1, L1, L2, T, lora_scale=1.0, dX=True, dL1=None, dL2=None,
                         workspace=None, stream=None):
    """qlora_linear_bwd with X as the packed pair (codes, scales) x8 and the forward's T [M, r]."""
    _need(dY, "dY", torch.bfloat16, ndim=2)
    M, N = dY.shape
    _need(L1, "L1", torch.bfloat16, ndim=2)
    K, r = L1.shape
    _packed(codes, c2, c1, N, K)
    _need(L2, "L2", torch.bfloat16, shape=(r, N))
    _mx8_packed(x8, "x8", M, K)
    _need(T, "T", torch.bfloat16, numel=M * r)
    dX = _opt_out(dX, "dX", torch.bfloat16, (M, K), dY, stream)
    dL1 = _out(dL1, "dL1", torch.float32, (K, r), dY, stream)
    dL2 = _out(dL2, "dL2", torch.float32, (r, N), dY, stream)
    ws = _workspace(int(lib().qlora_linear_bwd_mx8_workspace(M, K, N, r)), dY, workspace, stream)
    p = _ptrs(stream, *x8, dY, codes, c2, c1, L1, L2, T, dX, dL1, dL2, ws)
    _check("qlora_linear_bwd_mx8", lib().qlora_linear_bwd_mx8(
        *p[:3], M, K, N, *p[3:8], r, float(lora_scale), *p[8:], ws.numel(), _stream(stream)))
    return dX, dL1, dL2
