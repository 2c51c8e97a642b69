"""GPU parity of the norm and its backward against the oracle.

Tolerances, derived from the rounding points (U = 2^-24, a row of n columns):
  S is the fp32 sum rounded to X's type: equal;
  1 / rms: the fp32 sum of n squares is off by at most n U of itself (any order), half of which
  reaches the root, and is rounded once: (n / 2 + 1) U; Y takes two more roundings: by d = (n / 2 + 3) U
  of itself before it is rounded to bf16 (2^-8 of it);
  a value in 8 bits is what one of [y - d |y|, y + d |y|] is rounded to;
  dX: with n_ = S / rms, the mean of n_ d over n terms is off by (n + n / 2 + 4) U mean|n_ d|, the
  rest by a few U of each term: (n / 2 + 8) U (|inv d| + |inv n_ mean|);
  dw: M roundings of a sum, each term off by (n / 2 + 4) U.
"""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import assert_bitexact

pytestmark = pytest.mark.gpu
DEV = "cuda"
X8 = O.mx8
U = 2.0 ** -24
EPS = 1e-5


def qlib():
    import bit_quantized_lora_blockwise_amd as q
    return q


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rows_of(seed, rows, cols, dtype, wdtype):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(rows, cols, generator=g)
    X[:, ::17] *= 10
    if rows > 2:
        X[1] = 0                                             # a row of padding
        X[2] *= 1e-4                                         # one that eps matters to
    R = 0.3 * torch.randn(rows, cols, generator=g)
    if rows > 2:
        R[1] = 0
    w = 1 + 0.2 * torch.randn(cols, generator=g)
    return X.to(dtype).to(DEV), R.to(dtype).to(DEV), w.to(wdtype).to(DEV)


def within(got, ref, tol, name):
    g = f64(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert np.all(np.isfinite(g)), f"{name}: non-finite"
    over = np.abs(g - ref) - tol
    print(f"{name}: max err/tol {np.max(np.abs(g - ref) / np.maximum(tol, 1e-300)):.3f}", flush=True)
    assert np.all(over <= 0), f"{name}: {np.count_nonzero(over > 0)} of {over.size} past the tolerance, worst {over.max():.3e}"


def packed_between(packed, y, d, cols, name):
    """Every value is the rounding of one in [y - d, y + d], over a scale that one of these has."""
    codes, scales = (t.cpu().numpy() for t in packed)
    lo, hi = X8.exponents(np.maximum(np.abs(y) - d, 0)), X8.exponents(np.abs(y) + d)
    e = scales.astype(int) - 127
    assert ((e >= lo) & (e <= hi)).all(), f"{name}: scales"
    v = X8.values(codes, scales, cols)
    # a block at the border of two scales may pass the end of the smaller by d: nearest() holds it there
    below, above = X8.rounded(y - d, e), X8.rounded(y + d, e)
    assert ((v >= below) & (v <= above)).all(), f"{name}: {np.count_nonzero((v < below) | (v > above))} values"
    assert not codes[:, cols:].any(), f"{name}: padding"


BF, F32 = torch.bfloat16, torch.float32
CASES = [(1, 1, BF, BF), (1, 4096, BF, BF), (3, 7, F32, F32), (5, 512, BF, F32), (4, 513, BF, BF), (9, 1000, F32, BF),
         (2, 2048, BF, BF), (3, 2049, F32, F32), (6, 4099, BF, BF), (3, 8192, BF, BF), (2, 8200, F32, F32),
         (2, 16384, BF, BF), (1, 22016, BF, BF), (3, 32768, F32, F32), (333, 100, BF, BF), (700, 31, F32, F32)]


@pytest.mark.parametrize("rows,cols,dtype,wdtype", CASES)
@pytest.mark.parametrize("residual", [False, True])
def test_forward(rows, cols, dtype, wdtype, residual):
    q = qlib()
    X, R, w = rows_of(rows * 31 + cols, rows, cols, dtype, wdtype)
    Y, S, y8 = q.rms_norm_fwd(X, w, EPS, residual=R if residual else None, mx8=True)
    if residual:
        assert torch.equal(S, (X.float() + R.float()).to(dtype))
    else:
        assert S is None
        S = X
    y = X8.norm_forward(f64(S), f64(w), EPS)
    d = (cols / 2 + 3) * U * np.abs(y)
    within(Y, y, 2.0**-8 * np.abs(y) + d, "Y")
    packed_between(y8, y, d, cols, "Y8")
    # each output alone
    only, _, none = q.rms_norm_fwd(X, w, EPS, residual=R if residual else None)
    assert none is None and torch.equal(only, Y)
    none, _, alone = q.rms_norm_fwd(X, w, EPS, residual=R if residual else None, Y=False, mx8=True)
    assert none is None and torch.equal(alone[0], y8[0]) and torch.equal(alone[1], y8[1])


@pytest.mark.parametrize("rows,cols,dtype,wdtype", CASES)
@pytest.mark.parametrize("beside", [False, True])
def test_backward(rows, cols, dtype, wdtype, beside):
    q = qlib()
    S, dS, w = rows_of(rows * 37 + cols, rows, cols, dtype, wdtype)
    dY = (0.01 * torch.randn(rows, cols, generator=torch.Generator().manual_seed(cols))).to(BF).to(DEV)
    dX, dW = q.rms_norm_bwd(dY, S, w, EPS, dS=dS if beside else None)
    s, k, g, b = f64(S), f64(w), f64(dY), f64(dS) if beside else 0.0
    rx, rw = X8.norm_backward(g, s, k, EPS, b)
    inv = 1 / np.sqrt((s * s).mean(1, keepdims=True) + EPS)
    n, dd = s * inv, g * k
    tol = (cols / 2 + 8) * U * inv * (np.abs(dd) + np.abs(n) * np.abs((n * dd).mean(1, keepdims=True)))
    tol += inv * np.abs(n) * (1.5 * cols + 4) * U * np.abs(n * dd).mean(1, keepdims=True)
    tol += (2.0**-8 if dtype == BF else 2 * U) * np.abs(rx) + U * np.abs(b)
    within(dX, rx, tol, "dX")
    within(dW, rw, (rows + cols / 2 + 4) * U * np.abs(n * g).sum(0), "dW")
    alone, none = q.rms_norm_bwd(dY, S, w, EPS, dS=dS if beside else None, dW=False)
    assert none is None and torch.equal(alone, dX)
    none, alone = q.rms_norm_bwd(dY, S, w, EPS, dX=False)
    assert none is None and torch.equal(alone, dW)
    assert torch.equal(q.rms_norm_bwd(dY, S, w, EPS)[1], dW), "sums in a fixed order"


@pytest.mark.parametrize("cols", [100, 1001, 4096, 8193])
def test_in_place(cols):
    q = qlib()
    X, R, w = rows_of(cols, 37, cols, BF, BF)
    Y, S, _ = q.rms_norm_fwd(X, w, EPS, residual=R)
    for over in (0, 1):
        x, r = X.clone(), R.clone()
        y, s, _ = q.rms_norm_fwd(x, w, EPS, residual=r, S=(x, r)[over])
        assert s is (x, r)[over] and torch.equal(s, S) and torch.equal(y, Y)
    dY, dS = (0.01 * R).contiguous(), X.clone()
    dX, dW = q.rms_norm_bwd(dY, S, w, EPS, dS=dS)
    for over in (0, 1):
        s, d = S.clone(), dS.clone()
        a, b = q.rms_norm_bwd(dY, s, w, EPS, dS=d, dX=(s, d)[over])
        assert a is (s, d)[over] and torch.equal(a, dX) and torch.equal(b, dW)


def test_more_rows_than_shares():
    """Rows that several work groups take in turns, and few columns."""
    q = qlib()
    rows, cols = 5000, 40
    S, dS, w = rows_of(11, rows, cols, BF, BF)
    dY = (0.01 * torch.randn(rows, cols, generator=torch.Generator().manual_seed(5))).to(BF).to(DEV)
    dX, dW = q.rms_norm_bwd(dY, S, w, EPS, dS=dS)
    rx, rw = X8.norm_backward(f64(dY), f64(S), f64(w), EPS, f64(dS))
    s = f64(S)
    n = s / np.sqrt((s * s).mean(1, keepdims=True) + EPS)
    within(dW, rw, (rows + cols / 2 + 4) * U * np.abs(n * f64(dY)).sum(0), "dW")
    err = np.linalg.norm(f64(dX) - rx) / np.linalg.norm(rx)
    assert err <= 2.0**-8, err


def test_on_another_stream_and_captured():
    q = qlib()
    X, R, w = rows_of(9, 64, 1024, BF, BF)
    dY = (0.01 * R).contiguous()
    Y, S, y8 = q.rms_norm_fwd(X, w, EPS, residual=R, mx8=True)
    dX, dW = q.rms_norm_bwd(dY, S, w, EPS, dS=R)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    Y2, S2, p2 = q.rms_norm_fwd(X, w, EPS, residual=R, mx8=True, stream=st)
    dX2, dW2 = q.rms_norm_bwd(dY, S2, w, EPS, dS=R, stream=st)
    st.synchronize()
    for a, b in ((Y, Y2), (S, S2), (y8[0], p2[0]), (y8[1], p2[1]), (dX, dX2), (dW, dW2)):
        assert torch.equal(a, b)
    x, r = X.clone(), R.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, s, p = q.rms_norm_fwd(x, w, EPS, residual=r, mx8=True)
        a, b = q.rms_norm_bwd(dY, s, w, EPS, dS=r)
    for k in range(3):
        x.copy_(X * (k + 1))
        graph.replay()
        ey, es, ep = q.rms_norm_fwd(x, w, EPS, residual=r, mx8=True)
        ea, eb = q.rms_norm_bwd(dY, es, w, EPS, dS=r)
        torch.cuda.synchronize()
        for u, v in ((y, ey), (s, es), (p[0], ep[0]), (p[1], ep[1]), (a, ea), (b, eb)):
            assert torch.equal(u, v), k
