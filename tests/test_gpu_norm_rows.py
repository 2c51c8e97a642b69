"""The norm over many and over wide rows: several rows a work group in turn for every number of threads a row, and
matrices past 2^31 elements.  Tolerances as in test_gpu_norm."""
import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_norm import BF, EPS, F32, U, X8, f64, packed_between, qlib, rows_of, within

pytestmark = pytest.mark.gpu
DEV = "cuda"


def backward_bounds(s, k, g, b, dtype):
    """(dX, its bound, n): of test_gpu_norm.test_backward."""
    cols = s.shape[1]
    rx, _ = X8.norm_backward(g, s, k, EPS, b)
    inv = 1 / np.sqrt((s * s).mean(1, keepdims=True) + EPS)
    n, dd = s * inv, g * k
    tol = (cols / 2 + 8) * U * inv * (np.abs(dd) + np.abs(n) * np.abs((n * dd).mean(1, keepdims=True)))
    tol += inv * np.abs(n) * (1.5 * cols + 4) * U * np.abs(n * dd).mean(1, keepdims=True)
    return rx, tol + (2.0**-8 if dtype == BF else 2 * U) * np.abs(rx) + U * np.abs(b), n


# up to 512 work groups share the rows (of four rows each up to 1024 columns): two to four turns here
@pytest.mark.parametrize("rows,cols,dtype", [
    (4200, 515, BF), (4100, 1000, F32), (1100, 1025, BF), (1600, 2048, F32), (1300, 2050, BF), (1030, 4096, BF),
    (1100, 4104, F32), (1030, 8192, BF), (600, 8200, BF), (600, 8201, F32), (520, 16384, BF), (1030, 16390, BF),
    (520, 22016, F32), (520, 32767, BF)])
def test_backward_in_turns(rows, cols, dtype):
    q = qlib()
    S, dS, w = rows_of(rows * 41 + cols, rows, cols, dtype, BF)
    dY = (0.01 * torch.randn(rows, cols, generator=torch.Generator().manual_seed(cols))).to(BF).to(DEV)
    dX, dW = q.rms_norm_bwd(dY, S, w, EPS, dS=dS)
    again = q.rms_norm_bwd(dY, S, w, EPS, dS=dS)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dW), "the same call twice"
    g = f64(dY)
    rx, tol, n = backward_bounds(f64(S), f64(w), g, f64(dS), dtype)
    within(dX, rx, tol, "dX")
    within(dW, (n * g).sum(0), (rows + cols / 2 + 4) * U * np.abs(n * g).sum(0), "dW")
    # in place, the next row's loads in flight
    a, b = q.rms_norm_bwd(dY, s := S.clone(), w, EPS, dS=dS, dX=s)
    assert a is s and torch.equal(a, dX) and torch.equal(b, dW)


@pytest.mark.parametrize("rows,cols", [(66000, 32768), (2**21 + 3, 1030)])
def test_past_two_to_the_31_elements(rows, cols):
    q = qlib()
    assert rows * cols > 2**31
    g = torch.Generator(DEV).manual_seed(rows)
    n = lambda std: std * torch.randn(rows, cols, generator=g, device=DEV, dtype=BF)  # noqa: E731
    X, R, dY = n(1.0), n(0.3), n(0.01)
    w = (1 + 0.2 * torch.randn(cols, generator=g, device=DEV)).to(BF)
    Y, S, y8 = q.rms_norm_fwd(X, w, EPS, residual=R, mx8=True)
    dX, dW = q.rms_norm_bwd(dY, S, w, EPS, dS=R)
    at = 2**31 // cols
    for r in (slice(0, 5), slice(at - 2, at + 3), slice(rows - 5, rows)):
        assert torch.equal(S[r], (X[r].float() + R[r].float()).to(BF))
        s, k, gy = f64(S[r]), f64(w), f64(dY[r])
        y = X8.norm_forward(s, k, EPS)
        d = (cols / 2 + 3) * U * np.abs(y)
        within(Y[r], y, 2.0**-8 * np.abs(y) + d, "Y")
        packed_between([t[r] for t in y8], y, d, cols, "Y8")
        rx, tol, _ = backward_bounds(s, k, gy, f64(R[r]), BF)
        within(dX[r], rx, tol, "dX")
    ref, mag = torch.zeros(cols, dtype=torch.float64, device=DEV), torch.zeros(cols, dtype=torch.float64, device=DEV)
    step = max(1, 2**26 // cols)
    for i in range(0, rows, step):
        s = S[i:i + step].double()
        t = s / torch.sqrt(s.square().mean(1, keepdim=True) + EPS) * dY[i:i + step].double()
        ref += t.sum(0)
        mag += t.abs().sum(0)
    # a work group adds up every 512th row, and at most 64 additions join the work groups' shares
    within(dW, ref.cpu().numpy(), (rows / 512 + 64 + cols / 2 + 4) * U * mag.cpu().numpy(), "dW")
