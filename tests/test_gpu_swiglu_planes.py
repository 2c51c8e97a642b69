"""The bits that the gated product and its backward keep of T, dZ and B between their products.

The sums are made short or exact here, so that what is left of the tolerances is the rounding in question
(U = 2^-24, half a step of bf16 2^-8):
  dX of a gated product of up to 1024 columns takes dZ to 16 bits for any number of rows (test_gpu_swiglu's
  bounds with 2^-16 |dZ| |W| in place of 2^-8).
"""
import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_swiglu import Block, S, U, check_backward, f64, qlib
from test_gpu_norm import within

pytestmark = pytest.mark.gpu
DEV = "cuda"
X8 = O.mx8


@pytest.mark.parametrize("M,K,F,r", [
    # rows on either side of every path of dX at one F: few rows, large tiles, several rounds of them, slices
    (64, 64, 16, 8), (65, 64, 16, 8), (513, 128, 16, 8), (2000, 64, 3, 5), (800, 2048, 37, 12), (1600, 1024, 136, 64),
    (1000, 16640, 20, 8), (1, 128, 1024, 8), (2, 128, 1024, 8), (300, 704, 1024, 9), (1100, 1024, 1000, 8),
    (300, 4096, 1023, 64)])
def test_dz_keeps_its_bits_at_every_number_of_rows(M, K, F, r):
    q = qlib()
    b = Block(M * 1031 + K + F, M, K, F, r)
    x8 = q.mx8_quantize(b.X)
    _, T, gu8 = q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S, T_out=True, mx8=True)
    check_backward(q, b, x8, gu8, T, *q.qlora_swiglu_bwd(x8, b.d, *b.base, b.L1, b.L2, gu8, T, S), dz_bits=2.0**-16)


def sparse(b, n=6):
    """dH with n columns that are not zero: sums over the F columns have n terms, the zeros add nothing."""
    keep = torch.zeros(b.F, dtype=torch.bool)
    keep[torch.linspace(0, b.F - 1, n).long()] = True
    b.d *= keep.to(DEV)
    return n


def dx_bound(b, gu8, T, n, dz_bits):
    """dX in 64 bits, and how far it may be off before it is rounded, for n columns of dH that are not zero: dZ's own
    fp32 form as in check_backward, dz_bits of dZ, 2^-16 of B, and the sums' n + r terms a plane and a half."""
    M, F, r = b.M, b.F, b.r
    gu = X8.values(gu8[0].cpu().numpy(), gu8[1].cpu().numpy(), F)
    g, u, dh, l1, l2 = gu[:M], gu[M:], f64(b.d), f64(b.L1), f64(b.L2)
    dz = X8.swiglu_dz(dh, g, u)
    e = (np.abs(g) + 4) * 2.0**-23
    off = np.stack([e * np.abs(dh * u) * X8.sigmoid(g) * (1 + np.abs(g)) ** 2, e * np.abs(dz[1])]) + 4 * U * np.abs(dz)
    rx, tol, sums = 0.0, 0.0, (4 * n + 4 * r + 8) * U
    for h in range(2):
        w, B = b.W[h * F:(h + 1) * F], S * dz[h] @ l2[h].T
        ob = S * (off[h] @ np.abs(l2[h]).T) + (3 * n + 8) * U * S * (np.abs(dz[h]) @ np.abs(l2[h]).T)
        rx = rx + dz[h] @ w + B @ l1[h].T
        tol = tol + ((dz_bits + sums) * np.abs(dz[h]) + off[h]) @ np.abs(w)
        tol = tol + ((2.0**-16 + sums) * np.abs(B) + ob) @ np.abs(l1[h]).T
    return rx, tol


@pytest.mark.parametrize("M,K,F,r", [(2, 128, 1024, 8), (64, 256, 1024, 64), (300, 704, 1024, 9), (1100, 1024, 1000, 8),
                                     (600, 64, 513, 64), (4100, 2048, 1024, 8)])
def test_dz_keeps_its_bits_in_long_reductions(M, K, F, r):
    q = qlib()
    b = Block(M * 1033 + K + F, M, K, F, r)
    n = sparse(b)
    _, T, gu8 = q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S, T_out=True, mx8=True)
    dX = q.qlora_swiglu_bwd(q.mx8_quantize(b.X), b.d, *b.base, b.L1, b.L2, gu8, T, S)[0]
    rx, tol = dx_bound(b, gu8, T, n, 2.0**-16)
    within(dX, rx, 2.0**-8 * np.abs(rx) + tol, "dX")


def test_two_planes_of_many_rows():
    """Planes of dZ past 2^31 bytes together, which every size of the contract may have: first and last rows."""
    q = qlib()
    M, K, F, r = 520000, 64, 1024, 4
    g = torch.Generator(DEV).manual_seed(9)
    n = lambda *shape, std=1.0: (std * torch.randn(*shape, generator=g, device=DEV)).to(torch.bfloat16)  # noqa: E731
    W = n(2 * F, K, std=0.02)
    codes, absmax = q.nf4_quantize(W)
    base = (codes, *q.nf4_double_quant(absmax))
    X, L1, L2, d = n(M, K), n(2, K, r, std=0.1), n(2, r, F, std=0.05), n(M, F, std=0.01)
    x8 = q.mx8_quantize(X)
    _, T, gu8 = q.qlora_swiglu_fwd(X, *base, F, L1, L2, S, T_out=True, mx8=True)
    dX, dL1, _ = q.qlora_swiglu_bwd(x8, d, *base, L1, L2, gu8, T, S)
    assert torch.isfinite(dL1).all()
    w = f64(q.nf4_dequantize(*base, 2 * F, K))
    for rows in (slice(0, 200), slice(M - 200, M)):
        gu = [X8.values(gu8[0].view(2, M, -1)[h, rows].cpu().numpy(), gu8[1].view(2, M, -1)[h, rows].cpu().numpy(), F)
              for h in range(2)]
        dz = X8.swiglu_dz(f64(d[rows]), *gu)
        B = np.stack([S * dz[h] @ f64(L2[h]).T for h in range(2)])
        rx = sum(dz[h] @ w[h * F:(h + 1) * F] + B[h] @ f64(L1[h]).T for h in range(2))
        tol = 2.0**-8 * np.abs(rx)
        for h in range(2):
            # dZ's own fp32 form is off by less than 2^-18 of its terms here (test_gpu_swiglu), 2^-16 its planes
            tol += (2.0**-15 + 4 * F * U) * (np.abs(dz[h]) @ np.abs(w[h * F:(h + 1) * F]))
            tol += (2.0**-15 + 4 * F * U) * (S * np.abs(dz[h]) @ np.abs(f64(L2[h])).T @ np.abs(f64(L1[h])).T)
        within(dX[rows], rx, tol, "dX")
