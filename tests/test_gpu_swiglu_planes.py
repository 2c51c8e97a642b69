"""The bits that the gated product and its backward keep of T, dZ and B between their products.

The sums are made short or exact here, so that what is left of the tolerances is the rounding in question
(U = 2^-24, half a step of bf16 2^-8):
  T enters the gated product with 24 bits, with or without 8-bit copies.  X and L1 are whole numbers, so that T's
  sums of K <= 512 terms are whole numbers below 2^24 and exact in any order, and the base is zero: G and U are
  s T L2 of r terms in three planes, off by (3 r + 8) U S |T| |L2|.  Two planes lose 2^-18 of T and more, eight
  times that.  H = silu(G) U carries 1.1 of G's error, U's, and its own exponential and product, (|G| + 4) 2^-23.
  dX takes B with 16 bits: a zero base leaves B L1^T; one plane loses 2^-9.
  dX of a gated product of up to 1024 columns takes dZ to 16 bits for any number of rows (test_gpu_swiglu's
  bounds with 2^-16 |dZ| |W| in place of 2^-8).
A result in bf16 or 8 bits has to be the rounding of a value within those bounds.
"""
import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_swiglu import Block, S, U, check_backward, f64, qlib
from test_gpu_norm import packed_between, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
X8 = O.mx8


def rounds_between(got, ref, tol, name):
    """Every value is the bf16 rounding of one in [ref - tol, ref + tol]."""
    lo, hi = (torch.from_numpy(v).to(torch.bfloat16).float() for v in (ref - tol, ref + tol))
    v = got.float().cpu()
    out = (v < lo) | (v > hi)
    print(f"{name}: {int(out.sum())} of {out.numel()} outside", flush=True)
    assert not out.any(), f"{name}: {int(out.sum())} of {out.numel()}"


def over_zero(seed, M, K, F, r):
    """A gated block over a base of zeros."""
    q = qlib()
    b = Block(seed, M, K, F, r)
    codes, absmax = q.nf4_quantize(torch.zeros(2 * F, K, dtype=torch.bfloat16, device=DEV))
    b.base = (codes, *q.nf4_double_quant(absmax))
    b.W = f64(q.nf4_dequantize(*b.base, 2 * F, K))
    assert not b.W.any()
    return b


def whole_numbers(b, seed):
    """X and L1 whole, T = X L1 below 2^24 and exact; L2 so small that G and U are about one."""
    g = torch.Generator().manual_seed(seed)
    whole = lambda m, *shape: torch.randint(-m, m + 1, shape, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    b.X, b.L1 = whole(255, b.M, b.K), whole(127, 2, b.K, b.r)
    assert b.K * 255 * 127 < 1 << 24
    b.L2 = (torch.randn(2, b.r, b.F, generator=g) * 4e-6).to(torch.bfloat16).to(DEV)
    return np.stack([f64(b.X) @ f64(b.L1[h]) for h in range(2)])


@pytest.mark.parametrize("M,K,F,r", [
    # up to 16 rows (decoding without copies), few rows from T's slices and from its planes, half and whole large tiles
    (1, 512, 20000, 1), (16, 512, 4000, 3), (16, 512, 1000, 6), (32, 512, 16000, 1), (70, 512, 4000, 1),
    (2100, 512, 128, 1), (1300, 512, 1100, 3), (1300, 64, 3000, 17)])
def test_t_keeps_its_bits(M, K, F, r):
    q = qlib()
    b = over_zero(M * 1039 + K + F, M, K, F, r)
    t = whole_numbers(b, M + F)
    gu = [S * t[h] @ f64(b.L2[h]) for h in range(2)]
    d = [(3 * r + 8) * U * S * np.abs(t[h]) @ np.abs(f64(b.L2[h])) for h in range(2)]
    (g, u), (dg, du) = gu, d
    h = g * X8.sigmoid(g) * u
    dh = 1.1 * np.abs(u) * dg + np.abs(g * X8.sigmoid(g)) * du + 1.1 * dg * du + (np.abs(g) + 4) * 2.0**-23 * np.abs(h)
    H, T, gu8 = q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S, T_out=True, mx8=True)
    assert torch.equal(T.float().cpu(), torch.from_numpy(t).to(torch.bfloat16).float())
    packed_between(gu8, np.concatenate(gu), np.concatenate(d), F, "GU")
    rounds_between(H, h, dh, "H")
    H, T2, _ = q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S, T_out=True)
    assert torch.equal(T2, T)
    rounds_between(H, h, dh, "H alone")


@pytest.mark.parametrize("M,K,F,r", [
    # few rows with B in slices and in planes, slices of the reduction, large tiles; one and two planes of dZ
    (40, 128, 1100, 8), (40, 128, 100, 8), (64, 4096, 1030, 64), (300, 4096, 1100, 5), (4100, 2048, 1030, 8),
    (800, 2048, 37, 12), (1100, 1024, 1000, 8)])
def test_b_keeps_its_bits(M, K, F, r):
    q = qlib()
    b = over_zero(M * 1049 + K + F, M, K, F, r)
    n = sparse(b)
    _, T, gu8 = q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S, T_out=True, mx8=True)
    dX = q.qlora_swiglu_bwd(q.mx8_quantize(b.X), b.d, *b.base, b.L1, b.L2, gu8, T, S)[0]
    rounds_between(dX, *dx_bound(b, gu8, T, n, 0.0), "dX")


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


@pytest.mark.parametrize("M,K,F,r", [(40, 128, 100, 8), (800, 2048, 37, 12), (1000, 16640, 20, 8), (1100, 1024, 1000, 8),
                                     (600, 64, 33, 3)])
def test_two_planes_in_a_given_workspace_and_captured(M, K, F, r):
    """Few rows, large tiles, several rounds of them with the gradients beside, slices: from scratch memory full of
    NaN, and captured, then replayed between eager calls."""
    q = qlib()
    b = Block(M * 1051 + K + F, M, K, F, r)
    x8 = q.mx8_quantize(b.X)
    _, T, gu8 = q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S, T_out=True, mx8=True)
    d = b.d.clone()
    ws = torch.full((q.lib().qlora_swiglu_bwd_workspace(M, K, F, r),), 255, dtype=torch.uint8, device=DEV)

    def run(**kw):
        return q.qlora_swiglu_bwd(x8, d, *b.base, b.L1, b.L2, gu8, T, S, **kw)

    want = run()
    for u, v in zip(run(workspace=ws), want):
        assert torch.isfinite(v).all() and torch.equal(u, v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(workspace=ws)
    for k in range(3):
        d.copy_(b.d * (0.5 + k))
        graph.replay()
        eager = run()
        torch.cuda.synchronize()
        for u, v in zip(held, eager):
            assert torch.equal(u, v), k
