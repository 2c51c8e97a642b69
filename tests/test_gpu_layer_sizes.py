"""The layers at sizes where an operand, or a few of them together, pass 2^31 or 2^32 bytes: against float64 on the
rows and columns that hold anything.  The other elements are zeros, which add exactly, so that a sum's bound counts
its non-zero terms alone:
  a sum of n exact products in fp32, in any order: (n + 4) 2^-24 sum |a b| (scaling and the slices' sum included);
  a bf16 result v: 2^-8 |v| on top (half an ulp); G enters dX after its own bf16 rounding.
"""
import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
X4 = O.mx4
U = 2.0 ** -24
BF = torch.bfloat16


def qlib():
    import bit_quantized_lora_blockwise_amd as q
    return q


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def dev(a, dtype=BF):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(dtype).to(DEV)


def within(got, ref, tol, name):
    g = f64(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert np.all(np.isfinite(g)), f"{name}: non-finite"
    print(f"{name}: max err/tol {np.max(np.abs(g - ref) / np.maximum(tol, 1e-300)):.3f}", flush=True)
    assert np.all(np.abs(g - ref) <= tol), f"{name}: worst {np.max(np.abs(g - ref) - tol):.3e} past the tolerance"


def mask_at(rows, cols, p, seed, offset):
    """D (0 or the scale) at rows x cols, both arrays of indices."""
    m, k = np.meshgrid(np.asarray(rows, np.uint64), np.asarray(cols, np.uint64), indexing="ij")
    w = X4.philox4x32([k // np.uint64(8), m, offset % 2**32, offset // 2**32], (seed % 2**32, seed // 2**32))
    w = np.stack([np.broadcast_to(x, m.shape) for x in w], -1)
    u = np.take_along_axis(w, ((k % np.uint64(8)) // np.uint64(2)).astype(np.int64)[..., None], -1)[..., 0]
    u = np.where(k % np.uint64(2), u >> np.uint64(16), u & np.uint64(0xFFFF))
    cut = X4.cut_of(p)
    return np.where(u >= cut, 65536 / (65536 - cut), 0.0)


def test_mask_at_is_the_oracles():
    rows, cols = np.array([0, 3, 6]), np.array([1, 8, 30])
    full = X4.dropped(np.ones((7, 31)), 0.3, 2**33 + 5, 2**34 + 7)
    assert np.array_equal(mask_at(rows, cols, 0.3, 2**33 + 5, 2**34 + 7), full[np.ix_(rows, cols)])


@pytest.mark.parametrize("layer", ["mx4", "nf4"])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_planes_of_g_past_2_32_bytes(layer, p):
    """12 million rows of rank 64: G's three planes are 4.6 GB together.  Rows all along the matrices hold values."""
    q = qlib()
    M, K, N, r, s, seed, off = 12_000_000, 64, 64, 64, 2.0, 2**40 + 9, 3
    rows = np.unique(np.linspace(0, M - 1, 200).astype(np.int64))
    n = len(rows)
    rng = np.random.default_rng(5)
    print(f"[{layer} M={M} p={p}]", flush=True)
    at = torch.from_numpy(rows).to(DEV)

    def spread(a):
        full = torch.zeros((M, a.shape[1]), dtype=BF, device=DEV)
        full[at] = dev(a)
        return full

    X, dY, T = (spread(rng.standard_normal((n, c))) for c in (K, N, r))
    L1, L2 = dev(rng.standard_normal((K, r)) * 0.1), dev(rng.standard_normal((r, N)) * 0.1)
    W = dev(rng.standard_normal((N, K)) * 0.05)
    kw = dict(p=p, seed=seed, offset=off)
    if layer == "mx4":
        dX, dL1, dL2 = q.mx4_linear_bwd(X, dY, *q.mx4_quantize(W, transpose=True), L1, L2, s, T=T, **kw)
        Wt, dyv = X4.rounded(f64(W).T), X4.rounded(f64(dY[at]))
    else:
        codes, absmax = q.nf4_quantize(W)
        base = (codes, *q.nf4_double_quant(absmax))
        dX, dL1, dL2 = q.qlora_linear_bwd_dropout(X, dY, *base, L1, L2, s, T=T, **kw)
        Wt, dyv = f64(q.nf4_dequantize(*base, N, K)).T, f64(dY[at])
    x, dy, t, l1, l2 = (f64(v) for v in (X[at], dY[at], T[at], L1, L2))
    D = mask_at(rows, np.arange(K), p, seed, off)
    G = s * dy @ l2.T
    errG = (N + 4) * U * s * (np.abs(dy) @ np.abs(l2).T)
    within(dL1, (x * D).T @ G, (n + 4) * U * (np.abs(x * D).T @ np.abs(G)) + np.abs(x * D).T @ errG, "dL1")
    within(dL2, s * t.T @ dy, (n + 4) * U * s * (np.abs(t).T @ np.abs(dy)), "dL2")
    ref = dyv @ Wt.T + D * (G @ l1.T)
    tol = 2.0**-8 * np.abs(ref) + (N + 4) * U * (np.abs(dyv) @ np.abs(Wt).T)
    tol += D * (((2.0**-8 + 70 * U) * np.abs(G) + errG) @ np.abs(l1).T)
    within(dX[at], ref, tol, "dX")
    assert int((dX != 0).any(1).sum()) <= n


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("K", [2**25, 2**25 + 2**22])
def test_l1_of_2_32_bytes(K, p):
    """17 rows of 2^25 columns and more over NF4: L1 is 4.3 GB, and past 2^31 elements.  dX and dL1 in blocks of columns
    all along the matrix."""
    q = qlib()
    M, N, r, s, seed, off = 17, 8, 64, 1.5, 7, 2**33 + 1
    rng = np.random.default_rng(6)
    print(f"[nf4 M={M} K={K} p={p}]", flush=True)
    X = torch.empty((M, K), dtype=BF, device=DEV).normal_()
    L1 = torch.empty((K, r), dtype=BF, device=DEV).normal_()
    W = torch.empty((N, K), dtype=BF, device=DEV).normal_(0, 0.05)
    dY, T, L2 = (dev(rng.standard_normal(shape)) for shape in ((M, N), (M, r), (r, N)))
    codes, absmax = q.nf4_quantize(W)
    base = (codes, *q.nf4_double_quant(absmax))
    Wq = q.nf4_dequantize(*base, N, K)
    dX, dL1, _ = q.qlora_linear_bwd_dropout(X, dY, *base, L1, L2, s, p=p, seed=seed, offset=off, T=T)
    dy, l2 = f64(dY), f64(L2)
    G = s * dy @ l2.T
    errG = (N + 4) * U * s * (np.abs(dy) @ np.abs(l2).T)
    for k in (0, 2**22 - 32, 2**24 + 64, 2**24 + 2**23, K - 128):
        c = slice(k, k + 128)
        D = mask_at(np.arange(M), np.arange(k, k + 128), p, seed, off)
        x, l1, w = f64(X[:, c]), f64(L1[c]), f64(Wq[:, c])
        ref = dy @ w + D * (G @ l1.T)
        tol = 2.0**-8 * np.abs(ref) + (N + 4) * U * (np.abs(dy) @ np.abs(w))
        tol += D * (((2.0**-8 + 70 * U) * np.abs(G) + errG) @ np.abs(l1).T)
        within(dX[:, c], ref, tol, f"dX {k}")
        within(dL1[c], (x * D).T @ G, (M + 4) * U * (np.abs(x * D).T @ np.abs(G)) + np.abs(x * D).T @ errG, f"dL1 {k}")


def test_bf16_base_dx_of_2_27_columns():
    """The widest dX over a bf16 base, 7 rows of nearly 2^27 columns: rows past the end of a tile of 256 stay unwritten."""
    q = qlib()
    M, K, N, r, s = 7, 2**27 - 64, 8, 8, 1.0
    rng = np.random.default_rng(7)
    W = torch.empty((N, K), dtype=BF, device=DEV).normal_(0, 0.05)
    L1 = torch.empty((K, r), dtype=BF, device=DEV).normal_()
    dY, G = dev(rng.standard_normal((M, N))), dev(rng.standard_normal((M, r)))
    dX = q.lora_linear_dx(dY, W, G, L1)
    dy, g = f64(dY), f64(G)
    for k in (0, 2**24, 2**26 - 64, 2**26 + 2**25, K - 128):
        c = slice(k, k + 128)
        l1, w = f64(L1[c]), f64(W[:, c])
        ref = dy @ w + g @ l1.T
        tol = 2.0**-8 * np.abs(ref) + (N + 4) * U * (np.abs(dy) @ np.abs(w)) + (r + 4) * U * (np.abs(g) @ np.abs(l1).T)
        within(dX[:, c], ref, tol, f"dX {k}")


@pytest.mark.parametrize("N", [2**25 + 5, 2**25 + 8])
@pytest.mark.parametrize("call", ["grad_in", "linear", "linear_dropout"])
def test_l2_past_2_32_bytes(call, N):
    """3 rows of more than 2^25 columns: L2 is 4.3 GB.  2000 columns of dY all along the matrix hold values; dL1 shows
    the layers' G."""
    q = qlib()
    M, K, r, s = 3, 64, 64, 2.0
    rng = np.random.default_rng(8)
    cols = np.unique(np.linspace(0, N - 1, 2000).astype(np.int64))
    n = len(cols)
    print(f"[{call} N={N}]", flush=True)
    at = torch.from_numpy(cols).to(DEV)
    L2 = torch.empty((r, N), dtype=BF, device=DEV).normal_()
    dY = torch.zeros((M, N), dtype=BF, device=DEV)
    dY[:, at] = dev(rng.standard_normal((M, n)))
    dy, l2 = f64(dY[:, at]), f64(L2[:, at])
    G = s * dy @ l2.T
    errG = (n + 4) * U * s * (np.abs(dy) @ np.abs(l2).T)
    if call == "grad_in":
        within(q.qlora_lora_grad_in(dY, L2, s), G, 2.0**-8 * np.abs(G) + errG, "G")
        return
    X, L1, T = (dev(rng.standard_normal(shape)) for shape in ((M, K), (K, r), (M, r)))
    W = torch.empty((N, K), dtype=BF, device=DEV).normal_(0, 0.05)
    codes, absmax = q.nf4_quantize(W)
    base = (codes, *q.nf4_double_quant(absmax))
    x = f64(X)
    if call == "linear":
        _, dL1, dL2 = q.qlora_linear_bwd(X, dY, *base, L1, L2, s, T=T, dX=False)
        errG = errG + 2.0**-8 * np.abs(G)                   # that layer's G is rounded to bf16
    else:
        _, dL1, dL2 = q.qlora_linear_bwd_dropout(X, dY, *base, L1, L2, s, T=T, dX=False, p=0.1, seed=1, offset=2)
        x = x * mask_at(np.arange(M), np.arange(K), 0.1, 1, 2)
    within(dL1, x.T @ G, (M + 4) * U * (np.abs(x).T @ np.abs(G)) + np.abs(x).T @ errG, "dL1")
    t = f64(T)
    within(dL2[:, at], s * t.T @ dy, (M + 4) * U * s * (np.abs(t).T @ np.abs(dy)), "dL2")


@pytest.mark.parametrize("K", [2**29 - 64, 2**29 + 128])
def test_one_row_of_2_29_columns(K):
    """One row over NF4, on both sides of the few-rows kernel's longest launch."""
    q = qlib()
    M, N, r, s, p, seed, off = 1, 3, 2, 1.5, 0.3, 5, 6
    rng = np.random.default_rng(9)
    X = torch.empty((M, K), dtype=BF, device=DEV).normal_()
    L1 = torch.empty((K, r), dtype=BF, device=DEV).normal_()
    W = torch.empty((N, K), dtype=BF, device=DEV).normal_(0, 0.05)
    dY, T, L2 = (dev(rng.standard_normal(shape)) for shape in ((M, N), (M, r), (r, N)))
    codes, absmax = q.nf4_quantize(W)
    base = (codes, *q.nf4_double_quant(absmax))
    Wq = q.nf4_dequantize(*base, N, K)
    dX, dL1, _ = q.qlora_linear_bwd_dropout(X, dY, *base, L1, L2, s, p=p, seed=seed, offset=off, T=T)
    dy, l2 = f64(dY), f64(L2)
    G = s * dy @ l2.T
    errG = (N + 4) * U * s * (np.abs(dy) @ np.abs(l2).T)
    for k in (0, 2**27 - 64, 2**28 + 64, K - 128):
        c = slice(k, k + 128)
        D = mask_at(np.arange(M), np.arange(k, k + 128), p, seed, off)
        x, l1, w = f64(X[:, c]), f64(L1[c]), f64(Wq[:, c])
        ref = dy @ w + D * (G @ l1.T)
        tol = 2.0**-8 * np.abs(ref) + (N + 4) * U * (np.abs(dy) @ np.abs(w))
        tol += D * (((2.0**-8 + 70 * U) * np.abs(G) + errG) @ np.abs(l1).T)
        within(dX[:, c], ref, tol, f"dX {k}")
        within(dL1[c], (x * D).T @ G, (M + 4) * U * (np.abs(x * D).T @ np.abs(G)) + np.abs(x * D).T @ errG, f"dL1 {k}")


@pytest.mark.parametrize("M", [3, 20])
@pytest.mark.parametrize("call", ["linear", "linear_t", "linear_dropout"])
def test_forward_of_l2_past_2_32_bytes(call, M):
    """Few rows to more than 2^25 columns: Y in blocks of columns all along the matrix."""
    q = qlib()
    K, N, r, s = 64, 2**25 + 8, 64, 0.5
    rng = np.random.default_rng(10)
    print(f"[{call} M={M} N={N}]", flush=True)
    L2 = torch.empty((r, N), dtype=BF, device=DEV).normal_()
    W = torch.empty((N, K), dtype=BF, device=DEV).normal_(0, 0.05)
    X, L1 = dev(rng.standard_normal((M, K))), dev(rng.standard_normal((K, r)) * 0.1)
    codes, absmax = q.nf4_quantize(W)
    base = (codes, *q.nf4_double_quant(absmax))
    Wq = q.nf4_dequantize(*base, N, K)
    x = f64(X)
    if call == "linear_dropout":
        Y, T = q.qlora_linear_fwd_dropout(X, *base, N, L1, L2, s, T_out=True, p=0.1, seed=1, offset=2)
    elif call == "linear":
        Y, T = q.qlora_linear_fwd(X, *base, N, L1, L2, s, T_out=True)
    else:
        T = q.qlora_lora_down(X, L1)
        Y = q.qlora_linear_fwd_t(X, *base, N, T, L2, s)
    D = mask_at(np.arange(M), np.arange(K), 0.1, 1, 2) if call == "linear_dropout" else np.ones((M, K))
    rT = (x * D) @ f64(L1)
    within(T, rT, 2.0**-8 * np.abs(rT) + (K + 4) * U * (np.abs(x * D) @ np.abs(f64(L1))), "T")
    t = f64(T)
    for n in (0, 2**22 + 16, 2**23, 2**24 - 64, 2**24 + 2**23, N - 128):
        c = slice(n, n + 128)
        w, l2 = f64(Wq[c]), f64(L2[:, c])
        ref = x @ w.T + s * (t @ l2)
        tol = 2.0**-8 * np.abs(ref) + (K + 4) * U * (np.abs(x) @ np.abs(w).T) + 70 * U * s * (np.abs(t) @ np.abs(l2))
        within(Y[:, c], ref, tol, f"Y {n}")
