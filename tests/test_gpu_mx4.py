"""GPU parity of the microscaled 4-bit layer and of the adapter dropout against the
float64 oracle.

Tolerances, elementwise, derived from the rounding points:
  codes, scale bytes, dequantised values, dropout: equal;
  a sum of n exact products in fp32, in any order: n 2^-24 sum |a b|;
  a bf16 result v: 2^-8 |v| on top (half an ulp);
  T enters Y after its bf16 rounding, G enters dX after its: 2^-8 |T| |L2| s and
  2^-8 |G| |L1| on top; dL1 also carries G's own fp32 sums.
"""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import assert_bitexact, bits

pytestmark = pytest.mark.gpu
DEV = "cuda"
X4 = O.mx4
U = 2.0 ** -24


def qlib():
    import bit_quantized_lora_blockwise_amd as q
    return q


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def dev(a, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(dtype).to(DEV)


def within(got, ref, tol, name):
    g = f64(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    assert np.all(np.isfinite(g)), f"{name}: non-finite"
    over = np.abs(g - ref) - tol
    print(f"{name}: max err/tol {np.max(np.abs(g - ref) / np.maximum(tol, 1e-300)):.3f}", flush=True)
    assert np.all(over <= 0), f"{name}: {np.count_nonzero(over > 0)} of {over.size} past the tolerance, worst {over.max():.3e}"


def wild(rng, rows, cols):
    """Values whose blocks differ in size by many powers of two, with zeros of both signs, ties and single spikes."""
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-30, 30, (rows, 1)))
    x *= np.where(rng.random((rows, cols)) < 0.02, 1000.0, 1.0)
    x[rng.random((rows, cols)) < 0.1] = 0.0
    x[rng.random((rows, cols)) < 0.05] *= -0.0
    if rows > 2:
        x[1] = 0.0
        x[2] = np.resize([0.25, -0.75, 1.25, 1.75, 2.5, -3.5, 5.0, 4.0, 7.9], cols)
    return x.astype(np.float32)


SHAPES = [(1, 1), (1, 4096), (3, 31), (5, 32), (2, 33), (17, 127), (16, 128), (33, 129), (333, 1000), (64, 1096),
          (130, 8), (1000, 3)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantize(rows, cols, dtype, transpose):
    q = qlib()
    x = dev(wild(np.random.default_rng(rows * 1000 + cols), rows, cols), dtype)
    codes, scales = q.mx4_quantize(x, transpose=transpose)
    ref = f64(x).T if transpose else f64(x)
    rc, rs = X4.quantize(ref)
    pc, ps = X4.pack(rc, rs)
    assert_bitexact(codes.cpu().numpy(), pc, "codes")
    assert_bitexact(scales.cpu().numpy(), ps, "scales")
    v = q.mx4_dequantize(codes, scales, *ref.shape)
    assert_bitexact(f64(v), X4.values(rc, rs, ref.shape[1]), "values")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantize_rows_apart(dtype, transpose):
    """A slice of a wider matrix: aligned rows 16 bytes apart or not."""
    q = qlib()
    for width, cols in ((512, 200), (301, 77)):
        x = dev(wild(np.random.default_rng(width), 37, width), dtype)[:, :cols]
        assert not x.is_contiguous()
        a = q.mx4_quantize(x, transpose=transpose)
        b = q.mx4_quantize(x.contiguous(), transpose=transpose)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantize_special_values(dtype, transpose):
    """Infinities and NaN mark their block alone; the largest and the smallest finite values, subnormals among them."""
    q = qlib()
    x = np.ones((40, 160), np.float32)
    x[0, 3], x[1, 40], x[2, 159], x[35, 64] = np.inf, -np.inf, np.nan, np.nan
    top = float(torch.finfo(dtype).max)
    x[4, :32], x[5, 32:64] = top, -top
    for i, e in enumerate(range(-149, -110, 3)):
        x[6 + i] = 2.0 ** e * np.resize([1, 1.5, -0.5, 0.25], 160)
    x = dev(x, dtype)
    codes, scales = q.mx4_quantize(x, transpose=transpose)
    ref = f64(x).T if transpose else f64(x)
    rc, rs = X4.quantize(ref)
    pc, ps = X4.pack(rc, rs)
    assert_bitexact(codes.cpu().numpy(), pc, "codes")
    assert_bitexact(scales.cpu().numpy(), ps, "scales")
    g, r = f64(q.mx4_dequantize(codes, scales, *ref.shape)), X4.values(rc, rs, ref.shape[1])
    assert np.array_equal(np.isnan(g), np.isnan(r)) and np.array_equal(g[~np.isnan(g)], r[~np.isnan(r)])


def test_quantize_every_bf16():
    """Every finite bf16 once, 32 of neighbouring magnitude to a block."""
    q = qlib()
    u = np.concatenate([np.arange(0x7F80), 0x8000 + np.arange(0x7F80)]).astype(np.uint32) << 16
    x = u.view(np.float32).reshape(-1, 64)
    rc, rs = X4.quantize(x)
    pc, ps = X4.pack(rc, rs)
    codes, scales = q.mx4_quantize(dev(x))
    assert_bitexact(codes.cpu().numpy(), pc, "codes")
    assert_bitexact(scales.cpu().numpy(), ps, "scales")


def test_quantize_past_2_31_bytes():
    """A matrix, its packed form and its values past 2^31 bytes: rows at both ends against the oracle."""
    q = qlib()
    rows, cols = 16400, 131072
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV).normal_()
    for transpose in (False, True):
        codes, scales = q.mx4_quantize(x, transpose=transpose)
        v = q.mx4_dequantize(codes, scales, *((cols, rows) if transpose else (rows, cols)))
        for at in (0, 8191, rows - 33, rows - 1):
            if transpose:
                b = at // 32 * 32
                got, src = v[:, b:b + 32].t(), x[b:b + 32]
                ref = X4.rounded(f64(src).T).T
            else:
                got, src = v[at:at + 1], x[at:at + 1]
                ref = X4.rounded(f64(src))
            assert_bitexact(f64(got), ref, f"row {at} transpose {transpose}")
        del codes, scales, v


DROP_SHAPES = [(1, 1), (3, 777), (1, 4096), (64, 8), (37, 1000), (257, 513)]


@pytest.mark.parametrize("rows,cols", DROP_SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.999])
def test_dropout(rows, cols, dtype, p):
    q = qlib()
    seed, offset = 0x9E3779B97F4A7C15, 2**40 + 11
    x = dev(np.random.default_rng(rows + cols).standard_normal((rows, cols)), dtype)
    y = q.lora_dropout(x, p, seed, offset)
    keep = torch.from_numpy(X4.keep(rows, cols, p, seed, offset)).to(DEV)
    scale = torch.tensor(65536 / (65536 - X4.cut_of(p)), dtype=torch.float32, device=DEV)
    ref = torch.where(keep, (x.float() * scale), torch.zeros((), device=DEV)).to(dtype)
    assert torch.equal(y, ref)


def test_dropout_drops_non_finite_and_takes_rows_apart():
    q = qlib()
    x = torch.full((9, 40), float("nan"), dtype=torch.bfloat16, device=DEV)
    x[:, ::2] = float("inf")
    y = q.lora_dropout(x, 0.5, 3, 4)
    keep = torch.from_numpy(X4.keep(9, 40, 0.5, 3, 4)).to(DEV)
    assert torch.equal(y.float().isfinite(), ~keep) and bool((y[~keep] == 0).all())
    w = dev(np.random.default_rng(0).standard_normal((33, 96)))
    assert torch.equal(q.lora_dropout(w[:, :56], 0.3, 1, 2), q.lora_dropout(w[:, :56].contiguous(), 0.3, 1, 2))
    assert torch.equal(q.lora_dropout(w[:, :51], 0.3, 1, 2), q.lora_dropout(w[:, :51].contiguous(), 0.3, 1, 2))


MATMUL = [(1, 1, 1), (1, 5, 4096), (2, 300, 32), (7, 64, 129), (31, 33, 1000), (64, 256, 384), (100, 1000, 77),
          (257, 513, 640), (300, 260, 2100)]


@pytest.mark.parametrize("M,N,K", MATMUL)
def test_matmul(M, N, K):
    q = qlib()
    rng = np.random.default_rng(M + 7 * N + 13 * K)
    a, b = dev(rng.standard_normal((M, K))), dev(rng.standard_normal((N, K)) * np.exp2(rng.integers(-4, 4, (N, 1))))
    ac, bc = q.mx4_quantize(a), q.mx4_quantize(b)
    c = q.mx4_matmul(*ac, M, *bc, N, K)
    av, bv = X4.rounded(f64(a)), X4.rounded(f64(b))
    ref = av @ bv.T
    within(c, ref, 2.0**-8 * np.abs(ref) + K * U * (np.abs(av) @ np.abs(bv).T), f"matmul {M}x{N}x{K}")
    assert torch.equal(c, q.mx4_matmul(*ac, M, *bc, N, K))


def test_matmul_nan_blocks_stay_in_their_row_and_column():
    q = qlib()
    a, b = torch.ones((70, 300), device=DEV), torch.ones((140, 300), device=DEV)
    a[3, 290], a[69, 0], b[5, 40] = float("nan"), float("inf"), float("-inf")
    c = q.mx4_matmul(*q.mx4_quantize(a), 70, *q.mx4_quantize(b), 140, 300)
    nan = torch.zeros((70, 140), dtype=torch.bool, device=DEV)
    nan[3], nan[69], nan[:, 5] = True, True, True
    assert torch.equal(c.isnan(), nan) and bool((c[~nan] == 300).all())


# M, K, N, r: single tokens, decode sizes and both sides of them, lengths inside and past a block, ranks of every alignment
LAYER = [(1, 1, 1, 1), (1, 4096, 300, 64), (1, 1000, 77, 5), (4, 2048, 512, 16), (15, 520, 130, 12), (16, 1024, 1000, 64),
         (17, 256, 64, 8), (33, 97, 129, 3), (77, 1000, 777, 12), (130, 520, 333, 5), (257, 640, 513, 33),
         (300, 1152, 264, 64)]


def layer_data(M, K, N, r):
    rng = np.random.default_rng(M * 31 + K * 7 + N * 3 + r)
    X = rng.standard_normal((M, K)) * np.where(rng.random(K) < 0.02, 10.0, 1.0)
    if M > 3:
        X[2] = 0.0
    return {"X": dev(X), "dY": dev(rng.standard_normal((M, N)) * 0.1), "L1": dev(rng.standard_normal((K, r)) / K**0.5),
            "L2": dev(rng.standard_normal((r, N)) * 0.1), "W": dev(rng.standard_normal((N, K)) * 0.05)}


def check_forward(Y, T, d, xv, Wv, s, p, seed, off):
    X, L1, L2 = (f64(d[k]) for k in ("X", "L1", "L2"))
    K = X.shape[1]
    rY, rT = X4.linear_forward(xv, Wv, L1, L2, s, p, seed, off, T=X4.dropped(X, p, seed, off) @ L1)
    rT = X4.dropped(X, p, seed, off) @ L1
    sumT = np.abs(X4.dropped(X, p, seed, off)) @ np.abs(L1)
    tolT = 2.0**-8 * np.abs(rT) + (K + 4) * U * sumT
    within(T, rT, tolT, "T")
    tolY = 2.0**-8 * np.abs(rY) + (K + 4) * U * (np.abs(xv) @ np.abs(Wv).T) + s * (tolT @ np.abs(L2)) \
        + 70 * U * s * (np.abs(rT) @ np.abs(L2))
    within(Y, rY, tolY, "Y")


def check_backward(dX, dL1, dL2, T, d, dyv, Wtv, s, p, seed, off):
    X, dY, L1, L2 = (f64(d[k]) for k in ("X", "dY", "L1", "L2"))
    M, N = dY.shape
    rdX, rdL1, rdL2, G = X4.linear_backward(X, dY, dyv, Wtv, L1, L2, s, p, seed, off, f64(T))
    scale = 65536 / (65536 - X4.cut_of(p))
    errG = (N + 4) * U * s * (np.abs(dY) @ np.abs(L2).T)
    Xd = np.abs(X4.dropped(X, p, seed, off))
    within(dL1, rdL1, (M + 4) * U * (Xd.T @ np.abs(G)) + Xd.T @ errG, "dL1")
    within(dL2, rdL2, (M + 4) * U * s * (np.abs(f64(T)).T @ np.abs(dY)), "dL2")
    if dX is not None:
        tol = 2.0**-8 * np.abs(rdX) + (N + 4) * U * (np.abs(dyv) @ np.abs(Wtv).T)
        tol += scale * ((2.0**-8 + 70 * U) * np.abs(G) + errG) @ np.abs(L1).T
        within(dX, rdX, tol, "dX")


@pytest.mark.parametrize("M,K,N,r", LAYER)
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_layer(M, K, N, r, p):
    q = qlib()
    s, seed, off = 2.0, 0xDEADBEEF12345678, 2**32 + 3
    print(f"[mx4 layer] M={M} K={K} N={N} r={r} p={p}", flush=True)
    d = layer_data(M, K, N, r)
    w = q.mx4_quantize(d["W"])
    wt = q.mx4_quantize(d["W"], transpose=True)
    kw = dict(p=p, seed=seed, offset=off)
    Y, T = q.mx4_linear_fwd(d["X"], *w, N, d["L1"], d["L2"], s, T_out=True, **kw)
    Y2, none = q.mx4_linear_fwd(d["X"], *w, N, d["L1"], d["L2"], s, **kw)
    assert none is None and torch.equal(Y, Y2)
    check_forward(Y, T, d, X4.rounded(f64(d["X"])), X4.rounded(f64(d["W"])), s, p, seed, off)
    dX, dL1, dL2 = q.mx4_linear_bwd(d["X"], d["dY"], *wt, d["L1"], d["L2"], s, T=T, **kw)
    check_backward(dX, dL1, dL2, T, d, X4.rounded(f64(d["dY"])), X4.rounded(f64(d["W"]).T), s, p, seed, off)
    # T formed again, dX left out, run to run: the same bits
    again = q.mx4_linear_bwd(d["X"], d["dY"], *wt, d["L1"], d["L2"], s, dX=False, **kw)
    assert again[0] is None and torch.equal(again[1], dL1)
    if p > 0 or M > 16:
        assert torch.equal(again[2], dL2)
    dX2, _, _ = q.mx4_linear_bwd(d["X"], d["dY"], *wt, d["L1"], d["L2"], s, T=T, **kw)
    assert torch.equal(dX, dX2)


# the persistent kernel: several tiles a work group with the fewest reduction steps and with many, each direction, rows
# of C and ranks that are whole 16-byte pieces or not
LARGE = [(2100, 700, 8200, 16), (2100, 8200, 700, 24), (2093, 701, 8197, 5), (2093, 8197, 701, 5), (2100, 3912, 3920, 64)]


@pytest.mark.parametrize("M,K,N,r", LARGE)
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_large_layer(M, K, N, r, p):
    test_layer(M, K, N, r, p)


@pytest.mark.parametrize("M,N,K", [(2100, 8200, 700), (2093, 8197, 1301), (4352, 4360, 1024)])
def test_large_matmul(M, N, K):
    test_matmul(M, N, K)


NF4 = [(1, 64, 1, 1), (1, 4096, 300, 64), (16, 512, 136, 8), (17, 512, 200, 12), (32, 512, 512, 8), (33, 704, 71, 20),
       (48, 128, 1000, 64), (63, 1024, 96, 3), (130, 576, 333, 5), (300, 1152, 264, 64), (260, 320, 520, 16),
       (520, 4224, 72, 8)]


@pytest.mark.parametrize("M,K,N,r", NF4)
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_nf4_layer(M, K, N, r, p):
    q = qlib()
    s, seed, off = 1.5, 77, 2**45 + 1
    print(f"[nf4 dropout] M={M} K={K} N={N} r={r} p={p}", flush=True)
    d = layer_data(M, K, N, r)
    codes, absmax = q.nf4_quantize(d["W"])
    base = (codes, *q.nf4_double_quant(absmax))
    Wv = f64(q.nf4_dequantize(*base, N, K))
    kw = dict(p=p, seed=seed, offset=off)
    Y, T = q.qlora_linear_fwd_dropout(d["X"], *base, N, d["L1"], d["L2"], s, T_out=True, **kw)
    check_forward(Y, T, d, f64(d["X"]), Wv, s, p, seed, off)
    dX, dL1, dL2 = q.qlora_linear_bwd_dropout(d["X"], d["dY"], *base, d["L1"], d["L2"], s, T=T, **kw)
    check_backward(dX, dL1, dL2, T, d, f64(d["dY"]), Wv.T.copy(), s, p, seed, off)
    if p == 0:
        Y0, T0 = q.qlora_linear_fwd(d["X"], *base, N, d["L1"], d["L2"], s, T_out=True)
        dX0, _, _ = q.qlora_linear_bwd(d["X"], d["dY"], *base, d["L1"], d["L2"], s, T=T)
        assert torch.equal(Y, Y0) and torch.equal(T, T0) and torch.equal(dX, dX0)


def test_gradients_against_differences():
    """dL1 and dL2 of the calls against differences of the calls' own forward.  Y is linear in L1 for a fixed L2, up to
    the bf16 rounding of T and Y: a step along a random direction in L1 changes sum(Y dY) by <dL1, step>.  The step (bf16
    numbers, twice as large as L1) makes the change large beside the roundings: each Y is rounded by at most 2^-9 |Y| and
    each T by 2^-9 |T|, independently, so that the sum's error is a random walk over M N (and M r) terms; eight standard
    deviations are allowed."""
    q = qlib()
    M, K, N, r, s, kw = 96, 384, 160, 8, 1.0, dict(p=0.2, seed=5, offset=6)
    d = layer_data(M, K, N, r)
    w, wt = q.mx4_quantize(d["W"]), q.mx4_quantize(d["W"], transpose=True)
    zero = torch.zeros_like(w[0])                       # a base of zeros: the adapter alone
    T = q.mx4_linear_fwd(d["X"], zero, w[1], N, d["L1"], d["L2"], s, T_out=True, **kw)[1]
    _, dL1, dL2 = q.mx4_linear_bwd(d["X"], d["dY"], *wt, d["L1"], d["L2"], s, T=T, **kw)
    dY = f64(d["dY"])
    for name, g in (("L1", dL1), ("L2", dL2)):
        step = dev(np.random.default_rng(1).standard_normal(g.shape) * (2 * f64(d[name]).std()))
        ends = []
        for sign in (1, -1):
            moved = dict(d)
            moved[name] = (sign * step).contiguous()
            ends.append(q.mx4_linear_fwd(d["X"], zero, w[1], N, moved["L1"], moved["L2"], s, T_out=True, **kw))
        num = ((f64(ends[0][0]) - f64(ends[1][0])) * dY).sum() / 2
        want = (f64(g) * f64(step)).sum()
        Gm = s * dY @ f64(d["L2"]).T
        walk = 2.0**-9 * np.sqrt((f64(ends[0][0]) ** 2 * dY**2).sum() + (f64(ends[0][1]) ** 2 * Gm**2).sum()
                                 + (f64(T) ** 2 * Gm**2).sum())
        print(f"{name}: {num:.6f} against {want:.6f}, allowed {8 * walk:.6f}", flush=True)
        assert abs(num - want) <= 8 * walk
        assert abs(want) > 8 * walk                     # the comparison says something


def test_dx_mask_is_the_forwards():
    """With a base of zeros, dX is zero exactly where the forward's mask dropped X."""
    q = qlib()
    M, K, N, r = 70, 264, 136, 16
    d = layer_data(M, K, N, r)
    wt = q.mx4_quantize(torch.zeros_like(d["W"]), transpose=True)
    T = torch.zeros((M, r), dtype=torch.bfloat16, device=DEV)
    dX, _, _ = q.mx4_linear_bwd(d["X"], d["dY"], *wt, d["L1"], d["L2"], 1.0, p=0.4, seed=8, offset=9, T=T)
    y = q.lora_dropout(torch.ones((M, K), dtype=torch.bfloat16, device=DEV), 0.4, 8, 9)
    assert torch.equal(dX != 0, y != 0)


def test_non_finite_tokens_stay_in_their_rows():
    q = qlib()
    for M in (5, 40):
        d = layer_data(M, 256, 192, 8)
        w, wt = q.mx4_quantize(d["W"]), q.mx4_quantize(d["W"], transpose=True)
        ref, _ = q.mx4_linear_fwd(d["X"], *w, 192, d["L1"], d["L2"])
        X = d["X"].clone()
        X[1, 7], X[4, 255] = float("nan"), float("inf")
        Y, _ = q.mx4_linear_fwd(X, *w, 192, d["L1"], d["L2"])
        rows = [i for i in range(M) if i not in (1, 4)]
        assert bool(Y[1].isnan().all()) and bool(Y[4].isnan().all()) and torch.equal(Y[rows], ref[rows])
        dY = d["dY"].clone()
        dY[3, 100] = float("nan")
        T = torch.zeros((M, 8), dtype=torch.bfloat16, device=DEV)
        g0 = q.mx4_linear_bwd(d["X"], d["dY"], *wt, d["L1"], d["L2"], T=T)[0]
        g1 = q.mx4_linear_bwd(d["X"], dY, *wt, d["L1"], d["L2"], T=T)[0]
        rows = [i for i in range(M) if i != 3]
        assert bool(g1[3].isnan().all()) and torch.equal(g1[rows], g0[rows])


def test_streams_workspaces_and_graph():
    """A call on a stream of its own with a caller's workspace and outputs equals the plain call, also captured into a
    graph and replayed after its input changed (eager work between the replays)."""
    q = qlib()
    for M in (4, 64):
        d = layer_data(M, 512, 320, 16)
        w, wt = q.mx4_quantize(d["W"]), q.mx4_quantize(d["W"], transpose=True)
        kw = dict(p=0.1, seed=1, offset=2)
        ws = torch.empty(int(max(q.lib().mx4_linear_fwd_workspace(M, 512, 320, 16),
                                 q.lib().mx4_linear_bwd_workspace(M, 512, 320, 16))), dtype=torch.uint8, device=DEV)
        X = d["X"].clone()
        Y, T = torch.empty((M, 320), dtype=torch.bfloat16, device=DEV), torch.empty((M, 16), dtype=torch.bfloat16, device=DEV)
        dX, dL1, dL2 = torch.empty_like(X), torch.empty((512, 16), device=DEV), torch.empty((16, 320), device=DEV)

        def call(stream):
            q.mx4_linear_fwd(X, *w, 320, d["L1"], d["L2"], 1.5, Y=Y, T_out=T, workspace=ws, stream=stream, **kw)
            q.mx4_linear_bwd(X, d["dY"], *wt, d["L1"], d["L2"], 1.5, T=T, dX=dX, dL1=dL1, dL2=dL2, workspace=ws,
                             stream=stream, **kw)

        def plain():
            y, t = q.mx4_linear_fwd(X, *w, 320, d["L1"], d["L2"], 1.5, T_out=True, **kw)
            return y, t, *q.mx4_linear_bwd(X, d["dY"], *wt, d["L1"], d["L2"], 1.5, T=t, **kw)

        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        call(st)
        st.synchronize()
        for a, b in zip((Y, T, dX, dL1, dL2), plain()):
            assert torch.equal(a, b)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(torch.cuda.current_stream())
        for i in range(3):
            X.copy_(d["X"] * (i + 1))
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip((Y, T, dX, dL1, dL2), plain()):
                assert torch.equal(a, b), i


@pytest.mark.parametrize("M", [8, 1024])
def test_own_workspace_outlives_a_call_on_another_stream(M):
    q = qlib()
    K, N, r = 1024, 2048, 16
    d = layer_data(M, K, N, r)
    w = q.mx4_quantize(d["W"])
    wt = q.mx4_quantize(d["W"], transpose=True)
    args = dict(p=0.1, seed=5)
    Y, T = q.mx4_linear_fwd(d["X"], *w, N, d["L1"], d["L2"], T_out=True, **args)
    grads = q.mx4_linear_bwd(d["X"], d["dY"], *wt, d["L1"], d["L2"], T=T, **args)
    size = max(q.lib().mx4_linear_fwd_workspace(M, K, N, r), q.lib().mx4_linear_bwd_workspace(M, K, N, r))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                # the calls below wait behind this
    Y2, _ = q.mx4_linear_fwd(d["X"], *w, N, d["L1"], d["L2"], stream=side, **args)
    grads2 = q.mx4_linear_bwd(d["X"], d["dY"], *wt, d["L1"], d["L2"], T=T, stream=side, **args)
    junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(Y, Y2)
    for a, b in zip(grads, grads2):
        assert torch.equal(a, b)
    del junk


@pytest.mark.parametrize("rows,cols,dtype", [(16500, 8200, torch.bfloat16), (16411, 8203, torch.bfloat16),
                                             (8300, 8203, torch.float32), (8208, 8192, torch.float32)])
def test_larger_than_the_last_level_cache(rows, cols, dtype):
    """The same bits as on parts of the matrix small enough to go through the cache."""
    q = qlib()
    X = torch.randn(rows, cols, device=DEV, dtype=torch.float32).to(dtype)
    assert X.numel() * X.element_size() > 256 << 20
    parts = [slice(0, 70), slice(rows // 2, rows // 2 + 33), slice(rows - 41, rows)]
    cparts = [slice(0, 64), slice(cols - 72, cols)]
    D = q.lora_dropout(X, 0.3, 7, 9)
    assert torch.equal(D[:70], q.lora_dropout(X[:70], 0.3, 7, 9))
    assert torch.equal(D[:, :64], q.lora_dropout(X[:, :64], 0.3, 7, 9))
    kept = D != 0
    assert abs(kept[:, -72:].float().mean().item() - 0.7) < 0.01
    scale = 65536 / (65536 - X4.cut_of(0.3))
    assert torch.equal(D[kept], (X[kept].float() * scale).to(dtype))
    codes, scales = q.mx4_quantize(X)
    for s in parts:
        c, e = q.mx4_quantize(X[s].clone())
        assert torch.equal(codes[:, s], c) and torch.equal(scales[:, s], e)
    tc, te = q.mx4_quantize(X, transpose=True)
    for s in cparts:
        c, e = q.mx4_quantize(X[:, s].clone(), transpose=True)
        assert torch.equal(tc[:, s], c) and torch.equal(te[:, s], e)
    V = q.mx4_dequantize(codes, scales, rows, cols)
    for s in parts:
        n = s.stop - s.start
        assert torch.equal(V[s], q.mx4_dequantize(codes[:, s].contiguous(), scales[:, s].contiguous(), n, cols))


@pytest.mark.parametrize("M,K,N,r", [(5, 512, 136, 8), (16, 256, 72, 7), (33, 704, 71, 20), (64, 1024, 264, 64), (65, 512, 136, 12), (200, 1088, 136, 16), (300, 8192, 80, 5)])
def test_nf4_layer_forms_t_and_g_again_alike(M, K, N, r):
    """Without T the backward forms the forward's, and dX does not change the gradients."""
    q = qlib()
    d = layer_data(M, K, N, r)
    codes, absmax = q.nf4_quantize(d["W"])
    base = (codes, *q.nf4_double_quant(absmax))
    kw = dict(p=0.2, seed=3, offset=4)
    Y, T = q.qlora_linear_fwd_dropout(d["X"], *base, N, d["L1"], d["L2"], 1.5, T_out=True, **kw)
    Y2, _ = q.qlora_linear_fwd_dropout(d["X"], *base, N, d["L1"], d["L2"], 1.5, **kw)
    assert torch.equal(Y, Y2)
    dX, dL1, dL2 = q.qlora_linear_bwd_dropout(d["X"], d["dY"], *base, d["L1"], d["L2"], 1.5, T=T, **kw)
    none, dL1b, dL2b = q.qlora_linear_bwd_dropout(d["X"], d["dY"], *base, d["L1"], d["L2"], 1.5, dX=False, **kw)
    assert none is None and torch.equal(dL1, dL1b) and torch.equal(dL2, dL2b)


@pytest.mark.parametrize("M,K,N,r", [(700, 1100, 60, 20), (1030, 260, 200, 33), (2000, 70, 24, 64), (520, 9000, 40, 8)])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_narrow_layer(M, K, N, r, p):
    """Many rows, few columns on one side or the other."""
    test_layer(M, K, N, r, p)


@pytest.mark.parametrize("M,K,N,r", [(4, 512, 136, 8), (40, 512, 72, 5), (200, 320, 264, 64), (700, 1024, 512, 16),
                                     (600, 320, 2048, 20)])
@pytest.mark.parametrize("layer", ["mx4", "nf4"])
def test_dropped_places_hold_anything(layer, M, K, N, r):
    """Infinities and NaN in places that the mask drops do not reach T or dL1; the same bits as with zeros there."""
    q = qlib()
    d = layer_data(M, K, N, r)
    kw = dict(p=0.3, seed=11, offset=5)
    kept = q.lora_dropout(torch.ones((M, K), dtype=torch.bfloat16, device=DEV), **kw) != 0
    zero = torch.where(kept, d["X"], torch.zeros_like(d["X"]))
    odd = torch.tensor([float("nan"), float("inf"), float("-inf")], dtype=torch.bfloat16, device=DEV)
    junk = odd[torch.arange(M * K, device=DEV).reshape(M, K) % 3]
    bad = torch.where(kept, d["X"], junk)
    if layer == "mx4":
        w, wt = q.mx4_quantize(d["W"]), q.mx4_quantize(d["W"], transpose=True)
        fwd = lambda X: q.mx4_linear_fwd(X, *w, N, d["L1"], d["L2"], 1.5, T_out=True, **kw)
        bwd = lambda X, T: q.mx4_linear_bwd(X, d["dY"], *wt, d["L1"], d["L2"], 1.5, T=T, **kw)
    else:
        codes, absmax = q.nf4_quantize(d["W"])
        base = (codes, *q.nf4_double_quant(absmax))
        fwd = lambda X: q.qlora_linear_fwd_dropout(X, *base, N, d["L1"], d["L2"], 1.5, T_out=True, **kw)
        bwd = lambda X, T: q.qlora_linear_bwd_dropout(X, d["dY"], *base, d["L1"], d["L2"], 1.5, T=T, **kw)
    T = fwd(zero)[1]
    assert torch.isfinite(T.float()).all() and torch.equal(T, fwd(bad)[1])
    for a, b in zip(bwd(zero, T), bwd(bad, T)):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)
    for a, b in zip(bwd(zero, None), bwd(bad, None)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("layer,M,K,N", [("mx4", 700, 512, 1024), ("mx4", 2100, 1024, 8200), ("mx4", 2100, 8200, 700), ("nf4", 8, 512, 328),
                                         ("nf4", 40, 512, 320), ("nf4", 600, 512, 2048), ("nf4", 2100, 8256, 320)])
def test_graph_replays(layer, M, K, N):
    """Forward, backward and dropout captured together: every replay equals the eager calls on the input it then has."""
    q = qlib()
    r = 16
    d = layer_data(M, K, N, r)
    kw = dict(p=0.1, seed=1, offset=2)
    X = d["X"].clone()
    if layer == "mx4":
        w, wt = q.mx4_quantize(d["W"]), q.mx4_quantize(d["W"], transpose=True)
    else:
        codes, absmax = q.nf4_quantize(d["W"])
        base = (codes, *q.nf4_double_quant(absmax))

    def calls():
        H = q.lora_dropout(X, **kw)
        if layer == "mx4":
            y, t = q.mx4_linear_fwd(H, *w, N, d["L1"], d["L2"], 1.5, T_out=True, **kw)
            return y, t, *q.mx4_linear_bwd(H, d["dY"], *wt, d["L1"], d["L2"], 1.5, T=t, **kw)
        y, t = q.qlora_linear_fwd_dropout(H, *base, N, d["L1"], d["L2"], 1.5, T_out=True, **kw)
        return y, t, *q.qlora_linear_bwd_dropout(H, d["dY"], *base, d["L1"], d["L2"], 1.5, T=t, **kw)

    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = calls()
    for i in range(3):
        X.copy_(d["X"] * (i + 1))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, calls()):
            assert torch.equal(a, b), i
