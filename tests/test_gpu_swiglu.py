"""GPU parity of the gated product, of its backward and of the linear's backward from 8-bit
activations against the oracle.

Tolerances, elementwise, derived from the rounding points (U = 2^-24, half a step of bf16 2^-8):
  a sum of n exact products in fp32, in any order: n U sum |a b|;
  T in the product as two bf16 planes at least: 2^-16 |T| on top;
  H = silu(G) U: |silu'| <= 1.1, so G and U off by dg and du move it by 1.1 |U| dg + |silu(G)| du + 1.1 dg du,
  silu's own exponential, sum and reciprocal by E = (|G| + 4) 2^-23 of it (the exponent's rounding is
  relative to G), rounding to bf16 by 2^-8;
  a value in 8 bits is the rounding of one in [g - dg, g + dg];
  dZ: dU = dH G sig by E |dU|, dG = dH U sig (1 + G (1 - sig)) by E |dH U| sig (1 + |G|) (1 + |G|): the
  factor's two terms may cancel, and 1 - sig carries sig's error times G;
  B and dL1, dL2 carry those and their own sums, three planes lose 2^-24; dX takes dZ in bf16 and B as
  two bf16 planes: 2^-8 |dZ| |W| (2^-16 for few terms, whose planes' products double the sum's terms) and
  2^-16 |B| |L1| on top (a linear's dX takes B in bf16).
"""
import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import bits
from test_gpu_norm import packed_between, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
X8 = O.mx8
U = 2.0 ** -24
S = 2.0


def qlib():
    import bit_quantized_lora_blockwise_amd as q
    return q


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Block:
    """Inputs of one gated block over an NF4 base, on the GPU and as float64."""

    def __init__(self, seed, M, K, F, r, halves=2):
        q = qlib()
        g = torch.Generator().manual_seed(seed)
        n = lambda *shape, std=1.0: (std * torch.randn(*shape, generator=g)).to(torch.bfloat16)  # noqa: E731
        self.M, self.K, self.F, self.r = M, K, F, r
        X = n(M, K)
        X[:, :: max(2, K // 3)] *= 10
        if M > 4:
            X[3] = 0
        self.X = X.to(DEV)
        W = n(halves * F, K, std=0.02).to(DEV)
        codes, absmax = q.nf4_quantize(W)
        self.base = (codes, *q.nf4_double_quant(absmax))
        self.W = f64(q.nf4_dequantize(*self.base, halves * F, K))
        self.L1, self.L2 = n(halves, K, r, std=K ** -0.5).to(DEV), n(halves, r, F, std=0.05).to(DEV)
        self.d = n(M, F, std=0.01).to(DEV)

    def forward(self):
        return X8.swiglu_forward(f64(self.X), self.W, f64(self.L1), f64(self.L2), S)

    def slack(self):
        """(dg, du, dT): how far the sums of G, U and T may be off."""
        x, w, F = np.abs(f64(self.X)), np.abs(self.W), self.F
        dz, dt = [], []
        for h in range(2):
            l1, l2 = np.abs(f64(self.L1[h])), np.abs(f64(self.L2[h]))
            t = np.abs(f64(self.X) @ f64(self.L1[h]))
            off = self.K * U * (x @ l1) + 2.0**-16 * t
            dt.append(self.K * U * (x @ l1))
            dz.append((self.K + 130) * U * (x @ w[h * F:(h + 1) * F].T + S * (t @ l2)) + S * (off @ l2))
        return dz[0], dz[1], np.stack(dt)


FORWARD = [(1, 64, 1, 1), (3, 4096, 48, 12), (9, 2048, 17, 5), (16, 4096, 64, 64), (24, 1024, 100, 37), (400, 64, 20, 64), (1, 4096, 512, 64), (2, 128, 33, 3), (16, 256, 100, 8), (17, 320, 129, 64), (5, 1088, 777, 12),
           (33, 64, 16, 5), (77, 1024, 777, 12), (130, 576, 128, 64), (257, 192, 300, 33), (300, 512, 130, 16), (64, 64, 3, 64),
           # eight rows in LDS at most 32 KB wide; then the large tiles: one round, several, one tile row, a step alone
           (2, 8192, 40, 16), (4, 4096, 65, 64), (1300, 128, 1100, 12), (4100, 64, 2000, 64), (34, 192, 20601, 8),
           (4100, 64, 300, 5)]


@pytest.mark.parametrize("M,K,F,r", FORWARD)
def test_forward(M, K, F, r):
    q = qlib()
    b = Block(M * 1009 + K + F, M, K, F, r)
    H, T, gu8 = q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S, T_out=True, mx8=True)
    h, g, u, t = b.forward()
    dg, du, dt = b.slack()
    within(T, t, dt + 2.0**-8 * np.abs(t), "T")
    packed_between(gu8, np.concatenate([g, u]), np.concatenate([dg, du]), F, "GU")
    e = (np.abs(g) + 4) * 2.0**-23
    tol = (1 + 2.0**-8) * (1.1 * np.abs(u) * dg + np.abs(g * X8.sigmoid(g)) * du + 1.1 * dg * du + e * np.abs(h)) + 2.0**-8 * np.abs(h)
    within(H, h, tol, "H")
    rel = np.linalg.norm(f64(H) - h) / np.linalg.norm(h)
    # half a step of bf16 is at most 2^-8 of a value, and so of the norm of any number of them; the fp32 sums' part
    # (2^-24 K at most) is far below what that bound leaves
    assert rel <= 2.0**-8, rel
    # without what the backward needs: H by another kernel for up to 16 rows, the same one beyond
    H2, none, no8 = q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S)
    assert none is None and no8 is None
    within(H2, h, tol, "H alone")
    H3, T3, _ = q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S, T_out=True)
    assert torch.equal(H2, H3) and torch.equal(T, T3)
    assert M <= 16 or torch.equal(H, H2)


def check_backward(q, b, x8, gu8, T, dX, dL1, dL2, dz_bits=2.0**-8):
    M, K, F, r = b.M, b.K, b.F, b.r
    x = X8.values(x8[0].cpu().numpy(), x8[1].cpu().numpy(), K)
    gu = X8.values(gu8[0].cpu().numpy(), gu8[1].cpu().numpy(), F)
    g, u, dh, t = gu[:M], gu[M:], f64(b.d), f64(T).reshape(2, M, r)
    l1, l2 = f64(b.L1), f64(b.L2)
    rx, r1, r2, dz, B = X8.swiglu_backward(x, dh, g, u, b.W, l1, l2, t, S)
    sig = X8.sigmoid(g)
    e = (np.abs(g) + 4) * 2.0**-23
    off = np.stack([e * np.abs(dh * u) * sig * (1 + np.abs(g)) ** 2, e * np.abs(dz[1])]) + 4 * U * np.abs(dz)
    tx = 2.0**-8 * np.abs(rx)
    for h in range(2):
        w, a1, a2 = np.abs(b.W[h * F:(h + 1) * F]), np.abs(l1[h]), np.abs(l2[h])
        ob = S * (off[h] @ a2.T) + (3 * F + 40) * U * S * (np.abs(dz[h]) @ a2.T)
        within(dL1[h], r1[h], np.abs(x).T @ ob + (3 * M + 40) * U * (np.abs(x).T @ np.abs(B[h])), f"dL1[{h}]")
        within(dL2[h], r2[h], S * (np.abs(t[h]).T @ off[h]) + (3 * M + 40) * U * S * (np.abs(t[h]).T @ np.abs(dz[h])),
               f"dL2[{h}]")
        if dX is not None:
            terms = 2 * F if dz_bits == 2.0**-8 else 4 * F
            tx = tx + ((dz_bits + (terms + 130) * U) * np.abs(dz[h]) + off[h]) @ w
            tx = tx + ((2.0**-16 + (2 * F + 260) * U) * np.abs(B[h]) + ob) @ a1.T
    if dX is not None:
        within(dX, rx, tx, "dX")
        rel = np.linalg.norm(f64(dX) - rx) / np.linalg.norm(rx)
        assert rel <= 2.0**-7, rel            # dZ's rounding to bf16 and the result's, 2^-8 each
    for got, ref, name in ((dL1, r1, "dL1"), (dL2, r2, "dL2")):
        rel = np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)
        print(name, "rel", rel, flush=True)
        assert rel <= 1e-5, (name, rel)


BACKWARD = [(1, 64, 1, 1), (1, 128, 40, 8), (2, 128, 33, 3), (16, 256, 100, 8), (17, 320, 129, 64), (33, 64, 16, 5),
            (130, 576, 777, 12), (257, 192, 300, 33), (520, 128, 68, 16), (300, 704, 130, 64), (64, 64, 3, 64),
            # dX in large tiles, rows of dZ padded; 260 of them, the gradients beside the last round
            (800, 2048, 37, 12), (1600, 1024, 136, 64), (1000, 16640, 20, 8),
            # its reduction in slices: of one row, of a whole tile and a part, of a length that ends inside a step
            (1, 128, 3500, 8), (33, 320, 3501, 12), (257, 576, 3333, 64), (300, 4096, 1100, 5)]


@pytest.mark.parametrize("M,K,F,r", BACKWARD)
def test_backward(M, K, F, r):
    q = qlib()
    b = Block(M * 1013 + K + F, M, K, F, r)
    x8 = q.mx8_quantize(b.X)
    _, T, gu8 = q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S, T_out=True, mx8=True)
    dX, dL1, dL2 = q.qlora_swiglu_bwd(x8, b.d, *b.base, b.L1, b.L2, gu8, T, S)
    check_backward(q, b, x8, gu8, T, dX, dL1, dL2)
    none, a1, a2 = q.qlora_swiglu_bwd(x8, b.d, *b.base, b.L1, b.L2, gu8, T, S, dX=False)
    assert none is None and torch.equal(a1, dL1) and torch.equal(a2, dL2)


@pytest.mark.parametrize("M,K,F,r", [(1, 64, 1, 1), (1, 320, 16, 54), (2, 192, 16, 1), (5, 512, 48, 37), (1, 128, 1024, 8),
                                     (40, 64, 25, 64), (300, 704, 3, 9)])
def test_backward_of_few_terms(M, K, F, r):
    """dX of up to 1024 values of dH takes dZ as two bf16 planes: 2^-16 of it in place of 2^-8."""
    q = qlib()
    b = Block(M * 1021 + K + F, M, K, F, r)
    x8 = q.mx8_quantize(b.X)
    _, T, gu8 = q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S, T_out=True, mx8=True)
    check_backward(q, b, x8, gu8, T, *q.qlora_swiglu_bwd(x8, b.d, *b.base, b.L1, b.L2, gu8, T, S), dz_bits=2.0**-16)


@pytest.mark.parametrize("level", [40.0, 100.0, 400.0])
def test_backward_of_far_gates(level):
    """Gates far on either side: sigmoids of 0 and 1, no NaN."""
    q = qlib()
    M, K, F, r = 40, 64, 96, 8
    b = Block(5, M, K, F, r)
    g = torch.Generator().manual_seed(6)
    gu = torch.cat([level * torch.randn(M, F, generator=g), torch.randn(M, F, generator=g)]).to(DEV)
    gu8, x8 = q.mx8_quantize(gu), q.mx8_quantize(b.X)
    T = torch.randn(2, M, r, generator=g).to(torch.bfloat16).to(DEV)
    dX, dL1, dL2 = q.qlora_swiglu_bwd(x8, b.d, *b.base, b.L1, b.L2, gu8, T, S)
    for t in (dX, dL1, dL2):
        assert torch.isfinite(t).all()
    check_backward(q, b, x8, gu8, T, dX, dL1, dL2)


LINEAR = [(1, 64, 1, 1), (1, 1088, 333, 5), (7, 128, 40, 8), (16, 64, 9, 64), (17, 320, 129, 33), (77, 1088, 333, 5),
          (130, 576, 776, 12), (600, 192, 300, 16), (257, 4096, 64, 64), (300, 64, 7, 3), (800, 2048, 37, 12),
          (800, 2048, 40, 12), (1000, 16640, 24, 8),
          # in slices
          (1, 64, 6152, 3), (40, 192, 7000, 16), (300, 4096, 2056, 64)]


@pytest.mark.parametrize("M,K,N,r", LINEAR)
def test_linear_backward(M, K, N, r):
    q = qlib()
    b = Block(M * 1019 + K + N, M, K, N, r, halves=1)
    L1, L2 = b.L1[0].contiguous(), b.L2[0].contiguous()
    x8 = q.mx8_quantize(b.X)
    T = q.qlora_lora_down(b.X, L1)
    dX, dL1, dL2 = q.qlora_linear_bwd_mx8(x8, b.d, *b.base, L1, L2, T, S)
    x = X8.values(x8[0].cpu().numpy(), x8[1].cpu().numpy(), K)
    l1, l2, dy, t = f64(L1), f64(L2), f64(b.d), f64(T)
    B = S * dy @ l2.T
    ob = (N + 40) * U * S * (np.abs(dy) @ np.abs(l2).T)
    r1, r2, rx = x.T @ B, S * t.T @ dy, dy @ b.W + B @ l1.T
    within(dL1, r1, np.abs(x).T @ ob + (3 * M + 40) * U * (np.abs(x).T @ np.abs(B)), "dL1")
    within(dL2, r2, (M + 40) * U * S * (np.abs(t).T @ np.abs(dy)), "dL2")
    within(dX, rx, 2.0**-8 * np.abs(rx) + (N + 130) * U * (np.abs(dy) @ np.abs(b.W)) +
           ((2.0**-8 + 130 * U) * np.abs(B) + ob) @ np.abs(l1).T, "dX")
    none, a1, a2 = q.qlora_linear_bwd_mx8(x8, b.d, *b.base, L1, L2, T, S, dX=False)
    assert none is None and torch.equal(a1, dL1) and torch.equal(a2, dL2)


def step(q, X, R, w, up, down, L, dO):
    """A pre-norm feed-forward block, forward and backward, from 8-bit activations."""
    Y, Sm, y8 = q.rms_norm_fwd(X, w, 1e-5, residual=R, mx8=True)
    F, K = down[1]
    H, T, gu8 = q.qlora_swiglu_fwd(Y, *up, F, L[0], L[1], S, T_out=True, mx8=True)
    O_, Td = q.qlora_linear_fwd(H, *down[0], K, L[2], L[3], S, T_out=True)
    h8 = q.mx8_quantize(H)
    dH, d3, d4 = q.qlora_linear_bwd_mx8(h8, dO, *down[0], L[2], L[3], Td, S)
    dY, d1, d2 = q.qlora_swiglu_bwd(y8, dH, *up, L[0], L[1], gu8, T, S)
    dX, dw = q.rms_norm_bwd(dY, Sm, w, 1e-5, dS=dO)
    return O_, dX, dw, d1, d2, d3, d4


def block_of(q, M, K, F, r):
    b, c = Block(3, M, K, F, r), Block(4, M, F, K, r, halves=1)
    g = torch.Generator().manual_seed(8)
    R = (0.3 * torch.randn(M, K, generator=g)).to(torch.bfloat16).to(DEV)
    w = (1 + 0.2 * torch.randn(K, generator=g)).to(torch.bfloat16).to(DEV)
    L = (b.L1, b.L2, c.L1[0].contiguous(), c.L2[0].contiguous())
    return b, c, (b.X, R, w, b.base, (c.base, (F, K)), L, c.d)


@pytest.mark.parametrize("M,K,F,r", [(64, 256, 320, 8), (300, 128, 192, 12)])
def test_block_step_against_autograd(M, K, F, r):
    """The whole block against autograd in 64 bits.  8 bits leave 2^-4 of a value at most, so each weight of a
    gradient's sums is off by a random share of that: the gradients' norm by less than 2^-4.  The output passes seven
    roundings to bf16 of 2^-8 at most: S and Y, which reach H twice, through G and through U, H, the down adapter's T
    and its own."""
    q = qlib()
    b, c, args = block_of(q, M, K, F, r)
    got = step(q, *args)
    X, R, w, _, _, L, dO = args
    d = [t.detach().double().cpu().requires_grad_() for t in (X, w, *L)]
    x, wt, a1, a2, a3, a4 = d
    Wu, Wd = torch.from_numpy(b.W), torch.from_numpy(c.W)
    s = x + R.double().cpu()
    y = s / torch.sqrt(s.square().mean(1, keepdim=True) + 1e-5) * wt
    G, Uu = (y @ Wu[h * F:(h + 1) * F].t() + S * (y @ a1[h]) @ a2[h] for h in range(2))
    h = torch.nn.functional.silu(G) * Uu
    o = h @ Wd.t() + S * (h @ a3) @ a4
    ((o + s) * dO.double().cpu()).sum().backward()
    ref = (o.detach(), x.grad, wt.grad, a1.grad, a2.grad, a3.grad, a4.grad)
    for k, (u, v) in enumerate(zip(got, ref)):
        rel = float((u.double().cpu() - v).norm() / v.norm())
        print("output", k, "rel", rel, flush=True)
        assert rel <= (7 * 2.0**-8 if k == 0 else 2.0**-4), (k, rel)


def test_block_step_on_another_stream_and_captured():
    q = qlib()
    _, _, args = block_of(q, 96, 128, 192, 8)
    want = step(q, *args)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = step(q, *args)
    st.synchronize()
    for a, v in zip(other, want):
        assert torch.equal(a, v)
    x = args[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(q, x, *args[1:])
    for k in range(3):
        x.copy_(args[0] * (0.5 + k))
        graph.replay()
        eager = step(q, x, *args[1:])
        torch.cuda.synchronize()
        for a, v in zip(held, eager):
            assert torch.equal(a, v), k


def test_calls_at_once_on_two_streams():
    """Two blocks in flight on streams of their own, sizes of every kind of dX, against one after the other."""
    q = qlib()
    sizes = [(96, 128, 192, 8), (40, 128, 6200, 8), (1000, 16640, 24, 8), (3, 4096, 65, 64)]
    work = []
    for n, (M, K, F, r) in enumerate(sizes):
        b = Block(41 + n, M, K, F, r)
        x8 = q.mx8_quantize(b.X)

        def run(b=b, x8=x8, F=F):
            H, T, gu8 = q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S, T_out=True, mx8=True)
            return (H, T, *gu8, *q.qlora_swiglu_bwd(x8, b.d, *b.base, b.L1, b.L2, gu8, T, S))

        work.append((run, run()))
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for n in range(len(work)):
        got = []
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                f, want = work[(n + k) % len(work)]
                got.append((f(), f(), want))
        torch.cuda.synchronize()
        for first, second, want in got:
            for u, v, x in zip(first, second, want):
                assert torch.equal(u, x) and torch.equal(v, x), n


@pytest.mark.parametrize("M,K,F", [(1000, 16640, 24), (40, 128, 100), (40, 128, 6200)])
def test_backward_captured(M, K, F):
    """Captured with the gradients beside dX, without and with dX in slices, then replayed between eager calls."""
    q = qlib()
    r = 8
    b, c = Block(31, M, K, F, r), Block(32, M, K, F, r, halves=1)
    x8 = q.mx8_quantize(b.X)
    _, T, gu8 = q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S, T_out=True, mx8=True)
    L1, L2 = c.L1[0].contiguous(), c.L2[0].contiguous()
    Tl = q.qlora_lora_down(b.X, L1)
    d = b.d.clone()

    def both():
        return (*q.qlora_swiglu_bwd(x8, d, *b.base, b.L1, b.L2, gu8, T, S),
                *q.qlora_linear_bwd_mx8(x8, d, *c.base, L1, L2, Tl, S))

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for k in range(3):
        d.copy_(b.d * (0.5 + k))
        graph.replay()
        eager = both()
        torch.cuda.synchronize()
        for u, v in zip(held, eager):
            assert torch.equal(u, v), k


def test_stream_given_by_argument_or_handle():
    """Calls on a stream that is passed, as a stream or as an object with its handle alone."""
    q = qlib()
    b = Block(27, 70, 128, 104, 8)
    w = torch.ones(128, device=DEV)

    def run(**kw):
        Y, Sm, y8 = q.rms_norm_fwd(b.X, w, 1e-5, residual=b.X, mx8=True, **kw)
        H, T, gu8 = q.qlora_swiglu_fwd(Y, *b.base, 104, b.L1, b.L2, S, T_out=True, mx8=True, **kw)
        g = q.qlora_swiglu_bwd(y8, b.d, *b.base, b.L1, b.L2, gu8, T, S, **kw)
        dX, dw = q.rms_norm_bwd(g[0], Sm, w, 1e-5, **kw)
        return (H, *g, dX, dw, q.mx8_dequantize(*q.mx8_quantize(dX, **kw), 70, 128, **kw))

    want = run()
    st = torch.cuda.Stream()

    class Handle:
        cuda_stream = st.cuda_stream

    for stream in (st, Handle()):
        st.wait_stream(torch.cuda.current_stream())
        got = run(stream=stream)
        st.synchronize()
        for a, v in zip(got, want):
            assert torch.equal(a, v)


@pytest.mark.parametrize("M,K,F,r", [(40, 128, 100, 8), (3, 64, 20, 5), (40, 128, 6200, 8), (1300, 128, 1100, 12), (600, 64, 72, 64)])
def test_given_outputs_and_workspace(M, K, F, r):
    q = qlib()
    b = Block(21, M, K, F, r)
    H, T, gu8 = q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S, T_out=True, mx8=True)
    L = q.lib()
    ws = torch.full((L.qlora_swiglu_fwd_workspace(M, K, F, r),), 255, dtype=torch.uint8, device=DEV)
    h, t = torch.empty_like(H), torch.empty_like(T)
    p = tuple(torch.full_like(v, 9) for v in gu8)
    got = q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S, H=h, T_out=t, mx8=p, workspace=ws)
    assert got[0] is h and got[1] is t and torch.equal(h, H) and torch.equal(t, T)
    assert torch.equal(p[0], gu8[0]) and torch.equal(p[1], gu8[1])
    x8 = q.mx8_quantize(b.X)
    want = q.qlora_swiglu_bwd(x8, b.d, *b.base, b.L1, b.L2, gu8, T, S)
    ws = torch.full((L.qlora_swiglu_bwd_workspace(M, K, F, r),), 255, dtype=torch.uint8, device=DEV)   # NaN all over
    outs = [torch.full_like(v, 7) for v in want]
    got = q.qlora_swiglu_bwd(x8, b.d, *b.base, b.L1, b.L2, gu8, T, S, dX=outs[0], dL1=outs[1], dL2=outs[2], workspace=ws)
    for a, o, v in zip(got, outs, want):
        assert a is o and torch.equal(a, v)
    bl = Block(22, M, K, F, r, halves=1)
    L1, L2 = bl.L1[0].contiguous(), bl.L2[0].contiguous()
    Tl = q.qlora_lora_down(bl.X, L1)
    want = q.qlora_linear_bwd_mx8(x8, bl.d, *bl.base, L1, L2, Tl, S)
    ws = torch.full((L.qlora_linear_bwd_mx8_workspace(M, K, F, r),), 255, dtype=torch.uint8, device=DEV)
    got = q.qlora_linear_bwd_mx8(x8, bl.d, *bl.base, L1, L2, Tl, S, workspace=ws)
    for a, v in zip(got, want):
        assert torch.equal(a, v)


def test_rows_that_are_not_finite_stay_alone():
    """A row with an infinity spoils its own outputs and sums over rows, nothing of other rows."""
    q = qlib()
    M, K, F, r = 40, 128, 100, 8
    b = Block(23, M, K, F, r)
    H, T, gu8 = q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S, T_out=True, mx8=True)
    x = b.X.clone()
    x[5, 7] = float("inf")
    h, t, p = q.qlora_swiglu_fwd(x, *b.base, F, b.L1, b.L2, S, T_out=True, mx8=True)
    rest = [i for i in range(M) if i != 5]
    assert torch.equal(h[rest], H[rest]) and torch.equal(t[:, rest], T[:, rest])
    assert torch.equal(p[0].view(2, M, -1)[:, rest], gu8[0].view(2, M, -1)[:, rest])
    assert (p[1].view(2, M, -1)[:, 5] == 255).all()
    x8, x8b = q.mx8_quantize(b.X), q.mx8_quantize(x)
    dX = q.qlora_swiglu_bwd(x8, b.d, *b.base, b.L1, b.L2, gu8, T, S)[0]
    dx = q.qlora_swiglu_bwd(x8b, b.d, *b.base, b.L1, b.L2, p, T, S)[0]
    assert torch.equal(dx[rest], dX[rest])


def test_decoding_row_by_row_is_the_batch():
    """Rows one at a time against all at once, within what the orders of the sums allow."""
    q = qlib()
    M, K, F, r = 20, 512, 200, 16
    b = Block(24, M, K, F, r)
    h, g, u, _ = b.forward()
    dg, du, _ = b.slack()
    e = (np.abs(g) + 4) * 2.0**-23
    tol = (1 + 2.0**-8) * (1.1 * np.abs(u) * dg + np.abs(g * X8.sigmoid(g)) * du + 1.1 * dg * du + e * np.abs(h)) + 2.0**-8 * np.abs(h)
    one = torch.cat([q.qlora_swiglu_fwd(b.X[i:i + 1].contiguous(), *b.base, F, b.L1, b.L2, S)[0] for i in range(M)])
    within(one, h, tol, "one at a time")
    assert np.count_nonzero(bits(one) != bits(q.qlora_swiglu_fwd(b.X, *b.base, F, b.L1, b.L2, S)[0])) <= one.numel() // 50


def test_tensors_of_another_device_are_refused(monkeypatch):
    q = qlib()
    b = Block(25, 20, 128, 40, 8)
    x8 = q.mx8_quantize(b.X)
    _, T, gu8 = q.qlora_swiglu_fwd(b.X, *b.base, 40, b.L1, b.L2, S, T_out=True, mx8=True)
    w = torch.ones(128, device=DEV)
    c = Block(26, 20, 128, 40, 8, halves=1)
    calls = [lambda: q.mx8_quantize(b.X), lambda: q.mx8_dequantize(*x8, 20, 128), lambda: q.rms_norm_fwd(b.X, w, 1e-5),
             lambda: q.rms_norm_bwd(b.X, b.X, w, 1e-5), lambda: q.qlora_swiglu_fwd(b.X, *b.base, 40, b.L1, b.L2, S),
             lambda: q.qlora_swiglu_bwd(x8, b.d, *b.base, b.L1, b.L2, gu8, T, S),
             lambda: q.qlora_linear_bwd_mx8(x8, c.d, *c.base, c.L1[0], c.L2[0], T[0], S)]
    for f in calls:
        f()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)      # the current device, as the binding asks for it
    for f in calls:
        with pytest.raises(ValueError, match="cuda:1"):
            f()
