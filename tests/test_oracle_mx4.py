"""CPU pins of the microscaled and dropout oracle: published vectors of the
generator, the element format by exhaustive comparison, and the layer's
gradients against differences of its forward."""
from fractions import Fraction

import numpy as np
import pytest

import oracle as O

X4 = O.mx4


# Random123's known-answer vectors of philox4x32 (counter, key, output)
KAT = [
    (7, [0] * 4, [0] * 2, [0x5F6FB709, 0x0D893F64, 0x4F121F81, 0x4F730A48]),
    (7, [0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x5207DDC2, 0x45165E59, 0x4D8EE751, 0x8C52F662]),
    (10, [0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    (10, [0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    (10, [0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
]


@pytest.mark.parametrize("rounds,ctr,key,out", KAT)
def test_philox_known_answers(rounds, ctr, key, out):
    assert [int(x) for x in X4.philox4x32(ctr, key, rounds)] == out


def test_mask_rate_and_independence():
    p, n = 0.1, 512
    k = X4.keep(n, n, p, 12345, 7)
    sd = np.sqrt(p * (1 - p) / k.size)
    assert abs(k.mean() - (1 - X4.cut_of(p) / 65536)) < 5 * sd
    for other in (X4.keep(n, n, p, 12346, 7), X4.keep(n, n, p, 12345, 8), X4.keep(n, n, p, 12345 + 2**32, 7),
                  X4.keep(n, n, p, 12345, 7 + 2**32)):
        both = (~k & ~other).mean()
        assert abs(both - p * p) < 5 * np.sqrt(p * p / k.size)
    assert X4.keep(4, 9, 0.0, 1, 1).all()
    assert np.array_equal(X4.keep(5, 13, p, 3, 4), X4.keep(9, 40, p, 3, 4)[:5, :13])   # a function of (m, k) alone


def _nearest(v, e):
    """Brute force in exact rationals, ties to the even code."""
    n = abs(Fraction(float(v))) / Fraction(2) ** int(e)
    d = [abs(n - Fraction(float(q))) for q in X4.E2M1]
    best = min(d)
    return min((c for c in range(8) if d[c] == best), key=lambda c: c % 2)


def test_quantize_against_rationals():
    rng = np.random.default_rng(0)
    X = (rng.standard_normal((8, 64)) * np.exp2(rng.integers(-126, 100, (8, 1)))).astype(np.float32)
    X[0, :9] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0, -5.0]
    X[0, 9:32] = 0
    X[7] = 0
    codes, scales = X4.quantize(X)
    assert np.all(scales[7] == 4) and np.all(codes[7] == 0)
    for i in range(8):
        for b in range(2):
            blk = X[i, 32 * b:32 * b + 32]
            top = Fraction(float(np.abs(blk).max()))
            e = -123
            if top:
                e = next(j for j in range(-160, 200) if Fraction(2) ** j <= top < Fraction(2) ** (j + 1)) - 2
                e = max(e, -123)
            assert int(scales[i, b]) == e + 127
            for j in range(32):
                c = int(codes[i, 32 * b + j])
                assert c & 7 == _nearest(blk[j], e)
                assert (c >> 3) == int(np.signbit(blk[j]))


def test_quantize_special_blocks_and_padding():
    X = np.ones((2, 70), np.float32)
    X[0, 3], X[1, 65] = np.inf, np.nan
    codes, scales = X4.quantize(X)
    assert codes.shape == (2, 128) and scales.shape == (2, 4)
    assert scales[0].tolist() == [255, 125, 125, 4] and scales[1].tolist() == [125, 125, 255, 4]
    assert not codes[0, :32].any() and not codes[:, 70:].any()
    v = X4.values(codes, scales, 70)
    assert np.isnan(v[0, :32]).all() and np.all(v[0, 32:] == 1)
    pc, ps = X4.pack(codes, scales)
    assert pc.shape == (4, 2, 16) and ps.shape == (1, 2, 4)
    assert pc[1, 0, 0] == (codes[0, 32] | codes[0, 33] << 4) and ps[0, 1, 2] == 255


def test_quantize_idempotent():
    rng = np.random.default_rng(1)
    v = X4.rounded(rng.standard_normal((5, 96)))
    top = np.abs(v.reshape(5, 3, 32)).max(2)
    w = X4.rounded(v)
    same = np.exp2(np.floor(np.log2(top))) * 2 > top     # always: a block's largest value keeps its exponent
    assert same.all() and np.array_equal(v, w)


@pytest.mark.parametrize("p", [0.0, 0.3])
def test_gradients_against_differences(p):
    """Y is linear in L1, in L2 and (with the base's quantisation passed straight
    through) in X, so central differences are exact up to rounding."""
    rng = np.random.default_rng(3)
    M, K, N, r, s = 5, 24, 7, 3, 1.5
    X, dY = rng.standard_normal((M, K)), rng.standard_normal((M, N))
    L1, L2, W = rng.standard_normal((K, r)), rng.standard_normal((r, N)), rng.standard_normal((N, K))
    args = (s, p, 99, 2**33 + 5)
    T = X4.dropped(X, p, 99, 2**33 + 5) @ L1
    dX, dL1, dL2, _ = X4.linear_backward(X, dY, dY, W.T.copy(), L1, L2, *args, T)
    loss = lambda X, L1, L2: float((X4.linear_forward(X, W, L1, L2, *args)[0] * dY).sum())  # noqa: E731
    h = 1e-3
    for g, which, at in ((dX, 0, X), (dL1, 1, L1), (dL2, 2, L2)):
        num = np.empty_like(at)
        for i in np.ndindex(at.shape):
            a = [X, L1, L2]
            up, dn = at.copy(), at.copy()
            up[i] += h
            dn[i] -= h
            a[which] = up
            hi = loss(*a)
            a[which] = dn
            num[i] = (hi - loss(*a)) / (2 * h)
        assert np.allclose(g, num, rtol=1e-8, atol=1e-8)
