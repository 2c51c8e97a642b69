"""The oracle of the 8-bit activations, the norm and the gated product against pins and differences (CPU)."""
import numpy as np
import pytest

import oracle as O

X8 = O.mx8


def test_every_code_keeps_its_value():
    assert X8.E4M3[1] == 2.0**-9 and X8.E4M3[8] == 2.0**-6 and X8.E4M3[126] == 448 and X8.E4M3[120] == 256
    assert np.array_equal(X8.nearest(X8.E4M3), np.arange(127))
    mid = (X8.E4M3[1:] + X8.E4M3[:-1]) / 2
    even = np.arange(126) + np.arange(126) % 2
    assert np.array_equal(X8.nearest(mid), even)
    assert np.array_equal(X8.nearest(mid * (1 + 1e-12)), np.arange(1, 127))
    assert np.array_equal(X8.nearest(mid * (1 - 1e-12)), np.arange(126))


@pytest.mark.parametrize("top,e", [(448.0, 0), (448.0000001, 1), (256.0, 0), (224.0, -1), (1.75, -8), (1.0, -8),
                                   (1.75 * 2.0**-108, -117 + 1), (2.0**-120, -117), (0.0, -117), (3.3e38, 120)])
def test_scale_is_the_least_that_holds_the_block(top, e):
    x = np.zeros((1, 40))
    x[0, 3] = -top
    assert X8.exponents(x).tolist() == [[e, -117]]


def test_rounding_stays_within_half_a_step():
    x = np.random.default_rng(0).standard_normal((50, 77)) * np.exp2(np.arange(50) - 25)[:, None]
    e = np.repeat(X8.exponents(x), 32, 1)[:, :77]
    err = np.abs(X8.rounded(x) - x)
    assert (err <= np.maximum(2.0**-4 * np.abs(x), 2.0**-10 * np.exp2(e))).all()


def test_blocks_that_are_not_finite():
    x = np.ones((3, 64))
    x[0, 5], x[1, 40], x[2, 0] = np.inf, np.nan, -np.inf
    codes, scales = X8.quantize(x)
    assert scales.tolist() == [[255, 119], [119, 255], [255, 119]]
    v = X8.values(codes, scales, 64)
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 1).all() and np.isnan(v[1, 32:]).all()


def _differences(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        up = f()
        x[i] = keep - h
        g[i] = (up - f()) / (2 * h)
        x[i] = keep
    return g


def test_norm_gradients_against_differences():
    rng = np.random.default_rng(1)
    S, w, dY, dS = rng.standard_normal((3, 7)), 1 + rng.random(7), rng.standard_normal((3, 7)), rng.standard_normal((3, 7))
    loss = lambda: (X8.norm_forward(S, w, 1e-3) * dY).sum() + (S * dS).sum()  # noqa: E731
    dX, dw = X8.norm_backward(dY, S, w, 1e-3, dS)
    assert np.allclose(dX, _differences(loss, S), atol=1e-8)
    assert np.allclose(dw, _differences(loss, w), atol=1e-8)


def test_swiglu_gradients_against_differences():
    rng = np.random.default_rng(2)
    M, K, F, r, s = 3, 5, 4, 2, 1.5
    X, W = rng.standard_normal((M, K)), rng.standard_normal((2 * F, K))
    L1, L2, dH = rng.standard_normal((2, K, r)), rng.standard_normal((2, r, F)), rng.standard_normal((M, F))
    loss = lambda: (X8.swiglu_forward(X, W, L1, L2, s)[0] * dH).sum()  # noqa: E731
    H, G, U, T = X8.swiglu_forward(X, W, L1, L2, s)
    dX, dL1, dL2, _, _ = X8.swiglu_backward(X, dH, G, U, W, L1, L2, T, s)
    for got, x in ((dX, X), (dL1, L1), (dL2, L2)):
        assert np.allclose(got, _differences(loss, x), atol=1e-6, rtol=1e-6)
