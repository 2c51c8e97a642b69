"""CPU oracle of the 8-bit activations, of the norm and of the gated product (TEST
INFRASTRUCTURE ONLY, like the rest of this package).

Written from the definitions in float64: E4M3 elements with one power-of-two scale per
32 (OCP Microscaling Formats v1.0), the nearest found in the list of every E4M3 value;
the norm and the gated product as functions of real numbers, and their derivatives.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
# magnitudes of the codes 0 .. 126 (127 is NaN): 3 mantissa bits, bias 7, subnormals in steps of 2^-9
E4M3 = np.array([c / 512 if c < 8 else 2.0 ** (c // 8 - 7) * (1 + c % 8 / 8) for c in range(127)])


def nearest(v):
    """Codes (magnitudes) nearest to v >= 0, ties to the even code, at most 448."""
    v = np.minimum(np.asarray(v, np.float64), E4M3[-1])
    lo = np.clip(np.searchsorted(E4M3, v, side="right") - 1, 0, 125)
    d0, d1 = v - E4M3[lo], E4M3[lo + 1] - v
    return lo + ((d1 < d0) | ((d1 == d0) & (lo % 2 == 1)))


def exponents(X, cols=None):
    """Scale exponents [rows, Kp/32] of finite rows."""
    X = np.asarray(X, np.float64)
    rows, n = X.shape
    kp = -(-n // BLOCK) * BLOCK
    top = np.abs(np.pad(X, ((0, 0), (0, kp - n)))).reshape(rows, -1, BLOCK).max(2)
    e = np.full(top.shape, -200)
    while (low := 448.0 * np.exp2(e) < top).any():
        e = e + low
    return np.maximum(e, -117)


def quantize(X, e=None):
    """Codes [rows, Kp] and scale bytes [rows, Kp/32] of the rows of X (finite or not), with exponents `e` if given."""
    X = np.asarray(X, np.float64)
    rows, cols = X.shape
    kp = -(-cols // BLOCK) * BLOCK
    v = np.pad(X, ((0, 0), (0, kp - cols))).reshape(rows, -1, BLOCK)
    bad = ~np.isfinite(v).all(2)
    fin = np.where(bad[..., None], 0.0, v)
    if e is None:
        e = exponents(fin.reshape(rows, kp))
    code = nearest(np.abs(fin) / np.exp2(e)[..., None]) + 128 * np.signbit(fin)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(rows, kp).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, scales, cols):
    """float64 [rows, cols] that codes and scale bytes stand for."""
    mag = E4M3[np.minimum(codes & 127, 126)] * np.where(codes & 128, -1.0, 1.0)
    s = np.exp2(scales.astype(np.float64) - 127)
    s[scales == 255] = np.nan
    return (mag * np.repeat(s, BLOCK, axis=1))[:, :cols]


def rounded(X, e=None):
    """The values that the rows of X stand for once packed."""
    return values(*quantize(X, e), np.shape(X)[1])


def norm_forward(S, w, eps):
    return S / np.sqrt((S * S).mean(1, keepdims=True) + eps) * w


def norm_backward(dY, S, w, eps, dS=0.0):
    """(dX, dw) of norm_forward at S, dS the gradient that reaches S beside it."""
    inv = 1 / np.sqrt((S * S).mean(1, keepdims=True) + eps)
    d = dY * w
    return inv * d - inv**3 * S * (S * d).mean(1, keepdims=True) + dS, (S * inv * dY).sum(0)


def sigmoid(g):
    return 1 / (1 + np.exp(-g))


def swiglu_forward(X, W, L1, L2, s):
    """(H, G, U, T): W [2 F, K], L1 [2, K, r], L2 [2, r, F]."""
    F = W.shape[0] // 2
    T = [X @ L1[h] for h in range(2)]
    G, U = (X @ W[h * F:(h + 1) * F].T + s * (T[h] @ L2[h]) for h in range(2))
    return G * sigmoid(G) * U, G, U, np.stack(T)


def swiglu_dz(dH, G, U):
    sig = sigmoid(G)
    return np.stack([dH * U * sig * (1 + G * (1 - sig)), dH * G * sig])


def swiglu_backward(X, dH, G, U, W, L1, L2, T, s):
    """(dX, dL1, dL2, dZ, B)."""
    F = W.shape[0] // 2
    dZ = swiglu_dz(dH, G, U)
    B = np.stack([s * dZ[h] @ L2[h].T for h in range(2)])
    dX = sum(dZ[h] @ W[h * F:(h + 1) * F] + B[h] @ L1[h].T for h in range(2))
    return dX, np.stack([X.T @ B[h] for h in range(2)]), s * np.stack([T[h].T @ dZ[h] for h in range(2)]), dZ, B
