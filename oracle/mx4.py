"""CPU oracle of the microscaled 4-bit layer and of the adapter dropout (TEST
INFRASTRUCTURE ONLY, like the rest of this package).

Written from the definitions: E2M1 elements with one power-of-two scale per 32
(OCP Microscaling Formats v1.0), the nearest element found by comparing with
every E2M1 value; Philox4x32 (Salmon et al., SC 2011) in unsigned 64-bit words;
the layer in float64 with its two rounding points (the packed operands and, as a
result, T).
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK, PAD = 32, 128


def quantize(X):
    """Codes [rows, Kp] (0..15) and scale bytes [rows, Kp/32] of the rows of X (finite or not)."""
    X = np.asarray(X, np.float64)
    rows, cols = X.shape
    kp = -(-cols // PAD) * PAD
    v = np.zeros((rows, kp))
    v[:, :cols] = X
    v = v.reshape(rows, kp // BLOCK, BLOCK)
    bad = ~np.isfinite(v).all(2)
    top = np.where(bad, 0.0, np.abs(np.where(np.isfinite(v), v, 0.0)).max(2))
    e = np.frexp(top)[1] - 1 - 2                       # floor(log2 top) - 2
    e = np.where(top == 0, -123, np.maximum(e, -123))
    n = np.abs(np.where(bad[..., None], 0.0, v)) / np.exp2(e)[..., None]
    dist = np.abs(n[..., None] - E2M1)
    best = dist.min(-1, keepdims=True)
    # of two equally near values the one with the even code
    code = np.argmin(np.where(dist == best, np.arange(8) % 2, 2), -1)
    code = np.where(bad[..., None], 0, code + 8 * np.signbit(v))
    byte = np.where(bad, 255, e + 127)
    return code.reshape(rows, kp).astype(np.uint8), byte.astype(np.uint8)


def values(codes, scales, cols):
    """float64 [rows, cols] that codes and scale bytes stand for."""
    mag = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.exp2(scales.astype(np.float64) - 127)
    s[scales == 255] = np.nan
    return (mag * np.repeat(s, BLOCK, axis=1))[:, :cols]


def pack(codes, scales):
    """The packed layout: codes [Kp/32, rows, 16], scales [Kp/128, rows, 4]."""
    rows, kp = codes.shape
    by = (codes[:, 0::2] | (codes[:, 1::2] << 4)).reshape(rows, kp // BLOCK, 16)
    return np.ascontiguousarray(by.transpose(1, 0, 2)), np.ascontiguousarray(
        scales.reshape(rows, kp // PAD, 4).transpose(1, 0, 2))


def rounded(X):
    """The values that the rows of X stand for once quantised."""
    return values(*quantize(X), np.shape(X)[1])


def philox4x32(counter, key, rounds=7):
    """Output words of Philox4x32: counter a list of four arrays (or numbers) below 2^32, key two numbers."""
    low = np.uint64(0xFFFFFFFF)
    c = [np.asarray(x, np.uint64) for x in counter]
    k = [int(key[0]), int(key[1])]
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]),
             a & low]
        k = [(k[0] + 0x9E3779B9) % 2**32, (k[1] + 0xBB67AE85) % 2**32]
    return c


def cut_of(p):
    return min(int(np.floor(p * 65536 + 0.5)), 65535)


def keep(rows, cols, p, seed, offset):
    """True where element (m, k) is kept."""
    octs = -(-cols // 8)
    q, m = np.meshgrid(np.arange(octs), np.arange(rows))
    w = philox4x32([q, m, offset % 2**32, offset // 2**32], (seed % 2**32, seed // 2**32))
    w = np.stack([np.broadcast_to(x, q.shape) for x in w], -1)          # [rows, octs, 4]
    u = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(rows, octs * 8)[:, :cols]
    return u >= cut_of(p)


def dropped(X, p, seed, offset):
    """D o X in float64."""
    X = np.asarray(X, np.float64)
    c = cut_of(p)
    return np.where(keep(*X.shape, p, seed, offset), X * (65536 / (65536 - c)), 0.0)


def linear_forward(X, Wv, L1, L2, s, p, seed, offset, T=None):
    """(Y, T) unrounded in float64: X as given, Wv the values of the base; the adapter term from `T` when given."""
    Tx = dropped(X, p, seed, offset) @ np.asarray(L1, np.float64)
    return X @ Wv.T + s * ((Tx if T is None else T) @ L2), Tx


def linear_backward(X, dY, dYv, Wtv, L1, L2, s, p, seed, offset, T):
    """(dX, dL1, dL2, G) in float64: dYv the gradient that the base sees, Wtv [K, N] the base's values."""
    G = s * (dY @ L2.T)
    branch = np.where(keep(*X.shape, p, seed, offset), (G @ L1.T) * (65536 / (65536 - cut_of(p))), 0.0)
    return dYv @ Wtv.T + branch, dropped(X, p, seed, offset).T @ G, s * (T.T @ dY), G
