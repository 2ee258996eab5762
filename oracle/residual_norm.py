"""Residual addition with dropout and RMS norm, forward and back, in float64.  (Test infrastructure.)

The generator is Philox 4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as
1, 2, 3", SC 2011): ten rounds of two 32 x 32 -> 64-bit products on a 128-bit counter under a 64-bit
key that a Weyl sequence advances.
"""
import numpy as np

from . import mx_quant

_LOW = np.uint64(0xFFFFFFFF)
_32 = np.uint64(32)


def philox(counter, key):
    """counter [..., 4], key [2] (32-bit numbers) -> [..., 4]."""
    c = [np.asarray(counter[..., i], dtype=np.uint64) for i in range(4)]
    k = [np.uint64(key[0]), np.uint64(key[1])]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> _32) ^ c[1] ^ k[0], b & _LOW, (a >> _32) ^ c[3] ^ k[1], a & _LOW]
        k = [(k[0] + np.uint64(0x9E3779B9)) & _LOW, (k[1] + np.uint64(0xBB67AE85)) & _LOW]
    return np.stack(c, axis=-1)


def numbers(n, seed, step, stream):
    """The 16-bit numbers of elements 0..n-1 (n a multiple of 8)."""
    b = np.arange(n // 8, dtype=np.uint64)
    one = np.ones_like(b)
    seed = int(seed) & (2 ** 64 - 1)
    w = philox(np.stack([b & _LOW, b >> _32, one * np.uint64(step & 0xFFFFFFFF), one * np.uint64(stream)], axis=-1),
               (seed & 0xFFFFFFFF, seed >> 32))
    return np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], axis=-1).reshape(-1).astype(np.int64)


def below(p):
    """16-bit numbers under this are dropped."""
    return min(65535, int(np.rint(float(np.float32(p)) * 65536)))


def keep(T, K, p, seed, step, stream):
    """What dropout multiplies a [T, K] tensor by."""
    d = below(p)
    if d == 0:
        return np.ones((T, K))
    return np.where(numbers(T * K, seed, step, stream) >= d, 65536 / (65536 - d), 0.0).reshape(T, K)


def forward(x, residual, weight, eps, kept=1.0, mask=None):
    """-> s, n (before any rounding)."""
    s = np.where(np.asarray(kept) == 0, 0.0, x * kept) if x is not None else 0.0
    s = s + (0.0 if residual is None else residual)
    if mask is not None:
        s = np.where(mask[:, None] != 0, s, 0.0)
    with np.errstate(invalid="ignore"):
        n = s / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps) * weight
    return s, n


def row_quantize(n):
    """-> codes, scales of a row each: max |n| / 448, at least 2^-120."""
    scale = np.maximum(np.abs(n).max(axis=1) / 448, 2.0 ** -120)
    return mx_quant.e4m3_encode(n / scale[:, None]), scale


def backward(d_out, d_stream, s, weight, eps, kept=1.0, mask=None):
    """-> d_residual, d_x, d_weight from the stored stream s."""
    live = np.ones((len(s), 1), bool) if mask is None else mask[:, None] != 0
    s, d_out = np.where(live, s, 0.0), np.where(live, d_out, 0.0)
    r = 1 / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    g = d_out * weight
    ds = r * (g - s * r * r * (g * s).mean(axis=1, keepdims=True))
    ds = ds + (0.0 if d_stream is None else np.where(live, d_stream, 0.0))
    return ds, np.where(np.asarray(kept) == 0, 0.0, ds * kept), (d_out * s * r).sum(axis=0)
