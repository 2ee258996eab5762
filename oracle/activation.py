"""Float64 oracle of the expert activation, its MXFP8 checkpoint and its backward pass."""
import numpy as np

from . import formats, mx_quant


def _sigmoid(x):
    e = np.exp(-np.abs(x))  # at most 1: nothing overflows, and no difference cancels for x < 0
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


def forward(z, row_w, gated):
    """z [R, N1] -> h [R, I]."""
    z = np.asarray(z, dtype=np.float64)
    if gated:
        I = z.shape[1] // 2
        a = z[:, :I] * _sigmoid(z[:, :I]) * z[:, I:]
    else:
        a = np.maximum(z, 0.0) ** 2
    return a if row_w is None else _weighted(row_w, a)


def _weighted(w, a):
    w = np.asarray(w, dtype=np.float64)[:, None]
    return np.where(w == 0, 0.0, w * a)


def held(z):
    """The checkpoint's codes, scales and the values they stand for."""
    codes, scales = mx_quant.mx_quantize(np.asarray(z, dtype=np.float64))
    return codes, scales, formats.dequant_mxfp8(codes, scales)


def backward(v, dh, row_w, gated):
    """v: the checkpoint's values [R, N1]; dh [R, I] -> (dz [R, N1], h [R, I], d_row_w [R])."""
    dh = np.asarray(dh, dtype=np.float64)
    w = np.ones(len(dh)) if row_w is None else np.asarray(row_w, dtype=np.float64)
    t = w[:, None] * dh
    if gated:
        I = v.shape[1] // 2
        g, u = v[:, :I], v[:, I:]
        s = _sigmoid(g)
        a = g * s * u
        dz = np.concatenate([t * u * s * (1 + g * (1 - s)), t * g * s], axis=1)
    else:
        r = np.maximum(v, 0.0)
        a = r * r
        dz = 2 * t * r
    out = w == 0
    dz = np.where(out[:, None], 0.0, dz)
    return dz, np.where(out[:, None], 0.0, w[:, None] * a), np.where(out, 0.0, np.sum(dh * a, axis=1))
