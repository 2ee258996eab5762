"""Low-rank adapters of many requests beside a dense product, in float64.  (Test infrastructure.)"""
import numpy as np


def row_adapters(M, row_offsets, adapter):
    """A row's adapter: -1 none, -2 of no request."""
    ids = np.full(M, -2)
    for i, a in enumerate(adapter):
        ids[row_offsets[i]:row_offsets[i + 1]] = a
    return ids


def adapter_gemm(x, a, b, scale, row_offsets, adapter, base):
    """-> out, and the sum of magnitudes of what is added (rows of no request: base)."""
    ids = row_adapters(len(x), row_offsets, adapter)
    out, mag = base.astype(np.float64).copy(), np.zeros(base.shape)
    for l in set(ids[ids >= 0]):
        m = ids == l
        s = 1.0 if scale is None else scale[l]
        v = x[m] @ a[l].T
        out[m] += s * (v @ b[l].T)
        mag[m] = abs(s) * ((np.abs(x[m]) @ np.abs(a[l]).T) @ np.abs(b[l]).T)
    return out, mag
