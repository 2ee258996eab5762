"""Float64 oracle of the router losses and of the logits' gradient."""
import numpy as np


def router_loss(logits, ids, w, dw, mask, balance_coef, z_coef):
    """logits [T, E], ids [T, k], w / dw [T, k] or None, mask [T] or None ->
    (counts [E], prob_mean [E], (total, balance, z), d_logits [T, E])."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    k = ids.shape[1]
    counts = np.zeros(E, dtype=np.int64)
    p = np.zeros((T, E))
    lse = np.zeros(T)
    rows = [t for t in range(T) if mask is None or mask[t]]
    n = len(rows)
    for t in rows:
        for e in ids[t]:
            if 0 <= e < E:
                counts[e] += 1
        m = x[t].max()
        if m == -np.inf:
            continue
        ex = np.exp(x[t] - m)
        p[t] = ex / ex.sum()
        lse[t] = m + np.log(ex.sum())
    d = np.zeros((T, E))
    if n == 0:
        return counts, np.zeros(E), (0.0, 0.0, 0.0), d
    f = counts * (E / (n * k))
    mean = p.sum(axis=0) / n
    balance, z = float(f @ mean), float((lse ** 2).sum() / n)
    for t in rows:
        if p[t].sum() == 0:
            continue
        d[t] = balance_coef / n * p[t] * (f - f @ p[t]) + 2 * z_coef / n * lse[t] * p[t]
        if dw is not None:
            good = [j for j in range(k) if 0 <= ids[t, j] < E]
            s = sum(float(w[t, j]) * float(dw[t, j]) for j in good)
            for j in good:
                d[t, ids[t, j]] += float(w[t, j]) * (float(dw[t, j]) - s)
    return counts, mean, (balance_coef * balance + z_coef * z, balance, z), d
