"""Float64 oracle of one training step of a MoE layer with a dense shared expert.

The activations' gradients, the activations of the weight gradients and the routing weights'
gradients are taken at the values that ``held`` gives for the bf16 pre-activations (an MXFP8
checkpoint's values; the identity differentiates the step exactly); the forward pass uses the
pre-activations themselves.
"""
import numpy as np

from .activation import _sigmoid


def bf16_round(a):
    """float64 -> the nearest bf16 value, ties to even (8 significant bits; no subnormals met)."""
    m, e = np.frexp(np.asarray(a, dtype=np.float64))
    return np.ldexp(np.rint(m * 256.0), e - 8)


def _swiglu(v):
    g, u = np.split(v, 2, axis=1)
    return g * _sigmoid(g) * u


def _swiglu_grad(v, d):
    g, u = np.split(v, 2, axis=1)
    s = _sigmoid(g)
    return np.concatenate([d * u * s * (1 + g * (1 - s)), d * g * s], axis=1)


def forward(W, x, ids):
    """W: wr [E, K], w1 [E, 2I, K], w2 [E, K, I], ws1 [2Is, K], bs1, ws2 [K, Is], bs2; x [T, K];
    ids [T, k] -> (y [T, K], what ``backward`` takes)."""
    T, k = ids.shape
    logits = x @ W["wr"].T
    top = np.take_along_axis(logits, ids, axis=1)
    w = np.exp(top - top.max(axis=1, keepdims=True))
    w /= w.sum(axis=1, keepdims=True)
    gu = np.zeros((T * k, W["w1"].shape[1]))
    y = np.zeros_like(x)
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        gu[t * k + j] = x[t] @ W["w1"][e].T
        np.add.at(y, t, (w[t, j][:, None] * _swiglu(gu[t * k + j])) @ W["w2"][e].T)
    gs = x @ W["ws1"].T + W["bs1"]
    y += _swiglu(gs) @ W["ws2"].T + W["bs2"]
    return y, {"x": x, "ids": ids, "logits": logits, "w": w, "gu": gu, "gs": gs}


def backward(W, kept, dy, balance_coef, z_coef, mask=None, held=lambda v: v):
    """dy [T, K] -> gradients of every weight, "dx", "d_logits" [T, E], "loss" (total, balance, z)
    and "counts".  mask [T]: 0 for tokens that the losses and the routing weights' gradient leave
    out."""
    x, ids, logits, w = kept["x"], kept["ids"], kept["logits"], kept["w"]
    T, k = ids.shape
    E = logits.shape[1]
    v, vs = held(kept["gu"]), held(kept["gs"])
    g = {n: np.zeros_like(a) for n, a in W.items()}
    dx = np.zeros_like(x)
    dw = np.zeros((T, k))
    a = _swiglu(v)
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        p, wt = t * k + j, w[t, j][:, None]
        dh = dy[t] @ W["w2"][e]
        dgu = _swiglu_grad(v[p], wt * dh)
        dw[t, j] = (dh * a[p]).sum(axis=1)
        g["w2"][e] = dy[t].T @ (wt * a[p])
        g["w1"][e] = dgu.T @ x[t]
        np.add.at(dx, t, dgu @ W["w1"][e])
    dgs = _swiglu_grad(vs, dy @ W["ws2"])
    g["ws2"], g["bs2"] = dy.T @ _swiglu(vs), dy.sum(axis=0)
    g["ws1"], g["bs1"] = dgs.T @ x, dgs.sum(axis=0)
    dx += dgs @ W["ws1"]
    live = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    n = max(int(live.sum()), 1)
    counts = np.bincount(ids[live].reshape(-1), minlength=E)
    m = logits.max(axis=1, keepdims=True)
    p = np.exp(logits - m)
    lse = m + np.log(p.sum(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    f = counts * (E / (n * k))
    balance, z = float(f @ p[live].sum(axis=0)) / n, float((lse[live] ** 2).sum()) / n
    dl = balance_coef / n * p * (f - (p @ f)[:, None]) + 2 * z_coef / n * lse * p
    dr = w * (dw - (w * dw).sum(axis=1, keepdims=True))
    np.add.at(dl, (np.arange(T)[:, None], ids), dr)
    dl[~live] = 0.0
    g["wr"] = dl.T @ x
    dx += dl @ W["wr"]
    return {**g, "dx": dx, "d_logits": dl, "loss": (balance_coef * balance + z_coef * z, balance, z), "counts": counts}
