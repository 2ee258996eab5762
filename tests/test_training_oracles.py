"""The float64 oracles of the training operators against things other than themselves: central
differences of the functions they are the gradients of, closed forms and torch's autograd."""
import numpy as np
import pytest

from oracle import activation, router_loss

torch = pytest.importorskip("torch")


def _router_value(x, ids, dw, mask, a, b):
    """The scalar whose gradient router_loss returns: the loss plus sum dw * softmax(chosen)."""
    _, _, (total, _, _), _ = router_loss.router_loss(x, ids, None, None, mask, a, b)
    if dw is not None:
        for t in range(len(x)):
            if mask is None or mask[t]:
                c = x[t][ids[t]]
                w = np.exp(c - c.max())
                total += float((w / w.sum()) @ dw[t])
    return total


@pytest.mark.parametrize("masked,upstream", [(False, False), (True, True)])
def test_router_gradient_is_the_difference_quotient(masked, upstream):
    rng = np.random.default_rng(3)
    T, E, k = 5, 7, 3
    x = rng.standard_normal((T, E))
    ids = np.argsort(-x, axis=1)[:, :k]
    dw = rng.standard_normal((T, k)) if upstream else None
    c = np.take_along_axis(x, ids, axis=1)
    w = np.exp(c - c.max(axis=1, keepdims=True))
    w /= w.sum(axis=1, keepdims=True)
    mask = np.array([1, 0, 1, 1, 1]) if masked else None
    d = router_loss.router_loss(x, ids, w, dw, mask, 0.7, 0.3)[3]
    h = 1e-5
    for t in range(T):
        for e in range(E):
            xp, xm = x.copy(), x.copy()
            xp[t, e] += h
            xm[t, e] -= h
            q = (_router_value(xp, ids, dw, mask, 0.7, 0.3) - _router_value(xm, ids, dw, mask, 0.7, 0.3)) / (2 * h)
            assert abs(q - d[t, e]) < 1e-9, (t, e)


def test_router_closed_forms():
    # equal logits, each token choosing another expert: f = 1, P = 1/E, balance 1, z = log(E)^2
    E = 4
    counts, mean, (total, bal, z), d = router_loss.router_loss(
        np.zeros((E, E)), np.arange(E)[:, None], None, None, None, 2.0, 0.0)
    assert counts.tolist() == [1] * E and np.allclose(mean, 0.25) and abs(bal - 1) < 1e-15
    assert abs(z - np.log(E) ** 2) < 1e-15 and total == 2 * bal and np.allclose(d, 0)
    # every token on one expert with probability one: balance E
    x = np.full((3, E), -40.0)
    x[:, 2] = 0
    _, _, (_, bal, _), _ = router_loss.router_loss(x, np.full((3, 1), 2), None, None, None, 1.0, 0.0)
    assert abs(bal - E) < 1e-12


@pytest.mark.parametrize("gated", [True, False])
def test_activation_gradient_is_autograds(gated):
    rng = np.random.default_rng(4)
    R, I = 6, 32
    v = rng.standard_normal((R, 2 * I if gated else I)) * 3
    dh = rng.standard_normal((R, I))
    w = rng.uniform(0.1, 1, R)
    dz, h, dw = activation.backward(v, dh, w, gated)
    tv = torch.tensor(v, requires_grad=True)
    tw = torch.tensor(w, requires_grad=True)
    act = torch.nn.functional.silu(tv[:, :I]) * tv[:, I:] if gated else torch.relu(tv).square()
    out = tw[:, None] * act
    out.backward(torch.tensor(dh))
    assert np.allclose(dz, tv.grad.numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(dw, tw.grad.numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(h, out.detach().numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(activation.forward(v, w, gated), h)


def test_activation_row_of_weight_zero_is_zeros():
    v = np.full((2, 64), np.nan)
    v[1] = 1.0
    dz, h, dw = activation.backward(v, np.ones((2, 32)), np.array([0.0, 1.0]), True)
    assert not dz[0].any() and not h[0].any() and dw[0] == 0 and np.isfinite(dz[1]).all()


def test_checkpoint_values_are_within_half_a_step():
    """E4M3 has three mantissa bits and saturates at 448 / 512 of the block's binade: a value is
    held within 2^-4 of itself, 1/8 of the block's largest power of two, or half the subnormal step."""
    rng = np.random.default_rng(5)
    z = (rng.standard_normal((4, 96)) * np.exp2(rng.integers(-6, 6, (4, 96)))).astype(np.float32)
    _, _, v = activation.held(z)
    blk = np.abs(z).reshape(4, 3, 32).max(axis=2, keepdims=True)
    top = np.exp2(np.floor(np.log2(blk)))
    err = np.abs(v - z).reshape(4, 3, 32)
    a = np.abs(z).reshape(4, 3, 32)
    bound = np.where(a >= 1.75 * top, a - 1.75 * top, np.maximum(a * 2.0 ** -4, top * 2.0 ** -18))
    assert np.all(err <= bound * (1 + 1e-12))
