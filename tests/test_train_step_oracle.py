"""The training step's oracle, at unquantised pre-activations, against torch's autograd."""
import numpy as np
import pytest

from oracle import train_step

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("masked", [False, True])
def test_gradients_are_autograd_s(masked):
    E, K, I, Is, k, T = 6, 12, 8, 10, 2, 17
    rng = np.random.default_rng(1)
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    W = {"wr": n(E, K), "w1": n(E, 2 * I, K), "w2": n(E, K, I), "ws1": n(2 * Is, K), "bs1": n(2 * Is), "ws2": n(K, Is),
         "bs2": n(K)}
    x, dy = n(T, K), n(T, K)
    mask = (rng.random(T) < 0.7).astype(np.uint8) if masked else None
    ids = np.argsort(-(x @ W["wr"].T), axis=1)[:, :k]
    y, kept = train_step.forward(W, x, ids)
    got = train_step.backward(W, kept, dy, 0.7, 0.3, mask)
    D = {m: torch.from_numpy(a).requires_grad_(True) for m, a in W.items()}
    xd, it = torch.from_numpy(x).requires_grad_(True), torch.from_numpy(ids)
    logits = xd @ D["wr"].t()
    logits.retain_grad()
    w = torch.softmax(logits.gather(1, it), dim=1)
    live = torch.ones(T, dtype=torch.bool) if mask is None else torch.from_numpy(mask).bool()
    wl = torch.where(live[:, None], w, w.detach())
    swiglu = lambda v: torch.nn.functional.silu(v.chunk(2, -1)[0]) * v.chunk(2, -1)[1]  # noqa: E731
    h = swiglu(torch.einsum("tk,tjnk->tjn", xd, D["w1"][it]))
    out = (torch.einsum("tji,tjki->tjk", h, D["w2"][it]) * wl[..., None]).sum(1)
    out = out + swiglu(xd @ D["ws1"].t() + D["bs1"]) @ D["ws2"].t() + D["bs2"]
    counts = torch.bincount(it[live].reshape(-1), minlength=E)
    nl = int(live.sum())
    bal = (counts.double() * E / (nl * k) * torch.softmax(logits[live], 1).mean(0)).sum()
    z = (torch.logsumexp(logits[live], 1) ** 2).mean()
    ((out * torch.from_numpy(dy)).sum() + 0.7 * bal + 0.3 * z).backward()
    close = lambda a, b: np.testing.assert_allclose(a, b, rtol=1e-10, atol=1e-10)  # noqa: E731
    close(y, out.detach().numpy())
    for m in W:
        close(got[m], D[m].grad.numpy())
    close(got["dx"], xd.grad.numpy())
    close(got["d_logits"], logits.grad.numpy())
    close(got["loss"], (0.7 * bal.item() + 0.3 * z.item(), bal.item(), z.item()))
    assert np.array_equal(got["counts"], counts.numpy())


def test_bf16_rounding():
    v = np.random.default_rng(2).standard_normal(10000) * 100
    v[:2] = 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8  # ties
    want = torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16).double().numpy()
    assert np.array_equal(train_step.bf16_round(v.astype(np.float32)), want)
