"""The training operators together: one step of a bf16 MoE layer with a shared expert against
float64 autograd, and moe_pair_sum against its sum.

Bounds.  Everything between two kernels is rounded to bf16 (2^-9 relative), a handful of times:
2e-2 in norm is generous.  What comes from a checkpoint is up to half an E4M3 step, 2^-4, off in
each of g and u, so a gradient that depends on both is within 2 * 2^-4.
"""
import numpy as np
import pytest

import synth
from helpers import bf16_half_ulp, bf16_to_np
from oracle import formats

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF16, HELD = 2e-2, 0.125


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_grouped_align_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.build()
    m.load()
    return m


def near(got, ref, tol, what):
    e = float((got.double() - ref).norm() / ref.norm())
    assert e <= tol, (what, e)


@pytest.mark.parametrize("T,masked", [(300, False), (700, True), (3, False)])
def test_training_step(moe, T, masked):
    from mixture_experts_grouped_align_gb300.train import TrainLayer
    E, K, I, Is, k = 64, 256, 128, 384, 4
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    W = {"wr": rnd(E, K, std=0.1), "w1": rnd(E, 2 * I, K, std=0.08), "w2": rnd(E, K, I, std=0.08),
         "ws1": rnd(2 * Is, K, std=0.08), "bs1": rnd(2 * Is, std=0.1), "ws2": rnd(K, Is, std=0.08), "bs2": rnd(K, std=0.1)}
    x, dy = rnd(T, K), rnd(T, K)
    mask = (torch.rand(T, generator=g, device="cuda") < 0.8).to(torch.uint8) if masked else None
    L = TrainLayer(W["wr"], W["w1"], W["w2"], W["ws1"], W["bs1"], W["ws2"], W["bs2"], k, max_rows=T + 5, balance_coef=2.0,
                   z_coef=0.5)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    L.forward(x, y)
    L.backward(dy, dx, mask)
    torch.cuda.synchronize()
    assert int(L.status[0]) == 0
    # the same layer in float64 (the routing that the GPU chose)
    D = {n: w.double().requires_grad_(True) for n, w in W.items()}
    xd = x.double().requires_grad_(True)
    logits = xd @ D["wr"].t()
    ids = L.ids[:T].long()
    w = torch.softmax(logits.gather(1, ids), dim=1)
    gu = torch.einsum("tk,tjnk->tjn", xd, D["w1"][ids])
    h = torch.nn.functional.silu(gu[..., :I]) * gu[..., I:]
    routed = (torch.einsum("tji,tjki->tjk", h, D["w2"][ids]) * w[..., None]).sum(1)
    gs = xd @ D["ws1"].t() + D["bs1"]
    yd = (torch.nn.functional.silu(gs[:, :Is]) * gs[:, Is:]) @ D["ws2"].t() + D["bs2"] + routed
    # the token's mask leaves its routing weights' gradient out as well
    live = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask.bool()
    n = int(live.sum())
    counts = torch.bincount(ids[live].reshape(-1), minlength=E)
    p = torch.softmax(logits, dim=1)[live]
    bal = (counts.double() * E / (n * k) * p.mean(0)).sum()
    z = (torch.logsumexp(logits[live], dim=1) ** 2).mean()
    wl = torch.where(live[:, None], w, w.detach())
    routed2 = (torch.einsum("tji,tjki->tjk", h, D["w2"][ids]) * wl[..., None]).sum(1)
    total = ((yd - routed + routed2) * dy.double()).sum() + 2.0 * bal + 0.5 * z
    total.backward()
    near(y, yd, BF16, "y")
    assert torch.equal(L.counts.long(), counts)
    assert abs(float(L.loss[1]) - float(bal)) < 1e-2 * float(bal) and abs(float(L.loss[2]) - float(z)) < 1e-2 * float(z)
    near(L.grads["bs2"], D["bs2"].grad, 1e-5, "bs2")
    near(L.grads["ws2"], D["ws2"].grad, HELD, "ws2")
    near(L.grads["ws1"], D["ws1"].grad, HELD, "ws1")
    near(L.grads["bs1"], D["bs1"].grad, HELD, "bs1")
    near(L.grads["w1"], D["w1"].grad, HELD, "w1")
    near(L.grads["w2t"].transpose(1, 2), D["w2"].grad, HELD, "w2")
    near(L.grads["wr"], D["wr"].grad, HELD, "wr")
    near(dx, xd.grad, HELD, "dx")


@pytest.mark.parametrize("T,k,K,residual", [(1, 1, 8, False), (1, 8, 2880, True), (37, 5, 264, True), (1000, 4, 2880, False),
                                            (513, 33, 136, True)])
def test_pair_sum(moe, T, k, K, residual):
    rng = np.random.default_rng(T + k)
    bf = lambda a: synth.to_bf16_bits(a)  # noqa: E731
    o, r = bf(rng.standard_normal((T * k, K))), bf(rng.standard_normal((T, K)))
    dev = lambda b: torch.from_numpy(b.view(np.int16).copy()).view(torch.bfloat16).cuda()  # noqa: E731
    y = torch.full((T * K + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_pair_sum(dev(o), dev(r) if residual else None, T, k, K, y)
    torch.cuda.synchronize()
    assert bool((y[T * K:] == 7).all())
    ov, rv = formats.bf16_decode(o).reshape(T, k, K), formats.bf16_decode(r) if residual else np.zeros((T, K))
    ref, mag = ov.sum(1) + rv, np.abs(ov).sum(1) + np.abs(rv)
    got = bf16_to_np(y[:T * K]).reshape(T, K)
    assert np.all(np.abs(got - ref) <= bf16_half_ulp(np.abs(ref) + mag * 2.0 ** -18) * (1 + 2.0 ** -6) + (k + 1) * 2.0 ** -24 * mag)


def test_pair_sum_in_place_and_empty(moe):
    o = torch.randn((40, 64), device="cuda").to(torch.bfloat16)
    r = torch.randn((10, 64), device="cuda").to(torch.bfloat16)
    y = torch.empty_like(r)
    moe.moe_pair_sum(o, r, 10, 4, 64, y)
    moe.moe_pair_sum(o, r, 10, 4, 64, r)
    assert moe.moe_pair_sum(None, None, 0, 4, 64, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(r, y)
