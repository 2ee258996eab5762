"""Training steps of TrainLayer on the GPU against the float64 oracle at the checkpoint's values.

Bounds.  A value stored between two kernels in bf16 is within 2^-9 of itself, in norm too.  No
output has more than eight such roundings before it, so 8 * 2^-9 = 1.6e-2; a pre-activation whose
fp32 sum lies at a rounding's border may fall to the checkpoint's next value, for fewer than one in
10^4 of them: 1e-3 in norm.  2e-2 holds for both together.
"""
import numpy as np
import pytest

from helpers import bf16_to_np
from oracle import activation, train_step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TOL = 2e-2


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_grouped_align_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.build()
    m.load()
    return m


def held(v):
    return activation.held(train_step.bf16_round(v))[2]


def make(seed, E, K=256, I=128, Is=384):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    W = {"wr": rnd(E, K, std=0.1), "w1": rnd(E, 2 * I, K, std=0.08), "w2": rnd(E, K, I, std=0.08),
         "ws1": rnd(2 * Is, K, std=0.08), "bs1": rnd(2 * Is, std=0.1), "ws2": rnd(K, Is, std=0.08), "bs2": rnd(K, std=0.1)}
    return W, rnd


def layer(W, k, rows, coef=(2.0, 0.5), **kw):
    from mixture_experts_grouped_align_gb300.train import TrainLayer
    return TrainLayer(W["wr"], W["w1"], W["w2"], W["ws1"], W["bs1"], W["ws2"], W["bs2"], k, max_rows=rows,
                      balance_coef=coef[0], z_coef=coef[1], **kw)


def near(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    e = float(np.linalg.norm(got - ref) / np.linalg.norm(ref))
    assert e <= tol, (what, e)


def compare(L, W, x, dy, y, dx, mask=None, full=None):
    """The layer's results of a step against the oracle's (``full``: other expected gradients)."""
    T = len(x)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    Wd, xd, dyd, ids = {n: f(w) for n, w in W.items()}, f(x), f(dy), L.ids[:T].cpu().numpy().astype(np.int64)
    ry, kept = train_step.forward(Wd, xd, ids)
    r = full(Wd, kept, dyd) if full else train_step.backward(Wd, kept, dyd, *L.coef, mask, held)
    if y is not None:
        near(bf16_to_np(y), ry, TOL, "y")
    for n in ("wr", "w1", "ws1", "bs1", "ws2", "bs2"):
        if np.any(r[n]):
            near(f(L.grads[n]), r[n], TOL, n)
        else:
            assert not L.grads[n].any(), n
    near(f(L.grads["w2t"].transpose(1, 2)), r["w2"], TOL, "w2") if np.any(r["w2"]) else None
    near(bf16_to_np(dx), r["dx"], TOL, "dx")
    assert np.array_equal(L.counts.cpu().numpy(), r["counts"])
    near(L.loss.cpu().numpy(), r["loss"], 1e-4, "loss")
    assert int(L.status[0]) == 0
    return r


def step(L, x, dy, mask=None):
    y, dx = torch.empty_like(x), torch.empty_like(x)
    L.forward(x, y)
    L.backward(dy, dx, mask)
    torch.cuda.synchronize()
    return y, dx


def test_weights_changed_between_steps(moe):
    """An optimiser's in-place update: the second step's gradients are those of the new weights."""
    T, k = 300, 4
    W, rnd = make(1, 64)
    L = layer(W, k, T)
    for _ in range(2):
        x, dy = rnd(T, 256), rnd(T, 256)
        y, dx = step(L, x, dy)
        compare(L, W, x, dy, y, dx)
        for n, w in W.items():
            w.copy_(w + rnd(*w.shape, std=float(w.float().std())))


@pytest.mark.parametrize("T,masked", [(300, False), (700, True), (3, False), (1, False)])
def test_step_at_the_checkpoint_s_values(moe, T, masked):
    W, rnd = make(T, 64)
    x, dy = rnd(T, 256), rnd(T, 256)
    mask = torch.from_numpy((np.random.default_rng(T).random(T) < 0.8).astype(np.uint8)).cuda() if masked else None
    L = layer(W, 4, T + 5)
    y, dx = step(L, x, dy, mask)
    compare(L, W, x, dy, y, dx, None if mask is None else mask.cpu().numpy())


@pytest.mark.parametrize("coef", [(2.0, 0.0), (0.0, 0.5), (2.0, 0.5)])
def test_gradients_of_the_losses_alone(moe, coef):
    """dy = 0: what reaches x and the router's weights comes from the balance and z losses."""
    T = 300
    W, rnd = make(5, 64)
    x, dy = rnd(T, 256), torch.zeros((T, 256), dtype=torch.bfloat16, device="cuda")
    L = layer(W, 4, T, coef)
    y, dx = step(L, x, dy)
    r = compare(L, W, x, dy, y, dx)
    # fp32 logits within 1e-6 of their magnitude, probabilities and gradients with them
    near(L.d_logits[:T].double().cpu().numpy(), r["d_logits"], 1e-4, "d_logits")


def test_padding_rows_have_no_part_in_any_gradient(moe):
    """Tokens of mask 0 whose dy is zero, as padding's is: every gradient is the whole one."""
    T, k = 500, 4
    W, rnd = make(6, 64)
    x, dy = rnd(T, 256), rnd(T, 256)
    mask = (np.random.default_rng(6).random(T) < 0.7).astype(np.uint8)
    dy[torch.from_numpy(mask == 0).cuda()] = 0
    L = layer(W, k, T)

    def full(Wd, kept, dyd):  # the output's gradient through every weight, and the losses' alone
        a = train_step.backward(Wd, kept, dyd, 0.0, 0.0, None, held)
        b = train_step.backward(Wd, kept, np.zeros_like(dyd), *L.coef, mask, held)
        return {n: b[n] if n in ("loss", "counts") else a[n] + b[n] for n in a}

    y, dx = step(L, x, dy, torch.from_numpy(mask).cuda())
    compare(L, W, x, dy, y, dx, full=full)


@pytest.mark.parametrize("E,k", [(6, 2), (8, 2), (60, 6), (160, 8)])
def test_any_number_of_experts(moe, E, k):
    T = 257
    W, rnd = make(E, E)
    L = layer(W, k, T)
    for _ in range(2):
        x, dy = rnd(T, 256), rnd(T, 256)
        y, dx = step(L, x, dy)
        compare(L, W, x, dy, y, dx)
        W["wr"].copy_(rnd(E, 256, std=0.1))


def test_layers_that_share_scratch(moe):
    """Two layers of different sizes, both forward before either goes back."""
    k, T = 4, 300
    (Wa, rnd), (Wb, _) = make(21, 64), make(22, 60, I=192, Is=128)
    A = layer(Wa, k, T)
    B = layer(Wb, k, T + 50, scratch=A.scratch)
    x, dy = [rnd(T, 256) for _ in range(2)], [rnd(T, 256) for _ in range(2)]
    y, dx = [torch.empty_like(x[0]) for _ in range(2)], [torch.empty_like(x[0]) for _ in range(2)]
    for _ in range(2):
        A.forward(x[0], y[0])
        B.forward(x[1], y[1])
        B.backward(dy[1], dx[1])
        A.backward(dy[0], dx[0])
        torch.cuda.synchronize()
        compare(A, Wa, x[0], dy[0], y[0], dx[0])
        compare(B, Wb, x[1], dy[1], y[1], dx[1])


def test_a_layer_holds_checkpoints_and_not_pre_activations(moe):
    """What a further layer holds beside its gradients is below the bf16 pre-activations' bytes."""
    E, K, I, Is, k, T = 8, 256, 512, 512, 8, 4096
    W, _ = make(23, E, K, I, Is)
    A = layer(W, k, T)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    B = layer(W, k, T, scratch=A.scratch)
    more = torch.cuda.memory_allocated() - before
    grads = sum(t.numel() * 4 for t in B.grads.values())
    bf16 = 2 * (T * k * 2 * I + T * 2 * Is)
    assert more - grads < 0.6 * bf16, (more, grads, bf16)
    assert A.scratch.nbytes() > bf16


def test_a_step_without_tokens(moe):
    W, rnd = make(24, 64)
    L = layer(W, 4, 10)
    x, dy = rnd(10, 256), rnd(10, 256)
    step(L, x, dy)  # leaves gradients behind
    y, dx = step(L, x[:0], dy[:0])
    assert y.shape == dx.shape == (0, 256) and int(L.status[0]) == 0
    assert not L.loss.any() and not L.counts.any() and not any(g.any() for g in L.grads.values())
    y, dx = step(L, x, dy)
    compare(L, W, x, dy, y, dx)
