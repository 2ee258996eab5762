"""The norm, the adapters and the layers together: blocks in a residual stream, in training against
float64 autograd and in serving against the float64 oracle of each step.

Bounds as for the training layer: what lies between two kernels is bf16, 2e-2 in norm is generous, and
what depends on two values of an MXFP8 checkpoint is within 2 * 2^-4; the second block's gradients pass
through both.
"""
import numpy as np
import pytest

import synth
from helpers import bf16_to_np, dev
from oracle import adapter as adapter_oracle
from oracle import formats, layer as layer_oracle, residual_norm, route
from oracle.train_step import bf16_round

torch = pytest.importorskip("torch")
BF16, HELD = 2e-2, 0.125


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_grouped_align_gb300 as m
    m.build()
    m.load()
    return m


def near(got, ref, tol, what):
    e = float((got.double() - ref).norm() / ref.norm())
    assert e <= tol, (what, e)


def layer64(D, x, ids, I, Is, live):
    """The training layer in float64, with the routing that the GPU chose; a token that is not live has constant
    routing weights."""
    logits = x @ D["wr"].t()
    w = torch.softmax(logits.gather(1, ids), dim=1)
    w = torch.where(live[:, None], w, w.detach())
    gu = torch.einsum("tk,tjnk->tjn", x, D["w1"][ids])
    h = torch.nn.functional.silu(gu[..., :I]) * gu[..., I:]
    gs = x @ D["ws1"].t() + D["bs1"]
    y = (torch.nn.functional.silu(gs[:, :Is]) * gs[:, Is:]) @ D["ws2"].t() + D["bs2"]
    return y + (torch.einsum("tji,tjki->tjk", h, D["w2"][ids]) * w[..., None]).sum(1)


@pytest.mark.gpu
@pytest.mark.parametrize("T,masked,f32,p", [(150, False, False, 0.1), (90, True, True, 0.25), (3, False, True, 0.0)])
def test_training_blocks(moe, T, masked, f32, p):
    from mixture_experts_grouped_align_gb300.train import TrainBlock, TrainLayer
    E, K, I, Is, k, eps = 64, 256, 64, 128, 4, 1e-5
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    st = torch.float32 if f32 else torch.bfloat16
    rng = torch.tensor([12345 + T, 7], device="cuda")
    Ws, blocks, scratch = [], [], None
    for i in range(2):
        W = {"wr": rnd(E, K, std=0.1), "w1": rnd(E, 2 * I, K, std=0.08), "w2": rnd(E, K, I, std=0.1),
             "ws1": rnd(2 * Is, K, std=0.08), "bs1": rnd(2 * Is, std=0.1), "ws2": rnd(K, Is, std=0.08), "bs2": rnd(K, std=0.1)}
        L = TrainLayer(*(W[n] for n in ("wr", "w1", "w2", "ws1", "bs1", "ws2", "bs2")), k, T + 3, 0.0, 0.0, scratch=scratch)
        scratch = L.scratch
        W["norm"] = (1 + 0.2 * torch.randn(K, generator=g, device="cuda")).to(torch.bfloat16)
        Ws.append(W)
        blocks.append(TrainBlock(L, W["norm"], eps, p, rng, i, f32))
    res = rnd(T, K).to(st)
    mask = (torch.rand(T, generator=g, device="cuda") < 0.8).to(torch.uint8) if masked else None
    live = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask.bool()
    y = [torch.empty((T, K), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    s = [None, None]
    _, s[0] = blocks[0].forward(None, res, y[0], mask)
    _, s[1] = blocks[1].forward(y[0], s[0], y[1], mask)
    dy = rnd(T, K)
    dst = rnd(T, K).to(st)
    dy[~live] = 0
    dst[~live] = 0
    d_stream, d_branch = dst.clone(), torch.empty_like(dy)
    blocks[1].backward(dy, d_stream, d_stream, d_branch)           # in place
    d_res = torch.empty_like(res)
    blocks[0].backward(d_branch, d_stream, d_res)
    torch.cuda.synchronize()
    # the same in float64
    Ds = [{n: w.double().requires_grad_(True) for n, w in W.items()} for W in Ws]
    r64 = res.double().requires_grad_(True)
    stream, branch, outs = r64, None, []
    for i in range(2):
        if branch is not None:
            kept = residual_norm.keep(T, K, p, 12345 + T, 7, i)
            stream = stream + branch * torch.from_numpy(kept).cuda()
        stream = torch.where(live[:, None], stream, 0.0)
        n = stream / torch.sqrt((stream ** 2).mean(1, keepdim=True) + eps) * Ds[i]["norm"]
        branch = layer64(Ds[i], n, blocks[i].layer.ids[:T].long(), I, Is, live)
        outs.append((branch, stream))
    ((outs[1][0] * dy.double()).sum() + (outs[1][1] * dst.double()).sum()).backward()
    for i in range(2):
        near(y[i][live], outs[i][0][live].detach(), BF16 * (i + 1), f"y {i}")
        near(s[i], outs[i][1].detach(), BF16, f"stream {i}")
        near(blocks[i].grad_norm, Ds[i]["norm"].grad, HELD, f"norm weight {i}")
        for n in ("ws1", "ws2", "bs2", "w1"):
            near(blocks[i].layer.grads[n], Ds[i][n].grad, HELD * (2 - i), f"{n} {i}")
    near(d_res, r64.grad, HELD, "d_residual")
    assert (d_res[~live] == 0).all()


@pytest.mark.gpu
def test_training_block_refusals(moe):
    from mixture_experts_grouped_align_gb300 import MoeError
    from mixture_experts_grouped_align_gb300.train import TrainBlock, TrainLayer
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
    K = 64
    L = TrainLayer(z(8, K), z(8, 128, K), z(8, K, 64), z(128, K), z(128), z(K, 64), z(K), 2, 10)
    for args in ((None, z(K)), (L, z(K + 64)), (L, z(K).float()), (L, z(K).cpu())):
        with pytest.raises(MoeError):
            TrainBlock(*args)
    with pytest.raises(MoeError, match="rng"):
        TrainBlock(L, z(K), dropout=0.1)
    B = TrainBlock(L, z(K))
    with pytest.raises(MoeError, match="forward"):
        B.backward(z(4, K), None, z(4, K))
    for args in ((None, z(11, K), z(11, K)), (None, z(4, K).float(), z(4, K)), (z(3, K), z(4, K), z(4, K)), (None, z(4, K), z(3, K)),
                 (None, z(4, K + 64), z(4, K)), (None, z(4, K), B.normed[:4]), (None, z(4, K), z(4, K), z(4, dtype=torch.float32))):
        with pytest.raises(MoeError):
            B.forward(*args)
    B.forward(z(4, K), z(4, K), z(4, K))
    t = z(4, K)
    for args in ((z(4, K), None, z(4, K)), (z(4, K), None, z(3, K), z(4, K)), (z(4, K), z(4, K).float(), z(4, K), z(4, K)),
                 (z(4, K), None, t, t), (z(3, K), None, z(4, K), z(4, K))):
        with pytest.raises(MoeError):
            B.backward(*args)


def serve_weights(quant, seed, E=16, K=256, I=256, k=2):
    w = synth.Workload("blocks", T=8, K=K, I=I, E=E, k=k, quant=quant, seed=seed, weight_std=0.05, bias=True)
    lay = synth.make_layer(w)
    rng = np.random.default_rng(seed)
    Is, r, L = 192, 16, 5
    bits = lambda *s, std: synth.to_bf16_bits(rng.standard_normal(s) * std)  # noqa: E731
    D = {"norm": synth.to_bf16_bits(1 + 0.2 * rng.standard_normal(K)), "wr": bits(E, K, std=0.2), "ws1": bits(2 * Is, K, std=0.06),
         "bs1": bits(2 * Is, std=0.1), "ws2": bits(K, Is, std=0.08), "bs2": bits(K, std=0.1), "a1": bits(L, r, K, std=K ** -0.5),
         "b1": bits(L, 2 * Is, r, std=0.2), "a2": bits(L, r, Is, std=Is ** -0.5), "b2": bits(L, K, r, std=0.2)}
    return w, lay, D, rng.uniform(0.5, 2, L).astype(np.float32)


def serve_block(w, lay, D, scale, which, max_rows, **kw):
    from mixture_experts_grouped_align_gb300.runner import DeviceLayer, ServeBlock
    L = DeviceLayer(w.quant, w.E, w.K, w.I, w.k, *(dev(lay[n]) for n in ("w1", "w1_scale", "b1", "w2", "w2_scale", "b2")),
                    max_rows=max_rows)
    G = {n: dev(b) for n, b in D.items()}
    sc = torch.from_numpy(scale).cuda()
    ad = [(G["a1"], G["b1"], sc) if "1" in which else None, (G["a2"], G["b2"], sc) if "2" in which else None]
    shared = (G["ws1"], G["bs1"], G["ws2"], G["bs2"]) if which is not None else None
    return ServeBlock(L, G["norm"], G["wr"], shared, ad, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("quant", ["bf16", "mxfp4", "mxfp8"])
@pytest.mark.parametrize("T,which", [(1, "12"), (7, "1"), (40, "12"), (300, "2"), (300, "12"), (700, "")])
def test_serving_block(moe, quant, T, which):
    w, lay, D, scale = serve_weights(quant, T)
    B = serve_block(w, lay, D, scale, which, T)
    V = {n: formats.bf16_decode(b) for n, b in D.items()}
    rng = np.random.default_rng(T + 1)
    x, res = (synth.to_bf16_bits(rng.standard_normal((T, w.K)) * s) for s in (1, 2))
    R = min(T, 20)
    off = np.concatenate([[0], np.sort(rng.choice(T - 1, R - 1, replace=False) + 1), [T]]) if T > 1 else np.array([0, 1])
    ad = rng.integers(-1, 5, R)
    y = torch.empty((T, w.K), dtype=torch.bfloat16, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    _, s = B.step(dev(x), dev(res), T, y, i32(off), i32(ad))
    torch.cuda.synchronize()
    assert int(B.status[0]) == 0 and int(B.layer.status[0]) == 0
    # each step from what the one before it left
    s64, n64 = residual_norm.forward(formats.bf16_decode(x), formats.bf16_decode(res), V["norm"], 1e-5)
    fro = lambda a, b: np.linalg.norm(a - b) / np.linalg.norm(b)  # noqa: E731
    assert fro(bf16_to_np(s), s64) < 3e-3 and fro(bf16_to_np(B.normed[:T]), n64) < 3e-3
    n = bf16_to_np(B.normed[:T])
    logits = B.logits[:T].cpu().numpy()
    assert fro(logits, n @ V["wr"].T) < 1e-5
    ids, wt = route.route(logits, w.k)
    xin = n
    if quant == "mxfp8":
        xin = formats.dequant_mxfp8(B.codes[:T].cpu().numpy(), B.scales[:T].cpu().numpy())
        assert fro(xin, n64) < 2.0 ** -4
    W = layer_oracle.ExpertWeights(quant, *(lay[n_] for n_ in ("w1", "w1_scale", "b1", "w2", "w2_scale", "b2")))
    ref = bf16_round(layer_oracle.moe_layer(xin, ids, wt, W))
    gs = n @ V["ws1"].T + V["bs1"]
    if "1" in which:
        gs = bf16_round(adapter_oracle.adapter_gemm(n, V["a1"], V["b1"], scale, off, ad, bf16_round(gs))[0])
    g, u = np.split(gs, 2, axis=1)
    hs = bf16_round(g / (1 + np.exp(-g)) * u)
    ref = bf16_round(ref + hs @ V["ws2"].T + V["bs2"])
    if "2" in which:
        ref = adapter_oracle.adapter_gemm(hs, V["a2"], V["b2"], scale, off, ad, ref)[0]
    assert fro(bf16_to_np(y), ref) < 1e-2


@pytest.mark.gpu
@pytest.mark.parametrize("quant", ["bf16", "mxfp8"])
def test_serving_block_in_a_graph(moe, quant):
    """Decode steps replayed with other tokens, offsets and adapters than were captured."""
    T = 24
    w, lay, D, scale = serve_weights(quant, 5)
    B = serve_block(w, lay, D, scale, "12", T, stream_f32=True)
    rng = np.random.default_rng(6)
    new = lambda: dev(synth.to_bf16_bits(rng.standard_normal((T, w.K))))  # noqa: E731
    x, res, y = new(), torch.randn((T, w.K), device="cuda"), new()
    off, ad = (torch.arange(n, dtype=torch.int32, device="cuda") for n in (T + 1, T))
    ad.remainder_(5)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        B.step(x, res, T, y, off, ad)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        B.step(x, res, T, y, off, ad)
    for _ in range(3):
        x.copy_(new())
        res.normal_()
        ad.copy_(torch.from_numpy(rng.integers(-1, 5, T)).int())
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        y.zero_()
        B.step(x, res, T, y, off, ad)
        torch.cuda.synchronize()
        assert torch.equal(got, y)


def test_serving_block_refusals(moe):
    """Shapes that do not fit the layer are refused when the block is made."""
    from mixture_experts_grouped_align_gb300 import MoeError
    from mixture_experts_grouped_align_gb300.runner import DeviceLayer, ServeBlock
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    E, K, I, Is = 8, 64, 64, 32
    L = DeviceLayer("bf16", E, K, I, 2, z(E, 2 * I, K), None, None, z(E, K, I), None, None, 16, device="cpu")
    shared = (z(2 * Is, K), z(2 * Is), z(K, Is), z(K))
    good = dict(layer=L, norm_w=z(K), wr=z(E, K), shared=shared, adapters=((z(3, 8, K), z(3, 2 * Is, 8), None), None))
    assert ServeBlock(**good).workspace.numel() >= 256
    for kw in (dict(norm_w=z(K + 8)), dict(wr=z(E, K + 8)), dict(wr=z(E + 1, K)), dict(shared=None),
               dict(shared=(z(2 * Is, K + 8), *shared[1:])), dict(adapters=(None, (z(3, 8, K), z(3, K, 8), None))),
               dict(adapters=((z(3, 8, K), z(2, 2 * Is, 8), None), None))):
        with pytest.raises(MoeError):
            ServeBlock(**{**good, **kw})
    B = ServeBlock(**good, max_requests=4)
    i = torch.zeros(6, dtype=torch.int32)
    with pytest.raises(MoeError, match="requests"):
        B.step(None, z(5, K), 5, z(5, K), i, i[:5])
    with pytest.raises(MoeError, match="rows"):
        B.step(None, z(17, K), 17, z(17, K))


@pytest.mark.parametrize("max_requests", [4, 512, 2000])
def test_serving_block_workspace_holds_every_batch(moe, max_requests):
    """Whatever the rows and requests of a batch, also more requests than rows and more than 1024."""
    from mixture_experts_grouped_align_gb300 import moe_adapter_gemm_workspace_size
    from mixture_experts_grouped_align_gb300.runner import DeviceLayer, ServeBlock
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    E, K, I, Is, r = 8, 64, 64, 32, 16
    L = DeviceLayer("bf16", E, K, I, 2, z(E, 2 * I, K), None, None, z(E, K, I), None, None, 2050, device="cpu")
    B = ServeBlock(L, z(K), z(E, K), (z(2 * Is, K), z(2 * Is), z(K, Is), z(K)), (None, (z(3, r, Is), z(3, K, r), None)),
                   max_requests=max_requests)
    for T in (1, 100, 255, 256, 257, 300, 511, 512, 1000, 1792, 2048, 2050):
        for R in {1, 3, 300, 1000, 1024, 1025, 2000}:
            if R <= max_requests:
                assert B.workspace.numel() >= moe_adapter_gemm_workspace_size(T, R, r), (T, R)
