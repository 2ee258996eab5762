"""TrainLayer refuses weights that its kernels would read wrongly, before it allocates anything."""
import pytest

torch = pytest.importorskip("torch")

E, K, I, Is = 64, 128, 64, 192
SHAPES = {"wr": (E, K), "w1": (E, 2 * I, K), "w2": (E, K, I), "ws1": (2 * Is, K), "bs1": (2 * Is,), "ws2": (K, Is), "bs2": (K,)}


def weights(device="cpu"):
    return {n: torch.zeros(s, dtype=torch.bfloat16, device=device) for n, s in SHAPES.items()}


def layer(W, rows=8):
    from mixture_experts_grouped_align_gb300.train import TrainLayer
    return TrainLayer(W["wr"], W["w1"], W["w2"], W["ws1"], W["bs1"], W["ws2"], W["bs2"], 2, rows)


def spoilt(t, how):
    if how == "type":
        return t.half()
    if how == "shape":
        return t[: t.shape[0] // 2].clone()
    if how == "strides":
        return torch.empty((2 * t.shape[0], *t.shape[1:]), dtype=t.dtype, device=t.device)[::2]
    if how == "expanded":
        return torch.zeros((), dtype=t.dtype, device=t.device).expand(t.shape)
    if how == "address":
        return torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape)
    return None


HOW = ["type", "shape", "strides", "expanded", "nothing"]


@pytest.mark.parametrize("how", HOW)
@pytest.mark.parametrize("name", list(SHAPES))
def test_weights_are_refused_by_name(name, how):
    from mixture_experts_grouped_align_gb300 import MoeError
    W = weights()
    W[name] = spoilt(W[name], how)
    with pytest.raises((MoeError, ValueError) if how == "shape" else MoeError, match=None if how == "shape" else f"{name}:"):
        layer(W)


def test_host_weights_are_refused():
    from mixture_experts_grouped_align_gb300 import MoeError
    with pytest.raises(MoeError, match="CUDA device"):
        layer(weights())


@pytest.mark.parametrize("name,shape", [("K", (E, 96)), ("I", (E, K, 96)), ("Is", (K, 96)), ("k", (1, K)), ("E", (1025, K))])
def test_sizes_are_refused(name, shape):
    W = weights()
    W[{"I": "w2", "Is": "ws2"}.get(name, "wr")] = torch.zeros(shape, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="multiples of 64" if name in ("K", "I", "Is") else "1024"):
        layer(W)


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("how", ["type", "strides", "expanded", "address"])
def test_device_weights_are_refused_by_name(name, how):
    from mixture_experts_grouped_align_gb300 import MoeError
    W = weights("cuda")
    W[name] = spoilt(W[name], how)
    with pytest.raises(MoeError, match=f"{name}:"):
        layer(W)


@pytest.mark.gpu
def test_operands_of_a_step_are_refused_before_anything_is_launched(monkeypatch):
    import mixture_experts_grouped_align_gb300 as moe
    from mixture_experts_grouped_align_gb300 import MoeError, train
    moe.build()
    moe.load()
    T = 6
    W = weights("cuda")
    L = layer(W)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(MoeError, match="forward"):
        L.backward(x, torch.empty_like(x))
    L.forward(x, torch.empty_like(x))
    torch.cuda.synchronize()

    def launched(*a, **kw):
        raise AssertionError("launched")

    for n in ("moe_grouped_gemm", "moe_act_backward", "moe_wgrad", "moe_router_loss", "moe_dense_gemm", "moe_pair_sum",
              "moe_dense_bias_grad", "moe_align", "moe_act_checkpoint"):
        monkeypatch.setattr(train, n, launched)
    new = lambda: torch.empty_like(x)  # noqa: E731
    for how in ("type", "shape", "strides", "expanded", "address", "nothing"):
        bad = spoilt(x, how)
        for args in ((bad, new()), (new(), bad)):
            with pytest.raises(MoeError):
                L.backward(*args)
        with pytest.raises(MoeError):
            L.forward(x, bad)
        if how != "shape":  # half the elements are as many whole rows
            with pytest.raises(MoeError):
                L.forward(bad, new())
    for args in ((x.cpu(), new()), (new(), x.cpu()), (new()[:3], new()), (new(), new(), torch.ones(T, device="cuda")),
                 (new(), new(), torch.ones(T - 1, dtype=torch.uint8, device="cuda")), (new(), x)):
        with pytest.raises(MoeError):
            L.backward(*args)
    dy = new()
    with pytest.raises(MoeError):
        L.backward(dy, dy)
    with pytest.raises(MoeError):
        L.forward(x, x)
    with pytest.raises(MoeError):
        L.forward(torch.empty((9, K), dtype=torch.bfloat16, device="cuda"), torch.empty((9, K), dtype=torch.bfloat16, device="cuda"))
    keep = L.w2
    L.w2 = spoilt(keep, "strides")
    for call in (lambda: L.forward(x, new()), lambda: L.backward(new(), new())):
        with pytest.raises(MoeError, match="w2"):
            call()
