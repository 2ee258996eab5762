"""ServeBlock refuses, before it launches anything, operands that its kernels would read or write past, and
outputs over rows that it still reads.  On the CPU: the refusals name the operand and come first."""
import pytest

torch = pytest.importorskip("torch")

E, K, I, Is, T = 8, 64, 64, 64, 5


def z(*s, dtype=torch.bfloat16, **kw):
    return torch.zeros(s, dtype=dtype, **kw)


def parts():
    from mixture_experts_grouped_align_gb300.runner import DeviceLayer
    L = DeviceLayer("bf16", E, K, I, 2, z(E, 2 * I, K), None, None, z(E, K, I), None, None, 16, device="cpu")
    return dict(layer=L, norm_w=z(K), wr=z(E, K), shared=(z(2 * Is, K), z(2 * Is), z(K, Is), z(K)),
                adapters=((z(3, 8, K), z(3, 2 * Is, 8), z(3, dtype=torch.float32)), None))


@pytest.fixture(scope="module")
def block():
    from mixture_experts_grouped_align_gb300 import build
    from mixture_experts_grouped_align_gb300.runner import ServeBlock
    build()
    return ServeBlock(**parts())


def refused(match, fn, *a, **kw):
    from mixture_experts_grouped_align_gb300 import MoeError
    with pytest.raises(MoeError, match=match):
        fn(*a, **kw)


@pytest.mark.parametrize("y", [z(T - 1, K), z(T, K, dtype=torch.float32), z(K, T + 1).t(), z(T * K + 8)[1:], None])
def test_y(block, y):
    refused("^(.*: )?y: need", block.step, z(T, K), z(T, K), T, y)


@pytest.mark.parametrize("branch", [z(T - 1, K), z(T, K, dtype=torch.float32), z(K, T).t()])
def test_branch(block, branch):
    refused("branch: need", block.step, branch, z(T, K), T, z(T, K))


@pytest.mark.parametrize("residual", [z(T - 1, K), z(T, K, dtype=torch.float32), z(K, T).t()])
def test_residual(block, residual):
    refused("residual: need", block.step, None, residual, T, z(T, K))


@pytest.mark.parametrize("off,ad", [(z(3, dtype=torch.int32), z(3, dtype=torch.int32)), (z(4, dtype=torch.int64), z(3, dtype=torch.int32)),
                                    (z(4, dtype=torch.int32), z(3, dtype=torch.int64)), (None, z(3, dtype=torch.int32))])
def test_tables(block, off, ad):
    refused("row_offsets: need|adapter: need", block.step, None, z(T, K), T, z(T, K), off, ad)


def test_overlaps(block):
    refused("y and the block", block.step, None, z(T, K), T, block.normed[:T])
    refused("y and the block", block.step, None, z(T, K), T, block.stream[1:T + 1])
    refused("branch and the block", block.step, block.stream[:T], z(T, K), T, z(T, K))
    refused("branch and the block", block.step, block.normed[1:T + 1], z(T, K), T, z(T, K))
    refused("residual and the block", block.step, None, block.normed[:T], T, z(T, K))
    refused("residual and the block", block.step, None, block.stream[1:T + 1], T, z(T, K))


@pytest.mark.parametrize("name", ["norm_w", "wr"])
def test_weights_on_another_device(name):
    from mixture_experts_grouped_align_gb300.runner import ServeBlock
    p = parts()
    refused(f"{name}: need", ServeBlock, **{**p, name: p[name].to("meta")})
    refused(f"{name}: need", ServeBlock, **{**p, name: p[name].float()})


def test_shared_weights_and_adapters_that_do_not_fit():
    from mixture_experts_grouped_align_gb300.runner import ServeBlock
    p = parts()
    ws1, bs1, ws2, bs2 = p["shared"]
    for what, shared in (("ws1", (ws1.float(), bs1, ws2, bs2)), ("bs1", (ws1, bs1[:Is], ws2, bs2)), ("ws2", (ws1, bs1, ws2.to("meta"), bs2)),
                         ("bs2", (ws1, bs1, ws2, z(K - 8)))):
        refused(f"{what}: need", ServeBlock, **{**p, "shared": shared})
    a, b, scale = p["adapters"][0]
    for what, pair in (("a: need", (a.float(), b, scale)), ("b: need", (a, b.to("meta"), scale)), ("scale: need", (a, b, scale[:2])),
                       ("scale: need", (a, b, scale.double()))):
        refused(what, ServeBlock, **{**p, "adapters": (pair, None)})


def test_shared_width_with_adapters_before_the_activation():
    """The pre-activations with adapters in them pass through moe_act_checkpoint, whose rows are multiples of 32."""
    from mixture_experts_grouped_align_gb300.runner import ServeBlock
    p = parts()
    n = 40
    shared = (z(2 * n, K), z(2 * n), z(K, n), z(K))
    refused("multiple of 32", ServeBlock, **{**p, "shared": shared, "adapters": ((z(3, 8, K), z(3, 2 * n, 8), None), None)})
    for adapters in ((None, None), (None, (z(3, 8, n), z(3, K, 8), None))):  # neither needs it
        assert ServeBlock(**{**p, "shared": shared, "adapters": adapters}).Is == n
