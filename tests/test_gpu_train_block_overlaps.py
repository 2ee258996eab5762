"""TrainBlock refuses operands that share memory with what a pass still reads: the stored stream, from which
the backward pass has the norm again, and the norm's rows.  What the kernels allow in place stays allowed."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
K, T = 64, 4


def z(*s, dtype=torch.bfloat16):
    return torch.zeros(s, dtype=dtype, device="cuda")


@pytest.fixture(scope="module")
def block():
    import mixture_experts_grouped_align_gb300 as moe
    from mixture_experts_grouped_align_gb300.train import TrainBlock, TrainLayer
    moe.build()
    moe.load()
    L = TrainLayer(z(8, K), z(8, 128, K), z(8, K, 64), z(128, K), z(128), z(K, 64), z(K), 2, 10)
    return TrainBlock(L, z(K))


def refused(fn, *a):
    from mixture_experts_grouped_align_gb300 import MoeError
    with pytest.raises(MoeError, match="must not overlap"):
        fn(*a)


def test_forward(block):
    B = block
    refused(B.forward, z(T, K), z(T, K), B.stream[:T])            # y over the stream
    refused(B.forward, z(T, K), z(T, K), B.stream[T - 1:2 * T - 1])
    refused(B.forward, B.stream[:T], z(T, K), z(T, K))            # branch
    refused(B.forward, z(T, K), B.stream[1:T + 1], z(T, K))       # residual, shifted
    refused(B.forward, z(T, K), B.normed[:T], z(T, K))
    t = z(T, K)
    B.forward(z(T, K), B.stream[:T], t)                           # the residual in place
    B.forward(t, z(T, K), t)                                      # y over the branch, which is done with


def test_backward(block):
    B = block
    B.forward(z(T, K), z(T, K), z(T, K))
    both = z(2 * T, K)
    refused(B.backward, z(T, K), both[:T], both[1:T + 1], z(T, K))   # d_residual over d_stream, shifted
    refused(B.backward, z(T, K), both[:T], z(T, K), both[:T])        # d_branch over d_stream
    refused(B.backward, z(T, K), None, B.stream[:T], z(T, K))        # d_residual over the stream
    refused(B.backward, z(T, K), None, z(T, K), B.stream[:T])        # d_branch over the stream
    refused(B.backward, z(T, K), None, B.stream[2:T + 2], z(T, K))
    dy, ds = z(T, K), z(T, K)
    B.backward(dy, ds, ds, dy)                                       # both in place
    torch.cuda.synchronize()
