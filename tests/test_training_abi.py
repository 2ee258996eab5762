"""Refusals of the training operators' calls: argument errors come back from the host, before
any launch (no GPU needed)."""
import pytest

import mixture_experts_grouped_align_gb300 as moe

torch = pytest.importorskip("torch")

P = 1 << 20  # a well aligned pointer that nothing dereferences


@pytest.fixture(scope="module", autouse=True)
def lib():
    moe.build()
    return moe.load()


def refused(status, fn, *a, **kw):
    with pytest.raises(moe.MoeError) as e:
        fn(*a, **kw)
    assert e.value.status == status, e.value
    assert len(str(e.value)) > 20


def router(logits=P, ids=P, w=P, dw=P, mask=None, T=4, k=2, E=8, counts=P, mean=P, loss=P, d=P, ws=P, nbytes=1 << 24):
    return moe.moe_router_loss(logits, ids, w, dw, mask, T, k, E, 0.01, 0.001, counts, mean, loss, d,
                               moe.Ctx(stream=0, workspace=ws, workspace_bytes=nbytes))


@pytest.mark.parametrize("status,kw", [
    (-2, dict(k=0)), (-2, dict(k=33, E=64)), (-2, dict(E=1025)), (-2, dict(k=9, E=8)), (-1, dict(T=-1)),
    (-2, dict(T=1 << 31, k=1)), (-1, dict(logits=None)), (-1, dict(ids=None)), (-1, dict(loss=None)),
    (-1, dict(w=None)), (-1, dict(logits=P + 4)), (-1, dict(d=P + 8)), (-1, dict(mask=P + 1)),
    (-3, dict(ws=None)), (-3, dict(nbytes=256)),
])
def test_router_loss_refusals(status, kw):
    refused(status, router, **kw)


def test_router_loss_workspace_size():
    assert moe.moe_router_loss_workspace_size(0) == 0 and moe.moe_router_loss_workspace_size(1025) == 0
    assert 0 < moe.moe_router_loss_workspace_size(1) < moe.moe_router_loss_workspace_size(1024) <= 4 << 20


def forward(gu=P, w=None, rows=4, I=64, act="swiglu", h=P, codes=P, scales=P):
    return moe.moe_act_checkpoint(gu, w, rows, I, act, h, codes, scales, moe.Ctx(stream=0))


def backward(codes=P, scales=P, dh=P, w=None, rows=4, I=64, act="swiglu", d=P, h=P, dw=P):
    return moe.moe_act_backward(codes, scales, dh, w, rows, I, act, d, h, dw, moe.Ctx(stream=0))


@pytest.mark.parametrize("fn,status,kw", [
    (forward, -2, dict(I=0)), (forward, -2, dict(I=48)), (forward, -1, dict(rows=-1)), (forward, -1, dict(act=7)),
    (forward, -1, dict(rows=1 << 31)), (forward, -1, dict(gu=None)), (forward, -1, dict(codes=None)),
    (forward, -1, dict(scales=None)), (forward, -1, dict(gu=P + 2)), (forward, -1, dict(h=P + 2)),
    (backward, -2, dict(I=31)), (backward, -1, dict(rows=-3)), (backward, -1, dict(act=3)),
    (backward, -1, dict(codes=None)), (backward, -1, dict(dh=None)), (backward, -1, dict(d=None)),
    (backward, -1, dict(dw=P + 4)), (backward, -1, dict(w=P + 4)),
])
def test_activation_refusals(fn, status, kw):
    refused(status, fn, **kw)


def test_empty_calls_return_ok():
    assert forward(gu=None, codes=None, scales=None, h=None, rows=0) == 0
    assert backward(codes=None, scales=None, dh=None, d=None, rows=0) == 0


def test_binding_refuses_what_the_abi_cannot_see():
    """Host tensors, other types, strides and short buffers never reach the library as pointers."""
    gu = torch.zeros((4, 128), dtype=torch.bfloat16)
    refused(-1, forward, gu=gu)                                     # host memory
    refused(-1, forward, gu=gu.float())                             # another type
    refused(-1, forward, gu=torch.zeros((128, 4), dtype=torch.bfloat16).t())  # strides
    refused(-1, backward, dh=torch.zeros((3, 64), dtype=torch.bfloat16))      # short
    refused(-1, router, logits=torch.zeros((4, 8)))


def dense(x=P, w=P, lay="nk", bias=None, residual=None, scale=1.0, M=4, N=64, K=64, act="none", out=P, f32=False):
    return moe.moe_dense_gemm(x, w, lay, bias, residual, scale, M, N, K, act, out, moe.Ctx(stream=0), out_f32=f32)


@pytest.mark.parametrize("status,kw", [
    (-1, dict(act=3)), (-1, dict(lay=2)), (-1, dict(M=-1)), (-1, dict(N=0)), (-1, dict(K=0)), (-2, dict(K=12)),
    (-2, dict(K=1 << 30)), (-2, dict(M=1 << 30)), (-2, dict(N=1 << 29)), (-2, dict(lay="kn", N=60)),
    (-1, dict(x=None)), (-1, dict(w=None)), (-1, dict(out=None)), (-1, dict(x=P + 2)), (-1, dict(w=P + 8)),
    (-1, dict(bias=P + 2)), (-1, dict(residual=P + 4)), (-1, dict(out=P + 8)),
])
def test_dense_gemm_refusals(status, kw):
    refused(status, dense, **kw)


@pytest.mark.parametrize("kw", [dict(dz=None), dict(d=None), dict(M=-1), dict(N=0), dict(dz=P + 2), dict(d=P + 4)])
def test_bias_grad_refusals(kw):
    a = {"dz": P, "M": 4, "N": 64, "d": P} | kw
    refused(-1, moe.moe_dense_bias_grad, a["dz"], a["M"], a["N"], a["d"], moe.Ctx(stream=0))


def test_dense_binding_refusals():
    assert dense(x=None, w=None, out=None, M=0) == 0
    refused(-1, dense, x=torch.zeros((4, 64), dtype=torch.bfloat16))
    # a residual in another type than the output
    refused(-1, dense, residual=torch.zeros((4, 64), dtype=torch.bfloat16), f32=True)


@pytest.mark.parametrize("status,kw", [(-1, dict(T=-1)), (-1, dict(k=0)), (-1, dict(k=1025)), (-2, dict(K=12)),
                                       (-2, dict(T=1 << 30, k=4)), (-1, dict(o=None)), (-1, dict(y=None)), (-1, dict(o=P + 2)),
                                       (-1, dict(r=P + 8))])
def test_pair_sum_refusals(status, kw):
    a = {"o": P, "r": None, "T": 4, "k": 2, "K": 64, "y": P} | kw
    refused(status, moe.moe_pair_sum, a["o"], a["r"], a["T"], a["k"], a["K"], a["y"], moe.Ctx(stream=0))
