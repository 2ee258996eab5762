"""Refusals of the residual norm's calls come back from the host, before any launch (no GPU needed)."""
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


def forward(x=P, res=P, mask=None, w=P, T=4, K=64, eps=1e-5, p=0.0, rng=None, sid=0, stream=P, out=P, codes=None, scales=None, **kw):
    return moe.moe_residual_norm(x, res, mask, w, T, K, eps, p, rng, sid, stream, out, codes, scales, moe.Ctx(stream=0), **kw)


def backward(d_out=P, d_st=P, st=P, mask=None, w=P, T=4, K=64, eps=1e-5, p=0.0, rng=None, sid=0, dr=P, dx=P, dw=P, ws=P,
             nbytes=1 << 24):
    return moe.moe_residual_norm_backward(d_out, d_st, st, mask, w, T, K, eps, p, rng, sid, dr, dx, dw,
                                          moe.Ctx(stream=0, workspace=ws, workspace_bytes=nbytes))


@pytest.mark.parametrize("fn", [forward, backward])
@pytest.mark.parametrize("status,kw", [
    (-1, dict(T=-1)), (-1, dict(K=0)), (-2, dict(K=12)), (-2, dict(K=16392)), (-2, dict(T=1 << 31)), (-1, dict(eps=0.0)),
    (-1, dict(eps=-1.0)), (-1, dict(eps=float("nan"))), (-1, dict(eps=float("inf"))), (-1, dict(p=1.0, rng=P)),
    (-1, dict(p=-0.1, rng=P)), (-1, dict(p=float("nan"), rng=P)), (-1, dict(p=0.1)), (-1, dict(p=0.1, rng=P + 8)),
    (-1, dict(w=None)), (-1, dict(w=P + 2)), (-1, dict(mask=P + 1)),
])
def test_common_refusals(fn, status, kw):
    refused(status, fn, **kw)


@pytest.mark.parametrize("status,kw", [
    (-1, dict(x=None, res=None)), (-1, dict(stream=None, out=None)), (-1, dict(x=P + 2)), (-1, dict(res=P + 4)),
    (-1, dict(stream=P + 8)), (-1, dict(out=P + 2)), (-1, dict(codes=P)), (-1, dict(scales=P, scale_mode="mx")),
    (-1, dict(codes=P, scale_mode="row")), (-1, dict(codes=P, scales=P, scale_mode=3)),
    (-1, dict(codes=P, scales=P, scale_mode=0)), (-2, dict(K=72, codes=P, scales=P, scale_mode="mx")),
    (-1, dict(codes=P + 8, scales=P, scale_mode="mx")), (-1, dict(codes=P, scales=P + 4, scale_mode="row")),
])
def test_forward_refusals(status, kw):
    refused(status, forward, **kw)


@pytest.mark.parametrize("status,kw", [
    (-1, dict(d_out=None)), (-1, dict(st=None)), (-1, dict(dr=None, dx=None, dw=None)), (-1, dict(d_out=P + 2)),
    (-1, dict(d_st=P + 2)), (-1, dict(dr=P + 2)), (-1, dict(dx=P + 2)), (-1, dict(dw=P + 4)), (-3, dict(ws=None)),
    (-3, dict(nbytes=256)),
])
def test_backward_refusals(status, kw):
    refused(status, backward, **kw)


def test_empty_calls_and_workspace_size():
    assert forward(x=None, res=None, w=None, stream=None, out=None, T=0) == 0
    assert backward(d_out=None, st=None, w=None, dr=None, dx=None, dw=None, T=0) == 0
    size = moe.moe_residual_norm_workspace_size
    assert size(0) == size(12) == size(16392) == 0 and 0 < size(8) < size(16384) <= 64 << 20


def test_binding_refuses_what_the_abi_cannot_see():
    t = torch.zeros((4, 64), dtype=torch.bfloat16)
    refused(-1, forward, x=t)                                            # host memory
    refused(-1, forward, res=t.float(), stream=P)                        # the stream is fp32 then, but on the host
    refused(-1, forward, w=torch.zeros(32, dtype=torch.bfloat16))        # short
    refused(-1, forward, p=0.1, rng=torch.zeros(2, dtype=torch.int32))   # another type
    refused(-1, backward, d_out=t)
    with pytest.raises(OverflowError):
        forward(sid=1 << 32)
    with pytest.raises(KeyError):
        forward(codes=P, scales=P, scale_mode="block")
