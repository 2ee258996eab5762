"""Refusals of moe_adapter_gemm come back from the host, before any launch (no GPU needed); its oracle."""
import numpy as np
import pytest

import mixture_experts_grouped_align_gb300 as moe
from oracle import adapter as oracle

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


def call(x=P, a=P, b=P, scale=P, off=P, ad=P, base=P, M=4, N=64, K=64, r=16, L=2, R=3, out=P, ctx=None, **kw):
    return moe.moe_adapter_gemm(x, a, b, scale, off, ad, base, M, N, K, r, L, R, out,
                                ctx or moe.Ctx(stream=0, workspace=P, workspace_bytes=1 << 30), **kw)


@pytest.mark.parametrize("status,kw", [
    (-1, dict(M=-1)), (-1, dict(N=0)), (-1, dict(K=0)), (-1, dict(r=0)), (-1, dict(L=0)), (-1, dict(R=-1)),
    (-2, dict(N=12)), (-2, dict(K=20)), (-2, dict(r=12)), (-2, dict(r=136)), (-2, dict(M=1 << 30)), (-2, dict(N=1 << 30)),
    (-2, dict(K=1 << 30)), (-2, dict(R=1 << 30)), (-1, dict(x=None)), (-1, dict(a=None)), (-1, dict(b=None)),
    (-1, dict(off=None)), (-1, dict(ad=None)), (-1, dict(out=None)), (-1, dict(x=P + 2)), (-1, dict(a=P + 2)),
    (-1, dict(b=P + 8)), (-1, dict(scale=P + 4)), (-1, dict(off=P + 4)), (-1, dict(ad=P + 4)), (-1, dict(base=P + 2)),
    (-1, dict(out=P + 2)),
])
def test_refusals(status, kw):
    refused(status, call, **kw)


def test_plan_and_workspace_size():
    plan = moe.moe_adapter_gemm_plan
    assert plan(1, 2880, 2880, 16, 8, 1) == plan(64, 5760, 2880, 16, 100, 64) == "few"
    assert plan(8192, 4096, 7168, 32, 8, 16) == plan(58879, 2880, 2880, 64, 6, 16) == "long"
    assert plan(58879, 2880, 2880, 64, 1 << 20, 16) == "few"  # adapters of more than 2^31 rows
    assert plan(100000, 2880, 2880, 16, 6, 1025) == "few"     # more requests than the other kernels' tables
    for kw in (dict(M=0), dict(R=0), dict(N=12), dict(r=136)):
        with pytest.raises(moe.MoeError):
            plan(**{**dict(M=8, N=64, K=64, r=8, L=2, R=2), **kw})
    size = moe.moe_adapter_gemm_workspace_size
    assert size(0, 1, 16) == size(1, 0, 16) == size(1, 1, 0) == size(1, 1, 136) == size(1 << 30, 1, 16) == 0
    assert 0 < size(1, 1, 8) < 1 << 20 and size(58879, 16, 64) < 64 << 20
    refused(-3, call, ctx=moe.Ctx(stream=0, workspace=P, workspace_bytes=64))
    refused(-3, call, ctx=moe.Ctx(stream=0))


def test_empty_calls():
    assert call(x=None, out=None, M=0) == 0
    assert call(x=None, off=None, ad=None, out=None, R=0) == 0


def test_binding_refuses_what_the_abi_cannot_see():
    t = torch.zeros((4, 64), dtype=torch.bfloat16)
    refused(-1, call, x=t)                                          # host memory
    refused(-1, call, base=torch.zeros((4, 64)))                    # another type than out's
    refused(-1, call, off=torch.zeros(4, dtype=torch.int64))


def test_oracle_against_rows():
    rng = np.random.default_rng(1)
    x, a, b = rng.standard_normal((7, 8)), rng.standard_normal((3, 2, 8)), rng.standard_normal((3, 4, 2))
    base, scale = rng.standard_normal((7, 4)), np.array([2.0, 0.5, -1.0])
    got, _ = oracle.adapter_gemm(x, a, b, scale, [1, 3, 3, 6], [2, 1, -1], base)
    for m, l in enumerate([None, 2, 2, None, None, None, None]):
        want = base[m].copy()
        if l is not None:
            for n in range(4):
                want[n] += scale[l] * sum(b[l][n][j] * sum(a[l][j][k] * x[m][k] for k in range(8)) for j in range(2))
        assert np.allclose(got[m], want)
    assert list(oracle.row_adapters(7, [1, 3, 3, 6], [2, 1, -1])) == [-2, 2, 2, -1, -1, -1, -2]
