"""moe_dense_gemm_plan refuses what moe_dense_gemm refuses (no GPU needed)."""
import pytest

import mixture_experts_grouped_align_gb300 as moe


@pytest.fixture(scope="module", autouse=True)
def lib():
    moe.build()
    return moe.load()


@pytest.mark.parametrize("status,kw", [(-1, dict(M=0)), (-1, dict(M=-1)), (-1, dict(N=0)), (-1, dict(K=0)), (-2, dict(K=12)),
                                       (-1, dict(activation=3)), (-2, dict(K=1 << 30)), (-2, dict(M=1 << 30)), (-2, dict(N=1 << 29))])
def test_refusals(status, kw):
    with pytest.raises(moe.MoeError) as e:
        moe.moe_dense_gemm_plan(**({"M": 4, "N": 64, "K": 64} | kw))
    assert e.value.status == status


def test_null_plan_is_refused():
    assert moe.load().moe_dense_gemm_plan(4, 64, 64, 2, 0, None) == -1
