"""The workspace size of the adapters' call is 0 for what the call refuses (no GPU needed)."""
import pytest

import mixture_experts_grouped_align_gb300 as moe


@pytest.mark.parametrize("M,R,r", [(1, 1, 12), (1, 1, 4), (300, 2, 100), (1, 1 << 30, 16), (1000, 1 << 30, 16), (-1, 1, 16), (1, -1, 16),
                                   (1, 1, -8)])
def test_no_size_for_what_is_refused(moe_lib, M, R, r):
    assert moe.moe_adapter_gemm_workspace_size(M, R, r) == 0
    with pytest.raises(moe.MoeError):
        moe.moe_adapter_gemm_plan(M, 64, 64, r, 2, R)


@pytest.mark.parametrize("M,R,r", [(1, 1, 8), (300, 2, 104), (1, (1 << 30) - 1, 16), ((1 << 30) - 1, 1, 8)])
def test_a_size_for_what_is_taken(moe_lib, M, R, r):
    assert moe.moe_adapter_gemm_workspace_size(M, R, r) >= M * r * 4
    assert moe.moe_adapter_gemm_plan(M, 64, 64, r, 2, R) in ("few", "long")


@pytest.fixture(scope="module")
def moe_lib():
    moe.build()
    return moe.load()
