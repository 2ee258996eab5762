"""Names given as strings: subclasses of str (enums, numpy strings) are names too (no GPU needed)."""
import enum

import numpy as np
import pytest

import mixture_experts_grouped_align_gb300 as moe

P = 1 << 20


class Act(str, enum.Enum):
    SWIGLU = "swiglu"
    RELU2 = "relu2"
    NONE = "none"


@pytest.fixture(scope="module", autouse=True)
def lib():
    moe.build()
    return moe.load()


@pytest.mark.parametrize("name", [Act.RELU2, np.str_("relu2")])
def test_activation_names(name):
    assert moe._act(name) == moe.ACTIVATION["relu2"] and moe._act(np.int32(1)) == 1
    # rows == 0: answered on the host
    assert moe.moe_act_checkpoint(None, None, 0, 64, name, None, None, None, moe.Ctx(stream=0)) == 0


@pytest.mark.parametrize("layout", ["kn", np.str_("kn"), moe.W_LAYOUT["kn"]])
def test_layout_names(layout):
    assert moe.moe_dense_gemm(None, None, layout, None, None, 1.0, 0, 64, 64, Act.NONE, None, moe.Ctx(stream=0)) == 0
    with pytest.raises(moe.MoeError):  # the name was understood: [K, N] weights need N a multiple of 8
        moe.moe_dense_gemm(P, P, layout, None, None, 1.0, 4, 60, 64, Act.NONE, P, moe.Ctx(stream=0))


class Pointer(int):
    pass


def test_pointers_of_int_subclasses():
    with pytest.raises(moe.MoeError):  # an argument error of the library, not an attribute of the pointer
        moe.moe_dense_gemm(P, P, "nk", None, None, 1.0, 4, 64, 12, "none", Pointer(P), moe.Ctx(stream=0))
