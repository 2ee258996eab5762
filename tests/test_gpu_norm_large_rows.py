"""Rows whose sum of squares is above fp32's range: their norm is 0, in every format, and so is what passes
through it backward, also where s times the weight overflows.  A row with an infinity is NaN in its scale.
No tolerances: zeros, and d_stream as it is.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TOPS = [1.0, 1e25, 1e37, 1e38, 3e38]  # of |s|; weights of 1 to 8


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_grouped_align_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.build()
    m.load()
    return m


def inputs(T, K, f32):
    rng = np.random.default_rng(T + K)
    s = np.sign(rng.uniform(-1, 1, (T, K))) * np.resize(TOPS, T)[:, None]
    s = torch.from_numpy(s).to(torch.float32 if f32 else torch.bfloat16).cuda()
    assert torch.isfinite(s).all()
    w = torch.from_numpy(rng.uniform(1, 8, K)).bfloat16().cuda()
    return s, w, torch.from_numpy(np.resize(TOPS, T) > 1).cuda()


SIZES = [(15, 64), (15, 256), (25, 2880), (7000, 256), (900, 7168), (140, 12288)]


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("quant", [None, "mx", "row"])
def test_forward(moe, T, K, f32, quant):
    s, w, large = inputs(T, K, f32)
    s[2, 3] = float("inf")
    o = torch.full((T, K), 7.0, dtype=torch.bfloat16, device="cuda")
    codes = torch.full((T, K), 0xA5, dtype=torch.uint8, device="cuda") if quant else None
    sc = {None: None, "mx": torch.full((T, K // 32), 0xA5, dtype=torch.uint8, device="cuda"),
          "row": torch.full((T,), 7.0, device="cuda")}[quant]
    moe.moe_residual_norm(None, s, None, w, T, K, 1e-5, 0.0, None, 0, None, o, codes, sc)
    torch.cuda.synchronize()
    zero = large.clone()
    zero[2] = False
    assert (o[zero] == 0).all() and torch.isnan(o[2, 3])
    assert (o[~large].float().abs() > 0.9).all() and (o[~large].float().abs() < 8.1).all()
    if quant:
        assert (codes[zero] & 0x7F == 0).all() and (codes[~large] & 0x7F != 0).all()
    if quant == "mx":
        assert (sc[zero] == 0).all() and sc[2, 0] == 255
    if quant == "row":
        assert (sc[zero] == 2.0 ** -120).all() and torch.isnan(sc[2]) and (codes[2] & 0x7F == 0x7F).all()


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("f32", [False, True])
def test_backward(moe, T, K, f32):
    s, w, large = inputs(T, K, f32)
    g = torch.Generator(device="cuda").manual_seed(T)
    do = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    ds = torch.randn((T, K), generator=g, device="cuda").to(s.dtype)
    dr, dx = torch.full_like(s, 7.0), torch.full((T, K), 7.0, dtype=torch.bfloat16, device="cuda")
    dw, dw_rest = (torch.full((K,), 7.0, device="cuda") for _ in range(2))
    ws = torch.full((moe.moe_residual_norm_workspace_size(K),), 0xFF, dtype=torch.uint8, device="cuda")
    ctx = moe.Ctx(workspace=ws)
    moe.moe_residual_norm_backward(do, ds, s, None, w, T, K, 1e-5, 0.0, None, 0, dr, dx, dw, ctx)
    # the weight's gradient is that of the other rows alone
    moe.moe_residual_norm_backward(do, ds, s, (~large).to(torch.uint8), w, T, K, 1e-5, 0.0, None, 0, None, None, dw_rest, ctx)
    torch.cuda.synchronize()
    assert torch.equal(dr[large], ds[large]) and torch.equal(dx[large], ds[large].bfloat16())
    assert torch.isfinite(dr).all() and torch.equal(dw, dw_rest)
