"""SwiGLU of moe_dense_gemm with fp32 outputs: silu(z) u to fp32 precision, not to that of a bf16 output.

One product per sum (the other elements of x are zero), so z and u are exact.  Bound, in units of
2^-23 of the result: the exponential is within 2 ulp, the sum 1 + e adds half a unit, and so do the division
and the product with u: 3.5, and 4 with the terms of second order.  Below z = -88 the exponential
overflows and the result is 0, at most 88 e^-88 |u| < 6e-37 |u| away."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,kernel", [(200, 264, "split"), (37, 66, "split"), (4096, 4104, "pairs"), (4097, 4101, "pairs")])
def test_fp32_swiglu(M, N, kernel):
    import mixture_experts_grouped_align_gb300 as moe
    moe.build()
    moe.load()
    K = 8
    assert moe.moe_dense_gemm_plan(M, N, K, "swiglu", True)["kernel"] == kernel
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[:, 3] = torch.rand(M, generator=g, device="cuda") + 0.5
    w = torch.zeros((2 * N, K), dtype=torch.bfloat16, device="cuda")
    w[:N, 3] = (torch.rand(N, generator=g, device="cuda") - 0.5) * 140
    w[N:, 3] = torch.randn(N, generator=g, device="cuda")
    out = torch.empty((M, N), device="cuda")
    moe.moe_dense_gemm(x, w, "nk", None, None, 1.0, M, N, K, "swiglu", out)
    z = x[:, 3:4].double() * w[:, 3].double()[None]
    z, u = z[:, :N], z[:, N:]
    e = torch.exp(-z.abs())
    ref = z * torch.where(z >= 0, torch.ones_like(e), e) / (1 + e) * u
    assert bool(((out.double() - ref).abs() <= 4 * 2.0 ** -23 * ref.abs() + 6e-37 * u.abs()).all())
