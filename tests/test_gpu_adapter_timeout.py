"""Failure detection of moe_adapter_gemm's kernels for long requests, without a GPU fault: with the
stall self-test switch on, both launch with their copy and MMA roles off, so that the other roles wait
on barriers that nothing arrives on.  Every wait is bounded: the call must report MOE_ERR_TIMEOUT in
the device status word within a second, and the next call on the same workspace must be right.

Bounds: those of the kernel's own tests (2^-13 of the sum of magnitudes, and the output's rounding).
"""
import time

import numpy as np
import pytest

import synth
from helpers import bf16_half_ulp, bf16_to_np
from oracle import adapter as oracle, formats

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
MOE_ERR_TIMEOUT = -7


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_grouped_align_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.build()
    m.load()
    yield m
    m.moe_debug_stall_tensor_kernels(0)


def bf(a):
    bits = synth.to_bf16_bits(np.asarray(a, dtype=np.float64))
    return torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16).cuda(), formats.bf16_decode(bits)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("has_base", [False, True])
def test_stalled_waits_time_out_and_the_next_call_is_right(moe, f32, has_base):
    """Four requests, one without an adapter; tiles of 128 rows and shorter ones, runs that cut them."""
    rng = np.random.default_rng(31)
    M, N, K, r, L = 9000, 384, 320, 24, 3
    offsets, ids = [0, 3000, 5560, 7001, 9000], [2, -1, 0, 2]
    assert moe.moe_adapter_gemm_plan(M, N, K, r, L, 4) == "long"
    (x, xv), (a, av), (b, bv) = bf(rng.standard_normal((M, K))), bf(rng.standard_normal((L, r, K)) / 16), bf(rng.standard_normal((L, N, r)))
    base = torch.from_numpy(rng.standard_normal((M, N)).astype(np.float32)).cuda().to(torch.float32 if f32 else torch.bfloat16)
    out = torch.empty_like(base)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = torch.full((moe.moe_adapter_gemm_workspace_size(M, 4, r),), 0xFF, dtype=torch.uint8, device="cuda")
    off, ad = (torch.tensor(t, dtype=torch.int32, device="cuda") for t in (offsets, ids))
    ctx = moe.Ctx(workspace=ws, dev_status=status)

    def call():
        moe.moe_adapter_gemm(x, a, b, None, off, ad, base if has_base else None, M, N, K, r, L, 4, out, ctx)
        torch.cuda.synchronize()

    call()
    assert int(status[0]) == 0
    try:
        moe.moe_debug_stall_tensor_kernels(5_000)  # 5 us limit on every wait
        t0 = time.perf_counter()
        call()
        elapsed = time.perf_counter() - t0
    finally:
        moe.moe_debug_stall_tensor_kernels(0)
    assert int(status[0]) == MOE_ERR_TIMEOUT
    assert elapsed < 1.0, elapsed
    status.zero_()
    out.fill_(float("nan"))
    call()
    assert int(status[0]) == 0
    base64 = base.double().cpu().numpy() if has_base else np.zeros((M, N))
    ref, mag = oracle.adapter_gemm(xv, av, bv, None, offsets, ids, base64)
    got = out.double().cpu().numpy() if f32 else bf16_to_np(out)
    half = np.abs(ref) * 2.0 ** -24 if f32 else bf16_half_ulp(ref) * (1 + 2.0 ** -7)
    assert np.all(np.abs(got - ref) - half <= mag * 2.0 ** -13)
