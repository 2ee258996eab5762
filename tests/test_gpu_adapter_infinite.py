"""Adapters of rows whose x, or whose products with A, are infinite: the formula's infinities, with their
signs, and the other rows' values.  All weights are positive, so that no sum meets infinities of both signs.

Bounds of the finite rows: positive terms, so a relative error holds: chains of fewer than 128 additions of at
most 2^-23, 2^-16 in all, v's two bf16 numbers 2^-17, and the output's half step: 2^-8 for bf16, 2^-24 for fp32.
"""
import numpy as np
import pytest

import synth
from helpers import bf16_to_np
from oracle import adapter as oracle, formats

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_grouped_align_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.build()
    m.load()
    return m


def bf(a):
    bits = synth.to_bf16_bits(np.asarray(a, dtype=np.float64))
    return torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16).cuda(), formats.bf16_decode(bits)


# up to four rows of an adapter, tiles of more, long requests
@pytest.mark.parametrize("offsets,plan", [([0, 1, 2, 3], "few"), ([0, 9, 20, 40], "few"), ([0, 3000, 9000, 9400], "long")])
@pytest.mark.parametrize("r", [8, 24, 128])
@pytest.mark.parametrize("f32", [False, True])
def test_infinite_rows(moe, offsets, plan, r, f32):
    rng = np.random.default_rng(r + offsets[-1])
    M, N, K, L, ids = offsets[-1], 136, 72, 3, [0, 2, 1]
    assert moe.moe_adapter_gemm_plan(M, N, K, r, L, 3) == plan
    xs = rng.uniform(0.5, 1.5, (M, K))
    inf, over = [0, M - 1], M // 2
    xs[inf[0], 5], xs[inf[1], K - 1] = np.inf, -np.inf
    xs[over, 8:12] = 3e38
    x, xv = bf(xs)
    a, av = bf(rng.uniform(0.5, 1, (L, r, K)))
    b, bv = bf(rng.uniform(0.5, 1, (L, N, r)))
    sv = np.array([2.0, 1.0, -0.5], dtype=np.float32)
    out = torch.empty((M, N), dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_adapter_gemm_workspace_size(M, 3, r), dtype=torch.uint8, device="cuda")
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")  # noqa: E731
    moe.moe_adapter_gemm(x, a, b, torch.from_numpy(sv).cuda(), i32(offsets), i32(ids), None, M, N, K, r, L, 3, out,
                         moe.Ctx(workspace=ws))
    torch.cuda.synchronize()
    got = out.cpu().numpy().astype(np.float64) if f32 else bf16_to_np(out)
    ref, _ = oracle.adapter_gemm(xv, av, bv, sv.astype(np.float64), offsets, ids, np.zeros((M, N)))
    sign = np.sign(sv[oracle.row_adapters(M, offsets, ids)])
    assert (ref[over] * sign[over] > 3.5e38).all()  # above fp32's range, by sums above it
    assert (got[inf[0]] == np.inf * sign[inf[0]]).all() and (got[inf[1]] == -np.inf * sign[inf[1]]).all()
    assert (got[over] == np.inf * sign[over]).all()
    fine = np.setdiff1d(np.arange(M), inf + [over])
    tol = 2.0 ** -16 + 2.0 ** -17 + (2.0 ** -24 if f32 else 2.0 ** -8 * (1 + 2.0 ** -7))
    assert np.all(np.abs(got[fine] - ref[fine]) <= np.abs(ref[fine]) * tol)


@pytest.mark.parametrize("rows,plan", [(1, "few"), (9, "few"), (9000, "long")])
def test_sums_next_to_the_largest_number(moe, rows, plan):
    """v above bf16's largest number and within fp32's: its first bf16 number rounds to an infinity, which the
    others must not meet with one of the other sign."""
    M, N, K, r = rows, 64, 8, 8
    assert moe.moe_adapter_gemm_plan(M, N, K, r, 1, 1) == plan
    xs = np.zeros((M, K))
    xs[:, 0], xs[:, 1] = 3.38e38, 2.2e36  # bf16 numbers whose sum is about 3.398e38
    (x, xv), (a, _), (b, _) = bf(xs), bf(np.ones((1, r, K))), bf(np.full((1, N, r), 2.0 ** -10))
    assert 3.3961e38 < xv[0].sum() < 3.4028e38
    out = torch.empty((M, N), dtype=torch.float32, device="cuda")
    ws = torch.empty(moe.moe_adapter_gemm_workspace_size(M, 1, r), dtype=torch.uint8, device="cuda")
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")  # noqa: E731
    moe.moe_adapter_gemm(x, a, b, None, i32([0, M]), i32([0]), None, M, N, K, r, 1, 1, out, moe.Ctx(workspace=ws))
    torch.cuda.synchronize()
    got, want = out.cpu().numpy().astype(np.float64), xv[0].sum() * r * 2.0 ** -10
    assert np.all(np.abs(got - want) <= want * 2.0 ** -20)
