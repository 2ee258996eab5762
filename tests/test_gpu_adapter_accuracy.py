"""What moe_adapter_gemm keeps of v = x A^T, held against v itself, not against the magnitudes that cancel in
it: on tiles of up to four rows, of more, on more tiles than CTAs, and on long requests.

1. Whole numbers x, a < 128 with sums below 2^24 are exact in fp32 in any order, and a B of single ones copies
   v.  Three bf16 numbers carry 24 bits: fp32 outputs equal v.  Two carry it within 2^-17: bf16 outputs beside
   a base of -bf16(v) have what is left of v within that and their half step (with one they would be 0).
2. Positive sums of 7168 products, where a truncating accumulator loses up to 2^-23 of the sum with every MMA of
   16 of K, always towards zero.  Long requests: fp32 outputs empty it every 48 MMAs, 48 x 2^-23; then eleven
   additions, v's parts, the second product's nine MMAs and the output: 16 x 2^-23 more, in all 2^-17.  Few rows:
   a warp's share is 56 MMAs at rank 16, and eight shares, 32 pieces and the same rest: below 2^-16.
"""
import numpy as np
import pytest

import synth
from helpers import bf16_half_ulp, bf16_to_np
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


def call(moe, x, a, b, offsets, ids, base, out, plan):
    (M, K), (L, N, r), R = x.shape, b.shape, len(ids)
    assert moe.moe_adapter_gemm_plan(M, N, K, r, L, R) == plan
    i32 = lambda t: torch.tensor(np.asarray(t), dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.full((moe.moe_adapter_gemm_workspace_size(M, R, r),), 0xFF, dtype=torch.uint8, device="cuda")
    moe.moe_adapter_gemm(x, a, b, None, i32(offsets), i32(ids), base, M, N, K, r, L, R, out, moe.Ctx(workspace=ws))
    torch.cuda.synchronize()
    return out.cpu().numpy().astype(np.float64) if out.dtype == torch.float32 else bf16_to_np(out)


SHAPES = [([0, 1, 2, 3], [2, 0, 1], 3, "few"), ([0, 20, 21, 45], [0, 1, 0], 3, "few"),
          (list(range(401)), [(i * 7) % 190 for i in range(400)], 190, "few"), ([0, 3000, 3100, 9000], [1, 0, 2], 3, "long")]


@pytest.mark.parametrize("offsets,ids,L,plan", SHAPES)
@pytest.mark.parametrize("r", [8, 24, 64, 128])
@pytest.mark.parametrize("f32", [False, True])
def test_v_is_carried(moe, offsets, ids, L, plan, r, f32):
    rng = np.random.default_rng(r + offsets[-1])
    M, K, N = offsets[-1], 512, 136
    x, xv = bf(rng.integers(0, 128, (M, K)))
    a, av = bf(rng.integers(0, 128, (L, r, K)))
    sel = np.zeros((L, N, r))
    sel[:, np.arange(N), np.arange(N) % r] = 1
    b, bv = bf(sel)
    v, _ = oracle.adapter_gemm(xv, av, bv, None, offsets, ids, np.zeros((M, N)))
    assert 2 ** 20 < v.max() < 2 ** 24 and (v % 2 == 1).any()  # more bits than two bf16 numbers have
    if f32:
        got = call(moe, x, a, b, offsets, ids, None, torch.empty((M, N), dtype=torch.float32, device="cuda"), plan)
        assert np.array_equal(got, v)
        return
    base, base_v = bf(-v)
    ref = v + base_v
    assert np.abs(ref).max() > v.max() * 2.0 ** -10
    got = call(moe, x, a, b, offsets, ids, base, torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), plan)
    # the rounding of what is kept: half a step of a number up to 2^-17 v larger
    assert np.all(np.abs(got - ref) <= v * 2.0 ** -17 + bf16_half_ulp(np.abs(ref) + v * 2.0 ** -17))


@pytest.mark.parametrize("offsets,ids,L,plan,tol", [
    (list(range(401)), [(i * 7) % 190 for i in range(400)], 190, "few", 2.0 ** -16), ([0, 1, 2, 3], [2, 0, 1], 3, "few", 2.0 ** -16),
    ([0, 20, 21, 45], [0, 1, 0], 3, "few", 2.0 ** -16), ([0, 3000, 3100, 9000], [1, 0, 2], 3, "long", 2.0 ** -17)])
def test_long_positive_sums(moe, offsets, ids, L, plan, tol):
    rng = np.random.default_rng(offsets[-1])
    M, K, N, r = offsets[-1], 7168, 136, 16
    x, xv = bf(rng.uniform(0.5, 1.5, (M, K)))
    a, av = bf(rng.uniform(0.5, 1.5, (L, r, K)) / K)
    b, bv = bf(rng.uniform(0.5, 1.5, (L, N, r)))
    ref, _ = oracle.adapter_gemm(xv, av, bv, None, offsets, ids, np.zeros((M, N)))
    got = call(moe, x, a, b, offsets, ids, None, torch.empty((M, N), dtype=torch.float32, device="cuda"), plan)
    assert np.all(np.abs(got - ref) <= ref * tol)
