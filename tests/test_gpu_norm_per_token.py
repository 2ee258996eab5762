"""The residual norm's row-scaled codes as the operand of the per-token FP8 product, as they are used: padding
rows (zeros) and rows whose values are tiny among them.  The product is held against the float64 oracle on the
codes that the norm wrote, and the pair of calls against float64 products of the norm without its rounding:
a code is within 2^-4 of its value, or within half a step of 2^-9 of its row's scale, so the error's norm is
below 2^-4 of the product of the operands' magnitudes; of independent signs it stays below 2^-4 of the result's.
"""
import numpy as np
import pytest

import synth
from helpers import assert_close_bf16, bf16_to_np, dev
from oracle import formats, per_token, residual_norm

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,f32", [(1, 256, False), (77, 2688, True), (300, 7168, False)])
def test_norm_into_the_per_token_product(T, K, f32):
    import mixture_experts_grouped_align_gb300 as moe
    moe.build()
    moe.load()
    rng = np.random.default_rng(T)
    E, N, eps = 3, 128, 1e-5
    sizes = np.array([T - T // 2 - T // 3, T // 2, T // 3], dtype=np.int32)
    x = synth.to_bf16_bits(rng.standard_normal((T, K)))
    res = rng.standard_normal((T, K)) * 2
    xv = formats.bf16_decode(x)
    if T > 1:
        xv = xv.copy()
        xv[5] = 0
        x = synth.to_bf16_bits(xv)
        res[5] *= 2.0 ** -60
    mask = np.ones(T, np.uint8)
    mask[T // 2 + 1:T // 2 + 4] = 0
    if f32:
        rv = res.astype(np.float32)
        r, rv = torch.from_numpy(rv).cuda(), rv.astype(np.float64)
    else:
        bits = synth.to_bf16_bits(res)
        r, rv = dev(bits), formats.bf16_decode(bits)
    nw = synth.to_bf16_bits(rng.uniform(0.5, 1.5, K))
    w = rng.integers(0, 256, (E, N, K), dtype=np.uint8)
    w = np.where((w & 0x7F) == 0x7F, w - 1, w).astype(np.uint8)
    sw = rng.uniform(2.0 ** -10, 2.0 ** -6, E).astype(np.float32)
    codes = torch.empty((T, K), dtype=torch.uint8, device="cuda")
    scales = torch.empty(T, dtype=torch.float32, device="cuda")
    out = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    ctx = moe.Ctx(dev_status=status)
    moe.moe_residual_norm(dev(x), r, dev(mask), dev(nw), T, K, eps, 0.0, None, 0, None, None, codes, scales, ctx)
    moe.moe_gemm_per_token(E, N, K, codes, scales, dev(w), dev(sw), None, dev(sizes), T, out, ctx)
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    got = bf16_to_np(out)
    ref = per_token.gemm_per_token(codes.cpu().numpy(), scales.cpu().numpy(), w, sw, None, sizes)
    assert_close_bf16(got, ref)
    _, n = residual_norm.forward(xv, rv, formats.bf16_decode(nw), eps, 1.0, mask)
    wv, group = formats.e4m3_decode(w) * sw[:, None, None], np.repeat(np.arange(E), sizes)
    full = np.stack([wv[g] @ n[t] for t, g in enumerate(group)])
    for t in range(T):
        assert np.linalg.norm(got[t] - full[t]) <= 2.0 ** -4 * np.linalg.norm(full[t]), t
    assert (got[mask == 0] == 0).all()
