"""Row-scaled codes of rows so small that 448 / max |s w| or max |s w| itself leaves fp32's normal range,
against the float64 oracle: the smallest scale 2^-120 and those above it, on each kernel.

Bounds.  n = (s r) w: the sum of squares has at most 70 roundings of 2^-24 one after another (ordinary rows; in
the others it vanishes beside eps), half of that is in r, and five more follow: |n| 2^-18, and 2^-149 below
the normal numbers.  The scale: 2^-17.  Codes lie between those of n less and n plus its bound, by the scale
that was stored and 2^-22 for its reciprocal and the product.
"""
import numpy as np
import pytest

import synth
from helpers import bf16_to_np
from oracle import formats, mx_quant, residual_norm

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
# largest |s| of a row, weights near 1: above and below 448 / FLT_MAX = 1.32e-36, 2^-120 * 448 eps^(1/2) for
# each eps, 2^-126 = 1.18e-38, and down to the smallest subnormal number; ordinary rows and zeros between
TOPS = [1.0, 1.6e-36, 1.33e-36, 1.31e-36, 0.0, 1.2e-36, 1.08e-36, 1.05e-36, 9e-37, 3.5e-37, 3.3e-37, 1e-37, 1.2e-38, 2.0, 1.1e-38,
        1e-39, 1.4e-40, 1e-41, 1e-43, 3e-45]


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


@pytest.mark.parametrize("T,K,f32", [(40, 64, True), (45, 256, False), (40, 256, True), (40, 2880, True), (60, 2880, False), (40, 12288, False),
                                     (6400, 256, True), (3200, 512, False), (1700, 1024, True), (700, 2880, False), (900, 7168, False),
                                     (140, 12288, False)])
@pytest.mark.parametrize("eps", [1e-5, 1e-6, 1e-12, 1e-30])
@pytest.mark.parametrize("out", [False, True])
def test_row_codes_of_tiny_rows(moe, T, K, f32, eps, out):
    rng = np.random.default_rng(T + K)
    shape = rng.uniform(-1, 1, (T, K))
    shape[:, ::7] = 0.0
    shape[:, 1] = 1.0
    res = shape * np.resize(TOPS, T)[:, None]
    if f32:
        rv = res.astype(np.float32)
        r, rv = torch.from_numpy(rv).cuda(), rv.astype(np.float64)
    else:
        r, rv = bf(res)
    w, wv = bf(rng.uniform(0.9, 1.0, K))
    mask = (rng.random(T) < 0.9).astype(np.uint8)
    m = torch.from_numpy(mask).cuda()
    codes = torch.full((T, K), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((T,), float("nan"), dtype=torch.float32, device="cuda")
    o = torch.full((T, K), float("nan"), dtype=torch.bfloat16, device="cuda") if out else None
    moe.moe_residual_norm(None, r, m, w, T, K, eps, 0.0, None, 0, None, o, codes, scales)
    torch.cuda.synchronize()
    _, n = residual_norm.forward(None, rv, wv, float(np.float32(eps)), 1.0, mask)
    dn = np.abs(n) * 2.0 ** -18 + 2.0 ** -149
    unit = scales.cpu().numpy().astype(np.float64)
    want = np.maximum(np.abs(n).max(axis=1) / 448, 2.0 ** -120)
    assert np.all(np.abs(unit - want) <= want * 2.0 ** -17)
    got = formats.e4m3_decode(codes.cpu().numpy())
    lo, hi = (formats.e4m3_decode(mx_quant.e4m3_encode((n + s * (dn + np.abs(n) * 2.0 ** -22)) / unit[:, None])) for s in (-1, 1))
    assert np.all((lo <= got) & (got <= hi))  # NaN is neither
    assert np.all(got[n == 0] == 0)
    if out:
        assert np.all(np.abs(bf16_to_np(o) - n) <= np.abs(n) * (2.0 ** -8 * (1 + 2.0 ** -17) + 2.0 ** -18) + 2.0 ** -133)
