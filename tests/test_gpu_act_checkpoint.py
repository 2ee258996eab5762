"""moe_act_checkpoint and moe_act_backward on the GPU against the float64 oracle.

The checkpoint is compared bit for bit (the quantiser is exact but for its one rounding).  bf16
outputs: half an ulp of the output (2^(e - 8) in the binade of 2^e) plus the fp32 evaluation, whose sigmoid is
within 2 + 1.173 |g| + 4 ulp of 2^-23; with |g| <= 64 in these tests that is below 2^-16 of the
terms' magnitudes.  d_row_w: 2^-16 of the sum of magnitudes (the same terms, and a sum of I of
them in lanes and a tree).
"""
import numpy as np
import pytest

import synth
from helpers import bf16_half_ulp, bf16_to_np
from oracle import activation, formats

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


def near_bf16(got, ref, mag):
    """Within half a bf16 ulp of ref (a subnormal step at the least) and 2^-16 of mag."""
    return np.abs(got - ref) <= bf16_half_ulp(ref) * (1 + 2.0 ** -7) + mag * 2.0 ** -16


def run(moe, z, dh, w, gated, again=True):
    R, I = dh.shape
    zt, zv = bf(z)
    dt, dv = bf(dh)
    wt = None if w is None else torch.from_numpy(w.astype(np.float32)).cuda()
    N1 = z.shape[1]
    h = torch.full((R, I), float("nan"), dtype=torch.bfloat16, device="cuda")
    codes = torch.full((R, N1), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((R, N1 // 32), 0xA5, dtype=torch.uint8, device="cuda")
    act = "swiglu" if gated else "relu2"
    moe.moe_act_checkpoint(zt, wt, R, I, act, h, codes, scales)
    dz = torch.full((R, N1), float("nan"), dtype=torch.bfloat16, device="cuda")
    h2 = torch.full((R, I), float("nan"), dtype=torch.bfloat16, device="cuda") if again else None
    dw = torch.full((R,), float("nan"), device="cuda") if again else None
    moe.moe_act_backward(codes, scales, dt, wt, R, I, act, dz, h2, dw)
    torch.cuda.synchronize()
    return zv, dv, h, codes, scales, dz, h2, dw


def check(moe, z, dh, w, gated):
    zv, dv, h, codes, scales, dz, h2, dw = run(moe, z, dh, w, gated)
    wf = None if w is None else w.astype(np.float32).astype(np.float64)
    out = np.zeros(len(zv), bool) if w is None else wf == 0
    oc, os_, v = activation.held(np.where(out[:, None], 0.0, zv))
    assert np.array_equal(scales.cpu().numpy(), os_)
    assert np.array_equal(codes.cpu().numpy(), oc)
    ref = activation.forward(zv, wf, gated)
    assert np.all(near_bf16(bf16_to_np(h), ref, np.abs(ref)))
    rz, rh, rw = activation.backward(v, dv, wf, gated)
    assert np.all(near_bf16(bf16_to_np(h2), rh, np.abs(rh)))
    mag = np.abs(rz)
    if gated:  # s (1 + g (1 - s)) cancels near its zero: its terms' magnitudes
        I = dv.shape[1]
        g, u = v[:, :I], v[:, I:]
        t = np.abs((1.0 if wf is None else wf[:, None]) * dv)
        mag[:, :I] = t * np.abs(u) * activation._sigmoid(g) * (1 + np.abs(g))
    assert np.all(near_bf16(bf16_to_np(dz), rz, mag))
    a = np.abs(rh) if wf is None else np.abs(activation.backward(v, dv, np.ones(len(v)), gated)[1]) * ~out[:, None]
    assert np.all(np.abs(dw.cpu().numpy() - rw) <= 2.0 ** -16 * (np.abs(dv) * a).sum(axis=1) + 1e-38)


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("R,I", [(1, 32), (1, 2880), (3, 64), (9, 96), (33, 160), (168, 928), (5, 5760),
                                 (1023, 288), (1024, 288), (1500, 512)])
def test_matches_oracle(moe, R, I, weighted, gated):
    rng = np.random.default_rng(R * 10000 + I)
    z = rng.standard_normal((R, 2 * I if gated else I)) * 2
    dh = rng.standard_normal((R, I)) * 0.05
    w = None
    if weighted:
        w = rng.uniform(0.01, 1, R)
        w[R // 2] = 0.0
    check(moe, z, dh, w, gated)


@pytest.mark.parametrize("gated", [True, False])
def test_blocks_of_many_octaves_zeros_and_extremes(moe, gated):
    rng = np.random.default_rng(21)
    R, I = 40, 64
    z = rng.standard_normal((R, 2 * I if gated else I)) * np.exp2(rng.integers(-30, 5, (R, 2 * I if gated else I)))
    z[0] = 0.0
    z[1] = -0.0
    z[2, :32] = 2.0 ** -126                    # the smallest normal
    z[3, :32] = 2.0 ** -133                    # a bf16 subnormal
    z[4] = 64.0
    z[5] = -64.0
    check(moe, z, rng.standard_normal((R, I)), None, gated)


def test_non_finite_values_stay_in_their_block(moe):
    rng = np.random.default_rng(22)
    R, I = 6, 96
    z = rng.standard_normal((R, 2 * I))
    dh = rng.standard_normal((R, I))
    clean = run(moe, z, dh, None, True)
    z[1, 33] = np.nan                          # gate, block 1
    z[2, I + 64] = np.inf                      # up, block 2
    got = run(moe, z, dh, None, True)
    oc, os_, _ = activation.held(got[0])
    assert np.array_equal(got[3].cpu().numpy(), oc) and np.array_equal(got[4].cpu().numpy(), os_)
    bad = np.zeros((R, I), bool)
    bad[1, 32:64] = True
    bad[2, 64:96] = True
    for i in (2, 6):
        a, b = bf16_to_np(clean[i]), bf16_to_np(got[i])
        assert np.array_equal(a[~bad], b[~bad])
    assert np.isnan(bf16_to_np(got[6])[1, 32:64]).all()
    assert np.isfinite(got[7].cpu().numpy()[[0, 3, 4, 5]]).all()


def test_rows_of_weight_zero_are_left_out_whatever_they_hold(moe):
    rng = np.random.default_rng(23)
    for R, I in ((4, 320), (2000, 64)):
        z = rng.standard_normal((R, 2 * I))
        dh = rng.standard_normal((R, I))
        z[1], dh[1] = np.nan, np.inf
        w = np.full(R, 0.5)
        w[1] = 0.0
        zv, dv, h, codes, scales, dz, h2, dw = run(moe, z, dh, w, True)
        for t in (h, dz, h2, codes, scales):
            assert not t[1].float().abs().any()
        assert float(dw[1]) == 0.0 and torch.isfinite(dz.float()).all() and torch.isfinite(dw).all()


def test_optional_outputs_and_streams(moe):
    rng = np.random.default_rng(24)
    z, dh = rng.standard_normal((70, 512)), rng.standard_normal((70, 256))
    full = run(moe, z, dh, None, True)
    part = run(moe, z, dh, None, True, again=False)
    assert torch.equal(full[5], part[5])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        other = run(moe, z, dh, None, True)
    for i in (2, 3, 4, 5, 6, 7):
        assert torch.equal(full[i], other[i])


def test_gradient_is_the_difference_quotient(moe):
    """d_gu against central differences of sum(dh * h) at the checkpoint's own values."""
    rng = np.random.default_rng(25)
    R, I = 3, 32
    z = rng.standard_normal((R, 2 * I))
    dh = rng.standard_normal((R, I))
    w = rng.uniform(0.2, 1, R).astype(np.float32)
    _, dv, _, codes, scales, dz, _, dw = run(moe, z, dh, w, True)
    v = formats.dequant_mxfp8(codes.cpu().numpy(), scales.cpu().numpy())
    f = lambda v, w: np.sum(dv * activation.forward(v, w, True), axis=1)  # noqa: E731
    h = 1e-5
    got = bf16_to_np(dz)
    for c in range(2 * I):
        vp, vm = v.copy(), v.copy()
        vp[:, c] += h
        vm[:, c] -= h
        q = (f(vp, w.astype(np.float64)) - f(vm, w.astype(np.float64))) / (2 * h)
        # half a bf16 ulp, and the quotient's own error (h^2 and rounding over h)
        assert np.all(np.abs(got[:, c] - q) <= 2.0 ** -8 * np.abs(q) + 1e-4 * 2.0 ** -8 + 1e-8)
    q = (f(v, w + 1e-3) - f(v, w - 1e-3)) / 2e-3
    assert np.allclose(dw.cpu().numpy(), q, rtol=1e-4, atol=1e-4)


def test_offsets_past_32_bits(moe):
    """More than 2^31 pre-activations: rows on both sides of the wrap against the oracle."""
    R, I = 400_000, 2880
    g = torch.Generator(device="cuda").manual_seed(26)
    z = torch.randn((R, 2 * I), generator=g, device="cuda", dtype=torch.bfloat16)
    dh = torch.randn((R, I), generator=g, device="cuda", dtype=torch.bfloat16)
    h, dz, codes = torch.empty_like(dh), torch.empty_like(z), torch.empty((R, 2 * I), dtype=torch.uint8, device="cuda")
    scales, dw = torch.empty((R, 2 * I // 32), dtype=torch.uint8, device="cuda"), torch.empty(R, device="cuda")
    moe.moe_act_checkpoint(z, None, R, I, "swiglu", h, codes, scales)
    moe.moe_act_backward(codes, scales, dh, None, R, I, "swiglu", dz, None, dw)
    torch.cuda.synchronize()
    wrap = 2 ** 31 // (2 * I)
    rows = torch.tensor([0, 1, wrap - 1, wrap, wrap + 1, 2 ** 32 // (2 * I) % R, R - 1], device="cuda")
    zv, dv = bf16_to_np(z[rows].contiguous()), bf16_to_np(dh[rows].contiguous())
    oc, os_, v = activation.held(zv)
    assert np.array_equal(codes[rows].cpu().numpy(), oc) and np.array_equal(scales[rows].cpu().numpy(), os_)
    ref = activation.forward(zv, None, True)
    assert np.all(near_bf16(bf16_to_np(h[rows].contiguous()), ref, np.abs(ref)))
    rz, _, rw = activation.backward(v, dv, None, True)
    gate, u = v[:, :I], v[:, I:]
    mag = np.abs(rz)
    mag[:, :I] = np.abs(dv * u) * activation._sigmoid(gate) * (1 + np.abs(gate))
    assert np.all(near_bf16(bf16_to_np(dz[rows].contiguous()), rz, mag))
    a = np.abs(gate * activation._sigmoid(gate) * u)
    assert np.all(np.abs(dw[rows].cpu().numpy() - rw) <= 2.0 ** -16 * (np.abs(dv) * a).sum(axis=1))


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("R,I", [(2000, 512), (5000, 544), (1700, 2048), (20000, 352), (3000, 1056)])
def test_rows_of_several_turns(moe, R, I, gated):
    """A warp per row with two or four turns of columns, whole and ragged."""
    rng = np.random.default_rng(I)
    z = rng.standard_normal((R, 2 * I if gated else I)) * 2
    w = rng.uniform(0.01, 1, R)
    w[::7] = 0.0
    check(moe, z, rng.standard_normal((R, I)) * 0.05, w, gated)


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("R,I", [(100001, 32), (50003, 64), (33341, 96), (25009, 128), (20011, 160), (16673, 192), (14293, 224),
                                 (12503, 256), (8347, 384), (6257, 512), (4201, 768), (2301, 1408)])
def test_narrow_rows_in_turns(moe, R, I, gated):
    """Several rows a warp with up to four turns of columns each, the last rows and columns ragged."""
    rng = np.random.default_rng(R)
    z = rng.standard_normal((R, 2 * I if gated else I)) * np.exp2(rng.integers(-6, 4, (R, 1)))
    w = rng.random(R) + 0.1
    w[rng.random(R) < 0.1] = 0.0
    check(moe, z, rng.standard_normal((R, I)), w, gated)
