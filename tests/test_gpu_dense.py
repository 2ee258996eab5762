"""moe_dense_gemm and moe_dense_bias_grad on the GPU against float64.

Bounds.  Products of bf16 are exact in fp32.  An MMA adds 16 of them to the accumulator and may
lose one unit of 2^-23 of the largest magnitude in flight for each of them, and the accumulator
one more: |z error| <= (K + K/16 + 32) 2^-23 S, S = sum_k |x_k w_k| + |b|, is generous for every
order of summation.  silu' is below 1.1 and silu(z) below |z|, the fast exponential is within
2 + 1.173 |z| ulp; relu^2 has the slope 2 |z|.  Then one rounding to the output type (bf16: half
an ulp; fp32: 2^-24 relative).
"""
import numpy as np
import pytest

import synth
from helpers import bf16_half_ulp
from oracle import formats

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


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


def reference(x, w, bias, act, residual, scale):
    """float64 result and its bound (before the output's rounding); w [N1, K]."""
    K = x.shape[1]
    z = x @ w.T + (0 if bias is None else bias)
    S = np.abs(x) @ np.abs(w).T + (0 if bias is None else np.abs(bias))
    e = (K + K / 16 + 32) * 2.0 ** -23 * S
    if act == "swiglu":
        n = z.shape[1] // 2
        g, u = z[:, :n], z[:, n:]
        s = sigmoid(g)
        out = g * s * u
        err = 1.1 * e[:, :n] * (np.abs(u) + e[:, n:]) + np.abs(g * s) * e[:, n:] + \
            (8 + 1.2 * np.abs(g)) * 2.0 ** -23 * np.abs(out)
    elif act == "relu2":
        out = np.maximum(z, 0) ** 2
        err = 2 * np.maximum(z, 0) * e + e * e + 2.0 ** -23 * out
    else:
        out, err = z, e
    if residual is not None:
        err = err + 2.0 ** -22 * (np.abs(out) + np.abs(scale * residual))
        out = out + scale * residual
    return out, err


def near(got, ref, err, f32):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    half = np.abs(ref) * 2.0 ** -24 + 1e-38 if f32 else bf16_half_ulp(np.abs(ref) + err)
    bad = np.abs(got - ref) > err + half * (1 + 2.0 ** -6)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], float(np.max(np.abs(got - ref) - err - half)))


def make(M, N, K, act, layout, bias, residual, f32, seed):
    rng = np.random.default_rng(seed)
    n1 = 2 * N if act == "swiglu" else N
    xt, x = bf(rng.standard_normal((M, K)))
    wt, w = bf(rng.standard_normal((n1, K)) * 0.05)
    if layout == "kn":
        wt = wt.t().contiguous()
    bt, b = bf(rng.standard_normal(n1)) if bias else (None, None)
    rt = r = None
    if residual:
        if f32:
            r = rng.standard_normal((M, N)).astype(np.float32)
            rt, r = torch.from_numpy(r).cuda(), r.astype(np.float64)
        else:
            rt, r = bf(rng.standard_normal((M, N)))
    return xt, x, wt, w, bt, b, rt, r


def run(moe, M, N, K, act, layout, bias, residual, f32, seed=0, scale=0.75):
    xt, x, wt, w, bt, b, rt, r = make(M, N, K, act, layout, bias, residual, f32, seed)
    guard = 64  # elements behind the output that must stay as they are
    buf = torch.full((M * N + guard,), 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    moe.moe_dense_gemm(xt, wt, layout, bt, rt, scale, M, N, K, act, buf, moe.Ctx(dev_status=status))
    torch.cuda.synchronize()
    assert int(status[0]) == 0 and bool((buf[M * N:] == 7).all())
    ref, err = reference(x, w, b, act, r, scale)
    near(buf[:M * N].view(M, N), ref, err, f32)


# few rows or columns: the split kernel, at each of its row tiles
@pytest.mark.parametrize("act", ["none", "relu2", "swiglu"])
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (1, 1856, 2688), (2, 136, 64), (17, 264, 520), (33, 128, 1000),
                                   (64, 328, 2880), (65, 40, 72), (129, 256, 136), (200, 904, 264), (257, 8, 4104)])
def test_few_rows(moe, M, N, K, layout, act):
    run(moe, M, N, K, act, layout, True, False, False, seed=M + N)


# more tiles than SMs: the tiled kernel, several tiles a block, ragged in every direction
@pytest.mark.parametrize("act", ["none", "relu2", "swiglu"])
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("M,N,K", [(2500, 2056, 72), (4097, 4104, 8), (1291, 5128, 328)])
def test_many_tiles(moe, M, N, K, layout, act):
    run(moe, M, N, K, act, layout, True, True, False, seed=K)


@pytest.mark.parametrize("M,N,K", [(1, 264, 136), (70, 1000, 264), (300, 128, 3000), (2500, 2056, 72), (4099, 256, 1024)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("residual", [False, True])
def test_fp32_outputs(moe, M, N, K, act, residual):
    run(moe, M, N, K, act, "nk", residual, residual, True, seed=N)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("act", ["none", "swiglu", "relu2"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 8), (5, 31, 64), (40, 7, 136), (130, 129, 72), (3000, 1999, 72), (2600, 2001, 24),
                                   (1501, 3502, 40)])
def test_odd_widths(moe, M, N, K, act, f32):
    run(moe, M, N, K, act, "nk", True, True, f32, seed=M)


@pytest.mark.parametrize("M,N,K,f32", [(9, 264, 128, False), (3000, 2056, 72, False), (3000, 2056, 72, True), (3000, 1999, 72, True)])
def test_accumulates_in_place(moe, M, N, K, f32):
    xt, x, wt, w, _, _, rt, r = make(M, N, K, "none", "nk", False, True, f32, 5)
    out = rt.clone()
    moe.moe_dense_gemm(xt, wt, "nk", None, out, 1.0, M, N, K, "none", out)
    torch.cuda.synchronize()
    ref, err = reference(x, w, None, "none", r, 1.0)
    near(out, ref, err, f32)


@pytest.mark.parametrize("M,N,K", [(50, 264, 520), (3000, 2056, 136)])
def test_non_finite_rows_stay_rows(moe, M, N, K):
    """NaN and infinity in a row of x reach that row of out only; past-the-end rows stay out."""
    xt, _, wt, _, _, _, _, _ = make(M, N, K, "none", "nk", False, False, False, 6)
    clean = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_dense_gemm(xt, wt, "nk", None, None, 1.0, M, N, K, "none", clean)
    xt[3, 5] = float("nan")
    xt[M - 1, 0] = float("inf")
    out = torch.empty_like(clean)
    moe.moe_dense_gemm(xt, wt, "nk", None, None, 1.0, M, N, K, "none", out)
    torch.cuda.synchronize()
    keep = [i for i in range(M) if i not in (3, M - 1)]
    assert torch.equal(out[keep], clean[keep]) and torch.isnan(out[3]).all() and not torch.isfinite(out[M - 1]).any()


@pytest.mark.parametrize("M,N,K", [(64, 2880, 2880), (4096, 2056, 264)])
def test_same_bits_again_on_another_stream_and_in_a_graph(moe, M, N, K):
    xt, _, wt, _, bt, _, rt, _ = make(M, N, K, "none", "nk", True, True, False, 7)
    outs = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    moe.moe_dense_gemm(xt, wt, "nk", bt, rt, 1.0, M, N, K, "none", outs[0])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        moe.moe_dense_gemm(xt, wt, "nk", bt, rt, 1.0, M, N, K, "none", outs[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        moe.moe_dense_gemm(xt, wt, "nk", bt, rt, 1.0, M, N, K, "none", outs[2], moe.Ctx(stream=s))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_offsets_past_32_bits(moe):
    """More than 2^31 output elements: the last rows are where 32-bit offsets would go wrong."""
    M, N, K = (1 << 20) + 77, 2056, 64
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn((N, K), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    moe.moe_dense_gemm(x, w, "nk", None, None, 1.0, M, N, K, "none", out)
    torch.cuda.synchronize()
    rows = torch.tensor([0, 1, M // 2, M - 129, M - 78, M - 2, M - 1], device="cuda")
    ref, err = reference(x[rows].double().cpu().numpy(), w.double().cpu().numpy(), None, "none", None, 1.0)
    near(out[rows], ref, err, False)
    d = torch.empty(N, device="cuda")
    moe.moe_dense_bias_grad(out, M, N, d)
    torch.cuda.synchronize()
    cols = torch.tensor([0, 1, 2048, N - 1], device="cuda")
    want, mag = out[:, cols].double().sum(0), out[:, cols].double().abs().sum(0)
    assert bool(((d[cols].double() - want).abs() <= mag * (M / 128 + 64) * 2.0 ** -24).all())


def test_gradients_are_the_difference_quotients(moe):
    """dx through moe_dense_gemm on the other layout and db through moe_dense_bias_grad, against
    differences of sum(dz * out) in float64."""
    M, N, K = 24, 40, 64
    xt, x, wt, w, bt, b, _, _ = make(M, N, K, "none", "nk", True, False, False, 9)
    dzt, dz = bf(np.random.default_rng(10).standard_normal((M, N)))
    dx = torch.empty((M, K), dtype=torch.float32, device="cuda")
    db = torch.empty(N, device="cuda")
    moe.moe_dense_gemm(dzt, wt, "kn", None, None, 1.0, M, K, N, "none", dx)
    moe.moe_dense_bias_grad(dzt, M, N, db)
    torch.cuda.synchronize()
    f = lambda x, b: float((dz * (x @ w.T + b)).sum())  # noqa: E731
    h = 1e-3
    rng = np.random.default_rng(11)
    for _ in range(20):
        i, k, n = rng.integers(M), rng.integers(K), rng.integers(N)
        xp, xm = x.copy(), x.copy()
        xp[i, k] += h
        xm[i, k] -= h
        assert abs((f(xp, b) - f(xm, b)) / (2 * h) - float(dx[i, k])) < 1e-4
        bp, bm = b.copy(), b.copy()
        bp[n] += h
        bm[n] -= h
        assert abs((f(x, bp) - f(x, bm)) / (2 * h) - float(db[n])) < 1e-4


@pytest.mark.parametrize("M,N", [(0, 64), (1, 1), (7, 31), (16, 128), (129, 130), (1000, 256), (8191, 520), (5, 7168)])
def test_bias_grad(moe, M, N):
    rng = np.random.default_rng(M + N)
    t, v = bf(rng.standard_normal((max(M, 1), N)))
    buf = torch.full((N + 16,), 7.0, device="cuda")
    moe.moe_dense_bias_grad(t if M else None, M, N, buf)
    torch.cuda.synchronize()
    v = v[:M]
    got = buf.cpu().numpy().astype(np.float64)
    assert (got[N:] == 7).all()
    # at most M / 128 additions in a thread, 16 of threads and 8 of CTAs, each within 2^-24
    assert np.all(np.abs(got[:N] - v.sum(axis=0)) <= (M / 128 + 32) * 2.0 ** -24 * np.abs(v).sum(axis=0) + 1e-38)


@pytest.mark.parametrize("M,N", [(2000, 8), (2300, 31), (2001, 40), (2047, 1999), (9001, 2048), (60001, 72)])
def test_bias_grad_of_many_rows(moe, M, N):
    rng = np.random.default_rng(M + N)
    t, v = bf(rng.standard_normal((M, N)) + 1)
    buf = torch.full((N + 16,), 7.0, device="cuda")
    moe.moe_dense_bias_grad(t, M, N, buf)
    again = torch.full((N + 16,), 7.0, device="cuda")
    moe.moe_dense_bias_grad(t, M, N, again)
    torch.cuda.synchronize()
    assert torch.equal(buf, again)
    got = buf.cpu().numpy().astype(np.float64)
    assert (got[N:] == 7).all()
    # at most M / 256 additions in a thread, 64 of threads and 8 of CTAs, each within 2^-24
    assert np.all(np.abs(got[:N] - v.sum(axis=0)) <= (M / 256 + 72) * 2.0 ** -24 * np.abs(v).sum(axis=0))


@pytest.mark.parametrize("M,N,K", [(40, 264, 520), (3000, 2056, 136)])
def test_waits_that_run_out_are_reported(moe, M, N, K):
    """With the copy and MMA roles off, both kernels give up, say so, and leave the context usable."""
    xt, x, wt, w, _, _, _, _ = make(M, N, K, "none", "nk", False, False, False, 12)
    out = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    moe.moe_debug_stall_tensor_kernels(2_000_000)
    try:
        moe.moe_dense_gemm(xt, wt, "nk", None, None, 1.0, M, N, K, "none", out, moe.Ctx(dev_status=status))
        torch.cuda.synchronize()
        assert int(status[0]) == -7
    finally:
        moe.moe_debug_stall_tensor_kernels(0)
    status.zero_()
    moe.moe_dense_gemm(xt, wt, "nk", None, None, 1.0, M, N, K, "none", out, moe.Ctx(dev_status=status))
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    ref, err = reference(x, w, None, "none", None, 1.0)
    near(out, ref, err, False)


@pytest.mark.parametrize("act,residual", [("none", True), ("swiglu", False), ("swiglu", True), ("relu2", False)])
@pytest.mark.parametrize("M,N,K", [(2500, 2056, 1600), (2049, 1999, 904), (3000, 2052, 776)])
def test_fp32_outputs_of_several_accumulators(moe, M, N, K, act, residual):
    """Long sums on the pairs' kernel: chunks of K added up by the epilogue, a ragged last one."""
    run(moe, M, N, K, act, "nk", True, residual, True, seed=K)


@pytest.mark.parametrize("M,N,layout", [(500, 128, "nk"), (4099, 256, "nk"), (4096, 4096, "nk"), (4096, 4096, "kn"), (33, 264, "kn")])
def test_fp32_outputs_keep_their_precision(moe, M, N, layout):
    """An accumulator takes at most 14 stages of 64, each of which costs it 6e-8 of its value at the
    most; the sums over accumulators round to nearest: below 1e-6 in all, whatever K is."""
    K = 7168
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn((N, K) if layout == "nk" else (K, N), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty((M, N), device="cuda")
    moe.moe_dense_gemm(x, w, layout, None, None, 1.0, M, N, K, "none", out)
    torch.cuda.synchronize()
    ref = x.double() @ (w.double().t() if layout == "nk" else w.double())
    assert float((out.double() - ref).norm() / ref.norm()) < 1e-6
