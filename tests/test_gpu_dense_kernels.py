"""moe_dense_gemm's two kernels on the GPU, each named: every case says which kernel its shape is for
and asks moe_dense_gemm_plan before it runs.  Bounds and references are test_gpu_dense's."""
import pytest

from test_gpu_dense import make, moe, near, reference, run  # noqa: F401 (moe is a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def plan(moe, M, N, K, act, f32, kernel):  # noqa: F811
    p = moe.moe_dense_gemm_plan(M, N, K, act, f32)
    assert p["kernel"] == kernel, (M, N, K, act, f32, p)
    return p


ACTS = ["none", "relu2", "swiglu"]
PAIRS = [(4096, 4104, 1032), (4097, 4104, 200), (2500, 4104, 520)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("M,N,K", PAIRS)
def test_pairs(moe, M, N, K, layout, act):  # noqa: F811
    """Several stages of K and several tiles a pair, ragged in every direction, with bias and residual."""
    plan(moe, M, N, K, act, False, "pairs")
    run(moe, M, N, K, act, layout, True, True, False, seed=K)


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_pairs_without_residual_and_in_fp32(moe, layout, act):  # noqa: F811
    M, N, K = PAIRS[2]
    for f32 in (False, True):
        plan(moe, M, N, K, act, f32, "pairs")
        run(moe, M, N, K, act, layout, False, False, f32, seed=1)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(4097, 4101, 1032), (5000, 3501, 328), (4096, 4100, 264)])
def test_pairs_of_odd_widths(moe, M, N, K, act, f32):  # noqa: F811
    """Rows of out that are no multiple of 16 bytes: stored without the box."""
    plan(moe, M, N, K, act, f32, "pairs")
    run(moe, M, N, K, act, "nk", True, True, f32, seed=M)


@pytest.mark.parametrize("M,N,K,f32,kernel", [(4096, 4104, 1032, False, "pairs"), (4096, 4104, 1032, True, "pairs"),
                                              (4097, 4101, 1032, False, "pairs"), (4097, 4101, 1032, True, "pairs"),
                                              (300, 2880, 2880, False, "split"), (700, 4104, 264, True, "split")])
def test_accumulates_in_place(moe, M, N, K, f32, kernel):  # noqa: F811
    plan(moe, M, N, K, "none", f32, kernel)
    xt, x, wt, w, _, _, rt, r = make(M, N, K, "none", "nk", False, True, f32, 5)
    out = rt.clone()
    moe.moe_dense_gemm(xt, wt, "nk", None, out, 1.0, M, N, K, "none", out)
    torch.cuda.synchronize()
    ref, err = reference(x, w, None, "none", r, 1.0)
    near(out, ref, err, f32)


@pytest.mark.parametrize("M,N,K,kernel", [(4096, 4104, 1032, "pairs"), (300, 2880, 2880, "split")])
def test_non_finite_rows_stay_rows(moe, M, N, K, kernel):  # noqa: F811
    plan(moe, M, N, K, "none", False, kernel)
    xt, _, wt, _, _, _, _, _ = make(M, N, K, "none", "nk", False, False, False, 6)
    clean, out = (torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_dense_gemm(xt, wt, "nk", None, None, 1.0, M, N, K, "none", clean)
    xt[3, 5] = float("nan")
    xt[M - 1, 0] = float("inf")
    moe.moe_dense_gemm(xt, wt, "nk", None, None, 1.0, M, N, K, "none", out)
    torch.cuda.synchronize()
    keep = [i for i in range(M) if i not in (3, M - 1)]
    assert torch.equal(out[keep], clean[keep]) and torch.isnan(out[3]).all() and not torch.isfinite(out[M - 1]).any()


@pytest.mark.parametrize("M,N,K,kernel", [(4096, 4104, 1032, "pairs"), (300, 2880, 2880, "split")])
def test_same_bits_again_on_another_stream_and_in_a_graph(moe, M, N, K, kernel):  # noqa: F811
    plan(moe, M, N, K, "none", False, kernel)
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


@pytest.mark.parametrize("act,f32", [("none", False), ("none", True), ("swiglu", False), ("swiglu", True)])
@pytest.mark.parametrize("M,N,K,kernel", [(4096, 4104, 1032, "pairs"), (300, 2880, 2880, "split")])
def test_waits_that_run_out_are_reported(moe, M, N, K, act, f32, kernel):  # noqa: F811
    """With the copy and MMA roles off the kernel gives up, says so, and leaves the context usable."""
    plan(moe, M, N, K, act, f32, kernel)
    xt, x, wt, w, _, _, _, _ = make(M, N, K, act, "nk", False, False, f32, 12)
    out = torch.zeros((M, N), dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    moe.moe_debug_stall_tensor_kernels(2_000_000)
    try:
        moe.moe_dense_gemm(xt, wt, "nk", None, None, 1.0, M, N, K, act, out, moe.Ctx(dev_status=status))
        torch.cuda.synchronize()
        assert int(status[0]) == -7
    finally:
        moe.moe_debug_stall_tensor_kernels(0)
    status.zero_()
    moe.moe_dense_gemm(xt, wt, "nk", None, None, 1.0, M, N, K, act, out, moe.Ctx(dev_status=status))
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    ref, err = reference(x, w, None, act, None, 1.0)
    near(out, ref, err, f32)


SPLIT = [(64, 2880, 2880), (100, 2880, 2880), (129, 2048, 2048), (300, 2880, 2880), (500, 520, 2880), (257, 520, 4104),
         (2000, 512, 2048), (1100, 7168, 264), (3000, 2056, 136), (4000, 928, 264), (333, 4104, 2688), (2500, 2056, 1600),
         (700, 4104, 264), (600, 2056, 1000)]


def test_split_shapes_reach_what_they_are_for(moe):  # noqa: F811
    """Row tiles above 64, alone and in clusters, two weight tiles, rows that leave in two phases."""
    seen = [p for s in SPLIT for act in ("none", "swiglu") for p in [moe.moe_dense_gemm_plan(*s, act)] if p["kernel"] == "split"]
    assert len({p["rows"] for p in seen if p["rows"] > 64}) >= 5
    assert len({p["cluster"] for p in seen if p["rows"] > 64}) >= 4
    assert any(p["weight_tiles"] == 2 for p in seen) and any(p["phase"] < p["rows"] for p in seen)


@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("M,N,K", SPLIT)
def test_split(moe, M, N, K, layout):  # noqa: F811
    plan(moe, M, N, K, "none", False, "split")
    run(moe, M, N, K, "none", layout, True, True, False, seed=M)


@pytest.mark.parametrize("act,f32", [("swiglu", False), ("relu2", False), ("swiglu", True), ("none", True)])
@pytest.mark.parametrize("M,N,K", [(100, 2880, 2880), (500, 520, 2880), (257, 520, 4104), (2000, 512, 2048), (4000, 928, 264),
                                   (700, 4104, 264), (600, 2056, 1000)])
def test_split_activations(moe, M, N, K, act, f32):  # noqa: F811
    plan(moe, M, N, K, act, f32, "split")
    run(moe, M, N, K, act, "nk", True, False, f32, seed=N)
