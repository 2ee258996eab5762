"""moe_adapter_gemm on the GPU against the float64 oracle.

Bounds, relative to the sum of magnitudes |x| |a| |b|: the first product adds K exact products of bf16 in
fp32, in chains (a lane's, the tensor core's, at most 2^-23 of the running magnitude an addition); the
chains of the sizes here have fewer than 600 links: 2^-13.7, taken as 2^-13.  Two bf16 numbers carry it
within 2^-17; the second product's chain has at most 16 links.  Errors of independent signs stay far
below: the mean over all elements is held to 2^-18.  The output's rounding comes on top.
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


def i32(a):
    return torch.tensor(list(a), dtype=torch.int32, device="cuda")


def np64(t):
    return bf16_to_np(t) if t.dtype == torch.bfloat16 else t.cpu().numpy().astype(np.float64)


class Case:
    def __init__(self, M, N, K, r, L, offsets, adapter, f32=False, base="apart", scaled=True, seed=0):
        rng = np.random.default_rng(seed + M * 31 + N * 7 + K + r)
        self.M, self.N, self.K, self.r, self.L, self.R, self.f32, self.base_is = M, N, K, r, L, len(adapter), f32, base
        self.offsets, self.adapter = list(offsets), list(adapter)
        self.x, self.xv = bf(rng.standard_normal((M, K)))
        self.a, self.av = bf(rng.standard_normal((L, r, K)) * K ** -0.5)
        self.b, self.bv = bf(rng.standard_normal((L, N, r)) * r ** -0.5)
        self.scale = torch.from_numpy(rng.uniform(-2, 2, L).astype(np.float32)).cuda() if scaled else None
        dt = torch.float32 if f32 else torch.bfloat16
        if f32:
            self.base = torch.from_numpy(rng.standard_normal((M, N)).astype(np.float32)).cuda()
        else:
            self.base, _ = bf(rng.standard_normal((M, N)))
        self.out = self.base.clone() if base == "out" else torch.full((M, N), float("nan"), dtype=dt, device="cuda")

    def run(self, moe, ctx=None, plan=None):
        if plan:
            assert moe.moe_adapter_gemm_plan(self.M, self.N, self.K, self.r, self.L, self.R) == plan
        base = {"apart": self.base, "out": self.out, None: None}[self.base_is]
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        ws = torch.full((moe.moe_adapter_gemm_workspace_size(self.M, self.R, self.r),), 0xFF, dtype=torch.uint8, device="cuda")
        moe.moe_adapter_gemm(self.x, self.a, self.b, self.scale, i32(self.offsets), i32(self.adapter), base, self.M, self.N,
                             self.K, self.r, self.L, self.R, self.out, ctx or moe.Ctx(workspace=ws, dev_status=status))
        torch.cuda.synchronize()
        return int(status[0])

    def check(self):
        base = np64(self.base) if self.base_is else np.zeros((self.M, self.N))
        scale = None if self.scale is None else np64(self.scale)
        ref, mag = oracle.adapter_gemm(self.xv, self.av, self.bv, scale, self.offsets, self.adapter, base)
        got, ids = np64(self.out), oracle.row_adapters(self.M, self.offsets, self.adapter)
        outside = ids == -2
        if self.base_is == "out":
            assert torch.equal(self.out[torch.from_numpy(ids < 0).cuda()], self.base[torch.from_numpy(ids < 0).cuda()])
        else:
            assert np.isnan(got[outside]).all()  # not written
            assert np.array_equal(got[ids == -1], base[ids == -1])
        m = ids >= 0
        half = np.abs(ref) * 2.0 ** -24 if self.f32 else bf16_half_ulp(ref) * (1 + 2.0 ** -7)
        err = np.abs(got[m] - ref[m]) - half[m]
        assert np.all(err <= mag[m] * 2.0 ** -13)
        if m.any() and self.f32:
            assert np.mean(np.abs(got[m] - ref[m])) <= np.mean(mag[m]) * 2.0 ** -18


def lengths(*n):
    return np.concatenate([[0], np.cumsum(n)]).tolist()


def decode(M, L, bare=0.2, seed=0):
    rng = np.random.default_rng(seed + M)
    ad = rng.integers(0, L, M)
    ad[rng.random(M) < bare] = -1
    return list(range(M + 1)), ad.tolist()


@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 128])
@pytest.mark.parametrize("M", [1, 7, 33])
def test_one_token_a_request(moe, M, r):
    c = Case(M, 264, 200, r, 5, *decode(M, 5))
    assert c.run(moe) == 0
    c.check()


@pytest.mark.parametrize("N,K", [(8, 8), (64, 2880), (2880, 64), (2888, 1000), (4096, 264)])
@pytest.mark.parametrize("f32", [False, True])
def test_sizes(moe, N, K, f32):
    c = Case(20, N, K, 16, 30, *decode(20, 30), f32=f32)
    c.run(moe)
    c.check()


@pytest.mark.parametrize("M,L", [(100, 1), (250, 5), (511, 100), (512, 3), (513, 3), (1500, 40)])
def test_many_requests(moe, M, L):
    c = Case(M, 136, 72, 16, L, *decode(M, L))
    c.run(moe)
    c.check()


PROMPTS = [lengths(600), lengths(1, 2, 130, 0, 128, 127, 129, 5), [3, 3, 300, 301, 900], lengths(*[17] * 60),
           lengths(300, 300, 300, 300)]
# long enough, for their sizes, for the other kernels: tiles that end in each of their boxes' rows, requests
# without rows, rows of no request
LONG = [lengths(9000), lengths(1, 2, 8000, 0, 128, 127, 129, 5, 31, 32, 33, 1000), [3, 3, 300, 5001, 11900], lengths(*[600] * 16)]


@pytest.mark.parametrize("offsets", PROMPTS)
@pytest.mark.parametrize("r,N,K", [(16, 264, 200), (64, 520, 136), (128, 72, 328), (8, 1032, 72)])
def test_prompts(moe, offsets, r, N, K):
    R = len(offsets) - 1
    c = Case(offsets[-1] + 9, N, K, r, 3, offsets, [(i * 2) % 4 - 1 for i in range(R)], seed=1)
    c.run(moe, plan="few")
    c.check()


@pytest.mark.parametrize("offsets", LONG)
@pytest.mark.parametrize("r,N,K", [(16, 264, 200), (64, 520, 136), (128, 72, 328), (8, 1032, 72), (40, 136, 264), (72, 200, 136)])
def test_long_prompts(moe, offsets, r, N, K):
    R = len(offsets) - 1
    c = Case(offsets[-1] + 9, N, K, r, 3, offsets, [(i * 2 + 1) % 4 - 1 for i in range(R)], seed=1)
    c.run(moe, plan="long")
    c.check()


@pytest.mark.parametrize("base", ["apart", "out", None])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("offsets,plan", [([0, 1, 2, 3, 4, 9], "few"), ([5, 400, 400, 900, 1111, 1130], "few"),
                                          ([5, 4000, 4000, 4900, 6111, 9130], "long")])
def test_base(moe, base, f32, offsets, plan):
    c = Case(offsets[-1] + 20, 328, 136, 24, 4, offsets, [1, 3, -1, 0, 1], f32=f32, base=base, scaled=f32, seed=2)
    c.run(moe, plan=plan)
    c.check()


def test_long_rows_of_fp32(moe):
    for offsets, plan in (([0, 1, 2, 3], "few"), ([0, 700, 1400, 1500], "long")):
        c = Case(offsets[-1], 520, 7168, 32, 2, offsets, [0, 1, 0], f32=True, seed=3)
        c.run(moe, plan=plan)
        c.check()


def test_same_bits_twice(moe):
    for (offsets, ad), plan in ((decode(90, 7), "few"), (([0, 1200, 1800, 3000], [1, 0, 1]), "long")):
        outs = []
        for _ in range(2):
            c = Case(offsets[-1], 1032, 2056, 32, 7, offsets, ad, seed=4)
            c.run(moe, plan=plan)
            outs.append(c.out)
        assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))


@pytest.mark.parametrize("M,L,r,N,K", [(256, 256, 16, 264, 4104), (500, 150, 64, 520, 2056), (700, 30, 32, 4096, 4096)])
@pytest.mark.parametrize("f32", [False, True])
def test_more_tiles_than_ctas(moe, M, L, r, N, K, f32):
    """Whole tiles in turn, and pieces of them; the rows of the first case have an adapter each."""
    offsets, ad = decode(M, L)
    c = Case(M, N, K, r, L, offsets, ad if L < M else list(range(L)), f32=f32, seed=21)
    c.run(moe, plan="few")
    c.check()


def test_adapters_that_are_not_finite_stay_with_their_requests(moe):
    for offsets, ad, plan in (([0, 1, 2, 3, 4], [0, 1, 0, 2], "few"), ([0, 3, 4, 130, 140], [0, 1, 2, 1], "few"),
                              ([0, 100, 230, 20000, 20070], [0, 1, 0, 2], "long")):
        c = Case(offsets[-1], 136, 136, 16, 3, offsets, ad, seed=5)
        clean = Case(offsets[-1], 136, 136, 16, 3, offsets, ad, seed=5)
        c.a[1, 3, 5] = float("inf")
        c.b[1, 7] = float("nan")
        c.run(moe, plan=plan)
        clean.run(moe)
        mine = torch.from_numpy(oracle.row_adapters(c.M, offsets, ad) == 1).cuda()
        assert torch.equal(c.out[~mine], clean.out[~mine])
        assert not torch.isfinite(c.out[mine]).all(dim=1).any()


def test_rows_without_an_adapter_are_not_read(moe):
    for offsets, plan in (([2, 4, 6, 8], "few"), ([10, 300, 700, 20000], "long")):
        c = Case(offsets[-1] + 10, 136, 136, 16, 3, offsets, [0, -1, 1], seed=6)
        ids = torch.from_numpy(oracle.row_adapters(c.M, offsets, c.adapter)).cuda()
        c.x[ids < 0] = float("nan")
        c.run(moe, plan=plan)
        c.check()


@pytest.mark.parametrize("offsets,adapter,status,rows", [
    ([0, 2, 4, 6], [0, 5, 1], -5, {0: 0, 1: 0, 2: -1, 3: -1, 4: 1, 5: 1}),
    ([0, 2, 4, 6], [0, -2, 1], -5, {0: 0, 1: 0, 2: -1, 3: -1, 4: 1, 5: 1}),
    ([0, 2, 4, 99], [0, 1, 1], -3, {0: 0, 1: 0, 2: 1, 3: 1, 4: -2, 5: -2}),
    ([-4, 2, 4, 6], [0, 1, 1], -3, {0: -2, 1: -2, 2: 1, 3: 1, 4: 1, 5: 1}),
    ([0, 4, 2, 3], [0, 1, 1], -3, {0: 0, 1: 0}),  # the last one overlaps the first
])
@pytest.mark.parametrize("M,plan", [(6, "few"), (900, "few"), (60000, "long")])
def test_data_errors_are_reported(moe, offsets, adapter, status, rows, M, plan):
    if M > 6:
        offsets = [o * (M // 6) for o in offsets]
    c = Case(M, 64, 64, 8, 2, offsets, adapter, seed=7)
    assert c.run(moe, plan=plan) == status
    got = np64(c.out)
    for m, l in rows.items():
        m = m * (M // 6)
        if l == -2:
            assert np.isnan(got[m]).all()
            continue
        want = np64(c.base)[m] + (0 if l < 0 else float(c.scale[l]) * (c.xv[m] @ c.av[l].T) @ c.bv[l].T)
        assert np.allclose(got[m], want, rtol=2.0 ** -7, atol=2.0 ** -7)


def test_captured_calls_follow_the_tables(moe):
    """A graph's replays take the offsets and adapters that memory holds by then; another stream."""
    for M, plans in ((40, [([0, 1, 20, 40], [0, 1, 2]), ([0, 20, 20, 33], [2, 0, 0])]),
                     (9000, [([0, 1, 2000, 4000], [0, 1, 2]), ([0, 5200, 5200, 8933], [2, 0, 0])])):
        c = Case(M, 264, 264, 16, 3, *plans[0], seed=8)
        assert moe.moe_adapter_gemm_plan(M, 264, 264, 16, 3, 3) == ("few" if M < 100 else "long")
        off, ad = i32(plans[0][0]), i32(plans[0][1])
        s = torch.cuda.Stream()
        ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
        ctx = moe.Ctx(stream=s, workspace=ws)

        def run(ctx):
            moe.moe_adapter_gemm(c.x, c.a, c.b, c.scale, off, ad, c.base, c.M, c.N, c.K, c.r, c.L, 3, c.out, ctx)

        s.wait_stream(torch.cuda.current_stream())
        run(ctx)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            run(ctx)
        for offsets, adapter in plans:
            off.copy_(i32(offsets))
            ad.copy_(i32(adapter))
            c.out.fill_(float("nan"))
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            c.offsets, c.adapter = offsets, adapter
            c.check()


def test_offsets_past_32_bits(moe):
    """The last adapters of tables of more than 2^31 elements."""
    L, r, K, N = 1030, 128, 16392, 64
    a = torch.zeros((L, r, K), dtype=torch.bfloat16, device="cuda")
    b = torch.zeros((L, N, r), dtype=torch.bfloat16, device="cuda")
    x, xv = bf(np.random.default_rng(9).standard_normal((600, K)))
    w, wv = bf(np.random.default_rng(10).standard_normal((r, K)) * K ** -0.5)
    u, uv = bf(np.random.default_rng(11).standard_normal((N, r)))
    a[L - 1], b[L - 1] = w, u
    out = torch.empty((600, N), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 25, dtype=torch.uint8, device="cuda")
    assert moe.moe_adapter_gemm_plan(600, N, K, r, L, 2) == "long" and moe.moe_adapter_gemm_plan(5, N, K, r, L, 2) == "few"
    for M, off, ad in ((5, [0, 2, 5], [L - 1, 0]), (600, [0, 300, 600], [L - 1, 0])):
        moe.moe_adapter_gemm(x, a, b, None, i32(off), i32(ad), None, M, N, K, r, L, 2, out, moe.Ctx(workspace=ws))
        torch.cuda.synchronize()
        want = (xv[:off[1]] @ wv.T) @ uv.T
        assert np.all(np.abs(np64(out[:off[1]]) - want) <= bf16_half_ulp(want) * 1.01 + 2.0 ** -9)
        assert (out[off[1]:off[2]] == 0).all()


@pytest.mark.parametrize("R,r,f32", [(16, 16, True), (16, 64, True), (3, 128, True), (16, 16, False), (1000, 64, False),
                                     (1000, 64, True)])
def test_long_prompts_under_load(moe, R, r, f32):
    """Twenty calls in a graph, replayed, each with many boxes of base in flight on every SM: the same
    bits as the first call alone, which are right.  (1000 requests: their tables leave less room for boxes.)"""
    M, N, K = 20000, 1024, 512
    offsets = np.linspace(0, M, R + 1).astype(int).tolist()
    c = Case(M, N, K, r, 4, offsets, [(i * 3) % 4 for i in range(R)], f32=f32)
    assert c.run(moe, plan="long") == 0
    c.check()
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    size = moe.moe_adapter_gemm_workspace_size(M, R, r)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(c.out) for _ in range(20)]
    off, ids = i32(offsets), i32(c.adapter)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        for i, o in enumerate(outs):
            moe.moe_adapter_gemm(c.x, c.a, c.b, c.scale, off, ids, c.base, M, N, K, r, 4, R, o,
                                 moe.Ctx(stream=stream, workspace=ws[i % 2], dev_status=status))
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert int(status[0]) == 0
        for o in outs:
            assert torch.equal(o, c.out)


def test_calls_at_once(moe):
    """Calls of both kinds on two streams at once, each with a workspace of its own: the bits of a call alone."""
    cases = [Case(6000, 1032, 520, 32, 4, lengths(2500, 0, 1500, 2000), [2, 1, -1, 0], seed=31),
             Case(6000, 520, 1032, 64, 4, lengths(3000, 3000), [1, 3], f32=True, seed=32),
             Case(300, 4096, 2056, 16, 40, *decode(300, 40), seed=33), Case(64, 2880, 2880, 128, 9, *decode(64, 9), f32=True, seed=34)]
    for c, plan in zip(cases, ("long", "long", "few", "few")):
        assert c.run(moe, plan=plan) == 0
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls, status = [], torch.zeros(4, dtype=torch.int32, device="cuda")
    for i in range(24):
        c, s = cases[(i // 2 + (i % 2) * 2) % 4], streams[i % 2]  # another case on the other stream
        ws = torch.empty(moe.moe_adapter_gemm_workspace_size(c.M, c.R, c.r), dtype=torch.uint8, device="cuda")
        calls.append((c, torch.full_like(c.out, float("nan")), i32(c.offsets), i32(c.adapter),
                      moe.Ctx(stream=s, workspace=ws, dev_status=status)))
    torch.cuda.synchronize()
    for c, out, off, ids, ctx in calls:
        moe.moe_adapter_gemm(c.x, c.a, c.b, c.scale, off, ids, c.base, c.M, c.N, c.K, c.r, c.L, c.R, out, ctx)
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    for c, out, *_ in calls:
        assert torch.equal(out, c.out)
