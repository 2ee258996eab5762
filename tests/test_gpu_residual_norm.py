"""moe_residual_norm and its backward pass on the GPU against the float64 oracle.

Bounds.  The stream: a product and a sum of fp32 (2^-22 of their magnitudes) and its type's rounding.
n: the sum of squares adds K positive terms, at most 32 of a thread, 5 shuffles and 32 warps, so 70
roundings of 2^-24; half of that in r, and five more: below |n| 2^-18, and the stream's error times r w.
bf16 adds half a step.  8-bit outputs lie between the codes of n less and n plus these bounds.  ds: the
same for its two sums, 2^-17 of its terms' magnitudes; d_weight: chains of fewer than 256 additions,
2^-16 of the magnitudes.
"""
import numpy as np
import pytest

import synth
from helpers import bf16_half_ulp, bf16_to_np
from oracle import formats, mx_quant, residual_norm

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
EPS, STREAM_ID = 1e-5, 11


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_grouped_align_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.build()
    m.load()
    return m


def bf(a):
    """-> bf16 device tensor and its values."""
    bits = synth.to_bf16_bits(np.asarray(a, dtype=np.float64))
    return torch.from_numpy(bits.view(np.int16).copy()).view(torch.bfloat16).cuda(), formats.bf16_decode(bits)


def typed(a, f32):
    if not f32:
        return bf(a)
    v = np.asarray(a, dtype=np.float32)
    return torch.from_numpy(v.copy()).cuda(), v.astype(np.float64)


def np64(t):
    return bf16_to_np(t) if t.dtype == torch.bfloat16 else t.cpu().numpy().astype(np.float64)


def rounding(ref, f32):
    """What storing ref costs."""
    return np.abs(ref) * 2.0 ** -24 + 2.0 ** -149 if f32 else bf16_half_ulp(ref) * (1 + 2.0 ** -7)


def nans(shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


class Case:
    """Inputs of T rows of K, and what the oracle makes of them."""

    def __init__(self, T, K, f32=False, p=0.0, branch=True, masked=False, seed=0, quant=None, scale=1.0):
        rng = np.random.default_rng(seed + 7919 * T + K)
        self.T, self.K, self.f32, self.p, self.quant = T, K, f32, p, quant
        self.x, xv = bf(rng.standard_normal((T, K)) * scale) if branch else (None, None)
        self.res, rv = typed(rng.standard_normal((T, K)) * 2 * scale, f32)
        self.w, self.wv = bf(1 + 0.3 * rng.standard_normal(K))
        mask = (rng.random(T) < 0.7).astype(np.uint8) if masked else None
        self.mask = None if mask is None else torch.from_numpy(mask).cuda()
        self.mask_np = mask
        state = (int(rng.integers(-2 ** 63, 2 ** 63 - 1)), int(rng.integers(0, 2 ** 40)))
        self.rng = torch.tensor(state, device="cuda")
        self.kept = residual_norm.keep(T, K, p, *state, STREAM_ID) if p and branch else 1.0
        self.s, self.n = residual_norm.forward(xv, rv, self.wv, EPS, self.kept, mask)
        live = 1.0 if mask is None else (mask[:, None] != 0)
        self.ds = ((0.0 if xv is None else np.abs(xv * self.kept)) + np.abs(rv)) * live * 2.0 ** -22
        r = 1 / np.sqrt((self.s ** 2).mean(axis=1, keepdims=True) + EPS)
        self.dn = np.abs(self.n) * 2.0 ** -18 + self.ds * r * np.abs(self.wv)
        self.gr = rng

    def run(self, moe, stream=True, out=True, in_place=False, ctx=None):
        T, K = self.T, self.K
        st = (self.res.clone() if in_place else nans((T, K), self.res.dtype)) if stream else None
        res = st if in_place else self.res
        x = self.x.clone() if in_place else self.x
        o = (x if in_place else nans((T, K), torch.bfloat16)) if out else None
        codes = torch.full((T, K), 0xA5, dtype=torch.uint8, device="cuda") if self.quant else None
        scales = {None: None, "mx": torch.full((T, K // 32), 0xA5, dtype=torch.uint8, device="cuda"),
                  "row": nans((T,), torch.float32)}[self.quant]
        moe.moe_residual_norm(x, res, self.mask, self.w, T, K, EPS, self.p, self.rng, STREAM_ID, st, o, codes, scales, ctx)
        torch.cuda.synchronize()
        return st, o, codes, scales

    def check(self, st, o, codes, scales):
        if st is not None:
            assert np.all(np.abs(np64(st) - self.s) <= rounding(self.s, self.f32) + self.ds)
        if o is not None:
            assert np.all(np.abs(np64(o) - self.n) <= rounding(self.n, False) + self.dn)
        if self.quant == "mx":
            sc = scales.cpu().numpy().astype(np.int64) - 127
            lo, hi = np.abs(self.n) - self.dn, np.abs(self.n) + self.dn
            exps = [mx_quant.block_exponent(np.maximum(v, 0).reshape(self.T, -1, 32).max(axis=2)) for v in (lo, hi)]
            assert np.all((exps[0] <= sc) & (sc <= exps[1]))
            unit = np.repeat(np.exp2(sc.astype(np.float64)), 32, axis=1)
            self.check_codes(codes, unit, 0.0)
        if self.quant == "row":
            unit = np64(scales)
            want = np.maximum(np.abs(self.n).max(axis=1) / 448, 2.0 ** -120)
            assert np.all(np.abs(unit - want) <= want * 2.0 ** -17)
            self.check_codes(codes, unit[:, None], 2.0 ** -21)

    def check_codes(self, codes, unit, rel):
        got = formats.e4m3_decode(codes.cpu().numpy())
        lo, hi = (formats.e4m3_decode(mx_quant.e4m3_encode((self.n + sign * (self.dn + np.abs(self.n) * rel)) / unit))
                  for sign in (-1, 1))
        assert np.all((lo <= got) & (got <= hi))


# a size of every kernel: few and many rows, groups of 8, 16 and 32 lanes, blocks of one, two and four eights a thread
SIZES = [(1, 8), (1, 16384), (3, 64), (5, 136), (37, 256), (300, 520), (28, 2688), (1, 7168), (64, 2880), (100, 12288),
         (30000, 64), (7000, 256), (4000, 512), (2000, 1000), (900, 2880), (130, 16384), (1001, 1856), (900, 7168)]


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("f32", [False, True])
def test_forward(moe, T, K, f32):
    c = Case(T, K, f32, p=0.1, masked=T > 2)
    c.check(*c.run(moe))


@pytest.mark.parametrize("T,K", [s for s in SIZES if s[1] % 32 == 0])
@pytest.mark.parametrize("quant", ["mx", "row"])
def test_codes(moe, T, K, quant):
    c = Case(T, K, T % 2 == 0, quant=quant, masked=T > 2, seed=1)
    c.check(*c.run(moe, stream=T % 3 != 0, out=T % 2 == 0))


def test_row_codes_of_other_widths(moe):
    for T, K in ((3, 8), (33, 1000), (200, 4104)):
        c = Case(T, K, quant="row", seed=2)
        c.check(*c.run(moe))


@pytest.mark.parametrize("T,K,quant,f32", [(700, 2880, "mx", False), (700, 2880, "row", True), (1700, 1024, "row", False),
                                           (3100, 520, "row", False), (900, 7168, "row", False), (900, 7168, "mx", False),
                                           (901, 4104, "row", True), (140, 12288, "row", False), (140, 12288, "mx", False)])
@pytest.mark.parametrize("out", [False, True])
def test_codes_of_many_rows(moe, T, K, quant, f32, out):
    """Two eights a thread, blocks that walk over rows, stores after the sums: with and without the bf16 rows."""
    c = Case(T, K, f32, p=0.1 if out else 0.0, quant=quant, masked=True, seed=13)
    c.check(*c.run(moe, out=out))
    c = Case(T, K, f32, branch=False, quant=quant, seed=14)
    c.check(*c.run(moe, stream=False, out=out))


@pytest.mark.parametrize("branch,stream,out,quant", [(False, False, True, None), (False, True, True, "mx"),
                                                     (True, True, False, None), (True, False, False, "row")])
def test_parts_of_the_call(moe, branch, stream, out, quant):
    c = Case(50, 2048, branch=branch, quant=quant, seed=3)
    st, o, codes, scales = c.run(moe, stream, out)
    assert (st is not None, o is not None) == (stream, out)
    c.check(st, o, codes, scales)


@pytest.mark.parametrize("T,K", [(9, 64), (40, 2880), (2000, 1000), (900, 2880)])
def test_in_place(moe, T, K):
    c = Case(T, K, p=0.25, masked=True, seed=4)
    apart, inside = c.run(moe), c.run(moe, in_place=True)
    c.check(*inside)
    assert torch.equal(apart[0], inside[0]) and torch.equal(apart[1], inside[1])


def test_x_alone_starts_a_stream(moe):
    c = Case(20, 512, p=0.5, seed=5)
    _, xv = c.x, np64(c.x)
    st = nans((20, 512), torch.float32)
    moe.moe_residual_norm(c.x, None, None, c.w, 20, 512, EPS, 0.5, c.rng, STREAM_ID, st, None)
    assert np.array_equal(np64(st), xv * c.kept)  # gain 2: exact


def test_probabilities(moe):
    """Next to 0: nothing dropped, by 2^-17; next to 1: at most all but one in 65536 numbers."""
    T, K = 64, 4096
    x, _ = bf(np.ones((T, K)))
    w, _ = bf(np.ones(K))
    rng = torch.tensor([5, 6], device="cuda")
    st = nans((T, K), torch.float32)
    for p, below in ((1e-9, 0), (2.0 ** -16, 1), (0.99999999 - 1e-7, 65535), (0.3, 19661)):
        assert residual_norm.below(p) == below
        moe.moe_residual_norm(x, None, None, w, T, K, EPS, p, rng, STREAM_ID, st, None)
        want = np.where(residual_norm.numbers(T * K, 5, 6, STREAM_ID) >= below, np.float32(65536 / (65536 - below)), 0)
        assert np.array_equal(st.cpu().numpy().reshape(-1), want.astype(np.float32))


def test_zeros_extremes_and_non_finite_rows(moe):
    T, K = 8, 256
    rng = np.random.default_rng(9)
    res = rng.standard_normal((T, K))
    res[0] = 0.0
    res[1] *= 2.0 ** -100
    res[2] *= 2.0 ** 50
    w, wv = bf(np.ones(K))
    clean, _ = typed(res, True)
    res[3, 7] = np.nan
    res[4, 40] = np.inf
    res[5, 3] = -np.inf
    dirty, dv = typed(res, True)
    outs = []
    for r in (clean, dirty):
        for quant in ("mx", "row"):
            o, codes = nans((T, K), torch.bfloat16), torch.full((T, K), 1, dtype=torch.uint8, device="cuda")
            sc = torch.full((T, K // 32), 1, dtype=torch.uint8, device="cuda") if quant == "mx" else nans((T,), torch.float32)
            moe.moe_residual_norm(None, r, None, w, T, K, EPS, 0.0, None, 0, None, o, codes, sc)
            outs.append((o, codes, sc))
    for (a, b) in ((outs[0], outs[2]), (outs[1], outs[3])):
        for u, v in zip(a, b):  # other rows are the same
            keep = [0, 1, 2, 6, 7]
            assert torch.equal(u[keep].view(torch.uint8), v[keep].view(torch.uint8))
    o, codes, sc = outs[2]
    assert torch.isnan(o[3]).all() and torch.isnan(o[4, 40]) and torch.isnan(o[5, 3])
    assert (sc[3] == 255).all() and (codes[3] == 0x7F).all() and sc[4, 1] == 255 and sc[5, 0] == 255
    o, codes, sc = outs[3]
    assert torch.isnan(sc[3:6]).all() and (codes[3:6] & 0x7F == 0x7F).all()
    o, codes, sc = outs[1]
    assert (o[0] == 0).all() and (codes[0] == 0).all() and sc[0] == 2.0 ** -120
    assert (outs[0][2][0] == 0).all()
    assert abs(float(o[2].float().square().mean()) - 1) < 0.01 and torch.isfinite(o[:3]).all()
    assert float(o[1].float().abs().max()) < 2.0 ** -85


def backward(moe, c, use=("d_stream", "d_residual", "d_x", "d_weight"), in_place=False, ctx=None):
    T, K = c.T, c.K
    st, _ = typed(c.s, c.f32)
    do, dov = bf(c.gr.standard_normal((T, K)) * 0.05)
    dst, dsv = typed(c.gr.standard_normal((T, K)) * 0.05, c.f32) if "d_stream" in use else (None, None)
    dr = (dst.clone() if in_place else nans((T, K), c.res.dtype)) if "d_residual" in use else None
    dx = (do.clone() if in_place else nans((T, K), torch.bfloat16)) if "d_x" in use else None
    dw = nans((K,), torch.float32) if "d_weight" in use else None
    ws = torch.full((moe.moe_residual_norm_workspace_size(K),), 0xFF, dtype=torch.uint8, device="cuda")
    moe.moe_residual_norm_backward(dx if in_place else do, dr if in_place else dst, st, c.mask, c.w, T, K, EPS, c.p, c.rng,
                                   STREAM_ID, dr, dx, dw, ctx or moe.Ctx(workspace=ws))
    torch.cuda.synchronize()
    sv = np64(st)
    rr, rx, rw = residual_norm.backward(dov, dsv, sv, c.wv, EPS, c.kept, c.mask_np)
    live = np.ones((T, 1), bool) if c.mask_np is None else c.mask_np[:, None] != 0
    r = 1 / np.sqrt((sv * sv).mean(axis=1, keepdims=True) + EPS)
    g = np.abs(dov * c.wv)
    mag = (r * g + np.abs(sv) * r ** 3 * (g * np.abs(sv)).mean(axis=1, keepdims=True) +
           (0.0 if dsv is None else np.abs(dsv))) * live * 2.0 ** -17
    if dr is not None:
        assert np.all(np.abs(np64(dr) - rr) <= rounding(rr, c.f32) + mag)
    if dx is not None:
        assert np.all(np.abs(np64(dx) - rx) <= rounding(rx, False) + mag * c.kept * (1 + 2.0 ** -7))
    if dw is not None:
        assert np.all(np.abs(np64(dw) - rw) <= (np.abs(dov * sv * r) * live).sum(axis=0) * 2.0 ** -16)
    return dr, dx, dw


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("f32", [False, True])
def test_backward(moe, T, K, f32):
    backward(moe, Case(T, K, f32, p=0.1, masked=T > 2, seed=6))


@pytest.mark.parametrize("T,K,f32", [(3000, 1024, False), (4000, 768, True), (2500, 1536, False)])
def test_backward_of_many_narrow_rows(moe, T, K, f32):
    """More than four blocks on an SM."""
    backward(moe, Case(T, K, f32, p=0.1, masked=True, seed=15))


@pytest.mark.parametrize("use", [("d_residual",), ("d_x",), ("d_weight",), ("d_stream", "d_x"), ("d_stream", "d_residual")])
def test_parts_of_the_backward_call(moe, use):
    backward(moe, Case(60, 928, p=0.1, seed=7), use)


@pytest.mark.parametrize("T,K", [(9, 64), (40, 2880), (2000, 1000), (900, 2880)])
def test_backward_in_place(moe, T, K):
    a = backward(moe, Case(T, K, p=0.25, masked=True, seed=8))
    b = backward(moe, Case(T, K, p=0.25, masked=True, seed=8), in_place=True)
    assert all(torch.equal(u, v) for u, v in zip(a, b))  # and the same bits twice


def test_no_rows(moe):
    K = 64
    w, _ = bf(np.ones(K))
    e = torch.empty((0, K), dtype=torch.bfloat16, device="cuda")
    dw = nans((K,), torch.float32)
    moe.moe_residual_norm(e, e, None, w, 0, K, EPS, 0.0, None, 0, e, e)
    moe.moe_residual_norm_backward(e, None, e, None, w, 0, K, EPS, 0.0, None, 0, e, e, dw)
    assert (dw == 0).all()
    c = Case(5, K, seed=10)  # no row counts
    c.mask = torch.zeros(5, dtype=torch.uint8, device="cuda")
    st, o, _, _ = c.run(moe)
    assert (st == 0).all() and (o == 0).all()
    c.mask_np = np.zeros(5, np.uint8)
    dr, dx, dw = backward(moe, c)
    assert (dr == 0).all() and (dx == 0).all() and (dw == 0).all()


def test_rows_that_do_not_count_are_not_read(moe):
    T, K = 40, 928
    a, b = Case(T, K, p=0.1, masked=True, seed=11, quant="mx"), Case(T, K, p=0.1, masked=True, seed=11, quant="mx")
    pad = a.mask == 0
    for t in (b.x, b.res):
        t[pad] = float("nan")
    for u, v in zip(a.run(moe), b.run(moe)):
        assert torch.equal(u, v)
    ws = torch.empty(moe.moe_residual_norm_workspace_size(K), dtype=torch.uint8, device="cuda")
    got = []
    for dirty in (False, True):
        st, do = a.res.clone(), a.x.clone()
        if dirty:
            st[pad], do[pad] = float("nan"), float("inf")
        o = [nans((T, K), torch.bfloat16), nans((T, K), torch.bfloat16), nans((K,), torch.float32)]
        moe.moe_residual_norm_backward(do, do, st, a.mask, a.w, T, K, EPS, 0.1, a.rng, 0, *o, moe.Ctx(workspace=ws))
        got.append(o)
    for u, v in zip(*got):
        assert torch.equal(u, v)


def test_captured_calls_draw_by_the_state_in_memory(moe):
    """A graph's replays follow rng; streams other than the default one and their own workspaces."""
    T, K = 70, 2688
    c = Case(T, K, p=0.2, seed=12)
    s = torch.cuda.Stream()
    ws = torch.empty(moe.moe_residual_norm_workspace_size(K), dtype=torch.uint8, device="cuda")
    new = lambda: nans((T, K), torch.bfloat16)  # noqa: E731
    st, o, dr, dx, dw = new(), new(), new(), new(), nans((K,), torch.float32)

    def step(ctx):
        moe.moe_residual_norm(c.x, c.res, None, c.w, T, K, EPS, 0.2, c.rng, STREAM_ID, st, o, None, None, ctx)
        moe.moe_residual_norm_backward(o, None, st, None, c.w, T, K, EPS, 0.2, c.rng, STREAM_ID, dr, dx, dw, ctx)

    ctx = moe.Ctx(stream=s, workspace=ws)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(ctx)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(ctx)
    for n in range(3):
        c.rng[1] = 100 + n
        for t in (st, o, dr, dx, dw):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (st, o, dr, dx, dw)]
        kept = residual_norm.keep(T, K, 0.2, int(c.rng[0]), 100 + n, STREAM_ID)
        assert np.array_equal(np64(st) != np64(c.res), (kept != 0) & (np64(st) != np64(c.res)))
        assert np.all(np64(dx)[kept == 0] == 0) and np.all(np64(dr)[kept == 0] != 0)
        step(moe.Ctx(workspace=ws))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (st, o, dr, dx, dw)))


def test_calls_at_once(moe):
    """Forward and backward passes on two streams at once, each with a workspace of its own."""
    cases = [Case(900, 7168, p=0.1, masked=True, quant="mx", seed=41), Case(2500, 1536, True, p=0.25, quant="row", seed=42)]
    alone = []

    def outputs(c):
        T, K = c.T, c.K
        st, dr = (nans((T, K), c.res.dtype) for _ in range(2))
        o, dx = (nans((T, K), torch.bfloat16) for _ in range(2))
        codes = torch.empty((T, K), dtype=torch.uint8, device="cuda")
        scales = torch.empty((T, K // 32), dtype=torch.uint8, device="cuda") if c.quant == "mx" else nans((T,), torch.float32)
        ws = torch.full((moe.moe_residual_norm_workspace_size(K),), 0xFF, dtype=torch.uint8, device="cuda")
        return st, o, codes, scales, dr, dx, nans((K,), torch.float32), ws

    def run(c, b, stream):
        st, o, codes, scales, dr, dx, dw, ws = b
        ctx = moe.Ctx(stream=stream, workspace=ws)
        moe.moe_residual_norm(c.x, c.res, c.mask, c.w, c.T, c.K, EPS, c.p, c.rng, STREAM_ID, st, o, codes, scales, ctx)
        moe.moe_residual_norm_backward(c.x, None, st, c.mask, c.w, c.T, c.K, EPS, c.p, c.rng, STREAM_ID, dr, dx, dw, ctx)

    for c in cases:
        alone.append(outputs(c))
        run(c, alone[-1], torch.cuda.current_stream())
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    many = [(i % 2, outputs(cases[i % 2])) for i in range(12)]
    torch.cuda.synchronize()
    for i, b in many:
        run(cases[i], b, streams[i])
    torch.cuda.synchronize()
    for i, b in many:
        for got, want in zip(b[:-1], alone[i][:-1]):
            assert torch.equal(got, want)
