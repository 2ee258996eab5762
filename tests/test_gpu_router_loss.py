"""moe_router_loss on the GPU against the float64 oracle.

Bounds.  The kernel's exponential is within 2 + 1.173 |x - max| ulp (the CUDA math library's
bound for the fast exponential), so a probability (an exponential over a sum of at most 1024 of
them) is within 2 (2 + 1.173 D) + 32 + 8 ulp with D the row's range above which terms matter
(they are weighted by themselves), 40 roundings of sums included: C = 64 + 3 D ulp of 2^-23 in
each factor.  Gradients are sums of such terms: |err| <= C 2^-23 * (the sum of the terms'
magnitudes).  Counts are exact.
"""
import numpy as np
import pytest

from oracle import route as oroute
from oracle import router_loss as orl

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
A, B = 0.01, 0.001


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_grouped_align_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.build()
    m.load()
    return m


def call(moe, x, ids, w=None, dw=None, mask=None, a=A, b=B, ctx=None, in_place=False, outputs=True):
    T, E = x.shape
    k = ids.shape[1]
    up = lambda v, t=None: None if v is None else torch.from_numpy(np.ascontiguousarray(v)).cuda()  # noqa: E731
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = torch.full((moe.moe_router_loss_workspace_size(E),), 255, dtype=torch.uint8, device="cuda")
    xd = up(x)
    counts = torch.full((E,), -7, dtype=torch.int32, device="cuda") if outputs else None
    mean = torch.full((E,), float("nan"), device="cuda") if outputs else None
    loss = torch.full((3,), float("nan"), device="cuda")
    d = xd if in_place else (torch.full((T, E), float("nan"), device="cuda") if outputs else None)
    moe.moe_router_loss(xd, up(ids), up(w), up(dw), up(mask), T, k, E, a, b, counts, mean, loss, d,
                        ctx or moe.Ctx(workspace=ws, dev_status=status))
    torch.cuda.synchronize()
    g = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    return g(counts), g(mean), g(loss), g(d), int(status[0])


def make(T, E, k, seed, allowed=None, scale=1.0):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((T, E)) * scale + rng.standard_normal(E) * 0.5).astype(np.float32)
    if allowed is not None:
        for t in range(T):
            x[t, rng.permutation(E)[allowed:]] = -np.inf
    ids, w = oroute.route(x, k)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    return x, ids.astype(np.int32), w.astype(np.float32), dw


def check(got, x, ids, w, dw, mask, a=A, b=B, z_fits=True):
    counts, mean, loss, d, _ = got
    oc, om, ol, od = orl.router_loss(x, ids, w, dw, mask, a, b)
    T, E = x.shape
    k = ids.shape[1]
    n = T if mask is None else int((mask != 0).sum())
    assert np.array_equal(counts, oc)
    if n == 0:
        assert not d.any() and not mean.any() and not loss.any()
        return
    below = np.where(np.isfinite(x), x.max(axis=1, keepdims=True) - np.where(np.isfinite(x), x, 0.0), 0.0)
    D = float(below[below < 70].max())  # a term below that is under 2^-100 of its row
    C = (64 + 3 * D) * 2.0 ** -23
    assert np.all(np.abs(mean - om) <= C * om + 1e-30)
    f = oc * (E / (n * k))
    assert abs(loss[1] - ol[1]) <= 2 * C * abs(f @ om)
    if z_fits:
        assert abs(loss[2] - ol[2]) <= 2 * C * (abs(ol[2]) + 1e-3)
    assert abs(loss[0] - ol[0]) <= 3 * C * (abs(a * ol[1]) + abs(b) * (ol[2] + 1e-3))
    # magnitudes of the gradient's terms, in float64
    live = np.ones(T, bool) if mask is None else mask != 0
    mag = np.zeros((T, E))
    m = x.max(axis=1, keepdims=True)
    ok = live & np.isfinite(m[:, 0])
    p = np.zeros((T, E))
    p[ok] = np.exp(x[ok] - m[ok])
    p[ok] /= p[ok].sum(axis=1, keepdims=True)
    lse = np.zeros((T, 1))
    lse[ok] = m[ok] + np.log(np.exp(x[ok] - m[ok]).sum(axis=1, keepdims=True))
    g = np.abs(f - 1)
    mag += abs(a) / n * p * (g + p @ g[:, None]) + 2 * abs(b) / n * (np.abs(lse) + 1) * p
    if dw is not None:
        good = (ids >= 0) & (ids < E)
        wa, da = np.where(good, w, 0), np.abs(np.where(good, dw, 0))
        u = wa * (da + (wa * da).sum(axis=1, keepdims=True))
        for t in np.nonzero(ok)[0]:
            np.add.at(mag[t], ids[t][good[t]], u[t][good[t]])
    assert np.all(np.abs(d - od) <= 2 * C * mag + 1e-30), np.max(np.abs(d - od) - 2 * C * mag)


@pytest.mark.parametrize("T,E,k,allowed,upstream", [
    (1, 1, 1, None, True), (1, 8, 2, None, True), (3, 31, 5, None, True), (64, 128, 4, None, False),
    (65, 60, 6, 20, True), (128, 128, 4, None, True), (129, 128, 4, None, True), (257, 130, 6, 44, True),
    (500, 256, 8, None, True), (333, 257, 8, None, True), (700, 512, 8, 100, False), (301, 1001, 6, None, True),
    (150, 1024, 32, None, True), (2000, 8, 1, None, False), (2001, 33, 32, None, True), (5000, 64, 8, None, True),
])
def test_matches_oracle(moe, T, E, k, allowed, upstream):
    x, ids, w, dw = make(T, E, k, T + E, allowed)
    dw = dw if upstream else None
    check(call(moe, x, ids, w, dw), x, ids, w, dw, None)


@pytest.mark.parametrize("T,E,k", [(40, 16, 2), (900, 130, 6), (3000, 128, 4)])
def test_masked_tokens_count_for_nothing(moe, T, E, k):
    """Interior and trailing masked tokens whose logits, ids and gradients are poison."""
    x, ids, w, dw = make(T, E, k, 7)
    rng = np.random.default_rng(8)
    mask = (rng.random(T) < 0.7).astype(np.uint8) * 3
    mask[-5:] = 0
    ox, oi, ow, od = x.copy(), ids.copy(), w.copy(), dw.copy()
    off = mask == 0
    for v, bad in ((x, np.nan), (w, np.inf), (dw, np.nan)):
        v[off] = bad
    x[np.nonzero(off)[0][0]] = np.inf
    ids[off] = 1 << 30
    got = call(moe, x, ids, w, dw, mask)
    assert got[4] == 0 and not got[3][off].any()
    check(got, np.where(off[:, None], ox, x), np.where(off[:, None], oi, ids), np.where(off[:, None], ow, w),
          np.where(off[:, None], od, dw), mask)


@pytest.mark.parametrize("T", [0, 1, 30, 2000])
def test_no_token_left(moe, T):
    x, ids, w, dw = make(max(T, 1), 64, 4, 9)
    x, ids, w, dw = x[:T], ids[:T], w[:T], dw[:T]
    got = call(moe, x, ids, w, dw, np.zeros(T, np.uint8) if T else None)
    assert not got[0].any() and not got[1].any() and not got[2].any() and not got[3].any()


@pytest.mark.parametrize("E", [16, 130, 256])
def test_rows_that_the_mask_leaves_empty(moe, E):
    x, ids, w, dw = make(300, E, 4, 10)
    x[5] = -np.inf
    x[299] = -np.inf
    x[17] = np.float32(-3.4028235e38)          # the type's lowest value everywhere: uniform
    x[18, : E // 2] = np.float32(-3.4028235e38)
    w[5] = np.nan                               # what a softmax over -inf leaves
    got = call(moe, x, ids, w, dw)
    assert not got[3][5].any() and not got[3][299].any()
    assert np.isfinite(got[3]).all() and np.isfinite(got[2][1])
    # lse^2 of the lowest value overflows fp32 (loss[2]); with the z loss off nothing else does
    wz = w.copy()
    wz[5] = 0
    check(call(moe, x, ids, wz, dw, b=0.0), x, ids, wz, dw, None, b=0.0, z_fits=False)


def test_nan_and_infinite_logits_stay_in_their_row(moe):
    x, ids, w, dw = make(200, 128, 4, 11)
    x[3, 9] = np.nan
    x[8, 100] = np.inf
    got = call(moe, x, ids, w, dw)
    assert np.isnan(got[3][3]).all() and np.isnan(got[3][8]).any() and np.isnan(got[2][0])
    keep = [t for t in range(200) if t not in (3, 8)]
    assert np.isfinite(got[3][keep]).all()


@pytest.mark.parametrize("T", [20, 1500])
def test_invalid_and_repeated_choices(moe, T):
    x, ids, w, dw = make(T, 64, 4, 12)
    ids[2, 1] = -1
    ids[7, 0] = 64
    ids[9] = 5                                   # the same expert four times
    got = call(moe, x, ids, w, dw)
    assert got[4] == -5
    check(got, x, ids, w, dw, None)


def test_loss_only_in_place_and_large_logits(moe):
    x, ids, w, dw = make(700, 128, 4, 13, scale=30.0)
    full = call(moe, x, ids, w, dw)
    check(full, x, ids, w, dw, None)
    only = call(moe, x, ids, outputs=False)
    assert np.array_equal(only[2], full[2])
    inp = call(moe, x, ids, w, dw, in_place=True)
    assert np.array_equal(inp[3], full[3])


def test_same_bits_again_and_on_another_stream(moe):
    x, ids, w, dw = make(9000, 128, 4, 14)
    a = call(moe, x, ids, w, dw)
    s = torch.cuda.Stream()
    ws = torch.zeros(moe.moe_router_loss_workspace_size(128), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        b = call(moe, x, ids, w, dw, ctx=moe.Ctx(stream=s, workspace=ws))
        c = call(moe, x, ids, w, dw, ctx=moe.Ctx(stream=s, workspace=ws))
    for i in range(4):
        assert np.array_equal(a[i], b[i]) and np.array_equal(a[i], c[i])


def test_gradient_is_the_loss_difference(moe):
    """A step along the gradient changes the loss by the gradient's square, to first order."""
    x, ids, _, _ = make(64, 32, 2, 15)
    _, _, l0, d, _ = call(moe, x, ids, a=1.0, b=1.0)
    gg = float((d.astype(np.float64) ** 2).sum())
    h = 1e-2 / np.sqrt(gg)
    lp = orl.router_loss(x + h * d.astype(np.float64), ids, None, None, None, 1.0, 1.0)[2][0]
    lm = orl.router_loss(x - h * d.astype(np.float64), ids, None, None, None, 1.0, 1.0)[2][0]
    # the quotient's own error is of second order in the step's length 1e-2
    assert abs((lp - lm) / (2 * h) - gg) <= 1e-3 * gg


def test_offsets_past_32_bits(moe):
    """More than 2^31 logits: rows on both sides of the wrap, against torch in float64."""
    T, E, k = 2_200_000, 1000, 4
    g = torch.Generator(device="cuda").manual_seed(16)
    x = torch.randn((T, E), generator=g, device="cuda")
    val, ids = x.topk(k, dim=1)
    w, dw = torch.softmax(val, 1), torch.randn((T, k), generator=g, device="cuda")
    ids = ids.to(torch.int32)
    counts, loss, d = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(3, device="cuda"), torch.empty_like(x)
    ws = torch.empty(moe.moe_router_loss_workspace_size(E), dtype=torch.uint8, device="cuda")
    moe.moe_router_loss(x, ids, w, dw, None, T, k, E, 1.0, 0.0, counts, None, loss, d, moe.Ctx(workspace=ws))
    torch.cuda.synchronize()
    assert torch.equal(counts.long(), torch.bincount(ids.long().reshape(-1), minlength=E))
    rows = torch.tensor([0, 1, 2147483, 2147484, T // 2, T - 1], device="cuda")
    p = torch.softmax(x[rows].double(), 1)
    f = counts.double() * E / (T * k)
    ref = p / T * (f - (p @ f)[:, None])
    wr, dr = w[rows].double(), dw[rows].double()
    ref.scatter_add_(1, ids[rows].long(), wr * (dr - (wr * dr).sum(1, keepdim=True)))
    # the terms are of order 1 and within a few ulp each
    assert float((d[rows].double() - ref).abs().max()) < 2.0 ** -20


@pytest.mark.parametrize("E,k", [(12, 5), (16, 8), (31, 7), (60, 12), (200, 20), (700, 32)])
def test_more_choices_than_lanes(moe, E, k):
    x, ids, w, dw = make(900, E, k, 17)
    ids[3, 0] = ids[3, 1]
    check(call(moe, x, ids, w, dw), x, ids, w, dw, None)


@pytest.mark.parametrize("T,E,k", [(2000, 513, 4), (4001, 1001, 6), (3000, 1024, 8)])
def test_many_experts_and_tokens(moe, T, E, k):
    """Wide rows over every SM, with masked tokens: the losses come from a launch of their own."""
    x, ids, w, dw = make(T, E, k, 18)
    mask = (np.random.default_rng(19).random(T) < 0.8).astype(np.uint8)
    got = call(moe, x, ids, w, dw, mask)
    check(got, x, ids, w, dw, mask)
    again = call(moe, x, ids, w, dw, mask)
    assert all(np.array_equal(a, b) for a, b in zip(got[:4], again[:4]))
    got = call(moe, x, ids, w, dw, np.zeros(T, np.uint8))
    assert not got[0].any() and not got[1].any() and not got[2].any() and not got[3].any()


@pytest.mark.parametrize("T,E,k", [(1, 1001, 6), (12, 1024, 32), (13, 513, 4), (90, 700, 8), (97, 1001, 6)])
def test_many_experts_few_tokens(moe, T, E, k):
    x, ids, w, dw = make(T, E, k, 20)
    check(call(moe, x, ids, w, dw), x, ids, w, dw, None)
