"""Rows that do not count are zeros whatever the norm's weight holds, forward and back; where the weight is
finite the rows that count keep their values.  No tolerances: zeros, and bits equal to those of a weight
whose odd entries are 1."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
EPS = 1e-5
# narrow rows, a block a row, blocks that walk over rows (bf16, with codes or dropout), two eights a thread
SIZES = [(20, 64), (21, 256), (7000, 256), (900, 2880), (900, 7168), (140, 12288)]


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_grouped_align_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.build()
    m.load()
    return m


class Inputs:
    def __init__(self, T, K, f32):
        g = torch.Generator(device="cuda").manual_seed(T + K)
        self.dt = torch.float32 if f32 else torch.bfloat16
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.x, self.res, self.do, self.ds = rnd(T, K).bfloat16(), rnd(T, K).to(self.dt), rnd(T, K).bfloat16(), rnd(T, K).to(self.dt)
        self.mask = (torch.rand(T, generator=g, device="cuda") < 0.6).to(torch.uint8)
        self.clean = torch.ones(K, dtype=torch.bfloat16, device="cuda")
        self.dirty, self.odd = self.clean.clone(), torch.zeros(K, dtype=torch.bool, device="cuda")
        for i, v in ((3, "nan"), (K // 2, "inf"), (K - 1, "-inf")):
            self.dirty[i], self.odd[i] = float(v), True
        self.rng = torch.tensor([3, 4], device="cuda")


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("quant,p", [(None, 0.0), (None, 0.1), ("mx", 0.0), ("row", 0.0)])
def test_forward(moe, T, K, f32, quant, p):
    c = Inputs(T, K, f32)
    got = []
    for w in (c.dirty, c.clean):
        st, o = torch.full((T, K), 7.0, dtype=c.dt, device="cuda"), torch.full((T, K), 7.0, dtype=torch.bfloat16, device="cuda")
        codes = torch.full((T, K), 0xA5, dtype=torch.uint8, device="cuda") if quant else None
        sc = {None: None, "mx": torch.full((T, K // 32), 0xA5, dtype=torch.uint8, device="cuda"),
              "row": torch.full((T,), 7.0, device="cuda")}[quant]
        moe.moe_residual_norm(c.x, c.res, c.mask, w, T, K, EPS, p, c.rng, 1, st, o, codes, sc)
        torch.cuda.synchronize()
        got.append((st, o, codes, sc))
    (st, o, codes, sc), (st1, o1, codes1, sc1) = got
    pad, keep = c.mask == 0, c.mask != 0
    assert torch.equal(st, st1) and (st[pad] == 0).all()
    assert (o[pad] == 0).all()
    assert torch.equal(o[keep][:, ~c.odd], o1[keep][:, ~c.odd]) and not torch.isfinite(o[keep][:, c.odd]).any()
    if quant:
        assert (codes[pad] & 0x7F == 0).all() and torch.equal(sc[pad], sc1[pad])
    if quant == "mx":
        whole = ~c.odd.view(-1, 32).any(dim=1)  # blocks without an odd weight
        assert torch.equal(sc[keep][:, whole], sc1[keep][:, whole])


@pytest.mark.parametrize("T,K", SIZES)
@pytest.mark.parametrize("f32", [False, True])
def test_backward(moe, T, K, f32):
    c = Inputs(T, K, f32)
    got = []
    for w in (c.dirty, c.clean):
        dr, dx = torch.full((T, K), 7.0, dtype=c.dt, device="cuda"), torch.full((T, K), 7.0, dtype=torch.bfloat16, device="cuda")
        dw = torch.full((K,), 7.0, device="cuda")
        ws = torch.full((moe.moe_residual_norm_workspace_size(K),), 0xFF, dtype=torch.uint8, device="cuda")
        moe.moe_residual_norm_backward(c.do, c.ds, c.res, c.mask, w, T, K, EPS, 0.1, c.rng, 1, dr, dx, dw, moe.Ctx(workspace=ws))
        torch.cuda.synchronize()
        got.append((dr, dx, dw))
    (dr, dx, dw), (_, _, dw1) = got
    pad = c.mask == 0
    assert (dr[pad] == 0).all() and (dx[pad] == 0).all()
    assert torch.equal(dw, dw1)  # the weight's gradient does not go by the weight
    assert np.isfinite(dw.cpu().numpy()).all()
