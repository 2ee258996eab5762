"""Workloads of what stands around an expert layer: the residual norm with dropout and 8-bit
outputs, its backward pass, and the low-rank adapters of many requests beside a dense product.

``listed`` names the workloads that are timed, ``draw`` gives further ones of the same ranges,
``prepare`` makes a workload's inputs on the GPU, ``run`` is one pass (elementary torch
operations in 32 bits, or the library's kernels where ``own`` is true), ``work`` the bytes
and operations a pass cannot do without, and ``exact`` the results in 64 bits.
"""
import math

import torch

own = False

SCRATCH_BYTES = 64 << 20  # the device scratch a program keeps for its calls
EPS = 1e-5


# ---------------------------------------------------------------------------- the workloads

def _norm(name, T, K, quant, out16=True, stream="bf16", branch=True):
    """The norm of T rows of K: ``branch``: a layer's output is added to the residual first.
    quant: "none", "mx" (a power of two per 32 values) or "row" (a scale per row), beside or
    (out16 false) instead of the bf16 rows."""
    return {"name": name, "op": "norm", "T": T, "K": K, "quant": quant, "out16": out16, "stream": stream,
            "branch": branch}


def _train(name, T, K, p, real, stream="bf16"):
    """Dropout of probability p, residual addition and norm, forward and back; the first ``real``
    rows are tokens, the others padding."""
    return {"name": name, "op": "train", "T": T, "K": K, "p": p, "real": real, "stream": stream}


def _adapter(name, M, requests, adapters, rank, N, K, bare, out="bf16"):
    """M rows of ``requests`` requests, each of which uses one of ``adapters`` adapters or, with
    probability ``bare``, none."""
    return {"name": name, "op": "adapter", "M": M, "requests": requests, "adapters": adapters, "rank": rank, "N": N,
            "K": K, "bare": bare, "out": out}


def listed():
    return [
        # one token into an MXFP8 layer: bf16 rows for the router, codes for the experts
        _norm("norm_token", 1, 7168, "mx"),
        # a decode batch of the 2880-wide layer
        _norm("norm_decode", 64, 2880, "none"),
        # an odd batch into the per-token FP8 product alone, residual stream in 32 bits
        _norm("norm_row", 1001, 2688, "row", out16=False, stream="f32"),
        # a prefill chunk into an MXFP8 layer
        _norm("norm_prefill", 8192, 7168, "mx"),
        # a tiny training batch
        _train("train_small", 28, 2688, 0.1, 28),
        # sixteen packed requests, padded to their bucket, residual stream in 32 bits
        _train("train_padded", 61440, 2880, 0.05, 58879, stream="f32"),
        # one training micro-batch of the wide layer
        _train("train_wide", 8192, 7168, 0.1, 8192),
        # one token with its adapter
        _adapter("adapter_token", 1, 1, 8, 16, 2880, 2880, 0.0),
        # a decode batch, a request a token, most with adapters of their own
        _adapter("adapter_decode", 64, 64, 100, 16, 5760, 2880, 0.1),
        # a larger decode batch over a few popular adapters
        _adapter("adapter_popular", 250, 250, 5, 64, 4096, 7168, 0.2),
        # prompts of uneven lengths in one chunk
        _adapter("adapter_prompts", 8192, 16, 8, 32, 4096, 7168, 0.1),
        # sixteen long prompts through a square projection
        _adapter("adapter_long", 58879, 16, 6, 64, 2880, 2880, 0.0),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "train", "adapter"])
    stream = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        quant = rng.choice(["none", "mx", "mx", "row"])
        K = rng.choice([64, 256, 928, 1856, 2048, 2688, 2880, 4096, 5120, 7168, 12288] +
                       ([] if quant == "mx" else [136, 520, 4104]))
        T = _logint(rng, 1, min(61440, 8192 * 7168 // K))
        c = _norm("", T, K, quant, quant == "none" or rng.random() < 0.7, stream, rng.random() < 0.85)
    elif op == "train":
        K = rng.choice([64, 136, 256, 520, 928, 1856, 2048, 2688, 2880, 4104, 7168, 12288])
        T = _logint(rng, 1, min(61440, 8192 * 7168 // K))
        real = T if rng.random() < 0.6 else max(1, T - rng.randrange(T // 8 + 1))
        c = _train("", T, K, rng.choice([0.0, 0.05, 0.1, 0.25]), real, stream)
    else:
        N = rng.choice([64, 256, 520, 928, 1856, 2048, 2880, 4096, 4104, 5760, 7168])
        K = rng.choice([64, 256, 520, 928, 1856, 2048, 2688, 2880, 4096, 4104, 7168])
        rank = rng.choice([8, 16, 16, 24, 32, 64, 128])
        out = "f32" if rng.random() < 0.2 else "bf16"
        # no more bytes or operations than the largest listed one
        most = min(58879 * 6 * 2880 // (2 * K + (8 if out == "f32" else 4) * N), 58879 * 2 * 2880 * 64 // (rank * (N + K)))
        M = _logint(rng, 1, min(58879, most))
        requests = M if M <= 512 and rng.random() < 0.6 else min(M, _logint(rng, 1, 128))
        adapters = _logint(rng, 1, 200 if M <= 512 else 12)
        c = _adapter("", M, requests, adapters, rank, N, K, rng.choice([0.0, 0.1, 0.5]), out)
    del c["name"]
    return c


# ------------------------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    bf, f32 = torch.bfloat16, torch.float32
    s = {"case": case, "ws": torch.empty(SCRATCH_BYTES, dtype=torch.uint8, device="cuda"), "ctx": {}}
    new = lambda *shape, dtype=bf: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if case["op"] == "adapter":
        M, N, K, L, r, R = (case[k] for k in ("M", "N", "K", "adapters", "rank", "requests"))
        host = torch.Generator().manual_seed(int(seed))
        # the requests' lengths: uneven parts of M, one row each at least
        cuts = torch.randperm(M - 1, generator=host)[:R - 1].sort().values + 1
        edges = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([M])])
        # popular adapters first: the square of a uniform number
        pick = (torch.rand(R, generator=host).square() * L).long().clamp(max=L - 1)
        pick[torch.rand(R, generator=host) < case["bare"]] = -1
        s["row_offsets"], s["adapter"] = edges.int().cuda(), pick.int().cuda()
        s["x"] = _normal(g, (M, K), 1.0, bf)
        # adapters whose product is a part of the projection's output
        s["a"] = _normal(g, (L, r, K), K ** -0.5, bf)
        s["b"] = _normal(g, (L, N, r), r ** -0.5, bf)
        s["scale"] = torch.rand(L, generator=g, device="cuda").mul_(0.5).add_(0.25)
        s["base"] = _normal(g, (M, N), 1.0, f32 if case["out"] == "f32" else bf)  # the shared projection's output
        s["out"] = torch.empty_like(s["base"])
        return s
    T, K = case["T"], case["K"]
    dt = f32 if case["stream"] == "f32" else bf
    # a residual stream with a few large channels, as they grow over the layers
    grow = 1.0 + 20.0 * (torch.rand((1, K), generator=g, device="cuda") < 0.01).float()
    s["residual"] = (_normal(g, (T, K), 2.0) * grow).to(dt)
    s["weight"] = (1.0 + _normal(g, (K,), 0.2)).to(bf)
    if case["op"] == "norm":
        s["x"] = _normal(g, (T, K), 1.0, bf) if case["branch"] else None
        s["out"] = {"stream": new(T, K, dtype=dt) if case["branch"] else None,
                    "out": new(T, K) if case["out16"] else None}
        s["codes"] = new(T, K, dtype=torch.uint8) if case["quant"] != "none" else None
        s["scales"] = {"none": None, "mx": new(T, K // 32, dtype=torch.uint8) if K % 32 == 0 else None,
                       "row": new(T, dtype=f32)}[case["quant"]]
        return s
    s["x"] = _normal(g, (T, K), 1.0, bf)
    s["d_out"] = _normal(g, (T, K), 0.02, bf)
    s["d_stream"] = _normal(g, (T, K), 0.02).to(dt)
    real = case["real"]
    if real < T:  # what the bucket padding writes, and gradients that nothing reads
        for n in ("x", "residual", "d_out", "d_stream"):
            s[n][real:] = 0.0
    s["mask"] = (torch.arange(T, device="cuda") < real).to(torch.uint8) if real < T else None
    s["rng"] = torch.tensor([int(seed) * 0x9E3779B97F4A7C15 % (1 << 63), int(seed) % 1000], device="cuda")
    s["out"] = {"stream": new(T, K, dtype=dt), "out": new(T, K), "d_residual": new(T, K, dtype=dt), "d_x": new(T, K),
                "d_weight": new(K, dtype=f32)}
    return s


# ------------------------------------------------------------------------------- the passes

def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "train": _own_train, "adapter": _own_adapter}[op](state)
    return {"norm": _plain_norm, "train": _plain_train, "adapter": _plain_adapter}[op](state)


LAYER = 3  # which of a model's dropouts this is: a word of the generator's counter


def _ctx(moe, state):
    """The call context of the current stream, made once per stream."""
    stream = torch.cuda.current_stream().cuda_stream
    c = state["ctx"].get(stream)
    if c is None:
        c = state["ctx"][stream] = moe.Ctx(stream=stream, workspace=state["ws"])
    return c


def _held(s):
    """8-bit outputs as the numbers that their codes and scales stand for."""
    scales = s["scales"]
    return {"codes": s["codes"].view(torch.float8_e4m3fn),
            "scales": scales.view(torch.float8_e8m0fnu) if scales.dtype == torch.uint8 else scales}


def _own_norm(s):
    import mixture_experts_grouped_align_gb300 as moe
    c, o = s["case"], s["out"]
    moe.moe_residual_norm(s["x"], s["residual"], None, s["weight"], c["T"], c["K"], EPS, 0.0, None, 0, o["stream"],
                          o["out"], s["codes"], s["scales"], _ctx(moe, s))
    return o if s["codes"] is None else {**o, **_held(s)}


def _own_train(s):
    import mixture_experts_grouped_align_gb300 as moe
    c, o = s["case"], s["out"]
    ctx = _ctx(moe, s)
    moe.moe_residual_norm(s["x"], s["residual"], s["mask"], s["weight"], c["T"], c["K"], EPS, c["p"], s["rng"], LAYER,
                          o["stream"], o["out"], None, None, ctx)
    moe.moe_residual_norm_backward(s["d_out"], s["d_stream"], o["stream"], s["mask"], s["weight"], c["T"], c["K"], EPS,
                                   c["p"], s["rng"], LAYER, o["d_residual"], o["d_x"], o["d_weight"], ctx)
    return o


def _own_adapter(s):
    import mixture_experts_grouped_align_gb300 as moe
    c = s["case"]
    moe.moe_adapter_gemm(s["x"], s["a"], s["b"], s["scale"], s["row_offsets"], s["adapter"], s["base"], c["M"], c["N"],
                         c["K"], c["rank"], c["adapters"], c["requests"], s["out"], _ctx(moe, s))
    return s["out"]


def _plain_norm(s):
    """s = residual + x;  n = s (mean(s^2) + eps)^(-1/2) w;  n rounded to bf16, and to E4M3 under
    scales of 32 values or of a row."""
    c = s["case"]
    v = s["residual"].float()
    stream = None
    if s["x"] is not None:
        v = v + s["x"].float()
        stream = v.to(s["residual"].dtype)
    n = v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
    r = {"stream": stream, "out": n.to(torch.bfloat16) if c["out16"] else None}
    if c["quant"] == "mx":
        b = n.reshape(c["T"], -1, 32)
        e = (torch.frexp(b.abs().amax(dim=2, keepdim=True)).exponent - 9).clamp(-127, 127).float()
        r["codes"] = _plain_e4m3(b * torch.exp2(-e)).reshape(n.shape).to(torch.float8_e4m3fn)
        r["scales"] = torch.exp2(e[:, :, 0]).to(torch.float8_e8m0fnu)
    elif c["quant"] == "row":
        top = n.abs().amax(dim=1, keepdim=True)
        r["codes"] = _plain_e4m3(n * (448.0 / top)).to(torch.float8_e4m3fn)
        r["scales"] = (top / 448.0)[:, 0]
    return r


def _plain_e4m3(q):
    """q rounded to four significant bits, ties to even, no finer than 2^-9, at most 448."""
    step = torch.exp2((torch.frexp(q).exponent - 1).clamp(min=-6).float() - 3)
    return (torch.round(q / step) * step).clamp(-448.0, 448.0)


def _plain_keep(rng, T, K, p):
    """1 / (1 - p) where a [T, K] element is kept and 0 where it is dropped: ten rounds of the
    counter-based generator Philox 4x32 on (index / 8, step, layer) under the seed give eight 16-bit
    numbers, and those below 65536 p are dropped."""
    low = 0xFFFFFFFF
    d = min(65535, round(p * 65536))
    i = torch.arange(T * K // 8, device=rng.device)
    x0, x1, x2, x3 = i & low, i >> 32, (rng[1] & low).expand_as(i), torch.full_like(i, LAYER)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low

    for _ in range(10):
        p0, p1 = x0 * 0xD2511F53, x2 * 0xCD9E8D57
        x0, x1, x2, x3 = ((p1 >> 32) & low) ^ x1 ^ k0, p1 & low, ((p0 >> 32) & low) ^ x3 ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    x = torch.stack([x0, x1, x2, x3], dim=1)
    u = torch.stack([x & 0xFFFF, x >> 16], dim=2).reshape(T, K)
    return torch.where(u >= d, 65536.0 / (65536 - d), 0.0)


def _plain_train(s):
    """Forward as above with the dropped branch; backward from the stream as it is stored:
    ds = r g - v r^3 mean(g v) + dstream with g = dout w and r = (mean(v^2) + eps)^(-1/2)."""
    c = s["case"]
    bf = torch.bfloat16
    live = 1.0 if s["mask"] is None else s["mask"][:, None].float()
    w = s["weight"].float()
    keep = _plain_keep(s["rng"], c["T"], c["K"], c["p"]) * live
    v = s["residual"].float() * live + s["x"].float() * keep
    stream = v.to(s["residual"].dtype)
    out = v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS) * w
    v, do = stream.float(), s["d_out"].float() * live
    r = 1 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    g = do * w
    ds = r * (g - v * (r * r * (g * v).mean(dim=1, keepdim=True))) + s["d_stream"].float() * live
    return {"stream": stream, "out": out.to(bf), "d_residual": ds.to(stream.dtype), "d_x": (ds * keep).to(bf),
            "d_weight": (do * (v * r)).sum(dim=0)}


def _plain_adapter(s):
    """out = base + scale (x A^T) B^T with each row's adapter: all adapters side by side, with zeros
    where the row's is another."""
    c = s["case"]
    L, r, N = c["adapters"], c["rank"], c["N"]
    lengths = (s["row_offsets"][1:] - s["row_offsets"][:-1]).long()
    mine = s["adapter"].long().repeat_interleave(lengths, output_size=c["M"])
    pick = torch.where(mine[:, None] == torch.arange(L, device=mine.device), s["scale"], 0.0)
    v = (s["x"].float() @ s["a"].float().reshape(L * r, -1).t()).reshape(-1, L, r) * pick[:, :, None]
    b = s["b"].float().transpose(1, 2).reshape(L * r, N)
    return (s["base"].float() + v.reshape(-1, L * r) @ b).to(s["base"].dtype)


# ---------------------------------------------------------------------------- floors and truth

def work(case):
    if case["op"] == "adapter":
        M, N, K, r = case["M"], case["N"], case["K"], case["rank"]
        rows = max(1.0, M * (1 - case["bare"]))
        used = min(case["adapters"], case["requests"])
        size = 4 if case["out"] == "f32" else 2
        # the rows of x with an adapter, base and out, the adapters in use
        return {"bytes": rows * 2 * K + M * 2 * size * N + 2 * used * r * (K + N), "flops": 2 * rows * r * (K + N)}
    T, K = case["T"], case["K"]
    size = 4 if case["stream"] == "f32" else 2
    if case["op"] == "norm":
        b = size * T * K + (2 + size if case["branch"] else 0) * T * K + 2 * K + (2 * T * K if case["out16"] else 0)
        b += {"none": 0, "mx": T * K + T * K // 32, "row": T * K + 4 * T}[case["quant"]]
        return {"bytes": b, "flops": 8 * T * K}
    real = case["real"]
    # forward: x and residual read, stream and rows written; backward: the rows' and the stream's
    # gradients and the stream read, the residual's and the branch's gradients written
    read = (2 + size + 2 + 2 * size) * real * K
    written = (2 * size + 4) * T * K
    return {"bytes": read + written + 8 * K + (2 * T if real < T else 0), "flops": 30 * real * K}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "train": _exact_train, "adapter": _exact_adapter}[case["op"]](case, s)


def _exact_norm(case, s):
    parts = {"stream": [], "out": [], "codes": [], "scales": []}
    # the finite values of E4M3, and the middles between neighbours
    e4m3 = torch.tensor([(m / 8.0 * 2.0 ** -6) if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                         for e in range(16) for m in range(8)][:127], dtype=torch.float64, device="cuda")
    mid = (e4m3[1:] + e4m3[:-1]) / 2

    def nearest(y):
        m = y.abs().contiguous()
        lo, hi = torch.bucketize(m, mid, right=False), torch.bucketize(m, mid, right=True)
        return e4m3[torch.where((lo != hi) & (lo % 2 == 1), hi, lo)] * torch.sign(y)

    for i in range(0, case["T"], 4096):
        v = s["residual"][i:i + 4096].double()
        if case["branch"]:
            v = v + s["x"][i:i + 4096].double()
            parts["stream"].append(v)
        n = v * torch.rsqrt(v.square().sum(dim=1, keepdim=True) / case["K"] + EPS) * s["weight"].double()
        parts["out"].append(n)
        if case["quant"] == "mx":
            b = n.reshape(len(n), -1, 32)
            e = torch.floor(torch.log2(b.abs().amax(dim=2, keepdim=True)) + 1e-12) - 8
            parts["codes"].append(nearest(b / torch.exp2(e)).reshape(n.shape))
            parts["scales"].append(torch.exp2(e).squeeze(2))
        elif case["quant"] == "row":
            unit = n.abs().amax(dim=1) / 448
            parts["codes"].append(nearest(n / unit[:, None]))
            parts["scales"].append(unit)
    r = {k: torch.cat(v) if v else None for k, v in parts.items()}
    if not case["out16"]:
        r["out"] = None
    return r if case["quant"] != "none" else {"stream": r["stream"], "out": r["out"]}


def _exact_kept(s, T, K, p, rows):
    """Which elements of some rows are kept: the generator's rounds in 16-bit limbs."""
    def wide(a, b):  # the high and the low word of a product of 32-bit numbers
        t = (a & 0xFFFF) * (b & 0xFFFF)
        u = (a >> 16) * (b & 0xFFFF) + (t >> 16)
        v = (a & 0xFFFF) * (b >> 16) + (u & 0xFFFF)
        return (a >> 16) * (b >> 16) + (u >> 16) + (v >> 16), ((v & 0xFFFF) << 16) | (t & 0xFFFF)

    seed, step = (int(v) for v in s["rng"].cpu())
    n = torch.arange(rows.start * K // 8, rows.stop * K // 8, device="cuda")
    c = [n % (1 << 32), n // (1 << 32), torch.full_like(n, step), torch.full_like(n, LAYER)]
    key = [seed % (1 << 32), seed >> 32]
    for _ in range(10):
        h0, l0 = wide(c[0], 0xD2511F53)
        h1, l1 = wide(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ key[0], l1, h0 ^ c[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
    u = torch.empty((len(n), 8), dtype=torch.int64, device="cuda")
    for j in range(4):
        u[:, 2 * j], u[:, 2 * j + 1] = c[j] % 65536, c[j] // 65536
    return u.reshape(len(rows), K) >= min(65535, round(p * 65536))


def _exact_train(case, s):
    T, K, p = case["T"], case["K"], case["p"]
    gain = 65536 / (65536 - min(65535, round(p * 65536)))
    dt = s["residual"].dtype
    w = s["weight"].double()
    parts = {"stream": [], "out": [], "d_residual": [], "d_x": []}
    dw = torch.zeros(K, dtype=torch.float64, device="cuda")
    for i in range(0, T, 4096):
        j = min(T, i + 4096)
        live = torch.arange(i, j, device="cuda")[:, None] < case["real"]
        kept = _exact_kept(s, T, K, p, range(i, j)) & live
        x = torch.where(kept, s["x"][i:j].double(), 0.0)
        res = torch.where(live, s["residual"][i:j].double(), 0.0)
        v = res + x * gain
        parts["stream"].append(v)
        parts["out"].append(v / (v.square().mean(dim=1, keepdim=True) + EPS).sqrt() * w)
        # the backward pass is a call of its own: its input is the stream in the type it is held in,
        # a product and a sum of 32 bits, each rounded
        v = (res.float() + x.float() * gain).to(dt).double()
        do = torch.where(live, s["d_out"][i:j].double(), 0.0)
        rms = (v.square().mean(dim=1, keepdim=True) + EPS).sqrt()
        h = v / rms
        g = do * w
        ds = (g - h * (g * h).mean(dim=1, keepdim=True)) / rms + torch.where(live, s["d_stream"][i:j].double(), 0.0)
        parts["d_residual"].append(ds)
        parts["d_x"].append(torch.where(kept, ds * gain, 0.0))
        dw += (do * h).sum(dim=0)
    return {**{k: torch.cat(v) for k, v in parts.items()}, "d_weight": dw}


def _exact_adapter(case, s):
    out = s["base"].double()
    edges, pick = s["row_offsets"].tolist(), s["adapter"].tolist()
    for lo, hi, a in zip(edges[:-1], edges[1:], pick):
        if a >= 0:
            v = s["x"][lo:hi].double() @ s["a"][a].double().mT
            out[lo:hi] += s["scale"][a].double() * (v @ s["b"][a].double().mT)
    return out
