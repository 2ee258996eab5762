"""Workloads of the training and dense operators: the router's auxiliary losses, the expert
activation with an 8-bit checkpoint, and the dense matrix product with a fused epilogue.

``listed`` names the workloads that are timed, ``draw`` gives further ones of the same ranges,
``prepare`` makes a workload's inputs on the GPU, ``run`` is one pass (elementary torch
operations in 32 bits, or the library's kernels where ``own`` is true), ``work`` the bytes
and operations a pass cannot do without, and ``exact`` the results in 64 bits.
"""
import math

import torch

own = False

SCRATCH_BYTES = 64 << 20  # the device scratch a program keeps for its calls


# ---------------------------------------------------------------------------- the workloads

def _router(name, T, E, k, real, allowed, upstream):
    """T rows of E logits, the first ``real`` of them tokens; each token may choose among
    ``allowed`` experts (the others' logits are -inf); ``upstream``: with a gradient of the
    routing weights."""
    return {"name": name, "op": "router", "T": T, "E": E, "k": k, "real": real, "allowed": allowed,
            "upstream": upstream}


def _act(name, rows, I, act, weighted):
    return {"name": name, "op": "act", "rows": rows, "I": I, "act": act, "weighted": weighted}


def _dense(name, M, N, K, act="none", bias=False, residual=False, out="bf16", form="forward"):
    return {"name": name, "op": "dense", "M": M, "N": N, "K": K, "act": act, "bias": bias,
            "residual": residual, "out": out, "form": form}


def listed():
    return [
        # a 64-token batch of the 128-expert layer: the latency of the call
        _router("router_small", 64, 128, 4, 64, 128, False),
        # an odd batch whose tokens may use a third of the experts each, odd expert count
        _router("router_limited", 1001, 130, 6, 1001, 44, True),
        # one training micro-batch of the 256-expert layer
        _router("router_train", 8192, 256, 8, 8192, 256, True),
        # sixteen packed requests, padded to their bucket: the pad rows count for nothing
        _router("router_padded", 61440, 128, 4, 58879, 128, True),
        # 28 tokens of the six-expert layer: pairs of a tiny batch
        _act("act_small", 168, 928, "swiglu", True),
        # ungated experts, odd number of rows
        _act("act_relu2", 12345, 1856, "relu2", False),
        # every pair of a training micro-batch of the large layer
        _act("act_train", 65536, 2048, "swiglu", True),
        # one token through an ungated dense layer: the weights' stream
        _dense("dense_token", 1, 1856, 2688, act="relu2", bias=True),
        # a decode batch through a gated dense expert
        _dense("dense_decode", 64, 2880, 2880, act="swiglu", bias=True),
        # the router's projection, whose logits stay in 32 bits
        _dense("dense_router", 4099, 256, 7168, out="f32"),
        # a training micro-batch through a gated dense expert
        _dense("dense_up", 8192, 2048, 7168, act="swiglu", bias=True),
        # its backward pass: the input's gradient joined to the residual path's, and the bias's
        _dense("dense_backward", 8191, 7168, 4096, residual=True, form="backward"),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "act", "dense"])
    if op == "router":
        E = rng.choice([8, 31, 60, 64, 128, 130, 160, 256, 384, 512, 1001])
        k = min(rng.choice([1, 2, 4, 6, 8]), E // 4)
        T = _logint(rng, 1, min(61440, 61440 * 128 // E))
        real = T if rng.random() < 0.5 else max(1, T - rng.randrange(T // 8 + 1))
        allowed = E if rng.random() < 0.6 else rng.randint(max(k, E // 4), E)
        return {k2: v for k2, v in _router("", T, E, k, real, allowed, rng.random() < 0.7).items() if k2 != "name"}
    if op == "act":
        I = rng.choice([64, 96, 160, 352, 512, 928, 1408, 1856, 2048, 2880, 5760])
        rows = _logint(rng, 1, min(100000, 65536 * 2048 // I))
        return {k2: v for k2, v in _act("", rows, I, rng.choice(["swiglu", "swiglu", "relu2"]),
                                        rng.random() < 0.6).items() if k2 != "name"}
    form = rng.choice(["forward", "forward", "forward", "backward"])
    N = rng.choice([8, 64, 136, 256, 520, 928, 1856, 2048, 2880, 4104, 7168])
    K = rng.choice([64, 136, 256, 520, 928, 1856, 2048, 2688, 2880, 4104, 7168])
    act = rng.choice(["none", "none", "swiglu", "relu2"]) if form == "forward" else "none"
    gates = 2 if act == "swiglu" else 1
    M = _logint(rng, 1, min(16384, max(1, 8191 * 7168 * 4096 // (N * gates * K))))
    out = "f32" if act == "none" and form == "forward" and rng.random() < 0.3 else "bf16"
    return {k2: v for k2, v in _dense("", M, N, K, act, form == "forward" and rng.random() < 0.5, rng.random() < 0.4,
                                      out, form).items() if k2 != "name"}


# ------------------------------------------------------------------------------- the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case, "ws": torch.empty(SCRATCH_BYTES, dtype=torch.uint8, device="cuda"), "ctx": {}}
    bf = torch.bfloat16
    if case["op"] == "router":
        T, E, k, real = case["T"], case["E"], case["k"], case["real"]
        # logits of an unevenly loaded router: an offset for each expert
        x = _normal(g, (T, E), 1.0) + _normal(g, (1, E), 0.5)
        if case["allowed"] < E:
            order = torch.rand((T, E), generator=g, device="cuda").argsort(dim=1)
            x = x.masked_fill(order >= case["allowed"], float("-inf"))
        if real < T:
            x[real:] = 0.0  # what the bucket padding writes
        val, ids = x.topk(k, dim=1)
        s["logits"], s["ids"] = x, ids.to(torch.int32)
        s["w"] = torch.softmax(val, dim=1)
        s["dw"] = _normal(g, (T, k), 1e-3) if case["upstream"] else None
        s["mask"] = (torch.arange(T, device="cuda") < real).to(torch.uint8) if real < T else None
        s["coef"] = (0.01, 0.001)
        s["out"] = {"counts": torch.empty(E, dtype=torch.int32, device="cuda"),
                    "prob_mean": torch.empty(E, device="cuda"), "loss": torch.empty(3, device="cuda"),
                    "d_logits": torch.empty((T, E), device="cuda")}
    elif case["op"] == "act":
        R, I = case["rows"], case["I"]
        N1 = 2 * I if case["act"] == "swiglu" else I
        # pre-activations and gradients as the products before and after leave them
        s["gu"] = _normal(g, (R, N1), 1.5, bf)
        s["dh"] = _normal(g, (R, I), 0.02, bf)
        s["row_w"] = torch.rand(R, generator=g, device="cuda").mul_(0.5).add_(0.01) if case["weighted"] else None
        s["codes"] = torch.empty((R, N1), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty((R, N1 // 32), dtype=torch.uint8, device="cuda")
        s["out"] = {"h": torch.empty((R, I), dtype=bf, device="cuda"),
                    "d_gu": torch.empty((R, N1), dtype=bf, device="cuda"),
                    "h_again": torch.empty((R, I), dtype=bf, device="cuda"),
                    "d_row_w": torch.empty(R, device="cuda") if case["weighted"] else None}
    else:
        M, N, K = case["M"], case["N"], case["K"]
        N1 = 2 * N if case["act"] == "swiglu" else N
        dt = torch.float32 if case["out"] == "f32" else bf
        s["x"] = _normal(g, (M, K), 1.0, bf)
        # the weight as the forward pass stores it: [N1, K]; the backward pass contracts over
        # the rows of the [K, N] weight of the layer it goes back through
        s["weight"] = _normal(g, (K, N) if case["form"] == "backward" else (N1, K), 0.02, bf)
        s["bias"] = _normal(g, (N1,), 0.02, bf) if case["bias"] else None
        s["residual"] = _normal(g, (M, N), 1.0, dt) if case["residual"] else None
        s["out"] = {"out": torch.empty((M, N), dtype=dt, device="cuda")}
        if case["form"] == "backward":
            s["out"]["d_bias"] = torch.empty(K, device="cuda")
    return s


# ------------------------------------------------------------------------------- the passes

def run(state):
    op = state["case"]["op"]
    if own:
        return {"router": _own_router, "act": _own_act, "dense": _own_dense}[op](state)
    return {"router": _plain_router, "act": _plain_act, "dense": _plain_dense}[op](state)


def _ctx(moe, state):
    """The call context of the current stream, made once per stream."""
    stream = torch.cuda.current_stream().cuda_stream
    c = state["ctx"].get(stream)
    if c is None:
        c = state["ctx"][stream] = moe.Ctx(stream=stream, workspace=state["ws"])
    return c


def _own_router(s):
    import mixture_experts_grouped_align_gb300 as moe
    c, o = s["case"], s["out"]
    moe.moe_router_loss(s["logits"], s["ids"], s["w"], s["dw"], s["mask"], c["T"], c["k"], c["E"], s["coef"][0],
                        s["coef"][1], o["counts"], o["prob_mean"], o["loss"], o["d_logits"], _ctx(moe, s))
    return o


def _own_act(s):
    import mixture_experts_grouped_align_gb300 as moe
    c, o = s["case"], s["out"]
    ctx = _ctx(moe, s)
    moe.moe_act_checkpoint(s["gu"], s["row_w"], c["rows"], c["I"], c["act"], o["h"], s["codes"], s["scales"], ctx)
    moe.moe_act_backward(s["codes"], s["scales"], s["dh"], s["row_w"], c["rows"], c["I"], c["act"], o["d_gu"],
                         o["h_again"], o["d_row_w"], ctx)
    return o


def _own_dense(s):
    import mixture_experts_grouped_align_gb300 as moe
    c, o = s["case"], s["out"]
    ctx = _ctx(moe, s)
    back = c["form"] == "backward"
    moe.moe_dense_gemm(s["x"], s["weight"], "kn" if back else "nk", s["bias"], s["residual"], 1.0, c["M"], c["N"],
                       c["K"], c["act"], o["out"], ctx)
    if back:
        moe.moe_dense_bias_grad(s["x"], c["M"], c["K"], o["d_bias"], ctx)
    return o


def _plain_router(s):
    """loss = a E sum_e f_e P_e + b mean(lse^2) over the real tokens, with its gradient and
    that of the routing weights (a softmax over the chosen logits)."""
    x, ids, w = s["logits"], s["ids"].long(), s["w"]
    T, E = x.shape
    k = ids.shape[1]
    a, b = s["coef"]
    live = torch.ones(T, device=x.device) if s["mask"] is None else (s["mask"] != 0).float()
    n = live.sum()
    counts = torch.zeros(E, device=x.device).index_add_(0, ids.reshape(-1), live[:, None].expand(T, k).reshape(-1))
    top = x.max(dim=1, keepdim=True).values
    ex = torch.exp(x - top)
    total = ex.sum(dim=1, keepdim=True)
    p = ex / total * live[:, None]
    lse = (top + torch.log(total)) * live[:, None]
    f = counts * (E / (n * k))
    prob_mean = p.sum(dim=0) / n
    balance = (f * prob_mean).sum()
    z = (lse * lse).sum() / n
    d = (a / n) * p * (f - (f * p).sum(dim=1, keepdim=True)) + (2 * b / n) * lse * p
    if s["dw"] is not None:
        dw = s["dw"] * live[:, None]
        d = d.scatter_add(1, ids, w * (dw - (w * dw).sum(dim=1, keepdim=True)))
    return {"counts": counts.to(torch.int32), "prob_mean": prob_mean,
            "loss": torch.stack([a * balance + b * z, balance, z]), "d_logits": d}


def _plain_mxfp8(v):
    """The values that MXFP8 holds for v [R, n]: per 32 columns a scale 2^(floor(log2 max) - 8)
    and E4M3 codes, ties to even, saturated at 448."""
    b = v.reshape(v.shape[0], -1, 32)
    top = b.abs().amax(dim=2, keepdim=True)
    e = (torch.frexp(top).exponent - 9).clamp(-127, 127).float()
    q = b * torch.exp2(-e)
    step = torch.exp2((torch.frexp(q).exponent - 1).clamp(min=-6).float() - 3)
    q = (torch.round(q / step) * step).clamp(-448.0, 448.0)
    return (q * torch.exp2(e)).reshape(v.shape)


def _plain_act(s):
    c = s["case"]
    gu, dh = s["gu"].float(), s["dh"].float()
    w = torch.ones(c["rows"], device=gu.device) if s["row_w"] is None else s["row_w"]
    w = w[:, None]
    held = _plain_mxfp8(gu)
    if c["act"] == "swiglu":
        g, u = gu.chunk(2, dim=1)
        h = g / (1 + torch.exp(-g)) * u
        g, u = held.chunk(2, dim=1)
        sig = 1 / (1 + torch.exp(-g))
        again = g * sig * u
        t = w * dh
        d_gu = torch.cat([t * u * sig * (1 + g * (1 - sig)), t * g * sig], dim=1)
    else:
        h = gu.clamp(min=0.0) * gu.clamp(min=0.0)
        r = held.clamp(min=0.0)
        again = r * r
        d_gu = w * dh * 2 * r
    bf = torch.bfloat16
    return {"h": (w * h).to(bf), "d_gu": d_gu.to(bf), "h_again": (w * again).to(bf),
            "d_row_w": None if s["row_w"] is None else (dh * again).sum(dim=1)}


def _plain_dense(s):
    c = s["case"]
    back = c["form"] == "backward"
    x, wt = s["x"].float(), s["weight"].float()
    z = x @ (wt if back else wt.t())
    if s["bias"] is not None:
        z = z + s["bias"].float()
    if c["act"] == "swiglu":
        g, u = z.chunk(2, dim=1)
        z = g / (1 + torch.exp(-g)) * u
    elif c["act"] == "relu2":
        z = z.clamp(min=0.0) * z.clamp(min=0.0)
    if s["residual"] is not None:
        z = z + s["residual"].float()
    r = {"out": z.to(s["out"]["out"].dtype)}
    if back:
        r["d_bias"] = x.sum(dim=0)
    return r


# ---------------------------------------------------------------------------- floors and truth

def work(case):
    if case["op"] == "router":
        T, E, k = case["T"], case["E"], case["k"]
        b = 4 * T * E * 2 + 4 * T * k * (3 if case["upstream"] else 1) + 8 * E + 12
        return {"bytes": b + (T if case["real"] < T else 0), "flops": 12 * T * E}
    if case["op"] == "act":
        R, I = case["rows"], case["I"]
        N1 = 2 * I if case["act"] == "swiglu" else I
        held = R * N1 + R * N1 // 32
        # the pre-activation, the gradient and the outputs once, the checkpoint written and read
        return {"bytes": 2 * R * N1 * 2 + 3 * 2 * R * I + 2 * held + (12 * R if case["weighted"] else 0),
                "flops": 40 * R * I}
    M, N, K = case["M"], case["N"], case["K"]
    N1 = 2 * N if case["act"] == "swiglu" else N
    size = 4 if case["out"] == "f32" else 2
    b = 2 * M * K + 2 * N1 * K + size * M * N * (2 if case["residual"] else 1) + (2 * N1 if case["bias"] else 0)
    return {"bytes": b + (4 * K if case["form"] == "backward" else 0), "flops": 2 * M * N1 * K}


def exact(case, seed):
    s = prepare(case, seed)
    return {"router": _exact_router, "act": _exact_act, "dense": _exact_dense}[case["op"]](case, s)


def _exact_router(case, s):
    x = s["logits"].double()
    T, E, k = case["T"], case["E"], case["k"]
    live = torch.ones(T, dtype=torch.bool, device=x.device) if s["mask"] is None else s["mask"].bool()
    n = int(live.sum())
    a, b = s["coef"]
    ids = s["ids"].long()
    counts = torch.bincount(ids[live].reshape(-1), minlength=E)
    lse = torch.logsumexp(x[live], dim=1)
    p = torch.softmax(x[live], dim=1)
    load = counts.double() / (n * k) * E
    mean = p.mean(dim=0)
    balance, z = torch.dot(load, mean), (lse ** 2).mean()
    # d balance / d logit through the softmax's Jacobian, d z / d logit = 2 lse p / n
    grad = torch.zeros(T, E, dtype=torch.float64, device=x.device)
    part = a / n * (p * load - p * (p @ load)[:, None]) + (2 * b / n) * p * lse[:, None]
    if s["dw"] is not None:
        w, dw = s["w"].double()[live], s["dw"].double()[live]
        up = w * dw - w * (w * dw).sum(dim=1, keepdim=True)
        part.scatter_add_(1, ids[live], up)
    grad[live] = part
    return {"counts": counts.to(torch.int32), "prob_mean": mean,
            "loss": torch.stack([a * balance + b * z, balance, z]), "d_logits": grad}


def _exact_act(case, s):
    R = case["rows"]
    wide = case["act"] == "swiglu"
    e4m3 = torch.tensor([(m / 8.0 * 2.0 ** -6) if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                         for e in range(16) for m in range(8)][:127], dtype=torch.float64, device="cuda")
    mid = (e4m3[1:] + e4m3[:-1]) / 2

    def hold(v):  # nearest table value, ties to the even code
        b = v.reshape(v.shape[0], -1, 32)
        top = b.abs().amax(dim=2, keepdim=True)
        # the nudge keeps a maximum that is a power of two on its own side of the logarithm's rounding
        e = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=1e-300)) + 1e-9) - 8, -127.0).clamp(-127, 127)
        y = b / torch.exp2(e)
        m = y.abs().contiguous()
        lo, hi = torch.bucketize(m, mid, right=False), torch.bucketize(m, mid, right=True)
        code = torch.where((lo != hi) & (lo % 2 == 1), hi, lo)
        return (e4m3[code] * torch.sign(y) * torch.exp2(e)).reshape(v.shape)

    parts = {"h": [], "d_gu": [], "h_again": [], "d_row_w": []}
    for r in range(0, R, 4096):
        gu, dh = s["gu"][r:r + 4096].double(), s["dh"][r:r + 4096].double()
        w = 1.0 if s["row_w"] is None else s["row_w"][r:r + 4096].double()[:, None]
        if wide:
            I = case["I"]
            gate = torch.sigmoid(gu[:, :I])
            held = hold(gu)
            g, u = held[:, :I], held[:, I:]
            sg = torch.sigmoid(g)
            parts["h"].append(w * gu[:, :I] * gate * gu[:, I:])
            again = g * sg * u
            parts["d_gu"].append(torch.cat([w * dh * u * (sg + g * sg * torch.sigmoid(-g)), w * dh * g * sg], dim=1))
        else:
            r1 = torch.relu(hold(gu))
            parts["h"].append(w * torch.relu(gu) ** 2)
            again = r1 ** 2
            parts["d_gu"].append(2 * w * dh * r1)
        parts["h_again"].append(w * again)
        parts["d_row_w"].append((dh * again).sum(dim=1))
    if s["row_w"] is None:
        parts["d_row_w"] = None
    return {n: None if v is None else torch.cat(v) for n, v in parts.items()}


def _exact_dense(case, s):
    x, wt = s["x"].double(), s["weight"].double()
    r = torch.matmul(x, wt) if case["form"] == "backward" else torch.matmul(x, wt.mT)
    if case["bias"]:
        r += s["bias"].double()
    if case["act"] == "swiglu":
        r = r[:, :case["N"]] * torch.sigmoid(r[:, :case["N"]]) * r[:, case["N"]:]
    elif case["act"] == "relu2":
        r = torch.relu(r).square()
    if case["residual"]:
        r += s["residual"].double()
    out = {"out": r}
    if case["form"] == "backward":
        out["d_bias"] = x.sum(dim=0)
    return out
