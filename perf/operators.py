"""Cases and plain forms of the operators that train the MoE block in bf16:
the norms around the block with its gate and residual scale, the experts'
products over ragged groups in all three directions, the gated activation
between them, and the gradient norm with clipping over many tensors.

``run`` computes a case either in its plain form (elementary torch operations
in float32, rounded once at the end) or, with ``own`` set, by the package's
entry points.  ``exact`` gives the same outputs from the definition in float64.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# The layer's shape: hidden width 7168, expert width 2048 (gate and up rows:
# 4096), top 8 of 256 experts.  One of eight GPUs holds 32 of the experts and
# the shared one, and a token has one pick among its 32 on average.
WIDTH, INNER = 7168, 2048
LARGEST_FLOPS = 2.0 * 16384 * (2 * INNER) * WIDTH
LARGEST_WEIGHTS = 33 * (2 * INNER) * WIDTH


def listed():
    return [
        # one token of a request being answered passes the boundary between two
        # blocks: the latency of a call
        {"name": "norm_one_token", "op": "norm", "rows": 1, "width": WIDTH, "stream": "bf16",
         "gate": "channel"},
        # the same boundary for a training or prefill batch, gated per token
        {"name": "norm_batch", "op": "norm", "rows": 8192, "width": WIDTH, "stream": "bf16",
         "gate": "token"},
        # its backward pass with a gate per channel, whose gradient sums over the batch
        {"name": "norm_backward_batch", "op": "norm_backward", "rows": 8192, "width": WIDTH,
         "stream": "bf16", "gate": "channel"},
        # a float32 residual stream of an odd width and a ragged number of rows,
        # with a gate for every element
        {"name": "norm_backward_odd", "op": "norm_backward", "rows": 1021, "width": 2049,
         "stream": "f32", "gate": "full"},
        # decode: 16 tokens, all their experts on this card; the weights' stream
        {"name": "gemm_decode", "op": "gemm", "tokens": 16, "experts": 32, "picks": 8, "skew": 0.0,
         "n": 2 * INNER, "k": WIDTH, "layout": "nk", "gather": True, "out": "bf16"},
        # the first product of a training or prefill batch, rows gathered by token
        {"name": "gemm_batch", "op": "gemm", "tokens": 8192, "experts": 32, "picks": 1,
         "skew": 0.0, "n": 2 * INNER, "k": WIDTH, "layout": "nk", "gather": True, "out": "bf16"},
        # its input gradient, with an uneven load over the experts
        {"name": "dgrad_batch", "op": "gemm", "tokens": 8192, "experts": 32, "picks": 1,
         "skew": 0.8, "n": WIDTH, "k": 2 * INNER, "layout": "kn", "gather": False, "out": "bf16"},
        # its weight gradients, in float32 for the optimizer
        {"name": "wgrad_batch", "op": "wgrad", "tokens": 8192, "experts": 32, "picks": 1,
         "skew": 0.4, "n": 2 * INNER, "k": WIDTH, "gather": True, "out": "f32"},
        # the activation of one token's nine expert rows: latency
        {"name": "swiglu_one_token", "op": "swiglu", "rows": 9, "width": INNER, "dtype": "bf16"},
        # its backward pass for the rows of a whole layer's batch
        {"name": "swiglu_backward_batch", "op": "swiglu_backward", "rows": 8192 * 9,
         "width": INNER, "dtype": "bf16"},
        # the gradients of a small layer, every expert's its own tensors: latency
        {"name": "clip_small", "op": "clip", "form": "layer", "experts": 17, "routed": 16,
         "width": 256, "inner": 128, "dtype": "f32"},
        # the gradients of one GPU's experts, as the weight gradients leave them
        {"name": "clip_shard", "op": "clip", "form": "layer", "experts": 33, "routed": 256,
         "width": WIDTH, "inner": INNER, "dtype": "f32"},
    ]


def _spread(rng, lo, hi, step=1):
    """A size between lo and hi, even over its logarithm, a multiple of step."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(max(v, lo), hi)


def draw(rng):
    while True:
        case = _drawn(rng)
        sizes = {v for v in case.values() if type(v) is int}
        sizes |= {2 * case.get("width", 0), case.get("tokens", 0) * (case.get("picks", 0) + 1)}
        if 3072 not in sizes:       # a size of no configuration here
            return case


def _drawn(rng):
    op = rng.choice(["norm", "norm_backward", "gemm", "gemm", "wgrad", "swiglu",
                     "swiglu_backward", "clip"])
    if op in ("norm", "norm_backward"):
        width = _spread(rng, 64, 8192, rng.choice([1, 8, 128]) if rng.random() < 0.9 else 64)
        return {"op": op, "rows": _spread(rng, 1, max(2, min(16384, 8192 * WIDTH // width))),
                "width": width, "stream": rng.choice(["bf16", "f32"]),
                "gate": rng.choice(["none", "channel", "token", "full"])}
    if op in ("gemm", "wgrad"):
        experts = rng.randint(1, 32)
        picks = rng.randint(1, min(8, experts))
        n = _spread(rng, 128, WIDTH, rng.choice([8, 128]))
        k = _spread(rng, 128, WIDTH, rng.choice([8, 128]))
        while (experts + 1) * n * k > LARGEST_WEIGHTS:
            experts, picks = max(1, experts // 2), max(1, picks // 2)
        most = int(LARGEST_FLOPS / (2.0 * n * k * (picks + 1)))
        case = {"op": op, "tokens": _spread(rng, 1, max(2, min(8192, most))), "experts": experts,
                "picks": picks, "skew": rng.choice([0.0, 0.4, 0.8]), "n": n, "k": k,
                "gather": rng.random() < 0.5, "out": rng.choice(["bf16", "f32"])}
        if op == "gemm":
            case["layout"] = rng.choice(["nk", "kn"])
        return case
    if op in ("swiglu", "swiglu_backward"):
        return {"op": op, "rows": _spread(rng, 1, 8192 * 9),
                "width": _spread(rng, 64, INNER, rng.choice([1, 8, 128])),
                "dtype": rng.choice(["bf16", "f32"]) if rng.random() < 0.5 else "bf16"}
    return {"op": "clip", "form": "spread", "count": _spread(rng, 1, 200),
            "most": _spread(rng, 1000, 1 << 23), "sizes": rng.randrange(1 << 30),
            "dtype": rng.choice(["f32", "bf16", "mixed"])}


# ---------------------------------------------------------------------------
# inputs


def _normal(gen, shape, dtype, std=1.0):
    t = torch.empty(shape, dtype=dtype, device=DEV)
    return t.normal_(0.0, std, generator=gen)


def _norm_inputs(case, gen):
    T, H = case["rows"], case["width"]
    sdt, bdt = DTYPES[case["stream"]], torch.bfloat16
    s = {"alpha": 1.0, "beta": 0.5}
    # a residual stream has a few channels much larger than the others
    loud = torch.ones(H, device=DEV)
    loud[torch.randint(0, H, (max(1, H // 100),), device=DEV, generator=gen)] = 10.0
    s["x"] = (_normal(gen, (T, H), torch.float32) * loud).to(sdt)
    s["b"] = _normal(gen, (T, H), bdt, 0.3)
    s["w_pre"] = 1.0 + _normal(gen, (H,), torch.float32, 0.1)
    s["w_post"] = 1.0 + _normal(gen, (H,), torch.float32, 0.1)
    shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[case["gate"]]
    s["gate"] = None
    if shape is not None:
        gate = torch.rand(shape, dtype=torch.float32, device=DEV, generator=gen)
        s["gate"] = gate.to(bdt) if case["gate"] == "full" else gate
    if case["op"] == "norm":
        s["r"], s["h"] = torch.empty_like(s["x"]), torch.empty_like(s["b"])
        return s
    s["r"] = s.pop("x")     # any stored stream will do
    s["dr"] = _normal(gen, (T, H), sdt, 0.1)
    s["dh"] = _normal(gen, (T, H), bdt, 0.1)
    return s


def _groups(case, gen):
    """Rows by expert, as the permutation lays them out: each token's picks
    among the experts (uneven by `skew`), and the shared expert's rows last."""
    T, E, picks = case["tokens"], case["experts"], case["picks"]
    lean = -case["skew"] * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    noise = torch.rand((T, E), device=DEV, generator=gen).clamp_(1e-9, 1.0 - 1e-7)
    idx = (lean - torch.log(-torch.log(noise))).topk(picks, 1).indices
    order = torch.argsort(idx.reshape(-1), stable=True)
    token_of = torch.cat([order // picks, torch.arange(T, device=DEV)]).to(torch.int32)
    counts = torch.bincount(idx.reshape(-1), minlength=E).tolist() + [T]
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    return token_of, torch.tensor(offsets, dtype=torch.int32, device=DEV), counts


def _grouped_inputs(case, gen):
    token_of, offsets, counts = _groups(case, gen)
    R, G, n, k = offsets_rows(case), case["experts"] + 1, case["n"], case["k"]
    s = {"offsets": offsets, "counts": counts, "rows": R,
         "index": token_of if case["gather"] else None}
    src = case["tokens"] if case["gather"] else R
    odt = DTYPES[case["out"]]
    if case["op"] == "gemm":
        s["a"] = _normal(gen, (src, k), torch.bfloat16)
        s["w"] = _normal(gen, (G, n, k) if case["layout"] == "nk" else (G, k, n), torch.bfloat16,
                         0.02)
        s["out"] = torch.empty((R, n), dtype=odt, device=DEV)
    else:
        s["dy"] = _normal(gen, (R, n), torch.bfloat16, 0.1)
        s["x"] = _normal(gen, (src, k), torch.bfloat16)
        s["out"] = torch.empty((G, n, k), dtype=odt, device=DEV)
    return s


def offsets_rows(case):
    return case["tokens"] * (case["picks"] + 1)


def _swiglu_inputs(case, gen):
    R, I, dt = case["rows"], case["width"], DTYPES[case["dtype"]]
    s = {"a": _normal(gen, (R, 2 * I), dt, 1.5)}
    if case["op"] == "swiglu":
        s["h"] = torch.empty((R, I), dtype=dt, device=DEV)
    else:
        s["dh"] = _normal(gen, (R, I), dt, 0.1)
        s["row_gate"] = torch.rand(R, device=DEV, generator=gen)
    return s


def _clip_sizes(case):
    """(numel, dtype) of every gradient."""
    kinds = {"f32": ("f32", "f32"), "bf16": ("bf16", "bf16"), "mixed": ("f32", "bf16")}
    small, large = kinds[case["dtype"]]
    if case["form"] == "layer":
        H, I = case["width"], case["inner"]
        return ([(H, small), (H, small), (case["routed"] * H, small)]
                + [(2 * I * H, large)] * case["experts"] + [(H * I, large)] * case["experts"])
    r = random.Random(case["sizes"])
    sizes = [_spread(r, 1, case["most"]) for _ in range(case["count"])]
    return [(n, r.choice([small, large])) for n in sizes]


def _clip_inputs(case, gen):
    sizes = _clip_sizes(case)
    s = {"max_norm": 1.0, "grads": [], "outs": []}
    at = {}
    for kind in ("f32", "bf16"):    # the gradients lie one behind the other in one buffer a type
        total = sum(n for n, d in sizes if d == kind)
        s["in_" + kind] = _normal(gen, (total,), DTYPES[kind], 0.01)
        s["out_" + kind] = torch.empty(total, dtype=DTYPES[kind], device=DEV)
        at[kind] = 0
    for n, kind in sizes:
        for name, buf in (("grads", "in_"), ("outs", "out_")):
            s[name].append(s[buf + kind][at[kind]:at[kind] + n])
        at[kind] += n
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    if op in ("norm", "norm_backward"):
        s = _norm_inputs(case, gen)
    elif op in ("gemm", "wgrad"):
        s = _grouped_inputs(case, gen)
    elif op in ("swiglu", "swiglu_backward"):
        s = _swiglu_inputs(case, gen)
    else:
        s = _clip_inputs(case, gen)
        if own:     # the list of gradients that a training program keeps
            import fp8_block_scaled_sigmoid_amd as moe
            s["list"] = moe.GradList(s["grads"], s["outs"])
    s["case"] = dict(case)
    return s


# ---------------------------------------------------------------------------
# one pass


def run(state):
    op = state["case"]["op"]
    return (_RUN_OWN if own else _RUN_PLAIN)[op](state)


def _own_norm(s):
    import fp8_block_scaled_sigmoid_amd as moe
    r, h = moe.moe_block_norm(s["x"], s["b"], w_pre=s["w_pre"], w_post=s["w_post"], gate=s["gate"],
                              alpha=s["alpha"], beta=s["beta"], eps=EPS, r=s["r"], h=s["h"])
    return {"r": r, "h": h}


def _own_norm_backward(s):
    import fp8_block_scaled_sigmoid_amd as moe
    dx, db, dw_pre, dw_post, dgate = moe.moe_block_norm_backward(
        s["r"], dr=s["dr"], dh=s["dh"], b=s["b"], w_pre=s["w_pre"], w_post=s["w_post"],
        gate=s["gate"], alpha=s["alpha"], beta=s["beta"], eps=EPS)
    return {"dx": dx, "db": db, "dw_pre": dw_pre, "dw_post": dw_post, "dgate": dgate}


def _own_gemm(s):
    import fp8_block_scaled_sigmoid_amd as moe
    return moe.moe_grouped_gemm_bf16(s["a"], s["w"], s["offsets"], s["rows"],
                                     b_kn=s["case"]["layout"] == "kn", a_row_index=s["index"],
                                     out=s["out"])


def _own_wgrad(s):
    import fp8_block_scaled_sigmoid_amd as moe
    return moe.moe_grouped_wgrad_bf16(s["dy"], s["x"], s["offsets"], s["rows"],
                                      b_row_index=s["index"], out=s["out"])


def _own_swiglu(s):
    import fp8_block_scaled_sigmoid_amd as moe
    return moe.moe_swiglu(s["a"], h=s["h"])


def _own_swiglu_backward(s):
    import fp8_block_scaled_sigmoid_amd as moe
    da, dgate, hg = moe.moe_swiglu_backward(s["a"], s["dh"], row_gate=s["row_gate"])
    return {"da": da, "dgate": dgate, "hg": hg}


def _own_clip(s):
    import fp8_block_scaled_sigmoid_amd as moe
    result = moe.moe_grad_clip(s["list"], s["max_norm"])
    return {"result": result, "f32": s["out_f32"], "bf16": s["out_bf16"]}


def _plain_norm(s):
    x, b = s["x"].float(), s["b"].float()
    n = b * torch.rsqrt((b * b).mean(1, keepdim=True) + EPS) * s["w_post"]
    if s["gate"] is not None:
        n = n * s["gate"].float()
    r = s["alpha"] * x + s["beta"] * n
    h = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * s["w_pre"]
    return {"r": r.to(s["x"].dtype), "h": h.to(s["b"].dtype)}


def _plain_norm_backward(s):
    r, b, dh = s["r"].float(), s["b"].float(), s["dh"].float()
    inv_r = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
    inv_b = torch.rsqrt((b * b).mean(1, keepdim=True) + EPS)
    r_hat, b_hat = r * inv_r, b * inv_b
    dw_pre = (dh * r_hat).sum(0)
    v = dh * s["w_pre"]
    d = s["dr"].float() + inv_r * (v - r_hat * (v * r_hat).mean(1, keepdim=True))
    dn = s["beta"] * d
    dgate = None
    if s["gate"] is not None:
        dgate = dn * (b_hat * s["w_post"])
        dn = dn * s["gate"].float()
        kind = s["case"]["gate"]
        if kind == "channel":
            dgate = dgate.sum(0)
        elif kind == "token":
            dgate = dgate.sum(1, keepdim=True)
        else:
            dgate = dgate.to(s["gate"].dtype)
    dw_post = (dn * b_hat).sum(0)
    v = dn * s["w_post"]
    db = inv_b * (v - b_hat * (v * b_hat).mean(1, keepdim=True))
    return {"dx": (s["alpha"] * d).to(s["r"].dtype), "db": db.to(s["b"].dtype), "dw_pre": dw_pre,
            "dw_post": dw_post, "dgate": dgate}


def _plain_gemm(s):
    a = s["a"] if s["index"] is None else s["a"][s["index"]]
    kn = s["case"]["layout"] == "kn"
    rows = a.split(s["counts"])
    return torch.cat([part.float() @ (s["w"][g].float() if kn else s["w"][g].float().t())
                      for g, part in enumerate(rows) if len(part)]).to(s["out"].dtype)


def _plain_wgrad(s):
    x = s["x"] if s["index"] is None else s["x"][s["index"]]
    return torch.stack([d.float().t() @ part.float()
                        for d, part in zip(s["dy"].split(s["counts"]),
                                           x.split(s["counts"]))]).to(s["out"].dtype)


def _plain_swiglu(s):
    g, u = s["a"].float().chunk(2, 1)
    return (g / (1.0 + torch.exp(-g)) * u).to(s["a"].dtype)


def _plain_swiglu_backward(s):
    dt = s["a"].dtype
    g, u = s["a"].float().chunk(2, 1)
    dh = s["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    silu = g * sig
    h = silu * u
    w = s["row_gate"][:, None]
    da = torch.cat([w * dh * u * (sig + silu * (1.0 - sig)), w * dh * silu], 1)
    return {"da": da.to(dt), "dgate": (h * dh).sum(1), "hg": (w * h).to(dt)}


def _plain_clip(s):
    squares = [g.float().square().sum() for g in s["grads"]]
    norm = torch.stack(squares).sum().sqrt()
    coef = torch.where(torch.isfinite(norm), (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0),
                       torch.ones_like(norm))
    [o.copy_(g.float() * coef) for g, o in zip(s["grads"], s["outs"])]
    return {"result": torch.stack([norm, coef]), "f32": s["out_f32"], "bf16": s["out_bf16"]}


_RUN_OWN = {"norm": _own_norm, "norm_backward": _own_norm_backward, "gemm": _own_gemm,
            "wgrad": _own_wgrad, "swiglu": _own_swiglu, "swiglu_backward": _own_swiglu_backward,
            "clip": _own_clip}
_RUN_PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "gemm": _plain_gemm,
              "wgrad": _plain_wgrad, "swiglu": _plain_swiglu,
              "swiglu_backward": _plain_swiglu_backward, "clip": _plain_clip}


# ---------------------------------------------------------------------------
# what a pass cannot do without


def _experts_hit(case):
    """Experts with rows, on average for an even load (and the shared one)."""
    E = case["experts"]
    return E * (1.0 - (1.0 - case["picks"] / E) ** case["tokens"]) + 1.0


def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        T, H = case["rows"], case["width"]
        sb = 4 if case["stream"] == "f32" else 2
        gate = {"none": 0, "channel": 4 * H, "token": 4 * T, "full": 2 * T * H}[case["gate"]]
        if op == "norm":        # read x, b; write r, h
            return {"bytes": T * H * (2 * sb + 4) + 8 * H + gate, "flops": 10.0 * T * H}
        # read r, dr, b, dh and the gate; write dx, db, the weights' and the gate's gradients
        return {"bytes": T * H * (3 * sb + 6) + 16 * H + 2 * gate, "flops": 30.0 * T * H}
    if op in ("gemm", "wgrad"):
        R, n, k = offsets_rows(case), case["n"], case["k"]
        src = case["tokens"] if case["gather"] else R
        ob = 4 if case["out"] == "f32" else 2
        if op == "gemm":
            moved = 2 * src * k + 2 * _experts_hit(case) * n * k + ob * R * n
        else:
            moved = 2 * R * n + 2 * src * k + ob * (case["experts"] + 1) * n * k
        return {"bytes": moved, "flops": 2.0 * R * n * k}
    if op in ("swiglu", "swiglu_backward"):
        R, I = case["rows"], case["width"]
        b = 4 if case["dtype"] == "f32" else 2
        if op == "swiglu":      # read a, write h
            return {"bytes": 3 * b * R * I, "flops": 8.0 * R * I}
        # read a and dh, write da and the gated h
        return {"bytes": 6 * b * R * I + 8 * R, "flops": 20.0 * R * I}
    sizes = _clip_sizes(case)
    moved = sum(2 * n * (4 if d == "f32" else 2) for n, d in sizes)
    return {"bytes": moved, "flops": 3.0 * sum(n for n, _ in sizes)}


# ---------------------------------------------------------------------------
# the definitions in float64


def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s, case)


def _rms(v, w):
    return v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + EPS) * w


def _boundary(x, b, w_post, gate, alpha, beta):
    y = _rms(b, w_post)
    return alpha * x + beta * (y if gate is None else gate * y)


def _exact_norm(s, case):
    x, b, wp, wq = (s[n].double() for n in ("x", "b", "w_post", "w_pre"))
    gate = None if s["gate"] is None else s["gate"].double()
    r = _boundary(x, b, wp, gate, s["alpha"], s["beta"])
    return {"r": r, "h": _rms(r, wq)}


def _exact_norm_backward(s, case):
    # through automatic differentiation of the forward definition: first the
    # norm that reads r, then the sum that made r (x enters it linearly)
    r, w_pre, b, w_post = (s[n].double().requires_grad_(True)
                           for n in ("r", "w_pre", "b", "w_post"))
    dr, dw_pre = torch.autograd.grad(_rms(r, w_pre), (r, w_pre), s["dh"].double())
    dr = dr + s["dr"].double()
    x = torch.zeros_like(dr, requires_grad=True)
    inputs = [x, b, w_post]
    gate = None
    if s["gate"] is not None:
        gate = s["gate"].double().requires_grad_(True)
        inputs.append(gate)
    got = torch.autograd.grad(_boundary(x, b, w_post, gate, s["alpha"], s["beta"]), inputs, dr)
    return {"dx": got[0], "db": got[1], "dw_pre": dw_pre, "dw_post": got[2],
            "dgate": got[3] if gate is not None else None}


def _bounds(s):
    edge = s["offsets"].tolist()
    return list(zip(edge[:-1], edge[1:]))


def _exact_gemm(s, case):
    out = torch.zeros(s["rows"], case["n"], dtype=torch.float64, device=DEV)
    for g, (lo, hi) in enumerate(_bounds(s)):
        if hi > lo:
            a = s["a"][lo:hi] if s["index"] is None else s["a"][s["index"][lo:hi].long()]
            w = s["w"][g].double()
            out[lo:hi] = torch.mm(a.double(), w if case["layout"] == "kn" else w.t().contiguous())
    return out


def _exact_wgrad(s, case):
    out = torch.zeros(case["experts"] + 1, case["n"], case["k"], dtype=torch.float64, device=DEV)
    for g, (lo, hi) in enumerate(_bounds(s)):
        if hi > lo:
            x = s["x"][lo:hi] if s["index"] is None else s["x"][s["index"][lo:hi].long()]
            out[g] = torch.mm(s["dy"][lo:hi].double().t().contiguous(), x.double())
    return out


def _silu_times(a):
    I = a.shape[1] // 2
    return a[:, :I] * torch.sigmoid(a[:, :I]) * a[:, I:]


def _exact_swiglu(s, case):
    return _silu_times(s["a"].double())


def _exact_swiglu_backward(s, case):
    a = s["a"].double().requires_grad_(True)
    gate = s["row_gate"].double().requires_grad_(True)
    h = gate[:, None] * _silu_times(a)
    da, dgate = torch.autograd.grad(h, (a, gate), s["dh"].double())
    return {"da": da, "dgate": dgate, "hg": h.detach()}


def _exact_clip(s, case):
    total = torch.zeros((), dtype=torch.float64, device=DEV)
    for kind in ("f32", "bf16"):
        for part in s["in_" + kind].split(1 << 26):
            total = total + part.double().pow(2).sum()
    norm = torch.sqrt(total)
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return {"result": torch.stack([norm, coef]), "f32": s["in_f32"].double() * coef,
            "bf16": s["in_bf16"].double() * coef}


_EXACT = {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "gemm": _exact_gemm,
          "wgrad": _exact_wgrad, "swiglu": _exact_swiglu,
          "swiglu_backward": _exact_swiglu_backward, "clip": _exact_clip}
