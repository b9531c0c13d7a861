"""Operators around and of the expert layer: routing, the order of the rows by
expert with the copies into and out of it, and 8-bit floating point products
with a scale for each block of 128.  Cases, plain forms and 64-bit definitions.

Routing: each token chooses k of E experts by its logits, as softmax or sigmoid
scores; a bias per expert may be added for the choice (not for the weight), and
the choice may be limited to the best of several groups of neighbouring experts.
An expert whose logit is -inf is never chosen; where fewer than k can be, the
remaining slots hold expert -1 with weight 0.

Order: pair n * k + j is slot j of token n.  The pairs sorted by expert (stably)
are the rows of the grouped products; offs are the experts' borders, rows the
pair of each row (-1 past the last), pos the row of each pair (-1 for expert -1).

fp8: e4m3 elements; along the contraction 128 elements of a row (activations), or
128 rows by 128 elements (weights), share the fp32 scale max(amax / 448, 2^-126).
"""
import math
import random

import torch


own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
BLOCK = 128


def _ssg():
    import structured_sparse_gemm_amd as ssg
    return ssg


# ----------------------------------------------------------------- cases

def listed():
    return [
        # a decode batch through the router of a mixture of a few dozen experts
        {"name": "route_decode", "op": "route", "dtype": "bf16", "N": 32, "E": 64, "k": 4, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_score": "max", "renorm": True, "scale": 1.0, "pad": 0,
         "grad": False},
        # a training micro-batch, many experts in groups, a bias that balances them, with the gradient
        {"name": "route_train", "op": "route", "dtype": "f32", "N": 8192, "E": 256, "k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "group_score": "top2", "renorm": True, "scale": 2.5, "pad": 100,
         "grad": True},
        # the rows of a decode batch put in the order of their experts
        {"name": "dispatch_decode", "op": "dispatch", "dtype": "bf16", "N": 16, "k": 4, "E": 64, "D": 4096, "pad": 0},
        # those of a prefill chunk, with padding at its end
        {"name": "dispatch_prefill", "op": "dispatch", "dtype": "bf16", "N": 8192, "k": 8, "E": 256, "D": 2048,
         "pad": 77},
        # a decode batch's expert outputs summed back
        {"name": "combine_decode", "op": "combine", "dtype": "f16", "N": 16, "k": 4, "E": 64, "D": 4096, "pad": 0,
         "grad": False},
        # a training micro-batch's, with the gradients of the expert outputs and of the weights
        {"name": "combine_train", "op": "combine", "dtype": "bf16", "N": 4096, "k": 4, "E": 64, "D": 4096, "pad": 50,
         "grad": True},
        # a prefill chunk's activations on their way to an 8-bit product
        {"name": "quantize_tokens", "op": "quantize", "dtype": "bf16", "R": 2048, "K": 8192, "block": 1,
         "transpose": False},
        # a weight of a training step, transposed for the gradient of its input
        {"name": "quantize_weight", "op": "quantize", "dtype": "bf16", "R": 11008, "K": 4096, "block": 128,
         "transpose": True},
        # one token through a square projection
        {"name": "mm_one_token", "op": "mm", "x": "bf16", "out": "bf16", "M": 4096, "K": 4096, "N": 1},
        # a linear layer's training step: output and both gradients, all operands quantised in it
        {"name": "mm_step", "op": "step", "x": "bf16", "out": "bf16", "M": 11008, "K": 4096, "N": 2048},
        # a decode batch of 16 tokens, four experts each, spread over 64 experts
        {"name": "experts_decode", "op": "grouped", "x": "bf16", "out": "bf16", "E": 64, "M": 2048, "K": 4096, "N": 64},
        # a prefill chunk routed over 32 experts
        {"name": "experts_prefill", "op": "grouped", "x": "bf16", "out": "bf16", "E": 32, "M": 4096, "K": 2048,
         "N": 16384},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _inner(rng, lo, hi):
    """A reduction length or row count: mostly what weights have, sometimes any number."""
    v = _log_int(rng, lo, hi)
    return v if rng.random() < 0.25 else max(64, v // 64 * 64) if rng.random() < 0.7 else max(8, v // 8 * 8)


def _draw_route(rng):
    groups = rng.choice([1, 1, 2, 4, 8, 16, 5])
    E = groups * max(2, _log_int(rng, max(2, 8 // groups), 512 // groups))
    top = rng.randint(max(1, groups // 4), groups)
    k = min(rng.choice([1, 2, 4, 6, 8, 8, 10, 16]), top * (E // groups))
    N = _log_int(rng, 1, 16384)
    return {"op": "route", "dtype": rng.choice(["f16", "bf16", "f32", "f32"]), "N": N, "E": E, "k": k,
            "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
            "top_groups": top, "group_score": rng.choice(["max", "top2"]), "renorm": rng.random() < 0.7,
            "scale": rng.choice([1.0, 2.5, 16.0]), "pad": rng.choice([0, 0, N // 9]), "grad": rng.random() < 0.5}


def draw(rng):
    op = rng.choice(["route", "route", "dispatch", "dispatch", "combine", "combine", "quantize", "quantize", "mm", "mm",
                     "step", "grouped", "grouped"])
    if op == "route":
        return _draw_route(rng)
    if op in ("dispatch", "combine"):
        dt = rng.choice(["f16", "bf16", "bf16", "f32"])
        E, k, D = _log_int(rng, 2, 512), rng.choice([1, 2, 4, 6, 8, 8]), _inner(rng, 64, 8192)
        k = min(k, E)
        limit = 60_000_000 if op == "combine" else 120_000_000
        N = min(_log_int(rng, 1, 16384), max(1, limit // (k * D) * 2 // SIZE[dt]))
        case = {"op": op, "dtype": dt, "N": N, "k": k, "E": E, "D": D, "pad": rng.choice([0, 0, N // 9])}
        if op == "combine":
            case["grad"] = rng.random() < 0.5
        return case
    if op == "quantize":
        R = _log_int(rng, 1, 12000)
        return {"op": op, "dtype": rng.choice(["f16", "bf16", "f32"]), "R": R,
                "K": _inner(rng, 64, min(28672, max(128, 40_000_000 // R))), "block": rng.choice([1, 128]),
                "transpose": rng.random() < 0.4}
    M, K = _inner(rng, 64, 16384), _inner(rng, 64, 12288)
    N = _log_int(rng, 1, 8192) if rng.random() < 0.6 else rng.randint(1, 80)
    x = rng.choice(["f16", "bf16"])
    out = rng.choice(["f32", x])
    if op in ("mm", "step"):
        return {"op": op, "x": x, "out": out, "M": M, "K": K,
                "N": min(N, max(1, (130_000_000_000 if op == "mm" else 80_000_000_000) // (M * K)))}
    E = _log_int(rng, 1, 96)
    while E * M * K > 400_000_000:                      # what the experts of one layer hold
        M, K = max(33, M // 2), max(40, K // 2)
    return {"op": op, "x": x, "out": out, "E": E, "M": M, "K": K, "N": min(N, max(1, 100_000_000_000 // (M * K)))}


# ----------------------------------------------------------------- inputs

def _sizes(E, N, seed):
    """Rows per expert as a router leaves them: skewed, some experts empty."""
    r = random.Random(1_000_003 * seed + 7 * E + N)
    weight = [math.exp(0.7 * r.gauss(0.0, 1.0)) for _ in range(E)]
    count = [0] * E
    for e in r.choices(range(E), weight, k=N):
        count[e] += 1
    return count


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, R, K, dtype):
    """Normal values with a spread of channel magnitudes."""
    x = _randn(gen, R, K)
    return x.mul_(_randn(gen, K).mul_(0.5).exp_()).to(dtype)


def _logits(gen, N, E, pad):
    """Router logits: some experts are liked better; the last `pad` tokens are padding."""
    l = _randn(gen, N, E).add_(_randn(gen, E).mul_(0.7))
    if pad:
        l[N - pad:] = -math.inf
    return l


def _choices(gen, case):
    """[N, k] distinct experts of each token, -1 for padding."""
    N, pad = case["N"], case["pad"]
    e = _logits(gen, N, case["E"], 0).topk(case["k"], dim=1).indices.to(torch.int32)
    if pad:
        e[N - pad:] = -1
    return e


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7919 * int(seed) + 13)
    s, op = dict(case), case["op"]
    if op == "route":
        N, E = case["N"], case["E"]
        s["logits"] = _logits(gen, N, E, case["pad"]).to(DTYPES[case["dtype"]])
        s["b"] = _randn(gen, E).mul_(0.1) if case["bias"] else None
        if case["grad"]:
            s["dw"] = _randn(gen, N, case["k"])
        return s
    if op in ("dispatch", "combine"):
        dt = DTYPES[case["dtype"]]
        s["experts"] = _choices(gen, case)
        N, k, D = case["N"], case["k"], case["D"]
        if op == "dispatch":
            s["X"] = _activations(gen, N, D, dt)
            return s
        offs, s["rows"], s["pos"] = _order(s["experts"], case["E"])
        # what the expert products hand over: zeros in the rows of nobody
        s["Y"] = _randn(gen, N * k, D).masked_fill_(s["rows"][:, None] < 0, 0.0).to(dt)
        s["w"] = torch.softmax(_randn(gen, N, k), dim=1).masked_fill_(s["experts"] < 0, 0.0)
        if case["grad"]:
            s["dO"] = _randn(gen, N, D).to(dt)
        return s
    if op == "quantize":
        R, K, dt = case["R"], case["K"], DTYPES[case["dtype"]]
        s["A"] = _activations(gen, R, K, dt) if case["block"] == 1 else _randn(gen, R, K).mul_(0.02).to(dt)
        return s
    M, N, K, xt = case["M"], case["N"], case["K"], DTYPES[case["x"]]
    s["X"] = _activations(gen, N, K, xt)
    if op == "step":
        s["W"] = _randn(gen, M, K).mul_(0.02).to(xt)
        s["dY"] = _randn(gen, N, M).to(xt)
        return s
    E = case.get("E", 1)
    parts = [_quantize(_randn(gen, M, K).mul_(0.02), 128) for _ in range(E)]
    if op == "mm":
        s["W"], s["scales"] = parts[0][0].to(torch.float8_e4m3fn), parts[0][1]
        return s
    s["W"] = torch.stack([p[0].to(torch.float8_e4m3fn) for p in parts])
    s["scales"] = torch.stack([p[1] for p in parts])
    sizes = _sizes(E, N, int(seed))
    offs = [0]
    for n in sizes:
        offs.append(offs[-1] + n)
    s["offs"] = torch.tensor(offs, dtype=torch.int32, device="cuda")
    # the plain form's table of rows: row i of expert e, or N where there is none
    at = torch.arange(max(max(sizes), 1), device="cuda")
    counts = s["offs"][1:] - s["offs"][:-1]
    s["table"] = torch.where(at[None, :] < counts[:, None], at[None, :] + s["offs"][:-1, None], N)
    return s


# ----------------------------------------------------------------- plain forms

def _scores(l, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    top = l.amax(dim=1, keepdim=True)
    e = torch.exp(l - torch.where(top == -math.inf, torch.zeros_like(top), top))
    return e / e.sum(dim=1, keepdim=True).clamp_min(torch.finfo(l.dtype).tiny)


def _route(s):
    """(weights, experts): the choice is made in 64 bits, the weights in 32."""
    l, N, E, k, G = s["logits"], s["N"], s["E"], s["k"], s["groups"]
    gone = l == -math.inf
    s64 = _scores(l.double(), s["score"])
    c = l.double() if s["b"] is None else s64 + s["b"].double()
    c = c.masked_fill(gone, -math.inf)
    if G > 1:
        by = c if s["group_score"] == "max" else (s64 if s["b"] is None else c).masked_fill(gone, -math.inf)
        best = torch.sort(by.view(N, G, E // G), dim=2, descending=True).values
        score = best[:, :, 0]
        if s["group_score"] == "top2" and E // G > 1:
            score = score + best[:, :, 1].masked_fill(best[:, :, 1] == -math.inf, 0.0)
        rank = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        keep = torch.zeros(N, G, dtype=torch.bool, device=l.device).scatter_(1, rank, True)
        c = c.masked_fill(~keep.repeat_interleave(E // G, dim=1), -math.inf)
    value, index = torch.sort(c, dim=1, descending=True, stable=True)
    value, index = value[:, :k], index[:, :k]
    none = value == -math.inf
    w = _scores(l.float(), s["score"]).gather(1, index).masked_fill(none, 0.0)
    if s["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp_min(torch.finfo(torch.float32).tiny)
    return w * s["scale"], index.to(torch.int32).masked_fill(none, -1)


def _route_backward(s, experts):
    l = s["logits"].float()
    p, none = _scores(l, s["score"]), experts < 0
    at = experts.long().clamp_min(0)
    g = (s["dw"] * s["scale"]).masked_fill(none, 0.0)
    pj = p.gather(1, at).masked_fill(none, 0.0)
    if s["renorm"]:
        total = pj.sum(dim=1, keepdim=True).clamp_min(torch.finfo(torch.float32).tiny)
        g = (g - (g * pj).sum(dim=1, keepdim=True) / total) / total
    g = torch.zeros_like(l).scatter_add_(1, at, g.masked_fill(none, 0.0))
    d = p * (1.0 - p) * g if s["score"] == "sigmoid" else p * (g - (g * p).sum(dim=1, keepdim=True))
    return d.to(s["logits"].dtype)


def _order(experts, E):
    """(offs, rows, pos) of [N, k] experts."""
    flat = experts.flatten().long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    there = key[order] < E
    offs = torch.searchsorted(key[order].contiguous(), torch.arange(E + 1, device=flat.device))
    pos = torch.empty_like(flat).scatter_(0, order, torch.arange(flat.numel(), device=flat.device))
    return (offs.to(torch.int32), torch.where(there, order, -1).to(torch.int32),
            torch.where(key < E, pos, -1).to(torch.int32).view_as(experts))


def _round_e4m3(q):
    """Nearest e4m3 value of 64-bit q, ties to even: steps of 2^(exponent - 3),
    2^-9 at least; at most 448."""
    q = q.clamp(-448.0, 448.0)
    step = torch.exp2((torch.frexp(q).exponent - 4).clamp_min(-9).double())
    return torch.round(q / step) * step


def _quantize(a, block):
    """(elements as fp32 values, scales) of [R, K]."""
    R, K = a.shape
    nb, rb = -(-K // BLOCK), -(-R // block)
    v = torch.nn.functional.pad(a.float(), (0, nb * BLOCK - K, 0, rb * block - R))
    v = v.view(rb, block, nb, BLOCK)
    scale = (v.abs().amax(dim=(1, 3)).double() / 448.0).float().clamp_min(2.0 ** -126)
    q = _round_e4m3(v.double() / scale.double()[:, None, :, None])
    return q.view(rb * block, nb * BLOCK)[:R, :K].float(), scale


def _dequantize(e, scale, block):
    """fp32 values of [R, K] elements."""
    R, K = e.shape
    s = scale if block == 1 else scale.repeat_interleave(block, dim=0)[:R]
    return e.float() * s.repeat_interleave(BLOCK, dim=1)[:, :K]


def _through8(a, block):
    return _dequantize(*_quantize(a, block), block)


def _by_expert(x, table):
    """[E, cap, C] fp32: the rows of each expert, zeros where it has fewer than cap."""
    return torch.cat([x.float(), x.new_zeros(1, x.shape[1], dtype=torch.float32)])[table]


def _run_own(s):
    ssg, op = _ssg(), s["op"]
    if op == "route":
        w, e = ssg.route(s["logits"], s["k"], score=s["score"], bias=s["b"], groups=s["groups"],
                         top_groups=s["top_groups"], group_score=s["group_score"], renorm=s["renorm"], scale=s["scale"])
        out = {"weights": w, "experts": e}
        if s["grad"]:
            out["dlogits"] = ssg.route_backward(s["dw"], s["logits"], e, score=s["score"], renorm=s["renorm"],
                                                scale=s["scale"])
        return out
    if op == "dispatch":
        offs, rows, pos = ssg.expert_order(s["experts"], s["E"])
        return {"offs": offs, "rows": rows, "pos": pos, "X": ssg.expert_gather(s["X"], pos, rows)}
    if op == "combine":
        out = {"O": ssg.expert_combine(s["Y"], s["pos"], s["w"])}
        if s["grad"]:
            out["dY"], out["dw"] = ssg.expert_combine_backward(s["dO"], s["Y"], s["pos"], s["rows"], s["w"])
        return out
    if op == "quantize":
        e, scales = ssg.fp8_quantize(s["A"], block=s["block"], transpose=s["transpose"])
        return {"values": ssg.fp8_dequantize(e, scales, dtype=s["A"].dtype), "scales": scales}
    out = DTYPES[s["out"]]
    if op == "mm":
        return ssg.mm_fp8(s["X"], s["W"], s["scales"], out_dtype=out)
    if op == "grouped":
        return ssg.grouped_mm_fp8(s["X"], s["W"], s["scales"], s["offs"], out_dtype=out)
    w, ws = ssg.fp8_quantize(s["W"], block=128)
    wt, wts = ssg.fp8_quantize(s["W"], block=128, transpose=True)
    xt, xts = ssg.fp8_quantize(s["X"], transpose=True)
    dyt, dyts = ssg.fp8_quantize(s["dY"], transpose=True)
    return {"Y": ssg.mm_fp8(s["X"], w, ws, out_dtype=out), "dX": ssg.mm_fp8(s["dY"], wt, wts, out_dtype=out),
            "dW": ssg.mm_fp8(dyt, xt, xts, xscales=dyts, out_dtype=torch.float32)}


def run(state):
    if own:
        return _run_own(state)
    s, op = state, state["op"]
    if op == "route":
        w, e = _route(s)
        out = {"weights": w, "experts": e}
        if s["grad"]:
            out["dlogits"] = _route_backward(s, e)
        return out
    if op == "dispatch":
        offs, rows, pos = _order(s["experts"], s["E"])
        x = s["X"][rows.long().clamp_min(0) // s["k"]]
        return {"offs": offs, "rows": rows, "pos": pos, "X": x.masked_fill_(rows[:, None] < 0, 0.0)}
    if op == "combine":
        N, k, D, dt = s["N"], s["k"], s["D"], s["Y"].dtype
        gone, at = s["pos"] < 0, s["pos"].long().clamp_min(0)
        w = s["w"].masked_fill(gone, 0.0)
        y = s["Y"][at.flatten()].view(N, k, D).float()
        out = {"O": (w[:, :, None] * y).sum(dim=1).to(dt)}
        if s["grad"]:
            pair = s["rows"].long().clamp_min(0)
            d = w.flatten()[pair, None] * s["dO"][pair // k].float()
            out["dY"] = d.masked_fill_(s["rows"][:, None] < 0, 0.0).to(dt)
            out["dw"] = (y * s["dO"].float()[:, None, :]).sum(dim=2).masked_fill(gone, 0.0)
        return out
    if op == "quantize":
        A = s["A"].t().contiguous() if s["transpose"] else s["A"]
        e, scale = _quantize(A, s["block"])
        return {"values": _dequantize(e, scale, s["block"]).to(A.dtype), "scales": scale}
    out = DTYPES[s["out"]]
    if op == "mm":
        return (_through8(s["X"], 1) @ _dequantize(s["W"], s["scales"], 128).t()).to(out)
    if op == "grouped":
        W = torch.stack([_dequantize(w, c, 128) for w, c in zip(s["W"], s["scales"])])
        y = torch.bmm(_by_expert(_through8(s["X"], 1), s["table"]), W.transpose(1, 2).contiguous())
        Y = y.new_zeros(s["N"] + 1, s["M"])
        Y[s["table"].flatten()] = y.flatten(0, 1)
        return Y[:s["N"]].to(out)
    W, X, dY = _through8(s["W"], 128), s["X"], s["dY"]
    dW = _through8(dY.t().contiguous(), 1) @ _through8(X.t().contiguous(), 1).t()
    return {"Y": (_through8(X, 1) @ W.t()).to(out), "dX": (_through8(dY, 1) @ W).to(out), "dW": dW}


# ----------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "route":
        n, pairs = case["N"] * case["E"] * SIZE[case["dtype"]], case["N"] * case["k"]
        g = case["grad"]
        return {"bytes": (2 if g else 1) * n + (12 if g else 8) * pairs + (4 * case["E"] if case["bias"] else 0),
                "flops": (12 if g else 6) * case["N"] * case["E"]}
    if op in ("dispatch", "combine"):
        P, d = case["N"] * case["k"], case["D"] * SIZE[case["dtype"]]
        if op == "dispatch":
            return {"bytes": 12 * P + 4 * (case["E"] + 1) + case["N"] * d + P * d, "flops": P}
        if not case["grad"]:
            return {"bytes": 8 * P + P * d + case["N"] * d, "flops": 2 * P * case["D"]}
        return {"bytes": 16 * P + 2 * P * d + 2 * case["N"] * d, "flops": 5 * P * case["D"]}
    if op == "quantize":
        # the matrix in, elements and scales out and in again, the values out
        n, b = case["R"] * case["K"], case["block"]
        return {"bytes": 2 * n * SIZE[case["dtype"]] + 2 * n + 8 * n // (b * BLOCK), "flops": 4 * n}
    M, N, K = case["M"], case["N"], case["K"]
    x, o = SIZE[case["x"]], SIZE[case["out"]]
    if op == "mm":
        return {"bytes": M * K + N * K * x + N * M * o + 4 * M * K // (BLOCK * BLOCK), "flops": 2 * M * N * K}
    if op == "grouped":
        busy = min(case["E"], N)                       # at most so many experts have rows
        return {"bytes": busy * (M * K + 4 * M * K // (BLOCK * BLOCK)) + N * K * x + N * M * o, "flops": 2 * M * N * K}
    return {"bytes": (M * K + N * K + N * M) * x + (N * M + N * K) * o + 4 * M * K, "flops": 6 * M * N * K}


# ----------------------------------------------------------------- the definition in 64 bits

def _exact_route(case, s):
    """Token by token on the host, experts chosen one after the other."""
    N, E, k, G = case["N"], case["E"], case["k"], case["groups"]
    S = E // G
    l = s["logits"].double().cpu()
    bias = s["b"].double().cpu().tolist() if s["b"] is not None else None
    if case["score"] == "sigmoid":
        score = torch.special.expit(l)
    else:
        score = torch.softmax(l, dim=1)
    weights, experts = torch.zeros(N, k, dtype=torch.float64), torch.full((N, k), -1, dtype=torch.int32)
    d = torch.zeros(N, E, dtype=torch.float64)
    g_all = s["dw"].double().cpu() * case["scale"] if case["grad"] else None
    for n in range(N):
        row, sc = l[n].tolist(), score[n].tolist()
        live = [e for e in range(E) if row[e] != -math.inf]
        if not live:
            continue
        c = {e: sc[e] + bias[e] if bias else row[e] for e in live}
        if G > 1:
            val = c if case["group_score"] == "max" or bias else {e: sc[e] for e in live}
            most = 1 if case["group_score"] == "max" else 2
            total = []
            for g in range(G):
                v = sorted((val[e] for e in range(g * S, g * S + S) if e in val), reverse=True)[:most]
                total.append(math.fsum(v) if v else -math.inf)
            stay = set(sorted(range(G), key=lambda g: (-total[g], g))[:case["top_groups"]])
            live = [e for e in live if e // S in stay]
        pick = sorted(live, key=lambda e: (-c[e], e))[:k]
        sj = torch.tensor([sc[e] for e in pick], dtype=torch.float64)
        total = sj.sum()
        m = len(pick)
        if m:
            weights[n, :m] = (sj / total if case["renorm"] else sj) * case["scale"]
            experts[n, :m] = torch.tensor(pick, dtype=torch.int32)
        if case["grad"] and m:
            g = g_all[n, :m]
            if case["renorm"]:
                g = (g - (g * sj).sum() / total) / total
            if case["score"] == "sigmoid":
                d[n, pick] = g * sj * (1.0 - sj)
            else:
                d[n] = -score[n] * (g * sj).sum()
                d[n, pick] += sj * g
    out = {"weights": weights.cuda(), "experts": experts.cuda()}
    if case["grad"]:
        out["dlogits"] = d.cuda()
    return out


def _exact_order(experts, E):
    """Each pair's row: the pairs of smaller experts, and those before it of its own."""
    flat = experts.flatten().tolist()
    start = [0] * (E + 1)
    for e in flat:
        if 0 <= e < E:
            start[e + 1] += 1
    for e in range(E):
        start[e + 1] += start[e]
    offs, at = list(start), list(start)
    rows, pos = [-1] * len(flat), []
    for i, e in enumerate(flat):
        p = -1
        if 0 <= e < E:
            p = at[e]
            at[e] += 1
            rows[p] = i
        pos.append(p)
    return offs, rows, pos


def _exact8(a, block):
    """Values of the 8-bit form of [R, K] in 64 bits, and its scales."""
    R, K = a.shape
    a = a.double()
    out = torch.zeros_like(a)
    rb, nb = -(-R // block), -(-K // BLOCK)
    scales = torch.zeros(rb, nb, dtype=torch.float64, device=a.device)
    for b in range(nb):
        cols = slice(b * BLOCK, min(K, (b + 1) * BLOCK))
        top = a[:, cols].abs().max(dim=1).values
        if block > 1:
            top = torch.nn.functional.pad(top, (0, rb * block - R)).view(rb, block).max(dim=1).values
        sc = torch.maximum(top / 448.0, torch.full_like(top, 2.0 ** -126)).float().double()   # held in fp32
        scales[:, b] = sc
        q = a[:, cols] / sc.repeat_interleave(block)[:R, None]
        mag = q.abs()
        e = torch.floor(torch.log2(mag.clamp_min(2.0 ** -6)))
        e = torch.where(mag >= torch.exp2(e + 1), e + 1, torch.where(mag < torch.exp2(e), e - 1, e)).clamp_min(-6.0)
        unit = torch.exp2(e - 3)
        low = torch.floor(mag / unit)
        rest = mag / unit - low
        up = (rest > 0.5) | ((rest == 0.5) & (low % 2 == 1))
        out[:, cols] = torch.sign(q) * ((low + up) * unit).clamp_max(448.0) * sc.repeat_interleave(block)[:R, None]
    return out, scales


def _exact_values(e, scales):
    """64-bit values of [M, K] elements with a scale for each 128 x 128."""
    rows = torch.arange(e.shape[0], device=e.device) // BLOCK
    cols = torch.arange(e.shape[1], device=e.device) // BLOCK
    return e.float().double() * scales.double()[rows][:, cols]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "route":
        return _exact_route(case, s)
    if op == "dispatch":
        offs, rows, pos = _exact_order(s["experts"], case["E"])
        r = torch.tensor(rows, dtype=torch.int64, device="cuda")
        X = torch.zeros(len(rows), case["D"], dtype=torch.float64, device="cuda")
        X[r >= 0] = s["X"].double()[r[r >= 0] // case["k"]]
        return {"offs": torch.tensor(offs, dtype=torch.int32, device="cuda"), "rows": r.to(torch.int32),
                "pos": torch.tensor(pos, dtype=torch.int32, device="cuda").view(case["N"], case["k"]), "X": X}
    if op == "combine":
        N, k = case["N"], case["k"]
        out = {"O": torch.zeros(N, case["D"], dtype=torch.float64, device="cuda")}
        if case["grad"]:
            out["dY"] = torch.zeros(N * k, case["D"], dtype=torch.float64, device="cuda")
            out["dw"] = torch.zeros(N, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            n = (s["pos"][:, j] >= 0).nonzero().flatten()
            p, w = s["pos"][n, j].long(), s["w"][n, j].double()[:, None]
            y = s["Y"][p].double()
            out["O"][n] += w * y
            if case["grad"]:
                out["dY"][p] = w * s["dO"][n].double()
                out["dw"][n, j] = (y * s["dO"][n].double()).sum(dim=1)
        return out
    if op == "quantize":
        v, scales = _exact8(s["A"].t() if case["transpose"] else s["A"], case["block"])
        return {"values": v, "scales": scales}
    if op == "mm":
        return _exact8(s["X"], 1)[0] @ _exact_values(s["W"], s["scales"]).t()
    if op == "step":
        X, dY, W = s["X"], s["dY"], _exact8(s["W"], 128)[0]
        return {"Y": _exact8(X, 1)[0] @ W.t(), "dX": _exact8(dY, 1)[0] @ W,
                "dW": _exact8(dY.t(), 1)[0] @ _exact8(X.t(), 1)[0].t()}
    Y = torch.zeros(case["N"], case["M"], dtype=torch.float64, device="cuda")
    ends, X = s["offs"].tolist(), _exact8(s["X"], 1)[0]
    for e, (a, b) in enumerate(zip(ends[:-1], ends[1:])):
        if b > a:
            Y[a:b] = X[a:b] @ _exact_values(s["W"][e], s["scales"][e]).t()
    return Y
