"""Operators of the 4-bit microscaled weights and the expert-grouped products:
cases, plain forms and 64-bit definitions.

Format (mx4): along K, blocks of 32 elements share a power-of-two scale
2^(s - 127) stored as the byte s; each element is an E2M1 float (sign, two
exponent bits, one fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two per byte,
the even element in the low nibble.  A matrix [R, K] is a byte tensor
[R, 16 * ceil(K / 32)] of elements (zeros past K) and one of scales
[R, ceil(K / 32)].

Expert-grouped: the rows of the activations are sorted by expert, and rows
offs[e] .. offs[e + 1] - 1 meet the weight of expert e.
"""
import math
import random

import torch


own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 32


def _ssg():
    import structured_sparse_gemm_amd as ssg
    return ssg


# ----------------------------------------------------------------- cases

def listed():
    return [
        # activations of a decode step on their way to a 4-bit product, and back for an error estimate
        {"name": "quantize_decode", "op": "quantize", "dtype": "f16", "R": 16, "K": 4096},
        # a 7B-class FFN weight quantised when a checkpoint is loaded
        {"name": "quantize_weight", "op": "quantize", "dtype": "bf16", "R": 11008, "K": 4096},
        # one token through a square projection
        {"name": "mm_one_token", "op": "mm", "x": "bf16", "out": "bf16", "M": 4096, "K": 4096, "N": 1},
        # a decode batch through the 7B-class FFN weight
        {"name": "mm_decode", "op": "mm", "x": "f16", "out": "f32", "M": 11008, "K": 4096, "N": 16},
        # a prefill chunk with 16-bit activations kept for accuracy
        {"name": "mm_prefill_a16", "op": "mm", "x": "bf16", "out": "bf16", "M": 8192, "K": 8192, "N": 1000},
        # a prefill chunk through the 70B-class FFN weight, activations quantised on the way in
        {"name": "mm_prefill_a4", "op": "mm", "x": "mx4", "out": "bf16", "M": 28672, "K": 8192, "N": 2048},
        # a decode batch of 16 tokens, four experts each, spread over 64 experts
        {"name": "experts_mx4_decode", "op": "grouped_mx4", "x": "bf16", "out": "bf16", "E": 64, "M": 2048, "K": 4096,
         "N": 64},
        # a prefill chunk routed over 32 experts, activations quantised on the way in
        {"name": "experts_mx4_prefill", "op": "grouped_mx4", "x": "mx4", "out": "bf16", "E": 32, "M": 4096, "K": 2048,
         "N": 16384},
        # 16-bit experts: one token that goes to two of eight experts
        {"name": "experts_one_token", "op": "grouped", "x": "f16", "out": "f16", "E": 8, "M": 4096, "K": 4096, "N": 2},
        # 16-bit experts, a prefill chunk
        {"name": "experts_prefill", "op": "grouped", "x": "bf16", "out": "bf16", "E": 8, "M": 4096, "K": 4096,
         "N": 8192},
        # gradients of the expert weights and of their inputs, a training micro-batch
        {"name": "experts_grads", "op": "grads", "x": "bf16", "out": "bf16", "E": 8, "M": 4096, "K": 2048, "N": 8192},
        # the same with many small experts, ragged sizes, gradients accumulated by the optimiser in fp32
        {"name": "experts_grads_ragged", "op": "grads", "x": "f16", "out": "f32", "E": 40, "M": 1000, "K": 1416,
         "N": 2047},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _inner(rng, lo, hi):
    """A reduction length or row count: mostly what weights have, sometimes any number."""
    v = _log_int(rng, lo, hi)
    return v if rng.random() < 0.25 else max(32, v // 32 * 32) if rng.random() < 0.7 else max(8, v // 8 * 8)


def draw(rng):
    op = rng.choice(["quantize", "mm", "mm", "grouped_mx4", "grouped_mx4", "grouped", "grouped", "grads", "grads"])
    if op == "quantize":
        R = _log_int(rng, 1, 12000)
        return {"op": op, "dtype": rng.choice(["f16", "bf16", "f32"]), "R": R,
                "K": _inner(rng, 64, min(28672, 48_000_000 // R))}
    M, K = _inner(rng, 64, 16384), _inner(rng, 64, 12288)
    N = _log_int(rng, 1, 8192) if rng.random() < 0.6 else rng.randint(1, 80)
    if op == "mm":
        x = rng.choice(["f16", "bf16", "mx4"])
        return {"op": op, "x": x, "out": rng.choice(["f32", "bf16"] if x == "mx4" else ["f32", x]), "M": M, "K": K,
                "N": min(N, max(1, 200_000_000_000 // (M * K)))}
    E = _log_int(rng, 1, 96)
    while E * M * K > 400_000_000:                      # what the experts of one layer hold
        M, K = max(33, M // 2), max(40, K // 2)
    N = min(N, max(1, 100_000_000_000 // (M * K)))
    if op == "grouped_mx4":
        x = rng.choice(["f16", "bf16", "mx4"])
        return {"op": op, "x": x, "out": rng.choice(["f32", "bf16"] if x == "mx4" else ["f32", x]), "E": E, "M": M,
                "K": K, "N": N}
    x = rng.choice(["f16", "bf16"])
    return {"op": op, "x": x, "out": rng.choice(["f32", x]), "E": E, "M": M, "K": K, "N": N}


# ----------------------------------------------------------------- inputs

def _sizes(E, N, seed):
    """Rows per expert as a router leaves them: skewed, some experts empty."""
    r = random.Random(1_000_003 * seed + 7 * E + N)
    weight = [math.exp(0.7 * r.gauss(0.0, 1.0)) for _ in range(E)]
    count = [0] * E
    for e in r.choices(range(E), weight, k=N):
        count[e] += 1
    return count


def _activations(gen, R, K, dtype):
    """Normal values with a spread of channel magnitudes."""
    x = torch.randn(R, K, generator=gen, device="cuda", dtype=torch.float32)
    channel = torch.randn(K, generator=gen, device="cuda", dtype=torch.float32).mul_(0.5).exp_()
    return x.mul_(channel).to(dtype)


def _weights(gen, shape, dtype):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(0.02).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7919 * int(seed) + 13)
    s = dict(case)
    if case["op"] == "quantize":
        s["A"] = _activations(gen, case["R"], case["K"], DTYPES[case["dtype"]])
        return s
    xt = DTYPES[case["x"] if case["x"] != "mx4" else "bf16"]
    s["X"] = _activations(gen, case["N"], case["K"], xt)
    if case["op"] == "mm":
        s["W"], s["scales"] = _quantize(_weights(gen, (case["M"], case["K"]), torch.float32))
        return s
    sizes = _sizes(case["E"], case["N"], int(seed))
    s["sizes"] = sizes
    offs = [0]
    for n in sizes:
        offs.append(offs[-1] + n)
    s["offs"] = torch.tensor(offs, dtype=torch.int32, device="cuda")
    # the plain form's table of rows: row i of expert e, or N where there is none
    cap = max(max(sizes), 1)
    at = torch.arange(cap, device="cuda")
    counts = s["offs"][1:] - s["offs"][:-1]
    s["rows"] = torch.where(at[None, :] < counts[:, None], at[None, :] + s["offs"][:-1, None], case["N"])
    if case["op"] == "grouped_mx4":
        parts = [_quantize(_weights(gen, (case["M"], case["K"]), torch.float32)) for _ in range(case["E"])]
        s["W"], s["scales"] = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
    else:
        s["W"] = _weights(gen, (case["E"], case["M"], case["K"]), xt)
    if case["op"] == "grads":
        s["dY"] = torch.randn(case["N"], case["M"], generator=gen, device="cuda", dtype=torch.float32).to(xt)
    return s


# ----------------------------------------------------------------- plain forms

def _padded(a, cols):
    return a if a.shape[1] == cols else torch.nn.functional.pad(a, (0, cols - a.shape[1]))


def _quantize(a):
    """(elements, scales) of a [R, K] matrix: uint8 [R, 16 nb] and uint8 [R, nb]."""
    R, K = a.shape
    nb = -(-K // BLOCK)
    v = _padded(a.float(), nb * BLOCK).view(R, nb, BLOCK)
    top = v.abs().amax(dim=2)
    # floor(log2 top) from the exponent field (top is 0 or normal here)
    s = ((top.view(torch.int32) >> 23) - 2).clamp_(min=0)
    # 2^(127 - s), exact, as two factors: s may be 253
    half = (127 - s) >> 1
    up = _pow2(half)[:, :, None], _pow2(127 - s - half)[:, :, None]
    m = v.abs() * up[0] * up[1]
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = (code.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)).view(R, nb * BLOCK)
    return code[:, 0::2] | (code[:, 1::2] << 4), s.to(torch.uint8)


def _pow2(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _dequantize(elements, scales, K):
    """fp32 values of the last two dimensions [R, 16 nb] and [R, nb]."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=elements.device)
    code = torch.stack([elements & 15, elements >> 4], dim=-1).flatten(-2)
    s = scales.to(torch.int32)
    f = torch.where(s == 0, torch.full_like(s, 1 << 22), s << 23).view(torch.float32)
    v = table[code.to(torch.int32)].unflatten(-1, (-1, BLOCK)) * f[..., None]
    return v.flatten(-2)[..., :K]


def _by_expert(x, rows):
    """[E, cap, C] fp32: the rows of each expert, zeros where it has fewer than cap."""
    return torch.cat([x.float(), x.new_zeros(1, x.shape[1], dtype=torch.float32)])[rows]


def _back(y, rows, N):
    out = y.new_zeros(N + 1, y.shape[2])
    out[rows.flatten()] = y.flatten(0, 1)
    return out[:N]


def run(state):
    op = state["op"]
    out = DTYPES[state["out"]] if "out" in state else None
    if own:
        ssg = _ssg()
        if op == "quantize":
            vals, scales = ssg.mx4_quantize(state["A"])
            return {"values": ssg.mx4_dequantize(vals, scales, state["K"], dtype=state["A"].dtype),
                    "scales": scales.to(torch.int32)}
        if op in ("mm", "grouped_mx4"):
            X, xs = state["X"], None
            if state["x"] == "mx4":
                X, xs = ssg.mx4_quantize(X)
            if op == "mm":
                return ssg.mm_mx4(X, state["W"], state["scales"], xscales=xs, out_dtype=out)
            return ssg.grouped_mm_mx4(X, state["W"], state["scales"], state["offs"], xscales=xs, out_dtype=out)
        if op == "grouped":
            return ssg.grouped_mm(state["X"], state["W"], state["offs"], out_dtype=out)
        return {"dX": ssg.grouped_mm_dx(state["dY"], state["W"], state["offs"], out_dtype=out),
                "dW": ssg.grouped_mm_dw(state["dY"], state["X"], state["offs"], out_dtype=out)}
    if op == "quantize":
        vals, scales = _quantize(state["A"])
        return {"values": _dequantize(vals, scales, state["K"]).to(state["A"].dtype), "scales": scales.to(torch.int32)}
    X = state["X"]
    if state["x"] == "mx4":
        X = _dequantize(*_quantize(X), state["K"])
    if op == "mm":
        return (X.float() @ _dequantize(state["W"], state["scales"], state["K"]).t()).to(out)
    rows, N = state["rows"], state["N"]
    if op == "grads":
        dy = _by_expert(state["dY"], rows)
        return {"dX": _back(torch.bmm(dy, state["W"].float()), rows, N).to(out),
                "dW": torch.bmm(dy.transpose(1, 2).contiguous(), _by_expert(X, rows)).to(out)}
    W = _dequantize(state["W"], state["scales"], state["K"]) if op == "grouped_mx4" else state["W"].float()
    return _back(torch.bmm(_by_expert(X, rows), W.transpose(1, 2)), rows, N).to(out)


# ----------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, K = case["op"], case["K"]
    nb = -(-K // BLOCK)
    size = {"f16": 2, "bf16": 2, "f32": 4}
    if op == "quantize":
        # the matrix in, elements and scales out and in again, the values out
        n = case["R"] * K
        return {"bytes": 2 * n * size[case["dtype"]] + 2 * case["R"] * nb * 17, "flops": 4 * n}
    M, N, E = case["M"], case["N"], case.get("E", 1)
    busy = min(E, N)                                   # at most so many experts have rows
    x, y = N * K * 2, N * M * size[case["out"]]
    if op in ("mm", "grouped_mx4"):
        return {"bytes": busy * M * nb * 17 + x + y, "flops": 2 * M * N * K}
    if op == "grouped":
        return {"bytes": busy * M * K * 2 + x + y, "flops": 2 * M * N * K}
    o = size[case["out"]]
    return {"bytes": 2 * N * M * 2 + busy * M * K * 2 + x + N * K * o + E * M * K * o, "flops": 4 * M * N * K}


# ----------------------------------------------------------------- the definition in 64 bits

def _exact_round(a):
    """(values, scale bytes) of the 4-bit form of [R, K], from the definition: every
    block divided by 2^(floor(log2 max) - 2), each quotient to the nearest E2M1
    value (ties to the even one), saturating at 6."""
    R, K = a.shape
    nb = -(-K // BLOCK)
    v = torch.zeros(R, nb * BLOCK, dtype=torch.float64, device=a.device)
    v[:, :K] = a.double()
    v = v.view(R, nb, BLOCK)
    top = v.abs().max(dim=2).values
    e = (torch.frexp(top).exponent - 1 - 2).clamp(-127, 127)
    e = torch.where(top == 0, torch.full_like(e, -127), e)
    scale = torch.ldexp(torch.ones_like(top), e)
    q = v / scale[:, :, None]
    step = torch.ldexp(torch.full_like(q, 0.5), (torch.frexp(q).exponent - 1).clamp(0, 2))
    q = (torch.round(q / step) * step).clamp(-6.0, 6.0)
    return (q * scale[:, :, None]).view(R, nb * BLOCK)[:, :K], e + 127


def _exact_values(elements, scales, K):
    mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=elements.device)
    v = torch.zeros(*elements.shape[:-1], elements.shape[-1] * 2, dtype=torch.float64, device=elements.device)
    for half, nib in ((0, elements & 0xF), (1, elements >> 4)):
        v[..., half::2] = mag[(nib & 7).long()] * (1.0 - 2.0 * (nib >> 3).double())
    return (v * torch.exp2(scales.double() - 127.0).repeat_interleave(BLOCK, dim=-1))[..., :K]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        values, scales = _exact_round(s["A"])
        return {"values": values, "scales": None}
    X = _exact_round(s["X"])[0] if case["x"] == "mx4" else s["X"].double()
    if case["op"] == "mm":
        return X @ _exact_values(s["W"], s["scales"], case["K"]).t()
    ends = s["offs"].tolist()
    if case["op"] == "grads":
        dX = torch.zeros(case["N"], case["K"], dtype=torch.float64, device="cuda")
        dW = torch.zeros(case["E"], case["M"], case["K"], dtype=torch.float64, device="cuda")
        for e, (a, b) in enumerate(zip(ends[:-1], ends[1:])):
            if b > a:
                dy = s["dY"][a:b].double()
                dX[a:b] = dy @ s["W"][e].double()
                dW[e] = dy.t() @ X[a:b]
        return {"dX": dX, "dW": dW}
    Y = torch.zeros(case["N"], case["M"], dtype=torch.float64, device="cuda")
    for e, (a, b) in enumerate(zip(ends[:-1], ends[1:])):
        if b > a:
            W = s["W"][e].double() if case["op"] == "grouped" else _exact_values(s["W"][e], s["scales"][e], case["K"])
            Y[a:b] = X[a:b] @ W.t()
    return Y
