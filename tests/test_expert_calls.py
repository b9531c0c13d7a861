"""The calls around the experts' products and of 8-bit floats: marshalled by the
compiled module and by the Python binding, with operands that either refuses."""
import pytest
import torch

import structured_sparse_gemm_amd as ssg
from structured_sparse_gemm_amd import _abi
from structured_sparse_gemm_amd._abi import (SSG_ERR_DTYPE as DTYPE, SSG_ERR_NULL as NULL, SSG_ERR_SHAPE as SHAPE,
                                             SSG_ERR_STRIDE as STRIDE)

F8 = torch.float8_e4m3fn


def status(f, *args, **kw):
    with pytest.raises(ssg.SsgError) as e:
        f(*args, **kw)
    return e.value.status


def calls(device):
    """(name, function, arguments of the public call, those of the compiled one)."""
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g)
    N, E, k, C, M = 6, 8, 2, 256, 24
    l, X, dO, bias, dw = r(N, E).half(), r(N, C).bfloat16(), r(N, C).bfloat16(), r(E), r(N, k)
    experts = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(N)]).int()
    flat = experts.reshape(-1)
    rows = torch.sort(flat, stable=True).indices.int()
    pos = torch.argsort(rows.long()).int().reshape(N, k)
    offs = torch.zeros(E + 1, dtype=torch.int32)
    offs[1:] = torch.bincount(flat.long(), minlength=E).cumsum(0)
    Y, w = r(N * k, C).bfloat16(), r(N, k)
    W, ws, W3, ws3 = r(M, C).to(F8), r(1, 2).abs(), r(E, M, C).to(F8), r(E, 1, 2).abs()
    x8, xs = r(N, C).to(F8), r(N, 2).abs()
    l, X, dO, bias, dw, experts, rows, pos, offs, Y, w, W, ws, W3, ws3, x8, xs = (
        t.to(device) for t in (l, X, dO, bias, dw, experts, rows, pos, offs, Y, w, W, ws, W3, ws3, x8, xs))
    t, half = torch, Y[::2]
    return [
        ("route", ssg.route, (l, k, "sigmoid", bias, 4, 2, "top2", True, 2.5), None),
        ("route", ssg.route, (l, k, "softmax", None, 1, 1, "max", False, 1.0), None),
        ("route_backward", ssg.route_backward, (dw, l, experts, "softmax", True, 1.0), None),
        ("expert_order", ssg.expert_order, (experts, E), None),
        ("expert_gather", ssg.expert_gather, (X, pos, rows), None),
        ("expert_combine", ssg.expert_combine, (Y, pos, w, t.float32), None),
        ("expert_combine", ssg.expert_combine, (Y, pos, None, None), None),
        ("expert_combine_backward", ssg.expert_combine_backward, (dO, Y, pos, rows, w), None),
        ("fp8_quantize", ssg.fp8_quantize, (X, 1, False), None),
        ("fp8_quantize", ssg.fp8_quantize, (X[:, :250], 1, True), None),
        ("fp8_quantize", ssg.fp8_quantize, (X.view(2, 3, C), 128, False), None),
        ("fp8_dequantize", ssg.fp8_dequantize, (W, ws, t.float16), None),
        ("fp8_dequantize", ssg.fp8_dequantize, (W3, ws3, t.float32), None),
        ("fp8_product", ssg.mm_fp8, (X, W, ws, None, t.bfloat16), (X, None, W, ws, None, t.bfloat16)),
        ("fp8_product", ssg.mm_fp8, (x8, W, ws, xs, t.float32), (x8, xs, W, ws, None, t.float32)),
        ("fp8_product", ssg.grouped_mm_fp8, (Y, W3, ws3, offs, None, t.float32), (Y, None, W3, ws3, offs, t.float32)),
        ("fp8_product", ssg.grouped_mm_fp8, (half, W3, ws3, offs, None, t.float16),
         (half, None, W3, ws3, offs, t.float16)),
    ]


def result(v):
    return v if isinstance(v, tuple) else (v,)


def test_compiled_calls_leave_host_tensors_and_others_to_the_binding():
    compiled = _abi.torch_calls()
    assert compiled is not None
    for name, f, args, c in calls("cpu"):
        c = c or args
        g = getattr(compiled, name)
        assert g(*c) is None and g(*c[:-1]) is None and g(*c, 1) is None
        for i in range(len(c)):
            assert g(*c[:i], None, *c[i + 1:]) is None and g(*c[:i], 1 << 70, *c[i + 1:]) is None
        assert status(f, *args) == NULL, name


@pytest.mark.gpu
def test_both_marshallings_give_the_same_results():
    compiled, stream = _abi.torch_calls(), torch.cuda.current_stream()
    for name, f, args, c in calls("cuda"):
        by_hand = getattr(compiled, name)(*(c or args))
        assert by_hand is not None, name
        for got in (f(*args), f(*args, stream=stream)):
            for a, b in zip(result(by_hand), result(got)):
                assert a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride(), name
                assert torch.equal(a.flatten().view(torch.uint8), b.flatten().view(torch.uint8)), name


# operands that may have a column less: fewer experts, choices, elements
SMALLER = {("route", 0), ("route_backward", 1), ("expert_order", 0), ("expert_gather", 0), ("expert_combine", 0),
           ("fp8_quantize", 0), ("fp8_dequantize", 0)}


def damaged(args):
    """(argument's place, its damaged form, status) for each tensor of a call."""
    for i, t in enumerate(args):
        if not isinstance(t, torch.Tensor):
            continue
        yield i, t.to(torch.int64), DTYPE
        yield i, t.reshape(-1)[:0], SHAPE
        yield i, t[..., :-1].contiguous(), SHAPE
        if t.dim() > 1 and t.dtype != torch.float32:
            yield i, t[..., :1].expand(t.shape), STRIDE


@pytest.mark.gpu
def test_operands_of_other_types_shapes_and_strides_are_refused_on_the_device():
    compiled = _abi.torch_calls()
    for name, f, args, c in calls("cuda"):
        for i, bad, want in damaged(args):
            other = args[:i] + (bad,) + args[i + 1:]
            if want == SHAPE and bad.dim() > 1 and (name, i) in SMALLER:
                continue
            c2 = other if c is None else tuple(bad if t is args[i] else t for t in c)
            assert getattr(compiled, name)(*c2) is None, (name, i, want)
            with pytest.raises(ssg.SsgError) as e:
                f(*other)
            assert e.value.status == want, (name, i, want)


@pytest.mark.gpu
def test_numbers_out_of_range_are_refused_before_anything_is_allocated():
    l, e = torch.zeros(4, 8).cuda(), torch.zeros(4, 2, dtype=torch.int32).cuda()
    for k in (-1, 9, 1 << 40):
        assert status(ssg.route, l, k) == SHAPE
    for E in (-1, 1 << 20, 1 << 40):
        assert status(ssg.expert_order, e, E) == SHAPE
    assert status(ssg.route, l, 2, groups=1 << 40) == SHAPE and status(ssg.route, l, 2, groups=3) == SHAPE
