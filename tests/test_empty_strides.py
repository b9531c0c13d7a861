"""Matrices without rows have no stride that could be wrong: slices of transposed tensors
are taken by every call, and by both marshallings."""
import pytest
import torch

import structured_sparse_gemm_amd as ssg
from structured_sparse_gemm_amd import _abi

F8 = torch.float8_e4m3fn


def none(cols, dtype, device):
    """[0, cols] with columns apart."""
    t = torch.zeros(cols, 4, device=device).to(dtype)[:, :0].t()
    assert t.shape == (0, cols) and t.stride(1) == 4
    return t


def calls(device):
    h, f, i = torch.float16, torch.float32, torch.int32
    w, ws = torch.zeros(8, 128, device=device).to(F8), torch.ones(1, 1, device=device)
    offs, x = torch.zeros(4, dtype=i, device=device), none(128, h, device)
    W = torch.zeros(3, 8, 128, dtype=h, device=device)
    pos, rows = torch.zeros(0, 2, dtype=i, device=device), torch.zeros(0, dtype=i, device=device)
    return [("mm_fp8", ssg.mm_fp8, (x, w, ws), (0, 8)), ("grouped_mm", ssg.grouped_mm, (x, W, offs), (0, 8)),
            ("expert_gather", ssg.expert_gather, (x, pos, rows), (0, 128)),
            ("expert_combine", ssg.expert_combine, (x, pos, none(2, f, device)), (0, 128)),
            ("expert_order", ssg.expert_order, (none(2, i, device), 8), (9,)), ("route", ssg.route, (none(8, f, device), 2), (0, 2))]


def test_strides_of_no_rows_are_not_refused():
    for name, f, args, _ in calls("cpu"):
        with pytest.raises(ssg.SsgError) as e:
            f(*args)
        assert e.value.status == _abi.SSG_ERR_NULL, name         # not on a device, and nothing else


@pytest.mark.gpu
def test_results_of_no_rows():
    s = torch.cuda.current_stream()
    for name, f, args, shape in calls("cuda"):
        for got in (f(*args), f(*args, stream=s)):
            assert (got[0] if isinstance(got, tuple) else got).shape == shape, name
    compiled, (x, w, ws) = _abi.torch_calls(), calls("cuda")[0][2]
    assert compiled.fp8_product(x, None, w, ws, None, torch.float32).shape == (0, 8)
