"""Products of more tiles than a launch holds are refused on the host, before anything is
enqueued."""
import ctypes

import pytest

from structured_sparse_gemm_amd import _abi

FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: every call below is refused first
SHAPE = _abi.SSG_ERR_SHAPE


@pytest.fixture(scope="module")
def lib():
    return _abi.load()


@pytest.mark.parametrize("x", [_abi.SSG_E4M3, _abi.SSG_BF16])
@pytest.mark.parametrize("y", [_abi.SSG_F32, _abi.SSG_BF16])
@pytest.mark.parametrize("wblock", [1, 128])
def test_more_tiles_than_a_launch_holds(lib, x, y, wblock):
    E, M, N, K = 1 << 19, 1 << 17, 1 << 14, 128
    e4 = x == _abi.SSG_E4M3
    args = (x, y, E, M, N, K, FAKE, K, FAKE if e4 else None, 1, N, FAKE, K, M * K, wblock, FAKE, 1, M, M, FAKE)
    assert lib.ssg_grouped_mm_fp8(*args, FAKE, M, FAKE, 1 << 62, None) == SHAPE
    assert lib.ssg_grouped_mm_fp8(*args, FAKE, M, None, _abi.SSG_WS_ASK, None) == SHAPE
    M = N = 1 << 28
    args = (x, y, M, N, K, FAKE, K, FAKE if e4 else None, 1, N, FAKE, K, wblock, FAKE, 1, M)
    assert lib.ssg_mm_fp8(*args, FAKE, M, FAKE, 1 << 62, None) == SHAPE
    assert b"size too large" in lib.ssg_last_error()
    assert lib.ssg_mm_fp8_workspace_bytes(*args) == 0
    kernel = (ctypes.c_int64 * 4)()
    assert lib.ssg_mm_fp8_select_kernel(x, y, wblock, 0, M, N, K, kernel) == SHAPE


def test_scales_that_would_fill_more_than_a_launch_are_refused(lib):
    # scales by rows, of matrices that repeat: 2^32 of them to rearrange
    E, M, N, K = 1 << 10, 1 << 15, 1 << 19, 16384
    args = (_abi.SSG_E4M3, _abi.SSG_BF16, E, M, N, K, FAKE, K, FAKE, 1, N, FAKE, K, 0, 1, FAKE, 128, 1, 0, FAKE)
    assert lib.ssg_grouped_mm_fp8(*args, FAKE, M, FAKE, 1 << 62, None) == SHAPE
