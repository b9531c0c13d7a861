"""Operands that the mx4 and expert-grouped calls have to refuse, or take, by
their strides and extents.  Refusals come before anything is enqueued."""
import contextlib
import ctypes
import sys
import warnings

import pytest
import torch

import structured_sparse_gemm_amd as ssg
from structured_sparse_gemm_amd import _abi
from tests import _mm as D

SHAPE, STRIDE, WORKSPACE = _abi.SSG_ERR_SHAPE, _abi.SSG_ERR_STRIDE, _abi.SSG_ERR_WORKSPACE


def status(f, *a, **k):
    with pytest.raises(ssg.SsgError) as e:
        f(*a, **k)
    return e.value.status


def repeated(t):
    """t's shape, every row the first one: row stride 0."""
    return t[..., :1, :].expand(t.shape)


def overlapping(t):
    """t's shape, every row one element after the one before."""
    strides = list(t.stride())
    strides[-2] = 1
    return t.as_strided(t.shape, strides)


def operands(device):
    X, dY = (torch.ones(6, c, dtype=torch.float16, device=device) for c in (64, 8))
    W = torch.ones(2, 8, 64, dtype=torch.float16, device=device)
    e, s = (torch.zeros(2, 8, c, dtype=torch.uint8, device=device) for c in (32, 2))
    xe, xs = (torch.zeros(6, c, dtype=torch.uint8, device=device) for c in (32, 2))
    return X, dY, W, e, s, xe, xs, torch.tensor([0, 2, 6], dtype=torch.int32, device=device)


def calls_with(bad, device):
    """Every call with one operand in the layout `bad`; each is a function to
    call, and what it would call in the compiled marshalling (None: no such call)."""
    X, dY, W, e, s, xe, xs, offs = operands(device)
    f16, f32 = torch.float16, torch.float32
    Y, dX, dW = (torch.empty(n, device=device) for n in ((6, 8), (6, 64), (2, 8, 64)))
    prod, grp = "mx4_product", "grouped_product"
    return [
        (ssg.mx4_quantize, (bad(X),), ("mx4_quantize", bad(X))),
        (ssg.mx4_dequantize, (bad(xe), xs, 64), ("mx4_dequantize", bad(xe), xs, 64, f32)),
        (ssg.mx4_dequantize, (xe, bad(xs), 64), ("mx4_dequantize", xe, bad(xs), 64, f32)),
        (ssg.mm_mx4, (bad(X), e[0], s[0]), (prod, bad(X), None, e[0], s[0], None, f32)),
        (ssg.mm_mx4, (X, bad(e[0]), s[0]), (prod, X, None, bad(e[0]), s[0], None, f32)),
        (ssg.mm_mx4, (X, e[0], bad(s[0])), (prod, X, None, e[0], bad(s[0]), None, f32)),
        (ssg.mm_mx4, (bad(xe), e[0], s[0], xs), (prod, bad(xe), xs, e[0], s[0], None, f32)),
        (ssg.mm_mx4, (xe, e[0], s[0], bad(xs)), (prod, xe, bad(xs), e[0], s[0], None, f32)),
        (ssg.grouped_mm_mx4, (bad(X), e, s, offs), (prod, bad(X), None, e, s, offs, f32)),
        (ssg.grouped_mm_mx4, (X, bad(e), s, offs), (prod, X, None, bad(e), s, offs, f32)),
        (ssg.grouped_mm_mx4, (X, e, bad(s), offs), (prod, X, None, e, bad(s), offs, f32)),
        (ssg.grouped_mm, (bad(X), W, offs), (grp, 0, bad(X), W, offs, f16)),
        (ssg.grouped_mm, (X, bad(W), offs), (grp, 0, X, bad(W), offs, f16)),
        (ssg.grouped_mm_dx, (bad(dY), W, offs), (grp, 1, bad(dY), W, offs, f16)),
        (ssg.grouped_mm_dx, (dY, bad(W), offs), (grp, 1, dY, bad(W), offs, f16)),
        (ssg.grouped_mm_dw, (bad(dY), X, offs), (grp, 2, bad(dY), X, offs, f16)),
        (ssg.grouped_mm_dw, (dY, bad(X), offs), (grp, 2, dY, bad(X), offs, f16)),
        # outputs
        (ssg.ssg_mx4_quantize, (X, bad(xe), xs), None),
        (ssg.ssg_mx4_quantize, (X, xe, bad(xs)), None),
        (ssg.ssg_mx4_dequantize, (xe, xs, bad(dX)), None),
        (ssg.ssg_mm_mx4, (X, e[0], s[0], bad(Y)), None),
        (ssg.ssg_grouped_mm_mx4, (X, e, s, offs, bad(Y)), None),
        (ssg.ssg_grouped_mm, (X, W, offs, bad(Y)), None),
        (ssg.ssg_grouped_mm_dx, (dY, W, offs, bad(dX)), None),
        (ssg.ssg_grouped_mm_dw, (dY, X, offs, bad(dW)), None),
    ]


class NoLibrary:
    """Takes every call and does nothing."""
    def __getattr__(self, name):
        return lambda *args: 0


@pytest.fixture
def host_tensors(monkeypatch):
    """Host tensors get as far as the library, and no call leaves the binding."""
    monkeypatch.setattr(ssg, "_lib", NoLibrary)
    for name in ("_on_device", "_ptr"):
        monkeypatch.setattr(ssg, name, lambda t, name: None if t is None else t.data_ptr())
    for name in ("_raw_stream", "_stream"):
        monkeypatch.setattr(ssg, name, lambda t, stream: None)


@pytest.mark.parametrize("bad", [repeated, overlapping])
def test_rows_that_repeat_or_overlap_are_refused(bad, host_tensors):
    for f, args, _ in calls_with(lambda t: t, "cpu"):
        f(*args)
    for i, (f, args, _) in enumerate(calls_with(bad, "cpu")):
        assert status(f, *args) == STRIDE, (i, f.__name__)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [repeated, overlapping])
def test_rows_that_repeat_or_overlap_are_refused_on_the_device(bad):
    compiled = _abi.torch_calls()
    for i, (f, args, call) in enumerate(calls_with(bad, "cuda")):
        if call is not None:
            assert getattr(compiled, call[0])(*call[1:]) is None, (i, call[0])
        assert status(f, *args) == STRIDE, (i, f.__name__)


@pytest.mark.gpu
def test_strides_without_a_meaning():
    # a single row, and rows of one column, whatever their strides; one weight
    # for every expert
    gen = torch.Generator().manual_seed(5)
    x, w = torch.randn(1, 64, generator=gen).half(), torch.randn(1, 8, 64, generator=gen).half()
    offs = torch.tensor([0, 0, 1], dtype=torch.int32).cuda()
    X, W = x.cuda().as_strided((1, 64), (0, 1)), w.cuda().expand(2, 8, 64)
    D.check(ssg.grouped_mm(X, W, offs), (x.double() @ w[0].double().t()).numpy(),
            (x.double().abs() @ w[0].double().abs().t()).numpy(), 64, "one row")
    dY = torch.randn(5, 3, generator=gen).half().cuda()
    one = torch.ones(2, 1, 3, dtype=torch.float16).cuda().transpose(1, 2)       # [2, 3, 1], strides (3, 1, 3)
    offs = torch.tensor([0, 2, 5], dtype=torch.int32).cuda()
    got = ssg.grouped_mm_dx(dY, one, offs, out_dtype=torch.float32)
    ref = dY.double().cpu()
    D.check(got, ref.sum(1, keepdim=True).numpy(), ref.abs().sum(1, keepdim=True).numpy(), 3, "one column")


@pytest.mark.parametrize("bad", [repeated, overlapping])
def test_rows_of_sparse_operands_that_repeat_or_overlap_are_refused(bad, host_tensors):
    A, B, C = torch.ones(8, 64, dtype=torch.float16), torch.ones(64, 4, dtype=torch.float16), torch.empty(8, 4)
    v, m = torch.ones(8, 32, dtype=torch.float16), torch.full((8, 8), 0x44, dtype=torch.uint8)
    calls = [(ssg.ssg_prune_2to4, 0, A, A.clone()), (ssg.ssg_prune_2to4, 1, A, A.clone()),
             *((ssg.ssg_compress_2to4, at, A, v, m) for at in range(3)),
             (ssg.ssg_decompress_2to4, 2, v, m, A), (ssg.ssg_compress_2to4_prefill, 0, A, v, m),
             (ssg.ssg_spmm_2to4_packed, 3, v, m, 8, B, C), (ssg.ssg_spmm_2to4_packed, 4, v, m, 8, B, C),
             (ssg.ssg_spmm_2to4_packed_bt, 3, v, m, 8, A, C), (ssg.ssg_spmm_2to4_prefill, 3, v, m, 8, B, C),
             (ssg.ssg_spmm_2to4_prefill_bt, 3, v, m, 8, A, C)]
    for i, (f, at, *args) in enumerate(calls):
        f(*args)
        args[at] = bad(args[at])
        assert status(f, *args) == STRIDE, (i, f.__name__)


def test_weight_gradients_that_share_elements_are_refused():
    lib, at = _abi.load(), ctypes.c_void_p(0x1000)     # never dereferenced: no rows, or refused

    def dw(E, M, K, ld, stride):
        # rows of odd length need a workspace: without one, nothing is enqueued
        assert K % 2 == 1
        return lib.ssg_grouped_mm_dw(0, 3, E, M, 300, K, at, M + 1, at, K, at, at, ld, stride, None, 0, None)

    def apart(E, M, K, ld, stride):
        starts = [e * stride + m * ld for e in range(E) for m in range(M)]
        cells = [a + k for a in starts for k in range(K)]
        return len(set(cells)) == len(cells)

    seen = set()
    for E, M, K in [(2, 3, 5), (3, 2, 5), (4, 4, 3), (2, 1, 5), (5, 3, 1)]:
        for ld in (K, K + 1, 2 * K, 3 * K + 1, 5 * K):
            for stride in [*range(-2, 5 * K), M * ld - ld, M * ld - ld + K - 1, M * ld - ld + K, M * ld, -M * ld]:
                ok = apart(E, M, K, ld, stride)
                seen.add(ok)
                assert dw(E, M, K, ld, stride) == (WORKSPACE if ok else STRIDE), (E, M, K, ld, stride)
    assert seen == {False, True}
    assert dw(1, 3, 5, 5, 0) == WORKSPACE                  # one matrix: the stride means nothing


@pytest.mark.gpu
def test_weight_gradients_in_any_layout_that_keeps_them_apart():
    gen = torch.Generator().manual_seed(6)
    dY, X = (torch.randn(70, c, generator=gen).half() for c in (12, 24))
    offs = D.offsets([30, 0, 40])
    ref = D.grouped_dw(dY.double().numpy(), X.double().numpy(), offs)
    between = torch.empty(12, 3, 24).cuda().transpose(0, 1)      # every matrix's row m side by side
    apart = torch.empty(3, 15, 30).cuda()[:, :12, :24]
    for dW in (between, apart):
        ssg.ssg_grouped_mm_dw(dY.cuda(), X.cuda(), offs.cuda(), dW)
        D.check(dW, *ref, 40, "dW")
    inside = torch.empty(500).cuda().as_strided((3, 12, 24), (24, 24, 1))
    for dW in (torch.empty(1, 12, 24).cuda().expand(3, 12, 24), inside):
        assert status(ssg.ssg_grouped_mm_dw, dY.cuda(), X.cuda(), offs.cuda(), dW) == STRIDE


@pytest.mark.parametrize("cols", [1, 15, 17, 31, 33])
def test_mx4_activations_that_end_inside_a_block_are_refused(cols, host_tensors):
    nb = (2 * cols + 31) // 32
    X, xs = torch.zeros(6, 64, dtype=torch.uint8)[:, :cols], torch.zeros(6, nb, dtype=torch.uint8)
    W, s = torch.zeros(2, 8, 16 * nb, dtype=torch.uint8), torch.zeros(2, 8, nb, dtype=torch.uint8)
    offs = torch.zeros(3, dtype=torch.int32)
    assert status(ssg.mm_mx4, X, W[0], s[0], xs) == SHAPE
    assert status(ssg.grouped_mm_mx4, X, W, s, offs, xs) == SHAPE
    assert status(ssg.ssg_mm_mx4_workspace_bytes, X, W[0], s[0], xs) == SHAPE


@pytest.mark.gpu
def test_mx4_activations_that_end_inside_a_block_are_refused_on_the_device():
    X, xs = torch.zeros(6, 64, dtype=torch.uint8).cuda()[:, :17], torch.zeros(6, 2, dtype=torch.uint8).cuda()
    W, s = torch.zeros(2, 8, 32, dtype=torch.uint8).cuda(), torch.zeros(2, 8, 2, dtype=torch.uint8).cuda()
    offs, compiled = torch.zeros(3, dtype=torch.int32).cuda(), _abi.torch_calls()
    for w, t, o in ((W[0], s[0], None), (W, s, offs)):
        assert compiled.mx4_product(X, xs, w, t, o, torch.float32) is None
    assert status(ssg.mm_mx4, X, W[0], s[0], xs) == SHAPE
    assert status(ssg.grouped_mm_mx4, X, W, s, offs, xs) == SHAPE


def test_no_experts_need_no_copy_of_their_weights():
    # the copy of an absent stack would begin at a null pointer: it shows as workspace
    lib, at = _abi.load(), ctypes.c_void_p(0x1000)
    for N in (200, 5000):
        assert lib.ssg_grouped_mm_workspace_bytes(0, 0, 64, N, 33, at, 33, None, 33, 0, at) == -(-N * 80 // 256) * 256
        assert lib.ssg_grouped_mm_dx_workspace_bytes(0, 0, 64, N, 33, at, 64, None, 33, 0, at) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 200, 3000])
@pytest.mark.parametrize("K", [33, 64, 100])
def test_no_experts(N, K):
    offs = torch.zeros(1, dtype=torch.int32).cuda()
    for f, cols, out in ((ssg.grouped_mm, K, 66), (ssg.grouped_mm_dx, 66, K)):
        X = torch.ones(N, cols, dtype=torch.float16).cuda()
        Y = f(X, torch.empty(0, 66, K, dtype=torch.float16).cuda(), offs)
        assert Y.shape == (N, out) and (Y == 0).all()
    nb = (K + 31) // 32
    W, s = torch.empty(0, 66, 16 * nb, dtype=torch.uint8).cuda(), torch.empty(0, 66, nb, dtype=torch.uint8).cuda()
    Xe, Xs = (torch.full((N, c), v, dtype=torch.uint8).cuda() for c, v in ((16 * nb, 0x22), (nb, 127)))
    for Y in (ssg.grouped_mm_mx4(torch.ones(N, K, dtype=torch.bfloat16).cuda(), W, s, offs),
              ssg.grouped_mm_mx4(Xe, W, s, offs, xscales=Xs)):
        assert Y.shape == (N, 66) and (Y == 0).all()


EMPTY = [(0, 5, 70), (3, 0, 70), (3, 5, 0), (0, 0, 0), (2, 0, 0)]


def back_and_forth(E, R, K, device):
    nb = (K + 31) // 32
    e, s = ssg.mx4_quantize(torch.zeros(E, R, K, dtype=torch.bfloat16, device=device))
    assert e.shape == (E, R, 16 * nb) and s.shape == (E, R, nb)
    assert ssg.mx4_dequantize(e, s, K).shape == (E, R, K)


@pytest.mark.parametrize("E,R,K", EMPTY)
def test_empty_stacks(E, R, K, host_tensors):
    back_and_forth(E, R, K, "cpu")


@pytest.mark.gpu
@pytest.mark.parametrize("E,R,K", EMPTY)
def test_empty_stacks_on_the_device(E, R, K):
    back_and_forth(E, R, K, "cuda")


def test_scales_of_another_stack_are_refused(host_tensors):
    e = torch.zeros(2, 3, 32, dtype=torch.uint8)
    for s in (torch.zeros(3, 2, 2, dtype=torch.uint8), torch.zeros(6, 2, dtype=torch.uint8)):
        assert status(ssg.mx4_dequantize, e, s, 64) == SHAPE


@pytest.mark.gpu
def test_stacks_are_read_on_the_stream_that_the_call_names():
    # weights that `side` is still about to write, in stacks whose rows are not
    # equally far apart
    gen = torch.Generator().manual_seed(8)
    wide = torch.randn(4, 40, 96, generator=gen).bfloat16().cuda()
    e, s = ssg.mx4_quantize(wide[:, :30])
    values = ssg.mx4_dequantize(e, s, 96)
    late = torch.zeros(4, 40, 96, dtype=torch.bfloat16).cuda()
    le, ls = (torch.zeros(4, 40, c, dtype=torch.uint8).cuda() for c in (48, 3))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(wide)
        le[:, :30].copy_(e)
        ls[:, :30].copy_(s)
    e2, s2 = ssg.mx4_quantize(late[:, :30], stream=side)
    got = ssg.mx4_dequantize(le[:, :30], ls[:, :30], 96, stream=side)
    side.synchronize()
    assert torch.equal(e2, e) and torch.equal(s2, s) and torch.equal(got, values)


def test_copies_of_stacks_are_made_on_the_stream_that_the_call_names(host_tensors, monkeypatch):
    inside, copied = [], []
    real = torch.Tensor.reshape

    @contextlib.contextmanager
    def on_stream(like, stream):
        inside.append(stream)
        yield
        inside.pop()

    monkeypatch.setattr(ssg, "_on_stream", on_stream, raising=False)
    monkeypatch.setattr(torch.Tensor, "reshape", lambda t, *a: (copied.append(list(inside)), real(t, *a))[1])
    wide = torch.zeros(4, 40, 96, dtype=torch.bfloat16)
    e, s = ssg.mx4_quantize(wide[:, :30], stream=77)
    assert copied == [[77]]
    ssg.mx4_dequantize(e[:, :9], s[:, :9], 96, stream=78)
    assert copied[1:] == [[78], [78]]


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 40, 300])
def test_contractions_of_no_elements(N):
    def empty(*shape, dtype=torch.uint8):
        return torch.empty(*shape, dtype=dtype).cuda()

    offs = torch.tensor([0, 0, N], dtype=torch.int32).cuda()
    e, s = empty(2, 70, 0), empty(2, 70, 0)
    for X, xs in ((empty(N, 0, dtype=torch.float16), None), (empty(N, 0, dtype=torch.bfloat16), None),
                  (empty(N, 0), empty(N, 0))):
        for Y in (ssg.mm_mx4(X, e[0], s[0], xs), ssg.grouped_mm_mx4(X, e, s, offs, xs)):
            assert Y.shape == (N, 70) and (Y == 0).all()
    h = empty(N, 0, dtype=torch.float16)
    Y = ssg.grouped_mm(h, empty(2, 70, 0, dtype=torch.float16), offs)
    assert Y.shape == (N, 70) and (Y == 0).all()
    dX = ssg.grouped_mm_dx(h, empty(2, 0, 70, dtype=torch.float16), offs)
    assert dX.shape == (N, 70) and (dX == 0).all()


def failed(lib):
    """A failure for ssg_last_error() to tell."""
    at = ctypes.c_void_p(0x1000)                               # never dereferenced
    assert lib.ssg_mx4_quantize(3, 4, 64, at, 63, at, 32, at, 2, None) == STRIDE
    return lib.ssg_last_error()


def test_asking_for_a_workspace_records_no_error():
    lib, at = _abi.load(), ctypes.c_void_p(0x1000)
    product = (0, 3, 2, 70, 600, 333, at, 333, at, 333, 70 * 333, at, at, 70)      # odd rows: copied to a workspace
    before = failed(lib)
    assert lib.ssg_grouped_mm(*product, None, _abi.SSG_WS_ASK, None) == WORKSPACE
    assert lib.ssg_last_error() == before
    assert lib.ssg_grouped_mm(*product, None, 0, None) == WORKSPACE
    assert b"workspace" in lib.ssg_last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("stream", [False, True])
def test_a_call_that_succeeds_records_no_error(stream):
    lib = _abi.load()
    before = failed(lib)
    X, W = torch.ones(600, 333, dtype=torch.float16).cuda(), torch.ones(2, 70, 333, dtype=torch.float16).cuda()
    offs = torch.tensor([0, 100, 600], dtype=torch.int32).cuda()
    assert ssg.ssg_grouped_mm_workspace_bytes(X, W, offs) > 0
    Y = ssg.grouped_mm(X, W, offs, stream=torch.cuda.current_stream() if stream else None)
    assert (Y == 333).all() and lib.ssg_last_error() == before


def test_missing_compiled_marshalling_is_told(monkeypatch):
    monkeypatch.delattr(ssg, "_torch_calls", raising=False)
    monkeypatch.setitem(sys.modules, ssg.__name__ + "._torch_calls", None)     # its import fails
    monkeypatch.setattr(ssg, "_calls", None)
    with pytest.warns(RuntimeWarning, match="compiled marshalling"):
        assert _abi.torch_calls() is None
    with pytest.warns(RuntimeWarning):
        first = ssg._compiled()
    with warnings.catch_warnings():
        warnings.simplefilter("error")                                         # once only
        assert ssg._compiled() is first and first.mx4_quantize(None) is None


def test_workspaces_that_are_not_one_piece_are_refused(host_tensors):
    X, dY, W, e, s, xe, xs, offs = operands("cpu")
    v, B, C = torch.ones(8, 32).half(), torch.ones(64, 4).half(), torch.empty(8, 4)
    m = torch.full((8, 8), 0x44, dtype=torch.uint8)
    calls = [lambda ws: ssg.ssg_mm_mx4(X, e[0], s[0], torch.empty(6, 8), ws=ws),
             lambda ws: ssg.ssg_grouped_mm(X, W, offs, torch.empty(6, 8), ws=ws),
             lambda ws: ssg.ssg_grouped_mm_dw(dY, X, offs, torch.empty(2, 8, 64), ws=ws),
             lambda ws: ssg.ssg_spmm_2to4(v, m, B, C, ws=ws)]
    for call in calls:
        for ws in (torch.empty(4096, dtype=torch.uint8), torch.empty(32, 128).t(), torch.empty(0), torch.empty(3, 0)):
            call(ws)
        # one byte that claims to be 4096, and every second one of 8192
        assert status(call, torch.empty(1, dtype=torch.uint8).expand(4096)) == STRIDE
        assert status(call, torch.empty(8192, dtype=torch.uint8)[::2]) == STRIDE
        assert status(call, torch.empty(4096, dtype=torch.uint8, device="meta")) == _abi.SSG_ERR_NULL


def test_limits():
    # the largest operands that the header allows, and the smallest that it does not
    lib, at, k = _abi.load(), ctypes.c_void_p(0x1000), (ctypes.c_int64 * 4)()

    def choice(op, E=1, M=64, N=64, K=64):
        return lib.ssg_mm_select_kernel(op, 0, E, M, N, K, k)

    for op in range(5):
        for size in ("M", "N", "K"):
            assert choice(op, **{size: 2 ** 29}) == SHAPE
        assert choice(op, N=2 ** 29 - 1) == 0
        if op > 0:
            assert choice(op, E=2 ** 20 - 1) == 0 and choice(op, E=2 ** 20) == SHAPE
    assert choice(0, K=2 ** 21 - 1) == 0 and choice(0, K=2 ** 21) == STRIDE
    assert choice(3, M=2 ** 21) == STRIDE and choice(4, K=2 ** 21) == STRIDE and choice(2, M=2 ** 21) == 0
    # (no rows: nothing is enqueued)
    for ld, rc in ((2 ** 21 - 1, 0), (2 ** 21, STRIDE)):
        assert lib.ssg_mm_mx4(0, 3, 8, 0, 64, at, ld, None, 0, at, 32, at, 2, at, 8, None, 0, None) == rc
    assert lib.ssg_mm_mx4(0, 3, 8, 0, 64, at, 64, None, 0, at, 32, at, 2, at, 2 ** 40, None, 0, None) == 0


def test_operands_off_the_current_device_do_not_meet_its_null_stream(monkeypatch):
    class Tensor:
        device = torch.device("cuda:1")

    class Stream:
        def __init__(self, raw):
            self.cuda_stream = raw

    current = {"raw": 0, "device": 0}
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: current["raw"], raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream(current["raw"]))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current["device"])
    for handle in (ssg._stream, ssg._raw_stream):
        current.update(raw=0, device=0)
        assert status(handle, Tensor, None) == _abi.SSG_ERR_NULL
        assert status(handle, Tensor, Stream(0)) == _abi.SSG_ERR_NULL
        assert handle(Tensor, Stream(5)) == 5                # a stream knows its device
        current.update(raw=7)
        assert handle(Tensor, None) == 7
        current.update(raw=0, device=1)
        assert handle(Tensor, None) is None


# clamped to the rows that there are: [0, 3, 3, N], [N, N, N, N], [0, 0, 0, 0]; and
# offsets that descend, whose results are anything inside the outputs
@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(20, 96), (400, 96), (400, 97)])
@pytest.mark.parametrize("offs", [[-5, 3, 3, 1 << 30], [2000, 2000, 3000, 4000], [-9, -8, -7, -6], [17, 3, 400, 2]])
def test_offsets_out_of_range_are_clamped(N, K, offs):
    M, E = 70, 3
    gen = torch.Generator().manual_seed(N + K)
    X, W, dY = (torch.randn(*n, generator=gen).half() for n in ((N, K), (E, M, K), (N, M)))
    clamped = torch.tensor(offs, dtype=torch.int32).clamp(0, N)
    og = torch.tensor(offs, dtype=torch.int32).cuda()
    e, s = D.random_mx4((E, M, K), 3)
    We, Ws = torch.from_numpy(e).cuda(), torch.from_numpy(s).cuda()
    Xe, Xs = ssg.mx4_quantize(X.cuda())
    x, w, d = (t.double().numpy() for t in (X, W, dY))
    outs = {name: torch.full((rows + 2, cols + 2), 7.0).cuda() for name, rows, cols in
            (("Y", N, M), ("dX", N, K), ("dW", E * M, K), ("w4", N, M), ("mx", N, M))}
    inner = {name: t[1:-1, 1:-1] for name, t in outs.items()}
    dW = inner["dW"].unflatten(0, (E, M))
    ssg.ssg_grouped_mm(X.cuda(), W.cuda(), og, inner["Y"])
    ssg.ssg_grouped_mm_dx(dY.cuda(), W.cuda(), og, inner["dX"])
    ssg.ssg_grouped_mm_dw(dY.cuda(), X.cuda(), og, dW)
    ssg.ssg_grouped_mm_mx4(X.cuda(), We, Ws, og, inner["w4"])
    ssg.ssg_grouped_mm_mx4(Xe, We, Ws, og, inner["mx"], xscales=Xs)
    for t in outs.values():
        assert (t[0] == 7).all() and (t[-1] == 7).all() and (t[:, 0] == 7).all() and (t[:, -1] == 7).all()
    if sorted(offs) != offs:
        return
    w4 = D.mx4_values(e, s, K)
    x4 = D.mx4_values(Xe.cpu().numpy(), Xs.cpu().numpy(), K)
    D.check(inner["Y"], *D.grouped(x, w, clamped), K, "Y")
    D.check(inner["dX"], *D.grouped_dx(d, w, clamped), M, "dX")
    D.check(dW, *D.grouped_dw(d, x, clamped), N, "dW")
    D.check(inner["w4"], *D.grouped(x, w4, clamped), K, "mx4 weights")
    D.check(inner["mx"], *D.grouped(x4, w4, clamped), K, "mx4 x mx4")
