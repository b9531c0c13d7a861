// fp8_abi.cpp -- the C ABI of 8-bit floats with a scale for each block of 128:
// host-side checks, the choice of kernel, and the workspace (activations rounded
// in the call, operands and scales in another layout, partials of a split
// contraction).
#include "ssgemm.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "fp8.hpp"
#include "ssg_abi.hpp"

namespace {

using ssg::abi_failf;
using ssg::Fp8Matrix;
using ssg::MmFp8Args;

typedef long long ll;

constexpr int64_t kMaxDim = (int64_t)1 << 29;
constexpr int kCUs = 256;

int hip_status(hipError_t e) {
    return e == hipSuccess ? SSG_OK : abi_failf(SSG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
}

bool al(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
int64_t blocks(int64_t n) { return (n + ssg::kFp8Block - 1) / ssg::kFp8Block; }

int source(int dt) {
    return dt == SSG_F16 ? ssg::SRC8_F16 : dt == SSG_BF16 ? ssg::SRC8_BF16 : dt == SSG_F32 ? ssg::SRC8_F32 : -1;
}
int64_t float_bytes(int dt) { return dt == SSG_F32 ? 4 : 2; }

// ------------------------------------------------------------------ checks

int check_mat(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld) {
    if (rows > 0 && cols > 0 && !p) return abi_failf(SSG_ERR_NULL, "%s is NULL", name);
    if (ld < cols) return abi_failf(SSG_ERR_STRIDE, "row stride of %s: %lld < %lld", name, (ll)ld, (ll)cols);
    return SSG_OK;
}

// Scales are read (and written) one by one where their layout asks for it; their
// strides only have to be addressable.
int check_scales(const char* name, const void* p, int64_t rows, int64_t nb, int64_t row, int64_t blk) {
    if (rows > 0 && nb > 0 && !p) return abi_failf(SSG_ERR_NULL, "%s is NULL", name);
    if (row < 0 || blk < 0 || row >= kMaxDim || blk >= kMaxDim)
        return abi_failf(SSG_ERR_STRIDE, "strides of %s: %lld, %lld", name, (ll)row, (ll)blk);
    return SSG_OK;
}

// No two elements of an output of n[] elements, `stride`[] apart, share a place: by
// rising stride, each is beyond what the smaller ones reach.
bool apart(const int64_t (&n)[3], const int64_t (&stride)[3]) {
    if (n[0] == 0 || n[1] == 0 || n[2] == 0) return true;
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return stride[a] < stride[b]; });
    int64_t reach = 0;
    for (int d : order) {
        if (n[d] <= 1) continue;
        if (stride[d] <= reach || stride[d] > INT64_MAX / 4 / n[d]) return false;
        reach += (n[d] - 1) * stride[d];
    }
    return true;
}

int check_fp8(int dtype, int64_t B, int64_t R, int64_t K, int block, const void* A, int64_t lda, bool transpose,
              const void* e, int64_t lde, int64_t stridee, const void* s, int64_t row, int64_t blk, int64_t mat) {
    if (source(dtype) < 0) return abi_failf(SSG_ERR_DTYPE, "element type %d", dtype);
    if (block != 1 && block != ssg::kFp8Block) return abi_failf(SSG_ERR_FORMAT, "%d rows to a scale (1 or 128)", block);
    if (B < 0 || R < 0 || K < 0 || B >= (1 << 20) || R >= kMaxDim || K >= kMaxDim)
        return abi_failf(SSG_ERR_SHAPE, "size B=%lld R=%lld K=%lld", (ll)B, (ll)R, (ll)K);
    const int64_t er = transpose ? K : R, ec = transpose ? R : K;
    int rc;
    if ((rc = check_mat("the matrix", A, B * R, K, lda)) || (rc = check_mat("elems", e, B * er, ec, lde)) ||
        (rc = check_scales("scales", s, B * er, ec, row, blk)))
        return rc;
    const int64_t rows = block == 1 ? er : blocks(er);
    if (!apart({B, rows, blocks(ec)}, {mat, row, blk}))
        return abi_failf(SSG_ERR_STRIDE, "scales overlap: strides %lld, %lld, %lld", (ll)mat, (ll)row, (ll)blk);
    if (!apart({B, er, ec}, {stridee, lde, 1}))
        return abi_failf(SSG_ERR_STRIDE, "elems overlap: strides %lld, %lld", (ll)stridee, (ll)lde);
    // workgroups of a launch are counted in 32 bits
    if (B > 0 && blocks(R) > 0 && blocks(K) * ((R + 15) / 16) > 0xffffffffLL / B)
        return abi_failf(SSG_ERR_SHAPE, "size too large: B=%lld R=%lld K=%lld", (ll)B, (ll)R, (ll)K);
    return SSG_OK;
}

// ------------------------------------------------------------------ the products

struct Call {
    MmFp8Args a;
    int x;                             // type of X
    int64_t ldx;                       // bytes
};

int mm_args(int x, int y, int64_t E, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const float* xs, int64_t xsr,
            int64_t xsk, const uint8_t* W, int64_t ldw, int64_t stridew, int wblock, const float* wsc, int64_t wsr,
            int64_t wsk, int64_t strides, const int32_t* offs, bool grouped, Call* out) {
    if (x != SSG_E4M3 && source(x) < 0) return abi_failf(SSG_ERR_DTYPE, "activations of type %d", x);
    if (source(y) < 0) return abi_failf(SSG_ERR_DTYPE, "output of type %d", y);
    if (wblock != 1 && wblock != ssg::kFp8Block) return abi_failf(SSG_ERR_FORMAT, "%d rows to a scale (1 or 128)", wblock);
    if (E < 0 || M < 0 || N < 0 || K < 0)
        return abi_failf(SSG_ERR_SHAPE, "negative size E=%lld M=%lld N=%lld K=%lld", (ll)E, (ll)M, (ll)N, (ll)K);
    if (E >= (1 << 20) || M >= kMaxDim || N >= kMaxDim || K >= kMaxDim)
        return abi_failf(SSG_ERR_SHAPE, "size too large: E=%lld M=%lld N=%lld K=%lld", (ll)E, (ll)M, (ll)N, (ll)K);
    const int64_t xb = x == SSG_E4M3 ? 1 : float_bytes(x);
    int rc;
    if ((rc = check_mat("X", X, N, K, ldx)) || (rc = check_mat("W", W, E * M, K, ldw))) return rc;
    // a tile's rows are addressed with 31 bits
    if (ldx * xb >= (int64_t)1 << 22) return abi_failf(SSG_ERR_STRIDE, "rows of X are 2^22 bytes apart or more");
    if (ldw >= (int64_t)1 << 22) return abi_failf(SSG_ERR_STRIDE, "rows of W are 2^22 bytes apart or more");
    if (x == SSG_E4M3) {
        if ((rc = check_scales("xscales", xs, N, K, xsr, xsk))) return rc;
    } else if (xs) {
        return abi_failf(SSG_ERR_FORMAT, "xscales with activations that are not e4m3");
    }
    if ((rc = check_scales("wscales", wsc, E * M, K, wsr, wsk))) return rc;
    if (grouped && !offs) return abi_failf(SSG_ERR_NULL, "offs is NULL");
    Call c{};
    ssg::MmArgs& m = c.a.m;
    m.mode = ssg::MM_FP8;
    m.Q = M; m.P = N; m.C = K;
    m.q = W; m.ldq = ldw; m.strideq = stridew;
    m.p = (const uint8_t*)X; m.ldp = ldx * xb;
    m.E = E; m.offs = grouped ? offs : nullptr;
    m.splits = 1;
    c.a.w = {wsc, wsr, wsk, strides};
    c.a.x = {xs, xsr, xsk, 0};
    c.a.w_rows = wblock == 1 && M > 1;
    c.a.x_src = -1;
    m.out = y == SSG_F32 ? ssg::OUT_F32 : y == SSG_F16 ? ssg::OUT_F16 : ssg::OUT_BF16;
    c.x = x;
    *out = c;
    return SSG_OK;
}

// ------------------------------------------------------------------ the choice of kernel
//
// Times in us of the launches that a plan would make, from what they measured on
// this chip.  Every kernel handles every product it can be chosen for, so a wrong
// estimate costs time only.  Over 17014 random products with 16-bit outputs (dense and
// of 2 to 64 experts, 128 .. 16384 weight rows, lengths of 256 to 12288, 100 .. 8192
// tokens), the kernels of few rows and the tiles timed, the choice is 2.4% slower than
// the best in the geometric mean; over 25272 of 1 .. 300 tokens, 128 .. 160000 weight rows
// and both widths of output, 3.8%; in both not at all in the median.

struct Plan {
    bool fits;                         // every launch has fewer than 2^32 threads
    bool few;
    int rt, nt, size, splits;
    bool round, copy_q, copy_p, planes_q, planes_p;
    int64_t at_x, ldx, at_xs, xplane, at_q, ldq, at_p, ldp, at_ws, wplane, at_part;
    size_t bytes;
};

// Few rows: 16 rt weight rows x 16 nt tokens a workgroup.  One round of the chip
// takes start + length / 1024 * first; a further one, and (several workgroups share a
// CU) the part `second` of one more, `each` + length / 4096 * more.  Fitted to 15768
// products of up to 300 tokens: 1.8% slower than the best of the six.
struct FewShape {
    int rt, nt;
    double first, each, more, second;
};
constexpr FewShape kFew[6] = {{1, 1, 0.77, 0.56, 2.96, 0.40}, {2, 1, 1.27, 0.75, 4.58, 0.63},
                              {4, 1, 2.39, 1.30, 8.79, 0.73}, {1, 2, 1.00, 0.85, 3.37, 0.44},
                              {2, 2, 1.63, 1.28, 5.63, 0.51}, {4, 2, 3.01, 3.08, 11.4, 0.69}};
// Those that round their activations.  The others leave that to a launch before.
constexpr FewShape kRounding[2] = {{1, 1, 1.05, 0.95, 1.71, 0.66}, {2, 1, 1.64, 1.07, 4.18, 0.69}};
constexpr double kStart = 3.2, kRoundLaunch = 2.4;
// Weights from memory; of tiles with one workgroup on a CU.
constexpr double kBytesPerUs = 5.2e6, kBytesPerUsAlone = 4.2e6;

// Tiles: a block of the contraction takes `one` us where a CU has one workgroup, `two`
// where it has two (128 x 128, two on a CU).
constexpr double kPairOne = 1.25, kPairTwo = 1.9;
// 256 x 256, 16-bit outputs: a whole round, and a last one of tiles as they are, cut in
// two and in four.
constexpr double kLarge[3] = {3.1, 1.9, 1.35};

Plan plan(const Call& c) {
    const ssg::MmArgs& m = c.a.m;
    Plan p{};
    p.splits = 1;
    p.nt = p.rt = 1;
    // experts that have rows, if rows choose them at random, and their rows
    const double E = m.offs ? std::max<double>(1, (double)m.E) : 1;
    const double busy = m.offs ? std::max(1.0, E * (1 - std::exp(-(double)m.P / E))) : 1;
    const double avg = (double)m.P / busy;
    const int64_t nb = blocks(m.C);
    auto row_tiles = [&](int t) {
        if (!m.offs || E == 1) return (double)((m.P + t - 1) / t);
        return busy * std::max(1.0, avg / t + 0.6);
    };
    auto ceil_div = [](int64_t n, int64_t d) { return (double)((n + d - 1) / d); };
    const double length = (double)m.C, bytes = busy * (double)m.Q * (double)m.C;
    const bool may_round = (c.x == SSG_F16 || c.x == SSG_BF16) && m.P <= ssg::kFp8RoundTokens &&
                           m.P * nb * ssg::kFp8Block <= ssg::kFp8RoundBytes;
    const double launch = c.x != SSG_E4M3 ? kRoundLaunch : 0;
    double best = 1e30;
    if (avg <= 300) {
        for (int i = 0; i < 6; ++i) {
            const bool rounds_x = may_round && i < 2;
            const FewShape& f = rounds_x ? kRounding[i] : kFew[i];
            if (c.a.w_rows && f.rt > 1) continue;      // (not built)
            if (ceil_div(m.Q, 16 * f.rt) * (double)ssg::mm_tile_bound(m, 16 * f.nt) >= (1 << 23)) continue;
            const double rounds = ceil_div(m.Q, 16 * f.rt) * row_tiles(16 * f.nt) / kCUs;
            const double more = rounds <= 1 ? 0 : rounds - 1 + f.second;
            const double us = (rounds_x ? 0 : launch) + kStart +
                              std::max(bytes / kBytesPerUs,
                                       length / 1024 * f.first + more * (f.each + length / 4096 * f.more));
            if (us < best) {
                best = us;
                p.few = true;
                p.rt = f.rt;
                p.nt = f.nt;
            }
        }
    }
    // (fp32 outputs, and a scale for each weight row: 128 x 128)
    for (int size = m.out == ssg::OUT_F32 || c.a.w_rows ? 1 : 0; size <= 1; ++size) {
        const int tp = size == 0 ? 256 : 128, tq = tp;
        const double tiles = row_tiles(tp) * ceil_div(m.Q, tq);
        for (int splits = 1; splits <= 8; splits *= 2) {
            if (splits > 1 && (size == 0 || nb < 2 * splits)) break;
            if (ceil_div(m.Q, tq) * (double)ssg::mm_tile_bound(m, tp) * splits >= (1 << 23) - kCUs) break;
            const double n = tiles * splits, len = std::ceil((double)nb / splits);
            double block;
            if (size == 0) {
                const double whole = std::floor(n / kCUs), rest = n - whole * kCUs;
                block = whole * kLarge[0] + (rest <= 0           ? 0
                                             : rest <= kCUs / 4 ? kLarge[2]
                                             : rest <= kCUs / 2 ? kLarge[1]
                                                                : kLarge[0]);
            } else {
                const double r = std::ceil(n / kCUs), pairs = std::floor(r / 2);
                block = pairs * kPairTwo + (r - 2 * pairs) * kPairOne;
            }
            double us = launch + kStart +
                        std::max(bytes / (n <= kCUs ? kBytesPerUsAlone : kBytesPerUs), 0.8 + block * len);
            if (splits > 1) us += 3 + (double)splits * m.P * m.Q * 14 / 3e6;
            if (us < best) {
                best = us;
                p.few = false;
                p.size = size;
                p.splits = splits;
            }
        }
    }
    // (more tiles than a launch holds, of every size; the sizes of copies are then not computed)
    p.fits = best < 1e30;
    if (!p.fits) return p;
    int64_t at = 0;
    auto take = [&](int64_t n) {
        const int64_t r = at;
        at += up(n, 256);
        return r;
    };
    const bool in_kernel = p.few && p.rt <= 2 && p.nt == 1 && may_round;
    p.round = c.x != SSG_E4M3 && !in_kernel;
    if (p.round) {
        p.ldx = up(m.C, 16);
        p.xplane = up(m.P, 4);
        p.at_x = take(m.P * p.ldx);
        p.at_xs = take(nb * p.xplane * 4);
    }
    if (!p.few) {
        // tiles load rows 16 bytes at a time from any dword
        p.copy_q = !al(m.q, 4) || m.ldq % 4 || (m.E > 1 && m.strideq % 4);
        p.copy_p = !p.round && (!al(m.p, 4) || m.ldp % 4);
        p.planes_q = c.a.w_rows && c.a.w.row != 1;
        p.planes_p = !p.round && c.a.x.row != 1 && m.P > 1;
        if (p.copy_q) {
            p.ldq = up(m.C, 16);
            p.at_q = take(m.E * m.Q * p.ldq);
        }
        if (p.copy_p) {
            p.ldp = up(m.C, 16);
            p.at_p = take(m.P * p.ldp);
        }
        if (p.planes_q) {
            p.wplane = up(m.Q, 4);
            p.at_ws = take(m.E * nb * p.wplane * 4);
        }
        if (p.planes_p) {
            p.xplane = up(m.P, 4);
            p.at_xs = take(nb * p.xplane * 4);
        }
    }
    if (p.splits > 1) p.at_part = take((int64_t)p.splits * m.P * m.Q * 4);
    p.fits &= !p.round || nb * ((m.P + 15) / 16) <= 0xffffffffLL;
    p.fits &= !p.planes_q || m.E * nb * p.wplane < (int64_t)1 << 32;
    p.fits &= !p.planes_p || nb * p.xplane < (int64_t)1 << 32;
    p.bytes = p.fits ? (size_t)at : 0;
    return p;
}

int too_large(const Call& c) {
    const ssg::MmArgs& m = c.a.m;
    return abi_failf(SSG_ERR_SHAPE, "size too large: E=%lld M=%lld N=%lld K=%lld", (ll)m.E, (ll)m.Q, (ll)m.P, (ll)m.C);
}

int run(Call c, void* ws, size_t ws_bytes, hipStream_t s) {
    ssg::MmArgs& m = c.a.m;
    if (m.P == 0 || m.Q == 0) return SSG_OK;
    const Plan p = plan(c);
    if (!p.fits) return too_large(c);
    if (p.bytes > 0) {
        if (!ws && ws_bytes == SSG_WS_ASK) return SSG_ERR_WORKSPACE;
        if (!ws || ws_bytes < p.bytes)
            return abi_failf(SSG_ERR_WORKSPACE, "workspace %zu < %zu bytes", ws ? ws_bytes : (size_t)0, p.bytes);
        if (!al(ws, 16)) return abi_failf(SSG_ERR_WORKSPACE, "workspace must be 16-byte aligned");
    }
    uint8_t* const w = (uint8_t*)ws;
    const int64_t nb = blocks(m.C);
    hipError_t e = hipSuccess;
    m.splits = p.splits;
    if (p.splits > 1) m.part = (float*)(w + p.at_part);
    if (p.round) {
        if (m.C > 0) {
            Fp8Matrix q{};
            q.type = source(c.x);
            q.mats = 1; q.R = m.P; q.K = m.C;
            q.a = m.p; q.lda = m.ldp / float_bytes(c.x);
            q.block = 1;
            q.e = w + p.at_x; q.lde = p.ldx;
            q.s = (float*)(w + p.at_xs); q.row = 1; q.blk = p.xplane;
            e = ssg::launch_fp8_quantize(q, s);
        }
        m.p = w + p.at_x;
        m.ldp = p.ldx;
        c.a.x = {(const float*)(w + p.at_xs), 1, p.xplane, 0};
    } else if (c.x != SSG_E4M3) {
        c.a.x_src = source(c.x);
    }
    if (p.few) {
        if (e == hipSuccess) e = ssg::launch_mm_fp8_few(c.a, p.rt, p.nt, s);
    } else {
        if (p.copy_q && e == hipSuccess) {
            e = ssg::launch_mm_repack(m.q, m.E, m.strideq, m.Q, m.C, m.ldq, w + p.at_q, p.ldq, 0, m.offs, s);
            m.q = w + p.at_q;
            m.ldq = p.ldq;
            m.strideq = m.Q * p.ldq;
        }
        if (p.copy_p && e == hipSuccess) {
            e = ssg::launch_mm_repack(m.p, 1, 0, m.P, m.C, m.ldp, w + p.at_p, p.ldp, 0, nullptr, s);
            m.p = w + p.at_p;
            m.ldp = p.ldp;
        }
        if (p.planes_q && e == hipSuccess) {
            e = ssg::launch_fp8_planes(c.a.w, m.E, m.Q, nb, (float*)(w + p.at_ws), p.wplane, s);
            c.a.w = {(const float*)(w + p.at_ws), 1, p.wplane, nb * p.wplane};
        }
        if (p.planes_p && e == hipSuccess) {
            e = ssg::launch_fp8_planes(c.a.x, 1, m.P, nb, (float*)(w + p.at_xs), p.xplane, s);
            c.a.x = {(const float*)(w + p.at_xs), 1, p.xplane, 0};
        }
        if (e == hipSuccess) e = ssg::launch_mm_fp8_tiles(c.a, p.size, s);
    }
    if (e == hipSuccess && p.splits > 1) e = ssg::launch_mm_reduce(m, s);
    return hip_status(e);
}

int check_y(const void* Y, int64_t N, int64_t M, int64_t ldy, Call* c) {
    const int rc = check_mat("Y", Y, N, M, ldy);
    if (rc) return rc;
    c->a.m.y = const_cast<void*>(Y);
    c->a.m.ldy = ldy;
    return SSG_OK;
}

size_t bytes_of(int rc, const Call& c) { return rc || c.a.m.P == 0 || c.a.m.Q == 0 ? 0 : plan(c).bytes; }

}  // namespace

extern "C" {

int64_t ssg_fp8_scale_cols(int64_t K) { return blocks(K); }

int ssg_fp8_quantize(int dtype, int64_t B, int64_t R, int64_t K, const void* A, int64_t lda, int64_t stridea, int block,
                     int transpose, uint8_t* elems, int64_t lde, int64_t stridee, float* scales, int64_t row,
                     int64_t blk, int64_t strides, void* stream) {
    const int rc = check_fp8(dtype, B, R, K, block, A, lda, transpose != 0, elems, lde, stridee, scales, row,
                             blk, strides);
    if (rc || B == 0 || R == 0 || K == 0) return rc;
    Fp8Matrix a{source(dtype), B, R, K, A, lda, stridea, block, transpose != 0, elems, lde, stridee, scales, row, blk, strides};
    return hip_status(ssg::launch_fp8_quantize(a, (hipStream_t)stream));
}

int ssg_fp8_dequantize(int dtype, int64_t B, int64_t R, int64_t K, const uint8_t* elems, int64_t lde, int64_t stridee,
                       int block, const float* scales, int64_t row, int64_t blk, int64_t strides, void* D, int64_t ldd,
                       int64_t strided, void* stream) {
    if (source(dtype) < 0) return abi_failf(SSG_ERR_DTYPE, "element type %d", dtype);
    if (block != 1 && block != ssg::kFp8Block) return abi_failf(SSG_ERR_FORMAT, "%d rows to a scale (1 or 128)", block);
    if (B < 0 || R < 0 || K < 0 || B >= (1 << 20) || R >= kMaxDim || K >= kMaxDim)
        return abi_failf(SSG_ERR_SHAPE, "size B=%lld R=%lld K=%lld", (ll)B, (ll)R, (ll)K);
    int rc;
    if ((rc = check_mat("elems", elems, B * R, K, lde)) || (rc = check_scales("scales", scales, B * R, K, row, blk)) ||
        (rc = check_mat("D", D, B * R, K, ldd)))
        return rc;
    if (B == 0 || R == 0 || K == 0) return SSG_OK;
    if (!apart({B, R, K}, {strided, ldd, 1}))
        return abi_failf(SSG_ERR_STRIDE, "D overlaps: strides %lld, %lld", (ll)strided, (ll)ldd);
    Fp8Matrix a{source(dtype), B, R, K, D, ldd, strided, block, false, const_cast<uint8_t*>(elems), lde, stridee,
                const_cast<float*>(scales), row, blk, strides};
    return hip_status(ssg::launch_fp8_dequantize(a, (hipStream_t)stream));
}

size_t ssg_mm_fp8_workspace_bytes(int x, int y, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx,
                                  const float* xs, int64_t xsr, int64_t xsk, const uint8_t* W, int64_t ldw, int wblock, const float* wsc,
                                  int64_t wsr, int64_t wsk) {
    Call c{};
    return bytes_of(mm_args(x, y, 1, M, N, K, X, ldx, xs, xsr, xsk, W, ldw, 0, wblock, wsc, wsr, wsk, 0, nullptr, false, &c), c);
}

int ssg_mm_fp8(int x, int y, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const float* xs, int64_t xsr,
               int64_t xsk, const uint8_t* W, int64_t ldw, int wblock, const float* wsc, int64_t wsr, int64_t wsk,
               void* Y, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
    Call c{};
    int rc = mm_args(x, y, 1, M, N, K, X, ldx, xs, xsr, xsk, W, ldw, 0, wblock, wsc, wsr, wsk, 0, nullptr, false, &c);
    if (rc || (rc = check_y(Y, N, M, ldy, &c))) return rc;
    return run(c, ws, ws_bytes, (hipStream_t)stream);
}

size_t ssg_grouped_mm_fp8_workspace_bytes(int x, int y, int64_t E, int64_t M, int64_t N, int64_t K, const void* X,
                                          int64_t ldx, const float* xs, int64_t xsr, int64_t xsk, const uint8_t* W, int64_t ldw,
                                          int64_t stridew, int wblock, const float* wsc, int64_t wsr, int64_t wsk,
                                          int64_t strides, const int32_t* offs) {
    Call c{};
    return bytes_of(mm_args(x, y, E, M, N, K, X, ldx, xs, xsr, xsk, W, ldw, stridew, wblock, wsc, wsr, wsk, strides, offs, true, &c), c);
}

int ssg_grouped_mm_fp8(int x, int y, int64_t E, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx,
                       const float* xs, int64_t xsr, int64_t xsk, const uint8_t* W, int64_t ldw, int64_t stridew,
                       int wblock, const float* wsc, int64_t wsr, int64_t wsk, int64_t strides, const int32_t* offs,
                       void* Y, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
    Call c{};
    int rc = mm_args(x, y, E, M, N, K, X, ldx, xs, xsr, xsk, W, ldw, stridew, wblock, wsc, wsr, wsk, strides, offs, true, &c);
    if (rc || (rc = check_y(Y, N, M, ldy, &c))) return rc;
    return run(c, ws, ws_bytes, (hipStream_t)stream);
}

int ssg_mm_fp8_select_kernel(int x, int y, int wblock, int64_t E, int64_t M, int64_t N, int64_t K, int64_t kernel[4]) {
    if (!kernel) return abi_failf(SSG_ERR_NULL, "kernel is NULL");
    // an address at a 16-byte border stands for every operand; nothing reads it
    void* const p = reinterpret_cast<void*>((uintptr_t)256);
    const bool grouped = E > 0;
    const int64_t ld = up(K, 16), nb = blocks(K), rows = wblock == 1 ? M : blocks(M);
    Call c{};
    const int rc = mm_args(x, y, grouped ? E : 1, M, N, K, p, ld, x == SSG_E4M3 ? (float*)p : nullptr, 1, up(N, 4),
                           (uint8_t*)p, ld, M * ld, wblock, (float*)p, wblock == 1 ? 1 : nb, wblock == 1 ? up(M, 4) : 1,
                           rows * nb, (int32_t*)p, grouped, &c);
    if (rc) return rc;
    const Plan q = plan(c);
    if (!q.fits) return too_large(c);
    kernel[0] = q.few ? 0 : 1;
    kernel[1] = q.few ? 16 * q.rt : q.size == 0 ? 256 : 128;
    kernel[2] = q.few ? 16 * q.nt : q.size == 0 ? 256 : 128;
    kernel[3] = q.splits;
    return SSG_OK;
}

}  // extern "C"
