// mm_abi.cpp -- the C ABI of the mx4 format and of the dense and grouped
// matrix products: host-side checks, the choice of kernel, and the workspace
// (partials of a split contraction, operands repacked into aligned rows).
#include "ssgemm.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "mm_args.hpp"
#include "ssg_abi.hpp"

namespace {

using ssg::MmArgs;

int fail(int status, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return ssg::abi_fail(status, buf);
}

int hip_status(hipError_t e, const char* what) {
    return e == hipSuccess ? SSG_OK : fail(SSG_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

typedef long long ll;

constexpr int64_t kMaxDim = (int64_t)1 << 29;   // rows: three scale planes are addressed with 31 bits
constexpr int kCUs = 256;

bool al(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
int64_t blocks(int64_t K) { return (K + ssg::kMxBlock - 1) / ssg::kMxBlock; }

bool float16_type(int dt) { return dt == SSG_F16 || dt == SSG_BF16; }
int64_t float_bytes(int dt) { return dt == SSG_F32 ? 4 : 2; }
int to_dt(int dt) { return dt == SSG_F16 ? ssg::DT_F16 : ssg::DT_BF16; }
int to_out(int dt) { return dt == SSG_F32 ? ssg::OUT_F32 : dt == SSG_F16 ? ssg::OUT_F16 : ssg::OUT_BF16; }

// ------------------------------------------------------------------ the choice of kernel
//
// Times in us of the launches that a plan would make, from what they measured
// on this chip: a workgroup's time on its CU times the workgroups a CU gets,
// but no less than the weights take from memory.  Every kernel handles every
// product it can be chosen for, so a wrong estimate costs time only.  Over 250
// random products of each kind (1 .. 64 experts, 64 .. 16384 rows, contractions
// of 64 .. 12288, 1 .. 8192 tokens), all kernels timed, the choice is 2 to 3%
// (gradients of the rows: 1%) slower than the best one in the geometric mean.

constexpr double kBytesPerUs = 5.2e6, kCopyBytesPerUs = 4.5e6;

// Skinny: 16 rt weight rows (rt = 1 .. 4) x 16 nt tokens a workgroup of a
// 4096-long contraction, by operand types (16-bit, mx4 x mx4, mx4 x 16-bit) and
// nt; 0: not built.  Measured at 4096 and 11008 x 4096 with 16 and 32 tokens
// (fp16 x mx4 at 11008 x 4096 x 16: 21, 19, 13, 15 us for rt = 1 .. 4; at 4096 x
// 4096: 10, 12, 13, 14); 16-bit weights with rt > 1 are priced up to where many
// workgroups measured (11008 x 4096 x 16: 30, 33, -, 32 us).
constexpr double kSkinnyUs[3][2][4] = {{{8.4, 19.0, 0, 36.0}, {13.0, 16.0, 0, 27.0}},
                                       {{4.4, 4.7, 6.0, 6.8}, {6.0, 6.5, 0, 8.0}},
                                       {{6.0, 7.8, 9.2, 10.3}, {10.6, 11.9, 0, 14.1}}};

// The same for other lengths, in parts of it: the start, and the rest by
// length / 4096.  Workgroups that share their scales (rt >= 3) start once for
// every 4096 elements.
struct SkinnyShape {
    double start, length, shared_start, shared_length;
};
constexpr SkinnyShape kSkinnyShape[3] = {{0.2, 0.7, 0, 0}, {0.3, 0.9, 0.9, 0.45}, {0.1, 0.7, 0.7, 0.2}};

struct Plan {
    bool skinny;
    int rt, nt;                        // skinny: 16-row groups of weights and tokens
    int size, splits;                  // tiles
    bool copy_q, copy_p, copy_s;
    int64_t at_q, at_p, at_qs, at_ps, at_part;   // workspace offsets
    int64_t ldq, ldp, lds, plane_q, plane_p;     // strides of the copies and the scale planes
    size_t bytes;
};

// Rows and row bytes of an operand as stored.
int64_t q_rows(const MmArgs& a) { return a.pt ? a.C : a.qt ? a.C : a.Q; }
int64_t q_bytes(const MmArgs& a) {
    if (a.mode != ssg::MM_16) return blocks(a.C) * 16;
    return (a.qt ? a.Q : a.C) * 2;
}
int64_t p_rows(const MmArgs& a) { return a.pt ? a.C : a.P; }
int64_t p_bytes(const MmArgs& a) {
    if (a.mode == ssg::MM_MX4) return blocks(a.C) * 16;
    return (a.pt ? a.P : a.C) * 2;
}
int64_t q_mats(const MmArgs& a) { return a.pt ? 1 : a.E; }   // (E is 1 without offsets)

Plan plan(const MmArgs& a) {
    Plan p{};
    p.splits = 1;
    // experts that have rows, if rows choose them at random, and their rows
    const double E = a.offs ? std::max<double>(1, (double)a.E) : 1;
    const double busy = a.offs && !a.pt ? std::max(1.0, E * (1 - std::exp(-(double)a.P / E))) : 1;
    const double avg = (double)a.P / busy;
    auto row_tiles = [&](int t) {
        if (a.pt) return (double)((a.P + t - 1) / t) * E;
        if (!a.offs || E == 1) return (double)((a.P + t - 1) / t);
        return busy * std::max(1.0, avg / t + 0.6);
    };
    auto ceil_div = [](int64_t n, int64_t d) { return (double)((n + d - 1) / d); };
    const double bytes = a.pt ? 0 : busy * (double)a.Q * (double)a.C * (a.mode == ssg::MM_16 ? 2 : 0.53);
    const double floor_us = bytes / kBytesPerUs;
    const int64_t qb = q_bytes(a), pb = p_bytes(a), nb = blocks(a.C);
    // Tiles load rows 16 bytes at a time.  16-bit operands may begin at any dword
    // (an odd contraction length ends inside one); others at 16 bytes.  The
    // kernel finds the end of transposed rows of part chunks with 31 bits.
    const int64_t q_al = a.mode != ssg::MM_16 ? 16 : a.qt || a.C % 2 == 0 ? 4 : 0;
    const int64_t p_al = a.mode != ssg::MM_16 ? 16 : a.pt || a.C % 2 == 0 ? 4 : 0;
    auto far = [](int64_t rows, int64_t ld) { return rows * ld >= (int64_t)1 << 31; };
    p.copy_q = q_al == 0 || (qb % 16 && (q_al == 16 || (a.qt && far(q_rows(a), a.ldq)))) || !al(a.q, q_al) ||
               a.ldq % q_al || a.strideq % q_al;
    p.copy_p = p_al == 0 || (pb % 16 && (p_al == 16 || (a.pt && far(p_rows(a), a.ldp)))) || !al(a.p, p_al) ||
               a.ldp % p_al;
    const double copies = (p.copy_q ? 4 + 2 * bytes / kCopyBytesPerUs : 0) +
                          (p.copy_p ? 4 + 2 * (double)p_rows(a) * (double)pb / kCopyBytesPerUs : 0);
    double best = 1e30;
    if (!a.qt && !a.pt && avg <= 160) {
        for (int nt = 1; nt <= (avg > 16 ? 2 : 1); ++nt)
            for (int rt = 1; rt <= 4; ++rt) {
                const double full = kSkinnyUs[a.mode][nt - 1][rt - 1];
                if (full == 0) continue;
                const double wgs = ceil_div(a.Q, 16 * rt) * row_tiles(16 * nt);
                const double fill = std::min(1.0, avg / (16 * nt));   // tokens of a tile that exist
                const bool shared = rt >= 3 && a.mode != ssg::MM_16;  // scales through LDS, 4096 elements a round
                const SkinnyShape& h = kSkinnyShape[a.mode];
                auto one = [&](int64_t C) {
                    const double len = (double)C / 4096;
                    const double parts = shared ? h.shared_start * std::ceil(len) + h.shared_length * len
                                                : h.start + h.length * len;
                    return full * parts * (0.7 + 0.3 * fill);
                };
                const double more = std::max(0.0, std::ceil(wgs / kCUs) - 1) * 0.8;
                const double us = 3.5 + std::max((1 + more) * one(a.C), floor_us);
                if (us < best) {
                    best = us;
                    p.skinny = true;
                    p.nt = nt;
                    p.rt = rt;
                    p.splits = 1;
                }
                // few rows of long weights: several workgroups a row, each with
                // at least one step a wave (shared scales: one round)
                const int64_t unit = shared ? 4096 : 8 * (a.mode == ssg::MM_MX4 ? 256 : 128);
                for (int splits = 2; splits <= 8 && unit * splits <= a.C && wgs * splits <= kCUs; splits *= 2) {
                    const int64_t rounds = (a.C + unit - 1) / unit;
                    const double us2 = 3.5 + std::max(one((rounds + splits - 1) / splits * unit), floor_us) + 8 +
                                       (double)splits * a.P * a.Q * 8 / 3e6;
                    if (us2 >= best) continue;
                    best = us2;
                    p.skinny = true;
                    p.nt = nt;
                    p.rt = rt;
                    p.splits = splits;
                }
            }
    }
    // Tiles: a stage takes as long as its products at the rate of a full chip
    // (smaller tiles for a last round of at most half, and less for one that
    // leaves CUs idle), or its latency.  A split adds the pass over its partials.
    const int64_t stages = (a.pt ? (int64_t)((double)a.C / E) : a.C) / (a.mode == ssg::MM_MX4 ? 128 : 32) + 1;
    for (int k = 0; k < 3; ++k) {
        const ssg::MmTileSize& t = ssg::kMmTileSizes[k];
        const double tiles = row_tiles(t.p) * ceil_div(a.Q, t.q);
        const double stage = t.q * t.p * (a.mode == ssg::MM_MX4 ? 1.3 : 1.1) / t.rate / 78000;
        for (int splits = 1; splits <= 8; splits *= 2) {
            if (splits > 1 && (a.pt || k == 0 || stages / splits < 8)) break;
            const double n = tiles * splits, whole = std::floor(n / kCUs), rest = n - whole * kCUs;
            double us;
            if (k == 0) {
                const double cut = rest <= 0           ? 0
                                   : rest <= kCUs / 4 ? 0.3
                                   : rest <= kCUs / 2 ? 0.55
                                                      : 0.35 + 0.65 * rest / kCUs;
                us = (whole * stage + (cut > 0 ? std::max(t.latency, cut * stage) : 0)) * stages;
            } else {
                const double m = n <= kCUs ? 1 : n / kCUs + 0.25;
                us = std::max(t.latency * std::ceil(m / t.per_cu), m * stage) * (double)(stages / splits);
            }
            us = 6.5 + std::max(us, floor_us) + copies;
            if (splits > 1) us += 4 + (double)splits * a.P * a.Q * 8 / 3e6;
            if (a.mode == ssg::MM_MX4) us += 5;   // the scale planes
            if (us < best) {
                best = us;
                p.skinny = false;
                p.size = k;
                p.splits = splits;
            }
        }
    }
    if (p.skinny) {
        if (p.splits > 1) p.bytes = (size_t)((int64_t)p.splits * a.P * a.Q * 4);
        return p;
    }
    int64_t at = 0;
    auto take = [&](int64_t n) {
        const int64_t r = at;
        at += up(n, 256);
        return r;
    };
    if (p.copy_q) {
        p.ldq = up(qb, 16);
        p.at_q = take(q_mats(a) * q_rows(a) * p.ldq);
    }
    if (p.copy_p) {
        p.ldp = up(pb, 16);
        p.at_p = take(p_rows(a) * p.ldp);
    }
    // scales against 16-bit activations: whole dwords
    if (a.mode == ssg::MM_W4 && (nb % 4 || !al(a.qs, 4) || a.ldqs % 4 || a.strideqs % 4)) {
        p.copy_s = true;
        p.lds = up(nb, 16);
        p.at_qs = take(a.E * a.Q * p.lds);
    }
    // scale planes, padded so that the last tile's pieces stay inside
    if (a.mode == ssg::MM_MX4) {
        p.plane_q = up(a.Q, 256);
        p.at_qs = take(a.E * up(nb, 4) * p.plane_q);
        p.plane_p = up(a.P, 16) + 256;
        p.at_ps = take(up(nb, 4) * p.plane_p);
    }
    if (p.splits > 1) p.at_part = take((int64_t)p.splits * a.P * a.Q * 4);
    p.bytes = (size_t)at;
    return p;
}

int run(MmArgs a, void* ws, size_t ws_bytes, hipStream_t s) {
    if (a.P == 0 || a.Q == 0 || (a.pt && a.E == 0)) return SSG_OK;
    const Plan p = plan(a);
    if (p.bytes > 0) {
        if (!ws && ws_bytes == SSG_WS_ASK) return SSG_ERR_WORKSPACE;
        if (!ws || ws_bytes < p.bytes)
            return fail(SSG_ERR_WORKSPACE, "workspace %zu < %zu bytes", ws ? ws_bytes : (size_t)0, p.bytes);
        if (!al(ws, 16)) return fail(SSG_ERR_WORKSPACE, "workspace must be 16-byte aligned");
    }
    uint8_t* const w = (uint8_t*)ws;
    hipError_t e = hipSuccess;
    a.splits = p.splits;
    if (p.skinny) {
        if (p.splits > 1) a.part = (float*)w;
        e = ssg::launch_mm_skinny(a, p.rt, p.nt, s);
        if (e == hipSuccess && p.splits > 1) e = ssg::launch_mm_reduce(a, s);
        return hip_status(e, "kernel launch");
    }
    if (p.copy_q) {
        e = ssg::launch_mm_repack(a.q, q_mats(a), a.strideq, q_rows(a), q_bytes(a), a.ldq, w + p.at_q, p.ldq, 0,
                                  a.pt ? nullptr : a.offs, s);
        a.q = w + p.at_q;
        a.ldq = p.ldq;
        a.strideq = q_rows(a) * p.ldq;
    }
    if (p.copy_p && e == hipSuccess) {
        e = ssg::launch_mm_repack(a.p, 1, 0, p_rows(a), p_bytes(a), a.ldp, w + p.at_p, p.ldp, 0, nullptr, s);
        a.p = w + p.at_p;
        a.ldp = p.ldp;
    }
    if (p.copy_s && e == hipSuccess) {
        // past the row's blocks: 1.0, for elements that are zero
        e = ssg::launch_mm_repack(a.qs, a.E, a.strideqs, a.Q, blocks(a.C), a.ldqs, w + p.at_qs, p.lds, 127, a.offs, s);
        a.qs = w + p.at_qs;
        a.ldqs = p.lds;
        a.strideqs = a.Q * p.lds;
    }
    if (a.mode == ssg::MM_MX4 && e == hipSuccess) {
        const int64_t nb = blocks(a.C);
        e = ssg::launch_mm_planes({a.qs, a.E, a.strideqs, a.Q, nb, a.ldqs, w + p.at_qs, p.plane_q},
                                  {a.ps, 1, 0, a.P, nb, a.ldps, w + p.at_ps, p.plane_p}, s);
        a.qs = w + p.at_qs;
        a.ldqs = p.plane_q;
        a.strideqs = up(nb, 4) * p.plane_q;
        a.ps = w + p.at_ps;
        a.ldps = p.plane_p;
    }
    if (p.splits > 1) a.part = (float*)(w + p.at_part);
    if (e == hipSuccess) e = ssg::launch_mm_tiles(a, p.size, s);
    if (e == hipSuccess && p.splits > 1) e = ssg::launch_mm_reduce(a, s);
    return hip_status(e, "kernel launch");
}

// ------------------------------------------------------------------ checks

int check_sizes(int64_t E, int64_t M, int64_t N, int64_t K) {
    if (E < 0 || M < 0 || N < 0 || K < 0)
        return fail(SSG_ERR_SHAPE, "negative size E=%lld M=%lld N=%lld K=%lld", (ll)E, (ll)M, (ll)N, (ll)K);
    if (E >= (1 << 20) || M >= kMaxDim || N >= kMaxDim || K >= kMaxDim)
        return fail(SSG_ERR_SHAPE, "size too large: E=%lld M=%lld N=%lld K=%lld", (ll)E, (ll)M, (ll)N, (ll)K);
    return SSG_OK;
}

// A matrix of `rows` rows of `need` elements, `ld` apart; a tile's 256 rows have
// to be addressable with 31 bits.
int check_mat(const char* name, const void* p, int64_t rows, int64_t need, int64_t ld, int64_t es) {
    if (rows > 0 && need > 0 && !p) return fail(SSG_ERR_NULL, "%s is NULL", name);
    if (ld < need) return fail(SSG_ERR_STRIDE, "row stride of %s: %lld < %lld", name, (ll)ld, (ll)need);
    if (ld * es >= (int64_t)1 << 22) return fail(SSG_ERR_STRIDE, "rows of %s are 2^22 bytes apart or more", name);
    return SSG_OK;
}

int check_out(int x, int y) {
    const bool ok = x == SSG_MX4 ? y == SSG_F32 || float16_type(y) : float16_type(x) && (y == SSG_F32 || y == x);
    return ok ? SSG_OK : fail(SSG_ERR_DTYPE, "unsupported (input, output) types (%d, %d)", x, y);
}

int check_y(const char* name, const void* y, int64_t rows, int64_t cols, int64_t ld) {
    if (rows > 0 && cols > 0 && !y) return fail(SSG_ERR_NULL, "%s is NULL", name);
    if (ld < cols) return fail(SSG_ERR_STRIDE, "row stride of %s: %lld < %lld", name, (ll)ld, (ll)cols);
    return SSG_OK;
}

// The matrices of an output stack may lie one after the other or between each
// other's rows, but must not share elements.  d matrices on, a row is moved by
// d * stride: the rows nearest to it are the two around that many.
int check_apart(const char* name, int64_t E, int64_t rows, int64_t cols, int64_t ld, int64_t stride) {
    if (rows == 0 || cols == 0) return SSG_OK;
    const int64_t s = stride < 0 ? -stride : stride;
    if (s >= (rows - 1) * ld + cols) return SSG_OK;
    for (int64_t d = 1; d < E; ++d) {
        const int64_t m = d * s / ld, r = d * s - m * ld;
        if (m >= rows) break;
        if (r < cols || (m + 1 < rows && ld - r < cols))
            return fail(SSG_ERR_STRIDE, "matrices of %s overlap: stride %lld", name, (ll)stride);
    }
    return SSG_OK;
}

// X [N, K] (16-bit or mx4) against mx4 weights [E][M, K].
int mx4_args(int x, int64_t E, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const uint8_t* xs,
             int64_t ldxs, const uint8_t* W, int64_t ldw, int64_t stridew, const uint8_t* S, int64_t lds,
             int64_t strides, const int32_t* offs, bool grouped, MmArgs* out) {
    if (x != SSG_MX4 && !float16_type(x)) return fail(SSG_ERR_DTYPE, "activations of type %d", x);
    int rc = check_sizes(E, M, N, K);
    if (rc) return rc;
    const int64_t nb = blocks(K);
    if ((rc = check_mat("X", X, N, x == SSG_MX4 ? nb * 16 : K, ldx, x == SSG_MX4 ? 1 : 2))) return rc;
    if (x == SSG_MX4) {
        if ((rc = check_mat("xscales", xs, N, nb, ldxs, 1))) return rc;
    } else if (xs) {
        return fail(SSG_ERR_FORMAT, "xscales with 16-bit activations");
    }
    if ((rc = check_mat("W", W, E * M, nb * 16, ldw, 1))) return rc;
    if ((rc = check_mat("scales", S, E * M, nb, lds, 1))) return rc;
    if (grouped && !offs) return fail(SSG_ERR_NULL, "offs is NULL");
    MmArgs a{};
    a.mode = x == SSG_MX4 ? ssg::MM_MX4 : ssg::MM_W4;
    a.dt = to_dt(x);
    a.Q = M; a.P = N; a.C = K;
    a.q = W; a.ldq = ldw; a.strideq = stridew;
    a.qs = S; a.ldqs = lds; a.strideqs = strides;
    a.p = (const uint8_t*)X; a.ldp = x == SSG_MX4 ? ldx : ldx * 2;
    a.ps = xs; a.ldps = ldxs;
    a.E = E; a.offs = grouped ? offs : nullptr;
    a.splits = 1;
    *out = a;
    return SSG_OK;
}

enum Kind { FORWARD, DX, DW };

// The 16-bit products; A and B are (X, W), (dY, W) or (dY, X).
int grouped_args(Kind kind, int x, int64_t E, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                 const void* B, int64_t ldb, int64_t strideb, const int32_t* offs, MmArgs* out) {
    if (!float16_type(x)) return fail(SSG_ERR_DTYPE, "operands of type %d", x);
    int rc = check_sizes(E, M, N, K);
    if (rc) return rc;
    if ((rc = check_mat(kind == FORWARD ? "X" : "dY", A, N, kind == FORWARD ? K : M, lda, 2))) return rc;
    if ((rc = check_mat(kind == DW ? "X" : "W", B, kind == DW ? N : E * M, K, ldb, 2))) return rc;
    if (!offs) return fail(SSG_ERR_NULL, "offs is NULL");
    MmArgs a{};
    a.mode = ssg::MM_16;
    a.dt = to_dt(x);
    a.qt = kind != FORWARD;
    a.pt = kind == DW;
    a.Q = kind == FORWARD ? M : K;
    a.P = kind == DW ? M : N;
    a.C = kind == FORWARD ? K : kind == DX ? M : N;
    a.q = (const uint8_t*)B; a.ldq = ldb * 2; a.strideq = kind == DW ? 0 : strideb * 2;
    a.p = (const uint8_t*)A; a.ldp = lda * 2;
    a.E = E; a.offs = offs;
    a.splits = 1;
    *out = a;
    return SSG_OK;
}

size_t bytes_of(int rc, const MmArgs& a) {
    if (rc || a.P == 0 || a.Q == 0) return 0;
    return plan(a).bytes;
}

int check_mx4(int dtype, int64_t R, int64_t K, const void* A, int64_t lda, const void* elems, int64_t lde,
              const void* scales, int64_t lds) {
    if (dtype != SSG_F32 && !float16_type(dtype)) return fail(SSG_ERR_DTYPE, "element type %d", dtype);
    if (R < 0 || K < 0 || K >= kMaxDim) return fail(SSG_ERR_SHAPE, "size R=%lld K=%lld", (ll)R, (ll)K);
    if (R > 0 && K > 0 && (!A || !elems || !scales)) return fail(SSG_ERR_NULL, "a pointer is NULL");
    if (lda < K) return fail(SSG_ERR_STRIDE, "row stride %lld < K=%lld", (ll)lda, (ll)K);
    if (lde < blocks(K) * 16) return fail(SSG_ERR_STRIDE, "element row stride %lld < %lld", (ll)lde, (ll)blocks(K) * 16);
    if (lds < blocks(K)) return fail(SSG_ERR_STRIDE, "scale row stride %lld < %lld", (ll)lds, (ll)blocks(K));
    return SSG_OK;
}

}  // namespace

extern "C" {

int64_t ssg_mx4_elem_cols(int64_t K) { return blocks(K) * 16; }
int64_t ssg_mx4_scale_cols(int64_t K) { return blocks(K); }

int ssg_mx4_quantize(int dtype, int64_t R, int64_t K, const void* A, int64_t lda, uint8_t* elems, int64_t lde,
                     uint8_t* scales, int64_t lds, void* stream) {
    const int rc = check_mx4(dtype, R, K, A, lda, elems, lde, scales, lds);
    if (rc || R == 0 || K == 0) return rc;
    return hip_status(ssg::launch_mx4_quantize(dtype == SSG_F32 ? 2 : dtype == SSG_F16 ? 0 : 1, R, K, A, lda, elems,
                                               lde, scales, lds, (hipStream_t)stream), "kernel launch");
}

int ssg_mx4_dequantize(int dtype, int64_t R, int64_t K, const uint8_t* elems, int64_t lde, const uint8_t* scales,
                       int64_t lds, void* D, int64_t ldd, void* stream) {
    const int rc = check_mx4(dtype, R, K, D, ldd, elems, lde, scales, lds);
    if (rc || R == 0 || K == 0) return rc;
    return hip_status(ssg::launch_mx4_dequantize(dtype == SSG_F32 ? 2 : dtype == SSG_F16 ? 0 : 1, R, K, elems, lde,
                                                 scales, lds, D, ldd, (hipStream_t)stream), "kernel launch");
}

size_t ssg_mm_mx4_workspace_bytes(int x, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx,
                                  const uint8_t* xscales, int64_t ldxs, const uint8_t* W, int64_t ldw,
                                  const uint8_t* scales, int64_t lds) {
    MmArgs a{};
    return bytes_of(mx4_args(x, 1, M, N, K, X, ldx, xscales, ldxs, W, ldw, 0, scales, lds, 0, nullptr, false, &a), a);
}

int ssg_mm_mx4(int x, int y, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const uint8_t* xscales,
               int64_t ldxs, const uint8_t* W, int64_t ldw, const uint8_t* scales, int64_t lds, void* Y, int64_t ldy,
               void* ws, size_t ws_bytes, void* stream) {
    MmArgs a{};
    int rc = mx4_args(x, 1, M, N, K, X, ldx, xscales, ldxs, W, ldw, 0, scales, lds, 0, nullptr, false, &a);
    if (rc || (rc = check_out(x, y)) || (rc = check_y("Y", Y, N, M, ldy))) return rc;
    a.out = to_out(y);
    a.y = Y;
    a.ldy = ldy;
    return run(a, ws, ws_bytes, (hipStream_t)stream);
}

size_t ssg_grouped_mm_mx4_workspace_bytes(int x, int64_t E, int64_t M, int64_t N, int64_t K, const void* X,
                                          int64_t ldx, const uint8_t* xscales, int64_t ldxs, const uint8_t* W,
                                          int64_t ldw, int64_t stridew, const uint8_t* scales, int64_t lds,
                                          int64_t strides, const int32_t* offs) {
    MmArgs a{};
    return bytes_of(mx4_args(x, E, M, N, K, X, ldx, xscales, ldxs, W, ldw, stridew, scales, lds, strides, offs, true, &a), a);
}

int ssg_grouped_mm_mx4(int x, int y, int64_t E, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx,
                       const uint8_t* xscales, int64_t ldxs, const uint8_t* W, int64_t ldw, int64_t stridew,
                       const uint8_t* scales, int64_t lds, int64_t strides, const int32_t* offs, void* Y, int64_t ldy,
                       void* ws, size_t ws_bytes, void* stream) {
    MmArgs a{};
    int rc = mx4_args(x, E, M, N, K, X, ldx, xscales, ldxs, W, ldw, stridew, scales, lds, strides, offs, true, &a);
    if (rc || (rc = check_out(x, y)) || (rc = check_y("Y", Y, N, M, ldy))) return rc;
    a.out = to_out(y);
    a.y = Y;
    a.ldy = ldy;
    return run(a, ws, ws_bytes, (hipStream_t)stream);
}

size_t ssg_grouped_mm_workspace_bytes(int x, int64_t E, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx,
                                      const void* W, int64_t ldw, int64_t stridew, const int32_t* offs) {
    MmArgs a{};
    return bytes_of(grouped_args(FORWARD, x, E, M, N, K, X, ldx, W, ldw, stridew, offs, &a), a);
}

int ssg_grouped_mm(int x, int y, int64_t E, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const void* W,
                   int64_t ldw, int64_t stridew, const int32_t* offs, void* Y, int64_t ldy, void* ws, size_t ws_bytes,
                   void* stream) {
    MmArgs a{};
    int rc = grouped_args(FORWARD, x, E, M, N, K, X, ldx, W, ldw, stridew, offs, &a);
    if (rc || (rc = check_out(x, y)) || (rc = check_y("Y", Y, N, M, ldy))) return rc;
    a.out = to_out(y);
    a.y = Y;
    a.ldy = ldy;
    return run(a, ws, ws_bytes, (hipStream_t)stream);
}

size_t ssg_grouped_mm_dx_workspace_bytes(int x, int64_t E, int64_t M, int64_t N, int64_t K, const void* dY,
                                         int64_t lddy, const void* W, int64_t ldw, int64_t stridew,
                                         const int32_t* offs) {
    MmArgs a{};
    return bytes_of(grouped_args(DX, x, E, M, N, K, dY, lddy, W, ldw, stridew, offs, &a), a);
}

int ssg_grouped_mm_dx(int x, int y, int64_t E, int64_t M, int64_t N, int64_t K, const void* dY, int64_t lddy,
                      const void* W, int64_t ldw, int64_t stridew, const int32_t* offs, void* dX, int64_t lddx,
                      void* ws, size_t ws_bytes, void* stream) {
    MmArgs a{};
    int rc = grouped_args(DX, x, E, M, N, K, dY, lddy, W, ldw, stridew, offs, &a);
    if (rc || (rc = check_out(x, y)) || (rc = check_y("dX", dX, N, K, lddx))) return rc;
    a.out = to_out(y);
    a.y = dX;
    a.ldy = lddx;
    return run(a, ws, ws_bytes, (hipStream_t)stream);
}

size_t ssg_grouped_mm_dw_workspace_bytes(int x, int64_t E, int64_t M, int64_t N, int64_t K, const void* dY,
                                         int64_t lddy, const void* X, int64_t ldx, const int32_t* offs) {
    MmArgs a{};
    return bytes_of(grouped_args(DW, x, E, M, N, K, dY, lddy, X, ldx, 0, offs, &a), a);
}

int ssg_grouped_mm_dw(int x, int y, int64_t E, int64_t M, int64_t N, int64_t K, const void* dY, int64_t lddy,
                      const void* X, int64_t ldx, const int32_t* offs, void* dW, int64_t lddw, int64_t stridedw,
                      void* ws, size_t ws_bytes, void* stream) {
    MmArgs a{};
    int rc = grouped_args(DW, x, E, M, N, K, dY, lddy, X, ldx, 0, offs, &a);
    if (rc || (rc = check_out(x, y)) || (rc = check_y("dW", dW, E * M, K, lddw)) ||
        (rc = check_apart("dW", E, M, K, lddw, stridedw)))
        return rc;
    a.out = to_out(y);
    a.y = dW;
    a.ldy = lddw;
    a.stridey = stridedw;
    return run(a, ws, ws_bytes, (hipStream_t)stream);
}

int ssg_mm_select_kernel(int op, int x, int64_t E, int64_t M, int64_t N, int64_t K, int64_t kernel[4]) {
    if (!kernel) return fail(SSG_ERR_NULL, "kernel is NULL");
    // an address at a 16-byte border stands for every operand; nothing reads it
    void* const p = reinterpret_cast<void*>((uintptr_t)256);
    const uint8_t* const b = (const uint8_t*)p;
    const int32_t* const offs = (const int32_t*)p;
    const int64_t nb = blocks(K);
    MmArgs a{};
    int rc;
    switch (op) {
        case SSG_OP_MM_MX4:
        case SSG_OP_GROUPED_MM_MX4: {
            const bool mx = x == SSG_MX4, grouped = op == SSG_OP_GROUPED_MM_MX4;
            rc = mx4_args(x, grouped ? E : 1, M, N, K, p, mx ? nb * 16 : K, mx ? b : nullptr, mx ? nb : 0, b, nb * 16,
                          M * nb * 16, b, nb, M * nb, offs, grouped, &a);
            break;
        }
        case SSG_OP_GROUPED_MM: rc = grouped_args(FORWARD, x, E, M, N, K, p, K, p, K, M * K, offs, &a); break;
        case SSG_OP_GROUPED_MM_DX: rc = grouped_args(DX, x, E, M, N, K, p, M, p, K, M * K, offs, &a); break;
        case SSG_OP_GROUPED_MM_DW: rc = grouped_args(DW, x, E, M, N, K, p, M, p, K, 0, offs, &a); break;
        default: return fail(SSG_ERR_ALGO, "unknown operator %d", op);
    }
    if (rc) return rc;
    const Plan q = plan(a);
    kernel[0] = q.skinny ? 0 : 1;
    kernel[1] = q.skinny ? 16 * q.rt : ssg::kMmTileSizes[q.size].q;
    kernel[2] = q.skinny ? 16 * q.nt : ssg::kMmTileSizes[q.size].p;
    kernel[3] = q.splits;
    return SSG_OK;
}

}  // extern "C"
