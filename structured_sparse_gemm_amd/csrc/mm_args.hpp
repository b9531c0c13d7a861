// mm_args.hpp -- arguments and device helpers shared by the dense and mx4
// matrix products (mm_skinny.hip, mm_tiles*.hip, mm_prep.hip).
//
// Every product here is Y[p, q] = sum_c P[p, c] Q[q, c] for each expert, with
// q the contiguous direction of Y.  Q is the MFMA's A operand (its rows are
// the accumulator's register direction, so a lane holds four consecutive q
// and stores them together), P its B operand.
#pragma once

#include "ssg_device.hpp"
#include "ssg_stream.hpp"

namespace ssg {

// What the two operands hold: 16-bit floats both; mx4 both; mx4 weights (Q)
// against 16-bit activations (P).
enum MmMode { MM_16 = 0, MM_MX4 = 1, MM_W4 = 2 };
enum MmOut { OUT_F32 = 0, OUT_F16 = 1, OUT_BF16 = 2 };

constexpr int kMxBlock = 32;           // elements that share one scale byte

struct MmArgs {
    int mode, dt, out;                 // MmMode, DT_F16 / DT_BF16 of 16-bit operands, MmOut
    int qt, pt;                        // operand stored [c][q] / [c][p] instead of [q][c] / [p][c]
    int64_t Q, P, C;                   // columns of Y; rows of Y (all tokens; M for dW); contraction length
    const uint8_t* q;                  // strides in bytes
    int64_t ldq, strideq;
    const uint8_t* p;
    int64_t ldp;
    const uint8_t* qs;                 // scale bytes of mx4 operands
    int64_t ldqs, strideqs;
    const uint8_t* ps;
    int64_t ldps;
    int64_t E;
    const int32_t* offs;               // E + 1 row offsets, or nullptr: one expert that has every row
    void* y;
    int64_t ldy, stridey;              // elements
    float* part;                       // split contraction: fp32 partials [splits][P][Q], else nullptr
    int splits;
};

// Tiles of T rows that the experts' rows can need at most: every segment may
// end in a partial one.
int64_t mm_tile_bound(const MmArgs& a, int T);
hipError_t launch_mm_skinny(const MmArgs& a, int rt, int nt, hipStream_t s);
// Tile sizes of the tiled kernels, the workgroups a CU holds at once, the
// matrix rate of a chip full of them relative to the largest, and the time of
// a stage (us) when a CU has one workgroup that waits for nothing else.
struct MmTileSize {
    int q, p, per_cu;
    double rate, latency;
};
constexpr MmTileSize kMmTileSizes[3] = {{256, 256, 1, 1.0, 0.26}, {128, 128, 2, 0.65, 0.26}, {128, 64, 3, 0.48, 0.2}};
// Scales [mats][rows][nb], ld bytes a row, to planes [mats][ceil(nb / 4)][4][plane]
// for the tiled products of two mx4 operands (which take the planes' size as
// ldqs / ldps).
struct MmPlanes {
    const uint8_t* src;
    int64_t mats, stride, rows, nb, ld;
    uint8_t* dst;
    int64_t plane;
};
hipError_t launch_mm_planes(const MmPlanes& q, const MmPlanes& p, hipStream_t s);
hipError_t launch_mm_tiles(const MmArgs& a, int size, hipStream_t s);
// Y = the sum of the partials in split order, in the output type.
hipError_t launch_mm_reduce(const MmArgs& a, hipStream_t s);
// Matrices of `rows` rows of n bytes to rows of ldd bytes (a multiple of 16),
// `fill` past n; matrix e is left out if offs is given and offs[e + 1] <= offs[e].
hipError_t launch_mm_repack(const void* src, int64_t mats, int64_t stride, int64_t rows, int64_t n, int64_t lds,
                            void* dst, int64_t ldd, int fill, const int32_t* offs, hipStream_t s);
hipError_t launch_mx4_quantize(int src, int64_t R, int64_t K, const void* A, int64_t lda, void* elems, int64_t lde,
                               void* scales, int64_t lds, hipStream_t s);
hipError_t launch_mx4_dequantize(int dst, int64_t R, int64_t K, const void* elems, int64_t lde, const void* scales,
                                 int64_t lds, void* D, int64_t ldd, hipStream_t s);

// ---------------------------------------------------------------------------
// Experts' rows.  Segment 0 is the rows before offs[0], segment s the rows of
// expert s - 1, segment E + 1 the rows from offs[E] on; the first and last are
// nobody's and get zeros.  The offsets live on the device, so the host cannot
// check them: they are clamped to [0, P], and a segment that would end before
// it begins is empty, so that no offsets reach past the operands.
// ---------------------------------------------------------------------------
struct MmTile {
    int e;                             // expert, or -1: rows that get zeros
    int64_t r0, v0, r1;                // the tile begins at r0, its rows are v0 .. r1 - 1
};

// Tiles of an mx4 operand begin at multiples of 16 rows, where the pieces of
// its scale planes are aligned; the rows before the segment are left out.
__device__ __forceinline__ int64_t mm_align(const MmArgs& a, int64_t row) {
    return a.mode == MM_MX4 ? row & ~(int64_t)15 : row;
}

__device__ __forceinline__ void mm_segment(const MmArgs& a, int64_t s, int64_t* lo, int64_t* hi) {
    auto at = [&](int64_t i) -> int64_t {
        if (i < 0) return 0;
        if (i > a.E) return a.P;
        const int64_t v = a.offs[i];
        return v < 0 ? 0 : (v > a.P ? a.P : v);
    };
    *lo = at(s - 1);
    *hi = at(s);
    if (s > a.E + 1) *lo = *hi = a.P;
}

// Inclusive prefix sum over the wave.
__device__ __forceinline__ int wave_scan(int v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(v, d);
        if (lane >= d) v += u;
    }
    return v;
}

// Tiles of T rows over all segments.
__device__ __forceinline__ int mm_count_tiles(const MmArgs& a, int T) {
    if (!a.offs) return (int)((a.P + T - 1) / T);
    const int lane = threadIdx.x & 63;
    int total = 0;
    for (int64_t s0 = 0; s0 < a.E + 2; s0 += 64) {
        int64_t lo, hi;
        mm_segment(a, s0 + lane, &lo, &hi);
        total += __builtin_amdgcn_readlane(wave_scan(hi > lo ? (int)((hi - mm_align(a, lo) + T - 1) / T) : 0), 63);
    }
    return total;
}

// Tile t; false past the last one.
__device__ __forceinline__ bool mm_find_tile(const MmArgs& a, int T, int t, MmTile* out) {
    if (!a.offs) {
        out->e = 0;
        out->r0 = out->v0 = (int64_t)t * T;
        out->r1 = out->r0 + T < a.P ? out->r0 + T : a.P;
        return out->r0 < a.P;
    }
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int64_t s0 = 0; s0 < a.E + 2; s0 += 64) {
        int64_t lo, hi;
        mm_segment(a, s0 + lane, &lo, &hi);
        const int n = hi > lo ? (int)((hi - mm_align(a, lo) + T - 1) / T) : 0;
        const int inc = wave_scan(n);
        const uint64_t hit = __ballot(t < before + inc);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const int first = before + __builtin_amdgcn_readlane(inc, l) - __builtin_amdgcn_readlane(n, l);
            const int slo = __builtin_amdgcn_readlane((int)lo, l), shi = __builtin_amdgcn_readlane((int)hi, l);
            const int64_t s = s0 + l;
            out->e = s == 0 || s == a.E + 1 ? -1 : (int)(s - 1);
            out->r0 = mm_align(a, slo) + (int64_t)(t - first) * T;
            out->v0 = out->r0 > slo ? out->r0 : slo;
            out->r1 = out->r0 + T < shi ? out->r0 + T : shi;
            return true;
        }
        before += __builtin_amdgcn_readlane(inc, 63);
    }
    return false;
}

// ---------------------------------------------------------------------------
// mx4 elements and scales.
// ---------------------------------------------------------------------------
// 2^(s - 127): exact for every s (s = 0 is the subnormal 2^-127), NaN for 255.
__device__ __forceinline__ float e8m0_to_f32(uint32_t s) {
    return __uint_as_float(s == 0 ? 0x00400000u : s == 255u ? 0x7FC00000u : s << 23);
}

// Scale bytes whose blocks are exact in the 16-bit type, whatever their
// elements: magnitudes 0.5 * 2^(s - 127) to 6 * 2^(s - 127) have to stay
// normal and finite (fp16: 2^-14 .. 6 * 2^13; bf16: 2^-126 .. 6 * 2^124).
// Weights lie well inside; products that meet another scale take the elements
// unscaled and scale their fp32 sums instead.
template <int DT> constexpr uint32_t kSafeLo = DT == DT_F16 ? 127 - 13 : 2;
template <int DT> constexpr uint32_t kSafeHi = DT == DT_F16 ? 127 + 13 : 127 + 124;
template <int DT> __device__ __forceinline__ bool mx4_unsafe(uint32_t s) {
    return s - kSafeLo<DT> > kSafeHi<DT> - kSafeLo<DT>;
}

// Blocks of zeros have the scale 0, which is not safe, and are exact all the
// same (under every scale but the NaN): rows of zeros (padding, pruned rows, an
// expert not trained yet) are ordinary.  So the main loops note unsafe scales
// alone (looking at the elements there, too, costs the largest tile registers
// that it does not have: 155 instead of 125 us for 32 experts of 4096 x 2048 with 4096
// rows), and where one was met, this pass decides whether it matters (8192 x 8192
// with two rows of zeros and 1000 bf16 rows: 167 us, without them 130, and 411
// where every unsafe scale counted; 11008 x 4096 and 16 fp16 rows: 15.3, 13.2, 23.5):
// thread t of n looks for an unsafe scale whose block is not all zeros, in `rows`
// rows and blocks [first + k step, first + k step + len) below nb, k = 0, 1, ..
template <int DT>
__device__ __forceinline__ bool mx4_not_exact(const uint8_t* q, int64_t ldq, const uint8_t* qs, int64_t ldqs,
                                              uint32_t rows, uint32_t first, uint32_t len, uint32_t step, uint32_t nb,
                                              uint32_t t, uint32_t n) {
    if (first >= nb) return false;
    const uint32_t parts = (len + 3) / 4, per = ((nb - first + step - 1) / step) * parts;
    bool bad = false;
    for (uint32_t u = t; u < rows * per; u += n) {
        const uint32_t row = u / per, c = u - row * per, k = c / parts, in = (c - k * parts) * 4;
        const uint32_t b = first + k * step + in, left = min(len - in, nb > b ? nb - b : 0u);
        const uint8_t *s = qs + row * ldqs + b, *e = q + row * ldq + (int64_t)b * 16;
        uint32_t v = 0x7F7F7F7Fu;
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
            if (j < left) v = (v & ~(0xFFu << (8 * j))) | ((uint32_t)s[j] << (8 * j));
#pragma unroll 1                           // registers that the main loop would pay for
        for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t sc = (v >> (8 * j)) & 0xFFu;
            if (!mx4_unsafe<DT>(sc)) continue;
            uint4 d;
            __builtin_memcpy(&d, e + j * 16, 16);
            bad |= sc == 255u || ((d.x | d.y | d.z | d.w) & 0x77777777u) != 0;
        }
    }
    return bad;
}

// Eight 16-bit values of eight elements (one dword) times `scale`, a power of
// two; the even element of each byte is its low nibble.
template <int DT>
__device__ __forceinline__ uint4 mx4_widen(uint32_t d, float scale) {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    if constexpr (DT == DT_F16) {
        union { f16x2 v[4]; uint4 u; } r;
        r.v[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, scale, 0);
        r.v[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, scale, 1);
        r.v[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, scale, 2);
        r.v[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, scale, 3);
        return r.u;
    } else {
        union { bf16x2 v[4]; uint4 u; } r;
        r.v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 0);
        r.v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 1);
        r.v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 2);
        r.v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 3);
        return r.u;
    }
}

// 16 x 16 x 32 product of 16-bit operands: lane (i = l % 16, g = l / 16) holds
// row i, elements 8g .. 8g + 7 of both; register r of the result is row
// 4g + r of the first operand and row i of the second.
template <int DT>
__device__ __forceinline__ f32x4 mfma16(uint4 a, uint4 b, f32x4 c) {
    if constexpr (DT == DT_F16) {
        union { uint4 u; f16x8 v; } x{a}, y{b};
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(x.v, y.v, c, 0, 0, 0);
    } else {
        union { uint4 u; bf16x8 v; } x{a}, y{b};
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.v, y.v, c, 0, 0, 0);
    }
}

// 16 x 16 x 128 product of mx4 operands: lane (i, g) holds 32 elements of row
// i (one block) of both, their scales are bytes QSEL of qs and PSEL of ps.
template <int QSEL, int PSEL>
__device__ __forceinline__ f32x4 mfma_mx4(uint4 a, uint4 b, f32x4 c, uint32_t qs, uint32_t ps) {
    const i32x8 x = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const i32x8 y = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, QSEL, (int)qs, PSEL, (int)ps);
}

// Four consecutive outputs of row p from column q on, rounded to nearest even
// for 16-bit outputs (half a step of the type, the only rounding after the
// fp32 sums); any alignment.
__device__ __forceinline__ void mm_store4(void* y, int out, int64_t at, int n, f32x4 v) {
    typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    if (out == OUT_F32) {
        float* d = reinterpret_cast<float*>(y) + at;
        if (n >= 4) __builtin_memcpy(d, &v, 16);
        else
            for (int r = 0; r < 4; ++r)
                if (r < n) d[r] = v[r];
        return;
    }
    union { f16x4 h; bf16x4 b; uint2 u; uint16_t s[4]; } w;
    if (out == OUT_F16) w.h = __builtin_convertvector(v, f16x4);
    else w.b = __builtin_convertvector(v, bf16x4);
    uint16_t* d = reinterpret_cast<uint16_t*>(y) + at;
    if (n >= 4) __builtin_memcpy(d, &w.u, 8);
    else
        for (int r = 0; r < 4; ++r)
            if (r < n) d[r] = w.s[r];
}

}  // namespace ssg
