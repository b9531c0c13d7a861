// fp8.hpp -- 8-bit floats (e4m3) with an fp32 scale for each block of 128: device
// helpers, arguments and launchers (fp8_quantize.hip, mm_fp8_few.hip,
// mm_fp8_tiles.hip).
#pragma once

#include "mm_args.hpp"

namespace ssg {

constexpr int kFp8Block = 128;
enum Fp8Src { SRC8_F16 = 0, SRC8_BF16 = 1, SRC8_F32 = 2 };

struct Fp8Scales {
    const float* p;
    int64_t row, blk, mat;             // strides in elements: of rows (or blocks of rows), of blocks, of matrices
};

// Y = X W^T: m describes the elements (q: W, p: X), their scales here.
struct MmFp8Args {
    MmArgs m;
    Fp8Scales w, x;
    bool w_rows;                       // a scale for each row of W, else for each 128 rows
    int x_src;                         // few rows: Fp8Src of X that the kernel rounds itself, or -1
};
// Activations that the few-row kernel may round: at most so many tokens, and bytes of
// them rounded (in whole blocks).
constexpr int kFp8RoundTokens = 16, kFp8RoundBytes = 32768;
hipError_t launch_mm_fp8_few(const MmFp8Args& a, int rt, int nt, hipStream_t s);
hipError_t launch_mm_fp8_tiles(const MmFp8Args& a, int size, hipStream_t s);

struct Fp8Matrix {
    int type;                          // Fp8Src of the matrix
    int64_t mats, R, K;                // of the matrix in its own type
    const void* a;
    int64_t lda, stridea;              // elements
    int block;                         // rows that share a scale: 1 or 128
    bool transpose;                    // the 8-bit form is that of the transpose, [K, R]
    uint8_t* e;
    int64_t lde, stridee;              // bytes
    float* s;
    int64_t row, blk, mat;             // strides of the scales, as in Fp8Scales
};
hipError_t launch_fp8_quantize(const Fp8Matrix& a, hipStream_t s);
hipError_t launch_fp8_dequantize(const Fp8Matrix& a, hipStream_t s);
// Scales [rows][nb] of `mats` matrices to planes [nb][plane] (zeros past the rows).
hipError_t launch_fp8_planes(const Fp8Scales& src, int64_t mats, int64_t rows, int64_t nb, float* dst, int64_t plane,
                             hipStream_t s);

// ---------------------------------------------------------------------------
// Rounding.  A block with largest magnitude m has the scale
// s = max(m / 448, 2^-126) (448 is the largest e4m3 number; the bound keeps 1 / s
// finite and gives blocks of zeros a scale), and its elements are the e4m3 numbers
// nearest to x / s, ties to even.
//
// The nearest to the exact quotient, so that every kernel (and a definition in
// 64 bits) gives the same bytes: x times the reciprocal r of s is off by up to two
// steps of fp32, which matters where x / s lies at or next to the border of two codes,
// and it often does: with 16-bit x whole blocks have quotients of few digits.  So
// q = |x| r is rounded to a multiple of 64 steps (borders have five digits: where x / s
// is near one, q becomes the border itself), the sign of |x| - q s, which one fused
// multiply-add gives exactly, says on which side x / s lies, and q takes one step to
// that side; then the conversion's rounding is right.  Eight instructions an element
// without a branch; comparing the doubtful ones in fp64 needed fewer for most, and
// 40 us instead of 23 for 11008 x 4096 of bf16, transposed.
// NaN stays NaN and does not enter m; an infinity makes the scale infinite, and
// with it every product that meets the block (0 * inf) NaN.
// ---------------------------------------------------------------------------
// A magnitude as it enters a maximum: a signalling NaN becomes a quiet one, which the
// maximum passes over (of a signalling one it makes a NaN, and forgets what was before).
__device__ __forceinline__ float fp8_mag(float x) { return __builtin_canonicalizef(fabsf(x)); }

__device__ __forceinline__ float fp8_scale(float top) { return fmaxf(top / 448.0f, 0x1p-126f); }

struct Fp8Recip {
    float s, r;
};
// (r is within a step; of an infinite scale 0, and what is multiplied by it stays a number)
__device__ __forceinline__ Fp8Recip fp8_recip(float s) { return {fminf(s, 0x1.fffffep127f), __builtin_amdgcn_rcpf(s)}; }

// Eight codes, in element order.
__device__ __forceinline__ uint2 fp8_pack8(float (&v)[8], Fp8Recip b) {
    if (b.s < 0x1p-80f) {              // so that |x| - q s does not underflow
        b.s *= 0x1p64f;
        b.r *= 0x1p-64f;
#pragma unroll
        for (float& x : v) x *= 0x1p64f;
    }
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // (a NaN's payload could carry into the sign: the last 32 would become numbers)
        const uint32_t near = (min(__float_as_uint(fabsf(v[e]) * b.r), 0x7FC00000u) + 32u) & ~63u;
        const float side = __builtin_fmaf(-__uint_as_float(near), b.s, fabsf(v[e]));
        int step;                      // its sign: between -1 and 1 as integers (the compiler makes two compares of it)
        asm("v_med3_i32 %0, %1, -1, 1" : "=v"(step) : "v"(side));
        q[e] = copysignf(__uint_as_float(near + (uint32_t)step), v[e]);
    }
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// 16 bytes of 16-bit elements as eight fp32 values.
template <int SRC>
__device__ __forceinline__ void fp8_widen8(uint4 d, float (&v)[8]) {
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (SRC == SRC8_BF16) {
            v[2 * e] = __uint_as_float(w[e] << 16);
            v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        } else {
            v[2 * e] = f16_bits_to_f32((uint16_t)w[e]);
            v[2 * e + 1] = f16_bits_to_f32((uint16_t)(w[e] >> 16));
        }
    }
}

// ---------------------------------------------------------------------------
// 16 x 16 x 128 products of e4m3 operands: lane (i = l % 16, g = l / 16) holds 32
// elements of row i of both, the same ones for the same g; the result as in mfma16.
//
// The elements are widened to fp16, where each is exact, and take four 16-bit
// instructions, whose sums are fp32's.  The 8-bit instruction would take half the
// time, but adds eight neighbouring products at a time, aligned to the largest
// exponent among them and cut 13 bits below it (a check of the instruction, and of
// its form for 32 elements: 2^16 + 2^3 is kept, 2^16 + 2^2 is not, and only within
// eight).  What it loses is up to 7 * 2^-13 of the largest of eight products, which
// no output's rounding hides where terms cancel: of 2000 sums of 4096 normal numbers
// (this rule followed in 64 bits) 3.0% are off by more than half a step of fp16 and
// 0.4% of bf16.
// ---------------------------------------------------------------------------
// 32 elements as fp16, eight a 16 bytes.
struct Fp8Wide {
    uint4 v[4];
};
__device__ __forceinline__ uint4 fp8_widen_part(uint32_t lo, uint32_t hi) {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    union { f16x2 h[4]; uint4 u; } w;
    w.h[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    w.h[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    w.h[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    w.h[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return w.u;
}
__device__ __forceinline__ Fp8Wide fp8_widen(uint4 lo, uint4 hi) {
    return {{fp8_widen_part(lo.x, lo.y), fp8_widen_part(lo.z, lo.w), fp8_widen_part(hi.x, hi.y),
             fp8_widen_part(hi.z, hi.w)}};
}
__device__ __forceinline__ f32x4 fp8_mfma(const Fp8Wide& a, const Fp8Wide& b) {
    f32x4 d = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) d = mfma16<DT_F16>(a.v[k], b.v[k], d);
    return d;
}

}  // namespace ssg
