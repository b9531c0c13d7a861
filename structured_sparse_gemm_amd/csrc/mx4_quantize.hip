// mx4_quantize.hip -- 4-bit microscaled floating point: rows to blocks of 32
// E2M1 elements with one power-of-two scale byte, and back.
//
// A block with largest magnitude m gets the scale 2^(s - 127),
// s = max(floor(log2 m) - 2 + 127, 0): the top of the element range, 6 = 1.5 *
// 2^2, then meets the block's top binade.  Each element is x / scale rounded to the nearest of
// 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code), saturating at 6.  Dividing
// by a power of two is exact in fp32 here (the quotient is below 8, and where
// it is subnormal it rounds to 0 anyway), so the codes are those of exact
// arithmetic.  Infinities saturate in a block whose scale makes 6 overflow (they
// read back as infinities); a block with a NaN gets the scale 255 and reads
// back as NaN throughout.
//
// Both passes are bound by memory.  Four lanes share a block, 8 elements each:
// a lane's 16-bit input is one 16-byte load, its elements one 4-byte store, and
// the maximum takes two lane exchanges.  11008 x 4096 bf16: 23 us there (114 MB,
// 4.9 TB/s), 18 us back (6.3: part of the elements is still in the cache).
#include <algorithm>

#include "mm_args.hpp"
#include "ssg_kernels.hpp"

namespace ssg {

namespace {

constexpr int kThreads = 256;
enum Src { SRC_F16 = 0, SRC_BF16 = 1, SRC_F32 = 2 };
constexpr int src_bytes(int s) { return s == SRC_F32 ? 4 : 2; }

template <int S>
__device__ __forceinline__ float src_to_f32(const uint8_t* p) {
    if constexpr (S == SRC_F32) {
        float f;
        __builtin_memcpy(&f, p, 4);
        return f;
    } else {
        uint16_t b;
        __builtin_memcpy(&b, p, 2);
        return S == SRC_F16 ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
    }
}

// Thread i: chunk i % cpr (8 elements) of row i / cpr.
template <int S>
__global__ void __launch_bounds__(kThreads) k_mx4_quantize(uint32_t total, uint32_t cpr, int64_t K, const uint8_t* A,
                                                           int64_t lda, uint8_t* elems, int64_t lde, uint8_t* scales,
                                                           int64_t lds) {
    constexpr int ES = src_bytes(S);
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= total) return;            // total is a multiple of 4: a block's lanes stay together
    const uint32_t row = i / cpr, c = i - row * cpr;
    const uint8_t* src = A + row * lda + (int64_t)c * 8 * ES;
    const int64_t left = K - (int64_t)c * 8;
    float v[8];
    if (left >= 8) {
        uint8_t raw[8 * ES];
        __builtin_memcpy(raw, src, 8 * ES);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = src_to_f32<S>(raw + e * ES);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < left ? src_to_f32<S>(src + e * ES) : 0.0f;
    }
    uint32_t top = 0;                  // magnitudes order as their bits do, NaN above infinity
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    int s = (int)(top >> 23) - 2;
    s = s < 0 ? 0 : s;
    uint32_t d = 0;
    if (top > 0x7F800000u) {
        s = 255;
    } else {
        float m[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = __builtin_ldexpf(v[e], 127 - s);
            m[e] = __builtin_amdgcn_fmed3f(x, -6.0f, 6.0f);
        }
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, m[0], m[1], 1.0f, 0);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, m[2], m[3], 1.0f, 1);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, m[4], m[5], 1.0f, 2);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, m[6], m[7], 1.0f, 3);
    }
    __builtin_memcpy(elems + row * lde + (int64_t)c * 4, &d, 4);
    if ((c & 3) == 0) scales[row * lds + (c >> 2)] = (uint8_t)s;
}

// Thread i: elements 8 (i % cpr) .. + 7 of row i / cpr.
template <int S>
__global__ void __launch_bounds__(kThreads) k_mx4_dequantize(uint32_t total, uint32_t cpr, int64_t K,
                                                             const uint8_t* elems, int64_t lde, const uint8_t* scales,
                                                             int64_t lds, uint8_t* D, int64_t ldd) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    constexpr int ES = src_bytes(S);
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= total) return;
    const uint32_t row = i / cpr, c = i - row * cpr;
    uint32_t d;
    __builtin_memcpy(&d, elems + row * lde + (int64_t)c * 4, 4);
    const uint32_t s = scales[row * lds + (c >> 2)];
    f32x2 v[4];
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 0);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 1);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 2);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 3);
    uint8_t raw[8 * ES];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = s == 255u ? __uint_as_float(0x7FC00000u) : __builtin_ldexpf(v[e >> 1][e & 1], (int)s - 127);
        if constexpr (S == SRC_F32) {
            __builtin_memcpy(raw + e * ES, &x, 4);
        } else if constexpr (S == SRC_F16) {
            const _Float16 h = (_Float16)x;
            __builtin_memcpy(raw + e * ES, &h, 2);
        } else {
            const __bf16 h = (__bf16)x;
            __builtin_memcpy(raw + e * ES, &h, 2);
        }
    }
    uint8_t* dst = D + row * ldd + (int64_t)c * 8 * ES;
    const int64_t left = K - (int64_t)c * 8;
    if (left >= 8) {
        __builtin_memcpy(dst, raw, 8 * ES);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left) __builtin_memcpy(dst + e * ES, raw + e * ES, ES);
    }
}

// Slabs of rows, so that a launch counts its chunks in 32 bits.
template <typename F>
hipError_t by_slabs(int64_t R, int64_t cpr, F&& launch) {
    const int64_t slab = std::max<int64_t>(1, ((int64_t)1 << 30) / cpr);
    for (int64_t r = 0; r < R; r += slab) {
        const int64_t n = std::min(slab, R - r) * cpr;
        launch(r, (uint32_t)n, (uint32_t)((n + kThreads - 1) / kThreads));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_mx4_quantize(int src, int64_t R, int64_t K, const void* A, int64_t lda, void* elems, int64_t lde,
                               void* scales, int64_t lds, hipStream_t s) {
    const int64_t cpr = (K + kMxBlock - 1) / kMxBlock * 4, es = src == SRC_F32 ? 4 : 2;
    return by_slabs(R, cpr, [&](int64_t r, uint32_t n, uint32_t grid) {
        const uint8_t* a = (const uint8_t*)A + r * lda * es;
        uint8_t *e = (uint8_t*)elems + r * lde, *sc = (uint8_t*)scales + r * lds;
        auto* k = src == SRC_F16 ? k_mx4_quantize<SRC_F16> : src == SRC_BF16 ? k_mx4_quantize<SRC_BF16>
                                                                              : k_mx4_quantize<SRC_F32>;
        hipLaunchKernelGGL(k, dim3(grid), dim3(kThreads), 0, s, n, (uint32_t)cpr, K, a, lda * es, e, lde, sc, lds);
    });
}

hipError_t launch_mx4_dequantize(int dst, int64_t R, int64_t K, const void* elems, int64_t lde, const void* scales,
                                 int64_t lds, void* D, int64_t ldd, hipStream_t s) {
    const int64_t cpr = (K + 7) / 8, es = dst == SRC_F32 ? 4 : 2;
    return by_slabs(R, cpr, [&](int64_t r, uint32_t n, uint32_t grid) {
        const uint8_t *e = (const uint8_t*)elems + r * lde, *sc = (const uint8_t*)scales + r * lds;
        uint8_t* d = (uint8_t*)D + r * ldd * es;
        auto* k = dst == SRC_F16 ? k_mx4_dequantize<SRC_F16> : dst == SRC_BF16 ? k_mx4_dequantize<SRC_BF16>
                                                                                : k_mx4_dequantize<SRC_F32>;
        hipLaunchKernelGGL(k, dim3(grid), dim3(kThreads), 0, s, n, (uint32_t)cpr, K, e, lde, sc, lds, d, ldd * es);
    });
}

}  // namespace ssg
