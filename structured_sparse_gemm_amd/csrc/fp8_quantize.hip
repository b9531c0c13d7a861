// fp8_quantize.hip -- matrices to e4m3 elements with an fp32 scale for each 128
// elements of a row, or each 128 rows by 128 elements, as they are or transposed;
// and back.  (The rounding: fp8.hpp.)
//
// Bound by memory: a 16-bit element is read once and a byte written.
// * Rows as they are: 16 lanes share a block, 8 elements each; the maximum takes
//   four exchanges between lanes.  A workgroup has 16 rows of a block, so that it
//   writes 16 neighbouring scales of a block-major array.
// * 128 x 128 tiles, where the scale is shared by rows or the output is
//   transposed: a thread has 8 rows of 8 columns in registers, so every byte is
//   read once whatever the scale covers.  A transposed tile turns in LDS (8 bytes,
//   8 rows of a column, at a time) and leaves in whole lines.
#include <algorithm>

#include "fp8.hpp"
#include "lanes.hpp"

namespace ssg {

namespace {

constexpr int kThreads = 256;

template <int SRC> constexpr int kBytes = SRC == SRC8_F32 ? 4 : 2;

// Elements c .. c + 7 of a row, zeros from n on.
template <int SRC>
__device__ __forceinline__ void load8(const uint8_t* row, int64_t c, int64_t n, float (&v)[8]) {
    if (c + 8 <= n) {
        if constexpr (SRC == SRC8_F32) {
            __builtin_memcpy(v, row + c * 4, 32);
        } else {
            uint4 d;
            __builtin_memcpy(&d, row + c * 2, 16);
            fp8_widen8<SRC>(d, v);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = 0.0f;
        if (c + e >= n) continue;
        if constexpr (SRC == SRC8_F32) {
            __builtin_memcpy(&v[e], row + (c + e) * 4, 4);
        } else {
            uint16_t b;
            __builtin_memcpy(&b, row + (c + e) * 2, 2);
            v[e] = SRC == SRC8_F16 ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
        }
    }
}

// n of the bytes of v (element order) to any address.
__device__ __forceinline__ void store8(uint8_t* at, int64_t n, uint2 v) {
    if (n >= 8) {
        __builtin_memcpy(at, &v, 8);
        return;
    }
    const uint64_t w = ((uint64_t)v.y << 32) | v.x;
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n) at[e] = (uint8_t)(w >> (8 * e));
}

__device__ __forceinline__ float top8(const float (&v)[8], float top) {
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));   // (a NaN does not count)
    return top;
}

// Rows as they are: workgroup (16 rows, one block).
template <int SRC>
__global__ void __launch_bounds__(kThreads) k_quantize_rows(Fp8Matrix a, uint32_t first, uint32_t nb, uint32_t rg) {
    const uint32_t id = first + blockIdx.x, m = id / (nb * rg), in = id - m * nb * rg, g = in / nb, b = in - g * nb;
    const int64_t r = (int64_t)g * 16 + threadIdx.x / 16, c = (int64_t)b * kFp8Block + threadIdx.x % 16 * 8;
    const int64_t rr = r < a.R ? r : a.R - 1;
    const uint8_t* row = (const uint8_t*)a.a + (m * a.stridea + rr * a.lda) * kBytes<SRC>;
    float v[8];
    load8<SRC>(row, c, a.K, v);
    const float s = fp8_scale(lanes_max<16>(top8(v, 0.0f)));
    const uint2 q = fp8_pack8(v, fp8_recip(s));
    if (r >= a.R) return;
    if (c < a.K) store8(a.e + m * a.stridee + r * a.lde + c, a.K - c, q);
    if (threadIdx.x % 16 == 0) a.s[m * a.mat + r * a.row + b * a.blk] = s;
}

// 128 x 128 tiles.  Thread (c = t % 16, g = t / 16): columns 8 c .. + 7 of rows 8 g .. + 7.
template <int SRC, bool WIDE, bool TR>
__global__ void __launch_bounds__(kThreads) k_quantize_tiles(Fp8Matrix a, uint32_t first, uint32_t nb, uint32_t nr) {
    __shared__ __attribute__((aligned(16))) float top_of[TR && !WIDE ? 16 : 1][kFp8Block];
    __shared__ __attribute__((aligned(16))) uint8_t turn[TR ? kFp8Block * 144 : 16];   // rows of 144 bytes: over all banks
    const uint32_t id = first + blockIdx.x, m = id / (nb * nr), in = id - m * nb * nr, rb = in / nb, cb = in - rb * nb;
    const int t = threadIdx.x, c = t % 16, g = t / 16;
    const int64_t r0 = (int64_t)rb * kFp8Block, c0 = (int64_t)cb * kFp8Block;
    const uint8_t* const base = (const uint8_t*)a.a + m * a.stridea * kBytes<SRC>;
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 8 * g + i;
        if (r < a.R) {
            load8<SRC>(base + r * a.lda * kBytes<SRC>, c0 + 8 * c, a.K, v[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
        }
    }
    float* const sc = a.s + m * a.mat;
    if constexpr (WIDE) {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = top8(v[i], top);
        top = lanes_max<64>(top);
        if ((t & 63) == 0) top_of[0][t >> 6] = top;
        __syncthreads();
        top = fmaxf(fmaxf(top_of[0][0], top_of[0][1]), fmaxf(top_of[0][2], top_of[0][3]));
        const float s = fp8_scale(top);
        const Fp8Recip rc = fp8_recip(s);
        if (t == 0) sc[(TR ? cb : rb) * a.row + (TR ? rb : cb) * a.blk] = s;
        if constexpr (!TR) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t r = r0 + 8 * g + i, at = c0 + 8 * c;
                const uint2 q = fp8_pack8(v[i], rc);
                if (r < a.R && at < a.K) store8(a.e + m * a.stridee + r * a.lde + at, a.K - at, q);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = v[i][e];
                *reinterpret_cast<uint2*>(turn + (8 * c + e) * 144 + 8 * g) = fp8_pack8(u, rc);
            }
        }
    } else {
        static_assert(TR || WIDE, "rows as they are have their own kernel");
        // a scale for each column of the tile
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i][e]));
            top_of[g][8 * c + e] = top;
        }
        __syncthreads();
        if (t < kFp8Block) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, top_of[i][t]);
            const float s = fp8_scale(top);
            top_of[0][t] = s;          // (column t is this thread's alone)
            if (c0 + t < a.K) sc[(c0 + t) * a.row + rb * a.blk] = s;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = v[i][e];
            *reinterpret_cast<uint2*>(turn + (8 * c + e) * 144 + 8 * g) = fp8_pack8(u, fp8_recip(top_of[0][8 * c + e]));
        }
    }
    if constexpr (TR) {
        __syncthreads();
        // row c0 + k of the output: bytes r0 .. r0 + 127, 16 a thread
        for (int u = t; u < kFp8Block * 8; u += kThreads) {
            const int k = u >> 3;
            const int64_t at = r0 + (u & 7) * 16, n = a.R - at;
            if (c0 + k >= a.K || n <= 0) continue;
            uint4 d = *reinterpret_cast<const uint4*>(turn + k * 144 + (u & 7) * 16);
            uint8_t* const dst = a.e + m * a.stridee + (c0 + k) * a.lde + at;
            if (n >= 16) {
                __builtin_memcpy(dst, &d, 16);
            } else {
                store8(dst, n, make_uint2(d.x, d.y));
                if (n > 8) store8(dst + 8, n - 8, make_uint2(d.z, d.w));
            }
        }
    }
}

// Eight elements a thread: element times scale in fp32, then in the type.
template <int DST>
__global__ void __launch_bounds__(kThreads) k_dequantize(Fp8Matrix a, int64_t r0, uint32_t total, uint32_t cpr) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= total) return;
    const uint32_t rl = i / cpr;
    const int64_t c = (int64_t)(i - rl * cpr) * 8, flat = r0 + rl, m = flat / a.R, r = flat - m * a.R, left = a.K - c;
    const uint8_t* const src = a.e + m * a.stridee + r * a.lde + c;
    uint2 d = make_uint2(0, 0);
    if (left >= 8) {
        __builtin_memcpy(&d, src, 8);
    } else {
        uint64_t w = 0;
        for (int e = 0; e < left; ++e) w |= (uint64_t)src[e] << (8 * e);
        d = make_uint2((uint32_t)w, (uint32_t)(w >> 32));
    }
    const float s = a.s[m * a.mat + (a.block == 1 ? r : r / kFp8Block) * a.row + c / kFp8Block * a.blk];
    f32x2 f[4];
    f[0] = __builtin_amdgcn_cvt_pk_f32_fp8((int)d.x, false);
    f[1] = __builtin_amdgcn_cvt_pk_f32_fp8((int)d.x, true);
    f[2] = __builtin_amdgcn_cvt_pk_f32_fp8((int)d.y, false);
    f[3] = __builtin_amdgcn_cvt_pk_f32_fp8((int)d.y, true);
    uint8_t raw[8 * kBytes<DST>];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float x = f[e >> 1][e & 1] * s;
        // (the product as the products take it: fp16 would be rounded from the exact one)
        asm("" : "+v"(x));
        if constexpr (DST == SRC8_F32) {
            __builtin_memcpy(raw + 4 * e, &x, 4);
        } else if constexpr (DST == SRC8_F16) {
            const _Float16 h = (_Float16)x;
            __builtin_memcpy(raw + 2 * e, &h, 2);
        } else {
            const __bf16 h = (__bf16)x;
            __builtin_memcpy(raw + 2 * e, &h, 2);
        }
    }
    uint8_t* const dst = (uint8_t*)const_cast<void*>(a.a) + (m * a.stridea + r * a.lda + c) * kBytes<DST>;
    if (left >= 8) {
        __builtin_memcpy(dst, raw, 8 * kBytes<DST>);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left) __builtin_memcpy(dst + e * kBytes<DST>, raw + e * kBytes<DST>, kBytes<DST>);
    }
}

// Thread: one scale of the planes, rows fastest.
__global__ void __launch_bounds__(kThreads) k_planes(Fp8Scales src, int64_t total, int64_t rows, int64_t nb, float* dst,
                                                     int64_t plane) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= total) return;
    const int64_t r = i % plane, mb = i / plane, b = mb % nb, m = mb / nb;
    dst[i] = r < rows ? src.p[m * src.mat + r * src.row + b * src.blk] : 0.0f;
}

// f(first, number) for slabs of `total` workgroups, each a launch of fewer than 2^32 threads.
template <typename F>
hipError_t by_slabs(int64_t total, F&& f) {
    constexpr int64_t kSlab = (int64_t)1 << 23;
    for (int64_t i = 0; i < total; i += kSlab) {
        f((uint32_t)i, dim3((unsigned)std::min(kSlab, total - i)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int SRC>
hipError_t quantize(const Fp8Matrix& a, hipStream_t s) {
    const int64_t nb = (a.K + kFp8Block - 1) / kFp8Block;
    const int64_t nr = a.block == 1 && !a.transpose ? (a.R + 15) / 16 : (a.R + kFp8Block - 1) / kFp8Block;
    if (a.mats * nb * nr >= (int64_t)1 << 32) return hipErrorInvalidValue;
    return by_slabs(a.mats * nb * nr, [&](uint32_t i, dim3 grid) {
        const uint32_t n = (uint32_t)nb, r = (uint32_t)nr;
        if (a.block == 1 && !a.transpose) hipLaunchKernelGGL(k_quantize_rows<SRC>, grid, dim3(kThreads), 0, s, a, i, n, r);
        else if (a.block == 1) hipLaunchKernelGGL((k_quantize_tiles<SRC, false, true>), grid, dim3(kThreads), 0, s, a, i, n, r);
        else if (a.transpose) hipLaunchKernelGGL((k_quantize_tiles<SRC, true, true>), grid, dim3(kThreads), 0, s, a, i, n, r);
        else hipLaunchKernelGGL((k_quantize_tiles<SRC, true, false>), grid, dim3(kThreads), 0, s, a, i, n, r);
    });
}

}  // namespace

hipError_t launch_fp8_quantize(const Fp8Matrix& a, hipStream_t s) {
    return a.type == SRC8_F16 ? quantize<SRC8_F16>(a, s) : a.type == SRC8_BF16 ? quantize<SRC8_BF16>(a, s)
                                                                               : quantize<SRC8_F32>(a, s);
}

hipError_t launch_fp8_dequantize(const Fp8Matrix& a, hipStream_t s) {
    const int64_t cpr = (a.K + 7) / 8, slab = std::max<int64_t>(1, ((int64_t)1 << 30) / cpr), R = a.mats * a.R;
    for (int64_t r = 0; r < R; r += slab) {
        const uint32_t n = (uint32_t)(std::min(slab, R - r) * cpr);
        auto* k = a.type == SRC8_F16 ? k_dequantize<SRC8_F16> : a.type == SRC8_BF16 ? k_dequantize<SRC8_BF16>
                                                                                    : k_dequantize<SRC8_F32>;
        hipLaunchKernelGGL(k, dim3((n + kThreads - 1) / kThreads), dim3(kThreads), 0, s, a, r, n, (uint32_t)cpr);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_fp8_planes(const Fp8Scales& src, int64_t mats, int64_t rows, int64_t nb, float* dst, int64_t plane,
                             hipStream_t s) {
    const int64_t total = mats * nb * plane;
    if (total == 0) return hipSuccess;
    if ((total + kThreads - 1) / kThreads >= (int64_t)1 << 24) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_planes, dim3((unsigned)((total + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, src, total,
                       rows, nb, dst, plane);
    return hipGetLastError();
}

}  // namespace ssg
