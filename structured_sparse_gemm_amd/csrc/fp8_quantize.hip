// fp8_quantize.hip -- matrices to e4m3 elements with an fp32 scale for each 128
// elements of a row, or each 128 rows by 128 elements, as they are or transposed;
// and back.  (The rounding: fp8.hpp.)
//
// Bound by memory: a 16-bit element is read once and a byte written.  16384 x 8192 of bf16
// (402 MB) take 80 us, 5.0 TB/s, the rate of a copy; 11008 x 4096 (135 MB) 23 to 26 us in
// all four forms where the cache holds it, and from HBM, with the cache full of others'
// writes, 43 to 47; 1024 x 4096 4.7 us, one row 2.4 us.
// * Rows as they are: 16 lanes share a block, 8 elements each; the maximum takes
//   four exchanges between lanes.  A workgroup has 16 or 64 rows of a block, so that
//   it writes as many neighbouring scales of a block-major array.
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

// Eight neighbouring elements as they lie in memory.
template <int SRC>
struct Eight {
    uint32_t w[2 * kBytes<SRC>];
    __device__ __forceinline__ float operator[](int e) const {
        if constexpr (SRC == SRC8_F32) return __uint_as_float(w[e]);
        else if constexpr (SRC == SRC8_BF16) return __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
        else return f16_bits_to_f32((uint16_t)(e & 1 ? w[e >> 1] >> 16 : w[e >> 1]));
    }
    __device__ __forceinline__ float top(float t) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) t = fmaxf(t, fp8_mag((*this)[e]));   // (a NaN does not count)
        return t;
    }
};

// What follows begins from the words as loaded: the compiler keeps neither their
// widened forms nor both sides of a choice (tiles of 16-bit types: 74 registers, 96 without).
template <int SRC, int N>
__device__ __forceinline__ void pin(Eight<SRC> (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (uint32_t& w : v[i].w) asm volatile("" : "+v"(w));
}

// Elements c .. c + 7 of the rows r, r + STEP, .., zeros outside the matrix.  Where the
// columns are whole eights nothing depends on a branch (rows outside are read from
// inside, and masked), so that all loads are on their way before the first is used:
// with a branch a row 11008 x 4096 of bf16, transposed, took 48 us instead of 40 (and
// takes 23 since the rounding is cheap).
template <int SRC, int STEP, int N>
__device__ __forceinline__ void load_rows(const Fp8Matrix& a, int64_t m, int64_t r, int64_t c, bool eights,
                                          Eight<SRC> (&v)[N]) {
    const bool in = r < a.R && c < a.K;
    const int n = !in ? 0 : (int)min((a.R - r + STEP - 1) / STEP, (int64_t)N);
    const uint8_t* const p =
        (const uint8_t*)a.a + (m * a.stridea + (in ? r * a.lda + c : 0)) * kBytes<SRC>;
    const int64_t step = a.lda * kBytes<SRC> * STEP;
    if (eights) {
#pragma unroll
        for (int i = 0; i < N; ++i) __builtin_memcpy(v[i].w, p + (uint32_t)(i < n ? i : 0) * step, sizeof v[i].w);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint32_t keep = i < n ? ~0u : 0u;
            asm("" : "+v"(keep));
#pragma unroll
            for (uint32_t& w : v[i].w) w &= keep;
        }
        return;
    }
    // (one element at a time: 64 loads on their way would take twice the registers)
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint32_t bits = 0;
            if (i < n && c + e < a.K) __builtin_memcpy(&bits, p + i * step + e * kBytes<SRC>, kBytes<SRC>);
            asm volatile("" : "+v"(bits));
            if constexpr (SRC == SRC8_F32) v[i].w[e] = bits;
            else v[i].w[e >> 1] = e & 1 ? v[i].w[e >> 1] | bits << 16 : bits;
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

// Rows as they are: workgroup (16 PER rows, one block).
template <int SRC, int PER>
__global__ void __launch_bounds__(kThreads) k_quantize_rows(Fp8Matrix a, uint32_t first, uint32_t nb, uint32_t rg) {
    const uint32_t id = first + blockIdx.x, m = id / (nb * rg), in = id - m * nb * rg, g = in / nb, b = in - g * nb;
    const int64_t r0 = (int64_t)g * 16 * PER + threadIdx.x / 16, c = (int64_t)b * kFp8Block + threadIdx.x % 16 * 8;
    Eight<SRC> v[PER];
    load_rows<SRC, 16>(a, m, r0, c, (int64_t)(b + 1) * kFp8Block <= a.K || a.K % 8 == 0, v);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int64_t r = r0 + 16 * i;
        const float s = fp8_scale(lanes_max<16>(v[i].top(0.0f)));
        float u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = v[i][e];
        const uint2 q = fp8_pack8(u, fp8_recip(s));
        if (r >= a.R) continue;
        if (c < a.K) store8(a.e + m * a.stridee + r * a.lde + c, a.K - c, q);
        if (threadIdx.x % 16 == 0) a.s[m * a.mat + r * a.row + b * a.blk] = s;
    }
}

// 128 x 128 tiles.  Thread (c = t % 16, g = t / 16): columns 8 c .. + 7 of rows 8 g .. + 7.
//
// A tile that turns: row k of the transpose is 16 pieces of 8 bytes, piece g at place
// g ^ (k / 16); rows are 144 bytes apart.  So the 64 writes of a wave (16 rows 8 apart,
// 4 pieces) fall on 32 banks, four each, as few as 512 bytes take, and 16 bytes that are
// read (two pieces) stay together, at most changed about.
template <int SRC, bool WIDE, bool TR>
__global__ void __launch_bounds__(kThreads) k_quantize_tiles(Fp8Matrix a, uint32_t first, uint32_t nb, uint32_t nr) {
    static_assert(TR || WIDE, "rows as they are have their own kernel");
    __shared__ __attribute__((aligned(16))) float top_of[WIDE ? 1 : 16][kFp8Block];
    __shared__ __attribute__((aligned(16))) uint8_t turn[TR ? kFp8Block * 144 : 16];
    const uint32_t id = first + blockIdx.x, m = id / (nb * nr), in = id - m * nb * nr, rb = in / nb, cb = in - rb * nb;
    const int t = threadIdx.x, c = t % 16, g = t / 16;
    const int64_t r0 = (int64_t)rb * kFp8Block, c0 = (int64_t)cb * kFp8Block;
    Eight<SRC> v[8];
    load_rows<SRC, 1>(a, m, r0 + 8 * g, c0 + 8 * c, c0 + kFp8Block <= a.K || a.K % 8 == 0, v);
    pin(v);
    float* const sc = a.s + m * a.mat;
    float s8[WIDE ? 1 : 8];            // the scales of this thread's columns
    if constexpr (WIDE) {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = v[i].top(top);
        top = lanes_max<64>(top);
        if ((t & 63) == 0) top_of[0][t >> 6] = top;
        __syncthreads();
        s8[0] = fp8_scale(fmaxf(fmaxf(top_of[0][0], top_of[0][1]), fmaxf(top_of[0][2], top_of[0][3])));
        if (t == 0) sc[(TR ? cb : rb) * a.row + (TR ? rb : cb) * a.blk] = s8[0];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fp8_mag(v[i][e]));
            s8[e] = top;
        }
        __builtin_memcpy(&top_of[g][8 * c], s8, sizeof s8);
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
        __builtin_memcpy(s8, &top_of[0][8 * c], sizeof s8);
    }
    pin(v);
    if constexpr (!TR) {
        const Fp8Recip rc = fp8_recip(s8[0]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = r0 + 8 * g + i, at = c0 + 8 * c;
            float u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = v[i][e];
            const uint2 q = fp8_pack8(u, rc);
            if (r < a.R && at < a.K) store8(a.e + m * a.stridee + r * a.lde + at, a.K - at, q);
        }
    } else {
        uint8_t* const put = turn + 8 * c * 144 + 8 * (g ^ (c >> 1));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = v[i][e];
            *reinterpret_cast<uint2*>(put + e * 144) = fp8_pack8(u, fp8_recip(s8[WIDE ? 0 : e]));
        }
        __syncthreads();
        // row c0 + k of the output: bytes r0 .. r0 + 127, 16 a thread
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = i * 32 + (t >> 3), j = t & 7, x = k >> 4;
            const int64_t at = r0 + j * 16, n = a.R - at;
            if (c0 + k >= a.K || n <= 0) continue;
            uint4 d = *reinterpret_cast<const uint4*>(turn + k * 144 + (j ^ (x >> 1)) * 16);
            if (x & 1) d = make_uint4(d.z, d.w, d.x, d.y);
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

// Rows as they are: 16 a workgroup up to so many workgroups, which the chip holds at
// once, 64 from there on.  bf16, 16 and 64: 512 x 4096 3.5 and 3.9 us, 1024 x 4096 4.7
// and 4.8, 16384 x 8192 97 and 80 (the rate of a copy).
constexpr int64_t kFewGroups = 2048;

template <int SRC>
hipError_t quantize(const Fp8Matrix& a, hipStream_t s) {
    const int64_t nb = (a.K + kFp8Block - 1) / kFp8Block;
    const bool rows = a.block == 1 && !a.transpose;
    const bool few = rows && a.mats * nb * ((a.R + 15) / 16) <= kFewGroups;
    const int64_t per = few ? 16 : rows ? 64 : kFp8Block, nr = (a.R + per - 1) / per;
    if (a.mats * nb * nr >= (int64_t)1 << 32) return hipErrorInvalidValue;
    return by_slabs(a.mats * nb * nr, [&](uint32_t i, dim3 grid) {
        const uint32_t n = (uint32_t)nb, r = (uint32_t)nr;
        if (few) hipLaunchKernelGGL((k_quantize_rows<SRC, 1>), grid, dim3(kThreads), 0, s, a, i, n, r);
        else if (rows) hipLaunchKernelGGL((k_quantize_rows<SRC, 4>), grid, dim3(kThreads), 0, s, a, i, n, r);
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
