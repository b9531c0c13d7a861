// mm_prep.hip -- the passes beside the tiled products: the sum of a split
// contraction's partials, and operands repacked into 16-byte aligned rows.
#include <algorithm>

#include "mm_args.hpp"
#include "ssg_kernels.hpp"

namespace ssg {

namespace {

constexpr int kThreads = 256;

// Four columns a thread; the splits are added in order, so the result does
// not depend on which workgroup ended first.
__global__ void __launch_bounds__(kThreads) k_mm_reduce(MmArgs a) {
    const int64_t cpr = (a.Q + 3) / 4, n = a.P * cpr;
    const bool vin = a.Q % 4 == 0;
    const bool vec = a.ldy % 4 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0;
    for (int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x; t < n; t += (int64_t)gridDim.x * kThreads) {
        const int64_t p = t / cpr, q = (t - p * cpr) * 4;
        const int m = a.Q - q < 4 ? (int)(a.Q - q) : 4;
        f32x4 v = {0, 0, 0, 0};
        for (int s = 0; s < a.splits; ++s) {
            const float* src = a.part + (s * a.P + p) * a.Q + q;
            if (vin) v += *reinterpret_cast<const f32x4*>(src);
            else
                for (int r = 0; r < 4; ++r)
                    if (r < m) v[r] += src[r];
        }
        mm_store4(a.y, a.out, p * a.ldy + q, m, vec, v);
    }
}

// One 16-byte chunk a thread.
__global__ void __launch_bounds__(kThreads) k_mm_repack(const uint8_t* src, int64_t rows, int64_t n, int64_t lds,
                                                        uint8_t* dst, int64_t ldd, int fill) {
    const int64_t cpr = ldd / 16, total = rows * cpr;
    for (int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x; t < total; t += (int64_t)gridDim.x * kThreads) {
        const int64_t r = t / cpr, b = (t - r * cpr) * 16;
        const uint8_t* at = src + r * lds + b;
        uint8_t v[16];
        if (b + 16 <= n) {
            __builtin_memcpy(v, at, 16);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = b + j < n ? at[j] : (uint8_t)fill;
        }
        *reinterpret_cast<uint4*>(dst + r * ldd + b) = *reinterpret_cast<uint4*>(v);
    }
}

unsigned grid_of(int64_t n) { return (unsigned)std::min<int64_t>((n + kThreads - 1) / kThreads, 16384); }

}  // namespace

hipError_t launch_mm_tiles_16(const MmArgs& a, int size, hipStream_t s);
hipError_t launch_mm_tiles_mx4(const MmArgs& a, int size, hipStream_t s);

hipError_t launch_mm_tiles(const MmArgs& a, int size, hipStream_t s) {
    return a.mode == MM_16 ? launch_mm_tiles_16(a, size, s) : launch_mm_tiles_mx4(a, size, s);
}

hipError_t launch_mm_reduce(const MmArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(k_mm_reduce, dim3(grid_of(a.P * ((a.Q + 3) / 4))), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_mm_repack(const void* src, int64_t rows, int64_t n, int64_t lds, void* dst, int64_t ldd, int fill,
                            hipStream_t s) {
    if (rows * ldd == 0) return hipSuccess;
    hipLaunchKernelGGL(k_mm_repack, dim3(grid_of(rows * (ldd / 16))), dim3(kThreads), 0, s, (const uint8_t*)src, rows,
                       n, lds, (uint8_t*)dst, ldd, fill);
    return hipGetLastError();
}

}  // namespace ssg
