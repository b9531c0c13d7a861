// mm_prep.hip -- the passes beside the tiled products: the sum of a split
// contraction's partials, operands repacked into 16-byte aligned rows, and
// scales brought into planes.
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
        mm_store4(a.y, a.out, p * a.ldy + q, m, v);
    }
}

// One 16-byte chunk a thread.
__global__ void __launch_bounds__(kThreads) k_mm_repack(const uint8_t* src, int64_t stride, int64_t rows, int64_t n,
                                                        int64_t lds, uint8_t* dst, int64_t ldd, int fill,
                                                        const int32_t* offs, int64_t total) {
    const int64_t cpr = ldd / 16, per = rows * cpr;
    for (int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x; t < total; t += (int64_t)gridDim.x * kThreads) {
        const int64_t e = t / per, u = t - e * per, r = u / cpr, b = (u - r * cpr) * 16;
        if (offs && offs[e + 1] <= offs[e]) continue;      // an expert that no product reads
        const uint8_t* at = src + e * stride + r * lds + b;
        uint8_t v[16];
        if (b + 16 <= n) {
            __builtin_memcpy(v, at, 16);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = b + j < n ? at[j] : (uint8_t)fill;
        }
        *reinterpret_cast<uint4*>(dst + t * 16) = *reinterpret_cast<uint4*>(v);
    }
}

__host__ __device__ inline int64_t mm_plane_threads(int64_t nb, int64_t plane) {
    return plane / 4 * ((nb + 63) / 64 * 4);
}

// Scales [rows][nb] to planes [blocks / 4][4][plane]: a thread takes 4 rows by
// 16 blocks, transposes them in registers, and writes 16 dwords of 4 rows each.
// Four consecutive threads read 64 bytes of the same rows, every fourth writes
// consecutive rows (with the rows consecutive alone, 28672 x 256 scales took 7.7 us
// instead of 6.2).  Rows and blocks past the end get 127
// (1.0): their elements are zeros.
__global__ void __launch_bounds__(kThreads) k_mm_planes(MmPlanes jq, MmPlanes jp, int64_t nq, int64_t total) {
    for (int64_t n = (int64_t)blockIdx.x * kThreads + threadIdx.x; n < total; n += (int64_t)gridDim.x * kThreads) {
        const MmPlanes& j = n < nq ? jq : jp;
        const uint8_t* const src = j.src;
        uint8_t* const dst = j.dst;
        const int64_t t = n < nq ? n : n - nq, nb = j.nb, ld = j.ld, rows = j.rows, stride = j.stride, plane = j.plane;
        const int64_t r4 = plane / 4, planes = (nb + 3) / 4 * 4, per_mat = mm_plane_threads(nb, plane);
        const int64_t e = t / per_mat, u = t - e * per_mat, cb = u / (4 * r4), v0 = u - cb * 4 * r4;
        const int64_t r = v0 / 4 * 4, b = (cb * 4 + v0 % 4) * 16;
        if (b >= planes) continue;
        uint32_t v[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint8_t* at = src + e * stride + (r + k) * ld + b;
            uint4 w = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
            if (r + k < rows) {
                if (b + 16 <= nb) {
                    __builtin_memcpy(&w, at, 16);
                } else {
                    uint8_t x[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] = b + j < nb ? at[j] : 127;
                    __builtin_memcpy(&w, x, 16);
                }
            }
            v[k][0] = w.x; v[k][1] = w.y; v[k][2] = w.z; v[k][3] = w.w;
        }
        uint8_t* out = dst + (e * planes + b) * plane + r;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            if (b + j >= planes) break;
            uint32_t w = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) w |= ((v[k][j >> 2] >> (8 * (j & 3))) & 0xFFu) << (8 * k);
            *reinterpret_cast<uint32_t*>(out + j * plane) = w;
        }
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

hipError_t launch_mm_repack(const void* src, int64_t mats, int64_t stride, int64_t rows, int64_t n, int64_t lds,
                            void* dst, int64_t ldd, int fill, const int32_t* offs, hipStream_t s) {
    const int64_t total = mats * rows * (ldd / 16);
    if (total == 0) return hipSuccess;
    hipLaunchKernelGGL(k_mm_repack, dim3(grid_of(total)), dim3(kThreads), 0, s, (const uint8_t*)src, stride, rows, n,
                       lds, (uint8_t*)dst, ldd, fill, offs, total);
    return hipGetLastError();
}

hipError_t launch_mm_planes(const MmPlanes& q, const MmPlanes& p, hipStream_t s) {
    auto threads = [](const MmPlanes& j) { return j.mats * mm_plane_threads(j.nb, j.plane); };
    const int64_t nq = threads(q), total = nq + threads(p);
    if (total == 0) return hipSuccess;
    hipLaunchKernelGGL(k_mm_planes, dim3(grid_of(total)), dim3(kThreads), 0, s, q, p, nq, total);
    return hipGetLastError();
}

}  // namespace ssg
