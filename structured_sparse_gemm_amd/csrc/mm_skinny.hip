// mm_skinny.hip -- products of few rows (single tokens, decode batches) with
// 16-bit or mx4 weights, dense or grouped by expert.
//
// Bound by reading the weights once.  A workgroup owns 16 * RT weight rows and
// 16 * NT tokens of one expert; its 8 waves split the contraction, each wave
// loads both operands from memory straight into MFMA operand registers (no
// LDS, no barrier in the loop: with at most 32 tokens nothing is worth
// sharing between waves), and the waves' fp32 sums meet once in LDS, added in
// wave order.  Any length, stride and alignment is taken: rows and tokens past
// the end repeat the last one (their results are not stored), and the last
// steps of a row load under guards.
//
// A wave's step is kStep contraction elements:
// * 16-bit: lane (i, g) loads 16 bytes of row i, elements 32 u + 8 g, u < 8.
// * mx4: lane (i, g) loads one 32-element block (16 bytes) of row i, block
//   4 t + g, t < 4, and one dword of scales, blocks 4 g .. 4 g + 3 of the
//   step, which the lanes of a row then exchange.  Against 16-bit activations
//   dword j of the block meets elements 8 j .. 8 j + 7 of the same block of
//   the token: the order of the contraction is free as long as both operands
//   agree.
#include <algorithm>

#include "mm_args.hpp"
#include "ssg_kernels.hpp"

namespace ssg {

namespace {

constexpr int kWaves = 8, kThreads = kWaves * 64;

// 8 16-bit elements from element k of a row of n; those past the end are zero.
__device__ __forceinline__ uint4 ld8(const uint8_t* row, int64_t k, int64_t n) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (k + 8 <= n) {
        __builtin_memcpy(&v, row + k * 2, 16);
    } else if (k < n) {
        uint16_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            h[e] = 0;
            if (k + e < n) __builtin_memcpy(&h[e], row + (k + e) * 2, 2);
        }
        __builtin_memcpy(&v, h, 16);
    }
    return v;
}

__device__ __forceinline__ uint4 ld16(const uint8_t* p) {
    uint4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

template <int MODE> constexpr int kStep = MODE == MM_16 ? 256 : 512;

template <int MODE, int DT, int RT, int NT>
struct Skinny {
    const MmArgs& a;
    const uint8_t* qrow[RT];
    const uint8_t* prow[NT];
    const uint8_t* qsrow[RT];
    const uint8_t* psrow[NT];
    int64_t nb;                        // scale bytes of a row
    int i, g;
    f32x4 acc[RT][NT];

    // scales of blocks 4 g .. 4 g + 3 of the step whose first block is b0; 127 (1.0) past the end
    template <bool FULL>
    __device__ __forceinline__ uint32_t ld_scales(const uint8_t* row, int64_t b0) const {
        const int64_t b = b0 + 4 * g;
        uint32_t v = 0x7F7F7F7Fu;
        if (FULL || b + 4 <= nb) {
            __builtin_memcpy(&v, row + b, 4);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (b + e < nb) v = (v & ~(0xFFu << (8 * e))) | ((uint32_t)row[b + e] << (8 * e));
        }
        return v;
    }

    template <bool FULL>
    __device__ __forceinline__ uint4 ld_block(const uint8_t* row, int64_t b) const {
        if (FULL || b < nb) return ld16(row + b * 16);
        return make_uint4(0, 0, 0, 0);
    }

    template <bool FULL>
    __device__ __forceinline__ void step(int64_t k0) {
        if constexpr (MODE == MM_16) {
            uint4 w[RT][8], x[NT][8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int64_t k = k0 + 32 * u + 8 * g;
#pragma unroll
                for (int r = 0; r < RT; ++r) w[r][u] = FULL ? ld16(qrow[r] + k * 2) : ld8(qrow[r], k, a.C);
#pragma unroll
                for (int t = 0; t < NT; ++t) x[t][u] = FULL ? ld16(prow[t] + k * 2) : ld8(prow[t], k, a.C);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int t = 0; t < NT; ++t) acc[r][t] = mfma16<DT>(w[r][u], x[t][u], acc[r][t]);
        } else if constexpr (MODE == MM_MX4) {
            const int64_t b0 = k0 / kMxBlock;
            uint4 w[RT][4], x[NT][4];
            uint32_t ws[RT], xs[NT];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
#pragma unroll
                for (int r = 0; r < RT; ++r) w[r][u] = ld_block<FULL>(qrow[r], b0 + 4 * u + g);
#pragma unroll
                for (int t = 0; t < NT; ++t) x[t][u] = ld_block<FULL>(prow[t], b0 + 4 * u + g);
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) ws[r] = ld_scales<FULL>(qsrow[r], b0);
#pragma unroll
            for (int t = 0; t < NT; ++t) xs[t] = ld_scales<FULL>(psrow[t], b0);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint32_t sw[RT], sx[NT];
#pragma unroll
                for (int r = 0; r < RT; ++r) sw[r] = (uint32_t)__shfl((int)ws[r], 16 * u + i) >> (8 * g);
#pragma unroll
                for (int t = 0; t < NT; ++t) sx[t] = (uint32_t)__shfl((int)xs[t], 16 * u + i) >> (8 * g);
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int t = 0; t < NT; ++t) acc[r][t] = mfma_mx4<0, 0>(w[r][u], x[t][u], acc[r][t], sw[r], sx[t]);
            }
        } else {
            const int64_t b0 = k0 / kMxBlock;
            uint4 w[RT][4];
            uint32_t ws[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                ws[r] = ld_scales<FULL>(qsrow[r], b0);
#pragma unroll
                for (int u = 0; u < 4; ++u) w[r][u] = ld_block<FULL>(qrow[r], b0 + 4 * u + g);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint4 x[NT][4];
                const int64_t k = k0 + 32 * (4 * u + g);
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[t][j] = FULL ? ld16(prow[t] + (k + 8 * j) * 2) : ld8(prow[t], k + 8 * j, a.C);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const uint32_t s = ((uint32_t)__shfl((int)ws[r], 16 * u + i) >> (8 * g)) & 0xFFu;
                    const uint32_t d[4] = {w[r][u].x, w[r][u].y, w[r][u].z, w[r][u].w};
                    if (__builtin_expect(!__any(s - kSafeLo<DT> > kSafeHi<DT> - kSafeLo<DT>), 1)) {
                        const float f = __uint_as_float(s << 23);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint4 v = mx4_widen<DT>(d[j], f);
#pragma unroll
                            for (int t = 0; t < NT; ++t) acc[r][t] = mfma16<DT>(v, x[t][j], acc[r][t]);
                        }
                    } else {
                        // one block of each row at a time, unscaled, its sum scaled in fp32
                        for (int b = 0; b < 4; ++b) {
                            f32x4 sum[NT];
#pragma unroll
                            for (int t = 0; t < NT; ++t) sum[t] = f32x4{0, 0, 0, 0};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint4 z = make_uint4(0, 0, 0, 0);
                                const uint4 v = g == b ? mx4_widen<DT>(d[j], 1.0f) : z;
#pragma unroll
                                for (int t = 0; t < NT; ++t) sum[t] = mfma16<DT>(v, g == b ? x[t][j] : z, sum[t]);
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float f = e8m0_to_f32((uint32_t)__shfl((int)s, 16 * b + 4 * g + e));
#pragma unroll
                                for (int t = 0; t < NT; ++t) acc[r][t][e] += f * sum[t][e];
                            }
                        }
                    }
                }
            }
        }
    }
};

template <int MODE, int DT, int RT, int NT>
__global__ void __launch_bounds__(kThreads) k_mm_skinny(MmArgs a, uint32_t nq) {
    __shared__ f32x4 red[kWaves][RT * NT * 64];
    const uint32_t tt = blockIdx.x / nq, qt = blockIdx.x - tt * nq;
    MmTile tile;
    if (!mm_find_tile(a, 16 * NT, (int)tt, &tile)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t q0 = (int64_t)qt * 16 * RT;
    Skinny<MODE, DT, RT, NT> k{a};
    k.i = lane & 15;
    k.g = lane >> 4;
    k.nb = (a.C + kMxBlock - 1) / kMxBlock;
    const int64_t e = tile.e < 0 ? 0 : tile.e;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int64_t row = std::min<int64_t>(q0 + 16 * r + k.i, a.Q - 1);
        k.qrow[r] = a.q + e * a.strideq + row * a.ldq;
        if constexpr (MODE != MM_16) k.qsrow[r] = a.qs + e * a.strideqs + row * a.ldqs;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t row = std::max(tile.v0, std::min<int64_t>(tile.r0 + 16 * t + k.i, tile.r1 - 1));
        k.prow[t] = a.p + row * a.ldp;
        if constexpr (MODE == MM_MX4) k.psrow[t] = a.ps + row * a.ldps;
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) k.acc[r][t] = f32x4{0, 0, 0, 0};
    if (tile.e >= 0) {
        constexpr int S = kStep<MODE>;
        // a block that K ends inside is whole in an mx4 operand, not in a 16-bit one
        const int64_t whole = MODE == MM_MX4 ? k.nb * kMxBlock : a.C;
        for (int64_t k0 = (int64_t)wave * S; k0 < a.C; k0 += kWaves * S) {
            if (k0 + S <= whole) k.template step<true>(k0);
            else k.template step<false>(k0);
        }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) red[wave][(r * NT + t) * 64 + lane] = k.acc[r][t];
    __syncthreads();
    for (int o = threadIdx.x; o < RT * NT * 64; o += kThreads) {
        f32x4 v = red[0][o];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += red[w][o];
        const int l = o & 63, r = (o >> 6) / NT, t = (o >> 6) % NT;
        const int64_t p = tile.r0 + 16 * t + (l & 15), q = q0 + 16 * r + 4 * (l >> 4);
        if (p >= tile.v0 && p < tile.r1 && q < a.Q) {
            const int64_t left = a.Q - q;
            const bool vec = a.ldy % 4 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0;
            mm_store4(a.y, a.out, p * a.ldy + q, left < 4 ? (int)left : 4, vec, v);
        }
    }
}

template <int MODE, int DT, int RT, int NT>
hipError_t go(const MmArgs& a, hipStream_t s) {
    const int64_t nq = (a.Q + 16 * RT - 1) / (16 * RT);
    const int64_t tiles = mm_tile_bound(a, 16 * NT);
    if (nq * tiles >= (int64_t)1 << 31) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_mm_skinny<MODE, DT, RT, NT>), dim3((unsigned)(nq * tiles)), dim3(kThreads), 0, s, a,
                       (uint32_t)nq);
    return hipGetLastError();
}

template <int MODE, int DT>
hipError_t pick(const MmArgs& a, int rt, int nt, hipStream_t s) {
    if (nt == 1) return rt == 1 ? go<MODE, DT, 1, 1>(a, s) : go<MODE, DT, 2, 1>(a, s);
    return rt == 1 ? go<MODE, DT, 1, 2>(a, s) : go<MODE, DT, 2, 2>(a, s);
}

}  // namespace

int64_t mm_tile_bound(const MmArgs& a, int T) {
    if (!a.offs) return (a.P + T - 1) / T;
    // a segment's partial tile, and the rows an mx4 tile begins before it
    return (a.P + (a.mode == MM_MX4 ? 15 * (a.E + 2) : 0)) / T + a.E + 2;
}

hipError_t launch_mm_skinny(const MmArgs& a, int rt, int nt, hipStream_t s) {
    switch (a.mode) {
        case MM_16: return a.dt == DT_F16 ? pick<MM_16, DT_F16>(a, rt, nt, s) : pick<MM_16, DT_BF16>(a, rt, nt, s);
        case MM_MX4: return pick<MM_MX4, DT_F16>(a, rt, nt, s);
        default: return a.dt == DT_F16 ? pick<MM_W4, DT_F16>(a, rt, nt, s) : pick<MM_W4, DT_BF16>(a, rt, nt, s);
    }
}

}  // namespace ssg
