// mm_fp8_few.hip -- products of few rows with e4m3 weights that have an fp32 scale
// for each block of 128; dense or grouped by expert.
//
// Bound by reading the weights once.  A workgroup owns 16 * RT weight rows and
// 16 * NT tokens of one expert.  Its 8 waves take the blocks of the contraction
// in turn, each loads both operands of a block from memory straight into MFMA
// registers, multiplies them (as fp16: the matrix units have time) into fresh
// sums and adds those, times the two scales, to its own; the waves' sums meet in
// LDS in wave order.
//
// 16-bit activations are rounded here, on their way to the registers: a lane has
// 32 elements of a token's block, and three other lanes the rest, so the maximum
// takes two exchanges.  A launch of its own for that costs a decode step more
// than every workgroup's repeating it.
#include <algorithm>

#include "fp8.hpp"
#include "lanes.hpp"

namespace ssg {

namespace {

constexpr int kWaves = 8, kThreads = kWaves * 64;

// 16 bytes of a row from byte k on, zeros from n on.
template <bool FULL>
__device__ __forceinline__ uint4 ld_bytes(const uint8_t* row, int64_t k, int64_t n) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (FULL || k + 16 <= n) {
        __builtin_memcpy(&v, row + k, 16);
    } else if (k < n) {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (k + e < n) w[e >> 2] |= (uint32_t)row[k + e] << (8 * (e & 3));
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
}

// The larger of a value in the four lanes that share a token (16 apart).
__device__ __forceinline__ float max_of_groups(float v) {
    uint32_t a, b;
    lane_pair<false>(__float_as_uint(v), &a, &b);
    v = fmaxf(__uint_as_float(a), __uint_as_float(b));
    lane_pair<true>(__float_as_uint(v), &a, &b);
    return fmaxf(__uint_as_float(a), __uint_as_float(b));
}

// XS: Fp8Src of the activations (F16, BF16), or -1 for e4m3.  WR: a scale for each weight row.
template <int XS, bool WR, int RT, int NT>
struct Few {
    static constexpr bool ROUND = XS >= 0;
    static constexpr int XL = ROUND ? 4 : 2;           // 16-byte loads of a token's block
    // Blocks whose loads go out together: 16 rows are 2 KiB a block and wave.
    static constexpr int AHEAD = RT * NT == 1 ? 4 : RT * NT == 2 ? 2 : 1;
    struct Ops {
        uint4 w[RT][2], x[NT][XL];
        float ws[RT][WR ? 4 : 1], xs[ROUND ? 1 : NT];
    };

    const MmFp8Args& a;
    const uint8_t *q[RT], *p[NT];      // this lane's rows
    const float *ws[RT][WR ? 4 : 1], *xs[NT];
    int g;
    f32x4 acc[RT][NT];

    template <bool FULL>
    __device__ __forceinline__ void load(int64_t b, Ops& o) const {
        const int64_t k = b * kFp8Block + 16 * g, n = a.m.C;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            o.w[r][0] = ld_bytes<FULL>(q[r], k, n);
            o.w[r][1] = ld_bytes<FULL>(q[r], k + 64, n);
#pragma unroll
            for (int e = 0; e < (WR ? 4 : 1); ++e) o.ws[r][e] = ws[r][e][b * a.w.blk];
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int u = 0; u < XL; ++u)
                o.x[t][u] = ROUND ? ld_bytes<FULL>(p[t], 2 * k + (u >> 1) * 128 + (u & 1) * 16, 2 * n)
                                  : ld_bytes<FULL>(p[t], k + u * 64, n);
            if constexpr (!ROUND) o.xs[t] = xs[t][b * a.x.blk];
        }
    }

    __device__ __forceinline__ void products(const Ops& o) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            uint4 x0, x1;
            float s;
            if constexpr (ROUND) {
                float v[4][8], top = 0.0f;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    fp8_widen8<XS>(o.x[t][u], v[u]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[u][e]));
                }
                s = fp8_scale(max_of_groups(top));
                const Fp8Recip rc = fp8_recip(s);
                uint2 c[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) c[u] = fp8_pack8(v[u], rc);
                x0 = make_uint4(c[0].x, c[0].y, c[1].x, c[1].y);
                x1 = make_uint4(c[2].x, c[2].y, c[3].x, c[3].y);
            } else {
                x0 = o.x[t][0];
                x1 = o.x[t][1];
                s = o.xs[t];
            }
            const Fp8Wide x = fp8_widen(x0, x1);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const f32x4 d = fp8_mfma_exact(fp8_widen(o.w[r][0], o.w[r][1]), x);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[r][t][e] = fmaf(d[e], s * o.ws[r][WR ? e : 0], acc[r][t][e]);
            }
        }
    }

    __device__ __forceinline__ void run(int64_t n, int64_t by) {
        const int64_t whole = a.m.C / kFp8Block, all = (a.m.C + kFp8Block - 1) / kFp8Block;
        if constexpr (AHEAD > 1) {
            for (; n + (AHEAD - 1) * by < whole; n += AHEAD * by) {
                Ops o[AHEAD];
#pragma unroll
                for (int d = 0; d < AHEAD; ++d) load<true>(n + d * by, o[d]);
#pragma unroll
                for (int d = 0; d < AHEAD; ++d) products(o[d]);
            }
        }
        Ops o;
        for (; n < whole; n += by) {
            load<true>(n, o);
            products(o);
        }
        if (n < all) {
            load<false>(n, o);
            products(o);
        }
    }
};

template <int XS, bool WR, int RT, int NT>
__global__ void __launch_bounds__(kThreads, 2) k_mm_fp8_few(MmFp8Args a, uint32_t nq) {
    __shared__ __attribute__((aligned(16))) f32x4 red[kWaves][RT * NT * 64];
    const MmArgs& m = a.m;
    const uint32_t per = gridDim.x / (uint32_t)m.splits, split = blockIdx.x / per, id = blockIdx.x - split * per;
    const uint32_t tt = id / nq, qt = id - tt * nq;
    MmTile tile;
    if (!mm_find_tile(m, 16 * NT, (int)tt, &tile)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i = lane & 15;
    const int64_t q0 = (int64_t)qt * 16 * RT, e = tile.e < 0 ? 0 : tile.e;
    Few<XS, WR, RT, NT> k{a};
    k.g = lane >> 4;
    // rows and tokens past the end repeat the last one; their sums are not stored
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int64_t row = std::min<int64_t>(q0 + 16 * r + i, m.Q - 1);
        k.q[r] = m.q + e * m.strideq + row * m.ldq;
#pragma unroll
        for (int f = 0; f < (WR ? 4 : 1); ++f) {
            const int64_t sr = WR ? std::min<int64_t>(q0 + 16 * r + 4 * k.g + f, m.Q - 1) : (q0 + 16 * r) / kFp8Block;
            k.ws[r][f] = a.w.p + e * a.w.mat + sr * a.w.row;
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t row = std::min<int64_t>(tile.r0 + 16 * t + i, tile.r1 - 1);
        k.p[t] = m.p + row * m.ldp;
        k.xs[t] = a.x.p + row * a.x.row;
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) k.acc[r][t] = f32x4{0, 0, 0, 0};
    if (tile.e >= 0) k.run((int64_t)split * kWaves + wave, (int64_t)m.splits * kWaves);
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
        if (p < tile.r1 && q < m.Q) {
            const int n = m.Q - q < 4 ? (int)(m.Q - q) : 4;
            if (m.part) mm_store4(m.part, OUT_F32, ((int64_t)split * m.P + p) * m.Q + q, n, v);
            else mm_store4(m.y, m.out, p * m.ldy + q, n, v);
        }
    }
}

template <int XS, bool WR, int RT, int NT>
hipError_t go(const MmFp8Args& a, hipStream_t s) {
    const int64_t nq = (a.m.Q + 16 * RT - 1) / (16 * RT), tiles = mm_tile_bound(a.m, 16 * NT);
    if (nq * tiles * a.m.splits >= (int64_t)1 << 23) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_mm_fp8_few<XS, WR, RT, NT>), dim3((unsigned)(nq * tiles * a.m.splits)), dim3(kThreads), 0, s,
                       a, (uint32_t)nq);
    return hipGetLastError();
}

template <int XS>
hipError_t pick(const MmFp8Args& a, int rt, int nt, hipStream_t s) {
    if (a.w_rows) return nt == 1 ? go<XS, true, 1, 1>(a, s) : go<XS, true, 1, 2>(a, s);
    if (rt == 1) return nt == 1 ? go<XS, false, 1, 1>(a, s) : go<XS, false, 1, 2>(a, s);
    if (rt == 2) return nt == 1 ? go<XS, false, 2, 1>(a, s) : go<XS, false, 2, 2>(a, s);
    return nt == 1 ? go<XS, false, 4, 1>(a, s) : go<XS, false, 4, 2>(a, s);
}

}  // namespace

hipError_t launch_mm_fp8_few(const MmFp8Args& a, int rt, int nt, hipStream_t s) {
    switch (a.x_src) {
        case SRC8_F16: return pick<SRC8_F16>(a, rt, nt, s);
        case SRC8_BF16: return pick<SRC8_BF16>(a, rt, nt, s);
        default: return pick<-1>(a, rt, nt, s);
    }
}

}  // namespace ssg
