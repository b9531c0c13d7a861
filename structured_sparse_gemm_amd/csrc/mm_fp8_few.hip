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
// A few 16-bit activations are rounded here, by every workgroup into LDS: up to
// kFp8RoundBytes of them cost less than a launch of their own (rounding them in
// the lanes that multiply them, 16 rows whatever the tokens, took longer: 11.5
// instead of 7 us for one token through 4096 x 4096, 24 instead of 8 for 16).  The
// weights' first loads come after it; of one token's 6.5 us the bytes need 3.3.
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

// XS: Fp8Src of activations that are rounded here (F16, BF16), or -1 for e4m3.  WR: a
// scale for each weight row.
template <int XS, bool WR, int RT, int NT>
struct Few {
    static constexpr bool ROUND = XS >= 0;
    // One block's loads at a time: what hides them is the other workgroups of the CU,
    // four of 16 x 16 (64 registers).  With four blocks of 16 rows or two of 32 on their
    // way, and half as many workgroups, 40 experts of 2048 x 4096 took 100 us instead of
    // 76, 53 of 1024 x 2048 31 instead of 24, one token the same.
    struct Ops {
        uint4 w[RT][2], x[NT][2];
        float ws[RT][WR ? 4 : 1], xs[NT];
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
        // (rounded activations end with zeros)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if constexpr (ROUND) continue;
            o.x[t][0] = ld_bytes<FULL>(p[t], k, n);
            o.x[t][1] = ld_bytes<FULL>(p[t], k + 64, n);
            o.xs[t] = xs[t][b * a.x.blk];
        }
    }

    __device__ __forceinline__ void products(int64_t b, Ops& o) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if constexpr (ROUND) {
                o.x[t][0] = *reinterpret_cast<const uint4*>(p[t] + b * kFp8Block + 16 * g);
                o.x[t][1] = *reinterpret_cast<const uint4*>(p[t] + b * kFp8Block + 16 * g + 64);
                o.xs[t] = xs[t][b];
            }
            const Fp8Wide x = fp8_widen(o.x[t][0], o.x[t][1]);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const f32x4 d = fp8_mfma(fp8_widen(o.w[r][0], o.w[r][1]), x);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[r][t][e] = fmaf(d[e], o.xs[t] * o.ws[r][WR ? e : 0], acc[r][t][e]);
            }
        }
    }

    __device__ __forceinline__ void run(int64_t n) {       // blocks n, n + kWaves, ..
        const int64_t whole = a.m.C / kFp8Block, all = (a.m.C + kFp8Block - 1) / kFp8Block;
        for (; n < whole; n += kWaves) {
            Ops o;
            load<true>(n, o);
            products(n, o);
        }
        // the block that the contraction ends in is the turn of one wave
        if (whole < all && n == whole) {
            Ops o;
            load<false>(whole, o);
            products(whole, o);
        }
    }
};

template <int XS, bool WR, int RT, int NT>
__global__ void __launch_bounds__(kThreads, RT * NT > 1 ? 2 : WR ? 6 : 8) k_mm_fp8_few(MmFp8Args a, uint32_t nq) {
    constexpr bool ROUND = XS >= 0;
    constexpr int kRed = kWaves * RT * NT * 64 * 16;
    // sums of the waves; before them rounded activations (rows 16 bytes further apart
    // than long, over the banks) and their scales
    constexpr int kRows = kFp8RoundBytes + 16 * kFp8RoundTokens, kX = ROUND ? kRows + kFp8RoundBytes / kFp8Block * 4 : 0;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kRed > kX ? kRed : kX];
    f32x4(*const red)[RT * NT * 64] = reinterpret_cast<f32x4(*)[RT * NT * 64]>(lds);
    const MmArgs& m = a.m;
    const uint32_t tt = blockIdx.x / nq, qt = blockIdx.x - tt * nq;
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
    const int64_t nb = (m.C + kFp8Block - 1) / kFp8Block;
    if constexpr (ROUND) {
        // 16 threads a block of a token, 8 elements each (at most kFp8RoundTokens
        // tokens, and blocks of them in kFp8RoundBytes: the caller's choice)
        const int64_t tokens = tile.r1 - tile.r0, ld = nb * kFp8Block + 16;
        float* const sc = reinterpret_cast<float*>(lds + kRows);
        for (int64_t u = threadIdx.x / 16; u < tokens * nb; u += kThreads / 16) {
            const int64_t t = u / nb, b = u - t * nb, c = b * kFp8Block + threadIdx.x % 16 * 8;
            const uint8_t* const row = m.p + (tile.r0 + t) * m.ldp;
            float v[8];
            uint4 d = make_uint4(0, 0, 0, 0);
            if (c + 8 <= m.C) {
                __builtin_memcpy(&d, row + 2 * c, 16);
            } else {
                uint16_t h[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < m.C) __builtin_memcpy(&h[j], row + 2 * (c + j), 2);
                __builtin_memcpy(&d, h, 16);
            }
            fp8_widen8<XS>(d, v);
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, fp8_mag(v[j]));
            const float s = fp8_scale(lanes_max<16>(top));
            *reinterpret_cast<uint2*>(lds + t * ld + c) = fp8_pack8(v, fp8_recip(s));
            if (threadIdx.x % 16 == 0) sc[u] = s;
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int64_t row = std::min<int64_t>(16 * t + i, tokens - 1);
            k.p[t] = lds + row * ld;
            k.xs[t] = sc + row * nb;
        }
    } else {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int64_t row = std::min<int64_t>(tile.r0 + 16 * t + i, tile.r1 - 1);
            k.p[t] = m.p + row * m.ldp;
            k.xs[t] = a.x.p + row * a.x.row;
        }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) k.acc[r][t] = f32x4{0, 0, 0, 0};
    if (tile.e >= 0) k.run(wave);
    if constexpr (ROUND) __syncthreads();              // the activations give way to the sums
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
            mm_store4(m.y, m.out, p * m.ldy + q, n, v);
        }
    }
}

template <int XS, bool WR, int RT, int NT>
hipError_t go(const MmFp8Args& a, hipStream_t s) {
    const int64_t nq = (a.m.Q + 16 * RT - 1) / (16 * RT), tiles = mm_tile_bound(a.m, 16 * NT);
    if (nq * tiles >= (int64_t)1 << 23) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_mm_fp8_few<XS, WR, RT, NT>), dim3((unsigned)(nq * tiles)), dim3(kThreads), 0, s, a, (uint32_t)nq);
    return hipGetLastError();
}

template <int XS, bool WR>
hipError_t pick(const MmFp8Args& a, int rt, int nt, hipStream_t s) {
    if constexpr (XS >= 0 && WR) return go<XS, WR, 1, 1>(a, s);
    else if constexpr (XS >= 0) return rt == 1 ? go<XS, WR, 1, 1>(a, s) : go<XS, WR, 2, 1>(a, s);
    else if constexpr (WR) return nt == 1 ? go<XS, WR, 1, 1>(a, s) : go<XS, WR, 1, 2>(a, s);
    else if (rt == 1) return nt == 1 ? go<XS, WR, 1, 1>(a, s) : go<XS, WR, 1, 2>(a, s);
    else if (rt == 2) return nt == 1 ? go<XS, WR, 2, 1>(a, s) : go<XS, WR, 2, 2>(a, s);
    else return nt == 1 ? go<XS, WR, 4, 1>(a, s) : go<XS, WR, 4, 2>(a, s);
}

}  // namespace

hipError_t launch_mm_fp8_few(const MmFp8Args& a, int rt, int nt, hipStream_t s) {
    switch (a.x_src) {
        case SRC8_F16: return a.w_rows ? pick<SRC8_F16, true>(a, rt, nt, s) : pick<SRC8_F16, false>(a, rt, nt, s);
        case SRC8_BF16: return a.w_rows ? pick<SRC8_BF16, true>(a, rt, nt, s) : pick<SRC8_BF16, false>(a, rt, nt, s);
        default: return a.w_rows ? pick<-1, true>(a, rt, nt, s) : pick<-1, false>(a, rt, nt, s);
    }
}

}  // namespace ssg
