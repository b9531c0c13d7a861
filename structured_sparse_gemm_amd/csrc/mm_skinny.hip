// mm_skinny.hip -- products of few rows (single tokens, decode batches) with
// 16-bit or mx4 weights, dense or grouped by expert.
//
// Bound by reading the weights once.  A workgroup owns 16 * RT weight rows and
// 16 * NT tokens of one expert; its 8 waves split the contraction, each wave
// loads both operands from memory straight into MFMA operand registers (not
// through LDS: with at most 32 tokens no element is worth sharing between
// waves), and the waves' fp32 sums meet once in LDS, added in
// wave order.  Any length, stride and alignment is taken: rows and tokens past
// the end repeat the last one (their results are not stored), and the last
// steps of a row load under guards.
//
// Measured (copy of 1 GiB: 5.2 TB/s): mx4 4096 x 4096, one bf16 token 5.9 us
// (8.9 MB; 3 to 4 us of it pass before the first weight arrives); mx4 11008 x
// 4096, 16 fp16 tokens 12.3 us; 36 of 64 mx4 experts of 2048 x 4096 43.8 us (159
// MB needed, 199 read from memory by the counters: 4.5 TB/s); two fp16
// experts of 4096 x 4096 14.1 us (67 MB, 4.8 TB/s).
//
// A wave's step is kStep contraction elements:
// * 16-bit: lane (i, g) loads 16 bytes of row i, elements 32 u + 8 g, u < 8.
// * mx4: lane (i, g) loads one 32-element block (16 bytes) of row i, block
//   4 t + g, t < 4, and one dword of scales, blocks 4 g .. 4 g + 3 of the
//   step, which the lanes of a row then exchange.  Against 16-bit activations
//   the four lane groups also exchange the blocks' dwords (four lane-swap
//   instructions), after which register j holds dword g of block 4 t + j and
//   meets elements 8 g .. 8 g + 7 of that block of the token, 64 contiguous
//   bytes a row and load.
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

// 16 bytes at a wave-uniform address plus a lane's 32-bit offset: the load
// takes both as they are, without a 64-bit address a lane.
__device__ __forceinline__ uint4 ld16(const uint8_t* base, uint32_t off, int imm) {
    uint4 v;
    __builtin_memcpy(&v, base + off + imm, 16);
    return v;
}

// Lane groups of 16 as rows, d[0 .. 3] as columns: the transpose.
__device__ __forceinline__ void transpose4(uint32_t (&d)[4]) {
    // swap the lower group of one pair of registers with the upper one of the
    // other: first over two groups (32 lanes), then over one
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const auto r = __builtin_amdgcn_permlane32_swap(d[k], d[k + 2], false, false);
        d[k] = r[0];
        d[k + 2] = r[1];
    }
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
        const auto r = __builtin_amdgcn_permlane16_swap(d[k], d[k + 1], false, false);
        d[k] = r[0];
        d[k + 1] = r[1];
    }
}

template <int MODE> constexpr int kStep = MODE == MM_MX4 ? 256 : 128;
constexpr int kRound = 4096;           // mx4: elements whose scales a workgroup holds at once, at most
constexpr int kScaleRow = kRound / kMxBlock + 16;  // LDS bytes of a row's scales; the pad spreads 16 rows over the banks

template <int MODE, int DT, int RT, int NT>
struct Skinny {
    static constexpr bool MX = MODE == MM_MX4, W4 = MODE == MM_W4;
    static constexpr int S = kStep<MODE>;
    static constexpr int UW = MODE == MM_16 ? S / 32 : S / 128;      // 16-byte loads of a weight row
    static constexpr int UX = MX ? S / 128 : S / 32;                 // and of a token row
    // Scales read by the lanes that use them are four bytes a row and load, and
    // as many memory requests as the elements: 44032 x 4096 with 16 tokens took
    // 46 us (bf16) and 35 us (mx4).  Through LDS, 16 bytes a thread for 4096
    // elements of every row, it takes 37 and 31; with fewer than 48 rows a
    // workgroup the barriers cost more than the requests.
    static constexpr bool SHARED = MODE != MM_16 && RT >= 3;
    // Steps whose loads go out together: small 16-bit workgroups leave a wave
    // with little in flight (fp16 4096 x 4096, one token: 9.6 us instead of 11.5;
    // 11008 x 4096: 21.6 instead of 23.4).  mx4 workgroups gain nothing.
    static constexpr int AHEAD = MODE != MM_16 ? 1 : RT * NT == 1 ? 4 : RT * NT == 2 ? 2 : 1;

    // One step's operands.
    struct Ops {
        uint4 w[RT][UW], x[NT][UX];
        uint32_t ws[RT], xs[NT];       // scales, where the workgroup does not share them
    };

    const MmArgs& a;
    const uint8_t *q, *p, *qs, *ps;    // the tile's first rows (wave-uniform)
    uint32_t qo[RT], po[NT], qso[RT], pso[NT];   // this lane's rows
    int64_t qrows, prows, prow0;       // rows of W from q on; the tile's rows from p on, and the first of them
    uint8_t* sc;                       // LDS: scales of 16 RT weight rows, then of 16 NT tokens (mx4 x mx4)
    int64_t nb;                        // scale bytes of a row
    int i, g;
    bool odd;                          // met a scale that the 16-bit type may not hold
    f32x4 acc[RT][NT];

    // The scales of 128 blocks from `first` on, 16 bytes a thread: from memory,
    // and into LDS.
    static constexpr int SROWS = 16 * RT + (MX ? 16 * NT : 0);
    static constexpr int SPT = (SROWS * 8 + kThreads - 1) / kThreads;
    __device__ __forceinline__ void load_scales(int64_t first, uint4 (&v)[SPT]) const {
#pragma unroll
        for (int j = 0; j < SPT; ++j) {
            const int t = j * kThreads + threadIdx.x, row = t >> 3;
            const int64_t b = first + (t & 7) * 16;
            const bool is_q = row < 16 * RT;
            const int64_t r = is_q ? std::min<int64_t>(row, qrows - 1)
                                   : std::max<int64_t>(prow0, std::min<int64_t>(row - 16 * RT, prows - 1));
            const uint8_t* at = is_q ? qs + r * a.ldqs : ps + r * a.ldps;
            v[j] = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);   // 1.0 past the end
            if (row >= SROWS) continue;
            if (b + 16 <= nb) {
                __builtin_memcpy(&v[j], at + b, 16);
            } else if (b < nb) {
                uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (b + e < nb) w[e >> 2] = (w[e >> 2] & ~(0xFFu << (8 * (e & 3)))) | ((uint32_t)at[b + e] << (8 * (e & 3)));
                v[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
    __device__ __forceinline__ void store_scales(const uint4 (&v)[SPT]) const {
#pragma unroll
        for (int j = 0; j < SPT; ++j) {
            const int t = j * kThreads + threadIdx.x, row = t >> 3;
            if (row < SROWS) *reinterpret_cast<uint4*>(sc + row * kScaleRow + (t & 7) * 16) = v[j];
        }
    }

    // scales of blocks b + 4 lg .. + 3; 1.0 past the end
    template <bool FULL>
    __device__ __forceinline__ uint32_t ld_scales(const uint8_t* base, uint32_t off, int64_t b, int lg) const {
        uint32_t v = 0x7F7F7F7Fu;
        if (FULL || b + 4 * lg + 4 <= nb) {
            __builtin_memcpy(&v, base + b + (off + 4 * lg), 4);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (b + 4 * lg + e < nb) v = (v & ~(0xFFu << (8 * e))) | ((uint32_t)(base + b)[off + 4 * lg + e] << (8 * e));
        }
        return v;
    }

    // block b + g, in a row of n blocks
    template <bool FULL>
    __device__ __forceinline__ uint4 ld_block(const uint8_t* base, uint32_t off, int64_t b, int imm) const {
        if (FULL || b + imm / 16 + g < nb) return ld16(base + b * 16, off + 16 * g, imm);
        return make_uint4(0, 0, 0, 0);
    }

    // elements k + 8 g .. + 7 of a 16-bit row.  HALF: rows may begin inside a
    // dword, where a 16-byte load is cut into many (3 fp16 experts of 4928 x
    // 2605, 37 rows: 59 us): the dwords that hold the elements, moved together.
    template <bool FULL, bool HALF>
    __device__ __forceinline__ uint4 ld_row(const uint8_t* base, uint32_t off, int64_t k, int imm) const {
        if constexpr (FULL && HALF) {
            const uint32_t b = (uint32_t)reinterpret_cast<uintptr_t>(base) & 2, m = (b + off) & 2;
            const uint32_t at = off + b - m + 16 * g;
            const uint4 v = ld16(base - b + k * 2, at, imm);
            uint32_t last;
            __builtin_memcpy(&last, base - b + k * 2 + at + imm + (m ? 16 : 12), 4);
            return make_uint4(__builtin_amdgcn_alignbit(v.y, v.x, 8 * m), __builtin_amdgcn_alignbit(v.z, v.y, 8 * m),
                              __builtin_amdgcn_alignbit(v.w, v.z, 8 * m), __builtin_amdgcn_alignbit(last, v.w, 8 * m));
        } else if constexpr (FULL) {
            return ld16(base + k * 2, off + 16 * g, imm);
        } else {
            return ld8(base + off, k + imm / 2 + 8 * g, a.C);
        }
    }

    template <bool FULL, bool HALF = false>
    __device__ __forceinline__ void load(int64_t k0, Ops& o) const {
        const int64_t b0 = k0 / kMxBlock;
        if constexpr (MODE == MM_16) {
#pragma unroll
            for (int u = 0; u < UW; ++u)
#pragma unroll
                for (int r = 0; r < RT; ++r) o.w[r][u] = ld_row<FULL, HALF>(q, qo[r], k0, 64 * u);
        } else {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int u = 0; u < UW; ++u) o.w[r][u] = ld_block<FULL>(q, qo[r], b0, 64 * u);
            if constexpr (!SHARED) {
                // (mx4 x mx4: two groups of four blocks, from lane groups 0 and 1; the others repeat them)
#pragma unroll
                for (int r = 0; r < RT; ++r) o.ws[r] = ld_scales<FULL>(qs, qso[r], b0, MX ? g & 1 : 0);
            }
        }
        if constexpr (MX) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < UX; ++u) o.x[t][u] = ld_block<FULL>(p, po[t], b0, 64 * u);
            if constexpr (!SHARED) {
#pragma unroll
                for (int t = 0; t < NT; ++t) o.xs[t] = ld_scales<FULL>(ps, pso[t], b0, g & 1);
            }
        } else {
#pragma unroll
            for (int u = 0; u < UX; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t) o.x[t][u] = ld_row<FULL, HALF>(p, po[t], k0, 64 * u);
        }
    }

    // Scale dword (blocks 4 u .. 4 u + 3 of the step) of this lane's row: row
    // tile r of the weights, or RT + t of the tokens; `at` is the LDS offset in
    // a row's scales of the step's first block
    __device__ __forceinline__ uint32_t scales(uint32_t own, int tile, int at, int u) const {
        if constexpr (SHARED) return *reinterpret_cast<const uint32_t*>(sc + (16 * tile + i) * kScaleRow + at + 4 * u);
        else return MX ? (uint32_t)__shfl((int)own, 16 * u + i) : own;
    }

    template <bool ODD>
    __device__ __forceinline__ void products(const Ops& o, int at) {
        if constexpr (MODE == MM_16) {
#pragma unroll
            for (int u = 0; u < UW; ++u)
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int t = 0; t < NT; ++t) acc[r][t] = mfma16<DT>(o.w[r][u], o.x[t][u], acc[r][t]);
        } else if constexpr (MX) {
            uint32_t sx[NT][UW];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int u = 0; u < UW; ++u)
                    sx[t][u] = scales(o.xs[t], RT + t, at, u) >> (8 * g);
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int u = 0; u < UW; ++u) {
                    const uint32_t sw = scales(o.ws[r], r, at, u) >> (8 * g);
#pragma unroll
                    for (int t = 0; t < NT; ++t) acc[r][t] = mfma_mx4<0, 0>(o.w[r][u], o.x[t][u], acc[r][t], sw, sx[t][u]);
                }
        } else {
#pragma unroll
            for (int u = 0; u < UW; ++u)
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    uint32_t d[4] = {o.w[r][u].x, o.w[r][u].y, o.w[r][u].z, o.w[r][u].w};
                    transpose4(d);
                    const uint32_t s4 = scales(o.ws[r], r, at, u);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t s = (s4 >> (8 * j)) & 0xFFu;
                        if constexpr (!ODD) {
                            odd |= mx4_unsafe<DT>(s);
                            const uint4 v = mx4_widen<DT>(d[j], __uint_as_float(s << 23));
#pragma unroll
                            for (int t = 0; t < NT; ++t) acc[r][t] = mfma16<DT>(v, o.x[t][4 * u + j], acc[r][t]);
                        } else {
                            const uint4 v = mx4_widen<DT>(d[j], 1.0f);
                            f32x4 f;
#pragma unroll
                            for (int e = 0; e < 4; ++e) f[e] = e8m0_to_f32((uint32_t)__shfl((int)s, 4 * g + e));
#pragma unroll
                            for (int t = 0; t < NT; ++t)
                                acc[r][t] += f * mfma16<DT>(v, o.x[t][4 * u + j], f32x4{0, 0, 0, 0});
                        }
                    }
                }
        }
    }

    // Whether an unsafe scale that was met matters: groups of `len` blocks, `step`
    // apart from `first` on, by thread t of n.
    __device__ __forceinline__ bool not_exact(uint32_t first, uint32_t len, uint32_t step, int t, int n) const {
        return mx4_not_exact<DT>(q, a.ldq, qs, a.ldqs, (uint32_t)std::min<int64_t>(qrows, 16 * RT), first, len, step,
                                 (uint32_t)nb, t, n);
    }

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[r][t] = f32x4{0, 0, 0, 0};
    }

    // This wave's part of the contraction: steps n, n + by, ..  ODD
    // (mx4 weights against 16-bit activations): the elements unscaled, their
    // sums scaled in fp32.  HALF: see ld_row.
    template <bool ODD, bool HALF = false>
    __device__ __forceinline__ void run_steps(int64_t n, int64_t by) {
        // a block that K ends inside is whole in an mx4 operand, not in a 16-bit one
        const int64_t whole = (MX ? nb * kMxBlock : a.C) / S, steps = (a.C + S - 1) / S;
        Ops o;
        if constexpr (!ODD && !HALF && AHEAD > 1) {
            for (; n + (AHEAD - 1) * by < whole; n += AHEAD * by) {
                Ops b[AHEAD];
#pragma unroll
                for (int d = 0; d < AHEAD; ++d) load<true>((n + d * by) * S, b[d]);
#pragma unroll
                for (int d = 0; d < AHEAD; ++d) products<ODD>(b[d], 0);
            }
        }
        for (; n < whole; n += by) {
            load<true, HALF>(n * S, o);
            products<ODD>(o, 0);
        }
        if (n < steps) {
            load<false>(n * S, o);
            products<ODD>(o, 0);
        }
    }

    __device__ __forceinline__ int slice_of(int64_t rounds) const {
        return (int)(((a.C + rounds * kWaves - 1) / (rounds * kWaves) + S - 1) / S * S);
    }

    // The same with shared scales: slice `wave` of every round of this split.  Every wave
    // takes part in the barriers.
    template <bool ODD, bool HALF = false>
    __device__ __forceinline__ void run_rounds(int wave, int split) {
        const int64_t whole = MX ? nb * kMxBlock : a.C;
        // rounds of equal length, a wave's slices of them whole steps
        const int64_t rounds = (a.C + kRound - 1) / kRound;
        const int slice = slice_of(rounds);
        for (int64_t n = split; n < rounds; n += a.splits) {
            const int64_t k0 = (n * kWaves + wave) * slice;
            uint4 v[SPT];
            load_scales(n * kWaves * slice / kMxBlock, v);
            Ops o;
            if (k0 < a.C) {            // the first step's loads are under way while the scales arrive
                if (k0 + S <= whole) load<true, HALF>(k0, o);
                else load<false>(k0, o);
            }
            if (n > split) lds_barrier();  // every wave has read the last round's scales
            store_scales(v);
            lds_barrier();
#pragma unroll 1                           // unrolled, its registers cost half the waves
            for (int h = 0; h < slice; h += S) {
                const int64_t k = k0 + h;
                if (k >= a.C) break;
                if (h > 0) {
                    if (k + S <= whole) load<true, HALF>(k, o);
                    else load<false>(k, o);
                }
                products<ODD>(o, (wave * slice + h) / kMxBlock);
            }
        }
    }
};

template <int MODE, int DT, int RT, int NT>
// (two workgroups of 64 rows x 16 tokens on a CU: within 128 registers)
__global__ void __launch_bounds__(kThreads, RT == 4 && NT == 1 ? 4 : 2) k_mm_skinny(MmArgs a, uint32_t nq) {
    using K = Skinny<MODE, DT, RT, NT>;
    constexpr int kRed = kWaves * RT * NT * 64 * 16, kSc = K::SHARED ? K::SROWS * kScaleRow : 0;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kRed > kSc ? kRed : kSc];   // the scales, then the waves' sums
    f32x4(*const red)[RT * NT * 64] = reinterpret_cast<f32x4(*)[RT * NT * 64]>(lds);
    const uint32_t per = gridDim.x / (uint32_t)a.splits, split = blockIdx.x / per, id = blockIdx.x - split * per;
    const uint32_t tt = id / nq, qt = id - tt * nq;
    MmTile tile;
    if (!mm_find_tile(a, 16 * NT, (int)tt, &tile)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t q0 = (int64_t)qt * 16 * RT;
    K k{a};
    k.sc = lds;
    k.qrows = a.Q - q0;
    k.prow0 = tile.v0 - tile.r0;
    k.prows = tile.r1 - tile.r0;
    k.i = lane & 15;
    k.g = lane >> 4;
    k.nb = (a.C + kMxBlock - 1) / kMxBlock;
    const int64_t e = tile.e < 0 ? 0 : tile.e;
    k.q = a.q + e * a.strideq + q0 * a.ldq;
    k.p = a.p + tile.r0 * a.ldp;
    k.qs = MODE != MM_16 ? a.qs + e * a.strideqs + q0 * a.ldqs : nullptr;
    k.ps = MODE == MM_MX4 ? a.ps + tile.r0 * a.ldps : nullptr;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int64_t row = std::min<int64_t>(16 * r + k.i, a.Q - 1 - q0);
        k.qo[r] = (uint32_t)(row * a.ldq);
        k.qso[r] = (uint32_t)(row * a.ldqs);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int64_t row = std::max(tile.v0, std::min<int64_t>(tile.r0 + 16 * t + k.i, tile.r1 - 1)) - tile.r0;
        k.po[t] = (uint32_t)(row * a.ldp);
        k.pso[t] = (uint32_t)(row * a.ldps);
    }
    k.zero();
    // 16-bit rows that may begin inside a dword
    const bool half = (MODE != MM_MX4 && (reinterpret_cast<uintptr_t>(k.p) | a.ldp) & 2) ||
                      (MODE == MM_16 && (reinterpret_cast<uintptr_t>(k.q) | a.ldq) & 2);
    if (tile.e >= 0 && a.C > 0) {      // (no contraction: no rounds to share out, the sums are zero)
        k.odd = false;
        if constexpr (K::SHARED) {
            if (half) k.template run_rounds<false, MODE != MM_MX4>(wave, (int)split);
            else k.template run_rounds<false>(wave, (int)split);
            if constexpr (MODE == MM_W4) {
                if (__syncthreads_or(k.odd)) {
                    const uint32_t round = kWaves * k.slice_of((a.C + kRound - 1) / kRound) / kMxBlock;
                    if (__syncthreads_or(k.not_exact((uint32_t)split * round, round, (uint32_t)a.splits * round,
                                                     threadIdx.x, kThreads))) {
                        k.zero();
                        k.template run_rounds<true>(wave, (int)split);
                    }
                }
            }
            __syncthreads();           // the scales give way to the sums
        } else {
            // splits take the steps in turn
            const int64_t first = (int64_t)split * kWaves + wave, by = (int64_t)a.splits * kWaves;
            if (half) k.template run_steps<false, MODE != MM_MX4>(first, by);
            else k.template run_steps<false>(first, by);
            if constexpr (MODE == MM_W4) {
                constexpr uint32_t B = K::S / kMxBlock;
                if (__any(k.odd) && __any(k.not_exact((uint32_t)first * B, B, (uint32_t)by * B, lane, 64))) {
                    k.zero();
                    k.template run_steps<true>(first, by);
                }
            }
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
            const int n = left < 4 ? (int)left : 4;
            if (a.part) mm_store4(a.part, OUT_F32, ((int64_t)split * a.P + p) * a.Q + q, n, v);
            else mm_store4(a.y, a.out, p * a.ldy + q, n, v);
        }
    }
}

template <int MODE, int DT, int RT, int NT>
hipError_t go(const MmArgs& a, hipStream_t s) {
    const int64_t nq = (a.Q + 16 * RT - 1) / (16 * RT);
    const int64_t tiles = mm_tile_bound(a, 16 * NT);
    if (nq * tiles * a.splits >= (int64_t)1 << 31) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_mm_skinny<MODE, DT, RT, NT>), dim3((unsigned)(nq * tiles * a.splits)), dim3(kThreads), 0, s, a,
                       (uint32_t)nq);
    return hipGetLastError();
}

template <int MODE, int DT>
hipError_t pick(const MmArgs& a, int rt, int nt, hipStream_t s) {
    if (rt == 1) return nt == 1 ? go<MODE, DT, 1, 1>(a, s) : go<MODE, DT, 1, 2>(a, s);
    if (rt == 2) return nt == 1 ? go<MODE, DT, 2, 1>(a, s) : go<MODE, DT, 2, 2>(a, s);
    if (rt == 3) return go<MODE, DT, 3, 1>(a, s);   // one token tile only (mm_abi.cpp)
    return nt == 1 ? go<MODE, DT, 4, 1>(a, s) : go<MODE, DT, 4, 2>(a, s);
}

}  // namespace

int64_t mm_tile_bound(const MmArgs& a, int T) {
    if (!a.offs) return (a.P + T - 1) / T;
    // n rows need (n - 1) / T + 1 tiles, rounded down; an mx4 tile begins up to 15
    // rows before them.  No more segments than rows have any: idle workgroups
    // are not free (2 tokens, 28 experts: 2 of 30 tiles had rows, and 6496
    // workgroups took 15 us)
    const int64_t some = std::min(a.P, a.E + 2);
    return (a.P + (a.mode == MM_MX4 ? 14 : -1) * some) / T + some;
}

hipError_t launch_mm_skinny(const MmArgs& a, int rt, int nt, hipStream_t s) {
    switch (a.mode) {
        case MM_16: return a.dt == DT_F16 ? pick<MM_16, DT_F16>(a, rt, nt, s) : pick<MM_16, DT_BF16>(a, rt, nt, s);
        case MM_MX4: return pick<MM_MX4, DT_F16>(a, rt, nt, s);
        default: return a.dt == DT_F16 ? pick<MM_W4, DT_F16>(a, rt, nt, s) : pick<MM_W4, DT_BF16>(a, rt, nt, s);
    }
}

}  // namespace ssg
