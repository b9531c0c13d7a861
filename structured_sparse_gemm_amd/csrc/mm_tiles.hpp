// mm_tiles.hpp -- tiled products of many rows: 16-bit x 16-bit in the three
// layouts of a linear layer and its gradients, mx4 x mx4, and mx4 weights x
// 16-bit activations; dense or grouped by expert.
//
// Bound by the matrix cores.  A workgroup owns a TQ x TP tile of one expert's
// Y; both operands stream through LDS in stages of 128 bytes per row (64
// 16-bit elements, 256 mx4 elements), two stages, brought by direct-to-LDS
// loads whose out-of-range offsets read as zero, so ragged edges need no
// branch.  Every wave multiplies 16-row fragments out of registers while the
// reads of the next half-stage are in flight; one barrier a stage.
//
// * Operand stored along the contraction ([row][c]): 16-byte chunk c of tile
//   row r sits at chunk c ^ ((r / 2) % 8) of the row's 128 bytes, so the 16
//   lanes an LDS cycle serves (16 rows, one chunk) meet 16 different 16-byte
//   bank groups.
// * Operand stored across it ([c][row], the weights of the input gradient and
//   both operands of the weight gradient): 64 contraction rows of T columns;
//   the transposing reads (ds_read_b64_tr_b16) hand each lane 4 consecutive
//   contraction elements of its column.  A read touches 32 bytes of 8
//   contraction rows per cycle; 32-byte unit u of row c sits at unit
//   u ^ (c % 4 + 4 * ((c / 8) % 2)), which spreads those 8 over all banks.
// * mx4 x mx4: the lane group g of a fragment takes the 32-element blocks
//   2g and 2g + 1 of a stage, one per half-stage, so that its two scale bytes
//   are one 16-bit read and the MFMA's byte select picks between them.
// * mx4 x 16-bit: a stage's 32 weight bytes a row stay 4-bit in LDS; a wave
//   widens its fragment (4 conversions) on the way into the MFMA, scaled
//   where the scale is in the type's safe range, else unscaled with the
//   product's fp32 sum scaled instead.
//
// Workgroups are dealt round-robin to the 8 XCDs; tile numbers are dealt so
// that each XCD gets a contiguous range, walked 8 row tiles at a time, which
// keeps the operand panels of the tiles in flight in its L2.  The number of
// tiles of a grouped product is known on the device only: the grid covers the
// worst case and surplus workgroups leave after counting.
#pragma once

#include <type_traits>

#include "mm_args.hpp"

namespace ssg {

constexpr int kMmGroupP = 8;           // row tiles walked together

template <int MODE, int TQ, int TP, int WQ, int WP>
struct MmLay {
    static constexpr int NW = WQ * WP;
    static constexpr int FQ = TQ / WQ / 16, FP = TP / WP / 16;       // fragments per wave
    static constexpr int CE = MODE == MM_MX4 ? 256 : 64;             // contraction elements per stage
    static constexpr int QROW = MODE == MM_W4 ? 32 : 128;            // bytes per row per stage
    static constexpr int Q_BYTES = TQ * QROW, P_BYTES = TP * 128;
    static constexpr int QS_BYTES = MODE == MM_MX4 ? TQ * 8 : MODE == MM_W4 ? TQ * 4 : 0;
    static constexpr int PS_BYTES = MODE == MM_MX4 ? TP * 8 : 0;
    static constexpr int P_AT = Q_BYTES, QS_AT = P_AT + P_BYTES, PS_AT = QS_AT + QS_BYTES;
    static constexpr int STAGE = PS_AT + PS_BYTES;
    static constexpr int LDS = 2 * STAGE;
    // loads per wave and stage; scales of small tiles are loaded by several waves alike
    static constexpr int QL = Q_BYTES / 1024 / NW, PL = P_BYTES / 1024 / NW;
    static constexpr int up(int bytes) { return bytes == 0 ? 0 : bytes / 256 >= NW ? bytes / 256 / NW : 1; }
    static constexpr int QSL = up(QS_BYTES), PSL = up(PS_BYTES);
    static_assert(QL >= 1 && PL >= 1 && Q_BYTES % (1024 * NW) == 0 && P_BYTES % (1024 * NW) == 0, "loads");
    static_assert(LDS <= 160 * 1024, "LDS");
};

typedef __attribute__((address_space(3))) i16x4 mm_lds_i16x4;

// A wave-uniform address, in scalar registers.
__device__ __forceinline__ const uint8_t* mm_uniform(const uint8_t* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<const uint8_t*>(((uint64_t)hi << 32) | lo);
}

// One operand's loads.  T rows (or columns, TR) of the tile.
template <bool TR, int T, int ROWB, int L>
struct MmLoad {
    const uint8_t* base;               // tile origin at the first stage
    int64_t ld;                        // row bytes
    int64_t left;                      // bytes (TR: rows) of the contraction from the first stage on
    uint32_t off[L];

    __device__ __forceinline__ static int swz_row(int r) { return ROWB == 128 ? (r >> 1) & 7 : 0; }
    __device__ __forceinline__ static int swz_c(int c) { return ((c & 3) | ((c >> 1) & 4)) & (T / 16 - 1); }

    // rows: valid rows of the tile (TR: valid bytes of a row, a multiple of 16 or past them whole chunks)
    __device__ __forceinline__ void init(int wave, int lane, int64_t rows) {
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int slot = (wave * L + j) * 64 + lane;
            if constexpr (TR) {
                constexpr int CPR = T / 8;
                const int c = slot / CPR, pos = slot % CPR;
                const int chunk = (((pos >> 1) ^ swz_c(c)) << 1) | (pos & 1);
                off[j] = 16 * chunk < rows ? (uint32_t)(c * ld + 16 * chunk) : kOob;
            } else {
                constexpr int CPR = ROWB / 16;
                const int r = slot / CPR, chunk = (slot % CPR) ^ swz_row(r);
                off[j] = r < rows ? (uint32_t)(r * ld + 16 * chunk) : kOob;
            }
        }
    }

    // Bring stage `it` (counted from the first) to LDS address dst.
    __device__ __forceinline__ void issue(int64_t it, uint32_t dst, int wave, int lane) const {
        const int64_t at = TR ? it * 64 * ld : it * ROWB;
        const int64_t rem64 = left - (TR ? it * 64 : it * ROWB);
        const int rem = rem64 > 0x10000 ? 0x10000 : (int)rem64;
        const __amdgpu_buffer_rsrc_t r = rsrc(mm_uniform(base + at), 0x7fffffff);
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int slot = (wave * L + j) * 64 + lane;
            bool ok;
            if constexpr (TR) ok = slot / (T / 8) < rem;
            else ok = 16 * ((slot % (ROWB / 16)) ^ swz_row(slot / (ROWB / 16))) < rem;
            dma<16>(r, dst + (wave * L + j) * 1024, ok ? off[j] : kOob);
        }
    }
};

// Scale dwords of T rows, W dwords a row, dword arrays [w][row].  Rows past
// the tile's last repeat it, so that every scale a wave meets is a real one.
template <int T, int W, int L>
struct MmScales {
    const uint8_t* base;
    int64_t left;                      // scale bytes of a row from the first stage on
    uint32_t off[L];

    __device__ __forceinline__ void init(int wave, int lane, int64_t rows, int64_t ld) {
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int slot = ((wave * L + j) * 64 + lane) % (T * W);
            const int w = slot / T, r = slot % T;
            off[j] = (uint32_t)((r < rows ? r : rows - 1) * ld + 4 * w);
        }
    }

    // `at`: byte of the row, a multiple of 4 like the row's length
    __device__ __forceinline__ void issue(int64_t at, uint32_t dst, int wave, int lane) const {
        const int64_t rem64 = left - at;
        const int rem = rem64 > 0x10000 ? 0x10000 : (int)rem64;
        const __amdgpu_buffer_rsrc_t r = rsrc(mm_uniform(base + at), 0x7fffffff);
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int piece = (wave * L + j) % (T * W / 64);
            const int w = (piece * 64 + lane) / T;
            dma<4>(r, dst + piece * 256, 4 * w < rem ? off[j] : kOob);
        }
    }
};

// Two bytes of each of N fragments (64 LDS bytes apart), two fragments a register.
template <int N>
__device__ __forceinline__ void read_u16s(const uint8_t* at, uint32_t* out) {
#pragma unroll
    for (int x = 0; x < N; x += 2) {
        out[x / 2] = *reinterpret_cast<const uint16_t*>(at + x * 64);
        if (x + 1 < N) out[x / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(at + (x + 1) * 64) << 16;
    }
}

// f(0), .., f(N - 1) with constant arguments.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void mm_for(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        mm_for<N, I + 1>(f);
    }
}

template <int NM, int ND>
__device__ __forceinline__ void mm_interleave() {
    if constexpr (NM > 0) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if constexpr (ND > 0) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        mm_interleave<NM - 1, ND - 1>();
    }
}

template <int MODE, int DT, bool QT, bool PT, int TQ, int TP, int WQ, int WP>
__global__ void __launch_bounds__(WQ* WP * 64, 2) k_mm_tiles(MmArgs a, uint32_t nq, uint32_t np) {
    using L = MmLay<MODE, TQ, TP, WQ, WP>;
    constexpr bool GC = PT;            // the experts divide the contraction (weight gradient)
    __shared__ __attribute__((aligned(1024))) uint8_t lds[L::LDS];
    const uint32_t lds32 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const lds_void*)lds);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;

    // which tile
    const uint32_t rows = GC ? np : a.offs ? (uint32_t)mm_count_tiles(a, TP) : np;
    const uint32_t per_split = rows * nq * (GC ? (uint32_t)a.E : 1u), total = per_split * (uint32_t)a.splits;
    const uint32_t chunk = (total + 7) / 8;
    uint32_t id = (blockIdx.x & 7) * chunk + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= chunk || id >= total) return;
    const int split = (int)(id / per_split);
    id -= split * per_split;
    uint32_t e_gc = 0;
    if constexpr (GC) {
        e_gc = id / (rows * nq);
        id -= e_gc * rows * nq;
    }
    const uint32_t grp = id / (kMmGroupP * nq), in = id - grp * kMmGroupP * nq;
    const uint32_t gsz = rows - grp * kMmGroupP < (uint32_t)kMmGroupP ? rows - grp * kMmGroupP : (uint32_t)kMmGroupP;
    const uint32_t qt = in / gsz, pt = grp * kMmGroupP + in - qt * gsz;

    MmTile tile;
    int64_t c_at = 0, c_len = a.C;     // this expert's part of the contraction (GC: token rows)
    if constexpr (GC) {
        int64_t lo = 0, hi = a.C;
        if (a.offs) {
            const int64_t v0 = a.offs[e_gc], v1 = a.offs[e_gc + 1];
            lo = v0 < 0 ? 0 : (v0 > a.C ? a.C : v0);
            hi = v1 < lo ? lo : (v1 > a.C ? a.C : v1);
        }
        c_at = lo;
        c_len = hi - lo;
        tile.e = (int)e_gc;
        tile.r0 = (int64_t)pt * TP;
        tile.r1 = tile.r0 + TP < a.P ? tile.r0 + TP : a.P;
    } else {
        if (!mm_find_tile(a, TP, (int)pt, &tile)) return;
    }
    const int64_t q0 = (int64_t)qt * TQ, e = tile.e < 0 ? 0 : tile.e;
    const int64_t nst_all = (c_len + L::CE - 1) / L::CE;
    const int64_t st0 = nst_all * split / a.splits, st1 = nst_all * (split + 1) / a.splits;
    const int nst = tile.e < 0 ? 0 : (int)(st1 - st0);

    constexpr int ES = 2;
    const int64_t rowb = MODE == MM_MX4 ? (a.C + kMxBlock - 1) / kMxBlock * 16 : a.C * ES;   // contraction bytes, [row][c]
    MmLoad<QT, TQ, L::QROW, L::QL> lq;
    MmLoad<PT, TP, 128, L::PL> lp;
    lq.ld = a.ldq;
    lp.ld = a.ldp;
    if constexpr (QT) {
        lq.base = a.q + (GC ? c_at * a.ldq : e * a.strideq + st0 * 64 * a.ldq) + q0 * ES;
        lq.left = GC ? c_len : c_len - st0 * 64;
        lq.init(wave, lane, (a.Q - q0) * ES);
    } else {
        const int64_t qrowb = MODE == MM_W4 ? (a.C + kMxBlock - 1) / kMxBlock * 16 : rowb;
        lq.base = a.q + e * a.strideq + q0 * a.ldq + st0 * L::QROW;
        lq.left = qrowb - st0 * L::QROW;
        lq.init(wave, lane, a.Q - q0);
    }
    if constexpr (PT) {
        lp.base = a.p + c_at * a.ldp + tile.r0 * ES;
        lp.left = c_len;
        lp.init(wave, lane, (a.P - tile.r0) * ES);
    } else {
        lp.base = a.p + tile.r0 * a.ldp + st0 * 128;
        lp.left = rowb - st0 * 128;
        lp.init(wave, lane, tile.r1 - tile.r0);
    }
    constexpr int QSW = MODE == MM_MX4 ? 2 : 1;
    MmScales<TQ, QSW, MODE == MM_16 ? 1 : L::QSL> lqs;
    MmScales<TP, 2, MODE == MM_MX4 ? L::PSL : 1> lps;
    const int64_t nb = (a.C + kMxBlock - 1) / kMxBlock;
    if constexpr (MODE != MM_16) {
        lqs.base = a.qs + e * a.strideqs + q0 * a.ldqs;
        lqs.left = nb;
        lqs.init(wave, lane, a.Q - q0, a.ldqs);
    }
    if constexpr (MODE == MM_MX4) {
        lps.base = a.ps + tile.r0 * a.ldps;
        lps.left = nb;
        lps.init(wave, lane, tile.r1 - tile.r0, a.ldps);
    }
    constexpr int VM = L::QL + L::PL + L::QSL + L::PSL;
    // stage `it` of this split into slot it % 2; one past the last writes zeros that nobody reads
    auto issue = [&](int it) {
        const uint32_t dst = lds32 + (it & 1) * L::STAGE;
        lq.issue(it, dst, wave, lane);
        lp.issue(it, dst + L::P_AT, wave, lane);
        if constexpr (MODE == MM_MX4) {
            lqs.issue((st0 + it) * 8, dst + L::QS_AT, wave, lane);
            lps.issue((st0 + it) * 8, dst + L::PS_AT, wave, lane);
        }
        // 16-bit activations: a stage needs 2 scale bytes; its dword holds those of two stages
        if constexpr (MODE == MM_W4) lqs.issue((st0 + it) / 2 * 4, dst + L::QS_AT, wave, lane);
    };

    const int wq = wave % WQ, wp = wave / WQ;
    const int fq0 = wq * L::FQ, fp0 = wp * L::FP;    // first fragments of this wave
    f32x4 acc[L::FQ][L::FP];
#pragma unroll
    for (int x = 0; x < L::FQ; ++x)
#pragma unroll
        for (int y = 0; y < L::FP; ++y) acc[x][y] = f32x4{0, 0, 0, 0};

    struct Ops {
        uint4 q[MODE == MM_W4 ? 1 : L::FQ];
        uint32_t qd[MODE == MM_W4 ? L::FQ : 1];
        uint4 p[L::FP];
    };
    struct Sc {
        uint32_t q[(L::FQ + 1) / 2], p[(L::FP + 1) / 2];   // two bytes a fragment, two fragments a register
    };
    auto frag_row = [&](const uint8_t* at, int f, int s) -> uint4 {
        const int c = MODE == MM_MX4 ? 2 * g + s : 4 * s + g;
        return *reinterpret_cast<const uint4*>(at + f * 2048 + i * 128 + ((c ^ ((i >> 1) & 7)) << 4));
    };
    auto frag_tr = [&](const uint8_t* at, int f, int s, auto tc) -> uint4 {
        constexpr int T = decltype(tc)::value;
        const int fx = (((i >> 2) & 3) | ((g & 1) << 2)) & (T / 16 - 1);
        const uint8_t* p = at + (32 * s + 8 * g + (i >> 2)) * (T * 2) + ((f ^ fx) << 5) + ((i & 3) << 3);
        union { i16x4 v[2]; uint4 u; } r;
        r.v[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((mm_lds_i16x4*)(p));
        r.v[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((mm_lds_i16x4*)(p + 4 * T * 2));
        return r.u;
    };
    auto read_ops = [&](const uint8_t* st, int s, Ops& o) {
#pragma unroll
        for (int x = 0; x < L::FQ; ++x) {
            if constexpr (MODE == MM_W4)
                o.qd[x] = *reinterpret_cast<const uint32_t*>(st + ((fq0 + x) * 16 + i) * 32 + s * 16 + g * 4);
            else if constexpr (QT) o.q[x] = frag_tr(st, fq0 + x, s, std::integral_constant<int, TQ>{});
            else o.q[x] = frag_row(st, fq0 + x, s);
        }
#pragma unroll
        for (int y = 0; y < L::FP; ++y) {
            if constexpr (PT) o.p[y] = frag_tr(st + L::P_AT, fp0 + y, s, std::integral_constant<int, TP>{});
            else o.p[y] = frag_row(st + L::P_AT, fp0 + y, s);
        }
    };
    auto read_sc = [&](const uint8_t* st, int64_t stage, Sc& o) {
        if constexpr (MODE == MM_MX4) {
            const uint8_t* at = st + (g >> 1) * (TQ * 4) + (g & 1) * 2 + L::QS_AT + i * 4;
            read_u16s<L::FQ>(at + fq0 * 64, o.q);
            at = st + (g >> 1) * (TP * 4) + (g & 1) * 2 + L::PS_AT + i * 4;
            read_u16s<L::FP>(at + fp0 * 64, o.p);
        }
        if constexpr (MODE == MM_W4) {
            const uint8_t* at = st + L::QS_AT + i * 4 + (stage & 1) * 2;
            read_u16s<L::FQ>(at + fq0 * 64, o.q);
        }
    };
    bool odd = false;                  // MM_W4: this lane met a scale outside the safe range
    auto mmas = [&](const Ops& o, const Sc& sc, auto half) {
        constexpr int S = decltype(half)::value;
        if constexpr (MODE == MM_16) {
#pragma unroll
            for (int y = 0; y < L::FP; ++y)
#pragma unroll
                for (int x = 0; x < L::FQ; ++x) acc[x][y] = mfma16<DT>(o.q[x], o.p[y], acc[x][y]);
        } else if constexpr (MODE == MM_MX4) {
            mm_for<L::FP>([&](auto yc) {
                mm_for<L::FQ>([&](auto xc) {
                    constexpr int x = decltype(xc)::value, y = decltype(yc)::value;
                    acc[x][y] = mfma_mx4<2 * (x & 1) + S, 2 * (y & 1) + S>(o.q[x], o.p[y], acc[x][y], sc.q[x / 2],
                                                                           sc.p[y / 2]);
                });
            });
        } else {
            uint4 w[L::FQ];
#pragma unroll
            for (int x = 0; x < L::FQ; ++x) {
                const uint32_t v = (sc.q[x / 2] >> (16 * (x & 1) + 8 * S)) & 0xFFu;
                odd |= v - kSafeLo<DT> > kSafeHi<DT> - kSafeLo<DT>;
                w[x] = mx4_widen<DT>(o.qd[x], __uint_as_float(v << 23));
            }
#pragma unroll
            for (int y = 0; y < L::FP; ++y)
#pragma unroll
                for (int x = 0; x < L::FQ; ++x) acc[x][y] = mfma16<DT>(w[x], o.p[y], acc[x][y]);
        }
    };
    constexpr int NMMA = L::FQ * L::FP;
    constexpr int NRD = L::FQ * (QT ? 2 : 1) + L::FP * (PT ? 2 : 1);
    constexpr int NSC = MODE == MM_MX4 ? L::FQ + L::FP : 0;

    if (nst > 0) {
        using H0 = std::integral_constant<int, 0>;
        using H1 = std::integral_constant<int, 1>;
        issue(0);
        issue(1);
        wait_vm<VM>();
        lds_barrier();
        Ops o0, o1;
        Sc sc, sn;
        read_ops(lds, 0, o0);
        read_sc(lds, st0, sc);
        for (int it = 0; it < nst; ++it) {
            read_ops(lds + (it & 1) * L::STAGE, 1, o1);
            mmas(o0, sc, H0{});
            if constexpr (MODE != MM_W4) mm_interleave<NMMA, NRD>();
            // stage it + 1 has landed, and this wave has read all of stage it
            wait_vm<0>();
            lds_barrier();
            issue(it + 2);
            const uint8_t* nx = lds + ((it + 1) & 1) * L::STAGE;
            read_ops(nx, 0, o0);
            read_sc(nx, st0 + it + 1, sn);
            mmas(o1, sc, H1{});
            if constexpr (MODE != MM_W4) mm_interleave<NMMA, NRD + NSC>();
            sc = sn;
        }
        wait_vm<0>();                  // no load of this workgroup may land after it ends
    }

    if constexpr (MODE == MM_W4) {
        // Scales that the 16-bit type cannot hold (they never come from weights
        // of ordinary magnitude): this wave's products once more, a block at a
        // time from memory, unscaled, each sum scaled in fp32.  Kept out of the
        // main loop, where a second path would double the accumulators.
        if (__any(odd)) {
#pragma unroll
            for (int x = 0; x < L::FQ; ++x)
#pragma unroll
                for (int y = 0; y < L::FP; ++y) acc[x][y] = f32x4{0, 0, 0, 0};
            const int64_t b1 = st1 * 2 < nb ? st1 * 2 : nb;
            for (int64_t b = st0 * 2; b < b1; ++b) {
                uint4 pv[L::FP];
#pragma unroll
                for (int y = 0; y < L::FP; ++y) {
                    const int64_t r = tile.r0 + (fp0 + y) * 16 + i, at = b * 64 + g * 16;
                    pv[y] = make_uint4(0, 0, 0, 0);
                    if (r < tile.r1 && at < rowb) pv[y] = *reinterpret_cast<const uint4*>(a.p + r * a.ldp + at);
                }
#pragma unroll
                for (int x = 0; x < L::FQ; ++x) {
                    const int64_t r = q0 + (fq0 + x) * 16 + i, row = r < a.Q ? r : a.Q - 1;
                    const uint32_t d = *reinterpret_cast<const uint32_t*>(a.q + e * a.strideq + row * a.ldq + b * 16 + g * 4);
                    const uint32_t sv = a.qs[e * a.strideqs + row * a.ldqs + b];
                    const uint4 w = mx4_widen<DT>(d, 1.0f);
                    f32x4 f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) f[k] = e8m0_to_f32((uint32_t)__shfl((int)sv, 4 * g + k));
#pragma unroll
                    for (int y = 0; y < L::FP; ++y) acc[x][y] += f * mfma16<DT>(w, pv[y], f32x4{0, 0, 0, 0});
                }
            }
        }
    }

    // lane (i, g), register r: row p = i, column q = 4g + r of its fragment pair
    const bool vec = a.part ? a.Q % 4 == 0 : a.ldy % 4 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0 &&
                                                 (a.stridey % 4 == 0);
#pragma unroll
    for (int y = 0; y < L::FP; ++y) {
        const int64_t p = tile.r0 + (fp0 + y) * 16 + i;
        if (p >= tile.r1) continue;
#pragma unroll
        for (int x = 0; x < L::FQ; ++x) {
            const int64_t q = q0 + (fq0 + x) * 16 + 4 * g;
            if (q >= a.Q) continue;
            const int n = a.Q - q < 4 ? (int)(a.Q - q) : 4;
            if (a.part) mm_store4(a.part, OUT_F32, ((int64_t)split * a.P + p) * a.Q + q, n, vec, acc[x][y]);
            else mm_store4(a.y, a.out, (GC ? e * a.stridey : 0) + p * a.ldy + q, n, vec, acc[x][y]);
        }
    }
}

template <int MODE, int DT, bool QT, bool PT, int TQ, int TP, int WQ, int WP>
hipError_t mm_tiles_go(const MmArgs& a, hipStream_t s) {
    const int64_t nq = (a.Q + TQ - 1) / TQ, np = (a.P + TP - 1) / TP;
    const int64_t tiles = PT ? np * a.E : mm_tile_bound(a, TP);
    const int64_t total = tiles * nq * a.splits;
    if (total >= (int64_t)1 << 31) return hipErrorInvalidValue;
    const unsigned grid = (unsigned)((total + 7) / 8 * 8);
    hipLaunchKernelGGL((k_mm_tiles<MODE, DT, QT, PT, TQ, TP, WQ, WP>), dim3(grid), dim3(WQ * WP * 64), 0, s, a,
                       (uint32_t)nq, (uint32_t)np);
    return hipGetLastError();
}

template <int MODE, int DT, bool QT, bool PT>
hipError_t mm_tiles_size(const MmArgs& a, int size, hipStream_t s) {
    switch (size) {
        // mx4 weights stay 4-bit until a wave multiplies them: 128 x 64 a wave holds
        // fewer 16-bit fragments than 64 x 128, which would spill
        case 0: return mm_tiles_go<MODE, DT, QT, PT, 256, 256, MODE == MM_W4 ? 2 : 4, MODE == MM_W4 ? 4 : 2>(a, s);
        case 1: return mm_tiles_go<MODE, DT, QT, PT, 128, 128, 2, 2>(a, s);
        default: return mm_tiles_go<MODE, DT, QT, PT, 128, 64, 4, 1>(a, s);
    }
}

}  // namespace ssg
