// mm_tiles.hpp -- tiled products of many rows: 16-bit x 16-bit in the three
// layouts of a linear layer and its gradients, mx4 x mx4, and mx4 weights x
// 16-bit activations; dense or grouped by expert.
//
// Bound by the matrix cores.  A workgroup owns a TQ x TP tile of one expert's
// Y; both operands stream through LDS in stages of 64 bytes per row (32 16-bit
// elements, 128 mx4 elements), brought by direct-to-LDS loads whose
// out-of-range offsets read as zero, so ragged edges need no branch.  A wave
// reads the 16-row fragments of stage i + 1 into registers while it multiplies
// those of stage i, so stage i's slot is free as soon as the barrier that opens
// stage i has passed: with a ring of 4 slots the loads run up to four
// stages ahead, which covers their latency (two whole stages of 128 bytes a
// row, the same LDS, left it exposed: bf16 8 x 4096 x 4096 with 8192 tokens
// took 345 us).
//
// * Operand stored along the contraction ([row][c]): of a group of 64 tile
//   rows, row 4 i + f is row i of fragment f.  A lane then holds 16
//   consecutive columns of Y (whole 16-byte stores), and the scale bytes of
//   its four fragments are one dword.  16-byte chunk c of fragment row i sits
//   at chunk c ^ mm_swz(i) of its 64 bytes; the permutation is the fastest of
//   all parity pairs of row bits under the LDS read probe (as fast as a
//   lane-contiguous read).
// * Operand stored across it ([c][row], the weights of the input gradient and
//   both operands of the weight gradient): 32 contraction rows of T columns;
//   the transposing reads (ds_read_b64_tr_b16) hand each lane 4 consecutive
//   contraction elements of its column.  A read touches 32 bytes of 8
//   contraction rows per cycle; 32-byte unit u of row c sits at unit
//   u ^ (c % 4 + 4 * ((c / 8) % 2)), which spreads those 8 over all banks.
// * mx4 x mx4: lane group g of a fragment takes block g of the stage; the
//   scales were brought into planes [stage][g][row] beforehand, so a stage's
//   are 1 KiB an operand in contiguous pieces (read from their rows they are
//   four bytes a row and triple the number of memory requests: 357 us against
//   the products' own time at 28672 x 8192 x 2048).
// * mx4 x 16-bit: weights come 64 bytes and one dword of scales a row (128
//   elements) every fourth stage and stay 4-bit in LDS; a wave widens its
//   fragment (4 conversions) on the way into the MFMA.
//
// Measured, by card: 16-bit 4096^3 108 to 114 us, 1.2 to 1.27 PFLOP/s (the vendor's
// product 94 to 97 us), its input gradient 109 to 127 us, weight gradient 111 to
// 127; mx4 x mx4 44 us, 3.1 PFLOP/s; mx4 x 16-bit 104 to 109 us.  8192^3: 1.29 to
// 1.39 PFLOP/s (vendor: 1.3 to 1.6 on the same cards), mx4 x mx4 4.2 to 4.3.  The
// matrix units are busy 39 to 49% of the cycles of the cases of a layer's size.
//
// Workgroups are dealt round-robin to the 8 XCDs; tile numbers are dealt so
// that each XCD gets a contiguous range, walked 8 row tiles at a time, which
// keeps the operand panels of the tiles in flight in its L2.  The number of
// tiles of a grouped product is known on the device only: the grid covers the
// worst case and surplus workgroups leave after counting.  The tiles of the
// last, partly filled round of the chip's 256 CUs are cut in two or in four
// where that many fit in one round.
#pragma once

#include <type_traits>

#include "mm_args.hpp"

namespace ssg {

constexpr int kMmGroupP = 8;           // row tiles walked together
constexpr int kMmCUs = 256;

__device__ __forceinline__ int mm_swz(int i) { return ((i ^ (i >> 1)) & 1) | ((i >> 1) & 2); }

typedef __attribute__((address_space(3))) i16x4 mm_lds_i16x4;

// A wave-uniform address, in scalar registers.
__device__ __forceinline__ const uint8_t* mm_uniform(const uint8_t* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<const uint8_t*>(((uint64_t)hi << 32) | lo);
}

// A 16-byte direct-to-LDS load: lane l's bytes from offset voff of the buffer
// (base, hi, bytes, flags) land at LDS address dst + IMM + 16 l; dwords past
// the buffer's bytes read as zero.  The kernel counts these loads itself
// (wait_vm); GFX9 needs one wait state between the write of M0 and the load.
template <int IMM>
__device__ __forceinline__ void mm_dma(i32x4 buf, uint32_t dst, uint32_t voff) {
    asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds" ::"s"(dst), "n"(IMM),
                 "v"(voff), "s"(buf)
                 : "memory", "m0", "scc");
}

// A tile of T rows by 64 bytes (TR: 32 contraction rows by T columns) as
// 1 KiB loads, L a wave.  Stages are opened in order.  Scalar instructions
// between the products are not free (a dozen more a stage cost 8% of the
// rate), so each kind has the cheapest ends that are exact for it:
//   MASK: rows of mx4 elements and of a TR operand.  Lanes past the tile's rows
//     or columns, past the contraction in the ragged stage, and whole stages
//     past the last read zeros.
//   else: rows of 16-bit elements along the contraction.  Rows past the tile's
//     are past the buffer and read as zero; what the last stage brings of the
//     next row is cleared in LDS (clear()); stages past the last bring what
//     nobody reads.
template <bool TR, int T, int L, bool MASK>
struct MmLoad {
    static_assert(MASK || !TR, "a TR operand's ends are masked");
    uint32_t lo, hi;                   // origin of the next stage
    int lim, dec;                      // bytes from there that may be read, and how many fewer a stage later
    int64_t step;                      // bytes from a stage to the next
    int last, ragged, tail;            // stages; the one that ends inside its 64 bytes (TR: 32 rows), and where
    int at;                            // MASK: this lane's place in a stage (TR: of load 0)
    uint32_t off[L];

    // tile row of an LDS fragment row
    __device__ __forceinline__ static int row_of(int slot) { return (slot & ~63) + 4 * (slot & 15) + ((slot >> 4) & 3); }
    __device__ __forceinline__ static int swz_c(int c) { return ((c & 3) | ((c >> 1) & 4)) & (T / 16 - 1); }

    // rows: the tile's rows from `base` on (TR: contraction rows from the first
    // stage on); bytes: what a row holds from `base` on; nst: stages of this
    // workgroup.  Rows of 16-bit elements need 4-byte alignment; a dword that
    // the last one ends inside is read whole (it lies in the same aligned
    // memory), and where rows may end inside a chunk (TR: bytes % 16) the
    // buffer ends with the last of them (those of 2^31 bytes and more come
    // here as copies with whole chunks).
    __device__ __forceinline__ void init(const uint8_t* base, int64_t ld, int64_t rows, int64_t bytes, int nst,
                                         int wave, int lane) {
        const uint64_t p = reinterpret_cast<uint64_t>(base);
        lo = __builtin_amdgcn_readfirstlane((uint32_t)p);
        hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
        step = TR ? 32 * ld : 64;
        last = nst;
        const int64_t n = TR ? rows : (rows < T ? rows : T), end = n > 0 ? (n - 1) * ld + (bytes + 3) / 4 * 4 : 0;
        const bool exact = !MASK || (TR && bytes % 16 != 0 && end <= 0x7fffffff);
        lim = exact ? (int)end : 0x7fffffff;
        dec = exact ? (int)step : 0;
        const int64_t left = TR ? rows : bytes;
        constexpr int U = TR ? 32 : 64;
        ragged = left < (int64_t)nst * U ? nst - 1 : -1;
        tail = (int)(left - (int64_t)(nst - 1) * U < U ? left - (int64_t)(nst - 1) * U : U);
        at = TR ? (wave * L * 64 + lane) / (T / 8) : 16 * ((lane & 3) ^ mm_swz(lane >> 2));
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int unit = (wave * L + j) * 64 + lane;
            if constexpr (TR) {
                constexpr int CPR = T / 8;
                const int c = unit / CPR, pos = unit % CPR;
                const int chunk = (((pos >> 1) ^ swz_c(c)) << 1) | (pos & 1);
                off[j] = 16 * chunk < bytes ? (uint32_t)(c * ld + 16 * chunk) : kOob;
            } else {
                const int slot = unit >> 2, r = row_of(slot);
                off[j] = !MASK || r < rows ? (uint32_t)(r * ld + 16 * ((unit & 3) ^ mm_swz(slot & 15))) : kOob;
            }
        }
    }

    // Buffer of stage `it`, the next.
    __device__ __forceinline__ i32x4 open(int it) {
        const i32x4 r = {(int)lo, (int)hi, MASK ? (it < last ? lim : 0) : (lim > 0 ? lim : 0), 0x00020000};
        const uint64_t p = (((uint64_t)hi << 32) | lo) + step;
        lo = (uint32_t)p;
        hi = (uint32_t)(p >> 32);
        if constexpr (TR || !MASK) lim -= dec;
        return r;
    }
    // Load J of stage `it` to LDS address dst + AT + (this wave's part).  No
    // branch: it would cut the block that the products are scheduled in.
    template <int J, int AT>
    __device__ __forceinline__ void load(i32x4 r, int it, uint32_t dst) const {
        if constexpr (MASK) {
            const int end = (it == ragged ? tail : 64) - (TR ? J * (64 / (T / 8)) : 0);
            mm_dma<AT + J * 1024>(r, dst, at < end ? off[J] : kOob);
        } else {
            mm_dma<AT + J * 1024>(r, dst, off[J]);
        }
    }
    // The contraction may end inside the last stage: this wave's own chunks
    // (which have landed) from there on become zeros.
    __device__ __forceinline__ void clear(uint8_t* st, int wave, int lane) const {
        const int n = tail - 16 * ((lane & 3) ^ mm_swz(lane >> 2));   // bytes of the lane's chunk that stay
        if (n >= 16) return;
#pragma unroll
        for (int j = 0; j < L; ++j) {
            uint32_t* const d = reinterpret_cast<uint32_t*>(st + (wave * L + j) * 1024 + lane * 16);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (4 * k >= n) d[k] = 0;
        }
    }
};

// The scale planes of T rows, 4 a stage: T / 16 lanes of 16 bytes a plane,
// one load for the workgroup (every wave that issues it brings the same bytes).
struct MmScales {
    const uint8_t* next;
    int64_t step;
    int last;
    uint32_t off;

    __device__ __forceinline__ void init(const uint8_t* base, int64_t plane, int T, int nst, int lane) {
        next = mm_uniform(base);
        step = 4 * plane;
        last = nst;
        const int pl = lane / (T / 16), at = lane % (T / 16);
        off = pl < 4 ? (uint32_t)(pl * plane + 16 * at) : kOob;
    }
    // (past the last stage: zeros that nobody reads)
    __device__ __forceinline__ void issue(int it, uint32_t dst) {
        const uint8_t* p = next;
        next += step;
        dma<16>(rsrc(p, it < last ? 0x7fffffff : 0), dst, off);
    }
};

// mx4 weights against 16-bit activations: one dword of scales of each of T
// rows, in fragment order, for four stages; a wave brings 64 rows.
template <int T>
struct MmRowScales {
    const uint8_t* next;
    int last;
    uint32_t off, dst;

    // rows past the last repeat it, so that every scale a wave meets is a real one
    __device__ __forceinline__ void init(const uint8_t* base, int64_t ld, int groups, int wave, int lane, int64_t rows) {
        next = mm_uniform(base);
        last = groups;
        const int piece = wave % (T / 64), r = piece * 64 + 4 * (lane & 15) + (lane >> 4);
        off = (uint32_t)((r < rows ? r : rows - 1) * ld);
        dst = piece * 256;
    }
    __device__ __forceinline__ void issue(int grp, uint32_t at) {
        const uint8_t* p = next;
        next += 4;
        dma<4>(rsrc(p, grp < last ? 0x7fffffff : 0), at + dst, off);
    }
};

// f(0), .., f(N - 1) with constant arguments.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void mm_for(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        mm_for<N, I + 1>(f);
    }
}

// What a workgroup computes: rows [v0, r1) of the tile that begins at row r0
// and column q0, of expert e (-1: zeros), over stages [st0, st0 + nst) of the
// contraction that begins at c_at and is c_len long.
struct MmWork {
    int e, split;
    int64_t r0, v0, r1, q0, c_at, c_len, st0;
    int nst;
};

template <int MODE, int TQ, int TP, int WQ, int WP>
struct MmLay {
    static constexpr int NW = WQ * WP;
    // stages in the ring (eight of the small tile's gain nothing: 18.5 against
    // 18.9 us at 4096 x 4096 with 32 tokens, bf16)
    static constexpr int kRing = 4;
    static constexpr int FQ = TQ / WQ / 16, FP = TP / WP / 16;       // fragments per wave
    static constexpr bool W4 = MODE == MM_W4, MX = MODE == MM_MX4;
    static constexpr int Q_BYTES = TQ * 64, P_BYTES = TP * 64;
    static constexpr int QS_BYTES = MX || W4 ? 1024 : 0, PS_BYTES = MX ? 1024 : 0;
    // a ring slot holds a stage's P (and Q); mx4 weights against 16-bit
    // activations have slots of their own, each for four stages
    static constexpr int P_AT = W4 ? 0 : Q_BYTES, QS_AT = P_AT + P_BYTES, PS_AT = QS_AT + (W4 ? 0 : QS_BYTES);
    static constexpr int STAGE = PS_AT + PS_BYTES;
    static constexpr int W_AT = kRing * STAGE, W_SLOT = Q_BYTES + QS_BYTES;
    static constexpr int WS = kRing / 4 + 1;                          // those slots
    static constexpr int LDS = kRing * STAGE + (W4 ? WS * W_SLOT : 0);
    static constexpr int QL = Q_BYTES / 1024 / NW, PL = P_BYTES / 1024 / NW;
    static constexpr int VM = W4 ? PL : QL + PL + (MX ? 1 : 0);      // loads per wave and stage
    static constexpr int VMW = W4 ? QL + 1 : 0;                       // and per four stages of weights
    static_assert(QL >= 1 && PL >= 1 && Q_BYTES % (1024 * NW) == 0 && P_BYTES % (1024 * NW) == 0, "loads");
    static_assert(FQ % 4 == 0 && (FP % 4 == 0 || FP == 2 || FP == 1), "fragments");
    static_assert(LDS <= 160 * 1024, "LDS");
};

// 16 bytes of outputs (n of the elements that they hold exist) to any address.
template <int ES>
__device__ __forceinline__ void mm_store_chunk(uint8_t* at, int64_t n, uint4 v) {
    if (n * ES >= 16) {
        __builtin_memcpy(at, &v, 16);
    } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 16 / ES; ++k) {
            if (k < n) {
                if constexpr (ES == 4) __builtin_memcpy(at + 4 * k, &w[k], 4);
                else {
                    const uint16_t h = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
                    __builtin_memcpy(at + 2 * k, &h, 2);
                }
            }
        }
    }
}

template <int MODE, int DT, bool QT, bool PT, int TQ, int TP, int WQ, int WP>
__device__ __forceinline__ void mm_tile(const MmArgs& a, const MmWork& w, uint8_t* lds) {
    using L = MmLay<MODE, TQ, TP, WQ, WP>;
    constexpr bool W4 = L::W4, MX = L::MX;
    const uint32_t lds32 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const lds_void*)lds);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int64_t e = w.e < 0 ? 0 : w.e;
    const int64_t nb = (a.C + kMxBlock - 1) / kMxBlock;
    constexpr int ES = 2;

    MmLoad<QT, TQ, L::QL, MODE != MM_16 || QT> lq;
    MmLoad<PT, TP, L::PL, MODE != MM_16 || PT> lp;
    const int groups = (w.nst + 3) / 4;              // W4: a load of weights covers four stages
    const int64_t qrow = MX || W4 ? nb * 16 : QT ? a.Q * ES : a.C * ES, prow = MX ? nb * 16 : PT ? a.P * ES : a.C * ES;
    if constexpr (QT) {
        lq.init(a.q + (PT ? w.c_at * a.ldq : e * a.strideq) + w.st0 * 32 * a.ldq + w.q0 * ES, a.ldq,
                w.c_len - w.st0 * 32, qrow - w.q0 * ES, w.nst, wave, lane);
    } else {
        const int64_t at = W4 ? w.st0 / 4 * 64 : w.st0 * 64;         // W4: splits begin at whole groups of four stages
        lq.init(a.q + e * a.strideq + w.q0 * a.ldq + at, a.ldq, a.Q - w.q0, qrow - at, W4 ? groups : w.nst, wave, lane);
    }
    if constexpr (PT)
        lp.init(a.p + (w.c_at + w.st0 * 32) * a.ldp + w.r0 * ES, a.ldp, w.c_len - w.st0 * 32, prow - w.r0 * ES, w.nst,
                wave, lane);
    else
        lp.init(a.p + w.r0 * a.ldp + w.st0 * 64, a.ldp, w.r1 - w.r0, prow - w.st0 * 64, w.nst, wave, lane);
    // one scale load a wave: mx4 x mx4, those of Q from even waves and of P from odd ones
    MmScales ls;
    MmRowScales<TQ> lw;
    const bool odd_wave = MX && (wave & 1);
    if constexpr (MX) {
        const uint8_t* const qs = a.qs + e * a.strideqs + w.st0 * 4 * a.ldqs + w.q0;
        const uint8_t* const ps = a.ps + w.st0 * 4 * a.ldps + w.r0;
        ls.init(odd_wave ? ps : qs, odd_wave ? a.ldps : a.ldqs, odd_wave ? TP : TQ, w.nst, lane);
    }
    if constexpr (W4)
        lw.init(a.qs + e * a.strideqs + w.q0 * a.ldqs + w.st0, a.ldqs, groups, wave, lane, a.Q - w.q0);
    const int sdst = odd_wave ? L::PS_AT : L::QS_AT;
    // load U of stage `it` into its ring slot; past the last stage: zeros, or what nobody reads
    i32x4 rq, rp;
    const uint32_t wave_q = lds32 + wave * L::QL * 1024, wave_p = lds32 + wave * L::PL * 1024;
    auto load = [&](auto uc, int it) {
        constexpr int U = decltype(uc)::value, NQ = W4 ? 0 : L::QL;
        const uint32_t slot = (it & (L::kRing - 1)) * L::STAGE;
        if constexpr (U < NQ) {
            if constexpr (U == 0) rq = lq.open(it);
            lq.template load<U, 0>(rq, it, slot + wave_q);
        } else if constexpr (U < NQ + L::PL) {
            if constexpr (U == NQ) rp = lp.open(it);
            lp.template load<U - NQ, L::P_AT>(rp, it, slot + wave_p);
        } else if constexpr (MX) {
            ls.issue(it, lds32 + slot + sdst);
        }
    };
    auto issue = [&](int it) { mm_for<L::VM>([&](auto u) { load(u, it); }); };
    auto issue_w = [&](int grp) {
        const uint32_t slot = grp % L::WS * L::W_SLOT;
        rq = lq.open(grp);
        mm_for<L::QL>([&](auto u) { lq.template load<decltype(u)::value, L::W_AT>(rq, grp, slot + wave_q); });
        lw.issue(grp, lds32 + L::W_AT + slot + L::Q_BYTES);
    };

    const int wq = wave % WQ, wp = wave / WQ;
    const int fq0 = wq * L::FQ, fp0 = wp * L::FP;    // first fragments of this wave
    f32x4 acc[L::FQ][L::FP];
#pragma unroll
    for (int x = 0; x < L::FQ; ++x)
#pragma unroll
        for (int y = 0; y < L::FP; ++y) acc[x][y] = f32x4{0, 0, 0, 0};

    constexpr int SQ = W4 ? L::FQ : MX ? L::FQ / 4 : 1, SP = MX ? (L::FP + 3) / 4 : 1;
    struct Ops {
        uint4 q[W4 ? 1 : L::FQ];
        uint32_t qd[W4 ? L::FQ : 1];
        uint4 p[L::FP];
        uint32_t qs[MX ? SQ : 1], ps[SP];   // scale bytes, four fragments a register
    };
    uint32_t wsc[W4 ? L::FQ : 1];      // W4: scale bytes of a fragment's rows, four stages a register
    auto frag_row = [&](const uint8_t* at, int f) -> uint4 {
        return *reinterpret_cast<const uint4*>(at + f * 1024 + i * 64 + ((g ^ mm_swz(i)) << 4));
    };
    auto frag_tr = [&](const uint8_t* at, int f, auto tc) -> uint4 {
        constexpr int T = decltype(tc)::value;
        const int fx = (((i >> 2) & 3) | ((g & 1) << 2)) & (T / 16 - 1);
        const uint8_t* p = at + (8 * g + (i >> 2)) * (T * 2) + ((f ^ fx) << 5) + ((i & 3) << 3);
        union { i16x4 v[2]; uint4 u; } r;
        r.v[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((mm_lds_i16x4*)(p));
        r.v[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((mm_lds_i16x4*)(p + 4 * T * 2));
        return r.u;
    };
    // read U of stage `it`'s operands: scales, Q fragments, P fragments
    constexpr int NS = MX ? SQ + SP : 0, NRD = NS + L::FQ + L::FP;
    auto read = [&](auto uc, int it, Ops& o) {
        constexpr int U = decltype(uc)::value;
        const uint8_t* st = lds + (it & (L::kRing - 1)) * L::STAGE;
        const uint8_t* ws = lds + L::W_AT + (it >> 2) % L::WS * L::W_SLOT;   // W4 only
        const int b = it & 3;                                              // W4: block of the group
        if constexpr (U < NS) {
            if constexpr (U < SQ)
                o.qs[U] = *reinterpret_cast<const uint32_t*>(st + L::QS_AT + g * TQ + (fq0 + 4 * U) * 16 + 4 * i);
            else {
                constexpr int Y = U - SQ;
                o.ps[Y] = *reinterpret_cast<const uint32_t*>(st + L::PS_AT + g * TP + ((fp0 + 4 * Y) & ~3) * 16 + 4 * i);
                if constexpr (L::FP < 4) o.ps[Y] >>= 8 * (fp0 & 3);
            }
        } else if constexpr (U < NS + L::FQ) {
            constexpr int X = U - NS;
            if constexpr (W4)
                o.qd[X] = *reinterpret_cast<const uint32_t*>(ws + (fq0 + X) * 1024 + i * 64 + ((b ^ mm_swz(i)) << 4) + g * 4);
            else if constexpr (QT) o.q[X] = frag_tr(st, fq0 + X, std::integral_constant<int, TQ>{});
            else o.q[X] = frag_row(st, fq0 + X);
        } else {
            constexpr int Y = U - NS - L::FQ;
            if constexpr (PT) o.p[Y] = frag_tr(st + L::P_AT, fp0 + Y, std::integral_constant<int, TP>{});
            else o.p[Y] = frag_row(st + L::P_AT, fp0 + Y);
        }
    };
    auto row_scales = [&](int it, int x) -> uint32_t {   // W4
        return *reinterpret_cast<const uint32_t*>(lds + L::W_AT + (it >> 2) % L::WS * L::W_SLOT + L::Q_BYTES +
                                                  (fq0 + x) * 64 + i * 4);
    };
    bool odd = false;                  // W4: this lane met a scale outside the safe range
    // a stage's products in NG groups: those of one P fragment with every Q
    // fragment, or (W4) those of one Q fragment, widened a group ahead
    constexpr int NG = W4 ? L::FQ : L::FP;
    auto widen = [&](auto xc, int b, const Ops& o) -> uint4 {
        constexpr int X = decltype(xc)::value;
        const uint32_t s = (wsc[X] >> (8 * b)) & 0xFFu;
        odd |= mx4_unsafe<DT>(s);
        return mx4_widen<DT>(o.qd[X], __uint_as_float(s << 23));
    };
    auto mmas = [&](auto gc, const Ops& o, uint4 v) {
        constexpr int G = decltype(gc)::value;
        if constexpr (W4) {
#pragma unroll
            for (int y = 0; y < L::FP; ++y) acc[G][y] = mfma16<DT>(v, o.p[y], acc[G][y]);
        } else {
            mm_for<L::FQ>([&](auto xc) {
                constexpr int X = decltype(xc)::value;
                if constexpr (MX) acc[X][G] = mfma_mx4<X % 4, G % 4>(o.q[X], o.p[G], acc[X][G], o.qs[X / 4], o.ps[G / 4]);
                else acc[X][G] = mfma16<DT>(o.q[X], o.p[G], acc[X][G]);
            });
        }
    };

    // the stage that the contraction of 16-bit rows ends inside of, or -1
    const int part = MODE == MM_16 && !PT && a.C % 32 != 0 && (w.st0 + w.nst) * 32 >= a.C ? w.nst - 1 : -1;
    auto clear_part = [&]() {
        uint8_t* const st = lds + (part & (L::kRing - 1)) * L::STAGE;
        if constexpr (!QT) lq.clear(st, wave, lane);
        if constexpr (!PT) lp.clear(st + L::P_AT, wave, lane);
    };
    if (w.nst > 0) {
        // (W4) the weights of group m follow the activations of stage 4 m - 1,
        // here and in the loop
        if constexpr (W4) issue_w(0);
#pragma unroll
        for (int s = 0; s < L::kRing; ++s) {
            issue(s);
            if (W4 && s % 4 == 3) issue_w(s / 4 + 1);
        }
        wait_vm<(L::kRing - 1) * L::VM + L::kRing / 4 * L::VMW>();
        if (MODE == MM_16 && !PT && part == 0) clear_part();
        lds_barrier();
        Ops o[2];
        mm_for<NRD>([&](auto u) { read(u, 0, o[0]); });
        if constexpr (W4) {
#pragma unroll
            for (int x = 0; x < L::FQ; ++x) wsc[x] = row_scales(0, x);
        }
        // One stage: stage it + 1 has landed and every wave has read stage it.
        // Its products in FP groups, the first half of which also read the next
        // stage's operands, and all of which share the loads of stage it + ring:
        // issued in one burst after the barrier, the loads' scalar instructions
        // kept the matrix unit waiting in all waves at once.
        constexpr int V = (L::kRing - 2) * L::VM;
        constexpr int RPG = (NRD + (NG + 1) / 2 - 1) / ((NG + 1) / 2), LPG = (L::VM + NG - 1) / NG;
        auto stage = [&](int it, Ops& cur, Ops& nxt, auto bc) {
            constexpr int B = decltype(bc)::value;   // W4: stage of the group
            constexpr bool last_of_4 = W4 && B == 3;
            wait_vm<V + (L::kRing / 4 - (B < 3 ? 0 : 1)) * L::VMW>();
            if (MODE == MM_16 && !PT && it + 1 == part) clear_part();
            lds_barrier();
            uint4 v = make_uint4(0, 0, 0, 0), vn = v;
            if constexpr (W4) v = widen(std::integral_constant<int, 0>{}, B, cur);
            mm_for<NG>([&](auto gc) {
                constexpr int G = decltype(gc)::value;
                mmas(gc, cur, v);
                if constexpr (W4 && G + 1 < NG) vn = widen(std::integral_constant<int, G + 1>{}, B, cur);
                mm_for<RPG>([&](auto k) {
                    constexpr int U = G * RPG + decltype(k)::value;
                    if constexpr (U < NRD) read(std::integral_constant<int, U>{}, it + 1, nxt);
                });
                mm_for<LPG>([&](auto k) {
                    constexpr int U = G * LPG + decltype(k)::value;
                    if constexpr (U < L::VM) load(std::integral_constant<int, U>{}, it + L::kRing);
                });
                v = vn;
                __builtin_amdgcn_sched_barrier(0);
            });
            if constexpr (last_of_4) {
                // every scale of this group is used: those of the next
#pragma unroll
                for (int x = 0; x < L::FQ; ++x) wsc[x] = row_scales(it + 1, x);
            }
            if constexpr (last_of_4) issue_w((it >> 2) + L::WS);
        };
        if constexpr (W4) {
            // so the weights issued after the next stage's activations, one
            // group for each four stages of the ring, may be outstanding with
            // the activations; the last stage of a group needs the oldest of them
            for (int gr = 0; gr < groups; ++gr) {
                stage(4 * gr, o[0], o[1], std::integral_constant<int, 0>{});
                stage(4 * gr + 1, o[1], o[0], std::integral_constant<int, 1>{});
                stage(4 * gr + 2, o[0], o[1], std::integral_constant<int, 2>{});
                stage(4 * gr + 3, o[1], o[0], std::integral_constant<int, 3>{});
            }
        } else {
            int it = 0;
            for (; it + 2 <= w.nst; it += 2) {
                stage(it, o[0], o[1], std::integral_constant<int, 0>{});
                stage(it + 1, o[1], o[0], std::integral_constant<int, 0>{});
            }
            if (it < w.nst) mm_for<NG>([&](auto gc) { mmas(gc, o[0], make_uint4(0, 0, 0, 0)); });
        }
        wait_vm<0>();                  // no load of this workgroup may land after it ends
    }

    if constexpr (W4) {
        // Scales that the 16-bit type cannot hold (they never come from weights
        // of ordinary magnitude, but for blocks of zeros, which do not count):
        // this wave's products once more, a block at a time from memory,
        // unscaled, each sum scaled in fp32.  Kept out of the main loop, where a
        // second path would double the accumulators.
        auto matters = [&]() {
            const int64_t row = w.q0 + fq0 * 16, rows = a.Q - row < L::FQ * 16 ? a.Q - row : L::FQ * 16;
            return rows > 0 && mx4_not_exact<DT>(a.q + e * a.strideq + row * a.ldq, a.ldq,
                                                 a.qs + e * a.strideqs + row * a.ldqs, a.ldqs, (uint32_t)rows,
                                                 (uint32_t)w.st0, w.nst, w.nst,
                                                 (uint32_t)(w.st0 + w.nst < nb ? w.st0 + w.nst : nb), lane, 64);
        };
        if (__any(odd) && __any(matters())) {
#pragma unroll
            for (int x = 0; x < L::FQ; ++x)
#pragma unroll
                for (int y = 0; y < L::FP; ++y) acc[x][y] = f32x4{0, 0, 0, 0};
            const int64_t b1 = w.st0 + w.nst < nb ? w.st0 + w.nst : nb;
            for (int64_t b = w.st0; b < b1; ++b) {
                uint4 pv[L::FP];
#pragma unroll
                for (int y = 0; y < L::FP; ++y) {
                    const int64_t r = w.r0 + (fp0 + y) / 4 * 64 + 4 * i + (fp0 + y) % 4, at = b * 64 + g * 16;
                    pv[y] = make_uint4(0, 0, 0, 0);
                    if (r < w.r1 && at < prow) pv[y] = *reinterpret_cast<const uint4*>(a.p + r * a.ldp + at);
                }
#pragma unroll
                for (int x = 0; x < L::FQ; ++x) {
                    const int64_t r = w.q0 + (fq0 + x) / 4 * 64 + 4 * i + x % 4, row = r < a.Q ? r : a.Q - 1;
                    const uint32_t d = *reinterpret_cast<const uint32_t*>(a.q + e * a.strideq + row * a.ldq + b * 16 + g * 4);
                    const uint32_t sv = a.qs[e * a.strideqs + row * a.ldqs + b];
                    const uint4 v = mx4_widen<DT>(d, 1.0f);
                    f32x4 f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) f[k] = e8m0_to_f32((uint32_t)__shfl((int)sv, 4 * g + k));
#pragma unroll
                    for (int y = 0; y < L::FP; ++y) acc[x][y] += f * mfma16<DT>(v, pv[y], f32x4{0, 0, 0, 0});
                }
            }
        }
    }

    // Lane (i, g), register r of fragments (x, y) is row 16 y + i of the wave's
    // rows (PT) or 4 i + y % 4 of 64, column 16 x + 4 g + r (QT) or
    // 16 g + 4 r + x % 4 of 64.  A wave turns its outputs in 8 KiB of LDS, 64
    // columns of 64 (16-bit) or 32 (fp32) rows at a time, into 16-byte pieces of
    // rows, so that a store covers whole cache lines: written from the registers
    // as they are (8 bytes a lane, 16 rows a store), the weight gradient of 8 x
    // 4096 x 4096 with few rows took 88 us.  16-byte chunk c of row r sits at
    // chunk c ^ (r % chunks).  (fp32 columns of QT are whole 16 bytes a lane and 64
    // a row already: 65 us as they are, 89 through LDS at 40 x 1000 x 1416.)
    lds_barrier();                     // every wave has read its last stage
    void* const out = a.part ? (void*)(a.part + (int64_t)w.split * a.P * a.Q) : a.y;
    const int64_t ldo = a.part ? a.Q : a.ldy, oat = PT && !a.part ? e * a.stridey : 0;
    uint8_t* const turn = lds + wave * 8192;
    auto write_out = [&](auto es, auto half) {
        constexpr int ES = decltype(es)::value, NY = ES == 2 ? 4 : 2;       // fragments of rows a time
        constexpr int CH = 64 * ES / 16, YN = NY < L::FP ? NY : L::FP;      // chunks a row
        constexpr bool HALF = decltype(half)::value;
        if constexpr (QT && ES == 4) {
#pragma unroll
            for (int y = 0; y < L::FP; ++y) {
                const int fy = fp0 + y;
                const int64_t p = w.r0 + (PT ? fy * 16 + i : fy / 4 * 64 + 4 * i + fy % 4);
                if (p < w.v0 || p >= w.r1) continue;
#pragma unroll
                for (int x = 0; x < L::FQ; ++x) {
                    const int64_t q = w.q0 + (fq0 + x) * 16 + 4 * g;
                    if (q < a.Q) mm_store4(out, OUT_F32, oat + p * ldo + q, a.Q - q < 4 ? (int)(a.Q - q) : 4, acc[x][y]);
                }
            }
            return;
        }
#pragma unroll
        for (int xg = 0; xg < L::FQ; xg += 4) {
#pragma unroll
            for (int yg = 0; yg < L::FP; yg += YN) {
#pragma unroll
                for (int yy = 0; yy < YN; ++yy) {
                    // LDS row of this lane's outputs
                    const int row = PT ? yy * 16 + i : YN == 4 ? 4 * i + yy : YN * i + yy;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const f32x4 v = QT ? acc[xg + k][yg + yy]
                                           : f32x4{acc[xg][yg + yy][k], acc[xg + 1][yg + yy][k], acc[xg + 2][yg + yy][k],
                                                   acc[xg + 3][yg + yy][k]};
                        const int col = QT ? 16 * k + 4 * g : 16 * g + 4 * k;
                        const int at = col * ES, ch = (at >> 4) ^ (row & (CH - 1));
                        uint8_t* const d = turn + row * (64 * ES) + (ch << 4) + (at & 15);
                        if constexpr (ES == 4) {
                            *reinterpret_cast<f32x4*>(d) = v;
                        } else {
                            typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
                            typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                            // one rounding to nearest even after the fp32 sums
                            if constexpr (HALF) *reinterpret_cast<f16x4*>(d) = __builtin_convertvector(v, f16x4);
                            else *reinterpret_cast<bf16x4*>(d) = __builtin_convertvector(v, bf16x4);
                        }
                    }
                }
                constexpr int RPI = 64 / CH;                                // rows a store
#pragma unroll
                for (int n = 0; n < YN * 16 / RPI; ++n) {
                    const int row = n * RPI + lane / CH, c = lane % CH;
                    const uint4 v = *reinterpret_cast<const uint4*>(turn + row * (64 * ES) + ((c ^ (row & (CH - 1))) << 4));
                    // row of the tile: the wave's rows are 16 FP from 16 fp0 on (PT), or
                    // every (4 / YN)th of the 64-row groups its fragments belong to
                    const int f = fp0 + yg;
                    const int64_t p = w.r0 + (PT ? f * 16 + row : f / 4 * 64 + (YN == 4 ? row : row / YN * 4 + row % YN + f % 4));
                    const int64_t q = w.q0 + (fq0 + xg) * 16 + c * (16 / ES);
                    if (p >= w.v0 && p < w.r1 && q < a.Q)
                        mm_store_chunk<ES>(reinterpret_cast<uint8_t*>(out) + (oat + p * ldo + q) * ES, a.Q - q, v);
                }
            }
        }
    };
    if (a.part || a.out == OUT_F32) write_out(std::integral_constant<int, 4>{}, std::false_type{});
    else if (a.out == OUT_F16) write_out(std::integral_constant<int, 2>{}, std::true_type{});
    else write_out(std::integral_constant<int, 2>{}, std::false_type{});
}

// Tile (pt, qt) of T.p x T.q tiles, walked kMmGroupP row tiles at a time.
__device__ __forceinline__ void mm_walk(uint32_t id, uint32_t np, uint32_t nq, uint32_t* pt, uint32_t* qt) {
    const uint32_t grp = id / (kMmGroupP * nq), in = id - grp * kMmGroupP * nq;
    const uint32_t left = np - grp * kMmGroupP, gsz = left < (uint32_t)kMmGroupP ? left : (uint32_t)kMmGroupP;
    *qt = in / gsz;
    *pt = grp * kMmGroupP + in - *qt * gsz;
}

// The expert with the n-th most rows (ties by number).  A tile of the weight
// gradient takes as long as its expert has rows, so the large ones go first:
// begun last, one alone would keep the launch going.  (Up to 64 experts, a lane
// each; more go in their own order.)
__device__ __forceinline__ uint32_t mm_by_size(const MmArgs& a, uint32_t n) {
    if (!a.offs || a.E > 64) return n;
    const int lane = threadIdx.x & 63;
    int64_t lo = 0, hi = 0;
    if (lane < a.E) {
        lo = a.offs[lane];
        hi = a.offs[lane + 1];
    }
    const int rows = lane < a.E ? (int)(hi > lo ? hi - lo : 0) : -1;
    uint32_t rank = 0;
    for (int k = 0; k < (int)a.E; ++k) {
        const int r = __builtin_amdgcn_readlane(rows, k);
        rank += r > rows || (r == rows && k < lane);
    }
    const uint64_t hit = __ballot(lane < a.E && rank == n);
    return hit ? (uint32_t)__builtin_ctzll(hit) : n;
}

// The work of tile `id` of TQ x TP tiles; false if it is none.
template <bool GC, int TQ, int TP>
__device__ __forceinline__ bool mm_work(const MmArgs& a, uint32_t id, uint32_t np, uint32_t nq, int split, int ce,
                                        MmWork* w) {
    uint32_t pt, qt;
    w->c_at = 0;
    w->c_len = a.C;
    if constexpr (GC) {
        uint32_t e = id / (np * nq);
        mm_walk(id - e * np * nq, np, nq, &pt, &qt);
        e = mm_by_size(a, e);
        int64_t lo = 0, hi = a.C;
        if (a.offs) {
            const int64_t v0 = a.offs[e], v1 = a.offs[e + 1];
            lo = v0 < 0 ? 0 : (v0 > a.C ? a.C : v0);
            hi = v1 < lo ? lo : (v1 > a.C ? a.C : v1);
        }
        w->e = (int)e;
        w->c_at = lo;
        w->c_len = hi - lo;
        w->r0 = w->v0 = (int64_t)pt * TP;
        w->r1 = w->r0 + TP < a.P ? w->r0 + TP : a.P;
    } else {
        mm_walk(id, np, nq, &pt, &qt);
        MmTile t;
        if (!mm_find_tile(a, TP, (int)pt, &t)) return false;
        w->e = t.e;
        w->r0 = t.r0;
        w->v0 = t.v0;
        w->r1 = t.r1;
    }
    w->q0 = (int64_t)qt * TQ;
    const int64_t n = (w->c_len + ce - 1) / ce;
    const int64_t u = a.mode == MM_W4 ? 4 : 1, nu = (n + u - 1) / u;   // splits of whole groups
    w->split = split;
    w->st0 = nu * split / a.splits * u;
    const int64_t st1 = nu * (split + 1) / a.splits * u;
    w->nst = w->e < 0 ? 0 : (int)((st1 < n ? st1 : n) - w->st0);
    return true;
}

// Tile number of this workgroup among n, so that an XCD (every eighth
// workgroup) has a contiguous range; false for the surplus.
__device__ __forceinline__ bool mm_xcd(uint32_t b, uint32_t n, uint32_t* id) {
    const uint32_t chunk = (n + 7) / 8;
    *id = (b & 7) * chunk + (b >> 3);
    return (b >> 3) < chunk && *id < n;
}

// The same for the weight gradient, whose experts differ in time: every XCD has
// a range of every expert's `per` tiles, the experts one after the other.  (A
// range of all tiles is whole experts: 272 us instead of 150 for 8 x 4096 x 2048
// with 8192 tokens.)
__device__ __forceinline__ bool mm_xcd_experts(uint32_t b, uint32_t per, uint32_t E, uint32_t* id) {
    const uint32_t chunk = (per + 7) / 8, slot = b >> 3, e = slot / chunk, in = (b & 7) * chunk + slot % chunk;
    *id = e * per + in;
    return e < E && in < per;
}

// Large products: 256 x 256 tiles, the last round's cut where they fit.
template <int MODE, int DT, bool QT, bool PT>
__global__ void __launch_bounds__(512, 2) k_mm_large(MmArgs a, uint32_t nq, uint32_t np) {
    constexpr bool GC = PT;
    // 128 x 64 a wave holds fewer 16-bit fragments of mx4 weights than 64 x 128
    constexpr int WQ = MODE == MM_W4 ? 2 : 4, WP = 8 / WQ;
    using A = MmLay<MODE, 256, 256, WQ, WP>;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[A::LDS];
    constexpr int CE = MODE == MM_MX4 ? 128 : 32;
    const uint32_t rows = GC || !a.offs ? np : (uint32_t)mm_count_tiles(a, 256);
    const uint32_t total = rows * nq * (GC ? (uint32_t)a.E : 1u);
    const uint32_t full = total / kMmCUs * kMmCUs, rem = total - full;
    const uint32_t cut = rem <= kMmCUs / 4 ? 4 : rem <= kMmCUs / 2 ? 2 : 1;
    uint32_t id, part = 0, parts = 1;
    if (GC && full > 0) {
        if (!mm_xcd_experts(blockIdx.x, rows * nq, (uint32_t)a.E, &id)) return;
    } else if (blockIdx.x < full) {
        if (!mm_xcd(blockIdx.x, full, &id)) return;
    } else {
        if (!mm_xcd(blockIdx.x - full, rem * cut, &id)) return;
        parts = cut;
        part = id % cut;
        id = full + id / cut;
    }
    MmWork w;
    if (!mm_work<GC, 256, 256>(a, id, rows, nq, 0, CE, &w)) return;
    if (parts > 1) {
        // rows of the upper or lower half, and (in four) columns of one half
        const int64_t mid = w.r0 + 128;
        if (part & 1) {
            w.r0 = mid;
            w.v0 = w.v0 > mid ? w.v0 : mid;
        } else {
            w.r1 = w.r1 < mid ? w.r1 : mid;
        }
        if (part & 2) w.q0 += 128;
        if (w.v0 >= w.r1 || w.q0 >= a.Q) return;
    }
    if (parts == 4) mm_tile<MODE, DT, QT, PT, 128, 128, 2, 4>(a, w, lds);
    else if (parts == 2 || w.r1 - w.r0 <= 128) mm_tile<MODE, DT, QT, PT, 256, 128, 4, 2>(a, w, lds);
    else mm_tile<MODE, DT, QT, PT, 256, 256, WQ, WP>(a, w, lds);
}

// Small products: one tile size, the contraction split where tiles are few.
template <int MODE, int DT, bool QT, bool PT, int TQ, int TP, int WQ, int WP>
__global__ void __launch_bounds__(WQ* WP * 64, 2) k_mm_tiles(MmArgs a, uint32_t nq, uint32_t np) {
    constexpr bool GC = PT;
    using L = MmLay<MODE, TQ, TP, WQ, WP>;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[L::LDS];
    constexpr int CE = MODE == MM_MX4 ? 128 : 32;
    const uint32_t rows = GC || !a.offs ? np : (uint32_t)mm_count_tiles(a, TP);
    const uint32_t per = rows * nq * (GC ? (uint32_t)a.E : 1u);
    uint32_t id;
    if (GC ? !mm_xcd_experts(blockIdx.x, rows * nq, (uint32_t)a.E, &id)
           : !mm_xcd(blockIdx.x, per * (uint32_t)a.splits, &id))
        return;
    const int split = (int)(id / per);
    MmWork w;
    if (!mm_work<GC, TQ, TP>(a, id - split * per, rows, nq, split, CE, &w)) return;
    mm_tile<MODE, DT, QT, PT, TQ, TP, WQ, WP>(a, w, lds);
}

template <int MODE, int DT, bool QT, bool PT>
hipError_t mm_tiles_size(const MmArgs& a, int size, hipStream_t s) {
    const MmTileSize t = kMmTileSizes[size];
    const int64_t nq = (a.Q + t.q - 1) / t.q, np = (a.P + t.p - 1) / t.p;
    // (the weight gradient deals every expert's tiles to 8 XCDs)
    const int64_t tiles = PT ? (np * nq + 7) / 8 * 8 * a.E : mm_tile_bound(a, t.p) * nq;
    // cutting the last round adds at most 3 workgroups for each of 64 tiles
    const int64_t total = tiles * a.splits + (size == 0 ? 3 * kMmCUs / 4 : 0);
    if (total >= (int64_t)1 << 31) return hipErrorInvalidValue;
    const dim3 grid((unsigned)((total + 7) / 8 * 8));
    const uint32_t q = (uint32_t)nq, p = (uint32_t)np;
    switch (size) {
        case 0: hipLaunchKernelGGL((k_mm_large<MODE, DT, QT, PT>), grid, dim3(512), 0, s, a, q, p); break;
        case 1: hipLaunchKernelGGL((k_mm_tiles<MODE, DT, QT, PT, 128, 128, 2, 2>), grid, dim3(256), 0, s, a, q, p); break;
        default: hipLaunchKernelGGL((k_mm_tiles<MODE, DT, QT, PT, 128, 64, 2, 2>), grid, dim3(256), 0, s, a, q, p); break;
    }
    return hipGetLastError();
}

}  // namespace ssg
