// mm_fp8_tiles.hip -- tiled products of e4m3 operands with fp32 scales for each
// block of 128 along the contraction; dense or grouped by expert.
//
// Y[p, q] = sum over blocks of xs[p, b] ws[q, b] (sum over the block of x w): the
// inner sum is four MFMAs from zero, of elements widened to fp16 (fp8_mfma), and
// the vector unit adds it, times the scales, to the tile's sums.  So a fragment's
// 64 matrix cycles have four multiply-adds (with a scale for each weight row four
// multiplications more) and its share of the widening: 16 conversions a fragment
// of either operand.
//
// A workgroup owns a TQ x TP tile of one expert's Y; both operands stream through
// LDS a block (128 bytes of every row) at a time by direct-to-LDS loads.  A wave
// has the weights' widened fragments of a block in registers and goes through the
// tokens' one by one, with the LDS reads of the next fragments and of the next
// block's weights, the multiply-adds of the fragment before and a few of the loads
// of blocks to come between the MFMAs.
//
// 256 x 256 tiles fill LDS with two blocks, so a block is freed in halves: its
// weights once every wave has them (before it starts on the block), the first four
// token fragments of each wave after the first half, the others after the second.
// Smaller tiles have three or four blocks in LDS (or two, and two workgroups on a CU).
//
// Measured, 16-bit outputs: 8192^3 in 820 us, 1.34 PFLOP/s, with 256 x 256 tiles and 945
// with 128 x 128 in pairs; 4096^3 118 and 144; 11008 x 4096 with 2048 tokens 164 and 182.
// (fp32 outputs, 128 x 128 in pairs: 970, 145 and 193.)
//
// LDS image, the row order of fragments, the order of tiles and the cut of the
// last round are those of mm_tiles.hpp: a block is two of its 64-byte stages, and a
// lane's 32 elements are chunk g of both.
#include "fp8.hpp"
#include "mm_tiles.hpp"

namespace ssg {

namespace {

// A 16-byte direct-to-LDS load: lane l's bytes from offset voff + OFF of the
// buffer land at LDS address dst + IMM + 16 l (see mm_dma; the instruction adds
// its offset to both addresses).
template <int IMM, int OFF>
__device__ __forceinline__ void dma16(i32x4 buf, uint32_t dst, uint32_t voff) {
    asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, 0 offen offset:%4 lds" ::"s"(dst),
                 "n"(IMM - OFF), "v"(voff), "s"(buf), "n"(OFF)
                 : "memory", "m0", "scc");
}
__device__ __forceinline__ void dma4(i32x4 buf, uint32_t dst, uint32_t voff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(dst), "v"(voff), "s"(buf)
                 : "memory", "m0");
}

// A buffer that begins `step` bytes a block after `base` and ends `lim` bytes after it.
struct Walk {
    uint32_t lo, hi;
    int64_t step;
    int lim;

    __device__ __forceinline__ void init(const void* base, int64_t st, int64_t bytes) {
        const uint64_t p = reinterpret_cast<uint64_t>(base);
        lo = __builtin_amdgcn_readfirstlane((uint32_t)p);
        hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
        step = st;
        lim = __builtin_amdgcn_readfirstlane((int)bytes);
    }
    __device__ __forceinline__ i32x4 at(int b, bool moves) const {
        const uint64_t p = (((uint64_t)hi << 32) | lo) + (uint64_t)(b * step);
        const int n = moves ? max(lim - b * kFp8Block, 0) : lim;
        return i32x4{(int)(uint32_t)p, (int)(uint32_t)(p >> 32), n, 0x00020000};
    }
};

template <int TQ, int TP, int WQ, int WP, int SL>
struct Fp8Lay {
    static constexpr int NW = WQ * WP, FQ = TQ / WQ / 16, FP = TP / WP / 16;
    static constexpr int NPH = FP > 4 ? 2 : 1, YP = FP / NPH;        // halves of a block, token fragments of each
    static constexpr int Q_BYTES = TQ * 128, P_BYTES = TP * 128;
    static constexpr int P_AT = Q_BYTES, SLOT = P_AT + P_BYTES;
    static constexpr int SLOTS = SL;                                  // blocks in LDS
    static constexpr bool PRE = NPH == 2 || SLOTS > 2;               // the next one is there while this one is multiplied
    // Scales in four slots: they are loaded with a block's first part and read until its end.
    static constexpr int S_AT = SLOTS * SLOT, WS_AT = 1024, S_SLOT = 2048;
    static constexpr int LDS = S_AT + 4 * S_SLOT;
    static constexpr int QL = TQ / 16 * 2 / NW, PL = YP * WP * 2 / NW;   // loads of a wave: weights, tokens of a half
    static constexpr int ALL = QL + PL + 1;                              // of a block of one half, with a scale load
    static_assert(NPH == 1 || SLOTS == 2, "halves");
    static_assert(FQ == 4 && QL % 2 == 0 && PL % 2 == 0 && TQ <= 256 && TP <= 256, "tile");
    static_assert(NW * 8192 <= LDS && LDS <= 160 * 1024, "LDS");
};

// LDS row (of fragment f = slot / 16) to tile row, as in mm_tiles.hpp
__device__ __forceinline__ int row_of(int slot) { return (slot & ~63) + 4 * (slot & 15) + ((slot >> 4) & 3); }

template <bool WR, int TQ, int TP, int WQ, int WP, int SL>
__device__ __forceinline__ void fp8_tile(const MmFp8Args& a, const MmWork& w, uint8_t* lds) {
    using L = Fp8Lay<TQ, TP, WQ, WP, SL>;
    const MmArgs& m = a.m;
    const uint32_t lds32 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const lds_void*)lds);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4, wq = wave % WQ, wp = wave / WQ;
    const int64_t e = w.e < 0 ? 0 : w.e;

    Walk bq, bp, bs;
    auto span = [](int64_t rows, int64_t most, int64_t ld, int64_t bytes) {
        const int64_t n = rows < most ? rows : most;
        return n > 0 ? (n - 1) * ld + (bytes + 3) / 4 * 4 : 0;
    };
    const int64_t left = m.C - w.st0 * kFp8Block;      // bytes of a row from the first block on
    bq.init(m.q + e * m.strideq + w.q0 * m.ldq + w.st0 * kFp8Block, kFp8Block, span(m.Q - w.q0, TQ, m.ldq, left));
    bp.init(m.p + w.r0 * m.ldp + w.st0 * kFp8Block, kFp8Block, span(w.r1 - w.r0, TP, m.ldp, left));
    // a scale load a wave: the tokens' from even waves, the weights' from odd ones
    const bool odd = wave & 1;
    uint32_t far = 0;                  // the second scale of the tile's weights
    if (!odd) {
        const int64_t n = w.r1 - w.r0 < TP ? w.r1 - w.r0 : TP;
        bs.init(a.x.p + w.r0 + w.st0 * a.x.blk, a.x.blk * 4, n * 4);
    } else if (WR) {
        const int64_t n = m.Q - w.q0 < TQ ? m.Q - w.q0 : TQ;
        bs.init(a.w.p + e * a.w.mat + w.q0 + w.st0 * a.w.blk, a.w.blk * 4, n * 4);
    } else {
        // lane l: that of 128 rows l % 2 of the tile
        const int64_t first = w.q0 / kFp8Block, last = (m.Q + kFp8Block - 1) / kFp8Block - 1;
        bs.init(a.w.p + e * a.w.mat + first * a.w.row + w.st0 * a.w.blk, a.w.blk * 4, 0x7fffffff);
        far = last > first ? (uint32_t)(a.w.row * 4) : 0;
    }
    // A wave's pieces (a fragment's 16 rows x 64 bytes), and the lane's place in them:
    // computed where they are needed, from a lane number that the compiler takes for a new
    // one (kept over the loop they cost registers that the large tile does not have).
    auto here = [] {
        int l = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
        asm volatile("" : "+v"(l));
        return l;
    };
    auto chunk_of = [](int l) { return 16 * ((l & 3) ^ mm_swz(l >> 2)); };
    auto qf = [&](int j) { return wave * (L::QL / 2) + j; };
    auto pf = [&](int h, int j) {
        const int n = wave * (L::PL / 2) + j;
        return n / L::YP * L::FP + h * L::YP + n % L::YP;
    };
    auto off_of = [&](int l, int f, int64_t ld) {
        return (uint32_t)row_of(f * 16 + (l >> 2)) * (uint32_t)ld + chunk_of(l);
    };
    auto slot_at = [&](int b) { return (uint32_t)(L::SLOTS == 3 ? b % 3 : b & (L::SLOTS - 1)) * L::SLOT; };
    auto slot_of = [&](int b) { return lds32 + slot_at(b); };
    auto scales_of = [&](int b) { return L::S_AT + (b & 3) * L::S_SLOT; };
    auto issue_q = [&](int b) {
        const i32x4 r = bq.at(b, true);
        const uint32_t s = slot_of(b);
        const int l = here();
#pragma unroll
        for (int j = 0; j < L::QL / 2; ++j) {
            const uint32_t off = off_of(l, qf(j), m.ldq);
            dma16<0, 0>(r, s + qf(j) * 1024, off);
            dma16<TQ * 64, 64>(r, s + qf(j) * 1024, off);
        }
    };
    auto issue_p = [&](auto hc, int b) {
        constexpr int H = decltype(hc)::value;
        const i32x4 r = bp.at(b, true);
        const uint32_t s = slot_of(b);
        const int l = here();
#pragma unroll
        for (int j = 0; j < L::PL / 2; ++j) {
            const uint32_t off = off_of(l, pf(H, j), m.ldp);
            dma16<L::P_AT, 0>(r, s + pf(H, j) * 1024, off);
            dma16<L::P_AT + TP * 64, 64>(r, s + pf(H, j) * 1024, off);
        }
    };
    // (past the last block the walk may leave the scales: nothing is read)
    auto issue_s = [&](int b) {
        i32x4 r = bs.at(b, false);
        if (b >= w.nst) r[2] = 0;
        const uint32_t s = lds32 + scales_of(b);
        const int l = here();
        if (!odd) dma16<0, 0>(r, s, 16 * l);
        else if (WR) dma16<L::WS_AT, 0>(r, s, 16 * l);
        else dma4(r, s + L::WS_AT, l & 1 ? far : 0);
    };
    using H0 = std::integral_constant<int, 0>;
    using H1 = std::integral_constant<int, L::NPH - 1>;
    auto issue_block = [&](int b) {    // of one half
        issue_q(b);
        issue_p(H0{}, b);
        issue_s(b);
    };
    // The contraction ends inside the last block: the wave's own pieces (which have
    // landed) become zeros from there on.
    const int last = w.nst - 1;
    const int64_t tail64 = left - (int64_t)last * kFp8Block;
    const int tail = tail64 < kFp8Block ? (int)tail64 : kFp8Block;
    auto clear = [&](uint8_t* piece, int half) {
        const int l = here(), n = tail - 64 * half - chunk_of(l);   // bytes of the lane's chunk that stay
        uint4* const d = reinterpret_cast<uint4*>(piece + l * 16);
        uint4 v = *d;
        auto mask = [&](int k) { return n >= 4 * k + 4 ? ~0u : n <= 4 * k ? 0u : (1u << (8 * (n - 4 * k))) - 1; };
        v.x &= mask(0);
        v.y &= mask(1);
        v.z &= mask(2);
        v.w &= mask(3);
        *d = v;
    };
    auto clear_q = [&](uint8_t* s) {
#pragma unroll
        for (int j = 0; j < L::QL / 2; ++j) {
            clear(s + qf(j) * 1024, 0);
            clear(s + TQ * 64 + qf(j) * 1024, 1);
        }
    };
    auto clear_p = [&](auto hc, uint8_t* s) {
        constexpr int H = decltype(hc)::value;
#pragma unroll
        for (int j = 0; j < L::PL / 2; ++j) {
            clear(s + L::P_AT + pf(H, j) * 1024, 0);
            clear(s + L::P_AT + TP * 64 + pf(H, j) * 1024, 1);
        }
    };

    f32x4 acc[L::FQ][L::FP];
#pragma unroll
    for (int x = 0; x < L::FQ; ++x)
#pragma unroll
        for (int y = 0; y < L::FP; ++y) acc[x][y] = f32x4{0, 0, 0, 0};

    const int fq0 = wq * L::FQ, fp0 = wp * L::FP;
    const int at_lane = i * 64 + ((g ^ mm_swz(i)) << 4);
    struct Raw {
        uint4 lo, hi;
    };
    auto frag = [](const uint8_t* at, int rows) -> Raw {
        return {*reinterpret_cast<const uint4*>(at), *reinterpret_cast<const uint4*>(at + rows * 64)};
    };
    // Where a block is in LDS: this lane's fragments in its slot, and its scales.
    struct Place {
        const uint8_t *slot, *sc;
    };
    auto place = [&](int b) -> Place { return {lds + slot_at(b) + at_lane, lds + scales_of(b)}; };
    // weights of a block: fragments, and scales (of 128 rows, or of rows
    // 16 g + 4 r + x of the wave's 64: [r][x])
    struct Weights {
        Raw q[L::FQ];
        float s;
        f32x4 r[WR ? 4 : 1];
    };
    const int q_at = fq0 * 1024, p_at = L::P_AT + fp0 * 1024;
    const int ws_at = L::WS_AT + (WR ? (wq * 64 + 16 * g) * 4 : wq * 64 / kFp8Block * 4);
    const int xs_at = (fp0 / 4 * 64 + 4 * i + fp0 % 4) * 4;
    auto read_q = [&](auto xc, const Place& at, Weights& w_) {
        constexpr int X = decltype(xc)::value;
        w_.q[X] = frag(at.slot + q_at + X * 1024, TQ);
        if constexpr (WR) w_.r[X] = *reinterpret_cast<const f32x4*>(at.sc + ws_at + 16 * X);
        else if constexpr (X == 0) w_.s = *reinterpret_cast<const float*>(at.sc + ws_at);
    };
    struct Tokens {
        Raw p;
        float s;
    };
    auto read_p = [&](auto yc, const Place& at) -> Tokens {
        constexpr int Y = decltype(yc)::value;
        return {frag(at.slot + p_at + Y * 1024, TP), *reinterpret_cast<const float*>(at.sc + xs_at + (Y / 4 * 64 + Y % 4) * 4)};
    };

    Weights wt[2];                     // of blocks (even, odd)
    Fp8Wide qx[L::FQ], px[2];          // the block's weights; tokens of fragments y (even, odd)
    Tokens tok[2];                     // as they are read
    f32x4 t[4];                        // sums of the last MFMAs, by step number
    float f[2];                        // of the tokens of fragments (even, odd): their scale, times the weights' if that is one
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = f32x4{0, 0, 0, 0};
    f[0] = f[1] = 0.0f;
    if constexpr (WR) {
#pragma unroll
        for (int k = 0; k < 4; ++k) wt[1].r[k] = f32x4{0, 0, 0, 0};
    }
    // One step: fragment Y of the tokens with X of the weights, and the multiply-adds of two steps before.
    auto add = [&](auto yc, auto xc, const Weights& of) {
        constexpr int Y = decltype(yc)::value, X = decltype(xc)::value, K = Y * L::FQ + X;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            acc[X][Y][r] = WR ? fmaf(t[K & 3][r] * f[Y & 1], of.r[WR ? r : 0][X], acc[X][Y][r])
                              : fmaf(t[K & 3][r], f[Y & 1], acc[X][Y][r]);
        asm volatile("" : "+v"(acc[X][Y]));            // here: the compiler would collect them behind the next branch
    };
    // Fragment Y of the tokens of a block at `at` (the next one: `to`) with weights
    // `cur`, four steps; `loads` issues its share of the loads.
    auto group = [&](auto yc, const Place& at, const Place& to, const Weights& cur, Weights& nxt, auto&& loads) {
        constexpr int Y = decltype(yc)::value;
        f[Y & 1] = WR ? tok[Y & 1].s : cur.s * tok[Y & 1].s;
        mm_for<L::FQ>([&](auto xc) {
            constexpr int X = decltype(xc)::value, K = Y * L::FQ + X, J = (K + L::FQ * L::FP - 2) % (L::FQ * L::FP);
            t[K & 3] = fp8_mfma(qx[X], px[Y & 1]);
            add(std::integral_constant<int, J / L::FQ>{}, std::integral_constant<int, J % L::FQ>{}, K >= 2 ? cur : nxt);
            if constexpr (X == 0) {
                if constexpr (Y + 1 < L::FP) tok[(Y + 1) & 1] = read_p(std::integral_constant<int, Y + 1>{}, at);
                else if constexpr (L::PRE) tok[0] = read_p(std::integral_constant<int, 0>{}, to);
            } else if constexpr (X == 1) {
                loads();
            } else if constexpr (X == 2 && L::PRE) {
                // the next block's weights, over the two fragments before the last, in which
                // they are widened
                constexpr int G = L::FP > 2 ? 2 : 1, N = L::FQ / G, AT = (Y - (L::FP - 1 - G)) * N;
                if constexpr (AT >= 0 && AT < L::FQ)
                    mm_for<N>([&](auto n) { read_q(std::integral_constant<int, (AT < 0 ? 0 : AT) + decltype(n)::value>{}, to, nxt); });
            }
            // what has had its last use, and the next tokens
            if constexpr (Y + 1 == L::FP && L::PRE) qx[X] = fp8_widen(nxt.q[X].lo, nxt.q[X].hi);
            if constexpr (X == 3 && (Y + 1 < L::FP || L::PRE))
                px[(Y + 1) & 1] = fp8_widen(tok[(Y + 1) & 1].p.lo, tok[(Y + 1) & 1].p.hi);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    auto read_block = [&](const Place& at, Weights& w_) {  // weights and first tokens
        mm_for<L::FQ>([&](auto xc) { read_q(xc, at, w_); });
        tok[0] = read_p(std::integral_constant<int, 0>{}, at);
        mm_for<L::FQ>([&](auto xc) {
            constexpr int X = decltype(xc)::value;
            qx[X] = fp8_widen(w_.q[X].lo, w_.q[X].hi);
        });
        px[0] = fp8_widen(tok[0].p.lo, tok[0].p.hi);
    };
    auto none = [] {};
    auto by_twos = [&](auto&& block) {                 // block(b, this one's weights, the next one's)
        int b = 0;
        for (; b + 2 <= w.nst; b += 2) {
            block(b, wt[0], wt[1]);
            block(b + 1, wt[1], wt[0]);
        }
        if (b < w.nst) block(b, wt[0], wt[1]);
    };

    if (w.nst > 0) {
        auto tail_first = [&](int b) {                 // weights and first tokens of block b have landed
            if (b != last || tail == kFp8Block) return;
            uint8_t* const s = lds + slot_at(b);
            clear_q(s);
            clear_p(H0{}, s);
        };
        if constexpr (L::NPH == 2) {
            issue_q(0);
            issue_p(H0{}, 0);
            issue_s(0);
            issue_p(H1{}, 0);
            issue_q(1);
            issue_p(H0{}, 1);
            issue_s(1);
            wait_vm<2 * L::PL + L::QL + 1>();
            tail_first(0);
            lds_barrier();
            // 128 registers hold sums here and 64 the weights, so all else has one place each.
            // A fragment's MFMAs go through the contraction's four parts, the four weights'
            // fragments in each: a part of the tokens that was multiplied is overwritten
            // with the next fragment's, widened from `raw`, whose halves are read again as
            // soon as they are free (two fragments ahead of their products).  The last
            // fragment goes weight by weight, each replaced by the next block's.
            Raw raw;
            uint4(&p4)[4] = px[0].v;
            float ws, ts[2], fs[2] = {0.0f, 0.0f};     // scales: weights, tokens of fragments (even, odd), products
            // this lane's place in the slot that is read, and in its scales
            uint32_t at = at_lane, sc = L::S_AT + xs_at;
            static_assert((L::SLOT & (L::SLOT - 1)) == 0 && L::S_AT % (4 * L::S_SLOT) == 0, "places");
            // (pinned where they are: moved behind the next branch they would cost the registers of both forms)
            auto wide = [&](auto kc, uint4& d) {
                constexpr int K = decltype(kc)::value;
                const uint4& h = K < 2 ? raw.lo : raw.hi;
                d = K & 1 ? fp8_widen_part(h.z, h.w) : fp8_widen_part(h.x, h.y);
                asm volatile("" : "+v"(d.x), "+v"(d.y), "+v"(d.z), "+v"(d.w));
            };
            auto wide_all = [&](uint4(&d)[4]) { mm_for<4>([&](auto kc) { wide(kc, d[decltype(kc)::value]); }); };
            auto read_lo = [&](int off) { raw.lo = *reinterpret_cast<const uint4*>(lds + at + off); };
            auto read_hi = [&](int off) { raw.hi = *reinterpret_cast<const uint4*>(lds + at + off); };
            auto p_lo = [&](int y) { read_lo(p_at + y * 1024); };
            auto p_hi = [&](int y) { read_hi(p_at + y * 1024 + TP * 64); };
            auto q_lo = [&](int x) { read_lo(q_at + x * 1024); };
            auto q_hi = [&](int x) { read_hi(q_at + x * 1024 + TQ * 64); };
            auto p_scale = [&](int y) { return *reinterpret_cast<const float*>(lds + sc + (y / 4 * 64 + y % 4) * 4); };
            auto q_scale = [&](int b) { return *reinterpret_cast<const float*>(lds + scales_of(b) + ws_at); };
            mm_for<4>([&](auto xc) {
                constexpr int X = decltype(xc)::value;
                q_lo(X);
                q_hi(X);
                wide_all(qx[X].v);
            });
            p_lo(0);
            p_hi(0);
            ts[0] = p_scale(0);
            wide_all(p4);
            p_lo(1);
            p_hi(1);
            ts[1] = p_scale(1);
            ws = q_scale(0);
            // the multiply-adds of fragment Y
            auto put = [&](auto xc, auto yc) {
                constexpr int X = decltype(xc)::value, Y = decltype(yc)::value;
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[X][Y][r] = fmaf(t[X][r], fs[Y & 1], acc[X][Y][r]);
                asm volatile("" : "+v"(acc[X][Y]));
            };
            auto mma = [&](auto xc, auto kc) {
                constexpr int X = decltype(xc)::value, K = decltype(kc)::value;
                t[X] = mfma16<DT_F16>(qx[X].v[K], p4[K], K ? t[X] : f32x4{0, 0, 0, 0});
            };
            auto fragment = [&](auto yc, int b, auto&& loads) {
                constexpr int Y = decltype(yc)::value;
                const std::integral_constant<int, (Y + 7) % 8> before{};
                fs[Y & 1] = ws * ts[Y & 1];
                if constexpr (Y < 7) {
                    mm_for<4>([&](auto kc) {
                        constexpr int K = decltype(kc)::value;
                        mm_for<4>([&](auto xc) {
                            if constexpr (K == 0) put(xc, before);
                            mma(xc, kc);
                        });
                        __builtin_amdgcn_sched_barrier(0);
                        wide(kc, p4[K]);
                        if constexpr (K == 1) {
                            loads();
                            if constexpr (Y < 6) {
                                p_lo(Y + 2);
                            } else {                   // from here on the next block is read
                                at ^= L::SLOT;
                                sc = ((sc + L::S_SLOT) & (4 * L::S_SLOT - 1)) | L::S_AT;
                                q_lo(0);
                            }
                        } else if constexpr (K == 3) {
                            if constexpr (Y < 6) p_hi(Y + 2);
                            else q_hi(0);
                            ts[Y & 1] = p_scale(Y < 6 ? Y + 2 : 0);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    });
                } else {
                    ws = q_scale(b + 1);
                    mm_for<4>([&](auto xc) {
                        constexpr int X = decltype(xc)::value;
                        put(xc, before);
                        mm_for<4>([&](auto kc) { mma(xc, kc); });
                        __builtin_amdgcn_sched_barrier(0);
                        wide_all(qx[X].v);
                        __builtin_amdgcn_sched_barrier(0);
                        if constexpr (X < 3) {
                            q_lo(X + 1);
                            q_hi(X + 1);
                        } else {
                            p_lo(0);
                            p_hi(0);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    });
                    wide_all(p4);
                    p_lo(1);
                    p_hi(1);
                    ts[1] = p_scale(1);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            for (int b = 0; b < w.nst; ++b) {
                // the second half of this block has landed; every wave has its weights, and
                // has read the second half of the last block
                wait_vm<L::QL + L::PL + 1>();
                if (b == last && tail < kFp8Block) clear_p(H1{}, lds + slot_at(b));
                lds_barrier();
                fragment(std::integral_constant<int, 0>{}, b, [&] { issue_p(H1{}, b + 1); });
                fragment(std::integral_constant<int, 1>{}, b, [&] { issue_q(b + 2); });
                fragment(std::integral_constant<int, 2>{}, b, none);
                fragment(std::integral_constant<int, 3>{}, b, none);
                // the next block's weights and first half have landed; every wave has read this one's
                wait_vm<L::QL + L::PL>();
                tail_first(b + 1);
                lds_barrier();
                fragment(std::integral_constant<int, 4>{}, b, [&] { issue_p(H0{}, b + 2); });
                fragment(std::integral_constant<int, 5>{}, b, [&] { issue_s(b + 2); });
                fragment(std::integral_constant<int, 6>{}, b, none);
                fragment(std::integral_constant<int, 7>{}, b, none);
            }
            mm_for<4>([&](auto xc) { put(xc, std::integral_constant<int, 7>{}); });
        } else if constexpr (L::PRE) {
            mm_for<L::SLOTS - 1>([&](auto b) { issue_block(decltype(b)::value); });
            wait_vm<(L::SLOTS - 2) * L::ALL>();
            tail_first(0);
            lds_barrier();
            read_block(place(0), wt[0]);
            by_twos([&](int b, const Weights& cur, Weights& nxt) {
                const Place at = place(b), to = place(b + 1);
                wait_vm<(L::SLOTS - 3) * L::ALL>();    // the next block has landed, every wave is done with the last one
                tail_first(b + 1);
                lds_barrier();
                mm_for<L::FP>([&](auto yc) {
                    if constexpr (decltype(yc)::value == 0) group(yc, at, to, cur, nxt, [&] { issue_block(b + L::SLOTS - 1); });
                    else group(yc, at, to, cur, nxt, none);
                });
            });
        } else {
            issue_block(0);
            by_twos([&](int b, Weights& cur, Weights& nxt) {
                const Place at = place(b);
                wait_vm<0>();
                tail_first(b);
                lds_barrier();
                read_block(at, cur);
                mm_for<L::FP>([&](auto yc) {
                    if constexpr (decltype(yc)::value == 0) group(yc, at, at, cur, nxt, [&] { issue_block(b + 1); });
                    else group(yc, at, at, cur, nxt, none);
                });
            });
        }
        // the last two steps
        constexpr int N = L::FQ * L::FP;
        auto rest = [&](const Weights& of) {
            add(std::integral_constant<int, (N - 2) / L::FQ>{}, std::integral_constant<int, (N - 2) % L::FQ>{}, of);
            add(std::integral_constant<int, (N - 1) / L::FQ>{}, std::integral_constant<int, (N - 1) % L::FQ>{}, of);
        };
        if constexpr (L::NPH == 1) {
            if (last & 1) rest(wt[1]);
            else rest(wt[0]);
        }
        wait_vm<0>();                  // no load of this workgroup may land after it ends
    }

    // The wave's outputs, turned in 8 KiB of LDS into 16-byte pieces of rows (as in
    // mm_tiles.hpp): lane (i, g), register r of fragments (x, y) is row
    // 4 i + y % 4 of 64, column 16 g + 4 r + x of 64.
    lds_barrier();                     // every wave has read its last block
    const int ln = here(), oi = ln & 15, og = ln >> 4;
    void* const out = m.part ? (void*)(m.part + (int64_t)w.split * m.P * m.Q) : m.y;
    const int64_t ldo = m.part ? m.Q : m.ldy;
    uint8_t* const turn = lds + wave * 8192;
    auto write_out = [&](auto es, auto half) {
        constexpr int ES = decltype(es)::value, NY = ES == 2 ? 4 : 2, YN = NY < L::FP ? NY : L::FP;
        constexpr int CH = 64 * ES / 16, RPI = 64 / CH;                   // chunks a row, rows a store
#pragma unroll
        for (int yg = 0; yg < L::FP; yg += YN) {
#pragma unroll
            for (int yy = 0; yy < YN; ++yy) {
                const int row = YN * oi + yy;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x4 v = {acc[0][yg + yy][k], acc[1][yg + yy][k], acc[2][yg + yy][k], acc[3][yg + yy][k]};
                    const int at = (16 * og + 4 * k) * ES, ch = (at >> 4) ^ (row & (CH - 1));
                    uint8_t* const d = turn + row * (64 * ES) + (ch << 4) + (at & 15);
                    if constexpr (ES == 4) {
                        *reinterpret_cast<f32x4*>(d) = v;
                    } else {
                        typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
                        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                        // one rounding to nearest even after the fp32 sums
                        if constexpr (decltype(half)::value) *reinterpret_cast<f16x4*>(d) = __builtin_convertvector(v, f16x4);
                        else *reinterpret_cast<bf16x4*>(d) = __builtin_convertvector(v, bf16x4);
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < YN * 16 / RPI; ++n) {
                const int row = n * RPI + ln / CH, c = ln % CH, f = fp0 + yg;
                const uint4 v = *reinterpret_cast<const uint4*>(turn + row * (64 * ES) + ((c ^ (row & (CH - 1))) << 4));
                const int64_t p = w.r0 + f / 4 * 64 + row / YN * 4 + row % YN + f % 4;
                const int64_t col = w.q0 + fq0 * 16 + c * (16 / ES);
                if (p >= w.v0 && p < w.r1 && col < m.Q)
                    mm_store_chunk<ES>(reinterpret_cast<uint8_t*>(out) + (p * ldo + col) * ES, m.Q - col, v);
            }
        }
    };
    if (m.part || m.out == OUT_F32) write_out(std::integral_constant<int, 4>{}, std::false_type{});
    else if (m.out == OUT_F16) write_out(std::integral_constant<int, 2>{}, std::true_type{});
    else write_out(std::integral_constant<int, 2>{}, std::false_type{});
}

// Large products: 256 x 256 tiles, the last round's cut where they fit (k_mm_large).
// Not with a scale for each weight row, whose registers these tiles do not have, and not
// with fp32 outputs, of which a tile has twice the bytes to write.
__global__ void __launch_bounds__(512, 2) k_mm_fp8_large(MmFp8Args a, uint32_t nq, uint32_t np) {
    using Half = Fp8Lay<256, 128, 4, 2, 3>;            // the largest of the three
    __shared__ __attribute__((aligned(1024))) uint8_t lds[Half::LDS];
    static_assert(Fp8Lay<256, 256, 4, 2, 2>::LDS <= sizeof lds && Fp8Lay<128, 128, 2, 4, 4>::LDS <= sizeof lds, "LDS");
    const uint32_t rows = a.m.offs ? (uint32_t)mm_count_tiles(a.m, 256) : np, total = rows * nq;
    const uint32_t full = total / kMmCUs * kMmCUs, rem = total - full;
    const uint32_t cut = rem <= kMmCUs / 4 ? 4 : rem <= kMmCUs / 2 ? 2 : 1;
    uint32_t id, part = 0, parts = 1;
    if (blockIdx.x < full) {
        if (!mm_xcd(blockIdx.x, full, &id)) return;
    } else {
        if (!mm_xcd(blockIdx.x - full, rem * cut, &id)) return;
        parts = cut;
        part = id % cut;
        id = full + id / cut;
    }
    MmWork w;
    if (!mm_work<false, 256, 256>(a.m, id, rows, nq, 0, kFp8Block, &w)) return;
    if (parts > 1) {
        // the upper or lower half, and (in four) columns of one half
        const int64_t mid = w.r0 + 128;
        if (part & 1) {
            w.r0 = mid;
            w.v0 = w.v0 > mid ? w.v0 : mid;
        } else {
            w.r1 = w.r1 < mid ? w.r1 : mid;
        }
        if (part & 2) w.q0 += 128;
        if (w.v0 >= w.r1 || w.q0 >= a.m.Q) return;
    }
    if (parts == 4) fp8_tile<false, 128, 128, 2, 4, 4>(a, w, lds);
    else if (parts == 2 || w.r1 - w.r0 <= 128) fp8_tile<false, 256, 128, 4, 2, 3>(a, w, lds);
    else fp8_tile<false, 256, 256, 4, 2, 2>(a, w, lds);
}

// Small products: one tile size, the contraction split where tiles are few.
template <bool WR, int TQ, int TP, int WQ, int WP, int SL>
__global__ void __launch_bounds__(WQ* WP * 64, 2) k_mm_fp8_tiles(MmFp8Args a, uint32_t nq, uint32_t np) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[Fp8Lay<TQ, TP, WQ, WP, SL>::LDS];
    const uint32_t rows = a.m.offs ? (uint32_t)mm_count_tiles(a.m, TP) : np, per = rows * nq;
    uint32_t id;
    if (!mm_xcd(blockIdx.x, per * (uint32_t)a.m.splits, &id)) return;
    const int split = (int)(id / per);
    MmWork w;
    if (!mm_work<false, TQ, TP>(a.m, id - split * per, rows, nq, split, kFp8Block, &w)) return;
    fp8_tile<WR, TQ, TP, WQ, WP, SL>(a, w, lds);
}

// (a launch of q x p tiles of tq x tp, and `more` workgroups)
template <typename K>
hipError_t go(K kernel, const MmFp8Args& a, int tq, int tp, int threads, int more, hipStream_t s) {
    const int64_t nq = (a.m.Q + tq - 1) / tq, np = (a.m.P + tp - 1) / tp;
    const int64_t total = mm_tile_bound(a.m, tp) * nq * a.m.splits + more;
    if (total >= (int64_t)1 << 23) return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((total + 7) / 8 * 8)), dim3(threads), 0, s, a, (uint32_t)nq, (uint32_t)np);
    return hipGetLastError();
}

template <bool WR>
hipError_t pick(const MmFp8Args& a, int size, hipStream_t s) {
    if (size == 1) return go(k_mm_fp8_tiles<WR, 128, 128, 2, 2, 2>, a, 128, 128, 256, 0, s);
    if (WR) return hipErrorInvalidValue;
    // cutting the last round adds at most 3 workgroups for each of 64 tiles
    return go(k_mm_fp8_large, a, 256, 256, 512, 3 * kMmCUs / 4, s);
}

}  // namespace

hipError_t launch_mm_fp8_tiles(const MmFp8Args& a, int size, hipStream_t s) {
    return a.w_rows ? pick<true>(a, size, s) : pick<false>(a, size, s);
}

}  // namespace ssg
