// mm_fp8_tiles.hip -- tiled products of e4m3 operands with fp32 scales for each
// block of 128 along the contraction; dense or grouped by expert.
//
// Y[p, q] = sum over blocks of xs[p, b] ws[q, b] (sum over the block of x w): the
// inner sum is one MFMA from zero (16 x 16 x 128), and the vector unit adds it,
// times the scales, to the tile's sums while the matrix unit has the next.  With
// a scale for 128 weight rows that is a multiplication for each token and four
// multiply-adds a fragment, half of the MFMA's time; with one for each weight row
// four multiplications more.
//
// A workgroup owns a TQ x TP tile of one expert's Y; both operands stream through
// LDS a block (128 bytes of every row) at a time by direct-to-LDS loads.  A wave
// has the weights' fragments of a block in registers and goes through the tokens'
// one by one: a fragment's MFMAs are issued with the multiply-adds of two MFMAs
// before, the LDS reads of the next fragment and of the next block's weights, and
// a few of the loads of blocks to come between them.
//
// 256 x 256 tiles fill LDS with two blocks, so a block is freed in halves: its
// weights once every wave has them (before it starts on the block), the first four
// token fragments of each wave after the first half, the others after the second.
// Smaller tiles have three blocks in LDS (or two, and two workgroups on a CU).
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
    int64_t lim;

    __device__ __forceinline__ void init(const void* base, int64_t st, int64_t bytes) {
        const uint64_t p = reinterpret_cast<uint64_t>(base);
        lo = __builtin_amdgcn_readfirstlane((uint32_t)p);
        hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
        step = st;
        lim = bytes;
    }
    __device__ __forceinline__ i32x4 at(int b, bool moves) const {
        const uint64_t p = (((uint64_t)hi << 32) | lo) + (uint64_t)(b * step);
        int64_t n = moves ? lim - b * step : lim;
        n = n < 0 ? 0 : n > 0x7fffffff ? 0x7fffffff : n;
        return i32x4{(int)(uint32_t)p, (int)(uint32_t)(p >> 32), (int)n, 0x00020000};
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

// EX: exact products (fp8_mfma_exact).
template <bool WR, bool EX, int TQ, int TP, int WQ, int WP, int SL>
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
    uint32_t soff;
    if (!odd) {
        const int64_t n = w.r1 - w.r0 < TP ? w.r1 - w.r0 : TP;
        bs.init(a.x.p + w.r0 + w.st0 * a.x.blk, a.x.blk * 4, n * 4);
        soff = 16 * lane;
    } else if (WR) {
        const int64_t n = m.Q - w.q0 < TQ ? m.Q - w.q0 : TQ;
        bs.init(a.w.p + e * a.w.mat + w.q0 + w.st0 * a.w.blk, a.w.blk * 4, n * 4);
        soff = 16 * lane;
    } else {
        // lane l: that of 128 rows l % 2 of the tile
        const int64_t first = w.q0 / kFp8Block, last = (m.Q + kFp8Block - 1) / kFp8Block - 1;
        bs.init(a.w.p + e * a.w.mat + first * a.w.row + w.st0 * a.w.blk, a.w.blk * 4, 0x7fffffff);
        soff = (uint32_t)(((lane & 1) < last - first ? (lane & 1) : last - first) * a.w.row * 4);
    }
    // a wave's pieces (a fragment's 16 rows x 64 bytes): lane's offset in the first
    // fragment's rows, and what the next fragments add
    const int chunk = 16 * ((lane & 3) ^ mm_swz(lane >> 2));
    uint32_t qoff[L::QL / 2], poff[L::NPH][L::PL / 2];
    int qf[L::QL / 2], pf[L::NPH][L::PL / 2];
#pragma unroll
    for (int j = 0; j < L::QL / 2; ++j) {
        qf[j] = wave * (L::QL / 2) + j;
        qoff[j] = (uint32_t)(row_of(qf[j] * 16 + (lane >> 2)) * m.ldq + chunk);
    }
#pragma unroll
    for (int h = 0; h < L::NPH; ++h)
#pragma unroll
        for (int j = 0; j < L::PL / 2; ++j) {
            const int n = wave * (L::PL / 2) + j;
            pf[h][j] = n / L::YP * L::FP + h * L::YP + n % L::YP;
            poff[h][j] = (uint32_t)(row_of(pf[h][j] * 16 + (lane >> 2)) * m.ldp + chunk);
        }
    auto slot_at = [&](int b) { return (uint32_t)(L::SLOTS == 3 ? b % 3 : b & (L::SLOTS - 1)) * L::SLOT; };
    auto slot_of = [&](int b) { return lds32 + slot_at(b); };
    auto scales_of = [&](int b) { return L::S_AT + (b & 3) * L::S_SLOT; };
    auto issue_q = [&](int b) {
        const i32x4 r = bq.at(b, true);
        const uint32_t s = slot_of(b);
#pragma unroll
        for (int j = 0; j < L::QL / 2; ++j) {
            dma16<0, 0>(r, s + qf[j] * 1024, qoff[j]);
            dma16<TQ * 64, 64>(r, s + qf[j] * 1024, qoff[j]);
        }
    };
    auto issue_p = [&](auto hc, int b) {
        constexpr int H = decltype(hc)::value;
        const i32x4 r = bp.at(b, true);
        const uint32_t s = slot_of(b);
#pragma unroll
        for (int j = 0; j < L::PL / 2; ++j) {
            dma16<L::P_AT, 0>(r, s + pf[H][j] * 1024, poff[H][j]);
            dma16<L::P_AT + TP * 64, 64>(r, s + pf[H][j] * 1024, poff[H][j]);
        }
    };
    // (past the last block the walk may leave the scales: nothing is read)
    auto issue_s = [&](int b) {
        i32x4 r = bs.at(b, false);
        if (b >= w.nst) r[2] = 0;
        const uint32_t s = lds32 + scales_of(b);
        if (!odd) dma16<0, 0>(r, s, soff);
        else if (WR) dma16<L::WS_AT, 0>(r, s, soff);
        else dma4(r, s + L::WS_AT, soff);
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
        const int n = tail - 64 * half - chunk;        // bytes of the lane's chunk that stay
        uint4* const d = reinterpret_cast<uint4*>(piece + lane * 16);
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
            clear(s + qf[j] * 1024, 0);
            clear(s + TQ * 64 + qf[j] * 1024, 1);
        }
    };
    auto clear_p = [&](auto hc, uint8_t* s) {
        constexpr int H = decltype(hc)::value;
#pragma unroll
        for (int j = 0; j < L::PL / 2; ++j) {
            clear(s + L::P_AT + pf[H][j] * 1024, 0);
            clear(s + L::P_AT + TP * 64 + pf[H][j] * 1024, 1);
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
    Fp8Wide qx[EX ? L::FQ : 1], px[EX ? 2 : 1];
    Tokens tok[2];                     // of fragments y (even, odd)
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
            if constexpr (EX) t[K & 3] = fp8_mfma_exact(qx[X], px[Y & 1]);
            else t[K & 3] = fp8_mfma(cur.q[X].lo, cur.q[X].hi, tok[Y & 1].p.lo, tok[Y & 1].p.hi);
            add(std::integral_constant<int, J / L::FQ>{}, std::integral_constant<int, J % L::FQ>{}, K >= 2 ? cur : nxt);
            if constexpr (X == 0) {
                if constexpr (Y + 1 < L::FP) tok[(Y + 1) & 1] = read_p(std::integral_constant<int, Y + 1>{}, at);
                else if constexpr (L::PRE) tok[0] = read_p(std::integral_constant<int, 0>{}, to);
            } else if constexpr (X == 1) {
                loads();
            } else if constexpr (X == 2 && L::PRE) {
                // the next block's weights, over the last FQ fragments; exact products widen
                // them in the last one, and have them a fragment earlier
                constexpr int N = (EX ? 2 : 1) * (L::FP < L::FQ ? L::FQ / L::FP : 1);
                constexpr int AT = (Y - (L::FP - L::FQ / N - (EX && L::FP > 2))) * N;
                if constexpr (AT >= 0 && AT < L::FQ)
                    mm_for<N>([&](auto n) { read_q(std::integral_constant<int, (AT < 0 ? 0 : AT) + decltype(n)::value>{}, to, nxt); });
            }
            if constexpr (EX) {
                // what has had its last use, and the next tokens
                if constexpr (Y + 1 == L::FP && L::PRE) qx[X] = fp8_widen(nxt.q[X].lo, nxt.q[X].hi);
                if constexpr (X == 3 && (Y + 1 < L::FP || L::PRE)) px[(Y + 1) & 1] = fp8_widen(tok[(Y + 1) & 1].p.lo, tok[(Y + 1) & 1].p.hi);
            }
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    auto widen_block = [&](const Weights& w_) {        // weights and first tokens that were read ahead
        if constexpr (EX) {
            mm_for<L::FQ>([&](auto xc) {
                constexpr int X = decltype(xc)::value;
                qx[X] = fp8_widen(w_.q[X].lo, w_.q[X].hi);
            });
            px[0] = fp8_widen(tok[0].p.lo, tok[0].p.hi);
        }
    };
    auto read_block = [&](const Place& at, Weights& w_) {
        mm_for<L::FQ>([&](auto xc) { read_q(xc, at, w_); });
        tok[0] = read_p(std::integral_constant<int, 0>{}, at);
        widen_block(w_);
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
            read_block(place(0), wt[0]);
            by_twos([&](int b, const Weights& cur, Weights& nxt) {
                const Place at = place(b), to = place(b + 1);
                auto go = [&](auto yc, auto&& loads) { group(yc, at, to, cur, nxt, loads); };
                // the second half of this block has landed; every wave has its weights, and
                // has read the second half of the last block
                wait_vm<L::QL + L::PL + 1>();
                if (b == last && tail < kFp8Block) clear_p(H1{}, lds + slot_at(b));
                lds_barrier();
                go(std::integral_constant<int, 0>{}, [&] { issue_p(H1{}, b + 1); });
                go(std::integral_constant<int, 1>{}, [&] { issue_q(b + 2); });
                go(std::integral_constant<int, 2>{}, none);
                go(std::integral_constant<int, 3>{}, none);
                // the next block's weights and first half have landed; every wave has read this one's
                wait_vm<L::QL + L::PL>();
                tail_first(b + 1);
                lds_barrier();
                go(std::integral_constant<int, 4>{}, [&] { issue_p(H0{}, b + 2); });
                go(std::integral_constant<int, 5>{}, [&] { issue_s(b + 2); });
                go(std::integral_constant<int, 6>{}, none);
                go(std::integral_constant<int, 7>{}, none);
            });
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
        if (last & 1) rest(wt[1]);
        else rest(wt[0]);
        wait_vm<0>();                  // no load of this workgroup may land after it ends
    }

    // The wave's outputs, turned in 8 KiB of LDS into 16-byte pieces of rows (as in
    // mm_tiles.hpp): lane (i, g), register r of fragments (x, y) is row
    // 4 i + y % 4 of 64, column 16 g + 4 r + x of 64.
    lds_barrier();                     // every wave has read its last block
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
                const int row = YN * i + yy;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const f32x4 v = {acc[0][yg + yy][k], acc[1][yg + yy][k], acc[2][yg + yy][k], acc[3][yg + yy][k]};
                    const int at = (16 * g + 4 * k) * ES, ch = (at >> 4) ^ (row & (CH - 1));
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
                const int row = n * RPI + lane / CH, c = lane % CH, f = fp0 + yg;
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
// (Not with a scale for each weight row: at 8192^3 256 x 128 takes 671 us, 128 x 128 in
// pairs 651.)
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
    if (parts == 4) fp8_tile<false, false, 128, 128, 2, 4, 4>(a, w, lds);
    else if (parts == 2 || w.r1 - w.r0 <= 128) fp8_tile<false, false, 256, 128, 4, 2, 3>(a, w, lds);
    else fp8_tile<false, false, 256, 256, 4, 2, 2>(a, w, lds);
}

// Small products: one tile size, the contraction split where tiles are few.
template <bool WR, bool EX, int TQ, int TP, int WQ, int WP, int SL>
__global__ void __launch_bounds__(WQ* WP * 64, 2) k_mm_fp8_tiles(MmFp8Args a, uint32_t nq, uint32_t np) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[Fp8Lay<TQ, TP, WQ, WP, SL>::LDS];
    const uint32_t rows = a.m.offs ? (uint32_t)mm_count_tiles(a.m, TP) : np, per = rows * nq;
    uint32_t id;
    if (!mm_xcd(blockIdx.x, per * (uint32_t)a.m.splits, &id)) return;
    const int split = (int)(id / per);
    MmWork w;
    if (!mm_work<false, TQ, TP>(a.m, id - split * per, rows, nq, split, kFp8Block, &w)) return;
    fp8_tile<WR, EX, TQ, TP, WQ, WP, SL>(a, w, lds);
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
    if (a.exact) return go(k_mm_fp8_tiles<WR, true, 128, 128, 2, 2, 2>, a, 128, 128, 256, 0, s);
    if (size == 1) return go(k_mm_fp8_tiles<WR, false, 128, 128, 2, 2, 2>, a, 128, 128, 256, 0, s);
    if (size == 2) return go(k_mm_fp8_tiles<WR, false, 128, 128, 2, 4, 4>, a, 128, 128, 512, 0, s);
    if (WR) return hipErrorInvalidValue;
    // cutting the last round adds at most 3 workgroups for each of 64 tiles
    return go(k_mm_fp8_large, a, 256, 256, 512, 3 * kMmCUs / 4, s);
}

}  // namespace

hipError_t launch_mm_fp8_tiles(const MmFp8Args& a, int size, hipStream_t s) {
    return a.w_rows ? pick<true>(a, size, s) : pick<false>(a, size, s);
}

}  // namespace ssg
