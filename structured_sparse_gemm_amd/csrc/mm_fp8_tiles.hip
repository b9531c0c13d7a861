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
// LDS a block (128 bytes of every row) at a time by direct-to-LDS loads, two
// slots.  A slot is freed in two phases: a wave keeps its weight fragments of the
// block in registers and goes through the tokens' fragments in two halves, so
// after the first half the weights' part and the first tokens' part of the slot
// take the loads of the block after next, after the second half the rest.  Every
// load thus has one and a half blocks' time to arrive in LDS for two.  (Tiles of few
// token fragments have one phase.)
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

template <int TQ, int TP, int WQ, int WP>
struct Fp8Lay {
    static constexpr int NW = WQ * WP, FQ = TQ / WQ / 16, FP = TP / WP / 16;
    static constexpr int NPH = FP > 4 ? 2 : 1, YP = FP / NPH;        // phases of a block, token fragments of each
    static constexpr int Q_BYTES = TQ * 128, P_BYTES = TP * 128;
    static constexpr int P_AT = Q_BYTES, SLOT = P_AT + P_BYTES;
    // Scales: read in both phases of a block, but loaded with its first part, so
    // the block after next must not take their place.
    static constexpr int S_AT = 2 * SLOT, WS_AT = 1024, S_SLOT = 2048;
    static constexpr int LDS = S_AT + 4 * S_SLOT;
    static constexpr int QL = TQ / 16 * 2 / NW, PL = YP * WP * 2 / NW;   // loads of a wave: weights, tokens of a phase
    static constexpr int FIRST = QL + PL + 1;                            // and in all, with a scale load
    static_assert(FQ == 4 && QL % 2 == 0 && PL % 2 == 0 && TQ <= 256 && TP <= 256, "tile");
    static_assert(NW * 8192 <= LDS && LDS <= 160 * 1024, "LDS");
};

// LDS row (of fragment f = slot / 16) to tile row, as in mm_tiles.hpp
__device__ __forceinline__ int row_of(int slot) { return (slot & ~63) + 4 * (slot & 15) + ((slot >> 4) & 3); }

// EX: exact products (fp8_mfma_exact).
template <bool WR, bool EX, int TQ, int TP, int WQ, int WP>
__device__ __forceinline__ void fp8_tile(const MmFp8Args& a, const MmWork& w, uint8_t* lds) {
    using L = Fp8Lay<TQ, TP, WQ, WP>;
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
    auto slot_of = [&](int b) { return lds32 + (b & 1) * L::SLOT; };
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
    auto issue_first = [&](int b) {
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
        if (n >= 16) return;
        uint32_t* const d = reinterpret_cast<uint32_t*>(piece + lane * 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int keep = n - 4 * k;
            if (keep <= 0) d[k] = 0;
            else if (keep < 4) d[k] &= (1u << (8 * keep)) - 1;
        }
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
    auto frag = [&](const uint8_t* at, int f) -> uint4 {
        return *reinterpret_cast<const uint4*>(at + f * 1024 + i * 64 + ((g ^ mm_swz(i)) << 4));
    };
    uint4 q[EX ? 1 : L::FQ][2];
    Fp8Wide qx[EX ? L::FQ : 1];
    float ws = 0.0f;
    f32x4 wr[WR ? 4 : 1];              // scales of rows 16 g + 4 r + x of the wave's 64: [r][x]
    auto phase = [&](auto hc, int b) {
        constexpr int H = decltype(hc)::value;
        const uint8_t *const s = lds + (b & 1) * L::SLOT, *const sc = lds + scales_of(b);
        if constexpr (H == 0) {
#pragma unroll
            for (int x = 0; x < L::FQ; ++x) {
                const uint4 a0 = frag(s, fq0 + x), a1 = frag(s + TQ * 64, fq0 + x);
                if constexpr (EX) {
                    qx[x] = fp8_widen(a0, a1);
                } else {
                    q[x][0] = a0;
                    q[x][1] = a1;
                }
            }
            if constexpr (WR) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    wr[r] = *reinterpret_cast<const f32x4*>(sc + L::WS_AT + (wq * 64 + 16 * g + 4 * r) * 4);
            } else {
                ws = *reinterpret_cast<const float*>(sc + L::WS_AT + (wq * 64 / kFp8Block) * 4);
            }
        }
#pragma unroll
        for (int yy = 0; yy < L::YP; ++yy) {
            const int y = H * L::YP + yy, f = fp0 + y;
            const uint4 p0 = frag(s + L::P_AT, f), p1 = frag(s + L::P_AT + TP * 64, f);
            const float xs = *reinterpret_cast<const float*>(sc + (f / 4 * 64 + 4 * i + f % 4) * 4);
            Fp8Wide px;
            if constexpr (EX) px = fp8_widen(p0, p1);
#pragma unroll
            for (int x = 0; x < L::FQ; ++x) {
                f32x4 d;
                if constexpr (EX) d = fp8_mfma_exact(qx[x], px);
                else d = fp8_mfma(q[x][0], q[x][1], p0, p1);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[x][y][r] = fmaf(d[r], xs * (WR ? wr[WR ? r : 0][x] : ws), acc[x][y][r]);
            }
        }
    };

    if (w.nst > 0) {
        uint8_t* const last_slot = lds + (last & 1) * L::SLOT;
        if constexpr (L::NPH == 2) {
            issue_first(0);
            issue_p(H1{}, 0);
            issue_first(1);
            constexpr int V = L::FIRST + L::PL;
            for (int b = 0; b < w.nst; ++b) {
                // newer than what this phase reads: the other half's loads and the next block's first
                wait_vm<V>();
                if (b == last && tail < kFp8Block) {
                    clear_q(last_slot);
                    clear_p(H0{}, last_slot);
                }
                lds_barrier();         // this half has landed, every wave has read the last one
                issue_p(H1{}, b + 1);
                phase(H0{}, b);
                wait_vm<V>();
                if (b == last && tail < kFp8Block) clear_p(H1{}, last_slot);
                lds_barrier();
                issue_first(b + 2);
                phase(H1{}, b);
            }
        } else {
            issue_first(0);
            for (int b = 0; b < w.nst; ++b) {
                wait_vm<0>();
                if (b == last && tail < kFp8Block) {
                    clear_q(last_slot);
                    clear_p(H0{}, last_slot);
                }
                lds_barrier();
                issue_first(b + 1);
                phase(H0{}, b);
            }
        }
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
template <bool WR>
__global__ void __launch_bounds__(512, 2) k_mm_fp8_large(MmFp8Args a, uint32_t nq, uint32_t np) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[Fp8Lay<256, 256, 4, 2>::LDS];
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
    if (parts == 4) fp8_tile<WR, false, 128, 128, 2, 4>(a, w, lds);
    else if (parts == 2 || w.r1 - w.r0 <= 128) fp8_tile<WR, false, 256, 128, 4, 2>(a, w, lds);
    else fp8_tile<WR, false, 256, 256, 4, 2>(a, w, lds);
}

// Small products: one tile size, the contraction split where tiles are few.
template <bool WR, bool EX, int TQ, int TP, int WQ, int WP>
__global__ void __launch_bounds__(WQ* WP * 64, 2) k_mm_fp8_tiles(MmFp8Args a, uint32_t nq, uint32_t np) {
    __shared__ __attribute__((aligned(1024))) uint8_t lds[Fp8Lay<TQ, TP, WQ, WP>::LDS];
    const uint32_t rows = a.m.offs ? (uint32_t)mm_count_tiles(a.m, TP) : np, per = rows * nq;
    uint32_t id;
    if (!mm_xcd(blockIdx.x, per * (uint32_t)a.m.splits, &id)) return;
    const int split = (int)(id / per);
    MmWork w;
    if (!mm_work<false, TQ, TP>(a.m, id - split * per, rows, nq, split, kFp8Block, &w)) return;
    fp8_tile<WR, EX, TQ, TP, WQ, WP>(a, w, lds);
}

template <bool WR, bool EX>
hipError_t go(const MmFp8Args& a, int size, hipStream_t s) {
    const MmTileSize t = kFp8TileSizes[EX][size];
    const int64_t nq = (a.m.Q + t.q - 1) / t.q, np = (a.m.P + t.p - 1) / t.p;
    const int64_t total = mm_tile_bound(a.m, t.p) * nq * a.m.splits + (size == 0 ? 3 * kMmCUs / 4 : 0);
    if (total >= (int64_t)1 << 23) return hipErrorInvalidValue;
    const dim3 grid((unsigned)((total + 7) / 8 * 8));
    const uint32_t q = (uint32_t)nq, p = (uint32_t)np;
    if (size == 0) {
        if constexpr (EX) hipLaunchKernelGGL((k_mm_fp8_tiles<WR, true, 256, 128, 4, 2>), grid, dim3(512), 0, s, a, q, p);
        else hipLaunchKernelGGL((k_mm_fp8_large<WR>), grid, dim3(512), 0, s, a, q, p);
    } else {
        hipLaunchKernelGGL((k_mm_fp8_tiles<WR, EX, 128, 128, 2, 2>), grid, dim3(256), 0, s, a, q, p);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mm_fp8_tiles(const MmFp8Args& a, int size, hipStream_t s) {
    if (a.exact) return a.w_rows ? go<true, true>(a, size, s) : go<false, true>(a, size, s);
    return a.w_rows ? go<true, false>(a, size, s) : go<false, false>(a, size, s);
}

}  // namespace ssg
