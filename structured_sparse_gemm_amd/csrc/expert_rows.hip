// expert_rows.hip -- the rows of the expert-grouped products: their order by
// expert, the copies of token rows into it, the weighted sums of expert rows
// back, and the gradients of these.
//
// Pair n * k + j is slot j of token n.  Sorted stably by expert, the pairs are
// the rows of the grouped products: rows offs[e] .. offs[e + 1] - 1 are expert
// e's, rows[r] is the pair of row r and pos[n, j] the row of a pair.  A pair
// whose expert is outside 0 .. E - 1 (a slot that the router left empty, a
// padded token) has no row: pos is -1, and as many rows at the end have -1.
// The kernels below check both against their ranges, so that other contents
// give wrong results but no access out of range.
#include <algorithm>
#include <type_traits>

#include "experts.hpp"
#include "lanes.hpp"
#include "ssg_device.hpp"

namespace ssg {

namespace {

// ------------------------------------------------------------------ the order
//
// A counting sort.  The pairs are cut into chunks, a workgroup each, and a
// chunk into 16 runs, a wave each; LDS holds the counts of every run by expert,
// which scans over runs, chunks and experts turn into the row that the run's
// next pair of an expert takes.  A wave goes through its run 64 pairs at a time;
// ballots over the bits of the expert give each lane the lanes with the same
// one, so the rows within a run keep the pairs' order, and nothing depends on
// the order of atomics (they only count).
//
// Up to kOneChunk pairs a single workgroup does it in one launch.  Above, one
// launch counts the chunks, and in the next each workgroup sums the counts of
// all chunks by itself (as many as 256 x E words, from the caches), which costs
// less than a third launch for that scan.
constexpr int kOrderThreads = 1024, kRuns = kOrderThreads / 64;
constexpr int kHeld = 4;               // pairs of a lane in registers between the two passes
constexpr int64_t kOneChunk = 4096, kMostChunk = 4096;
constexpr int kMaxChunks = 256;

// Pairs of a chunk: few chunks have few counts to sum, many have short runs.  32 chunks,
// of 1024 to 4096 pairs (more beyond): 8192, 65536 and 262144 pairs of 256 experts take
// 7.6, 9.3 and 13.2 us; the first in one workgroup 11.4, the second in chunks of 4096
// 10.3, the third of 1024 21.8.
inline int64_t chunk_pairs(int64_t P) {
    if (P <= kOneChunk) return P;
    auto up = [](int64_t n) { return (n + kOrderThreads - 1) / kOrderThreads * kOrderThreads; };
    return std::max(std::min(up((P + 31) / 32), kMostChunk), up((P + kMaxChunks - 1) / kMaxChunks));
}

struct OrderArgs {
    int64_t P, chunk;
    int k, E, bits;
    const int32_t* experts;
    int64_t lde;
    int32_t *offs, *rows, *pos;
    uint32_t* counts;                  // [chunks][E], where there are several
};

// Expert of pair i, E for none.
__device__ __forceinline__ uint32_t expert_of(const OrderArgs& a, int64_t i) {
    int32_t e;
    if (a.lde == a.k) {
        e = a.experts[i];
    } else {
        const int64_t n = i / a.k;
        e = a.experts[n * a.lde + (i - n * a.k)];
    }
    return (uint32_t)e < (uint32_t)a.E ? (uint32_t)e : (uint32_t)a.E;
}

__global__ void __launch_bounds__(kOrderThreads) k_order_count(OrderArgs a) {
    __shared__ uint32_t n[kMaxExperts];
    for (int e = threadIdx.x; e < a.E; e += kOrderThreads) n[e] = 0;
    __syncthreads();
    const int64_t i0 = blockIdx.x * a.chunk, i1 = i0 + a.chunk < a.P ? i0 + a.chunk : a.P;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kOrderThreads) {
        const uint32_t e = expert_of(a, i);
        if (e < (uint32_t)a.E) atomicAdd(&n[e], 1u);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kOrderThreads) a.counts[(int64_t)blockIdx.x * a.E + e] = n[e];
}

__global__ void __launch_bounds__(kOrderThreads) k_order(OrderArgs a) {
    extern __shared__ uint32_t lds[];
    uint32_t* const next = lds;                    // [kRuns][E]: counts, then the row of the run's next pair
    __shared__ uint32_t waves[kRuns], total_rows;
    if (threadIdx.x == 0) total_rows = 0;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int64_t i0 = blockIdx.x * a.chunk, i1 = i0 + a.chunk < a.P ? i0 + a.chunk : a.P;
    const int64_t run = ((i1 - i0 + kRuns - 1) / kRuns + 63) / 64 * 64;
    const int64_t r0 = i0 + wave * run, r1 = r0 + run < i1 ? r0 + run : i1;
    for (int e = t; e < kRuns * a.E; e += kOrderThreads) next[e] = 0;
    __syncthreads();
    uint32_t* const mine = next + wave * a.E;
    // the experts of the first pairs stay in registers for the second pass
    uint32_t held[kHeld];
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
        const int64_t i = r0 + 64 * u + lane;
        held[u] = i < r1 ? expert_of(a, i) : (uint32_t)a.E;
    }
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
        if (held[u] < (uint32_t)a.E) atomicAdd(&mine[held[u]], 1u);
    for (int64_t i = r0 + 64 * kHeld + lane; i < r1; i += 64) {
        const uint32_t e = expert_of(a, i);
        if (e < (uint32_t)a.E) atomicAdd(&mine[e], 1u);
    }
    // thread e: pairs of expert e in all chunks, and in those before this one
    uint32_t total = 0, before = 0;
    if (a.counts && t < a.E) {
        const int chunks = (int)gridDim.x;
        constexpr int B = 16;          // loads on their way
        for (int c0 = 0; c0 < chunks; c0 += B) {
            uint32_t v[B];
#pragma unroll
            for (int c = 0; c < B; ++c) v[c] = a.counts[(int64_t)(c0 + c < chunks ? c0 + c : c0) * a.E + t];
#pragma unroll
            for (int c = 0; c < B; ++c) {
                if (c0 + c >= chunks) v[c] = 0;
                total += v[c];
                before += c0 + c < (int)blockIdx.x ? v[c] : 0;
            }
        }
    }
    __syncthreads();
    if (t < a.E) {
        uint32_t sum = 0;
        for (int w = 0; w < kRuns; ++w) {
            const uint32_t v = next[w * a.E + t];
            next[w * a.E + t] = before + sum;
            sum += v;
        }
        if (!a.counts) total = sum;
    }
    // first row of expert t
    uint32_t inc = total;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t u = (uint32_t)__shfl_up((int)inc, d);
        if (lane >= d) inc += u;
    }
    if (lane == 63) waves[wave] = inc;
    __syncthreads();
    uint32_t start = inc - total;
    for (int w = 0; w < wave; ++w) start += waves[w];
    if (t < a.E) {
        for (int w = 0; w < kRuns; ++w) next[w * a.E + t] += start;
        if (blockIdx.x == 0) a.offs[t] = (int32_t)start;
        if (t == a.E - 1) total_rows = start + total;
    }
    __syncthreads();
    if (blockIdx.x == 0 && t == 0) a.offs[a.E] = (int32_t)total_rows;
    auto place = [&](int64_t i, uint32_t e) {      // the pairs i .. i + 63, lane's expert e
        const bool in = i + lane < r1;
        uint64_t same = __ballot(in && e < (uint32_t)a.E);
        const bool there = (same >> lane) & 1;
        for (int b = 0; b < a.bits; ++b) {
            const bool bit = (e >> b) & 1;
            const uint64_t set = __ballot(bit);
            same &= bit ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        uint32_t at = 0;
        if (there) at = mine[e] + rank;
        __builtin_amdgcn_wave_barrier();           // a wave's LDS accesses stay in order
        if (there && rank == 0) mine[e] += __popcll(same);
        __builtin_amdgcn_wave_barrier();
        if (in) a.pos[i + lane] = there ? (int32_t)at : -1;
        if (there) a.rows[at] = (int32_t)(i + lane);
    };
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
        if (r0 + 64 * u < r1) place(r0 + 64 * u, held[u]);
    for (int64_t i = r0 + 64 * kHeld; i < r1; i += 64) place(i, i + lane < r1 ? expert_of(a, i + lane) : (uint32_t)a.E);
    for (int64_t r = i0 + t; r < i1; r += kOrderThreads)
        if (r >= total_rows) a.rows[r] = -1;
}

// ------------------------------------------------------------------ the rows
//
// Gather and the combine's gradient are bound by memory (from HBM 4.9 and 5.4 TB/s), the
// combine by latency: 4096 tokens of 4 x 4096 in 57 us, 3.0 TB/s, since a slot's place,
// weight and row are each waited for before the next slot's (the gradient has four slots
// on their way).  A workgroup has a token and kTile columns of its row, so a
// token's row is read (gather, the combine's gradient) or written (combine) once
// and its k expert rows meet it there: in the order of the rows, every token row
// would be read k times.  A thread has 16 bytes of a row; rows that are not all
// aligned to 16 bytes go element by element, neighbouring lanes neighbouring
// elements.
constexpr int kThreads = 256;

template <int DT> struct Elem;
template <> struct Elem<FT_F16> { typedef _Float16 type; };
template <> struct Elem<FT_BF16> { typedef __bf16 type; };
template <> struct Elem<FT_F32> { typedef float type; };

// N elements of a row from `at` on (N = 1: any alignment that the type has).
template <int DT, int N>
__device__ __forceinline__ void load_row(const void* p, int64_t at, float (&v)[N]) {
    typedef typename Elem<DT>::type E;
    E e[N];
    if constexpr (N == 1) e[0] = reinterpret_cast<const E*>(p)[at];
    else *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(reinterpret_cast<const E*>(p) + at);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (float)e[i];
}

// (a 16-bit type: rounded to nearest even)
template <int DT, int N>
__device__ __forceinline__ void store_row(void* p, int64_t at, const float (&v)[N]) {
    typedef typename Elem<DT>::type E;
    E e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = (E)v[i];
    if constexpr (N == 1) {
        reinterpret_cast<E*>(p)[at] = e[0];
    } else {
#pragma unroll
        for (int c = 0; c < N * (int)sizeof(E) / 16; ++c)
            reinterpret_cast<uint4*>(reinterpret_cast<E*>(p) + at)[c] = reinterpret_cast<const uint4*>(e)[c];
    }
}

// out[pos[n, j]] = X[n]; rows of nobody are zeros.  T: what a thread copies.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_gather(RowsArgs a, int64_t n0, int64_t cols, uint32_t tiles) {
    const uint32_t b = blockIdx.x / tiles;
    const int64_t n = n0 + b, c = (int64_t)(blockIdx.x - b * tiles) * kThreads + threadIdx.x;
    if (c >= cols) return;
    const T v = reinterpret_cast<const T*>(a.x)[n * a.ldx + c];
    T* const out = reinterpret_cast<T*>(a.o);
    for (int j = 0; j < a.k; ++j) {
        const int64_t pair = n * a.k + j;
        const int32_t p = a.pos[pair], r = a.rows[pair];
        if ((uint32_t)p < (uint64_t)a.P) out[p * a.ldo + c] = v;
        if ((uint32_t)r >= (uint64_t)a.P) out[pair * a.ldo + c] = T{};
    }
}

// out[n] = sum_j w[n, j] Y[pos[n, j]], in slot order, in fp32.
template <int DT, int OUT, int N>
__global__ void __launch_bounds__(kThreads) k_combine(RowsArgs a, int64_t n0, uint32_t tiles) {
    const uint32_t b = blockIdx.x / tiles;
    const int64_t n = n0 + b, c = ((int64_t)(blockIdx.x - b * tiles) * kThreads + threadIdx.x) * N;
    if (c >= a.D) return;
    float sum[N];
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        const int32_t p = a.pos[n * a.k + j];
        if ((uint32_t)p >= (uint64_t)a.P) continue;
        const float w = a.w ? a.w[n * a.ldw + j] : 1.0f;
        float v[N];
        load_row<DT, N>(a.y, p * a.ldy + c, v);
#pragma unroll
        for (int i = 0; i < N; ++i) sum[i] = fmaf(w, v[i], sum[i]);
    }
    store_row<OUT, N>(a.o, n * a.ldo + c, sum);
}

// dY[pos[n, j]] = w[n, j] dO[n], dw[n, j] = <dO[n], Y[pos[n, j]]>; rows of nobody
// are zeros, and so is dw of a pair without a row.  A workgroup has a token; a
// thread's products are added in column order, the threads' sums in lane and
// wave order.  JB slots at a time, for the registers that hold their sums.
template <int DT, int N>
__global__ void __launch_bounds__(kThreads) k_combine_backward(RowsArgs a, int64_t n0) {
    constexpr int JB = 4, kWaves = kThreads / 64;
    __shared__ float part[kWaves][JB];
    const int64_t n = n0 + blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int j0 = 0; j0 < a.k; j0 += JB) {
        int64_t p[JB];
        float w[JB], dot[JB];
        bool clear[JB];
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            const int64_t pair = n * a.k + j0 + j;
            const bool in = j0 + j < a.k;
            const int32_t q = in ? a.pos[pair] : -1;
            p[j] = (uint32_t)q < (uint64_t)a.P ? q : -1;
            w[j] = p[j] >= 0 ? a.w[n * a.ldw + j0 + j] : 0.0f;
            clear[j] = in && (uint32_t)a.rows[pair] >= (uint64_t)a.P;
            dot[j] = 0.0f;
        }
        for (int64_t c = (int64_t)threadIdx.x * N; c < a.D; c += kThreads * N) {
            float d[N], y[JB][N];
            load_row<DT, N>(a.x, n * a.ldx + c, d);
#pragma unroll
            for (int j = 0; j < JB; ++j)
                if (p[j] >= 0) load_row<DT, N>(a.y, p[j] * a.ldy + c, y[j]);
#pragma unroll
            for (int j = 0; j < JB; ++j) {
                float g[N];
                if (p[j] >= 0) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        dot[j] = fmaf(d[i], y[j][i], dot[j]);
                        g[i] = w[j] * d[i];
                    }
                    store_row<DT, N>(a.o, p[j] * a.ldo + c, g);
                }
                if (clear[j]) {
#pragma unroll
                    for (int i = 0; i < N; ++i) g[i] = 0.0f;
                    store_row<DT, N>(a.o, (n * a.k + j0 + j) * a.ldo + c, g);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            const float s = lanes_sum<64>(dot[j]);
            if (lane == 0) part[wave][j] = s;
        }
        __syncthreads();
        if (threadIdx.x < JB && j0 + threadIdx.x < a.k) {
            float s = 0.0f;
#pragma unroll
            for (int v = 0; v < kWaves; ++v) s += part[v][threadIdx.x];
            a.dw[n * a.lddw + j0 + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

bool al16(const void* p, int64_t ld_bytes) { return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)ld_bytes) % 16 == 0; }

// f(first token, workgroups) for slabs of tokens: a launch has fewer than 2^32 threads.
template <typename F>
hipError_t by_tokens(int64_t N, int64_t tiles, F&& f) {
    const int64_t most = ((int64_t)1 << 32) / kThreads - 1, slab = most / tiles;   // (tiles < 2^22)
    for (int64_t n = 0; n < N; n += slab) {
        f(n, dim3((unsigned)((N - n < slab ? N - n : slab) * tiles)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename T>
hipError_t gather(RowsArgs a, hipStream_t s) {
    const int64_t es = ft_bytes(a.dt), per = (int64_t)sizeof(T) / es, cols = a.D / per;
    a.ldx /= per;
    a.ldo /= per;
    const int64_t tiles = (cols + kThreads - 1) / kThreads;
    if (tiles == 0) return hipSuccess;
    return by_tokens(a.N, tiles, [&](int64_t n, dim3 grid) {
        hipLaunchKernelGGL((k_gather<T>), grid, dim3(kThreads), 0, s, a, n, cols, (uint32_t)tiles);
    });
}

template <int DT, int OUT, int N>
hipError_t combine(const RowsArgs& a, hipStream_t s) {
    const int64_t tiles = (a.D + kThreads * N - 1) / (kThreads * N);
    if (tiles == 0) return hipSuccess;
    return by_tokens(a.N, tiles, [&](int64_t n, dim3 grid) {
        hipLaunchKernelGGL((k_combine<DT, OUT, N>), grid, dim3(kThreads), 0, s, a, n, (uint32_t)tiles);
    });
}

template <int DT>
hipError_t combine_out(const RowsArgs& a, hipStream_t s) {
    constexpr int N = 16 / ft_bytes(DT);
    const bool vec = a.D % N == 0 && al16(a.y, a.ldy * ft_bytes(DT)) && al16(a.o, a.ldo * ft_bytes(a.out));
    if (a.out == FT_F32) return vec ? combine<DT, FT_F32, N>(a, s) : combine<DT, FT_F32, 1>(a, s);
    return vec ? combine<DT, DT, N>(a, s) : combine<DT, DT, 1>(a, s);
}

template <int DT>
hipError_t combine_backward(const RowsArgs& a, hipStream_t s) {
    constexpr int ES = ft_bytes(DT), N = 16 / ES;
    const bool vec = a.D % N == 0 && al16(a.x, a.ldx * ES) && al16(a.y, a.ldy * ES) && al16(a.o, a.ldo * ES);
    return by_tokens(a.N, 1, [&](int64_t n, dim3 grid) {
        if (vec) hipLaunchKernelGGL((k_combine_backward<DT, N>), grid, dim3(kThreads), 0, s, a, n);
        else hipLaunchKernelGGL((k_combine_backward<DT, 1>), grid, dim3(kThreads), 0, s, a, n);
    });
}

}  // namespace

int expert_order_chunks(int64_t pairs) {
    if (pairs <= kOneChunk) return 1;
    const int64_t c = chunk_pairs(pairs);
    return (int)((pairs + c - 1) / c);
}

hipError_t launch_expert_order(int64_t N, int k, int E, const int32_t* experts, int64_t lde, int32_t* offs,
                               int32_t* rows, int32_t* pos, uint32_t* counts, hipStream_t s) {
    OrderArgs a{};
    a.P = N * k;
    a.chunk = chunk_pairs(a.P);
    a.k = k;
    a.E = E;
    while ((1 << a.bits) < E) ++a.bits;
    a.experts = experts;
    a.lde = lde;
    a.offs = offs;
    a.rows = rows;
    a.pos = pos;
    const int chunks = expert_order_chunks(a.P);
    if (chunks > 1) {
        a.counts = counts;
        hipLaunchKernelGGL(k_order_count, dim3(chunks), dim3(kOrderThreads), 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(k_order, dim3(chunks), dim3(kOrderThreads), kRuns * E * sizeof(uint32_t), s, a);
    return hipGetLastError();
}

hipError_t launch_expert_gather(const RowsArgs& a, hipStream_t s) {
    const int64_t es = ft_bytes(a.dt);
    if (a.D * es % 16 == 0 && al16(a.x, a.ldx * es) && al16(a.o, a.ldo * es)) return gather<uint4>(a, s);
    return es == 4 ? gather<uint32_t>(a, s) : gather<uint16_t>(a, s);
}

hipError_t launch_expert_combine(const RowsArgs& a, hipStream_t s) {
    return a.dt == FT_F16 ? combine_out<FT_F16>(a, s) : a.dt == FT_BF16 ? combine_out<FT_BF16>(a, s)
                                                                        : combine_out<FT_F32>(a, s);
}

hipError_t launch_expert_combine_backward(const RowsArgs& a, hipStream_t s) {
    return a.dt == FT_F16 ? combine_backward<FT_F16>(a, s) : a.dt == FT_BF16 ? combine_backward<FT_BF16>(a, s)
                                                                             : combine_backward<FT_F32>(a, s);
}

}  // namespace ssg
