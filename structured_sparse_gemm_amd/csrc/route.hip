// route.hip -- which experts a token goes to, and with what weights; and the
// gradient of the weights with respect to the logits.
//
// s = softmax(l) or sigmoid(l) over a token's E logits.  The choice is made by
// c = s + bias (without a bias by l itself, which orders as s does); of groups
// of E / G neighbouring experts the best top_groups stay, by their largest c or
// the sum of their two largest; then the k largest c, ties to the lower expert.
// Weights are scale * s, with renorm scale * s / (sum over the chosen s).
// An expert whose logit or bias is -inf is never chosen; NaN ranks first.
//
// The choice must not depend on how a score is rounded, or two implementations
// (a training and a serving one) would send a token to different experts: with a
// bias, or sums of two scores, scores of 24 bits are near enough to each other
// that of 8192 tokens x 256 experts some choices change.  So c is held in 64
// bits there and in the logits' own bits elsewhere, and compared as an
// unsigned key of that width: 0 stands for "never", so removing a chosen expert
// is storing 0.
//
// Bound by instructions, not by memory: 8192 x 256 fp32 logits are 8 MB, 2 us, and
// take 14.5 us with sigmoids, a bias, 4 of 8 groups and 8 choices (a third of it the
// scores in 64 bits, which every token pays for and few need), 8.4 us for 8 choices by
// softmax; one token 5.6 and 3.6 us.  The gradient, 17 MB, takes 5.8: its rows go through
// LDS one element a lane at a time, and the waves wait 61% of their cycles.
// L lanes share a token, V neighbouring experts a lane; a group has a power of
// two of the lanes to itself, so that its best are found by exchanges among
// them.  Every choice is a maximum over the lane's keys, one over the lanes
// (lanes.hpp) and a ballot for the lowest lane that has it.
#include <type_traits>

#include "experts.hpp"
#include "lanes.hpp"
#include "ssg_device.hpp"

namespace ssg {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

__device__ __forceinline__ float load_float(const void* p, int dt, int64_t at) {
    if (dt == FT_F32) return reinterpret_cast<const float*>(p)[at];
    const uint16_t b = reinterpret_cast<const uint16_t*>(p)[at];
    return dt == FT_F16 ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
}

// p[at + first + v] for v < count, `other` beyond (p[at] is there): no load waits for
// another, nor for a branch of its own.
template <int V>
__device__ __forceinline__ void load_floats(const void* p, int dt, int64_t at, int first, int count, float other,
                                            float (&x)[V]) {
    if (dt == FT_F32) {
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = reinterpret_cast<const float*>(p)[at + (v < count ? first + v : 0)];
    } else {
        uint16_t b[V];
#pragma unroll
        for (int v = 0; v < V; ++v) b[v] = reinterpret_cast<const uint16_t*>(p)[at + (v < count ? first + v : 0)];
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = dt == FT_F16 ? f16_bits_to_f32(b[v]) : bf16_bits_to_f32(b[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = v < count ? x[v] : other;
}

__device__ __forceinline__ void store_float(void* p, int dt, int64_t at, float v) {
    if (dt == FT_F32) reinterpret_cast<float*>(p)[at] = v;
    else if (dt == FT_F16) reinterpret_cast<_Float16*>(p)[at] = (_Float16)v;
    else reinterpret_cast<__bf16*>(p)[at] = (__bf16)v;
}

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xFF800000u); }

// Keys that order as the numbers do (+0 and -0 alike), NaN above all, 0 for -inf.
__device__ __forceinline__ uint32_t key32(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    if (v != v) return 0xFFFFFFFFu;
    const uint32_t k = b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
    return v == neg_inf() ? 0u : k;
}
__device__ __forceinline__ uint64_t key64(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    if (v != v) return ~0ull;
    const uint64_t k = b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
    return v == -__builtin_inf() ? 0ull : k;
}

// exp in 64 bits, off by 2^-51: x = n log 2 + r, the series of exp(r) for |r| <= log(2) / 2
// up to r^12 / 12! (the next term is 2^-52 of it).
__device__ __forceinline__ double exp64(double x) {
    const double n = __builtin_rint(fmin(fmax(x, -2000.0), 2000.0) * 0x1.71547652b82fep+0);
    const double r = fma(n, -0x1.abc9e3b39803fp-56, fma(n, -0x1.62e42fefa39efp-1, x));
    double p = 1.0 / 479001600;
    constexpr double c[12] = {1.0 / 39916800, 1.0 / 3628800, 1.0 / 362880, 1.0 / 40320, 1.0 / 5040, 1.0 / 720,
                              1.0 / 120,      1.0 / 24,      1.0 / 6,      1.0 / 2,     1.0,        1.0};
#pragma unroll
    for (double k : c) p = fma(p, r, k);
    p = ldexp(p, (int)n);
    return x > 2000.0 ? __builtin_inf() : x < -2000.0 ? 0.0 : p;   // (NaN stays NaN by r)
}

// Weights of the chosen logits x (lane j of L has slot j; `there`: slot filled):
// the scores, or their shares of the sum.  The shares are taken relative to the
// largest, so that they are numbers also where every score is below fp32's range.
template <int L>
__device__ __forceinline__ float chosen_weight(const RouteArgs& a, float x, bool there, float row_max, float row_sum) {
    float s;
    if (a.sigmoid) {
        const float top = a.renorm ? lanes_max<L>(there ? x : neg_inf()) : 0.0f;
        // below -60 a sigmoid is the exponential to 26 digits
        s = top < -60.0f ? expf(x - top) : 1.0f / (1.0f + expf(-x));
    } else if (a.renorm) {
        s = expf(x - lanes_max<L>(there ? x : neg_inf()));
    } else {
        s = expf(x - row_max) / row_sum;
    }
    if (!there) s = 0.0f;
    if (a.renorm) s /= lanes_sum<L>(s);
    return there ? s : 0.0f;
}

// How many of the groups (of 2^lg lanes; L lanes a token) come before this lane's.
template <int L, typename Key>
__device__ __forceinline__ int group_rank(Key key, int group, int groups, int seg, int lg) {
    int rank = 0;
    for (int h = 0; h < groups; ++h) {
        union { Key k; uint32_t w[sizeof(Key) / 4]; } o;
        o.k = key;
#pragma unroll
        for (uint32_t& w : o.w) {
            // (the lane is the same for the whole wave where it has one token)
            if constexpr (L == 64) w = (uint32_t)__builtin_amdgcn_readlane((int)w, h << lg);
            else w = (uint32_t)__shfl((int)w, seg * L + (h << lg));
        }
        rank += o.k > key || (o.k == key && h < group);
    }
    return rank;
}

template <int L, int V, bool WIDE>
__global__ void __launch_bounds__(kThreads) k_route(RouteArgs a, int64_t n0, int S, int lg_shift) {
    using Key = typename std::conditional<WIDE, uint64_t, uint32_t>::type;
    constexpr int T = 64 / L;                      // tokens of a wave
    __shared__ int32_t res[kWaves * T][L];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % L, seg = lane / L;
    const int64_t n = n0 + ((int64_t)blockIdx.x * kWaves + wave) * T + seg, nr = n < a.N ? n : a.N - 1;
    const int group = l >> lg_shift, base = (l & ((1 << lg_shift) - 1)) * V;
    const int first = group * S + base;
    const int count = group < a.groups ? (S - base < V ? (S - base > 0 ? S - base : 0) : V) : 0;

    float x[V], b[WIDE ? V : 1];
    load_floats<V>(a.logits, a.dt, nr * a.ldl, first, count, neg_inf(), x);
    if constexpr (WIDE)
        if (a.bias) load_floats<V>(a.bias, FT_F32, 0, first, count, neg_inf(), b);

    float row_max = 0.0f, row_sum = 1.0f;
    double sum64 = 1.0;
    if (!a.sigmoid) {
        row_max = neg_inf();
#pragma unroll
        for (int v = 0; v < V; ++v) row_max = fmaxf(row_max, x[v]);
        row_max = lanes_max<L>(row_max);
        if (row_max == neg_inf()) row_max = 0.0f;
        if (!WIDE && !a.renorm) {
            row_sum = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) row_sum += expf(x[v] - row_max);
            row_sum = lanes_sum<L>(row_sum);
        }
    }
    Key key[V];
    if constexpr (WIDE) {
        double s[V];
        if (a.sigmoid) {
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = 1.0 / (1.0 + exp64(-(double)x[v]));
        } else {
            sum64 = 0.0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[v] = exp64((double)x[v] - (double)row_max);
                sum64 += s[v];
            }
            sum64 = lanes_sum<L>(sum64);
            row_sum = (float)sum64;
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] /= sum64;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            double c = x[v];
            if (a.bias) {
                c = x[v] == neg_inf() || b[v] == neg_inf() ? (double)neg_inf() : s[v] + (double)b[v];
            }
            key[v] = key64(c);
            // what the group's score is taken of
            s[v] = key[v] == 0 ? -__builtin_inf() : a.bias || !a.top2 ? c : s[v];
        }
        if (a.groups > 1) {
            // the group's two largest, over its lanes
            double m1 = -__builtin_inf(), m2 = m1;
            bool nan = false;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                nan |= s[v] != s[v];
                m2 = fmax(m2, fmin(m1, s[v]));
                m1 = fmax(m1, s[v]);
            }
            uint32_t any_nan = nan;
            lane_steps<L == 64 ? 6 : 4>(lg_shift, [&](auto step) {
                constexpr int ST = decltype(step)::value;
                const double o1 = lane_partner<ST>(m1), o2 = lane_partner<ST>(m2);
                any_nan |= lane_partner<ST>(any_nan);
                m2 = fmax(fmin(m1, o1), fmax(m2, o2));
                m1 = fmax(m1, o1);
            });
            if (a.top2 && m2 != -__builtin_inf()) m1 += m2;
            const uint64_t gk = any_nan ? ~0ull : group < a.groups ? key64(m1) : 0;
            const int rank = group_rank<L>(gk, group, a.groups, seg, lg_shift);
            if (rank >= a.top_groups) {
#pragma unroll
                for (int v = 0; v < V; ++v) key[v] = 0;
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = key32(x[v]);
        if (a.groups > 1) {
            uint32_t gk = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) gk = gk > key[v] ? gk : key[v];
            lane_steps<L == 64 ? 6 : 4>(lg_shift, [&](auto step) { gk = max(gk, lane_partner<decltype(step)::value>(gk)); });
            const int rank = group_rank<L>(gk, group, a.groups, seg, lg_shift);
            if (rank >= a.top_groups) {
#pragma unroll
                for (int v = 0; v < V; ++v) key[v] = 0;
            }
        }
    }

    int32_t* const out = res[wave * T + seg];
    out[l] = -1;
    __syncthreads();
    if constexpr (WIDE) {
        // The upper words decide nearly always: a maximum of 32 bits over the lanes, and
        // the lower words only where two keys share it in a token.
        uint32_t hi[V], lo[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            hi[v] = (uint32_t)(key[v] >> 32);
            lo[v] = (uint32_t)key[v];
        }
        constexpr uint64_t kOnes = L == 64 ? 1 : 0x0001000100010001ull;    // a token's lowest lane
        for (int j = 0; j < a.k; ++j) {
            uint32_t best = hi[0];
#pragma unroll
            for (int v = 1; v < V; ++v) best = max(best, hi[v]);
            const uint32_t top = lanes_max<L>(best);
            uint64_t seen = 0, twice = 0;              // lanes with a key that has it, or two
            int at = 0;
#pragma unroll
            for (int v = V - 1; v >= 0; --v) {
                const bool has = hi[v] == top;
                const uint64_t lanes = __ballot(has);
                twice |= seen & lanes;
                seen |= lanes;
                at = has ? v : at;
            }
            twice |= seen & (seen - kOnes);            // (every token has one: nothing is borrowed)
            if (twice == 0) {
                if (best == top && top != 0) out[j] = first + at;
#pragma unroll
                for (int v = 0; v < V; ++v) hi[v] = hi[v] == top ? 0u : hi[v];
                continue;
            }
            uint32_t low = 0;
            at = 0;
#pragma unroll
            for (int v = V - 1; v >= 0; --v) {
                if (hi[v] == top && lo[v] >= low) {
                    low = lo[v];
                    at = v;
                }
            }
            const uint32_t top_low = lanes_max<L>(low);
            const uint64_t hit = __ballot(best == top && low == top_low) >> (seg * L);
            if (l == __builtin_ctzll(hit) && top != 0) {
                out[j] = first + at;
#pragma unroll
                for (int v = 0; v < V; ++v) hi[v] = v == at ? 0u : hi[v];
            }
        }
    } else {
        for (int j = 0; j < a.k; ++j) {
            uint32_t best = key[0];
            int at = 0;
#pragma unroll
            for (int v = 1; v < V; ++v) {
                if (key[v] > best) {
                    best = key[v];
                    at = v;
                }
            }
            const uint32_t top = lanes_max<L>(best);
            const uint64_t hit = __ballot(best == top) >> (seg * L);
            if (top != 0 && l == __builtin_ctzll(hit)) {
                out[j] = first + at;
#pragma unroll
                for (int v = 0; v < V; ++v) key[v] = v == at ? 0u : key[v];
            }
        }
    }
    __syncthreads();
    const int e = l < a.k ? out[l] : -1;
    const bool there = e >= 0;
    const float chosen = there ? load_float(a.logits, a.dt, nr * a.ldl + e) : 0.0f;
    const float w = chosen_weight<L>(a, chosen, there, row_max, row_sum) * a.scale;
    if (n < a.N && l < a.k) {
        a.weights[n * a.ldw + l] = w;
        a.experts[n * a.lde + l] = e;
    }
}

// The gradient, g = scale * dweights, q the shares of the chosen (renorm):
//   softmax           dl_i = p_i (g_i - sum_j g_j p_j), g_i = 0 if not chosen
//   softmax, renorm   dl_j = q_j (g_j - sum g q), 0 elsewhere
//   sigmoid           dl_j = g_j s_j (1 - s_j), 0 elsewhere
//   sigmoid, renorm   dl_j = q_j (1 - s_j) (g_j - sum g q), 0 elsewhere
// A wave has a token; the slots' values meet the row in LDS (experts that a
// token names twice add up; those out of range and masked ones count for nothing).
__global__ void __launch_bounds__(kThreads) k_route_backward(RouteArgs a, int64_t n0) {
    __shared__ float rows[kWaves][kMaxExperts];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = n0 + (int64_t)blockIdx.x * kWaves + wave;
    if (n >= a.N) return;              // (no barrier below: a wave's LDS accesses stay in order)
    float* const row = rows[wave];
    const int64_t at = n * a.ldl;
    const bool dense = !a.sigmoid && !a.renorm;
    float m = 0.0f, sum = 1.0f;
    if (dense) {
        m = neg_inf();
        for (int i = lane; i < a.E; i += 64) m = fmaxf(m, load_float(a.logits, a.dt, at + i));
        m = lanes_max<64>(m);
        if (m == neg_inf()) m = 0.0f;
        sum = 0.0f;
        for (int i = lane; i < a.E; i += 64) sum += expf(load_float(a.logits, a.dt, at + i) - m);
        sum = lanes_sum<64>(sum);
        if (sum == 0.0f) sum = 1.0f;   // a row of -inf
    }
    const int e = lane < a.k ? a.experts[n * a.lde + lane] : -1;
    bool there = e >= 0 && e < a.E;
    const float x = there ? load_float(a.logits, a.dt, at + e) : 0.0f;
    there = there && x != neg_inf();
    const float g = there ? a.scale * a.weights[n * a.ldw + lane] : 0.0f;
    const float q = chosen_weight<64>(a, x, there, m, sum);
    const float mean = lanes_sum<64>(there ? g * q : 0.0f);
    float v = g;
    if (!dense) {
        v = q * (a.renorm ? g - mean : g);
        if (a.sigmoid) v *= 1.0f / (1.0f + expf(x));
    }
    for (int i = lane; i < a.E; i += 64) row[i] = 0.0f;
    __builtin_amdgcn_wave_barrier();
    if (there) atomicAdd(&row[e], v);
    __builtin_amdgcn_wave_barrier();
    for (int i = lane; i < a.E; i += 64) {
        float d = row[i];
        if (dense) d = expf(load_float(a.logits, a.dt, at + i) - m) / sum * (d - mean);
        store_float(a.dlogits, a.dt, n * a.ldd + i, d);
    }
}

// f(first token, workgroups): a launch has fewer than 2^32 threads.
template <typename F>
hipError_t by_tokens(int64_t N, int64_t per, F&& f) {
    const int64_t slab = (((int64_t)1 << 32) / kThreads - 1) * per;
    for (int64_t n = 0; n < N; n += slab) {
        f(n, dim3((unsigned)(((N - n < slab ? N - n : slab) + per - 1) / per)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int L, int V>
hipError_t go(const RouteArgs& a, bool wide, int S, int lg_shift, hipStream_t s) {
    return by_tokens(a.N, kWaves * (64 / L), [&](int64_t n, dim3 grid) {
        if (wide) hipLaunchKernelGGL((k_route<L, V, true>), grid, dim3(kThreads), 0, s, a, n, S, lg_shift);
        else hipLaunchKernelGGL((k_route<L, V, false>), grid, dim3(kThreads), 0, s, a, n, S, lg_shift);
    });
}

int log2_up(int v) {
    int b = 0;
    while ((1 << b) < v) ++b;
    return b;
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
    const bool wide = a.bias || (a.groups > 1 && a.top2);
    const int S = a.E / a.groups, gb = log2_up(a.groups);
    // 16 lanes a token where its experts fit 8 a lane: a choice then serves four tokens.
    // (With 16 a lane one token takes twice the time, 12 us for 6, and 32768 tokens of
    // 256 experts no less: 44 us for 45.)
    const int per16 = gb <= 4 ? (S + (16 >> gb) - 1) / (16 >> gb) : 99;
    if (per16 <= 8 && a.k <= 16) {
        const int sh = 4 - gb;
        if (per16 <= 1) return go<16, 1>(a, wide, S, sh, s);
        if (per16 <= 2) return go<16, 2>(a, wide, S, sh, s);
        if (per16 <= 4) return go<16, 4>(a, wide, S, sh, s);
        return go<16, 8>(a, wide, S, sh, s);
    }
    const int sh = 6 - gb, per = (S + (64 >> gb) - 1) / (64 >> gb);
    if (per <= 1) return go<64, 1>(a, wide, S, sh, s);
    if (per <= 2) return go<64, 2>(a, wide, S, sh, s);
    if (per <= 4) return go<64, 4>(a, wide, S, sh, s);
    if (per <= 8) return go<64, 8>(a, wide, S, sh, s);
    if (per <= 16) return go<64, 16>(a, wide, S, sh, s);
    return go<64, 32>(a, wide, S, sh, s);
}

hipError_t launch_route_backward(const RouteArgs& a, hipStream_t s) {
    return by_tokens(a.N, kWaves, [&](int64_t n, dim3 grid) {
        hipLaunchKernelGGL(k_route_backward, grid, dim3(kThreads), 0, s, a, n);
    });
}

}  // namespace ssg
