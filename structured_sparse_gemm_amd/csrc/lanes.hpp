// lanes.hpp -- reductions over 16 or all 64 lanes of a wave in registers (lane
// permutations of the vector unit, no LDS).  Every lane ends with the result,
// and with the same bits: the exchanges are symmetric, and each step adds the
// same two numbers in both lanes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace ssg {

// Lane i's value from lane i ^ 1, i ^ 2, 7 - i of 8, 15 - i of 16.
template <int STEP>
__device__ __forceinline__ uint32_t lane_swap16(uint32_t v) {
    constexpr int ctrl = STEP == 0 ? 0xB1 : STEP == 1 ? 0x4E : STEP == 2 ? 0x141 : 0x140;
    return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, ctrl, 0xF, 0xF, false);
}

// r[0] and r[1] hold, in every lane, the values of the two partners (16, 32 lanes apart).
template <bool WIDE>
__device__ __forceinline__ void lane_pair(uint32_t v, uint32_t* a, uint32_t* b) {
    const auto r = WIDE ? __builtin_amdgcn_permlane32_swap(v, v, false, false)
                        : __builtin_amdgcn_permlane16_swap(v, v, false, false);
    *a = r[0];
    *b = r[1];
}

// The value of the lane that step S = 0 .. 5 of a reduction over 2^(S + 1) neighbouring
// lanes pairs this one with (any lane of the other half, once both halves agree).
template <int S, typename T>
__device__ __forceinline__ T lane_partner(T v) {
    union U { T t; uint32_t w[sizeof(T) / 4]; } u;
    u.t = v;
#pragma unroll
    for (uint32_t& w : u.w) {
        if constexpr (S < 4) {
            w = lane_swap16<S>(w);
        } else {
            uint32_t a, b;
            lane_pair<S == 5>(w, &a, &b);
            w ^= a ^ b;
        }
    }
    return u.t;
}
// f(step) for the steps of a reduction over 2^n neighbouring lanes (n the same in all lanes).
template <int MAX, typename F>
__device__ __forceinline__ void lane_steps(int n, F&& f) {
    if (n > 0) f(std::integral_constant<int, 0>{});
    if (n > 1) f(std::integral_constant<int, 1>{});
    if (n > 2) f(std::integral_constant<int, 2>{});
    if (n > 3) f(std::integral_constant<int, 3>{});
    if constexpr (MAX > 4) {
        if (n > 4) f(std::integral_constant<int, 4>{});
        if (n > 5) f(std::integral_constant<int, 5>{});
    }
}

template <typename T> struct LaneBits;
template <> struct LaneBits<uint32_t> {
    static __device__ __forceinline__ uint32_t to(uint32_t v) { return v; }
    static __device__ __forceinline__ uint32_t from(uint32_t v) { return v; }
};
template <> struct LaneBits<float> {
    static __device__ __forceinline__ uint32_t to(float v) { return __float_as_uint(v); }
    static __device__ __forceinline__ float from(uint32_t v) { return __uint_as_float(v); }
};

template <int L, typename T, typename F>
__device__ __forceinline__ T lanes_reduce(T v, F&& f) {
    static_assert(L == 16 || L == 64, "lanes");
    if constexpr (sizeof(T) == 8) {
        union U { T t; uint32_t w[2]; } u, p, q;
        u.t = v;
        auto step = [&](auto sc) {
            constexpr int S = decltype(sc)::value;
            p.w[0] = lane_swap16<S>(u.w[0]);
            p.w[1] = lane_swap16<S>(u.w[1]);
            u.t = f(u.t, p.t);
        };
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
        if constexpr (L == 64) {
            lane_pair<false>(u.w[0], &p.w[0], &q.w[0]);
            lane_pair<false>(u.w[1], &p.w[1], &q.w[1]);
            u.t = f(p.t, q.t);
            lane_pair<true>(u.w[0], &p.w[0], &q.w[0]);
            lane_pair<true>(u.w[1], &p.w[1], &q.w[1]);
            u.t = f(p.t, q.t);
        }
        return u.t;
    } else {
        using B = LaneBits<T>;
        v = f(v, B::from(lane_swap16<0>(B::to(v))));
        v = f(v, B::from(lane_swap16<1>(B::to(v))));
        v = f(v, B::from(lane_swap16<2>(B::to(v))));
        v = f(v, B::from(lane_swap16<3>(B::to(v))));
        if constexpr (L == 64) {
            uint32_t a, b;
            lane_pair<false>(B::to(v), &a, &b);
            v = f(B::from(a), B::from(b));
            lane_pair<true>(B::to(v), &a, &b);
            v = f(B::from(a), B::from(b));
        }
        return v;
    }
}
template <int L, typename T> __device__ __forceinline__ T lanes_sum(T v) {
    return lanes_reduce<L>(v, [](T a, T b) { return a + b; });
}
template <int L, typename T> __device__ __forceinline__ T lanes_max(T v) {
    return lanes_reduce<L>(v, [](T a, T b) { return a > b ? a : b; });
}

}  // namespace ssg
