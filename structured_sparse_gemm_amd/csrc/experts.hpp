// experts.hpp -- arguments and launchers of the operators around the
// expert-grouped products (route.hip, expert_rows.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssg {

constexpr int kMaxExperts = 1024, kMaxChoices = 64, kMaxGroups = 64;

enum FloatType { FT_F16 = 0, FT_BF16 = 1, FT_F32 = 2 };
constexpr int ft_bytes(int t) { return t == FT_F32 ? 4 : 2; }

struct RouteArgs {
    int dt;                            // FloatType of the logits and their gradient
    int64_t N;
    int E, k;
    const void* logits;
    int64_t ldl;                       // strides in elements
    const float* bias;                 // [E] or nullptr
    int groups, top_groups;
    bool sigmoid, top2, renorm;        // else softmax; group score max; scores as they are
    float scale;
    float* weights;
    int64_t ldw;
    int32_t* experts;
    int64_t lde;
    // gradient: weights and experts are read
    void* dlogits;
    int64_t ldd;
};
hipError_t launch_route(const RouteArgs& a, hipStream_t s);
hipError_t launch_route_backward(const RouteArgs& a, hipStream_t s);

// Chunks of pairs that the order is built from; their counts are the workspace.
int expert_order_chunks(int64_t pairs);
hipError_t launch_expert_order(int64_t N, int k, int E, const int32_t* experts, int64_t lde, int32_t* offs,
                               int32_t* rows, int32_t* pos, uint32_t* counts, hipStream_t s);

struct RowsArgs {
    int dt, out;                       // FloatType of the matrices; of the combined rows
    int64_t N, P, D;                   // tokens, expert rows, columns
    int k;
    const int32_t *pos, *rows;         // [N, k]; [P]
    const float* w;                    // [N, k] or nullptr
    int64_t ldw;
    const void* x;                     // token rows: X, dO
    int64_t ldx;                       // strides in elements
    const void* y;                     // expert rows: Y
    int64_t ldy;
    void* o;                           // output rows
    int64_t ldo;
    float* dw;
    int64_t lddw;
};
hipError_t launch_expert_gather(const RowsArgs& a, hipStream_t s);
hipError_t launch_expert_combine(const RowsArgs& a, hipStream_t s);
hipError_t launch_expert_combine_backward(const RowsArgs& a, hipStream_t s);

}  // namespace ssg
