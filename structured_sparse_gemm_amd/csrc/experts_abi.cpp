// experts_abi.cpp -- the C ABI of the operators around the expert-grouped
// products: routing, the order of the rows, gather, combine, and gradients.
#include "ssgemm.h"

#include <hip/hip_runtime.h>

#include <cstdint>

#include "experts.hpp"
#include "ssg_abi.hpp"

namespace {

using ssg::abi_failf;

typedef long long ll;

constexpr int64_t kMaxRows = (int64_t)1 << 29, kMaxPairs = 0x7fffffff;

int hip_status(hipError_t e) {
    return e == hipSuccess ? SSG_OK : abi_failf(SSG_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
}

int float_type(int dt) {
    return dt == SSG_F16 ? ssg::FT_F16 : dt == SSG_BF16 ? ssg::FT_BF16 : dt == SSG_F32 ? ssg::FT_F32 : -1;
}

int check_mat(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld) {
    if (rows > 0 && cols > 0 && !p) return abi_failf(SSG_ERR_NULL, "%s is NULL", name);
    if (ld < cols) return abi_failf(SSG_ERR_STRIDE, "row stride of %s: %lld < %lld", name, (ll)ld, (ll)cols);
    return SSG_OK;
}

int check_pairs(int64_t N, int64_t k) {
    if (N < 0 || N >= kMaxRows || k < 0 || k > ssg::kMaxChoices)
        return abi_failf(SSG_ERR_SHAPE, "N=%lld (below 2^29), k=%lld (0 .. %d)", (ll)N, (ll)k, ssg::kMaxChoices);
    if (N * k > kMaxPairs) return abi_failf(SSG_ERR_SHAPE, "N * k = %lld >= 2^31", (ll)(N * k));
    return SSG_OK;
}

int route_args(int dt, int64_t N, int64_t E, const void* logits, int64_t ldl, int score, int64_t k, int64_t groups,
               int64_t top_groups, int group_score, int renorm, float scale, ssg::RouteArgs* out) {
    if (float_type(dt) < 0) return abi_failf(SSG_ERR_DTYPE, "logits of type %d", dt);
    if (score != SSG_SCORE_SOFTMAX && score != SSG_SCORE_SIGMOID) return abi_failf(SSG_ERR_ALGO, "unknown score %d", score);
    if (group_score != SSG_GROUP_MAX && group_score != SSG_GROUP_TOP2)
        return abi_failf(SSG_ERR_ALGO, "unknown group score %d", group_score);
    int rc = check_pairs(N, k);
    if (rc) return rc;
    if (E < 1 || E > ssg::kMaxExperts) return abi_failf(SSG_ERR_SHAPE, "E=%lld (1 .. %d)", (ll)E, ssg::kMaxExperts);
    if (groups < 1 || groups > ssg::kMaxGroups || E % groups)
        return abi_failf(SSG_ERR_SHAPE, "%lld groups (1 .. %d, dividing E=%lld)", (ll)groups, ssg::kMaxGroups, (ll)E);
    if (top_groups < 1 || top_groups > groups)
        return abi_failf(SSG_ERR_SHAPE, "top_groups=%lld of %lld groups", (ll)top_groups, (ll)groups);
    if (k < 1 || k > E / groups * top_groups)
        return abi_failf(SSG_ERR_SHAPE, "k=%lld of %lld experts", (ll)k, (ll)(E / groups * top_groups));
    if ((rc = check_mat("logits", logits, N, E, ldl))) return rc;
    ssg::RouteArgs a{};
    a.dt = float_type(dt);
    a.N = N;
    a.E = (int)E;
    a.k = (int)k;
    a.logits = logits;
    a.ldl = ldl;
    a.groups = (int)groups;
    a.top_groups = (int)top_groups;
    a.sigmoid = score == SSG_SCORE_SIGMOID;
    a.top2 = group_score == SSG_GROUP_TOP2;
    a.renorm = renorm != 0;
    a.scale = scale;
    *out = a;
    return SSG_OK;
}

// What gather, combine and its gradient have in common.
int rows_args(int dt, int64_t N, int64_t k, int64_t D, const int32_t* pos, ssg::RowsArgs* out) {
    if (float_type(dt) < 0) return abi_failf(SSG_ERR_DTYPE, "rows of type %d", dt);
    const int rc = check_pairs(N, k);
    if (rc) return rc;
    if (D < 0 || D >= kMaxRows) return abi_failf(SSG_ERR_SHAPE, "D=%lld (below 2^29)", (ll)D);
    if (N * k > 0 && !pos) return abi_failf(SSG_ERR_NULL, "pos is NULL");
    ssg::RowsArgs a{};
    a.dt = a.out = float_type(dt);
    a.N = N;
    a.P = N * k;
    a.D = D;
    a.k = (int)k;
    a.pos = pos;
    *out = a;
    return SSG_OK;
}

}  // namespace

extern "C" {

int ssg_route(int dt, int64_t N, int64_t E, const void* logits, int64_t ldl, const float* bias, int score, int64_t k,
              int64_t groups, int64_t top_groups, int group_score, int renorm, float scale, float* weights, int64_t ldw,
              int32_t* experts, int64_t lde, void* stream) {
    ssg::RouteArgs a{};
    int rc = route_args(dt, N, E, logits, ldl, score, k, groups, top_groups, group_score, renorm, scale, &a);
    if (rc || (rc = check_mat("weights", weights, N, k, ldw)) || (rc = check_mat("experts", experts, N, k, lde)))
        return rc;
    if (N == 0) return SSG_OK;
    a.bias = bias;
    a.weights = weights;
    a.ldw = ldw;
    a.experts = experts;
    a.lde = lde;
    return hip_status(ssg::launch_route(a, (hipStream_t)stream));
}

int ssg_route_backward(int dt, int64_t N, int64_t E, const float* dweights, int64_t lddw, const void* logits,
                       int64_t ldl, const int32_t* experts, int64_t lde, int score, int64_t k, int renorm, float scale,
                       void* dlogits, int64_t ldd, void* stream) {
    ssg::RouteArgs a{};
    int rc = route_args(dt, N, E, logits, ldl, score, k, 1, 1, SSG_GROUP_MAX, renorm, scale, &a);
    if (rc || (rc = check_mat("dweights", dweights, N, k, lddw)) || (rc = check_mat("experts", experts, N, k, lde)) ||
        (rc = check_mat("dlogits", dlogits, N, E, ldd)))
        return rc;
    if (N == 0) return SSG_OK;
    a.weights = const_cast<float*>(dweights);
    a.ldw = lddw;
    a.experts = const_cast<int32_t*>(experts);
    a.lde = lde;
    a.dlogits = dlogits;
    a.ldd = ldd;
    return hip_status(ssg::launch_route_backward(a, (hipStream_t)stream));
}

size_t ssg_expert_order_workspace_bytes(int64_t N, int64_t k, int64_t E) {
    if (N < 0 || k < 0 || E < 0 || E > ssg::kMaxExperts || check_pairs(N, k)) return 0;
    const int chunks = ssg::expert_order_chunks(N * k);
    return chunks > 1 ? (size_t)chunks * (size_t)E * sizeof(uint32_t) : 0;
}

int ssg_expert_order(int64_t N, int64_t k, int64_t E, const int32_t* experts, int64_t lde, int32_t* offs, int32_t* rows,
                     int32_t* pos, void* ws, size_t ws_bytes, void* stream) {
    int rc = check_pairs(N, k);
    if (rc) return rc;
    if (E < 0 || E > ssg::kMaxExperts) return abi_failf(SSG_ERR_SHAPE, "E=%lld (0 .. %d)", (ll)E, ssg::kMaxExperts);
    if ((rc = check_mat("experts", experts, N, k, lde))) return rc;
    if (!offs) return abi_failf(SSG_ERR_NULL, "offs is NULL");
    if (N * k > 0 && (!rows || !pos)) return abi_failf(SSG_ERR_NULL, "rows or pos is NULL");
    const size_t need = ssg_expert_order_workspace_bytes(N, k, E);
    if (need > 0) {
        if (!ws && ws_bytes == SSG_WS_ASK) return SSG_ERR_WORKSPACE;
        if (!ws || ws_bytes < need)
            return abi_failf(SSG_ERR_WORKSPACE, "workspace %zu < %zu bytes", ws ? ws_bytes : (size_t)0, need);
        if (reinterpret_cast<uintptr_t>(ws) % 4) return abi_failf(SSG_ERR_WORKSPACE, "workspace must be 4-byte aligned");
    }
    return hip_status(ssg::launch_expert_order(N, (int)k, (int)E, experts, lde, offs, rows, pos, (uint32_t*)ws,
                                               (hipStream_t)stream));
}

int ssg_expert_gather(int dt, int64_t N, int64_t k, int64_t D, const void* X, int64_t ldx, const int32_t* pos,
                      const int32_t* rows, void* Y, int64_t ldy, void* stream) {
    ssg::RowsArgs a{};
    int rc = rows_args(dt, N, k, D, pos, &a);
    if (rc || (rc = check_mat("X", X, N, D, ldx)) || (rc = check_mat("Y", Y, N * k, D, ldy))) return rc;
    if (N * k > 0 && !rows) return abi_failf(SSG_ERR_NULL, "rows is NULL");
    if (N * k == 0 || D == 0) return SSG_OK;
    a.rows = rows;
    a.x = X;
    a.ldx = ldx;
    a.o = Y;
    a.ldo = ldy;
    return hip_status(ssg::launch_expert_gather(a, (hipStream_t)stream));
}

int ssg_expert_combine(int dt, int out, int64_t N, int64_t k, int64_t D, const void* Y, int64_t ldy, const int32_t* pos,
                       const float* weights, int64_t ldw, void* O, int64_t ldo, void* stream) {
    ssg::RowsArgs a{};
    int rc = rows_args(dt, N, k, D, pos, &a);
    if (rc) return rc;
    if (out != dt && out != SSG_F32) return abi_failf(SSG_ERR_DTYPE, "unsupported (input, output) types (%d, %d)", dt, out);
    if ((rc = check_mat("Y", Y, N * k, D, ldy)) || (rc = check_mat("O", O, N, D, ldo))) return rc;
    if (weights && ldw < k) return abi_failf(SSG_ERR_STRIDE, "row stride of weights: %lld < %lld", (ll)ldw, (ll)k);
    if (N == 0 || D == 0) return SSG_OK;
    a.out = float_type(out);
    a.y = Y;
    a.ldy = ldy;
    a.w = weights;
    a.ldw = ldw;
    a.o = O;
    a.ldo = ldo;
    return hip_status(ssg::launch_expert_combine(a, (hipStream_t)stream));
}

int ssg_expert_combine_backward(int dt, int64_t N, int64_t k, int64_t D, const void* dO, int64_t lddo, const void* Y,
                                int64_t ldy, const int32_t* pos, const int32_t* rows, const float* weights, int64_t ldw,
                                void* dY, int64_t lddy, float* dweights, int64_t lddw, void* stream) {
    ssg::RowsArgs a{};
    int rc = rows_args(dt, N, k, D, pos, &a);
    if (rc || (rc = check_mat("dO", dO, N, D, lddo)) || (rc = check_mat("Y", Y, N * k, D, ldy)) ||
        (rc = check_mat("weights", weights, N, k, ldw)) || (rc = check_mat("dY", dY, N * k, D, lddy)) ||
        (rc = check_mat("dweights", dweights, N, k, lddw)))
        return rc;
    if (N * k > 0 && !rows) return abi_failf(SSG_ERR_NULL, "rows is NULL");
    if (N * k == 0) return SSG_OK;
    a.rows = rows;
    a.w = weights;
    a.ldw = ldw;
    a.x = dO;
    a.ldx = lddo;
    a.y = Y;
    a.ldy = ldy;
    a.o = dY;
    a.ldo = lddy;
    a.dw = dweights;
    a.lddw = lddw;
    return hip_status(ssg::launch_expert_combine_backward(a, (hipStream_t)stream));
}

}  // extern "C"
