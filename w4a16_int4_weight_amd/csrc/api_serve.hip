// C ABI of the operators that decode with mixtures of int4 experts and draw tokens
// (include/w4a16_serve.h): argument validation, workspace layout, launches.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/w4a16_serve.h"
#include "api_common.h"
#include "launch.h"
#include "split_k.h"

namespace {

using w4a16::aligned;
using w4a16::check_device;
using w4a16::check_shape;
using w4a16::kMaxK;
using w4a16::packed_size;

constexpr int64_t kMaxRows = int64_t(1) << 31;
constexpr int64_t kRouteRowsPerPass = 16384;        // 8 E bytes a row
constexpr int64_t kPairsPerPass = 16384;            // 4 (F + K) bytes a pair
constexpr int64_t kMaxMoeWidth = int64_t(1) << 15;  // a pass's rows of h are addressed in 32 bits
constexpr int64_t kMaxVocabulary = int64_t(1) << 28;

bool known(w4a16_dtype d) { return d == W4A16_FP16 || d == W4A16_BF16; }
bool known_act(w4a16_act a) { return a == W4A16_ACT_SILU || a == W4A16_ACT_GELU || a == W4A16_ACT_GELU_TANH; }
bool known_score(w4a16_score s) { return s == W4A16_SCORE_SOFTMAX || s == W4A16_SCORE_SIGMOID; }

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

w4a16_status from_hip(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_HIP; }

w4a16_status check_workspace(const void* ws, size_t bytes, size_t need) {
    if (need == 0) return W4A16_OK;
    if (!ws) return W4A16_ERR_NULL;
    if (!aligned(ws, 16)) return W4A16_ERR_ALIGN;
    return bytes < need ? W4A16_ERR_BUFFER_SIZE : W4A16_OK;
}

// ---------------------------------------------------------------- router

w4a16_status check_route(int64_t M, int64_t K, int64_t E, int64_t T) {
    if (M < 0 || M >= kMaxRows || K <= 0 || K % 128 != 0 || K > kMaxK) return W4A16_ERR_SHAPE;
    if (E < 1 || E > w4a16::kMaxExperts || T < 1 || T > E || T > w4a16::kMaxChosen) return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

size_t route_workspace(int64_t M, int64_t E) {
    return w4a16::kSplitCounterBytes + round256(w4a16::route_logits_bytes(M < kRouteRowsPerPass ? M : kRouteRowsPerPass, E));
}

struct Router {
    const void* router;
    const float* bias;
    w4a16_score score;
    int normalize;
    float scale;
};

w4a16_status check_router(const Router& r, const int32_t* ids, const float* weights) {
    if (!r.router || !ids || !weights) return W4A16_ERR_NULL;
    if (!aligned(r.router, 16) || !aligned(r.bias, 4) || !aligned(ids, 4) || !aligned(weights, 4)) return W4A16_ERR_ALIGN;
    return W4A16_OK;
}

hipError_t run_route(const void* x, const Router& r, w4a16_dtype dtype, int64_t M, int64_t K, int64_t E, int64_t T, int32_t* ids,
                     float* weights, uint8_t* ws, hipStream_t s) {
    for (int64_t r0 = 0; r0 < M; r0 += kRouteRowsPerPass) {
        w4a16::RouteCall q{};
        q.x = static_cast<const uint16_t*>(x) + r0 * K;
        q.router = static_cast<const uint16_t*>(r.router);
        q.bias = r.bias;
        q.M = M - r0 < kRouteRowsPerPass ? M - r0 : kRouteRowsPerPass;
        q.K = K;
        q.E = E;
        q.T = T;
        q.sigmoid = r.score == W4A16_SCORE_SIGMOID;
        q.normalize = r.normalize != 0;
        q.scale = r.scale;
        q.ids = ids + r0 * T;
        q.weights = weights + r0 * T;
        q.bf16 = dtype == W4A16_BF16;
        q.counters = reinterpret_cast<uint32_t*>(ws);
        q.logits = ws + w4a16::kSplitCounterBytes;
        const hipError_t err = w4a16::launch_route(q, s);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

// ---------------------------------------------------------------- experts

struct Experts {
    const void* gate_up;
    size_t gate_up_bytes, gate_up_stride;
    const void* down;
    size_t down_bytes, down_stride;
};

w4a16_status check_moe(int64_t M, int64_t K, int64_t F, int64_t E, int64_t T, int64_t group_size, int64_t* G_up, int64_t* G_down) {
    if (M < 0 || M >= kMaxRows || F <= 0 || F % 128 != 0 || F > kMaxMoeWidth || K > kMaxMoeWidth) return W4A16_ERR_SHAPE;
    if (E < 1 || E > w4a16::kMaxExperts || T < 1 || T > w4a16::kMaxChosen) return W4A16_ERR_SHAPE;
    const w4a16_status st = check_shape(K, 2 * F, group_size, G_up);
    return st != W4A16_OK ? st : check_shape(F, K, group_size, G_down);
}

// metadata has one word per min(G, 128) rows, so a group of all rows reads as groups of 128
int64_t unit_group(int64_t group_size) { return group_size == -1 ? w4a16::kRowsPerBlock : group_size; }

int64_t moe_rows(int64_t M, int64_t T) { return M < kPairsPerPass / T ? M : kPairsPerPass / T; }

size_t moe_scratch(int64_t M, int64_t K, int64_t F, int64_t E, int64_t T, int64_t G) {
    return w4a16::moe_small(M, K, T) ? w4a16::moe_small_scratch(M, K, F, E, T) : w4a16::moe_tile_layout(M, K, F, E, T, G).end;
}

size_t moe_workspace(int64_t M, int64_t K, int64_t F, int64_t E, int64_t T, int64_t group_size) {
    const int64_t G = unit_group(group_size);
    const int64_t full = moe_rows(M, T), tail = M % full;
    size_t need = moe_scratch(full, K, F, E, T, G);
    if (tail) {
        const size_t rest = moe_scratch(tail, K, F, E, T, G);
        if (rest > need) need = rest;
    }
    return w4a16::kSplitCounterBytes + need;
}

w4a16_status check_experts(const Experts& e, const void* x, const int32_t* ids, const float* weights, const void* residual,
                           const void* y, int64_t K, int64_t F, int64_t E, int64_t G_up, int64_t G_down) {
    if (!x || !ids || !weights || !e.gate_up || !e.down || !y) return W4A16_ERR_NULL;
    if (!aligned(x, 16) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(e.gate_up, 16) || !aligned(e.down, 16) ||
        !aligned(residual, 16) || !aligned(y, 16) || e.gate_up_stride % 16 != 0 || e.down_stride % 16 != 0)
        return W4A16_ERR_ALIGN;
    const size_t up = packed_size(K, 2 * F, G_up), down = packed_size(F, K, G_down), n = (size_t)(E - 1);
    if (e.gate_up_stride < up || e.down_stride < down || e.gate_up_bytes < up || e.down_bytes < down)
        return W4A16_ERR_BUFFER_SIZE;
    if ((e.gate_up_bytes - up) / e.gate_up_stride < n || (e.down_bytes - down) / e.down_stride < n) return W4A16_ERR_BUFFER_SIZE;
    return W4A16_OK;
}

hipError_t run_moe(const void* x, const int32_t* ids, const float* weights, const Experts& e, w4a16_dtype dtype, const void* residual,
                   void* y, int64_t M, int64_t K, int64_t F, int64_t E, int64_t T, int64_t group_size, w4a16_act act, uint8_t* ws,
                   hipStream_t s) {
    const int64_t rows = moe_rows(M, T);
    for (int64_t r0 = 0; r0 < M; r0 += rows) {
        w4a16::MoeCall q{};
        q.x = static_cast<const uint16_t*>(x) + r0 * K;
        q.ids = ids + r0 * T;
        q.weights = weights + r0 * T;
        q.gate_up = static_cast<const uint8_t*>(e.gate_up);
        q.down = static_cast<const uint8_t*>(e.down);
        q.gate_up_stride = (int64_t)e.gate_up_stride;
        q.down_stride = (int64_t)e.down_stride;
        q.residual = residual ? static_cast<const uint16_t*>(residual) + r0 * K : nullptr;
        q.y = static_cast<uint16_t*>(y) + r0 * K;
        q.M = M - r0 < rows ? M - r0 : rows;
        q.K = K;
        q.F = F;
        q.E = E;
        q.T = T;
        q.G = unit_group(group_size);
        q.act = (int)act;
        q.bf16 = dtype == W4A16_BF16;
        uint8_t* scratch = ws + w4a16::kSplitCounterBytes;
        const hipError_t err = w4a16::moe_small(q.M, K, T) ? w4a16::launch_moe_small(q, reinterpret_cast<uint32_t*>(ws), scratch, s)
                                                        : w4a16::launch_moe_tile(q, scratch, s);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

// The two operators share a workspace: the router's l is done with when the experts begin.
w4a16_status moe_impl(const void* x, const Router* router, int32_t* ids_out, float* weights_out, const int32_t* ids,
                      const float* weights, const Experts& experts, w4a16_dtype dtype, const void* residual, void* y, int64_t M,
                      int64_t K, int64_t F, int64_t E, int64_t T, int64_t group_size, w4a16_act act, void* workspace,
                      size_t workspace_bytes, void* stream) {
    int64_t G_up = 0, G_down = 0;
    w4a16_status st = check_moe(M, K, F, E, T, group_size, &G_up, &G_down);
    if (st != W4A16_OK) return st;
    if (router) {
        st = check_route(M, K, E, T);
        if (st != W4A16_OK) return st;
        if (!known_score(router->score)) return W4A16_ERR_PATH;
        if (!isfinite(router->scale)) return W4A16_ERR_SHAPE;
    }
    if (!known(dtype)) return W4A16_ERR_DTYPE;
    if (!known_act(act)) return W4A16_ERR_PATH;
    if (M == 0) return W4A16_OK;
    if (router) {
        st = check_router(*router, ids_out, weights_out);
        if (st != W4A16_OK) return st;
    }
    st = check_experts(experts, x, ids, weights, residual, y, K, F, E, G_up, G_down);
    if (st != W4A16_OK) return st;
    size_t need = moe_workspace(M, K, F, E, T, group_size);
    if (router && route_workspace(M, E) > need) need = route_workspace(M, E);
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != W4A16_OK) return st;
    st = check_device();
    if (st != W4A16_OK) return st;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (router) {
        const hipError_t err = run_route(x, *router, dtype, M, K, E, T, ids_out, weights_out, ws, s);
        if (err != hipSuccess) return W4A16_ERR_HIP;
    }
    return from_hip(run_moe(x, ids, weights, experts, dtype, residual, y, M, K, F, E, T, group_size, act, ws, s));
}

}  // namespace

extern "C" {

size_t w4a16_route_workspace_bytes(int64_t M, int64_t K, int64_t E, int64_t T) {
    if (M <= 0 || check_route(M, K, E, T) != W4A16_OK) return 0;
    return route_workspace(M, E);
}

w4a16_status w4a16_route(const void* x, const void* router, const float* bias, w4a16_dtype dtype, int64_t M, int64_t K,
                         int64_t E, int64_t T, w4a16_score score, int normalize, float scale, int32_t* ids,
                         float* weights, void* workspace, size_t workspace_bytes, void* stream) {
    w4a16_status st = check_route(M, K, E, T);
    if (st != W4A16_OK) return st;
    if (!known(dtype)) return W4A16_ERR_DTYPE;
    if (!known_score(score)) return W4A16_ERR_PATH;
    if (!isfinite(scale)) return W4A16_ERR_SHAPE;
    if (M == 0) return W4A16_OK;
    if (!x) return W4A16_ERR_NULL;
    if (!aligned(x, 16)) return W4A16_ERR_ALIGN;
    const Router r{router, bias, score, normalize, scale};
    st = check_router(r, ids, weights);
    if (st != W4A16_OK) return st;
    st = check_workspace(workspace, workspace_bytes, route_workspace(M, E));
    if (st != W4A16_OK) return st;
    st = check_device();
    if (st != W4A16_OK) return st;
    return from_hip(run_route(x, r, dtype, M, K, E, T, ids, weights, static_cast<uint8_t*>(workspace),
                              static_cast<hipStream_t>(stream)));
}

size_t w4a16_moe_workspace_bytes(int64_t M, int64_t K, int64_t F, int64_t E, int64_t T, int64_t group_size) {
    int64_t G_up = 0, G_down = 0;
    if (M <= 0 || check_moe(M, K, F, E, T, group_size, &G_up, &G_down) != W4A16_OK) return 0;
    return moe_workspace(M, K, F, E, T, group_size);
}

w4a16_status w4a16_moe(const void* x, const int32_t* ids, const float* weights, const void* gate_up,
                       size_t gate_up_bytes, size_t gate_up_stride, const void* down, size_t down_bytes,
                       size_t down_stride, w4a16_dtype dtype, const void* residual, void* y, int64_t M, int64_t K,
                       int64_t F, int64_t E, int64_t T, int64_t group_size, w4a16_act act, void* workspace,
                       size_t workspace_bytes, void* stream) {
    const Experts e{gate_up, gate_up_bytes, gate_up_stride, down, down_bytes, down_stride};
    return moe_impl(x, nullptr, nullptr, nullptr, ids, weights, e, dtype, residual, y, M, K, F, E, T, group_size, act, workspace,
                    workspace_bytes, stream);
}

size_t w4a16_moe_layer_workspace_bytes(int64_t M, int64_t K, int64_t F, int64_t E, int64_t T, int64_t group_size) {
    const size_t moe = w4a16_moe_workspace_bytes(M, K, F, E, T, group_size), route = w4a16_route_workspace_bytes(M, K, E, T);
    if (moe == 0 || route == 0) return 0;
    return moe > route ? moe : route;
}

w4a16_status w4a16_moe_layer(const void* x, const void* router, const float* bias, w4a16_score score, int normalize,
                             float scale, const void* gate_up, size_t gate_up_bytes, size_t gate_up_stride,
                             const void* down, size_t down_bytes, size_t down_stride, w4a16_dtype dtype,
                             const void* residual, int32_t* ids, float* weights, void* y, int64_t M, int64_t K,
                             int64_t F, int64_t E, int64_t T, int64_t group_size, w4a16_act act, void* workspace,
                             size_t workspace_bytes, void* stream) {
    const Router r{router, bias, score, normalize, scale};
    const Experts e{gate_up, gate_up_bytes, gate_up_stride, down, down_bytes, down_stride};
    return moe_impl(x, &r, ids, weights, ids, weights, e, dtype, residual, y, M, K, F, E, T, group_size, act, workspace,
                    workspace_bytes, stream);
}

size_t w4a16_sample_workspace_bytes(int64_t M, int64_t V) {
    if (M <= 0 || M >= kMaxRows || V < 1 || V > kMaxVocabulary) return 0;
    const size_t need = w4a16::sample_workspace(M, V);
    return need ? w4a16::kSplitCounterBytes + need : 0;
}

w4a16_status w4a16_sample(const void* logits, w4a16_logits type, int64_t row_stride, const float* u, int64_t M, int64_t V,
                          const w4a16_sampling* how, int32_t* ids, float* logprob, void* workspace,
                          size_t workspace_bytes, void* stream) {
    if (M < 0 || M >= kMaxRows || V < 1 || V > kMaxVocabulary || row_stride < V || row_stride > (int64_t(1) << 40))
        return W4A16_ERR_SHAPE;
    if (type != W4A16_LOGITS_FP16 && type != W4A16_LOGITS_BF16 && type != W4A16_LOGITS_FP32) return W4A16_ERR_DTYPE;
    if (!how) return W4A16_ERR_NULL;
    if (M == 0) return W4A16_OK;
    if (!logits || !u || !ids) return W4A16_ERR_NULL;
    if (!aligned(logits, type == W4A16_LOGITS_FP32 ? 4 : 2) || !aligned(u, 4) || !aligned(ids, 4) || !aligned(logprob, 4) ||
        !aligned(how->temperatures, 4) || !aligned(how->top_ks, 4) || !aligned(how->top_ps, 4) || !aligned(how->min_ps, 4))
        return W4A16_ERR_ALIGN;
    w4a16_status st = check_workspace(workspace, workspace_bytes, w4a16_sample_workspace_bytes(M, V));
    if (st != W4A16_OK) return st;
    st = check_device();
    if (st != W4A16_OK) return st;
    w4a16::SampleCall q{};
    q.logits = logits;
    q.kind = (int)type;
    q.ld = row_stride;
    q.M = M;
    q.V = V;
    q.u = u;
    q.temperature = how->temperature;
    q.top_p = how->top_p;
    q.min_p = how->min_p;
    q.top_k = how->top_k;
    q.temperatures = how->temperatures;
    q.top_ks = how->top_ks;
    q.top_ps = how->top_ps;
    q.min_ps = how->min_ps;
    q.ids = ids;
    q.logprob = logprob;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    return from_hip(w4a16::launch_sample(q, ws ? ws + w4a16::kSplitCounterBytes : nullptr, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
