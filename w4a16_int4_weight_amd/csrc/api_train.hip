// C ABI of the operators that train through packed int4 weights and score with them
// (include/w4a16_train.h): argument validation, workspace layout, launches.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/w4a16_train.h"
#include "api_common.h"
#include "launch.h"
#include "split_k.h"

namespace {

using w4a16::aligned;
using w4a16::check_device;
using w4a16::check_shape;
using w4a16::kMaxMK;
using w4a16::packed_size;

constexpr int64_t kMaxRowElements = int64_t(1) << 22;     // a 256-row tile is addressed in 32 bits
constexpr int64_t kGatedRowsPerPass = 8192;            // of a backward: 4 F bytes a row

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

bool known(w4a16_dtype d) { return d == W4A16_FP16 || d == W4A16_BF16; }

// Row counts and sizes common to every entry: M rows of K and of `cols` elements
w4a16_status check_rows(int64_t M, int64_t K, int64_t cols) {
    if (M < 0 || M >= (int64_t(1) << 31) || M * K > kMaxMK || M * cols > kMaxMK) return W4A16_ERR_SHAPE;
    return W4A16_OK;
}

w4a16_status check_workspace(const void* ws, size_t bytes, size_t need) {
    if (need == 0) return W4A16_OK;
    if (!ws) return W4A16_ERR_NULL;
    if (!aligned(ws, 16)) return W4A16_ERR_ALIGN;
    return bytes < need ? W4A16_ERR_BUFFER_SIZE : W4A16_OK;
}

w4a16_status from_hip(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_ERR_HIP; }

// ---------------------------------------------------------------- dx = dy W^T

w4a16_status check_gemm_grad(int64_t M, int64_t K, int64_t N, int64_t group_size, int64_t* G) {
    const w4a16_status st = check_shape(K, N, group_size, G);
    if (st != W4A16_OK) return st;
    if (N > kMaxRowElements) return W4A16_ERR_SHAPE;
    return check_rows(M, K, N);
}

size_t gemm_grad_workspace(int64_t M, int64_t K, int64_t N) {
    const size_t part = w4a16::plan_grad(M, K, N, false).part_bytes;
    return part ? w4a16::kSplitCounterBytes + part : 0;
}

// ---------------------------------------------------------------- gated block

w4a16_status check_gated(int64_t M, int64_t K, int64_t F, int64_t group_size, int64_t* G) {
    if (F <= 0 || F % 8 != 0 || F > kMaxRowElements / 2) return W4A16_ERR_SHAPE;
    const w4a16_status st = check_shape(K, 2 * F, group_size, G);
    if (st != W4A16_OK) return st;
    return check_rows(M, K, F);
}

struct GatedLayout {
    size_t partials, tops, rowmax, factor, scale_max, d, d_rest, d32, gpart, end;
};

// one pass over M rows: the forward's K-split partials and, for the gradient, dg | du and
// the transposed product's partials
GatedLayout gated_layout(int64_t M, int64_t K, int64_t F, int64_t G, bool grad, bool bf16) {
    GatedLayout l{};
    const size_t partial = w4a16::plan_product(M, K, 2 * F, G, true).partial_bytes;
    l.partials = w4a16::kSplitCounterBytes;
    size_t at = l.partials + round256(partial);
    if (grad) {
        l.tops = at;
        at += round256((size_t)w4a16::gated_tiles(M, K, F, G) * M * 4);
        l.rowmax = at;
        at += round256((size_t)M * 4);
        l.factor = at;
        at += round256((size_t)w4a16::gated_tiles(M, K, F, G) * M * 4);
        l.scale_max = at;
        at += round256(w4a16::kScaleParts * 4);
        l.d = at;
        at += round256((size_t)M * 4 * F);
        l.d_rest = at;
        if (w4a16::grad_takes_rest(w4a16::plan_grad(M, K, 2 * F, false), bf16)) at += round256((size_t)M * 4 * F);
        l.d32 = at;
        if (w4a16::small_product(M, K)) at += round256((size_t)M * 8 * F);
        l.gpart = at;
        at += round256(w4a16::plan_grad(M, K, 2 * F, false).part_bytes);
    } else if (partial == 0) {
        at = 0;
    }
    l.end = at;
    return l;
}

// (of both types: fp16's, which may keep d_rest)
size_t gated_workspace(int64_t M, int64_t K, int64_t F, int64_t G, bool grad) {
    if (!grad) return gated_layout(M, K, F, G, false, false).end;
    const int64_t full = M < kGatedRowsPerPass ? M : kGatedRowsPerPass;
    size_t need = gated_layout(full, K, F, G, true, false).end;
    if (M > full && M % full) {
        const size_t tail = gated_layout(M % full, K, F, G, true, false).end;
        if (tail > need) need = tail;
    }
    return need;
}

bool known_act(w4a16_act a) { return a == W4A16_ACT_SILU || a == W4A16_ACT_GELU || a == W4A16_ACT_GELU_TANH; }

// ---------------------------------------------------------------- losses

w4a16_status check_loss(int64_t M, int64_t K, int64_t V, int64_t group_size, int64_t T, int64_t* G) {
    const w4a16_status st = check_shape(K, V, group_size, G);
    if (st != W4A16_OK) return st;
    if (T < 1 || T > w4a16::max_loss_targets()) return W4A16_ERR_SHAPE;
    return check_rows(M, K, T);
}

w4a16_status loss_impl(const void* x, const int32_t* ids, const float* top, bool distill, const void* packed,
                       size_t packed_bytes, w4a16_dtype dtype, int64_t M, int64_t K, int64_t V, int64_t group_size,
                       int64_t T, float tau, const float* dloss, float* loss, float* lse, void* dx, void* workspace,
                       size_t workspace_bytes, void* stream) {
    int64_t G = 0;
    w4a16_status st = check_loss(M, K, V, group_size, T, &G);
    if (st != W4A16_OK) return st;
    if (!(tau > 0.f) || isinf(tau)) return W4A16_ERR_SHAPE;
    if (!known(dtype)) return W4A16_ERR_DTYPE;
    if (M == 0) return W4A16_OK;
    if (!x || !ids || !packed || !loss || !lse || (distill && !top)) return W4A16_ERR_NULL;
    if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(ids, 4) || !aligned(top, 4) || !aligned(dloss, 4) ||
        !aligned(loss, 4) || !aligned(lse, 4) || !aligned(dx, 16))
        return W4A16_ERR_ALIGN;
    if (packed_bytes < packed_size(K, V, G)) return W4A16_ERR_BUFFER_SIZE;
    st = check_workspace(workspace, workspace_bytes, w4a16::loss_workspace(M, K, V, G, T, distill, dx != nullptr));
    if (st != W4A16_OK) return st;
    st = check_device();
    if (st != W4A16_OK) return st;
    w4a16::LossCall q{};
    q.x = static_cast<const uint16_t*>(x);
    q.ids = ids;
    q.top = distill ? top : nullptr;
    q.packed = static_cast<const uint8_t*>(packed);
    q.dloss = dloss;
    q.loss = loss;
    q.lse = lse;
    q.dx = static_cast<uint16_t*>(dx);
    q.M = M;
    q.K = K;
    q.V = V;
    q.G = G;
    q.T = T;
    q.tau = tau;
    q.bf16 = dtype == W4A16_BF16;
    q.workspace = workspace;
    return from_hip(w4a16::launch_loss(q, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t w4a16_gemm_grad_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t group_size) {
    int64_t G = 0;
    if (M <= 0 || check_gemm_grad(M, K, N, group_size, &G) != W4A16_OK) return 0;
    return gemm_grad_workspace(M, K, N);
}

w4a16_status w4a16_gemm_grad(const void* dy, const void* packed, size_t packed_bytes, w4a16_dtype dtype, void* dx,
                             int64_t M, int64_t K, int64_t N, int64_t group_size, void* workspace,
                             size_t workspace_bytes, void* stream) {
    int64_t G = 0;
    w4a16_status st = check_gemm_grad(M, K, N, group_size, &G);
    if (st != W4A16_OK) return st;
    if (!known(dtype)) return W4A16_ERR_DTYPE;
    if (M == 0) return W4A16_OK;
    if (!dy || !packed || !dx) return W4A16_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(packed, 16) || !aligned(dx, 16)) return W4A16_ERR_ALIGN;
    if (packed_bytes < packed_size(K, N, G)) return W4A16_ERR_BUFFER_SIZE;
    st = check_workspace(workspace, workspace_bytes, gemm_grad_workspace(M, K, N));
    if (st != W4A16_OK) return st;
    st = check_device();
    if (st != W4A16_OK) return st;
    const bool bf16 = dtype == W4A16_BF16;
    const w4a16::GradPlan plan = w4a16::plan_grad(M, K, N, false);
    float* part = plan.part_bytes
                      ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w4a16::kSplitCounterBytes) : nullptr;
    w4a16::GradCall q{};
    q.d = static_cast<const uint16_t*>(dy);
    q.ld = N;
    q.packed = static_cast<const uint8_t*>(packed);
    q.dx = part ? nullptr : static_cast<uint16_t*>(dx);
    q.part = part;
    q.M = M;
    q.K = K;
    q.N = N;
    q.G = G;
    q.n0 = 0;
    q.n = N;
    q.bf16 = bf16;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t err = w4a16::launch_grad(plan, q, s);
    if (err == hipSuccess && part)
        err = w4a16::launch_grad_finish(part, plan.splits, M, K, static_cast<uint16_t*>(dx), bf16, nullptr, nullptr, s);
    return from_hip(err);
}

size_t w4a16_gated_workspace_bytes(int64_t M, int64_t K, int64_t F, int64_t group_size, int grad) {
    int64_t G = 0;
    if (M <= 0 || check_gated(M, K, F, group_size, &G) != W4A16_OK) return 0;
    return gated_workspace(M, K, F, G, grad != 0);
}

w4a16_status w4a16_gated(const void* x, const void* packed, size_t packed_bytes, w4a16_dtype dtype, void* h, int64_t M,
                         int64_t K, int64_t F, int64_t group_size, w4a16_act act, void* workspace,
                         size_t workspace_bytes, void* stream) {
    int64_t G = 0;
    w4a16_status st = check_gated(M, K, F, group_size, &G);
    if (st != W4A16_OK) return st;
    if (!known(dtype)) return W4A16_ERR_DTYPE;
    if (!known_act(act)) return W4A16_ERR_PATH;
    if (M == 0) return W4A16_OK;
    if (!x || !packed || !h) return W4A16_ERR_NULL;
    if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(h, 16)) return W4A16_ERR_ALIGN;
    if (packed_bytes < packed_size(K, 2 * F, G)) return W4A16_ERR_BUFFER_SIZE;
    st = check_workspace(workspace, workspace_bytes, gated_workspace(M, K, F, G, false));
    if (st != W4A16_OK) return st;
    st = check_device();
    if (st != W4A16_OK) return st;
    const GatedLayout l = gated_layout(M, K, F, G, false, dtype == W4A16_BF16);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    w4a16::GatedCall q{};
    q.x = static_cast<const uint16_t*>(x);
    q.packed = static_cast<const uint8_t*>(packed);
    q.h = static_cast<uint16_t*>(h);
    q.M = M;
    q.K = K;
    q.F = F;
    q.G = G;
    q.act = (int)act;
    q.bf16 = dtype == W4A16_BF16;
    q.counters = reinterpret_cast<uint32_t*>(ws);
    q.partials = ws ? reinterpret_cast<float*>(ws + l.partials) : nullptr;
    return from_hip(w4a16::launch_gated(q, static_cast<hipStream_t>(stream)));
}

w4a16_status w4a16_gated_grad(const void* x, const void* dh, const void* packed, size_t packed_bytes, w4a16_dtype dtype,
                              void* dx, int64_t M, int64_t K, int64_t F, int64_t group_size, w4a16_act act,
                              void* workspace, size_t workspace_bytes, void* stream) {
    int64_t G = 0;
    w4a16_status st = check_gated(M, K, F, group_size, &G);
    if (st != W4A16_OK) return st;
    if (!known(dtype)) return W4A16_ERR_DTYPE;
    if (!known_act(act)) return W4A16_ERR_PATH;
    if (M == 0) return W4A16_OK;
    if (!x || !dh || !packed || !dx) return W4A16_ERR_NULL;
    if (!aligned(x, 16) || !aligned(dh, 16) || !aligned(packed, 16) || !aligned(dx, 16)) return W4A16_ERR_ALIGN;
    if (packed_bytes < packed_size(K, 2 * F, G)) return W4A16_ERR_BUFFER_SIZE;
    st = check_workspace(workspace, workspace_bytes, gated_workspace(M, K, F, G, true));
    if (st != W4A16_OK) return st;
    st = check_device();
    if (st != W4A16_OK) return st;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const bool bf16 = dtype == W4A16_BF16;
    hipStream_t s = static_cast<hipStream_t>(stream);
    for (int64_t r0 = 0; r0 < M; r0 += kGatedRowsPerPass) {
        const int64_t rows = M - r0 < kGatedRowsPerPass ? M - r0 : kGatedRowsPerPass;
        const GatedLayout l = gated_layout(rows, K, F, G, true, bf16);
        w4a16::GatedCall q{};
        q.x = static_cast<const uint16_t*>(x) + r0 * K;
        q.dh = static_cast<const uint16_t*>(dh) + r0 * F;
        q.packed = static_cast<const uint8_t*>(packed);
        q.d = reinterpret_cast<uint16_t*>(ws + l.d);
        const w4a16::GradPlan plan = w4a16::plan_grad(rows, K, 2 * F, false);
        if (w4a16::grad_takes_rest(plan, bf16)) q.d_rest = reinterpret_cast<uint16_t*>(ws + l.d_rest);
        q.d32 = reinterpret_cast<float*>(ws + l.d32);
        q.tops = reinterpret_cast<float*>(ws + l.tops);
        float* rowmax = reinterpret_cast<float*>(ws + l.rowmax);
        float* scale_max = reinterpret_cast<float*>(ws + l.scale_max);
        q.M = rows;
        q.K = K;
        q.F = F;
        q.G = G;
        q.act = (int)act;
        q.bf16 = bf16;
        q.counters = reinterpret_cast<uint32_t*>(ws);
        q.partials = reinterpret_cast<float*>(ws + l.partials);
        hipError_t err = w4a16::launch_gated(q, s);
        if (err == hipSuccess)
            err = w4a16::launch_gated_tops(q, rowmax, reinterpret_cast<uint32_t*>(ws + l.factor), scale_max, s);
        if (err != hipSuccess) return W4A16_ERR_HIP;
        float* part = plan.part_bytes ? reinterpret_cast<float*>(ws + l.gpart) : nullptr;
        uint16_t* out = static_cast<uint16_t*>(dx) + r0 * K;
        w4a16::GradCall g{};
        g.d = q.d;
        g.scaled = true;
        g.d_rest = q.d_rest;
        g.rowmax = rowmax;
        g.tile_columns = w4a16::gated_tile_columns(rows, K);
        g.tile_factor = g.tile_columns ? reinterpret_cast<uint32_t*>(ws + l.factor) : nullptr;
        g.scale_max = scale_max;
        g.ld = 2 * F;
        g.packed = q.packed;
        g.dx = part ? nullptr : out;
        g.part = part;
        g.M = rows;
        g.K = K;
        g.N = 2 * F;
        g.G = G;
        g.n = 2 * F;
        g.bf16 = bf16;
        err = w4a16::launch_grad(plan, g, s);
        if (err == hipSuccess && part) err = w4a16::launch_grad_finish(part, plan.splits, rows, K, out, bf16, rowmax, scale_max, s);
        if (err != hipSuccess) return W4A16_ERR_HIP;
    }
    return W4A16_OK;
}

size_t w4a16_cross_entropy_workspace_bytes(int64_t M, int64_t K, int64_t V, int64_t group_size, int grad) {
    int64_t G = 0;
    if (M <= 0 || check_loss(M, K, V, group_size, 1, &G) != W4A16_OK) return 0;
    return w4a16::loss_workspace(M, K, V, G, 1, false, grad != 0);
}

w4a16_status w4a16_cross_entropy(const void* x, const int32_t* labels, const void* packed, size_t packed_bytes,
                                 w4a16_dtype dtype, int64_t M, int64_t K, int64_t V, int64_t group_size,
                                 const float* dloss, float* loss, float* lse, void* dx, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    return loss_impl(x, labels, nullptr, false, packed, packed_bytes, dtype, M, K, V, group_size, 1, 1.f, dloss, loss, lse,
                     dx, workspace, workspace_bytes, stream);
}

size_t w4a16_distill_workspace_bytes(int64_t M, int64_t K, int64_t V, int64_t group_size, int64_t T, int grad) {
    int64_t G = 0;
    if (M <= 0 || check_loss(M, K, V, group_size, T, &G) != W4A16_OK) return 0;
    return w4a16::loss_workspace(M, K, V, G, T, true, grad != 0);
}

w4a16_status w4a16_distill(const void* x, const int32_t* top_ids, const float* top_logits, const void* packed,
                           size_t packed_bytes, w4a16_dtype dtype, int64_t M, int64_t K, int64_t V, int64_t group_size,
                           int64_t T, float temperature, const float* dloss, float* loss, float* lse, void* dx,
                           void* workspace, size_t workspace_bytes, void* stream) {
    return loss_impl(x, top_ids, top_logits, true, packed, packed_bytes, dtype, M, K, V, group_size, T, temperature, dloss,
                     loss, lse, dx, workspace, workspace_bytes, stream);
}

}  // extern "C"
