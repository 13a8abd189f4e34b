/*
 * w4a16_train.h - C ABI of the operators that train through frozen int4 weights, and
 * score with them, on the packed buffers of w4a16.h (same library, same conventions:
 * caller-owned device pointers, asynchronous on `stream`, every argument checked on the
 * host before anything is launched, status codes, nothing thrown or allocated).
 *
 *   W[k, n] = (q[k, n] - z[g, n]) * s[g, n], g = k div G, as in w4a16.h. The weights are
 *   frozen: gradients go to the activations (adapters, norms and embeddings train).
 *
 * Sums, softmax statistics and losses are held in fp32; 16-bit results are rounded once,
 * to nearest even. Every result is bit-for-bit reproducible for fixed inputs and shape.
 * M = 0 is a valid no-op. Group sizes as w4a16_gemm: -1, 32, 64, multiples of 128.
 *
 * Workspaces follow the contract of w4a16_workspace_bytes: zero-filled before first use,
 * the first 512 bytes zero again after every call, so one allocation as large as the
 * largest need serves calls of every entry point, w4a16_gemm's included, in order on one
 * stream; calls that overlap in time need workspaces of their own. 16-byte alignment.
 * The *_workspace_bytes functions return 0 for an unsupported shape or where none is
 * needed.
 */
#ifndef W4A16_TRAIN_H
#define W4A16_TRAIN_H

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* dx = dy . W^T, the gradient of y = x . W (w4a16_gemm) with respect to x:
 *   dx[m, k] = sum_n dy[m, n] * W[k, n]
 *   dy  [M, N] row-major, `dtype`, 16-byte aligned; read only.
 *   dx  [M, K] row-major, `dtype`, written in full, 16-byte aligned; must not overlap dy.
 * W's values enter the product rounded once to `dtype`. N <= 2^22, M * N <= 2^32. */
size_t w4a16_gemm_grad_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t group_size);
w4a16_status w4a16_gemm_grad(const void* dy, const void* packed, size_t packed_bytes, w4a16_dtype dtype, void* dx,
                             int64_t M, int64_t K, int64_t N, int64_t group_size, void* workspace,
                             size_t workspace_bytes, void* stream);

typedef enum {
    W4A16_ACT_SILU = 0,         /* g / (1 + e^-g)                                   */
    W4A16_ACT_GELU = 1,         /* g Phi(g), Phi the normal distribution function   */
    W4A16_ACT_GELU_TANH = 2,    /* g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2  */
    W4A16_ACT_RANGE_MIN_ = -0x7FFFFFFF - 1,
    W4A16_ACT_RANGE_MAX_ = 0x7FFFFFFF
} w4a16_act;

/* Gated feed-forward block on one packed weight of K rows and 2F columns: columns
 * 0 .. F-1 are the gate projection's, F .. 2F-1 the up projection's.
 *   h = a(x Wg) * (x Wu)                      x [M, K], h [M, F]
 * g, u and the activation stay in fp32; h is rounded once. F % 8 == 0, F <= 2^21.
 * An unknown activation gives W4A16_ERR_PATH. x, h 16-byte aligned, not overlapping.
 *
 * w4a16_gated_grad is its backward to x: it forms both projections again from x and
 * returns dx = dg Wg^T + du Wu^T, dg = dh u a'(g), du = dh a(g). dg and du are rounded once
 * to fp16 at a power of two of their row's largest value, and so are the weights at one of
 * the largest scale (a scale less than 2^-21 of it loses bits, one below 2^-31 is taken as
 * 0). With fp16 tensors what dg's and du's rounding leaves is kept in a second fp16 value
 * where the product's tiles have up to 128 rows, in practice up to several hundred rows: the
 * error against exact arithmetic, in the norm, is 2.9e-4 there and 3.5e-4 above (2.1e-4: the
 * result's own rounding; bf16: 1.7e-3, all of it the result's). dh [M, F]. 8192 rows at a
 * time. */
size_t w4a16_gated_workspace_bytes(int64_t M, int64_t K, int64_t F, int64_t group_size, int grad);
w4a16_status w4a16_gated(const void* x, const void* packed, size_t packed_bytes, w4a16_dtype dtype, void* h, int64_t M,
                         int64_t K, int64_t F, int64_t group_size, w4a16_act act, void* workspace,
                         size_t workspace_bytes, void* stream);
w4a16_status w4a16_gated_grad(const void* x, const void* dh, const void* packed, size_t packed_bytes, w4a16_dtype dtype,
                              void* dx, int64_t M, int64_t K, int64_t F, int64_t group_size, w4a16_act act,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Softmax cross entropy over a packed head W [K, V] without the logits:
 *   loss[m] = lse[m] - z[m, labels[m]],  z = x W,  lse[m] = log sum_v e^{z[m, v]}
 *   dx[m]   = dloss[m] * sum_v (e^{z[m, v] - lse[m]} - [v = labels[m]]) W_v
 *   labels  int32 [M]; a label outside [0, V) gives loss 0 and dx 0 (lse is still given).
 *   dloss   fp32 [M] or NULL (1). Read only when dx is given.
 *   loss, lse  fp32 [M], written in full.
 *   dx      [M, K] `dtype`, written in full, or NULL: no gradient. 16-byte aligned.
 * The vocabulary is taken in pieces: the largest buffer holds the unnormalised
 * probabilities of one piece (`dtype`, at most 256 MiB, 4096 rows at a time). The target
 * columns' part of dx is taken in fp32. A row's label is left out of its sum, so that the
 * loss, log(1 + sum_{v != label} e^{z_v - z_label}), is never negative, and small losses and
 * gradients are right relative to themselves. No pointer may overlap another that is
 * written. */
size_t w4a16_cross_entropy_workspace_bytes(int64_t M, int64_t K, int64_t V, int64_t group_size, int grad);
w4a16_status w4a16_cross_entropy(const void* x, const int32_t* labels, const void* packed, size_t packed_bytes,
                                 w4a16_dtype dtype, int64_t M, int64_t K, int64_t V, int64_t group_size,
                                 const float* dloss, float* loss, float* lse, void* dx, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* Distillation from a teacher's top logits, over the same head:
 *   p[m, :] = softmax of top_logits[m, :] / t over the entries whose id is in [0, V)
 *   loss[m] = t^2 sum_j p_j (log p_j - log q[m, id_j]),  q = softmax(x W / t)
 *   dx[m]   = dloss[m] * t * sum_v (q_v - sum_{j: id_j = v} p_j) W_v
 * lse is that of x W / t. T = 1 .. 256 entries a row, ids in any order; an id outside
 * [0, V) is none (lists of different lengths are padded with -1), an id given twice
 * counts with both weights, a logit of -infinity weighs nothing. A row with nothing left
 * has loss 0 and dx 0. temperature t > 0, finite. top_ids int32, top_logits fp32 [M, T].
 * The remaining arguments are those of w4a16_cross_entropy. */
size_t w4a16_distill_workspace_bytes(int64_t M, int64_t K, int64_t V, int64_t group_size, int64_t T, int grad);
w4a16_status w4a16_distill(const void* x, const int32_t* top_ids, const float* top_logits, const void* packed,
                           size_t packed_bytes, w4a16_dtype dtype, int64_t M, int64_t K, int64_t V, int64_t group_size,
                           int64_t T, float temperature, const float* dloss, float* loss, float* lse, void* dx,
                           void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_TRAIN_H */
