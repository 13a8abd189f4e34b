/*
 * w4a16_serve.h - C ABI of the operators that decode with mixtures of int4 experts and draw
 * the next token, beside those of w4a16.h (same library, same conventions: caller-owned
 * device pointers, asynchronous on `stream`, every argument checked on the host before
 * anything is launched, status codes, nothing thrown or allocated).
 *
 * Sums and softmax statistics are held in fp32 or fp64; results are rounded once, to nearest
 * even. Every result is bit-for-bit reproducible for fixed inputs and shape. M = 0 is a
 * valid no-op. No pointer may overlap another that is written, unless said so.
 *
 * Workspaces follow the contract of w4a16_workspace_bytes: zero-filled before first use, the
 * first 512 bytes zero again after every call, so one allocation as large as the largest need
 * serves calls of every entry point in order on one stream; calls that overlap in time need
 * workspaces of their own. 16-byte alignment. The *_workspace_bytes functions return 0 for an
 * unsupported shape or where none is needed.
 */
#ifndef W4A16_SERVE_H
#define W4A16_SERVE_H

#include "w4a16.h"
#include "w4a16_train.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    W4A16_SCORE_SOFTMAX = 0,    /* s = softmax over the experts                     */
    W4A16_SCORE_SIGMOID = 1,    /* s = 1 / (1 + e^-l), each expert by itself        */
    W4A16_SCORE_RANGE_MIN_ = -0x7FFFFFFF - 1,
    W4A16_SCORE_RANGE_MAX_ = 0x7FFFFFFF
} w4a16_score;

/* The router of a mixture of E experts: T of them for each row.
 *   l[m, e] = sum_k x[m, k] * router[e, k],  s = score(l)
 *   ids[m, :]      the T experts of the largest l (of the largest s + bias[e] where a bias is
 *                  given), the largest first, ties to the lowest expert; what is no number
 *                  there comes last
 *   weights[m, j]  s of expert ids[m, j] (without the bias); with `normalize` over the sum of
 *                  the row's T (0 where that sum is 0); times `scale`
 *   x [M, K], router [E, K] row-major, `dtype`, 16-byte aligned. bias fp32 [E] or NULL.
 *   ids int32, weights fp32 [M, T], written in full.
 * K % 128 == 0, K <= 2^20, 1 <= T <= min(E, 32), E <= 1024. l is summed in fp64, so that the
 * choice is that of exact arithmetic up to rounding in the 53rd bit. A row in which some s is
 * no number (that expert's l is none, or +infinity or all -infinity under softmax), chosen or
 * not, still gets T different experts, with weights that are all no numbers. An unknown
 * score gives W4A16_ERR_PATH; scale must be finite. */
size_t w4a16_route_workspace_bytes(int64_t M, int64_t K, int64_t E, int64_t T);
w4a16_status w4a16_route(const void* x, const void* router, const float* bias, w4a16_dtype dtype, int64_t M, int64_t K,
                         int64_t E, int64_t T, w4a16_score score, int normalize, float scale, int32_t* ids,
                         float* weights, void* workspace, size_t workspace_bytes, void* stream);

/* The experts' gated feed-forward blocks, weighed and summed, on packed int4 weights:
 *   y[m] = residual[m] + sum_j weights[m, j] * (a(x[m] Wg) * (x[m] Wu)) Wd
 * Wg | Wu and Wd those of expert ids[m, j]. An id outside [0, E) is none (entries dropped, rows
 * of padding); an id given twice in a row counts with both weights.
 *   gate_up  E packed buffers of K rows and 2F columns (gate, then up, as w4a16_gated has
 *            them), expert e's at gate_up + e * gate_up_stride bytes
 *   down     E packed buffers of F rows and K columns, at down + e * down_stride
 *            both strides multiples of 16 and at least w4a16_packed_bytes of one expert
 *   gate_up_bytes, down_bytes  at least (E - 1) * stride + one expert
 *   group_size the same for both; it must suit K and F.
 *   ids int32, weights fp32 [M, T], 1 <= T <= 32
 *   residual [M, K] `dtype` or NULL (0); may be y itself
 *   y        [M, K] `dtype`, written in full, 16-byte aligned
 * F % 128 == 0 (a row block of the down projection), K and F <= 2^15, E <= 1024. g, u and the activation stay in fp32, h between
 * the projections in two bf16 values (16 bits), the sum over experts in fp32. Only the
 * experts that some row names are read. A row of x that is not finite gives a row of y that is
 * not (where it names an expert), and touches no other. Made for few rows: up to 16, with M T <= 256 and K <= 4096, take two
 * launches, more take four and are met 16384 / T rows at a time. The workspace holds 4 (F + K) bytes for
 * each of at most 16384 entries of ids (1.2 GB where K = 4096 and F = 14336 and the rows fill a pass, 4.3 GB
 * at the widest), or, where two launches serve, 4 M F for each expert that may be named (at most
 * min(E, M T)). */
size_t w4a16_moe_workspace_bytes(int64_t M, int64_t K, int64_t F, int64_t E, int64_t T, int64_t group_size);
w4a16_status w4a16_moe(const void* x, const int32_t* ids, const float* weights, const void* gate_up,
                       size_t gate_up_bytes, size_t gate_up_stride, const void* down, size_t down_bytes,
                       size_t down_stride, w4a16_dtype dtype, const void* residual, void* y, int64_t M, int64_t K,
                       int64_t F, int64_t E, int64_t T, int64_t group_size, w4a16_act act, void* workspace,
                       size_t workspace_bytes, void* stream);

/* w4a16_route and w4a16_moe in one call; ids and weights are written as by w4a16_route. */
size_t w4a16_moe_layer_workspace_bytes(int64_t M, int64_t K, int64_t F, int64_t E, int64_t T, int64_t group_size);
w4a16_status w4a16_moe_layer(const void* x, const void* router, const float* bias, w4a16_score score, int normalize,
                             float scale, const void* gate_up, size_t gate_up_bytes, size_t gate_up_stride,
                             const void* down, size_t down_bytes, size_t down_stride, w4a16_dtype dtype,
                             const void* residual, int32_t* ids, float* weights, void* y, int64_t M, int64_t K,
                             int64_t F, int64_t E, int64_t T, int64_t group_size, w4a16_act act, void* workspace,
                             size_t workspace_bytes, void* stream);

typedef enum {
    W4A16_LOGITS_FP16 = 0,
    W4A16_LOGITS_BF16 = 1,
    W4A16_LOGITS_FP32 = 2,
    W4A16_LOGITS_RANGE_MIN_ = -0x7FFFFFFF - 1,
    W4A16_LOGITS_RANGE_MAX_ = 0x7FFFFFFF
} w4a16_logits;

/* How a row's token is drawn: one value for all rows, or (pointer not NULL) fp32 / int32 [M],
 * one per row, in its place. */
typedef struct {
    float temperature;          /* t; not above 0: the largest logit (the lowest v of it), whatever
                                   the rest says, with logprob 0 */
    int32_t top_k;              /* below 1, or V and above: all                             */
    float top_p;                /* 1 and above or no number: all; not above 0: the first    */
    float min_p;                /* not above 0: all; above 1: as 1                          */
    const float* temperatures;
    const int32_t* top_ks;
    const float* top_ps;
    const float* min_ps;
} w4a16_sampling;

/* Draws one token a row from its logits z, given one uniform random number u a row:
 *   w[v] = e^((z[v] - max z) / t)
 *   kept: the top_k largest z (ties to the lowest v); of these, in falling order, the shortest
 *         run whose weights reach top_p of their sum (at least one); of these w[v] >= min_p
 *   ids[m]      the first v, in rising order, with (sum of kept w up to v) > u * (their sum)
 *   logprob[m]  log of w over that sum (fp32 [M], or NULL: not wanted)
 * A logit that is no number counts as -infinity, which is never drawn; +infinity excludes
 * all others. A row with nothing to draw gives id -1, logprob -infinity. u below 0 (or no
 * number) counts as 0, 1 and above draws the last token kept.
 *   logits  [M, V], `type`, row m at logits + m * row_stride elements (row_stride >= V), aligned
 *           to its element; read only.
 * 1 <= V <= 2^28. Weights and their sums are in fp64; top_p's sums in 64-bit fixed point, a
 * step of 2^-62 V (V rounded up to a power of two; at least 2^-51) of the largest weight. */
size_t w4a16_sample_workspace_bytes(int64_t M, int64_t V);
w4a16_status w4a16_sample(const void* logits, w4a16_logits type, int64_t row_stride, const float* u, int64_t M, int64_t V,
                          const w4a16_sampling* how, int32_t* ids, float* logprob, void* workspace,
                          size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_SERVE_H */
