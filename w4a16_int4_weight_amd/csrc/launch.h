// Host-side launchers of the W4A16 kernels. Arguments are assumed validated by the
// C ABI layer (api.hip): shapes supported by the tile layout, pointers aligned.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a16 {

// AWQ tensors of columns [n0, n0 + N) of a K x Nt weight -> those columns of the
// packed tile layout of the K x Nt weight (n0 % 16 == 0; N % 16 == 0 unless
// n0 + N == Nt). G: resolved group size (32, 64, or a multiple of 128 dividing K).
hipError_t launch_repack(const int32_t* qweight, const int32_t* qzeros, const uint16_t* scales,
                         uint8_t* packed, int64_t K, int64_t N, int64_t G, int64_t n0, int64_t Nt,
                         hipStream_t stream);
// The same from GPTQ-standard tensors (codes packed along K, standard order).
hipError_t launch_repack_gptq(const int32_t* qweight, const int32_t* qzeros, const uint16_t* scales,
                              uint8_t* packed, int64_t K, int64_t N, int64_t G, int64_t n0, int64_t Nt,
                              hipStream_t stream);

// Weight-streaming split-K GEMV for 1 <= M <= 16: K split over the waves of a
// workgroup, and for outputs of at most 128 column blocks (K >= 6144, M >= 6) also
// over 2-4 workgroups per block when the caller's workspace holds their partials.
struct GemvPlan {
    int kb_per_wave;       // row blocks per wave (multiple of 4)
    int waves;             // waves per workgroup (waves_k per column block)
    int waves_k;           // waves splitting K for one 16-column block
    bool staged;           // activations staged in LDS
    int chunks_per_thread; // 16-byte activation chunks each thread stages
    int sub;               // metadata units per 128-row block (128 / G for G = 32, 64; else 1)
    size_t lds_bytes;
    int splits;            // workgroups per column block along K
    int kb_per_split;      // row blocks per such workgroup
    size_t workspace_bytes;   // [counters][splits x blocks x 1 KiB fp32 partials] when splits > 1
};
GemvPlan plan_gemv(int64_t M, int64_t K, int64_t N, int64_t G, size_t workspace_bytes);

// `workspace` (or NULL) holds `workspace_bytes` bytes whose counter part is zero; the
// kernel uses it only if plan_gemv splits K over workgroups with that many bytes, and
// leaves the counters zero.
hipError_t launch_gemv(const uint16_t* x, const uint8_t* packed, const uint16_t* bias, uint16_t* y,
                       int64_t M, int64_t K, int64_t N, int64_t G, bool bf16, void* workspace,
                       size_t workspace_bytes, hipStream_t stream);

// Decode GEMV for M = 1 over equal shares of 8-column half blocks, one workgroup per
// compute unit (G >= 128). ok = false when the shape does not fit it (then the
// GEMV above runs).
struct StripPlan {
    bool ok;
    int grid;          // workgroups
    int items;         // code loads in flight per lane
    size_t lds_bytes;
};
StripPlan plan_gemv_strip(int64_t M, int64_t K, int64_t N, int64_t G);

hipError_t launch_gemv_strip(const StripPlan& plan, const uint16_t* x, const uint8_t* packed, const uint16_t* bias,
                             uint16_t* y, int64_t K, int64_t N, int64_t G, bool bf16, hipStream_t stream);

// Decode GEMV for 2 <= M <= 16 on the matrix cores over equal shares of 8-column half
// blocks, one workgroup per compute unit (G >= 128). ok = false when the shape does
// not fit it or the GEMV above is faster on it.
struct SmallPlan {
    bool ok;
    int P;             // units (row-block pairs) per half block
    int grid;          // workgroups
    int smax;          // most half blocks of any workgroup
    int JP;            // most units of one half block per wave
};
SmallPlan plan_gemv_small(int64_t M, int64_t K, int64_t N, int64_t G);

hipError_t launch_gemv_small(const SmallPlan& plan, const uint16_t* x, const uint8_t* packed, const uint16_t* bias,
                             uint16_t* y, int64_t M, int64_t K, int64_t N, int64_t G, bool bf16, hipStream_t stream);

// Tied-embedding gather: out[t, :] = dequantised column ids[t] of the packed [K, N]
// weight (zeros for ids outside [0, N)).
hipError_t launch_embedding(const int32_t* ids, int64_t T, const uint8_t* packed, uint16_t* out, int64_t K,
                            int64_t N, int64_t G, bool bf16, hipStream_t stream);

// LDS-staged dequantise -> MFMA GEMM for any M >= 1: tile shape and K split chosen
// from the shape; workspace_bytes > 0 when K is split over workgroups.
struct GemmPlan {
    int mr;            // row fragments of 16 per tile (tile rows = 16 * mr)
    int cbw;           // 16-column blocks per wave (tile columns = 16 * waves * cbw)
    int waves;         // waves per workgroup, side by side along N (4 or 8)
    int tiles_m, tiles_n;
    int splits;        // workgroups per tile along K
    int sub;           // metadata units per 128-row block (128 / G for G = 32, 64; else 1)
    size_t workspace_bytes;   // [kSplitCounterBytes of tile counters][splits x M x N fp32 partials]
};
GemmPlan plan_gemm(int64_t M, int64_t K, int64_t N, int64_t G);

// `workspace` must hold plan_gemm(M, K, N, G).workspace_bytes bytes whose counter part is
// zero; the kernel leaves it zero.
hipError_t launch_gemm(const uint16_t* x, const uint8_t* packed, const uint16_t* bias, uint16_t* y,
                       int64_t M, int64_t K, int64_t N, int64_t G, bool bf16, void* workspace,
                       hipStream_t stream);

// W4A8 activations after quantisation (one caller buffer, see w4a8_activation_bytes):
// codes [M x K] E4M3 bytes in operand order, row_scale [M] fp32, block_sum [M x K/128]
// fp32 (sum of each 128-element block's decoded codes).
struct W4A8Act {
    uint8_t* codes;
    float* row_scale;
    float* block_sum;
};
hipError_t launch_w4a8_quantize(const uint16_t* x, int64_t M, int64_t K, bool bf16, const W4A8Act& a,
                                hipStream_t stream);
// Tiles of launch_gemm (plan_gemm, G >= 128), plus a 256 x 256 tile for outputs of at
// least two rounds of it; the workspace never exceeds plan_gemm's.
hipError_t launch_w4a8_gemm(const W4A8Act& a, const uint8_t* packed, const uint16_t* bias, uint16_t* y, int64_t M,
                            int64_t K, int64_t N, int64_t G, bool bf16, void* workspace, hipStream_t stream);

// Tiles of the training and scoring products (csrc/tile_product.h): `cols` columns of the
// weight (2F for a gated block), 16 mr rows and 256 columns (8 waves of 2 column blocks) each.
constexpr int kProductColumns = 256;
struct ProductPlan {
    int mr, sub;
    int tiles_m, tiles_n, splits;
    size_t partial_bytes;  // fp32 partial tiles of a K split (0 without one)
};
ProductPlan plan_product(int64_t M, int64_t K, int64_t cols, int64_t G, bool gated);

// Gated block: h = a(x Wg) (x Wu) when d is NULL; else d = [dg, du] [M, 2F] from dh, fp16,
// each row of a column tile scaled by the power of two of its `tops`.
// act: 0 silu, 1 gelu, 2 gelu's tanh form. counters / partials as plan_product asks.
struct GatedCall {
    const uint16_t* x;
    const uint16_t* dh;
    const uint8_t* packed;
    uint16_t* h;
    uint16_t* d;
    uint16_t* d_rest;      // NULL, or [M, 2F]: what d's rounding leaves, at the same scales
    float* d32;            // what small_product shapes write instead
    float* tops;           // [gated_tiles(...)][M] largest |d| of a row in each share of the columns
    int64_t M, K, F, G;
    int act;
    bool bf16;
    uint32_t* counters;
    float* partials;
};
hipError_t launch_gated(const GatedCall& call, hipStream_t stream);
int gated_tiles(int64_t M, int64_t K, int64_t F, int64_t G);
int gated_tile_columns(int64_t M, int64_t K);       // 0: d's rows have one scale
// Between a backward's products: the rows' largest |d| from `tops`, the factors [tile][M] (two
// fp16) that bring the tiles to their row's scale, and the largest |scale| of the weight in
// kScaleParts parts.
constexpr int kScaleParts = 64;
hipError_t launch_gated_tops(const GatedCall& call, float* rowmax, uint32_t* factor, float* scale_max, hipStream_t stream);

// Up to 16 rows (csrc/product_small.hip): the gated block, and the head's statistics for
// cross entropy: the labels' logits and (max, sum) per row and workgroup, part
// [small_workgroups][M] pairs. No workspace besides.
bool small_product(int64_t M, int64_t K);
int small_workgroups(int64_t units);
hipError_t launch_gated_small(const GatedCall& call, hipStream_t stream);
hipError_t launch_ce_small(const uint16_t* x, const int32_t* labels, const uint8_t* packed, int64_t M, int64_t K, int64_t V,
                           int64_t G, bool bf16, float* zsel, float* part, hipStream_t stream);

// dx = D W^T: D [M, columns n0 .. n0 + n) of the weight, row stride ld, of the weight's type. The sum over columns is split over
// `splits` workgroups and may be cut into calls: with `part` set, partial tiles
// [splits][M][K] fp32 are written (or, with `add`, added to); grad_finish sums them.
struct GradCall {
    const uint16_t* d;
    int64_t ld;
    const uint8_t* packed;
    uint16_t* dx;          // NULL when `part` is set
    float* part;
    bool add;
    int64_t M, K, N, G;    // N: columns of the weight
    int64_t n0, n;         // n0 % 64 == 0
    bool bf16;
    // when *hot is set: D's rows are multiplied by factor[tile][M], tile of factor_columns
    // columns from n0, and what `add` adds to by before[M]. hot may be NULL.
    const int* hot;
    const float* factor;
    const float* before;
    int factor_columns;
    // `scaled`: D is fp16 at its rows' scales (rowmax), times tile_factor[tile][M] where that
    // is not NULL, tile of tile_columns columns from 0 and from N / 2; the weights are taken
    // in fp16, scaled from the largest |scale| (scale_max)
    bool scaled;
    const uint16_t* d_rest;   // added to d
    const float* rowmax;
    const uint32_t* tile_factor;
    int tile_columns;
    const float* scale_max;
};
struct GradPlan {
    int bm;                // rows of a tile: 16, 32, 64, 128 or 256
    int tiles_m, tiles_k;
    int splits;
    size_t part_bytes;     // [splits][M][K] fp32 when splits > 1
};
// Whether a scaled product of this type takes d_rest: fp16, tiles of up to 128 rows.
bool grad_takes_rest(const GradPlan& plan, bool bf16);
// `forced`: the sum comes in several calls, so partials are needed at any split.
GradPlan plan_grad(int64_t M, int64_t K, int64_t n, bool forced);
hipError_t launch_grad(const GradPlan& plan, const GradCall& call, hipStream_t stream);
// dx[m, k] = sum_s part[s][m][k], rounded once (rowmax, scale_max: of a `scaled` product)
hipError_t launch_grad_finish(const float* part, int splits, int64_t M, int64_t K, uint16_t* dx, bool bf16,
                              const float* rowmax, const float* scale_max, hipStream_t stream);

// Cross entropy (top NULL, T = 1) or distillation over the packed head. lse and loss
// [M] fp32; dx (or NULL) with dloss (or NULL: 1). The workspace holds loss_workspace(...)
// bytes whose counter part is zero; the kernels leave it zero.
struct LossCall {
    const uint16_t* x;
    const int32_t* ids;    // [M, T]
    const float* top;      // [M, T] teacher logits
    const uint8_t* packed;
    const float* dloss;
    float* loss;
    float* lse;
    uint16_t* dx;
    int64_t M, K, V, G, T;
    float tau;
    bool bf16;
    void* workspace;
};
int max_loss_targets();
size_t loss_workspace(int64_t M, int64_t K, int64_t V, int64_t G, int64_t T, bool distill, bool grad);
hipError_t launch_loss(const LossCall& call, hipStream_t stream);

// Router of a mixture of experts (csrc/route.hip): counters zero, left zero; logits of
// route_logits_bytes.
constexpr int kMaxExperts = 1024;
constexpr int kMaxChosen = 32;         // experts of a row
struct RouteCall {
    const uint16_t* x;
    const uint16_t* router;
    const float* bias;
    int64_t M, K, E, T;
    int sigmoid, normalize;
    float scale;
    int32_t* ids;
    float* weights;
    bool bf16;
    uint32_t* counters;
    void* logits;
};
size_t route_logits_bytes(int64_t M, int64_t E);
hipError_t launch_route(const RouteCall& call, hipStream_t stream);

// Mixture of experts on packed weights. M T pairs are indexed in 32 bits, and h's rows
// (2 M T F elements) within 4 GiB.
struct MoeCall {
    const uint16_t* x;
    const int32_t* ids;
    const float* weights;
    const uint8_t* gate_up;
    const uint8_t* down;
    int64_t gate_up_stride, down_stride;
    const uint16_t* residual;   // or NULL
    uint16_t* y;
    int64_t M, K, F, E, T, G;
    int act;
    bool bf16;
};
// csrc/moe.hip, where moe_small: counters zero, left zero; scratch of moe_small_scratch bytes
bool moe_small(int64_t M, int64_t K, int64_t T);
size_t moe_small_scratch(int64_t M, int64_t K, int64_t F, int64_t E, int64_t T);
hipError_t launch_moe_small(const MoeCall& call, uint32_t* counters, uint8_t* scratch, hipStream_t stream);
// csrc/moe_tile.hip: scratch of layout.end bytes, nothing in it kept between calls
struct MoeTileLayout {
    int mr, slots;
    size_t list, slot, h, out, end;
};
MoeTileLayout moe_tile_layout(int64_t M, int64_t K, int64_t F, int64_t E, int64_t T, int64_t G);
hipError_t launch_moe_tile(const MoeCall& call, uint8_t* scratch, hipStream_t stream);

// Draws a token from each row's logits (csrc/sample.hip). kind: 0 fp16, 1 bf16, 2 fp32.
struct SampleCall {
    const void* logits;
    int kind;
    int64_t ld, M, V;
    const float* u;
    float temperature, top_p, min_p;
    int32_t top_k;
    const float* temperatures;
    const int32_t* top_ks;
    const float* top_ps;
    const float* min_ps;
    int32_t* ids;
    float* logprob;             // or NULL
};
// scratch of sample_workspace bytes (NULL where that is 0), nothing in it kept between calls
size_t sample_workspace(int64_t M, int64_t V);
hipError_t launch_sample(const SampleCall& call, void* scratch, hipStream_t stream);

}  // namespace w4a16
