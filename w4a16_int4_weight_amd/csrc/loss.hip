// Losses over the packed output head that never form the logits in memory.
//
//   z_v = x . W_v / tau,  lse = log sum_v e^{z_v},  q_v = e^{z_v - lse}
//   loss = tau^2 sum_j p_j (log p_j - z_{id_j} + lse)          (p: the row's targets)
//   dx   = dloss tau sum_v (q_v - sum_{j: id_j = v} p_j) W_v
//
// Cross entropy is one target of weight 1 at tau = 1. The targets' own logits are short
// dot products with single columns, taken by a kernel of their own; the vocabulary is
// met in tiles of x W.
//
// Every row has a reference r from the start, its largest target logit. Each tile leaves,
// per row, the sum of P = e^{z - r} (fp32), and a last kernel joins them in a fixed order.
// With a gradient each tile is still formed once (bf16): P goes to a piece buffer as it is
// formed, the product with W^T of that piece follows, and at the end
// dx = e^{r - lse} (P W^T). r need only lie within 40 of the row's maximum: P is bf16, of
// fp32's range. A row that goes higher in some tile takes that tile's maximum as the tile's
// reference, and the product with W^T brings the row's tiles to a common one ("hot": rare,
// right for any logits, off the usual path: 4096 x 2048 x 131072 takes 5790 us instead of
// 4700 on one set of inputs). A row without a target, whose reference is column 0's logit and may lie anywhere,
// takes references of its own for its log-sum but makes nothing hot: its gradient is zero.
// fp16 has not that range: there the statistics come first, in a product of their own, and
// P = 2^15 q is formed with r = lse - 15 log 2, in fp16 (the target term of a loss in fp16
// is 8 times finer than bf16's rounding).
// The targets' columns are zero in P and enter at the end in fp32, (q_t - p_t) W_t: for a
// confident row that difference is small, and of two rounded numbers it would be lost.
// A row's only target is left out of its tiles' sums too: with w = sum_{v != t} e^{z_v - z_t}
// the loss is log(1 + w) and q_t - 1 = -w / (1 + w), neither a difference of large numbers
// (lse - z_t, two sums of different order, came out at -1.5e-5 for losses of 1e-9, and 19%
// off at 2e-3 where logits are in the hundreds).
//
// Roundings: P once and W once, to the operand type; dx once. Measured on 4096 x 2048 x
// 131072 with its gradient: 9490 us with the tile formed twice and the scheduling left to
// the compiler, 4900 us so (4730 where every call has the same inputs; two products of 2.2
// TFLOP, about 900 TFLOP/s each); bound as tile_product.h and gemm_grad.hip have it.
#include "device_common.h"
#include "launch.h"
#include "tile_product.h"

namespace w4a16 {
namespace {

constexpr float kHeadroom = 40.f;           // far inside fp32's range, sums and gains too
constexpr int kShiftBits = 15;              // fp16: P = 2^15 q

struct LossArgs {
    ProductArgs p;
    float inv_tau;
    float2* part;            // [tiles_n][M] (reference, sum) of a tile's row, from this launch's first tile
    const float* ref;        // [M]
    const int32_t* only;     // [M] the column of a row's only target, left out (or -1), or NULL
    uint16_t* q;             // [M, ldq] P
    int ldq;
    const int32_t* live;     // [M] whether the row has a target, and so a gradient
    int* hot;                // set when a tile took a reference of its own for a live row
};

// kSums: the rows' sums over the tile; kOut: P of the tile to the piece buffer
template <class P, bool kSums, bool kOut>
__device__ __forceinline__ void loss_epilogue(const LossArgs& a, typename P::Shared& sh, int m0, int n_tile,
                                              f32x4 (&acc)[P::MR][P::CBW]) {
    constexpr int kRow = P::BN * 2 + 16;
    constexpr int kChunks = P::BN / 8;
    static_assert(P::BM * kRow + P::W * P::BM * 4 + 64 <= (int)sizeof(typename P::Shared), "LDS");
    const int tid = threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
    const int c = lane & 15, h = lane >> 4;
    const int M = a.p.M;
    uint8_t* tile = reinterpret_cast<uint8_t*>(&sh);
    float* red = reinterpret_cast<float*>(tile + P::BM * kRow);                // [W][BM]
    int* flag = reinterpret_cast<int*>(red + P::W * P::BM);
    const int n0 = a.p.n_begin + n_tile * P::BN;
    const int nw = n0 + w * 16 * P::CBW;
    const bool whole = nw + 16 * P::CBW <= a.p.N;
    float ref[P::MR];
#pragma unroll
    for (int r = 0; r < P::MR; ++r) {
        const int m = m0 + 16 * r + c;
        ref[r] = a.ref[m < M ? m : M - 1];
    }
    if (a.only) {
        // a target lies in few waves' columns (128 rows x 32 columns of 131072: in 3% of them)
        int at[P::MR];
        bool mine = false;
#pragma unroll
        for (int r = 0; r < P::MR; ++r) {
            const int m = m0 + 16 * r + c;
            at[r] = a.only[m < M ? m : M - 1] - nw;
            mine |= (unsigned)at[r] < 16u * P::CBW;
        }
        if (__any(mine)) {
#pragma unroll
            for (int r = 0; r < P::MR; ++r) {
                if (!__any((unsigned)at[r] < 16u * P::CBW)) continue;
#pragma unroll
                for (int j = 0; j < P::CBW; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[r][j][e] = at[r] == 16 * j + 4 * h + e ? -INFINITY : acc[r][j][e];
            }
        }
    }
    auto emit = [&](const float* rf) -> bool {       // true: a sum is out of range (or no number)
        bool high = false;
#pragma unroll
        for (int r = 0; r < P::MR; ++r) {
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < P::CBW; ++j) {
                float q[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    q[e] = __expf(fmaf(acc[r][j][e], a.inv_tau, -rf[r]));
                    if (!whole && nw + 16 * j + 4 * h + e >= a.p.N) q[e] = 0.f;
                    sum += q[e];
                }
                if constexpr (kOut)
                    *reinterpret_cast<uint2*>(tile + (16 * r + c) * kRow + 2 * (16 * (w * P::CBW + j) + 4 * h)) =
                        make_uint2(pack2_rne<P::kBF16>(q[0], q[1]), pack2_rne<P::kBF16>(q[2], q[3]));
            }
            if constexpr (kSums) {
                high |= !(sum < 2e17f);              // e^40
                sum = quarter_sum(sum);
                if (h == 0) red[w * P::BM + 16 * r + c] = sum;
            }
        }
        return high;
    };
    if constexpr (kSums) {
        if (tid == 0) *flag = 0;
        __syncthreads();
    }
    const bool high = emit(ref);
    if constexpr (kSums) {
        if (high) *flag = 1;
        __syncthreads();
        if (*flag) {
            // the row's maximum over the tile takes the reference's place where it is higher
            __syncthreads();
#pragma unroll
            for (int r = 0; r < P::MR; ++r) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < P::CBW; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (whole || nw + 16 * j + 4 * h + e < a.p.N) top = fmaxf(top, acc[r][j][e] * a.inv_tau);
                top = quarter_max(top);
                if (h == 0) red[w * P::BM + 16 * r + c] = top;
            }
            __syncthreads();
            bool hot = false;
#pragma unroll
            for (int r = 0; r < P::MR; ++r) {
                float top = -INFINITY;
                for (int i = 0; i < P::W; ++i) top = fmaxf(top, red[i * P::BM + 16 * r + c]);
                if (top > ref[r] + kHeadroom - 8.f) {
                    const int m = m0 + 16 * r + c;
                    ref[r] = top;
                    if (a.hot) hot |= a.live[m < M ? m : M - 1] != 0;
                }
            }
            __syncthreads();
            emit(ref);
            if (hot) __hip_atomic_store(a.hot, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
        }
        // (reference, sum): lane c of wave 0 holds the references of rows 16 r + c
        if (w == 0) {
#pragma unroll
            for (int r = 0; r < P::MR; ++r) {
                const int m = m0 + 16 * r + c;
                if (h != 0 || m >= M) continue;
                float sum = red[16 * r + c];
                for (int i = 1; i < P::W; ++i) sum += red[i * P::BM + 16 * r + c];
                a.part[(size_t)n_tile * M + m] = make_float2(ref[r], sum);
            }
        }
    } else {
        __syncthreads();
    }
    if constexpr (!kOut) return;
    for (int i = tid; i < P::BM * kChunks; i += P::kThreads) {
        const int row = i / kChunks, ch = i % kChunks;
        const int m = m0 + row, n = n0 + 8 * ch;
        if (m < M && n < a.p.n_end)
            *reinterpret_cast<uint4*>(a.q + (size_t)m * a.ldq + (n - a.p.n_begin)) =
                *reinterpret_cast<const uint4*>(tile + row * kRow + 16 * ch);
    }
}

template <class P, bool kProb>
__global__ __launch_bounds__(P::kThreads) void loss_kernel(const LossArgs a) {
    __shared__ typename P::Shared sh;
    int m_tile, n_tile, split;
    if (!product_tile(a.p, (int)blockIdx.x, &m_tile, &n_tile, &split)) return;
    f32x4 acc[P::MR][P::CBW];
    P::run(a.p, sh, m_tile, n_tile, split, acc);
    if (a.p.splits > 1 && !reduce_splits<P::MR, P::CBW, P::W>(acc, a.p.counters, a.p.partials,
                                                              m_tile * a.p.tiles_n + n_tile, split, a.p.splits))
        return;
    loss_epilogue<P, P::kBF16 || !kProb, kProb>(a, sh, m_tile * P::BM, n_tile, acc);
}

// One wave: x . W_id of kCols columns in fp32, (q - z) s exactly. Lane: row block lane / 4
// (+ 16, ...), rows 8 (lane % 4) + 32 i of it. Several columns at a time share the loads of
// x and hide each other's latency.
template <bool kBF16, int kCols>
__device__ __forceinline__ void column_dots(const uint16_t* __restrict__ x, const uint8_t* __restrict__ packed, int K, int Np,
                                            int UW, int sub, const int (&id)[kCols], int lane, float (&total)[kCols]) {
    const int KB = K / kRowsPerBlock;
    const int h = lane & 3;
    const uint8_t* codes[kCols];
    const uint32_t* meta[kCols];
#pragma unroll
    for (int n = 0; n < kCols; ++n) {
        codes[n] = packed + (size_t)(id[n] >> 4) * KB * kBlockBytes + 16 * (16 * h + (id[n] & 15));
        meta[n] = reinterpret_cast<const uint32_t*>(packed + (size_t)K * Np / 2) + (size_t)id[n] * UW;
        total[n] = 0.f;
    }
    for (int kb = lane >> 2; kb < KB; kb += 16) {
        uint4 q[kCols];
        uint32_t md[kCols][4];
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
            q[n] = *reinterpret_cast<const uint4*>(codes[n] + (size_t)kb * kBlockBytes);
#pragma unroll
            for (int i = 0; i < 4; ++i) md[n][i] = meta[n][kb * sub + ((i * sub) >> 2)];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 xv = *reinterpret_cast<const uint4*>(x + (size_t)kb * kRowsPerBlock + 32 * i + 8 * h);
#pragma unroll
            for (int n = 0; n < kCols; ++n) {
                const uint32_t d = i == 0 ? q[n].x : i == 1 ? q[n].y : i == 2 ? q[n].z : q[n].w;
                const float z = (float)((md[n][i] >> 16) & 0xFu);
                float a = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t xp = e == 0 ? xv.x : e == 1 ? xv.y : e == 2 ? xv.z : xv.w;
                    a = fmaf(half_bits_to_f32<kBF16>(xp & 0xFFFFu), (float)((d >> (4 * e)) & 0xFu) - z, a);
                    a = fmaf(half_bits_to_f32<kBF16>(xp >> 16), (float)((d >> (4 * e + 16)) & 0xFu) - z, a);
                }
                total[n] = fmaf(half_bits_to_f32<kBF16>(md[n][i] & 0xFFFFu), a, total[n]);
            }
        }
    }
    for (int s = 32; s > 0; s >>= 1)
#pragma unroll
        for (int n = 0; n < kCols; ++n) total[n] += __shfl_xor(total[n], s);
}
template <bool kBF16>
__device__ __forceinline__ float column_dot(const uint16_t* x, const uint8_t* packed, int K, int Np, int UW, int sub, int id, int lane) {
    const int ids[1] = {id};
    float total[1];
    column_dots<kBF16, 1>(x, packed, K, Np, UW, sub, ids, lane, total);
    return total[0];
}

constexpr int kMaxTargets = 256;

struct TargetArgs {
    const uint16_t* x;
    const uint8_t* packed;
    const int32_t* ids;      // [M, T] as given
    const float* top;        // [M, T] teacher logits, or NULL: one target of weight 1
    int M, K, N, T, UW, sub;
    float inv_tau;
    int32_t* out_ids;        // [M, T] each column once, -1: none (distillation)
    float* weight;           // [M, T]
    float* ent;              // [M] sum p log p
    float* zsel;             // [M, T]
    float* ref;              // [M] the largest target logit, without a target column 0's
    int32_t* live;           // [M] whether the row has a target (where `hot` is used)
    int* hot;
};

// Cross entropy: a wave a row.
template <bool kBF16>
__global__ __launch_bounds__(256) void label_kernel(const TargetArgs a) {
    const int m = (int)blockIdx.x * 4 + ((int)threadIdx.x >> 6), lane = (int)threadIdx.x & 63;
    if (a.hot && blockIdx.x == 0 && threadIdx.x == 0) *a.hot = 0;
    if (m >= a.M) return;
    int id = a.ids[m];
    const bool live = id >= 0 && id < a.N;
    if (!live) id = 0;
    const float z = a.inv_tau * column_dot<kBF16>(a.x + (size_t)m * a.K, a.packed, a.K, (int)padded_cols(a.N), a.UW, a.sub, id, lane);
    if (lane == 0) {
        a.zsel[m] = z;
        a.ref[m] = z;
        if (a.hot) a.live[m] = live;
    }
}

// Distillation: a workgroup a row. The teacher's list -> target weights, p = softmax of
// t / tau over the row's valid ids (0 where the id is none or t is -inf; all 0 if nothing is
// left). An id that comes more than once keeps its first entry, with the sum of the weights,
// so that later steps meet each column once; ent = sum p log p is of the entries as given.
template <bool kBF16>
__global__ __launch_bounds__(256) void targets_kernel(const TargetArgs a) {
    __shared__ int sid[kMaxTargets], first_id[kMaxTargets];
    __shared__ float sp[kMaxTargets];
    __shared__ float wave_top[4];
    const int m = (int)blockIdx.x, tid = (int)threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int T = a.T;
    if (a.hot && m == 0 && tid == 0) *a.hot = 0;
    if (w == 0) {
        float top = -INFINITY;
        for (int j = lane; j < T; j += 64) {
            const int id = a.ids[(size_t)m * T + j];
            const bool ok = id >= 0 && id < a.N;
            const float v = ok ? a.top[(size_t)m * T + j] * a.inv_tau : -INFINITY;
            sid[j] = ok ? id : -1;
            sp[j] = v;
            top = fmaxf(top, v);
        }
        for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
        const float ref = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        for (int j = lane; j < T; j += 64) {
            sp[j] = __expf(sp[j] - ref);
            sum += sp[j];
        }
        for (int s = 32; s > 0; s >>= 1) sum += __shfl_xor(sum, s);
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        float en = 0.f;
        for (int j = lane; j < T; j += 64) {
            sp[j] *= inv;
            if (sp[j] > 0.f) en += sp[j] * logf(sp[j]);
        }
        for (int s = 32; s > 0; s >>= 1) en += __shfl_xor(en, s);
        if (lane == 0) {
            a.ent[m] = en;
            if (a.hot) a.live[m] = sum != 0.f;
            if (T == 1 && sp[0] == 0.f) sid[0] = -1;         // an only target that weighs nothing is none
        }
    }
    __syncthreads();
    for (int j = tid; j < T; j += 256) {
        const int id = sid[j];
        float p = sp[j];
        bool first = id >= 0;
        for (int i = 0; i < T; ++i) {
            if (i == j || sid[i] != id) continue;
            if (i < j) first = false;
            p += sp[i];
        }
        first_id[j] = first ? id : -1;
        a.out_ids[(size_t)m * T + j] = first ? id : -1;
        a.weight[(size_t)m * T + j] = first ? p : 0.f;
    }
    __syncthreads();
    const uint16_t* x = a.x + (size_t)m * a.K;
    float top = -INFINITY;
    for (int j0 = 4 * w; j0 < T; j0 += 16) {
        int id[4];
        float z[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) id[n] = j0 + n < T && first_id[j0 + n] >= 0 ? first_id[j0 + n] : 0;
        column_dots<kBF16, 4>(x, a.packed, a.K, (int)padded_cols(a.N), a.UW, a.sub, id, lane, z);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (j0 + n >= T || first_id[j0 + n] < 0) continue;
            z[n] *= a.inv_tau;
            if (lane == 0) a.zsel[(size_t)m * T + j0 + n] = z[n];
            top = fmaxf(top, z[n]);
        }
    }
    if (lane == 0) wave_top[w] = top;
    __syncthreads();
    if (w == 0) {
        top = fmaxf(fmaxf(wave_top[0], wave_top[1]), fmaxf(wave_top[2], wave_top[3]));
        if (top == -INFINITY)
            top = a.inv_tau * column_dot<kBF16>(x, a.packed, a.K, (int)padded_cols(a.N), a.UW, a.sub, 0, lane);
        if (lane == 0) a.ref[m] = top;
    }
}

// Between a piece's two products: the targets' places in P become zero (T = 0: they are),
// and where a tile took a reference of its own the rows' tiles are given the factors that bring them, and
// the sums of the pieces before, to the row's highest reference.
__global__ __launch_bounds__(256) void settle_kernel(const int32_t* __restrict__ ids, int M, int T, int N, int n0, int n,
                                                     uint16_t* __restrict__ q, int ldq, const int* __restrict__ hot,
                                                     const float2* __restrict__ part, int tiles, float* __restrict__ ref,
                                                     float* __restrict__ factor, float* __restrict__ before) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at < (int64_t)M * T) {
        const int id = ids[at];
        if (id >= n0 && id < n0 + n && id < N) q[(at / T) * (int64_t)ldq + (id - n0)] = 0;
    }
    if (!hot || *hot == 0 || at >= M) return;
    const int m = (int)at;
    const float old = ref[m];
    float top = old;
    for (int t = 0; t < tiles; ++t) top = fmaxf(top, part[(size_t)t * M + m].x);
    for (int t = 0; t < tiles; ++t) factor[(size_t)t * M + m] = __expf(part[(size_t)t * M + m].x - top);
    before[m] = __expf(old - top);
    ref[m] = top;
}

// Rows: 16 rows a workgroup, 16 threads a row; the tiles' statistics and the targets'
// terms are added in an order that depends on the shape alone.
struct RowArgs {
    const float2* part;
    int tiles, M, N, T;
    const int32_t* ids;
    const float* weight;
    const float* ent;
    const float* zsel;
    float tau;
    const float* dloss;
    float* loss;
    float* lse;
    float* coef;             // [M] dloss tau, 0 for a row without a target, or NULL
    float* gain;             // [M] the factor of P W^T in dx
    const float* ref;        // [M] P's reference (bf16) ...
    float* next_ref;         // ... or that of the P to come (fp16)
    float* rest;             // [M] q_t - 1 (kOnly)
};
// kOnly: one target a row, which the sums leave out
template <bool kOnly>
__global__ __launch_bounds__(256) void rows_kernel(const RowArgs a) {
    __shared__ float2 sv[16][17];
    const int i = (int)threadIdx.x & 15, g = (int)threadIdx.x >> 4;
    const int m = (int)blockIdx.x * 16 + i;
    const int M = a.M;
    const int mc = m < M ? m : M - 1;
    [[maybe_unused]] bool live = false;
    [[maybe_unused]] float z = 0.f;
    if constexpr (kOnly) {
        const int id = a.ids[mc];
        live = id >= 0 && id < a.N;
        if (live) z = a.zsel[mc];
    }
    // (a maximum passes over what is no number; the sums carry it, also where nothing else is left)
    auto join = [](float2 v, float2 o) {
        const float top = fmaxf(v.x, o.x);
        return make_float2(top, top == -INFINITY ? v.y + o.y : v.y * __expf(v.x - top) + o.y * __expf(o.x - top));
    };
    float2 v = make_float2(-INFINITY, 0.f);
    for (int t0 = g; t0 < a.tiles; t0 += 128) {           // 8 loads in flight
        float2 o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int t = t0 + 16 * k;
            o[k] = t < a.tiles ? a.part[(size_t)t * M + mc] : make_float2(-INFINITY, 0.f);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) v = join(v, o[k]);
    }
    sv[g][i] = v;
    __syncthreads();
    v = sv[0][i];
    for (int k = 1; k < 16; ++k) v = join(v, sv[k][i]);
    float lse = v.x + logf(v.y);
    if constexpr (kOnly) {
        if (g != 0 || m >= M) return;
        const float others = lse;                // log of the sum without the target
        float loss = 0.f;
        if (live) {
            const float far = v.x - z;
            lse = far > 0.f ? v.x + logf(v.y + __expf(-far)) : z + log1pf(v.y * __expf(far));
            loss = far > 30.f ? lse - z : log1pf(v.y * __expf(far));
        }
        const float p = a.weight && live ? a.weight[m] : 1.f;        // 1, or no number
        a.loss[m] = a.tau * a.tau * loss * p;
        a.lse[m] = lse;
        if (a.coef) {
            const float cf = live ? a.tau * (a.dloss ? a.dloss[m] : 1.f) * p : 0.f;
            const float rest = expm1f(-loss);
            a.coef[m] = cf;
            a.rest[m] = rest;
            if (a.next_ref) {
                // 2^15 of what the others have: the largest of them fills fp16 however little it is
                const bool some = others - lse > -60.f;
                a.next_ref[m] = (some ? others : lse) - kShiftBits * 0.6931471806f;
                a.gain[m] = cf * (some && live ? -rest : 1.f) * (1.f / (1 << kShiftBits));
            } else {
                a.gain[m] = cf * __expf(a.ref[m] - lse);
            }
        }
        return;
    }
    __syncthreads();
    float sum = 0.f, mass = 0.f;
    for (int j = g; j < a.T; j += 16) {
        const int id = a.ids[(size_t)mc * a.T + j];
        if (id < 0 || id >= a.N) continue;
        const float p = a.weight[(size_t)mc * a.T + j];
        if (p == 0.f) continue;
        sum += p * (lse - a.zsel[(size_t)mc * a.T + j]);
        mass += p;
    }
    sv[g][i] = make_float2(sum, mass);
    __syncthreads();
    if (g == 0 && m < M) {
        sum = 0.f;
        mass = 0.f;
        for (int k = 0; k < 16; ++k) {
            sum += sv[k][i].x;
            mass += sv[k][i].y;
        }
        const bool some = mass != 0.f;
        sum += a.ent[m];
        a.loss[m] = some ? a.tau * a.tau * sum : 0.f;
        a.lse[m] = lse;
        if (a.coef) {
            const float cf = some ? a.tau * (a.dloss ? a.dloss[m] : 1.f) : 0.f;
            a.coef[m] = cf;
            a.gain[m] = a.next_ref ? cf * (1.f / (1 << kShiftBits)) : cf * __expf(a.ref[m] - lse);
            if (a.next_ref) a.next_ref[m] = lse - kShiftBits * 0.6931471806f;
        }
    }
}

// dx[m] = gain[m] sum_s part[s][m] + sum_j coef[m] (q_j - p_j) W[:, id_j], one rounding. A
// thread takes 8 elements of a row (one code word per target); where there are many splits
// and targets, kShare threads share them and their sums meet in LDS, in a fixed order.
struct FinishArgs {
    const float* part;
    int splits, M, K, N, T, UW, sub;
    const uint8_t* packed;
    const float *coef, *gain, *lse, *zsel, *weight;
    const float* rest;       // q_t - 1 of a row's only target, or NULL
    const int32_t* ids;
    uint16_t* dx;
};
template <bool kBF16, int kShare>
__global__ __launch_bounds__(256) void finish_kernel(const FinishArgs a) {
    constexpr int kWide = 256 / kShare;                    // threads along a row
    __shared__ int sid[kMaxTargets];
    __shared__ float sc[kMaxTargets];
    __shared__ float sums[kShare > 1 ? kShare : 1][kShare > 1 ? kWide * 8 + 4 : 1];
    const int m = (int)blockIdx.x, tid = (int)threadIdx.x;
    const int g = tid / kWide, at = tid % kWide;
    const int k0 = 8 * ((int)blockIdx.y * kWide + at);
    const float coef = a.coef[m], gain = a.gain[m];
    for (int j = tid; j < a.T; j += 256) {
        const int id = a.ids[(size_t)m * a.T + j];
        const bool ok = id >= 0 && id < a.N;
        sid[j] = ok ? id : 0;
        const size_t at_j = (size_t)m * a.T + j;
        sc[j] = !ok ? 0.f : coef * (a.rest ? a.rest[m] : __expf(a.zsel[at_j] - a.lse[m]) - a.weight[at_j]);
    }
    __syncthreads();
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (k0 < a.K && coef != 0.f) {
        f32x4 s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
        const size_t MK = (size_t)a.M * a.K;
        const float* p = a.part + (size_t)m * a.K + k0;
#pragma unroll 4
        for (int s = g; s < a.splits; s += kShare) {
            s0 += *reinterpret_cast<const f32x4*>(p + s * MK);
            s1 += *reinterpret_cast<const f32x4*>(p + s * MK + 4);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = s0[e] * gain;
            v[e + 4] = s1[e] * gain;
        }
        const int KB = a.K / kRowsPerBlock, kb = k0 / kRowsPerBlock, i = (k0 >> 5) & 3, h = (k0 >> 3) & 3;
        const uint8_t* codes = a.packed + (size_t)kb * kBlockBytes + 256 * h + 4 * i;
        const uint32_t* meta = reinterpret_cast<const uint32_t*>(a.packed + (size_t)a.K * padded_cols(a.N) / 2) + kb * a.sub +
                               ((i * a.sub) >> 2);
#pragma unroll 8
        for (int j = g; j < a.T; j += kShare) {
            const int id = sid[j];
            const float cf = sc[j];
            const uint32_t d = *reinterpret_cast<const uint32_t*>(codes + (size_t)(id >> 4) * KB * kBlockBytes + 16 * (id & 15));
            const uint32_t md = meta[(size_t)id * a.UW];
            const float s = cf * half_bits_to_f32<kBF16>(md & 0xFFFFu);
            const float z = (float)((md >> 16) & 0xFu);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[tile_row_of_slot(e)] = fmaf((float)((d >> (4 * e)) & 0xFu) - z, s, v[tile_row_of_slot(e)]);
        }
    }
    if constexpr (kShare > 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[g][8 * at + e] = v[e];
        __syncthreads();
        static_assert(kShare == 8, "a thread sums one element");
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < kShare; ++i) t += sums[i][tid];
        const int k = (int)blockIdx.y * kWide * 8 + tid;
        if (k < a.K) a.dx[(size_t)m * a.K + k] = f32_to_half_bits<kBF16>(t);
    } else if (k0 < a.K) {
        *reinterpret_cast<uint4*>(a.dx + (size_t)m * a.K + k0) =
            make_uint4(pack2_rne<kBF16>(v[0], v[1]), pack2_rne<kBF16>(v[2], v[3]), pack2_rne<kBF16>(v[4], v[5]),
                       pack2_rne<kBF16>(v[6], v[7]));
    }
}

template <bool kBF16, int MR, int kSub, bool kProb>
void launch_cfg(LossArgs& a, hipStream_t s) {
    using P = TileProduct<kBF16, MR, kProductColumns / 128, 8, kSub, false>;
    const int64_t ids = product_ids(a.p.tiles_m, a.p.tiles_n, a.p.splits);
    hipLaunchKernelGGL((loss_kernel<P, kProb>), dim3((unsigned)ids), dim3(P::kThreads), 0, s, a);
}

template <bool kBF16, bool kProb>
void launch_typed(const ProductPlan& p, LossArgs& a, hipStream_t s) {
    if (p.sub == 4) {
        if (p.mr == 1) launch_cfg<kBF16, 1, 4, kProb>(a, s);
        else if (p.mr == 2) launch_cfg<kBF16, 2, 4, kProb>(a, s);
        else launch_cfg<kBF16, 4, 4, kProb>(a, s);
    } else if (p.sub == 2) {
        if (p.mr == 1) launch_cfg<kBF16, 1, 2, kProb>(a, s);
        else if (p.mr == 2) launch_cfg<kBF16, 2, 2, kProb>(a, s);
        else launch_cfg<kBF16, 4, 2, kProb>(a, s);
    } else if (p.mr == 1) launch_cfg<kBF16, 1, 1, kProb>(a, s);
    else if (p.mr == 2) launch_cfg<kBF16, 2, 1, kProb>(a, s);
    else if (p.mr == 4) launch_cfg<kBF16, 4, 1, kProb>(a, s);
    else launch_cfg<kBF16, 8, 1, kProb>(a, s);
}

void launch_any(const ProductPlan& p, LossArgs& a, bool bf16, bool prob, hipStream_t s) {
    if (bf16) prob ? launch_typed<true, true>(p, a, s) : launch_typed<true, false>(p, a, s);
    else prob ? launch_typed<false, true>(p, a, s) : launch_typed<false, false>(p, a, s);
}

constexpr int64_t kRowsPerPass = 4096;
constexpr int64_t kPieceBytes = int64_t(1) << 28;

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

// Where one pass over `M` rows keeps its pieces, in bytes from the workspace's start
struct LossLayout {
    ProductPlan stats, prob;   // stats: without a gradient, and fp16's
    GradPlan grad;
    int64_t piece, pieces;
    bool small;              // up to 16 rows without a gradient: one kernel before the rows'
    size_t hot, partials, part, zsel, ids, weight, ent, coef, gain, rest, ref, live, factor, before, q, gpart, end;
};

LossLayout loss_layout(int64_t M, int64_t K, int64_t V, int64_t G, int64_t T, bool bf16, bool distill, bool grad) {
    LossLayout l{};
    l.small = !distill && !grad && small_product(M, K);
    if (!l.small && !(grad && bf16)) l.stats = plan_product(M, K, V, G, false);
    size_t partial = l.stats.partial_bytes;
    int64_t tiles = l.small ? small_workgroups(padded_cols(V) / kColsPerBlock) : l.stats.tiles_n;       // bf16's: below
    if (grad) {
        // pieces of the vocabulary: P of a piece takes at most 256 MiB (it then stays in
        // the last-level cache between the two products)
        int64_t most = kPieceBytes / (2 * M) / 512 * 512;
        if (most < 512) most = 512;
        l.pieces = (V + most - 1) / most;
        l.piece = ((V + l.pieces - 1) / l.pieces + 511) / 512 * 512;
        l.pieces = (V + l.piece - 1) / l.piece;
        const int64_t last = V - (l.pieces - 1) * l.piece;
        l.prob = plan_product(M, K, l.pieces > 1 ? l.piece : last, G, false);
        const ProductPlan tail = plan_product(M, K, last, G, false);
        if (l.prob.partial_bytes > partial) partial = l.prob.partial_bytes;
        if (tail.partial_bytes > partial) partial = tail.partial_bytes;
        if (bf16) tiles = (l.pieces - 1) * l.prob.tiles_n + tail.tiles_n;
        l.grad = plan_grad(M, K, l.pieces > 1 ? l.piece : last, true);
    }
    size_t at = kSplitCounterBytes;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += round256(bytes);
        return here;
    };
    l.hot = take(4);         // (right behind the counters)
    l.partials = take(partial);
    l.part = take((size_t)tiles * M * 8);
    l.zsel = take((size_t)M * T * 4);
    l.ids = take(distill ? (size_t)M * T * 4 : 0);
    l.weight = take(distill ? (size_t)M * T * 4 : 0);
    l.ent = take(distill ? (size_t)M * 4 : 0);
    l.coef = take((size_t)M * 4);
    l.gain = take((size_t)M * 4);
    l.rest = take(grad && T == 1 ? (size_t)M * 4 : 0);
    l.ref = take((size_t)M * 4);
    l.live = take(grad && bf16 ? (size_t)M * 4 : 0);
    l.factor = take(grad && bf16 ? (size_t)l.prob.tiles_n * M * 4 : 0);
    l.before = take(grad && bf16 ? (size_t)M * 4 : 0);
    l.q = take(grad ? (size_t)M * l.piece * 2 : 0);
    l.gpart = take(grad ? l.grad.part_bytes : 0);
    l.end = at;
    return l;
}

}  // namespace

int max_loss_targets() { return kMaxTargets; }

size_t loss_workspace(int64_t M, int64_t K, int64_t V, int64_t G, int64_t T, bool distill, bool grad) {
    const int64_t full = M < kRowsPerPass ? M : kRowsPerPass;
    size_t need = 0;
    for (const bool bf16 : {false, true}) {       // one size for both types
        size_t n = loss_layout(full, K, V, G, T, bf16, distill, grad).end;
        if (n > need) need = n;
        if (M > full && M % full) {
            n = loss_layout(M % full, K, V, G, T, bf16, distill, grad).end;
            if (n > need) need = n;
        }
    }
    return need;
}

hipError_t launch_loss(const LossCall& q, hipStream_t stream) {
    uint8_t* ws = static_cast<uint8_t*>(q.workspace);
    const bool distill = q.top != nullptr;
    const bool grad = q.dx != nullptr;
    const bool sums_first = !grad || !q.bf16;
    const bool only = q.T == 1;
    for (int64_t r0 = 0; r0 < q.M; r0 += kRowsPerPass) {
        const int64_t M = q.M - r0 < kRowsPerPass ? q.M - r0 : kRowsPerPass;
        const LossLayout l = loss_layout(M, q.K, q.V, q.G, q.T, q.bf16, distill, grad);
        auto floats = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
        float2* part = reinterpret_cast<float2*>(ws + l.part);
        int* hot = grad && q.bf16 ? reinterpret_cast<int*>(ws + l.hot) : nullptr;
        float* ref = floats(l.ref);
        const int32_t* ids = q.ids + r0 * q.T;

        TargetArgs t{};
        t.x = q.x + r0 * q.K;
        t.packed = q.packed;
        t.ids = ids;
        t.M = (int)M;
        t.K = (int)q.K;
        t.N = (int)q.V;
        t.T = (int)q.T;
        t.UW = (int)padded_units(q.K, q.G);
        t.sub = units_per_block(q.G);
        t.inv_tau = 1.f / q.tau;
        t.zsel = floats(l.zsel);
        t.ref = ref;
        t.live = reinterpret_cast<int32_t*>(ws + l.live);
        t.hot = hot;
        if (distill) {
            t.top = q.top + r0 * q.T;
            t.out_ids = reinterpret_cast<int32_t*>(ws + l.ids);
            t.weight = floats(l.weight);
            t.ent = floats(l.ent);
            if (q.bf16) hipLaunchKernelGGL((targets_kernel<true>), dim3((unsigned)M), dim3(256), 0, stream, t);
            else hipLaunchKernelGGL((targets_kernel<false>), dim3((unsigned)M), dim3(256), 0, stream, t);
            ids = t.out_ids;
        } else if (!l.small) {
            const dim3 grid((unsigned)((M + 3) / 4));
            if (q.bf16) hipLaunchKernelGGL((label_kernel<true>), grid, dim3(256), 0, stream, t);
            else hipLaunchKernelGGL((label_kernel<false>), grid, dim3(256), 0, stream, t);
        }

        LossArgs a{};
        a.p.x = t.x;
        a.p.packed = q.packed;
        a.p.M = (int)M;
        a.p.K = (int)q.K;
        a.p.N = (int)q.V;
        a.p.counters = static_cast<uint32_t*>(q.workspace);
        a.p.partials = floats(l.partials);
        a.inv_tau = t.inv_tau;
        a.ref = ref;
        a.only = only ? ids : nullptr;
        a.live = t.live;
        a.hot = hot;
        auto product = [&](const ProductPlan& p, int64_t n0, int64_t n, bool prob) {
            a.p.n_begin = (int)n0;
            a.p.n_end = (int)(n0 + n);
            a.p.tiles_m = p.tiles_m;
            a.p.tiles_n = p.tiles_n;
            a.p.splits = p.splits;
            launch_any(p, a, q.bf16, prob, stream);
        };
        RowArgs rows{};
        rows.part = part;
        rows.M = (int)M;
        rows.N = (int)q.V;
        rows.T = (int)q.T;
        rows.ids = ids;
        rows.weight = t.weight;
        rows.ent = t.ent;
        rows.zsel = t.zsel;
        rows.tau = q.tau;
        rows.dloss = q.dloss ? q.dloss + r0 : nullptr;
        rows.loss = q.loss + r0;
        rows.lse = q.lse + r0;
        if (grad) {
            rows.coef = floats(l.coef);
            rows.gain = floats(l.gain);
            rows.rest = floats(l.rest);
            rows.ref = ref;
            if (!q.bf16) rows.next_ref = ref;
        }
        auto join_rows = [&]() {
            const dim3 grid((unsigned)((M + 15) / 16));
            if (only) hipLaunchKernelGGL((rows_kernel<true>), grid, dim3(256), 0, stream, rows);
            else hipLaunchKernelGGL((rows_kernel<false>), grid, dim3(256), 0, stream, rows);
        };
        if (sums_first) {
            a.part = part;
            if (l.small) {
                const hipError_t e = launch_ce_small(t.x, ids, q.packed, M, q.K, q.V, q.G, q.bf16, t.zsel, floats(l.part), stream);
                if (e != hipSuccess) return e;
                rows.tiles = small_workgroups(padded_cols(q.V) / kColsPerBlock);
            } else {
                product(l.stats, 0, q.V, false);
                rows.tiles = l.stats.tiles_n;
            }
            join_rows();
        }
        hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        if (!grad) continue;

        a.q = reinterpret_cast<uint16_t*>(ws + l.q);
        a.ldq = (int)l.piece;
        int tiles = 0;
        for (int64_t n0 = 0; n0 < q.V; n0 += l.piece) {
            const int64_t n = q.V - n0 < l.piece ? q.V - n0 : l.piece;
            const ProductPlan p = n == l.piece ? l.prob : plan_product(M, q.K, n, q.G, false);
            a.part = part + (size_t)tiles * M;
            product(p, n0, n, true);
            if (!only || hot)
                hipLaunchKernelGGL(settle_kernel, dim3((unsigned)((M * q.T + 255) / 256)), dim3(256), 0, stream, ids, (int)M,
                                   only ? 0 : (int)q.T, (int)q.V, (int)n0, (int)n, a.q, a.ldq, hot, a.part, p.tiles_n, ref,
                                   floats(l.factor), floats(l.before));
            tiles += p.tiles_n;
            GradCall g{};
            g.d = a.q;
            g.ld = l.piece;
            g.packed = q.packed;
            g.part = floats(l.gpart);
            g.add = n0 > 0;
            g.M = M;
            g.K = q.K;
            g.N = q.V;
            g.G = q.G;
            g.n0 = n0;
            g.n = n;
            g.bf16 = q.bf16;
            g.hot = hot;
            g.factor = floats(l.factor);
            g.before = floats(l.before);
            g.factor_columns = kProductColumns;
            err = launch_grad(l.grad, g, stream);
            if (err != hipSuccess) return err;
        }
        if (!sums_first) {
            rows.tiles = tiles;
            join_rows();
        }
        FinishArgs f{};
        f.part = floats(l.gpart);
        f.splits = l.grad.splits;
        f.M = (int)M;
        f.K = (int)q.K;
        f.N = (int)q.V;
        f.T = (int)q.T;
        f.UW = t.UW;
        f.sub = t.sub;
        f.packed = q.packed;
        f.coef = rows.coef;
        f.gain = rows.gain;
        f.lse = rows.lse;
        f.zsel = t.zsel;
        f.weight = t.weight;
        f.rest = only ? rows.rest : nullptr;
        f.ids = ids;
        f.dx = q.dx + r0 * q.K;
        // shared where a thread alone would meet 16 loads or more (65 rows, 20 targets, 64
        // splits: 24 -> 6.6 us; 1024 rows, 64 targets: 83 -> 80 us, bound by the lines the
        // columns' codes lie in), else one thread each (4096 rows, 1 target, 2 splits: 18 us)
        const bool share = f.splits + f.T >= 16;
        const dim3 finish_grid((unsigned)M, (unsigned)(share ? (q.K + 255) / 256 : (q.K + 2047) / 2048));
        if (q.bf16) {
            if (share) hipLaunchKernelGGL((finish_kernel<true, 8>), finish_grid, dim3(256), 0, stream, f);
            else hipLaunchKernelGGL((finish_kernel<true, 1>), finish_grid, dim3(256), 0, stream, f);
        } else {
            if (share) hipLaunchKernelGGL((finish_kernel<false, 8>), finish_grid, dim3(256), 0, stream, f);
            else hipLaunchKernelGGL((finish_kernel<false, 1>), finish_grid, dim3(256), 0, stream, f);
        }
        err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace w4a16
