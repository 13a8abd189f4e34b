// Losses over the packed output head that never form the logits in memory.
//
//   z_v = x . W_v / tau,  lse = log sum_v e^{z_v},  q_v = e^{z_v - lse}
//   loss = tau^2 sum_j p_j (log p_j - z_{id_j} + lse)          (p: the row's targets)
//   dx   = dloss tau sum_v (q_v - sum_{j: id_j = v} p_j) W_v
//
// Cross entropy is one target of weight 1 at tau = 1. Three steps:
//   1. statistics: each tile of x . W leaves per row its maximum m and sum e^{z - m}
//      (fp32) and the logits of the row's targets; the tile itself is dropped;
//   2. rows: the tiles' (m, sum) joined in a fixed order into lse, the loss, and the
//      row's factor dloss tau (0 for a row without a target: its dx is zero whatever x
//      holds);
//   3. with a gradient, piece by piece of the vocabulary: the tile again, q - p rounded
//      once to bf16 (for fp16 too: probabilities go below fp16's range) into a piece
//      buffer, and the product with W^T of that piece, added up in fp32.
// Recomputing the tile costs one product more than keeping e^{z - m} would, and gives
// q - p in fp32 before its one rounding: for a confident row q_target - 1 is small and a
// difference of two rounded numbers would lose it.
#include "device_common.h"
#include "launch.h"
#include "tile_product.h"

namespace w4a16 {
namespace {

struct LossArgs {
    ProductArgs p;
    float inv_tau;
    int T;
    const int32_t* ids;      // [M, T] targets, negative or past the head: none
    const float* weight;     // [M, T] or NULL (1)
    float* zsel;             // [M, T] logits of the targets
    float2* part;            // [tiles_n][M] (max, sum) of a tile's row
    const float* lse;        // [M]
    const float* coef;       // [M], 0: no gradient
    uint16_t* q;             // [M, ldq] bf16
    int ldq;
};

template <class P>
__device__ __forceinline__ void stats_epilogue(const LossArgs& a, typename P::Shared& sh, int m0, int n_tile,
                                               f32x4 (&acc)[P::MR][P::CBW]) {
    constexpr int kCols = 16 * P::CBW;                       // of a wave
    constexpr int kPitch = kCols + 1;
    const int tid = threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
    const int c = lane & 15, h = lane >> 4;
    const int M = a.p.M, N = a.p.N, T = a.T;
    float* scratch = reinterpret_cast<float*>(&sh) + w * 16 * kPitch;          // 16 rows of this wave
    float2* red = reinterpret_cast<float2*>(reinterpret_cast<float*>(&sh) + P::W * 16 * kPitch);   // [W][BM]
    static_assert(P::W * 16 * kPitch * 4 + P::W * P::BM * 8 <= (int)sizeof(typename P::Shared), "LDS");
    const int nw = a.p.n_begin + n_tile * P::BN + w * kCols;                   // the wave's first column
#pragma unroll
    for (int r = 0; r < P::MR; ++r) {
#pragma unroll
        for (int j = 0; j < P::CBW; ++j) acc[r][j] *= a.inv_tau;
        // targets among this wave's columns: row 16 r + c, entries h, h + 4, ...
        const int m = m0 + 16 * r + c;
        bool any = false;
        if (m < M) {
            for (int j = h; j < T; j += 4) {
                const int id = a.ids[(size_t)m * T + j];
                any |= id >= nw && id < nw + kCols && id < N;
            }
        }
        if (__any(any)) {
#pragma unroll
            for (int j = 0; j < P::CBW; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) scratch[c * kPitch + 16 * j + 4 * h + e] = acc[r][j][e];
            __builtin_amdgcn_wave_barrier();
            if (any) {
                for (int j = h; j < T; j += 4) {
                    const int id = a.ids[(size_t)m * T + j];
                    if (id >= nw && id < nw + kCols && id < N) a.zsel[(size_t)m * T + j] = scratch[c * kPitch + id - nw];
                }
            }
            __builtin_amdgcn_wave_barrier();
        }
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < P::CBW; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (nw + 16 * j + 4 * h + e >= N) acc[r][j][e] = -INFINITY;
                top = fmaxf(top, acc[r][j][e]);
            }
        top = quarter_max(top);
        const float ref = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < P::CBW; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += __expf(acc[r][j][e] - ref);
        sum = quarter_sum(sum);
        if (h == 0) red[w * P::BM + 16 * r + c] = make_float2(top, sum);
    }
    __syncthreads();
    if (tid < P::BM && m0 + tid < M) {
        float2 v = red[tid];
#pragma unroll
        for (int i = 1; i < P::W; ++i) {
            const float2 o = red[i * P::BM + tid];
            const float top = fmaxf(v.x, o.x);
            if (top != -INFINITY) v = make_float2(top, v.y * __expf(v.x - top) + o.y * __expf(o.x - top));
        }
        a.part[(size_t)n_tile * M + m0 + tid] = v;
    }
}

// q - p of the tile, bf16
template <class P>
__device__ __forceinline__ void prob_epilogue(const LossArgs& a, typename P::Shared& sh, int m0, int n_tile,
                                              f32x4 (&acc)[P::MR][P::CBW]) {
    constexpr int kRow = P::BN * 2 + 16;
    constexpr int kChunks = P::BN / 8;
    static_assert(P::BM * kRow <= (int)sizeof(typename P::Shared), "LDS");
    const int tid = threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
    const int c = lane & 15, h = lane >> 4;
    const int M = a.p.M, T = a.T;
    uint8_t* tile = reinterpret_cast<uint8_t*>(&sh);
    const int n0 = a.p.n_begin + n_tile * P::BN;
#pragma unroll
    for (int r = 0; r < P::MR; ++r) {
        const int row = 16 * r + c;
        const int m = m0 + row < M ? m0 + row : M - 1;
        const float lse = a.lse[m];
        const bool live = a.coef[m] != 0.f;
#pragma unroll
        for (int j = 0; j < P::CBW; ++j) {
            float q[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) q[e] = live ? __expf(acc[r][j][e] * a.inv_tau - lse) : 0.f;
            *reinterpret_cast<uint2*>(tile + row * kRow + 2 * (16 * (w * P::CBW + j) + 4 * h)) =
                make_uint2(pack2_rne<true>(q[0], q[1]), pack2_rne<true>(q[2], q[3]));
        }
    }
    __syncthreads();
    // the targets' entries, again in fp32 from the logit kept in step 1 (a row's ids are
    // distinct here, so no entry has two writers)
    for (int row = tid >> 2; row < P::BM; row += P::kThreads / 4) {
        const int m = m0 + row;
        if (m >= M || a.coef[m] == 0.f) continue;
        for (int j = tid & 3; j < T; j += 4) {
            const int id = a.ids[(size_t)m * T + j];
            if (id < n0 || id >= n0 + P::BN || id >= a.p.N) continue;
            const float p = a.weight ? a.weight[(size_t)m * T + j] : 1.f;
            *reinterpret_cast<uint16_t*>(tile + row * kRow + 2 * (id - n0)) =
                f32_to_half_bits<true>(__expf(a.zsel[(size_t)m * T + j] - a.lse[m]) - p);
        }
    }
    __syncthreads();
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
    if constexpr (kProb) prob_epilogue<P>(a, sh, m_tile * P::BM, n_tile, acc);
    else stats_epilogue<P>(a, sh, m_tile * P::BM, n_tile, acc);
}

// A teacher's list -> target weights, one wave a row: p = softmax of t / tau over the
// row's valid ids (0 where the id is none or t is -inf; all 0 if nothing is left). An id
// that comes more than once keeps its first entry, with the sum of the weights, so that
// later steps meet each column once; ent = sum p log p is of the entries as given.
constexpr int kMaxTargets = 256;
__global__ __launch_bounds__(64) void targets_kernel(const int32_t* __restrict__ ids, const float* __restrict__ t, int M,
                                                     int T, int N, float inv_tau, int32_t* __restrict__ out_ids,
                                                     float* __restrict__ out_p, float* __restrict__ ent) {
    __shared__ int sid[kMaxTargets];
    __shared__ float sp[kMaxTargets];
    const int m = (int)blockIdx.x, lane = (int)threadIdx.x;
    float top = -INFINITY;
    for (int j = lane; j < T; j += 64) {
        const int id = ids[(size_t)m * T + j];
        const bool ok = id >= 0 && id < N;
        const float v = ok ? t[(size_t)m * T + j] * inv_tau : -INFINITY;
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
    __syncthreads();
    for (int j = lane; j < T; j += 64) {
        const int id = sid[j];
        float p = sp[j];
        bool first = id >= 0;
        for (int i = 0; i < T; ++i) {
            if (i == j || sid[i] != id) continue;
            if (i < j) first = false;
            p += sp[i];
        }
        out_ids[(size_t)m * T + j] = first ? id : -1;
        out_p[(size_t)m * T + j] = first ? p : 0.f;
    }
    if (lane == 0) ent[m] = en;
}

// Rows: 16 rows a workgroup, 16 threads a row; the tiles' statistics and the targets'
// terms are added in an order that depends on the shape alone.
__global__ __launch_bounds__(256) void rows_kernel(const float2* __restrict__ part, int tiles, int M, int N, int T,
                                                   const int32_t* __restrict__ ids, const float* __restrict__ weight,
                                                   const float* __restrict__ ent, const float* __restrict__ zsel, float tau,
                                                   const float* __restrict__ dloss, float* __restrict__ loss,
                                                   float* __restrict__ lse_out, float* __restrict__ coef) {
    __shared__ float2 sv[16][17];
    const int i = (int)threadIdx.x & 15, g = (int)threadIdx.x >> 4;
    const int m = (int)blockIdx.x * 16 + i;
    const int mc = m < M ? m : M - 1;
    float2 v = make_float2(-INFINITY, 0.f);
    for (int t = g; t < tiles; t += 16) {
        const float2 o = part[(size_t)t * M + mc];
        const float top = fmaxf(v.x, o.x);
        if (top != -INFINITY) v = make_float2(top, v.y * __expf(v.x - top) + o.y * __expf(o.x - top));
    }
    sv[g][i] = v;
    __syncthreads();
    v = sv[0][i];
    for (int k = 1; k < 16; ++k) {
        const float2 o = sv[k][i];
        const float top = fmaxf(v.x, o.x);
        if (top != -INFINITY) v = make_float2(top, v.y * __expf(v.x - top) + o.y * __expf(o.x - top));
    }
    const float lse = v.x + logf(v.y);
    __syncthreads();
    float sum = 0.f, mass = 0.f;
    for (int j = g; j < T; j += 16) {
        const int id = ids[(size_t)mc * T + j];
        if (id < 0 || id >= N) continue;
        const float p = weight ? weight[(size_t)mc * T + j] : 1.f;
        if (p == 0.f) continue;
        sum += p * (lse - zsel[(size_t)mc * T + j]);
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
        const bool live = mass != 0.f;
        if (ent) sum += ent[m];
        loss[m] = live ? tau * tau * sum : 0.f;
        lse_out[m] = lse;
        if (coef) coef[m] = live ? tau * (dloss ? dloss[m] : 1.f) : 0.f;
    }
}

template <bool kBF16, int MR, int CBW, int kSub, bool kProb>
void launch_cfg(LossArgs& a, hipStream_t s) {
    using P = TileProduct<kBF16, MR, CBW, 8, kSub, false>;
    const int64_t ids = product_ids(a.p.tiles_m, a.p.tiles_n, a.p.splits);
    hipLaunchKernelGGL((loss_kernel<P, kProb>), dim3((unsigned)ids), dim3(P::kThreads), 0, s, a);
}

template <bool kBF16, bool kProb>
void launch_typed(const ProductPlan& p, LossArgs& a, hipStream_t s) {
    if (p.sub == 4) {
        if (p.mr == 1) launch_cfg<kBF16, 1, 2, 4, kProb>(a, s);
        else launch_cfg<kBF16, 4, 2, 4, kProb>(a, s);
    } else if (p.sub == 2) {
        if (p.mr == 1) launch_cfg<kBF16, 1, 2, 2, kProb>(a, s);
        else launch_cfg<kBF16, 4, 2, 2, kProb>(a, s);
    } else if (p.mr == 1) launch_cfg<kBF16, 1, 2, 1, kProb>(a, s);
    else if (p.mr == 2) launch_cfg<kBF16, 2, 2, 1, kProb>(a, s);
    else if (p.mr == 4) launch_cfg<kBF16, 4, 2, 1, kProb>(a, s);
    else launch_cfg<kBF16, 8, 2, 1, kProb>(a, s);
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
    ProductPlan stats, prob;
    GradPlan grad;
    int64_t piece, pieces;
    size_t partials, part, zsel, ids, weight, ent, coef, lse, q, gpart, end;
};

LossLayout loss_layout(int64_t M, int64_t K, int64_t V, int64_t G, int64_t T, bool distill, bool grad) {
    LossLayout l{};
    l.stats = plan_product(M, K, V, G, false);
    size_t partial = l.stats.partial_bytes;
    if (grad) {
        // pieces of the vocabulary: q of a piece takes at most 256 MiB (it then stays in
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
        l.grad = plan_grad(M, K, l.pieces > 1 ? l.piece : last, true);
    }
    size_t at = kSplitCounterBytes;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += round256(bytes);
        return here;
    };
    l.partials = take(partial);
    l.part = take((size_t)l.stats.tiles_n * M * 8);
    l.zsel = take((size_t)M * T * 4);
    l.ids = take(distill ? (size_t)M * T * 4 : 0);
    l.weight = take(distill ? (size_t)M * T * 4 : 0);
    l.ent = take(distill ? (size_t)M * 4 : 0);
    l.coef = take((size_t)M * 4);
    l.q = take(grad ? (size_t)M * l.piece * 2 : 0);
    l.gpart = take(grad ? l.grad.part_bytes : 0);
    l.end = at;
    return l;
}

}  // namespace

int max_loss_targets() { return kMaxTargets; }

size_t loss_workspace(int64_t M, int64_t K, int64_t V, int64_t G, int64_t T, bool distill, bool grad) {
    const int64_t full = M < kRowsPerPass ? M : kRowsPerPass;
    size_t need = loss_layout(full, K, V, G, T, distill, grad).end;
    if (M > full && M % full) {
        const size_t tail = loss_layout(M % full, K, V, G, T, distill, grad).end;
        if (tail > need) need = tail;
    }
    return need;
}

hipError_t launch_loss(const LossCall& q, hipStream_t stream) {
    uint8_t* ws = static_cast<uint8_t*>(q.workspace);
    const bool distill = q.top != nullptr;
    const bool grad = q.dx != nullptr;
    for (int64_t r0 = 0; r0 < q.M; r0 += kRowsPerPass) {
        const int64_t M = q.M - r0 < kRowsPerPass ? q.M - r0 : kRowsPerPass;
        const LossLayout l = loss_layout(M, q.K, q.V, q.G, q.T, distill, grad);
        LossArgs a{};
        a.p.x = q.x + r0 * q.K;
        a.p.packed = q.packed;
        a.p.M = (int)M;
        a.p.K = (int)q.K;
        a.p.N = (int)q.V;
        a.p.n_begin = 0;
        a.p.n_end = (int)q.V;
        a.p.counters = static_cast<uint32_t*>(q.workspace);
        a.p.partials = reinterpret_cast<float*>(ws + l.partials);
        a.inv_tau = 1.f / q.tau;
        a.T = (int)q.T;
        a.zsel = reinterpret_cast<float*>(ws + l.zsel);
        a.part = reinterpret_cast<float2*>(ws + l.part);
        float* coef = reinterpret_cast<float*>(ws + l.coef);
        const float* ent = nullptr;
        if (distill) {
            int32_t* ids = reinterpret_cast<int32_t*>(ws + l.ids);
            float* weight = reinterpret_cast<float*>(ws + l.weight);
            float* e = reinterpret_cast<float*>(ws + l.ent);
            hipLaunchKernelGGL(targets_kernel, dim3((unsigned)M), dim3(64), 0, stream, q.ids + r0 * q.T, q.top + r0 * q.T,
                               (int)M, (int)q.T, (int)q.V, a.inv_tau, ids, weight, e);
            a.ids = ids;
            a.weight = weight;
            ent = e;
        } else {
            a.ids = q.ids + r0 * q.T;
        }
        a.p.tiles_m = l.stats.tiles_m;
        a.p.tiles_n = l.stats.tiles_n;
        a.p.splits = l.stats.splits;
        launch_any(l.stats, a, q.bf16, false, stream);
        float* lse = q.lse + r0;
        hipLaunchKernelGGL(rows_kernel, dim3((unsigned)((M + 15) / 16)), dim3(256), 0, stream, a.part, l.stats.tiles_n, (int)M,
                           (int)q.V, (int)q.T, a.ids, a.weight, ent, a.zsel, q.tau, q.dloss ? q.dloss + r0 : nullptr,
                           q.loss + r0, lse, grad ? coef : nullptr);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        if (!grad) continue;
        a.lse = lse;
        a.coef = coef;
        a.q = reinterpret_cast<uint16_t*>(ws + l.q);
        a.ldq = (int)l.piece;
        for (int64_t n0 = 0; n0 < q.V; n0 += l.piece) {
            const int64_t n = q.V - n0 < l.piece ? q.V - n0 : l.piece;
            const ProductPlan p = n == l.piece ? l.prob : plan_product(M, q.K, n, q.G, false);
            a.p.n_begin = (int)n0;
            a.p.n_end = (int)(n0 + n);
            a.p.tiles_m = p.tiles_m;
            a.p.tiles_n = p.tiles_n;
            a.p.splits = p.splits;
            launch_any(p, a, q.bf16, true, stream);
            GradCall g{};
            g.d = a.q;
            g.ld = l.piece;
            g.packed = q.packed;
            g.part = reinterpret_cast<float*>(ws + l.gpart);
            g.add = n0 > 0;
            g.M = M;
            g.K = q.K;
            g.N = q.V;
            g.G = q.G;
            g.n0 = n0;
            g.n = n;
            g.op_bf16 = true;
            g.scale_bf16 = q.bf16;
            err = launch_grad(l.grad, g, stream);
            if (err != hipSuccess) return err;
        }
        err = launch_grad_finish(reinterpret_cast<const float*>(ws + l.gpart), l.grad.splits, M, q.K, coef, q.dx + r0 * q.K,
                                 q.bf16, stream);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

}  // namespace w4a16
