// Mixture of experts for more rows than the streaming kernels take (moe.hip): tiles of rows
// gathered by expert.
//
//   y[m] = residual[m] + sum_j w[m, j] h[m, j] Wd_e,   h[m, j] = a(x[m] Wg_e) * (x[m] Wu_e)
//
// A pair is an entry (m, j) of ids, number m T + j. Four launches: the pairs of each expert in
// rising order and the tiles of them (lists_kernel); the gated block of each tile, its rows of
// x gathered, h left in two bf16 values (16 bits: one bf16 would be off by as much as the
// result's own rounding, and fp16 overflows where bf16 models do not); the down projection,
// whose tile holds the upper halves of its rows in its first fragments and the lower halves in
// the others, so that one pass over the codes serves both, to fp32 rows of pairs; and each
// row's sum over its pairs in their order. No atomics on results: they do not depend on timing.
// The products are tile_product.h's.
//
// Measured (2048 x 1024, 64 experts, 8 a row): 77 rows 5 + 57 + 52 + 5 us (143 and 67 MB of codes: 2.5 and 1.3
// TB/s; 75 tiles of 8 column tiles are a round and a bit of two workgroups a compute unit), 512 rows 6 + 115 + 98
// + 7 us (64-row tiles, half the experts with a second one; 300 and, each half by itself, 350 TFLOP/s). A ring of 4
// stages: the same at 64 rows, 74 instead of 56 us at 16. Tiles of 32 rows for 512: 138 and 99 us,
// of 128 for the first product 127; tiles that begin at different row blocks: the same.
#include "device_common.h"
#include "gate.h"
#include "launch.h"
#include "tile_product.h"

namespace w4a16 {
namespace {

constexpr int kListThreads = 1024;

// Expert e's tiles take the slots from floor(pairs of lower experts / rows of a tile) + e on:
// at least as many as it has tiles, so that no expert waits for another's count; the last
// expert takes all that are left (entries that name no expert leave some). Slots without a tile
// have no rows.
struct Slot {
    int expert, first, rows, pad;       // the tile's pairs: list[first .. first + rows)
};

__global__ __launch_bounds__(kListThreads) void lists_kernel(const int32_t* __restrict__ ids, int pairs, int E, int tile_rows,
                                                            int32_t* __restrict__ list, Slot* __restrict__ slots, int all_slots) {
    __shared__ int wave_low[kListThreads / 64], wave_own[kListThreads / 64];
    const int tid = (int)threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int e = (int)blockIdx.x;
    int low = 0, own = 0;
    for (int i = tid; i < pairs; i += kListThreads) {
        const int id = ids[i];
        low += id >= 0 && id < e;
        own += id == e;
    }
    for (int s = 32; s > 0; s >>= 1) {
        low += __shfl_xor(low, s);
        own += __shfl_xor(own, s);
    }
    if (lane == 0) {
        wave_low[w] = low;
        wave_own[w] = own;
    }
    __syncthreads();
    low = own = 0;
#pragma unroll
    for (int k = 0; k < kListThreads / 64; ++k) {
        low += wave_low[k];
        own += wave_own[k];
    }
    const int slot0 = low / tile_rows + e, slot1 = e == E - 1 ? all_slots : (low + own) / tile_rows + e + 1;
    for (int s = slot0 + tid; s < slot1; s += kListThreads) {
        const int at = (s - slot0) * tile_rows, left = own - at;
        slots[s] = Slot{e, low + at, left < 0 ? 0 : left < tile_rows ? left : tile_rows, 0};
    }
    // the expert's pairs in rising order
    int at = low;
    for (int i0 = 0; i0 < pairs; i0 += kListThreads) {
        const int i = i0 + tid;
        const bool hit = i < pairs && ids[i] == e;
        const uint64_t mask = __ballot(hit);
        __syncthreads();
        if (lane == 0) wave_own[w] = __popcll(mask);
        __syncthreads();
        int before = at;
        for (int k = 0; k < kListThreads / 64; ++k) {
            before += k < w ? wave_own[k] : 0;
            at += wave_own[k];
        }
        if (hit) list[before + __popcll(mask & ((1ull << lane) - 1ull))] = i;
    }
}

// rows of x: those of the tile's pairs, the last one repeated
struct RowsOfPairs {
    static __device__ __forceinline__ const uint16_t* base(const ProductArgs& a, int) { return a.x; }
    static __device__ __forceinline__ int at(const ProductArgs& a, int, int row) {
        return a.rows[row < a.M ? row : a.M - 1] / a.row_div;
    }
};
// the two halves of h: upper ones in the first half of the tile's rows
template <int kHalf>
struct HalvesOfPairs {
    static __device__ __forceinline__ const uint16_t* base(const ProductArgs& a, int) { return a.x; }
    static __device__ __forceinline__ int at(const ProductArgs& a, int, int row) {
        const int r = row < kHalf ? row : row - kHalf;
        return 2 * a.rows[r < a.M ? r : a.M - 1] + (row < kHalf ? 0 : 1);
    }
};

struct MoeTileArgs {
    ProductArgs p;
    const Slot* slots;
    int64_t stride;         // bytes from one expert's weight to the next
    uint16_t* h;            // up: [pairs][2][F] bf16
    float* out;             // down: [pairs][N]
    int act;
};

// this workgroup's tile: false where its slot has none
__device__ __forceinline__ bool take_slot(const MoeTileArgs& a, ProductArgs* p, int* n_tile) {
    int slot, split;
    if (!product_tile(a.p, (int)blockIdx.x, &slot, n_tile, &split)) return false;
    const Slot s = a.slots[slot];
    *p = a.p;
    p->M = __builtin_amdgcn_readfirstlane(s.rows);
    if (p->M == 0) return false;
    p->rows = a.p.rows + __builtin_amdgcn_readfirstlane(s.first);
    p->packed = a.p.packed + (int64_t)__builtin_amdgcn_readfirstlane(s.expert) * a.stride;
    return true;
}

// The tile's h goes through LDS and leaves as whole rows.
template <class P, int kAct>
__device__ __forceinline__ void up_epilogue(const MoeTileArgs& a, const ProductArgs& p, typename P::Shared& sh, int f0,
                                            f32x4 (&acc)[P::MR][P::CBW]) {
    constexpr int BM = P::BM, BN = P::BN, HB = P::HB;
    constexpr int kRow = BN * 2 + 16;                        // bytes of a tile row, padded
    constexpr int kChunks = BN / 8;
    static_assert(2 * BM * kRow <= (int)sizeof(typename P::Shared), "both output tiles fit in LDS");
    const int tid = (int)threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63, c = lane & 15, h = lane >> 4;
    const int F = p.F;
    uint8_t* t0 = reinterpret_cast<uint8_t*>(&sh);
    uint8_t* t1 = t0 + BM * kRow;
#pragma unroll
    for (int r = 0; r < P::MR; ++r)
#pragma unroll
        for (int j = 0; j < HB; ++j) {
            float o[4], rest[4];
            uint32_t hi[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float g = acc[r][j][e];
                float slope;
                o[e] = g * gate_prob<kAct>(g, &slope) * acc[r][j + HB][e];
                hi[e] = f32_to_half_bits<true>(o[e]);
                rest[e] = o[e] - bf16_bits_to_f32(hi[e]);
            }
            const int at = (16 * r + c) * kRow + 2 * (16 * (w * HB + j) + 4 * h);     // 4 columns of a row
            *reinterpret_cast<uint2*>(t0 + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
            *reinterpret_cast<uint2*>(t1 + at) = make_uint2(pack2_rne<true>(rest[0], rest[1]), pack2_rne<true>(rest[2], rest[3]));
        }
    __syncthreads();
    for (int q = tid; q < BM * kChunks; q += P::kThreads) {
        const int row = q / kChunks, ch = q % kChunks;
        const int f = f0 + 8 * ch;
        if (row >= p.M || f >= F) continue;
        uint16_t* to = a.h + (size_t)2 * (size_t)p.rows[row] * F + f;
        *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(t0 + row * kRow + 16 * ch);
        *reinterpret_cast<uint4*>(to + F) = *reinterpret_cast<const uint4*>(t1 + row * kRow + 16 * ch);
    }
}

template <class P>
__global__ __launch_bounds__(P::kThreads) void up_kernel(const MoeTileArgs a) {
    __shared__ typename P::Shared sh;
    ProductArgs p;
    int n_tile;
    if (!take_slot(a, &p, &n_tile)) return;
    f32x4 acc[P::MR][P::CBW];
    P::run(p, sh, 0, n_tile, 0, acc);
    const int f0 = n_tile * P::BN;
    if (a.act == 0) up_epilogue<P, 0>(a, p, sh, f0, acc);
    else if (a.act == 1) up_epilogue<P, 1>(a, p, sh, f0, acc);
    else up_epilogue<P, 2>(a, p, sh, f0, acc);
}

template <class P>
__global__ __launch_bounds__(P::kThreads) void down_kernel(const MoeTileArgs a) {
    __shared__ typename P::Shared sh;
    ProductArgs p;
    int n_tile;
    if (!take_slot(a, &p, &n_tile)) return;
    f32x4 acc[P::MR][P::CBW];
    P::run(p, sh, 0, n_tile, 0, acc);
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int lane = (int)threadIdx.x & 63, c = lane & 15, h = lane >> 4;
#pragma unroll
    for (int r = 0; r < P::MR / 2; ++r) {
        const int row = 16 * r + c;
        if (row >= p.M) continue;
        float* to = a.out + (size_t)p.rows[row] * p.N;
#pragma unroll
        for (int j = 0; j < P::CBW; ++j) {
            const int n = n_tile * P::BN + 16 * (w * P::CBW + j) + 4 * h;
            if (n < p.N) *reinterpret_cast<f32x4*>(to + n) = acc[r][j] + acc[r + P::MR / 2][j];      // N % 128 == 0
        }
    }
}

// y[m, 8 columns a thread] = residual + the row's pairs in their order
template <bool kBF16>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ out, const int32_t* __restrict__ ids,
                                                   const float* __restrict__ weights, const uint16_t* residual, uint16_t* y,
                                                   int64_t chunks, int K, int E, int T) {
    const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (q >= chunks) return;
    const int per = K / 8;
    const int64_t m = q / per;
    const int n = (int)(q % per) * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    // four entries at a time, added in order; what names no expert has no row in `out`, and is read as another
    for (int j0 = 0; j0 < T; j0 += 4) {
        f32x4 lo[4], hi[4];
        float wt[4];
        bool in[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t at = m * T + (j0 + j < T ? j0 + j : T - 1);
            const int id = ids[at];
            in[j] = j0 + j < T && id >= 0 && id < E;
            wt[j] = weights[at];
            const f32x4* p = reinterpret_cast<const f32x4*>(out + (size_t)at * K + n);
            lo[j] = p[0];
            hi[j] = p[1];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (in[j]) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = fmaf(wt[j], lo[j][e], v[e]);
                    v[4 + e] = fmaf(wt[j], hi[j][e], v[4 + e]);
                }
            }
    }
    if (residual) {
        const uint4 r = *reinterpret_cast<const uint4*>(residual + m * K + n);
        const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += half_bits_to_f32<kBF16>((e & 1) ? rw[e / 2] >> 16 : rw[e / 2] & 0xFFFFu);
    }
    *reinterpret_cast<uint4*>(y + m * K + n) =
        make_uint4(pack2_rne<kBF16>(v[0], v[1]), pack2_rne<kBF16>(v[2], v[3]), pack2_rne<kBF16>(v[4], v[5]), pack2_rne<kBF16>(v[6], v[7]));
}

template <bool kBF16, int MR, int kSub>
void launch_pair(const MoeTileArgs& up, const MoeTileArgs& down, hipStream_t s) {
    using Up = TileProduct<kBF16, MR, kProductColumns / 128, 8, kSub, true, RowsOfPairs>;
    using Down = TileProduct<true, 2 * MR, kProductColumns / 128, 8, kSub, false, HalvesOfPairs<16 * MR>, kBF16>;
    hipLaunchKernelGGL((up_kernel<Up>), dim3((unsigned)product_ids(up.p.tiles_m, up.p.tiles_n, 1)), dim3(Up::kThreads), 0, s, up);
    hipLaunchKernelGGL((down_kernel<Down>), dim3((unsigned)product_ids(down.p.tiles_m, down.p.tiles_n, 1)), dim3(Down::kThreads), 0, s, down);
}

template <bool kBF16>
void launch_typed(int mr, int sub, const MoeTileArgs& up, const MoeTileArgs& down, hipStream_t s) {
    if (sub == 4) {
        if (mr == 1) launch_pair<kBF16, 1, 4>(up, down, s);
        else launch_pair<kBF16, 2, 4>(up, down, s);
    } else if (sub == 2) {
        if (mr == 1) launch_pair<kBF16, 1, 2>(up, down, s);
        else launch_pair<kBF16, 2, 2>(up, down, s);
    } else if (mr == 1) launch_pair<kBF16, 1, 1>(up, down, s);
    else if (mr == 2) launch_pair<kBF16, 2, 1>(up, down, s);
    else launch_pair<kBF16, 4, 1>(up, down, s);
}

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

// Rows of a tile (pairs of one expert): 16, 32 or 64, the least that holds the rows an expert
// meets on average (77 rows of 8: tiles of 16 56 us, of 32 69; 512 rows: 64 115, 32 138, 16 145) (the 128-row tile of the down projection's halves does not fit in LDS with
// finer groups than 128).
int tile_mr(int64_t M, int64_t E, int64_t T, int64_t G) {
    const int64_t each = M * T / (E < M * T ? E : M * T);
    if (each <= 16) return 1;
    return each <= 32 || units_per_block(G) > 1 ? 2 : 4;
}

}  // namespace

MoeTileLayout moe_tile_layout(int64_t M, int64_t K, int64_t F, int64_t E, int64_t T, int64_t G) {
    MoeTileLayout l{};
    const size_t pairs = (size_t)M * (size_t)T;
    l.mr = tile_mr(M, E, T, G);
    l.slots = (int)(pairs / (16 * l.mr) + E);
    l.list = 0;
    l.slot = l.list + round256(pairs * 4);
    l.h = l.slot + round256((size_t)l.slots * sizeof(Slot));
    l.out = l.h + round256(pairs * 4 * (size_t)F);
    l.end = l.out + round256(pairs * 4 * (size_t)K);
    return l;
}

hipError_t launch_moe_tile(const MoeCall& q, uint8_t* scratch, hipStream_t stream) {
    const MoeTileLayout l = moe_tile_layout(q.M, q.K, q.F, q.E, q.T, q.G);
    int32_t* list = reinterpret_cast<int32_t*>(scratch + l.list);
    Slot* slots = reinterpret_cast<Slot*>(scratch + l.slot);
    hipLaunchKernelGGL(lists_kernel, dim3((unsigned)q.E), dim3(kListThreads), 0, stream, q.ids, (int)(q.M * q.T), (int)q.E,
                       16 * l.mr, list, slots, l.slots);
    MoeTileArgs up{}, down{};
    up.p.x = q.x;
    up.p.packed = q.gate_up;
    up.p.K = (int)q.K;
    up.p.N = (int)(2 * q.F);
    up.p.F = (int)q.F;
    up.p.tiles_m = l.slots;
    up.p.tiles_n = (int)((q.F + kProductColumns / 2 - 1) / (kProductColumns / 2));
    up.p.splits = 1;
    up.p.rows = list;
    up.p.row_div = (int)q.T;
    up.slots = slots;
    up.stride = q.gate_up_stride;
    up.h = reinterpret_cast<uint16_t*>(scratch + l.h);
    up.act = q.act;
    down.p.x = up.h;
    down.p.packed = q.down;
    down.p.K = (int)q.F;
    down.p.N = (int)q.K;
    down.p.n_end = (int)q.K;
    down.p.tiles_m = l.slots;
    down.p.tiles_n = (int)((q.K + kProductColumns - 1) / kProductColumns);
    down.p.splits = 1;
    down.p.rows = list;
    down.slots = slots;
    down.stride = q.down_stride;
    down.out = reinterpret_cast<float*>(scratch + l.out);
    const int sub = units_per_block(q.G);
    if (q.bf16) launch_typed<true>(l.mr, sub, up, down, stream);
    else launch_typed<false>(l.mr, sub, up, down, stream);
    const int64_t chunks = q.M * (q.K / 8);
    const dim3 grid((unsigned)((chunks + 255) / 256));
    if (q.bf16) hipLaunchKernelGGL((join_kernel<true>), grid, dim3(256), 0, stream, down.out, q.ids, q.weights, q.residual, q.y, chunks, (int)q.K, (int)q.E, (int)q.T);
    else hipLaunchKernelGGL((join_kernel<false>), grid, dim3(256), 0, stream, down.out, q.ids, q.weights, q.residual, q.y, chunks, (int)q.K, (int)q.E, (int)q.T);
    return hipGetLastError();
}

}  // namespace w4a16
