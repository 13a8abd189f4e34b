// Gated feed-forward block on one packed [K, 2F] weight (gate columns 0 .. F-1, up
// columns F .. 2F-1, as checkpoints fuse them):
//
//   forward   h  = a(g) u,             g = x Wg, u = x Wu
//   backward  dg = dh u a'(g), du = dh a(g);   dx = dg Wg^T + du Wu^T
//
// Both projections of an output element sit in one lane: a wave owns HB gate column
// blocks and the HB matching up blocks, so g and u never leave its registers and the
// block costs one product and one pass over x. The backward recomputes them (keeping
// them would take 4 F bytes a token and round them to 16 bits), writes dg and du to the
// workspace in fp16, scaled by a power of two for each row of a tile, and one product with
// W^T follows, which brings a row's tiles to one scale (gemm_grad.hip): rounded to bf16 they
// would be off by as much as the result's own rounding, and fp32 took 8 F bytes a row.
//
// Measured: 512 rows x 2048 x 13312 37 us (757 TFLOP/s; 208 tiles, one round), 4096 rows 242
// us (923); the backward of 4096 rows 557 us (802 over both products; 525 where every call
// has the same inputs), fp16 503. Bound as tile_product.h has it: matrix cores 0.35 busy,
// vector units 0.39 with other work; a tile's start and end, which no other workgroup of its
// compute unit covers, take a tenth.
#include "device_common.h"
#include "gate.h"
#include "launch.h"
#include "tile_product.h"

namespace w4a16 {
namespace {

constexpr int kTargetWorkgroups = 256;      // one per compute unit

struct GatedArgs {
    ProductArgs p;
    uint16_t* h;            // forward: [M, F]
    const uint16_t* dh;     // backward: [M, F]
    uint16_t* d;            // backward: [M, 2F] fp16, dg then du
    uint16_t* d_rest;       // NULL or what d's rounding leaves
    float* tops;            // [column tiles][M] largest |d| of a row
    int act;
};

// The tile's results go through LDS and leave as whole rows. A backward forms dg and du in
// the accumulators, takes each row's largest over the workgroup's columns, and rounds them
// once, scaled by its power of two.
template <class P, bool kGrad, int kAct>
__device__ __forceinline__ void gated_epilogue(const GatedArgs& a, typename P::Shared& sh, int m0, int f0,
                                               f32x4 (&acc)[P::MR][P::CBW]) {
    constexpr int BM = P::BM, BN = P::BN, HB = P::HB;
    constexpr int kRow = BN * 2 + 16;                        // bytes of a tile row, padded
    constexpr int kChunks = BN / 8;
    static_assert((kGrad ? 2 : 1) * BM * kRow + P::W * BM * 4 <= (int)sizeof(typename P::Shared), "the output tiles fit in LDS");
    const int tid = threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
    const int c = lane & 15, h = lane >> 4;
    const int M = a.p.M, F = a.p.F;
    uint8_t* t0 = reinterpret_cast<uint8_t*>(&sh);
    uint8_t* t1 = t0 + BM * kRow;
    float* red = reinterpret_cast<float*>(t1 + BM * kRow);   // backward: [W][BM]
    auto place = [&](int r, int j) { return (16 * r + c) * kRow + 2 * (16 * (w * HB + j) + 4 * h); };     // 4 columns of a row
    if constexpr (!kGrad) {
#pragma unroll
        for (int r = 0; r < P::MR; ++r)
#pragma unroll
            for (int j = 0; j < HB; ++j) {
                float o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float g = acc[r][j][e];
                    float slope;
                    o[e] = g * gate_prob<kAct>(g, &slope) * acc[r][j + HB][e];
                }
                *reinterpret_cast<uint2*>(t0 + place(r, j)) = make_uint2(pack2_rne<P::kBF16>(o[0], o[1]), pack2_rne<P::kBF16>(o[2], o[3]));
            }
    } else {
        // dh of the lane's 4 columns, which lie wholly inside or outside (F % 8 == 0)
        uint2 dv[P::MR][HB];
#pragma unroll
        for (int r = 0; r < P::MR; ++r)
#pragma unroll
            for (int j = 0; j < HB; ++j) {
                const int m = m0 + 16 * r + c, f = f0 + 16 * (w * HB + j) + 4 * h;
                const uint2 v = *reinterpret_cast<const uint2*>(a.dh + (size_t)(m < M ? m : M - 1) * F + (f < F ? f : F - 4));
                dv[r][j] = m < M && f < F ? v : make_uint2(0u, 0u);
            }
#pragma unroll
        for (int r = 0; r < P::MR; ++r) {
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < HB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float g = acc[r][j][e], u = acc[r][j + HB][e];
                    const uint32_t dw = e < 2 ? dv[r][j].x : dv[r][j].y;
                    const float d = half_bits_to_f32<P::kBF16>(e & 1 ? dw >> 16 : dw & 0xFFFFu);
                    float slope;
                    const float pr = gate_prob<kAct>(g, &slope);
                    acc[r][j][e] = d * u * fmaf(g, slope, pr);
                    acc[r][j + HB][e] = d * (g * pr);
                    top = fmaxf(top, fmaxf(fabsf(acc[r][j][e]), fabsf(acc[r][j + HB][e])));
                }
            top = quarter_max(top);
            if (h == 0) red[w * BM + 16 * r + c] = top;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < P::MR; ++r) {
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < P::W; ++i) top = fmaxf(top, red[i * BM + 16 * r + c]);
            const int m = m0 + 16 * r + c;
            if (w == 0 && h == 0 && m < M) a.tops[(size_t)(f0 / BN) * M + m] = top;
            const float by = power_of_two(scale_exponent(top, kGradTop));
#pragma unroll
            for (int j = 0; j < P::CBW; ++j) acc[r][j] *= by;
        }
    }
    // (an fp16 backward's second pass: what the first one's rounding left)
    constexpr bool kRest = kGrad && !P::kBF16;
    for (int pass = 0; pass < (kRest && a.d_rest ? 2 : 1); ++pass) {
        if constexpr (kGrad) {
            if (pass) __syncthreads();
#pragma unroll
            for (int r = 0; r < P::MR; ++r)
#pragma unroll
                for (int j = 0; j < P::CBW; ++j) {
                    const f32x4 v = acc[r][j];
                    const uint2 o = make_uint2(pack2_rne<false>(v[0], v[1]), pack2_rne<false>(v[2], v[3]));
                    *reinterpret_cast<uint2*>((j < HB ? t0 : t1) + place(r, j % HB)) = o;
                    if constexpr (kRest) acc[r][j] = f32x4{v[0] - f16_bits_to_f32(o.x & 0xFFFFu), v[1] - f16_bits_to_f32(o.x >> 16),
                                      v[2] - f16_bits_to_f32(o.y & 0xFFFFu), v[3] - f16_bits_to_f32(o.y >> 16)};
                }
        }
        __syncthreads();
        for (int q = tid; q < BM * kChunks; q += P::kThreads) {
            const int row = q / kChunks, ch = q % kChunks;
            const int m = m0 + row, f = f0 + 8 * ch;
            if (m >= M || f >= F) continue;
            const uint4 v = *reinterpret_cast<const uint4*>(t0 + row * kRow + 16 * ch);
            if constexpr (!kGrad) {
                *reinterpret_cast<uint4*>(a.h + (size_t)m * F + f) = v;
            } else {
                uint16_t* d = pass ? a.d_rest : a.d;
                *reinterpret_cast<uint4*>(d + (size_t)m * 2 * F + f) = v;
                *reinterpret_cast<uint4*>(d + (size_t)m * 2 * F + F + f) = *reinterpret_cast<const uint4*>(t1 + row * kRow + 16 * ch);
            }
        }
    }
}

template <class P, bool kGrad>
__global__ __launch_bounds__(P::kThreads) void gated_kernel(const GatedArgs a) {
    __shared__ typename P::Shared sh;
    int m_tile, n_tile, split;
    if (!product_tile(a.p, (int)blockIdx.x, &m_tile, &n_tile, &split)) return;
    f32x4 acc[P::MR][P::CBW];
    P::run(a.p, sh, m_tile, n_tile, split, acc);
    if (a.p.splits > 1 && !reduce_splits<P::MR, P::CBW, P::W>(acc, a.p.counters, a.p.partials,
                                                              m_tile * a.p.tiles_n + n_tile, split, a.p.splits))
        return;
    const int m0 = m_tile * P::BM, f0 = n_tile * P::BN;
    if (a.act == 0) gated_epilogue<P, kGrad, 0>(a, sh, m0, f0, acc);
    else if (a.act == 1) gated_epilogue<P, kGrad, 1>(a, sh, m0, f0, acc);
    else gated_epilogue<P, kGrad, 2>(a, sh, m0, f0, acc);
}

// Workgroups 0 .. kScaleParts - 1: the weight's largest |scale|, a part each. The others: 16
// rows each, 16 threads a row: their largest |d| over the column tiles, and what brings each
// tile's values to the row's scale, two fp16 of one power of two.
template <bool kBF16>
__device__ __forceinline__ void scale_part(const uint32_t* __restrict__ meta, int64_t words, float* __restrict__ scale_max) {
    __shared__ float wave_top[4];
    const int tid = (int)threadIdx.x;
    float top = 0.f;
#pragma unroll 4
    for (int64_t k = (int64_t)blockIdx.x * 256 + tid; 4 * k < words; k += kScaleParts * 256) {
        const uint4 v = *reinterpret_cast<const uint4*>(meta + 4 * k);
        for (const uint32_t q : {v.x, v.y, v.z, v.w}) top = fmaxf(top, fabsf(half_bits_to_f32<kBF16>(q & 0xFFFFu)));
    }
    for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
    if ((tid & 63) == 0) wave_top[tid >> 6] = top;
    __syncthreads();
    if (tid == 0) scale_max[blockIdx.x] = fmaxf(fmaxf(wave_top[0], wave_top[1]), fmaxf(wave_top[2], wave_top[3]));
}
template <bool kBF16>
__global__ __launch_bounds__(256) void tops_kernel(const float* __restrict__ tops, int tiles, const uint32_t* __restrict__ meta,
                                                   int64_t words, int M, float* __restrict__ rowmax,
                                                   uint32_t* __restrict__ factor, float* __restrict__ scale_max) {
    if ((int)blockIdx.x < kScaleParts) {
        scale_part<kBF16>(meta, words, scale_max);
        return;
    }
    __shared__ float red[16][17];
    const int tid = (int)threadIdx.x, i = tid & 15, g = tid >> 4;
    const int m = ((int)blockIdx.x - kScaleParts) * 16 + i, mc = m < M ? m : M - 1;
    float top = 0.f;
#pragma unroll 4
    for (int t = g; t < tiles; t += 16) top = fmaxf(top, tops[(size_t)t * M + mc]);
    red[g][i] = top;
    __syncthreads();
    for (int k = 0; k < 16; ++k) top = fmaxf(top, red[k][i]);
    if (m >= M) return;
    if (g == 0) rowmax[m] = top;
    const int row = scale_exponent(top, kGradTop);
    for (int t = g; t < tiles; t += 16) {
        const float own = tops[(size_t)t * M + m];
        factor[(size_t)t * M + m] = own > 0.f ? 0x10001u * f32_to_half_bits<false>(power_of_two(row - scale_exponent(own, kGradTop))) : 0u;
    }
}

// The same after the small product, whose d is fp32: one row and 2048 of its values a
// workgroup, rounded to fp16 at the row's scale.
template <bool kBF16>
__global__ __launch_bounds__(256) void convert_kernel(const float* __restrict__ tops, int tiles, const uint32_t* __restrict__ meta,
                                                      int64_t words, int M, int N, const float* __restrict__ d32,
                                                      float* __restrict__ rowmax, uint16_t* __restrict__ d,
                                                      uint16_t* __restrict__ d_rest, float* __restrict__ scale_max) {
    if ((int)blockIdx.x < kScaleParts) {
        scale_part<kBF16>(meta, words, scale_max);
        return;
    }
    __shared__ float wave_top[4];
    const int tid = (int)threadIdx.x;
    const int m = ((int)blockIdx.x - kScaleParts) % M, n = 8 * ((((int)blockIdx.x - kScaleParts) / M) * 256 + tid);
    float top = tid < tiles ? tops[(size_t)tid * M + m] : 0.f;            // tiles <= 256
    for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
    if ((tid & 63) == 0) wave_top[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(wave_top[0], wave_top[1]), fmaxf(wave_top[2], wave_top[3]));
    if (tid == 0) rowmax[m] = top;
    if (n >= N) return;
    const float by = power_of_two(scale_exponent(top, kGradTop));
    const f32x4* p = reinterpret_cast<const f32x4*>(d32 + (size_t)m * N + n);
    const f32x4 lo = p[0] * by, hi = p[1] * by;
    const uint4 o = make_uint4(pack2_rne<false>(lo[0], lo[1]), pack2_rne<false>(lo[2], lo[3]), pack2_rne<false>(hi[0], hi[1]),
                               pack2_rne<false>(hi[2], hi[3]));
    *reinterpret_cast<uint4*>(d + (size_t)m * N + n) = o;
    if (!d_rest) return;
    auto rest = [](float a, float b, uint32_t v) {
        return pack2_rne<false>(a - f16_bits_to_f32(v & 0xFFFFu), b - f16_bits_to_f32(v >> 16));
    };
    *reinterpret_cast<uint4*>(d_rest + (size_t)m * N + n) =
        make_uint4(rest(lo[0], lo[1], o.x), rest(lo[2], lo[3], o.y), rest(hi[0], hi[1], o.z), rest(hi[2], hi[3], o.w));
}

template <bool kBF16, int MR, int kSub, bool kGrad>
void launch_cfg(GatedArgs& a, hipStream_t s) {
    using P = TileProduct<kBF16, MR, kProductColumns / 128, 8, kSub, true>;
    const int64_t ids = product_ids(a.p.tiles_m, a.p.tiles_n, a.p.splits);
    hipLaunchKernelGGL((gated_kernel<P, kGrad>), dim3((unsigned)ids), dim3(P::kThreads), 0, s, a);
}

template <bool kBF16, bool kGrad>
void launch_typed(const ProductPlan& p, GatedArgs& a, hipStream_t s) {
    if (p.sub == 4) {
        if (p.mr == 1) launch_cfg<kBF16, 1, 4, kGrad>(a, s);
        else if (p.mr == 2) launch_cfg<kBF16, 2, 4, kGrad>(a, s);
        else launch_cfg<kBF16, 4, 4, kGrad>(a, s);
    } else if (p.sub == 2) {
        if (p.mr == 1) launch_cfg<kBF16, 1, 2, kGrad>(a, s);
        else if (p.mr == 2) launch_cfg<kBF16, 2, 2, kGrad>(a, s);
        else launch_cfg<kBF16, 4, 2, kGrad>(a, s);
    } else if (p.mr == 1) launch_cfg<kBF16, 1, 1, kGrad>(a, s);
    else if (p.mr == 2) launch_cfg<kBF16, 2, 1, kGrad>(a, s);
    else if (p.mr == 4) launch_cfg<kBF16, 4, 1, kGrad>(a, s);
    else launch_cfg<kBF16, 8, 1, kGrad>(a, s);
}

}  // namespace

// Tile shape: 128, 64 or 32 rows by 256 columns of the weight, whose rounds over the compute
// units cost least, by area over the rate each shape was measured at with every compute unit
// busy (333 rows x 1024 x 5456: 132 tiles of 64 rows 17.0 us, 242 of 32 rows 13.4; 100 rows
// x 2048 x 13312: 18.6 against 20.8). Outputs of few tiles split K over workgroups, at least
// 4 row blocks each.
ProductPlan plan_product(int64_t M, int64_t K, int64_t cols, int64_t G, bool gated) {
    ProductPlan p{};
    if (gated && small_product(M, K)) return p;          // no tiles, no workspace
    p.sub = units_per_block(G);
    const int64_t KB = K / kRowsPerBlock;
    auto splits_of = [&](int64_t tiles) -> int64_t {
        if (tiles >= kTargetWorkgroups / 2 || KB < 8) return 1;
        const int64_t want = kTargetWorkgroups / tiles, most = KB / 4;
        return want < most ? want : most;
    };
    struct Shape { int mr; double rate; };
    // finer groups scale each fragment 2 or 4 times; their 128-row tile does not fit in LDS
    static constexpr Shape kShapes[] = {{8, 0.85}, {4, 0.7}, {2, 0.5}};
    if (M <= 16) {
        p.mr = 1;
    } else {
        double best = 0.0;
        for (const Shape& c : kShapes) {
            if (c.mr == 8 && (p.sub > 1 || M <= 64)) continue;
            const int64_t tm = (M + 16 * c.mr - 1) / (16 * c.mr);
            const int64_t tn = (cols + kProductColumns - 1) / kProductColumns;
            const int64_t tiles = tm * tn, rounds = (tiles + kTargetWorkgroups - 1) / kTargetWorkgroups;
            const int64_t splits = splits_of(tiles);
            // a 128-row tile takes 2.1 us a row block; a tile's start and end as much as one,
            // a split's meeting by its partial tiles
            const double cost = (double)rounds * ((double)KB / (double)splits * c.mr * 2.0 / c.rate + 20.0 +
                                                  (splits > 1 ? 4.0 * c.mr * (double)splits : 0.0));
            if (best == 0.0 || cost < best) {
                best = cost;
                p.mr = c.mr;
            }
        }
    }
    constexpr int64_t width = kProductColumns;
    p.tiles_m = (int)((M + 16 * p.mr - 1) / (16 * p.mr));
    p.tiles_n = (int)(gated ? (cols / 2 + width / 2 - 1) / (width / 2) : (cols + width - 1) / width);
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    static_assert(kTargetWorkgroups / 2 <= kMaxSplitTiles, "split tiles must fit the counter region");
    p.splits = (int)splits_of(tiles);
    p.partial_bytes = p.splits > 1 ? (size_t)p.splits * (size_t)tiles * (size_t)(16 * p.mr) * (size_t)width * 4 : 0;
    return p;
}

int gated_tiles(int64_t M, int64_t K, int64_t F, int64_t G) {
    return small_product(M, K) ? small_workgroups(F / 8) : plan_product(M, K, 2 * F, G, true).tiles_n;
}

int gated_tile_columns(int64_t M, int64_t K) {
    return small_product(M, K) ? 0 : kProductColumns / 2;
}

hipError_t launch_gated_tops(const GatedCall& q, float* rowmax, uint32_t* factor, float* scale_max, hipStream_t stream) {
    const int64_t N = 2 * q.F;
    const uint32_t* meta = reinterpret_cast<const uint32_t*>(q.packed + (size_t)q.K * padded_cols(N) / 2);
    const int64_t words = padded_cols(N) * padded_units(q.K, q.G);
    const int tiles = gated_tiles(q.M, q.K, q.F, q.G);
    const dim3 block(256);
    if (small_product(q.M, q.K)) {
        const dim3 grid((unsigned)(kScaleParts + q.M * ((N + 2047) / 2048)));
        if (q.bf16) hipLaunchKernelGGL((convert_kernel<true>), grid, block, 0, stream, q.tops, tiles, meta, words, (int)q.M, (int)N, q.d32, rowmax, q.d, q.d_rest, scale_max);
        else hipLaunchKernelGGL((convert_kernel<false>), grid, block, 0, stream, q.tops, tiles, meta, words, (int)q.M, (int)N, q.d32, rowmax, q.d, q.d_rest, scale_max);
    } else {
        const dim3 grid((unsigned)(kScaleParts + (q.M + 15) / 16));
        if (q.bf16) hipLaunchKernelGGL((tops_kernel<true>), grid, block, 0, stream, q.tops, tiles, meta, words, (int)q.M, rowmax, factor, scale_max);
        else hipLaunchKernelGGL((tops_kernel<false>), grid, block, 0, stream, q.tops, tiles, meta, words, (int)q.M, rowmax, factor, scale_max);
    }
    return hipGetLastError();
}

hipError_t launch_gated(const GatedCall& q, hipStream_t stream) {
    if (small_product(q.M, q.K)) return launch_gated_small(q, stream);
    const ProductPlan p = plan_product(q.M, q.K, 2 * q.F, q.G, true);
    GatedArgs a{};
    a.p.x = q.x;
    a.p.packed = q.packed;
    a.p.M = (int)q.M;
    a.p.K = (int)q.K;
    a.p.N = (int)(2 * q.F);
    a.p.F = (int)q.F;
    a.p.tiles_m = p.tiles_m;
    a.p.tiles_n = p.tiles_n;
    a.p.splits = p.splits;
    a.p.counters = q.counters;
    a.p.partials = q.partials;
    a.h = q.h;
    a.dh = q.dh;
    a.d = q.d;
    a.d_rest = q.d_rest;
    a.tops = q.tops;
    a.act = q.act;
    if (q.d) {
        if (q.bf16) launch_typed<true, true>(p, a, stream);
        else launch_typed<false, true>(p, a, stream);
    } else {
        if (q.bf16) launch_typed<true, false>(p, a, stream);
        else launch_typed<false, false>(p, a, stream);
    }
    return hipGetLastError();
}

}  // namespace w4a16
