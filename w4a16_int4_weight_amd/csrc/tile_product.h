// The forward product of the training and scoring operators: one workgroup's tile of
// x . W from the packed layout, left in registers as unrounded fp32 for the operator's
// own epilogue (activation, softmax statistics, probabilities).
//
// Mathematics. Per metadata unit (min(G, 128) rows) the tile is s (T - (b + z) X): the
// matrix cores form T = sum x (b + q) on operands that hold the codes themselves
// (b + q exactly: a code masked into the mantissa of b = 128 in bf16; in fp16
// 1024 + q - (1024 + z) is exact in 16 bits and leaves q - z, so b + z is 0 there), X is
// the sum of the same activations, and s and z enter in fp32. No weight is rounded to 16
// bits, so a logit carries fp32 error only. (A loss in fp32 needs that: with (q - z) s
// rounded to bf16 each logit is off by 2^-9 / sqrt(3) of its size, 100 times more than
// the sum itself loses.) It also costs less than rounding: 7 vector instructions decode
// 8 codes against 23 for fp32 fused multiply-adds and a pack, and the scale takes 8 per
// 16 x 16 tile of a 128-row block.
//
// Workgroup: W waves side by side along N, each owning CBW column blocks and all 16 MR
// rows. Per 128-row block of K an LDS ring holds the activations (16-byte chunks
// XOR-swizzled by row) and the waves' packed codes, filled by direct global -> LDS
// copies; a wave decodes its codes of the block into registers once and runs through
// its MR row fragments with them, so each weight is decoded once per 16 MR rows.
// X is summed by wave r for fragment r while it multiplies, passed on through LDS and
// taken off one block later, behind the barrier that the ring needs anyway.
#pragma once

#include <stddef.h>

#include "device_common.h"
#include "split_k.h"

namespace w4a16 {

struct ProductArgs {
    const uint16_t* x;
    const uint8_t* packed;
    int M, K;
    int N;                  // columns of the weight
    int F;                  // gated: columns of one half (N = 2 F)
    int n_begin, n_end;     // not gated: the columns of this launch (n_begin % 16 == 0)
    int tiles_m, tiles_n, splits;
    uint32_t* counters;     // K split: tile counters and partial tiles
    float* partials;
};

constexpr int kProductXcds = 8;

// Workgroup id -> tile. Ids id, id + 8, ... run on one XCD: it takes every 8th column
// tile and walks the row tiles of one in groups of 8, so that its L2 serves the codes of
// few column tiles and the activations of few row tiles at a time.
__device__ __forceinline__ bool product_tile(const ProductArgs& a, int id, int* m_tile, int* n_tile, int* split) {
    const int x = id % kProductXcds;
    int local = id / kProductXcds;
    *split = local % a.splits;
    local /= a.splits;
    const int per = (a.tiles_n + kProductXcds - 1) / kProductXcds;   // column tiles of an XCD
    const int chunk = local / (8 * per);
    const int gm = a.tiles_m - 8 * chunk < 8 ? a.tiles_m - 8 * chunk : 8;
    const int rem = local - chunk * 8 * per;
    *m_tile = 8 * chunk + rem % gm;
    *n_tile = (rem / gm) * kProductXcds + x;
    return *n_tile < a.tiles_n;
}
inline int64_t product_ids(int tiles_m, int tiles_n, int splits) {
    return (int64_t)tiles_m * ((tiles_n + kProductXcds - 1) / kProductXcds) * kProductXcds * splits;
}

template <bool kBF16>
__device__ __forceinline__ float product_dot2(uint32_t a, uint32_t b, float c) {
    if constexpr (kBF16)
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), c, false);
    else
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, a), __builtin_bit_cast(f16x2, b), c, false);
}

template <bool kBF16_, int MR_, int CBW_, int W_, int kSub_, bool kGated_>
struct TileProduct {
    static constexpr bool kBF16 = kBF16_, kGated = kGated_;
    static constexpr int MR = MR_, CBW = CBW_, W = W_, kSub = kSub_;
    static constexpr int BM = 16 * MR;
    static constexpr int HB = kGated ? CBW / 2 : CBW;      // column blocks of a wave per half
    static constexpr int BN = 16 * HB * W;                 // output columns of the tile
    static constexpr int kThreads = 64 * W;
    static constexpr int kXSlabs = BM / 4;                 // 1 KiB slabs (4 rows) of the x stage
    static constexpr int kSlabs = (kXSlabs + W - 1) / W;   // copied per wave (a wave without one of its own repeats one)
    static constexpr int kDma = kSlabs + CBW;              // copies per wave and stage
    static constexpr int kMeta = CBW * kSub;               // + these every 4th stage
    struct Stage {
        uint4 x[BM * 16];                 // chunk j of row r at chunk j ^ (r % 16)
        uint4 w[W * CBW * 64];
    };
    // two stages where three do not fit beside the metadata
    static constexpr int kStages = 3 * sizeof(Stage) + 2 * W * kMeta * 256 + 8192 <= 160 * 1024 ? 3 : 2;
    struct Shared {
        Stage ring[kStages];
        uint32_t meta[2][W][64 * kMeta];  // [column of the wave][unit of 4 row blocks]
        float xsum[2][kSub][BM];
    };
    static_assert(!kGated || CBW % 2 == 0, "a gated wave holds both halves");
    static_assert(MR <= W, "wave r sums the activations of fragment r");
    static_assert(sizeof(Shared) <= 160 * 1024, "LDS");

    // weight column of lane column c in block j of wave w (clamped into the weight)
    static __device__ __forceinline__ int column(const ProductArgs& a, int n_tile, int w, int j, int c) {
        if constexpr (kGated) {
            const int f = ((n_tile * W + w) * HB + j % HB) * 16 + c;
            return (j < HB ? 0 : a.F) + (f < a.F ? f : a.F - 1);
        } else {
            const int n = a.n_begin + ((n_tile * W + w) * CBW + j) * 16 + c;
            const int last = (int)padded_cols(a.N) - 1;
            return n < last ? n : last;
        }
    }

    static __device__ __forceinline__ void run(const ProductArgs& a, Shared& sh, int m_tile, int n_tile, int split,
                                               f32x4 (&acc)[MR][CBW]) {
        const int K = a.K;
        const int KB = K / kRowsPerBlock;
        const int UW = (int)padded_units(K, kRowsPerBlock / kSub);
        const int tid = threadIdx.x;
        const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int lane = tid & 63;
        const int c = lane & 15;
        const int h = lane >> 4;
        const int kb_begin = (int)((int64_t)KB * split / a.splits);
        const int nkb = (int)((int64_t)KB * (split + 1) / a.splits) - kb_begin;
        const int m0 = m_tile * BM;
        const uint32_t ring_base = lds_addr(&sh.ring[0]);
        const uint32_t meta_base = lds_addr(&sh.meta[0][w][0]);

        // copies: wave-uniform bases and per-lane byte offsets. Rows past M read row M - 1
        // and columns past the last read the last: they feed outputs that are not used.
        const uint8_t* xbase = uniform_ptr(a.x + (size_t)m0 * K);
        uint32_t xoff[kSlabs];
        int xslab[kSlabs];
#pragma unroll
        for (int t = 0; t < kSlabs; ++t) {
            xslab[t] = (w * kSlabs + t) % kXSlabs;
            const int row = 4 * xslab[t] + (lane >> 4);
            const int m = m0 + row < a.M ? m0 + row : a.M - 1;
            xoff[t] = 2u * ((uint32_t)(m - m0) * (uint32_t)K + 8u * (uint32_t)((lane & 15) ^ (row & 15)));
        }
        const uint8_t* wbase[CBW];
        const uint8_t* mbase[CBW];
        uint32_t woff[CBW];
#pragma unroll
        for (int j = 0; j < CBW; ++j) {
            const int first = column(a, n_tile, w, j, 0);
            const int n = column(a, n_tile, w, j, c);
            wbase[j] = uniform_ptr(a.packed + (size_t)(first >> 4) * KB * kBlockBytes);
            woff[j] = (uint32_t)((n >> 4) - (first >> 4)) * (uint32_t)KB * kBlockBytes + 16u * (uint32_t)(16 * h + (n & 15));
            mbase[j] = uniform_ptr(a.packed + (size_t)K * padded_cols(a.N) / 2 + (size_t)first * UW * 4);
        }
        auto issue = [&](int t) {
            const int kb = kb_begin + t;
            const uint32_t st = ring_base + (uint32_t)(t % kStages) * (uint32_t)sizeof(Stage);
#pragma unroll
            for (int j = 0; j < CBW; ++j)
                dma16(wbase[j] + (size_t)kb * kBlockBytes, woff[j],
                      st + (uint32_t)offsetof(Stage, w) + (uint32_t)(w * CBW + j) * 1024u);
#pragma unroll
            for (int q = 0; q < kSlabs; ++q)
                dma16(xbase + (size_t)kb * kRowsPerBlock * 2, xoff[q], st + (uint32_t)xslab[q] * 1024u);
            if ((t & 3) == 0) {
                const uint32_t dst = meta_base + (uint32_t)((t >> 2) & 1) * (uint32_t)(W * kMeta * 256);
#pragma unroll
                for (int i = 0; i < kMeta; ++i) {
                    const int wi = 64 * i + lane;
                    const int cl = (wi / (4 * kSub)) & 15, u = wi % (4 * kSub);
                    const int j = i / kSub;
                    const int n = column(a, n_tile, w, j, cl);
                    const int first = column(a, n_tile, w, j, 0);
                    const int ua = kb * kSub + u < UW ? kb * kSub + u : UW - 1;
                    dma4(mbase[j], ((uint32_t)(n - first) * (uint32_t)UW + (uint32_t)ua) * 4u, dst + (uint32_t)i * 256u);
                }
            }
        };

#pragma unroll
        for (int r = 0; r < MR; ++r)
#pragma unroll
            for (int j = 0; j < CBW; ++j) acc[r][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        float szp[CBW][kSub];             // s (b + z) of the block before
        if constexpr (kBF16) {
#pragma unroll
            for (int j = 0; j < CBW; ++j)
#pragma unroll
                for (int u = 0; u < kSub; ++u) szp[j][u] = 0.f;
            for (int i = tid; i < kSub * BM; i += kThreads) (&sh.xsum[1][0][0])[i] = 0.f;
        }
        auto take_off = [&](int t, int r) {           // the zero points of block t, fragment r
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                const f32x4 X = *reinterpret_cast<const f32x4*>(&sh.xsum[t & 1][u][16 * r + 4 * h]);
#pragma unroll
                for (int j = 0; j < CBW; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[r][j][e] = fmaf(-szp[j][u], X[e], acc[r][j][e]);
            }
        };

        issue(0);
        if constexpr (kStages == 3) {
            if (nkb > 1) issue(1);
        }
        for (int t = 0; t < nkb; ++t) {
            if (kStages == 2 || t + 1 >= nkb) wait_vmcnt<0>();
            else if (((t + 1) & 3) == 0) wait_vmcnt<kDma + kMeta>();
            else wait_vmcnt<kDma>();
            wait_lgkmcnt0();
            lds_barrier();
            if (t + kStages - 1 < nkb) issue(t + kStages - 1);

            const Stage& st = sh.ring[t % kStages];
            uint4 b[CBW][4];
            float s[CBW][kSub], sz[CBW][kSub];
#pragma unroll
            for (int j = 0; j < CBW; ++j) {
                const uint4 q = st.w[(w * CBW + j) * 64 + lane];
                uint32_t md[kSub];
#pragma unroll
                for (int u = 0; u < kSub; ++u) {
                    md[u] = sh.meta[(t >> 2) & 1][w][(16 * j + c) * 4 * kSub + (t & 3) * kSub + u];
                    s[j][u] = half_bits_to_f32<kBF16>(md[u] & 0xFFFFu);
                    sz[j][u] = s[j][u] * (128.f + (float)((md[u] >> 16) & 0xFu));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t d = i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w;
                    uint32_t p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = ((d >> (4 * e)) & 0x000F000Fu) | Magic<kBF16>::kBase2;
                    if constexpr (!kBF16) {
                        const _Float16 zb = (_Float16)(1024.0f + (float)((md[(i * kSub) / 4] >> 16) & 0xFu));
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            p[e] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, p[e]) - f16x2{zb, zb});
                    }
                    b[j][i] = make_uint4(p[0], p[1], p[2], p[3]);
                }
            }
#pragma unroll
            for (int r = 0; r < MR; ++r) {
                uint4 f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = st.x[(16 * r + c) * 16 + ((4 * i + h) ^ c)];
                if constexpr (kBF16) {
                    if (r == w) {
#pragma unroll
                        for (int u = 0; u < kSub; ++u) {
                            float X = 0.f;
#pragma unroll
                            for (int i = 0; i < 4 / kSub; ++i) {
                                const uint4 v = f[u * (4 / kSub) + i];
                                X = product_dot2<true>(v.x, 0x3F803F80u, X);
                                X = product_dot2<true>(v.y, 0x3F803F80u, X);
                                X = product_dot2<true>(v.z, 0x3F803F80u, X);
                                X = product_dot2<true>(v.w, 0x3F803F80u, X);
                            }
                            X += __shfl_xor(X, 16);
                            X += __shfl_xor(X, 32);
                            if (h == 0) sh.xsum[t & 1][u][16 * r + c] = X;
                        }
                    }
                    take_off(t + 1, r);               // block t - 1 (the same slot parity)
                }
#pragma unroll
                for (int j = 0; j < CBW; ++j) {
#pragma unroll
                    for (int u = 0; u < kSub; ++u) {
                        f32x4 T = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int i = 0; i < 4 / kSub; ++i)
                            T = mfma16x16x32<kBF16>(f[u * (4 / kSub) + i], b[j][u * (4 / kSub) + i], T);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[r][j][e] = fmaf(s[j][u], T[e], acc[r][j][e]);
                    }
                }
            }
            if constexpr (kBF16) {
#pragma unroll
                for (int j = 0; j < CBW; ++j)
#pragma unroll
                    for (int u = 0; u < kSub; ++u) szp[j][u] = sz[j][u];
            }
        }
        if constexpr (kBF16) {
            wait_lgkmcnt0();
            lds_barrier();
#pragma unroll
            for (int r = 0; r < MR; ++r) take_off(nkb - 1, r);
        }
        // the ring may be reused by the caller: every wave is done with it
        wait_lgkmcnt0();
        lds_barrier();
    }
};

}  // namespace w4a16
