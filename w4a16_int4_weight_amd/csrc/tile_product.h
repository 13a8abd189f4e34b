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
// What bounds it at 128 rows, by counters (4096 x 2048 x 32768 with the loss's epilogue): the
// matrix cores are busy 0.37 of the time, the vector units with other work (4 instructions
// an MFMA, epilogue included) 0.39, both at once 0.14, so that for the rest, 0.38, a SIMD
// issues neither: its two waves wait for each other at the barrier of a row block or for a
// tile's start and end. Groups of 32: 11 instructions an MFMA, matrix cores 0.11.
// Measured on 4096 x 2048 x 131072 with the loss's epilogue: 3530 us with the decoding and
// scaling left to the compiler's order, 2410 us in the order below and with the zero points
// on the matrix cores (bf16, 912 TFLOP/s; fp16, whose codes lose their zero point in 16 bits,
// 2230 us).
// X is summed by wave r for fragment r, passed on through LDS and taken off every fourth
// row block. The MFMA takes the weights as its first operand, so a lane holds four adjacent
// columns of one row.
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
    const int32_t* rows;    // gathered tiles: rows of x (RowsInOrder does not read it)
    int row_div;
};

// Which rows of x a tile's rows are: those of [m0, M) in order, the last one repeated. at() is
// relative to base().
struct RowsInOrder {
    static __device__ __forceinline__ const uint16_t* base(const ProductArgs& a, int m0) { return a.x + (size_t)m0 * a.K; }
    static __device__ __forceinline__ int at(const ProductArgs& a, int m0, int row) {
        return (m0 + row < a.M ? m0 + row : a.M - 1) - m0;
    }
};

constexpr int kProductXcds = 8;

// Workgroup id -> tile. Ids id, id + 8, ... run on one XCD, which takes a contiguous eighth
// of the tiles in an order that walks 8 row tiles of a column tile, then the next column
// tile's: its L2 serves the codes of few column tiles and the activations of few row tiles
// at a time. (Whole column tiles dealt to the XCDs left some with a round more than others:
// 242 tiles, 22 columns wide, took 25 us, two rounds, against 17.)
__device__ __forceinline__ bool product_tile(const ProductArgs& a, int id, int* m_tile, int* n_tile, int* split) {
    const int x = id % kProductXcds, total = a.tiles_m * a.tiles_n * a.splits;
    const int at = (int)((int64_t)total * x / kProductXcds) + id / kProductXcds;
    if (at >= (int)((int64_t)total * (x + 1) / kProductXcds)) return false;
    *split = at % a.splits;
    const int tile = at / a.splits;
    const int chunk = tile / (8 * a.tiles_n);
    const int gm = a.tiles_m - 8 * chunk < 8 ? a.tiles_m - 8 * chunk : 8;
    const int rem = tile - chunk * 8 * a.tiles_n;
    *m_tile = 8 * chunk + rem % gm;
    *n_tile = rem / gm;
    return true;
}
inline int64_t product_ids(int tiles_m, int tiles_n, int splits) {
    return ((int64_t)tiles_m * tiles_n * splits + kProductXcds - 1) / kProductXcds * kProductXcds;
}

template <bool kBF16>
__device__ __forceinline__ float product_dot2(uint32_t a, uint32_t b, float c) {
    if constexpr (kBF16)
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), c, false);
    else
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, a), __builtin_bit_cast(f16x2, b), c, false);
}

// sum and maximum over the four lanes c, c + 16, c + 32, c + 48, left in all four
__device__ __forceinline__ float quarter_sum(float v) {
    typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
    u32x2_t p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}
__device__ __forceinline__ float quarter_max(float v) {
    typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
    u32x2_t p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
    p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}

// kScaleBF16: the type of the weight's scales, where it is not that of x.
template <bool kBF16_, int MR_, int CBW_, int W_, int kSub_, bool kGated_, class Rows = RowsInOrder, bool kScaleBF16 = kBF16_>
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
    static constexpr int kUnits = 4 * kSub;                // metadata units of a group of 4 row blocks
    // Stages t and t + 1 are read in turn t, t + 2 is on its way. (Rings of 4 to 6 stages, where
    // they fit, measured the same for 64-row tiles and 15% slower for 16-row ones, which then
    // run one workgroup a compute unit instead of two.)
    static constexpr int kStages = 3;
    static constexpr int kMetaSlots = 2;                   // a group's is read until its last block is done
    struct Stage {
        uint4 x[BM * 16];                 // chunk j of row r at chunk j ^ (r % 16)
        uint4 w[W * CBW * 64];
    };
    struct Shared {
        Stage ring[kStages];
        uint32_t meta[kMetaSlots][W][64 * kMeta];  // [group of 4 row blocks][column of the wave][its units]
        float scale[W][kSub][16 * CBW];   // one row block's, passed between the lanes of a wave
        float xsum[2][kUnits][BM];        // [group % 2][unit]
    };
    static_assert(!kGated || CBW % 2 == 0, "a gated wave holds both halves");
    static_assert(MR <= W, "wave r sums the activations of fragment r");
    static_assert(sizeof(Shared) + 16 <= 160 * 1024, "LDS");

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

    // one row block's decoded operands and scales
    struct Operands {
        uint4 b[CBW][4];
        f32x4 s[CBW][kSub];               // columns 4 h .. 4 h + 3 of block j
    };

    // acc[r][j] register e of lane (c, h): row 16 r + c, column 16 j + 4 h + e of the wave
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
        const uint8_t* xbase = uniform_ptr(Rows::base(a, m0));
        uint32_t xoff[kSlabs];
        int xslab[kSlabs];
#pragma unroll
        for (int t = 0; t < kSlabs; ++t) {
            xslab[t] = (w * kSlabs + t) % kXSlabs;
            const int row = 4 * xslab[t] + (lane >> 4);
            xoff[t] = 2u * ((uint32_t)Rows::at(a, m0, row) * (uint32_t)K + 8u * (uint32_t)((lane & 15) ^ (row & 15)));
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
                const uint32_t dst = meta_base + (uint32_t)((t >> 2) % kMetaSlots) * (uint32_t)(W * kMeta * 256);
#pragma unroll
                for (int i = 0; i < kMeta; ++i) {
                    const int wi = 64 * i + lane;
                    const int cl = (wi / kUnits) & 15, u = wi % kUnits;
                    const int j = i / kSub;
                    const int n = column(a, n_tile, w, j, cl);
                    const int first = column(a, n_tile, w, j, 0);
                    const int ua = kb * kSub + u < UW ? kb * kSub + u : UW - 1;
                    dma4(mbase[j], ((uint32_t)(n - first) * (uint32_t)UW + (uint32_t)ua) * 4u, dst + (uint32_t)i * 256u);
                }
            }
        };
        // this wave's copies of stages t and t + 1 have landed (later ones may be on their way;
        // metadata copies among them only make the wait longer), and everyone's after the barrier
        auto arrive = [&](int t) {
            if (t + kStages - 2 < nkb) wait_vmcnt<(kStages - 3) * kDma>();
            else wait_vmcnt<0>();
            wait_lgkmcnt0();
            lds_barrier();
        };
        auto word = [](const uint4& q, int i) { return i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w; };
        // scales of block t: each lane converts its own column's and reads back those of the
        // four columns its accumulators hold
        auto scales = [&](Operands& o, int t, uint32_t (&md)[CBW][kSub]) {
#pragma unroll
            for (int j = 0; j < CBW; ++j)
#pragma unroll
                for (int u = 0; u < kSub; ++u) {
                    md[j][u] = sh.meta[(t >> 2) % kMetaSlots][w][(16 * j + c) * kUnits + (t & 3) * kSub + u];
                    sh.scale[w][u][16 * j + c] = half_bits_to_f32<kScaleBF16>(md[j][u] & 0xFFFFu);
                }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int j = 0; j < CBW; ++j)
#pragma unroll
                for (int u = 0; u < kSub; ++u) o.s[j][u] = *reinterpret_cast<const f32x4*>(&sh.scale[w][u][16 * j + 4 * h]);
            __builtin_amdgcn_wave_barrier();
        };
        auto decode = [&](Operands& o, int j, int i, uint32_t d, const uint32_t (&md)[CBW][kSub]) {
            uint32_t p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = ((d >> (4 * e)) & 0x000F000Fu) | Magic<kBF16>::kBase2;
            if constexpr (!kBF16) {
                const _Float16 zb = (_Float16)(1024.0f + (float)((md[j][(i * kSub) / 4] >> 16) & 0xFu));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    p[e] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, p[e]) - f16x2{zb, zb});
            }
            o.b[j][i] = make_uint4(p[0], p[1], p[2], p[3]);
        };
        // Zero points of the group of row blocks 4 g .. 4 g + n - 1, by the matrix cores:
        // acc -= sum over its units of s (128 + z) X. Lane quarter h takes unit 4 v + h of
        // MFMA v. X (24 bits) is cut into three bf16 values, s (128 + z) (16 bits) into two,
        // each exactly, and their six products fill six of a quarter's eight places. (An fp16
        // scale makes it 19 bits and three values: eight products, all but the smallest.)
        auto take_off = [&](int g, int n) {
#pragma unroll
            for (int v = 0; v < kSub; ++v) {
                const int u = 4 * v + h;
                const bool in = u < n * kSub;
                uint4 S[CBW];
#pragma unroll
                for (int j = 0; j < CBW; ++j) {
                    const uint32_t md = sh.meta[g % kMetaSlots][w][(16 * j + c) * kUnits + u];
                    const float f = -half_bits_to_f32<kScaleBF16>(md & 0xFFFFu) * (128.f + (float)((md >> 16) & 0xFu));
                    const float f1 = bf16_bits_to_f32(f32_to_half_bits<true>(f));
                    const uint32_t p = in ? pack2_rne<true>(f1, f - f1) : 0u;
                    uint32_t p3 = 0u;
                    if constexpr (!kScaleBF16) {
                        const float f3 = f - f1 - bf16_bits_to_f32(f32_to_half_bits<true>(f - f1));
                        p3 = in ? pack2_rne<true>(f3, f3) : 0u;
                    }
                    S[j] = make_uint4(p, p, p, p3);
                }
#pragma unroll
                for (int r = 0; r < MR; ++r) {
                    const float X = in ? sh.xsum[g & 1][u][16 * r + c] : 0.f;
                    const uint32_t x1 = f32_to_half_bits<true>(X);
                    const float r1 = X - bf16_bits_to_f32(x1);
                    const uint32_t x2 = f32_to_half_bits<true>(r1);
                    const uint32_t x3 = f32_to_half_bits<true>(r1 - bf16_bits_to_f32(x2));
                    const uint4 xx = make_uint4(x1 * 0x10001u, x2 * 0x10001u, x3 * 0x10001u, kScaleBF16 ? 0u : x1 | x2 << 16);
#pragma unroll
                    for (int j = 0; j < CBW; ++j) acc[r][j] = mfma16x16x32<true>(S[j], xx, acc[r][j]);
                }
            }
        };
#pragma unroll
        for (int r = 0; r < MR; ++r)
#pragma unroll
            for (int j = 0; j < CBW; ++j) acc[r][j] = f32x4{0.f, 0.f, 0.f, 0.f};

        // Tiles of one fragment. Block t on operands `cur`; block t + 1 is decoded into `nxt`
        // behind its MFMAs. Stages t and t + 1 are in LDS, t + 2 is on its way.
        [[maybe_unused]] auto block = [&](int t, Operands& cur, Operands& nxt) {
            arrive(t);
            if (t + kStages - 1 < nkb) issue(t + kStages - 1);
            if constexpr (kBF16) {
                if ((t & 3) == 0 && t > 0) take_off((t >> 2) - 1, 4);
            }
            const Stage& st = sh.ring[t % kStages];
            const Stage& sn = sh.ring[(t + 1) % kStages];
            uint4 q[CBW], f[4];
            uint32_t md[CBW][kSub];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = st.x[c * 16 + ((4 * i + h) ^ c)];
#pragma unroll
            for (int j = 0; j < CBW; ++j) q[j] = sn.w[(w * CBW + j) * 64 + lane];
            scales(nxt, t + 1, md);
            if constexpr (kBF16) {
                // X (every lane and wave of a row writes the same value)
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
                    sh.xsum[(t >> 2) & 1][(t & 3) * kSub + u][c] = quarter_sum(X);
                }
            }
            f32x4 T[CBW][kSub];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < CBW; ++j) {
                    const int u = i * kSub / 4;
                    const f32x4 zero = f32x4{0.f, 0.f, 0.f, 0.f};
                    T[j][u] = mfma16x16x32<kBF16>(cur.b[j][i], f[i], i % (4 / kSub) == 0 ? zero : T[j][u]);
                }
#pragma unroll
            for (int j = 0; j < CBW; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) decode(nxt, j, i, word(q[j], i), md);
#pragma unroll
            for (int j = 0; j < CBW; ++j)
#pragma unroll
                for (int u = 0; u < kSub; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[0][j][e] = fmaf(cur.s[j][u][e], T[j][u][e], acc[0][j][e]);
            // keep the decoding and the sums in this block: they would be moved down to
            // their next use, behind the barrier and away from the MFMAs that hide them
#pragma unroll
            for (int j = 0; j < CBW; ++j) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    asm volatile("" : "+v"(nxt.b[j][i].x), "+v"(nxt.b[j][i].y), "+v"(nxt.b[j][i].z), "+v"(nxt.b[j][i].w));
                asm volatile("" : "+v"(acc[0][j]));
            }
        };

        Operands ops[2];
        if constexpr (MR >= 2) {
            // Tiles of several fragments: one MFMA, then a few vector instructions, in this
            // order (sched_barrier keeps it): a wave hides two or three of them behind each
            // MFMA, not a burst. The last fragment of a block is multiplied behind the next
            // block's barrier, where the first reads of LDS are on their way; a fragment is
            // scaled behind the one after it.
            f32x4 T[2][CBW][kSub], sc[CBW][kSub];
            uint4 f[2][4];
            constexpr int kFma = 4 * CBW * kSub;
            constexpr int kN = 4 * CBW;                                  // MFMAs of a fragment
            auto read_scale = [&](int j, int u) {
                sc[j][u] = *reinterpret_cast<const f32x4*>(&sh.scale[w][u][16 * j + 4 * h]);
            };
            auto write_scale = [&](int j, int u, uint32_t m) {
                sh.scale[w][u][16 * j + c] = half_bits_to_f32<kScaleBF16>(m & 0xFFFFu);
            };
            // behind the last fragment of a block the next block's scales come in, each
            // after its last use
            auto scale_part = [&](int r, int from, int to) {
#pragma unroll
                for (int i = 0; i < kFma; ++i)
                    if (i >= from && i < to) {
                        const int u = i / (4 * CBW), j = i / 4 % CBW, e = i % 4;
                        acc[r][j][e] = fmaf(sc[j][u][e], T[r & 1][j][u][e], acc[r][j][e]);
                        if (r == MR - 1 && e == 3) read_scale(j, u);
                    }
            };
            auto mfma_slot = [&](const Operands& o, int r, int k) {
                const int i = k / CBW, j = k % CBW, u = i * kSub / 4;
                const f32x4 zero = f32x4{0.f, 0.f, 0.f, 0.f};
                T[r & 1][j][u] = mfma16x16x32<kBF16>(o.b[j][i], f[r & 1][i], i % (4 / kSub) == 0 ? zero : T[r & 1][j][u]);
            };
            auto wide_block = [&](int t, Operands& cur, Operands& nxt) {
                arrive(t);
                const Stage& st = sh.ring[t % kStages];
                const Stage& sn = sh.ring[(t + 1) % kStages];
                uint4 q[CBW];
                uint32_t md[CBW][kSub];
                [[maybe_unused]] uint4 xf[4];
                [[maybe_unused]] float X[kSub];
                [[maybe_unused]] const int rx = w % MR;
                static_assert(MR % 2 == 0, "fragment 0 and the last one use different registers");
#pragma unroll
                for (int i = 0; i < 4; ++i) f[0][i] = st.x[c * 16 + ((4 * i + h) ^ c)];
#pragma unroll
                for (int j = 0; j < CBW; ++j) {
                    q[j] = sn.w[(w * CBW + j) * 64 + lane];
#pragma unroll
                    for (int u = 0; u < kSub; ++u)
                        md[j][u] = sh.meta[((t + 1) >> 2) % kMetaSlots][w][(16 * j + c) * kUnits + ((t + 1) & 3) * kSub + u];
                }
                if constexpr (kBF16) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) xf[i] = st.x[(16 * rx + c) * 16 + ((4 * i + h) ^ c)];
                }
                if (t + kStages - 1 < nkb) issue(t + kStages - 1);
                __builtin_amdgcn_sched_barrier(0);
                // phase 0: the last fragment of block t - 1; phase p: fragment p - 1
#pragma unroll
                for (int p = 0; p < MR; ++p) {
                    const int r = p == 0 ? MR - 1 : p - 1;
                    Operands& o = p == 0 ? nxt : cur;
                    const int rs = p == 0 ? MR - 2 : p == 1 ? MR - 1 : p - 2;       // the fragment to scale
                    constexpr int kPhases = MR - 1;
#pragma unroll
                    for (int k = 0; k < kN; ++k) {
                        mfma_slot(o, r, k);
                        // the next fragment's operands
                        if (p >= 1 && k % CBW == 0) {
                            const int i = k / CBW;
                            f[p & 1][i] = st.x[(16 * p + c) * 16 + ((4 * i + h) ^ c)];
                        }
                        if (k >= 1) scale_part(rs, (k - 1) * kFma / (kN - 1), k * kFma / (kN - 1));
                        if (p >= 1) {
                            // words of block t + 1, a quarter (two codes a register) at a time
                            const int all = 16 * CBW, at = (p - 1) * kN + k, slots = kPhases * kN;
#pragma unroll
                            for (int d = 0; d < 16 * CBW; ++d)
                                if (d >= at * all / slots && d < (at + 1) * all / slots) {
                                    const int j = d / 16, i = d / 4 % 4, e = d % 4;
                                    const uint32_t wd = word(q[j], i);
                                    uint32_t v = ((wd >> (4 * e)) & 0x000F000Fu) | Magic<kBF16>::kBase2;
                                    if constexpr (!kBF16) {
                                        const _Float16 zb = (_Float16)(1024.0f + (float)((md[j][(i * kSub) / 4] >> 16) & 0xFu));
                                        v = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, v) - f16x2{zb, zb});
                                    }
                                    (e == 0 ? nxt.b[j][i].x : e == 1 ? nxt.b[j][i].y : e == 2 ? nxt.b[j][i].z : nxt.b[j][i].w) = v;
                                }
                        }
                        // the block's sums of activations, two terms a slot
                        if constexpr (kBF16) {
                            constexpr int kFrom = MR > 2 ? kN : 0;
                            const int at = p * kN + k - kFrom;
                            if (at >= 0 && at < 8) {
                                const int i = at / 2, u = i * kSub / 4;
                                if (i % (4 / kSub) == 0 && at % 2 == 0) X[u] = 0.f;
                                X[u] = product_dot2<true>(at % 2 ? xf[i].z : xf[i].x, 0x3F803F80u, X[u]);
                                X[u] = product_dot2<true>(at % 2 ? xf[i].w : xf[i].y, 0x3F803F80u, X[u]);
                            }
                            if (at >= 8 && at < 8 + kSub) {
                                const int u = at - 8;
                                X[u] = quarter_sum(X[u]);
                                sh.xsum[(t >> 2) & 1][(t & 3) * kSub + u][16 * rx + c] = X[u];
                            }
                        }
                        // the scales of block t + 1, through LDS
                        if (p == MR - 1 && k == kN - 1) {
#pragma unroll
                            for (int j = 0; j < CBW; ++j)
#pragma unroll
                                for (int u = 0; u < kSub; ++u) write_scale(j, u, md[j][u]);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                // keep the decoding and the sums in this block: they would be moved down to
                // their next use, behind the barrier and away from the MFMAs that hide them
#pragma unroll
                for (int j = 0; j < CBW; ++j) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        asm volatile("" : "+v"(nxt.b[j][i].x), "+v"(nxt.b[j][i].y), "+v"(nxt.b[j][i].z), "+v"(nxt.b[j][i].w));
#pragma unroll
                    for (int r = 0; r < MR; ++r) asm volatile("" : "+v"(acc[r][j]));
                }
            };
            for (int t = 0; t < kStages - 1 && t < nkb; ++t) issue(t);
            if (kStages - 1 <= nkb) wait_vmcnt<(kStages - 2) * kDma>();
            else wait_vmcnt<0>();
            {
                uint32_t md[CBW][kSub];
#pragma unroll
                for (int j = 0; j < CBW; ++j) {
#pragma unroll
                    for (int u = 0; u < kSub; ++u) {
                        md[j][u] = sh.meta[0][w][(16 * j + c) * kUnits + u];
                        write_scale(j, u, md[j][u]);
                    }
                    const uint4 q = sh.ring[0].w[(w * CBW + j) * 64 + lane];
#pragma unroll
                    for (int i = 0; i < 4; ++i) decode(ops[0], j, i, word(q, i), md);
                }
            }
            // nothing before block 0
#pragma unroll
            for (int j = 0; j < CBW; ++j) {
#pragma unroll
                for (int i = 0; i < 4; ++i) ops[1].b[j][i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int u = 0; u < kSub; ++u) {
                    sc[j][u] = f32x4{0.f, 0.f, 0.f, 0.f};
                    T[0][j][u] = T[1][j][u] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) f[1][i] = make_uint4(0u, 0u, 0u, 0u);
            auto last = [&](const Operands& o) {
#pragma unroll
                for (int k = 0; k < kN; ++k) mfma_slot(o, MR - 1, k);
                scale_part(MR - 2, 0, kFma);
                scale_part(MR - 1, 0, kFma);
            };
            int t = 0;
            for (; t + 1 < nkb; t += 2) {
                wide_block(t, ops[0], ops[1]);
                wide_block(t + 1, ops[1], ops[0]);
                if constexpr (kBF16) {
                    if ((t & 3) == 2 && t + 2 < nkb) {
                        wait_lgkmcnt0();
                        lds_barrier();
                        take_off(t >> 2, 4);
                    }
                }
            }
            if (t < nkb) {
                wide_block(t, ops[0], ops[1]);
                last(ops[0]);
            } else {
                last(ops[1]);
            }
        } else {
            for (int t = 0; t < kStages - 1 && t < nkb; ++t) issue(t);
            if (kStages - 1 <= nkb) wait_vmcnt<(kStages - 2) * kDma>();
            else wait_vmcnt<0>();
            {
                uint32_t md[CBW][kSub];
                scales(ops[0], 0, md);
#pragma unroll
                for (int j = 0; j < CBW; ++j) {
                    const uint4 q = sh.ring[0].w[(w * CBW + j) * 64 + lane];
#pragma unroll
                    for (int i = 0; i < 4; ++i) decode(ops[0], j, i, word(q, i), md);
                }
            }
            int t = 0;
            for (; t + 1 < nkb; t += 2) {
                block(t, ops[0], ops[1]);
                block(t + 1, ops[1], ops[0]);
            }
            if (t < nkb) block(t, ops[0], ops[1]);
        }
        wait_lgkmcnt0();
        lds_barrier();
        if constexpr (kBF16) {
            take_off((nkb - 1) >> 2, ((nkb - 1) & 3) + 1);
            wait_lgkmcnt0();
            lds_barrier();
        }
        // the ring may be reused by the caller: every wave is done with it
    }
};

}  // namespace w4a16
