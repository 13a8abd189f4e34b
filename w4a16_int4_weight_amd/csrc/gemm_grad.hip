// The product with the transposed weight, dx = D W^T, from the packed buffer the forward
// reads: D [M, N] (an output gradient, or the gradient an operator formed itself), W [K, N].
//
//   dx[m, k] = sum_n D[m, n] (q[k, n] - z[g, n]) s[g, n],   g = k div G
//
// The sum now runs along n, where neighbouring weights lie in different lanes of a packed
// block and every term has a scale of its own. A weight is decoded once per workgroup:
// each thread takes 16 bytes of the stage (32 codes of one column), forms (q - z) s rounded
// once to the operand type (at most half a step each, errors of both signs over a sum of N
// terms), and writes 8-row runs into LDS as rows of n. The transposing LDS read
// (ds_read_b64_tr_b16: lane l of 16 receives element l of four rows) then delivers matrix
// operands that run along n: no nibble is moved between lanes by hand, and one packed
// buffer serves both directions. fp32 accumulators, no rounding between.
//
// Workgroup: a tile of BM rows x 256 columns of dx, 8 waves as WM x WK. A stage is 64
// columns of W: D's rows by direct global -> LDS copies (16-byte chunks XOR-swizzled by
// row), the codes through registers one stage ahead; two stages alternate, and the next
// one is decoded between the products of the current one. Tiles of up to 128 rows, which
// run few stages, take both through registers and four stages ahead, so that a memory
// latency is paid once and not each stage. Small M, or few tiles: the sum
// is split over workgroups into fp32 partial tiles, added in split order by a second
// kernel (the result does not depend on the order of arrival).
//
// Measured with every compute unit busy (4096 x 8192 -> 4096, bf16): 257 us, 1070 TFLOP/s;
// bound by LDS and the decoding: the matrix cores are busy 0.43 of the time, LDS about 0.5 (a
// third of it bank conflicts), and the two vector instructions an MFMA run beside it in only
// 0.02: a stage is decoded, written and read in bursts.
// 4096 x 2048 -> 6656 has 416 tiles for 256 compute units: 144 us, the second round 0.6 full.
// Few rows are bound by the partial tiles' traffic and the latency of a few stages.
#include "device_common.h"
#include "launch.h"

namespace w4a16 {
namespace {

constexpr int kTargetWorkgroups = 256;      // one per compute unit
constexpr int kStageN = 64;
constexpr int kTileK = 256;

typedef short i16x4 __attribute__((ext_vector_type(4)));

struct GradArgs {
    const uint16_t* d;
    int64_t ld;
    const uint8_t* packed;
    uint16_t* dx;
    float* part;
    int M, K, N, KB, UW;
    int n0, n;              // this call's columns
    int tiles_m, tiles_k, splits;
    int add;
    const int* hot;         // factors of D's rows and of what `add` adds to
    const float* factor;
    const float* before;
    int factor_stages;      // stages of one column of `factor`
    const uint16_t* d_rest;
    const float* rowmax;
    const uint32_t* tile_factor;
    int tile_columns;
    const float* scale_max;
};


__device__ __forceinline__ int weight_exponent(const float* scale_max) {       // by every lane of a wave
    float top = scale_max[threadIdx.x & 63];
    for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
    return scale_exponent(top, kScaleTop);
}

// 8 codes -> 8 operand values (q - z) s in row order
template <bool kOpBF16, bool kScaleBF16>
struct Decode {
    static_assert(kOpBF16 && kScaleBF16, "bf16 operands from bf16 scales");
    float s, nzs;
    __device__ __forceinline__ explicit Decode(uint32_t md) {
        s = half_bits_to_f32<kScaleBF16>(md & 0xFFFFu);
        nzs = -(float)((md >> 16) & 0xFu) * s;
    }
    __device__ __forceinline__ uint4 operator()(uint32_t d) const {
        uint32_t lo = d & 0x0F0F0F0Fu, hi = (d >> 4) & 0x0F0F0F0Fu;    // rows 0,4,1,5 / 2,6,3,7
        asm volatile("" : "+v"(lo), "+v"(hi));
        const float r0 = fmaf((float)(lo & 0xFFu), s, nzs), r4 = fmaf((float)((lo >> 8) & 0xFFu), s, nzs);
        const float r1 = fmaf((float)((lo >> 16) & 0xFFu), s, nzs), r5 = fmaf((float)(lo >> 24), s, nzs);
        const float r2 = fmaf((float)(hi & 0xFFu), s, nzs), r6 = fmaf((float)((hi >> 8) & 0xFFu), s, nzs);
        const float r3 = fmaf((float)((hi >> 16) & 0xFFu), s, nzs), r7 = fmaf((float)(hi >> 24), s, nzs);
        return make_uint4(pack2_rne<true>(r0, r1), pack2_rne<true>(r2, r3), pack2_rne<true>(r4, r5),
                          pack2_rne<true>(r6, r7));
    }
};
template <>
struct Decode<false, false> : Dequant<false> {
    __device__ __forceinline__ explicit Decode(uint32_t md) : Dequant<false>(md) {}
};

// codes -> fp16 (q - z) (s 2^e), s of either type
template <bool kScaleBF16>
struct DecodeScaled : Dequant<false> {
    __device__ __forceinline__ DecodeScaled(uint32_t md, float by) {
        const _Float16 zb = (_Float16)(1024.0f + (float)((md >> 16) & 0xFu));
        const _Float16 s = (_Float16)(half_bits_to_f32<kScaleBF16>(md & 0xFFFFu) * by);
        zz = f16x2{zb, zb};
        ss = f16x2{s, s};
    }
};

// One stage: D rows [BM][8 chunks of 16 bytes], chunk j of row r at j ^ (r % 8); W rows
// [64 n][32 chunks of 8 k], chunk j of row n at j ^ swz(n). swz spreads the 8 lanes of a
// write (8 consecutive n, one chunk) over 8 chunks and the 16 rows of a transposing read
// (n % 8 in a half, all n / 8) evenly over 4 chunk pairs.
__device__ __forceinline__ int swz(int n) { return (n & 7) ^ (2 * ((n >> 3) & 3)); }

template <bool kOpBF16, bool kScaleBF16, int MR, int WM, int CK, int kSub, bool kScaled>
__global__ __launch_bounds__(512) void grad_kernel(const GradArgs a) {
    constexpr int WK = 8 / WM;
    constexpr int BM = 16 * MR * WM;
    static_assert(16 * CK * WK == kTileK, "the waves cover the tile's columns");
    constexpr int kSlabs = BM / 8;                    // 1 KiB slabs (8 rows) of the D stage
    // D through registers (else by direct copies), and stages on their way in registers
    constexpr bool kRegs = kScaled || BM <= 128;
    constexpr int kDepth = BM > 128 ? 1 : kScaled && !kScaleBF16 ? 2 : 4;       // (fp16 scaled: twice the D)
    // D as two fp16 values, d + d_rest. One fp16 rounding of D, one of W and the result's own
    // come to 1.7 times the last; without D's, to 1.4. (bf16's own rounding is 8 times
    // theirs.) It costs a second MFMA; a 256-row tile has neither the time nor the LDS.
    constexpr bool kRest = kScaled && !kScaleBF16 && BM <= 128;
    struct Stage {
        uint4 d[BM * 8];
        uint4 w[kStageN * 32];
        uint4 rest[kRest ? BM * 8 : 1];
    };
    __shared__ Stage ring[2];

    const int tid = threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
    const int c = lane & 15, h = lane >> 4;
    const int wm = w / WK, wk = w % WK;

    // ids id, id + 8, ... share an XCD, which takes whole splits' tiles in turn: column tiles
    // fastest, so that one stage of D, the wider operand, serves several of its workgroups
    // from its L2 (4096 x 8192 -> 4096: 270 -> 264 us against row tiles fastest)
    int id = (int)blockIdx.x;
    const int total = a.tiles_m * a.tiles_k * a.splits;
    id = xcd_share(id, total);
    const int k_tile = id % a.tiles_k;
    const int rest = id / a.tiles_k;
    const int m_tile = rest % a.tiles_m;
    const int split = rest / a.tiles_m;
    const int m0 = m_tile * BM, k0 = k_tile * kTileK;
    const int stages = (a.n + kStageN - 1) / kStageN;
    const int st_lo = (int)((int64_t)stages * split / a.splits);
    const int st_hi = (int)((int64_t)stages * (split + 1) / a.splits);

    // this thread's 16 bytes of a stage: column 16 nbi + cc, row block kbi of the tile,
    // lane quarter hh
    const int nbi = tid >> 7, kbi = (tid >> 6) & 1, hh = (tid >> 4) & 3, cc = tid & 15;
    const int kb = k0 / kRowsPerBlock + kbi;
    const int kbc = kb < a.KB ? kb : a.KB - 1;
    const int Np = (int)padded_cols(a.N);
    const int NB = Np / kColsPerBlock;
    const uint8_t* meta = a.packed + (size_t)a.K * Np / 2;

    [[maybe_unused]] int we = 0;
    [[maybe_unused]] float wscale = 1.f;
    if constexpr (kScaled) {
        we = weight_exponent(a.scale_max);
        wscale = power_of_two(we);
    }
    constexpr int kChunks = kRegs ? (BM * 8 + 511) / 512 : 1;
    struct Fetch {                                    // what a thread holds of a stage
        uint4 code;
        uint32_t md[kSub];
        uint4 dv[kChunks];                            // chunk tid + 512 i of D (row / 8, 8 columns)
        uint4 rest[kRest ? kChunks : 1];
        uint32_t df[kChunks];
    };
    Fetch fetch[kDepth];
    auto load_codes = [&](Fetch& x, int t) {
        const int n = a.n0 + t * kStageN + 16 * nbi + cc;
        const int nb = n / kColsPerBlock < NB ? n / kColsPerBlock : NB - 1;
        x.code = *reinterpret_cast<const uint4*>(a.packed + ((size_t)nb * a.KB + kbc) * kBlockBytes + 16 * (16 * hh + cc));
#pragma unroll
        for (int u = 0; u < kSub; ++u)
            x.md[u] = *reinterpret_cast<const uint32_t*>(meta + 4 * ((size_t)(nb * kColsPerBlock + cc) * a.UW + kbc * kSub + u));
    };
    auto store_codes = [&](const Fetch& x, int slot, int t) {
        const int row = 16 * nbi + cc;
        const bool in = t * kStageN + row < a.n;      // columns past the call's weigh zero
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t d = i == 0 ? x.code.x : i == 1 ? x.code.y : i == 2 ? x.code.z : x.code.w;
            const uint32_t md = in ? x.md[(i * kSub) / 4] : 0u;
            uint4 v;
            if constexpr (kScaled) v = DecodeScaled<kScaleBF16>(md, wscale)(d);
            else v = Decode<kOpBF16, kScaleBF16>(md)(d);
            ring[slot].w[row * 32 + ((16 * kbi + 4 * i + hh) ^ swz(row))] = v;
        }
    };
    // Direct copies: D rows m0 + 8 slab + lane / 8, 16-byte chunk (lane % 8) ^ (row % 8). Rows past M read
    // row M - 1. A stage that ends past the call's columns is read with a test per chunk
    // instead (n % 8 == 0), zero outside: what lies there may be no number.
    const uint8_t* dbase = uniform_ptr(a.d + (size_t)m0 * a.ld);
    auto issue_d = [&](int slot, int t) {
        const int nn = t * kStageN;
        if (nn + kStageN <= a.n) {
#pragma unroll
            for (int q = 0; q < (kSlabs + 7) / 8; ++q) {
                const int slab = w + 8 * q;
                if (kSlabs % 8 == 0 || slab < kSlabs) {
                    const int row = 8 * slab + (lane >> 3);
                    const int m = m0 + row < a.M ? row : a.M - 1 - m0;
                    dma16(dbase + (size_t)nn * 2, 2u * ((uint32_t)m * (uint32_t)a.ld + 8u * (uint32_t)((lane & 7) ^ (row & 7))),
                          lds_addr(&ring[slot].d[0]) + 1024u * (uint32_t)slab);
                }
            }
        } else {
            for (int q = tid; q < BM * 8; q += 512) {
                const int row = q >> 3, ch = q & 7;
                const int m = m0 + row < a.M ? m0 + row : a.M - 1;
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (nn + 8 * ch < a.n) v = *reinterpret_cast<const uint4*>(a.d + (size_t)m * a.ld + nn + 8 * ch);
                ring[slot].d[row * 8 + (ch ^ (row & 7))] = v;
            }
        }
    };

    // Through registers. Scaled D is multiplied by its tile's factor on the way (a power of
    // two, exact but for what falls below fp16's last place at the row's scale).
    [[maybe_unused]] uint32_t drow[kChunks];
    if constexpr (kRegs) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int row = ((tid + 512 * i) >> 3) % BM;
            drow[i] = (uint32_t)(m0 + row < a.M ? row : a.M - 1 - m0);
        }
    }
    const bool hot = a.hot && *a.hot != 0;
    auto load_d = [&](Fetch& x, int t) {
        const int n = t * kStageN + 8 * (tid & 7) < a.n ? t * kStageN + 8 * (tid & 7) : a.n - 8;      // n % 8 == 0
        const uint32_t* fac = nullptr;
        if constexpr (kScaled) {
            if (a.tile_factor) fac = a.tile_factor + (size_t)((n < a.n / 2 ? n : n - a.n / 2) / a.tile_columns) * a.M + m0;
        }
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            x.dv[i] = *reinterpret_cast<const uint4*>(dbase + 2 * ((size_t)drow[i] * a.ld + n));
            if constexpr (kRest)
                x.rest[i] = *reinterpret_cast<const uint4*>(a.d_rest + ((size_t)m0 + drow[i]) * a.ld + n);
            if constexpr (kScaled) x.df[i] = fac ? fac[drow[i]] : 0x3C003C00u;
        }
    };
    auto bf16_times = [](uint32_t p, float by) {
        return pack2_rne<true>(bf16_bits_to_f32(p & 0xFFFFu) * by, bf16_bits_to_f32(p >> 16) * by);
    };
    auto store_d = [&](const Fetch& x, int slot, int t) {
        const bool in = t * kStageN + 8 * (tid & 7) < a.n;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int q = tid + 512 * i;
            if (BM * 8 % 512 != 0 && q >= BM * 8) break;
            const int row = q >> 3, ch = q & 7;
            uint4 v = x.dv[i];
            if constexpr (kScaled) {
                const f16x2 by = __builtin_bit_cast(f16x2, x.df[i]);
                auto times = [&](uint32_t p) { return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, p) * by); };
                v = make_uint4(times(v.x), times(v.y), times(v.z), times(v.w));
                if constexpr (kRest) {
                    const uint4 l = x.rest[i];
                    ring[slot].rest[row * 8 + (ch ^ (row & 7))] =
                        in ? make_uint4(times(l.x), times(l.y), times(l.z), times(l.w)) : make_uint4(0u, 0u, 0u, 0u);
                }
            } else if constexpr (kOpBF16) {
                if (hot) {
                    const float by = a.factor[(size_t)(t / a.factor_stages) * a.M + m0 + drow[i]];
                    v = make_uint4(bf16_times(v.x, by), bf16_times(v.y, by), bf16_times(v.z, by), bf16_times(v.w, by));
                }
            }
            ring[slot].d[row * 8 + (ch ^ (row & 7))] = in ? v : make_uint4(0u, 0u, 0u, 0u);
        }
    };

    f32x4 acc[MR][CK];
#pragma unroll
    for (int r = 0; r < MR; ++r)
#pragma unroll
        for (int j = 0; j < CK; ++j) acc[r][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto load = [&](Fetch& x, int t) {
        load_codes(x, t);
        if constexpr (kRegs) load_d(x, t);
    };
    auto store = [&](const Fetch& x, int slot, int t) {
        if constexpr (kRegs) store_d(x, slot, t);
        else issue_d(slot, t);
        store_codes(x, slot, t);
    };
    // one stage; `next` holds stage t + 1 and takes stage t + 1 + kDepth
    auto stage = [&](int t, Fetch& next) {
        const int slot = (t - st_lo) & 1;
        if constexpr (!kRegs) wait_vmcnt<0>();        // this wave's copies of stage t
        wait_lgkmcnt0();                  // its decoded rows of stage t are written
        lds_barrier();                    // everyone's; and everyone has read stage t - 1
        if constexpr (kOpBF16 && !kRegs) {
            if (hot) {
                const float* fac = a.factor + (size_t)(t / a.factor_stages) * a.M;
                for (int q = tid; q < BM * 8; q += 512) {
                    const int row = q >> 3;
                    const float by = fac[m0 + row < a.M ? m0 + row : a.M - 1];
                    const uint4 v = ring[slot].d[q];
                    ring[slot].d[q] = make_uint4(bf16_times(v.x, by), bf16_times(v.y, by), bf16_times(v.z, by), bf16_times(v.w, by));
                }
                __syncthreads();
            }
        }
        if (t + 1 < st_hi) store(next, slot ^ 1, t + 1);
        if (t + 1 + kDepth < st_hi) load(next, t + 1 + kDepth);
        const Stage& st = ring[slot];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint4 b[CK], f[MR];
#pragma unroll
            for (int j = 0; j < CK; ++j) {
                // rows n = 32 i + 8 h + (0..3) and + (4..7), 16 columns k from 16 (wk CK + j):
                // lane c of the 16 points at row c / 4, columns 4 (c % 4)
                const int ch = 2 * (wk * CK + j) + ((c >> 1) & 1);
                i16x4 v[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int n = 32 * i + 8 * h + 4 * q + (c >> 2);
                    const uint8_t* p = reinterpret_cast<const uint8_t*>(&st.w[n * 32 + (ch ^ swz(n))]) + 8 * (c & 1);
                    v[q] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (__attribute__((address_space(3))) i16x4*)(const __attribute__((address_space(3))) void*)p);
                }
                const uint2 lo = __builtin_bit_cast(uint2, v[0]), hi = __builtin_bit_cast(uint2, v[1]);
                b[j] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
#pragma unroll
            for (int r = 0; r < MR; ++r) {
                const int row = 16 * (wm * MR + r) + c;
                f[r] = st.d[row * 8 + ((4 * i + h) ^ (row & 7))];
            }
            // transposed tiles: lane (c, h), register e -> row 16 r + c, column 16 j + 4 h + e
#pragma unroll
            for (int r = 0; r < MR; ++r)
#pragma unroll
                for (int j = 0; j < CK; ++j) acc[r][j] = mfma16x16x32<kOpBF16>(b[j], f[r], acc[r][j]);
            if constexpr (kRest) {
#pragma unroll
                for (int r = 0; r < MR; ++r) {
                    const int row = 16 * (wm * MR + r) + c;
                    const uint4 l = st.rest[row * 8 + ((4 * i + h) ^ (row & 7))];
#pragma unroll
                    for (int j = 0; j < CK; ++j) acc[r][j] = mfma16x16x32<kOpBF16>(b[j], l, acc[r][j]);
                }
            }
        }
    };
    if (st_lo < st_hi) {
#pragma unroll
        for (int u = 0; u < kDepth; ++u)
            if (st_lo + u < st_hi) load(fetch[u], st_lo + u);
        store(fetch[0], 0, st_lo);
        if (st_lo + kDepth < st_hi) load(fetch[0], st_lo + kDepth);
    }
    for (int t = st_lo; t < st_hi; t += kDepth) {
#pragma unroll
        for (int u = 0; u < kDepth; ++u)
            if (t + u < st_hi) stage(t + u, fetch[(u + 1) % kDepth]);
    }

#pragma unroll
    for (int r = 0; r < MR; ++r) {
        const int m = m0 + 16 * (wm * MR + r) + c;
        if (m >= a.M) continue;
#pragma unroll
        for (int j = 0; j < CK; ++j) {
            const int k = k0 + 16 * (wk * CK + j) + 4 * h;
            if (k >= a.K) continue;
            f32x4 v = acc[r][j];
            if (a.part) {
                f32x4* o = reinterpret_cast<f32x4*>(a.part + ((size_t)split * a.M + m) * a.K + k);
                if (a.add) v += hot ? *o * a.before[m] : *o;
                *o = v;
            } else {
                if constexpr (kScaled) v = times_power_of_two(v, -we - scale_exponent(a.rowmax[m], kGradTop));
                const uint2 o = make_uint2(pack2_rne<kScaleBF16>(v[0], v[1]), pack2_rne<kScaleBF16>(v[2], v[3]));
                *reinterpret_cast<uint2*>(a.dx + (size_t)m * a.K + k) = o;
            }
        }
    }
}

// dx = sum_s part[s], 8 values a thread; bandwidth-bound over the partials
template <bool kBF16>
__global__ __launch_bounds__(256) void grad_finish_kernel(const float* __restrict__ part, int splits, int64_t MK, int K,
                                                          const float* __restrict__ rowmax,
                                                          const float* __restrict__ scale_max, uint16_t* __restrict__ dx) {
    const int64_t at = 8 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    const int we = rowmax ? weight_exponent(scale_max) : 0;
    if (at >= MK) return;
    f32x4 s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
        const f32x4* p = reinterpret_cast<const f32x4*>(part + s * MK + at);
        s0 += p[0];
        s1 += p[1];
    }
    if (rowmax) {
        const int e = -we - scale_exponent(rowmax[at / K], kGradTop);
        s0 = times_power_of_two(s0, e);
        s1 = times_power_of_two(s1, e);
    }
    *reinterpret_cast<uint4*>(dx + at) = make_uint4(pack2_rne<kBF16>(s0[0], s0[1]), pack2_rne<kBF16>(s0[2], s0[3]),
                                                    pack2_rne<kBF16>(s1[0], s1[1]), pack2_rne<kBF16>(s1[2], s1[3]));
}

template <bool kOp, bool kSc, int kSub, bool kScaled>
void launch_sub(int bm, const GradArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.tiles_m * a.tiles_k * a.splits)), block(512);
    if (bm == 16) hipLaunchKernelGGL((grad_kernel<kOp, kSc, 1, 1, 2, kSub, kScaled>), grid, block, 0, s, a);
    else if (bm == 32) hipLaunchKernelGGL((grad_kernel<kOp, kSc, 2, 1, 2, kSub, kScaled>), grid, block, 0, s, a);
    else if (bm == 64) hipLaunchKernelGGL((grad_kernel<kOp, kSc, 4, 1, 2, kSub, kScaled>), grid, block, 0, s, a);
    else if (bm == 128) hipLaunchKernelGGL((grad_kernel<kOp, kSc, 4, 2, 4, kSub, kScaled>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((grad_kernel<kOp, kSc, 8, 2, 4, kSub, kScaled>), grid, block, 0, s, a);
}

// operands: bf16 or fp16 as the scales, or scaled fp16
template <bool kSc, bool kScaled>
void launch_typed(int bm, int sub, const GradArgs& a, hipStream_t s) {
    constexpr bool kOp = kSc && !kScaled;
    if (sub == 4) launch_sub<kOp, kSc, 4, kScaled>(bm, a, s);
    else if (sub == 2) launch_sub<kOp, kSc, 2, kScaled>(bm, a, s);
    else launch_sub<kOp, kSc, 1, kScaled>(bm, a, s);
}

}  // namespace

// Rows of a tile and the split of the sum, by what they cost: rounds of tiles over the
// compute units times the stages of each (us, measured with every compute unit busy; 4096 x
// 8192 -> 4096 takes 264 us in 256-row tiles, 376 in 128-row ones), plus a start and an end,
// plus the partial tiles written and read at 4 TB/s. Lower tiles need fewer splits: 180 x
// 4000 -> 1024 takes 21.3 us in 128-row tiles, 15.5 in 32-row ones; 64 x 32000 -> 2048, where
// the stages count, 6.7 us less in 64-row tiles than in 32-row ones. At least 4 stages a
// split.
GradPlan plan_grad(int64_t M, int64_t K, int64_t n, bool forced) {
    GradPlan p{};
    p.tiles_k = (int)((K + kTileK - 1) / kTileK);
    const int64_t stages = (n + kStageN - 1) / kStageN;
    const int64_t most = stages / 4 > 1 ? stages / 4 : 1;
    struct Shape { int bm; double stage; };
    static constexpr Shape kShapes[] = {{16, 0.85}, {32, 0.9}, {64, 1.1}, {128, 1.47}, {256, 2.06}};
    double best = 0.0;
    for (const Shape& c : kShapes) {
        if (c.bm > 16 && c.bm / 2 >= M) break;                     // half the rows would do
        const int64_t tm = (M + c.bm - 1) / c.bm, tiles = tm * p.tiles_k;
        int64_t s = kTargetWorkgroups / tiles;
        s = s < 1 ? 1 : s < most ? s : most;
        for (;; s /= 2) {
            const int64_t rounds = (tiles * s + kTargetWorkgroups - 1) / kTargetWorkgroups;
            const double part = forced || s > 1 ? 8.0e-6 * (double)s * (double)M * (double)K / 4.0 : 0.0;
            const double cost = (double)rounds * ((double)stages / (double)s * c.stage + 5.0) + part;
            if (best == 0.0 || cost < best) {
                best = cost;
                p.bm = c.bm;
                p.tiles_m = (int)tm;
                p.splits = (int)s;
            }
            if (s == 1) break;
        }
    }
    p.part_bytes = forced || p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)K * 4 : 0;
    return p;
}

bool grad_takes_rest(const GradPlan& plan, bool bf16) { return !bf16 && plan.bm <= 128; }

hipError_t launch_grad(const GradPlan& plan, const GradCall& q, hipStream_t stream) {
    GradArgs a{};
    a.d = q.d;
    a.ld = q.ld;
    a.packed = q.packed;
    a.dx = q.dx;
    a.part = q.part;
    a.add = q.add ? 1 : 0;
    a.M = (int)q.M;
    a.K = (int)q.K;
    a.N = (int)q.N;
    a.KB = (int)(q.K / kRowsPerBlock);
    a.UW = (int)padded_units(q.K, q.G);
    a.n0 = (int)q.n0;
    a.n = (int)q.n;
    a.tiles_m = plan.tiles_m;
    a.tiles_k = plan.tiles_k;
    a.splits = plan.splits;
    a.hot = q.hot;
    a.factor = q.factor;
    a.before = q.before;
    a.factor_stages = q.factor_columns / kStageN;
    if ((plan.splits > 1 || !q.dx) && !q.part) return hipErrorInvalidValue;
    if (q.scaled && grad_takes_rest(plan, q.bf16) != (q.d_rest != nullptr)) return hipErrorInvalidValue;
    a.d_rest = q.d_rest;
    a.rowmax = q.rowmax;
    a.tile_factor = q.tile_factor;
    a.tile_columns = q.tile_columns;
    a.scale_max = q.scale_max;
    const int sub = units_per_block(q.G);
    if (q.scaled) {
        if (q.bf16) launch_typed<true, true>(plan.bm, sub, a, stream);
        else launch_typed<false, true>(plan.bm, sub, a, stream);
    } else {
        if (q.bf16) launch_typed<true, false>(plan.bm, sub, a, stream);
        else launch_typed<false, false>(plan.bm, sub, a, stream);
    }
    return hipGetLastError();
}

hipError_t launch_grad_finish(const float* part, int splits, int64_t M, int64_t K, uint16_t* dx, bool bf16,
                              const float* rowmax, const float* scale_max, hipStream_t stream) {
    const int64_t MK = M * K;
    const dim3 grid((unsigned)((MK / 8 + 255) / 256)), block(256);
    if (bf16) hipLaunchKernelGGL((grad_finish_kernel<true>), grid, block, 0, stream, part, splits, MK, (int)K, rowmax, scale_max, dx);
    else hipLaunchKernelGGL((grad_finish_kernel<false>), grid, block, 0, stream, part, splits, MK, (int)K, rowmax, scale_max, dx);
    return hipGetLastError();
}

}  // namespace w4a16
