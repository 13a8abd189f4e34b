// The operators' product for up to 16 rows (decoding, scoring while serving): bound by the
// time to stream the packed codes, so the work is cut as for a matrix-vector product.
//
// A unit is 16 weight columns over the whole of K: one column block of the head, or 8 gate
// columns and their 8 up columns (half blocks are whole 128-byte lines). Workgroup g takes a
// contiguous share of the units; its 8 waves split K, JP consecutive row blocks each, and
// hold the activations of those in registers for good. Units come in batches: every code
// and metadata load of the next batch is on its way while one is multiplied (16x16x32
// MFMAs: rows x 16 columns), and the waves' partial sums meet in LDS, two buffers in turn,
// one barrier a batch, added in wave order. No K split over workgroups, no partial sums in
// memory, no atomics: results do not depend on timing.
//
// Per metadata unit: s (T - (16 + z) X), T = sum x (16 + q) on codes masked into the mantissa
// of bf16's 16.0 (one shift more per word than 128.0, as tile_product.h has it, and a ninth
// of what the difference loses; here the shifts hide behind the loads). X comes from the
// same MFMAs against ones, once for all units. fp16 takes q - z exactly in 16 bits.
//
// Measured: 2048 x 13312, one row or 16, 7.4 us a call, the kernel 6.3 (10 us with 16-row tiles
// and K split over workgroups); 2048 x 131072, one row, 35 us, 4.1 TB/s (the matrix-vector
// kernel of the product reads the same codes in 22 us: here a barrier a batch keeps the waves
// together, and the vector units decode half the time). With 512 workgroups instead of 256:
// 9.0 and 38.7 us a call.
#include "device_common.h"
#include "gate.h"
#include "launch.h"

namespace w4a16 {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kTargetWorkgroups = 256;      // one per compute unit

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

struct SmallArgs {
    const uint16_t* x;
    const uint8_t* packed;
    int M, K, N, F, KB, UW, U;
    // gated
    uint16_t* h;
    const uint16_t* dh;
    float* d32;
    float* tops;            // [workgroups][M]
    int act;
    // cross entropy
    const int32_t* labels;
    float* zsel;
    float2* part;           // [workgroups][M]
};

__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
}

template <bool kBF16, int kSub, int JP, bool kGated>
__global__ __launch_bounds__(kThreads) void small_kernel(const SmallArgs a) {
    constexpr int S = JP == 4 ? 2 : 4;                     // units of a batch
    constexpr int kWords = JP * kSub;                      // metadata words of a lane and unit
    __shared__ f32x4 part[2][S][kWaves][64];

    const int tid = (int)threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63, c = lane & 15, h = lane >> 4;
    const int nwg = (int)gridDim.x;
    const int g = xcd_share((int)blockIdx.x, nwg);
    const int lo = (int)((int64_t)g * a.U / nwg), hi = (int)((int64_t)(g + 1) * a.U / nwg);
    const int kb0 = w * JP;
    const int M = a.M, KB = a.KB;
    const uint8_t* meta = a.packed + (size_t)a.K * padded_cols(a.N) / 2;

    auto column = [&](int u) { return kGated ? (c >> 3) * a.F + 8 * u + (c & 7) : 16 * u + c; };
    struct Batch {
        uint4 q[S][JP];
        uint32_t md[S][kWords];
    };
    auto load = [&](Batch& b, int u0) {
        // a wave past the last row block loads nothing; metadata words past the column's
        // last belong to row blocks that are skipped
        if (kb0 >= KB) return;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int u = u0 + s < hi ? u0 + s : hi - 1;
            const int n = column(u);
            const uint8_t* at = a.packed + ((size_t)(n >> 4) * KB) * kBlockBytes + 16 * (16 * h + (n & 15));
#pragma unroll
            for (int j = 0; j < JP; ++j) b.q[s][j] = load_once(at + (size_t)(kb0 + j < KB ? kb0 + j : KB - 1) * kBlockBytes);
            const uint32_t* m = reinterpret_cast<const uint32_t*>(meta) + (size_t)n * a.UW;
#pragma unroll
            for (int j = 0; j < kWords; j += 4) {
                constexpr int kVec = kWords < 4 ? kWords : 4;
                const int w0 = kb0 * kSub + j + kVec <= a.UW ? kb0 * kSub + j : a.UW - kVec;
                if constexpr (kVec == 4) {
                    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(m + w0));
                    b.md[s][j] = v.x; b.md[s][j + 1] = v.y; b.md[s][j + 2] = v.z; b.md[s][j + 3] = v.w;
                } else if constexpr (kVec == 2) {
                    const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(m + w0));
                    b.md[s][j] = v.x; b.md[s][j + 1] = v.y;
                } else {
                    b.md[s][j] = __builtin_nontemporal_load(m + w0);
                }
            }
        }
    };

    // the activations of this wave's row blocks: row c (rows past M: row M - 1), and X
    uint4 xf[JP][4];
    const uint16_t* xr = a.x + (size_t)(c < M ? c : M - 1) * a.K + 8 * h;
#pragma unroll
    for (int j = 0; j < JP; ++j) {
        const int kb = kb0 + j < KB ? kb0 + j : KB - 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) xf[j][i] = *reinterpret_cast<const uint4*>(xr + (size_t)kb * kRowsPerBlock + 32 * i);
    }
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 X[JP][kSub];
    auto sums = [&]() {
        if constexpr (kBF16) {
            const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
#pragma unroll
            for (int j = 0; j < JP; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int u = i * kSub / 4;
                    X[j][u] = mfma16x16x32<true>(xf[j][i], ones, i % (4 / kSub) == 0 ? zero : X[j][u]);
                }
        }
    };
    // rows 4 h + e, column c of unit s
    auto multiply = [&](const Batch& b, int s) {
        f32x4 acc = zero;
#pragma unroll
        for (int j = 0; j < JP; ++j) {
            if (kb0 + j >= KB) continue;
            f32x4 T[kSub];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t d = i == 0 ? b.q[s][j].x : i == 1 ? b.q[s][j].y : i == 2 ? b.q[s][j].z : b.q[s][j].w;
                const int u = i * kSub / 4;
                uint32_t p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (kBF16) p[e] = ((e == 0 ? d << 3 : d >> (4 * e - 3)) & 0x00780078u) | 0x41804180u;
                    else p[e] = ((d >> (4 * e)) & 0x000F000Fu) | Magic<false>::kBase2;
                }
                if constexpr (!kBF16) {
                    const _Float16 zb = (_Float16)(1024.0f + (float)((b.md[s][j * kSub + u] >> 16) & 0xFu));
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        p[e] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, p[e]) - f16x2{zb, zb});
                }
                T[u] = mfma16x16x32<kBF16>(xf[j][i], make_uint4(p[0], p[1], p[2], p[3]), i % (4 / kSub) == 0 ? zero : T[u]);
            }
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                const uint32_t md = b.md[s][j * kSub + u];
                const float sc = half_bits_to_f32<kBF16>(md & 0xFFFFu);
                const float zb = 16.f + (float)((md >> 16) & 0xFu);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] = fmaf(sc, kBF16 ? fmaf(-zb, X[j][u][e], T[u][e]) : T[u][e], acc[e]);
            }
        }
        return acc;
    };
    auto total = [&](int buf, int s, int m, int col) {
        float v = 0.f;
        const int at = 16 * (m >> 2) + col, e = m & 3;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) v += reinterpret_cast<const float*>(&part[buf][s][i][at])[e];
        return v;
    };

    constexpr int kCols = kGated ? 8 : 16;
    constexpr int kRowStep = kThreads / (kCols * S);       // rows met at a time
    constexpr int kSlots = kGated || kRowStep >= 16 ? 1 : 16 / kRowStep;
    const int oc = tid % kCols, os = tid / kCols % S, om = tid / (kCols * S);
    [[maybe_unused]] float top[kSlots], sum[kSlots], most = 0.f;
    [[maybe_unused]] int label[kSlots];
    if constexpr (!kGated) {
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            top[k] = -INFINITY;
            sum[k] = 0.f;
            const int m = om + k * kRowStep;
            label[k] = m < M ? a.labels[m] : -1;
        }
    }

    auto turn = [&](Batch& cur, Batch& nxt, int u0, int buf) {
        if (u0 + S < hi) load(nxt, u0 + S);
#pragma unroll
        for (int s = 0; s < S; ++s) part[buf][s][w][lane] = multiply(cur, s);
        __syncthreads();
        const int u = u0 + os;
        if constexpr (kGated) {
            for (int m = om; m < M; m += kRowStep) {              // one row a thread: M <= 16 <= kRowStep
                if (u >= hi) continue;
                const float gv = total(buf, os, m, oc), uv = total(buf, os, m, oc + 8);
                const size_t f = (size_t)8 * u + oc;
                float slope;
                const float pr = a.act == 0 ? gate_prob<0>(gv, &slope) : a.act == 1 ? gate_prob<1>(gv, &slope) : gate_prob<2>(gv, &slope);
                if (a.d32) {
                    const float dv = half_bits_to_f32<kBF16>(a.dh[(size_t)m * a.F + f]);
                    const float dg = dv * uv * fmaf(gv, slope, pr), du = dv * (gv * pr);
                    a.d32[(size_t)m * 2 * a.F + f] = dg;
                    a.d32[(size_t)m * 2 * a.F + a.F + f] = du;
                    most = fmaxf(most, fmaxf(fabsf(dg), fabsf(du)));
                } else {
                    a.h[(size_t)m * a.F + f] = f32_to_half_bits<kBF16>(gv * pr * uv);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < kSlots; ++k) {
                const int m = om + k * kRowStep, n = 16 * u + oc;
                if (m >= M || u >= hi || n >= a.N) continue;
                float z = total(buf, os, m, oc);
                if (n == label[k]) {
                    a.zsel[m] = z;
                    z = -INFINITY;                               // the target is left out of the sum
                }
                const float t = fmaxf(top[k], z);                // passes over what is no number: the sum carries it
                if (top[k] != -INFINITY || z != -INFINITY) sum[k] = sum[k] * __expf(top[k] - t) + __expf(z - t);
                top[k] = t;
            }
        }
    };
    Batch b0, b1;
    load(b0, lo);
    sums();
    for (int u0 = lo; u0 < hi; u0 += 2 * S) {
        turn(b0, b1, u0, 0);
        if (u0 + S < hi) turn(b1, b0, u0 + S, 1);
    }
    if constexpr (kGated) {
        static_assert(kRowStep >= 16, "a thread meets one row");
        if (a.d32) {
#pragma unroll
            for (int s = 1; s < kCols * S; s *= 2) most = fmaxf(most, __shfl_xor(most, s));
            if (oc == 0 && os == 0 && om < M) a.tops[(size_t)g * M + om] = most;
        }
    }
    if constexpr (!kGated) {
        // a row's kCols S threads are neighbours in one wave
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
            float t = top[k], v = sum[k];
#pragma unroll
            for (int s = 1; s < kCols * S; s *= 2) {
                const float t2 = __shfl_xor(t, s), v2 = __shfl_xor(v, s);
                const float m2 = fmaxf(t, t2);
                v = m2 == -INFINITY ? v + v2 : v * __expf(t - m2) + v2 * __expf(t2 - m2);
                t = m2;
            }
            const int m = om + k * kRowStep;
            if (oc == 0 && os == 0 && m < M) a.part[(size_t)g * M + m] = make_float2(t, v);
        }
    }
}

template <bool kBF16, int kSub, bool kGated>
void launch_jp(const SmallArgs& a, int grid, hipStream_t s) {
    const int jp = (a.KB + kWaves - 1) / kWaves;
    if (jp <= 1) hipLaunchKernelGGL((small_kernel<kBF16, kSub, 1, kGated>), dim3(grid), dim3(kThreads), 0, s, a);
    else if (jp <= 2) hipLaunchKernelGGL((small_kernel<kBF16, kSub, 2, kGated>), dim3(grid), dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((small_kernel<kBF16, kSub, 4, kGated>), dim3(grid), dim3(kThreads), 0, s, a);
}

template <bool kGated>
void launch_any(const SmallArgs& a, int sub, bool bf16, int grid, hipStream_t s) {
    if (bf16) sub == 4 ? launch_jp<true, 4, kGated>(a, grid, s) : sub == 2 ? launch_jp<true, 2, kGated>(a, grid, s) : launch_jp<true, 1, kGated>(a, grid, s);
    else sub == 4 ? launch_jp<false, 4, kGated>(a, grid, s) : sub == 2 ? launch_jp<false, 2, kGated>(a, grid, s) : launch_jp<false, 1, kGated>(a, grid, s);
}

SmallArgs common(const uint16_t* x, const uint8_t* packed, int64_t M, int64_t K, int64_t N, int64_t G) {
    SmallArgs a{};
    a.x = x;
    a.packed = packed;
    a.M = (int)M;
    a.K = (int)K;
    a.N = (int)N;
    a.KB = (int)(K / kRowsPerBlock);
    a.UW = (int)padded_units(K, G);
    return a;
}

}  // namespace

bool small_product(int64_t M, int64_t K) { return M <= 16 && K <= 4 * kWaves * kRowsPerBlock; }

int small_workgroups(int64_t units) { return (int)(units < kTargetWorkgroups ? units : kTargetWorkgroups); }

hipError_t launch_gated_small(const GatedCall& q, hipStream_t stream) {
    SmallArgs a = common(q.x, q.packed, q.M, q.K, 2 * q.F, q.G);
    a.F = (int)q.F;
    a.U = (int)(q.F / 8);
    a.h = q.h;
    a.dh = q.dh;
    a.d32 = q.d ? q.d32 : nullptr;
    a.tops = q.tops;
    a.act = q.act;
    launch_any<true>(a, units_per_block(q.G), q.bf16, small_workgroups(a.U), stream);
    return hipGetLastError();
}

hipError_t launch_ce_small(const uint16_t* x, const int32_t* labels, const uint8_t* packed, int64_t M, int64_t K, int64_t V,
                           int64_t G, bool bf16, float* zsel, float* part, hipStream_t stream) {
    SmallArgs a = common(x, packed, M, K, V, G);
    a.U = (int)(padded_cols(V) / kColsPerBlock);
    a.labels = labels;
    a.zsel = zsel;
    a.part = reinterpret_cast<float2*>(part);
    launch_any<false>(a, units_per_block(G), bf16, small_workgroups(a.U), stream);
    return hipGetLastError();
}

}  // namespace w4a16
