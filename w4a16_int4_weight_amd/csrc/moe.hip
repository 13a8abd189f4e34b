// Mixture of experts for up to 16 rows: the routed experts' codes are streamed once, in two
// launches. More rows, or K over 4096: moe_tile.hip.
//
// Bound by the time to read the routed experts' codes, so both kernels deal equal shares of
// them to the compute units. Each workgroup first makes the list of the experts that some row
// names, from ids (at most 512), in LDS; nothing on the host depends on it. The activations
// of all rows are one operand of 16 rows: it costs the matrix cores the same whether one row
// of it counts or all.
//
// up_kernel: a unit is 8 gate and 8 up columns of one listed expert over the whole of K.
// Workgroup g takes a contiguous share of the units, each of its waves a contiguous run of
// that share's chunks of 4 blocks of 1 KiB, whether it ends inside a unit or not: a unit that began in one
// wave and goes on in the next meets in LDS at the end, the only barrier behind the first
// loads. h is multiplied by the row's weight for the expert, so that the down projections add
// up, and left in two bf16 values (16 bits: one would be off by as much as the result's own
// rounding; fp16 overflows where bf16 models do not).
//
// down_kernel: one sum over (listed expert, row of Wd). Workgroup (columns, split) takes 64
// columns and a share of that sum's row blocks, each wave every 8th of them; rows that an
// expert does not serve are zero operands and load nothing. The waves' sums meet in LDS, the
// splits' in the workspace in split order (split_k.h's way): results do not depend on timing.
//
// Per metadata unit: s (T - (16 + z) X), T = sum x (16 + q), as product_small.hip has it; fp16
// activations take q - z exactly in 16 bits.
#include "device_common.h"
#include "gate.h"
#include "launch.h"
#include "split_k.h"

namespace w4a16 {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kTargetWorkgroups = 256;      // one per compute unit
constexpr int kMaxRows = 16;
constexpr int kMaxEntries = kMaxRows * kMaxChosen;
constexpr int kDownBlocks = 4;              // 16-column blocks of a down workgroup
constexpr int kDownColumns = kDownBlocks * kColsPerBlock;
static_assert(kMaxEntries <= kThreads, "a thread an entry");

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

struct MoeArgs {
    const uint16_t* x;
    const int32_t* ids;
    const float* weights;
    const uint8_t* gate_up;
    const uint8_t* down;
    int64_t gate_up_stride, down_stride;
    const uint16_t* residual;
    uint16_t* y;
    uint16_t* h;            // [listed experts][M][2][F] bf16
    uint32_t* counters;
    float* partials;        // [column groups][splits][16][64]
    int M, K, F, E, T;
    int splits;
    int act;
};

// The experts that some row names, in rising order, and which rows name each.
struct Listed {
    uint32_t words[kMaxExperts / 32];
    int before[kMaxExperts / 32];
    int count;
    int id[kMaxEntries];                    // of each entry
    int16_t expert[kMaxEntries];
    uint32_t rows[kMaxEntries];             // bit m: row m names expert[i]
};

// an id's position among the listed experts
__device__ __forceinline__ int place(const Listed& l, int e) {
    return l.before[e >> 5] + __popc(l.words[e >> 5] & ((1u << (e & 31)) - 1u));
}

// id: the entry of this thread's number, -1 past the last
__device__ __forceinline__ void make_list(const MoeArgs& a, Listed& l, int id) {
    const int tid = (int)threadIdx.x;
    if (id >= a.E) id = -1;
    if (tid < kMaxExperts / 32) l.words[tid] = 0u;
    l.id[tid] = id;
    l.rows[tid] = 0u;
    __syncthreads();
    if (id >= 0) atomicOr(&l.words[id >> 5], 1u << (id & 31));
    __syncthreads();
    if (tid < 64) {
        const int own = tid < kMaxExperts / 32 ? __popc(l.words[tid]) : 0;
        int sum = own;
        for (int s = 1; s < 32; s <<= 1) {
            const int o = __shfl_up(sum, s);
            if (tid >= s) sum += o;
        }
        if (tid < kMaxExperts / 32) l.before[tid] = sum - own;
        if (tid == kMaxExperts / 32 - 1) l.count = sum;
    }
    __syncthreads();
    if (id >= 0) {
        const int i = place(l, id);
        l.expert[i] = (int16_t)id;          // (every entry that names it writes the same)
        atomicOr(&l.rows[i], 1u << (tid / a.T));
    }
    __syncthreads();
}

__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
}

__device__ __forceinline__ uint32_t word_of(const uint4& q, int i) { return i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w; }

// the operand of 8 codes: 16 + q in bf16, or q - z in fp16
template <bool kBF16>
__device__ __forceinline__ uint4 operand(uint32_t d, uint32_t md) {
    uint32_t p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (kBF16) p[e] = ((e == 0 ? d << 3 : d >> (4 * e - 3)) & 0x00780078u) | 0x41804180u;
        else p[e] = ((d >> (4 * e)) & 0x000F000Fu) | Magic<false>::kBase2;
    }
    if constexpr (!kBF16) {
        const _Float16 zb = (_Float16)(1024.0f + (float)((md >> 16) & 0xFu));
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, p[e]) - f16x2{zb, zb});
    }
    return make_uint4(p[0], p[1], p[2], p[3]);
}

// lane c of each 16 takes lane c + 8's (mod 16)
__device__ __forceinline__ uint32_t turn8(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, true);
}
__device__ __forceinline__ float turn8(float v) { return __uint_as_float(turn8(__float_as_uint(v))); }

template <bool kBF16, int kSub, int kAct>
__global__ __launch_bounds__(kThreads) void up_kernel(const MoeArgs a) {
    constexpr int C = 4, D = kSub == 4 ? 2 : 3;            // row blocks of a chunk, chunks on their way per wave
    extern __shared__ uint4 xs[];                          // [KB][4][64]: operands of the rows, then X [KB kSub][16]
    __shared__ Listed list;
    __shared__ uint8_t entry_of[kMaxEntries][kMaxRows];    // the first entry of a row that names a listed expert
    __shared__ float row_weight[kMaxEntries];              // of each first entry: all the row's weights for its expert
    __shared__ f32x4 begun[kWaves][64];                    // a wave's part of the unit that an earlier one began
    float* entry_weight = reinterpret_cast<float*>(&begun[0][0]);      // (done with before the first unit ends)

    const int tid = (int)threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63, c = lane & 15, h = lane >> 4;
    const int M = a.M, F = a.F, KB = a.K / kRowsPerBlock, UW = (int)padded_units(a.K, kRowsPerBlock / kSub);
    float* xsum = reinterpret_cast<float*>(xs + KB * 256);

    const int id = tid < M * a.T ? a.ids[tid] : -1;
    entry_weight[tid] = tid < M * a.T ? a.weights[tid] : 0.f;
    // rows past M are left as they are: they feed results that are not used
    {
        const int m = tid & 15;
        const uint16_t* xr = a.x + (size_t)m * a.K;
        if (m < M)
            for (int q = tid >> 4; q < a.K / 8; q += kThreads / 16)
                xs[(q >> 2) * 64 + 16 * (q & 3) + m] = *reinterpret_cast<const uint4*>(xr + 8 * q);
    }
    make_list(a, list, id);
    if (list.id[tid] >= 0) {
        const int m = tid / a.T, e0 = m * a.T;
        float sum = 0.f;
        bool first = true;
        for (int j = e0; j < e0 + a.T; ++j)
            if (list.id[j] == id) {
                sum += entry_weight[j];
                first = first && j >= tid;
            }
        if (first) {
            entry_of[place(list, id)][m] = (uint8_t)(tid - e0);
            row_weight[tid] = sum;
        }
    }

    const int per = F / 8, U = list.count * per;           // units of an expert, of all
    const int nwg = (int)gridDim.x, g = xcd_share((int)blockIdx.x, nwg);
    const int lo = (int)((int64_t)g * U / nwg), hi = (int)((int64_t)(g + 1) * U / nwg);
    const int per_unit = (KB + C - 1) / C, chunks = (hi - lo) * per_unit;
    auto first_of = [&](int wave) { return (int)((int64_t)chunks * wave / kWaves); };
    const int c0 = first_of(w), c1 = first_of(w + 1);

    // a chunk: C row blocks of a unit, those past the last one with scales of 0
    struct Chunk {
        uint4 q[C];
        uint4 md[kSub];
    };
    int lu = lo + c0 / per_unit, lk = c0 % per_unit;       // the chunk to load next
    const uint8_t* at;
    const uint4* meta;
    auto enter = [&]() {
        const int i = lu / per;
        const uint8_t* base = a.gate_up + (int64_t)__builtin_amdgcn_readfirstlane((int)list.expert[i]) * a.gate_up_stride;
        const int n = (c >> 3) * F + 8 * (lu - i * per) + (c & 7);
        at = base + ((size_t)(n >> 4) * KB) * kBlockBytes + 16 * (16 * h + (n & 15));
        meta = reinterpret_cast<const uint4*>(base + (size_t)a.K * F + (size_t)n * UW * 4);
    };
    auto issue = [&](Chunk& s) {
#pragma unroll
        for (int j = 0; j < C; ++j) s.q[j] = load_once(at + (size_t)(C * lk + j < KB ? C * lk + j : KB - 1) * kBlockBytes);
#pragma unroll
        for (int v = 0; v < kSub; ++v) s.md[v] = meta[lk * kSub + v < UW / 4 ? lk * kSub + v : UW / 4 - 1];
        if (++lk == per_unit) {                            // past the share's end the last unit repeats
            lk = 0;
            if (lu + 1 < hi) {
                ++lu;
                enter();
            }
        }
    };
    Chunk ring[D];
    if (c0 < c1) {
        enter();
#pragma unroll
        for (int d = 0; d < D; ++d) issue(ring[d]);
    }
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    if constexpr (kBF16) {
        const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
        for (int kb = w; kb < KB; kb += kWaves) {
            f32x4 X[kSub];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int u = i * kSub / 4;
                X[u] = mfma16x16x32<true>(xs[(kb * 4 + i) * 64 + lane], ones, i % (4 / kSub) == 0 ? zero : X[u]);
            }
            if (c == 0) {
#pragma unroll
                for (int u = 0; u < kSub; ++u) *reinterpret_cast<f32x4*>(xsum + (kb * kSub + u) * 16 + 4 * h) = X[u];
            }
        }
    }
    __syncthreads();

    // rows 4 h + e, column c of a finished unit: lanes c < 8 make h of rows 4 h, 4 h + 1, the others of the next two
    auto finish = [&](const f32x4 acc, int u) {
        const int i = u / per;
        const uint32_t rows = list.rows[i];
        const bool lower = c < 8;
        const f32x4 other = {turn8(acc[0]), turn8(acc[1]), turn8(acc[2]), turn8(acc[3])};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int m = 4 * h + e + (lower ? 0 : 2);
            if (!((rows >> m) & 1u)) continue;
            const float gv = lower ? acc[e] : other[2 + e], uv = lower ? other[e] : acc[2 + e];
            const float weight = row_weight[m * a.T + entry_of[i][m]];
            float slope;
            const float pr = gate_prob<kAct>(gv, &slope);
            const float o = gv * pr * uv * weight;
            const uint32_t top = f32_to_half_bits<true>(o);
            uint16_t* to = a.h + (((size_t)i * M + m) * 2) * F + 8 * (u - i * per) + (c & 7);
            to[0] = (uint16_t)top;
            to[F] = f32_to_half_bits<true>(o - bf16_bits_to_f32(top));
        }
    };
    int u = lo + c0 / per_unit, k = c0 % per_unit;         // the chunk to multiply next
    bool own = k == 0;                                     // the unit began in this wave
    f32x4 acc = zero;
    auto multiply = [&](const Chunk& s) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const bool in = C * k + j < KB;
            const int kb = in ? C * k + j : KB - 1;
            f32x4 T[kSub];
            uint32_t md[kSub];
#pragma unroll
            for (int v = 0; v < kSub; ++v) md[v] = word_of(s.md[(j * kSub + v) / 4], (j * kSub + v) % 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int v = i * kSub / 4;
                T[v] = mfma16x16x32<kBF16>(xs[(kb * 4 + i) * 64 + lane], operand<kBF16>(word_of(s.q[j], i), md[v]),
                                           i % (4 / kSub) == 0 ? zero : T[v]);
            }
#pragma unroll
            for (int v = 0; v < kSub; ++v) {
                const float sc = in ? half_bits_to_f32<kBF16>(md[v] & 0xFFFFu) : 0.f;
                if constexpr (kBF16) {
                    const float zb = 16.f + (float)((md[v] >> 16) & 0xFu);
                    const f32x4 X = *reinterpret_cast<const f32x4*>(xsum + (kb * kSub + v) * 16 + 4 * h);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[e] = fmaf(sc, fmaf(-zb, X[e], T[v][e]), acc[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[e] = fmaf(sc, T[v][e], acc[e]);
                }
            }
        }
        if (++k == per_unit) {
            if (own) finish(acc, u);
            else begun[w][lane] = acc;
            acc = zero;
            k = 0;
            own = true;
            ++u;
        }
    };
    for (int b = c0; b < c1; b += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (b + d < c1) multiply(ring[d]);
            issue(ring[d]);
        }
    }
    if (k && !own) begun[w][lane] = acc;
    __syncthreads();
    if (k && own) {
        // the waves that went on with the unit, in their order
        const int end = (u + 1 - lo) * per_unit;
        for (int v = w + 1; first_of(v) < end; ++v) acc += begun[v][lane];
        finish(acc, u);
    }
}

template <bool kBF16, int kSub>
__global__ __launch_bounds__(kThreads) void down_kernel(const MoeArgs a) {
    constexpr int CB = kDownBlocks;
    __shared__ f32x4 part[kWaves][CB][64];
    __shared__ Listed list;
    __shared__ int last;
    const int tid = (int)threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63, c = lane & 15, h = lane >> 4;
    const int M = a.M, K = a.K, F = a.F, FB = F / kRowsPerBlock, UW = (int)padded_units(F, kRowsPerBlock / kSub);
    const int groups = K / kDownColumns;
    const int group = (int)blockIdx.x % groups, split = (int)blockIdx.x / groups;
    make_list(a, list, tid < M * a.T ? a.ids[tid] : -1);

    const int all = list.count * FB;                       // row blocks of the whole sum
    const int lo = (int)((int64_t)all * split / a.splits), hi = (int)((int64_t)all * (split + 1) / a.splits);
    struct Batch {
        uint4 q[CB];
        uint32_t md[CB][kSub];
        uint4 x[2][4];
    };
    auto load = [&](Batch& b, int r) {
        const int i = r / FB, fb = r - i * FB;
        const uint8_t* base = a.down + (int64_t)__builtin_amdgcn_readfirstlane((int)list.expert[i]) * a.down_stride;
#pragma unroll
        for (int j = 0; j < CB; ++j) {
            const int nb = group * CB + j;
            b.q[j] = load_once(base + ((size_t)nb * FB + fb) * kBlockBytes + 16 * lane);
            const uint32_t* m = reinterpret_cast<const uint32_t*>(base + (size_t)F * K / 2) + (size_t)(16 * nb + c) * UW + fb * kSub;
#pragma unroll
            for (int u = 0; u < kSub; ++u) b.md[j][u] = __builtin_nontemporal_load(m + u);
        }
        const bool serves = (list.rows[i] >> c) & 1u;
        const uint16_t* x = a.h + (((size_t)i * M + c) * 2) * F + (size_t)fb * kRowsPerBlock + 8 * h;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                b.x[k][t] = serves ? *reinterpret_cast<const uint4*>(x + (size_t)k * F + 32 * t) : make_uint4(0u, 0u, 0u, 0u);
    };
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    f32x4 acc[CB];
#pragma unroll
    for (int j = 0; j < CB; ++j) acc[j] = zero;
    auto multiply = [&](const Batch& b) {
        const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
        f32x4 X[kSub];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int u = t * kSub / 4;
            X[u] = mfma16x16x32<true>(b.x[1][t], ones, t % (4 / kSub) == 0 ? zero : X[u]);
            X[u] = mfma16x16x32<true>(b.x[0][t], ones, X[u]);
        }
#pragma unroll
        for (int j = 0; j < CB; ++j) {
            f32x4 T[kSub];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int u = t * kSub / 4;
                const uint4 codes = operand<true>(word_of(b.q[j], t), 0u);
                T[u] = mfma16x16x32<true>(b.x[1][t], codes, t % (4 / kSub) == 0 ? zero : T[u]);
                T[u] = mfma16x16x32<true>(b.x[0][t], codes, T[u]);
            }
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                const float sc = half_bits_to_f32<kBF16>(b.md[j][u] & 0xFFFFu);
                const float zb = 16.f + (float)((b.md[j][u] >> 16) & 0xFu);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(sc, fmaf(-zb, X[u][e], T[u][e]), acc[j][e]);
            }
        }
    };
    constexpr int D = 2;                                   // row blocks on their way per wave
    Batch ring[D];
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (lo + w + d * kWaves < hi) load(ring[d], lo + w + d * kWaves);
    for (int r = lo + w; r < hi; r += D * kWaves) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (r + d * kWaves < hi) multiply(ring[d]);
            if (r + (d + D) * kWaves < hi) load(ring[d], r + (d + D) * kWaves);
        }
    }
#pragma unroll
    for (int j = 0; j < CB; ++j) part[w][j][lane] = acc[j];
    __syncthreads();
    // thread t: column t % 64 of the group, rows t / 64 and t / 64 + 8
    const int oc = tid % kDownColumns, om = tid / kDownColumns;
    auto total = [&](int m) {
        float v = 0.f;
        const int at = 16 * (m >> 2) + (oc & 15), e = m & 3;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) v += reinterpret_cast<const float*>(&part[i][oc >> 4][at])[e];
        return v;
    };
    static_assert(kThreads / kDownColumns * 2 == kMaxRows, "two rows a thread");
    float v[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (om + 8 * k < M) v[k] = total(om + 8 * k);
    if (a.splits > 1) {
        auto slot = [&](int s, int m) { return a.partials + (((size_t)group * a.splits + s) * kMaxRows + m) * kDownColumns + oc; };
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (om + 8 * k < M) __hip_atomic_store(slot(split, om + 8 * k), v[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __builtin_amdgcn_s_waitcnt(0);          // this wave's stores have completed
        __syncthreads();
        if (tid == 0)
            last = __hip_atomic_fetch_add(&a.counters[group], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(a.splits - 1);
        __syncthreads();
        if (!last) return;
        float sum[2] = {0.f, 0.f};
        for (int s0 = 0; s0 < a.splits; s0 += 8) {
            float got[8][2];
#pragma unroll
            for (int s = 0; s < 8; ++s)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    got[s][k] = s0 + s < a.splits && om + 8 * k < M
                                    ? __hip_atomic_load(slot(s0 + s, om + 8 * k), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.f;
#pragma unroll
            for (int s = 0; s < 8; ++s)
#pragma unroll
                for (int k = 0; k < 2; ++k) sum[k] += got[s][k];
        }
        v[0] = sum[0];
        v[1] = sum[1];
        if (tid == 0) __hip_atomic_store(&a.counters[group], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int m = om + 8 * k;
        if (m >= M) continue;
        const size_t at = (size_t)m * K + group * kDownColumns + oc;
        if (a.residual) v[k] += half_bits_to_f32<kBF16>(a.residual[at]);
        a.y[at] = f32_to_half_bits<kBF16>(v[k]);
    }
}

template <bool kBF16, int kSub>
hipError_t launch_sub(const MoeArgs& a, int grid, hipStream_t s) {
    const int KB = a.K / kRowsPerBlock;
    const size_t lds = (size_t)KB * (4096 + 64 * kSub);    // 136 KiB at most, beside 23.3 of the kernel's own
    if (a.act == 0) hipLaunchKernelGGL((up_kernel<kBF16, kSub, 0>), dim3(grid), dim3(kThreads), lds, s, a);
    else if (a.act == 1) hipLaunchKernelGGL((up_kernel<kBF16, kSub, 1>), dim3(grid), dim3(kThreads), lds, s, a);
    else hipLaunchKernelGGL((up_kernel<kBF16, kSub, 2>), dim3(grid), dim3(kThreads), lds, s, a);
    hipLaunchKernelGGL((down_kernel<kBF16, kSub>), dim3(a.K / kDownColumns * a.splits), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

int64_t most_listed(int64_t M, int64_t E, int64_t T) { return E < M * T ? E : M * T; }

// Workgroups that share 64 columns of the down projection: those that fill the chip, each with
// a row block for every wave where all entries name different experts.
int down_splits(int64_t M, int64_t K, int64_t F, int64_t E, int64_t T) {
    const int64_t want = kTargetWorkgroups / (K / kDownColumns), most = most_listed(M, E, T) * (F / kRowsPerBlock) / kWaves;
    const int64_t n = want < most ? want : most;
    return n < 1 ? 1 : (int)n;
}

size_t h_bytes(int64_t M, int64_t F, int64_t E, int64_t T) {
    return ((size_t)most_listed(M, E, T) * (size_t)(4 * M * F) + 255) / 256 * 256;
}

}  // namespace

bool moe_small(int64_t M, int64_t K) { return M <= kMaxRows && K <= 4096; }

size_t moe_small_scratch(int64_t M, int64_t K, int64_t F, int64_t E, int64_t T) {
    const int splits = down_splits(M, K, F, E, T);
    return h_bytes(M, F, E, T) + (splits > 1 ? (size_t)splits * kMaxRows * (size_t)K * 4 : 0);
}

hipError_t launch_moe_small(const MoeCall& q, uint32_t* counters, uint8_t* scratch, hipStream_t stream) {
    MoeArgs a{};
    a.x = q.x;
    a.ids = q.ids;
    a.weights = q.weights;
    a.gate_up = q.gate_up;
    a.down = q.down;
    a.gate_up_stride = q.gate_up_stride;
    a.down_stride = q.down_stride;
    a.residual = q.residual;
    a.y = q.y;
    a.h = reinterpret_cast<uint16_t*>(scratch);
    a.counters = counters;
    a.partials = reinterpret_cast<float*>(scratch + h_bytes(q.M, q.F, q.E, q.T));
    a.splits = down_splits(q.M, q.K, q.F, q.E, q.T);
    a.M = (int)q.M;
    a.K = (int)q.K;
    a.F = (int)q.F;
    a.E = (int)q.E;
    a.T = (int)q.T;
    a.act = q.act;
    const int64_t units = most_listed(q.M, q.E, q.T) * (q.F / 8);
    const int grid = (int)(units < kTargetWorkgroups ? units : kTargetWorkgroups);
    const int sub = units_per_block(q.G);
    if (q.bf16) return sub == 4 ? launch_sub<true, 4>(a, grid, stream) : sub == 2 ? launch_sub<true, 2>(a, grid, stream) : launch_sub<true, 1>(a, grid, stream);
    return sub == 4 ? launch_sub<false, 4>(a, grid, stream) : sub == 2 ? launch_sub<false, 2>(a, grid, stream) : launch_sub<false, 1>(a, grid, stream);
}

}  // namespace w4a16
