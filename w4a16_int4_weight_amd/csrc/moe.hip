// Mixture of experts for up to 16 rows and 256 entries: the routed experts' codes are streamed once, in two
// launches. More rows, or K over 4096: moe_tile.hip.
//
// Bound by the time to read the routed experts' codes, so both kernels deal equal shares of
// them to the compute units. Each workgroup first makes the list of the experts that some row
// names, from ids (at most 256), in LDS; nothing on the host depends on it. The activations
// of all rows are one operand of 16 rows: it costs the matrix cores the same whether one row
// of it counts or all.
//
// up_kernel: a unit is 16 gate and 16 up columns of one listed expert over the whole of K.
// Workgroup g takes a contiguous share of the units, each of its waves a contiguous run of
// that share's chunks of 4 row blocks, whether it ends inside a unit or not: a unit that began in one
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
//
// Measured (2048 x 1024, 64 experts, 8 a row): one row 11.0 + 8.7 us, of which a launch takes 1.5,
// the ids and their list 2, the first codes 2 to 3 (16.8 and 8.4 MB), and the splits' meeting 2.3;
// 16 rows 32 us for 132 MB (4.1 TB/s; with the loads alone 31) and 24 us for 66 MB (decoding takes the vector units
// 46% of its cycles, both halves of h the matrix cores 18%, and the two waves of a SIMD wait 42% of
// theirs). A barrier a batch
// of units, as product_small.hip has it, took 39 us for up_kernel at 16 rows; two workgroups a compute unit
// 48 (up) and 30 us (down); 8 columns a down workgroup and no splits 50 us.
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
constexpr int kMaxEntries = 256;            // M T: what LDS holds beside 16 rows of 4096
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
    uint4 words[kMaxExperts / 128];         // a bit an expert
    int id[kMaxEntries];                    // of each entry
    int16_t expert[kMaxEntries];
    uint32_t rows[kMaxEntries];             // bit m: row m names expert[i]
};

// id: the entry of this thread's number, -1 past the last. Returns how many experts are
// listed; `place`: the position of this thread's entry among them.
__device__ __forceinline__ int make_list(const MoeArgs& a, Listed& l, int id, int* place) {
    const int tid = (int)threadIdx.x;
    uint32_t* words = reinterpret_cast<uint32_t*>(l.words);
    if (tid < kMaxExperts / 32) words[tid] = 0u;
    if (tid < kMaxEntries) l.rows[tid] = 0u;
    __syncthreads();
    if (id >= a.E) id = -1;
    if (tid < kMaxEntries) l.id[tid] = id;
    if (id >= 0) atomicOr(&words[id >> 5], 1u << (id & 31));
    __syncthreads();
    int count = 0, before = 0;
#pragma unroll
    for (int k = 0; k < kMaxExperts / 128; ++k) {
        const uint4 q = l.words[k];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t v = e == 0 ? q.x : e == 1 ? q.y : e == 2 ? q.z : q.w;
            const int own = (id >> 5) - (4 * k + e);       // > 0: a word below the id's
            before += __popc(own > 0 ? v : own == 0 ? v & ((1u << (id & 31)) - 1u) : 0u);
            count += __popc(v);
        }
    }
    if (id >= 0) {
        l.expert[before] = (int16_t)id;     // (every entry that names it writes the same)
        atomicOr(&l.rows[before], 1u << (tid / a.T));
    }
    *place = before;
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(count);
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

template <bool kBF16, int kSub, int kAct>
__global__ __launch_bounds__(kThreads) void up_kernel(const MoeArgs a) {
    constexpr int C = 4;                                   // row blocks of a chunk
    extern __shared__ uint4 xs[];                          // [KB][4][64]: operands of the rows, then X [KB kSub][16]
    __shared__ Listed list;
    __shared__ uint8_t entry_of[kMaxEntries][kMaxRows];    // the first entry of a row that names a listed expert
    __shared__ float row_weight[kMaxEntries];              // of each first entry: all the row's weights for its expert
    __shared__ f32x4 begun[kWaves][2][64];                 // a wave's part of the unit that an earlier one began
    float* entry_weight = reinterpret_cast<float*>(&begun[0][0][0]);      // (done with before the first unit ends)

    const int tid = (int)threadIdx.x;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63, c = lane & 15, h = lane >> 4;
    const int M = a.M, F = a.F, KB = a.K / kRowsPerBlock, UW = (int)padded_units(a.K, kRowsPerBlock / kSub);
    float* xsum = reinterpret_cast<float*>(xs + KB * 256);

    const int id = tid < M * a.T ? a.ids[tid] : -1;
    if (tid < M * a.T) entry_weight[tid] = a.weights[tid];
    // the rows' 16-byte chunks, chunk by chunk, a row each in turn; rows past M are left as they
    // are: they feed results that are not used
    {
        const int chunks = M * (a.K / 8);
        for (int t0 = tid; t0 < chunks; t0 += 4 * kThreads) {
            uint4 v[4];
            int to[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = t0 + j * kThreads < chunks ? t0 + j * kThreads : chunks - 1;
                const int q = t / M, m = t - q * M;
                to[j] = (q >> 2) * 64 + 16 * (q & 3) + m;
                v[j] = *reinterpret_cast<const uint4*>(a.x + (size_t)m * a.K + 8 * q);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) xs[to[j]] = v[j];
        }
    }
    int place;
    const int listed = make_list(a, list, id, &place);
    if (tid < kMaxEntries && list.id[tid] >= 0) {
        const int m = tid / a.T, e0 = m * a.T;
        float sum = 0.f;
        bool first = true;
        for (int j = e0; j < e0 + a.T; ++j)
            if (list.id[j] == id) {
                sum += entry_weight[j];
                first = first && j >= tid;
            }
        if (first) {
            entry_of[place][m] = (uint8_t)(tid - e0);
            row_weight[tid] = sum;
        }
    }

    const int per = F / 16, U = listed * per;              // units of an expert, of all
    const int nwg = (int)gridDim.x, g = xcd_share((int)blockIdx.x, nwg);
    const int lo = (int)((int64_t)g * U / nwg), hi = (int)((int64_t)(g + 1) * U / nwg);
    const int per_unit = (KB + C - 1) / C, chunks = (hi - lo) * per_unit;
    auto first_of = [&](int wave) { return (int)((int64_t)chunks * wave / kWaves); };
    const int c0 = first_of(w), c1 = first_of(w + 1);

    // a chunk: C row blocks of a unit, those past the last one with scales of 0
    struct Chunk {
        uint4 q[2][C];                                     // gate, up
        uint4 md[2][kSub];
    };
    // The chunk to load next. An odd run's last turn loads one more: its last chunk's first
    // lines again (steps of 0), so that the waits count the same in every turn.
    int lu = lo + c0 / per_unit, lk = c0 % per_unit, left = c1 - c0;
    const uint8_t* at = a.gate_up;
    const uint4* meta = reinterpret_cast<const uint4*>(a.gate_up);
    size_t up_codes = 0, up_meta = 0;
    uint32_t step = 0, meta_step = 0;
    auto enter = [&]() {
        const int i = lu / per, nb = lu - i * per;
        const uint8_t* base = a.gate_up + (int64_t)__builtin_amdgcn_readfirstlane((int)list.expert[i]) * a.gate_up_stride;
        at = base + (size_t)nb * KB * kBlockBytes + 16 * lane;
        meta = reinterpret_cast<const uint4*>(base + (size_t)a.K * F) + (size_t)(16 * nb + c) * (UW / 4);
    };
    auto issue = [&](Chunk& s) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
#pragma unroll
            for (int j = 0; j < C; ++j)
                s.q[p][j] = load_once(at + p * up_codes + (size_t)((uint32_t)(C * lk + j < KB ? C * lk + j : KB - 1) * step));
#pragma unroll
            for (int v = 0; v < kSub; ++v)
                s.md[p][v] = meta[p * up_meta + (uint32_t)(lk * kSub + v < UW / 4 ? lk * kSub + v : UW / 4 - 1) * meta_step];
        }
        if (--left <= 0) {
            up_codes = up_meta = 0;
            step = meta_step = 0;
        } else if (++lk == per_unit) {
            lk = 0;
            ++lu;
            enter();
        }
    };
    Chunk r0, r1;
    if (left > 0) {
        up_codes = (size_t)(F / kColsPerBlock) * KB * kBlockBytes;
        up_meta = (size_t)F * UW / 4;
        step = kBlockBytes;
        meta_step = 1;
        enter();
        issue(r0);
        if (left > 0) issue(r1);
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

    // rows 4 h + e, column c of a finished unit
    auto finish = [&](const f32x4 (&acc)[2], int u) {
        const int i = u / per;
        const uint32_t rows = list.rows[i] >> (4 * h);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (!((rows >> e) & 1u)) continue;
            const int m = 4 * h + e;
            const float weight = row_weight[m * a.T + entry_of[i][m]];
            float slope;
            const float o = acc[0][e] * gate_prob<kAct>(acc[0][e], &slope) * acc[1][e] * weight;
            const uint32_t top = f32_to_half_bits<true>(o);
            uint16_t* to = a.h + (((size_t)i * M + m) * 2) * F + 16 * (u - i * per) + c;
            to[0] = (uint16_t)top;
            to[F] = f32_to_half_bits<true>(o - bf16_bits_to_f32(top));
        }
    };
    int u = lo + c0 / per_unit, k = c0 % per_unit;         // the chunk to multiply next
    bool own = k == 0;                                     // the unit began in this wave
    f32x4 acc[2] = {zero, zero};
    auto multiply = [&](const Chunk& s) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const bool in = C * k + j < KB;
            const int kb = in ? C * k + j : KB - 1;
            f32x4 T[2][kSub];
            uint32_t md[2][kSub];
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int v = 0; v < kSub; ++v) md[p][v] = word_of(s.md[p][(j * kSub + v) / 4], (j * kSub + v) % 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int v = i * kSub / 4;
                const uint4 x = xs[(kb * 4 + i) * 64 + lane];
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    T[p][v] = mfma16x16x32<kBF16>(x, operand<kBF16>(word_of(s.q[p][j], i), md[p][v]), i % (4 / kSub) == 0 ? zero : T[p][v]);
            }
#pragma unroll
            for (int v = 0; v < kSub; ++v) {
                [[maybe_unused]] f32x4 X;
                if constexpr (kBF16) X = *reinterpret_cast<const f32x4*>(xsum + (kb * kSub + v) * 16 + 4 * h);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const float sc = in ? half_bits_to_f32<kBF16>(md[p][v] & 0xFFFFu) : 0.f;
                    const float zb = 16.f + (float)((md[p][v] >> 16) & 0xFu);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[p][e] = fmaf(sc, kBF16 ? fmaf(-zb, X[e], T[p][v][e]) : T[p][v][e], acc[p][e]);
                }
            }
        }
        if (++k == per_unit) {
            if (own) {
                finish(acc, u);
            } else {
                begun[w][0][lane] = acc[0];
                begun[w][1][lane] = acc[1];
            }
            acc[0] = acc[1] = zero;
            k = 0;
            own = true;
            ++u;
        }
    };
    int b = c0;
    for (; b + 2 < c1; b += 2) {
        multiply(r0);
        issue(r0);
        multiply(r1);
        issue(r1);
    }
    if (b < c1) multiply(r0);
    if (b + 1 < c1) multiply(r1);
    if (k && !own) {
        begun[w][0][lane] = acc[0];
        begun[w][1][lane] = acc[1];
    }
    __syncthreads();
    if (k && own) {
        // the waves that went on with the unit, in their order
        const int end = (u + 1 - lo) * per_unit;
        for (int v = w + 1; first_of(v) < end; ++v) {
            acc[0] += begun[v][0][lane];
            acc[1] += begun[v][1][lane];
        }
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
    int place;
    const int listed = make_list(a, list, tid < M * a.T ? a.ids[tid] : -1, &place);

    const int all = listed * FB;                       // row blocks of the whole sum
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
    const size_t lds = (size_t)KB * (4096 + 64 * kSub);    // 136 KiB at most, beside 23.8 of the kernel's own
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

bool moe_small(int64_t M, int64_t K, int64_t T) { return M <= kMaxRows && M * T <= kMaxEntries && K <= 4096; }

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
    const int64_t units = most_listed(q.M, q.E, q.T) * (q.F / 16);
    const int grid = (int)(units < kTargetWorkgroups ? units : kTargetWorkgroups);
    const int sub = units_per_block(q.G);
    if (q.bf16) return sub == 4 ? launch_sub<true, 4>(a, grid, stream) : sub == 2 ? launch_sub<true, 2>(a, grid, stream) : launch_sub<true, 1>(a, grid, stream);
    return sub == 4 ? launch_sub<false, 4>(a, grid, stream) : sub == 2 ? launch_sub<false, 2>(a, grid, stream) : launch_sub<false, 1>(a, grid, stream);
}

}  // namespace w4a16
