// The router of a mixture of experts: l = x R^T in fp64, scores, the T largest of each row.
//
// The choice is discrete, so l is summed in fp64: a product of two 16-bit values is exact in
// fp32 (22 bits at most), and its sums here err in the 53rd bit. A wave forms one expert's l
// of one row, its lanes splitting K in 16-byte pieces; 8 waves of a workgroup take 8 experts
// of the same rows. The workgroup that finishes its rows' last experts (a counter, as
// split_k.h has it) reads the l of its rows back and chooses: a wave a row, each lane holding
// every 64th expert.
#include "device_common.h"
#include "launch.h"
#include "split_k.h"

namespace w4a16 {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kMaxPerLane = kMaxExperts / 64;

struct RouteArgs {
    const uint16_t* x;
    const uint16_t* router;
    const float* bias;
    int M, K, E, T;
    int group;              // rows of a workgroup
    int sigmoid, normalize;
    float scale;
    int32_t* ids;
    float* weights;
    uint32_t* counters;     // one per group of rows
    uint64_t* logits;       // fp64 bits [M][E]
};

__device__ __forceinline__ double wave_sum(double v) {
    for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
    return v;
}
__device__ __forceinline__ double wave_max(double v) {
    for (int s = 32; s > 0; s >>= 1) v = fmax(v, __shfl_xor(v, s));
    return v;
}

template <bool kBF16>
__device__ __forceinline__ double dot8(const uint4& a, const uint4& b, double acc) {
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc += (double)(half_bits_to_f32<kBF16>(aw[i] & 0xFFFFu) * half_bits_to_f32<kBF16>(bw[i] & 0xFFFFu));
        acc += (double)(half_bits_to_f32<kBF16>(aw[i] >> 16) * half_bits_to_f32<kBF16>(bw[i] >> 16));
    }
    return acc;
}

// one row by one wave
__device__ __forceinline__ void choose(const RouteArgs& a, int m) {
    const int lane = (int)threadIdx.x & 63;
    double l[kMaxPerLane], by[kMaxPerLane];
    double top = -INFINITY;
    const int n = (a.E - lane + 63) / 64;                // experts lane, lane + 64, ...
#pragma unroll
    for (int i = 0; i < kMaxPerLane; ++i) {
        l[i] = by[i] = -INFINITY;
        if (i < n) {
            const uint64_t* p = a.logits + (size_t)m * a.E + lane + 64 * i;
            l[i] = __builtin_bit_cast(double, __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
            top = fmax(top, l[i]);
        }
    }
    top = wave_max(top);
    double sum = 0.0;
    if (!a.sigmoid) {
#pragma unroll
        for (int i = 0; i < kMaxPerLane; ++i)
            if (i < n) sum += exp(l[i] - top);
        sum = wave_sum(sum);
    }
    auto score = [&](double v) { return a.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - top) / sum; };
#pragma unroll
    for (int i = 0; i < kMaxPerLane; ++i)
        if (i < n) {
            by[i] = a.bias ? score(l[i]) + (double)a.bias[lane + 64 * i] : l[i];
            if (!(by[i] > -INFINITY)) by[i] = -INFINITY;  // no number: behind all others
        }
    uint32_t taken = 0;
    double mine = 0.0, total = 0.0;                       // lane j keeps the j-th weight
    int my_id = 0;
    for (int j = 0; j < a.T; ++j) {
        // (value, expert) of the lane's best that is left; ties to the lowest expert
        double v = 0.0, lv = 0.0;
        int e = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < kMaxPerLane; ++i)
            if (i < n && !((taken >> i) & 1u) && (e == 0x7FFFFFFF || by[i] > v)) {
                v = by[i];
                lv = l[i];
                e = lane + 64 * i;
            }
        for (int s = 32; s > 0; s >>= 1) {
            const double v2 = __shfl_xor(v, s), l2 = __shfl_xor(lv, s);
            const int e2 = __shfl_xor(e, s);
            if (e2 != 0x7FFFFFFF && (e == 0x7FFFFFFF || v2 > v || (v2 == v && e2 < e))) {
                v = v2;
                lv = l2;
                e = e2;
            }
        }
        if ((e & 63) == lane) taken |= 1u << (e >> 6);
        const double w = score(lv);
        total += w;
        if (lane == j) {
            mine = w;
            my_id = e;
        }
    }
    if (lane < a.T) {
        const double w = a.normalize ? (total == 0.0 ? 0.0 : mine / total) : mine;
        a.ids[(size_t)m * a.T + lane] = my_id;
        a.weights[(size_t)m * a.T + lane] = (float)(w * (double)a.scale);
    }
}

template <bool kBF16>
__global__ __launch_bounds__(kThreads) void route_kernel(const RouteArgs a) {
    __shared__ int last;
    const int tid = (int)threadIdx.x, w = tid >> 6, lane = tid & 63;
    const int tiles = (a.E + kWaves - 1) / kWaves;
    const int g = (int)blockIdx.x / tiles, e = (int)blockIdx.x % tiles * kWaves + w;
    const int m0 = g * a.group, m1 = m0 + a.group < a.M ? m0 + a.group : a.M;
    if (e < a.E) {
        const uint16_t* r = a.router + (size_t)e * a.K;
        for (int m = m0; m < m1; ++m) {
            const uint16_t* x = a.x + (size_t)m * a.K;
            double acc = 0.0;
            for (int k = 8 * lane; k < a.K; k += 512)
                acc = dot8<kBF16>(*reinterpret_cast<const uint4*>(x + k), *reinterpret_cast<const uint4*>(r + k), acc);
            acc = wave_sum(acc);
            if (lane == 0)
                __hip_atomic_store(a.logits + (size_t)m * a.E + e, __builtin_bit_cast(uint64_t, acc), __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    __builtin_amdgcn_s_waitcnt(0);          // this wave's stores have completed
    __syncthreads();
    if (tid == 0)
        last = __hip_atomic_fetch_add(&a.counters[g], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(tiles - 1);
    __syncthreads();
    if (!last) return;
    for (int m = m0 + w; m < m1; m += kWaves) choose(a, m);
    if (tid == 0) __hip_atomic_store(&a.counters[g], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace

size_t route_logits_bytes(int64_t M, int64_t E) { return (size_t)M * (size_t)E * 8; }

hipError_t launch_route(const RouteCall& q, hipStream_t stream) {
    RouteArgs a{};
    a.x = q.x;
    a.router = q.router;
    a.bias = q.bias;
    a.M = (int)q.M;
    a.K = (int)q.K;
    a.E = (int)q.E;
    a.T = (int)q.T;
    a.sigmoid = q.sigmoid;
    a.normalize = q.normalize;
    a.scale = q.scale;
    a.ids = q.ids;
    a.weights = q.weights;
    a.counters = q.counters;
    a.logits = reinterpret_cast<uint64_t*>(q.logits);
    // one counter per group of rows
    a.group = (int)((q.M + kMaxSplitTiles - 1) / kMaxSplitTiles);
    const int groups = (a.M + a.group - 1) / a.group, tiles = (a.E + kWaves - 1) / kWaves;
    if (q.bf16) hipLaunchKernelGGL((route_kernel<true>), dim3(groups * tiles), dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((route_kernel<false>), dim3(groups * tiles), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace w4a16
