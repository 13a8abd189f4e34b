// The router of a mixture of experts: l = x R^T in fp64, scores, the T largest of each row.
//
// The choice is discrete, so l is summed in fp64: a product of two 16-bit values is exact in
// fp32 (22 bits at most), and its sums here err in the 53rd bit. A wave forms one expert's l
// of a group of rows, the expert's weights in registers, its lanes splitting K in 16-byte
// pieces; 8 waves of a workgroup take 8 experts of the same rows. The workgroup that finishes
// its rows' last experts (a counter, as split_k.h has it) reads the l of its rows back and
// chooses, a wave a row: each lane holds every 64th expert, the largest of all lanes comes by
// row shifts, its owner by a ballot.
#include "device_common.h"
#include "launch.h"
#include "split_k.h"
#include "wave.h"

namespace w4a16 {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kPieces = 4;                  // 16-byte pieces of the weights a lane holds: K up to 2048 at a time

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

template <bool kBF16>
__device__ __forceinline__ void dot8(const uint4& a, const uint4& b, double (&acc)[2]) {
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc[0] += (double)(half_bits_to_f32<kBF16>(aw[i] & 0xFFFFu) * half_bits_to_f32<kBF16>(bw[i] & 0xFFFFu));
        acc[1] += (double)(half_bits_to_f32<kBF16>(aw[i] >> 16) * half_bits_to_f32<kBF16>(bw[i] >> 16));
    }
}

// one row by one wave, N experts a lane
template <int N>
__device__ __forceinline__ void choose(const RouteArgs& a, int m) {
    const int lane = (int)threadIdx.x & 63;
    double l[N];
    double top = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = lane + 64 * i;
        const uint64_t* p = a.logits + (size_t)m * a.E + (e < a.E ? e : 0);
        l[i] = __builtin_bit_cast(double, __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (lane + 64 * i >= a.E) l[i] = -INFINITY;
        top = fmax(top, l[i]);
    }
    top = wave_max(top);
    // scores; softmax's are divided by their sum at the end, unless it leaves with `normalize`
    double s[N], sum = 0.0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        s[i] = a.sigmoid ? 1.0 / (1.0 + exp(-l[i])) : exp(l[i] - top);
        sum += lane + 64 * i < a.E ? s[i] : 0.0;
    }
    sum = a.sigmoid ? 1.0 : wave_sum(sum);
    // what the choice goes by: -infinity for no number, no number for what is taken or not there
    double by[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = lane + 64 * i;
        by[i] = a.bias ? s[i] / sum + (double)a.bias[e < a.E ? e : 0] : l[i];
        if (!(by[i] > -INFINITY)) by[i] = -INFINITY;
        if (e >= a.E) by[i] = NAN;
    }
    double mine = 0.0, total = 0.0;                       // lane j keeps the j-th
    int my_id = 0;
    for (int j = 0; j < a.T; ++j) {
        double best = by[0];
#pragma unroll
        for (int i = 1; i < N; ++i) best = fmax(best, by[i]);
        best = from_lane(wave_scan(best, (double)NAN, [](double x, double y) { return fmax(x, y); }), 63);
        // the lowest expert that has it
        bool found = false;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint64_t has = __ballot(by[i] == best);
            if (found || has == 0) continue;
            found = true;
            const int owner = __builtin_ctzll(has);
            const double w = from_lane(s[i], owner);
            total += w;
            if (lane == owner) by[i] = NAN;
            if (lane == j) {
                mine = w;
                my_id = owner + 64 * i;
            }
        }
    }
    if (lane < a.T) {
        const double w = a.normalize ? (total == 0.0 ? 0.0 : mine / total) : mine / sum;
        a.ids[(size_t)m * a.T + lane] = my_id;
        a.weights[(size_t)m * a.T + lane] = (float)(w * (double)a.scale);
    }
}

template <bool kBF16, int N>
__global__ __launch_bounds__(kThreads) void route_kernel(const RouteArgs a) {
    __shared__ int last;
    const int tid = (int)threadIdx.x, w = tid >> 6, lane = tid & 63;
    const int tiles = (a.E + kWaves - 1) / kWaves;
    const int g = (int)blockIdx.x / tiles, e = (int)blockIdx.x % tiles * kWaves + w;
    const int m0 = g * a.group, m1 = m0 + a.group < a.M ? m0 + a.group : a.M;
    if (e < a.E) {
        const uint4* r = reinterpret_cast<const uint4*>(a.router + (size_t)e * a.K);
        const int pieces = a.K / 8;
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        uint4 rw[kPieces];
#pragma unroll
        for (int p = 0; p < kPieces; ++p) rw[p] = lane + 64 * p < pieces ? r[lane + 64 * p] : none;
        for (int m = m0; m < m1; ++m) {
            const uint4* x = reinterpret_cast<const uint4*>(a.x + (size_t)m * a.K);
            double acc[2] = {0.0, 0.0};
            uint4 xw[kPieces];
#pragma unroll
            for (int p = 0; p < kPieces; ++p) xw[p] = lane + 64 * p < pieces ? x[lane + 64 * p] : none;
#pragma unroll
            for (int p = 0; p < kPieces; ++p) dot8<kBF16>(xw[p], rw[p], acc);
            for (int q = lane + 64 * kPieces; q < pieces; q += 64) dot8<kBF16>(x[q], r[q], acc);
            const double sum = wave_sum(acc[0] + acc[1]);
            if (lane == 0)
                __hip_atomic_store(a.logits + (size_t)m * a.E + e, __builtin_bit_cast(uint64_t, sum), __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    __builtin_amdgcn_s_waitcnt(0);          // this wave's stores have completed
    __syncthreads();
    if (tid == 0)
        last = __hip_atomic_fetch_add(&a.counters[g], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(tiles - 1);
    __syncthreads();
    if (!last) return;
    for (int m = m0 + w; m < m1; m += kWaves) choose<N>(a, m);
    if (tid == 0) __hip_atomic_store(&a.counters[g], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <bool kBF16>
void launch_typed(const RouteArgs& a, int grid, hipStream_t s) {
    const int n = (a.E + 63) / 64;
    if (n == 1) hipLaunchKernelGGL((route_kernel<kBF16, 1>), dim3(grid), dim3(kThreads), 0, s, a);
    else if (n == 2) hipLaunchKernelGGL((route_kernel<kBF16, 2>), dim3(grid), dim3(kThreads), 0, s, a);
    else if (n <= 4) hipLaunchKernelGGL((route_kernel<kBF16, 4>), dim3(grid), dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((route_kernel<kBF16, kMaxExperts / 64>), dim3(grid), dim3(kThreads), 0, s, a);
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
    if (q.bf16) launch_typed<true>(a, groups * tiles, stream);
    else launch_typed<false>(a, groups * tiles, stream);
    return hipGetLastError();
}

}  // namespace w4a16
