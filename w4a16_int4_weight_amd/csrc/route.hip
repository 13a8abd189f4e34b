// The router of a mixture of experts: l = x R^T in fp64, scores, the T largest of each row.
//
// The choice is discrete, so l is summed in fp64: a product of two 16-bit values is exact there
// (22 bits at most), and the sums err in the 53rd bit. A wave forms one expert's l
// of a group of rows, the expert's weights in registers, its lanes splitting K in 16-byte
// pieces; 8 waves of a workgroup take 8 experts of the same rows. The workgroup that finishes
// its rows' last experts (a counter, as split_k.h has it) reads the l of its rows back and
// chooses, a wave a row: each lane holds every 64th expert, the largest of all lanes comes by
// row shifts, its owner by a ballot.
//
// Many rows (tile_kernel): 16 rows x 16 experts a workgroup, on the fp64 matrix cores, whose waves
// split K. They multiply no faster than the vector units, but each operand is converted once
// for 16 products instead of once for each. A second launch chooses, a wave a row: choosing for a
// tile's 16 rows in its last workgroup took 7 us more.
//
// Bound by latency: one row x 64 experts of 2048 9.1 us (launch 1.5, loads 2, the meeting 2.5, choosing 2);
// 512 rows x 128 experts 16.7 + 4.4 us, a quarter of the fp64 matrix rate: each wave loads its whole share at
// once, so nothing overlaps the loads, and waves wait for them 82% of their time.
#include "device_common.h"
#include "launch.h"
#include "split_k.h"
#include "wave.h"

namespace w4a16 {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kTile = 16;                   // rows and experts of a tile
constexpr int kTileWaves = 16;
constexpr int kChooseRows = 4;              // of a workgroup, a wave each
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
        acc[0] = fma((double)half_bits_to_f32<kBF16>(aw[i] & 0xFFFFu), (double)half_bits_to_f32<kBF16>(bw[i] & 0xFFFFu), acc[0]);
        acc[1] = fma((double)half_bits_to_f32<kBF16>(aw[i] >> 16), (double)half_bits_to_f32<kBF16>(bw[i] >> 16), acc[1]);
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
    bool none = false;                                    // some score is no number: no weight of the row is one
#pragma unroll
    for (int i = 0; i < N; ++i) {
        s[i] = a.sigmoid ? 1.0 / (1.0 + exp(-l[i])) : exp(l[i] - top);
        sum += lane + 64 * i < a.E ? s[i] : 0.0;
        none = none || (lane + 64 * i < a.E && s[i] != s[i]);
    }
    none = __ballot(none) != 0;
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
        const double w = none ? NAN : a.normalize ? (total == 0.0 ? 0.0 : mine / total) : mine / sum;
        a.ids[(size_t)m * a.T + lane] = my_id;
        a.weights[(size_t)m * a.T + lane] = (float)(w * (double)a.scale);
    }
}

// The workgroup that ends a group of rows, of `tiles`, chooses for it.
template <int N>
__device__ __forceinline__ void finish(const RouteArgs& a, int g, int tiles, int m0, int m1) {
    __shared__ int last;
    const int tid = (int)threadIdx.x, w = tid >> 6;
    __builtin_amdgcn_s_waitcnt(0);          // this wave's stores have completed
    __syncthreads();
    if (tid == 0)
        last = __hip_atomic_fetch_add(&a.counters[g], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)(tiles - 1);
    __syncthreads();
    if (!last) return;
    for (int m = m0 + w; m < m1; m += kWaves) choose<N>(a, m);
    if (tid == 0) __hip_atomic_store(&a.counters[g], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <bool kBF16, int N>
__global__ __launch_bounds__(kThreads) void route_kernel(const RouteArgs a) {
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
    finish<N>(a, g, tiles, m0, m1);
}

typedef double f64x4 __attribute__((ext_vector_type(4)));

template <bool kBF16>
__global__ __launch_bounds__(64 * kTileWaves) void tile_kernel(const RouteArgs a) {
    __shared__ double part[kTileWaves][4][64];
    const int tid = (int)threadIdx.x, w = tid >> 6, lane = tid & 63, c = lane & 15, h = lane >> 4;
    const int tiles = (a.E + kTile - 1) / kTile;
    const int g = (int)blockIdx.x / tiles, e0 = (int)blockIdx.x % tiles * kTile;
    const int m0 = g * kTile;
    // rows and experts past the last: the last, into results that are not stored
    const uint16_t* x = a.x + (size_t)(m0 + c < a.M ? m0 + c : a.M - 1) * a.K + 8 * h;
    const uint16_t* r = a.router + (size_t)(e0 + c < a.E ? e0 + c : a.E - 1) * a.K + 8 * h;
    f64x4 acc[4] = {};                       // (one sum would wait for each product)
    // step e multiplies element 8 h + e of the chunk of 32, h the step's index of the four
    auto multiply = [&](const uint4& xq, const uint4& rq) {
        const uint32_t xw[4] = {xq.x, xq.y, xq.z, xq.w}, rw[4] = {rq.x, rq.y, rq.z, rq.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double u = half_bits_to_f32<kBF16>(e & 1 ? xw[e / 2] >> 16 : xw[e / 2] & 0xFFFFu);
            const double v = half_bits_to_f32<kBF16>(e & 1 ? rw[e / 2] >> 16 : rw[e / 2] & 0xFFFFu);
            acc[e % 4] = __builtin_amdgcn_mfma_f64_16x16x4f64(u, v, acc[e % 4], 0, 0, 0);
        }
    };
    // each wave takes chunks that follow each other: whole lines
    const int chunks = a.K / 32, per = (chunks + kTileWaves - 1) / kTileWaves;
    const int end = (w + 1) * per < chunks ? (w + 1) * per : chunks;
    for (int i = w * per; i < end; i += 4) {
        uint4 xq[4], rq[4];
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = i + j;
            xq[j] = k < end ? *reinterpret_cast<const uint4*>(x + 32 * k) : none;
            rq[j] = k < end ? *reinterpret_cast<const uint4*>(r + 32 * k) : none;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) multiply(xq[j], rq[j]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) part[w][e][lane] = (acc[0][e] + acc[1][e]) + (acc[2][e] + acc[3][e]);
    __syncthreads();
    if (tid < kTile * kTile) {
        // register e of lane (c, h): row 4 e + h, expert c
        double l = 0.0;
#pragma unroll
        for (int k = 0; k < kTileWaves; ++k) l += part[k][w][lane];
        const int m = m0 + 4 * w + h, e = e0 + c;
        if (m < a.M && e < a.E)
            a.logits[(size_t)m * a.E + e] = __builtin_bit_cast(uint64_t, l);
    }
}

template <int N>
__global__ __launch_bounds__(64 * kChooseRows) void choose_kernel(const RouteArgs a) {
    const int m = (int)blockIdx.x * kChooseRows + ((int)threadIdx.x >> 6);
    if (m < a.M) choose<N>(a, m);
}

template <bool kBF16, int N>
void launch_n(RouteArgs& a, hipStream_t s) {
    // Tiles from 33 of them on (K = 2048, us without and with them: 64 rows x 64 experts 13.6, 18.4;
    // 128 x 64 23.3, 18.6; 512 x 128 78, 19.6)
    const int tiles = (a.E + kTile - 1) / kTile, row_tiles = (a.M + kTile - 1) / kTile;
    if (tiles * row_tiles > 32) {
        hipLaunchKernelGGL((tile_kernel<kBF16>), dim3(row_tiles * tiles), dim3(64 * kTileWaves), 0, s, a);
        hipLaunchKernelGGL((choose_kernel<N>), dim3((a.M + kChooseRows - 1) / kChooseRows), dim3(64 * kChooseRows), 0, s, a);
        return;
    }
    a.group = (a.M + kMaxSplitTiles - 1) / kMaxSplitTiles;        // one counter per group of rows
    const int groups = (a.M + a.group - 1) / a.group, parts = (a.E + kWaves - 1) / kWaves;
    hipLaunchKernelGGL((route_kernel<kBF16, N>), dim3(groups * parts), dim3(kThreads), 0, s, a);
}

template <bool kBF16>
void launch_typed(RouteArgs& a, hipStream_t s) {
    const int n = (a.E + 63) / 64;
    if (n == 1) launch_n<kBF16, 1>(a, s);
    else if (n == 2) launch_n<kBF16, 2>(a, s);
    else if (n <= 4) launch_n<kBF16, 4>(a, s);
    else launch_n<kBF16, kMaxExperts / 64>(a, s);
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
    if (q.bf16) launch_typed<true>(a, stream);
    else launch_typed<false>(a, stream);
    return hipGetLastError();
}

}  // namespace w4a16
