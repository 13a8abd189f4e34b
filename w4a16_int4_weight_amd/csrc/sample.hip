// Draws a token from each row of logits: temperature, top-k, top-p, min-p, one uniform number.
//
//   w[v] = e^((z[v] - max z) / t);  kept: the k largest z, of these the shortest falling run
//   that reaches p of their weight, of these w >= min_p;  the token: the first v in rising
//   order whose running sum of kept w exceeds u times the whole.
//
// Logits are compared as whole numbers (order-preserving keys), thresholds are found digit by
// digit from the top: counts for k, sums of weights in 64-bit fixed point for p (whole numbers,
// so that the order of the additions changes nothing). Ties at a threshold go to the lowest
// index. The draw itself adds w in fp64, in index order by fixed pieces.
//
// One workgroup a row.
#include "device_common.h"
#include "launch.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kVec = 8;                         // consecutive logits of a thread
constexpr int kTile = kThreads * kVec;

struct SampleArgs {
    const void* logits;
    int64_t ld;
    int M, V;
    int unit_shift;         // a weight's fixed-point step is 2^-unit_shift
    const float* u;
    float temperature, top_p, min_p;
    int top_k;
    const float* temperatures;
    const int32_t* top_ks;
    const float* top_ps;
    const float* min_ps;
    int32_t* ids;
    float* logprob;
    int aligned;            // rows on 16-byte boundaries
};

// kKind: 0 fp16, 1 bf16, 2 fp32. Values of the type take the top kBits of an fp32 key.
template <int kKind> struct Logit {
    static constexpr int kBits = kKind == 0 ? 19 : kKind == 1 ? 16 : 32;
    static __device__ __forceinline__ float one(const void* row, int i) {
        if constexpr (kKind == 2) return static_cast<const float*>(row)[i];
        else return half_bits_to_f32<kKind == 1>(static_cast<const uint16_t*>(row)[i]);
    }
    // logits i .. i + 7; -infinity for what is no number and past the end
    static __device__ __forceinline__ void eight(const void* row, int i, int V, bool aligned, float (&z)[kVec]) {
        if (aligned && i + kVec <= V) {
            if constexpr (kKind == 2) {
                const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(row) + i);
                const f32x4 lo = p[0], hi = p[1];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    z[e] = lo[e];
                    z[4 + e] = hi[e];
                }
            } else {
                const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + i);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    z[2 * e] = half_bits_to_f32<kKind == 1>(w[e] & 0xFFFFu);
                    z[2 * e + 1] = half_bits_to_f32<kKind == 1>(w[e] >> 16);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) z[e] = i + e < V ? one(row, i + e) : -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) z[e] = z[e] == z[e] ? z[e] + 0.f : -INFINITY;      // -0 as 0
    }
    // rises with z
    static __device__ __forceinline__ uint32_t key(float z) {
        const uint32_t b = __float_as_uint(z);
        return ((b & 0x80000000u) ? ~b : b | 0x80000000u) >> (32 - kBits);
    }
};

struct Bins {
    uint32_t count[256];
    unsigned long long mass[256];
};

// the bin, from the top, in which `want` is reached, and what lies above it
struct Found {
    int bin;
    uint64_t above;
};

template <int kKind>
__global__ __launch_bounds__(kThreads) void sample_kernel(const SampleArgs a) {
    using L = Logit<kKind>;
    __shared__ Bins bins;
    __shared__ double wave_part[kWaves];
    __shared__ int wave_int[kWaves];
    __shared__ uint64_t box[2];
    __shared__ int ibox;
    const int tid = (int)threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int m = (int)blockIdx.x, V = a.V;
    const void* row = static_cast<const uint8_t*>(a.logits) + (int64_t)m * a.ld * (kKind == 2 ? 4 : 2);
    const bool aligned = a.aligned != 0;
    const float t = a.temperatures ? a.temperatures[m] : a.temperature;
    const bool greedy = !(t > 0.f);
    const int kk = greedy ? 1 : a.top_ks ? a.top_ks[m] : a.top_k;
    const bool limit_k = kk >= 1 && kk < V;
    const float pf = a.top_ps ? a.top_ps[m] : a.top_p;
    const bool limit_p = !greedy && pf < 1.f;
    const double p = (double)fmaxf(pf, 0.f);
    const float mf = a.min_ps ? a.min_ps[m] : a.min_p;
    const double min_w = mf > 0.f ? (double)fminf(mf, 1.f) : 0.0;
    float uf = a.u[m];
    uf = uf > 0.f ? uf : 0.f;
    const double inv_t = greedy ? 0.0 : 1.0 / (double)t;

    // ---- largest logit
    float top = -INFINITY;
    for (int i = kVec * tid; i < V; i += kTile) {
        float z[kVec];
        L::eight(row, i, V, aligned, z);
#pragma unroll
        for (int e = 0; e < kVec; ++e) top = fmaxf(top, z[e]);
    }
    for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
    if (lane == 0) wave_part[wv] = (double)top;
    __syncthreads();
    for (int k = 0; k < kWaves; ++k) top = fmaxf(top, (float)wave_part[k]);
    if (top == -INFINITY) {
        if (tid == 0) {
            a.ids[m] = -1;
            if (a.logprob) a.logprob[m] = -INFINITY;
        }
        return;
    }
    auto weight = [&](float z) -> double {
        return z == top ? 1.0 : z == -INFINITY ? 0.0 : exp(((double)z - (double)top) * inv_t);
    };
    const double unit = (double)(1ull << a.unit_shift);
    auto fixed = [&](double w) { return (unsigned long long)__double2ull_rn(w * unit); };

    constexpr int kPasses = (L::kBits + 7) / 8;
    auto shift_of = [](int pass) { return L::kBits - 8 * (pass + 1) > 0 ? L::kBits - 8 * (pass + 1) : 0; };
    auto clear = [&]() {
        __syncthreads();
        if (tid < 256) {
            bins.count[tid] = 0u;
            bins.mass[tid] = 0ull;
        }
        __syncthreads();
    };

    // ---- the k-th largest: key, and how many of its ties are kept
    uint32_t cut = 0;                 // keys above it are kept,
    int ties = 0x7FFFFFFF;            // of those equal to it the first `ties`
    if (limit_k) {
        uint32_t prefix = 0;
        int left = kk;
        for (int pass = 0; pass < kPasses; ++pass) {
            const int sh = shift_of(pass), width = (pass == kPasses - 1 ? L::kBits - 8 * pass : 8);
            clear();
            for (int i = kVec * tid; i < V; i += kTile) {
                float z[kVec];
                L::eight(row, i, V, aligned, z);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const uint32_t key = L::key(z[e]);
                    if ((pass == 0 || key >> (sh + width) == prefix) && i + e < V) atomicAdd(&bins.count[(key >> sh) & ((1u << width) - 1u)], 1u);
                }
            }
            __syncthreads();
            if (tid == 0) {
                int above = 0, b = (1 << width) - 1;
                while (b > 0 && above + (int)bins.count[b] < left) above += (int)bins.count[b--];
                box[0] = (uint64_t)b;
                ibox = left - above;
            }
            __syncthreads();
            prefix = prefix << width | (uint32_t)box[0];
            left = ibox;
        }
        cut = prefix;
        ties = left;
    }

    // ---- top-p's threshold within what is left
    if (limit_p) {
        const uint32_t kcut = cut;
        const int kties = ties;
        uint32_t prefix = 0;
        uint64_t above = 0;
        double target = 0.0;
        for (int pass = 0; pass < kPasses; ++pass) {
            const int sh = shift_of(pass), width = (pass == kPasses - 1 ? L::kBits - 8 * pass : 8);
            const uint32_t mask = (1u << width) - 1u;
            clear();
            for (int i = kVec * tid; i < V; i += kTile) {
                float z[kVec];
                L::eight(row, i, V, aligned, z);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const uint32_t key = L::key(z[e]);
                    if ((pass == 0 || key >> (sh + width) == prefix) && i + e < V && key >= kcut) {
                        atomicAdd(&bins.count[(key >> sh) & mask], 1u);
                        if (!limit_k || key > kcut) atomicAdd(&bins.mass[(key >> sh) & mask], fixed(weight(z[e])));
                    }
                }
            }
            __syncthreads();
            if (tid == 0) {
                if (limit_k && (pass == 0 || kcut >> (sh + width) == prefix)) {
                    // the ties of the k-th that are kept
                    const uint32_t b = L::kBits < 32 ? kcut << (32 - L::kBits) : kcut;
                    const float z = __uint_as_float((b & 0x80000000u) ? b & 0x7FFFFFFFu : ~(b | (uint32_t)((1ull << (32 - L::kBits)) - 1ull)));
                    bins.mass[(kcut >> sh) & mask] += (uint64_t)kties * fixed(weight(z));
                }
                uint64_t sum = above;
                if (pass == 0) {
                    uint64_t all = 0;
                    for (int b = 0; b <= (int)mask; ++b) all += bins.mass[b];
                    target = p * (double)all;
                    wave_part[0] = target;
                }
                int b = (int)mask, some = -1;
                for (; b >= 0; --b) {
                    if (bins.count[b]) {
                        some = b;
                        if ((double)(sum + bins.mass[b]) >= target) break;
                        if (b > 0) sum += bins.mass[b];
                    }
                }
                if (b < 0) {                     // (rounding) the last that holds any
                    b = some;
                    sum -= b > 0 ? bins.mass[b] : 0;
                }
                box[0] = (uint64_t)b;
                box[1] = sum;
                ibox = (int)bins.count[b];
            }
            __syncthreads();
            prefix = prefix << width | (uint32_t)box[0];
            above = box[1];
            target = wave_part[0];
        }
        const int there = limit_k && prefix == kcut ? kties : ibox;
        const uint32_t b = L::kBits < 32 ? prefix << (32 - L::kBits) : prefix;
        const float z = __uint_as_float((b & 0x80000000u) ? b & 0x7FFFFFFFu : ~(b | (uint32_t)((1ull << (32 - L::kBits)) - 1ull)));
        const uint64_t each = fixed(weight(z));
        // tie j (from 0) is kept while what lies before it is below the target
        double need = each ? ceil((target - (double)above) / (double)each) : (double)there;
        need = need < 1.0 ? 1.0 : need;
        cut = prefix;
        ties = need < (double)there ? (int)need : there;
    }

    // ---- the index up to which ties are kept
    int last_tie = 0x7FFFFFFF;
    if (ties != 0x7FFFFFFF) {
        int seen = 0;
        for (int i0 = 0; i0 < V; i0 += kTile) {
            const int i = i0 + kVec * tid;
            float z[kVec];
            L::eight(row, i, V, aligned, z);
            int n = 0;
#pragma unroll
            for (int e = 0; e < kVec; ++e) n += i + e < V && L::key(z[e]) == cut;
            int scan = n;
            for (int s = 1; s < 64; s <<= 1) {
                const int o = __shfl_up(scan, s);
                if (lane >= s) scan += o;
            }
            __syncthreads();
            if (lane == 63) wave_int[wv] = scan;
            if (tid == 0) ibox = -1;
            __syncthreads();
            int before = seen;
            for (int k = 0; k < kWaves; ++k) {
                before += k < wv ? wave_int[k] : 0;
                seen += wave_int[k];
            }
            before += scan - n;
            if (before < ties && before + n >= ties) {
                int at = before;
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (i + e < V && L::key(z[e]) == cut && ++at == ties) ibox = i + e;
            }
            __syncthreads();
            if (ibox >= 0) {
                last_tie = ibox;
                break;
            }
        }
        __syncthreads();
    }

    // ---- kept weights, tile by tile, in index order
    auto kept = [&](float z, int i) -> double {
        const uint32_t key = L::key(z);
        if (i >= V || key < cut || (key == cut && i > last_tie)) return 0.0;
        const double w = weight(z);
        return w >= min_w ? w : 0.0;
    };
    // -> this thread's running sum before its eight, and the tile's sum
    auto scan_tile = [&](int i0, double (&w)[kVec], double* before, double* all) {
        const int i = i0 + kVec * tid;
        float z[kVec];
        L::eight(row, i, V, aligned, z);
        double own = 0.0;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            w[e] = kept(z[e], i + e);
            own += w[e];
        }
        double scan = own;
        for (int s = 1; s < 64; s <<= 1) {
            const double o = __shfl_up(scan, s);
            if (lane >= s) scan += o;
        }
        __syncthreads();
        if (lane == 63) wave_part[wv] = scan;
        __syncthreads();
        double sum = 0.0, low = 0.0;
        for (int k = 0; k < kWaves; ++k) {
            if (k == wv) low = sum;
            sum += wave_part[k];
        }
        const double up = __shfl_up(scan, 1);
        *before = low + (lane ? up : 0.0);
        *all = sum;
    };
    double total = 0.0;
    for (int i0 = 0; i0 < V; i0 += kTile) {
        double w[kVec], before, all;
        scan_tile(i0, w, &before, &all);
        total += all;
    }
    // the first whose running sum exceeds the target; where none does, the last kept
    const double target = uf < 1.f ? (double)uf * total : INFINITY;
    __shared__ int found, last_kept;
    __shared__ double found_w, last_w;
    if (tid == 0) {
        found = 0x7FFFFFFF;
        last_kept = -1;
    }
    double sum = 0.0;
    for (int i0 = 0; i0 < V; i0 += kTile) {
        double w[kVec], before, all;
        scan_tile(i0, w, &before, &all);
        double at = sum + before;
        int mine = 0x7FFFFFFF, mine_last = -1;
        double mine_w = 0.0, mine_last_w = 0.0;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            at += w[e];
            if (w[e] > 0.0) {
                if (mine == 0x7FFFFFFF && at > target) {
                    mine = i0 + kVec * tid + e;
                    mine_w = w[e];
                }
                mine_last = i0 + kVec * tid + e;
                mine_last_w = w[e];
            }
        }
        if (mine != 0x7FFFFFFF) atomicMin(&found, mine);
        if (mine_last >= 0) atomicMax(&last_kept, mine_last);
        __syncthreads();
        if (found == mine && mine != 0x7FFFFFFF) found_w = mine_w;
        if (last_kept == mine_last && mine_last >= 0) last_w = mine_last_w;
        __syncthreads();
        if (found != 0x7FFFFFFF) break;
        sum += all;
    }
    if (tid == 0) {
        const bool hit = found != 0x7FFFFFFF;
        a.ids[m] = hit ? found : last_kept;
        if (a.logprob) a.logprob[m] = (float)log((hit ? found_w : last_w) / total);
    }
}

}  // namespace

hipError_t launch_sample(const SampleCall& q, hipStream_t stream) {
    SampleArgs a{};
    a.logits = q.logits;
    a.ld = q.ld;
    a.M = (int)q.M;
    a.V = (int)q.V;
    int bits = 0;
    while ((int64_t(1) << bits) < q.V) ++bits;
    a.unit_shift = 62 - bits;
    a.u = q.u;
    a.temperature = q.temperature;
    a.top_p = q.top_p;
    a.min_p = q.min_p;
    a.top_k = q.top_k;
    a.temperatures = q.temperatures;
    a.top_ks = q.top_ks;
    a.top_ps = q.top_ps;
    a.min_ps = q.min_ps;
    a.ids = q.ids;
    a.logprob = q.logprob;
    a.aligned = (reinterpret_cast<uintptr_t>(q.logits) & 15) == 0 && (q.ld * (q.kind == 2 ? 4 : 2)) % 16 == 0;
    const dim3 grid((unsigned)q.M), block(kThreads);
    if (q.kind == 0) hipLaunchKernelGGL((sample_kernel<0>), grid, block, 0, stream, a);
    else if (q.kind == 1) hipLaunchKernelGGL((sample_kernel<1>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((sample_kernel<2>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace w4a16
