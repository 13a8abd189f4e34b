// Draws a token from each row of logits: temperature, top-k, top-p, min-p, one uniform number.
//
//   w[v] = e^((z[v] - max z) / t);  kept: the k largest z, of these the shortest falling run
//   that reaches p of their weight, of these w >= min_p;  the token: the first v in rising
//   order whose running sum of kept w exceeds u times the whole.
//
// One workgroup a row; wave i takes the i-th contiguous piece, so that sums of waves are sums in
// index order. The row is met two or three times, from the L2 after the first:
//   - its largest, and every thread's;
//   - top-k up to 1024: the k-th largest of the threads' largest bounds the k-th of all from
//     below; the few logits from it on are put into a list in LDS, in index order, and all the
//     rest happens there. A random row of 131072 and k = 50 lists 51.
//   - top-p alone: the sum of all w, and w by sixteenths of an octave below the largest; the
//     logits down to the one where p is reached go into the list.
//   - neither: sums of w, then of the sixteenth, and so on, in which the token lies.
// Where a list would overflow, thresholds are found over the row itself, digit by digit.
//
// Logits are compared as whole numbers (order-preserving keys), thresholds found digit by digit
// from the top: counts for k, sums of weights in 64-bit fixed point for p (whole numbers, so that
// the order of the additions changes nothing). Ties at a threshold go to the lowest index. w and
// the sums of the draw are in fp64: next to a border 32 bits would give another token.
#include "device_common.h"
#include "launch.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kVec = 8;                         // consecutive logits of a lane
constexpr int kStep = 64 * kVec;                // of a wave
constexpr int kRoom = 512;                      // listed logits of a wave
constexpr int kOctaves = 16;                    // below the largest, 16 bins each
constexpr int kNone = 0x7FFFFFFF;

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
    static constexpr int kPasses = (kBits + 7) / 8;
    struct Eight {
        uint4 q[kKind == 2 ? 2 : 1];
    };
    // logits i .. i + 7; past the end -infinity
    static __device__ __forceinline__ Eight load(const void* row, int i, int V, bool aligned) {
        Eight r;
        if (aligned && i + kVec <= V) {
            if constexpr (kKind == 2) {
                const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(row) + i);
                r.q[0] = p[0];
                r.q[1] = p[1];
            } else {
                r.q[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + i);
            }
        } else {
            uint32_t w[kKind == 2 ? 8 : 4];
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                if constexpr (kKind == 2) {
                    w[e] = i + e < V ? static_cast<const uint32_t*>(row)[i + e] : 0xFF800000u;
                } else {
                    const uint32_t v = i + e < V ? static_cast<const uint16_t*>(row)[i + e] : kKind == 1 ? 0xFF80u : 0xFC00u;
                    w[e / 2] = e & 1 ? w[e / 2] | v << 16 : v;
                }
            }
            r.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
            if constexpr (kKind == 2) r.q[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
        return r;
    }
    // the e-th; -infinity for what is no number
    static __device__ __forceinline__ float at(const Eight& r, int e) {
        float z;
        if constexpr (kKind == 2) {
            const uint4& q = r.q[e / 4];
            z = __uint_as_float(e % 4 == 0 ? q.x : e % 4 == 1 ? q.y : e % 4 == 2 ? q.z : q.w);
        } else {
            const uint32_t w = e / 2 == 0 ? r.q[0].x : e / 2 == 1 ? r.q[0].y : e / 2 == 2 ? r.q[0].z : r.q[0].w;
            z = half_bits_to_f32<kKind == 1>(e & 1 ? w >> 16 : w & 0xFFFFu);
        }
        return fmaxf(z, -INFINITY);
    }
    // rises with z; either zero is the same
    static __device__ __forceinline__ uint32_t key(float z) {
        const uint32_t b = __float_as_uint(z + 0.f);
        return ((b & 0x80000000u) ? ~b : b | 0x80000000u) >> (32 - kBits);
    }
    static __device__ __forceinline__ float value(uint32_t key) {
        const uint32_t b = kBits < 32 ? key << (32 - kBits) : key;
        return __uint_as_float((b & 0x80000000u) ? b & 0x7FFFFFFFu : ~(b | (uint32_t)((1ull << (32 - kBits)) - 1ull)));
    }
};

// w of a logit in fp64: 2^x, x = (z - top) log2(e) / t, by Tang's scheme: x = n / 64 + f, 2^(n mod 64 / 64)
// from a table, 2^f by its series to the fifth power (|f| <= 1/128: 4e-17 left out).
struct Weight {
    double top, per;        // log2(e) / t
    const double* table;
    bool endless;           // the largest is +infinity: it alone weighs
    __device__ __forceinline__ double octaves(float z) const { return fmax(((double)z - top) * per, -1100.0); }
    __device__ __forceinline__ double power(double x) const {
        const double shifted = x * 64.0 + 6755399441055744.0;      // 1.5 * 2^52: its low bits are the nearest n
        const int n = (int)(uint32_t)__builtin_bit_cast(uint64_t, shifted);
        const double f = fma(shifted - 6755399441055744.0, -1.0 / 64.0, x);
        double p = 1.3333558146428443e-3;                          // ln2^5 / 5!, ln2^4 / 4!, ...
        p = fma(p, f, 9.618129107628477e-3);
        p = fma(p, f, 5.550410866482158e-2);
        p = fma(p, f, 0.2402265069591007);
        p = fma(p, f, 0.6931471805599453);
        const double s = table[n & 63];
        return ldexp(fma(s, p * f, s), n >> 6);
    }
    __device__ __forceinline__ double operator()(float z) const {
        return endless ? ((double)z == top ? 1.0 : 0.0) : power(octaves(z));
    }
};

struct Shared {
    uint32_t count[256];
    unsigned long long mass[256];
    double table[64];
    double part[kWaves], found_w;
    int listed[kWaves];
    int box[2];
    uint64_t above;
    uint32_t key[kWaves][kRoom];
    int index[kWaves][kRoom];
};

__device__ __forceinline__ double wave_sum(double v) {
    for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
    return v;
}
template <class T>
__device__ __forceinline__ T wave_before(T v, T* all) {            // sum of the lower lanes; of all
    const int lane = (int)threadIdx.x & 63;
    T sum = v;
    for (int s = 1; s < 64; s <<= 1) {
        const T o = __shfl_up(sum, s);
        if (lane >= s) sum += o;
    }
    *all = __shfl(sum, 63);
    const T up = __shfl_up(sum, 1);
    return lane ? up : T(0);
}

// The key of the left-th largest of what each(f) gives f, and how many of its equals are among
// the largest `left`. Every thread calls it, with at least `left` in all.
template <class L, class Each>
__device__ __forceinline__ void find_count(Shared& sh, Each each, int left, uint32_t* cut, int* ties) {
    const int tid = (int)threadIdx.x, lane = tid & 63;
    uint32_t prefix = 0;
    for (int pass = 0; pass < L::kPasses; ++pass) {
        const int sh_ = L::kBits - 8 * (pass + 1) > 0 ? L::kBits - 8 * (pass + 1) : 0;
        const int width = L::kBits - 8 * pass < 8 ? L::kBits - 8 * pass : 8;
        __syncthreads();
        if (tid < 256) sh.count[tid] = 0u;
        __syncthreads();
        each([&](uint32_t key) {
            if (pass == 0 || key >> (sh_ + width) == prefix) atomicAdd(&sh.count[(key >> sh_) & ((1u << width) - 1u)], 1u);
        });
        __syncthreads();
        if (tid < 64) {
            int own = 0, all;
#pragma unroll
            for (int j = 0; j < 4; ++j) own += (int)sh.count[255 - 4 * lane - j];
            int above = wave_before(own, &all);
            if (above < left && left <= above + own) {
                int b = 255 - 4 * lane;
                while (above + (int)sh.count[b] < left) above += (int)sh.count[b--];
                sh.box[0] = b;
                sh.box[1] = left - above;
            }
        }
        __syncthreads();
        prefix = prefix << width | (uint32_t)sh.box[0];
        left = sh.box[1];
    }
    *cut = prefix;
    *ties = left;
}

// The key at which weights, the largest first, reach `target`, what lies above it, and how many
// equals it has. each(f) gives f(key, weight in fixed point, count).
template <class L, class Each>
__device__ __forceinline__ void find_mass(Shared& sh, Each each, double target, uint32_t* cut, uint64_t* above_cut, int* there) {
    const int tid = (int)threadIdx.x, lane = tid & 63;
    uint32_t prefix = 0;
    uint64_t above = 0;
    target = fmax(target, 1.0);                  // at least the first
    for (int pass = 0; pass < L::kPasses; ++pass) {
        const int sh_ = L::kBits - 8 * (pass + 1) > 0 ? L::kBits - 8 * (pass + 1) : 0;
        const int width = L::kBits - 8 * pass < 8 ? L::kBits - 8 * pass : 8;
        __syncthreads();
        if (tid < 256) {
            sh.count[tid] = 0u;
            sh.mass[tid] = 0ull;
        }
        __syncthreads();
        each([&](uint32_t key, auto weight) {
            if (pass == 0 || key >> (sh_ + width) == prefix) {
                const uint32_t b = (key >> sh_) & ((1u << width) - 1u);
                atomicAdd(&sh.count[b], 1u);
                atomicAdd(&sh.mass[b], (unsigned long long)weight());
            }
        });
        __syncthreads();
        if (tid < 64) {
            uint64_t own = 0, all;
            int some = -1;                       // the lane's lowest bin that holds any
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                own += sh.mass[255 - 4 * lane - j];
                if (sh.count[255 - 4 * lane - j]) some = 255 - 4 * lane - j;
            }
            uint64_t sum = above + wave_before((uint64_t)own, &all);
            const bool here = (double)sum < target && (double)(sum + own) >= target;
            const uint64_t hit = __ballot(here), any = __ballot(some >= 0);
            if (hit ? here : lane == 63 - __builtin_clzll(any)) {
                int b = 255 - 4 * lane;
                while (b > some && (sh.count[b] == 0 || (double)(sum + sh.mass[b]) < target)) sum += sh.mass[b--];
                sh.box[0] = b;
                sh.box[1] = (int)sh.count[b];
                sh.above = sum;
            }
        }
        __syncthreads();
        prefix = prefix << width | (uint32_t)sh.box[0];
        above = sh.above;
    }
    *cut = prefix;
    *above_cut = above;
    *there = sh.box[1];
}

template <int kKind>
__global__ __launch_bounds__(kThreads) void sample_kernel(const SampleArgs a) {
    using L = Logit<kKind>;
    using Eight = typename L::Eight;
    constexpr int kAhead = kKind == 2 ? 2 : 4;                     // pieces of a lane loaded at a time
    __shared__ Shared sh;
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = (int)blockIdx.x, V = a.V;
    const void* row = static_cast<const uint8_t*>(a.logits) + (int64_t)m * a.ld * (kKind == 2 ? 4 : 2);
    const bool aligned = a.aligned != 0;
    const float t = a.temperatures ? a.temperatures[m] : a.temperature;
    const bool greedy = !(t > 0.f);
    const int kk = greedy ? 1 : a.top_ks ? a.top_ks[m] : a.top_k;
    const bool limit_k = kk >= 1 && kk < V;
    const float pf = a.top_ps ? a.top_ps[m] : a.top_p;
    const bool limit_p = pf < 1.f;
    const double p = (double)fmaxf(pf, 0.f);
    const float mf = a.min_ps ? a.min_ps[m] : a.min_p;
    const double min_w = mf > 0.f ? (double)fminf(mf, 1.f) : 0.0;
    const float uf = a.u[m];
    const int piece = (int)(((int64_t)V + kWaves * kStep - 1) / (kWaves * kStep)) * kStep;     // of a wave
    const int64_t from64 = (int64_t)wv * piece;
    const int from = from64 < V ? (int)from64 : V, to = V - from < piece ? V : from + piece;

    // f(logits, index of the first) for each eight of [i0, i1), in rising order of a lane
    auto walk = [&](int i0, int i1, auto f) {
        for (int i = i0 + kVec * lane; i - kVec * lane < i1; i += kAhead * kStep) {
            Eight r[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) r[j] = L::load(row, i + j * kStep, i1, aligned);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) f(r[j], i + j * kStep);
        }
    };

    // ---- the largest, of the thread and of all
    float mine = -INFINITY;
    walk(from, to, [&](const Eight& r, int) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) mine = fmaxf(mine, L::at(r, e));
    });
    if (tid < 64) sh.table[tid] = exp2((double)tid / 64.0);
    float top = mine;
    for (int s = 32; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor(top, s));
    if (lane == 0) sh.part[wv] = (double)top;
    __syncthreads();
    for (int k = 0; k < kWaves; ++k) top = fmaxf(top, (float)sh.part[k]);
    if (top == -INFINITY) {
        if (tid == 0) {
            a.ids[m] = -1;
            if (a.logprob) a.logprob[m] = -INFINITY;
        }
        return;
    }
    if (greedy) {
        // the lowest index that has it
        if (tid == 0) sh.box[0] = kNone;
        __syncthreads();
        int at = kNone;
        walk(from, to, [&](const Eight& r, int i) {
#pragma unroll
            for (int e = kVec - 1; e >= 0; --e)
                if (L::at(r, e) == top && i + e < at) at = i + e;
        });
        if (at != kNone) atomicMin(&sh.box[0], at);
        __syncthreads();
        if (tid == 0) {
            a.ids[m] = sh.box[0];
            if (a.logprob) a.logprob[m] = 0.f;
        }
        return;
    }
    const Weight weight{(double)top, 1.4426950408889634 / (double)t, sh.table, top == INFINITY};
    const double unit = (double)(1ull << a.unit_shift);
    // (unit <= 2^51: the sum's low 52 bits are the nearest whole number)
    auto fixed = [&](double w) { return __builtin_bit_cast(uint64_t, fma(w, unit, 4503599627370496.0)) & 0xFFFFFFFFFFFFFull; };
    const bool last_of_all = uf >= 1.f;
    const double share = uf > 0.f ? (double)uf : 0.0;
    auto answer = [&](int id, double w, double total) {
        a.ids[m] = id;
        if (a.logprob) a.logprob[m] = (float)log(w / total);
    };

    // ---- the list: logits that `take` wants, in index order; false where they are too many
    auto gather = [&](auto take) {
        int n = 0;
        walk(from, to, [&](const Eight& r, int i) {
            uint32_t hits = 0;
#pragma unroll
            for (int e = 0; e < kVec; ++e) hits |= take(L::at(r, e)) && i + e < to ? 1u << e : 0u;
            if (__ballot(hits != 0) == 0) return;
            int all;
            int at = n + wave_before((int)__popc(hits), &all);
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if ((hits >> e) & 1u) {
                    if (at < kRoom) {
                        sh.key[wv][at] = L::key(L::at(r, e));
                        sh.index[wv][at] = i + e;
                    }
                    ++at;
                }
            n += all;
        });
        __syncthreads();
        if (lane == 0) sh.listed[wv] = n;
        __syncthreads();
        bool fits = true;
        for (int k = 0; k < kWaves; ++k) fits = fits && sh.listed[k] <= kRoom;
        return fits;
    };

    bool listed = false;
    double whole = 0.0;                          // the weight of all, where it is known
    if (limit_k && kk <= kThreads) {
        uint32_t bound;
        int equals;
        find_count<L>(sh, [&](auto f) { f(L::key(mine)); }, kk, &bound, &equals);
        listed = gather([&](float z) { return L::key(z) >= bound; });
    } else if (limit_p && !limit_k && !weight.endless) {
        __syncthreads();
        if (tid < 256) sh.mass[tid] = 0ull;
        __syncthreads();
        double sum = 0.0;
        auto bin_of = [&](double x) { return (int)(x * -16.0); };
        walk(from, to, [&](const Eight& r, int) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const double x = weight.octaves(L::at(r, e)), w = weight.power(x);
                sum += w;
                if (x > (double)-kOctaves) atomicAdd(&sh.mass[bin_of(x)], (unsigned long long)fixed(w));
            }
        });
        sum = wave_sum(sum);
        if (lane == 0) sh.part[wv] = sum;
        if (tid == 0) sh.box[0] = -1;
        __syncthreads();
        for (int k = 0; k < kWaves; ++k) whole += sh.part[k];
        if (tid < 64) {
            uint64_t own = 0, all;
#pragma unroll
            for (int j = 0; j < 4; ++j) own += sh.mass[4 * lane + j];
            uint64_t above = wave_before((uint64_t)own, &all);
            // (a little more than p: the list only has to hold what is kept)
            const double want = p * whole * unit * (1.0 + 1e-9) + 1.0;
            if ((double)above < want && (double)(above + own) >= want) {
                int b = 4 * lane;
                while ((double)(above + sh.mass[b]) < want) above += sh.mass[b++];
                sh.box[0] = b;
            }
        }
        __syncthreads();
        const int bin = sh.box[0];
        if (bin >= 0) listed = gather([&](float z) {
            const double x = weight.octaves(z);
            return x > (double)-kOctaves && bin_of(x) <= bin;
        });
    }
    __syncthreads();

    if (listed) {
        const int n = sh.listed[wv];
        auto each = [&](auto f) {
            for (int j = lane; j < n; j += 64) f(sh.key[wv][j], sh.index[wv][j]);
        };
        uint32_t cut = 0;                        // keys above it are kept,
        int ties = kNone;                        // of those equal to it the first `ties`
        if (limit_k) find_count<L>(sh, [&](auto f) { each([&](uint32_t key, int) { f(key); }); }, kk, &cut, &ties);
        // sums of w over the entries down to the cut, ties in index order
        auto kept_sums = [&](bool floor, double* before, double* all) {
            int equals = 0;
            for (int j = lane; j < n; j += 64) equals += sh.key[wv][j] == cut;
            int wave_equals;
            wave_before(equals, &wave_equals);
            __syncthreads();
            if (lane == 0) sh.listed[wv] = wave_equals;
            __syncthreads();
            int seen = 0;
            for (int k = 0; k < wv; ++k) seen += sh.listed[k];
            // ties seen so far turn into the number of this wave's that are kept
            const int keep = ties == kNone ? kNone : ties > seen ? ties - seen : 0;
            double sum = 0.0;
            int met = 0;
            for (int j0 = 0; j0 < n; j0 += 64) {
                const int j = j0 + lane;
                const bool tie = j < n && sh.key[wv][j] == cut;
                const uint64_t mask = __ballot(tie);
                const int rank = met + __popcll(mask & ((1ull << lane) - 1ull));
                met += __popcll(mask);
                double w = 0.0;
                if (j < n && (sh.key[wv][j] > cut || (tie && rank < keep))) w = weight(L::value(sh.key[wv][j]));
                if (floor && w < min_w) w = 0.0;
                sum += wave_sum(w);
            }
            __syncthreads();
            if (lane == 0) sh.part[wv] = sum;
            __syncthreads();
            *before = *all = 0.0;
            for (int k = 0; k < kWaves; ++k) {
                if (k == wv) *before = *all;
                *all += sh.part[k];
            }
            return keep;
        };
        if (limit_p) {
            const uint32_t kcut = cut;
            const int kties = ties;
            if (limit_k) {
                double before;
                kept_sums(false, &before, &whole);
            }
            // the ties of the k-th count as often as they are kept: one entry brings them all
            const double target = p * whole * unit;
            uint64_t above;
            int there;
            const uint64_t tie_mass = limit_k ? (uint64_t)kties * fixed(weight(L::value(kcut))) : 0;
            find_mass<L>(sh, [&](auto f) {
                each([&](uint32_t key, int) {
                    if (!limit_k || key > kcut) f(key, [&] { return fixed(weight(L::value(key))); });
                });
                if (limit_k && tid == 0) f(kcut, [&] { return tie_mass; });
            }, target, &cut, &above, &there);
            if (limit_k && cut == kcut) there = kties;
            const uint64_t one = fixed(weight(L::value(cut)));
            // tie j (from 0) is kept while what lies before it is below the target
            double need = one ? ceil((target - (double)above) / (double)one) : (double)there;
            need = need < 1.0 ? 1.0 : need;
            ties = need < (double)there ? (int)need : there;
        }
        double before, total;
        const int keep = kept_sums(true, &before, &total);
        const double target = share * total;
        // the wave in which the running sum exceeds the target, or the last that keeps any
        int wave = -1, fallback = 0;
        double run = 0.0;
        for (int k = 0; k < kWaves; ++k) {
            if (sh.part[k] > 0.0) {
                fallback = k;
                if (!last_of_all && wave < 0 && run + sh.part[k] > target) wave = k;
            }
            run += sh.part[k];
        }
        const bool exact = wave >= 0;
        if (!exact) wave = fallback;
        if (wv != wave) return;
        double sum = before;
        int met = 0, last_id = -1;
        double last_w = 0.0;
        for (int j0 = 0; j0 < n; j0 += 64) {
            const int j = j0 + lane;
            const bool tie = j < n && sh.key[wv][j] == cut;
            const uint64_t mask = __ballot(tie);
            const int rank = met + __popcll(mask & ((1ull << lane) - 1ull));
            met += __popcll(mask);
            double w = 0.0, all;
            if (j < n && (sh.key[wv][j] > cut || (tie && rank < keep))) w = weight(L::value(sh.key[wv][j]));
            if (w < min_w) w = 0.0;
            const double low = wave_before(w, &all);
            const uint64_t over = exact ? __ballot(w > 0.0 && sum + low + w > target) : 0;
            if (over) {
                if (lane == __builtin_ctzll(over)) answer(sh.index[wv][j], w, total);
                return;
            }
            const uint64_t some = __ballot(w > 0.0);
            if (some) {
                const int from_lane = 63 - __builtin_clzll(some);
                last_id = __shfl(j < n ? sh.index[wv][j] : 0, from_lane);
                last_w = __shfl(w, from_lane);
            }
            sum += all;
        }
        if (lane == 0) answer(last_id, last_w, total);
        return;
    }

    // ---- over the row itself
    uint32_t cut = 0;
    int ties = kNone;
    auto each = [&](auto f) {
        walk(from, to, [&](const Eight& r, int i) {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (i + e < to) f(L::at(r, e));
        });
    };
    if (limit_k) find_count<L>(sh, [&](auto f) { each([&](float z) { f(L::key(z)); }); }, kk, &cut, &ties);
    if (limit_p) {
        const uint32_t kcut = cut;
        const int kties = ties;
        const uint64_t tie_mass = limit_k ? (uint64_t)kties * fixed(weight(L::value(kcut))) : 0;
        double sum = 0.0;
        each([&](float z) {
            if (!limit_k || L::key(z) > kcut) sum += weight(z);
        });
        sum = wave_sum(sum);
        __syncthreads();
        if (lane == 0) sh.part[wv] = sum;
        __syncthreads();
        whole = limit_k ? (double)kties * weight(L::value(kcut)) : 0.0;
        for (int k = 0; k < kWaves; ++k) whole += sh.part[k];
        const double target = p * whole * unit;
        uint64_t above;
        int there;
        find_mass<L>(sh, [&](auto f) {
            each([&](float z) {
                if (!limit_k || L::key(z) > kcut) f(L::key(z), [&] { return fixed(weight(z)); });
            });
            if (limit_k && tid == 0) f(kcut, [&] { return tie_mass; });
        }, target, &cut, &above, &there);
        if (limit_k && cut == kcut) there = kties;
        const uint64_t one = fixed(weight(L::value(cut)));
        double need = one ? ceil((target - (double)above) / (double)one) : (double)there;
        need = need < 1.0 ? 1.0 : need;
        ties = need < (double)there ? (int)need : there;
    }
    // the index of the last tie that is kept
    int last_tie = kNone;
    if (ties != kNone) {
        int equals = 0, wave_equals;
        each([&](float z) { equals += L::key(z) == cut; });
        wave_before(equals, &wave_equals);
        __syncthreads();
        if (lane == 0) sh.listed[wv] = wave_equals;
        if (tid == 0) sh.box[0] = kNone;
        __syncthreads();
        int seen = 0;
        for (int k = 0; k < wv; ++k) seen += sh.listed[k];
        if (seen < ties && seen + sh.listed[wv] >= ties)
            walk(from, to, [&](const Eight& r, int i) {
                int n = 0, all;
#pragma unroll
                for (int e = 0; e < kVec; ++e) n += i + e < to && L::key(L::at(r, e)) == cut;
                int at = seen + wave_before(n, &all);
                seen += all;
                if (at < ties && at + n >= ties) {
#pragma unroll
                    for (int e = 0; e < kVec; ++e)
                        if (i + e < to && L::key(L::at(r, e)) == cut && ++at == ties) sh.box[0] = i + e;
                }
            });
        __syncthreads();
        last_tie = sh.box[0];
    }
    const bool all_kept = ties == kNone && min_w == 0.0;
    auto kept = [&](float z, int i) -> double {
        if (!all_kept) {
            const uint32_t key = L::key(z);
            if (key < cut || (key == cut && i > last_tie)) return 0.0;
        }
        const double w = weight(z);
        return w >= min_w ? w : 0.0;
    };
    // Sums of the sixteen pieces of a range, then of those of the one in which the running sum
    // exceeds the target, until a piece is one step of a wave.
    int i0 = 0, i1 = V;
    double run = 0.0, total = 0.0, target = 0.0;
    bool exact = !last_of_all;
    for (int size = piece;;) {
        const int64_t b64 = (int64_t)i0 + (int64_t)wv * size;
        const int b = b64 < i1 ? (int)b64 : i1, e1 = i1 - b < size ? i1 : b + size;
        double sum = 0.0;
        walk(b, e1, [&](const Eight& r, int i) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) sum += i + e < e1 ? kept(L::at(r, e), i + e) : 0.0;
        });
        sum = wave_sum(sum);
        __syncthreads();
        if (lane == 0) sh.part[wv] = sum;
        __syncthreads();
        if (total == 0.0) {
            for (int k = 0; k < kWaves; ++k) total += sh.part[k];
            target = share * total;
        }
        int wave = -1, fallback = 0;
        double at = run, before = run, before_last = run;
        for (int k = 0; k < kWaves; ++k) {
            if (sh.part[k] > 0.0) {
                fallback = k;
                before_last = at;
                if (exact && wave < 0 && at + sh.part[k] > target) {
                    wave = k;
                    before = at;
                }
            }
            at += sh.part[k];
        }
        if (wave < 0) {
            exact = false;                       // (rounding, or u of 1) the last that is kept
            wave = fallback;
            before = before_last;
        }
        run = before;
        const int64_t n0 = (int64_t)i0 + (int64_t)wave * size;
        i1 = i1 - n0 < size ? i1 : (int)n0 + size;
        i0 = (int)n0;
        if (size <= kStep) break;
        size = (int)(((int64_t)size + kWaves * kStep - 1) / (kWaves * kStep)) * kStep;
    }
    if (wv != 0) return;
    const int i = i0 + kVec * lane;
    const Eight r = L::load(row, i, i1, aligned);
    double w[kVec], own = 0.0, all;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        w[e] = i + e < i1 ? kept(L::at(r, e), i + e) : 0.0;
        own += w[e];
    }
    double at = run + wave_before(own, &all);
    int hit = kNone, last_kept = -1;
    double hit_w = 0.0, last_w = 0.0;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        at += w[e];
        if (w[e] > 0.0) {
            if (hit == kNone && at > target) {
                hit = i + e;
                hit_w = w[e];
            }
            last_kept = i + e;
            last_w = w[e];
        }
    }
    const uint64_t over = exact ? __ballot(hit != kNone) : 0, some = __ballot(last_kept >= 0);
    if (over) {
        if (lane == __builtin_ctzll(over)) answer(hit, hit_w, total);
    } else if (lane == 63 - __builtin_clzll(some)) {
        answer(last_kept, last_w, total);
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
    a.unit_shift = 62 - bits < 51 ? 62 - bits : 51;
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
