// Draws a token from each row of logits: temperature, top-k, top-p, min-p, one uniform number.
//
//   w[v] = e^((z[v] - max z) / t);  kept: the k largest z, of these the shortest falling run
//   that reaches p of their weight, of these w >= min_p;  the token: the first v in rising
//   order whose running sum of kept w exceeds u times the whole.
//
// A row is cut into 16 contiguous pieces, so that sums of pieces are sums in index order. It is met
// two to four times, from the caches after the first:
//   1. the largest logit, and the largest of 256 groups;
//   2. top-k up to 192: the k-th largest of the groups' bounds the k-th of all from below, and the
//      few logits from it on are put into a list, in index order; all the rest happens there (a
//      random row of 131072 and k = 50 lists 56). Otherwise: the sums of w, and with top-p w by
//      32nds of an octave below the largest;
//   3. top-p alone: the logits of the 32nd in which p is reached are listed, those above it summed;
//   4. the draw: the piece whose sum of kept w holds the target, its sixteenth, and so on.
// A few rows take 16 workgroups each, in a launch for each of these; many rows one workgroup each,
// a wave a piece, in one launch. Bound by latency (a few rows: three or four launches of 3 to 10 us whose
// steps wait for each other) and by the vector units (many rows: 256 x 131072 in 45 to 50 us, 1.4 TB/s: 36 vector
// instructions a logit, 25 of them in fp64, fill 73% of the cycles). What the lists do not hold (top-k over 1024, lists of more than 512
// in a piece) is found over the row itself.
//
// Logits are compared as whole numbers (order-preserving keys). Lists of up to 256 are sorted by
// counting, an entry a thread; in longer ones and over the row thresholds are found digit by digit
// from the top: counts for k, sums of weights in 64-bit fixed point for p (whole numbers, so that the
// order of the additions changes nothing). Ties at a threshold go to the lowest index. w and the sums
// of the draw are in fp64: next to a border 32 bits would give another token.
#include "device_common.h"
#include "launch.h"
#include "wave.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kPieces = kWaves;
constexpr int kPieceThreads = 256;              // of a workgroup that takes one piece
constexpr int kVec = 8;                         // consecutive logits of a lane
constexpr int kStep = 64 * kVec;                // of a wave
constexpr int kRoom = 512;                      // listed logits of a piece
constexpr int kShort = 256;                     // and of all in a short list
constexpr int kGroups = 256;
constexpr int kGroupK = kGroups * 3 / 4;        // top-k up to here goes by the groups' largest
constexpr int kBins = 1024, kBinsPerOctave = 32;   // of weights, below the largest
constexpr int kNone = 0x7FFFFFFF;
// Of a launch of one workgroup a row: a grid's size is 32 bits of threads, and HIP launches what is
// left of a larger one without an error (2^22 + 3 rows of 1024 threads: the first three).
constexpr int kRowsPerLaunch = 1 << 20;

// what the launches for few rows leave to each other
struct Left {
    float group_max[kGroups];
    double sum[kPieces];                        // of all w (top-p) or of those that min-p keeps
    double above[kPieces];                      // top-p: of w above the list, and of those that min-p keeps
    double above_kept[kPieces];
    int listed[kPieces];
    unsigned long long mass[kBins];
    uint32_t key[kPieces][kRoom];
    int index[kPieces][kRoom];
};

static_assert(sizeof(Left) % 16 == 0, "read 16 bytes at a time");

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
    Left* left;             // [M], or NULL: one workgroup a row
};

// a row's settings
struct How {
    float t;
    bool greedy, limit_k, limit_p, by_groups, by_bins;
    int k;
    double p, min_w;
    __device__ __forceinline__ How(const SampleArgs& a, int m) {
        t = a.temperatures ? a.temperatures[m] : a.temperature;
        greedy = !(t > 0.f);
        k = greedy ? 1 : a.top_ks ? a.top_ks[m] : a.top_k;
        limit_k = k >= 1 && k < a.V;
        const float pf = a.top_ps ? a.top_ps[m] : a.top_p;
        limit_p = pf < 1.f;
        p = (double)fmaxf(pf, 0.f);
        const float mf = a.min_ps ? a.min_ps[m] : a.min_p;
        min_w = mf > 0.f ? (double)fminf(mf, 1.f) : 0.0;
        by_groups = limit_k && k <= kGroupK;
        by_bins = limit_p && !limit_k;
    }
};

// kKind: 0 fp16, 1 bf16, 2 fp32. Values of the type take the top kBits of an fp32 key.
template <int kKind> struct Logit {
    static constexpr int kBits = kKind == 0 ? 19 : kKind == 1 ? 16 : 32;
    static constexpr int kPasses = (kBits + 7) / 8;
    struct Eight {
        uint4 q[kKind == 2 ? 2 : 1];
    };
    // logits i .. i + 7; past the end -infinity
    static __device__ __forceinline__ Eight load(const void* row, int i, int V) {
        Eight r;
        if (i + kVec <= V) {
            // (rows may begin anywhere: one load of 16 bytes either way)
            const char* from = static_cast<const char*>(row) + (size_t)i * (kKind == 2 ? 4 : 2);
            __builtin_memcpy(&r.q[0], from, 16);
            if constexpr (kKind == 2) __builtin_memcpy(&r.q[1], from + 16, 16);
        } else {
            // (rolled: it is in every loop over the row, and rarely taken)
            const uint32_t none = kKind == 2 ? 0xFF800000u : kKind == 1 ? 0xFF80FF80u : 0xFC00FC00u;
            r.q[0] = make_uint4(none, none, none, none);
            if constexpr (kKind == 2) r.q[1] = r.q[0];
            if (i >= V) return r;
#pragma unroll 1
            for (int e = kVec - 1; e >= 0; --e) {
                if constexpr (kKind == 2) {
                    const uint32_t v = i + e < V ? static_cast<const uint32_t*>(row)[i + e] : 0xFF800000u;
                    r.q[1] = make_uint4(r.q[0].w, r.q[1].x, r.q[1].y, r.q[1].z);
                    r.q[0] = make_uint4(v, r.q[0].x, r.q[0].y, r.q[0].z);
                } else {
                    const uint32_t v = i + e < V ? static_cast<const uint16_t*>(row)[i + e] : kKind == 1 ? 0xFF80u : 0xFC00u;
                    uint4& q = r.q[0];
                    q = make_uint4(q.x << 16 | v, q.y << 16 | q.x >> 16, q.z << 16 | q.y >> 16, q.w << 16 | q.z >> 16);
                }
            }
        }
        return r;
    }
    static __device__ __forceinline__ float one(const void* row, int i) {
        if constexpr (kKind == 2) return fmaxf(static_cast<const float*>(row)[i], -INFINITY);
        else return fmaxf(half_bits_to_f32<kKind == 1>(static_cast<const uint16_t*>(row)[i]), -INFINITY);
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
    // the seven behind the first move up
    static __device__ __forceinline__ void next(Eight& r) {
        if constexpr (kKind == 2) {
            r.q[0] = make_uint4(r.q[0].y, r.q[0].z, r.q[0].w, r.q[1].x);
            r.q[1] = make_uint4(r.q[1].y, r.q[1].z, r.q[1].w, 0u);
        } else {
            uint4& q = r.q[0];
            q = make_uint4(q.x >> 16 | q.y << 16, q.y >> 16 | q.z << 16, q.z >> 16 | q.w << 16, q.w >> 16);
        }
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

// w of a logit in fp64: 2^x, x = (z - top) log2(e) / t = n + f, 2^f by its series to the twelfth
// power (|f| <= 1/2: 2e-16 left out). (A table of 64 powers and a series to the fifth: 1.4 times the
// time, in bank conflicts.)
struct Weight {
    double top, per;        // log2(e) / t
    bool endless;           // the largest is +infinity: it alone weighs
    __device__ __forceinline__ Weight(float largest, float t)
        : top((double)largest), per(1.4426950408889634 / (double)t), endless(largest == INFINITY) {}
    __device__ __forceinline__ double octaves(float z) const { return fmax(((double)z - top) * per, -1100.0); }
    __device__ __forceinline__ double power(double x) const {
        const double n = rint(x), f = x - n;
        double p = 2.5678435993488202e-11;                         // ln2^12 / 12!, ln2^11 / 11!, ...
        p = fma(p, f, 4.4455382718708115e-10);
        p = fma(p, f, 7.0549116208011234e-9);
        p = fma(p, f, 1.0178086009239699e-7);
        p = fma(p, f, 1.3215486790144307e-6);
        p = fma(p, f, 1.5252733804059841e-5);
        p = fma(p, f, 1.5403530393381608e-4);
        p = fma(p, f, 1.3333558146428443e-3);
        p = fma(p, f, 9.618129107628477e-3);
        p = fma(p, f, 5.550410866482158e-2);
        p = fma(p, f, 0.2402265069591007);
        p = fma(p, f, 0.6931471805599453);
        return ldexp(fma(p, f, 1.0), (int)n);
    }
    __device__ __forceinline__ double operator()(float z) const {
        return endless ? ((double)z == top ? 1.0 : 0.0) : power(octaves(z));
    }
};

// Weights in whole steps (unit <= 2^51: the sum's low 52 bits are the nearest whole number), and
// their bins below the largest.
__device__ __forceinline__ uint64_t fixed_point(double w, double unit) {
    return __builtin_bit_cast(uint64_t, fma(w, unit, 4503599627370496.0)) & 0xFFFFFFFFFFFFFull;
}
__device__ __forceinline__ int bin_of(double x) { return (int)(x * -(double)kBinsPerOctave); }
// a bound a little below (by = 1e-6) or above (by = -1e-6) a bin's lower end
__device__ __forceinline__ float bin_end(const Weight& w, int bin, double by) {
    const double low = w.top - (double)(bin + 1) / kBinsPerOctave / w.per * (1.0 + by);
    return (float)(low - by * (fabs(low) + 1e-3 * fabs(w.top)));
}

template <int kKind> struct Row {
    using L = Logit<kKind>;
    using Eight = typename L::Eight;
    const void* p;
    int V, lane;
    __device__ __forceinline__ Row(const SampleArgs& a, int m) {
        p = static_cast<const uint8_t*>(a.logits) + (int64_t)m * a.ld * (kKind == 2 ? 4 : 2);
        V = a.V;
        lane = (int)threadIdx.x & 63;
    }
    // logits of a piece, and of the part of it that one of `parts` waves takes
    __device__ __forceinline__ int piece() const { return (int)(((int64_t)V + kPieces * kStep - 1) / (kPieces * kStep)) * kStep; }
    __device__ __forceinline__ int start(int64_t i) const { return i < V ? (int)i : V; }
    // f(logits, index of the first) for each eight of [i0, i1) that this wave's lane has, in rising order
    template <int kAhead, class F>
    __device__ __forceinline__ void walk(int i0, int i1, F f) const {
        for (int i = i0 + kVec * lane; i - kVec * lane < i1; i += kAhead * kStep) {
            Eight r[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) r[j] = L::load(p, i + j * kStep, i1);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) f(r[j], i + j * kStep);
        }
    }
    // the same for a costly f, in less code
    template <class F>
    __device__ __forceinline__ void stroll(int i0, int i1, F f) const {
        for (int i = i0; i < i1; i += 4 * kStep) {
            Eight r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) r[j] = L::load(p, i + j * kStep + kVec * lane, i1);
#pragma unroll 1
            for (int j = 0; j < 4 && i + j * kStep < i1; ++j) {
                f(r[0], i + j * kStep + kVec * lane);
                r[0] = r[1];
                r[1] = r[2];
                r[2] = r[3];
            }
        }
    }
    // f(logit, its index), where speed matters least
    template <class F>
    __device__ __forceinline__ void each(int i0, int i1, F f) const {
        stroll(i0, i1, [&](Eight q, int i) {
#pragma unroll 1
            for (int e = 0; e < kVec; e += 2) {
                if (i + e < i1) f(L::at(q, 0), i + e);
                if (i + e + 1 < i1) f(L::at(q, 1), i + e + 1);
                L::next(q);
                L::next(q);
            }
        });
    }
    // this lane's sum of w (without bins: of those that min-p keeps); with them, w by bins too
    __device__ __forceinline__ double sum_of(int i0, int i1, const Weight& weight, const How& how, double unit, unsigned long long* mass) const {
        double sum = 0.0;
        if (how.by_bins) {
            stroll(i0, i1, [&](const Eight& r, int) {
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const double x = weight.octaves(L::at(r, e)), v = weight.power(x);
                    sum += v;
                    if (x > -(double)(kBins / kBinsPerOctave)) atomicAdd(&mass[bin_of(x)], (unsigned long long)fixed_point(v, unit));
                }
            });
        } else if (how.min_w > 0.0) {
            stroll(i0, i1, [&](const Eight& r, int) {
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const double v = weight.power(weight.octaves(L::at(r, e)));
                    sum += v >= how.min_w ? v : 0.0;
                }
            });
        } else {
            stroll(i0, i1, [&](const Eight& r, int) {
#pragma unroll
                for (int e = 0; e < kVec; ++e) sum += weight.power(weight.octaves(L::at(r, e)));
            });
        }
        return sum;
    }
    // of those from `high` on: all, and those that min-p keeps
    __device__ __forceinline__ void sum_above(int i0, int i1, float high, const Weight& weight, double min_w, double* above, double* kept) const {
        double all = 0.0, some = 0.0;
        stroll(i0, i1, [&](Eight r, int) {
            float most = -INFINITY;
#pragma unroll
            for (int e = 0; e < kVec; ++e) most = fmaxf(most, L::at(r, e));
            if (__ballot(most >= high) == 0) return;
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                const double w = weight.power(weight.octaves(L::at(r, e))), v = L::at(r, e) >= high ? w : 0.0;
                all += v;
                some += v >= min_w ? v : 0.0;
            }
        });
        *above = wave_sum(all);
        *kept = wave_sum(some);
    }
    // Entries of [i0, i1) from `low` up to below `high` (no number: all), in index order, from place n on; returns the
    // place behind the last (entries past `room` are only counted).
    __device__ __forceinline__ int gather(int i0, int i1, float low, float high, uint32_t* key, int* index, int room, int n) const {
        constexpr int kAhead = kKind == 2 ? 2 : 4;
        walk<kAhead>(i0, i1, [&](const Eight& r, int i) {
            if (i - kVec * lane >= i1) return;
            float most = -INFINITY;
#pragma unroll
            for (int e = 0; e < kVec; ++e) most = fmaxf(most, L::at(r, e));
            if (__ballot(most >= low) == 0) return;
            uint32_t hits = 0;
#pragma unroll
            for (int e = 0; e < kVec; ++e) hits |= L::at(r, e) >= low && !(L::at(r, e) >= high) && i + e < i1 ? 1u << e : 0u;
            int all;
            int at = n + wave_before((int)__popc(hits), &all);
#pragma unroll 1
            for (Eight q = r; hits; hits >>= 1) {
                if ((hits & 1u) && at < room) {
                    key[at] = L::key(L::at(q, 0));
                    index[at] = i;
                }
                at += (int)(hits & 1u);
                ++i;
                L::next(q);
            }
            n += all;
        });
        return n;
    }
};

struct Shared {
    uint32_t count[256];
    unsigned long long mass[kBins];
    double part[kPieces], above[kPieces], above_kept[kPieces];
    double sorted[kShort];
    int entry[kShort];      // of each rank
    int listed[kPieces];
    int box[2];
    uint64_t above_cut;
    uint4 short_key[kShort / 4];
    int short_index[kShort];
    uint32_t key[kPieces][kRoom];
    int index[kPieces][kRoom];
};

// The k-th largest of 256 keys, 4 a lane: bit by bit from the top, the largest bound that k reach.
template <int kBits>
__device__ __forceinline__ uint32_t kth_of(const uint32_t (&key)[4], int k) {
    uint32_t bound = 0;
#pragma unroll 1
    for (uint32_t bit = 1u << (kBits - 1); bit; bit >>= 1) {
        const uint32_t at = bound | bit;
        int n = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) n += __popcll(__ballot(key[j] >= at));
        if (n >= k) bound = at;
    }
    return bound;
}

// how many of the first n short keys come before the i-th: larger, or equal and earlier
__device__ __forceinline__ int rank_of(const uint4* keys, int n, int i) {
    const uint32_t key = reinterpret_cast<const uint32_t*>(keys)[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 4) {
        const uint4 q = keys[j / 4];
        rank += (j < n && (q.x > key || (q.x == key && j < i))) + (j + 1 < n && (q.y > key || (q.y == key && j + 1 < i))) +
                (j + 2 < n && (q.z > key || (q.z == key && j + 2 < i))) + (j + 3 < n && (q.w > key || (q.w == key && j + 3 < i)));
    }
    return rank;
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
                sh.above_cut = sum;
            }
        }
        __syncthreads();
        prefix = prefix << width | (uint32_t)sh.box[0];
        above = sh.above_cut;
    }
    *cut = prefix;
    *above_cut = above;
    *there = sh.box[1];
}

// The bins, the likeliest first, in which the weights reach `want` steps: on either side by what the bins' sums of V
// weights in whole steps, half a step each, and the whole's own rounding may be off. bins[0]: the first that may be it,
// [1]: the last; -1 where the bins do not reach it. For the first wave; mass is in LDS.
__device__ __forceinline__ void find_bins(const unsigned long long* mass, double want, int V, int* bins) {
    const int lane = (int)threadIdx.x & 63;
    constexpr int kEach = kBins / 64;
    uint64_t own = 0, all;
#pragma unroll
    for (int j = 0; j < kEach; ++j) own += mass[kEach * lane + j];
    const uint64_t above = wave_before(own, &all);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const double off = want * 1e-12 + (double)V, at = fmax(side ? want + off : want - off, 1.0);
        const uint64_t hit = __ballot((double)above < at && (double)(above + own) >= at);
        int bin = -1;
        if (hit) {
            const int from = __builtin_ctzll(hit);           // the lane whose bins hold it: one of them a lane
            const uint64_t one = lane < kEach ? mass[kEach * from + lane] : 0, low = from_lane(above, from) + wave_before(one, &all);
            bin = kEach * from + __builtin_ctzll(__ballot((double)(low + one) >= at));
        }
        if (lane == 0) bins[side] = bin;
    }
}

// The part, of n <= 64, in which the running sum from `run` on exceeds the target, and what lies before it; where
// none does (rounding, or not asked for: !exact) the last that is not 0, and exact becomes false.
__device__ __forceinline__ int pick_part(const double* part, int n, double target, double* run, bool* exact) {
    const int lane = (int)threadIdx.x & 63;
    double own = lane < n ? part[lane] : 0.0, all;
    const double low = *run + wave_before(own, &all);
    const uint64_t some = __ballot(own > 0.0), over = *exact ? __ballot(own > 0.0 && low + own > target) : 0;
    if (!over) *exact = false;
    const int at = over ? __builtin_ctzll(over) : some ? 63 - __builtin_clzll(some) : 0;
    *run = from_lane(low, at);
    return at;
}

// ---- few rows: a workgroup of 4 waves a piece

template <int kKind>
__global__ __launch_bounds__(kPieceThreads) void piece_max_kernel(const SampleArgs a) {
    const int m = (int)blockIdx.x / kPieces, c = (int)blockIdx.x % kPieces, w = (int)threadIdx.x >> 6;
    const Row<kKind> row(a, m);
    const int part = (row.piece() + 4 * kStep - 1) / (4 * kStep) * kStep;
    const int64_t base = (int64_t)c * row.piece();
    const int end = row.start(base + row.piece()), i0 = row.start(base + (int64_t)w * part);
    const int from = i0 < end ? i0 : end, to = end - from < part ? end : from + part;
    float most = -INFINITY;
    row.template walk<kKind == 2 ? 2 : 4>(from, to, [&](const auto& r, int) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) most = fmaxf(most, Logit<kKind>::at(r, e));
    });
    for (int s = 8; s > 0; s >>= 1) most = fmaxf(most, __shfl_xor(most, s));
    if (threadIdx.x < kBins / kPieces) a.left[m].mass[c * (kBins / kPieces) + (int)threadIdx.x] = 0ull;
    if ((threadIdx.x & 15) == 0) a.left[m].group_max[c * (kGroups / kPieces) + ((int)threadIdx.x >> 4)] = most;
}

// Each wave's list of a piece to its place behind those of the waves before it.
struct PieceList {
    uint32_t key[4][kRoom];
    int index[4][kRoom];
    int n[4];
};
__device__ __forceinline__ void leave_list(PieceList& l, Left& left, int c) {
    const int w = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
    __syncthreads();
    int first = 0;
    for (int k = 0; k < w; ++k) first += l.n[k];
    for (int j = lane; j < l.n[w] && first + j < kRoom; j += 64) {
        left.key[c][first + j] = l.key[w][j];
        left.index[c][first + j] = l.index[w][j];
    }
    if (threadIdx.x == kPieceThreads - 1) left.listed[c] = first + l.n[w];
}

template <int kKind>
__global__ __launch_bounds__(kPieceThreads) void piece_sum_kernel(const SampleArgs a) {
    __shared__ double wave_part[4];
    __shared__ unsigned long long mass[kBins];
    __shared__ PieceList list;
    using L = Logit<kKind>;
    const int m = (int)blockIdx.x / kPieces, c = (int)blockIdx.x % kPieces, tid = (int)threadIdx.x, w = tid >> 6, lane = tid & 63;
    const How how(a, m);
    const f32x4 groups = reinterpret_cast<const f32x4*>(a.left[m].group_max)[lane];
    const float top = wave_max(fmaxf(fmaxf(groups[0], groups[1]), fmaxf(groups[2], groups[3])));
    // (all, or left to the last launch)
    if (how.greedy || !(top > -INFINITY) || top == INFINITY || (how.limit_k && !how.by_groups)) return;
    const Row<kKind> row(a, m);
    const int part = (row.piece() + 4 * kStep - 1) / (4 * kStep) * kStep;
    const int64_t base = (int64_t)c * row.piece();
    const int end = row.start(base + row.piece()), i0 = row.start(base + (int64_t)w * part);
    const int from = i0 < end ? i0 : end, to = end - from < part ? end : from + part;
    if (how.by_groups) {
        const uint32_t keys[4] = {L::key(groups[0]), L::key(groups[1]), L::key(groups[2]), L::key(groups[3])};
        const int n = row.gather(from, to, L::value(kth_of<L::kBits>(keys, how.k)), NAN, list.key[w], list.index[w], kRoom, 0);
        if (lane == 0) list.n[w] = n;
        leave_list(list, a.left[m], c);
        return;
    }
    const Weight weight(top, how.t);
    const double unit = (double)(1ull << a.unit_shift);
    for (int b = tid; b < kBins; b += kPieceThreads) mass[b] = 0ull;
    __syncthreads();
    double sum = wave_sum(row.sum_of(from, to, weight, how, unit, mass));
    if (lane == 0) wave_part[w] = sum;
    __syncthreads();
    if (tid == 0) a.left[m].sum[c] = wave_part[0] + wave_part[1] + wave_part[2] + wave_part[3];
    if (how.by_bins)
        for (int b = tid; b < kBins; b += kPieceThreads)
            if (mass[b]) atomicAdd(&a.left[m].mass[b], mass[b]);
}

template <int kKind>
__global__ __launch_bounds__(kPieceThreads) void piece_cut_kernel(const SampleArgs a) {
    __shared__ double wave_part[4][2];
    __shared__ unsigned long long mass[kBins];
    __shared__ int bins[2];
    __shared__ PieceList list;
    const int m = (int)blockIdx.x / kPieces, c = (int)blockIdx.x % kPieces, tid = (int)threadIdx.x, w = tid >> 6, lane = tid & 63;
    const How how(a, m);
    if (how.greedy || !how.by_bins) return;
    Left& left = a.left[m];
    const f32x4 groups = reinterpret_cast<const f32x4*>(left.group_max)[lane];
    for (int b = tid; b < kBins; b += kPieceThreads) mass[b] = left.mass[b];
    double whole = 0.0;
#pragma unroll
    for (int k = 0; k < kPieces; ++k) whole += left.sum[k];
    const float top = wave_max(fmaxf(fmaxf(groups[0], groups[1]), fmaxf(groups[2], groups[3])));
    if (!(top > -INFINITY) || top == INFINITY) return;
    __syncthreads();
    const double unit = (double)(1ull << a.unit_shift);
    if (w == 0) find_bins(mass, how.p * whole * unit, a.V, bins);
    __syncthreads();
    if (bins[0] < 0 || bins[1] < 0) {
        if (tid == 0) left.listed[c] = kRoom + 1;              // over the row itself
        return;
    }
    const Row<kKind> row(a, m);
    const Weight weight(top, how.t);
    const int part = (row.piece() + 4 * kStep - 1) / (4 * kStep) * kStep;
    const int64_t base = (int64_t)c * row.piece();
    const int end = row.start(base + row.piece()), i0 = row.start(base + (int64_t)w * part);
    const int from = i0 < end ? i0 : end, to = end - from < part ? end : from + part;
    // what may be cut, and what surely is not
    const float low = bin_end(weight, bins[1], 1e-6), high = bins[0] > 0 ? bin_end(weight, bins[0] - 1, -1e-6) : INFINITY;
    const int n = row.gather(from, to, low, high, list.key[w], list.index[w], kRoom, 0);
    double above, above_kept;
    row.sum_above(from, to, high, weight, how.min_w, &above, &above_kept);
    if (lane == 0) {
        list.n[w] = n;
        wave_part[w][0] = above;
        wave_part[w][1] = above_kept;
    }
    leave_list(list, left, c);
    if (tid == 0) {
        left.above[c] = wave_part[0][0] + wave_part[1][0] + wave_part[2][0] + wave_part[3][0];
        left.above_kept[c] = wave_part[0][1] + wave_part[1][1] + wave_part[2][1] + wave_part[3][1];
    }
}

// ---- the row's token: by one workgroup, from its logits alone or (kLeft) with what the launches above left

template <int kKind, bool kLeft>
__global__ __launch_bounds__(kThreads) void sample_kernel(const SampleArgs a) {
    using L = Logit<kKind>;
    using Eight = typename L::Eight;
    __shared__ Shared sh;
    const int tid = (int)threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = (int)blockIdx.x;
    const Row<kKind> row(a, m);
    const How how(a, m);
    const float uf = a.u[m];
    const int piece = row.piece();
    const int from = row.start((int64_t)wv * piece), to = row.start((int64_t)(wv + 1) * piece);
    [[maybe_unused]] const Left* left = kLeft ? a.left + m : nullptr;

    // ---- 1. the largest, of the thread and of all
    float mine = -INFINITY;
    if constexpr (kLeft) {
        if (tid < kGroups) mine = left->group_max[tid];
    } else {
        row.template walk<kKind == 2 ? 3 : 8>(from, to, [&](const Eight& r, int) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) mine = fmaxf(mine, L::at(r, e));
        });
    }
    float top = wave_max(mine);
    if (lane == 0) sh.part[wv] = (double)top;
    __syncthreads();
    for (int k = 0; k < kWaves; ++k) top = fmaxf(top, (float)sh.part[k]);
    __syncthreads();
    if (top == -INFINITY) {
        if (tid == 0) {
            a.ids[m] = -1;
            if (a.logprob) a.logprob[m] = -INFINITY;
        }
        return;
    }
    if (how.greedy) {
        // the lowest index that has it
        if (tid == 0) sh.box[0] = kNone;
        __syncthreads();
        int at = kNone;
        row.template walk<kKind == 2 ? 2 : 4>(from, to, [&](const Eight& r, int i) {
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
    const Weight weight(top, how.t);
    const double unit = (double)(1ull << a.unit_shift), min_w = how.min_w;
    auto fixed = [&](double w) { return fixed_point(w, unit); };
    const bool last_of_all = uf >= 1.f;
    const double share = uf > 0.f ? (double)uf : 0.0;
    auto answer = [&](int id, double w, double total) {
        a.ids[m] = id;
        if (a.logprob) a.logprob[m] = (float)log(w / total);
    };
    auto sums_of_waves = [&](double v, double* part) {            // -> of all
        v = wave_sum(v);
        __syncthreads();
        if (lane == 0) part[wv] = v;
        __syncthreads();
        double all = 0.0;
        for (int k = 0; k < kWaves; ++k) all += part[k];
        return all;
    };
    auto lists_fit = [&](int n) {
        __syncthreads();
        if (lane == 0) sh.listed[wv] = n;
        __syncthreads();
        bool fits = true;
        for (int k = 0; k < kPieces; ++k) fits = fits && sh.listed[k] <= kRoom;
        return fits;
    };

    // ---- 2. and 3. lists and sums of the pieces. `listed`: the list holds what is kept (top-k) or
    // what may be cut (top-p); `summed`: sh.part holds the pieces' sums, sh.above what lies above the list
    bool listed = false, summed = false;
    double whole = 0.0;                          // the weight of all
    if (how.limit_k ? how.k <= kThreads : !weight.endless) {
        if (kLeft && how.by_groups && top != INFINITY) {
            int n = left->listed[wv];
            for (int j = lane; j < n && j < kRoom; j += 64) {
                sh.key[wv][j] = left->key[wv][j];
                sh.index[wv][j] = left->index[wv][j];
            }
            listed = lists_fit(n);
        } else if (how.limit_k) {
            uint32_t bound;
            if (how.by_groups && !kLeft) {
                float most = fmaxf(mine, __shfl_xor(mine, 1));
                most = fmaxf(most, __shfl_xor(most, 2));
                if ((lane & 3) == 0) reinterpret_cast<uint32_t*>(sh.short_key)[tid >> 2] = L::key(most);
                __syncthreads();
                const uint4 q = sh.short_key[lane];
                const uint32_t keys[4] = {q.x, q.y, q.z, q.w};
                bound = kth_of<L::kBits>(keys, how.k);
            } else {
                if constexpr (kLeft) {
                    mine = -INFINITY;
                    row.template walk<kKind == 2 ? 2 : 4>(from, to, [&](const Eight& r, int) {
#pragma unroll
                        for (int e = 0; e < kVec; ++e) mine = fmaxf(mine, L::at(r, e));
                    });
                }
                int equals;
                find_count<L>(sh, [&](auto f) { f(L::key(mine)); }, how.k, &bound, &equals);
            }
            listed = lists_fit(row.gather(from, to, L::value(bound), NAN, sh.key[wv], sh.index[wv], kRoom, 0));
        } else if constexpr (kLeft) {
            whole = 0.0;
            if (tid < kPieces) {
                sh.part[tid] = left->sum[tid];
                if (how.by_bins) {
                    sh.above[tid] = left->above[tid];
                    sh.above_kept[tid] = left->above_kept[tid];
                }
            }
            if (how.by_bins) {
                int n = left->listed[wv];
                for (int j = lane; j < n && j < kRoom; j += 64) {
                    sh.key[wv][j] = left->key[wv][j];
                    sh.index[wv][j] = left->index[wv][j];
                }
                listed = summed = lists_fit(n);
            } else {
                __syncthreads();
                summed = true;
            }
            for (int k = 0; k < kPieces; ++k) whole += sh.part[k];
        } else {
            sh.mass[tid] = 0ull;
            __syncthreads();
            whole = sums_of_waves(row.sum_of(from, to, weight, how, unit, sh.mass), sh.part);
            summed = true;
            if (how.by_bins) {
                if (wv == 0) find_bins(sh.mass, how.p * whole * unit, a.V, sh.box);
                __syncthreads();
                const int first = sh.box[0], last = sh.box[1];
                summed = first >= 0 && last >= 0;
                if (summed) {
                    const float low = bin_end(weight, last, 1e-6), high = first > 0 ? bin_end(weight, first - 1, -1e-6) : INFINITY;
                    listed = summed = lists_fit(row.gather(from, to, low, high, sh.key[wv], sh.index[wv], kRoom, 0));
                    double above = 0.0, above_kept = 0.0;
                    if (listed) row.sum_above(from, to, high, weight, min_w, &above, &above_kept);
                    if (lane == 0) {
                        sh.above[wv] = above;
                        sh.above_kept[wv] = above_kept;
                    }
                }
            }
        }
    }
    __syncthreads();

    uint32_t cut = 0;                            // keys above it are kept,
    int ties = kNone;                            // of those equal to it the first `ties`,
    int last_tie = kNone;                        // which end at this index
    int entries = 0, first_entry = 0;
    if (listed)
        for (int k = 0; k < kPieces; ++k) {
            if (k == wv) first_entry = entries;
            entries += sh.listed[k];
        }
    double over_list = 0.0;                      // the weight above the list
    if (summed && how.by_bins)
        for (int k = 0; k < kPieces; ++k) over_list += sh.above[k];
    bool cut_found = summed && !how.by_bins;     // only the draw is left
    if (listed && entries <= kShort) {
        // ---- a short list: the entries in falling order by counting, then back in index order
        for (int j = lane; j < sh.listed[wv]; j += 64) {
            reinterpret_cast<uint32_t*>(sh.short_key)[first_entry + j] = sh.key[wv][j];
            sh.short_index[first_entry + j] = sh.index[wv][j];
        }
        if (tid == 0) sh.box[0] = -1;
        __syncthreads();
        if (how.limit_k && tid >= kShort) return;
        // sums over the first four waves: of the lower threads, and of all
        auto before_of = [&](double v, double* all) {
            double own;
            double low = wave_before(v, &own);
            __syncthreads();
            if (lane == 0 && wv < kShort / 64) sh.sorted[kShort - 1 - wv] = own;
            __syncthreads();
            *all = 0.0;
            for (int k = 0; k < kShort / 64; ++k) {
                if (k == wv) low += *all;
                *all += sh.sorted[kShort - 1 - k];
            }
            __syncthreads();
            return low;
        };
        int rank = 0;
        double own_w = 0.0;
        if (tid < entries) {
            rank = rank_of(sh.short_key, entries, tid);
            own_w = weight(L::value(reinterpret_cast<uint32_t*>(sh.short_key)[tid]));
            sh.sorted[rank] = own_w;
            sh.entry[rank] = tid;
        }
        __syncthreads();
        const int at = tid < entries ? sh.entry[tid] : 0;            // thread r: the entry of rank r
        double w = tid < entries && (!how.limit_k || tid < how.k) ? sh.sorted[tid] : 0.0, all;
        const double above = before_of(w, &all) + over_list;
        const bool stays = tid < entries && (how.limit_k ? tid < how.k && (!how.limit_p || tid == 0 || above < how.p * all)
                                                         : above < how.p * whole || (tid == 0 && over_list == 0.0));
        if (how.by_bins) {
            // the last that stays is the cut
            if (stays) atomicMax(&sh.box[0], tid);
            __syncthreads();
            const int last = sh.box[0];
            if (tid == (last < 0 ? 0 : last) && tid < entries) {
                sh.box[1] = last < 0 ? -1 : sh.short_index[at];
                sh.count[0] = reinterpret_cast<uint32_t*>(sh.short_key)[at];
            }
            __syncthreads();
            cut = entries ? sh.count[0] : 0u;
            last_tie = entries ? sh.box[1] : kNone;
            cut_found = true;
        } else {
            if (!stays || w < min_w) w = 0.0;
            if (tid < entries) sh.sorted[at] = w;
            if (tid == 0) {
                sh.box[0] = kNone;
                sh.box[1] = -1;
            }
            __syncthreads();
            w = tid < entries ? sh.sorted[tid] : 0.0;
            double total;
            const double low = before_of(w, &total);
            if (w > 0.0) {
                if (!last_of_all && low + w > share * total) atomicMin(&sh.box[0], tid);
                atomicMax(&sh.box[1], tid);
            }
            __syncthreads();
            if (tid == (sh.box[0] != kNone ? sh.box[0] : sh.box[1])) answer(sh.short_index[tid], w, total);
            return;
        }
    } else if (listed) {
        const int n = sh.listed[wv];
        auto each = [&](auto f) {
            for (int j = lane; j < n; j += 64) f(sh.key[wv][j], sh.index[wv][j]);
        };
        if (how.limit_k) find_count<L>(sh, [&](auto f) { each([&](uint32_t key, int) { f(key); }); }, how.k, &cut, &ties);
        // how many of the equals of the cut this wave keeps
        auto keep_of = [&] {
            int equals = 0, wave_equals;
            for (int j = lane; j < n; j += 64) equals += sh.key[wv][j] == cut;
            wave_before(equals, &wave_equals);
            __syncthreads();
            if (lane == 0) sh.listed[wv] = wave_equals;
            __syncthreads();
            int seen = 0;
            for (int k = 0; k < wv; ++k) seen += sh.listed[k];
            return ties > seen ? ties - seen : 0;
        };
        // sum of w over the wave's entries that are kept; f(entry, w) for each round of 64
        auto kept_entries = [&](int keep, auto f) {
            int met = 0;
            for (int j0 = 0; j0 < n; j0 += 64) {
                const int j = j0 + lane;
                const bool tie = j < n && sh.key[wv][j] == cut;
                const uint64_t mask = __ballot(tie);
                const int rank = met + __popcll(mask & ((1ull << lane) - 1ull));
                met += __popcll(mask);
                double w = 0.0;
                if (j < n && (sh.key[wv][j] > cut || (tie && rank < keep))) w = weight(L::value(sh.key[wv][j]));
                if (f(j, w)) return;
            }
        };
        auto kept_sum = [&](int keep) {
            double sum = 0.0;
            kept_entries(keep, [&](int, double w) {
                sum += w;
                return false;
            });
            return sum;
        };
        if (how.limit_p) {
            const uint32_t kcut = cut;
            const int kties = ties;
            if (how.limit_k) whole = sums_of_waves(kept_sum(keep_of()), sh.part);
            const double target = (how.p * whole - over_list) * unit;
            uint64_t above;
            int there;
            // the ties of the k-th count as often as they are kept: one entry brings them all
            const uint64_t tie_mass = how.limit_k ? (uint64_t)kties * fixed(weight(L::value(kcut))) : 0;
            find_mass<L>(sh, [&](auto f) {
                each([&](uint32_t key, int) {
                    if (!how.limit_k || key > kcut) f(key, [&] { return fixed(weight(L::value(key))); });
                });
                if (how.limit_k && tid == 0) f(kcut, [&] { return tie_mass; });
            }, target, &cut, &above, &there);
            if (how.limit_k && cut == kcut) there = kties;
            const uint64_t one = fixed(weight(L::value(cut)));
            // tie j (from 0) is kept while what lies before it is below the target
            double need = one ? ceil((target - (double)above) / (double)one) : (double)there;
            const double least = how.limit_k || over_list == 0.0 ? 1.0 : 0.0;
            need = need < least ? least : need;
            ties = need < (double)there ? (int)need : there;
        }
        const int keep = keep_of();
        if (how.by_bins) {
            // the index of the last tie that is kept (none: -1)
            if (tid == 0) sh.box[0] = -1;
            __syncthreads();
            int met = 0;
            for (int j0 = 0; j0 < n; j0 += 64) {
                const int j = j0 + lane;
                const bool tie = j < n && sh.key[wv][j] == cut;
                const uint64_t mask = __ballot(tie);
                if (tie && met + __popcll(mask & ((1ull << lane) - 1ull)) < keep) atomicMax(&sh.box[0], sh.index[wv][j]);
                met += __popcll(mask);
            }
            // (what this wave's list had is overwritten: its length is still in n)
            __syncthreads();
            last_tie = sh.box[0];
            cut_found = true;
            if (lane == 0) sh.listed[wv] = n;
            __syncthreads();
        } else {
            double sum = 0.0;
            kept_entries(keep, [&](int, double w) {
                sum += w >= min_w ? w : 0.0;
                return false;
            });
            const double total = sums_of_waves(sum, sh.part);
            const double target = share * total;
            // the wave in which the running sum exceeds the target, or the last that keeps any
            bool exact = !last_of_all;
            double before = 0.0;
            const int wave = pick_part(sh.part, kWaves, target, &before, &exact);
            if (wv != wave) return;
            int last_id = -1;
            double at = before, last_w = 0.0;
            bool done = false;
            kept_entries(keep, [&](int j, double w) {
                double all;
                if (w < min_w) w = 0.0;
                const double low = wave_before(w, &all);
                const uint64_t over = exact ? __ballot(w > 0.0 && at + low + w > target) : 0;
                if (over) {
                    if (lane == __builtin_ctzll(over)) answer(sh.index[wv][j], w, total);
                    done = true;
                    return true;
                }
                const uint64_t some = __ballot(w > 0.0);
                if (some) {
                    const int from_lane = 63 - __builtin_clzll(some);
                    last_id = __shfl(j < n ? sh.index[wv][j] : 0, from_lane);
                    last_w = __shfl(w, from_lane);
                }
                at += all;
                return false;
            });
            if (!done && lane == 0) answer(last_id, last_w, total);
            return;
        }
    }

    // ---- thresholds over the row itself
    if (!cut_found) {
        auto each = [&](auto f) { row.each(from, to, [&](float z, int) { f(z); }); };
        if (how.limit_k) find_count<L>(sh, [&](auto f) { each([&](float z) { f(L::key(z)); }); }, how.k, &cut, &ties);
        if (how.limit_p) {
            const uint32_t kcut = cut;
            const int kties = ties;
            const uint64_t tie_mass = how.limit_k ? (uint64_t)kties * fixed(weight(L::value(kcut))) : 0;
            double sum = 0.0;
            each([&](float z) {
                if (!how.limit_k || L::key(z) > kcut) sum += weight(z);
            });
            whole = sums_of_waves(sum, sh.part) + (how.limit_k ? (double)kties * weight(L::value(kcut)) : 0.0);
            const double target = how.p * whole * unit;
            uint64_t above;
            int there;
            find_mass<L>(sh, [&](auto f) {
                each([&](float z) {
                    if (!how.limit_k || L::key(z) > kcut) f(L::key(z), [&] { return fixed(weight(z)); });
                });
                if (how.limit_k && tid == 0) f(kcut, [&] { return tie_mass; });
            }, target, &cut, &above, &there);
            if (how.limit_k && cut == kcut) there = kties;
            const uint64_t one = fixed(weight(L::value(cut)));
            double need = one ? ceil((target - (double)above) / (double)one) : (double)there;
            need = need < 1.0 ? 1.0 : need;
            ties = need < (double)there ? (int)need : there;
        }
        // the index of the last tie that is kept
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
                row.stroll(from, to, [&](const Eight& r, int i) {
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
    }
    const bool all_kept = cut == 0 && min_w == 0.0;
    auto kept = [&](float z, int i) -> double {
        if (!all_kept) {
            const uint32_t key = L::key(z);
            if (key < cut || (key == cut && i > last_tie)) return 0.0;
        }
        const double w = weight(z);
        return w >= min_w ? w : 0.0;
    };
    // ---- 4. sums of the pieces, then of the sixteenths of the one in which the running sum exceeds the
    // target, until one is a step of a wave
    if (!summed) {
        double sum = 0.0;
        row.each(from, to, [&](float z, int i) { sum += kept(z, i); });
        sums_of_waves(sum, sh.part);
    } else if (how.by_bins) {
        // what is surely kept, and what of the list is
        double sum = 0.0;
        for (int j = lane; j < sh.listed[wv]; j += 64) {
            const double w = sh.key[wv][j] > cut || (sh.key[wv][j] == cut && sh.index[wv][j] <= last_tie) ? weight(L::value(sh.key[wv][j])) : 0.0;
            sum += w >= min_w ? w : 0.0;
        }
        sum = wave_sum(sum);
        __syncthreads();
        if (lane == 0) sh.part[wv] = sum + sh.above_kept[wv];
        __syncthreads();
    }
    double total = 0.0;
    for (int k = 0; k < kPieces; ++k) total += sh.part[k];
    const double target = share * total;
    int i0 = 0, i1 = row.V;
    double run = 0.0;
    bool exact = !last_of_all;
    for (int size = piece;;) {
        const int wave = pick_part(sh.part, kPieces, target, &run, &exact);
        const int64_t n0 = (int64_t)i0 + (int64_t)wave * size;
        i1 = i1 - n0 < size ? i1 : (int)n0 + size;
        i0 = (int)n0;
        if (size <= kStep) break;
        size = (int)(((int64_t)size + kWaves * kStep - 1) / (kWaves * kStep)) * kStep;
        const int64_t b64 = (int64_t)i0 + (int64_t)wv * size;
        const int b = b64 < i1 ? (int)b64 : i1, e1 = i1 - b < size ? i1 : b + size;
        double sum = 0.0;
        row.each(b, e1, [&](float z, int i) { sum += kept(z, i); });
        sums_of_waves(sum, sh.part);
    }
    // the step's eight times 64, a logit a lane: the wave that has it answers
    const int i = i0 + tid;
    const double w = tid < kStep && i < i1 ? kept(L::one(row.p, i), i) : 0.0;
    double all;
    const double low = wave_before(w, &all);
    __syncthreads();
    if (lane == 0) sh.part[wv] = all;
    __syncthreads();
    if (wv != pick_part(sh.part, kStep / 64, target, &run, &exact)) return;
    const uint64_t over = exact ? __ballot(w > 0.0 && run + low + w > target) : 0, some = __ballot(w > 0.0);
    if (lane == (over ? __builtin_ctzll(over) : 63 - __builtin_clzll(some))) answer(i, w, total);
}

// Rows m0 and on of a call.
SampleArgs rows_from(SampleArgs a, int m0, int bytes) {
    a.logits = static_cast<const uint8_t*>(a.logits) + (int64_t)m0 * a.ld * bytes;
    a.M -= m0;
    a.u += m0;
    if (a.temperatures) a.temperatures += m0;
    if (a.top_ks) a.top_ks += m0;
    if (a.top_ps) a.top_ps += m0;
    if (a.min_ps) a.min_ps += m0;
    a.ids += m0;
    if (a.logprob) a.logprob += m0;
    return a;
}

template <int kKind>
void launch_kind(const SampleArgs& a, hipStream_t s) {
    if (a.left) {
        const dim3 pieces((unsigned)(a.M * kPieces)), block(kPieceThreads);
        hipLaunchKernelGGL((piece_max_kernel<kKind>), pieces, block, 0, s, a);
        hipLaunchKernelGGL((piece_sum_kernel<kKind>), pieces, block, 0, s, a);
        // (without settings of each row, the host knows which rows cut by bins: none or all)
        if (a.top_ks || a.top_ps || (a.top_p < 1.f && !(a.top_k >= 1 && a.top_k < a.V)))
            hipLaunchKernelGGL((piece_cut_kernel<kKind>), pieces, block, 0, s, a);
        hipLaunchKernelGGL((sample_kernel<kKind, true>), dim3((unsigned)a.M), dim3(kThreads), 0, s, a);
    } else {
        for (int64_t m0 = 0; m0 < a.M; m0 += kRowsPerLaunch) {
            const SampleArgs b = rows_from(a, (int)m0, kKind == 2 ? 4 : 2);
            hipLaunchKernelGGL((sample_kernel<kKind, false>), dim3((unsigned)(b.M < kRowsPerLaunch ? b.M : kRowsPerLaunch)), dim3(kThreads), 0, s, b);
        }
    }
}

// Pieces where one workgroup a row would leave most of the chip idle and the row is long enough to be worth the
// launches; one rule for all settings, which may differ from row to row. Both ways, us, bf16, calls of a graph (pieces /
// a workgroup a row), without limits, top-k 50 with top-p 0.9, top-p 0.95:
//   1 x 131072    16 / 36    18 / 24    36 / 108        64 x 131072   25 / 38    24 / 27    64 / 115
//   128 x 131072  34 / 40    31 / 28    90 / 116        128 x 65536   25 / 24    27 / 22    68 / 72
//   1 x 24600     13 / 14    16 / 16    28 / 34         64 x 24600    16 / 15    20 / 18    40 / 38
//   16 x 32768    13 / 16    17 / 18    33 / 43         64 x 32768    16 / 16    20 / 18    42 / 44
bool in_pieces(int64_t M, int64_t V) { return V > 24576 && (M <= 64 || (M <= 128 && V >= 65536)); }

}  // namespace

size_t sample_workspace(int64_t M, int64_t V) { return in_pieces(M, V) ? (size_t)M * sizeof(Left) : 0; }

hipError_t launch_sample(const SampleCall& q, void* scratch, hipStream_t stream) {
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
    // One launch where the pieces' own leave it all the work: for the largest logit alone (15 us against 18), and
    // for a top-k that the groups do not bound (1 and 64 rows of 131072, bf16, one launch / pieces: k = 200 38 / 43
    // and 42 / 49, 1000 50 / 54 and 52 / 59, 5000 147 / 149 and 151 / 155).
    const bool greedy = !q.temperatures && !(q.temperature > 0.f);
    const bool long_k = !q.top_ks && q.top_k > kGroupK && q.top_k < q.V;
    a.left = in_pieces(q.M, q.V) && !greedy && !long_k ? static_cast<Left*>(scratch) : nullptr;
    if (q.kind == 0) launch_kind<0>(a, stream);
    else if (q.kind == 1) launch_kind<1>(a, stream);
    else launch_kind<2>(a, stream);
    return hipGetLastError();
}

}  // namespace w4a16
