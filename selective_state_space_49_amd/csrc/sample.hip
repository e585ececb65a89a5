// sample.hip -- the next token from a row of logits and one uniform number.
//
//     w_i = exp((logit_i - max) / temperature);   in the order of falling logits, equal ones by index:
//     the first top_k; of those the ones before which less than top_p of their mass lies; of those
//     the ones with w >= min_p;  then, by index, the first at which the sum of w exceeds u times all.
//
// Masses are whole numbers, w times 2^shift rounded (44 bits for a vocabulary of up to 2^18): their sums
// do not depend on an order, so neither does the token. They stay below 2^53 within a wave, where they
// are added as doubles, and below 2^62 in a row. Of a row, what top_k and top_p keep is a beginning of
// the falling order, so it is told by its last token: a 64-bit number of the logit's rank and the index
// ("place") compares as that order does.
//
// A row is read three times (from the caches after the first): the largest and the smallest logit; the
// number of logits in each of 2047 equal steps below the largest, which says in which steps the kept
// ones end; the masses. Logits of those steps (some hundreds) go to a list that is sorted in LDS, where
// the end is exact. A list that is too long for LDS is not made: bfloat16 logits around 20 lie 1/8 apart, and
// thousands of 131072 are equal. The end is found in their steps then by their places' digits, 11 bits a pass
// from the highest that differ on (a row of 131072 around 20, top_p 0.9: 350 us, 93 around 0; 256 of them 412 and
// 119). So it is among all logits if the steps do not hold the end, or a logit is +infinity.
//
// A block has a row, so a batch takes as long as its slowest row and a row as long as its chain of passes: 256 rows
// of 131072 float32 logits, each with its own settings, in 126 us (1.1 TB/s; a compute unit has work 54 % of that
// time, and its vector units are busy half of it), one row of 32000 in 27 us with a top_k of some tens.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "ssm_layers.h"

namespace ssm {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64, kEntries = 2048, kBins = 2048, kList = 2048;
constexpr uint32_t kNone = 0x007fffffu;  // the key of -infinity
#define kInfinity __builtin_inff()

typedef unsigned long long u64;

// Whole numbers in the order of the logits; -0 is 0.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) { return __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key); }
__device__ __forceinline__ u64 place_of(uint32_t key, uint32_t i) { return (u64)key << 32 | (0xffffffffu - i); }
__device__ __forceinline__ uint32_t index_of(u64 place) { return 0xffffffffu - (uint32_t)place; }

// Places without the bits that are the same for all of a row: of a bfloat16's key the lower 16 (0, or all set
// below 0), and those above the largest index.
template <typename T>
struct Short {
    static constexpr int kCut = sizeof(T) == 2 ? 16 : 0;
    int bits;  // of an index
    __device__ __forceinline__ explicit Short(int64_t vocab) : bits(vocab > 1 ? 64 - __clzll((long long)(vocab - 1)) : 0) {}
    __device__ __forceinline__ u64 of(uint32_t key, uint32_t i) const { return (u64)(key >> kCut) << bits | (((1u << bits) - 1) - i); }
    // the place from which on all that are kept lie
    __device__ __forceinline__ u64 place(u64 c) const {
        const uint32_t high = (uint32_t)(c >> bits), key = kCut == 0 ? high : high << kCut | (high >> 15 ? 0u : 0xffffu);
        return place_of(key, ((1u << bits) - 1) - (uint32_t)(c & ((1ull << bits) - 1)));
    }
};

// ------------------------------------------------------------------ sums over a wave and a block
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 moved(u64 x) {  // 0 where no lane sends
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)x, CTRL, ROWS, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(x >> 32), CTRL, ROWS, 0xf, false);
    return (u64)hi << 32 | lo;
}
// Inclusive sums over the lanes: within rows of 16, then of the rows.
__device__ __forceinline__ u64 wave_scan(u64 x) {
    x += moved<0x111, 0xf>(x);
    x += moved<0x112, 0xf>(x);
    x += moved<0x114, 0xf>(x);
    x += moved<0x118, 0xf>(x);
    x += moved<0x142, 0xa>(x);
    x += moved<0x143, 0xc>(x);
    return x;
}
__device__ __forceinline__ u64 lane_of(u64 x, int lane) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), lane);
    return (u64)hi << 32 | lo;
}
__device__ __forceinline__ u64 wave_sum(u64 x) { return lane_of(wave_scan(x), 63); }
__device__ __forceinline__ u64 wave_sum(double x) {  // of whole numbers, below 2^53 in all
    const auto add = [](double a, u64 b) { return a + __longlong_as_double((long long)b); };
    const auto bits = [](double a) { return (u64)__double_as_longlong(a); };
    x = add(x, moved<0x111, 0xf>(bits(x)));
    x = add(x, moved<0x112, 0xf>(bits(x)));
    x = add(x, moved<0x114, 0xf>(bits(x)));
    x = add(x, moved<0x118, 0xf>(bits(x)));
    x = add(x, moved<0x142, 0xa>(bits(x)));
    x = add(x, moved<0x143, 0xc>(bits(x)));
    return (u64)__longlong_as_double((long long)lane_of(bits(x), 63));
}
// Inclusive sums over the block's threads, in their order; all: the whole sum.
__device__ __forceinline__ u64 block_scan(u64 x, u64 *part, u64 &all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    x = wave_scan(x);
    __syncthreads();
    if (lane == 63) part[wave] = x;
    __syncthreads();
    const u64 sums = wave_scan(part[lane % kWaves]);  // lanes 0 to 15 count
    all = lane_of(sums, kWaves - 1);
    return wave ? x + lane_of(sums, __builtin_amdgcn_readfirstlane(wave) - 1) : x;
}

// ------------------------------------------------------------------ a row
// 2^((x - max) inv2) as a multiple of 2^-shift, rounded, and 0 for -infinity: a polynomial on [-1/2, 1/2]
// (equal ripple, 1 at 0, off by 2.2e-14 at most), then the whole part by the exponent.
struct Masses {
    double max, inv2, least;  // 1 / temperature in units of log 2; the mass of the least weight
    int shift;
    // A step of the polynomial with its coefficient in scalar registers, which the compiler would copy to
    // vector registers for every step.
    static __device__ __forceinline__ double step(double p, double f, double c) {
        double r;
        asm("v_fma_f64 %0, %1, %2, %3" : "=v"(r) : "v"(p), "v"(f), "s"(c));
        return r;
    }
    __device__ __forceinline__ double operator()(float x) const {
        const double t = fmax(((double)x - max) * inv2, -1000.0);
        const double n = __builtin_rint(t), f = t - n;
        double p = f * 1.0210919981407892e-07 + 1.3258537495951731e-06;
        p = step(p, f, 1.5252645306585149e-05);
        p = step(p, f, 0.00015403439922121213);
        p = step(p, f, 0.0013333558250865102);
        p = step(p, f, 0.009618129182540224);
        p = step(p, f, 0.055504108664325015);
        p = step(p, f, 0.24022650695717282);
        p = step(p, f, 0.6931471805599514);
        p = __builtin_fma(p, f, 1.0);
        return __builtin_rint(__builtin_amdgcn_ldexp(p, (int)n + shift));
    }
    // Beside an infinity only such logits have a mass.
    __device__ __forceinline__ double any(float x) const {
        if (max == (double)kInfinity) return x == kInfinity ? (double)(1ull << shift) : 0.0;
        return (*this)(x);
    }
};

// The logits in vectors of 16 bytes, 64 of them (a tile) to a wave.
template <typename T>
struct Logits {
    static constexpr int E = 16 / sizeof(T), kTile = 64 * E;
    const T *p;
    int64_t V;
    int skip;  // elements of the first vector before the row
    int64_t tiles, per_entry;
    int entries;  // neighbouring tiles whose kept mass is one sum
    __device__ __forceinline__ Logits(const T *row, int64_t n) : p(row), V(n) {
        skip = (int)((uintptr_t)row % 16 / sizeof(T));
        tiles = (V + skip + kTile - 1) / kTile;
        per_entry = (tiles + kEntries - 1) / kEntries;
        entries = (int)((tiles + per_entry - 1) / per_entry);
    }
    __device__ __forceinline__ int64_t first(int64_t tile, int lane) const { return tile * kTile + lane * E - skip; }
    // Elements from i on; what is not of the row becomes -infinity.
    __device__ __forceinline__ void load(int64_t i, float (&x)[E]) const {
        if (i >= 0 && i + E <= V) {
            const uint4 r = *(const uint4 *)(p + i);
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if constexpr (sizeof(T) == 2) x[e] = __uint_as_float(e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
                else x[e] = __uint_as_float(w[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = i + e >= 0 && i + e < V ? (float)p[i + e] : -kInfinity;
        }
    }
    // fn(x, the index of x[0], tile) for the tiles from, from + step, .., a wave at a time; UNROLL of them are loaded at once.
    template <int UNROLL, typename F>
    __device__ __forceinline__ void each(int64_t from, int64_t to, int64_t step, F fn) const {
        const int lane = threadIdx.x & 63;
        for (int64_t t = from; t < to; t += UNROLL * step) {
            float x[UNROLL][E];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u)
                if (u == 0 || t + u * step < to) load(first(t + u * step, lane), x[u]);
#pragma unroll
            for (int u = 0; u < UNROLL; ++u)
                if (u == 0 || t + u * step < to) fn(x[u], first(t + u * step, lane), t + u * step);
        }
    }
};

struct Shared {
    u64 entry[kEntries];
    u64 list[kList];
    u64 bins[kBins];  // logits of a step, and above them the sum of their places in it, in 256ths
    u64 part[2 * kWaves];
    uint32_t few[4 * kWaves];
    uint32_t count;
};

struct Settings {
    float temperature, top_p, min_p, u;
    int64_t top_k;
    bool by_k, by_p;
    __device__ __forceinline__ Settings(const SampleArgs &p, int64_t r) {
        temperature = p.temperature ? p.temperature[r] : p.temperature_all;
        top_p = p.top_p ? p.top_p[r] : p.top_p_all;
        min_p = p.min_p ? p.min_p[r] : p.min_p_all;
        top_k = p.top_k ? p.top_k[r] : p.top_k_all;
        u = p.u[r];
        by_k = top_k > 0 && top_k < p.vocab;
        by_p = top_p < 1.0f;
    }
};

// 1. The largest logit, the smallest above -infinity, whether there is a NaN, and, where the temperature
// is 0, the lowest index of the largest.
struct Ends {
    float high, low;
    uint32_t bad, where;
    __device__ __forceinline__ void join(const Ends &o) {
        if (o.high > high || (o.high == high && o.where < where)) {
            high = o.high;
            where = o.where;
        }
        low = fminf(low, o.low);
        bad |= o.bad;
    }
};
template <typename T>
__device__ __forceinline__ Ends find_ends(const Logits<T> &l, bool greedy, uint32_t *few) {
    constexpr int E = Logits<T>::E;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Ends r{-kInfinity, kInfinity, 0, 0xffffffffu};
    bool bad = false;
    if (greedy) {
        l.template each<4>(wave, l.tiles, kWaves, [&](const float(&x)[E], int64_t i, int64_t) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                bad |= x[e] != x[e];
                if (x[e] > r.high) {
                    r.high = x[e];
                    r.where = (uint32_t)(i + e);
                }
            }
        });
    } else {
        l.template each<4>(wave, l.tiles, kWaves, [&](const float(&x)[E], int64_t, int64_t) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                bad |= x[e] != x[e];
                r.high = fmaxf(r.high, x[e]);
                r.low = fminf(r.low, x[e] > -kInfinity ? x[e] : kInfinity);
            }
        });
    }
    r.bad = __ballot(bad) != 0;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) r.join(Ends{__shfl_xor(r.high, d), __shfl_xor(r.low, d), 0, (uint32_t)__shfl_xor(r.where, d)});
    if (lane == 0) {
        few[wave] = __float_as_uint(r.high);
        few[kWaves + wave] = __float_as_uint(r.low);
        few[2 * kWaves + wave] = r.bad;
        few[3 * kWaves + wave] = r.where;
    }
    __syncthreads();
    const int w = lane % kWaves;
    r = Ends{__uint_as_float(few[w]), __uint_as_float(few[kWaves + w]), few[2 * kWaves + w], few[3 * kWaves + w]};
#pragma unroll
    for (int d = 1; d < kWaves; d *= 2)
        r.join(Ends{__shfl_xor(r.high, d), __shfl_xor(r.low, d), (uint32_t)__shfl_xor(r.bad, d), (uint32_t)__shfl_xor(r.where, d)});
    return r;
}
__device__ __forceinline__ bool is_lost(const Ends &e, const Settings &s) {
    return e.bad || !(e.high > -kInfinity) || !(s.temperature >= 0.0f) || s.u != s.u;
}

// The steps: up to 33.5 temperatures below the largest (from 32 on nothing has mass), or to the smallest
// logit if that is nearer. The last step is what is beyond, -infinity included.
struct Steps {
    float high, per;
    __device__ __forceinline__ Steps(const Ends &e, const Settings &s) : high(e.high) {
        const float far = fminf(33.5f * s.temperature, e.high - e.low);
        per = far > 0.0f ? fminf((kBins - 1.5f) / far, 1e30f) : 0.0f;
    }
    __device__ __forceinline__ float of(float x) const { return (high - x) * per; }
};

// 2. The number of logits in every step.
template <typename T>
__device__ __forceinline__ void count_steps(const Logits<T> &l, const Steps &st, u64 *bins) {
    constexpr int E = Logits<T>::E;
    l.template each<4>(threadIdx.x >> 6, l.tiles, kWaves, [&](const float(&x)[E], int64_t, int64_t) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float at = fminf(st.of(x[e]), (float)(kBins - 1));  // a NaN (-infinity where all are equal) too
            const int b = (int)at;
            atomicAdd(&bins[b], (u64)(uint32_t)((at - (float)b) * 256.0f) << 32 | 1ull);
        }
    });
}

// Where the kept ones end: the step of top_k's last (kBins: it keeps all that has mass) and the number
// before that step; the steps in which top_p's last lies. Where top_k keeps so few that the list holds them all
// with their last step (`whole`), they need no masses but in the list (one row of 32000 with 50 of them: 27
// us, 31 without this).
struct Plan {
    int end_k, p_from, p_to;
    u64 before_k;
    bool whole;
};
__device__ __forceinline__ Plan plan_ends(Shared &sh, const Settings &s, const Steps &st) {
    Plan pl{kBins, kBins, kBins, 0, false};
    const int tid = threadIdx.x, b = 2 * tid;
    const u64 b0 = sh.bins[b], b1 = sh.bins[b + 1];
    const uint32_t n0 = (uint32_t)b0, n1 = (uint32_t)b1;
    u64 all;
    if (s.by_k) {
        if (tid == 0) sh.few[0] = kBins;
        const u64 upto = block_scan((u64)n0 + n1, sh.part, all), start = upto - n0 - n1, k = (u64)s.top_k;
        if (start < k && upto >= k) {
            const bool second = start + n0 < k;
            sh.few[0] = b + second;
            sh.few[1] = (uint32_t)(start + (second ? n0 : 0));
            sh.few[3] = (uint32_t)(second ? upto : start + n0);
        }
        __syncthreads();
        if (sh.few[0] < kBins - 1) {
            pl.end_k = (int)sh.few[0];
            pl.before_k = sh.few[1];
            pl.whole = sh.few[3] <= kThreads;
        }
    }
    if (pl.whole) {
        pl.p_from = 0;
        pl.p_to = pl.end_k;
    } else if (s.by_p) {
        // Masses estimated by the middle of a step's logits: a step is 1/61 of a unit at most, so they
        // are right to (1/61)^2 / 8 = 3e-5. By the step's middle they were off by half a percent, and
        // one heavy token by more than the mass of many steps of light ones.
        const float width = st.per > 0.0f ? 1.0f / (st.per * s.temperature) : 0.0f;
        const auto guess = [&](int i, u64 bin) {
            const float n = (float)(uint32_t)bin, many = i < pl.end_k ? n : i == pl.end_k ? (float)((u64)s.top_k - pl.before_k) : 0.0f;
            return many > 0.0f ? (u64)(many * __expf(-((float)i + (float)(uint32_t)(bin >> 32) / (256.0f * n)) * width) * 0x1p36f) : 0ull;
        };
        const u64 g0 = guess(b, b0), g1 = guess(b + 1, b1);
        if (tid == 0) sh.few[2] = kBins;
        const u64 sum = block_scan(g0 + g1, sh.part, all);
        const double aim = (double)s.top_p * (double)all;
        if ((double)(sum - g0 - g1) < aim && !((double)sum < aim)) atomicMin(&sh.few[2], (uint32_t)(b + ((double)(sum - g1) < aim)));
        __syncthreads();
        const int c = s.top_p > 0.0f ? (int)sh.few[2] : 0;
        pl.p_from = max(c - 1, 0);
        pl.p_to = min(c + 1, kBins - 1);
    }
    return pl;
}

// 3. The masses of the entries: what is certainly kept, to its entry; sums (of a thread) of what
// lies before top_k's last step, and of the certain part of it; and the list.
template <typename T>
__device__ __forceinline__ void weigh(const Logits<T> &l, const Settings &s, const Steps &st, const Plan &pl,
                                      const Masses &mass, u64 *entry, u64 *list, uint32_t *count, u64 &all, u64 &kept) {
    constexpr int E = Logits<T>::E;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool filtered = s.by_k || s.by_p, choosy = mass.least > 0.0;
    const float end = pl.end_k < kBins ? (float)pl.end_k : kInfinity, past = pl.end_k < kBins ? (float)(pl.end_k + 1) : kInfinity;
    const float p0 = s.by_p ? (float)pl.p_from : end, p1 = s.by_p ? (pl.p_to < kBins - 1 ? (float)(pl.p_to + 1) : kInfinity) : end;
    const float last = s.by_k ? past : p1;  // of the list
    double sum = 0.0, sure = 0.0, mine = 0.0;
    const auto tile = [&](const float(&x)[E], int64_t i, int64_t) {
        if (!filtered) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const double m = mass(x[e]);
                mine += choosy && m < mass.least ? 0.0 : m;
            }
            return;
        }
        float at[E];
        bool some = false, listed = false;
        if (pl.whole) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                at[e] = st.of(x[e]);
                listed |= at[e] < past;
            }
            if (__ballot(listed) == 0) return;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (at[e] < past) {
                    const uint32_t n = atomicAdd(count, 1u);
                    if (n < kList) list[n] = place_of(key_of(x[e]), (uint32_t)(i + e));
                }
            return;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            at[e] = st.of(x[e]);
            some |= at[e] < end;
            listed |= at[e] >= p0 && at[e] < last;
        }
        if (__ballot(listed)) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (at[e] >= p0 && at[e] < last && (at[e] < p1 || at[e] >= end)) {
                    const uint32_t n = atomicAdd(count, 1u);
                    if (n < kList) list[n] = place_of(key_of(x[e]), (uint32_t)(i + e));
                }
        }
        if (__ballot(some) == 0) return;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const double m = mass(x[e]), yes = at[e] < p0 ? m : 0.0;
            if (s.by_p) sum += s.by_k && !(at[e] < end) ? 0.0 : m;
            if (choosy) {
                sure += yes;
                mine += m < mass.least ? 0.0 : yes;
            } else {
                mine += yes;
            }
        }
    };
    if (l.per_entry == 1) {
        for (int e = wave; e < l.entries; e += 4 * kWaves)
            l.template each<2>(e, std::min(e + 3 * kWaves + 1, l.entries), kWaves, [&](const float(&x)[E], int64_t i, int64_t t) {
                mine = 0.0;
                tile(x, i, t);
                if (s.by_p && !choosy) sure += mine;
                const u64 m = __ballot(mine > 0.0) ? wave_sum(mine) : 0;
                if (lane == 0) entry[t] = m;
            });
    } else {
        for (int e = wave; e < l.entries; e += kWaves) {
            mine = 0.0;
            l.template each<1>(e * l.per_entry, std::min<int64_t>((e + 1) * l.per_entry, l.tiles), 1, tile);
            if (s.by_p && !choosy) sure += mine;
            const u64 m = __ballot(mine > 0.0) ? wave_sum(mine) : 0;
            if (lane == 0) entry[e] = m;
        }
    }
    all = (u64)sum;
    kept = (u64)sure;
}

// ------------------------------------------------------------------ the end
// The list in falling order, by Batcher's bitonic network: a thread holds elements tid and tid + 1024.
// Neighbours within a wave meet by shuffles, others in LDS.
__device__ __forceinline__ void sort_list(u64 *list, int n) {
    const int tid = threadIdx.x;
    int size = 64;
    while (size < n) size *= 2;
    const int held = size > kThreads ? 2 : 1;
    u64 x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) x[h] = tid + h * kThreads < n ? list[tid + h * kThreads] : 0;
    __syncthreads();
    const bool works = tid < size;  // whole waves
    for (int k = 2; k <= size; k *= 2)
        for (int j = k / 2; j > 0; j /= 2) {
            if (j == kThreads) {  // the two of a thread, in the last round: falling
                const u64 hi = std::max(x[0], x[1]), lo = std::min(x[0], x[1]);
                x[0] = hi;
                x[1] = lo;
                continue;
            }
            if (j >= 64) {
                if (works) {
                    list[tid] = x[0];
                    if (held == 2) list[tid + kThreads] = x[1];
                }
                __syncthreads();
            }
            if (works) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == held) break;
                    const int i = tid + h * kThreads;
                    const u64 y = j < 64 ? (u64)__shfl_xor((long long)x[h], j) : list[i ^ j];
                    // the lower place of a pair takes the larger in a falling part
                    const bool larger = ((i & j) == 0) == ((i & k) == 0);
                    x[h] = larger ? std::max(x[h], y) : std::min(x[h], y);
                }
            }
            if (j >= 64) __syncthreads();
        }
    if (works) {
        list[tid] = x[0];
        if (held == 2) list[tid + kThreads] = x[1];
    }
    __syncthreads();
}

// The logits of a range of steps, or all.
struct Among {
    const Steps *st;
    float from, to;
    __device__ __forceinline__ bool operator()(float x, uint32_t key) const {
        if (!st) return key > kNone;
        const float at = st->of(x);
        return at >= from && at < to;
    }
};

// The mass of those of a range that are not behind place `least`.
template <typename T>
__device__ __noinline__ u64 mass_among(const Logits<T> &l, const Masses &mass, const Among &among, u64 least, Shared &sh) {
    const Short<T> sp(l.V);
    double m = 0.0;
    l.template each<1>(threadIdx.x >> 6, l.tiles, kWaves, [&](const float(&x)[Logits<T>::E], int64_t i, int64_t) {
#pragma unroll
        for (int e = 0; e < Logits<T>::E; ++e) {
            const uint32_t key = key_of(x[e]);
            if (among(x[e], key) && sp.of(key, (uint32_t)(i + e)) >= least) m += mass.any(x[e]);
        }
    });
    u64 all;
    block_scan((u64)m, sh.part, all);
    return all;
}

// Of those of a range that are not behind place `least`, in their order, the first at which their number (or,
// BY_MASS, their mass), and `before` that lies before them, reaches `want`; 0 if none does.
template <typename T, bool BY_MASS>
__device__ __noinline__ u64 first_to_reach(const Logits<T> &l, const Masses &mass, const Among &among, u64 least, u64 before, double want,
                                           Shared &sh) {
    constexpr int E = Logits<T>::E;
    const Short<T> sp(l.V);
    const int tid = threadIdx.x;
    const auto each = [&](auto fn) {
        l.template each<2>(tid >> 6, l.tiles, kWaves, [&](const float(&x)[E], int64_t i, int64_t) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const uint32_t key = key_of(x[e]);
                const u64 c = sp.of(key, (uint32_t)(i + e));
                if (among(x[e], key) && c >= least) fn(x[e], c);
            }
        });
    };
    u64 lo = ~0ull, hi = 0;
    each([&](float, u64 c) {
        lo = std::min(lo, c);
        hi = std::max(hi, c);
    });
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        lo = std::min(lo, (u64)__shfl_xor((long long)lo, d));
        hi = std::max(hi, (u64)__shfl_xor((long long)hi, d));
    }
    __syncthreads();
    if ((tid & 63) == 0) {
        sh.part[tid >> 6] = lo;
        sh.part[kWaves + (tid >> 6)] = hi;
    }
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) {
        lo = std::min(lo, sh.part[w]);
        hi = std::max(hi, sh.part[kWaves + w]);
    }
    if (lo > hi) return 0;
    for (;;) {
        const u64 differ = lo ^ hi;
        const int shift = differ >> 11 ? 53 - __clzll((long long)differ) : 0;
        const u64 base = lo >> shift;  // bins up to hi's: 2048 at most
        for (int b = tid; b < kBins; b += kThreads) sh.bins[b] = 0;
        if (tid == 0) sh.few[0] = kBins;
        __syncthreads();
        each([&](float x, u64 c) {
            if (c >= lo && c <= hi) atomicAdd(&sh.bins[(c >> shift) - base], BY_MASS ? (u64)mass.any(x) : 1ull);
        });
        __syncthreads();
        // from the last bin down, two a thread
        const u64 b0 = sh.bins[kBins - 1 - 2 * tid], b1 = sh.bins[kBins - 2 - 2 * tid];
        u64 all;
        const u64 upto = before + block_scan(b0 + b1, sh.part, all);
        const auto reached = [&](u64 sum) { return sum > 0 && !((double)sum < want); };
        if (reached(upto)) atomicMin(&sh.few[0], (uint32_t)(2 * tid + !reached(upto - b1)));
        __syncthreads();
        const int r = (int)sh.few[0];
        if (r == kBins) return 0;
        if (r / 2 == tid) sh.list[0] = r & 1 ? upto - b1 : upto - b1 - b0;
        __syncthreads();
        before = sh.list[0];
        const u64 bin = base + (u64)(kBins - 1 - r);
        if (shift == 0) return bin;
        lo = std::max(lo, bin << shift);
        hi = std::min(hi, (bin << shift) + ((1ull << shift) - 1));
    }
}

// The last kept place without a list, and the entries with it. st: where the plan holds (all: the mass before
// top_k's last step; kept: of that, what lies before top_p's steps), or null; 0 if its steps do not hold the end.
template <typename T>
__device__ __noinline__ u64 descend(const Logits<T> &l, const Masses &mass, const Settings &s, const Steps *st, const Plan &pl, u64 all,
                                    u64 kept, Shared &sh) {
    constexpr int E = Logits<T>::E;
    const auto steps = [&](int from, int to) { return Among{st, (float)from, to < kBins - 1 ? (float)(to + 1) : kInfinity}; };
    u64 last = 0;
    const bool cut = st ? pl.end_k < kBins : s.by_k;
    if (cut) last = first_to_reach<T, false>(l, mass, steps(pl.end_k, pl.end_k), 0, st ? pl.before_k : 0, (double)s.top_k, sh);
    if (s.by_p) {
        if (!st) all = mass_among(l, mass, steps(0, 0), last, sh);
        else if (cut) all += mass_among(l, mass, steps(pl.end_k, pl.end_k), last, sh);
        const double part = (double)s.top_p * (double)all;
        const bool before = st && pl.p_from > 0 && !((double)kept < part);
        const u64 at = before ? 0 : first_to_reach<T, true>(l, mass, steps(pl.p_from, pl.p_to), last, st ? kept : 0, part, sh);
        if (at == 0 && st && (before || pl.p_to < std::min(pl.end_k, kBins - 1)))
            return 0;
        last = std::max(last, at);
    }
    last = Short<T>(l.V).place(last);
    __syncthreads();
    for (int e = threadIdx.x >> 6; e < l.entries; e += kWaves) {
        double mine = 0.0;
        l.template each<1>(e * l.per_entry, std::min<int64_t>((e + 1) * l.per_entry, l.tiles), 1, [&](const float(&x)[E], int64_t i, int64_t) {
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const uint32_t key = key_of(x[k]);
                if (key > kNone && place_of(key, (uint32_t)(i + k)) >= last) {
                    const double w = mass.any(x[k]);
                    mine += w >= mass.least ? w : 0.0;
                }
            }
        });
        const u64 w = wave_sum(mine);
        if ((threadIdx.x & 63) == 0) sh.entry[e] = w;
    }
    __syncthreads();
    return last;
}

// The last kept place from the list, whose kept ones go to their entries; 0: the list does not tell. all:
// the mass before top_k's last step; kept: of that, what lies before the list.
template <typename T>
__device__ __forceinline__ u64 resolve(const Logits<T> &l, const Masses &mass, const Settings &s, const Steps &st, const Plan &pl, u64 all, u64 kept,
                       Shared &sh) {
    const int tid = threadIdx.x, n = (int)sh.count;
    if (n > kList || n == 0) return 0;
    sort_list(sh.list, n);
    // two of the list a thread
    u64 place[2], m[2], whole;
    bool in_p[2], in_k[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = 2 * tid + h;
        place[h] = i < n ? sh.list[i] : 0;
        const float x = logit_of((uint32_t)(place[h] >> 32));
        const int bin = i < n ? (int)fminf(st.of(x), (float)(kBins - 1)) : -1;
        m[h] = i < n ? (u64)mass(x) : 0;
        in_k[h] = bin == pl.end_k;
        in_p[h] = bin >= pl.p_from && bin <= pl.p_to;
    }
    if (pl.end_k < kBins) {
        const u64 mine = in_k[0] + in_k[1];
        u64 rank = pl.before_k + block_scan(mine, sh.part, whole) - mine;  // of the first of the two in that step
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (in_k[h] && rank++ >= (u64)s.top_k) {
                place[h] = m[h] = 0;
                in_p[h] = false;
            }
    }
    if (s.by_p) {
        if (pl.whole) {
            block_scan(m[0] + m[1], sh.part, all);
        } else if (pl.end_k < kBins) {  // and what top_k keeps of that step
            block_scan((in_k[0] ? m[0] : 0) + (in_k[1] ? m[1] : 0), sh.part, whole);
            all += whole;
        }
        const double part = (double)s.top_p * (double)all;
        const u64 x0 = in_p[0] ? m[0] : 0, x1 = in_p[1] ? m[1] : 0;
        const u64 upto = kept + block_scan(x0 + x1, sh.part, whole);
        // the end lies in these steps: not before them, and not after, unless nothing is left there
        if (!((double)kept < part || pl.p_from == 0) || ((double)(kept + whole) < part && pl.p_to < std::min(pl.end_k, kBins - 1))) return 0;
        const bool first = tid == 0 && pl.p_from == 0;  // it always stays
        if (!(in_p[0] && ((double)(upto - x0 - x1) < part || first))) place[0] = 0;
        if (!(in_p[1] && (double)(upto - x1) < part)) place[1] = 0;
    }
    u64 least = ~0ull;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (place[h]) {
            least = std::min(least, place[h]);
            if ((double)m[h] >= mass.least) atomicAdd(&sh.entry[(index_of(place[h]) + l.skip) / Logits<T>::kTile / l.per_entry], m[h]);
        }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) least = std::min(least, (u64)__shfl_xor((long long)least, d));
    __syncthreads();
    if ((tid & 63) == 0) sh.part[tid >> 6] = least;
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) least = std::min(least, sh.part[w]);
    return least == ~0ull ? 0 : least;
}

// 4. The entry in which the sum exceeds u times all, and the token in it.
template <typename T>
__device__ __forceinline__ void draw(const Logits<T> &l, const Masses &mass, const Settings &s, u64 last, Shared &sh, int64_t *token, float *logprob) {
    constexpr int E = Logits<T>::E;
    const int tid = threadIdx.x, lane = tid & 63;
    __syncthreads();
    const u64 m0 = 2 * tid < l.entries ? sh.entry[2 * tid] : 0, m1 = 2 * tid + 1 < l.entries ? sh.entry[2 * tid + 1] : 0;
    if (tid == 0) sh.few[0] = kEntries;
    u64 total;
    const u64 upto = block_scan(m0 + m1, sh.part, total);
    const double aim = (double)s.u * (double)total;
    const auto over = [&](u64 m, u64 sum) { return m > 0 && ((double)sum > aim || sum == total); };
    if (over(m1, upto)) atomicMin(&sh.few[0], (uint32_t)(2 * tid + 1));
    if (over(m0, upto - m1)) atomicMin(&sh.few[0], (uint32_t)(2 * tid));
    __syncthreads();
    const int e = (int)sh.few[0];
    if (e / 2 != tid) {  // that thread's wave goes on
        if (e / 128 != tid / 64) return;
    }
    u64 sum = lane_of(e & 1 ? upto - m1 : upto - m1 - m0, __builtin_amdgcn_readfirstlane(e / 2 % 64));
    for (int64_t t = e * l.per_entry; t < std::min<int64_t>((e + 1) * l.per_entry, l.tiles); ++t) {
        const int64_t i = l.first(t, lane);
        float x[E];
        l.load(i, x);
        u64 m[E], mine = 0;
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const uint32_t key = key_of(x[k]);
            const double w = key > kNone && place_of(key, (uint32_t)(i + k)) >= last ? mass.any(x[k]) : 0.0;
            m[k] = w >= mass.least ? (u64)w : 0;
            mine += m[k];
        }
        const u64 upto_lane = sum + wave_scan(mine);
        const uint64_t hit = __ballot(over(mine, upto_lane));
        if (hit) {
            if (lane == __ffsll((long long)hit) - 1) {
                u64 run = upto_lane - mine;
                bool found = false;
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    run += m[k];
                    if (!found && over(m[k], run)) {
                        found = true;
                        *token = i + k;
                        if (logprob) *logprob = (float)log((double)m[k] / (double)total);
                    }
                }
            }
            return;
        }
        sum = lane_of(upto_lane, 63);
    }
}

__device__ __forceinline__ bool settled(const Ends &e, const Settings &s, int64_t *token, float *logprob) {
    const bool lost = is_lost(e, s);
    if (!lost && s.temperature > 0.0f) return false;
    if (threadIdx.x == 0) {
        *token = lost ? (int64_t)-1 : (int64_t)e.where;
        if (logprob) *logprob = lost ? __uint_as_float(0x7fc00000u) : 0.0f;
    }
    return true;
}
__device__ __forceinline__ Masses masses_of(const Ends &e, const Settings &s, int shift) {
    return Masses{(double)e.high, 1.4426950408889634 / (double)s.temperature,
                  s.min_p > 0.0f ? fmin((double)s.min_p, 1.0) * (double)(1ull << shift) : 0.0, shift};
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_sample(SampleArgs p, int shift) {
    __shared__ Shared sh;
    const int64_t r = blockIdx.x;
    const Logits<T> l((const T *)p.logits + r * p.vocab, p.vocab);
    const Settings s(p, r);
    float *const logprob = p.logprob ? p.logprob + r : nullptr;
    if (s.by_k || s.by_p)
        for (int b = threadIdx.x; b < kBins; b += kThreads) sh.bins[b] = 0;
    if (threadIdx.x == 0) sh.count = 0;
    const Ends ends = find_ends(l, s.temperature == 0.0f, sh.few);
    if (settled(ends, s, p.tokens + r, logprob)) return;
    const Masses mass = masses_of(ends, s, shift);
    u64 last = 0;  // the last place that is kept
    // No steps hold the end: there is a +infinity, or float32 does not hold the distance of the smallest.
    bool lost = !(ends.high - ends.low < kInfinity);
    if (!lost) {
        const Steps st(ends, s);
        Plan pl{kBins, kBins, kBins, 0, false};
        if (s.by_k || s.by_p) {
            count_steps(l, st, sh.bins);
            __syncthreads();
            pl = plan_ends(sh, s, st);
        }
        u64 all, kept;
        weigh(l, s, st, pl, mass, sh.entry, sh.list, &sh.count, all, kept);
        if (s.by_p) {
            block_scan(all, sh.part, all);
            block_scan(kept, sh.part, kept);
        }
        __syncthreads();
        if (pl.end_k < kBins || s.by_p) {
            last = resolve(l, mass, s, st, pl, all, kept, sh);
            if (last == 0) {
                // of copies: what a call takes by address lies in memory, on the fast way too
                const Logits<T> l1 = l;
                const Masses mass1 = mass;
                const Settings s1 = s;
                const Steps st1 = st;
                const Plan pl1 = pl;
                last = descend(l1, mass1, s1, &st1, pl1, all, kept, sh);
                lost = last == 0;
            }
        }
    }
    if (lost) {
        const Logits<T> l1 = l;
        const Masses mass1 = mass;
        const Settings s1 = s;
        last = descend(l1, mass1, s1, nullptr, Plan{}, 0, 0, sh);
    }
    draw(l, mass, s, last, sh, p.tokens + r, logprob);
}

}  // namespace

size_t sample_ws(int64_t, int64_t) { return 0; }
hipError_t launch_sample(const SampleArgs &a, int io, hipStream_t s) {
    int shift = 44;  // sums of a row stay below 2^62, those of a wave's entry below 2^53
    while (((int64_t)1 << (62 - shift)) < a.vocab) --shift;
    if (io) k_sample<__bf16><<<a.rows, kThreads, 0, s>>>(a, shift);
    else k_sample<float><<<a.rows, kThreads, 0, s>>>(a, shift);
    return hipGetLastError();
}

}  // namespace ssm
