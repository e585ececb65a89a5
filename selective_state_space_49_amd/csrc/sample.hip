// sample.hip -- the next token from a row of logits and one uniform number.
//
//     w_i = exp((logit_i - max) / temperature);   in the order of falling logits, equal ones by index:
//     the first top_k; of those the ones before which less than top_p of their mass lies; of those
//     the ones with w >= min_p;  then, by index, the first at which the sum of w exceeds u times all.
//
// Masses are whole numbers, w times 2^shift rounded (46 bits for a vocabulary of 65536): their sums do
// not depend on an order, so neither does the token. Of a row, equal logits have equal masses, and the
// kept ones are those above one logit and the first few equal to it.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ssm_layers.h"

namespace ssm {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64, kEntries = 2048;
constexpr uint32_t kNone = 0x007fffffu;  // the key of -infinity

typedef unsigned long long u64;

// Whole numbers in the order of the logits; -0 is 0, a NaN is above all.
__device__ __forceinline__ uint32_t key_of(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) { return __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key); }

struct Row {
    uint32_t top;   // the largest key
    double max, inv, one;  // one: the mass of weight 1
    __device__ __forceinline__ double weight(uint32_t key) const {
        if (key == top) return 1.0;
        if (top == 0xff800000u) return 0.0;  // beside an infinity
        return exp(((double)logit_of(key) - max) * inv);
    }
    __device__ __forceinline__ u64 mass(uint32_t key) const {
        return key > kNone ? (u64)__double2ull_rn(weight(key) * one) : 0;
    }
};

__device__ __forceinline__ u64 shfl_xor(u64 x, int d) { return (u64)__shfl_xor((long long)x, d); }

struct Shared {
    u64 mass[kEntries];
    uint32_t ties[kEntries];
    u64 part[kWaves];
    uint32_t count[kWaves];
};

// The number and the mass of all keys from `from` on.
template <typename T>
__device__ void measure(const T *logits, int64_t V, const Row &row, uint32_t from, Shared &sh, u64 &count, u64 &mass) {
    u64 m = 0;
    uint32_t c = 0;
    for (int64_t i = threadIdx.x; i < V; i += kThreads) {
        const uint32_t k = key_of((float)logits[i]);
        if (k >= from && k > kNone) {
            ++c;
            m += row.mass(k);
        }
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        m += shfl_xor(m, d);
        c += __shfl_xor(c, d);
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        sh.part[threadIdx.x >> 6] = m;
        sh.count[threadIdx.x >> 6] = c;
    }
    __syncthreads();
    count = mass = 0;
    for (int w = 0; w < kWaves; ++w) {
        mass += sh.part[w];
        count += sh.count[w];
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_sample(SampleArgs p, int shift) {
    __shared__ Shared sh;
    __shared__ uint32_t first[kWaves];
    const int64_t r = blockIdx.x, V = p.vocab;
    const T *const logits = (const T *)p.logits + r * V;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float temperature = p.temperature ? p.temperature[r] : p.temperature_all;
    const float top_p = p.top_p ? p.top_p[r] : p.top_p_all, min_p = p.min_p ? p.min_p[r] : p.min_p_all;
    const int64_t top_k = p.top_k ? p.top_k[r] : p.top_k_all;
    const float u = p.u[r];

    // The largest key and its lowest index.
    uint32_t top = 0;
    int64_t where = 0;
    for (int64_t i = threadIdx.x; i < V; i += kThreads) {
        const uint32_t k = key_of((float)logits[i]);
        if (k > top) {
            top = k;
            where = i;
        }
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t k = __shfl_xor(top, d), w = __shfl_xor((uint32_t)where, d);
        if (k > top || (k == top && w < (uint32_t)where)) {
            top = k;
            where = w;
        }
    }
    if (lane == 0) {
        sh.count[wave] = top;
        first[wave] = (uint32_t)where;
    }
    __syncthreads();
    top = 0;
    for (int w = 0; w < kWaves; ++w)
        if (sh.count[w] > top || (sh.count[w] == top && first[w] < (uint32_t)where)) {
            top = sh.count[w];
            where = first[w];
        }
    __syncthreads();
    const bool lost = top <= kNone || top == 0xffffffffu || !(temperature >= 0.0f) || u != u;
    if (lost || temperature == 0.0f) {
        if (threadIdx.x == 0) {
            p.tokens[r] = lost ? -1 : where;
            if (p.logprob) p.logprob[r] = lost ? __uint_as_float(0x7fc00000u) : 0.0f;
        }
        return;
    }
    Row row{top, (double)logit_of(top), 1.0 / (double)temperature, __longlong_as_double((u64)(1023 + shift) << 52)};

    // What is kept: keys above `edge`, and the first `ties` equal to it.
    uint32_t edge = kNone;
    u64 ties = 0, count, all;
    measure(logits, V, row, kNone + 1, sh, count, all);
    if (top_k > 0 && (u64)top_k < count) {
        uint32_t c = 0;
        for (int bit = 31; bit >= 0; --bit) {
            u64 n, m;
            measure(logits, V, row, c | 1u << bit, sh, n, m);
            if (n >= (u64)top_k) c |= 1u << bit;
        }
        u64 above, m;
        measure(logits, V, row, c + 1, sh, above, m);
        edge = c;
        ties = top_k - above;
        all = m + ties * row.mass(c);
    }
    if (top_p < 1.0f) {
        const double part = (double)top_p * (double)all;
        uint32_t c = 0;
        for (int bit = 31; bit >= 0; --bit) {
            u64 n, m;
            measure(logits, V, row, c | 1u << bit, sh, n, m);
            if (n > 0 && (double)m >= part) c |= 1u << bit;
        }
        if (c > row.top) c = row.top;
        if (c >= edge && c > kNone) {
            u64 n, m, n0, m0;
            measure(logits, V, row, c + 1, sh, n, m);
            measure(logits, V, row, c, sh, n0, m0);
            const u64 w = row.mass(c);
            u64 most = n0 - n;                  // equal keys, those that top_k keeps
            if (c == edge && ties < most) most = ties;
            // of them the ones before which less than `part` lies
            u64 keep = w ? (u64)fmin(fmax((part - (double)m) / (double)w, 0.0), (double)most) : most;
            while (keep > 0 && !((double)(m + (keep - 1) * w) < part)) --keep;
            while (keep < most && (double)(m + keep * w) < part) ++keep;
            if (n == 0 && keep == 0) keep = 1;
            edge = c;
            ties = keep;
        }
    }
    const double least = min_p > 0.0f ? fmin((double)min_p, 1.0) : 0.0;

    // The mass of what is kept, entry by entry in the order of the indices.
    const int64_t size = 64 * ((V + 64 * kEntries - 1) / (64 * (int64_t)kEntries));
    const int entries = (int)((V + size - 1) / size);
    for (int e = wave; e < entries; e += kWaves) {
        u64 m = 0;
        uint32_t c = 0;
        for (int64_t i = e * size + lane; i < std::min<int64_t>(V, (e + 1) * size); i += 64) {
            const uint32_t k = key_of((float)logits[i]);
            if (k > edge && row.weight(k) >= least) m += row.mass(k);
            c += k == edge;
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            m += shfl_xor(m, d);
            c += __shfl_xor(c, d);
        }
        if (lane == 0) {
            sh.mass[e] = m;
            sh.ties[e] = c;
        }
    }
    __syncthreads();
    if (wave != 0) return;
    const u64 tie = edge > kNone && row.weight(edge) >= least ? row.mass(edge) : 0;
    u64 total = 0, seen = 0;
    for (int e = 0; e < entries; ++e) {
        const u64 n = min((u64)sh.ties[e], ties - min(ties, seen));
        seen += sh.ties[e];
        total += sh.mass[e] + n * tie;
    }
    const double aim = (double)u * (double)total;
    u64 sum = 0;
    seen = 0;
    int64_t token = where;
    u64 got = row.mass(top);
    bool done = false;
    for (int e = 0; e < entries && !done; ++e) {
        const u64 n = min((u64)sh.ties[e], ties - min(ties, seen)), m = sh.mass[e] + n * tie;
        const bool last = sum + m == total;  // for a u of 1 and more
        if (m > 0 && ((double)(sum + m) > aim || last)) {
            for (int64_t i0 = e * size; i0 < std::min<int64_t>(V, (e + 1) * size) && !done; i0 += 64) {
                const int64_t i = i0 + lane;
                const uint32_t k = i < V ? key_of((float)logits[i]) : 0;
                const uint64_t equal = __ballot(k == edge && k > kNone);
                const u64 mine = seen + __popcll(equal & ((1ull << lane) - 1));
                u64 x = 0;
                if (k > edge && row.weight(k) >= least) x = row.mass(k);
                else if (k == edge && k > kNone && mine < ties) x = tie;
                u64 upto = x;
#pragma unroll
                for (int d = 1; d < 64; d *= 2) {
                    const u64 below = (u64)__shfl_up((long long)upto, d);
                    if (lane >= d) upto += below;
                }
                upto += sum;
                const uint64_t over = __ballot(x > 0 && ((double)upto > aim || upto == total));
                seen += __popcll(equal);
                if (over) {
                    const int at = __ffsll((long long)over) - 1;
                    token = i0 + at;
                    got = (u64)__shfl((long long)x, at);
                    done = true;
                } else {
                    sum = (u64)__shfl((long long)upto, 63);
                }
            }
        } else {
            sum += m;
            seen += sh.ties[e];
        }
    }
    if (lane == 0) {
        p.tokens[r] = token;
        if (p.logprob) p.logprob[r] = (float)log((double)got / (double)total);
    }
}

}  // namespace

size_t sample_ws(int64_t, int64_t) { return 0; }
hipError_t launch_sample(const SampleArgs &a, int io, hipStream_t s) {
    int shift = 46;  // sums of a vocabulary stay below 2^62
    while (((int64_t)1 << (62 - shift)) < a.vocab) --shift;
    if (io) k_sample<__bf16><<<a.rows, kThreads, 0, s>>>(a, shift);
    else k_sample<float><<<a.rows, kThreads, 0, s>>>(a, shift);
    return hipGetLastError();
}

}  // namespace ssm
