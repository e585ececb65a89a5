// gated.hip -- the gated linear recurrence: forward, backward and the single token.
//
//     k_t = c softplus(decay) sigmoid(r_t),  a_t = exp(-k_t),  beta_t = sqrt(1 - a_t^2)
//     h_t = a_t h_{t-1} + beta_t sigmoid(i_t) x_t,  y_t = h_t       (h_{t-1} = 0 at a reset)
// Backward, with g_t = dLoss/dh_t:
//     g_t = dy_t + a_{t+1} g_{t+1}
//     dx = g beta si,  di = g beta x si (1 - si)
//     kd = k dLoss/dk = g (a^2 (k / beta) si x - k a h_{t-1}),  dr = kd (1 - sr)
//     ddecay = sum kd sigmoid(decay) / softplus(decay),  dh0 = a_1 g_1
#include <algorithm>
#include <type_traits>

#include "ssm_device.h"
#include "ssm_train.h"

namespace ssm {
namespace {

// 1 - a^2 = -expm1(-2k) with relative precision: its series below 2k = 1/4 (the first term
// left out is below 6e-8 of the sum), 1 - a a above, where nothing cancels by more than a
// factor of 5.
__device__ __forceinline__ float one_minus_a2(float k, float a) {
    const float x = k + k;
    float p = fmaf(x, -1.0f / 720.0f, 1.0f / 120.0f);
    p = fmaf(x, p, -1.0f / 24.0f);
    p = fmaf(x, p, 1.0f / 6.0f);
    p = fmaf(x, p, -0.5f);
    p = fmaf(x, p, 1.0f);
    return x < 0.25f ? x * p : fmaf(-a, a, 1.0f);
}
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.0f + e2(-v * kLog2e)); }
// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|) in (0, 1], with log(1 + e) =
// 2 atanh(s), s = e / (2 + e) <= 1/3: relative precision also where e is small, as it is for
// slow decays. The first term of the series left out is below 2e-8 of the sum.
__device__ __forceinline__ float softplus(float v) {
    const float e = e2(-fabsf(v) * kLog2e), s = e * rcp(2.0f + e), q = s * s;
    float p = fmaf(q, 1.0f / 13.0f, 1.0f / 11.0f);
    p = fmaf(q, p, 1.0f / 9.0f);
    p = fmaf(q, p, 1.0f / 7.0f);
    p = fmaf(q, p, 1.0f / 5.0f);
    p = fmaf(q, p, 1.0f / 3.0f);
    p = fmaf(q, p, 1.0f);
    return fmaxf(v, 0.0f) + (s + s) * p;
}

struct Gate {
    float sr, si, k, a, beta;
};
// ck = c softplus(decay)
__device__ __forceinline__ Gate gate(float r, float i, float ck) {
    Gate g;
    g.sr = sigmoid(r);
    g.si = sigmoid(i);
    g.k = ck * g.sr;
    g.a = e2(-g.k * kLog2e);
    g.beta = __builtin_amdgcn_sqrtf(one_minus_a2(g.k, g.a));
    return g;
}

// ---------------------------------------------------------------- tiles
// One pass over the data. A thread block owns a tile of R W steps x 64 CPL channels: W waves,
// each with R consecutive steps, a lane with CPL channels, every value of the tile in
// registers. A wave reduces its steps to the pair (P, H): the state leaving them is
// P h_in + H, P = prod a. The waves' pairs meet in LDS, the tiles' pairs in global memory:
// a tile publishes its pair, takes the state that enters it from its predecessors' words,
// publishes the state that leaves it, and only then walks its steps with the true state. (What
// leaves a tile with a reset does not depend on what enters: it is published at once.) So each
// input is read once, where summary and rescan passes read it twice. What bounds it is the
// bytes: 8 a step and channel in bfloat16 forwards, 14 backwards. 262144 steps of 4096 channels
// take 1.61 ms (8.6 GB at 5.3 TB/s, where a large copy moves 4.9), and 2 x 4096 steps of 8192
// channels, forwards with the stored states and backwards, 0.316 ms (1.5 GB at 4.7 TB/s).
//
// A published word is 64 bits, {H, P | flags}, written and read whole by relaxed atomics at
// device scope: P lies in [0, 1], which leaves the two top bits of its float free for
// "valid" and "final state" (P not needed), and nothing else has to be ordered. The words
// start at 0. Blocks take their tiles from a counter in the order of the walk, so the tile
// that a block waits for belongs to a block that already runs: every wait ends.
constexpr uint64_t kValid = 1ull << 63, kFinal = 1ull << 62;

__device__ __forceinline__ uint64_t pack_word(float P, float H, uint64_t flags) {
    // a NaN decay has made H a NaN too (a tile with a reset has no P), and P's bits must stay clear
    // of the flags
    const uint32_t p = P == P ? __float_as_uint(P) : 0u;
    return flags | (uint64_t)p << 32 | __float_as_uint(H);
}
__device__ __forceinline__ float word_H(uint64_t w) { return __uint_as_float((uint32_t)w); }
__device__ __forceinline__ float word_P(uint64_t w) { return __uint_as_float((uint32_t)(w >> 32) & 0x3fffffffu); }

// c after steps with the pair (P, H). Where a reset is among the steps nothing of c passes, a NaN
// neither. That is a mark of its own, the same for all channels: a P of 0 is not one, since products
// underflow (and 0 c is NaN where c is), and a P that is NaN may have a reset behind it.
__device__ __forceinline__ float through(bool cut, float P, float H, float c) { return cut ? H : fmaf(P, c, H); }

// The state that enters a tile of the walk, for a lane's CPL channels; word j is the j-th tile
// at words + j stride, and `carry` comes in as the state before the first. Reads the words
// of kAhead predecessors until a final state is among them with every word after it there,
// and takes it forward: c <- P c + H, tile by tile. The value does not depend on which final
// state was met, since that one was made by the same steps; composing pairs on the way
// back would round differently from run to run. The words come from beyond the L2s, and what
// the waiting waves read of them takes bandwidth from the data: 262144 steps of 4096 channels
// take 1.96, 1.64, 1.60, 1.61, 1.77 and 2.39 ms with a kAhead of 1, 2, 3, 4, 8 and 12. Where
// few channels run side by side (far, below), the walk itself is what takes time, a round trip
// for every kAhead tiles.
template <int CPL, int kAhead>
__device__ __forceinline__ void look_back(const uint64_t *words, int64_t stride, int64_t tile, bool in,
                                          float (&carry)[CPL]) {
    for (;;) {
        uint64_t w[kAhead][CPL];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const int64_t j = tile - 1 - q;
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                w[q][c] = j >= 0 ? __hip_atomic_load(words + j * stride + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                                 : pack_word(0.0f, carry[c], kValid | kFinal);
        }
        bool all = true;
        float state[CPL];
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            bool have = false;
            state[c] = 0.0f;
#pragma unroll
            for (int q = kAhead - 1; q >= 0; --q) {
                const float P = word_P(w[q][c]), H = word_H(w[q][c]);
                const bool valid = w[q][c] & kValid, last = w[q][c] & kFinal;
                state[c] = last ? H : fmaf(P, state[c], H);
                have = valid && (last || have);
            }
            all = all && have;
        }
        if (__all(all || !in)) {
#pragma unroll
            for (int c = 0; c < CPL; ++c) carry[c] = state[c];
            return;
        }
        __builtin_amdgcn_s_sleep(1);
    }
}

// CPL neighbouring elements of a row, at a uniform address plus the lane's byte offset.
template <typename IO, int CPL> struct Lane;
template <typename IO> struct Lane<IO, 1> {
    typedef IO raw;
    static __device__ __forceinline__ raw ld(const char *p, uint32_t off) { return *(const IO *)(p + off); }
    static __device__ __forceinline__ void get(raw w, float (&v)[1]) { v[0] = Io<IO>::ld(&w); }
    static __device__ __forceinline__ void st(char *p, uint32_t off, const float (&v)[1]) { Io<IO>::st((IO *)(p + off), v[0]); }
};
template <> struct Lane<bf16_bits, 2> {
    typedef uint32_t raw;
    static __device__ __forceinline__ raw ld(const char *p, uint32_t off) { return *(const uint32_t *)(p + off); }
    static __device__ __forceinline__ void get(raw w, float (&v)[2]) {
        v[0] = __uint_as_float(w << 16);
        v[1] = __uint_as_float(w & 0xffff0000u);
    }
    static __device__ __forceinline__ void st(char *p, uint32_t off, const float (&v)[2]) {
        *(uint32_t *)(p + off) = f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16;
    }
};

// fn(std::true_type) for a wave whose R steps are all there, else fn(std::false_type): the
// common case compiles without a test per step.
template <int R, typename F>
__device__ __forceinline__ void by_rows(int rows, F fn) {
    if (rows == R) fn(std::true_type{});
    else if (rows > 0) fn(std::false_type{});
}

// Where a block works: the j-th tile of the walk of batch row b, channels from d0. `first`: the blocks
// of the call's launches before this one (the counter goes on from launch to launch by itself).
struct Place {
    int64_t j, b, d0;
};
__device__ __forceinline__ Place take_tile(const GatedArgs &p, uint32_t *ticket, uint32_t first, int cols, int *sh) {
    uint32_t id = first + blockIdx.x;
    if (ticket) {
        if (threadIdx.x == 0) *sh = (int)__hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        id = (uint32_t)__builtin_amdgcn_readfirstlane(*sh);
    }
    const uint32_t per = (uint32_t)(cols * p.batch), j = id / per, rest = id - j * per, b = rest / cols;
    return {(int64_t)j, (int64_t)b, (int64_t)(rest - b * cols)};
}

constexpr int kWaves = 8;
constexpr int kFwdRows = 16, kBwdRows = 8;  // steps of a wave
constexpr int kFwdTile = kFwdRows * kWaves, kBwdTile = kBwdRows * kWaves;
static_assert(kFwdTile % SSM_GATED_STATE_EVERY == 0 && SSM_GATED_STATE_EVERY % kFwdRows == 0 &&
                  kBwdTile == SSM_GATED_STATE_EVERY,
              "states are stored where waves of the forward and tiles of the backward begin");

// The workspace: a counter (256 bytes), then the words [batch][tiles][D], then the
// backward's sums.
__host__ __device__ inline int64_t tiles_of(int64_t L, int tile) { return (L + tile - 1) / tile; }
size_t words_bytes(int64_t batch, int64_t L, int64_t D, int tile) {
    const int64_t n = tiles_of(L, tile);
    return n > 1 ? kTrainWsAlign + round_up((size_t)(batch * n * D) * 8, kTrainWsAlign) : 0;
}

// 16 steps of a wave, 128 of a tile: at two bfloat16 channels a lane, 48 loads of 4 bytes a
// lane are in flight before the first gate, and the 2 x 32 floats of (a, b) still leave room
// for four waves a SIMD.
template <typename IO, int CPL, bool RESET, int FAR>
__global__ void __launch_bounds__(64 * kWaves, 4) k_gated_fwd(GatedArgs p, uint32_t first, uint32_t *ticket,
                                                              uint64_t *words) {
    constexpr int R = kFwdRows, CW = 64 * CPL;
    __shared__ float sP[kWaves][CW], sH[kWaves][CW], sC[CW];
    __shared__ int sid, sCut[kWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cols = (int)((p.D + CW - 1) / CW);
    const Place at = take_tile(p, ticket, first, cols, &sid);
    const int64_t d = at.d0 * CW + lane * CPL, n_tiles = tiles_of(p.L, kFwdTile);
    const int64_t dc = min(d, p.D - CPL);  // lanes past the last channel work on it and store nothing
    const bool in = d < p.D;
    const int64_t t0 = at.j * kFwdTile + wave * R, row0 = at.b * p.L + t0;
    const int rows = (int)max((int64_t)0, min((int64_t)R, p.L - t0));

    typedef Lane<IO, CPL> Ld;
    typename Ld::raw x[R], r[R], i[R];
    const int64_t base = (row0 * p.D + at.d0 * CW) * (int64_t)sizeof(IO), step = p.D * (int64_t)sizeof(IO);
    const uint32_t off = (uint32_t)(dc - at.d0 * CW) * (uint32_t)sizeof(IO);
    float a[R][CPL], b[R][CPL], P[CPL], H[CPL], ck[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        P[c] = 1.0f;
        H[c] = 0.0f;
    }
    uint64_t cut = 0;
    by_rows<R>(rows, [&](auto full) {
        int64_t o = base;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            r[k] = Ld::ld((const char *)p.r + o, off);
            i[k] = Ld::ld((const char *)p.i + o, off);
            x[k] = Ld::ld((const char *)p.x + o, off);
            if (full || k + 1 < rows) o += step;  // a step past the end reads the last one
        }
        if (RESET) cut = __ballot(lane < rows && p.reset[row0 + min(lane, rows - 1)] != 0);
#pragma unroll
        for (int c = 0; c < CPL; ++c) ck[c] = p.c * softplus(p.decay[dc + c]);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const bool there = full || k < rows, z = RESET && (cut >> k & 1);
            float xv[CPL], rv[CPL], iv[CPL];
            Ld::get(x[k], xv);
            Ld::get(r[k], rv);
            Ld::get(i[k], iv);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                const Gate g = gate(rv[c], iv[c], ck[c]);
                a[k][c] = there ? (z ? 0.0f : g.a) : 1.0f;
                b[k][c] = there ? g.beta * g.si * xv[c] : 0.0f;
                H[c] = z ? b[k][c] : fmaf(a[k][c], H[c], b[k][c]);
                P[c] *= a[k][c];
            }
        }
    });
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        sP[wave][lane * CPL + c] = P[c];
        sH[wave][lane * CPL + c] = H[c];
    }
    if (RESET && lane == 0) sCut[wave] = cut != 0;
    __syncthreads();
    const auto cuts = [&](int w) { return RESET && sCut[w]; };
    // the first wave: the tile's pair, the state that enters the tile, the state that leaves
    if (wave == 0) {
        float tP[CPL], tH[CPL], carry[CPL];
        uint64_t *mine = words ? words + (at.b * n_tiles + at.j) * p.D + d : nullptr;
        bool tcut = cuts(0);
        for (int w = 1; w < kWaves; ++w) tcut = tcut || cuts(w);
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            tP[c] = P[c];
            tH[c] = H[c];
            carry[c] = p.h0 ? p.h0[at.b * p.D + dc + c] : 0.0f;
            for (int w = 1; w < kWaves; ++w) {
                tH[c] = through(cuts(w), sP[w][lane * CPL + c], sH[w][lane * CPL + c], tH[c]);
                tP[c] *= sP[w][lane * CPL + c];
            }
            if (in && (at.j > 0 || tcut) && at.j + 1 < n_tiles)
                __hip_atomic_store(mine + c, tcut ? pack_word(0.0f, tH[c], kValid | kFinal) : pack_word(tP[c], tH[c], kValid),
                                   __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        if (at.j > 0) look_back<CPL, FAR ? FAR : 3>(words + at.b * n_tiles * p.D + dc, p.D, at.j, in, carry);
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            const float out = through(tcut, tP[c], tH[c], carry[c]);
            sC[lane * CPL + c] = carry[c];
            if (!in) continue;
            if (at.j + 1 == n_tiles) {
                if (p.h_final) p.h_final[at.b * p.D + d + c] = out;
            } else if (!tcut) {
                __hip_atomic_store(mine + c, pack_word(0.0f, out, kValid | kFinal), __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
            }
        }
    }
    __syncthreads();
    if (rows == 0) return;
    float h[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        h[c] = sC[lane * CPL + c];
        for (int w = 0; w < wave; ++w) h[c] = through(cuts(w), sP[w][lane * CPL + c], sH[w][lane * CPL + c], h[c]);
    }
    if (!in) return;
    if (p.states && t0 % SSM_GATED_STATE_EVERY == 0)
#pragma unroll
        for (int c = 0; c < CPL; ++c)
            p.states[(at.b * tiles_of(p.L, SSM_GATED_STATE_EVERY) + t0 / SSM_GATED_STATE_EVERY) * p.D + d + c] = h[c];
    by_rows<R>(rows, [&](auto full) {
        char *y = (char *)p.y + base;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (!full && k >= rows) continue;
#pragma unroll
            for (int c = 0; c < CPL; ++c) h[c] = RESET && (cut >> k & 1) ? b[k][c] : fmaf(a[k][c], h[c], b[k][c]);
            Ld::st(y, off, h);
            y += step;
        }
    });
}

// The same from the right: u_t = a_t g_t is what step t passes to its left, g_t = dy_t +
// u_{t+1}. The states come from the stored row that enters the tile, through the waves'
// forward pairs.
template <typename IO, int CPL, bool RESET, int FAR>
__global__ void __launch_bounds__(64 * kWaves, 4) k_gated_bwd(GatedArgs p, uint32_t first, uint32_t *ticket,
                                                              uint64_t *words, float *sums) {
    constexpr int R = kBwdRows, CW = 64 * CPL;
    __shared__ float sP[kWaves][CW], sH[kWaves][CW], sU[kWaves][CW], sC[CW];
    __shared__ int sid, sCut[kWaves];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int cols = (int)((p.D + CW - 1) / CW);
    const Place at = take_tile(p, ticket, first, cols, &sid);
    const int64_t d = at.d0 * CW + lane * CPL, n_tiles = tiles_of(p.L, kBwdTile);
    const int64_t dc = min(d, p.D - CPL), tile = n_tiles - 1 - at.j;
    const bool in = d < p.D;
    const int64_t t0 = tile * kBwdTile + wave * R, row0 = at.b * p.L + t0;
    const int rows = (int)max((int64_t)0, min((int64_t)R, p.L - t0));

    typedef Lane<IO, CPL> Ld;
    typename Ld::raw x[R], dy[R];
    const int64_t base = (row0 * p.D + at.d0 * CW) * (int64_t)sizeof(IO), step = p.D * (int64_t)sizeof(IO);
    const uint32_t off = (uint32_t)(dc - at.d0 * CW) * (uint32_t)sizeof(IO);
    float ck[CPL], h[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        ck[c] = p.c * softplus(p.decay[dc + c]);
        h[c] = p.states[(at.b * n_tiles + tile) * p.D + dc + c];
    }
    float sr[R][CPL], si[R][CPL], a[R][CPL], beta[R][CPL], P[CPL], H[CPL], U[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        P[c] = 1.0f;
        H[c] = U[c] = 0.0f;
    }
    uint64_t cut = 0;
    by_rows<R>(rows, [&](auto full) {
        typename Ld::raw r[R], i[R];
        int64_t o = base;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            r[k] = Ld::ld((const char *)p.r + o, off);
            i[k] = Ld::ld((const char *)p.i + o, off);
            x[k] = Ld::ld((const char *)p.x + o, off);
            dy[k] = Ld::ld((const char *)p.dy + o, off);
            if (full || k + 1 < rows) o += step;  // a step past the end reads the last one
        }
        if (RESET) cut = __ballot(lane < rows && p.reset[row0 + min(lane, rows - 1)] != 0);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const bool there = full || k < rows, z = RESET && (cut >> k & 1);
            float xv[CPL], rv[CPL], iv[CPL];
            Ld::get(x[k], xv);
            Ld::get(r[k], rv);
            Ld::get(i[k], iv);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                const Gate g = gate(rv[c], iv[c], ck[c]);
                sr[k][c] = g.sr;
                si[k][c] = g.si;
                a[k][c] = g.a;
                beta[k][c] = g.beta;
                if (!there) continue;
                const float b = g.beta * g.si * xv[c];
                H[c] = z ? b : fmaf(g.a, H[c], b);
                P[c] *= g.a;
            }
        }
#pragma unroll
        for (int k = R - 1; k >= 0; --k) {
            if (!full && k >= rows) continue;
            float gv[CPL];
            Ld::get(dy[k], gv);
#pragma unroll
            for (int c = 0; c < CPL; ++c) U[c] = RESET && (cut >> k & 1) ? 0.0f : a[k][c] * (gv[c] + U[c]);
        }
    });
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        sP[wave][lane * CPL + c] = P[c];
        sH[wave][lane * CPL + c] = H[c];
        sU[wave][lane * CPL + c] = U[c];
    }
    if (RESET && lane == 0) sCut[wave] = cut != 0;
    __syncthreads();
    const auto cuts = [&](int w) { return RESET && sCut[w]; };
    if (wave == 0) {
        float tP[CPL], tU[CPL], carry[CPL];
        uint64_t *mine = words ? words + (at.b * n_tiles + at.j) * p.D + d : nullptr;
        bool tcut = false;
        for (int w = 0; w < kWaves; ++w) tcut = tcut || cuts(w);
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            tP[c] = 1.0f;
            tU[c] = 0.0f;
            carry[c] = p.dh_final ? p.dh_final[at.b * p.D + dc + c] : 0.0f;
            for (int w = kWaves - 1; w >= 0; --w) {
                tU[c] = through(cuts(w), sP[w][lane * CPL + c], sU[w][lane * CPL + c], tU[c]);
                tP[c] *= sP[w][lane * CPL + c];
            }
            if (in && (at.j > 0 || tcut) && at.j + 1 < n_tiles)
                __hip_atomic_store(mine + c, tcut ? pack_word(0.0f, tU[c], kValid | kFinal) : pack_word(tP[c], tU[c], kValid),
                                   __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        if (at.j > 0) look_back<CPL, FAR ? FAR : 2>(words + at.b * n_tiles * p.D + dc, p.D, at.j, in, carry);
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            const float out = through(tcut, tP[c], tU[c], carry[c]);
            sC[lane * CPL + c] = carry[c];
            if (!in) continue;
            if (at.j + 1 == n_tiles) {
                if (p.dh0) p.dh0[at.b * p.D + d + c] = out;
            } else if (!tcut) {
                __hip_atomic_store(mine + c, pack_word(0.0f, out, kValid | kFinal), __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
            }
        }
    }
    __syncthreads();
    float u[CPL], sum[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        u[c] = sC[lane * CPL + c];
        sum[c] = 0.0f;
        for (int w = kWaves - 1; w > wave; --w) u[c] = through(cuts(w), sP[w][lane * CPL + c], sU[w][lane * CPL + c], u[c]);
        for (int w = 0; w < wave; ++w) h[c] = through(cuts(w), sP[w][lane * CPL + c], sH[w][lane * CPL + c], h[c]);
    }
    by_rows<R>(rows, [&](auto full) {
        float before[R][CPL];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (!full && k >= rows) continue;
            float xv[CPL];
            Ld::get(x[k], xv);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                before[k][c] = h[c];
                const float b = beta[k][c] * si[k][c] * xv[c];
                h[c] = RESET && (cut >> k & 1) ? b : fmaf(a[k][c], h[c], b);
            }
        }
        int64_t o = base + (int64_t)(rows - 1) * step;
#pragma unroll
        for (int k = R - 1; k >= 0; --k) {
            if (!full && k >= rows) continue;
            float xv[CPL], gv[CPL], dx[CPL], di[CPL], dr[CPL];
            Ld::get(x[k], xv);
            Ld::get(dy[k], gv);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                const bool z = RESET && (cut >> k & 1);
                const float g = gv[c] + u[c], s = si[k][c], ak = a[k][c], kk = ck[c] * sr[k][c];
                const float kb = beta[k][c] > 0.0f ? kk * rcp(beta[k][c]) : 0.0f;
                const float ah = z ? 0.0f : ak * before[k][c];
                const float kd = g * (ak * ak * kb * s * xv[c] - kk * ah);
                dx[c] = g * beta[k][c] * s;
                di[c] = dx[c] * xv[c] * (1.0f - s);
                dr[c] = kd * (1.0f - sr[k][c]);
                sum[c] += kd;
                u[c] = z ? 0.0f : ak * g;
            }
            if (in) {
                Ld::st((char *)p.dx + o, off, dx);
                Ld::st((char *)p.di + o, off, di);
                Ld::st((char *)p.dr + o, off, dr);
            }
            o -= step;
        }
    });
    // the tile's sum of k dLoss/dk: the waves' sums in order
    __syncthreads();
#pragma unroll
    for (int c = 0; c < CPL; ++c) sP[wave][lane * CPL + c] = sum[c];
    __syncthreads();
    if (wave == 0 && in)
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            float s = 0.0f;
            for (int w = 0; w < kWaves; ++w) s += sP[w][lane * CPL + c];
            sums[(at.b * n_tiles + tile) * p.D + d + c] = s;
        }
}

// ddecay[d] = sigmoid(decay) / softplus(decay) * sum over the n tiles' sums: 16 threads for a
// channel, in double, so that the order of thousands of them costs nothing. Channels from d0.
__global__ void __launch_bounds__(1024) k_gated_ddecay(const float *sums, const float *decay, float *out, int64_t n,
                                                       int64_t D, int64_t d0) {
    __shared__ double sh[16][64];
    const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
    const int64_t d = d0 + (int64_t)blockIdx.x * 64 + x;
    double s = 0.0;
    if (d < D)
        for (int64_t j = y; j < n; j += 16) s += (double)sums[j * D + d];
    sh[y][x] = s;
    __syncthreads();
    if (y || d >= D) return;
    for (int j = 1; j < 16; ++j) s += sh[j][x];
    const float sp = softplus(decay[d]);  // 0 where exp(decay) underflows: the ratio tends to 1
    out[d] = (float)s * (sp > 0.0f ? 1.0f / (1.0f + expf(-decay[d])) / sp : 1.0f);
}

__global__ void __launch_bounds__(256) k_clear(uint4 *p, int64_t n) {
    for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < n; j += (int64_t)gridDim.x * 256) p[j] = make_uint4(0, 0, 0, 0);
}

// dst = src (or 0), n floats.
__global__ void __launch_bounds__(256) k_fill(float *dst, const float *src, int64_t n) {
    for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < n; j += (int64_t)gridDim.x * 256)
        dst[j] = src ? src[j] : 0.0f;
}
hipError_t fill(float *dst, const float *src, int64_t n, hipStream_t s) {
    if (dst && n > 0) k_fill<<<dim3((unsigned)std::min<int64_t>((n + 255) / 256, 1 << 20)), 256, 0, s>>>(dst, src, n);
    return hipGetLastError();
}

// One token. A lane has N neighbouring channels of a layer, makes their decays once for S
// sequences, and has the loads of all of them in flight. What bounds it is the bytes: 16 a
// channel in bfloat16, half of them the state: 28 layers x 256 sequences x 8192 channels take
// 170 us, 0.94 GB at 5.5 TB/s.
template <typename IO, int N, int S>
__global__ void __launch_bounds__(256) k_gated_step(GatedStepArgs p) {
    const int64_t d = ((int64_t)blockIdx.x * 256 + threadIdx.x) * N;
    if (d >= p.D) return;
    const int64_t s0 = (int64_t)blockIdx.y * S, left = p.n_seq - s0;
    const int64_t e0 = ((int64_t)blockIdx.z * p.n_seq + s0) * p.D + d;
    typedef IO iov __attribute__((ext_vector_type(N)));
    typedef float f32v __attribute__((ext_vector_type(N)));
    iov r[S], i[S], x[S];
    f32v h[S];
#pragma unroll
    for (int k = 0; k < S; ++k) {
        const int64_t e = e0 + min((int64_t)k, left - 1) * p.D;
        r[k] = *(const iov *)((const IO *)p.r + e);
        i[k] = *(const iov *)((const IO *)p.i + e);
        x[k] = *(const iov *)((const IO *)p.x + e);
        h[k] = *(const f32v *)(p.h + e);
    }
    const f32v dec = *(const f32v *)(p.decay + blockIdx.z * p.D + d);
    float ck[N];
#pragma unroll
    for (int c = 0; c < N; ++c) ck[c] = p.c * softplus(dec[c]);
#pragma unroll
    for (int k = 0; k < S; ++k) {
        if (k >= left) break;
        iov y;
#pragma unroll
        for (int c = 0; c < N; ++c) {
            const IO rc = r[k][c], ic = i[k][c], xc = x[k][c];
            const Gate g = gate(Io<IO>::ld(&rc), Io<IO>::ld(&ic), ck[c]);
            h[k][c] = fmaf(g.a, h[k][c], g.beta * g.si * Io<IO>::ld(&xc));
            IO yc;
            Io<IO>::st(&yc, h[k][c]);
            y[c] = yc;
        }
        *(f32v *)(p.h + e0 + k * p.D) = h[k];
        *(iov *)((IO *)p.y + e0 + k * p.D) = y;
    }
}

}  // namespace

size_t gated_fwd_ws(int64_t batch, int64_t L, int64_t D) { return words_bytes(batch, L, D, kFwdTile); }
size_t gated_bwd_ws(int64_t batch, int64_t L, int64_t D) {
    return words_bytes(batch, L, D, kBwdTile) +
           round_up((size_t)(batch * tiles_of(L, kBwdTile) * D) * sizeof(float), kTrainWsAlign);
}

namespace {

// Two bfloat16 channels a lane where every row of every array starts on 4 bytes, else one: a
// wave then covers 128 bytes of a row instead of 256.
bool pairs(const GatedArgs &a, int io) {
    return io && a.D % 2 == 0 && (((uintptr_t)a.x | (uintptr_t)a.r | (uintptr_t)a.i | (uintptr_t)a.y | (uintptr_t)a.dy |
                                   (uintptr_t)a.dx | (uintptr_t)a.dr | (uintptr_t)a.di) & 3) == 0;
}

// The words read at a time, 0 for two or three, by the blocks of 64 channels side by side: 12 up to
// 8 of them, 8 up to 32, with one channel a lane. Training on 262144 steps of 256 channels takes
// 0.68 ms with 12, 0.79 with 8 and 2.21 as for many channels, on 16384 steps of 4096 channels 0.39
// with 8 and 0.35 as for many; the forward alone on 262144 steps of 512 channels 0.30, 0.31 and
// 0.61, of 1024 channels 0.56, 0.48 and 0.69, of 2048 channels 1.08, 0.92 and 0.90.
int far(const GatedArgs &a) {
    const int64_t side = a.batch * tiles_of(a.D, 64);
    return side <= 8 ? 12 : side <= 32 ? 8 : 0;
}

// launch(first, n) for as many blocks as a launch may have, until `blocks` of them are enqueued or one
// launch fails: a grid's work-items are fewer than 2^32.
template <typename F>
hipError_t in_launches(int64_t blocks, int threads, F launch) {
    const int64_t most = 0xffffffffll / threads;
    for (int64_t first = 0; first < blocks; first += most) {
        launch(first, (unsigned)std::min(most, blocks - first));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename IO, int CPL, int FAR>
hipError_t run_fwd(const GatedArgs &a, uint32_t *ticket, uint64_t *words, hipStream_t s) {
    return in_launches(tiles_of(a.D, 64 * CPL) * a.batch * tiles_of(a.L, kFwdTile), 64 * kWaves, [&](int64_t first, unsigned n) {
        if (a.reset) k_gated_fwd<IO, CPL, true, FAR><<<dim3(n), 64 * kWaves, 0, s>>>(a, (uint32_t)first, ticket, words);
        else k_gated_fwd<IO, CPL, false, FAR><<<dim3(n), 64 * kWaves, 0, s>>>(a, (uint32_t)first, ticket, words);
    });
}
template <typename IO, int CPL, int FAR>
hipError_t run_bwd(const GatedArgs &a, uint32_t *ticket, uint64_t *words, float *sums, hipStream_t s) {
    return in_launches(tiles_of(a.D, 64 * CPL) * a.batch * tiles_of(a.L, kBwdTile), 64 * kWaves, [&](int64_t first, unsigned n) {
        if (a.reset) k_gated_bwd<IO, CPL, true, FAR><<<dim3(n), 64 * kWaves, 0, s>>>(a, (uint32_t)first, ticket, words, sums);
        else k_gated_bwd<IO, CPL, false, FAR><<<dim3(n), 64 * kWaves, 0, s>>>(a, (uint32_t)first, ticket, words, sums);
    });
}

// The counter and the words of a call with several tiles, cleared; null for one tile.
hipError_t set_up(const GatedArgs &a, int tile, uint32_t **ticket, uint64_t **words, hipStream_t s) {
    const size_t n = words_bytes(a.batch, a.L, a.D, tile);
    *ticket = n ? (uint32_t *)a.ws : nullptr;
    *words = n ? (uint64_t *)((char *)a.ws + kTrainWsAlign) : nullptr;
    if (n)
        k_clear<<<dim3((unsigned)std::min<size_t>((n / 16 + 255) / 256, 1 << 20)), 256, 0, s>>>((uint4 *)a.ws, (int64_t)(n / 16));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gated_fwd(const GatedArgs &a, int io, hipStream_t s) {
    if (a.L == 0) return fill(a.h_final, a.h0, a.batch * a.D, s);
    uint32_t *ticket;
    uint64_t *words;
    const hipError_t e = set_up(a, kFwdTile, &ticket, &words, s);
    if (e != hipSuccess) return e;
    const int ahead = far(a);
    if (ahead == 12) return io ? run_fwd<bf16_bits, 1, 12>(a, ticket, words, s) : run_fwd<float, 1, 12>(a, ticket, words, s);
    if (ahead == 8) return io ? run_fwd<bf16_bits, 1, 8>(a, ticket, words, s) : run_fwd<float, 1, 8>(a, ticket, words, s);
    if (!io) return run_fwd<float, 1, 0>(a, ticket, words, s);
    return pairs(a, io) ? run_fwd<bf16_bits, 2, 0>(a, ticket, words, s) : run_fwd<bf16_bits, 1, 0>(a, ticket, words, s);
}

hipError_t launch_gated_bwd(const GatedArgs &a, int io, hipStream_t s) {
    if (a.L == 0 || a.batch == 0) {
        const hipError_t e = fill(a.dh0, a.dh_final, a.batch * a.D, s);
        return e != hipSuccess ? e : fill(a.ddecay, nullptr, a.D, s);
    }
    uint32_t *ticket;
    uint64_t *words;
    hipError_t e = set_up(a, kBwdTile, &ticket, &words, s);
    if (e != hipSuccess) return e;
    float *sums = (float *)((char *)a.ws + words_bytes(a.batch, a.L, a.D, kBwdTile));
    const int ahead = far(a);
    if (ahead == 12) e = io ? run_bwd<bf16_bits, 1, 12>(a, ticket, words, sums, s) : run_bwd<float, 1, 12>(a, ticket, words, sums, s);
    else if (ahead == 8) e = io ? run_bwd<bf16_bits, 1, 8>(a, ticket, words, sums, s) : run_bwd<float, 1, 8>(a, ticket, words, sums, s);
    else if (!io) e = run_bwd<float, 1, 0>(a, ticket, words, sums, s);
    else if (pairs(a, io)) e = run_bwd<bf16_bits, 2, 0>(a, ticket, words, sums, s);
    else e = run_bwd<bf16_bits, 1, 0>(a, ticket, words, sums, s);
    if (e != hipSuccess) return e;  // there are no sums then
    return in_launches(tiles_of(a.D, 64), 1024, [&](int64_t first, unsigned n) {
        k_gated_ddecay<<<dim3(n), 1024, 0, s>>>(sums, a.decay, a.ddecay, a.batch * tiles_of(a.L, kBwdTile), a.D, first * 64);
    });
}

namespace {
template <typename IO, int N>
void run_step(const GatedStepArgs &a, hipStream_t s) {
    // four sequences a lane where that still leaves 8 waves for each of 256 compute units
    const int64_t lanes = tiles_of(a.D, N), waves = a.n_layers * tiles_of(a.n_seq, 4) * tiles_of(lanes, 64);
    const int per = waves >= 256 * 8 ? 4 : 1;
    const dim3 grid((unsigned)tiles_of(lanes, 256), (unsigned)tiles_of(a.n_seq, per), (unsigned)a.n_layers);
    if (per == 4) k_gated_step<IO, N, 4><<<grid, 256, 0, s>>>(a);
    else k_gated_step<IO, N, 1><<<grid, 256, 0, s>>>(a);
}
}  // namespace

hipError_t launch_gated_step(const GatedStepArgs &a, int io, hipStream_t s) {
    // four channels a lane, 16 bytes of state at a time, where every row allows it
    const uintptr_t any = (uintptr_t)a.x | (uintptr_t)a.r | (uintptr_t)a.i | (uintptr_t)a.y;
    const bool wide = a.D % 4 == 0 && any % (io ? 8 : 16) == 0 && ((uintptr_t)a.h | (uintptr_t)a.decay) % 16 == 0;
    if (io) wide ? run_step<bf16_bits, 4>(a, s) : run_step<bf16_bits, 1>(a, s);
    else wide ? run_step<float, 4>(a, s) : run_step<float, 1>(a, s);
    return hipGetLastError();
}

}  // namespace ssm
