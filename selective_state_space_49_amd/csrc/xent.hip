// xent.hip -- softmax cross entropy of a linear head over a vocabulary, without keeping the
// logits, and its gradients.
//
// Everything large is a matrix product on the matrix cores, C[n][m] = sum_k A(m, k) B(n, k)
// (k_product), where an operand's rows run along k, or (transposed) its rows are the k. What
// differs is the epilogue:
//   forward    A = weight, B = hidden: a wave's tile of logits leaves, per token, the
//              maximum and the sum of exponentials over its vocabulary rows; a small kernel
//              joins a token's pairs: M = max(m, m'), s e^(m-M) + s' e^(m'-M).
//   backward   for a piece of the vocabulary at a time: the same product again, with
//              G [token][vocab] = dlogits / w = exp(logit - lse) - onehot; then dweight rows =
//              G^T (w hidden), both transposed, and dhidden += w G weight, weight transposed.
// What bounds it is the matrix cores' power: 8192 tokens x 4096 x 32000 in bfloat16 take 1.72 ms
// forwards and 5.1 ms backwards, 1.25 PFLOP/s, with the cores 64 to 75 % busy and the clock at
// 1.5 to 1.75 of 2.4 GHz; with few tokens it is the weight's bytes (8 x 4096 x 32000: 0.29 ms for
// 1.05 GB), with little of both the launches (100 x 256 x 1000: 37 us for six).
// The matrix cores take 16 bits, here always bfloat16: its exponents are float32's, so that no value
// needs a scale, and none is lost beside a larger one. An operand is the sum of one to three
// parts, x = x1 + x2 + x3, each the rounded rest of the ones before (8, 16, 24 bits), and a
// product the sum of those partial products x_i y_j that the operands' bits reach, as one longer
// sum over k, the small ones first. In the gradients' products, a token's weight w stays out of
// G, whose values lie in [-1, 1]: dhidden takes it as a factor of its row.
//   float32: three parts of each operand and of G, six partial products; those left out are below
//   2^-23 of |x||y|. That is 200 TFLOP/s; the float32 matrix instruction's peak is 157. (Two float16
//   parts, scaled by the array's largest value, need three partial products, but lose what is
//   small beside that value: an entry of G below 2^-28 its relative precision, a token its
//   own beside one 10^6 times as large.)
//   bfloat16: its own bits. G is rounded to bfloat16, and w is a factor of dweight where all tokens
//   have one (a mean loss): 2.0e-3 of dweight, where its own rounding is 1.7e-3. (With w in G, the
//   large values w (p - 1) of all tokens round alike, 2.1e-3 by themselves.) Where tokens have
//   weights of their own, dweight takes them with hidden, as two parts, so that no weight is lost
//   beside a larger one (8192 x 4096 x 32000: 8.5 ms instead of 6.9).
//   G has a second part where there are few tokens (kFewTokens): an entry of it then carries a whole
//   row of a gradient, and its rounding, up to 2^-8, would be the row's (3.5e-3 of dweight for one
//   token; 1.7e-3 so), and where the weight's bytes, not the products, bound the call.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "ssm_device.h"
#include "ssm_train.h"

namespace ssm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
#define SSM_LDS __attribute__((address_space(3)))

constexpr int kBK = 64;        // k per stage
constexpr int kMostParts = 3;  // bfloat16 parts of a float32 operand
constexpr uint32_t kRsrcWord3 = 0x00027000;  // raw buffer, 32-bit data

// One operand, 16-byte aligned: rows of ld elements (a multiple of 64), its parts `plane` elements
// apart. Its rows run along k, all of ld there; or, transposed, row k holds the values of all
// m (or n), and `rows` of them are there to be read.
struct Operand {
    const uint16_t *p;
    int64_t ld, plane;
    int64_t rows;
};

// The tokens' targets and the weights of their losses, as the caller gave them.
struct Tokens {
    const int64_t *targets;
    int64_t ignore, V;
    const float *dloss, *dmean, *mean;
    // The vocabulary row; -1: ignored, -2: out of range.
    __device__ __forceinline__ int32_t target(int64_t t) const {
        const int64_t y = targets[t];
        return y == ignore ? -1 : y >= 0 && y < V ? (int32_t)y : -2;
    }
    // The weight that every token has without dloss.
    __device__ __forceinline__ float same() const { return dmean ? *dmean * mean[1] : 0.0f; }
    __device__ __forceinline__ float weight(int64_t t, float same) const {
        const int32_t y = target(t);
        return y == -1 ? 0.0f : y == -2 ? NAN : (dloss ? dloss[t] : 0.0f) + same;
    }
};

enum class Epi { Lse, Dlogits, Out };
enum class Factor { None, Same, Row };  // of Out: the tokens' one weight, the weight of token n

// Partial products: which parts of the operands the n of them take, two bits each.
struct Terms {
    int32_t n;
    uint32_t a, b;
};

struct ProductArgs {
    Operand a, b;
    int64_t M, N;           // of C
    int32_t steps;          // ceil(K / kBK)
    Terms terms;
    int32_t parts;          // Dlogits: of G
    int32_t tiles_m, tiles_n, splits;
    // Lse, Dlogits: m = vocabulary row - v0, n = token
    Tokens tokens;
    float2 *part;           // Lse: [tiles_m * waves][N]
    float *at;              // Lse: [N] logit of the target
    uint32_t *done;         // Lse: set to 0 for the launch that joins
    const float *lse;       // Dlogits: [N]
    int64_t v0;
    uint16_t *g;            // Dlogits: G [rows_g][ldg], its parts gplane apart; 0 outside of N x M
    int64_t ldg, rows_g, gplane;
    // Out: C [N][ldc] of float32 or bfloat16 at split * cstride
    void *c;
    int64_t ldc, cstride;
    bool c_bf16;
    float *sum;             // with `add`: C = sum + product
    bool add;
    Factor factor;
};

// The bfloat16 that holds the most of v, and what is left of it. A finite value that would round
// to infinity is cut off instead; of an infinity or a NaN nothing is left.
__device__ __forceinline__ uint16_t take_part(float &v) {
    uint32_t h = f32_to_bf16(v);
    float rest = v - bf16_to_f32(h);
    if ((h & 0x7f80u) == 0x7f80u) {
        const uint32_t u = __float_as_uint(v);
        const bool finite = (u & 0x7f800000u) != 0x7f800000u;
        h = finite ? u >> 16 : h;
        rest = finite ? v - bf16_to_f32(h) : 0.0f;
    }
    v = rest;
    return (uint16_t)h;
}

// Waves stand WM x WN over a BM x BN tile; each makes TM x TN blocks of 32 x 32 with
// v_mfma_f32_32x32x16. Operand tiles go from global memory straight to LDS, 16 bytes a lane, into
// one of D buffers.
template <int BM, int BN, int WM, int WN, int D>
struct Shape {
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int kWaves = WM * WN;
    static constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
    static constexpr int kStage = (BM + BN) * kBK * 2;  // bytes
    static constexpr int kRow = BM + 8;                 // staging of G: elements of a token's row
    static constexpr int kLds = std::max(D * kStage, BN * kRow * 2);
};

// One operand's way into LDS and into fragments: B of its m (or n), kBK of k a stage.
//   Along k: LDS rows of 128 bytes, one for each m; the 16-byte chunk c of row r lies at chunk
//   c ^ (r / 2 & 7), so the 16 rows that a group of lanes reads at one k fall on the 16 chunks of
//   LDS's 64 banks (two rows of 128 bytes fill them once).
//   Transposed: LDS rows of 2 B bytes, one for each k; chunk c of row r lies at c ^ 4 (r & 3). The
//   transposing read gives a group of 16 lanes 4 k of 16 m from 4 rows of 32 bytes, and two
//   groups together read all 256 bytes of the banks.
// Rows (of m, or of k in the last step) past the operand's end read its last one, columns past
// its width the last ones: those products are never used, or the other operand is 0 there.
template <int B, bool TR, int WAVES, int BLOCKS>
struct Feed {
    static constexpr int kLoads = B * kBK * 2 / (1024 * WAVES);  // of a wave in a stage
    static constexpr int kReads = TR ? 2 : 1;                    // for a fragment
    const char *base, *next;  // plane 0 and the next step's address, uniform
    int64_t stride;           // bytes of a step
    uint32_t off[kLoads], last[kLoads], frag[4];

    __device__ __forceinline__ Feed(const Operand &o, int64_t at, int64_t end, int steps, int lane, int wave, int block0) {
        if (TR) {
            constexpr int kLanes = B / 8;  // of a row
            const int64_t there = o.rows - (int64_t)(steps - 1) * kBK - 1;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int r = (j * WAVES + wave) * (64 / kLanes) + lane / kLanes;
                const int64_t c = min(at + ((lane % kLanes) ^ (r & 3) * 4) * 8, o.ld - 8);
                off[j] = (uint32_t)((r * o.ld + c) * 2);
                last[j] = (uint32_t)((min((int64_t)r, there) * o.ld + c) * 2);
            }
            base = (const char *)o.p;
            stride = o.ld * kBK * 2;
            const int i = lane & 15, r = i >> 2, low = (lane >> 4 & 1) * 2 + (i & 3) / 2;
#pragma unroll
            for (int k = 0; k < BLOCKS; ++k)
                frag[k] = ((lane >> 5) * 8 + r) * (B * 2) + (((block0 + k) ^ r) * 4 + low) * 16 + (i & 1) * 8;
        } else {
            static_assert(WAVES % 2 == 0, "a wave's 8 rows all start at an even or all at an odd multiple of 8");
            const uint32_t chunk = (uint32_t)((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7)) * 16u;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int64_t r = min((int64_t)((j * WAVES + wave) * 8 + (lane >> 3)), end - 1 - at);
                off[j] = (uint32_t)(r * o.ld * 2) + chunk;
            }
            base = (const char *)(o.p + at * o.ld);
            stride = kBK * 2;
            const int row = lane & 31, half = lane >> 5;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                frag[ks] = (uint32_t)(((2 * ks + half) ^ (row >> 1 & 7)) * 16 + row * 128) + block0 * 4096;
        }
    }
    __device__ __forceinline__ void enter(int64_t plane, int k) { next = base + plane * 2 + k * stride; }
    __device__ __forceinline__ void load(SSM_LDS char *to, bool final) {
        __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void *)next, 0, -1, kRsrcWord3);
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (SSM_LDS void *)(to + j * WAVES * 1024), 16,
                                                     TR && final ? last[j] : off[j], 0, 0, 0);
        next += stride;
    }
    // Block k's fragment of step ks: lane l holds row l % 32, 8 consecutive k of half l / 32.
    __device__ __forceinline__ bf16x8 read(const SSM_LDS char *at, int ks, int k) const {
        if constexpr (TR) {
            const SSM_LDS char *from = at + frag[k] + ks * 16 * B * 2;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SSM_LDS s16x4 *)from);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SSM_LDS s16x4 *)(from + 4 * B * 2));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            return *(const SSM_LDS bf16x8 *)(at + frag[ks] + k * 4096);
        }
    }
};

template <typename S, Epi E, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void epilogue(const ProductArgs &p, f32x16 (&acc)[S::TM][S::TN], SSM_LDS char *lds,
                                         int64_t m0, int64_t n0, int wm, int wn, int split);

template <int BM, int BN, int WM, int WN, int D, Epi E, bool TA, bool TB>
__device__ __forceinline__ void product_tile(const ProductArgs &p, SSM_LDS char *lds, int bid, int split) {
    using S = Shape<BM, BN, WM, WN, D>;
    static_assert((D & (D - 1)) == 0, "a step's buffer is its last bits");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;

    // Tiles of one XCD (blocks are dealt to the 8 of them in turn) are neighbours, in groups
    // of 8 tile rows, so that its L2 sees an operand row several times.
    const int nt = p.tiles_m * p.tiles_n, xcd = bid & 7, q = nt >> 3, rest = nt & 7;
    const int id = xcd * q + min(xcd, rest) + (bid >> 3);
    const int width = 8 * p.tiles_n, group = id / width, gm = min(p.tiles_m - group * 8, 8), in = id % width;
    const int64_t m0 = (int64_t)(group * 8 + in % gm) * BM, n0 = (int64_t)(in / gm) * BN;

    const int total = p.steps * p.terms.n;
    const int first = (int)((int64_t)total * split / p.splits), last = (int)((int64_t)total * (split + 1) / p.splits);

    typedef Feed<BM, TA, S::kWaves, S::TM> FeedA;
    typedef Feed<BN, TB, S::kWaves, S::TN> FeedB;
    FeedA fa(p.a, m0, p.M, p.steps, lane, wave, wm * S::TM);
    FeedB fb(p.b, n0, p.N, p.steps, lane, wave, wn * S::TN);
    // Stages are loaded in order: k is the next one's step within its partial product seg.
    int seg = first / p.steps, k = first - seg * p.steps;
    auto enter = [&]() {
        fa.enter((p.terms.a >> 2 * seg & 3) * p.a.plane, k);
        fb.enter((p.terms.b >> 2 * seg & 3) * p.b.plane, k);
    };
    auto buffer = [&](int kt) { return lds + (kt & (D - 1)) * S::kStage; };
    auto stage = [&](SSM_LDS char *to) {
        to += wave * 1024;
        ++k;
        fa.load(to, k == p.steps);
        fb.load(to + BM * kBK * 2, k == p.steps);
    };
    auto turn = [&]() {  // to the next partial product after its last step
        if (k < p.steps) return;
        k = 0;
        ++seg;
        enter();
    };

    f32x16 acc[S::TM][S::TN];
#pragma unroll
    for (int i = 0; i < S::TM; ++i)
#pragma unroll
        for (int j = 0; j < S::TN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    bf16x8 a[2][S::TM], b[2][S::TN];
    auto fetch = [&](int set, const SSM_LDS char *at, int ks) {
#pragma unroll
        for (int i = 0; i < S::TM; ++i) a[set][i] = fa.read(at, ks, i);
#pragma unroll
        for (int j = 0; j < S::TN; ++j) b[set][j] = fb.read(at + BM * kBK * 2, ks, j);
    };
    auto multiply = [&](int set) {
#pragma unroll
        for (int i = 0; i < S::TM; ++i)
#pragma unroll
            for (int j = 0; j < S::TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[set][i], b[set][j], acc[i][j], 0, 0, 0);
    };
    // All waves' loads into the next stage and reads of this one are done, but for the `newer`
    // youngest loads of each, which may still be on their way: loads complete in order.
    auto meet = [&](auto newer) {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0x0070 | (newer & 15) | (newer >> 4) << 14);  // vmcnt(newer) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
    };
    // One stage of k, from the meeting of all waves at its start to the next: every fragment is
    // read while the products of the one before it run, and the loads into the buffer that the
    // meeting has freed are issued behind the last products of the stage before.
    constexpr int kMul = S::TM * S::TN, kReads = S::TM * FeedA::kReads + S::TN * FeedB::kReads;
    constexpr int kPer = (kReads + kMul - 1) / kMul, kLoads = (FeedA::kLoads + FeedB::kLoads) / kMul;
    auto weave = [&](auto loads) {  // fragment reads (and the loads' share) between the products
#pragma unroll
        for (int j = 0; j < kMul; ++j) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if (j * kPer < kReads) __builtin_amdgcn_sched_group_barrier(0x100, kPer, 0);
            if (loads) __builtin_amdgcn_sched_group_barrier(0x020, kLoads, 0);
        }
    };
    constexpr int kStageLoads = FeedA::kLoads + FeedB::kLoads;
    // `begun`: the last products of the stage before are still to be made. `more`: another stage is
    // asked for. `ahead` of the stages after this one will have been. That the two buffers differ
    // has to be said: before a transposing read, the compiler waits for every load that may go to
    // the same place (8192 x 4096 x 32000: 7.25 ms with that wait, 6.81 without).
    auto step = [&](const SSM_LDS char *__restrict from, SSM_LDS char *__restrict to, auto begun, auto more, auto ahead) {
        fetch(0, from, 0);
        if (more) stage(to);
        if (begun) {
            multiply(1);
            weave(more);
            __builtin_amdgcn_sched_barrier(0);
        }
        fetch(1, from, 1);
        multiply(0);
        weave(std::false_type{});
        __builtin_amdgcn_sched_barrier(0);
        fetch(0, from, 2);
        multiply(1);
        weave(std::false_type{});
        __builtin_amdgcn_sched_barrier(0);
        fetch(1, from, 3);
        multiply(0);
        weave(std::false_type{});
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (ahead > 0) meet(std::integral_constant<int, (ahead - 1) * kStageLoads>{});
    };
    if (first < last) {
        typedef std::true_type yes;
        typedef std::false_type no;
        const int count = min(D, last - first);  // stages on their way at the start
        enter();
        for (int i = 0; i < count; ++i) {
            if (i) turn();
            stage(buffer(first + i));
        }
        // fn(left) for left = n .. 1
        auto each = [&](int n, auto fn) {
            if constexpr (D > 2) {
                if (n >= 4) fn(std::integral_constant<int, 4>{});
                if (n >= 3) fn(std::integral_constant<int, 3>{});
            }
            if (n >= 2) fn(std::integral_constant<int, 2>{});
            if (n >= 1) fn(std::integral_constant<int, 1>{});
        };
        int kt = first;
        auto next = [&](auto begun, auto more, auto ahead) {
            step(buffer(kt), buffer(kt + D - 1), begun, more, ahead);
            ++kt;
        };
        each(count, [&](auto left) {
            if (left != count) return;
            meet(std::integral_constant<int, (left - 1) * kStageLoads>{});
            next(no{}, no{}, std::integral_constant<int, left - 1>{});
        });
        while (kt + D - 1 < last) {
            turn();
            const int until = kt + min(last - D + 1 - kt, p.steps - k);
            while (kt < until) next(yes{}, yes{}, std::integral_constant<int, D - 1>{});
        }
        each(last - kt, [&](auto left) { next(yes{}, no{}, std::integral_constant<int, left - 1>{}); });
        multiply(1);
        meet(std::integral_constant<int, 0>{});  // the epilogue may use the LDS
    }
    epilogue<S, E, BM, BN, WM, WN>(p, acc, lds, m0, n0, wm, wn, split);
}

template <int BM, int BN, int WM, int WN, int D, Epi E, bool TA, bool TB>
__global__ void __launch_bounds__(64 * WM * WN, 1) k_product(ProductArgs p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host has no buffer descriptors
    __shared__ __attribute__((aligned(1024))) char lds[Shape<BM, BN, WM, WN, D>::kLds];
    product_tile<BM, BN, WM, WN, D, E, TA, TB>(p, (SSM_LDS char *)lds, blockIdx.x, blockIdx.y);
#endif
}

// Both gradients of a piece by small tiles in one launch: alone, each of them leaves compute units
// idle in its last round (100 x 256 x 1000: 44 us a training step in two launches, 37 in one).
template <int D>
__global__ void __launch_bounds__(256, 1) k_gradients(ProductArgs w, ProductArgs h) {
#ifdef __HIP_DEVICE_COMPILE__
    __shared__ __attribute__((aligned(1024))) char lds[Shape<128, 128, 2, 2, D>::kLds];
    const int nw = w.tiles_m * w.tiles_n, nh = h.tiles_m * h.tiles_n, id = blockIdx.x, at = id - nw * w.splits;
    if (at < 0) product_tile<128, 128, 2, 2, D, Epi::Out, true, true>(w, (SSM_LDS char *)lds, id % nw, id / nw);
    else product_tile<128, 128, 2, 2, D, Epi::Out, true, false>(h, (SSM_LDS char *)lds, at % nh, at / nh);
#endif
}

// A block's element e of lane l is row m = 8 (e / 4) + 4 (l / 32) + e % 4, column n = l % 32.
template <typename S, Epi E, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void epilogue(const ProductArgs &p, f32x16 (&acc)[S::TM][S::TN], SSM_LDS char *lds,
                                         int64_t m0, int64_t n0, int wm, int wn, int split) {
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int64_t mw = m0 + wm * S::TM * 32 + 4 * half;  // the lane's first row
    const int64_t nw = n0 + wn * S::TN * 32 + (lane & 31);
    if constexpr (E == Epi::Lse) {
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.done = 0;
        const int64_t slot = (m0 / BM) * WM + wm;
#pragma unroll
        for (int j = 0; j < S::TN; ++j) {
            const int64_t n = nw + j * 32;
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < S::TM; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float v = acc[i][j][e];
                    if (mw + i * 32 + 8 * (e / 4) + e % 4 < p.M) top = top > v || top != top ? top : v;
                }
            const float o = __shfl_xor(top, 32);
            top = top > o || top != top ? top : o;
            float s = 0.0f;
            // a maximum of -inf (no rows, or all of them) has no terms
            const float off = top == -INFINITY ? 0.0f : top * kLog2e;
#pragma unroll
            for (int i = 0; i < S::TM; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (mw + i * 32 + 8 * (e / 4) + e % 4 < p.M) s += e2(fmaf(acc[i][j][e], kLog2e, -off));
            s += __shfl_xor(s, 32);
            if (n >= p.N) continue;
            if (half == 0) p.part[slot * p.N + n] = make_float2(top, s);
            const int64_t t = p.tokens.targets[n] - p.v0 - mw;  // the lane's rows are t = 32 i + 8 (e / 4) + e % 4
            if (t >= 0 && t < S::TM * 32 && (t & 4) == 0) {
#pragma unroll
                for (int i = 0; i < S::TM; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (t == i * 32 + 8 * (e / 4) + e % 4) p.at[n] = acc[i][j][e];
            }
        }
    }
    if constexpr (E == Epi::Dlogits) {
        // Through LDS, a token's row of kRow elements, and out in whole rows. Each part starts from
        // the product again. The token's weight stays out of G (dhidden takes it as a factor,
        // dweight with hidden).
        auto make = [&](auto part) {
#pragma unroll
            for (int j = 0; j < S::TN; ++j) {
                const int64_t n = nw + j * 32;
                const bool in = n < p.N;
                const int32_t target = in ? p.tokens.target(n) : -1;
                const float lse = in ? p.lse[n] : 0.0f;
                const float scale = target == -2 ? NAN : 1.0f;  // out of range: loud
                const int t = (int)max((int64_t)-1, min((int64_t)S::TM * 32, target - p.v0 - mw));
                // an ignored token and the padding are exactly 0, whatever the logit
                const int rows = target == -1 ? 0 : (int)max((int64_t)0, min((int64_t)S::TM * 32, p.M - mw));
                SSM_LDS char *to = lds + (wn * S::TN * 32 + j * 32 + (lane & 31)) * (S::kRow * 2) +
                                   (wm * S::TM * 32 + 4 * half) * 2;
#pragma unroll
                for (int i = 0; i < S::TM; ++i)
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        const int at = i * 32 + 2 * e;
                        uint32_t v16[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float q = e2((acc[i][j][e + k] - lse) * kLog2e) - (t == at + k ? 1.0f : 0.0f);
                            float v = at + k < rows ? q * scale : 0.0f;
#pragma unroll
                            for (int before = 0; before < part; ++before) v -= bf16_to_f32(f32_to_bf16(v));
                            v16[k] = f32_to_bf16(v);
                        }
                        *(SSM_LDS u32x2 *)(to + at * 2) = u32x2{v16[0] | v16[1] << 16, v16[2] | v16[3] << 16};
                    }
            }
            __syncthreads();
            uint16_t *g = p.g + part * p.gplane;
            for (int c = threadIdx.x; c < BN * (BM / 8); c += S::kThreads) {  // 8 columns of a token
                const int n = c / (BM / 8), m = c % (BM / 8) * 8;
                if (n0 + n < p.rows_g && m0 + m < p.ldg)
                    *(u32x4 *)(g + (n0 + n) * p.ldg + m0 + m) = *(const SSM_LDS u32x4 *)(lds + n * (S::kRow * 2) + m * 2);
            }
            __syncthreads();
        };
        make(std::integral_constant<int, 0>{});
        if (p.parts > 1) make(std::integral_constant<int, 1>{});
        if (p.parts > 2) make(std::integral_constant<int, 2>{});
    }
    if constexpr (E == Epi::Out) {
        const float same = p.factor == Factor::None ? 1.0f : p.tokens.same();
        const size_t eb = p.c_bf16 ? 2 : 4;
        char *const c = (char *)p.c + (size_t)split * p.cstride * eb;
        // A wave turns 32 rows of C at a time in LDS and writes them along the rows: four elements
        // a lane where every row starts on four, else one: 99 us for 262 MB and 128 us for 142 MB.
        // (Writing each lane's own four, a row apart from the next lane's, took 112 us for the
        // 262 MB, and 201 us for the 142 MB element by element.)
        const bool wide = p.ldc % 4 == 0 && ((uintptr_t)c & (4 * eb - 1)) == 0;
        constexpr int kWide = S::TM * 32, kTurn = kWide + 4;
        SSM_LDS float *mine = (SSM_LDS float *)lds + (wn * WM + wm) * 32 * kTurn;
        static_assert(S::kWaves * 32 * kTurn * 4 <= S::kLds, "the turned rows fit");
#pragma unroll
        for (int j = 0; j < S::TN; ++j) {
            const int64_t first = n0 + (wn * S::TN + j) * 32, mb = m0 + wm * kWide;
            typedef float f32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
            for (int i = 0; i < S::TM; ++i)
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *(SSM_LDS f32x4 *)(mine + (lane & 31) * kTurn + 4 * half + i * 32 + 2 * e) =
                        f32x4{acc[i][j][e], acc[i][j][e + 1], acc[i][j][e + 2], acc[i][j][e + 3]};
            __syncthreads();
            if (wide) {
                constexpr int kLanes = kWide / 4, kRows = 64 / kLanes;
                const int64_t m = mb + lane % kLanes * 4;
#pragma unroll 4
                for (int r = lane / kLanes; r < 32; r += kRows) {
                    const int64_t n = first + r, at = n * p.ldc + m;
                    if (n >= p.N || m >= p.M) break;  // M = ldc: all four or none
                    const f32x4 from = *(const SSM_LDS f32x4 *)(mine + r * kTurn + lane % kLanes * 4);
                    const float row = p.factor == Factor::Row ? p.tokens.weight(n, same) : same;
                    float v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = from[k] * row;
                    if (p.add) {
                        const float4 s = *(const float4 *)(p.sum + at);
                        v[0] += s.x, v[1] += s.y, v[2] += s.z, v[3] += s.w;
                    }
                    if (p.c_bf16)
                        *(u32x2 *)(c + at * 2) = u32x2{f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16,
                                                       f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16};
                    else
                        *(float4 *)(c + at * 4) = make_float4(v[0], v[1], v[2], v[3]);
                }
            } else {
                const int last = (int)min((int64_t)32, p.N - first);
#pragma unroll 4
                for (int r = 0; r < last; ++r) {
                    const int64_t n = first + r;
                    const float row = p.factor == Factor::Row ? p.tokens.weight(n, same) : same;
#pragma unroll
                    for (int i = 0; i < kWide; i += 64) {
                        const int64_t m = mb + i + lane, at = n * p.ldc + m;
                        if (m >= p.M) continue;
                        float v = mine[r * kTurn + i + lane] * row;
                        if (p.add) v += p.sum[at];
                        if (p.c_bf16) ((bf16_bits *)c)[at] = f32_to_bf16(v);
                        else ((float *)c)[at] = v;
                    }
                }
            }
            __syncthreads();
        }
    }
}

// ---------------------------------------------------------------- operands
// What a row of an array is: a token may be ignored, and may then hold anything; in Used it is 0 in
// the copy, so that nothing of it reaches a sum; in Weighed the others are multiplied by their
// tokens' weights.
enum class Rows { All, Used, Weighed };

// An array to be copied. The arrays of a call share a launch: blocks first .. of its grid are this
// one's.
struct Array {
    const void *src;         // [rows][cols]
    int64_t rows, cols;
    Rows kind;
    uint16_t *dst;           // [parts][rows_out][ld], the parts `plane` apart
    int64_t rows_out, ld, plane;
    int parts;
    unsigned first, blocks;
};
struct Arrays {
    Array a[3];
    int n;
};

// dst[part][r][ld] for r < rows_out: the parts of src, and 0 past its columns and rows. 16 bytes of
// a row a thread; the loads may start at any element.
template <typename IO>
__global__ void __launch_bounds__(256) k_pack(Arrays arrays, Tokens tokens) {
    constexpr int N = 16 / sizeof(IO);
    typedef IO iov __attribute__((ext_vector_type(N), aligned(sizeof(IO))));
    int n = 0;
    while (n + 1 < arrays.n && blockIdx.x >= arrays.a[n + 1].first) ++n;
    const Array &a = arrays.a[n];
    const unsigned block = blockIdx.x - a.first;
    const IO *src = (const IO *)a.src;
    const int64_t rows = a.rows, cols = a.cols, across = a.ld / N, total = a.rows_out * across;
    const bool drop = a.kind != Rows::All, weigh = a.kind == Rows::Weighed;
    const float same = weigh ? tokens.same() : 0.0f;
    for (int64_t e = (int64_t)block * 256 + threadIdx.x; e < total; e += (int64_t)a.blocks * 256) {
        const int64_t r = e / across, c = (e - r * across) * N;
        const bool in = r < rows && c < cols && !(drop && tokens.target(r) == -1);
        iov from;
#pragma unroll
        for (int k = 0; k < N; ++k) from[k] = IO(0);
        if (in) {
            const IO *at = src + r * cols + c;
            if (c + N <= cols) {
                from = *(const iov *)at;
            } else {
#pragma unroll
                for (int k = 0; k < N; ++k)
                    if (c + k < cols) from[k] = at[k];
            }
        }
        uint16_t *to = a.dst + r * a.ld + c;
        typedef uint16_t u16xN __attribute__((ext_vector_type(N)));
        if constexpr (sizeof(IO) == 2)
            if (!weigh) {
                *(u16xN *)to = from;
                continue;
            }
        const float f = weigh && in ? tokens.weight(r, same) : 1.0f;
        float v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const IO x = from[k];
            v[k] = Io<IO>::ld(&x) * f;
        }
        for (int q = 0; q < a.parts; ++q) {
            u16xN h;
#pragma unroll
            for (int k = 0; k < N; ++k) h[k] = take_part(v[k]);
            *(u16xN *)(to + q * a.plane) = h;
        }
    }
}

// (m, s) += (m2, s2): sums of exponentials under their maxima.
__device__ __forceinline__ void join(float &m, float &s, float m2, float s2) {
    const float M = m > m2 || m != m ? m : m2;
    const float f = m == M ? 1.0f : e2((m - M) * kLog2e), g = m2 == M ? 1.0f : e2((m2 - M) * kLog2e);
    s = s * f + s2 * g;
    m = M;
}

// A block of 256 joins the n partial pairs of TX tokens, 256 / TX threads for each, and sums their
// losses. The block that ends last makes the means of the blocks' sums, in their order:
// mean[0] = mean loss over the tokens that are not ignored, mean[1] = 1 / their number.
struct Losses {
    double sum;
    int64_t n;
};
__device__ __forceinline__ void put(Losses *p, const Losses &v) {
    __hip_atomic_store(&p->sum, v.sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(&p->n, v.n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ Losses get(Losses *p) {
    return {__hip_atomic_load(&p->sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT),
            __hip_atomic_load(&p->n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)};
}
template <int TX>
__global__ void __launch_bounds__(256) k_xent_join(const float2 *part, int64_t n, const float *at, Tokens tokens, int64_t T,
                                                   float *loss, float *lse, Losses *sums, uint32_t *done, float *mean) {
    constexpr int TY = 256 / TX;
    __shared__ float2 sh[TY][TX];
    __shared__ Losses wave_sum[4];
    __shared__ bool is_last;
    const int x = threadIdx.x % TX, y = threadIdx.x / TX;
    const int64_t t = (int64_t)blockIdx.x * TX + x;
    float m = -INFINITY, s = 0.0f;
    if (t < T)
#pragma unroll 4
        for (int64_t j = y; j < n; j += TY) {
            const float2 q = part[j * T + t];
            join(m, s, q.x, q.y);
        }
    sh[y][x] = make_float2(m, s);
    for (int half = TY / 2; half > 0; half /= 2) {
        __syncthreads();
        if (y < half) {
            join(m, s, sh[y + half][x].x, sh[y + half][x].y);
            sh[y][x] = make_float2(m, s);
        }
    }
    Losses own{0.0, 0};
    if (y == 0 && t < T) {
        const float l = m + logf(s);
        const int32_t to = tokens.target(t);
        const float v = to == -1 ? 0.0f : to >= 0 ? l - at[t] : NAN;
        lse[t] = l;
        loss[t] = v;
        if (to != -1) own = {v, 1};
    }
    for (int o = TX / 2; o > 0; o >>= 1) {
        own.sum += __shfl_xor(own.sum, o);
        own.n += __shfl_xor(own.n, o);
    }
    if (threadIdx.x == 0) {
        put(sums + blockIdx.x, own);
        is_last = __hip_atomic_fetch_add(done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    }
    __syncthreads();
    if (!is_last) return;
    own = {0.0, 0};
#pragma unroll 4
    for (unsigned b = threadIdx.x; b < gridDim.x; b += 256) {
        const Losses q = get(sums + b);
        own.sum += q.sum;
        own.n += q.n;
    }
    for (int o = 32; o > 0; o >>= 1) {
        own.sum += __shfl_xor(own.sum, o);
        own.n += __shfl_xor(own.n, o);
    }
    if ((threadIdx.x & 63) == 0) wave_sum[threadIdx.x >> 6] = own;
    __syncthreads();
    if (threadIdx.x) return;
    for (int j = 1; j < 4; ++j) {
        own.sum += wave_sum[j].sum;
        own.n += wave_sum[j].n;
    }
    mean[0] = own.n ? (float)(own.sum / (double)own.n) : 0.0f;
    mean[1] = own.n ? (float)(1.0 / (double)own.n) : 0.0f;
}

// dst = (sum +) the n partial products in order; float32 or bfloat16. Two of them side by side.
struct JoinArgs {
    const float *part;
    int n;
    int64_t count;  // elements; 0: nothing to join
    const float *sum;
    void *dst;
    bool bf16;
};
struct JoinPair {
    JoinArgs j[2];
};
__global__ void __launch_bounds__(256) k_join_splits(JoinPair pair) {
    const JoinArgs &a = pair.j[blockIdx.y];
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= a.count) return;
    float v = a.sum ? a.sum[e] : 0.0f;
#pragma unroll 4
    for (int k = 0; k < a.n; ++k) v += a.part[k * a.count + e];
    if (a.bf16) ((bf16_bits *)a.dst)[e] = f32_to_bf16(v);
    else ((float *)a.dst)[e] = v;
}

template <typename IO>
__global__ void __launch_bounds__(256) k_zero(IO *p, int64_t n) {
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) p[e] = IO(0);
}

// ---------------------------------------------------------------- host
int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
unsigned blocks(int64_t n, int64_t per) { return (unsigned)((n + per - 1) / per); }

constexpr int kBig = 256, kSmall = 128;

// Tiles of 256 x 256 or 128 x 128 and a split of k, whichever takes less time on 256 compute
// units, in microseconds as measured: a step of k takes 1.72 with a large tile and 1.14 with two
// small ones, which share a compute unit (8192 x 8192 x 4096: 1250 against 950 TFLOP/s) but waste
// less at the edges and in the last round, or 0.9 with one alone; each round has its start and its
// end; the partial sums of a split go through memory and a launch that joins them (1000 x 1000 x
// 48000: 140 us in 8 parts of small tiles, 112 in 16 of large ones). A part has 2 steps at least.
struct Tiling {
    int tile, splits;
};
constexpr int64_t kCus = 256;
Tiling tiling(int64_t M, int64_t N, int64_t steps, bool may_split) {
    Tiling best{};
    double least = 0;
    for (const int tile : {kSmall, kBig}) {
        const int64_t n = (int64_t)blocks(M, tile) * blocks(N, tile);
        const int64_t most = !may_split ? 1 : std::min(std::min((tile == kBig ? 1 : 2) * kCus / n, steps / 2), (int64_t)128);
        for (int64_t s = 1; s <= std::max<int64_t>(most, 1); ++s) {
            const double k = (double)steps / (double)s;
            const int64_t rounds = (int64_t)blocks(n * s, kCus), pairs = rounds / 2;
            const double join = s == 1 ? 0.0 : 4.0 + 0.05 * (double)s + (double)s * (double)M * (double)N * 8.0 / 5e6;
            const double time = join + (tile == kBig ? (double)rounds * (8.0 + 1.72 * k)
                                                     : (double)pairs * (5.0 + 1.14 * k) + (double)(rounds % 2) * (5.0 + 0.9 * k));
            if (!best.tile || time < least) {
                best = {tile, (int)s};
                least = time;
            }
        }
    }
    return best;
}

template <Epi E, bool TA = false, bool TB = false>
hipError_t product(ProductArgs p, int tile, hipStream_t s) {
    p.tiles_m = (int32_t)blocks(p.M, tile);
    p.tiles_n = (int32_t)blocks(p.N, tile);
    const dim3 grid((unsigned)(p.tiles_m * p.tiles_n), (unsigned)p.splits);
    if (tile == kBig) k_product<256, 256, 2, 4, 2, E, TA, TB><<<grid, 512, 0, s>>>(p);
    else if ((int64_t)grid.x * grid.y <= kCus) k_product<128, 128, 2, 2, 4, E, TA, TB><<<grid, 256, 0, s>>>(p);
    else k_product<128, 128, 2, 2, 2, E, TA, TB><<<grid, 256, 0, s>>>(p);
    return hipGetLastError();
}

// A bump allocator over the workspace; with no base it only counts.
struct Arena {
    char *base;
    size_t used = 0;
    template <typename P>
    P *take(int64_t n) {
        P *p = base ? (P *)(base + used) : nullptr;
        used += round_up((size_t)n * sizeof(P), kTrainWsAlign);
        return p;
    }
};

// The partial products of operands of `a` and `b` parts: x_i y_j is left out where it is no larger
// than what the operands' own bits leave out. Small ones first.
Terms terms_of(int a, int b) {
    Terms t{};
    for (int sum = std::max(a, b) - 1; sum >= 0; --sum)
        for (int i = 0; i <= sum; ++i)
            if (i < a && sum - i < b) {
                t.a |= (uint32_t)i << 2 * t.n;
                t.b |= (uint32_t)(sum - i) << 2 * t.n;
                ++t.n;
            }
    return t;
}

// G in two parts up to here in bfloat16: one step of k for each part of dweight's sum. With more tokens
// the roundings of G's entries, each up to 2^-8, average out (2.0e-3 to 2.2e-3 of dweight from 100
// tokens on, where its own rounding is 1.7e-3), and a second part would double the products (256 x
// 4096 x 32000: 513 us instead of 426).
constexpr int64_t kFewTokens = 64;

// What a call lays out in its workspace.
struct Layout {
    int parts, parts_w, parts_g;  // of hidden and weight, of w hidden, of G
    Terms logits, to_w, to_h;    // of the products
    int64_t ldk, rows_t, piece;  // padded dim and tokens; vocabulary rows of a piece (V: all in one)
    Tiling lse, out_w, out_h;
    bool pack;                   // hidden and weight are copied: float32, or rows not in steps of 64
    uint16_t *hidden, *weight;   // the copies, of weight a piece's
    uint16_t *hidden_w, *g;      // for the gradients: (w) hidden, G
    uint32_t *done;
    Losses *losses;
    float *at, *sum, *split_w, *split_h;
    float2 *part;
    size_t bytes;
};

// G of a piece holds about 2^27 numbers of 16 bits, 256 MB: 8192 tokens take pieces of 16384 rows.
// dhidden's partial sum is read and written once for each piece, so that more of them cost more
// (2^26, 2^27 and 2^28 values: 7.32, 7.27 and 7.22 ms for 8192 x 4096 x 32000, 8.34, 8.05 and
// 8.05 ms for 2000 x 4096 x 128000), and larger ones would begin to be the whole array. A copy of
// weight, where there is one, is that of a piece too, of 512 MB at most.
constexpr int64_t kPieceValues = (int64_t)1 << 27, kCopyValues = (int64_t)1 << 28;

// Tokens of a block that joins: whole lines of the partial pairs and few blocks where there are
// many tokens, many threads for each where there are few.
int join_tokens(int64_t T) { return T >= 4096 ? 32 : T >= 256 ? 16 : 2; }

// pack: hidden and weight have to be copied; weighed: the tokens have weights of their own.
Layout lay_out(int64_t T, int64_t K, int64_t V, int io, bool bwd, bool pack, bool weighed, char *ws) {
    Layout l{};
    Arena a{ws};
    l.parts = io ? 1 : kMostParts;
    l.logits = terms_of(l.parts, l.parts);
    l.ldk = up(K, kBK);
    l.rows_t = up(T, kBK);
    l.pack = pack;
    const auto rows_of = [](int64_t most, int64_t numbers) { return std::max<int64_t>(1024, most / numbers / kBig * kBig); };
    l.piece = std::min(V, pack ? rows_of(kCopyValues, l.ldk * l.parts) : V);
    if (bwd) {
        l.parts_w = io ? (weighed ? 2 : 1) : kMostParts;
        l.parts_g = io ? (T <= kFewTokens ? 2 : 1) : kMostParts;
        l.piece = std::min(l.piece, rows_of(kPieceValues, l.rows_t * l.parts_g));
    }
    l.hidden = a.take<uint16_t>(pack ? T * l.ldk * l.parts : 0);
    l.weight = a.take<uint16_t>(pack ? l.piece * l.ldk * l.parts : 0);
    if (!bwd) {
        l.lse = tiling(V, T, l.ldk / kBK * l.logits.n, false);
        l.part = a.take<float2>((int64_t)blocks(V, l.lse.tile) * 2 * T);
        l.at = a.take<float>(T);
        l.losses = a.take<Losses>(blocks(T, join_tokens(T)));
        l.done = a.take<uint32_t>(1);
    } else {
        l.to_w = terms_of(l.parts_w, l.parts_g);
        l.to_h = terms_of(l.parts, l.parts_g);
        l.out_w = tiling(K, l.piece, l.rows_t / kBK * l.to_w.n, true);
        l.out_h = tiling(K, T, up(l.piece, kBK) / kBK * l.to_h.n, true);
        l.sum = a.take<float>(V > l.piece ? T * K : 0);
        l.hidden_w = a.take<uint16_t>(l.rows_t * l.ldk * l.parts_w);
        l.g = a.take<uint16_t>(l.rows_t * up(l.piece, kBK) * l.parts_g);
        l.split_w = a.take<float>(l.out_w.splits > 1 ? l.out_w.splits * l.piece * K : 0);
        l.split_h = a.take<float>(l.out_h.splits > 1 ? l.out_h.splits * T * K : 0);
    }
    l.bytes = a.used;
    return l;
}

// Copies are needed but of bfloat16 rows in steps of 64 from 16 bytes on.
bool packs(int64_t K, int io, const void *hidden, const void *weight) {
    return !io || K % kBK != 0 || ((uintptr_t)hidden | (uintptr_t)weight) % 16 != 0;
}

constexpr int64_t kMostBlocks = (int64_t)1 << 20;

// The arrays that a call copies, gathered and then launched together.
template <typename IO>
struct Copies {
    Arrays list{};
    static constexpr int kWide = 16 / sizeof(IO);  // elements of a load
    unsigned grid = 0;
    // src [rows][cols] to dst [parts][rows_out][ld]. Returns the copy as an operand.
    Operand add(const Layout &l, const void *src, int64_t rows, int64_t cols, uint16_t *dst, int64_t rows_out, int parts,
                Rows kind) {
        Array &a = list.a[list.n++];
        a.src = src;
        a.rows = rows;
        a.cols = cols;
        a.kind = kind;
        a.dst = dst;
        a.rows_out = rows_out;
        a.ld = l.ldk;
        a.plane = rows_out * l.ldk;
        a.parts = parts;
        a.first = grid;
        a.blocks = (unsigned)std::min<int64_t>((rows_out * l.ldk / kWide + 255) / 256, kMostBlocks);
        grid += a.blocks;
        return {dst, l.ldk, a.plane, rows_out};
    }
    hipError_t launch(const Tokens &tokens, hipStream_t s) {
        if (grid) k_pack<IO><<<dim3(grid), 256, 0, s>>>(list, tokens);
        list = {};
        grid = 0;
        return hipGetLastError();
    }
};

#define SSM_TRY(x)                                 \
    do {                                           \
        const hipError_t try_e = (x);              \
        if (try_e != hipSuccess) return try_e;     \
    } while (0)

// Rows v0 .. of weight as an operand, as they are or copied.
template <typename IO>
Operand weight_rows(const XentArgs &a, const Layout &l, int64_t v0, Copies<IO> &copies) {
    const int64_t nv = std::min(l.piece, a.V - v0);
    const IO *from = (const IO *)a.weight + v0 * a.K;
    if (l.pack) return copies.add(l, from, nv, a.K, l.weight, nv, l.parts, Rows::All);
    return {(const uint16_t *)from, l.ldk, 0, nv};
}

// The product of the logits but for its weight. `made`: a copy of hidden that is there already.
template <typename IO>
ProductArgs logits_product(const XentArgs &a, const Layout &l, const Tokens &tokens, const Operand *made, Copies<IO> &copies) {
    ProductArgs p{};
    p.tokens = tokens;
    if (made) p.b = *made;
    else if (l.pack) p.b = copies.add(l, a.hidden, a.T, a.K, l.hidden, a.T, l.parts, Rows::All);
    else p.b = {(const uint16_t *)a.hidden, l.ldk, 0, a.T};
    p.N = a.T;
    p.steps = (int32_t)(l.ldk / kBK);
    p.terms = l.logits;
    p.splits = 1;
    return p;
}

template <typename IO>
hipError_t xent_fwd(const XentArgs &a, int io, hipStream_t s) {
    if (a.T == 0) {
        k_zero<<<dim3(1), 256, 0, s>>>(a.mean, (int64_t)2);
        return hipGetLastError();
    }
    const Layout l = lay_out(a.T, a.K, a.V, io, false, packs(a.K, io, a.hidden, a.weight), false, (char *)a.ws);
    const Tokens tokens{a.targets, a.ignore, a.V, nullptr, nullptr, nullptr};
    Copies<IO> copies;
    ProductArgs p = logits_product<IO>(a, l, tokens, nullptr, copies);
    p.at = l.at;
    p.done = l.done;
    for (int64_t v0 = 0; v0 < a.V; v0 += l.piece) {  // a piece is whole tiles, or all there is
        p.a = weight_rows<IO>(a, l, v0, copies);
        p.M = p.a.rows;
        p.v0 = v0;
        p.part = l.part + v0 / l.lse.tile * 2 * a.T;
        SSM_TRY(copies.launch(tokens, s));
        SSM_TRY(product<Epi::Lse>(p, l.lse.tile, s));
    }
    const int64_t n = (int64_t)blocks(a.V, l.lse.tile) * 2;
    const int most = join_tokens(a.T);
    auto join = most == 32 ? k_xent_join<32> : most == 16 ? k_xent_join<16> : k_xent_join<2>;
    join<<<dim3(blocks(a.T, most)), 256, 0, s>>>(l.part, n, l.at, tokens, a.T, a.loss, a.lse, l.losses, l.done, a.mean);
    return hipGetLastError();
}

// One of the gradients' products: C [N][M] = (sum +) A B, through partial sums over k where it is
// split, which *join is to join.
ProductArgs gradient(ProductArgs p, Tiling t, float *split, void *dst, bool bf16, float *sum, bool add, JoinArgs *join) {
    p.tiles_m = (int32_t)blocks(p.M, t.tile);
    p.tiles_n = (int32_t)blocks(p.N, t.tile);
    p.splits = t.splits;
    p.ldc = p.M;
    p.sum = sum;
    p.add = add && t.splits == 1;
    p.c = t.splits == 1 ? dst : split;
    p.c_bf16 = bf16 && t.splits == 1;
    p.cstride = p.M * p.N;
    *join = t.splits > 1 ? JoinArgs{split, t.splits, p.M * p.N, add ? sum : nullptr, dst, bf16} : JoinArgs{};
    return p;
}

// dweight's product w and dhidden's h, where they are wanted.
hipError_t gradients(const ProductArgs *w, int tile_w, const ProductArgs *h, int tile_h, hipStream_t s) {
    if (w && h && tile_w == kSmall && tile_h == kSmall) {
        const int64_t n = (int64_t)w->tiles_m * w->tiles_n * w->splits + (int64_t)h->tiles_m * h->tiles_n * h->splits;
        if (n <= kCus) k_gradients<4><<<dim3((unsigned)n), 256, 0, s>>>(*w, *h);
        else k_gradients<2><<<dim3((unsigned)n), 256, 0, s>>>(*w, *h);
        return hipGetLastError();
    }
    if (w) SSM_TRY((product<Epi::Out, true, true>(*w, tile_w, s)));
    if (h) SSM_TRY((product<Epi::Out, true, false>(*h, tile_h, s)));
    return hipSuccess;
}

template <typename IO>
hipError_t xent_bwd(const XentArgs &a, int io, hipStream_t s) {
    if (a.T == 0) {
        if (a.dweight) k_zero<IO><<<dim3((unsigned)std::min((a.V * a.K + 255) / 256, kMostBlocks)), 256, 0, s>>>((IO *)a.dweight, a.V * a.K);
        return hipGetLastError();
    }
    const bool weighed = a.dloss != nullptr;  // else one weight for all tokens: a factor at the end
    const Layout l = lay_out(a.T, a.K, a.V, io, true, packs(a.K, io, a.hidden, a.weight), weighed, (char *)a.ws);
    const Tokens tokens{a.targets, a.ignore, a.V, a.dloss, a.dmean, a.mean};
    Copies<IO> copies;
    Operand hidden_w{};
    if (a.dweight)
        hidden_w = copies.add(l, a.hidden, a.T, a.K, l.hidden_w, l.rows_t, l.parts_w, weighed ? Rows::Weighed : Rows::Used);
    ProductArgs logits = logits_product<IO>(a, l, tokens, a.dweight && !weighed ? &hidden_w : nullptr, copies);
    logits.lse = a.lse;
    logits.parts = l.parts_g;
    logits.g = l.g;
    logits.rows_g = l.rows_t;
    for (int64_t v0 = 0; v0 < a.V; v0 += l.piece) {
        const int64_t nv = std::min(l.piece, a.V - v0), ldg = up(nv, kBK);
        ProductArgs p = logits;
        p.a = weight_rows<IO>(a, l, v0, copies);
        SSM_TRY(copies.launch(tokens, s));
        p.M = nv;
        p.v0 = v0;
        p.ldg = ldg;
        p.gplane = l.rows_t * ldg;
        SSM_TRY(product<Epi::Dlogits>(p, tiling(nv, a.T, p.steps * p.terms.n, false).tile, s));
        const Operand g{l.g, ldg, p.gplane, l.rows_t};
        JoinPair join{};
        ProductArgs to_w{}, to_h{};
        if (a.dweight) {
            ProductArgs q{};
            q.tokens = tokens;
            q.a = hidden_w;
            q.b = g;
            q.M = a.K;
            q.N = nv;
            q.steps = (int32_t)(l.rows_t / kBK);
            q.terms = l.to_w;
            q.factor = weighed ? Factor::None : Factor::Same;
            to_w = gradient(q, l.out_w, l.split_w, (IO *)a.dweight + v0 * a.K, io, nullptr, false, &join.j[0]);
        }
        if (a.dhidden) {
            ProductArgs q{};
            q.tokens = tokens;
            q.a = p.a;
            q.b = g;
            q.factor = Factor::Row;
            q.M = a.K;
            q.N = a.T;
            q.steps = (int32_t)(ldg / kBK);
            q.terms = l.to_h;
            const bool end = v0 + nv == a.V;
            to_h = gradient(q, l.out_h, l.split_h, end ? a.dhidden : l.sum, end && io, l.sum, v0 > 0, &join.j[1]);
        }
        const ProductArgs *const pw = a.dweight ? &to_w : nullptr, *const ph = a.dhidden ? &to_h : nullptr;
        SSM_TRY(gradients(pw, l.out_w.tile, ph, l.out_h.tile, s));
        const int64_t most = std::max(join.j[0].count, join.j[1].count);
        if (most > 0) k_join_splits<<<dim3(blocks(most, 256), 2), 256, 0, s>>>(join);
    }
    return hipGetLastError();
}

}  // namespace

size_t xent_fwd_ws(int64_t T, int64_t K, int64_t V, int io, const void *hidden, const void *weight) {
    return T > 0 ? lay_out(T, K, V, io, false, packs(K, io, hidden, weight), false, nullptr).bytes : 0;
}
size_t xent_bwd_ws(int64_t T, int64_t K, int64_t V, int io, const void *hidden, const void *weight, bool weighed) {
    return T > 0 ? lay_out(T, K, V, io, true, packs(K, io, hidden, weight), weighed, nullptr).bytes : 0;
}
// For any pointers: the most of all, since the tilings, and with them the splits, go by the partial
// products and the pieces.
size_t xent_fwd_ws_any(int64_t T, int64_t K, int64_t V, int io) {
    const void *const odd = (const void *)1;
    return std::max(xent_fwd_ws(T, K, V, io, nullptr, nullptr), xent_fwd_ws(T, K, V, io, odd, odd));
}
size_t xent_bwd_ws_any(int64_t T, int64_t K, int64_t V, int io) {
    size_t most = 0;
    for (const void *p : {(const void *)nullptr, (const void *)1})
        for (const bool weighed : {false, true}) most = std::max(most, xent_bwd_ws(T, K, V, io, p, p, weighed));
    return most;
}
bool xent_fits(int64_t T, int64_t K, int64_t V, int io, bool bwd) {
    const int64_t most = 0xffffffffll;
    const auto tiles = [](int64_t M, int64_t N, int tile) { return (int64_t)blocks(M, tile) * blocks(N, tile); };
    const auto fits = [&](int64_t M, int64_t N, int tile) { return tiles(M, N, tile) * (tile == kBig ? 512 : 256) <= most; };
    if (T == 0) return true;
    if ((int64_t)blocks(T, join_tokens(T)) * 256 > most) return false;
    // most calls, whichever tiles they take
    if (tiles(V, T, kSmall) < 1 << 22 && tiles(K, std::max(T, V), kSmall) < 1 << 22) return true;
    if (!bwd) return fits(V, T, lay_out(T, K, V, io, false, true, false, nullptr).lse.tile);
    for (const int kind : {0, 1, 2, 3}) {
        const Layout l = lay_out(T, K, V, io, true, kind & 1, kind & 2, nullptr);
        const int64_t longest = std::min(V, l.piece), last = (V - 1) % l.piece + 1;
        for (const int64_t nv : {longest, last})
            if (!fits(nv, T, tiling(nv, T, l.ldk / kBK * l.logits.n, false).tile)) return false;
        if (!fits(K, longest, l.out_w.tile) || !fits(K, T, l.out_h.tile)) return false;
        // both gradients in one launch
        if (l.out_w.tile == kSmall && l.out_h.tile == kSmall &&
            (tiles(K, longest, kSmall) * l.out_w.splits + tiles(K, T, kSmall) * l.out_h.splits) * 256 > most)
            return false;
    }
    return true;
}
hipError_t launch_xent_fwd(const XentArgs &a, int io, hipStream_t s) {
    return io ? xent_fwd<bf16_bits>(a, io, s) : xent_fwd<float>(a, io, s);
}
hipError_t launch_xent_bwd(const XentArgs &a, int io, hipStream_t s) {
    return io ? xent_bwd<bf16_bits>(a, io, s) : xent_bwd<float>(a, io, s);
}

}  // namespace ssm
