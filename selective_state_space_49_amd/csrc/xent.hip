// xent.hip -- softmax cross entropy of a linear head over a vocabulary, without keeping the
// logits, and its gradients.
//
// Everything large is a matrix product on the matrix cores, C[n][m] = sum_k A[m][k] B[n][k]
// with both operands' rows contiguous in k (k_product), and what differs is its epilogue:
//   forward    A = weight, B = hidden: a wave's tile of logits leaves, per token, the
//              maximum and the sum of exponentials over its vocabulary rows; a small kernel
//              joins a token's pairs: M = max(m, m'), s e^(m-M) + s' e^(m'-M).
//   backward   for a piece of the vocabulary at a time: the same product again, with
//              dlogits = w (exp(logit - lse) - onehot) written twice, as G [token][vocab] and
//              G^T; then dweight rows = G^T hidden (A = hidden^T, B = G^T) and
//              dhidden += G weight (A = weight^T, B = G).
// The matrix cores take 16 bits. Logits of bfloat16 operands are products of their own bits. In
// the gradients' products, a token's weight w stays out of G, whose values dlogits / w lie in
// [-1, 1]: dhidden takes it as a factor of its row.
//   bfloat16, every token of one weight (a mean loss): G, hidden^T and weight^T are bfloat16,
//   and w is a factor of dweight. (With w in G, the large values w (p - 1) of all tokens round
//   alike, and their error was 2.1e-3 where dweight's own rounding is 1.7e-3.)
//   otherwise: float16 planes, scaled by a power of two that brings the largest of the array to
//   2^14 .. 2^15, which leaves small values an absolute error of 2^-39 of the largest. dweight
//   takes w with hidden^T. One plane each for bfloat16 operands: 11 bits. Two for float32, x =
//   x1 + x2, the rounded value and the rounded rest, 22 bits, and a product is the sum of x1y1,
//   x1y2, x2y1 as a longer sum over k; x2y2 is below 2^-22 of x1y1. (Three bfloat16 parts need
//   six partial products for 24 bits.) float16 products take 9 % longer than bfloat16 ones
//   (489 against 450 us for 8192 x 8192 x 4096: the clock falls under their power).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "ssm_device.h"
#include "ssm_train.h"

namespace ssm {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
#define SSM_LDS __attribute__((address_space(3)))
#define SSM_GLB __attribute__((address_space(1)))

constexpr int kBK = 64;        // k per stage: rows of 128 bytes in LDS
constexpr int kParts = 2;      // float16 planes of a float32 operand
enum { kPeakW, kPeakH, kPeakWH, kPeakPiece };  // peaks of weight, hidden, w hidden, pieces of weight
constexpr int kPeak = 14;      // a scaled array's largest value is in 2^kPeak .. 2^(kPeak + 1)
constexpr uint32_t kRsrcWord3 = 0x00027000;  // raw buffer, 32-bit data

// One operand: rows of ld elements, contiguous in k, 16-byte aligned, ld a multiple of 64;
// planes `plane` elements apart.
struct Operand {
    const uint16_t *p;
    int64_t ld, plane;
    const uint32_t *peak;  // float16 planes: the largest value's bits; null: scaled by 2^kPeak
};

enum class Epi { Lse, Dlogits, Out };

struct ProductArgs {
    Operand a, b;
    int64_t M, N;           // rows of A and of B
    int32_t steps;          // ceil(K / kBK)
    int32_t terms;          // partial products: 1, or 3 of two planes each
    int32_t planes;         // Dlogits: float16 planes of G, 0: bfloat16
    int32_t tiles_m, tiles_n, splits;
    // Lse, Dlogits: m = vocabulary row - v0, n = token
    const int64_t *targets; // Lse: [N]
    const int32_t *target;  // Dlogits: [N]: vocabulary row, -1 ignored, -2 out of range
    float2 *part;           // Lse: [tiles_m * waves][N]
    float *at;              // Lse: [N] logit of the target
    const float *lse;       // Dlogits: [N]
    int64_t v0;
    uint16_t *g, *gt;       // Dlogits: G [N][ldg], G^T [M][ldgt], planes apart
    int64_t ldg, ldgt, gplane, gtplane;
    // Out: C [N][ldc] of float32 or bfloat16 at split * cstride
    void *c;
    int64_t ldc, cstride;
    bool c_bf16;
    float *sum;             // with `add`: C = sum + product
    bool add;
    const float *row;       // Out: a factor for each n, or null
    const float *scale;     // Out: a factor, or null
};

// The float16 that holds the most of v, and what is left of it.
__device__ __forceinline__ uint16_t take_f16(float &v) {
    const _Float16 h = (_Float16)v;
    v -= (float)h;
    return __builtin_bit_cast(uint16_t, h);
}

// The power of two that brings the value with these bits to 2^kPeak .. 2^(kPeak + 1), as an
// exponent.
__device__ __forceinline__ int scale_exp(uint32_t peak) {
    return peak == 0 ? 0 : min(kPeak + 127 - (int)(peak >> 23), 126);
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
template <bool F16>
__device__ __forceinline__ float unscale(const Operand &o) {
    return !F16 ? 1.0f : o.peak ? exp2i(-scale_exp(*o.peak)) : exp2i(-kPeak);
}

// Waves stand WM x WN over a BM x BN tile; each makes TM x TN blocks of 32 x 32 with
// v_mfma_f32_32x32x16_bf16. Operand tiles go from global memory straight to LDS, 16 bytes a
// lane, double buffered; the 16-byte chunk c of row r lies at chunk c ^ (r / 2 & 7), so the 16
// rows that a group of lanes reads at one k fall on the 16 chunks of LDS's 64 banks (two
// rows of 128 bytes fill them once).
template <int BM, int BN, int WM, int WN>
struct Shape {
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int kWaves = WM * WN;
    static constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
    static constexpr int kStage = (BM + BN) * kBK * 2;   // bytes
    static constexpr int kRow = BM + 2;                  // staging of G: elements of a token's row
    static constexpr int kLds = std::max(2 * kStage, BN * kRow * 2);
    static constexpr int kLoadsA = BM * kBK * 2 / (1024 * kWaves), kLoadsB = BN * kBK * 2 / (1024 * kWaves);
};

template <typename S, Epi E, bool F16, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void epilogue(const ProductArgs &p, f32x16 (&acc)[S::TM][S::TN], SSM_LDS char *lds,
                                         int64_t m0, int64_t n0, int wm, int wn, int split);

template <int BM, int BN, int WM, int WN, Epi E, bool F16>
__device__ __forceinline__ void product_tile(const ProductArgs &p, SSM_LDS char *lds) {
    using S = Shape<BM, BN, WM, WN>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;

    // Tiles of one XCD (blocks are dealt to the 8 of them in turn) are neighbours, in groups
    // of 8 tile rows, so that its L2 sees an operand row several times.
    const int nt = p.tiles_m * p.tiles_n, bid = blockIdx.x, xcd = bid & 7, q = nt >> 3, rest = nt & 7;
    const int id = xcd * q + min(xcd, rest) + (bid >> 3);
    const int width = 8 * p.tiles_n, group = id / width, gm = min(p.tiles_m - group * 8, 8), in = id % width;
    const int64_t m0 = (int64_t)(group * 8 + in % gm) * BM, n0 = (int64_t)(in / gm) * BN;

    const int total = p.steps * p.terms;
    const int split = blockIdx.y;
    const int first = (int)((int64_t)total * split / p.splits), last = (int)((int64_t)total * (split + 1) / p.splits);

    // A load instruction of a wave fills 8 rows of 8 chunks. Rows past the operand's end read
    // its last row: their products are never used.
    uint32_t va[S::kLoadsA], vb[S::kLoadsB];
    static_assert(S::kWaves % 2 == 0, "a wave's 8 rows all start at an even or all at an odd multiple of 8");
    const uint32_t chunk = (uint32_t)((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7)) * 16u;
#pragma unroll
    for (int j = 0; j < S::kLoadsA; ++j) {
        const int64_t r = min((int64_t)((j * S::kWaves + wave) * 8 + (lane >> 3)), p.M - 1 - m0);
        va[j] = (uint32_t)(r * p.a.ld * 2) + chunk;
    }
#pragma unroll
    for (int j = 0; j < S::kLoadsB; ++j) {
        const int64_t r = min((int64_t)((j * S::kWaves + wave) * 8 + (lane >> 3)), p.N - 1 - n0);
        vb[j] = (uint32_t)(r * p.b.ld * 2) + chunk;
    }
    const uint16_t *const pa = p.a.p + m0 * p.a.ld, *const pb = p.b.p + n0 * p.b.ld;
    // Stages are loaded in order: k is the next one's step within its partial product seg,
    // whose planes of (A, B) are (0,0) (0,1) (1,0).
    int seg = first / p.steps, k = first - seg * p.steps;
    __amdgpu_buffer_rsrc_t ra, rb;
    auto enter = [&]() {
        const int64_t oa = seg == 2 ? p.a.plane : 0, ob = seg == 1 ? p.b.plane : 0;
        ra = __builtin_amdgcn_make_buffer_rsrc((void *)(pa + oa), 0, -1, kRsrcWord3);
        rb = __builtin_amdgcn_make_buffer_rsrc((void *)(pb + ob), 0, -1, kRsrcWord3);
    };
    auto stage = [&](int kt) {
        SSM_LDS char *to = lds + (kt & 1) * S::kStage + wave * 1024;
#pragma unroll
        for (int j = 0; j < S::kLoadsA; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (SSM_LDS void *)(to + j * S::kWaves * 1024), 16, va[j],
                                                     k * (kBK * 2), 0, 0);
        to += BM * kBK * 2;
#pragma unroll
        for (int j = 0; j < S::kLoadsB; ++j)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (SSM_LDS void *)(to + j * S::kWaves * 1024), 16, vb[j],
                                                     k * (kBK * 2), 0, 0);
        ++k;
    };
    auto turn = [&]() {  // to the next partial product after its last step
        if (k < p.steps) return;
        k = 0;
        ++seg;
        enter();
    };

    // Fragments: lane l holds row l % 32 of a block, 8 consecutive k of half l / 32.
    const int row = lane & 31, half = lane >> 5;
    uint32_t fa[4], fb[4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
        const uint32_t c = (uint32_t)(((2 * ks + half) ^ (row >> 1 & 7)) * 16 + row * 128);
        fa[ks] = c + wm * S::TM * 4096;
        fb[ks] = c + wn * S::TN * 4096 + BM * kBK * 2;
    }
    f32x16 acc[S::TM][S::TN];
#pragma unroll
    for (int i = 0; i < S::TM; ++i)
#pragma unroll
        for (int j = 0; j < S::TN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    bf16x8 a[2][S::TM], b[2][S::TN];
    auto fetch = [&](int set, int kt, int ks) {
        const SSM_LDS char *at = lds + (kt & 1) * S::kStage;
#pragma unroll
        for (int i = 0; i < S::TM; ++i) a[set][i] = *(const SSM_LDS bf16x8 *)(at + fa[ks] + i * 4096);
#pragma unroll
        for (int j = 0; j < S::TN; ++j) b[set][j] = *(const SSM_LDS bf16x8 *)(at + fb[ks] + j * 4096);
    };
    auto multiply = [&](int set) {
#pragma unroll
        for (int i = 0; i < S::TM; ++i)
#pragma unroll
            for (int j = 0; j < S::TN; ++j)
                if constexpr (F16)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a[set][i]),
                                                                       __builtin_bit_cast(f16x8, b[set][j]), acc[i][j], 0,
                                                                       0, 0);
                else
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[set][i], b[set][j], acc[i][j], 0, 0, 0);
    };
    // Every wave's loads into the next stage and reads of this one are done.
    // But for the `newer` youngest loads, which may still be on their way: loads complete in order.
    auto meet = [&](auto newer) {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0x0070 | (newer & 15) | (newer >> 4) << 14);  // vmcnt(newer) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
    };
    // One stage of k: every fragment is read while the products of the one before it run. The
    // last one is in registers once all waves meet; then the stage's buffer is loaded again
    // and the next stage's first fragments are read behind the last products.
    constexpr int kFrag = S::TM + S::TN, kMul = S::TM * S::TN, kLoads = (S::kLoadsA + S::kLoadsB) / kMul;
    static_assert(kFrag <= kMul, "a fragment read for each product");
    auto weave = [&](auto loads) {  // one fragment read (and the loads' share) between products
#pragma unroll
        for (int j = 0; j < kMul; ++j) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if (j < kFrag) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            if (loads) __builtin_amdgcn_sched_group_barrier(0x020, kLoads, 0);
        }
    };
    typedef std::integral_constant<int, 0> none;
    auto step = [&](int kt, auto more, auto next) {
        fetch(1, kt, 1);
        multiply(0);
        fetch(0, kt, 2);
        multiply(1);
        fetch(1, kt, 3);
        multiply(0);
        weave(std::false_type{});
        weave(std::false_type{});
        weave(std::false_type{});
        if (next) {
            meet(none{});
            fetch(0, kt + 1, 0);
            if (more) stage(kt + 2);
        }
        multiply(1);
        if (next) weave(more);
    };
    if (first < last) {
        typedef std::true_type yes;
        typedef std::false_type no;
        enter();
        stage(first);
        if (first + 1 < last) {
            turn();
            stage(first + 1);
            meet(std::integral_constant<int, S::kLoadsA + S::kLoadsB>{});
        } else {
            meet(none{});
        }
        fetch(0, first, 0);
        int kt = first;
        while (kt + 2 < last) {
            turn();
            const int until = kt + min(last - 2 - kt, p.steps - k);
            for (; kt < until; ++kt) step(kt, yes{}, yes{});
        }
        if (kt + 1 < last) step(kt++, no{}, yes{});
        step(kt, no{}, no{});
        meet(none{});  // the epilogue may use the LDS
    }
    epilogue<S, E, F16, BM, BN, WM, WN>(p, acc, lds, m0, n0, wm, wn, split);
}

// Two products that do not wait for each other share a launch: blockIdx.z chooses.
struct ProductPair {
    ProductArgs p[2];
};
template <int BM, int BN, int WM, int WN, Epi E, bool F16>
__global__ void __launch_bounds__(64 * WM * WN, 1) k_product(ProductPair pair) {
    const ProductArgs &p = pair.p[blockIdx.z];
    if ((int)blockIdx.x >= p.tiles_m * p.tiles_n || (int)blockIdx.y >= p.splits) return;
    __shared__ __attribute__((aligned(1024))) char lds[Shape<BM, BN, WM, WN>::kLds];
    product_tile<BM, BN, WM, WN, E, F16>(p, (SSM_LDS char *)lds);
}

// A block's element e of lane l is row m = 8 (e / 4) + 4 (l / 32) + e % 4, column n = l % 32.
template <typename S, Epi E, bool F16, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void epilogue(const ProductArgs &p, f32x16 (&acc)[S::TM][S::TN], SSM_LDS char *lds,
                                         int64_t m0, int64_t n0, int wm, int wn, int split) {
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int64_t mw = m0 + wm * S::TM * 32 + 4 * half;  // the lane's first row
    const int64_t nw = n0 + wn * S::TN * 32 + (lane & 31);
    const float ua = unscale<F16>(p.a), ub = unscale<F16>(p.b);
    auto value = [&](float v) { return F16 ? v * ua * ub : v; };
    if constexpr (E == Epi::Lse) {
        const int64_t slot = (m0 / BM) * WM + wm;
#pragma unroll
        for (int j = 0; j < S::TN; ++j) {
            const int64_t n = nw + j * 32;
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < S::TM; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float v = acc[i][j][e] = value(acc[i][j][e]);
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
            const int64_t t = p.targets[n] - mw;  // the lane's rows are t = 32 i + 8 (e / 4) + e % 4
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
        // Through LDS, a token's row of kRow elements (an odd number of words, so that 8
        // tokens at one pair of columns fall on different banks), and out both ways. The
        // second plane starts from the product again. The token's weight stays out of G
        // (dhidden takes it as a factor, dweight with hidden^T), so that its values lie in
        // [-1, 1] and need no peak of their own.
        constexpr int kWords = S::kRow / 2;
        const float unit = p.planes ? (float)(1 << kPeak) : 1.0f;
        SSM_LDS uint32_t *words = (SSM_LDS uint32_t *)lds;
        for (int part = 0; part < max(p.planes, 1); ++part) {
#pragma unroll
            for (int j = 0; j < S::TN; ++j) {
                const int64_t n = nw + j * 32;
                const bool in = n < p.N;
                const int32_t target = in ? p.target[n] : -1;
                const float lse = in ? p.lse[n] : 0.0f;
                const float scale = target == -2 ? NAN : unit;  // out of range: loud
                const int t = (int)max((int64_t)-1, min((int64_t)S::TM * 32, target - p.v0 - mw));
                // an ignored token and the padding are exactly 0, whatever the logit
                const int rows = target == -1 ? 0 : (int)max((int64_t)0, min((int64_t)S::TM * 32, p.M - mw));
                SSM_LDS uint32_t *to = words + (wn * S::TN * 32 + j * 32 + (lane & 31)) * kWords +
                                       (wm * S::TM * 32 + 4 * half) / 2;
#pragma unroll
                for (int i = 0; i < S::TM; ++i)
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const int at = i * 32 + 8 * (e / 4) + e % 4;
                        uint32_t word = 0;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float q = e2((value(acc[i][j][e + k]) - lse) * kLog2e) - (t == at + k ? 1.0f : 0.0f);
                            float v = at + k < rows ? q * scale : 0.0f;
                            if (part > 0) take_f16(v);
                            word |= (uint32_t)(p.planes ? take_f16(v) : f32_to_bf16(v)) << (16 * k);
                        }
                        to[at / 2] = word;
                    }
            }
            __syncthreads();
            typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
            uint16_t *g = p.g + part * p.gplane, *gt = p.gt + part * p.gtplane;
            for (int c = threadIdx.x; c < BN * (BM / 8); c += S::kThreads) {  // 8 columns of a token
                const int n = c / (BM / 8), m = c % (BM / 8) * 8;
                if (n0 + n >= p.N || m0 + m >= p.ldg) continue;
                const SSM_LDS uint32_t *from = words + n * kWords + m / 2;
                *(u32x4 *)(g + (n0 + n) * p.ldg + m0 + m) = u32x4{from[0], from[1], from[2], from[3]};
            }
            if (p.gt)
                for (int c = threadIdx.x; c < (BM / 2) * (BN / 8); c += S::kThreads) {  // 8 tokens of 2 columns
                    // 8 lanes cover 64 tokens of one pair of columns: a whole line of G^T
                    const int m = (c / 8) % (BM / 2) * 2, n = (c / 8 / (BM / 2) * 8 + c % 8) * 8;
                    if (m0 + m >= p.M || n0 + n >= p.ldgt) continue;
                    uint32_t v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = words[(n + k) * kWords + m / 2];
                    u32x4 lo, hi;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        lo[k] = __builtin_amdgcn_perm(v[2 * k + 1], v[2 * k], 0x05040100);
                        hi[k] = __builtin_amdgcn_perm(v[2 * k + 1], v[2 * k], 0x07060302);
                    }
                    uint16_t *to = gt + (m0 + m) * p.ldgt + n0 + n;
                    *(u32x4 *)to = lo;
                    if (m0 + m + 1 < p.M) *(u32x4 *)(to + p.ldgt) = hi;
                }
            __syncthreads();
        }
    }
    if constexpr (E == Epi::Out) {
        const float scale = p.scale ? *p.scale : 1.0f;
        const bool vec = p.ldc % 4 == 0 && ((uintptr_t)p.c & 15) == 0;
#pragma unroll
        for (int j = 0; j < S::TN; ++j) {
            const int64_t n = nw + j * 32;
            if (n >= p.N) continue;
            const float row = p.row ? p.row[n] : scale;
#pragma unroll
            for (int i = 0; i < S::TM; ++i)
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const int64_t m = mw + i * 32 + 2 * e;
                    if (m >= p.M) continue;
                    const int64_t at = n * p.ldc + m;
                    float v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = value(acc[i][j][e + k]) * row;
                    if (p.add)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (m + k < p.M) v[k] += p.sum[at + k];
                    if (vec && m + 3 < p.M) {
                        if (p.c_bf16) {
                            uint2 w;
                            w.x = f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16;
                            w.y = f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16;
                            *(uint2 *)((bf16_bits *)p.c + split * p.cstride + at) = w;
                        } else {
                            *(float4 *)((float *)p.c + split * p.cstride + at) = make_float4(v[0], v[1], v[2], v[3]);
                        }
                    } else {
                        for (int k = 0; k < 4 && m + k < p.M; ++k) {
                            if (p.c_bf16) ((bf16_bits *)p.c)[split * p.cstride + at + k] = f32_to_bf16(v[k]);
                            else ((float *)p.c)[split * p.cstride + at + k] = v[k];
                        }
                    }
                }
        }
    }
}

// ---------------------------------------------------------------- operands
// dst[plane][r][ld] = src [rows][cols], 0 past its columns: a copy of bfloat16, or the scaled
// planes of float32.
template <typename IO>
__global__ void __launch_bounds__(256) k_pack(const IO *src, int64_t rows, int64_t cols, const uint32_t *peak,
                                              uint16_t *dst, int64_t ld, int64_t plane) {
    constexpr bool F32 = sizeof(IO) == 4;
    const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 2;
    if (c >= ld) return;
    const float scale = F32 ? exp2i(scale_exp(*peak)) : 1.0f;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
        const IO *from = src + r * cols + c;
        uint16_t *to = dst + r * ld + c;
        if constexpr (F32) {
            float v0 = c < cols ? from[0] * scale : 0.0f, v1 = c + 1 < cols ? from[1] * scale : 0.0f;
#pragma unroll
            for (int q = 0; q < kParts; ++q) {
                const uint32_t lo = take_f16(v0), hi = take_f16(v1);
                *(uint32_t *)(to + q * plane) = lo | hi << 16;
            }
        } else {
            const uint32_t lo = c < cols ? from[0] : 0, hi = c + 1 < cols ? from[1] : 0;
            *(uint32_t *)to = lo | hi << 16;
        }
    }
}

// dst[plane][c][ld] = src^T, src [rows][cols]: with a peak its scaled planes, without one a copy of
// bfloat16; 0 past its rows, and for the rows whose target is ignored: they may hold anything,
// and 0 times it must not reach a sum. w: a factor for each row of the planes. Blocks of 64 x 64 go through
// LDS, N columns a lane on the way in (2 where rows start on pairs), two rows on the way out.
template <typename IO, int N>
__global__ void __launch_bounds__(256) k_pack_t(const IO *src, int64_t rows, int64_t cols, const int32_t *target,
                                                const float *w, const uint32_t *peak, uint16_t *dst, int64_t ld,
                                                int64_t plane) {
    __shared__ float sh[64][65];
    const int64_t c0 = (int64_t)blockIdx.x * 64;
    typedef IO iov __attribute__((ext_vector_type(N)));
    constexpr int kLanes = 64 / N, kRows = 256 / kLanes;
    const int x = threadIdx.x % kLanes * N, y = threadIdx.x / kLanes;
    const float scale = peak ? exp2i(scale_exp(*peak)) : 1.0f;
    for (int64_t r0 = (int64_t)blockIdx.y * 64; r0 < ld; r0 += (int64_t)gridDim.y * 64) {
        iov from[64 / kRows];
#pragma unroll
        for (int k = 0; k < 64 / kRows; ++k) {
            const int64_t r = r0 + y + k * kRows;
            const bool in = r < rows && c0 + x < cols && !(target && target[r] == -1);
#pragma unroll
            for (int q = 0; q < N; ++q) from[k][q] = 0;
            if (in) from[k] = *(const iov *)(src + r * cols + c0 + x);
        }
#pragma unroll
        for (int k = 0; k < 64 / kRows; ++k) {
            const int64_t r = r0 + y + k * kRows;
            const float f = w && r < rows ? w[r] : 1.0f;  // 0 for an ignored row
#pragma unroll
            for (int q = 0; q < N; ++q) {
                const IO e = from[k][q];
                sh[y + k * kRows][x + q] = Io<IO>::ld(&e) * f * scale;
            }
        }
        __syncthreads();
        const int px = threadIdx.x & 31, py = threadIdx.x >> 5;  // two rows of src a lane
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int k = py + 8 * j;
            if (c0 + k >= cols) break;
            float v0 = sh[2 * px][k], v1 = sh[2 * px + 1][k];
            uint16_t *to = dst + (c0 + k) * ld + r0 + 2 * px;
            if (sizeof(IO) == 2 && !peak) {
                *(uint32_t *)to = f32_to_bf16(v0) | (uint32_t)f32_to_bf16(v1) << 16;
                continue;
            }
#pragma unroll
            for (int q = 0; q < (sizeof(IO) == 4 ? kParts : 1); ++q) {
                const uint32_t lo = take_f16(v0), hi = take_f16(v1);
                *(uint32_t *)(to + q * plane) = lo | hi << 16;
            }
        }
        __syncthreads();
    }
}

// peak = the bits of the largest finite |src| (times the row's w) over the rows whose target
// is not ignored. An integer maximum: its order does not matter. A block of 1024 has
// 1024 / across rows at a time, N columns a lane; few blocks, since each ends on one address.
constexpr int kPeakThreads = 1024, kPeakBlocks = 256;
template <typename IO, int N>
__global__ void __launch_bounds__(kPeakThreads) k_peak(const IO *src, int64_t rows, int64_t cols, int across,
                                                       const int32_t *target, const float *w, uint32_t *peak) {
    typedef IO iov __attribute__((ext_vector_type(N)));
    __shared__ uint32_t sh[kPeakThreads / 64];
    const int down = kPeakThreads / across;
    const int64_t c0 = (int64_t)(threadIdx.x % across) * N;
    uint32_t top = 0;
#pragma unroll 4
    for (int64_t r = (int64_t)blockIdx.x * down + threadIdx.x / across; r < rows; r += (int64_t)gridDim.x * down) {
        if (target && target[r] == -1) continue;
        const float f = w ? w[r] : 1.0f;
        for (int64_t c = c0; c < cols; c += across * N) {
            const iov v = *(const iov *)(src + r * cols + c);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const IO e = v[k];
                const uint32_t b = __float_as_uint(Io<IO>::ld(&e) * f) & 0x7fffffffu;
                top = b < 0x7f800000u ? max(top, b) : top;
            }
        }
    }
    for (int o = 32; o > 0; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o));
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x) return;
    for (int k = 1; k < kPeakThreads / 64; ++k) top = max(top, sh[k]);
    if (top) atomicMax(peak, top);
}

// target[t] = the row, -1 where ignored, -2 where out of range; w[t] = the loss's weight, all[0]
// the one that every token has without dloss; the peaks start at 0.
__global__ void __launch_bounds__(256) k_xent_tokens(const int64_t *targets, int64_t ignore, int64_t T, int64_t V,
                                                     const float *dloss, const float *dmean, const float *mean,
                                                     int32_t *target, float *w, float *all, uint32_t *peak, int64_t n_peaks) {
    const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
    for (int64_t k = t; k < n_peaks; k += (int64_t)gridDim.x * 256) peak[k] = 0;
    const float same = dmean ? *dmean * mean[1] : 0.0f;
    if (t == 0 && all) *all = same;
    if (t >= T) return;
    const int64_t y = targets[t];
    const int32_t to = y == ignore ? -1 : y >= 0 && y < V ? (int32_t)y : -2;
    target[t] = to;
    if (w) w[t] = to == -1 ? 0.0f : to == -2 ? NAN : (dloss ? dloss[t] : 0.0f) + same;
}

// (m, s) += (m2, s2): sums of exponentials under their maxima.
__device__ __forceinline__ void join(float &m, float &s, float m2, float s2) {
    const float M = m > m2 || m != m ? m : m2;
    const float f = m == M ? 1.0f : e2((m - M) * kLog2e), g = m2 == M ? 1.0f : e2((m2 - M) * kLog2e);
    s = s * f + s2 * g;
    m = M;
}

// 16 threads for a token join its n partial pairs.
__global__ void __launch_bounds__(256) k_xent_join(const float2 *part, int64_t n, const float *at,
                                                   const int64_t *targets, int64_t ignore, int64_t T, int64_t V,
                                                   float *loss, float *lse) {
    __shared__ float2 sh[16][16];
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
    const int64_t t = (int64_t)blockIdx.x * 16 + x;
    float m = -INFINITY, s = 0.0f;
    if (t < T)
        for (int64_t j = y; j < n; j += 16) {
            const float2 q = part[j * T + t];
            join(m, s, q.x, q.y);
        }
    sh[y][x] = make_float2(m, s);
    __syncthreads();
    if (y || t >= T) return;
    for (int j = 1; j < 16; ++j) join(m, s, sh[j][x].x, sh[j][x].y);
    const float l = m + logf(s);
    lse[t] = l;
    const int64_t to = targets[t];
    loss[t] = to == ignore ? 0.0f : to >= 0 && to < V ? l - at[t] : NAN;
}

// mean[0] = mean loss over the tokens that are not ignored, mean[1] = 1 / their number.
__global__ void __launch_bounds__(1024) k_xent_mean(const float *loss, const int64_t *targets, int64_t ignore,
                                                    int64_t T, float *mean) {
    __shared__ double sh[16];
    __shared__ int64_t sn[16];
    double s = 0.0;
    int64_t c = 0;
    for (int64_t t = threadIdx.x; t < T; t += 1024)
        if (targets[t] != ignore) {
            s += loss[t];
            ++c;
        }
    for (int o = 32; o > 0; o >>= 1) {
        s += __shfl_xor(s, o);
        c += __shfl_xor(c, o);
    }
    if ((threadIdx.x & 63) == 0) {
        sh[threadIdx.x >> 6] = s;
        sn[threadIdx.x >> 6] = c;
    }
    __syncthreads();
    if (threadIdx.x) return;
    for (int j = 1; j < 16; ++j) {
        s += sh[j];
        c += sn[j];
    }
    mean[0] = c ? (float)(s / (double)c) : 0.0f;
    mean[1] = c ? (float)(1.0 / (double)c) : 0.0f;
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
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e < n) p[e] = IO(0);
}

// ---------------------------------------------------------------- host
int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
unsigned blocks(int64_t n, int64_t per) { return (unsigned)((n + per - 1) / per); }

constexpr int kBig = 256, kSmall = 128;

// Tiles of 256 x 256 or 128 x 128 and a split of k, whichever takes less time on 256 compute
// units by their rounds: a compute unit makes a quarter of the work in about a third of the
// time with the small tiles (measured on 8192 x 8192 x 4096: 1250 against 950 TFLOP/s), which
// waste less at the edges and in the last round. Only small tiles are split (1000 x 1000 x 48000:
// 134 us in 8 parts of small tiles, 170 in 16 of large ones); a split keeps at least 8 steps of k.
struct Tiling {
    int tile, splits;
};
constexpr int64_t kCus = 256;
Tiling tiling(int64_t M, int64_t N, int64_t steps, bool may_split) {
    Tiling best{};
    double least = 0;
    for (const int tile : {kSmall, kBig}) {
        const int64_t n = (int64_t)blocks(M, tile) * blocks(N, tile), room = 2 * kCus / n;
        const int64_t s = !may_split || tile == kBig ? 1 : std::max<int64_t>(1, std::min(std::min(room, steps / 8), (int64_t)16));
        const double time = (double)blocks(n * s, kCus) / (double)s * (tile == kBig ? 3.0 : 1.0);
        if (!best.tile || time < least) {
            best = {tile, (int)s};
            least = time;
        }
    }
    return best;
}

void set_tiles(ProductArgs &p, int tile) {
    p.tiles_m = (int32_t)blocks(p.M, tile);
    p.tiles_n = (int32_t)blocks(p.N, tile);
}
template <Epi E, bool F16>
hipError_t product(const ProductPair &pair, int n, int tile, hipStream_t s) {
    int32_t tiles = 0, splits = 0;
    for (int k = 0; k < n; ++k) {
        tiles = std::max(tiles, pair.p[k].tiles_m * pair.p[k].tiles_n);
        splits = std::max(splits, pair.p[k].splits);
    }
    const dim3 grid((unsigned)tiles, (unsigned)splits, (unsigned)n);
    if (tile == kBig) k_product<256, 256, 2, 4, E, F16><<<grid, 512, 0, s>>>(pair);
    else k_product<128, 128, 2, 2, E, F16><<<grid, 256, 0, s>>>(pair);
    return hipGetLastError();
}
template <Epi E, bool F16>
hipError_t product(const ProductArgs &p, int tile, hipStream_t s) {
    ProductPair pair{};
    pair.p[0] = p;
    set_tiles(pair.p[0], tile);
    return product<E, F16>(pair, 1, tile, s);
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

// What a call lays out in its workspace.
struct Layout {
    int planes, terms;         // of an operand, of a product
    int64_t ldk, ldt, piece;   // padded dim, tokens; vocabulary rows of a piece
    Tiling lse, out_w, out_h;
    bool pack;                 // hidden and weight are copied: float32, or rows not in steps of 64
    uint16_t *hidden, *weight;
    int32_t *target;
    uint32_t *peak;
    int64_t peaks;
    float *at, *w, *all, *sum, *split_w, *split_h;
    float2 *part;
    uint16_t *ht, *wt, *g, *gt;
    size_t bytes;
};

// G and G^T of a piece hold about 2^26 values each: 8192 tokens take pieces of 8192 rows, whose
// three products are 512 and 1024 tiles of 256 x 256, whole rounds of the compute units.
constexpr int64_t kPieceValues = (int64_t)1 << 26;

Layout lay_out(int64_t T, int64_t K, int64_t V, int io, bool bwd, bool aligned, char *ws) {
    Layout l{};
    Arena a{ws};
    l.planes = io ? 1 : kParts;
    l.terms = io ? 1 : 3;
    l.ldk = up(K, kBK);
    l.ldt = up(T, kBK);
    l.pack = !io || K % kBK != 0 || !aligned;
    l.target = a.take<int32_t>(T);
    // sized as if the operands had to be copied: their alignment is not known to the query
    l.hidden = a.take<uint16_t>(T * l.ldk * l.planes);
    l.weight = a.take<uint16_t>(V * l.ldk * l.planes);
    l.peaks = kPeakPiece;
    if (!bwd) {
        l.lse = tiling(V, T, l.ldk / kBK * l.terms, false);
        l.part = a.take<float2>((int64_t)blocks(V, l.lse.tile) * 2 * T);
        l.at = a.take<float>(T);
    } else {
        l.piece = std::min(up(V, kBig), std::max<int64_t>(1024, kPieceValues / std::max<int64_t>(T, 1) / kBig * kBig));
        const int64_t most = std::min(V, l.piece);
        l.peaks += blocks(V, l.piece);
        l.out_w = tiling(K, most, l.ldt / kBK * l.terms, true);
        l.out_h = tiling(K, T, up(most, kBK) / kBK * l.terms, true);
        l.w = a.take<float>(T);
        l.all = a.take<float>(1);
        l.sum = a.take<float>(V > l.piece ? T * K : 0);
        l.ht = a.take<uint16_t>(K * l.ldt * l.planes);
        l.wt = a.take<uint16_t>(K * up(most, kBK) * l.planes);
        l.g = a.take<uint16_t>(T * up(most, kBK) * l.planes);
        l.gt = a.take<uint16_t>(most * l.ldt * l.planes);
        const int64_t sw = l.out_w.splits > 1 ? l.out_w.splits * most * K : 0;
        const int64_t sh = l.out_h.splits > 1 ? l.out_h.splits * T * K : 0;
        l.split_w = a.take<float>(sw);
        l.split_h = a.take<float>(sh);
    }
    l.peak = a.take<uint32_t>(l.peaks);
    l.bytes = a.used;
    return l;
}

template <typename IO>
hipError_t pack(const void *src, int64_t rows, int64_t cols, const uint32_t *peak, uint16_t *dst, int64_t ld,
                hipStream_t s) {
    k_pack<IO><<<dim3(blocks(ld, 512), (unsigned)std::min<int64_t>(rows, 65535)), 256, 0, s>>>((const IO *)src, rows, cols,
                                                                                               peak, dst, ld, rows * ld);
    return hipGetLastError();
}
template <typename IO>
hipError_t pack_t(const void *src, int64_t rows, int64_t cols, const int32_t *target, const float *w,
                  const uint32_t *peak, uint16_t *dst, int64_t ld, hipStream_t s) {
    const dim3 grid(blocks(cols, 64), (unsigned)std::min<int64_t>(ld / 64, 65535));
    if (cols % 2 == 0 && (uintptr_t)src % (2 * sizeof(IO)) == 0)
        k_pack_t<IO, 2><<<grid, 256, 0, s>>>((const IO *)src, rows, cols, target, w, peak, dst, ld, cols * ld);
    else
        k_pack_t<IO, 1><<<grid, 256, 0, s>>>((const IO *)src, rows, cols, target, w, peak, dst, ld, cols * ld);
    return hipGetLastError();
}
template <typename IO>
hipError_t find_peak(const void *src, int64_t rows, int64_t cols, const int32_t *target, const float *w, uint32_t *peak,
                     hipStream_t s) {
    const bool wide = cols % 4 == 0 && (uintptr_t)src % (4 * sizeof(IO)) == 0;
    const int64_t lanes = wide ? cols / 4 : cols;
    int across = 16;
    while (across < lanes && across < kPeakThreads) across *= 2;
    const dim3 grid((unsigned)std::min<int64_t>(blocks(rows, kPeakThreads / across), kPeakBlocks));
    if (wide) k_peak<IO, 4><<<grid, kPeakThreads, 0, s>>>((const IO *)src, rows, cols, across, target, w, peak);
    else k_peak<IO, 1><<<grid, kPeakThreads, 0, s>>>((const IO *)src, rows, cols, across, target, w, peak);
    return hipGetLastError();
}

#define SSM_TRY(x)                                 \
    do {                                           \
        const hipError_t try_e = (x);              \
        if (try_e != hipSuccess) return try_e;     \
    } while (0)

bool rows_aligned(const XentArgs &a) { return ((uintptr_t)a.hidden | (uintptr_t)a.weight) % 16 == 0; }

// The operands of the logits: hidden and weight as they are, or their packed copies.
template <typename IO>
hipError_t logits_operands(const XentArgs &a, const Layout &l, ProductArgs &p, hipStream_t s) {
    const uint16_t *h = (const uint16_t *)a.hidden, *w = (const uint16_t *)a.weight;
    if (sizeof(IO) == 4) {
        SSM_TRY(find_peak<IO>(a.hidden, a.T, a.K, l.target, nullptr, l.peak + kPeakH, s));
        SSM_TRY(find_peak<IO>(a.weight, a.V, a.K, nullptr, nullptr, l.peak + kPeakW, s));
    }
    if (l.pack) {
        SSM_TRY(pack<IO>(a.hidden, a.T, a.K, l.peak + kPeakH, l.hidden, l.ldk, s));
        SSM_TRY(pack<IO>(a.weight, a.V, a.K, l.peak + kPeakW, l.weight, l.ldk, s));
        h = l.hidden;
        w = l.weight;
    }
    p.a = {w, l.ldk, a.V * l.ldk, l.peak + kPeakW};
    p.b = {h, l.ldk, a.T * l.ldk, l.peak + kPeakH};
    p.steps = (int32_t)(l.ldk / kBK);
    p.terms = l.terms;
    p.splits = 1;
    p.target = l.target;
    p.targets = a.targets;
    return hipSuccess;
}

template <typename IO>
hipError_t xent_fwd(const XentArgs &a, int io, hipStream_t s) {
    if (a.T > 0) {
        const Layout l = lay_out(a.T, a.K, a.V, io, false, rows_aligned(a), (char *)a.ws);
        if (!io)  // for the peaks
            k_xent_tokens<<<dim3(blocks(a.T, 256)), 256, 0, s>>>(a.targets, a.ignore, a.T, a.V, nullptr, nullptr, nullptr,
                                                                l.target, nullptr, nullptr, l.peak, l.peaks);
        ProductArgs p{};
        SSM_TRY(logits_operands<IO>(a, l, p, s));
        p.M = a.V;
        p.N = a.T;
        p.part = l.part;
        p.at = l.at;
        SSM_TRY((product<Epi::Lse, sizeof(IO) == 4>(p, l.lse.tile, s)));
        k_xent_join<<<dim3(blocks(a.T, 16)), 256, 0, s>>>(l.part, (int64_t)blocks(a.V, l.lse.tile) * 2, l.at, a.targets,
                                                         a.ignore, a.T, a.V, a.loss, a.lse);
    }
    k_xent_mean<<<dim3(1), 1024, 0, s>>>(a.loss, a.targets, a.ignore, a.T, a.mean);
    return hipGetLastError();
}

// One of the gradients' products: C [N][M] = (sum +) A B^T, through partial sums over k where it
// is split.
struct Gradient {
    ProductArgs p;
    Tiling t;
    JoinArgs join;
};
Gradient gradient(ProductArgs p, Tiling t, float *split, void *dst, bool bf16, float *sum, bool add) {
    Gradient g{p, t, {}};
    g.p.splits = t.splits;
    g.p.ldc = p.M;
    g.p.sum = sum;
    g.p.add = add && t.splits == 1;
    g.p.c = t.splits == 1 ? dst : split;
    g.p.c_bf16 = bf16 && t.splits == 1;
    g.p.cstride = p.M * p.N;
    set_tiles(g.p, t.tile);
    if (t.splits > 1) g.join = {split, t.splits, p.M * p.N, add ? sum : nullptr, dst, bf16};
    return g;
}
// One or both of them, in one launch where their tiles agree.
hipError_t run_gradients(const Gradient *g, int n, bool f16, hipStream_t s) {
    if (n == 2 && g[0].t.tile != g[1].t.tile) {
        SSM_TRY(run_gradients(g, 1, f16, s));
        return run_gradients(g + 1, 1, f16, s);
    }
    ProductPair pair{};
    JoinPair join{};
    int64_t most = 0;
    for (int k = 0; k < n; ++k) {
        pair.p[k] = g[k].p;
        join.j[k] = g[k].join;
        most = std::max(most, g[k].join.count);
    }
    SSM_TRY((f16 ? product<Epi::Out, true>(pair, n, g[0].t.tile, s) : product<Epi::Out, false>(pair, n, g[0].t.tile, s)));
    if (most > 0) k_join_splits<<<dim3(blocks(most, 256), (unsigned)n), 256, 0, s>>>(join);
    return hipGetLastError();
}

template <typename IO>
hipError_t xent_bwd(const XentArgs &a, int io, hipStream_t s) {
    if (a.T == 0) {
        if (a.dweight) k_zero<IO><<<dim3(blocks(a.V * a.K, 256)), 256, 0, s>>>((IO *)a.dweight, a.V * a.K);
        return hipGetLastError();
    }
    const Layout l = lay_out(a.T, a.K, a.V, io, true, rows_aligned(a), (char *)a.ws);
    k_xent_tokens<<<dim3(blocks(a.T, 256)), 256, 0, s>>>(a.targets, a.ignore, a.T, a.V, a.dloss, a.dmean, a.mean,
                                                        l.target, l.w, l.all, l.peak, l.peaks);
    ProductArgs logits{};
    SSM_TRY(logits_operands<IO>(a, l, logits, s));
    logits.N = a.T;
    logits.lse = a.lse;
    // one weight for all tokens: it is a factor at the end, and bfloat16 serves for the rest
    const bool f16 = sizeof(IO) == 4 || a.dloss;
    logits.planes = f16 ? l.planes : 0;
    if (a.dweight) {
        uint32_t *peak = f16 ? l.peak + kPeakWH : nullptr;
        if (f16) SSM_TRY(find_peak<IO>(a.hidden, a.T, a.K, l.target, l.w, peak, s));
        SSM_TRY(pack_t<IO>(a.hidden, a.T, a.K, l.target, f16 ? l.w : nullptr, peak, l.ht, l.ldt, s));
    }
    for (int64_t v0 = 0; v0 < a.V; v0 += l.piece) {
        const int64_t nv = std::min(l.piece, a.V - v0), ldg = up(nv, kBK);
        ProductArgs p = logits;
        p.a.p += v0 * l.ldk;
        p.M = nv;
        p.v0 = v0;
        p.g = l.g;
        p.gt = a.dweight ? l.gt : nullptr;
        p.ldg = ldg;
        p.ldgt = l.ldt;
        p.gplane = a.T * ldg;
        p.gtplane = nv * l.ldt;
        SSM_TRY((product<Epi::Dlogits, sizeof(IO) == 4>(p, tiling(nv, a.T, p.steps * l.terms, false).tile, s)));
        Gradient grads[2];
        int n = 0;
        if (a.dweight) {
            ProductArgs q{};
            q.a = {l.ht, l.ldt, a.K * l.ldt, l.peak + kPeakWH};
            q.b = {l.gt, l.ldt, nv * l.ldt, nullptr};
            q.M = a.K;
            q.N = nv;
            q.steps = (int32_t)(l.ldt / kBK);
            q.terms = l.terms;
            q.scale = f16 ? nullptr : l.all;
            grads[n++] = gradient(q, l.out_w, l.split_w, (IO *)a.dweight + v0 * a.K, io, nullptr, false);
        }
        if (a.dhidden) {
            // float32 weights have their peak from the logits; a piece's is read twice here
            // while the caches still hold it
            const IO *piece = (const IO *)a.weight + v0 * a.K;
            uint32_t *peak = !f16 ? nullptr : l.peak + (sizeof(IO) == 4 ? (int64_t)kPeakW : kPeakPiece + v0 / l.piece);
            if (f16 && sizeof(IO) == 2) SSM_TRY(find_peak<IO>(piece, nv, a.K, nullptr, nullptr, peak, s));
            SSM_TRY(pack_t<IO>(piece, nv, a.K, nullptr, nullptr, peak, l.wt, ldg, s));
            ProductArgs q{};
            q.a = {l.wt, ldg, a.K * ldg, peak};
            q.b = {l.g, ldg, a.T * ldg, nullptr};
            q.row = l.w;
            q.M = a.K;
            q.N = a.T;
            q.steps = (int32_t)(ldg / kBK);
            q.terms = l.terms;
            const bool end = v0 + nv == a.V;
            grads[n++] = gradient(q, l.out_h, l.split_h, end ? a.dhidden : l.sum, end && io, l.sum, v0 > 0);
        }
        SSM_TRY(run_gradients(grads, n, f16, s));
    }
    return hipSuccess;
}

}  // namespace

size_t xent_fwd_ws(int64_t T, int64_t K, int64_t V, int io) {
    return T > 0 ? lay_out(T, K, V, io, false, false, nullptr).bytes : 0;
}
size_t xent_bwd_ws(int64_t T, int64_t K, int64_t V, int io) {
    return T > 0 ? lay_out(T, K, V, io, true, false, nullptr).bytes : 0;
}
hipError_t launch_xent_fwd(const XentArgs &a, int io, hipStream_t s) {
    return io ? xent_fwd<bf16_bits>(a, io, s) : xent_fwd<float>(a, io, s);
}
hipError_t launch_xent_bwd(const XentArgs &a, int io, hipStream_t s) {
    return io ? xent_bwd<bf16_bits>(a, io, s) : xent_bwd<float>(a, io, s);
}

}  // namespace ssm
