// linattn.hip -- linear attention with a decay for each head: a state S [K, V] for every sequence
// and head,
//     S_t = exp(g_t) S_{t-1} + k_t v_t^T,    o_t = scale q_t^T S_t.
//
// In chunks of C tokens, with G the sums of g from the chunk's start (inclusive):
//     o_i   = scale (e^{G_i} q_i S_in + sum_{j <= i} (q_i.k_j) e^{G_i - G_j} v_j)
//     S_out = e^{G_C} S_in + sum_j e^{G_C - G_j} k_j v_j^T.
// The gradients, with dS_out the gradient of what leaves the chunk (do times scale throughout):
//     dq_i  = e^{G_i} S_in do_i + sum_{j <= i} (do_i.v_j) e^{G_i - G_j} k_j
//     dk_j  = e^{G_C - G_j} dS_out v_j + sum_{i >= j} (do_i.v_j) e^{G_i - G_j} q_i
//     dv_j  = e^{G_C - G_j} dS_out^T k_j + sum_{i >= j} (q_i.k_j) e^{G_i - G_j} do_i
//     dS_in = e^{G_C} dS_out + sum_i e^{G_i} q_i do_i^T
//     dg_t  = <what passes from before t to t and after>
//           = sum_{j < t <= i} (q_i.k_j)(do_i.v_j) e^{G_i - G_j} + sum_{i >= t} e^{G_i} q_i S_in do_i
//             + sum_{j < t} e^{G_C - G_j} k_j dS_out v_j + e^{G_C} <S_in, dS_out>,
// a sum without a difference, so that dg keeps its precision where a decay is strong. A g below
// kCut (exp(g) is 0 in float32) is a cut: decays across it are 0 by a comparison of document
// numbers, and its g does not enter G. G is a sum in 64 bits.
//
// Everything is a product on the matrix cores: v_mfma_f32_32x32x16_bf16 for bfloat16 inputs, and
// v_mfma_f32_32x32x2_f32 for float32 ones. The state stays in a wave's accumulators for a whole
// sweep (all of K for 32 columns of V) and is an operand from there: lane l holds column l % 32 and
// of each 8 rows the 4 of its half, and the other operand is read in the same order of the
// contraction ("quads": 4 consecutive elements at 8 a + 4 (l / 32)).
// bfloat16: scores, and the state where it makes an output of bfloat16, enter a product as the sum of two
// bfloat16 parts, which hold 17 bits: an output's error is its own rounding. (Of one part, 8 bits, the errors
// were 2.35e-3 of norm where the rounding is 1.66e-3.) What goes into a float32 result (states, dg) takes
// factors in three parts, which hold 24 bits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "ssm_layers.h"

namespace ssm {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
#define SSM_LDS __attribute__((address_space(3)))

// How rows are read and written: whole vectors of 16 bytes that start on 16 bytes; vectors that start on any
// element, the last of a row ending with it (rows of a vector at least); or elements.
enum Access { kWide, kAny, kElements };

constexpr float kCut = -104.0f;  // exp of less is 0 in float32
constexpr double kLog2e = 1.4426950408889634;

// What depends on the inputs' type: tokens of a chunk (C), the contraction of a step (KS), a
// fragment (this lane's elements of a step), and the parts that hold a float32 factor of a float32 result and
// of an output.
template <typename T> struct Kind;
template <> struct Kind<__bf16> {
    static constexpr int C = 64, KS = 16, kParts = 3, kOut = 2;
    typedef bf16x8 Frag;
    typedef f32x8 Wide;
    typedef u32x2 Quad;
};
template <> struct Kind<float> {
    static constexpr int C = 32, KS = 8, kParts = 1, kOut = 1;
    typedef f32x4 Frag;
    typedef f32x4 Wide;
    typedef f32x4 Quad;
};

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma(f32x4 a, f32x4 b, f32x16 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
    return c;
}

// x as the sum of operands. Two of them are rounded: 2^-18 of x is left at most.
__device__ __forceinline__ void split(f32x8 x, bf16x8 (&p)[2]) {
    p[0] = __builtin_convertvector(x, bf16x8);
    p[1] = __builtin_convertvector(x - __builtin_convertvector(p[0], f32x8), bf16x8);
}
// Three by truncation: 8 bits of 24 each, and nothing is left.
__device__ __forceinline__ void split(f32x8 x, bf16x8 (&p)[3]) {
    u32x4 q[3];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float a = x[2 * e], b = x[2 * e + 1];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const uint32_t ha = __float_as_uint(a) & 0xffff0000u, hb = __float_as_uint(b) & 0xffff0000u;
            q[k][e] = __builtin_amdgcn_perm(hb, ha, 0x07060302u);
            a -= __uint_as_float(ha);
            b -= __uint_as_float(hb);
        }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) p[k] = __builtin_bit_cast(bf16x8, q[k]);
}
__device__ __forceinline__ void split(f32x4 x, f32x4 (&p)[1]) { p[0] = x; }
__device__ __forceinline__ f32x8 widened(bf16x8 x) { return __builtin_convertvector(x, f32x8); }
__device__ __forceinline__ f32x4 widened(f32x4 x) { return x; }

// The compiler would read every fragment of a chunk from LDS before the first product, and spill.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// Step s of an accumulator's 32 rows as a fragment's elements.
template <typename T>
__device__ __forceinline__ typename Kind<T>::Wide rows_of(const f32x16 &acc, int s) {
    typename Kind<T>::Wide w;
    constexpr int N = sizeof(w) / 4;
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = acc[s * N + e];
    return w;
}
// The weights of a fragment's tokens (step s of a float array in LDS).
__device__ __forceinline__ void weights_of(const float *w, int s, int half, f32x8 &out) {
    const f32x4 lo = *(const f32x4 *)(w + 16 * s + 4 * half), hi = *(const f32x4 *)(w + 16 * s + 8 + 4 * half);
    out = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ void weights_of(const float *w, int s, int half, f32x4 &out) {
    out = *(const f32x4 *)(w + 8 * s + 4 * half);
}

// ROWS x F elements in LDS, in quads of 4 whose places in a row are permuted (by exclusive or, 16 bytes at a
// time) so that both ways of reading meet no bank twice: 16 bytes of 16 rows (fragments whose lanes are
// rows), and 4 rows of 32 neighbouring columns (fragments whose lanes are columns). bfloat16: the two quads
// of a lane's fragment, 8 elements apart, lie next to each other.
template <typename T, int ROWS, int F>
struct Tile {
    typedef Kind<T> N;
    static constexpr int W = F / 4, kRow = F * (int)sizeof(T), kBytes = ROWS * kRow;
    static __device__ __forceinline__ int at(int row, int quad) {
        if constexpr (sizeof(T) == 2) {
            const int f = W == 32 ? (row & 3) << 2 | (row >> 2 & 3) : (row >> 1 & 1) << 2 | (row >> 2 & 3);
            const int place = (quad >> 2) * 2 + (quad & 1);
            return row * kRow + ((place ^ f) * 2 + (quad >> 1 & 1)) * 8;
        } else {
            const int f = W == 8 ? row >> 1 & 7
                                 : (row & 3) | (row >> 2 & 1) << 3 | (row >> 3 & 1) << 2 | (W == 32 ? (row >> 4 & 1) << 4 : 0);
            return row * kRow + (quad ^ f) * 16;
        }
    }
    // Rows start on multiples of their size, so a step or a block changes a lane's address by an exclusive
    // or and a constant, and a lane keeps one number for each way of reading.
    // lanes: rows; contraction: columns KS s .. KS s + KS - 1. from: at(row, half).
    static __device__ __forceinline__ typename N::Frag by_row(const char *t, int from, int s) {
        return *(const typename N::Frag *)(t + (from ^ s * 32));
    }
    // lanes: columns 32 block + l % 32; contraction: rows KS s .. KS s + KS - 1. from: column_base(lane).
    static __device__ __forceinline__ int column_base(int lane) {
        const int half = lane >> 5;
        if constexpr (sizeof(T) == 2) return at(4 * half + (lane >> 2 & 3), (lane >> 4 & 1) * 4 + (lane & 3));
        else return at(4 * half, lane >> 2 & 7) + (lane & 3) * 4;
    }
    static __device__ __forceinline__ typename N::Frag by_column(const char *t, int from, int block, int s) {
        if constexpr (sizeof(T) == 2) {
            const int c = block * 64;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SSM_LDS s16x4 *)(t + (from ^ c) + s * 16 * kRow));
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((SSM_LDS s16x4 *)(t + (from ^ c ^ 32) + (s * 16 + 8) * kRow));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            f32x4 f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = W == 8 ? (e >> 1 | (s & 1) << 2) * 16 : (e | (s & 1) << 2 | (W == 32 ? (s >> 1 & 1) << 4 : 0)) * 16 ^ block * 128;
                f[e] = *(const float *)(t + (from ^ c) + (8 * s + e) * kRow);
            }
            return f;
        }
    }
    static __device__ __forceinline__ f32x4 quad(const char *t, int row, int quad) {
        if constexpr (sizeof(T) == 2) return __builtin_convertvector(*(const bf16x4 *)(t + at(row, quad)), f32x4);
        else return *(const f32x4 *)(t + at(row, quad));
    }
    static __device__ __forceinline__ float one(const char *t, int row, int column) {
        return (float)*(const T *)(t + at(row, column / 4) + column % 4 * (int)sizeof(T));
    }
    // One quad of a row, from four float32 values.
    static __device__ __forceinline__ void put(char *t, int row, int quad, f32x4 x) {
        if constexpr (sizeof(T) == 2) *(bf16x4 *)(t + at(row, quad)) = __builtin_convertvector(x, bf16x4);
        else *(f32x4 *)(t + at(row, quad)) = x;
    }
};

// Scores in kOut parts: rows i and columns j <= i of the chunk (BELOW), or rows j and columns i >= j. Of their
// four tiles of 32 x 32 (bfloat16) one is empty, so the second parts of the row of tiles that has one tile lie
// in it, and those of the other 32 rows behind the first parts: two blocks of the sweep still share a compute
// unit, and the backward's tiles fit one.
template <typename T, int C, bool BELOW>
struct Scores {
    typedef Tile<T, C, C> P;
    static constexpr int kDown = 32 * P::kRow, kBytes = P::kBytes + (Kind<T>::kOut - 1) * kDown;
    static __device__ __forceinline__ int at(int row, int quad) { return P::at(row, quad); }
    static __device__ __forceinline__ int second(int row, int o) { return BELOW == (row < 32) ? o ^ 64 : o + (BELOW ? 1 : 2) * kDown; }
    static __device__ __forceinline__ void put(char *t, int row, int quad, f32x4 x) {
        if constexpr (Kind<T>::kOut == 1) {
            P::put(t, row, quad, x);
        } else {
            const int o = P::at(row, quad);
            const bf16x4 first = __builtin_convertvector(x, bf16x4);
            *(bf16x4 *)(t + o) = first;
            *(bf16x4 *)(t + second(row, o)) = __builtin_convertvector(x - __builtin_convertvector(first, f32x4), bf16x4);
        }
    }
    static __device__ __forceinline__ float one(const char *t, int row, int column) {
        const int o = at(row, column / 4), c = column % 4 * (int)sizeof(T);
        if constexpr (Kind<T>::kOut == 1) return *(const T *)(t + o + c);
        else return (float)*(const T *)(t + o + c) + (float)*(const T *)(t + second(row, o) + c);
    }
    // lanes: rows 32 tile + l % 32; contraction: step s. from: at(l % 32, half).
    static __device__ __forceinline__ typename Kind<T>::Frag by_row(const char *t, int from, int tile, int s, int part) {
        if (part == 0) return P::by_row(t + tile * kDown, from, s);
        if (BELOW == (tile == 0)) return P::by_row(t + tile * kDown, from, s ^ 2);
        return P::by_row(t + 2 * kDown, from, s);
    }
};

// A range of global memory by offsets in 32 bits: what lies outside reads as 0 and is not written. All of an
// offset is given as the vector one, since the scalar one is not compared with the range. kOut is outside of
// every range, and so is what is added to it here.
constexpr int kOut = (int)0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t range_of(const void *p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void *)p, 0, (int)bytes, 0x00020000);
}
// Four float32 or bfloat16 values at element e of a row that starts at byte `at`; `width` elements long.
template <typename T, Access ACC>
__device__ __forceinline__ void put_quad(__amdgpu_buffer_rsrc_t to, int at, int e, int width, f32x4 x) {
    if (ACC != kElements) {
        const int o = e + 4 <= width ? at + e * (int)sizeof(T) : kOut;
        if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, __builtin_convertvector(x, bf16x4)), to, o, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), to, o, 0, 0);
    }
    if (ACC == kElements || (ACC == kAny && e < width && e + 4 > width)) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int o = e + k < width ? at + (e + k) * (int)sizeof(T) : kOut;
            if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, (__bf16)x[k]), to, o, 0, 0);
            else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[k]), to, o, 0, 0);
        }
    }
}
// The last vector of a row is read so that it ends with the row; its elements from d on are the asked ones
// (d of a vector or more: none, the load was out of range), and what is past the row is 0.
template <typename T>
__device__ __forceinline__ u32x4 moved_down(u32x4 r, int d) {
    const int dwords = sizeof(T) == 2 ? d >> 1 : d;
    if constexpr (sizeof(T) == 2) {
        const uint32_t bits = (d & 1) * 16;
        r = u32x4{__builtin_amdgcn_alignbit(r[1], r[0], bits), __builtin_amdgcn_alignbit(r[2], r[1], bits),
                  __builtin_amdgcn_alignbit(r[3], r[2], bits), __builtin_amdgcn_alignbit(0u, r[3], bits)};
    }
    if (dwords & 1) r = u32x4{r[1], r[2], r[3], 0u};
    if (dwords & 2) r = u32x4{r[2], r[3], 0u, 0u};
    return r;
}

// Rows of a finished tile in LDS to global memory, 16 bytes a lane.
template <typename T, int ROWS, int F, int THREADS, Access ACC>
__device__ __forceinline__ void put_rows(const char *t, __amdgpu_buffer_rsrc_t to, int stride, int rows, int width, int tid, int c0 = 0) {
    constexpr int kElems = 16 / sizeof(T), kPerRow = F / kElems, kStep = THREADS / kPerRow, N = (ROWS + kStep - 1) / kStep;
    const int c = tid % kPerRow;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int row = tid / kPerRow + n * kStep;
        if (ROWS % kStep != 0 && row >= ROWS) break;
        u32x4 x;
        if constexpr (sizeof(T) == 2) {
            const u32x2 lo = *(const u32x2 *)(t + Tile<T, ROWS, F>::at(row, 2 * c)), hi = *(const u32x2 *)(t + Tile<T, ROWS, F>::at(row, 2 * c + 1));
            x = u32x4{lo[0], lo[1], hi[0], hi[1]};
        } else {
            x = *(const u32x4 *)(t + Tile<T, ROWS, F>::at(row, c));
        }
        const int e = c0 + c * kElems, o = row < rows ? row * stride + e * (int)sizeof(T) : kOut;
        if (ACC != kElements) __builtin_amdgcn_raw_buffer_store_b128(x, to, e + kElems <= width ? o : kOut, 0, 0);
        if (ACC == kElements || (ACC == kAny && e < width && e + kElems > width)) {
#pragma unroll
            for (int k = 0; k < kElems; ++k) {
                const int w = e + k < width ? o + k * (int)sizeof(T) : kOut;
                if constexpr (sizeof(T) == 2) __builtin_amdgcn_raw_buffer_store_b16((short)(x[k / 2] >> (k % 2 * 16)), to, w, 0, 0);
                else __builtin_amdgcn_raw_buffer_store_b32(x[k], to, w, 0, 0);
            }
        }
    }
}

// A tile's way from global memory to LDS through registers: rows of `width` elements, `stride` bytes
// apart, from column c0 on; rows past `rows` and columns past `width` become 0.
template <typename T, int ROWS, int F, int THREADS, Access ACC>
struct Stage {
    static constexpr int kElems = 16 / sizeof(T), kPerRow = F / kElems, kStep = THREADS / kPerRow;
    static constexpr int N = (ROWS + kStep - 1) / kStep;
    static_assert(THREADS % kPerRow == 0, "a thread keeps its column");
    u32x4 r[N];
    __device__ __forceinline__ void load(const T *p, int stride, int rows, int width, int tid, int c0 = 0) {
        const int row = tid / kPerRow, c = c0 + tid % kPerRow * kElems;
        const __amdgpu_buffer_rsrc_t from = range_of(p, rows > 0 ? (int64_t)(rows - 1) * stride + width * (int64_t)sizeof(T) : 0);
        const int o = row * stride + c * (int)sizeof(T);
        if constexpr (ACC == kWide) {
            const int at = c < width ? o : kOut;
#pragma unroll
            for (int n = 0; n < N; ++n) r[n] = __builtin_amdgcn_raw_buffer_load_b128(from, at + n * kStep * stride, 0, 0);
        } else if constexpr (ACC == kAny) {
            // moved down when it is stored: the loads stay on their way
            const int first = min(c, width - kElems), at = c - first < kElems ? row * stride + first * (int)sizeof(T) : kOut;
#pragma unroll
            for (int n = 0; n < N; ++n) r[n] = __builtin_amdgcn_raw_buffer_load_b128(from, at + n * kStep * stride, 0, 0);
        } else {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                u32x4 got = {0, 0, 0, 0};
#pragma unroll
                for (int k = 0; k < kElems; ++k) {
                    const int at = c + k < width ? o + k * (int)sizeof(T) : kOut;
                    if constexpr (sizeof(T) == 2) got[k / 2] |= (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(from, at + n * kStep * stride, 0, 0) << (k % 2 * 16);
                    else got[k] = __builtin_amdgcn_raw_buffer_load_b32(from, at + n * kStep * stride, 0, 0);
                }
                r[n] = got;
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    // Of what was read; a vector that ends with its row may hold its neighbours.
    __device__ __forceinline__ bool not_finite() const {
        if constexpr (sizeof(T) == 2) {
            typedef short s16x2 __attribute__((ext_vector_type(2)));
            s16x2 most = {0, 0};
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) most = __builtin_elementwise_max(most, __builtin_bit_cast(s16x2, r[n][e] & 0x7fff7fffu));
            return most[0] >= 0x7f80 || most[1] >= 0x7f80;
        } else {
            float z = 0.0f;
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) z = __builtin_fmaf(__uint_as_float(r[n][e]), 0.0f, z);
            return z != z;
        }
    }
    __device__ __forceinline__ void store(char *t, int tid, int width, int c0 = 0) const {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int row = tid / kPerRow + n * kStep, c = tid % kPerRow;
            if (ROWS % kStep != 0 && row >= ROWS) break;
            u32x4 x = r[n];
            if constexpr (ACC == kAny) x = moved_down<T>(x, c0 + c * kElems - min(c0 + c * kElems, width - kElems));
            if constexpr (sizeof(T) == 2) {
                *(u32x2 *)(t + Tile<T, ROWS, F>::at(row, 2 * c)) = u32x2{x[0], x[1]};
                *(u32x2 *)(t + Tile<T, ROWS, F>::at(row, 2 * c + 1)) = u32x2{x[2], x[3]};
            } else {
                *(u32x4 *)(t + Tile<T, ROWS, F>::at(row, c)) = x;
            }
        }
    }
};

template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double x) {  // by DPP, 0 where no lane sends
    const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(x), CTRL, ROWS, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(x), CTRL, ROWS, 0xf, false);
    return __hiloint2double(hi, lo);
}
__device__ __forceinline__ double lane_of(double x, int lane) {
    return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(x), lane), __builtin_amdgcn_readlane(__double2loint(x), lane));
}

// 2^x to float32's last place: the raw instruction takes a float32 x, whose whole part would cost the
// fraction its bits, and gives no denormals.
__device__ __forceinline__ float exp2_of(double x) {
    const double n = __builtin_rint(x);
    return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f((float)(x - n)), (int)fmin(fmax(n, -1000.0), 1000.0));
}

// The decays of a chunk, made by one wave: G in units of log 2, document numbers, and the decays
// from the start to a token, from a token to the end, and over all of it.
template <int C>
struct Decays {
    double G[C];
    float start[C], end[C];
    int doc[C];
    float whole;
    int odd;  // something in the chunk is not finite

    __device__ __forceinline__ void make(float g, int lane) {
        const bool cut = g < kCut, bad = !(g < __builtin_inff());
        double sum = cut || bad ? 0.0 : (double)g * kLog2e;
        sum += moved<0x111, 0xf>(sum);  // inclusive: within rows of 16 lanes, then of the rows
        sum += moved<0x112, 0xf>(sum);
        sum += moved<0x114, 0xf>(sum);
        sum += moved<0x118, 0xf>(sum);
        sum += moved<0x142, 0xa>(sum);
        sum += moved<0x143, 0xc>(sum);
        const uint64_t cuts = __ballot(cut);
        const uint64_t until = ~0ull >> (63 - lane), upto = cuts & until;
        // a g of NaN or infinity is one for its document, from there on
        const uint64_t bads = __ballot(bad) & until;
        if (bads > upto) sum = __builtin_nan("");
        const double all = lane_of(sum, C - 1);
        if (lane < C) {
            G[lane] = sum;
            doc[lane] = __popcll(upto);
            start[lane] = upto ? 0.0f : exp2_of(sum);
            end[lane] = upto == cuts ? exp2_of(all - sum) : 0.0f;
            if (lane == 0) {
                whole = cuts ? 0.0f : exp2_of(all);
                odd = 0;
            }
        }
    }
    // the decay from token j to token i, 0 for j > i and across a cut
    __device__ __forceinline__ float between(double Gi, int di, double Gj, int dj, bool causal) const {
        return causal && di == dj ? __builtin_amdgcn_exp2f((float)(Gi - Gj)) : 0.0f;
    }
};

// NaN if one of these is not finite, else 0.
__device__ __forceinline__ float not_finite(const f32x16 &x) {
    float z = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) z = __builtin_fmaf(x[r], 0.0f, z);
    return z;
}
template <int N>
__device__ __forceinline__ bool any_not_finite(const bf16x8 (&x)[N]) {
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    s16x2 most = {0, 0};
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const u32x4 w = __builtin_bit_cast(u32x4, x[n]);
#pragma unroll
        for (int e = 0; e < 4; ++e) most = __builtin_elementwise_max(most, __builtin_bit_cast(s16x2, w[e] & 0x7fff7fffu));
    }
    return __ballot(most[0] >= 0x7f80 || most[1] >= 0x7f80) != 0;
}
template <int N>
__device__ __forceinline__ bool any_not_finite(const f32x4 (&x)[N]) {
    float z = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) z = __builtin_fmaf(x[n][e], 0.0f, z);
    return __ballot(z != z) != 0;
}

// What a chunk's products on the matrix cores make of a value that is not finite: a NaN wherever its weight is 0,
// before it and in other documents too. The sweep makes a chunk that has one pair by pair and token by token,
// without those that do not meet: acc (lanes: tokens, rows: 32 columns of `tile` from quad `first` on) gets the scores'
// products with the rows of the tile,
template <typename T, int C, int F, bool BELOW, int TT>
__device__ __forceinline__ void pairs_add(f32x16 (&acc)[TT], const char *scores, const char *tile, int first, const Decays<C> &dec,
                                          int l31, int half) {
#pragma unroll 1
    for (int n = 0; n < C; ++n) {
        f32x4 x[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) x[a] = Tile<T, C, F>::quad(tile, n, first + 2 * a + half);
#pragma unroll
        for (int j = 0; j < TT; ++j) {
            const int token = j * 32 + l31;
            const bool meet = (BELOW ? n <= token : n >= token) && dec.doc[n] == dec.doc[token];
            const float p = meet ? Scores<T, C, BELOW>::one(scores, token, n) : 0.0f;
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][r] += meet ? x[r / 4][r % 4] * p : 0.0f;
        }
        fence();
    }
}
// and a state the tokens of document `doc`.
template <typename T, int C, int FK, int FV, int TILES>
__device__ __forceinline__ void state_add_tokens(f32x16 (&S)[TILES], const char *k_tile, const char *v_tile, int column, const float *w,
                                                 const Decays<C> &dec, int doc, int half) {
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) S[t][r] = dec.whole == 0.0f ? 0.0f : S[t][r] * dec.whole;
#pragma unroll 1
    for (int n = 0; n < C; ++n) {
        if (__builtin_amdgcn_readfirstlane(dec.doc[n]) != doc) continue;
        const float v = w[n] * Tile<T, C, FV>::one(v_tile, n, column);
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const f32x4 k = Tile<T, C, FK>::quad(k_tile, n, t * 8 + 2 * a + half);
#pragma unroll
                for (int e = 0; e < 4; ++e) S[t][4 * a + e] += k[e] * v;
            }
            fence();
        }
    }
}

// The backward leaves out the tokens that have such a value, and gives their documents NaN in this chunk: where
// `spoilt` is NaN and, if the chunk's first is one, by the tokens' weights in what leaves the chunk. One thread a token.
template <typename T, int C, int KP, int VP>
__device__ __forceinline__ void take_out(char *qt, char *kt, char *vt, char *dt, const Decays<C> &dec, float *spoilt, float *back, int tid) {
    if (tid < C) {
        const auto row = [&](auto tile, char *t, bool clear) {
            typedef decltype(tile) Of;
            float z = 0.0f;
#pragma unroll 1
            for (int q = 0; q < Of::W; ++q) {
                const f32x4 x = Of::quad(t, tid, q);
#pragma unroll
                for (int e = 0; e < 4; ++e) z = __builtin_fmaf(x[e], 0.0f, z);
                if (clear) Of::put(t, tid, q, f32x4{0, 0, 0, 0});
            }
            return z;
        };
        const Tile<T, C, KP> keys;
        const Tile<T, C, VP> values;
        const float z = row(keys, qt, false) + row(keys, kt, false) + row(values, vt, false) + row(values, dt, false);
        const uint64_t bad = __ballot(z != z);  // of the first wave
        if (z != z) {
            row(keys, qt, true);
            row(keys, kt, true);
            row(values, vt, true);
            row(values, dt, true);
        }
        float mine = 0.0f;
#pragma unroll 1
        for (int n = 0; n < C; ++n) {
            const float x = bad >> n & 1 ? __builtin_nanf("") : 0.0f;
            if (dec.doc[n] == dec.doc[tid]) mine += x;
        }
        spoilt[tid] = mine;
        if (dec.doc[tid] == 0) back[tid] += mine;
    }
}

// b, head and piece of a block. Blocks of one XCD (every eighth) take neighbouring work, which
// shares q and k: heads of a group and slices of V.
__device__ __forceinline__ uint32_t work_of_block() {
    const uint32_t n = gridDim.x, id = blockIdx.x, x = id % 8, per = n / 8, rem = n % 8;
    return x * per + min(x, rem) + id / 8;
}

struct SweepArgs {
    const void *q, *k, *v;
    const float *g, *first;   // first: the entering state of every sequence (null: 0)
    const float *seg_in;      // the entering state of every segment, or null
    float *seg_out, *seg_fac;  // the state pass: what a segment adds, and its decay
    void *o;
    float *last, *states;
    int64_t L, g_batch, g_token;  // strides of g (0, 0 for [H])
    int32_t H, Hk, K, V, nseg, nchunk, per_seg, slices;
    float scale;
    bool reverse;             // the state pass runs from the end, with weights scale e^{G_i}
};

// A state [K][V] and an accumulator whose lanes are columns of V: row 32 t + 8 (r / 4) + 4 half + r % 4.
template <int TILES>
__device__ __forceinline__ void state_load(f32x16 (&S)[TILES], const float *p, int K, int V, int v, int half) {
    const __amdgpu_buffer_rsrc_t from = range_of(p, p ? (int64_t)K * V * 4 : 0);
    const int at = v < V ? (4 * half * V + v) * 4 : kOut;
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            S[t][r] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(from, at + (t * 32 + 8 * (r / 4) + r % 4) * V * 4, 0, 0));
}
template <int TILES>
__device__ __forceinline__ void state_store(const f32x16 (&S)[TILES], float *p, int K, int V, int v, int half) {
    const __amdgpu_buffer_rsrc_t to = range_of(p, (int64_t)K * V * 4);
    const int at = v < V ? (4 * half * V + v) * 4 : kOut;
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[t][r]), to, at + (t * 32 + 8 * (r / 4) + r % 4) * V * 4, 0, 0);
}

// S = whole S + sum over the chunk's tokens of w_j k_j v_j^T: k by columns of its tile, the wave's v
// fragments weighed in float32 and split.
template <typename T, int C, int KP, int TILES>
__device__ __forceinline__ void state_add(f32x16 (&S)[TILES], const char *k_tile, const typename Kind<T>::Frag *v,
                                          const float *w, float whole, int half, int columns) {
    typedef Kind<T> N;
    if (__builtin_amdgcn_readfirstlane(__float_as_int(whole)) == 0) {
#pragma unroll
        for (int t = 0; t < TILES; ++t) S[t] = f32x16{};
    } else {
#pragma unroll
        for (int t = 0; t < TILES; ++t) S[t] *= whole;
    }
#pragma unroll
    for (int s = 0; s < C / N::KS; ++s) {
        typename N::Wide wv;
        weights_of(w, s, half, wv);
        typename N::Frag part[N::kParts];
        split(widened(v[s]) * wv, part);
        typename N::Frag a[TILES];
#pragma unroll
        for (int t = 0; t < TILES; ++t) a[t] = Tile<T, C, KP>::by_column(k_tile, columns, t, s);
#pragma unroll
        for (int p = 0; p < N::kParts; ++p)
#pragma unroll
            for (int t = 0; t < TILES; ++t) S[t] = mfma(a[t], part[p], S[t]);
        fence();
    }
}

// One sweep over a segment of a sequence's chunks for NW x 32 columns of one head's state. OUT: with
// outputs, from the segment's entering state; else what the segment adds to the state, from 0. A wave has all
// of K for its 32 columns, so its state never leaves the accumulators; the block's waves share the chunk's q, k
// and scores in LDS, and two blocks share a compute unit so that one's products run beside the other's decays
// and roundings. Those vector instructions and the reads of LDS bound it (busy 53 % and 41 % of the time, the matrix
// cores 32 %): 262144 tokens x 32 heads of 128 x 128 in bf16, 2.48 ms with outputs and 1.11 without, for 1.2 ms
// of bytes; 2 x 4096 tokens 108 and 44 us.
template <typename T, int KP, int NW, bool OUT, Access ACC>
__global__ void __launch_bounds__(64 * NW, 2) k_sweep(SweepArgs p) {
    typedef Kind<T> N;
    typedef typename N::Frag Frag;
    constexpr int C = N::C, KS = N::KS, VT = 32 * NW, TT = C / 32, KT = KP / 32, THREADS = 64 * NW;
    typedef Tile<T, C, KP> TK;
    typedef Tile<T, C, VT> TV;
    typedef Scores<T, C, true> TP;
    __shared__ __attribute__((aligned(256))) char lds[(OUT ? 2 : 1) * TK::kBytes + (OUT ? 2 : 1) * TV::kBytes + (OUT ? TP::kBytes : 0)];
    __shared__ Decays<C> decays[2];
    char *const kt = lds, *const vt = lds + TK::kBytes, *const qt = vt + TV::kBytes, *const pt = qt + TK::kBytes, *const ot = pt + TP::kBytes;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t work = work_of_block();
    const int slice = work % p.slices;
    work /= p.slices;
    const int share = p.H / p.Hk, sub = work % share;
    work /= share;
    int seg = work % p.nseg;
    work /= p.nseg;
    if (!OUT && p.reverse) seg += 1;  // a pass covers all segments but the one that nothing follows
    const int hk = work % p.Hk, h = hk * share + sub;
    const int64_t b = work / p.Hk, bh = b * p.H + h;
    const int c0 = seg * p.per_seg, c1 = min(c0 + p.per_seg, p.nchunk), n = c1 - c0;
    const int v0 = slice * VT;
    const int64_t KV = (int64_t)p.K * p.V;
    const int nseg_all = OUT ? p.nseg : p.nseg + 1;

    int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, l31 = lane & 31, vcol = v0 + wave * 32 + l31;
    f32x16 S[KT];
    {
        const float *from = nullptr;
        if (OUT) from = p.seg_in ? p.seg_in + (bh * nseg_all + seg) * KV : p.first ? p.first + bh * KV : nullptr;
        state_load<KT>(S, from, p.K, p.V, vcol, half);
    }
    Stage<T, C, KP, THREADS, ACC> kr, qr;
    Stage<T, C, VT, THREADS, ACC> vr;
    const int ks = p.Hk * p.K * (int)sizeof(T), vs = p.H * p.V * (int)sizeof(T);  // bytes of a token
    const bool rev = !OUT && p.reverse;
    const auto chunk = [&](int it) { return rev ? c1 - 1 - it : c0 + it; };
    const auto rows_at = [&](int c) { return (int)min((int64_t)C, p.L - (int64_t)c * C); };
    // Past the last chunk nothing is read, but the registers are written: a fetch that is left out would keep
    // their old contents alive through a chunk.
    auto fetch = [&](int it) {
        const int c = chunk(min(it, n - 1)), rows = it < n ? rows_at(c) : 0;
        const int64_t at = b * p.L + (int64_t)c * C;
        kr.load((const T *)((const char *)p.k + at * ks) + (int64_t)hk * p.K, ks, rows, p.K, tid);
        vr.load((const T *)((const char *)p.v + at * vs) + (int64_t)h * p.V, vs, rows, p.V, tid, v0);
        if (OUT) qr.load((const T *)((const char *)p.q + at * ks) + (int64_t)hk * p.K, ks, rows, p.K, tid);
    };
    // One wave makes the decays, a chunk ahead, from a g that was loaded another chunk ahead.
    const bool decides = wave == NW - 1;
    float g = 0.0f;
    const auto load_g = [&](int it) {
        if (it >= n) return;
        const int c = chunk(it);
        const int64_t t = (int64_t)c * C + lane;
        g = lane < rows_at(c) ? p.g[b * p.g_batch + t * p.g_token + h] : 0.0f;
    };
    const auto decide = [&](int it) {
        Decays<C> &d = decays[it & 1];
        d.make(g, lane);
        if (rev && lane < C) d.start[lane] *= p.scale;
    };
    // The outputs of a chunk wait in LDS until the next one's loads are due: stores that are issued before
    // loads are not waited for with them.
    const auto put_outputs = [&](int c) {
        const int rows = rows_at(c);
        put_rows<T, C, VT, THREADS, ACC>(ot, range_of((const char *)p.o + (b * p.L + (int64_t)c * C) * vs + (int64_t)h * p.V * (int)sizeof(T),
                                                      (int64_t)(rows - 1) * vs + p.V * (int64_t)sizeof(T)),
                                         vs, rows, p.V, tid, v0);
    };
    if (n > 0) {
        if (decides) {
            load_g(0);
            decide(0);
            load_g(1);
        }
        fetch(0);
    }
    double decayed = 0.0;  // the sum of G over the segment, in units of log 2
    bool cut = false;
    for (int it = 0; it < n; ++it) {
        const int c = chunk(it);
        // Lanes' addresses are made anew in every chunk: kept over the loop, they fill the registers.
        asm volatile("" : "+v"(tid));
        lane = tid & 63;
        half = lane >> 5;
        l31 = lane & 31;
        vcol = v0 + wave * 32 + l31;
        const Decays<C> &dec = decays[it & 1];
        kr.store(kt, tid, p.K);
        vr.store(vt, tid, p.V, v0);
        if (OUT) qr.store(qt, tid, p.K);
        __syncthreads();
        if (OUT) {
            if (p.states) state_store<KT>(S, p.states + (bh * p.nchunk + c) * KV, p.K, p.V, vcol, half);
            if (it > 0) put_outputs(c - 1);
        }
        fetch(it + 1);
        if (decides && it + 1 < n) {
            decide(it + 1);
            load_g(it + 2);
        }
        const int kcol = TK::column_base(lane), krow = TK::at(l31, half), prow = TP::at(l31, half);
        constexpr int kDown = 32 * TK::kBytes / C;  // 32 rows further
        if (OUT) {
            // scores q k^T e^{G_i - G_j}, lanes i, in quads of j
            for (int t = wave; t < TT * (TT + 1) / 2; t += NW) {
                const int it2 = t > 0, jt = t == 2, i = it2 * 32 + l31;
                f32x16 acc = {};
#pragma unroll
                for (int s = 0; s < KP / KS; ++s) {
                    acc = mfma(TK::by_row(kt + jt * kDown, krow, s), TK::by_row(qt + it2 * kDown, krow, s), acc);
                    if (s % 4 == 3) fence();
                }
                if (it2 == jt) {  // every token's q and k are in these
                    const float z = not_finite(acc);
                    if (z != z) decays[it & 1].odd = 1;
                }
                const double Gi = dec.G[i];
                const int di = dec.doc[i];
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    f32x4 x;
                    const int j0 = jt * 32 + 8 * a + 4 * half;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[e] = acc[4 * a + e] * (p.scale * dec.between(Gi, di, dec.G[j0 + e], dec.doc[j0 + e], j0 + e <= i));
                    TP::put(pt, i, j0 / 4, x);
                    fence();
                }
            }
            __syncthreads();
        }
        Frag v[C / KS];
        {
            const int vcolumn = TV::column_base(lane);
#pragma unroll
            for (int s = 0; s < C / KS; ++s) v[s] = TV::by_column(vt, vcolumn ^ (wave * 32 * (int)sizeof(T)), 0, s);
        }
        const bool odd = OUT && (__builtin_amdgcn_readfirstlane(dec.odd) != 0 || any_not_finite(v));
        if (OUT) {
            f32x16 o[TT] = {};
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int s = 0; s < 32 / KS; ++s) {
                    Frag a[N::kOut];
                    split(rows_of<T>(S[t], s), a);
                    Frag f[TT];
#pragma unroll
                    for (int i = 0; i < TT; ++i) f[i] = TK::by_row(qt + i * kDown, krow, t * (32 / KS) + s);
#pragma unroll
                    for (int e = 0; e < N::kOut; ++e)
#pragma unroll
                        for (int i = 0; i < TT; ++i) o[i] = mfma(a[e], f[i], o[i]);
                    if (s % 2) fence();
                }
#pragma unroll
            for (int i = 0; i < TT; ++i) {
                const float w = dec.start[i * 32 + l31] * p.scale;
#pragma unroll
                for (int r = 0; r < 16; ++r) o[i][r] = w == 0.0f ? 0.0f : o[i][r] * w;
            }
            if (odd) {
                pairs_add<T, C, VT, true>(o, pt, vt, wave * 8, dec, l31, half);
            } else {
#pragma unroll
                for (int s = 0; s < C / KS; ++s)
#pragma unroll
                    for (int e = 0; e < N::kOut; ++e)
#pragma unroll
                        for (int i = s / (32 / KS); i < TT; ++i) o[i] = mfma(v[s], TP::by_row(pt, prow, i, s, e), o[i]);
            }
#pragma unroll
            for (int i = 0; i < TT; ++i) {
#pragma unroll
                for (int a = 0; a < 4; ++a)
                    TV::put(ot, i * 32 + l31, wave * 8 + 2 * a + half, f32x4{o[i][4 * a], o[i][4 * a + 1], o[i][4 * a + 2], o[i][4 * a + 3]});
                fence();
            }
        }
        const float *const weights = rev ? dec.start : dec.end;
        const auto by_token = [&] { state_add_tokens<T, C, KP, VT>(S, kt, vt, wave * 32 + l31, weights, dec, rev ? 0 : dec.doc[C - 1], half); };
        if (odd) by_token();
        else state_add<T, C, KP, KT>(S, kt, v, weights, dec.whole, half, kcol);
        if (!OUT && dec.whole == 0.0f) {  // else every token is of the document that goes on
            float z = 0.0f;
#pragma unroll
            for (int t = 0; t < KT; ++t) z += not_finite(S[t]);
            if (__ballot(z != z)) by_token();
        }
        if (!OUT) {
            decayed += dec.G[C - 1];
            cut |= dec.whole == 0.0f;
        }
        __syncthreads();
    }
    if (OUT) {
        if (n > 0) put_outputs(c1 - 1);
        if (p.last && seg == p.nseg - 1) state_store<KT>(S, p.last + bh * KV, p.K, p.V, vcol, half);
    } else {
        const int64_t at = bh * nseg_all + seg;
        state_store<KT>(S, p.seg_out + at * KV, p.K, p.V, vcol, half);
        if (threadIdx.x == 0 && slice == 0) p.seg_fac[at] = cut ? 0.0f : exp2_of(decayed);
    }
}

// What the segments add becomes what enters them (forwards), or what comes back to them (reverse). Bound by the
// bytes of the segments' states: 64 heads of 128 x 128 in 7 segments, 59 MB, 11 us (5 TB/s).
__global__ void __launch_bounds__(256) k_join(float *seg, const float *fac, const float *first, int64_t KV, int64_t heads,
                                              int nseg, bool reverse) {
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= heads * KV) return;
    const int64_t bh = e / KV, at = e % KV;
    float cur = first ? first[e] : 0.0f;
    constexpr int N = 8;  // loads at once
    for (int i0 = 0; i0 < nseg; i0 += N) {
        float add[N], f[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int s = reverse ? nseg - 1 - (i0 + k) : i0 + k;
            const bool there = i0 + k + 1 < nseg;  // what the last one adds is not asked for
            add[k] = there ? seg[(bh * nseg + s) * KV + at] : 0.0f;
            f[k] = there ? fac[bh * nseg + s] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (i0 + k >= nseg) break;
            const int s = reverse ? nseg - 1 - (i0 + k) : i0 + k;
            seg[(bh * nseg + s) * KV + at] = cur;
            cur = f[k] == 0.0f ? add[k] : f[k] * cur + add[k];
        }
    }
}

struct BwdArgs {
    const void *q, *k, *v, *do_;
    const float *g, *states, *seg_in, *dlast;
    void *dq, *dk, *dv;  // dq, dk: of T [B, L, Hk, K], or float32 [B, L, H, K] where heads share
    float *dg, *dfirst;  // dg [B, L, H]
    int64_t L, g_batch, g_token;
    int32_t H, Hk, K, V, nseg, nchunk, per_seg;
    float scale;
};

// The gradients of a segment, from its end. VP / 32 waves hold dS by columns of V and make dv;
// KP / 32 waves hold it transposed, by columns of K, and make dk and dq: each role's gradients need dS as an
// operand in another order, and holding it twice costs a product where turning it around costs LDS that is
// already full. A chunk's tiles take 157 KB of LDS with all heads of 128, so a block has the compute unit to
// itself, and what bounds it are vector and LDS instructions between its barriers (busy 47 % and 27 % of the time, the
// matrix cores 25 %): 2 x 4096 tokens x 32 heads of 128 x 128 in bf16, 265 us (740 MB with states, 2.8 TB/s).
template <typename T, int KP, int VP, Access ACC>
__global__ void __launch_bounds__(2 * (KP + VP)) k_bwd(BwdArgs p) {
    typedef Kind<T> N;
    typedef typename N::Frag Frag;
    constexpr int C = N::C, KS = N::KS, TT = C / 32, KT = KP / 32, VW = VP / 32, NW = KT + VW, THREADS = 64 * NW;
    constexpr int kMost = KT > VW ? KT : VW;
    typedef Tile<T, C, KP> TK;
    typedef Tile<T, C, VP> TV;
    typedef Scores<T, C, true> TP;   // rows i
    typedef Scores<T, C, false> TQ;  // rows j
    typedef Tile<float, C, C> TM;
    __shared__ __attribute__((aligned(256))) char lds[3 * TK::kBytes + 3 * TV::kBytes + TP::kBytes + 2 * TQ::kBytes + TM::kBytes];
    __shared__ Decays<C> decays[2];
    __shared__ float backs[2][C];         // scale e^{G_i}
    __shared__ float came[KT][C], left[KT][C], through[KT];
    __shared__ float spoilt[C];           // NaN for the tokens of a document that has a value that is not finite
    char *const qt = lds, *const kt = qt + TK::kBytes, *const vt = kt + TK::kBytes, *const dt = vt + TV::kBytes;
    char *const at = dt + TV::kBytes, *const bt = at + TQ::kBytes, *const bn = bt + TQ::kBytes, *const mt = bn + TP::kBytes;
    char *const ov = mt + TM::kBytes, *const oq = ov + TV::kBytes;  // dv and dq on their way out

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    uint32_t work = work_of_block();
    const int share = p.H / p.Hk, sub = work % share;
    work /= share;
    const int seg = work % p.nseg;
    work /= p.nseg;
    const int hk = work % p.Hk, h = hk * share + sub;
    const int64_t b = work / p.Hk, bh = b * p.H + h;
    const int c0 = seg * p.per_seg, c1 = min(c0 + p.per_seg, p.nchunk), n = c1 - c0;
    const int64_t KV = (int64_t)p.K * p.V;
    const bool of_v = wave < VW;          // this wave makes dv
    const int part = of_v ? wave : wave - VW;
    int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, l31 = lane & 31;

    f32x16 S[kMost];                      // dS [k rows][col of V], or dS^T [v rows][col of K]
    f32x16(&SV)[KT] = reinterpret_cast<f32x16(&)[KT]>(S);
    f32x16(&SK)[VW] = reinterpret_cast<f32x16(&)[VW]>(S);
    {
        const float *from = p.seg_in ? p.seg_in + (bh * p.nseg + seg) * KV : p.dlast ? p.dlast + bh * KV : nullptr;
        if (of_v) {
            state_load<KT>(SV, from, p.K, p.V, part * 32 + l31, half);
        } else {
            const __amdgpu_buffer_rsrc_t rows = range_of(from, from ? KV * 4 : 0);
            const int at = ((part * 32 + l31) * p.V + 4 * half) * 4;
#pragma unroll
            for (int t = 0; t < VW; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int v = t * 32 + 8 * (r / 4) + r % 4;
                    SK[t][r] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rows, v + 4 * half < p.V ? at + 4 * v : kOut, 0, 0));
                }
        }
    }
    Stage<T, C, KP, THREADS, ACC> qr, kr;
    Stage<T, C, VP, THREADS, ACC> vr, dr;
    const int ks = p.Hk * p.K * (int)sizeof(T), vs = p.H * p.V * (int)sizeof(T);  // bytes of a token
    const bool shared = share > 1;
    const int ksz = shared ? 4 : (int)sizeof(T), dks = shared ? p.H * p.K * 4 : ks;  // of an element and a token of dq and dk
    const auto rows_at = [&](int c) { return (int)min((int64_t)C, p.L - (int64_t)c * C); };
    auto fetch = [&](int next) {
        const int c = max(next, c0), rows = next >= c0 ? rows_at(c) : 0;
        const int64_t from = b * p.L + (int64_t)c * C;
        qr.load((const T *)((const char *)p.q + from * ks) + (int64_t)hk * p.K, ks, rows, p.K, tid);
        kr.load((const T *)((const char *)p.k + from * ks) + (int64_t)hk * p.K, ks, rows, p.K, tid);
        vr.load((const T *)((const char *)p.v + from * vs) + (int64_t)h * p.V, vs, rows, p.V, tid);
        dr.load((const T *)((const char *)p.do_ + from * vs) + (int64_t)h * p.V, vs, rows, p.V, tid);
    };
    const auto range_v = [&](int c) {
        return range_of((const char *)p.dv + (b * p.L + (int64_t)c * C) * vs + (int64_t)h * p.V * (int)sizeof(T),
                        (int64_t)(rows_at(c) - 1) * vs + p.V * (int64_t)sizeof(T));
    };
    const auto range_k = [&](void *out, int c) {
        return range_of((const char *)out + (b * p.L + (int64_t)c * C) * dks + (int64_t)(shared ? h : hk) * p.K * ksz,
                        (int64_t)(rows_at(c) - 1) * dks + p.K * (int64_t)ksz);
    };
    // As in the sweep: dv and dq (of T) wait in LDS until the next chunk's loads are due.
    const auto put_outputs = [&](int c) {
        put_rows<T, C, VP, THREADS, ACC>(ov, range_v(c), vs, rows_at(c), p.V, tid);
        if (!shared) put_rows<T, C, KP, THREADS, ACC>(oq, range_k(p.dq, c), dks, rows_at(c), p.K, tid);
    };
    // And one wave makes the decays a chunk ahead.
    const bool decides = wave == VW - 1;
    float g = 0.0f;
    const auto load_g = [&](int c) {
        if (c >= c0) g = lane < rows_at(c) ? p.g[b * p.g_batch + ((int64_t)c * C + lane) * p.g_token + h] : 0.0f;
    };
    const auto decide = [&](int c) {
        decays[c & 1].make(g, lane);
        if (lane < C) backs[c & 1][lane] = decays[c & 1].start[lane] * p.scale;
    };
    if (n > 0) {
        if (decides) {
            load_g(c1 - 1);
            decide(c1 - 1);
            load_g(c1 - 2);
        }
        fetch(c1 - 1);
        __syncthreads();  // the decays say that nothing is odd before a lane may say so
    }
    for (int c = c1 - 1; c >= c0; --c) {
        const int64_t t0 = (int64_t)c * C;
        const int rows = rows_at(c);
        const Decays<C> &dec = decays[c & 1];
        const float *const back = backs[c & 1];
        asm volatile("" : "+v"(tid));  // addresses are made anew, as in the sweep
        lane = tid & 63;
        half = lane >> 5;
        l31 = lane & 31;
        qr.store(qt, tid, p.K);
        kr.store(kt, tid, p.K);
        vr.store(vt, tid, p.V);
        dr.store(dt, tid, p.V);
        if (qr.not_finite() || kr.not_finite() || vr.not_finite() || dr.not_finite()) decays[c & 1].odd = 1;
        __syncthreads();
        const bool odd = __builtin_amdgcn_readfirstlane(dec.odd) != 0;
        if (odd) {  // is made without the tokens that have it; what is left of their documents is spoilt at the end
            take_out<T, C, KP, VP>(qt, kt, vt, dt, dec, spoilt, backs[c & 1], tid);
            __syncthreads();
        }
        if (c + 1 < c1) put_outputs(c + 1);
        constexpr int kDown = 32 * TK::kBytes / C, vDown = 32 * TV::kBytes / C;  // 32 rows further
        const int krow = TK::at(l31, half), vrow = TV::at(l31, half), prow = TP::at(l31, half);
        // The state that entered this chunk, lanes k, in quads of v; half of V at a time.
        constexpr int kIn = VW * 2;
        f32x4 in[kIn];
        const auto load_in = [&](int part_v) {
            const __amdgpu_buffer_rsrc_t from = range_of(p.states + (bh * p.nchunk + c) * KV, KV * 4);
            const int at = ((part * 32 + l31) * p.V + 4 * half) * 4;
#pragma unroll
            for (int a = 0; a < kIn; ++a) {
                const int v = 8 * (a + part_v * kIn) + 4 * half;
                if constexpr (ACC == kWide) {
                    in[a] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(from, v < p.V ? at + 32 * (a + part_v * kIn) : kOut, 0, 0));
                } else if constexpr (ACC == kAny) {
                    const int first = min(v, p.V - 4);
                    in[a] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(from, v < p.V ? at + 4 * (first - 4 * half) : kOut, 0, 0));
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        in[a][e] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(from, v + e < p.V ? at + 32 * (a + part_v * kIn) + 4 * e : kOut, 0, 0));
                }
            }
        };
        if (!of_v) load_in(0);
        // Scores: q k^T and do v^T with their decays. Tiles below the diagonal, each twice: lanes j
        // (both products, and theirs for dg), and lanes i (do v^T).
        for (int task = wave; task < TT * (TT + 1); task += NW) {
            const int t = task >> 1, it = t > 0, jt = t == 2;
            if (task & 1) {
                const int i = it * 32 + l31;
                f32x16 acc = {};
#pragma unroll
                for (int s = 0; s < VP / KS; ++s) {
                    acc = mfma(TV::by_row(vt + jt * vDown, vrow, s), TV::by_row(dt + it * vDown, vrow, s), acc);
                    if (s % 4 == 3) fence();
                }
                const double Gi = dec.G[i];
                const int di = dec.doc[i];
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    f32x4 x;
                    const int j0 = jt * 32 + 8 * a + 4 * half;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[e] = acc[4 * a + e] * (p.scale * dec.between(Gi, di, dec.G[j0 + e], dec.doc[j0 + e], j0 + e <= i));
                    TP::put(bn, i, j0 / 4, x);
                    fence();
                }
            } else {
                const int j = jt * 32 + l31;
                f32x16 qk = {}, dov = {};
#pragma unroll
                for (int s = 0; s < KP / KS; ++s) {
                    qk = mfma(TK::by_row(qt + it * kDown, krow, s), TK::by_row(kt + jt * kDown, krow, s), qk);
                    if (s % 4 == 3) fence();
                }
#pragma unroll
                for (int s = 0; s < VP / KS; ++s) {
                    dov = mfma(TV::by_row(dt + it * vDown, vrow, s), TV::by_row(vt + jt * vDown, vrow, s), dov);
                    if (s % 4 == 3) fence();
                }
                const double Gj = dec.G[j];
                const int dj = dec.doc[j];
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    f32x4 x, y, m;
                    const int i0 = it * 32 + 8 * a + 4 * half;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float w = p.scale * dec.between(dec.G[i0 + e], dec.doc[i0 + e], Gj, dj, j <= i0 + e);
                        x[e] = qk[4 * a + e] * w;
                        y[e] = dov[4 * a + e] * w;
                        m[e] = j < i0 + e && w != 0.0f ? x[e] * dov[4 * a + e] : 0.0f;
                    }
                    TQ::put(at, j, i0 / 4, x);
                    TQ::put(bt, j, i0 / 4, y);
                    TM::put(mt, j, i0 / 4, m);
                    fence();
                }
            }
        }
        __syncthreads();
        const int kcol = TK::column_base(lane), vcol = TV::column_base(lane);
        float pairs = 0.0f;
        if (of_v) {
            if (decides && c > c0) {
                decide(c - 1);
                load_g(c - 2);
            }
            f32x16 acc[TT] = {};
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int s = 0; s < 32 / KS; ++s) {
                    Frag a[N::kOut];
                    split(rows_of<T>(SV[t], s), a);
#pragma unroll
                    for (int j = 0; j < TT; ++j) {
                        const Frag f = TK::by_row(kt + j * kDown, krow, t * (32 / KS) + s);
#pragma unroll
                        for (int e = 0; e < N::kOut; ++e) acc[j] = mfma(a[e], f, acc[j]);
                    }
                    if (s % 2) fence();
                }
            Frag d[C / KS];
#pragma unroll
            for (int s = 0; s < C / KS; ++s) d[s] = TV::by_column(dt, vcol ^ (part * 32 * (int)sizeof(T)), 0, s);
#pragma unroll
            for (int j = 0; j < TT; ++j) {
                const float w = dec.end[j * 32 + l31];
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[j][r] = w == 0.0f ? 0.0f : acc[j][r] * w;
#pragma unroll
                for (int s = j * (32 / KS); s < C / KS; ++s)
#pragma unroll
                    for (int e = 0; e < N::kOut; ++e) acc[j] = mfma(d[s], TQ::by_row(at, prow, j, s, e), acc[j]);
#pragma unroll
                for (int a = 0; a < 4; ++a)
                    TV::put(ov, j * 32 + l31, part * 8 + 2 * a + half, f32x4{acc[j][4 * a], acc[j][4 * a + 1], acc[j][4 * a + 2], acc[j][4 * a + 3]});
                fence();
            }
            if (wave == 0) {
                // dg's pairs. Row j becomes its sums from i on; then token t adds the rows before it.
                if (lane < C) {
                    float sum = 0.0f;
                    for (int a = C / 4 - 1; a >= 0; --a) {
                        f32x4 *const q4 = (f32x4 *)(mt + TM::at(lane, a));
                        f32x4 m = *q4;
#pragma unroll
                        for (int e = 3; e >= 0; --e) {
                            sum += m[e];
                            m[e] = sum;
                        }
                        *q4 = m;
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
                if (lane < C)
#pragma unroll 8
                    for (int j = 0; j < C - 1; ++j) {
                        const float m = *(const float *)(mt + TM::at(j, lane >> 2) + (lane & 3) * 4);
                        pairs += j < lane ? m : 0.0f;
                    }
            }
        } else {
            // What of dq comes from earlier chunks and what of dk comes from later ones, each with its share of
            // dg before the chunk's own part is added. The entering state is read in halves, so that its
            // second half and the next chunk's tiles are on their way while others are worked on.
            const auto own = [&](f32x16(&acc)[TT], const char *tile, const float *decay, float *share_of) {
#pragma unroll
                for (int j = 0; j < TT; ++j) {
                    const float w = decay[j * 32 + l31];
                    float sum = 0.0f;
#pragma unroll
                    for (int s = 0; s < 32 / KS; ++s) {  // this wave's 32 columns of k or q, in quads
                        const typename N::Wide x = widened(TK::by_row(tile + j * kDown, krow ^ (part * 32 * (int)sizeof(T)), s));
                        constexpr int E = sizeof(x) / 4;
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            const float r = w == 0.0f ? 0.0f : acc[j][s * E + e] * w;
                            acc[j][s * E + e] = r;
                            sum += x[e] * r;
                        }
                    }
                    sum += __shfl_xor(sum, 32);
                    if (half == 0) share_of[j * 32 + l31] = w == 0.0f ? 0.0f : sum;
                }
            };
            const auto put = [&](const f32x16(&acc)[TT], void *out) {
                const __amdgpu_buffer_rsrc_t to = range_k(out, c);
#pragma unroll
                for (int j = 0; j < TT; ++j) {
                    const int row = j * 32 + l31, width = row < rows ? p.K : 0;
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        const int e = part * 32 + 8 * a + 4 * half;
                        const f32x4 x = {acc[j][4 * a], acc[j][4 * a + 1], acc[j][4 * a + 2], acc[j][4 * a + 3]};
                        if (!shared) put_quad<T, ACC>(to, row * dks, e, width, x);
                        else put_quad<float, ACC>(to, row * dks, e, width, x);
                    }
                    fence();
                }
            };
            constexpr int Q = sizeof(typename N::Wide) / 16;  // quads of a fragment
            float x = 0.0f;
            const int column = kcol ^ (part * 32 * (int)sizeof(T));
            f32x16 aq[TT] = {};
            const auto add_in = [&](int part_v) {  // half of V's share of dq
#pragma unroll
                for (int t = 0; t < VW / 2; ++t)
#pragma unroll
                    for (int s = 0; s < 32 / KS; ++s) {
                        const typename N::Wide w = rows_of<T>(SK[t + part_v * (VW / 2)], s);
                        typename N::Wide u;
#pragma unroll
                        for (int e = 0; e < Q; ++e) {
                            const int a = (t * (32 / KS) + s) * Q + e, v = 8 * (a + part_v * kIn) + 4 * half;
                            f32x4 y = in[a];  // moved down here, not where it is waited for
                            if (ACC == kAny) y = __builtin_bit_cast(f32x4, moved_down<float>(__builtin_bit_cast(u32x4, y), v - min(v, p.V - 4)));
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                u[4 * e + k] = y[k];
                                x += y[k] * w[4 * e + k];
                            }
                        }
                        Frag pq[N::kParts];
                        split(u, pq);
#pragma unroll
                        for (int j = 0; j < TT; ++j) {
                            const Frag f = TV::by_row(dt + j * vDown, vrow, (t + part_v * (VW / 2)) * (32 / KS) + s);
#pragma unroll
                            for (int e = 0; e < N::kParts; ++e) aq[j] = mfma(pq[e], f, aq[j]);
                        }
                        fence();
                    }
            };
            add_in(0);
            load_in(1);
            fence();
            {
                f32x16 acc[TT] = {};
#pragma unroll
                for (int t = 0; t < VW; ++t)
#pragma unroll
                    for (int s = 0; s < 32 / KS; ++s) {
                        const typename N::Wide w = rows_of<T>(SK[t], s);
                        Frag pk[N::kParts];
                        split(w, pk);
#pragma unroll
                        for (int j = 0; j < TT; ++j) {
                            const Frag f = TV::by_row(vt + j * vDown, vrow, t * (32 / KS) + s);
#pragma unroll
                            for (int e = 0; e < N::kParts; ++e) acc[j] = mfma(pk[e], f, acc[j]);
                        }
                        fence();
                    }
                own(acc, kt, dec.end, left[part]);
#pragma unroll
                for (int s = 0; s < C / KS; ++s) {
                    const Frag f = TK::by_column(qt, column, 0, s);
#pragma unroll
                    for (int j = 0; j <= s / (32 / KS); ++j)
#pragma unroll
                        for (int e = 0; e < N::kOut; ++e) acc[j] = mfma(f, TQ::by_row(bt, prow, j, s, e), acc[j]);
                }
                put(acc, p.dk);
            }
            add_in(1);
            own(aq, qt, back, came[part]);
#pragma unroll
            for (int s = 0; s < C / KS; ++s) {
                const Frag f = TK::by_column(kt, column, 0, s);
#pragma unroll
                for (int j = s / (32 / KS); j < TT; ++j)
#pragma unroll
                    for (int e = 0; e < N::kOut; ++e) aq[j] = mfma(f, TP::by_row(bn, prow, j, s, e), aq[j]);
            }
            if (shared) {
                put(aq, p.dq);
            } else {
#pragma unroll
                for (int j = 0; j < TT; ++j)
#pragma unroll
                    for (int a = 0; a < 4; ++a)
                        TK::put(oq, j * 32 + l31, part * 8 + 2 * a + half, f32x4{aq[j][4 * a], aq[j][4 * a + 1], aq[j][4 * a + 2], aq[j][4 * a + 3]});
            }
            fence();
#pragma unroll
            for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d);
            if (lane == 0) through[part] = dec.whole == 0.0f ? 0.0f : x * dec.whole;
        }
        // Here the roles meet, so that the next chunk's registers are the same ones in both.
        fence();
        fetch(c - 1);
        fence();
        Frag f[C / KS];
        if (of_v) {
#pragma unroll
            for (int s = 0; s < C / KS; ++s) f[s] = TV::by_column(dt, vcol ^ (part * 32 * (int)sizeof(T)), 0, s);
            state_add<T, C, KP, KT>(SV, qt, f, back, dec.whole, half, kcol);
        } else {
#pragma unroll
            for (int s = 0; s < C / KS; ++s) f[s] = TK::by_column(qt, kcol ^ (part * 32 * (int)sizeof(T)), 0, s);
            state_add<T, C, VP, VW>(SK, dt, f, back, dec.whole, half, vcol);
        }
        __syncthreads();
        if (odd) {  // over what has been written: dk, and dq of shared heads, are in memory, the others wait in LDS
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "agent");  // other lanes write it again
            __syncthreads();
            for (int r = wave; r < rows; r += NW) {
                const float x = spoilt[r];
                if (x == 0.0f) continue;
                const f32x4 quad = {x, x, x, x};
                if (lane < VP / 4) TV::put(ov, r, lane, quad);
                if (lane < KP / 4 && !shared) TK::put(oq, r, lane, quad);
                for (int e = lane; e < p.K; e += 64) {
                    if (shared) {
                        *(float *)((char *)p.dk + ((b * p.L + t0 + r) * p.H + h) * p.K * 4 + e * 4) = x;
                        *(float *)((char *)p.dq + ((b * p.L + t0 + r) * p.H + h) * p.K * 4 + e * 4) = x;
                    } else {
                        ((T *)p.dk)[((b * p.L + t0 + r) * p.Hk + hk) * p.K + e] = (T)x;
                    }
                }
            }
            __syncthreads();
        }
        if (wave == 0) {  // dg
            float d = pairs, a = 0.0f, e = 0.0f;
            if (lane < C) {
#pragma unroll
                for (int w = 0; w < KT; ++w) {
                    a += came[w][lane];
                    e += left[w][lane];
                    d += through[w];
                }
            }
            float before = e;  // sums of what left before t, and of what came from t on
#pragma unroll
            for (int k = 1; k < C; k *= 2) {
                const float up = __shfl_up(before, k), down = __shfl_down(a, k);
                if (lane >= k) before += up;
                if (lane + k < C) a += down;
            }
            before = __shfl_up(before, 1);
            if (lane > 0) d += before;
            d += a;
            if (odd && lane < C) d += spoilt[lane];
            if (lane < C && t0 + lane < p.L) p.dg[(b * p.L + t0 + lane) * p.H + h] = d;
        }
    }
    if (n > 0) put_outputs(c0);
    if (p.dfirst && seg == 0 && of_v) state_store<KT>(SV, p.dfirst + bh * KV, p.K, p.V, part * 32 + l31, half);
}

// Gradients of shared heads: the sum over a group's heads, rounded once.
template <typename T>
__global__ void __launch_bounds__(256) k_groups(const float *dq, const float *dk, T *oq, T *ok, int64_t n, int32_t K, int32_t share) {
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) {
        const int64_t group = e / K, at = group * share * K + e % K;
        float q = 0.0f, k = 0.0f;
        for (int s = 0; s < share; ++s) {
            q += dq[at + (int64_t)s * K];
            k += dk[at + (int64_t)s * K];
        }
        oq[e] = (T)q;
        ok[e] = (T)k;
    }
}

// Gradient of a decay that all tokens of a head share: the sum over them, in 64 bits.
__global__ void __launch_bounds__(1024) k_decay_sum(const float *dg, float *out, int64_t tokens, int32_t H) {
    const int h = blockIdx.x;
    double sum = 0.0;
    int64_t t = threadIdx.x;
    for (; t + 7 * 1024 < tokens; t += 8 * 1024) {
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = dg[(t + k * 1024) * H + h];
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += x[k];
    }
    for (; t < tokens; t += 1024) sum += dg[t * H + h];
    __shared__ double part[16];
#pragma unroll
    for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 16; ++w) sum += part[w];
        out[h] = (float)sum;
    }
}

// One token: a block has 4 LANES columns of V of one head's state, LANES lanes of 4 for a row (which may start
// on any element; the row's last lane may have fewer). What bounds it are the state's bytes, read and
// written once: 4 layers x 256 sequences x 32 heads of 128 x 128, 4.3 GB, in 0.83 ms (5.2 TB/s).
typedef f32x4 __attribute__((aligned(4))) any_f32x4;
template <typename T, int LANES>
__global__ void __launch_bounds__(256) k_step(LinattnStepArgs p) {
    constexpr int kRows = 256 / LANES;
    const int slices = (p.V + 4 * LANES - 1) / (4 * LANES), slice = blockIdx.x % slices;
    const int64_t nh = blockIdx.x / slices, n = nh / p.H;
    const int h = (int)(nh % p.H), hk = h / (p.H / p.Hk);
    const int v = slice * 4 * LANES + threadIdx.x % LANES * 4, r0 = threadIdx.x / LANES, live = min(max(p.V - v, 0), 4);
    const float g = p.g[(p.per_token ? n : n / p.seqs) * p.H + h];
    const float a = g < kCut ? 0.0f : exp2_of((double)g * kLog2e);
    const T *const q = (const T *)p.q + (n * p.Hk + hk) * p.K, *const k = (const T *)p.k + (n * p.Hk + hk) * p.K;
    f32x4 x = {0, 0, 0, 0}, o = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < live) x[e] = (float)((const T *)p.v + nh * p.V)[v + e];
    float *const S = p.h + nh * p.K * p.V + v;
    const auto add = [&](f32x4 s, int r) {
        const float kr = (float)k[r], qr = (float)q[r];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[e] = (a == 0.0f ? 0.0f : a * s[e]) + kr * x[e];
            o[e] += qr * s[e];
        }
        return s;
    };
    if (live == 4) {
#pragma unroll 4
        for (int r = r0; r < p.K; r += kRows) {
            any_f32x4 *const at = (any_f32x4 *)(S + (int64_t)r * p.V);
            *at = add(*at, r);
        }
    } else if (live > 0) {
        for (int r = r0; r < p.K; r += kRows) {
            float *const at = S + (int64_t)r * p.V;
            f32x4 s = {0, 0, 0, 0};
            for (int e = 0; e < live; ++e) s[e] = at[e];
            s = add(s, r);
            for (int e = 0; e < live; ++e) at[e] = s[e];
        }
    }
    __shared__ f32x4 sum[kRows][LANES];
    sum[r0][threadIdx.x % LANES] = o;
    __syncthreads();
    if (threadIdx.x < LANES) {
        f32x4 t = {0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < kRows; ++r) t += sum[r][threadIdx.x];
        T *const out = (T *)p.o + nh * p.V + v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < live) out[e] = (T)(t[e] * p.scale);
    }
}

// ------------------------------------------------------------------ host side
bool aligned_to(const void *p, size_t n) { return (uintptr_t)p % n == 0; }
int chunk_of(int io) { return io ? Kind<__bf16>::C : Kind<float>::C; }
size_t up(size_t v) { return (v + 255) / 256 * 256; }

// Segments of a sequence: enough blocks for the GPU, of two chunks at least. A sweep over the segments' keys
// and values comes first where there are several; with few heads the time is that of a chunk after
// another, so short segments pay all the same (3 x 1001 tokens of 6 heads, float32: 73 us forwards and 149
// back with 8 chunks a segment, 46 and 63 with 2).
struct Plan {
    int64_t nchunk;
    int nseg, per_seg, slices;
};
Plan plan(int64_t B, int64_t L, int32_t H, int32_t V, int io, bool bwd) {
    Plan p;
    p.nchunk = (L + chunk_of(io) - 1) / chunk_of(io);
    const int vp = V > 64 ? 128 : 64;
    // Two blocks of 4 waves a compute unit. Two slices of V, which read q and k twice, where even the shortest
    // segments are too few.
    const int64_t want = bwd ? 256 : 512, most = std::max<int64_t>(p.nchunk / 2, 1);
    p.slices = !bwd && vp == 128 && B * H * most < want ? 2 : 1;
    // The fewest chunks one after another: rounds of blocks times a segment's chunks and one for its start; more
    // than one segment takes the first sweep, a quarter as long. Back, 9107 tokens x 21 heads of 32 x 128 in float32:
    // 448 us with 12 segments, 740 with the 13 that begin a second round; 8192 x 40 heads of 128 x 128 in bf16: 382
    // with 6, 517 with 7. Forwards, where blocks share compute units, 148 with 12 and 169 with 13; the most that
    // this rule loses there to the fewest segments that fill the GPU is 4 % (4096 x 300 heads: 658 with 5, 633 with 2).
    const int64_t blocks = std::max<int64_t>(B * H * p.slices, 1);
    int64_t per = std::max<int64_t>(p.nchunk, 1), best = ((blocks + want - 1) / want) * (per + 1) * 4;
    for (int64_t rounds = 1; rounds <= 4; ++rounds) {
        const int64_t n = std::min(rounds * want / blocks, most);  // the most segments that take so many rounds
        if (n < 2) continue;
        const int64_t chunks = (p.nchunk + n - 1) / n, cost = ((blocks * n + want - 1) / want) * (chunks + 1) * 5;
        if (cost < best) {
            best = cost;
            per = chunks;
        }
    }
    p.per_seg = (int)per;
    p.nseg = (int)std::max<int64_t>((p.nchunk + per - 1) / per, 1);
    return p;
}

template <typename T>
Access access(int32_t K, int32_t V, std::initializer_list<const void *> arrays) {
    constexpr int E = 16 / sizeof(T);
    if (K < E || V < E) return kElements;
    for (const void *p : arrays)
        if (!aligned_to(p, 16)) return kAny;
    return K % E == 0 && V % E == 0 ? kWide : kAny;
}

// Rows shorter than a vector are read by the kernels of the largest sizes only.
template <typename T, bool OUT>
void sweep(const SweepArgs &a, Access access, int64_t blocks, hipStream_t s) {
    const int width = (a.V > 64 ? 128 : 64) / a.slices;
    const auto go = [&](auto acc) {
        constexpr Access A = decltype(acc)::value;
        const auto keys = [&](auto kp) {
            constexpr int KP = decltype(kp)::value;
            if (width == 128) k_sweep<T, KP, 4, OUT, A><<<blocks, 256, 0, s>>>(a);
            else k_sweep<T, KP, 2, OUT, A><<<blocks, 128, 0, s>>>(a);
        };
        if constexpr (A != kElements) {
            if constexpr (sizeof(T) == 4)  // products in float32 are what bounds it
                if (a.K <= 32) return keys(std::integral_constant<int, 32>());
            if (a.K <= 64) return keys(std::integral_constant<int, 64>());
        }
        keys(std::integral_constant<int, 128>());
    };
    if (access == kWide) go(std::integral_constant<Access, kWide>());
    else if (access == kAny) go(std::integral_constant<Access, kAny>());
    else go(std::integral_constant<Access, kElements>());
}
template <typename T>
void bwd(const BwdArgs &a, Access access, int64_t blocks, hipStream_t s) {
    const auto go = [&](auto acc) {
        constexpr Access A = decltype(acc)::value;
        if (a.K > 64) {
            if (a.V > 64) k_bwd<T, 128, 128, A><<<blocks, 512, 0, s>>>(a);
            else k_bwd<T, 128, 64, A><<<blocks, 384, 0, s>>>(a);
        } else if (sizeof(T) == 4 && a.K <= 32) {
            if constexpr (sizeof(T) == 4) {
                if (a.V > 64) k_bwd<T, 32, 128, A><<<blocks, 320, 0, s>>>(a);
                else k_bwd<T, 32, 64, A><<<blocks, 192, 0, s>>>(a);
            }
        } else {
            if (a.V > 64) k_bwd<T, 64, 128, A><<<blocks, 384, 0, s>>>(a);
            else k_bwd<T, 64, 64, A><<<blocks, 256, 0, s>>>(a);
        }
    };
    if (access == kWide) go(std::integral_constant<Access, kWide>());
    else if (access == kAny) go(std::integral_constant<Access, kAny>());
    else k_bwd<T, 128, 128, kElements><<<blocks, 512, 0, s>>>(a);
}

template <typename T>
hipError_t run_fwd(const LinattnArgs &a, hipStream_t s) {
    const int io = sizeof(T) == 2;
    const Plan pl = plan(a.B, a.L, a.H, a.V, io, false);
    const int64_t heads = a.B * a.H, KV = (int64_t)a.K * a.V;
    float *const seg = (float *)a.ws, *const fac = pl.nseg > 1 ? seg + heads * pl.nseg * KV : nullptr;
    SweepArgs p{};
    p.q = a.q; p.k = a.k; p.v = a.v; p.g = a.g;
    p.L = a.L; p.H = a.H; p.Hk = a.Hk; p.K = a.K; p.V = a.V;
    p.g_batch = a.per_token ? a.L * a.H : 0;
    p.g_token = a.per_token ? a.H : 0;
    p.nchunk = (int)pl.nchunk; p.per_seg = pl.per_seg; p.slices = pl.slices;
    p.scale = a.scale;
    const Access acc = access<T>(a.K, a.V, {a.q, a.k, a.v, a.o});
    if (pl.nseg > 1) {
        SweepArgs q = p;
        q.nseg = pl.nseg - 1;
        q.seg_out = seg;
        q.seg_fac = fac;
        sweep<T, false>(q, acc, heads * q.nseg * q.slices, s);
        k_join<<<(heads * KV + 255) / 256, 256, 0, s>>>(seg, fac, a.h0, KV, heads, pl.nseg, false);
        p.seg_in = seg;
    }
    p.nseg = pl.nseg;
    p.first = a.h0;
    p.o = a.o; p.last = a.h_final; p.states = a.states;
    sweep<T, true>(p, acc, heads * p.nseg * p.slices, s);
    return hipGetLastError();
}

// The backward's workspace: the segments' gradients of the state and their decays, the gradients of
// shared heads, and dg by token.
struct BwdPlan {
    Plan seg, pass;
    size_t fac, dq, dk, dg, bytes;
};
BwdPlan bwd_plan(int64_t B, int64_t L, int32_t H, int32_t Hk, int32_t K, int32_t V, bool per_token, int io) {
    BwdPlan p;
    p.seg = plan(B, L, H, V, io, true);
    p.pass = p.seg;
    p.pass.slices = V > 64 ? 2 : 1;
    size_t at = 0;
    if (p.seg.nseg > 1) at = up((size_t)B * H * p.seg.nseg * K * V * 4);
    p.fac = at;
    if (p.seg.nseg > 1) at = up(at + (size_t)B * H * p.seg.nseg * 4);
    p.dq = at;
    if (H != Hk) at = up(at + (size_t)B * L * H * K * 4);
    p.dk = at;
    if (H != Hk) at = up(at + (size_t)B * L * H * K * 4);
    p.dg = at;
    if (!per_token) at = up(at + (size_t)B * L * H * 4);
    p.bytes = at;
    return p;
}

template <typename T>
hipError_t run_bwd(const LinattnArgs &a, hipStream_t s) {
    const int io = sizeof(T) == 2;
    const BwdPlan pl = bwd_plan(a.B, a.L, a.H, a.Hk, a.K, a.V, a.per_token, io);
    const int64_t heads = a.B * a.H, KV = (int64_t)a.K * a.V;
    char *const ws = (char *)a.ws;
    float *const seg = (float *)ws, *const fac = (float *)(ws + pl.fac);
    BwdArgs p{};
    p.q = a.q; p.k = a.k; p.v = a.v; p.do_ = a.do_; p.g = a.g; p.states = a.states;
    p.L = a.L; p.H = a.H; p.Hk = a.Hk; p.K = a.K; p.V = a.V;
    p.g_batch = a.per_token ? a.L * a.H : 0;
    p.g_token = a.per_token ? a.H : 0;
    p.nchunk = (int)pl.seg.nchunk; p.per_seg = pl.seg.per_seg; p.nseg = pl.seg.nseg;
    p.scale = a.scale;
    const Access acc = access<T>(a.K, a.V, {a.q, a.k, a.v, a.do_, a.states, a.dq, a.dk, a.dv});
    const bool shared = a.H != a.Hk;
    p.dq = shared ? ws + pl.dq : (char *)a.dq;
    p.dk = shared ? ws + pl.dk : (char *)a.dk;
    p.dv = a.dv;
    p.dg = a.per_token ? a.dg : (float *)(ws + pl.dg);
    p.dlast = a.dh_final;
    p.dfirst = a.dh0;
    if (heads > 0) {
        if (p.nseg > 1) {
            SweepArgs q{};
            q.k = a.q; q.v = a.do_; q.g = a.g;
            q.L = a.L; q.H = a.H; q.Hk = a.Hk; q.K = a.K; q.V = a.V;
            q.g_batch = p.g_batch; q.g_token = p.g_token;
            q.nchunk = p.nchunk; q.per_seg = p.per_seg; q.nseg = p.nseg - 1; q.slices = pl.pass.slices;
            q.scale = a.scale; q.reverse = true;
            q.seg_out = seg; q.seg_fac = fac;
            sweep<T, false>(q, acc, heads * q.nseg * q.slices, s);
            k_join<<<(heads * KV + 255) / 256, 256, 0, s>>>(seg, fac, a.dh_final, KV, heads, p.nseg, true);
            p.seg_in = seg;
        }
        const int64_t blocks = heads * p.nseg;
        bwd<T>(p, acc, blocks, s);
        if (shared && a.L > 0) {
            const int64_t n = a.B * a.L * a.Hk * a.K;
            k_groups<T><<<std::min<int64_t>((n + 255) / 256, 1 << 20), 256, 0, s>>>((const float *)p.dq, (const float *)p.dk, (T *)a.dq,
                                                                                    (T *)a.dk, n, a.K, a.H / a.Hk);
        }
    }
    if (!a.per_token) k_decay_sum<<<a.H, 1024, 0, s>>>(p.dg, a.dg, a.B * a.L, a.H);
    return hipGetLastError();
}

}  // namespace

int32_t linattn_state_every(int io) { return chunk_of(io); }
size_t linattn_fwd_ws(int64_t B, int64_t L, int32_t H, int32_t K, int32_t V, int io) {
    const Plan p = plan(B, L, H, V, io, false);
    return p.nseg > 1 ? (size_t)B * H * p.nseg * ((size_t)K * V + 1) * 4 : 0;
}
size_t linattn_bwd_ws(int64_t B, int64_t L, int32_t H, int32_t Hk, int32_t K, int32_t V, bool per_token, int io) {
    return bwd_plan(B, L, H, Hk, K, V, per_token, io).bytes;
}
hipError_t launch_linattn_fwd(const LinattnArgs &a, int io, hipStream_t s) {
    return io ? run_fwd<__bf16>(a, s) : run_fwd<float>(a, s);
}
hipError_t launch_linattn_bwd(const LinattnArgs &a, int io, hipStream_t s) {
    return io ? run_bwd<__bf16>(a, s) : run_bwd<float>(a, s);
}
hipError_t launch_linattn_step(const LinattnStepArgs &a, int io, hipStream_t s) {
    // Whole rows where there are heads enough for the GPU (13203 of 25 x 46 in bf16: 43 us, 64 in slices of
    // 32 columns; 32768 of 128 x 128: 833 us, 903 in slices). With few heads slices of 32 columns (32 heads of
    // 128 x 128: 4.7 us, 5.5 in slices of 16).
    const int64_t heads = a.layers * a.seqs * a.H;
    const int lanes = heads < 1024 || a.V <= 32 ? 8 : a.V <= 64 ? 16 : 32;
    const int64_t blocks = heads * ((a.V + 4 * lanes - 1) / (4 * lanes));
    const auto go = [&](auto n) {
        constexpr int N = decltype(n)::value;
        if (io) k_step<__bf16, N><<<blocks, 256, 0, s>>>(a);
        else k_step<float, N><<<blocks, 256, 0, s>>>(a);
    };
    if (lanes == 8) go(std::integral_constant<int, 8>());
    else if (lanes == 16) go(std::integral_constant<int, 16>());
    else go(std::integral_constant<int, 32>());
    return hipGetLastError();
}

}  // namespace ssm
