// rmsnorm.hip -- the root-mean-square norm with the residual's addition before it, as values or as
// codes of 8 bits with scales, and its gradients.
//
//     s = x + residual (rounded to the residual's type), r = 1 / sqrt(mean(s^2) + eps),
//     y = s r weight;   codes: scale = max |y| / most (448 or 127), code = y / scale rounded
//     n = s r:  ds' = r (weight dy - n mean(weight dy n)) + ds,   dweight = sum over rows of dy n
//
// A row stays in registers between its sum and its output, so every array is read or written once:
// bytes are the floor. A row of up to 1024 elements belongs to a wave or a part of one, a longer one to a
// block of 256 to 1024 threads. The sum of squares is held in 64 bits (a conversion and a multiply-add an element:
// the 64-bit rate of the vector units is that of 32 bits), so that r does not depend on the order,
// and codes are computed in 64 bits from s on: a value next to the border of two codes takes the
// right one.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "ssm_layers.h"

namespace ssm {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int E = 8;  // elements of a vector

__device__ __forceinline__ float widen(uint32_t bits16) { return __uint_as_float(bits16 << 16); }
__device__ __forceinline__ uint32_t narrow(float a, float b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// A thread's elements of a row: eight neighbours for each of its NV vectors. A vector may start on any
// element (the hardware reads and writes 16 bytes there); the last of a row may be shorter, then the
// one thread that has it goes by elements.
typedef u32x4 __attribute__((aligned(2))) any_u32x4;
typedef u32x2 __attribute__((aligned(1))) any_u32x2;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 __attribute__((aligned(4))) any_f32x4;

template <int TPR>
struct Piece {
    int first;
    __device__ __forceinline__ Piece() { first = threadIdx.x % TPR * E; }
    __device__ __forceinline__ int at(int n) const { return first + n * TPR * E; }
    // What is past the row's end is 0.
    template <typename T>
    __device__ __forceinline__ void load(const T *row, int n, int width, float (&x)[E]) const {
        const int from = at(n);
        if (from + E <= width) {
            if constexpr (sizeof(T) == 2) {
                const u32x4 r = *(const any_u32x4 *)(row + from);
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] = widen(e % 2 ? r[e / 2] >> 16 : r[e / 2] & 0xffff);
            } else {
                const f32x4 lo = *(const any_f32x4 *)(row + from), hi = *(const any_f32x4 *)(row + from + 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = lo[e];
                    x[4 + e] = hi[e];
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = 0.0f;
            if (from < width) {
#pragma unroll
                for (int e = 0; e < E - 1; ++e)
                    if (from + e < width) x[e] = (float)row[from + e];
            }
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T *row, int n, int width, const float (&x)[E]) const {
        const int to = at(n);
        if (to + E <= width) {
            if constexpr (sizeof(T) == 2) {
                *(any_u32x4 *)(row + to) = u32x4{narrow(x[0], x[1]), narrow(x[2], x[3]), narrow(x[4], x[5]), narrow(x[6], x[7])};
            } else {
                *(any_f32x4 *)(row + to) = f32x4{x[0], x[1], x[2], x[3]};
                *(any_f32x4 *)(row + to + 4) = f32x4{x[4], x[5], x[6], x[7]};
            }
        } else if (to < width) {
#pragma unroll
            for (int e = 0; e < E - 1; ++e)
                if (to + e < width) row[to + e] = (T)x[e];
        }
    }
};
template <typename T> __device__ __forceinline__ float stored(float x) {
    if constexpr (sizeof(T) == 2) return (float)(T)x;
    else return x;
}

// The sum, or the largest, over a row's TPR threads, the same bits in all of them.
template <int TPR, typename V, typename F>
__device__ __forceinline__ V over_row(V x, V *part, F join) {
#pragma unroll
    for (int d = 1; d < (TPR < 64 ? TPR : 64); d *= 2) x = join(x, __shfl_xor(x, d));
    if constexpr (TPR > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
        __syncthreads();
        x = part[0];
#pragma unroll
        for (int w = 1; w < TPR / 64; ++w) x = join(x, part[w]);
    }
    return x;
}
template <int TPR> __device__ __forceinline__ double row_sum(double x, double *part) {
    return over_row<TPR>(x, part, [](double a, double b) { return a + b; });
}

// The multiple of the code's step next to u, ties to even, by adding and taking away 1.5 x 2^52
// steps: a step is 2^-3 of the value's power of two, and 2^-9 at least.
__device__ __forceinline__ float to_e4m3(double u) {
    int ex = __double2hiint(u) >> 20 & 0x7ff;
    ex = min(max(ex, 1023 - 6), 1023 + 10);
    const double big = __hiloint2double((ex + 49) << 20 | 0x80000, 0);
    const float r = (float)((u + big) - big);
    return fminf(fmaxf(r, -448.0f), 448.0f);
}
// A scale, and its reciprocal (0 where there is none).
struct Scale {
    double s, inv;
    // y / s: the reciprocal's error would put a quotient in the middle of two codes beside it (73.5 / 49), so
    // what is left of y is added, after which a quotient that 64 bits hold is that one.
    __device__ __forceinline__ double of(double y) const {
        const double q = y * inv;
        return __builtin_fma(__builtin_fma(-q, s, y), inv, q);
    }
};
// Eight codes. A quotient rounded to float32 first gives the same code as the quotient itself unless
// float32 puts it onto the middle of two codes, or it is below the smallest normal one (2^-6, where
// steps differ): about 1 in 10^4, which take the long way.
__device__ __forceinline__ void code8(const double (&y)[E], Scale scale, int code, uint32_t (&c)[2]) {
    float f[E];
    if (code == 1) {
        bool hard = false;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            f[e] = (float)(y[e] * scale.inv);
            hard |= (__float_as_uint(f[e]) & 0xfffffu) == 0x80000u || !(fabsf(f[e]) >= 0x1p-6f);
            f[e] = __builtin_amdgcn_fmed3f(f[e], -448.0f, 448.0f);
        }
        if (hard) {
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = to_e4m3(scale.of(y[e]));
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * k], f[4 * k + 1], 0, false);
            c[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * k + 2], f[4 * k + 3], v, true);
        }
    } else {
        c[0] = c[1] = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float r = __builtin_amdgcn_fmed3f((float)__builtin_rint(scale.of(y[e])), -127.0f, 127.0f);
            c[e / 4] |= (uint32_t)((int)r & 0xff) << (e % 4 * 8);
        }
    }
}

// The largest |y|, NaN where one is: the hardware's maximum leaves NaN out, so they are told apart.
struct Top {
    double top = 0.0;
    bool bad = false;
    __device__ __forceinline__ void add(double y) {
        top = __builtin_fmax(top, __builtin_fabs(y));
        bad |= y != y;
    }
    // As a whole number that compares like it, a NaN above all.
    __device__ __forceinline__ long long bits() const { return bad ? 0x7ff8000000000000ll : __double_as_longlong(top); }
};
__device__ __forceinline__ long long larger(long long a, long long b) { return a > b ? a : b; }
// The largest over `lanes` neighbouring lanes (a power of two).
__device__ __forceinline__ long long over_lanes(long long x, int lanes) {
    for (int d = 1; d < lanes; d *= 2) x = larger(x, __shfl_xor(x, d));
    return x;
}
// The scale of values whose largest is top, and its reciprocal, by Newton's steps from the hardware's estimate
// (relative 2^-22, 2^-44, 2^-52).
__device__ __forceinline__ float scale_of(long long top, int code, Scale &to) {
    const Scale most = code == 1 ? Scale{448.0, 1.0 / 448.0} : Scale{127.0, 1.0 / 127.0};
    const double largest = __longlong_as_double(top);
    const float scale = (float)(largest < __builtin_inf() ? most.of(largest) : largest);
    const double s = (double)scale;
    double x = __builtin_amdgcn_rcp(s);
    x = __builtin_fma(x, __builtin_fma(-s, x, 1.0), x);
    x = __builtin_fma(x, __builtin_fma(-s, x, 1.0), x);
    to = scale == 0.0f || scale == __builtin_inff() ? Scale{0.0, 0.0} : Scale{s, x};
    return scale;
}

// MODE: values, codes with a scale for a row, codes with a scale for a group.
enum { kValues, kRowCodes, kGroupCodes };
template <typename T, typename R, int TPR, int NV, int MODE>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) k_fwd(NormArgs p) {
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    __shared__ double part[TPR > 64 ? TPR / 64 : 1];
    const Piece<TPR> own;
    const int tid = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    if (row >= p.rows) return;  // whole rows: one of several waves has the block to itself
    const int D = p.dim;
    const int64_t at0 = row * D;
    float s[NV][E];
#pragma unroll
    for (int n = 0; n < NV; ++n) own.load((const T *)p.x + at0, n, D, s[n]);
    if (p.residual) {
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float add[E];
            own.load((const R *)p.residual + at0, n, D, add);
#pragma unroll
            for (int e = 0; e < E; ++e) s[n][e] = stored<R>(s[n][e] + add[e]);
            own.store((R *)p.added + at0, n, D, s[n]);
        }
    }
    double sum = 0.0;
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int e = 0; e < E; ++e) sum = __builtin_fma((double)s[n][e], (double)s[n][e], sum);
    const double r = 1.0 / sqrt(row_sum<TPR>(sum, part) / D + p.eps);
    if (p.rstd && tid == 0) p.rstd[row] = (float)r;
    if constexpr (MODE == kValues) {
        const float rf = (float)r;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float w[E];
            own.load(p.weight, n, D, w);
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] = s[n][e] * rf * w[e];
            own.store((T *)p.y + at0, n, D, w);
        }
        return;
    }
    const int group = p.group, groups = group ? (D + group - 1) / group : 1;
    Scale by{0.0, 0.0};
    if constexpr (MODE == kRowCodes) {
        Top top;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float w[E];
            own.load(p.weight, n, D, w);
#pragma unroll
            for (int e = 0; e < E; ++e) top.add((double)s[n][e] * r * (double)w[e]);
        }
        const float scale = scale_of(over_row<TPR>(top.bits(), (long long *)part, larger), p.code, by);
        if (tid == 0) p.scales[row] = scale;
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        float w[E];
        own.load(p.weight, n, D, w);
        double y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = (double)s[n][e] * r * (double)w[e];
        if constexpr (MODE == kGroupCodes) {
            Top top;
#pragma unroll
            for (int e = 0; e < E; ++e) top.add(y[e]);
            const float scale = scale_of(over_lanes(top.bits(), group / E), p.code, by);
            const int at = own.at(n);
            if (at < D && at % group == 0) p.scales[row * groups + at / group] = scale;
        }
        uint32_t c[2];
        code8(y, by, p.code, c);
        uint8_t *const to = (uint8_t *)p.y + at0;
        const int at = own.at(n);
        if (at + E <= D) {
            *(any_u32x2 *)(to + at) = u32x2{c[0], c[1]};
        } else if (at < D) {
#pragma unroll
            for (int e = 0; e < E - 1; ++e)
                if (at + e < D) to[at + e] = (uint8_t)(c[e / 4] >> (e % 4 * 8));
        }
        __builtin_amdgcn_sched_barrier(0);  // a vector at a time: more rows fit a compute unit
    }
}

// Every row set (a block, or a wave of one) takes rows at a distance and keeps its sum of dweight; a wave that
// has several rows at a time adds theirs at the end. A sum of many rows in 32 bits would lose the bits of a row's
// share, so it is compensated (Kahan), which takes as many registers again and three operations an element;
// rows of more than 8192, which have no registers left, get a set for every 64 rows instead. A row of more than 16384 elements is read a second time, from
// the cache where it fits, after its sum: it does not fit the registers beside dweight's (2048 rows of 9216 in
// 35 us; 1024 of 20000 in 129, held in registers and memory behind them 177).
template <typename T, typename R, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) k_bwd(NormBwdArgs p, int sets) {
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    __shared__ double part[TPR > 64 ? TPR / 64 : 1];
    Piece<TPR> own;
    constexpr int kOfSet = TPR < 64 ? 64 / TPR : 1, KEPT = NV <= 2 ? NV : 1;
    constexpr bool kCompensated = TPR < 1024;
    const int line = blockIdx.x * kRows + threadIdx.x / TPR, set = line / kOfSet, D = p.dim;
    if (set >= sets) return;
    float dw[NV][E] = {}, lost[kCompensated ? NV : 1][E] = {};  // what the sums have too much
    for (int64_t row = line; row < p.rows; row += (int64_t)sets * kOfSet) {
        const int64_t at0 = row * D;
        const float r = p.rstd[row];
        const float *weight = p.weight;
        if constexpr (TPR == 1024) asm volatile("" : "+s"(weight), "+v"(own.first));  // for each row anew: no registers are left (9216: 35 us, 57)
        float n[KEPT][E], wd[KEPT][E];
        const auto load = [&](int k, float (&n)[E], float (&wd)[E], bool first) {
            float w[E];
            own.load((const R *)p.s + at0, k, D, n);
            own.load((const T *)p.dy + at0, k, D, wd);
            own.load(weight, k, D, w);
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                n[e] *= r;
                if constexpr (kCompensated) {
                    const float add = __builtin_fmaf(wd[e], n[e], -lost[k][e]), up = dw[k][e] + add;
                    lost[k][e] = (up - dw[k][e]) - add;
                    dw[k][e] = up;
                } else if (first) {
                    dw[k][e] += wd[e] * n[e];
                }
                wd[e] *= w[e];
                t += wd[e] * n[e];
            }
            return t;
        };
        double sum = 0.0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            sum += load(k, n[k % KEPT], wd[k % KEPT], true);
            if (KEPT < NV) __builtin_amdgcn_sched_barrier(0);
        }
        const float c = (float)(row_sum<TPR>(sum, part) / D);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if constexpr (KEPT < NV) load(k, n[0], wd[0], false);
            float g[E];
            if (p.ds) {
                own.load((const R *)p.ds + at0, k, D, g);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) g[e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) g[e] += (wd[k % KEPT][e] - n[k % KEPT][e] * c) * r;
            own.store((T *)p.dx + at0, k, D, g);
            if (p.dres) own.store((R *)p.dres + at0, k, D, g);
            if (KEPT < NV) __builtin_amdgcn_sched_barrier(0);
        }
    }
    if constexpr (TPR < 64) {
#pragma unroll
        for (int d = TPR; d < 64; d *= 2)
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int e = 0; e < E; ++e) dw[k][e] += __shfl_xor(dw[k][e], d);
        if ((threadIdx.x & 63) >= TPR) return;
    }
    float *const to = (float *)p.ws + (int64_t)set * D;
#pragma unroll
    for (int k = 0; k < NV; ++k) own.store(to, k, D, dw[k]);
}

// 16 columns by 16 rows of partial sums at a time; a thread's rows, then the 16 threads of a column.
__global__ void __launch_bounds__(256) k_dweight(const float *part, float *out, int sets, int D) {
    __shared__ double sum[16][17];
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4, at = blockIdx.x * 16 + x;
    double s = 0.0;
    if (at < D) {
#pragma unroll 8
        for (int r = y; r < sets; r += 16) s += part[(int64_t)r * D + at];
    }
    sum[y][x] = s;
    __syncthreads();
    if (y == 0 && at < D) {
#pragma unroll
        for (int k = 1; k < 16; ++k) s += sum[k][x];
        out[at] = (float)s;
    }
}

// 8 codes of a row a thread (a group is a multiple of 8); the row's last may be fewer.
__global__ void __launch_bounds__(256) k_values(const uint8_t *codes, const float *scales, float *out, int64_t rows, int D, int group,
                                                int code) {
    const uint32_t per_row = (D + 7) / 8, groups = group ? (D + group - 1) / group : 1;
    const int64_t n = rows * per_row, stride = (int64_t)gridDim.x * 256;
    for (int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x; v < n; v += stride) {
        const int64_t row = n <= 0xffffffff ? (uint32_t)v / per_row : v / per_row;
        const int at = (int)(v - row * per_row) * 8;
        const float scale = scales[row * groups + (group ? at / group : 0)];
        const uint8_t *const from = codes + row * D + at;
        float *const to = out + row * D + at;
        if (at + 8 <= D) {
            const u32x2 c = *(const any_u32x2 *)from;
            f32x4 x[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (code == 1) {
                    x[k] = f32x4{__builtin_amdgcn_cvt_f32_fp8((int)c[k], 0), __builtin_amdgcn_cvt_f32_fp8((int)c[k], 1),
                                 __builtin_amdgcn_cvt_f32_fp8((int)c[k], 2), __builtin_amdgcn_cvt_f32_fp8((int)c[k], 3)};
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[k][j] = (float)(int8_t)(c[k] >> (8 * j));
                }
                x[k] *= scale;
                *(any_f32x4 *)(to + 4 * k) = x[k];
            }
        } else {
            for (int e = 0; at + e < D; ++e) to[e] = (code == 1 ? __builtin_amdgcn_cvt_f32_fp8((int)from[e], 0) : (float)(int8_t)from[e]) * scale;
        }
    }
}

// Threads of a row: 16 up to 128 elements (heads), 32 up to 256, a wave up to 1024, 256 up to 4096, 512 up to 8192,
// 1024 up to 65536. 524288 rows of 128 in bf16: forward 53 us, backward 124; with a wave for a row 170 and 339.
constexpr int kNarrow = 128, kHalf = 256, kCompensatedDim = 8192;
template <typename F>
void by_size(int D, F go) {
    typedef std::integral_constant<int, 16> N;
    typedef std::integral_constant<int, 32> H;
    typedef std::integral_constant<int, 64> W;
    typedef std::integral_constant<int, 256> B;
    typedef std::integral_constant<int, 512> M;
    typedef std::integral_constant<int, 1024> L;
    if (D <= kNarrow) go(N(), std::integral_constant<int, 1>());
    else if (D <= kHalf) go(H(), std::integral_constant<int, 1>());
    else if (D <= 512) go(W(), std::integral_constant<int, 1>());
    else if (D <= 1024) go(W(), std::integral_constant<int, 2>());
    else if (D <= 2048) go(B(), std::integral_constant<int, 1>());
    else if (D <= 4096) go(B(), std::integral_constant<int, 2>());
    else if (D <= 8192) go(M(), std::integral_constant<int, 2>());
    else if (D <= 16384) go(L(), std::integral_constant<int, 2>());
    else if (D <= 32768) go(L(), std::integral_constant<int, 4>());
    else go(L(), std::integral_constant<int, 8>());
}

template <typename T, typename R>
void run_fwd(const NormArgs &a, hipStream_t s) {
    by_size(a.dim, [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value, kThreads = TPR < 256 ? 256 : TPR;
        const int groups = a.group ? (a.dim + a.group - 1) / a.group : 1;
        // A launch has fewer than 2^32 threads.
        const int64_t most = (int64_t)(1 << 21) * (kThreads / TPR);
        for (int64_t first = 0; first < a.rows; first += most) {
            NormArgs p = a;
            p.rows = std::min(a.rows - first, most);
            p.x = (const T *)a.x + first * a.dim;
            if (a.residual) {
                p.residual = (const R *)a.residual + first * a.dim;
                p.added = (R *)a.added + first * a.dim;
            }
            p.y = (char *)a.y + first * a.dim * (a.code ? 1 : (int)sizeof(T));
            if (a.rstd) p.rstd = a.rstd + first;
            if (a.scales) p.scales = a.scales + first * groups;
            const int64_t blocks = (p.rows + kThreads / TPR - 1) / (kThreads / TPR);
            if (a.code == 0) k_fwd<T, R, TPR, NV, kValues><<<blocks, kThreads, 0, s>>>(p);
            else if (a.group == 0) k_fwd<T, R, TPR, NV, kRowCodes><<<blocks, kThreads, 0, s>>>(p);
            else k_fwd<T, R, TPR, NV, kGroupCodes><<<blocks, kThreads, 0, s>>>(p);
        }
    });
}

// Row sets of the backward: enough for the GPU, each with several rows where there are many, but 64 at most
// where their sums are not compensated (1/64 of the rows' bytes for the sets' sums). A launch has fewer than
// 2^32 threads.
int row_sets(int64_t rows, int32_t dim) {
    const int64_t at_once = dim <= kNarrow ? 4 : dim <= kHalf ? 2 : 1;
    int64_t most = dim <= 1024 ? 2048 : 512;
    if (dim > kCompensatedDim) most = std::min<int64_t>(std::max<int64_t>(most, (rows + 63) / 64), 1 << 21);
    return (int)std::max<int64_t>(1, std::min<int64_t>((rows + at_once - 1) / at_once, most));
}

template <typename T, typename R>
void run_bwd(const NormBwdArgs &a, hipStream_t s) {
    const int sets = row_sets(a.rows, a.dim);
    by_size(a.dim, [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value, kThreads = TPR < 256 ? 256 : TPR;
        constexpr int kSets = TPR < 256 ? 256 / (TPR < 64 ? 64 : TPR) : 1;
        const int blocks = (sets + kSets - 1) / kSets;
        k_bwd<T, R, TPR, NV><<<blocks, kThreads, 0, s>>>(a, sets);
    });
    k_dweight<<<(a.dim + 15) / 16, 256, 0, s>>>((const float *)a.ws, a.dweight, sets, a.dim);
}

}  // namespace

hipError_t launch_rmsnorm_fwd(const NormArgs &a, int io, int res_io, hipStream_t s) {
    if (!io) run_fwd<float, float>(a, s);
    else if (res_io) run_fwd<__bf16, __bf16>(a, s);
    else run_fwd<__bf16, float>(a, s);
    return hipGetLastError();
}
size_t rmsnorm_bwd_ws(int64_t rows, int32_t dim) { return (size_t)row_sets(rows, dim) * dim * 4; }
hipError_t launch_rmsnorm_bwd(const NormBwdArgs &a, int io, int res_io, hipStream_t s) {
    if (!io) run_bwd<float, float>(a, s);
    else if (res_io) run_bwd<__bf16, __bf16>(a, s);
    else run_bwd<__bf16, float>(a, s);
    return hipGetLastError();
}
hipError_t launch_q8_values(const void *codes, const float *scales, float *out, int64_t rows, int32_t dim, int32_t group,
                            int code, hipStream_t s) {
    const int64_t blocks = std::min<int64_t>((rows * ((dim + 7) / 8) + 255) / 256, 1 << 20);
    k_values<<<blocks, 256, 0, s>>>((const uint8_t *)codes, scales, out, rows, dim, group, code);
    return hipGetLastError();
}

}  // namespace ssm
