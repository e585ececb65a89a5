// rmsnorm.hip -- the root-mean-square norm with the residual's addition before it, as values or as
// codes of 8 bits with scales, and its gradients.
//
//     s = x + residual (rounded to the residual's type), r = 1 / sqrt(mean(s^2) + eps),
//     y = s r weight;   codes: scale = max |y| / most (448 or 127), code = y / scale rounded
//     n = s r:  ds' = r (weight dy - n mean(weight dy n)) + ds,   dweight = sum over rows of dy n
//
// A row stays in registers between its sum and its output, so every array is read or written once:
// bytes are the floor. A row of up to 1024 elements belongs to a wave, a longer one to a block of 256
// or 1024 threads. The sum of squares is held in 64 bits (a conversion and a multiply-add an element:
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

// Eight elements of a row from `at` on; what is past `width` is 0.
template <typename T>
__device__ __forceinline__ void load8(const T *row, int at, int width, bool wide, float (&x)[E]) {
    if (wide) {
        if (at < width) {
            if constexpr (sizeof(T) == 2) {
                const u32x4 r = *(const u32x4 *)(row + at);
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] = widen(e % 2 ? r[e / 2] >> 16 : r[e / 2] & 0xffff);
            } else {
                const float4 lo = *(const float4 *)(row + at), hi = *(const float4 *)(row + at + 4);
                x[0] = lo.x; x[1] = lo.y; x[2] = lo.z; x[3] = lo.w;
                x[4] = hi.x; x[5] = hi.y; x[6] = hi.z; x[7] = hi.w;
            }
            return;
        }
    } else if (at < width) {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = at + e < width ? (float)row[at + e] : 0.0f;
        return;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.0f;
}
template <typename T>
__device__ __forceinline__ void store8(T *row, int at, int width, bool wide, const float (&x)[E]) {
    if (at >= width) return;
    if (wide) {
        if constexpr (sizeof(T) == 2) {
            *(u32x4 *)(row + at) = u32x4{narrow(x[0], x[1]), narrow(x[2], x[3]), narrow(x[4], x[5]), narrow(x[6], x[7])};
        } else {
            *(float4 *)(row + at) = make_float4(x[0], x[1], x[2], x[3]);
            *(float4 *)(row + at + 4) = make_float4(x[4], x[5], x[6], x[7]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (at + e < width) row[at + e] = (T)x[e];
    }
}
template <typename T> __device__ __forceinline__ float stored(float x) {
    if constexpr (sizeof(T) == 2) return (float)(T)x;
    else return x;
}

// The sum, or the largest, over a row's TPR threads, the same bits in all of them.
template <int TPR, typename V, typename F>
__device__ __forceinline__ V over_row(V x, V *part, F join) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) x = join(x, __shfl_xor(x, d));
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

template <typename T, typename R, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) k_fwd(NormArgs p, bool wide) {
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    __shared__ double part[TPR > 64 ? TPR / 64 : 1];
    const int tid = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
    if (row >= p.rows) return;  // whole waves: a row of several waves has the block to itself
    const int D = p.dim;
    const int64_t at0 = row * D;
    float s[NV][E];
    double sum = 0.0;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int at = (tid + n * TPR) * E;
        load8((const T *)p.x + at0, at, D, wide, s[n]);
        if (p.residual) {
            float add[E];
            load8((const R *)p.residual + at0, at, D, wide, add);
#pragma unroll
            for (int e = 0; e < E; ++e) s[n][e] = stored<R>(s[n][e] + add[e]);
            store8((R *)p.added + at0, at, D, wide, s[n]);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) sum = __builtin_fma((double)s[n][e], (double)s[n][e], sum);
    }
    const double r = 1.0 / sqrt(row_sum<TPR>(sum, part) / D + p.eps);
    if (p.rstd && tid == 0) p.rstd[row] = (float)r;
    if (p.code == 0) {
        const float rf = (float)r;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int at = (tid + n * TPR) * E;
            float w[E];
            load8(p.weight, at, D, wide, w);
#pragma unroll
            for (int e = 0; e < E; ++e) w[e] = s[n][e] * rf * w[e];
            store8((T *)p.y + at0, at, D, wide, w);
        }
        return;
    }
    const double most = p.code == 1 ? 448.0 : 127.0;
    const auto larger = [](long long a, long long b) { return a > b ? a : b; };
    long long all = 0;
    if (p.group == 0) {  // |y| as integers: a NaN is larger than all
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float w[E];
            load8(p.weight, (tid + n * TPR) * E, D, wide, w);
#pragma unroll
            for (int e = 0; e < E; ++e) all = larger(all, __double_as_longlong(fabs((double)s[n][e] * r * (double)w[e])));
        }
        all = over_row<TPR>(all, (long long *)part, larger);
    }
    const int groups = p.group ? (D + p.group - 1) / p.group : 1, lanes = p.group / E;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int at = (tid + n * TPR) * E;
        float w[E];
        load8(p.weight, at, D, wide, w);
        double y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = (double)s[n][e] * r * (double)w[e];
        long long top = all;
        if (p.group) {
#pragma unroll
            for (int e = 0; e < E; ++e) top = larger(top, __double_as_longlong(fabs(y[e])));
            for (int d = 1; d < lanes; d *= 2) top = larger(top, __shfl_xor(top, d));
        }
        const float scale = (float)(__longlong_as_double(top) / most);
        const double inv = scale == 0.0f ? 0.0 : 1.0 / (double)scale;
        if (at < D && (p.group ? at % p.group == 0 : at == 0)) p.scales[row * groups + (p.group ? at / p.group : 0)] = scale;
        uint32_t c[2];
        if (p.code == 1) {
            float f[E];
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = to_e4m3(y[e] * inv);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                int v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * k], f[4 * k + 1], 0, false);
                c[k] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * k + 2], f[4 * k + 3], v, true);
            }
        } else {
            c[0] = c[1] = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int q = (int)fmin(fmax(rint(y[e] * inv), -127.0), 127.0);
                c[e / 4] |= (uint32_t)(q & 0xff) << (e % 4 * 8);
            }
        }
        uint8_t *const to = (uint8_t *)p.y + at0 + at;
        if (wide) {
            if (at < D) *(u32x2 *)to = u32x2{c[0], c[1]};
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (at + e < D) to[e] = (uint8_t)(c[e / 4] >> (e % 4 * 8));
        }
    }
}

// Every row set (a block, or a wave of one) takes rows at a distance and keeps its sum of dweight.
template <typename T, typename R, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) k_bwd(NormBwdArgs p, int sets, bool wide) {
    constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
    __shared__ double part[TPR > 64 ? TPR / 64 : 1];
    const int tid = threadIdx.x % TPR, set = blockIdx.x * kRows + threadIdx.x / TPR, D = p.dim;
    if (set >= sets) return;
    float dw[NV][E] = {};
    for (int64_t row = set; row < p.rows; row += sets) {
        const int64_t at0 = row * D;
        const float r = p.rstd[row];
        float n[NV][E], wd[NV][E];
        double sum = 0.0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int at = (tid + k * TPR) * E;
            float w[E];
            load8((const R *)p.s + at0, at, D, wide, n[k]);
            load8((const T *)p.dy + at0, at, D, wide, wd[k]);
            load8(p.weight, at, D, wide, w);
            float t = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                n[k][e] *= r;
                dw[k][e] += wd[k][e] * n[k][e];
                wd[k][e] *= w[e];
                t += wd[k][e] * n[k][e];
            }
            sum += t;
        }
        const float c = (float)(row_sum<TPR>(sum, part) / D);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int at = (tid + k * TPR) * E;
            float g[E];
            if (p.ds) {
                load8((const R *)p.ds + at0, at, D, wide, g);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) g[e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) g[e] += (wd[k][e] - n[k][e] * c) * r;
            store8((T *)p.dx + at0, at, D, wide, g);
            if (p.dres) store8((R *)p.dres + at0, at, D, wide, g);
        }
    }
    float *const to = (float *)p.ws + (int64_t)set * D;
#pragma unroll
    for (int k = 0; k < NV; ++k) store8(to, (tid + k * TPR) * E, D, wide, dw[k]);
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

// WIDE: 8 codes a thread (a group is a multiple of 8), else one.
template <bool WIDE>
__global__ void __launch_bounds__(256) k_values(const uint8_t *codes, const float *scales, float *out, int64_t rows, int D, int group,
                                                int code) {
    constexpr int N = WIDE ? 8 : 1;
    const uint32_t per_row = D / N, groups = group ? (D + group - 1) / group : 1;
    const int64_t n = rows * per_row, stride = (int64_t)gridDim.x * 256;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += stride) {
        const int64_t row = n <= 0xffffffff ? (uint32_t)e / per_row : e / per_row;
        const int at = (int)(e - row * per_row) * N;
        const float scale = scales[row * groups + (group ? at / group : 0)];
        if constexpr (WIDE) {
            const u32x2 c = *(const u32x2 *)(codes + e * 8);
            float v[8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (code == 1) {
                    v[4 * k] = __builtin_amdgcn_cvt_f32_fp8((int)c[k], 0);
                    v[4 * k + 1] = __builtin_amdgcn_cvt_f32_fp8((int)c[k], 1);
                    v[4 * k + 2] = __builtin_amdgcn_cvt_f32_fp8((int)c[k], 2);
                    v[4 * k + 3] = __builtin_amdgcn_cvt_f32_fp8((int)c[k], 3);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[4 * k + j] = (float)(int8_t)(c[k] >> (8 * j));
                }
            }
            float4 *const to = (float4 *)(out + e * 8);
            to[0] = make_float4(v[0] * scale, v[1] * scale, v[2] * scale, v[3] * scale);
            to[1] = make_float4(v[4] * scale, v[5] * scale, v[6] * scale, v[7] * scale);
        } else {
            out[e] = (code == 1 ? __builtin_amdgcn_cvt_f32_fp8((int)codes[e], 0) : (float)(int8_t)codes[e]) * scale;
        }
    }
}

bool aligned_to(const void *p, size_t n) { return (uintptr_t)p % n == 0; }

// Threads of a row: a wave up to 1024 elements, 256 up to 8192, 1024 up to 65536.
template <typename F>
void by_size(int D, F go) {
    typedef std::integral_constant<int, 64> W;
    typedef std::integral_constant<int, 256> B;
    typedef std::integral_constant<int, 1024> L;
    if (D <= 512) go(W(), std::integral_constant<int, 1>());
    else if (D <= 1024) go(W(), std::integral_constant<int, 2>());
    else if (D <= 2048) go(B(), std::integral_constant<int, 1>());
    else if (D <= 4096) go(B(), std::integral_constant<int, 2>());
    else if (D <= 8192) go(B(), std::integral_constant<int, 4>());
    else if (D <= 16384) go(L(), std::integral_constant<int, 2>());
    else if (D <= 32768) go(L(), std::integral_constant<int, 4>());
    else go(L(), std::integral_constant<int, 8>());
}

template <typename T, typename R>
void run_fwd(const NormArgs &a, hipStream_t s) {
    const bool wide = a.dim % E == 0 && aligned_to(a.x, 16) && aligned_to(a.residual, 16) && aligned_to(a.added, 16) &&
                      aligned_to(a.weight, 16) && aligned_to(a.y, a.code ? 8 : 16);
    by_size(a.dim, [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value, kThreads = TPR < 256 ? 256 : TPR;
        const int64_t blocks = (a.rows + kThreads / TPR - 1) / (kThreads / TPR);
        k_fwd<T, R, TPR, NV><<<blocks, kThreads, 0, s>>>(a, wide);
    });
}

// Row sets of the backward: enough for the GPU, each with several rows where there are many.
int row_sets(int64_t rows, int32_t dim) {
    return (int)std::max<int64_t>(1, std::min<int64_t>(rows, dim <= 1024 ? 2048 : dim <= 8192 ? 512 : 256));
}

template <typename T, typename R>
void run_bwd(const NormBwdArgs &a, hipStream_t s) {
    const bool wide = a.dim % E == 0 && aligned_to(a.s, 16) && aligned_to(a.dy, 16) && aligned_to(a.ds, 16) &&
                      aligned_to(a.weight, 16) && aligned_to(a.dx, 16) && aligned_to(a.dres, 16);
    const int sets = row_sets(a.rows, a.dim);
    by_size(a.dim, [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value, kThreads = TPR < 256 ? 256 : TPR;
        const int blocks = (sets + kThreads / TPR - 1) / (kThreads / TPR);
        k_bwd<T, R, TPR, NV><<<blocks, kThreads, 0, s>>>(a, sets, wide);
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
    const bool wide = dim % 8 == 0 && aligned_to(codes, 8) && aligned_to(out, 16);
    const int64_t blocks = std::min<int64_t>((rows * dim / (wide ? 8 : 1) + 255) / 256, 1 << 20);
    if (wide) k_values<true><<<blocks, 256, 0, s>>>((const uint8_t *)codes, scales, out, rows, dim, group, code);
    else k_values<false><<<blocks, 256, 0, s>>>((const uint8_t *)codes, scales, out, rows, dim, group, code);
    return hipGetLastError();
}

}  // namespace ssm
