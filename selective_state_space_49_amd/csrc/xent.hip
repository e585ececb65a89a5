// xent.hip -- softmax cross entropy of a linear head over a vocabulary, without keeping the
// logits, and its gradients.
//
// Forward: each thread block makes a 64 x 64 tile of logits and leaves its rows' maximum and
// sum of exponentials; a second kernel joins a token's partial pairs (m, s), (m', s') to
// M = max(m, m'), s e^(m-M) + s' e^(m'-M).
// Backward: for a piece of the vocabulary at a time, dlogits = w (exp(logit - lse) - onehot)
// go to the workspace, and two products make this piece's rows of dweight and add to dhidden.
#include <math.h>

#include <algorithm>

#include "ssm_device.h"
#include "ssm_train.h"

namespace ssm {
namespace {

constexpr int kTile = 64, kDepth = 16;
constexpr int64_t kPiece = 2048;  // vocabulary rows of one piece of the backward

// acc[i][j] += sum_k A(row0 + 4 ty + i, k) B(col0 + 4 tx + j, k) for k < K, in 256 threads;
// la, lb load one element (0 outside).
template <typename LA, typename LB>
__device__ __forceinline__ void tile_product(float (&acc)[4][4], int64_t K, LA la, LB lb) {
    __shared__ float sa[kDepth][kTile + 1], sb[kDepth][kTile + 1];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    for (int64_t k0 = 0; k0 < K; k0 += kDepth) {
        for (int e = tid; e < kTile * kDepth; e += 256) {
            const int k = e % kDepth, m = e / kDepth;
            sa[k][m] = k0 + k < K ? la(m, k0 + k) : 0.0f;
            sb[k][m] = k0 + k < K ? lb(m, k0 + k) : 0.0f;
        }
        __syncthreads();
        for (int k = 0; k < kDepth; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][4 * ty + i], sb[k][4 * tx + j], acc[i][j]);
        __syncthreads();
    }
}

struct Shape {
    int64_t T, K, V;
};

template <typename IO>
__device__ __forceinline__ void logits_tile(float (&acc)[4][4], const void *hidden, const void *weight, Shape n,
                                            int64_t t0, int64_t v0) {
    tile_product(
        acc, n.K,
        [&](int m, int64_t k) { return t0 + m < n.T ? Io<IO>::ld((const IO *)hidden + (t0 + m) * n.K + k) : 0.0f; },
        [&](int m, int64_t k) { return v0 + m < n.V ? Io<IO>::ld((const IO *)weight + (v0 + m) * n.K + k) : 0.0f; });
}

// part[t][tile] = (max, sum of exp(logit - max)) over the tile's columns; at[t] = the
// target's logit.
template <typename IO>
__global__ void __launch_bounds__(256) k_xent_part(const void *hidden, const void *weight, const int64_t *targets,
                                                   Shape n, float2 *part, float *at) {
    const int64_t t0 = (int64_t)blockIdx.y * kTile, v0 = (int64_t)blockIdx.x * kTile;
    float acc[4][4] = {};
    logits_tile<IO>(acc, hidden, weight, n, t0, v0);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + 4 * ty + i;
        float m = -INFINITY;
        for (int j = 0; j < 4; ++j)
            if (v0 + 4 * tx + j < n.V) m = m > acc[i][j] || m != m ? m : acc[i][j];
        for (int o = 8; o > 0; o >>= 1) {
            const float w = __shfl_xor(m, o);
            m = m > w || m != m ? m : w;
        }
        float s = 0.0f;
        for (int j = 0; j < 4; ++j)
            if (v0 + 4 * tx + j < n.V) s += m == -INFINITY ? 0.0f : e2((acc[i][j] - m) * kLog2e);
        for (int o = 8; o > 0; o >>= 1) s += __shfl_xor(s, o);
        if (t >= n.T) continue;
        if (tx == 0) part[t * gridDim.x + blockIdx.x] = make_float2(m, s);
        const int64_t y = targets[t] - (v0 + 4 * tx);
        if (y >= 0 && y < 4) at[t] = y < 2 ? (y == 0 ? acc[i][0] : acc[i][1]) : (y == 2 ? acc[i][2] : acc[i][3]);
    }
}

// A wave per token joins its partial pairs.
__global__ void __launch_bounds__(64) k_xent_join(const float2 *part, const float *at, const int64_t *targets,
                                                  int64_t ignore, Shape n, int64_t tiles, float *loss, float *lse) {
    const int64_t t = blockIdx.x;
    float m = -INFINITY, s = 0.0f;
    for (int64_t j = threadIdx.x; j < tiles; j += 64) {
        const float2 q = part[t * tiles + j];
        const float M = m > q.x || m != m ? m : q.x;
        const float f = m == M ? 1.0f : e2((m - M) * kLog2e), g = q.x == M ? 1.0f : e2((q.x - M) * kLog2e);
        s = s * f + q.y * g;
        m = M;
    }
    for (int o = 32; o > 0; o >>= 1) {
        const float m2 = __shfl_xor(m, o), s2 = __shfl_xor(s, o);
        const float M = m > m2 || m != m ? m : m2;
        const float f = m == M ? 1.0f : e2((m - M) * kLog2e), g = m2 == M ? 1.0f : e2((m2 - M) * kLog2e);
        s = s * f + s2 * g;
        m = M;
    }
    if (threadIdx.x) return;
    const float l = m + logf(s);
    const int64_t y = targets[t];
    lse[t] = l;
    loss[t] = y == ignore ? 0.0f : y >= 0 && y < n.V ? l - at[t] : NAN;
}

// mean[0] = mean loss over the tokens that are not ignored, mean[1] = 1 / their number.
__global__ void __launch_bounds__(1024) k_xent_mean(const float *loss, const int64_t *targets, int64_t ignore,
                                                    int64_t T, float *mean) {
    __shared__ double sh[1024];
    __shared__ int64_t sn[1024];
    double s = 0.0;
    int64_t c = 0;
    for (int64_t t = threadIdx.x; t < T; t += 1024)
        if (targets[t] != ignore) {
            s += loss[t];
            ++c;
        }
    sh[threadIdx.x] = s;
    sn[threadIdx.x] = c;
    __syncthreads();
    for (int o = 512; o > 0; o >>= 1) {
        if ((int)threadIdx.x < o) {
            sh[threadIdx.x] += sh[threadIdx.x + o];
            sn[threadIdx.x] += sn[threadIdx.x + o];
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        mean[0] = sn[0] ? (float)(sh[0] / (double)sn[0]) : 0.0f;
        mean[1] = sn[0] ? (float)(1.0 / (double)sn[0]) : 0.0f;
    }
}

// g[t][v - v0] = w_t (exp(logit - lse_t) - [v == target]) for one piece of n_v columns.
template <typename IO>
__global__ void __launch_bounds__(256) k_xent_dlogits(XentArgs a, int64_t v0, int64_t n_v, float *g, int64_t ldg) {
    const int64_t t0 = (int64_t)blockIdx.y * kTile, c0 = (int64_t)blockIdx.x * kTile;
    float acc[4][4] = {};
    const Shape n{a.T, a.K, v0 + n_v};
    logits_tile<IO>(acc, a.hidden, a.weight, n, t0, v0 + c0);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + 4 * ty + i;
        if (t >= a.T) continue;
        const int64_t y = a.targets[t];
        const bool skip = y == a.ignore, bad = !skip && (y < 0 || y >= a.V);
        float w = (a.dloss ? a.dloss[t] : 0.0f) + (a.dmean ? *a.dmean * a.mean[1] : 0.0f);
        if (bad) w = NAN;
        for (int j = 0; j < 4; ++j) {
            const int64_t c = c0 + 4 * tx + j;
            if (c >= n_v) continue;
            const float q = e2((acc[i][j] - a.lse[t]) * kLog2e) - (y == v0 + c ? 1.0f : 0.0f);
            g[t * ldg + c] = skip ? 0.0f : w * q;
        }
    }
}

// dweight rows [v0, v0 + n_v) = g^T hidden.
template <typename IO>
__global__ void __launch_bounds__(256) k_xent_dweight(XentArgs a, int64_t v0, int64_t n_v, const float *g, int64_t ldg) {
    const int64_t r0 = (int64_t)blockIdx.y * kTile, c0 = (int64_t)blockIdx.x * kTile;
    float acc[4][4] = {};
    tile_product(
        acc, a.T, [&](int m, int64_t t) { return r0 + m < n_v ? g[t * ldg + r0 + m] : 0.0f; },
        [&](int m, int64_t t) {  // an ignored token's hidden row may hold anything
            return c0 + m < a.K && a.targets[t] != a.ignore ? Io<IO>::ld((const IO *)a.hidden + t * a.K + c0 + m) : 0.0f;
        });
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + 4 * ty + i, c = c0 + 4 * tx + j;
            if (r < n_v && c < a.K) Io<IO>::st((IO *)a.dweight + (v0 + r) * a.K + c, acc[i][j]);
        }
}

// sum (+)= g weight[v0 ..]; the last piece writes dhidden.
template <typename IO>
__global__ void __launch_bounds__(256) k_xent_dhidden(XentArgs a, int64_t v0, int64_t n_v, const float *g, int64_t ldg,
                                                      float *sum, bool first, bool last) {
    const int64_t r0 = (int64_t)blockIdx.y * kTile, c0 = (int64_t)blockIdx.x * kTile;
    float acc[4][4] = {};
    tile_product(
        acc, n_v, [&](int m, int64_t v) { return r0 + m < a.T ? g[(r0 + m) * ldg + v] : 0.0f; },
        [&](int m, int64_t v) {
            return c0 + m < a.K ? Io<IO>::ld((const IO *)a.weight + (v0 + v) * a.K + c0 + m) : 0.0f;
        });
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + 4 * ty + i, c = c0 + 4 * tx + j;
            if (r >= a.T || c >= a.K) continue;
            const float q = first ? acc[i][j] : sum[r * a.K + c] + acc[i][j];
            if (last) Io<IO>::st((IO *)a.dhidden + r * a.K + c, q);
            else sum[r * a.K + c] = q;
        }
}

template <typename IO>
__global__ void __launch_bounds__(256) k_zero(IO *p, int64_t n) {
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e < n) p[e] = IO(0);
}

unsigned tiles(int64_t n) { return (unsigned)((n + kTile - 1) / kTile); }

template <typename IO>
hipError_t xent_fwd(const XentArgs &a, hipStream_t s) {
    if (a.T > 0) {
        const Shape n{a.T, a.K, a.V};
        float2 *part = (float2 *)a.ws;
        float *at = (float *)(part + (size_t)a.T * tiles(a.V));
        k_xent_part<IO><<<dim3(tiles(a.V), tiles(a.T)), 256, 0, s>>>(a.hidden, a.weight, a.targets, n, part, at);
        k_xent_join<<<dim3((unsigned)a.T), 64, 0, s>>>(part, at, a.targets, a.ignore, n, tiles(a.V), a.loss, a.lse);
    }
    k_xent_mean<<<dim3(1), 1024, 0, s>>>(a.loss, a.targets, a.ignore, a.T, a.mean);
    return hipGetLastError();
}

template <typename IO>
hipError_t xent_bwd(const XentArgs &a, hipStream_t s) {
    if (a.T == 0) {
        if (a.dweight)
            k_zero<IO><<<dim3((unsigned)((a.V * a.K + 255) / 256)), 256, 0, s>>>((IO *)a.dweight, a.V * a.K);
        return hipGetLastError();
    }
    const int64_t ldg = std::min(a.V, kPiece);
    float *g = (float *)a.ws, *sum = g + (size_t)a.T * ldg;
    for (int64_t v0 = 0; v0 < a.V; v0 += kPiece) {
        const int64_t n_v = std::min(kPiece, a.V - v0);
        k_xent_dlogits<IO><<<dim3(tiles(n_v), tiles(a.T)), 256, 0, s>>>(a, v0, n_v, g, ldg);
        if (a.dweight) k_xent_dweight<IO><<<dim3(tiles(a.K), tiles(n_v)), 256, 0, s>>>(a, v0, n_v, g, ldg);
        if (a.dhidden)
            k_xent_dhidden<IO><<<dim3(tiles(a.K), tiles(a.T)), 256, 0, s>>>(a, v0, n_v, g, ldg, sum, v0 == 0,
                                                                           v0 + n_v == a.V);
    }
    return hipGetLastError();
}

}  // namespace

size_t xent_fwd_ws(int64_t T, int64_t, int64_t V, int) {
    return round_up((size_t)T * (tiles(V) * sizeof(float2) + sizeof(float)), kTrainWsAlign);
}
size_t xent_bwd_ws(int64_t T, int64_t K, int64_t V, int) {
    return round_up((size_t)T * (std::min(V, kPiece) + K) * sizeof(float), kTrainWsAlign);
}
hipError_t launch_xent_fwd(const XentArgs &a, int io, hipStream_t s) {
    return io ? xent_fwd<bf16_bits>(a, s) : xent_fwd<float>(a, s);
}
hipError_t launch_xent_bwd(const XentArgs &a, int io, hipStream_t s) {
    return io ? xent_bwd<bf16_bits>(a, s) : xent_bwd<float>(a, s);
}

}  // namespace ssm
