// gated.hip -- the gated linear recurrence: forward, backward and the single token.
//
//     k_t = c softplus(decay) sigmoid(r_t),  a_t = exp(-k_t),  beta_t = sqrt(1 - a_t^2)
//     h_t = a_t h_{t-1} + beta_t sigmoid(i_t) x_t,  y_t = h_t       (h_{t-1} = 0 at a reset)
// Backward, with g_t = dLoss/dh_t:
//     g_t = dy_t + a_{t+1} g_{t+1}
//     dx = g beta si,  di = g beta x si (1 - si)
//     kd = k dLoss/dk = g (a^2 (k / beta) si x - k a h_{t-1}),  dr = kd (1 - sr)
//     ddecay = sum kd sigmoid(decay) / softplus(decay),  dh0 = a_1 g_1
#include "ssm_device.h"
#include "ssm_train.h"

namespace ssm {
namespace {

// 1 - a^2 = -expm1(-2k) with relative precision: its series below 2k = 1/4 (the first term
// left out is below 5e-8 of the sum), 1 - a a above, where nothing cancels by more than a
// factor of 5.
__device__ __forceinline__ float one_minus_a2(float k, float a) {
    const float x = k + k;
    float p = fmaf(x, -1.0f / 6.0f, 1.0f);
    p = fmaf(x * p, -1.0f / 5.0f, 1.0f);
    p = fmaf(x * p, -1.0f / 4.0f, 1.0f);
    p = fmaf(x * p, -1.0f / 3.0f, 1.0f);
    p = fmaf(x * p, -1.0f / 2.0f, 1.0f);
    return x < 0.25f ? x * p : fmaf(-a, a, 1.0f);
}
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.0f + e2(-v * kLog2e)); }
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))); }

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

constexpr int kThreads = 64;

template <typename IO>
__global__ void __launch_bounds__(kThreads) k_gated_fwd(GatedArgs p) {
    const int64_t d = (int64_t)blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y;
    if (d >= p.D) return;
    const float ck = p.c * softplus(p.decay[d]);
    const int64_t rows = (p.L + SSM_GATED_STATE_EVERY - 1) / SSM_GATED_STATE_EVERY;
    float h = p.h0 ? p.h0[b * p.D + d] : 0.0f;
    for (int64_t t = 0; t < p.L; ++t) {
        const int64_t e = (b * p.L + t) * p.D + d;
        if (p.states && t % SSM_GATED_STATE_EVERY == 0)
            p.states[(b * rows + t / SSM_GATED_STATE_EVERY) * p.D + d] = h;
        const Gate g = gate(Io<IO>::ld((const IO *)p.r + e), Io<IO>::ld((const IO *)p.i + e), ck);
        const float in = g.beta * g.si * Io<IO>::ld((const IO *)p.x + e);
        h = p.reset && p.reset[b * p.L + t] ? in : fmaf(g.a, h, in);
        Io<IO>::st((IO *)p.y + e, h);
    }
    if (p.h_final) p.h_final[b * p.D + d] = h;
}

template <typename IO>
__global__ void __launch_bounds__(kThreads) k_gated_bwd(GatedArgs p) {
    const int64_t d = (int64_t)blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y;
    if (d >= p.D) return;
    const float ck = p.c * softplus(p.decay[d]);
    const int64_t rows = (p.L + SSM_GATED_STATE_EVERY - 1) / SSM_GATED_STATE_EVERY;
    float u = p.dh_final ? p.dh_final[b * p.D + d] : 0.0f, sum = 0.0f;
    float before[SSM_GATED_STATE_EVERY];
    for (int64_t row = rows - 1; row >= 0; --row) {
        const int64_t t0 = row * SSM_GATED_STATE_EVERY;
        const int n = (int)min((int64_t)SSM_GATED_STATE_EVERY, p.L - t0);
        float h = p.states[(b * rows + row) * p.D + d];
        for (int j = 0; j < n; ++j) {
            const int64_t e = (b * p.L + t0 + j) * p.D + d;
            before[j] = h;
            const Gate g = gate(Io<IO>::ld((const IO *)p.r + e), Io<IO>::ld((const IO *)p.i + e), ck);
            const float in = g.beta * g.si * Io<IO>::ld((const IO *)p.x + e);
            h = p.reset && p.reset[b * p.L + t0 + j] ? in : fmaf(g.a, h, in);
        }
        for (int j = n - 1; j >= 0; --j) {
            const int64_t e = (b * p.L + t0 + j) * p.D + d;
            const bool cut = p.reset && p.reset[b * p.L + t0 + j];
            const Gate g = gate(Io<IO>::ld((const IO *)p.r + e), Io<IO>::ld((const IO *)p.i + e), ck);
            const float x = Io<IO>::ld((const IO *)p.x + e);
            const float gt = Io<IO>::ld((const IO *)p.dy + e) + u;
            const float gb = gt * g.beta, kb = g.beta > 0.0f ? g.k / g.beta : 0.0f;
            const float ah = cut ? 0.0f : g.a * before[j];
            const float kd = gt * (g.a * g.a * kb * g.si * x - g.k * ah);
            Io<IO>::st((IO *)p.dx + e, gb * g.si);
            Io<IO>::st((IO *)p.di + e, gb * x * g.si * (1.0f - g.si));
            Io<IO>::st((IO *)p.dr + e, kd * (1.0f - g.sr));
            sum += kd;
            u = cut ? 0.0f : g.a * gt;
        }
    }
    if (p.dh0) p.dh0[b * p.D + d] = u;
    ((float *)p.ws)[b * p.D + d] = sum;
}

// ddecay[d] = sigmoid(decay) / softplus(decay) * sum over n partial rows, in order.
__global__ void __launch_bounds__(kThreads) k_gated_ddecay(const float *part, const float *decay, float *out,
                                                           int64_t n, int64_t D) {
    const int64_t d = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (d >= D) return;
    float s = 0.0f;
    for (int64_t j = 0; j < n; ++j) s += part[j * D + d];
    const float sp = softplus(decay[d]);  // 0 where exp(decay) underflows: the ratio tends to 1
    out[d] = s * (sp > 0.0f ? 1.0f / (1.0f + expf(-decay[d])) / sp : 1.0f);
}

// dst = src (or 0), n floats.
__global__ void __launch_bounds__(256) k_fill(float *dst, const float *src, int64_t n) {
    const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (j < n) dst[j] = src ? src[j] : 0.0f;
}
hipError_t fill(float *dst, const float *src, int64_t n, hipStream_t s) {
    if (dst && n > 0) k_fill<<<dim3((unsigned)((n + 255) / 256)), 256, 0, s>>>(dst, src, n);
    return hipGetLastError();
}

// One token: a lane per (layer, sequence, channel).
template <typename IO>
__global__ void __launch_bounds__(256) k_gated_step(GatedStepArgs p) {
    const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (d >= p.D) return;
    const int64_t e = ((int64_t)blockIdx.z * p.n_seq + blockIdx.y) * p.D + d;
    const float ck = p.c * softplus(p.decay[(int64_t)blockIdx.z * p.D + d]);
    const Gate g = gate(Io<IO>::ld((const IO *)p.r + e), Io<IO>::ld((const IO *)p.i + e), ck);
    const float h = fmaf(g.a, p.h[e], g.beta * g.si * Io<IO>::ld((const IO *)p.x + e));
    p.h[e] = h;
    Io<IO>::st((IO *)p.y + e, h);
}

}  // namespace

size_t gated_fwd_ws(int64_t, int64_t, int64_t) { return 0; }
size_t gated_bwd_ws(int64_t batch, int64_t L, int64_t D) {
    return L > 0 ? round_up((size_t)batch * D * sizeof(float), kTrainWsAlign) : 0;
}

hipError_t launch_gated_fwd(const GatedArgs &a, int io, hipStream_t s) {
    if (a.L == 0) return fill(a.h_final, a.h0, a.batch * a.D, s);
    const dim3 grid((unsigned)((a.D + kThreads - 1) / kThreads), (unsigned)a.batch);
    if (io) k_gated_fwd<bf16_bits><<<grid, kThreads, 0, s>>>(a);
    else k_gated_fwd<float><<<grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_gated_bwd(const GatedArgs &a, int io, hipStream_t s) {
    if (a.L == 0 || a.batch == 0) {
        const hipError_t e = fill(a.dh0, a.dh_final, a.batch * a.D, s);
        return e != hipSuccess ? e : fill(a.ddecay, nullptr, a.D, s);
    }
    const dim3 grid((unsigned)((a.D + kThreads - 1) / kThreads), (unsigned)a.batch);
    if (io) k_gated_bwd<bf16_bits><<<grid, kThreads, 0, s>>>(a);
    else k_gated_bwd<float><<<grid, kThreads, 0, s>>>(a);
    k_gated_ddecay<<<dim3(grid.x), kThreads, 0, s>>>((const float *)a.ws, a.decay, a.ddecay, a.batch, a.D);
    return hipGetLastError();
}

hipError_t launch_gated_step(const GatedStepArgs &a, int io, hipStream_t s) {
    const dim3 grid((unsigned)((a.D + 255) / 256), (unsigned)a.n_seq, (unsigned)a.n_layers);
    if (io) k_gated_step<bf16_bits><<<grid, 256, 0, s>>>(a);
    else k_gated_step<float><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace ssm
