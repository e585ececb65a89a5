// adamw.hip -- one AdamW step over many tensors, moments in float32 or in 8-bit codes.
//
// The launch's tensors travel in the kernel arguments, so a step needs no copy of a table and
// no workspace. A thread block of 256 works on kPer blocks of 256 values of one tensor, which
// it finds by bisection over the tensors' first thread blocks (uniform, in scalar registers).
// Every operation is one IEEE float32 operation in the order of ssm_scan.h (contraction is
// off, divisions and square roots are the correctly rounded ones): an 8-bit code flips where
// an input of its rounding moves by an ulp, so only a fixed order gives reproducible codes.
#include "ssm_device.h"
#include "ssm_train.h"

namespace ssm {
namespace {

constexpr int kBlock = SSM_ADAMW_BLOCK;
constexpr int kPer = 8;

__device__ __forceinline__ float ld_any(const void *p, int64_t e, bool bf16) {
    return bf16 ? Io<bf16_bits>::ld((const bf16_bits *)p + e) : ((const float *)p)[e];
}

// The largest of a value over the 256 threads; a NaN anywhere gives NaN.
__device__ __forceinline__ float block_max(float v, float *sh) {
    for (int o = 32; o > 0; o >>= 1) {
        const float w = __shfl_xor(v, o);
        v = v > w || v != v ? v : w;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = sh[0];
    for (int k = 1; k < 4; ++k) v = v > sh[k] || v != v ? v : sh[k];
    return v;
}

constexpr float kScaleMin = 1e-35f;

template <bool CODES>
__global__ void __launch_bounds__(kBlock) k_adamw(AdamwArgs a) {
    __shared__ float sh[4];
    int lo = 0, hi = a.n_tensors;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if ((int)blockIdx.x >= a.t[mid].block0) lo = mid;
        else hi = mid;
    }
    const AdamwTensor t = a.t[lo];
    const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
    const int64_t base = (int64_t)((int)blockIdx.x - t.block0) * (kPer * kBlock);
    for (int j = 0; j < kPer; ++j) {
        const int64_t e = base + j * kBlock + threadIdx.x;
        if (base + j * kBlock >= t.n) break;  // the same for every thread
        const bool in = e < t.n;
        const int64_t s = t.at + e;
        float m = 0.0f, v = 0.0f;
        if (CODES) {
            const float u = (float)((const int8_t *)a.m)[s] * (float)(1.0 / 127.0);
            float w = (float)((const uint8_t *)a.v)[s] * (float)(1.0 / 255.0);
            w = w * w;
            m = a.m_scale[s / kBlock] * (u * fabsf(u));
            v = a.v_scale[s / kBlock] * (w * w);
        } else if (in) {
            m = ((const float *)a.m)[s];
            v = ((const float *)a.v)[s];
        }
        if (in) {
            const float g = ld_any(t.g, e, t.io & 2) * gs;
            m = m * a.beta1 + g * a.omb1;
            v = v * a.beta2 + (g * a.omb2) * g;
            const float denom = sqrtf(v) * a.rs2 + a.eps;
            const float p = ld_any(t.p, e, t.io & 1) * a.keep - (m / denom) * a.rate;
            if (t.io & 1) Io<bf16_bits>::st((bf16_bits *)t.p + e, p);
            else ((float *)t.p)[e] = p;
        } else {
            m = v = 0.0f;
        }
        if (!CODES) {
            if (in) {
                ((float *)a.m)[s] = m;
                ((float *)a.v)[s] = v;
            }
            continue;
        }
        float ms = block_max(fabsf(m), sh), vs = block_max(v, sh);
        ms = ms < kScaleMin ? 0.0f : ms;
        vs = vs < kScaleMin ? 0.0f : vs;
        const float mi = ms == 0.0f ? 0.0f : 1.0f / ms, vi = vs == 0.0f ? 0.0f : 1.0f / vs;
        const float um = fminf(rintf(sqrtf(fabsf(m) * mi) * 127.0f), 127.0f);
        const float r = v * vi;
        float uv = fminf(rintf(sqrtf(sqrtf(r)) * 255.0f), 255.0f);
        if (r > 0.0f) uv = fmaxf(uv, 1.0f);
        // a NaN leaves fminf as 127 or 255: its block's scale is NaN or infinite, and so
        // are all its values
        ((int8_t *)a.m)[s] = (int8_t)(m < 0.0f ? -um : m > 0.0f ? um : m != m ? 127.0f : 0.0f);
        ((uint8_t *)a.v)[s] = (uint8_t)uv;
        if (threadIdx.x == 0) {
            a.m_scale[s / kBlock] = ms;
            a.v_scale[s / kBlock] = vs;
        }
    }
}

__global__ void __launch_bounds__(256) k_adamw_values(const int8_t *m, const uint8_t *v, const float *ms,
                                                      const float *vs, float *mo, float *vo, int64_t n) {
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (e >= n) return;
    const float u = (float)m[e] * (float)(1.0 / 127.0);
    float w = (float)v[e] * (float)(1.0 / 255.0);
    w = w * w;
    mo[e] = ms[e / kBlock] * (u * fabsf(u));
    vo[e] = vs[e / kBlock] * (w * w);
}

}  // namespace

int32_t adamw_blocks(int64_t n, bool) { return (int32_t)((n + kPer * kBlock - 1) / (kPer * kBlock)); }

hipError_t launch_adamw(const AdamwArgs &a, int32_t blocks, hipStream_t s) {
    if (a.m_scale) k_adamw<true><<<dim3((unsigned)blocks), kBlock, 0, s>>>(a);
    else k_adamw<false><<<dim3((unsigned)blocks), kBlock, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_adamw_values(const int8_t *m, const uint8_t *v, const float *ms, const float *vs, float *mo,
                               float *vo, int64_t n, hipStream_t s) {
    k_adamw_values<<<dim3((unsigned)((n + 255) / 256)), 256, 0, s>>>(m, v, ms, vs, mo, vo, n);
    return hipGetLastError();
}

}  // namespace ssm
