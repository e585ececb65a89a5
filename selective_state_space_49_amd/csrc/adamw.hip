// adamw.hip -- one AdamW step over many tensors, moments in float32 or in 8-bit codes.
//
// The launch's tensors travel in the kernel arguments, so a step needs no copy of a table and
// no workspace. A thread block works on kPer blocks of 256 values of one tensor, which it
// finds by bisection over the tensors' first thread blocks (uniform, in scalar registers). A
// wave has a block of 256 values, four a lane, so that a block's scale is a reduction within
// the wave and nothing meets in LDS.
//
// Every operation is one IEEE float32 operation in the order of ssm_scan.h (contraction is
// off, divisions and square roots are the correctly rounded ones): an 8-bit code flips where
// an input of its rounding moves by an ulp, so only a fixed order gives reproducible codes.
// With 8-bit moments an element has four square roots and a division, and the kernel is bound
// by its vector instructions (99 an element; 112 with the compiler's general forms): 236 M
// bfloat16 parameters take 0.53 ms, 2.4 GB at 4.5 TB/s. With float32 ones it is bound by the
// bytes: 282 tensors of 13.3 M parameters, 373 MB, take 86 us. The roots of the codes go through the hardware's approximation, and only
// where a rounding could depend on its last bits are they made again exactly (m_code, v_code);
// the root and the division of the update have short exact forms for the range in which all
// but exotic values lie (sqrt_in_range, div_in_range), and the general ones outside.
#include "ssm_device.h"
#include "ssm_train.h"

namespace ssm {
namespace {

constexpr int kBlock = SSM_ADAMW_BLOCK;
constexpr int kPer = 8;      // blocks of 256 values of a thread block: two for each of its waves
constexpr int kUnroll = kPer / 4;
constexpr float kScaleMin = 1e-35f;
static_assert(kBlock == 64 * 4, "a wave holds a block, four values a lane");

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef int8_t i8x4 __attribute__((ext_vector_type(4)));
typedef uint8_t u8x4 __attribute__((ext_vector_type(4)));

// The largest of non-negative values by their bits, which order like the values; a NaN's (its
// sign cleared) lie above all of them, so it stays.
__device__ __forceinline__ uint32_t bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
// Over the wave, uniform: rotations within rows of 16 lanes, then row to row (row_ror 0x120 + n,
// row_bcast 0x142 and 0x143), and the last lane has it.
__device__ __forceinline__ float wave_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)v, 63));
}

// Four values from e on; n of them exist. vec: all four, aligned.
__device__ __forceinline__ f32x4 load4(const void *p, int64_t e, bool bf16, bool vec, int n) {
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (vec) {
        if (!bf16) return *(const f32x4 *)((const float *)p + e);
        const u16x4 w = *(const u16x4 *)((const bf16_bits *)p + e);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = bf16_to_f32(w[c]);
        return v;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (c < n) v[c] = bf16 ? Io<bf16_bits>::ld((const bf16_bits *)p + e + c) : ((const float *)p)[e + c];
    return v;
}
__device__ __forceinline__ void store4(void *p, int64_t e, bool bf16, bool vec, int n, f32x4 v) {
    if (vec) {
        if (bf16) {
            u16x4 w;
#pragma unroll
            for (int c = 0; c < 4; ++c) w[c] = f32_to_bf16(v[c]);
            *(u16x4 *)((bf16_bits *)p + e) = w;
        } else {
            *(f32x4 *)((float *)p + e) = v;
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
        if (c < n) {
            if (bf16) Io<bf16_bits>::st((bf16_bits *)p + e + c, v[c]);
            else ((float *)p)[e + c] = v[c];
        }
}

__device__ __forceinline__ f32x4 m_values(i8x4 q, float scale) {
    f32x4 v;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float u = (float)q[c] * (float)(1.0 / 127.0);
        v[c] = scale * (u * fabsf(u));
    }
    return v;
}
__device__ __forceinline__ f32x4 v_values(u8x4 q, float scale) {
    f32x4 v;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        float w = (float)q[c] * (float)(1.0 / 255.0);
        w = w * w;
        v[c] = scale * (w * w);
    }
    return v;
}

// Correctly rounded sqrt(v) and m / d without the general forms' scaling and special cases:
// v is 0 or in [2^-96, 2^96], |m| is 0 or in [2^-60, 2^60], d in [2^-60, 2^60] (in_range).
// Each ends with the exact remainder of a value that is right to within an ulp, times an
// approximate root or reciprocal.
__device__ __forceinline__ float sqrt_in_range(float v) {
    const float y = __builtin_amdgcn_rsqf(fmaxf(v, 0x1p-100f));
    float g = v * y, h = 0.5f * y;
    const float r = fmaf(-g, h, 0.5f);
    g = fmaf(g, r, g);
    h = fmaf(h, r, h);
    return fmaf(fmaf(-g, g, v), h, g);
}
__device__ __forceinline__ float div_in_range(float m, float d) {
    float y = rcp(d);
    y = fmaf(fmaf(-d, y, 1.0f), y, y);
    float q = m * y;
    q = fmaf(fmaf(-d, q, m), y, q);
    return fmaf(fmaf(-d, q, m), y, q);
}
// Whether all four values are 0 or at least `least`, by their bits: 0 - 1 is the largest.
__device__ __forceinline__ bool none_below(f32x4 v, float least) {
    uint32_t low = 0xffffffffu;
#pragma unroll
    for (int c = 0; c < 4; ++c) low = min(low, bits(v[c]) - 1u);
    return low >= __float_as_uint(least) - 1u;
}

// rint(127 sqrt(r)), r in [0, 1], from an approximate root: it is within 2^-23 of the exact
// one, so u within 4e-5 of the u that the exact root gives. Only where that can reach a half
// between two integers (one wave in twenty has such a value) does the exact one decide.
__device__ __forceinline__ f32x4 m_code(f32x4 r) {
    f32x4 q;
    float far = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float u = __builtin_amdgcn_sqrtf(r[c]) * 127.0f;
        q[c] = rintf(u);
        far = fmaxf(far, fabsf(u - q[c]));
    }
    if (__any(far > 0.4999f))
#pragma unroll
        for (int c = 0; c < 4; ++c) q[c] = rintf(sqrtf(r[c]) * 127.0f);
    return q;
}
// rint(255 sqrt(sqrt(r))): the approximation is within 1e-4 (one wave in ten).
__device__ __forceinline__ f32x4 v_code(f32x4 r) {
    f32x4 q;
    float far = 0.0f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float u = __builtin_amdgcn_sqrtf(__builtin_amdgcn_sqrtf(r[c])) * 255.0f;
        q[c] = rintf(u);
        far = fmaxf(far, fabsf(u - q[c]));
    }
    if (__any(far > 0.4998f))
#pragma unroll
        for (int c = 0; c < 4; ++c) q[c] = rintf(sqrtf(sqrtf(r[c])) * 255.0f);
    return q;
}

template <bool CODES>
__global__ void __launch_bounds__(256) k_adamw(AdamwArgs a) {
    int lo = 0, hi = a.n_tensors;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if ((int)blockIdx.x >= a.t[mid].block0) lo = mid;
        else hi = mid;
    }
    const AdamwTensor t = a.t[lo];
    const bool p16 = t.io & 1, g16 = t.io & 2, vec = t.io & 4;
    const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t base = ((int64_t)((int)blockIdx.x - t.block0) * kPer + wave * kUnroll) * kBlock;

    f32x4 g[kUnroll], p[kUnroll], m[kUnroll], v[kUnroll];
    i8x4 mq[kUnroll];
    u8x4 vq[kUnroll];
    float ms[kUnroll], vs[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
        const int64_t b = base + j * kBlock, e = b + lane * 4, s = t.at + e;
        if (b >= t.n) break;
        const int n = (int)min((int64_t)4, t.n - e);  // of this lane's four; may be negative
        const bool four = vec && n == 4;
        g[j] = load4(t.g, e, g16, four, n);
        p[j] = load4(t.p, e, p16, four, n);
        if (CODES) {
            mq[j] = *(const i8x4 *)((const int8_t *)a.m + s);
            vq[j] = *(const u8x4 *)((const uint8_t *)a.v + s);
            ms[j] = a.m_scale[(t.at + b) / kBlock];
            vs[j] = a.v_scale[(t.at + b) / kBlock];
        } else {
            m[j] = load4(a.m, s, false, n == 4, n);
            v[j] = load4(a.v, s, false, n == 4, n);
        }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
        const int64_t b = base + j * kBlock, e = b + lane * 4, s = t.at + e;
        if (b >= t.n) break;
        const int n = (int)min((int64_t)4, t.n - e);
        const bool four = vec && n == 4;
        if (CODES) {
            m[j] = m_values(mq[j], ms[j]);
            v[j] = v_values(vq[j], vs[j]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float gc = g[j][c] * gs;
            m[j][c] = m[j][c] * a.beta1 + gc * a.omb1;
            v[j][c] = v[j][c] * a.beta2 + (gc * a.omb2) * gc;
        }
        if (b + kBlock > t.n)  // the tensor's last block, the same for every lane
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                m[j][c] = c < n ? m[j][c] : 0.0f;
                v[j][c] = c < n ? v[j][c] : 0.0f;
            }
        float mt = wave_max(max(max(bits(m[j][0]), bits(m[j][1])), max(bits(m[j][2]), bits(m[j][3]))));
        float vt = wave_max(max(max(bits(v[j][0]), bits(v[j][1])), max(bits(v[j][2]), bits(v[j][3]))));
        const bool in_range = a.plain && mt <= 0x1p60f && vt <= 0x1p96f;  // false for a NaN
        if (in_range && __all(none_below(m[j], 0x1p-60f) && none_below(v[j], 0x1p-96f))) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float denom = sqrt_in_range(v[j][c]) * a.rs2 + a.eps;
                p[j][c] = p[j][c] * a.keep - div_in_range(m[j][c], denom) * a.rate;
            }
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float denom = sqrtf(v[j][c]) * a.rs2 + a.eps;
                p[j][c] = p[j][c] * a.keep - (m[j][c] / denom) * a.rate;
            }
        }
        store4(t.p, e, p16, four, n, p[j]);
        if (!CODES) {
            store4(a.m, s, false, n == 4, n, m[j]);
            store4(a.v, s, false, n == 4, n, v[j]);
            continue;
        }
        mt = mt < kScaleMin ? 0.0f : mt;
        vt = vt < kScaleMin ? 0.0f : vt;
        // both reciprocals in one division, each in half of the lanes
        const float top = lane < 32 ? mt : vt, inv = top == 0.0f ? 0.0f : 1.0f / top;
        const float mi = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(inv), 0));
        const float vi = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(inv), 63));
        f32x4 mr, vr;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            mr[c] = fabsf(m[j][c]) * mi;
            vr[c] = v[j][c] * vi;
        }
        const f32x4 um = m_code(mr), uv = v_code(vr);
        // Codes are whole numbers up to 127 or 255 here: r <= 1 but for a rounding, which
        // rint takes back. A block with a NaN or an infinity gets some codes: its scale makes
        // every value of them NaN or infinite.
        uint32_t wm = 0, wv = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            wm = __builtin_amdgcn_cvt_pk_u8_f32(copysignf(um[c], m[j][c]) + 128.0f, c, wm);
            wv = __builtin_amdgcn_cvt_pk_u8_f32(vr[c] > 0.0f ? fmaxf(uv[c], 1.0f) : 0.0f, c, wv);
        }
        *(uint32_t *)((int8_t *)a.m + s) = wm ^ 0x80808080u;  // q + 128 as an unsigned byte
        *(uint32_t *)((uint8_t *)a.v + s) = wv;
        if (lane == 0) {
            a.m_scale[(t.at + b) / kBlock] = mt;
            a.v_scale[(t.at + b) / kBlock] = vt;
        }
    }
}

// Four codes of each moment a lane; bound by the bytes: 236 M parameters, 2.4 GB, take 0.39 ms.
__global__ void __launch_bounds__(256) k_adamw_values(const int8_t *m, const uint8_t *v, const float *ms,
                                                      const float *vs, float *mo, float *vo, int64_t from, int64_t n) {
    const int64_t e = from + (int64_t)blockIdx.x * 1024 + threadIdx.x * 4;
    if (e >= n) return;
    *(f32x4 *)(mo + e) = m_values(*(const i8x4 *)(m + e), ms[e / kBlock]);
    *(f32x4 *)(vo + e) = v_values(*(const u8x4 *)(v + e), vs[e / kBlock]);
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
    const int64_t most = (int64_t)1 << 33;  // a launch's work-items are fewer than 2^32
    for (int64_t from = 0; from < n; from += most) {
        const int64_t to = from + most < n ? from + most : n;
        k_adamw_values<<<dim3((unsigned)((to - from + 1023) / 1024)), 256, 0, s>>>(m, v, ms, vs, mo, vo, from, to);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace ssm
