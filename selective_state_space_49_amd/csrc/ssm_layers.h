// ssm_layers.h -- host-side launch interface of the layer operators beside the scan: linear
// attention with a decay for each head, the RMS norm with the residual's addition, sampling.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ssm_scan.h"

namespace ssm {

constexpr size_t kLayersWsAlign = 256;

// One call of the linear attention, already validated; device pointers, layouts as in ssm_scan.h.
struct LinattnArgs {
    const void *q, *k, *v;
    const float *g, *h0;
    void *o;
    float *h_final, *states;
    // the backward: states, do_, dh_final in, the gradients out
    const void *do_;
    const float *dh_final;
    void *dq, *dk, *dv;
    float *dg, *dh0;
    int64_t B, L;
    int32_t H, Hk, K, V;
    bool per_token;  // g is [B, L, H], not [H]
    float scale;
    void *ws;
};
int32_t linattn_state_every(int io);
size_t linattn_fwd_ws(int64_t B, int64_t L, int32_t H, int32_t K, int32_t V, int io);
size_t linattn_bwd_ws(int64_t B, int64_t L, int32_t H, int32_t Hk, int32_t K, int32_t V, bool per_token, int io);
hipError_t launch_linattn_fwd(const LinattnArgs &a, int io, hipStream_t s);
hipError_t launch_linattn_bwd(const LinattnArgs &a, int io, hipStream_t s);

struct LinattnStepArgs {
    float *h;
    const void *q, *k, *v;
    const float *g;
    void *o;
    int64_t layers, seqs;
    int32_t H, Hk, K, V;
    bool per_token;  // g is [layers, seqs, H], not [layers, H]
    float scale;
};
hipError_t launch_linattn_step(const LinattnStepArgs &a, int io, hipStream_t s);

// The norm's forward: y (io), or codes and scales where code is not 0.
struct NormArgs {
    const void *x, *residual;
    const float *weight;
    void *y, *added;
    float *rstd, *scales;
    int64_t rows;
    int32_t dim, group;
    double eps;
    int code;  // 0: y of io, 1: e4m3, 2: int8
};
hipError_t launch_rmsnorm_fwd(const NormArgs &a, int io, int res_io, hipStream_t s);

struct NormBwdArgs {
    const void *dy, *s, *ds;
    const float *weight, *rstd;
    void *dx, *dres;
    float *dweight;
    int64_t rows;
    int32_t dim;
    void *ws;
};
size_t rmsnorm_bwd_ws(int64_t rows, int32_t dim);
hipError_t launch_rmsnorm_bwd(const NormBwdArgs &a, int io, int res_io, hipStream_t s);
hipError_t launch_q8_values(const void *codes, const float *scales, float *out, int64_t rows, int32_t dim, int32_t group,
                            int code, hipStream_t s);

struct SampleArgs {
    const void *logits;
    const float *u;
    const float *temperature, *top_p, *min_p;  // null: the values below for every row
    const int32_t *top_k;
    float temperature_all, top_p_all, min_p_all;
    int32_t top_k_all;
    int64_t *tokens;
    float *logprob;
    int64_t rows, vocab;
    void *ws;
};
size_t sample_ws(int64_t rows, int64_t vocab);
hipError_t launch_sample(const SampleArgs &a, int io, hipStream_t s);

}  // namespace ssm
