// ssm_train.h -- host-side launch interface of the training operators beside the scan: the
// gated linear recurrence, the vocabulary cross entropy, the AdamW step.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ssm_scan.h"

namespace ssm {

inline size_t round_up(size_t v, size_t m) { return (v + m - 1) / m * m; }
constexpr size_t kTrainWsAlign = 256;

// One call of the gated recurrence, already validated; device pointers, layouts as in
// ssm_scan.h. bwd: dy is given, and the outputs of the backward.
struct GatedArgs {
    const void *x, *r, *i, *dy;
    const float *decay, *h0, *dh_final;
    const uint8_t *reset;
    float c;
    void *y, *dx, *dr, *di;
    float *h_final, *states, *ddecay, *dh0;
    int64_t batch, L, D;
    void *ws;
};
size_t gated_fwd_ws(int64_t batch, int64_t L, int64_t D);
size_t gated_bwd_ws(int64_t batch, int64_t L, int64_t D);
hipError_t launch_gated_fwd(const GatedArgs &a, int io, hipStream_t s);
hipError_t launch_gated_bwd(const GatedArgs &a, int io, hipStream_t s);

struct GatedStepArgs {
    float *h;
    const void *x, *r, *i;
    const float *decay;
    float c;
    void *y;
    int64_t n_layers, n_seq, D;
};
hipError_t launch_gated_step(const GatedStepArgs &a, int io, hipStream_t s);

// The cross entropy of a linear head.
struct XentArgs {
    const void *hidden, *weight;
    const int64_t *targets;
    int64_t ignore;
    float *loss, *lse, *mean;  // forward outputs; the backward reads lse and mean
    const float *dloss, *dmean;
    void *dhidden, *dweight;
    int64_t T, K, V;
    void *ws;
};
size_t xent_fwd_ws(int64_t T, int64_t K, int64_t V, int io, const void *hidden, const void *weight);
size_t xent_bwd_ws(int64_t T, int64_t K, int64_t V, int io, const void *hidden, const void *weight, bool weighed);
size_t xent_fwd_ws_any(int64_t T, int64_t K, int64_t V, int io);  // enough for any pointers
size_t xent_bwd_ws_any(int64_t T, int64_t K, int64_t V, int io);
// Whether every launch of a call stays below 2^32 work-items.
bool xent_fits(int64_t T, int64_t K, int64_t V, int io, bool bwd);
hipError_t launch_xent_fwd(const XentArgs &a, int io, hipStream_t s);
hipError_t launch_xent_bwd(const XentArgs &a, int io, hipStream_t s);

// One launch of the AdamW step: up to SSM_ADAMW_TENSORS tensors, passed by value.
struct AdamwTensor {
    void *p;
    const void *g;
    int64_t n;       // elements
    int64_t at;      // first element of its moments
    int32_t block0;  // first thread block that works on it
    int32_t io;      // bit 0: the parameter is bfloat16, bit 1: the gradient, bit 2: four
                     // values of each can be read at once
};
struct AdamwArgs {
    AdamwTensor t[SSM_ADAMW_TENSORS];
    int32_t n_tensors;
    void *m, *v;
    float *m_scale, *v_scale;  // null: moments in float32
    const float *grad_scale;
    float beta1, omb1, beta2, omb2, rs2, eps, keep, rate;  // in the order of the formula
    bool plain;                // eps >= 2^-60, rs2 <= 2^10: no extreme denominators
};
constexpr int64_t kAdamwMostBlocks = 0xffffff;  // of a launch: 256 threads each, fewer than 2^32 in all
int32_t adamw_blocks(int64_t n, bool codes);  // thread blocks of a tensor of n elements
hipError_t launch_adamw(const AdamwArgs &a, int32_t blocks, hipStream_t s);
hipError_t launch_adamw_values(const int8_t *m, const uint8_t *v, const float *ms, const float *vs,
                               float *mo, float *vo, int64_t n, hipStream_t s);

}  // namespace ssm
