// api_train.cpp -- the C ABI of the training operators: argument checks and dispatch.
//
// As in api.cpp, every check runs on the host before anything is enqueued, so a rejected
// call leaves all outputs untouched.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdio.h>

#include <algorithm>
#include <initializer_list>
#include <new>
#include <vector>

#include "ssm_scan.h"
#include "ssm_status.h"
#include "ssm_train.h"

namespace {

using ssm::aligned;
using ssm::fail;
using ssm::launch_status;
using ssm::ok;
using ssm::overlaps;

bool valid_io(int32_t io) { return io == SSM_F32 || io == SSM_BF16; }
size_t io_bytes(int32_t io) { return io == SSM_BF16 ? 2 : 4; }

struct Range {
    const char *name;
    const void *p;
    size_t bytes;
};

// No output may overlap an input or another output.
ssm_status check_apart(std::initializer_list<Range> in, std::initializer_list<Range> out) {
    for (auto o = out.begin(); o != out.end(); ++o) {
        for (const Range &r : in)
            if (overlaps(o->p, o->bytes, r.p, r.bytes))
                return fail(SSM_ERR_UNSUPPORTED, "%s must not overlap %s", o->name, r.name);
        for (auto q = out.begin(); q != o; ++q)
            if (overlaps(o->p, o->bytes, q->p, q->bytes))
                return fail(SSM_ERR_UNSUPPORTED, "%s must not overlap %s", o->name, q->name);
    }
    return SSM_OK;
}

ssm_status check_workspace(const void *ws, size_t have, size_t need) {
    if (need == 0) return SSM_OK;
    if (!ws) return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes required", need);
    if (have < need) return fail(SSM_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", have, need);
    if (!aligned(ws, ssm::kTrainWsAlign)) return fail(SSM_ERR_ALIGN, "workspace must be 256-byte aligned");
    return SSM_OK;
}

bool gated_shape_ok(int64_t batch, int64_t L, int64_t D) {
    return batch >= 0 && batch <= 65535 && L >= 0 && D >= 1 && D <= ((int64_t)1 << 28) &&
           (double)batch * (double)L * (double)D <= 4.0e17 &&
           // one thread block for at least 64 steps x 64 channels
           (double)batch * (double)(L / 64 + 1) * (double)(D / 64 + 1) <= 2147483647.0;
}

ssm_status check_gated(int64_t batch, int64_t L, int64_t D, ssm_dtype io, float c) {
    if (!valid_io(io)) return fail(SSM_ERR_DTYPE, "io dtype %d unknown", (int)io);
    if (!gated_shape_ok(batch, L, D))
        return fail(SSM_ERR_SHAPE, "batch must be in 0..65535, L >= 0, d_inner in 1..2^28, and their product within the grid");
    if (!(c > 0.0f) || isinf(c)) return fail(SSM_ERR_UNSUPPORTED, "c must be finite and positive");
    return SSM_OK;
}

bool xent_shape_ok(int64_t T, int64_t K, int64_t V, int io, bool bwd) {
    const int64_t most = (int64_t)1 << 30;
    return T >= 0 && T <= most && K >= 1 && K <= ((int64_t)1 << 22) && V >= 1 && V <= most &&
           // rows of a tile by 32-bit offsets, tiles of 128 x 128 by 32-bit numbers
           (double)(T / 128 + 1) * (double)(V / 128 + 1) <= 2147483647.0 &&
           (double)(K / 128 + 1) * (double)((T > V ? T : V) / 128 + 1) <= 2147483647.0 && (double)V * K <= 2.7e11 && ssm::xent_fits(T, K, V, io == SSM_BF16, bwd);
}

ssm_status check_xent(const void *hidden, const void *weight, const int64_t *targets, int64_t T, int64_t K,
                      int64_t V, ssm_dtype io, bool bwd) {
    if (!valid_io(io)) return fail(SSM_ERR_DTYPE, "io dtype %d unknown", (int)io);
    if (!xent_shape_ok(T, K, V, io, bwd)) return fail(SSM_ERR_SHAPE, "tokens must be in 0..2^29 - 1, dim in 1..2^22, vocab in 1..2^30, and their products within a launch");
    if (T > 0 && (!hidden || !weight || !targets)) return fail(SSM_ERR_NULL, "hidden, weight and targets are required");
    const size_t eb = io_bytes(io);
    if (!aligned(hidden, eb) || !aligned(weight, eb) || !aligned(targets, 8))
        return fail(SSM_ERR_ALIGN, "pointer alignment (targets 8 B, hidden and weight element)");
    return SSM_OK;
}

// What a step over many tensors writes, by address, to find what must not meet it.
struct Written {
    struct Piece {
        uintptr_t at, end;
        int32_t k;  // the tensor; < 0: of the state
    };
    std::vector<Piece> pieces;

    void add(const void *p, size_t bytes, int32_t k) {
        if (p && bytes) pieces.push_back({(uintptr_t)p, (uintptr_t)p + bytes, k});
    }
    // In the order of addresses, which tensors allocated one after another mostly have already. Two
    // pieces that meet, as neighbours; null: none do.
    const Piece *sort() {
        const auto before = [](const Piece &a, const Piece &b) { return a.at < b.at; };
        if (!std::is_sorted(pieces.begin(), pieces.end(), before)) std::sort(pieces.begin(), pieces.end(), before);
        for (size_t j = 1; j < pieces.size(); ++j)
            if (pieces[j].at < pieces[j - 1].end) return &pieces[j - 1];
        return nullptr;
    }
    // The piece that meets [p, p + bytes), after sort() has found none that meet each other.
    const Piece *meets(const void *p, size_t bytes) const {
        if (!p || !bytes) return nullptr;
        const auto it = std::lower_bound(pieces.begin(), pieces.end(), (uintptr_t)p,
                                         [](const Piece &a, uintptr_t at) { return a.end <= at; });
        return it != pieces.end() && it->at < (uintptr_t)p + bytes ? &*it : nullptr;
    }
};

// The step reads and writes its tensors in no order: none of what it writes may be written or read
// under another name, so a tensor given twice is refused.
ssm_status check_adamw_apart(int32_t n, void *const *params, const void *const *grads, const int64_t *sizes,
                             const int32_t *param_io, const int32_t *grad_io, const void *m, const void *v,
                             const float *ms, const float *vs, const float *grad_scale, int64_t total) {
    static const char *const state[] = {"exp_avg", "exp_avg_sq", "avg_scale", "avg_sq_scale"};
    const size_t moment = (size_t)total * (ms ? 1 : 4), scale = (size_t)(total / SSM_ADAMW_BLOCK) * 4;
    Written w;
    w.pieces.reserve((size_t)n + 4);
    for (int32_t k = 0; k < n; ++k)
        if (grads[k]) w.add(params[k], (size_t)sizes[k] * io_bytes(param_io[k]), k);
    w.add(m, moment, -1);
    w.add(v, moment, -2);
    w.add(ms, scale, -3);
    w.add(vs, scale, -4);
    const auto name = [&](const Written::Piece &p, char *to) {
        if (p.k < 0) snprintf(to, 32, "%s", state[-1 - p.k]);
        else snprintf(to, 32, "parameter %d", p.k);
        return to;
    };
    char a[32], b[32];
    if (const Written::Piece *p = w.sort())
        return fail(SSM_ERR_UNSUPPORTED, "%s must not overlap %s", name(p[0], a), name(p[1], b));
    for (int32_t k = 0; k < n; ++k)
        if (const Written::Piece *p = w.meets(grads[k], (size_t)sizes[k] * io_bytes(grad_io[k])))
            return fail(SSM_ERR_UNSUPPORTED, "gradient %d must not overlap %s", k, name(*p, a));
    if (const Written::Piece *p = w.meets(grad_scale, 4))
        return fail(SSM_ERR_UNSUPPORTED, "grad_scale must not overlap %s", name(*p, a));
    return SSM_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- gated recurrence
size_t ssm_gated_states_bytes(int64_t batch, int64_t L, int64_t d_inner) {
    if (!gated_shape_ok(batch, L, d_inner)) return 0;
    return (size_t)batch * ((L + SSM_GATED_STATE_EVERY - 1) / SSM_GATED_STATE_EVERY) * d_inner * sizeof(float);
}
size_t ssm_gated_fwd_workspace(int64_t batch, int64_t L, int64_t d_inner) {
    return gated_shape_ok(batch, L, d_inner) ? ssm::gated_fwd_ws(batch, L, d_inner) : 0;
}
size_t ssm_gated_bwd_workspace(int64_t batch, int64_t L, int64_t d_inner) {
    return gated_shape_ok(batch, L, d_inner) ? ssm::gated_bwd_ws(batch, L, d_inner) : 0;
}

ssm_status ssm_gated_fwd(const void *x, const void *r, const void *i, const float *decay, const float *h0,
                         const uint8_t *reset, float c, void *y, float *h_final, float *states, int64_t batch,
                         int64_t L, int64_t d_inner, ssm_dtype io, void *workspace, size_t workspace_bytes,
                         void *hip_stream) {
    ssm_status st = check_gated(batch, L, d_inner, io, c);
    if (st != SSM_OK) return st;
    if (batch > 0 && L > 0 && (!x || !r || !i || !decay || !y))
        return fail(SSM_ERR_NULL, "x, r, i, decay and y are required");
    const size_t eb = io_bytes(io);
    if (!aligned(x, eb) || !aligned(r, eb) || !aligned(i, eb) || !aligned(y, eb) || !aligned(decay, 4) ||
        !aligned(h0, 4) || !aligned(h_final, 4) || !aligned(states, 4))
        return fail(SSM_ERR_ALIGN, "pointer alignment (float32 arrays 4 B, x, r, i, y element)");
    const size_t nb = (size_t)(batch * L * d_inner) * eb, hb = (size_t)(batch * d_inner) * 4, db = (size_t)d_inner * 4;
    const size_t sb = ssm_gated_states_bytes(batch, L, d_inner), rb = (size_t)(batch * L);
    st = check_apart({{"x", x, nb}, {"r", r, nb}, {"i", i, nb}, {"decay", decay, db}, {"h0", h0, hb}, {"reset", reset, rb}},
                     {{"y", y, nb}, {"h_final", h_final, hb}, {"states", states, sb}});
    if (st != SSM_OK) return st;
    st = check_workspace(workspace, workspace_bytes, ssm::gated_fwd_ws(batch, L, d_inner));
    if (st != SSM_OK) return st;
    if (batch == 0) return ok();
    ssm::GatedArgs a{};
    a.x = x; a.r = r; a.i = i; a.decay = decay; a.h0 = h0; a.reset = reset; a.c = c;
    a.y = y; a.h_final = h_final; a.states = states;
    a.batch = batch; a.L = L; a.D = d_inner; a.ws = workspace;
    return launch_status(ssm::launch_gated_fwd(a, io == SSM_BF16, (hipStream_t)hip_stream), "gated recurrence launch");
}

ssm_status ssm_gated_bwd(const void *x, const void *r, const void *i, const float *decay, const float *states,
                         const uint8_t *reset, float c, const void *dy, const float *dh_final, void *dx, void *dr,
                         void *di, float *ddecay, float *dh0, int64_t batch, int64_t L, int64_t d_inner, ssm_dtype io,
                         void *workspace, size_t workspace_bytes, void *hip_stream) {
    ssm_status st = check_gated(batch, L, d_inner, io, c);
    if (st != SSM_OK) return st;
    if (!ddecay || (batch > 0 && L > 0 && (!x || !r || !i || !decay || !states || !dy || !dx || !dr || !di)))
        return fail(SSM_ERR_NULL, "x, r, i, decay, states, dy, dx, dr, di and ddecay are required");
    const size_t eb = io_bytes(io);
    if (!aligned(x, eb) || !aligned(r, eb) || !aligned(i, eb) || !aligned(dy, eb) || !aligned(dx, eb) ||
        !aligned(dr, eb) || !aligned(di, eb) || !aligned(decay, 4) || !aligned(states, 4) || !aligned(dh_final, 4) ||
        !aligned(ddecay, 4) || !aligned(dh0, 4))
        return fail(SSM_ERR_ALIGN, "pointer alignment (float32 arrays 4 B, the others element)");
    const size_t nb = (size_t)(batch * L * d_inner) * eb, hb = (size_t)(batch * d_inner) * 4, db = (size_t)d_inner * 4;
    const size_t sb = ssm_gated_states_bytes(batch, L, d_inner), rb = (size_t)(batch * L);
    st = check_apart({{"x", x, nb}, {"r", r, nb}, {"i", i, nb}, {"decay", decay, db}, {"states", states, sb},
                      {"reset", reset, rb}, {"dy", dy, nb}, {"dh_final", dh_final, hb}},
                     {{"dx", dx, nb}, {"dr", dr, nb}, {"di", di, nb}, {"ddecay", ddecay, db}, {"dh0", dh0, hb}});
    if (st != SSM_OK) return st;
    st = check_workspace(workspace, workspace_bytes, ssm::gated_bwd_ws(batch, L, d_inner));
    if (st != SSM_OK) return st;
    ssm::GatedArgs a{};
    a.x = x; a.r = r; a.i = i; a.decay = decay; a.reset = reset; a.c = c; a.dy = dy; a.dh_final = dh_final;
    a.states = (float *)states; a.dx = dx; a.dr = dr; a.di = di; a.ddecay = ddecay; a.dh0 = dh0;
    a.batch = batch; a.L = L; a.D = d_inner; a.ws = workspace;
    return launch_status(ssm::launch_gated_bwd(a, io == SSM_BF16, (hipStream_t)hip_stream),
                         "gated recurrence backward launch");
}

ssm_status ssm_gated_step(float *h, const void *x_t, const void *r_t, const void *i_t, const float *decay, float c,
                          void *y_t, int64_t n_layers, int64_t n_seq, int64_t d_inner, ssm_dtype io, void *hip_stream) {
    ssm_status st = check_gated(n_seq, 1, d_inner, io, c);
    if (st != SSM_OK) return st;
    if (n_layers < 0 || n_layers > 65535) return fail(SSM_ERR_SHAPE, "n_layers must be in 0..65535");
    if (n_layers == 0 || n_seq == 0) return ok();
    if (!h || !x_t || !r_t || !i_t || !decay || !y_t)
        return fail(SSM_ERR_NULL, "h, x_t, r_t, i_t, decay and y_t are required");
    const size_t eb = io_bytes(io);
    if (!aligned(h, 4) || !aligned(decay, 4) || !aligned(x_t, eb) || !aligned(r_t, eb) || !aligned(i_t, eb) || !aligned(y_t, eb))
        return fail(SSM_ERR_ALIGN, "pointer alignment (h, decay 4 B, x_t, r_t, i_t, y_t element)");
    const size_t n = (size_t)(n_layers * n_seq * d_inner);
    st = check_apart({{"x_t", x_t, n * eb}, {"r_t", r_t, n * eb}, {"i_t", i_t, n * eb},
                      {"decay", decay, (size_t)(n_layers * d_inner) * 4}},
                     {{"h", h, n * 4}, {"y_t", y_t, n * eb}});
    if (st != SSM_OK) return st;
    ssm::GatedStepArgs a{h, x_t, r_t, i_t, decay, c, y_t, n_layers, n_seq, d_inner};
    return launch_status(ssm::launch_gated_step(a, io == SSM_BF16, (hipStream_t)hip_stream), "gated step launch");
}

// ---------------------------------------------------------------- vocabulary cross entropy
size_t ssm_xent_fwd_workspace(int64_t tokens, int64_t dim, int64_t vocab, ssm_dtype io) {
    return valid_io(io) && xent_shape_ok(tokens, dim, vocab, io, false) ? ssm::xent_fwd_ws_any(tokens, dim, vocab, io == SSM_BF16) : 0;
}
size_t ssm_xent_fwd_workspace_for(const void *hidden, const void *weight, int64_t tokens, int64_t dim, int64_t vocab, ssm_dtype io) {
    return valid_io(io) && xent_shape_ok(tokens, dim, vocab, io, false)
               ? ssm::xent_fwd_ws(tokens, dim, vocab, io == SSM_BF16, hidden, weight) : 0;
}
size_t ssm_xent_bwd_workspace_for(const void *hidden, const void *weight, const float *dloss, int64_t tokens, int64_t dim,
                                  int64_t vocab, ssm_dtype io) {
    return valid_io(io) && xent_shape_ok(tokens, dim, vocab, io, true)
               ? ssm::xent_bwd_ws(tokens, dim, vocab, io == SSM_BF16, hidden, weight, dloss != nullptr) : 0;
}
size_t ssm_xent_bwd_workspace(int64_t tokens, int64_t dim, int64_t vocab, ssm_dtype io) {
    return valid_io(io) && xent_shape_ok(tokens, dim, vocab, io, true) ? ssm::xent_bwd_ws_any(tokens, dim, vocab, io == SSM_BF16) : 0;
}

ssm_status ssm_xent_fwd(const void *hidden, const void *weight, const int64_t *targets, int64_t ignore_index,
                        float *loss, float *lse, float *mean, int64_t tokens, int64_t dim, int64_t vocab,
                        ssm_dtype io, void *workspace, size_t workspace_bytes, void *hip_stream) {
    ssm_status st = check_xent(hidden, weight, targets, tokens, dim, vocab, io, false);
    if (st != SSM_OK) return st;
    if (!mean || (tokens > 0 && (!loss || !lse))) return fail(SSM_ERR_NULL, "loss, lse and mean are required");
    if (!aligned(loss, 4) || !aligned(lse, 4) || !aligned(mean, 4))
        return fail(SSM_ERR_ALIGN, "pointer alignment (loss, lse, mean 4 B)");
    const size_t eb = io_bytes(io), tb = (size_t)tokens * 4;
    st = check_apart({{"hidden", hidden, (size_t)(tokens * dim) * eb}, {"weight", weight, (size_t)(vocab * dim) * eb},
                      {"targets", targets, (size_t)tokens * 8}},
                     {{"loss", loss, tb}, {"lse", lse, tb}, {"mean", mean, 8}});
    if (st != SSM_OK) return st;
    st = check_workspace(workspace, workspace_bytes, ssm::xent_fwd_ws(tokens, dim, vocab, io == SSM_BF16, hidden, weight));
    if (st != SSM_OK) return st;
    ssm::XentArgs a{};
    a.hidden = hidden; a.weight = weight; a.targets = targets; a.ignore = ignore_index;
    a.loss = loss; a.lse = lse; a.mean = mean;
    a.T = tokens; a.K = dim; a.V = vocab; a.ws = workspace;
    return launch_status(ssm::launch_xent_fwd(a, io == SSM_BF16, (hipStream_t)hip_stream), "cross entropy launch");
}

ssm_status ssm_xent_bwd(const void *hidden, const void *weight, const int64_t *targets, int64_t ignore_index,
                        const float *lse, const float *mean, const float *dloss, const float *dmean, void *dhidden,
                        void *dweight, int64_t tokens, int64_t dim, int64_t vocab, ssm_dtype io, void *workspace,
                        size_t workspace_bytes, void *hip_stream) {
    ssm_status st = check_xent(hidden, weight, targets, tokens, dim, vocab, io, true);
    if (st != SSM_OK) return st;
    if (tokens > 0 && (!lse || (dmean && !mean))) return fail(SSM_ERR_NULL, "lse is required, and mean with dmean");
    const size_t eb = io_bytes(io), tb = (size_t)tokens * 4;
    if (!aligned(lse, 4) || !aligned(mean, 4) || !aligned(dloss, 4) || !aligned(dmean, 4) || !aligned(dhidden, eb) ||
        !aligned(dweight, eb))
        return fail(SSM_ERR_ALIGN, "pointer alignment (float32 arrays 4 B, dhidden and dweight element)");
    const size_t nh = (size_t)(tokens * dim) * eb, nw = (size_t)(vocab * dim) * eb;
    st = check_apart({{"hidden", hidden, nh}, {"weight", weight, nw}, {"targets", targets, (size_t)tokens * 8},
                      {"lse", lse, tb}, {"mean", mean, 8}, {"dloss", dloss, tb}, {"dmean", dmean, 4}},
                     {{"dhidden", dhidden, nh}, {"dweight", dweight, nw}});
    if (st != SSM_OK) return st;
    st = check_workspace(workspace, workspace_bytes, ssm::xent_bwd_ws(tokens, dim, vocab, io == SSM_BF16, hidden, weight, dloss != nullptr));
    if (st != SSM_OK) return st;
    if (!dhidden && !dweight) return ok();
    ssm::XentArgs a{};
    a.hidden = hidden; a.weight = weight; a.targets = targets; a.ignore = ignore_index;
    a.lse = (float *)lse; a.mean = (float *)mean; a.dloss = dloss; a.dmean = dmean;
    a.dhidden = dhidden; a.dweight = dweight;
    a.T = tokens; a.K = dim; a.V = vocab; a.ws = workspace;
    return launch_status(ssm::launch_xent_bwd(a, io == SSM_BF16, (hipStream_t)hip_stream),
                         "cross entropy backward launch");
}

// ---------------------------------------------------------------- AdamW
int64_t ssm_adamw_state_size(int32_t n_tensors, const int64_t *sizes) {
    if (n_tensors < 0 || (n_tensors > 0 && !sizes)) return 0;
    int64_t total = 0;
    for (int32_t k = 0; k < n_tensors; ++k) {
        if (sizes[k] < 0 || sizes[k] > ((int64_t)1 << 40)) return 0;
        total += (int64_t)ssm::round_up((size_t)sizes[k], SSM_ADAMW_BLOCK);
    }
    return total;
}

ssm_status ssm_adamw_step(int32_t n_tensors, void *const *params, const void *const *grads, const int64_t *sizes,
                          const int32_t *param_io, const int32_t *grad_io, void *exp_avg, void *exp_avg_sq,
                          float *avg_scale, float *avg_sq_scale, const float *grad_scale, double lr, double beta1,
                          double beta2, double eps, double weight_decay, int64_t step, void *hip_stream) {
    if (n_tensors < 0) return fail(SSM_ERR_SHAPE, "n_tensors must be >= 0");
    if (n_tensors > 0 && (!params || !grads || !sizes || !param_io || !grad_io))
        return fail(SSM_ERR_NULL, "params, grads, sizes, param_io and grad_io are required");
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !(lr >= 0.0) ||
        !(weight_decay >= 0.0) || isinf(eps) || isinf(lr) || isinf(weight_decay) || step < 1)
        return fail(SSM_ERR_UNSUPPORTED, "betas must be in [0, 1), lr, eps, weight_decay finite and >= 0, step >= 1");
    if ((avg_scale == nullptr) != (avg_sq_scale == nullptr))
        return fail(SSM_ERR_NULL, "avg_scale and avg_sq_scale are given together or not at all");
    const bool codes = avg_scale != nullptr;
    bool any = false;
    for (int32_t k = 0; k < n_tensors; ++k) {
        if (sizes[k] < 0 || sizes[k] > ((int64_t)1 << 40)) return fail(SSM_ERR_SHAPE, "tensor %d has an invalid size", k);
        if (!valid_io(param_io[k]) || !valid_io(grad_io[k])) return fail(SSM_ERR_DTYPE, "tensor %d has an unknown dtype", k);
        if (sizes[k] == 0 || !grads[k]) continue;
        any = true;
        if (!params[k]) return fail(SSM_ERR_NULL, "tensor %d has a gradient and no parameter", k);
        if (!aligned(params[k], io_bytes(param_io[k])) || !aligned(grads[k], io_bytes(grad_io[k])))
            return fail(SSM_ERR_ALIGN, "tensor %d is not aligned to its element", k);
    }
    if (!any) return ok();
    if (!exp_avg || !exp_avg_sq) return fail(SSM_ERR_NULL, "exp_avg and exp_avg_sq are required");
    if (!aligned(exp_avg, 16) || !aligned(exp_avg_sq, 16) || !aligned(avg_scale, 4) || !aligned(avg_sq_scale, 4) ||
        !aligned(grad_scale, 4))
        return fail(SSM_ERR_ALIGN, "pointer alignment (exp_avg, exp_avg_sq 16 B; scales 4 B)");
    try {
        const ssm_status st = check_adamw_apart(n_tensors, params, grads, sizes, param_io, grad_io, exp_avg, exp_avg_sq, avg_scale,
                                                avg_sq_scale, grad_scale, ssm_adamw_state_size(n_tensors, sizes));
        if (st != SSM_OK) return st;
    } catch (const std::bad_alloc &) {
        return fail(SSM_ERR_WORKSPACE, "no host memory for the table of %d tensors", n_tensors);
    }
    ssm::AdamwArgs a{};
    a.m = exp_avg; a.v = exp_avg_sq; a.m_scale = avg_scale; a.v_scale = avg_sq_scale; a.grad_scale = grad_scale;
    a.beta1 = (float)beta1; a.omb1 = (float)(1.0 - beta1);
    a.beta2 = (float)beta2; a.omb2 = (float)(1.0 - beta2);
    a.rs2 = (float)(1.0 / sqrt(1.0 - pow(beta2, (double)step)));
    a.eps = (float)eps;
    a.plain = a.eps >= 0x1p-60f && a.eps <= 1.0f && a.rs2 <= 0x1p10f;
    a.keep = (float)(1.0 - lr * weight_decay);
    a.rate = (float)(lr / (1.0 - pow(beta1, (double)step)));
    int64_t at = 0, blocks = 0;
    for (int32_t k = 0; k < n_tensors; ++k) {
        // A tensor longer than one launch's blocks may cover goes in parts.
        for (int64_t from = 0; grads[k] && from < sizes[k];) {
            const int64_t most = (int64_t)1 << 34;
            const int64_t n = sizes[k] - from < most ? sizes[k] - from : most;
            const int64_t nb = ssm::adamw_blocks(n, codes);
            if (a.n_tensors == SSM_ADAMW_TENSORS || (a.n_tensors > 0 && blocks + nb > ssm::kAdamwMostBlocks)) {
                const ssm_status st = launch_status(ssm::launch_adamw(a, (int32_t)blocks, (hipStream_t)hip_stream), "AdamW launch");
                if (st != SSM_OK) return st;
                a.n_tensors = 0;
                blocks = 0;
            }
            ssm::AdamwTensor &t = a.t[a.n_tensors++];
            t.p = (char *)params[k] + (size_t)from * io_bytes(param_io[k]);
            t.g = (const char *)grads[k] + (size_t)from * io_bytes(grad_io[k]);
            t.n = n;
            t.at = at + from;
            t.block0 = (int32_t)blocks;
            t.io = (param_io[k] == SSM_BF16 ? 1 : 0) | (grad_io[k] == SSM_BF16 ? 2 : 0) |
                   (aligned(t.p, 4 * io_bytes(param_io[k])) && aligned(t.g, 4 * io_bytes(grad_io[k])) ? 4 : 0);
            blocks += nb;
            from += n;
        }
        at += (int64_t)ssm::round_up((size_t)sizes[k], SSM_ADAMW_BLOCK);
    }
    if (a.n_tensors == 0) return ok();
    return launch_status(ssm::launch_adamw(a, (int32_t)blocks, (hipStream_t)hip_stream), "AdamW launch");
}

ssm_status ssm_adamw_values(const int8_t *exp_avg, const uint8_t *exp_avg_sq, const float *avg_scale,
                            const float *avg_sq_scale, float *avg_out, float *avg_sq_out, int64_t n, void *hip_stream) {
    if (n < 0 || n % SSM_ADAMW_BLOCK != 0 || n > ((int64_t)1 << 38))
        return fail(SSM_ERR_SHAPE, "n must be a multiple of %d in 0..2^38", SSM_ADAMW_BLOCK);
    if (n == 0) return ok();
    if (!exp_avg || !exp_avg_sq || !avg_scale || !avg_sq_scale || !avg_out || !avg_sq_out)
        return fail(SSM_ERR_NULL, "the codes, the scales and the outputs are required");
    if (!aligned(exp_avg, 16) || !aligned(exp_avg_sq, 16) || !aligned(avg_scale, 4) || !aligned(avg_sq_scale, 4) ||
        !aligned(avg_out, 16) || !aligned(avg_sq_out, 16))
        return fail(SSM_ERR_ALIGN, "pointer alignment (codes and outputs 16 B, scales 4 B)");
    const size_t sb = (size_t)(n / SSM_ADAMW_BLOCK) * 4, fb = (size_t)n * 4;
    ssm_status st = check_apart({{"exp_avg", exp_avg, (size_t)n}, {"exp_avg_sq", exp_avg_sq, (size_t)n},
                                 {"avg_scale", avg_scale, sb}, {"avg_sq_scale", avg_sq_scale, sb}},
                                {{"avg_out", avg_out, fb}, {"avg_sq_out", avg_sq_out, fb}});
    if (st != SSM_OK) return st;
    return launch_status(ssm::launch_adamw_values(exp_avg, exp_avg_sq, avg_scale, avg_sq_scale, avg_out, avg_sq_out, n,
                                                  (hipStream_t)hip_stream),
                         "AdamW values launch");
}

}  // extern "C"
