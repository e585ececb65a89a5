// api_layers.cpp -- the C ABI of the layer operators (linear attention, RMS norm, sampling):
// argument checks and dispatch.
//
// As in api.cpp, every check runs on the host before anything is enqueued, so a rejected
// call leaves all outputs untouched.
#include <hip/hip_runtime.h>

#include <math.h>

#include <algorithm>
#include <initializer_list>

#include "ssm_layers.h"
#include "ssm_scan.h"
#include "ssm_status.h"

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
    if (!aligned(ws, ssm::kLayersWsAlign)) return fail(SSM_ERR_ALIGN, "workspace must be 256-byte aligned");
    return SSM_OK;
}

// Blocks of at most 512 threads: fewer than 2^32 work-items in a launch; a chunk's rows, 64 x heads x 128
// values, by offsets in 31 bits; and arrays whose sizes in bytes fit 64 bits.
bool linattn_shape_ok(int64_t batch, int64_t L, int64_t heads, int64_t groups, int64_t K, int64_t V) {
    return batch >= 0 && L >= 0 && heads >= 1 && groups >= 1 && heads % groups == 0 && K >= 1 && K <= 128 && V >= 1 && V <= 128 &&
           heads <= 32768 && (double)batch * heads <= 1048576.0 && L <= ((int64_t)1 << 36) &&
           (double)batch * L * heads * 128 <= 8.8e12 && (double)batch * heads * 16384 * (double)(L / 32 + 1) <= 2.2e12;
}

ssm_status check_linattn(int64_t batch, int64_t L, int64_t heads, int64_t groups, int64_t K, int64_t V, ssm_dtype io, float scale) {
    if (!valid_io(io)) return fail(SSM_ERR_DTYPE, "io dtype %d unknown", (int)io);
    if (!linattn_shape_ok(batch, L, heads, groups, K, V))
        return fail(SSM_ERR_SHAPE, "batch and L >= 0, heads at most 2^15 and a multiple of groups, batch x heads at most 2^20, d_k and d_v in 1..128");
    if (!isfinite(scale)) return fail(SSM_ERR_UNSUPPORTED, "scale must be finite");
    return SSM_OK;
}

struct LinattnBytes {
    size_t qk, v, g, state, states;
};
LinattnBytes linattn_bytes(int64_t B, int64_t L, int64_t H, int64_t Hk, int64_t K, int64_t V, bool per_token, int io) {
    const int64_t every = ssm::linattn_state_every(io);
    const size_t state = (size_t)(B * H) * K * V * 4;
    return {(size_t)(B * L * Hk * K) * io_bytes(io), (size_t)(B * L * H * V) * io_bytes(io), (size_t)(per_token ? B * L * H : H) * 4,
            state, state * (size_t)((L + every - 1) / every)};
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- linear attention
size_t ssm_linattn_states_bytes(int64_t batch, int64_t L, int32_t heads, int32_t d_k, int32_t d_v, ssm_dtype io) {
    if (!valid_io(io) || !linattn_shape_ok(batch, L, heads, 1, d_k, d_v)) return 0;
    return linattn_bytes(batch, L, heads, 1, d_k, d_v, true, io).states;
}
size_t ssm_linattn_fwd_workspace(int64_t batch, int64_t L, int32_t heads, int32_t groups, int32_t d_k, int32_t d_v, ssm_dtype io) {
    if (!valid_io(io) || !linattn_shape_ok(batch, L, heads, groups, d_k, d_v)) return 0;
    return ssm::linattn_fwd_ws(batch, L, heads, d_k, d_v, io == SSM_BF16);
}
size_t ssm_linattn_bwd_workspace(int64_t batch, int64_t L, int32_t heads, int32_t groups, int32_t d_k, int32_t d_v, int32_t per_token,
                                 ssm_dtype io) {
    if (!valid_io(io) || !linattn_shape_ok(batch, L, heads, groups, d_k, d_v)) return 0;
    return ssm::linattn_bwd_ws(batch, L, heads, groups, d_k, d_v, per_token != 0, io == SSM_BF16);
}

ssm_status ssm_linattn_fwd(const void *q, const void *k, const void *v, const float *log_decay, int32_t per_token, const float *h0,
                           float scale, void *o, float *h_final, float *states, int64_t batch, int64_t L, int32_t heads,
                           int32_t groups, int32_t d_k, int32_t d_v, ssm_dtype io, void *workspace, size_t workspace_bytes,
                           void *hip_stream) {
    ssm_status st = check_linattn(batch, L, heads, groups, d_k, d_v, io, scale);
    if (st != SSM_OK) return st;
    if (batch > 0 && L > 0 && (!q || !k || !v || !log_decay || !o))
        return fail(SSM_ERR_NULL, "q, k, v, log_decay and o are required");
    const size_t eb = io_bytes(io);
    if (!aligned(q, eb) || !aligned(k, eb) || !aligned(v, eb) || !aligned(o, eb) || !aligned(log_decay, 4) || !aligned(h0, 4) ||
        !aligned(h_final, 4) || !aligned(states, 4))
        return fail(SSM_ERR_ALIGN, "pointer alignment (float32 arrays 4 B, q, k, v, o element)");
    const LinattnBytes n = linattn_bytes(batch, L, heads, groups, d_k, d_v, per_token != 0, io);
    st = check_apart({{"q", q, n.qk}, {"k", k, n.qk}, {"v", v, n.v}, {"log_decay", log_decay, n.g}, {"h0", h0, n.state}},
                     {{"o", o, n.v}, {"h_final", h_final, n.state}, {"states", states, n.states}});
    if (st != SSM_OK) return st;
    const size_t need = ssm::linattn_fwd_ws(batch, L, heads, d_k, d_v, io == SSM_BF16);
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != SSM_OK) return st;
    if (batch == 0) return ok();
    ssm::LinattnArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = log_decay; a.h0 = h0; a.o = o; a.h_final = h_final; a.states = states;
    a.B = batch; a.L = L; a.H = heads; a.Hk = groups; a.K = d_k; a.V = d_v;
    a.per_token = per_token != 0; a.scale = scale; a.ws = workspace;
    return launch_status(ssm::launch_linattn_fwd(a, io == SSM_BF16, (hipStream_t)hip_stream), "linear attention launch");
}

ssm_status ssm_linattn_bwd(const void *q, const void *k, const void *v, const float *log_decay, int32_t per_token,
                           const float *states, const void *d_o, const float *dh_final, float scale, void *dq, void *dk, void *dv,
                           float *dlog_decay, float *dh0, int64_t batch, int64_t L, int32_t heads, int32_t groups, int32_t d_k,
                           int32_t d_v, ssm_dtype io, void *workspace, size_t workspace_bytes, void *hip_stream) {
    ssm_status st = check_linattn(batch, L, heads, groups, d_k, d_v, io, scale);
    if (st != SSM_OK) return st;
    const bool some = batch > 0 && L > 0;
    if ((some && (!q || !k || !v || !log_decay || !states || !d_o || !dq || !dk || !dv)) || ((some || !per_token) && !dlog_decay))
        return fail(SSM_ERR_NULL, "q, k, v, log_decay, states, d_o, dq, dk, dv and dlog_decay are required");
    const size_t eb = io_bytes(io);
    for (const void *p : {q, k, v, d_o, (const void *)dq, (const void *)dk, (const void *)dv})
        if (!aligned(p, eb)) return fail(SSM_ERR_ALIGN, "q, k, v, d_o, dq, dk and dv must be aligned to their elements");
    for (const float *p : {log_decay, states, dh_final, (const float *)dlog_decay, (const float *)dh0})
        if (!aligned(p, 4)) return fail(SSM_ERR_ALIGN, "float32 arrays must be 4-byte aligned");
    const LinattnBytes n = linattn_bytes(batch, L, heads, groups, d_k, d_v, per_token != 0, io);
    st = check_apart({{"q", q, n.qk}, {"k", k, n.qk}, {"v", v, n.v}, {"log_decay", log_decay, n.g}, {"states", states, n.states},
                      {"d_o", d_o, n.v}, {"dh_final", dh_final, n.state}},
                     {{"dq", dq, n.qk}, {"dk", dk, n.qk}, {"dv", dv, n.v}, {"dlog_decay", dlog_decay, n.g}, {"dh0", dh0, n.state}});
    if (st != SSM_OK) return st;
    const size_t need = ssm::linattn_bwd_ws(batch, L, heads, groups, d_k, d_v, per_token != 0, io == SSM_BF16);
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != SSM_OK) return st;
    ssm::LinattnArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = log_decay; a.states = (float *)states; a.do_ = d_o; a.dh_final = dh_final;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dlog_decay; a.dh0 = dh0;
    a.B = batch; a.L = L; a.H = heads; a.Hk = groups; a.K = d_k; a.V = d_v;
    a.per_token = per_token != 0; a.scale = scale; a.ws = workspace;
    return launch_status(ssm::launch_linattn_bwd(a, io == SSM_BF16, (hipStream_t)hip_stream), "linear attention backward launch");
}

ssm_status ssm_linattn_step(float *h, const void *q_t, const void *k_t, const void *v_t, const float *log_decay, int32_t per_token,
                            float scale, void *o_t, int64_t n_layers, int64_t n_seq, int32_t heads, int32_t groups, int32_t d_k,
                            int32_t d_v, ssm_dtype io, void *hip_stream) {
    if (n_layers < 0 || n_seq < 0 || n_layers > (1 << 20) || n_seq > (1 << 20))
        return fail(SSM_ERR_SHAPE, "n_layers and n_seq must be in 0..2^20");
    ssm_status st = check_linattn(n_layers * n_seq, 1, heads, groups, d_k, d_v, io, scale);
    if (st != SSM_OK) return st;
    const int64_t n = n_layers * n_seq;
    if (n > 0 && (!h || !q_t || !k_t || !v_t || !log_decay || !o_t))
        return fail(SSM_ERR_NULL, "h, q_t, k_t, v_t, log_decay and o_t are required");
    const size_t eb = io_bytes(io);
    if (!aligned(q_t, eb) || !aligned(k_t, eb) || !aligned(v_t, eb) || !aligned(o_t, eb) || !aligned(log_decay, 4) || !aligned(h, 4))
        return fail(SSM_ERR_ALIGN, "pointer alignment (float32 arrays 4 B, q_t, k_t, v_t, o_t element)");
    const size_t qk = (size_t)(n * groups * d_k) * eb, vb = (size_t)(n * heads * d_v) * eb,
                 gb = (size_t)((per_token ? n : n_layers) * heads) * 4, hb = (size_t)(n * heads) * d_k * d_v * 4;
    st = check_apart({{"q_t", q_t, qk}, {"k_t", k_t, qk}, {"v_t", v_t, vb}, {"log_decay", log_decay, gb}}, {{"h", h, hb}, {"o_t", o_t, vb}});
    if (st != SSM_OK) return st;
    if (n == 0) return ok();
    ssm::LinattnStepArgs a{};
    a.h = h; a.q = q_t; a.k = k_t; a.v = v_t; a.g = log_decay; a.o = o_t;
    a.layers = n_layers; a.seqs = n_seq; a.H = heads; a.Hk = groups; a.K = d_k; a.V = d_v;
    a.per_token = per_token != 0; a.scale = scale;
    return launch_status(ssm::launch_linattn_step(a, io == SSM_BF16, (hipStream_t)hip_stream), "linear attention step launch");
}

// ---------------------------------------------------------------- RMS norm
static ssm_status check_norm(int64_t rows, int32_t dim, ssm_dtype io, ssm_dtype res_io) {
    if (!valid_io(io) || !valid_io(res_io)) return fail(SSM_ERR_DTYPE, "io dtype %d or %d unknown", (int)io, (int)res_io);
    if (io == SSM_F32 && res_io != SSM_F32) return fail(SSM_ERR_DTYPE, "a float32 x takes a float32 residual");
    if (rows < 0 || rows > INT32_MAX || dim < 1 || dim > 65536)
        return fail(SSM_ERR_SHAPE, "rows must be in 0..2^31 - 1 and dim in 1..65536");
    return SSM_OK;
}
static ssm_status check_group(int32_t group) {
    if (group != 0 && group != 32 && group != 64 && group != 128) return fail(SSM_ERR_UNSUPPORTED, "group must be 0, 32, 64 or 128");
    return SSM_OK;
}

static ssm_status norm_fwd(const void *x, const void *residual, const float *weight, double eps, void *y, size_t y_bytes, int code,
                           float *scales, int32_t group, void *residual_out, float *rstd, int64_t rows, int32_t dim, ssm_dtype io,
                           ssm_dtype res_io, void *hip_stream) {
    ssm_status st = check_norm(rows, dim, io, res_io);
    if (st != SSM_OK) return st;
    if (!(eps >= 0.0) || isinf(eps)) return fail(SSM_ERR_UNSUPPORTED, "eps must be finite and not negative");
    if ((residual == nullptr) != (residual_out == nullptr) && rows > 0)
        return fail(SSM_ERR_NULL, "residual and residual_out must be given together or not at all");
    if (rows > 0 && (!x || !weight || !y || (code && !scales))) return fail(SSM_ERR_NULL, "x, weight, y (and scales) are required");
    const size_t eb = io_bytes(io), rb = io_bytes(res_io);
    if (!aligned(x, eb) || !aligned(residual, rb) || !aligned(residual_out, rb) || !aligned(weight, 4) || !aligned(rstd, 4) ||
        !aligned(scales, 4) || (!code && !aligned(y, eb)))
        return fail(SSM_ERR_ALIGN, "pointer alignment (float32 arrays 4 B, the others one element)");
    const size_t n = (size_t)rows * dim, groups = group ? (dim + group - 1) / group : 1;
    // A row is read before it is written, by the threads that write it: residual_out may be the residual.
    const bool inplace = residual_out && residual_out == residual;
    st = check_apart({{"x", x, n * eb}, {"residual", inplace ? nullptr : residual, n * rb}, {"weight", weight, (size_t)dim * 4}},
                     {{code ? "codes" : "y", y, y_bytes}, {"residual_out", residual_out, n * rb}, {"rstd", rstd, (size_t)rows * 4},
                      {"scales", scales, (size_t)rows * groups * 4}});
    if (st != SSM_OK) return st;
    if (rows == 0) return ok();
    ssm::NormArgs a{};
    a.x = x; a.residual = residual; a.weight = weight; a.y = y; a.added = residual_out; a.rstd = rstd; a.scales = scales;
    a.rows = rows; a.dim = dim; a.group = group; a.eps = eps; a.code = code;
    return launch_status(ssm::launch_rmsnorm_fwd(a, io == SSM_BF16, res_io == SSM_BF16, (hipStream_t)hip_stream), "norm launch");
}

ssm_status ssm_rmsnorm_fwd(const void *x, const void *residual, const float *weight, double eps, void *y, void *residual_out,
                           float *rstd, int64_t rows, int32_t dim, ssm_dtype io, ssm_dtype res_io, void *hip_stream) {
    return norm_fwd(x, residual, weight, eps, y, valid_io(io) && rows > 0 ? (size_t)rows * dim * io_bytes(io) : 0, 0, nullptr, 0,
                    residual_out, rstd, rows, dim, io, res_io, hip_stream);
}
ssm_status ssm_rmsnorm_fwd_q8(const void *x, const void *residual, const float *weight, double eps, void *codes, float *scales,
                              ssm_code code, int32_t group, void *residual_out, int64_t rows, int32_t dim, ssm_dtype io,
                              ssm_dtype res_io, void *hip_stream) {
    if (code != SSM_E4M3 && code != SSM_INT8) return fail(SSM_ERR_DTYPE, "code %d unknown", (int)code);
    const ssm_status st = check_group(group);
    if (st != SSM_OK) return st;
    return norm_fwd(x, residual, weight, eps, codes, rows > 0 ? (size_t)rows * dim : 0, (int)code, scales, group, residual_out, nullptr,
                    rows, dim, io, res_io, hip_stream);
}
ssm_status ssm_q8_values(const void *codes, const float *scales, ssm_code code, int32_t group, float *out, int64_t rows, int32_t dim,
                         void *hip_stream) {
    if (code != SSM_E4M3 && code != SSM_INT8) return fail(SSM_ERR_DTYPE, "code %d unknown", (int)code);
    ssm_status st = check_group(group);
    if (st != SSM_OK) return st;
    st = check_norm(rows, dim, SSM_F32, SSM_F32);
    if (st != SSM_OK) return st;
    if (rows > 0 && (!codes || !scales || !out)) return fail(SSM_ERR_NULL, "codes, scales and out are required");
    if (!aligned(scales, 4) || !aligned(out, 4)) return fail(SSM_ERR_ALIGN, "float32 arrays must be 4-byte aligned");
    const size_t n = (size_t)rows * dim, groups = group ? (dim + group - 1) / group : 1;
    st = check_apart({{"codes", codes, n}, {"scales", scales, (size_t)rows * groups * 4}}, {{"out", out, n * 4}});
    if (st != SSM_OK) return st;
    if (rows == 0) return ok();
    return launch_status(ssm::launch_q8_values(codes, scales, out, rows, dim, group, (int)code, (hipStream_t)hip_stream), "values launch");
}

size_t ssm_rmsnorm_bwd_workspace(int64_t rows, int32_t dim) {
    return check_norm(rows, dim, SSM_F32, SSM_F32) == SSM_OK ? ssm::rmsnorm_bwd_ws(rows, dim) : 0;
}
ssm_status ssm_rmsnorm_bwd(const void *dy, const void *s, const void *ds, const float *weight, const float *rstd, void *dx,
                           void *dresidual, float *dweight, int64_t rows, int32_t dim, ssm_dtype io, ssm_dtype res_io,
                           void *workspace, size_t workspace_bytes, void *hip_stream) {
    ssm_status st = check_norm(rows, dim, io, res_io);
    if (st != SSM_OK) return st;
    if (!dweight || (rows > 0 && (!dy || !s || !weight || !rstd || !dx)))
        return fail(SSM_ERR_NULL, "dy, s, weight, rstd, dx and dweight are required");
    const size_t eb = io_bytes(io), rb = io_bytes(res_io), n = (size_t)rows * dim;
    if (!aligned(dy, eb) || !aligned(dx, eb) || !aligned(s, rb) || !aligned(ds, rb) || !aligned(dresidual, rb) || !aligned(weight, 4) ||
        !aligned(rstd, 4) || !aligned(dweight, 4))
        return fail(SSM_ERR_ALIGN, "pointer alignment (float32 arrays 4 B, the others one element)");
    st = check_apart({{"dy", dy, n * eb}, {"s", s, n * rb}, {"ds", ds, n * rb}, {"weight", weight, (size_t)dim * 4}, {"rstd", rstd, (size_t)rows * 4}},
                     {{"dx", dx, n * eb}, {"dresidual", dresidual, n * rb}, {"dweight", dweight, (size_t)dim * 4}});
    if (st != SSM_OK) return st;
    st = check_workspace(workspace, workspace_bytes, ssm::rmsnorm_bwd_ws(rows, dim));
    if (st != SSM_OK) return st;
    ssm::NormBwdArgs a{};
    a.dy = dy; a.s = s; a.ds = ds; a.weight = weight; a.rstd = rstd; a.dx = dx; a.dres = dresidual; a.dweight = dweight;
    a.rows = rows; a.dim = dim; a.ws = workspace;
    return launch_status(ssm::launch_rmsnorm_bwd(a, io == SSM_BF16, res_io == SSM_BF16, (hipStream_t)hip_stream), "norm backward launch");
}

// ---------------------------------------------------------------- sampling
static bool sample_shape_ok(int64_t rows, int64_t vocab) {
    return rows >= 0 && rows <= 65535 && vocab >= 1 && vocab <= ((int64_t)1 << 24);
}
size_t ssm_sample_workspace(int64_t rows, int64_t vocab) { return sample_shape_ok(rows, vocab) ? ssm::sample_ws(rows, vocab) : 0; }
ssm_status ssm_sample(const void *logits, const float *u, const float *temperature, float temperature_all, const int32_t *top_k,
                      int32_t top_k_all, const float *top_p, float top_p_all, const float *min_p, float min_p_all, int64_t *tokens,
                      float *logprob, int64_t rows, int64_t vocab, ssm_dtype io, void *workspace, size_t workspace_bytes,
                      void *hip_stream) {
    if (!valid_io(io)) return fail(SSM_ERR_DTYPE, "io dtype %d unknown", (int)io);
    if (!sample_shape_ok(rows, vocab)) return fail(SSM_ERR_SHAPE, "rows must be in 0..65535 and vocab in 1..2^24");
    if (!temperature && !(temperature_all >= 0.0f)) return fail(SSM_ERR_UNSUPPORTED, "temperature must not be negative");
    if (rows > 0 && (!logits || !u || !tokens)) return fail(SSM_ERR_NULL, "logits, u and tokens are required");
    if (!aligned(logits, io_bytes(io)) || !aligned(tokens, 8)) return fail(SSM_ERR_ALIGN, "pointer alignment (logits element, tokens 8 B)");
    for (const void *p : {(const void *)u, (const void *)temperature, (const void *)top_k, (const void *)top_p, (const void *)min_p,
                          (const void *)logprob})
        if (!aligned(p, 4)) return fail(SSM_ERR_ALIGN, "u, the settings and logprob must be 4-byte aligned");
    const size_t rb = (size_t)rows * 4;
    ssm_status st = check_apart({{"logits", logits, (size_t)rows * vocab * io_bytes(io)}, {"u", u, rb}, {"temperature", temperature, rb},
                                 {"top_k", top_k, rb}, {"top_p", top_p, rb}, {"min_p", min_p, rb}},
                                {{"tokens", tokens, (size_t)rows * 8}, {"logprob", logprob, rb}});
    if (st != SSM_OK) return st;
    st = check_workspace(workspace, workspace_bytes, ssm::sample_ws(rows, vocab));
    if (st != SSM_OK) return st;
    if (rows == 0) return ok();
    ssm::SampleArgs a{};
    a.logits = logits; a.u = u; a.temperature = temperature; a.top_p = top_p; a.min_p = min_p; a.top_k = top_k;
    a.temperature_all = temperature_all; a.top_p_all = top_p_all; a.min_p_all = min_p_all; a.top_k_all = top_k_all;
    a.tokens = tokens; a.logprob = logprob; a.rows = rows; a.vocab = vocab; a.ws = workspace;
    return launch_status(ssm::launch_sample(a, io == SSM_BF16, (hipStream_t)hip_stream), "sampling launch");
}

}  // extern "C"
