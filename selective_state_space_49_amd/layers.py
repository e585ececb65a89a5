"""Binding of the layer operators beside the scan: linear attention with a decay for each head, the
RMS norm with the residual's addition, and sampling from logits.

Like the rest of the binding, it marshals arguments only: shapes, dtypes and devices are
checked, outputs and workspaces are allocated with torch where the caller gives none, and
the C entry points of ``include/ssm_scan.h`` run on torch's current stream.
"""
from __future__ import annotations


import torch
from torch.autograd.function import once_differentiable

from . import SSM_BF16, load_library
from .training import _at, _called, _entry, _f32, _kind, _made, _need, _scratch, _stream, _table_module

# SSM_LINATTN_CHUNK_BF16 and _F32 of ssm_scan.h, by SSM_F32 and SSM_BF16.
LINATTN_CHUNK = (32, 64)
# ssm_code, and the dtype that holds it.
_CODES = {"e4m3": (1, torch.float8_e4m3fn), "int8": (2, torch.int8)}


def _int32(value, name):
    """A size that the library takes in 32 bits: ctypes would cut off what is above them."""
    if not -2 ** 31 <= value < 2 ** 31:
        raise ValueError(f"{name} must fit 32 bits, got {value}")
    return value


def _refuse_leaves_elsewhere(ctx):
    """A leaf's gradient is gathered on the stream of the oldest living graph that has it, and every other
    function of the graph works on the stream on which it was recorded. In a capture autograd makes such a
    stream wait for the captured one, and so a part of it; the default stream cannot be one, and that ends the
    process: an error instead, before the gradients leave. What is looked at are the functions that this node's
    gradients come to, directly or through others."""
    if torch.cuda.is_current_stream_capturing():
        if _table_module().leaves_elsewhere(ctx.next_functions, torch.cuda.current_stream().stream_id):
            raise RuntimeError("a backward pass cannot be captured while a graph that was built on the default "
                               "stream holds the same leaves: drop that graph's outputs first")


# ------------------------------------------------------------------ linear attention
def _sizes(*sizes):
    return [_int32(n, "heads, groups, d_k and d_v") for n in sizes]


def ssm_linattn_states_bytes(batch, L, heads, d_k, d_v, io=SSM_BF16) -> int:
    return int(load_library().ssm_linattn_states_bytes(batch, L, *_sizes(heads, d_k, d_v), io))


def ssm_linattn_fwd_workspace(batch, L, heads, groups, d_k, d_v, io=SSM_BF16) -> int:
    return int(load_library().ssm_linattn_fwd_workspace(batch, L, *_sizes(heads, groups, d_k, d_v), io))


def ssm_linattn_bwd_workspace(batch, L, heads, groups, d_k, d_v, per_token=True, io=SSM_BF16) -> int:
    return int(load_library().ssm_linattn_bwd_workspace(batch, L, *_sizes(heads, groups, d_k, d_v), int(per_token), io))


def _decay(log_decay, lead, heads, other, device):
    """The address of the decays and whether they are one for every token."""
    if log_decay.dim() == len(lead) + 1:
        return _need(log_decay, "log_decay", (*lead, heads), _f32, device), 1
    return _need(log_decay, "log_decay", other, _f32, device), 0


def _linattn_inputs(q, k, v, log_decay):
    """Sizes, io type, scale's default and the addresses of a call's inputs."""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError(f"q and v must be [batch, L, heads, dim], got {tuple(q.shape)} and {tuple(v.shape)}")
    b, L, Hk, K = q.shape
    H, V = v.shape[2:]
    _sizes(H, Hk, K, V)
    io, dev = q.dtype, q.device
    at, per_token = _decay(log_decay, (b, L), H, (H,), dev)
    return (b, L, H, Hk, K, V, _kind(q)), (_need(q, "q", q.shape, io, dev), _need(k, "k", (b, L, Hk, K), io, dev),
                                           _need(v, "v", (b, L, H, V), io, dev), at, per_token)


def ssm_linattn_fwd(q, k, v, log_decay, h0=None, *, scale=None, o=None, h_final=None, states=None, workspace=None,
                    want_h_final=True):
    """Linear attention S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale q_t^T S_t: o [b, L, H, V] and
    h_final [b, H, K, V] float32. q, k [b, L, groups, K]; v [b, L, H, V]; log_decay (g) [b, L, H] or
    [H] float32, -inf starts a document; scale defaults to K ** -0.5. states: see ssm_linattn_fwd_save."""
    return _linattn_fwd(q, k, v, log_decay, h0, scale, o, h_final, states, workspace, want_h_final, False)[:2]


def _linattn_fwd(q, k, v, log_decay, h0, scale, o, h_final, states, workspace, want_h_final, save):
    if workspace is None and q.is_cuda:
        got = _table_module().linattn_fwd(_entry("ssm_linattn_fwd"), _entry("ssm_linattn_fwd_workspace"), _stream(q), q, k, v,
                                          log_decay, h0, scale, o, h_final, states, bool(want_h_final), save)
        if got is not None:
            return _made(got)
    lib = load_library()
    (b, L, H, Hk, K, V, kind), inputs = _linattn_inputs(q, k, v, log_decay)
    dev, chunk = q.device, LINATTN_CHUNK[kind]
    scale = K ** -0.5 if scale is None else scale
    o = torch.empty_like(v) if o is None else o
    if h_final is None and want_h_final:
        h_final = torch.empty((b, H, K, V), dtype=_f32, device=dev)
    rows = (b, H, -(-L // chunk), K, V)
    if states is None and save:
        states = torch.empty(rows, dtype=_f32, device=dev)
    ws, ws_at, ws_bytes = _scratch(workspace, lib.ssm_linattn_fwd_workspace(b, L, H, Hk, K, V, kind), dev)
    _called(q, lib.ssm_linattn_fwd, *inputs, _need(h0, "h0", (b, H, K, V), _f32, dev), scale,
            _need(o, "o", (b, L, H, V), q.dtype, dev), _need(h_final, "h_final", (b, H, K, V), _f32, dev),
            _need(states, "states", rows, _f32, dev), b, L, H, Hk, K, V, kind, ws_at, ws_bytes,
            written=(o, h_final, states))
    return o, h_final, states


def ssm_linattn_fwd_save(q, k, v, log_decay, h0=None, *, scale=None, o=None, h_final=None, states=None, workspace=None):
    """The training forward: ssm_linattn_fwd, and the state that enters every chunk of 64 (float32: 32)
    steps, [b, H, ceil(L / chunk), K, V] float32, for ssm_linattn_bwd."""
    return _linattn_fwd(q, k, v, log_decay, h0, scale, o, h_final, states, workspace, True, True)


def ssm_linattn_bwd(q, k, v, log_decay, states, *, do, dh_final=None, scale=None, want_dh0=True, workspace=None):
    """Gradients of sum(do o) + sum(dh_final h_final): a dict of dq, dk, dv (the inputs' dtype), dg
    (float32, log_decay's shape) and dh0 [b, H, K, V] (float32; None unless want_dh0)."""
    if workspace is None and q.is_cuda:
        got = _table_module().linattn_bwd(_entry("ssm_linattn_bwd"), _entry("ssm_linattn_bwd_workspace"), _stream(q), q, k, v,
                                          log_decay, states, do, dh_final, scale, bool(want_dh0))
        if got is not None:
            return dict(zip(("dq", "dk", "dv", "dg", "dh0"), _made(got)))
    lib = load_library()
    (b, L, H, Hk, K, V, kind), inputs = _linattn_inputs(q, k, v, log_decay)
    dev = q.device
    scale = K ** -0.5 if scale is None else scale
    dq, dk, dv, dg = (torch.empty_like(t) for t in (q, k, v, log_decay))
    dh0 = torch.empty((b, H, K, V), dtype=_f32, device=dev) if want_dh0 else None
    ws, ws_at, ws_bytes = _scratch(workspace, lib.ssm_linattn_bwd_workspace(b, L, H, Hk, K, V, inputs[4], kind), dev)
    _called(q, lib.ssm_linattn_bwd, *inputs, _need(states, "states", (b, H, -(-L // LINATTN_CHUNK[kind]), K, V), _f32, dev),
            _need(do, "do", (b, L, H, V), q.dtype, dev), _need(dh_final, "dh_final", (b, H, K, V), _f32, dev), scale,
            _at(dq), _at(dk), _at(dv), _at(dg), _at(dh0), b, L, H, Hk, K, V, kind, ws_at, ws_bytes)
    return {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dh0": dh0}


def ssm_linattn_step(h, q_t, k_t, v_t, log_decay, *, scale=None, o_t=None):
    """One token for every (layer, sequence): h [Ln, S, H, K, V] float32 in place; q_t, k_t
    [Ln, S, groups, K]; v_t [Ln, S, H, V]; log_decay [Ln, S, H] or [Ln, H]. Returns o_t."""
    if q_t.is_cuda:
        got = _table_module().linattn_step(_entry("ssm_linattn_step"), _stream(q_t), h, q_t, k_t, v_t, log_decay, scale, o_t)
        if got is not None:
            return _made(got)
    if q_t.dim() != 4 or v_t.dim() != 4:
        raise ValueError(f"q_t and v_t must be [layers, seqs, heads, dim], got {tuple(q_t.shape)} and {tuple(v_t.shape)}")
    Ln, S, Hk, K = q_t.shape
    H, V = v_t.shape[2:]
    _sizes(H, Hk, K, V)
    io, dev = q_t.dtype, q_t.device
    kind = _kind(q_t)
    at, per_token = _decay(log_decay, (Ln, S), H, (Ln, H), dev)
    o_t = torch.empty_like(v_t) if o_t is None else o_t
    _called(q_t, load_library().ssm_linattn_step, _need(h, "h", (Ln, S, H, K, V), _f32, dev),
            _need(q_t, "q_t", q_t.shape, io, dev), _need(k_t, "k_t", (Ln, S, Hk, K), io, dev),
            _need(v_t, "v_t", (Ln, S, H, V), io, dev), at, per_token, K ** -0.5 if scale is None else scale,
            _need(o_t, "o_t", (Ln, S, H, V), io, dev), Ln, S, H, Hk, K, V, kind, written=(h, o_t))
    return o_t


class _LinearAttention(torch.autograd.Function):
    """ssm_linattn_fwd_save forwards, ssm_linattn_bwd backwards."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, h0, scale):
        if not any(ctx.needs_input_grad):
            return ssm_linattn_fwd(q, k, v, log_decay, h0, scale=scale)
        o, h_final, states = ssm_linattn_fwd_save(q, k, v, log_decay, h0, scale=scale)
        ctx.save_for_backward(q, k, v, log_decay, states)
        ctx.scale, ctx.has_h0 = scale, h0 is not None
        ctx.set_materialize_grads(False)
        return o, h_final

    @staticmethod
    @once_differentiable
    def backward(ctx, do, dh_final):
        _refuse_leaves_elsewhere(ctx)
        q, k, v, log_decay, states = ctx.saved_tensors
        do = torch.zeros_like(v) if do is None else do.to(v.dtype).contiguous()
        g = ssm_linattn_bwd(q, k, v, log_decay, states, do=do, scale=ctx.scale,
                            dh_final=None if dh_final is None else dh_final.float().contiguous(),
                            want_dh0=ctx.has_h0 and ctx.needs_input_grad[4])
        grads = (g["dq"], g["dk"], g["dv"], g["dg"], g["dh0"], None)
        return tuple(gr if need else None for gr, need in zip(grads, ctx.needs_input_grad))


def linear_attention(q, k, v, log_decay, h0=None, *, scale=None):
    """Linear attention as a differentiable function: (o, h_final), with gradients for q, k, v,
    log_decay and h0 (which have none of their own: a second derivative is refused)."""
    return _LinearAttention.apply(q, k, v, log_decay, h0, scale)


# ------------------------------------------------------------------ RMS norm
def ssm_rmsnorm_bwd_workspace(rows, dim) -> int:
    return int(load_library().ssm_rmsnorm_bwd_workspace(rows, _int32(dim, "dim")))


def _norm_inputs(x, weight, residual, residual_out):
    """Rows, dim, the types, residual_out, and the addresses of x, residual and weight."""
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    dim, dev = _int32(x.shape[-1], "dim"), x.device
    rows = x.numel() // dim if dim else 0
    kind, res_kind = _kind(x), _kind(x if residual is None else residual)
    if residual is not None and residual.dtype is not x.dtype and residual.dtype is not _f32:
        raise TypeError(f"residual: expected {x.dtype} or {_f32}, got {residual.dtype}")
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(residual)
    if residual is None and residual_out is not None:
        raise ValueError("residual_out needs a residual")
    at = (_need(x, "x", x.shape, x.dtype, dev),
          None if residual is None else _need(residual, "residual", x.shape, residual.dtype, dev),
          _need(weight, "weight", (dim,), _f32, dev))
    if residual_out is not None:
        _need(residual_out, "residual_out", x.shape, residual.dtype, dev)
    return rows, dim, kind, res_kind, residual_out, at


def ssm_rmsnorm_fwd(x, weight, residual=None, *, eps=1e-6, y=None, residual_out=None, rstd=None, want_rstd=True):
    """s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight over the last dimension. Returns y, s
    (residual_out, in the residual's dtype, which may be the residual itself; None without one) and
    rstd [...] float32, what ssm_rmsnorm_bwd needs. weight is float32, residual x's dtype or float32."""
    if x.is_cuda:
        got = _table_module().rmsnorm_fwd(_entry("ssm_rmsnorm_fwd"), _stream(x), x, weight, residual, eps, y, residual_out, rstd,
                                          bool(want_rstd))
        if got is not None:
            return _made(got)
    rows, dim, kind, res_kind, residual_out, at = _norm_inputs(x, weight, residual, residual_out)
    y = torch.empty_like(x) if y is None else y
    if rstd is None and want_rstd:
        rstd = torch.empty(x.shape[:-1], dtype=_f32, device=x.device)
    _called(x, load_library().ssm_rmsnorm_fwd, *at, eps, _need(y, "y", x.shape, x.dtype, x.device), _at(residual_out),
            _need(rstd, "rstd", x.shape[:-1], _f32, x.device), rows, dim, kind, res_kind, written=(y, residual_out, rstd))
    return y, residual_out, rstd


def _code(code):
    if code not in _CODES:
        raise ValueError(f"code must be 'e4m3' or 'int8', got {code!r}")
    return _CODES[code]


def ssm_rmsnorm_fwd_q8(x, weight, residual=None, *, eps=1e-6, code="e4m3", group=0, codes=None, scales=None,
                       residual_out=None):
    """ssm_rmsnorm_fwd with y in 8 bits: codes [..., D] (float8_e4m3fn or int8), scales [..., groups]
    float32 (one for the row with group 0, or for 32, 64 or 128 values) and s (None without a residual)."""
    number, dtype = _code(code)
    _int32(group, "group")
    if x.is_cuda:
        got = _table_module().rmsnorm_fwd_q8(_entry("ssm_rmsnorm_fwd_q8"), _stream(x), x, weight, residual, eps, number, group,
                                             codes, scales, residual_out)
        if got is not None:
            return _made(got)
    rows, dim, kind, res_kind, residual_out, at = _norm_inputs(x, weight, residual, residual_out)
    shape = (*x.shape[:-1], -(-dim // group) if group > 0 else 1)
    codes = torch.empty(x.shape, dtype=dtype, device=x.device) if codes is None else codes
    scales = torch.empty(shape, dtype=_f32, device=x.device) if scales is None else scales
    _called(x, load_library().ssm_rmsnorm_fwd_q8, *at, eps, _need(codes, "codes", x.shape, dtype, x.device),
            _need(scales, "scales", shape, _f32, x.device), number, group, _at(residual_out), rows, dim, kind, res_kind,
            written=(codes, scales, residual_out))
    return codes, scales, residual_out


def ssm_q8_values(codes, scales, *, group=None, out=None):
    """The float32 values that codes and scales of ssm_rmsnorm_fwd_q8 stand for. group: the one they
    were made with; by default it follows from the number of scales."""
    number = {dtype: n for n, dtype in _CODES.values()}.get(codes.dtype)
    if number is None:
        raise TypeError(f"codes must be float8_e4m3fn or int8, got {codes.dtype}")
    dim, dev = _int32(codes.shape[-1], "dim"), codes.device
    count = scales.shape[-1]
    if group is None:
        fits = [0] if count == 1 else [g for g in (32, 64, 128) if -(-dim // g) == count]
        if len(fits) != 1:
            raise ValueError(f"{count} scales for {dim} values: give the group")
        group = fits[0]
    _int32(group, "group")
    if codes.is_cuda:
        got = _table_module().q8_values(_entry("ssm_q8_values"), _stream(codes), codes, scales, group, out)
        if got is not None:
            return _made(got)
    shape = (*codes.shape[:-1], -(-dim // group) if group > 0 else 1)
    out = torch.empty(codes.shape, dtype=_f32, device=dev) if out is None else out
    _called(codes, load_library().ssm_q8_values, _need(codes, "codes", codes.shape, codes.dtype, dev),
            _need(scales, "scales", shape, _f32, dev), number, group, _need(out, "out", codes.shape, _f32, dev),
            codes.numel() // dim if dim else 0, dim, written=(out,))
    return out


def ssm_rmsnorm_bwd(dy, s, weight, rstd, *, ds=None, workspace=None):
    """Gradients of sum(dy y) + sum(ds s), with s and rstd as ssm_rmsnorm_fwd gave them (s is x where it
    had no residual): dx (dy's dtype), dresidual (s's dtype; dx itself where they are the same) and
    dweight [D] float32."""
    if workspace is None and dy.is_cuda:
        got = _table_module().rmsnorm_bwd(_entry("ssm_rmsnorm_bwd"), _entry("ssm_rmsnorm_bwd_workspace"), _stream(dy), dy, s, weight,
                                          rstd, ds)
        if got is not None:
            dx, dres, dweight = _made(got)
            return dx, dx if dres is None else dres, dweight
    lib = load_library()
    dim, dev = _int32(dy.shape[-1], "dim"), dy.device
    rows = dy.numel() // dim if dim else 0
    kind, res_kind = _kind(dy), _kind(s)
    at = (_need(dy, "dy", dy.shape, dy.dtype, dev), _need(s, "s", dy.shape, s.dtype, dev), _need(ds, "ds", dy.shape, s.dtype, dev),
          _need(weight, "weight", (dim,), _f32, dev), _need(rstd, "rstd", dy.shape[:-1], _f32, dev))
    dx, dweight = torch.empty_like(dy), torch.empty_like(weight)
    dres = dx if s.dtype is dy.dtype else torch.empty_like(s)
    ws, ws_at, ws_bytes = _scratch(workspace, lib.ssm_rmsnorm_bwd_workspace(rows, dim), dev)
    _called(dy, lib.ssm_rmsnorm_bwd, *at, _at(dx), None if dres is dx else _at(dres), _at(dweight), rows, dim, kind, res_kind,
            ws_at, ws_bytes)
    return dx, dres, dweight


class _RmsNorm(torch.autograd.Function):
    """ssm_rmsnorm_fwd forwards, ssm_rmsnorm_bwd backwards."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, added, rstd = ssm_rmsnorm_fwd(x, weight, residual, eps=eps)
        ctx.save_for_backward(x if added is None else added, weight, rstd)
        ctx.io = x.dtype
        ctx.set_materialize_grads(False)
        return (y, added) if added is not None else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, ds=None):
        _refuse_leaves_elsewhere(ctx)
        s, weight, rstd = ctx.saved_tensors
        dy = torch.zeros(s.shape, dtype=ctx.io, device=s.device) if dy is None else dy.to(ctx.io).contiguous()
        dx, dres, dweight = ssm_rmsnorm_bwd(dy, s, weight, rstd, ds=None if ds is None else ds.to(s.dtype).contiguous())
        grads = (dx, dweight, dres, None)
        return tuple(g if need else None for g, need in zip(grads, ctx.needs_input_grad))


def rms_norm(x, weight, residual=None, *, eps=1e-6):
    """The norm as a differentiable function: y, or (y, x + residual) with a residual, with gradients
    for x, weight and residual (which have none of their own: a second derivative is refused)."""
    return _RmsNorm.apply(x, weight, residual, eps)


# ------------------------------------------------------------------ sampling
def ssm_sample_workspace(rows, vocab) -> int:
    return int(load_library().ssm_sample_workspace(rows, vocab))


def _setting(value, name, rows, dtype, device):
    """A setting's address and its value: a tensor with one for every row, or a number for all."""
    if torch.is_tensor(value):
        return _need(value, name, (rows,), dtype, device), 0
    return None, value


def _top_k(value):
    """A top_k for all rows, in 32 bits: a whole number, of which 0 and less keep all."""
    if not float(value).is_integer():
        raise ValueError(f"top_k must be a whole number, got {value}")
    return max(0, min(int(value), 2 ** 31 - 1))


def ssm_sample(logits, u, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, tokens=None, logprob=None,
               want_logprob=False, workspace=None):
    """The next token [S] int64 of every row of logits [S, V], from one uniform number of [0, 1) a row
    (u [S] float32): temperature, then the top_k largest, then the fewest most likely that hold top_p,
    then those at least min_p times as likely as the first. A setting is a number, or a tensor [S]
    (float32; top_k int32). A temperature of 0 takes the largest logit. With want_logprob (or logprob)
    returns (tokens, logprob), the logarithm of the token's share of what was kept."""
    if workspace is None and logits.is_cuda:
        got = _table_module().sample(_entry("ssm_sample"), _entry("ssm_sample_workspace"), _stream(logits), logits, u, temperature,
                                     top_k, top_p, min_p, tokens, logprob, bool(want_logprob))
        if got is not None:
            tokens, logprob = _made(got)
            return tokens if logprob is None else (tokens, logprob)
    k_all = 0 if torch.is_tensor(top_k) else _top_k(top_k)
    lib = load_library()
    rows, vocab = logits.shape
    dev = logits.device
    kind = _kind(logits)
    t, t_all = _setting(temperature, "temperature", rows, _f32, dev)
    k = _setting(top_k, "top_k", rows, torch.int32, dev)[0]
    p, p_all = _setting(top_p, "top_p", rows, _f32, dev)
    m, m_all = _setting(min_p, "min_p", rows, _f32, dev)
    tokens = torch.empty(rows, dtype=torch.int64, device=dev) if tokens is None else tokens
    if logprob is None and want_logprob:
        logprob = torch.empty(rows, dtype=_f32, device=dev)
    ws, ws_at, ws_bytes = _scratch(workspace, lib.ssm_sample_workspace(rows, vocab), dev)
    _called(logits, lib.ssm_sample, _need(logits, "logits", logits.shape, logits.dtype, dev), _need(u, "u", (rows,), _f32, dev),
            t, t_all, k, k_all, p, p_all, m, m_all, _need(tokens, "tokens", (rows,), torch.int64, dev),
            _need(logprob, "logprob", (rows,), _f32, dev), rows, vocab, kind, ws_at, ws_bytes, written=(tokens, logprob))
    return tokens if logprob is None else (tokens, logprob)
