"""Plain 64-bit forms of the layer operators, for the tests: written from the formulas, step by
step, on the CPU, sharing nothing with the library."""
import math
from fractions import Fraction

import numpy as np
import torch


def f64(t):
    return None if t is None else t.detach().double().cpu()


def linattn(q, k, v, g, h0=None, scale=None, do=None, dh_final=None):
    """o, h_final, the state before every step and, with do, the gradients. g [b, L, H] or [H]."""
    shared = g.dim() == 1
    q, k, v, g, h0, do, dh_final = map(f64, (q, k, v, g, h0, do, dh_final))
    b, L, Hk, K = q.shape
    H, V = v.shape[2:]
    share = H // Hk
    scale = K ** -0.5 if scale is None else scale
    q, k = (t.repeat_interleave(share, 2) for t in (q, k))
    g = g.expand(b, L, H)
    a = torch.where(g < -104, 0.0, torch.exp(g))
    S = torch.zeros(b, H, K, V, dtype=torch.float64) if h0 is None else h0.clone()
    o, states = torch.zeros(b, L, H, V, dtype=torch.float64), []
    for t in range(L):
        states.append(S)
        S = a[:, t, :, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = scale * (q[:, t, :, :, None] * S).sum(2)
    out = {"o": o, "h_final": S, "states": states}
    if do is None:
        return out
    dS = torch.zeros_like(S) if dh_final is None else dh_final.clone()
    dq, dk, dv, dg = (torch.zeros_like(t) for t in (q, k, v, g.contiguous()))
    for t in range(L - 1, -1, -1):
        St = states[t + 1] if t + 1 < L else S
        d = scale * do[:, t]
        dS = dS + q[:, t, :, :, None] * d[:, :, None, :]
        dq[:, t] = (St * d[:, :, None, :]).sum(3)
        dk[:, t] = (dS * v[:, t, :, None, :]).sum(3)
        dv[:, t] = (dS * k[:, t, :, :, None]).sum(2)
        dg[:, t] = a[:, t] * (states[t] * dS).sum((2, 3))
        dS = a[:, t, :, None, None] * dS
    group = lambda t: t.view(b, L, Hk, share, K).sum(3)  # noqa: E731
    return out | {"dq": group(dq), "dk": group(dk), "dv": dv, "dg": dg.sum((0, 1)) if shared else dg, "dh0": dS}


def norm(x, weight, residual=None, eps=1e-6, dy=None, ds=None):
    """y, s (as stored), rstd and, with dy, dx and dweight."""
    s = x.float().cpu() if residual is None else (x.float().cpu() + residual.float().cpu()).to(residual.dtype)
    n, w = s.double(), f64(weight)
    r = 1 / torch.sqrt((n * n).mean(-1) + eps)
    n = n * r[..., None]
    out = {"y": n * w, "s": s, "rstd": r}
    if dy is not None:
        dy = f64(dy)
        out["dx"] = r[..., None] * (w * dy - n * (w * dy * n).mean(-1, keepdim=True))
        if ds is not None:
            out["dx"] = out["dx"] + f64(ds)
        out["dweight"] = (dy * n).reshape(-1, n.shape[-1]).sum(0)
    return out


def e4m3_values():
    """What the codes 0 to 126 stand for: steps of 2^-9 up to 2^-6, then eight to a power of two, up to 448."""
    return np.array([m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:119])


def coded(y, code, group):
    """The nearest codes' values and the scales of rows of y (float64), ties to even, one by one."""
    y = np.asarray(y, dtype=np.float64)
    table = e4m3_values() if code == "e4m3" else np.arange(128.0)
    rows, D = y.shape
    size = group or D
    scales = np.zeros((rows, -(-D // size)), dtype=np.float32)
    values, codes = np.zeros_like(y), np.zeros((rows, D), dtype=np.int64)
    for r in range(rows):
        for n, at in enumerate(range(0, D, size)):
            part = y[r, at:at + size]
            scale = np.float32(np.abs(part).max() / table[-1])
            scales[r, n] = scale
            if scale == 0:
                continue
            for j, x in enumerate(part):
                u = abs(x) / float(scale)
                i = min(int(np.searchsorted(table, u)), len(table) - 1)  # table[i] >= u
                if i > 0:
                    below, above = u - table[i - 1], table[i] - u
                    if below < above or (below == above and (i - 1) % 2 == 0):
                        i -= 1
                codes[r, at + j] = int(math.copysign(1, x)) * i
                values[r, at + j] = math.copysign(table[i], x) * float(scale)
    return values, scales, codes


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Token, log of its share, and the kept indices, of one row: by a sorted list."""
    x = [float(t) for t in logits.double().tolist()]
    V = len(x)
    f32 = lambda t: float(np.float32(t))  # noqa: E731
    temperature, top_p, min_p, u = f32(temperature), f32(top_p), f32(min_p), f32(u)
    if any(math.isnan(t) for t in x) or max(x) == -math.inf or not temperature >= 0 or math.isnan(u):
        return -1, math.nan, []
    order = sorted((i for i in range(V) if x[i] > -math.inf), key=lambda i: (-x[i], i))
    if temperature == 0:
        return order[0], 0.0, order[:1]
    top = x[order[0]]
    if top == math.inf:
        order = [i for i in order if x[i] == math.inf]
    w = {i: 1.0 if x[i] == top else math.exp((x[i] - top) / temperature) for i in order}
    w = {i: int(Fraction(t) * 2 ** 1100) for i, t in w.items()}  # whole numbers: sums without rounding
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        part, held, kept = Fraction(top_p) * sum(w[i] for i in order), 0, []
        for i in order:
            if kept and not held < part:
                break
            kept.append(i)
            held += w[i]
        order = kept
    order = sorted(i for i in order if w[i] >= Fraction(min(min_p, 1.0)) * 2 ** 1100)
    whole, held = sum(w[i] for i in order), 0
    aim = Fraction(min(max(u, -1.0), 2.0)) * whole
    token = order[-1]
    for i in order:
        held += w[i]
        if held > aim:
            token = i
            break
    return token, math.log(w[token] / whole), order
