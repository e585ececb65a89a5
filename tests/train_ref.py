"""Plain 64-bit forms of the training operators, for the tests: written from the formulas,
step by step, on the CPU, sharing nothing with the library."""
import numpy as np
import torch


def f64(t):
    return None if t is None else t.detach().double().cpu()


def gated(x, r, i, decay, h0=None, reset=None, c=8.0, dy=None, dh_final=None):
    """y, h_final, the state entering every step and, with dy, the gradients."""
    x, r, i, decay, h0, dy, dh_final = map(f64, (x, r, i, decay, h0, dy, dh_final))
    b, L, D = x.shape
    sr, si = 1 / (1 + torch.exp(-r)), 1 / (1 + torch.exp(-i))
    sp = torch.where(decay > 30, decay, torch.log1p(torch.exp(decay.clamp(max=30))))
    k = c * sp * sr
    a, beta = torch.exp(-k), torch.sqrt(-torch.expm1(-2 * k))
    live = torch.ones(b, L, 1, dtype=torch.bool) if reset is None else ~reset.bool().cpu()[:, :, None]
    h = torch.zeros(b, D, dtype=torch.float64) if h0 is None else h0
    y, before = torch.empty_like(x), torch.empty_like(x)
    for t in range(L):
        before[:, t] = h
        h = torch.where(live[:, t], a[:, t] * h, 0.0) + beta[:, t] * si[:, t] * x[:, t]
        y[:, t] = h
    out = {"y": y, "h_final": h, "before": before}
    if dy is None:
        return out
    g = torch.zeros(b, D, dtype=torch.float64) if dh_final is None else dh_final
    kd = torch.empty_like(x)
    out["dx"], out["di"], out["dr"] = (torch.empty_like(x) for _ in range(3))
    for t in range(L - 1, -1, -1):
        gt = g + dy[:, t]
        kb = torch.where(beta[:, t] > 0, k[:, t] / beta[:, t], 0.0)
        kd[:, t] = gt * (torch.exp(-2 * k[:, t]) * kb * si[:, t] * x[:, t]
                         - torch.where(live[:, t], k[:, t] * a[:, t] * before[:, t], 0.0))
        out["dx"][:, t] = gt * beta[:, t] * si[:, t]
        out["di"][:, t] = gt * beta[:, t] * x[:, t] * si[:, t] * (1 - si[:, t])
        out["dr"][:, t] = kd[:, t] * (1 - sr[:, t])
        g = torch.where(live[:, t], a[:, t] * gt, 0.0)
    ratio = torch.where(sp > 0, 1 / (1 + torch.exp(-decay)) / sp, 1.0)
    out["ddecay"], out["dh0"] = kd.sum((0, 1)) * ratio, g
    # the size of the terms that ddecay sums, for its tolerance
    out["ddecay_size"] = torch.sqrt((kd ** 2).sum((0, 1))) * ratio
    return out


def xent(hidden, weight, targets, ignore_index=-100, dloss=None, dmean=None):
    """loss, lse, mean, count, and dlogits, dhidden, dweight for the weights given."""
    hidden, weight, dloss = map(f64, (hidden, weight, dloss))
    targets = targets.cpu()
    T = hidden.shape[0]
    keep = targets != ignore_index
    logits = hidden @ weight.t()
    lse = torch.logsumexp(logits, 1)
    rows = torch.arange(T)
    at = torch.where(keep, targets, 0)
    loss = torch.where(keep, lse - logits[rows, at], 0.0)
    count = int(keep.sum())
    out = {"loss": loss, "lse": lse, "count": count, "mean": float(loss.sum() / count) if count else 0.0}
    w = torch.zeros(T, dtype=torch.float64)
    if dloss is not None:
        w += dloss
    if dmean is not None and count:
        w += float(dmean) / count
    g = torch.exp(logits - lse[:, None])
    g[rows, at] -= 1
    g = g * (w * keep)[:, None]
    out |= {"dlogits": g, "dhidden": g @ weight, "dweight": g.t() @ hidden}
    return out


BLOCK = 256


def adam_values(mq, vq, ms, vs):
    """Values of 8-bit moments (numpy), as float32 operations in the documented order."""
    u = mq.astype(np.float32) * np.float32(1 / 127)
    w = vq.astype(np.float32) * np.float32(1 / 255)
    w = w * w
    return (np.repeat(ms, BLOCK) * (u * np.abs(u))).astype(np.float32), (np.repeat(vs, BLOCK) * (w * w)).astype(np.float32)


def adam_codes(m, v):
    """8-bit codes and scales of float32 moments, as float32 operations in the documented order."""
    def scale(t):
        s = np.max(np.abs(t.reshape(-1, BLOCK)), axis=1)
        s = np.where(s < np.float32(1e-35), np.float32(0), s).astype(np.float32)
        with np.errstate(divide="ignore"):
            inv = np.where(s == 0, np.float32(0), np.float32(1) / s).astype(np.float32)
        return s, np.repeat(inv, BLOCK)
    ms, mi = scale(m)
    vs, vi = scale(v)
    qm = np.minimum(np.rint(np.sqrt(np.abs(m) * mi) * np.float32(127)), 127) * np.sign(m)
    r = v * vi
    qv = np.minimum(np.rint(np.sqrt(np.sqrt(r)) * np.float32(255)), 255)
    qv = np.where(r > 0, np.maximum(qv, 1), qv)
    return qm.astype(np.int8), qv.astype(np.uint8), ms, vs


def adam32(p, g, m, v, *, lr, beta1, beta2, eps, weight_decay, step, grad_scale=None):
    """The step on float32 numpy arrays, every operation a float32 one in the documented order."""
    f = np.float32
    g = g * f(1 if grad_scale is None else grad_scale)
    m = m * f(beta1) + g * f(1 - beta1)
    v = v * f(beta2) + (g * f(1 - beta2)) * g
    denom = np.sqrt(v) * f(1 / np.sqrt(1 - beta2 ** step)) + f(eps)
    p = p * f(1 - lr * weight_decay) - (m / denom) * f(lr / (1 - beta1 ** step))
    return p.astype(f), m.astype(f), v.astype(f)


def adam64(p, g, m, v, *, lr, beta1, beta2, eps, weight_decay, step, grad_scale=None):
    p, g, m, v = (np.asarray(t, dtype=np.float64) for t in (p, g, m, v))
    g = g * (1.0 if grad_scale is None else float(grad_scale))
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p - lr * weight_decay * p - lr * mh / (np.sqrt(vh) + eps), m, v
