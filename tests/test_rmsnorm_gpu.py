"""The RMS norm on the GPU against 64 bits.

Tolerances: s is one addition, rounded: equal bits. y in float32 is two multiplications with a root
rounded to 32 bits, 3 x 2^-24 relative; in bfloat16 rounded once more, 2^-9 and a little (a half step,
of values up to 1/2^8 above a power of two: 2^-8 of the value). rstd: 2^-24, and as much for a root in
64 bits, nothing. dx: the root, a mean and four operations on terms of both signs, 8 x 2^-24 of the
row's largest term. dweight: a row's product n dy, 3 x 2^-24, and sums in 32 bits of at most 64 rows
before 64 bits: 64 x 2^-24 of the sum of magnitudes. Codes and scales: equal."""
import math

import pytest
import torch

import selective_state_space_49_amd as ssm
from tests import layers_ref as ref
from tests.gpu_util import bitwise_equal, say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(F32, None), (F32, F32), (BF16, None), (BF16, BF16), (BF16, F32)]
SIZES = [(1, 1), (1, 4096), (3, 7), (5, 16), (65, 100), (33, 512), (7, 1000), (4, 1024), (9, 2047), (3, 2048), (2, 5001), (2, 8192),
         (2, 10000), (1, 16384), (1, 30001), (2, 65536), (700, 24), (129, 128), (70, 129), (37, 256), (8501, 40), (4200, 200)]
EPS = 1e-5


def make(rows, dim, io, res, seed=0):
    g = torch.Generator().manual_seed(seed + dim)
    rn = lambda dt, scale=1.0: (torch.randn(rows, dim, generator=g) * scale).to(dt)  # noqa: E731
    return {"x": rn(io), "residual": None if res is None else rn(res, 3.0), "weight": 1 + 0.2 * torch.randn(dim, generator=g),
            "dy": rn(io), "ds": None if res is None else rn(res)}


def dev(d):
    return {k: None if t is None else t.cuda() for k, t in d.items()}


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward_and_gradients(size, types):
    say("norm", size, types)
    d = make(*size, *types)
    c = dev(d)
    y, s, rstd = ssm.ssm_rmsnorm_fwd(c["x"], c["weight"], c["residual"], eps=EPS)
    dx, dres, dw = ssm.ssm_rmsnorm_bwd(c["dy"], c["x"] if s is None else s, c["weight"], rstd, ds=c["ds"])
    want = ref.norm(d["x"], d["weight"], d["residual"], EPS, d["dy"], d["ds"])
    if s is not None:
        assert bitwise_equal(s.cpu(), want["s"])
    assert float((rstd.double().cpu() / want["rstd"] - 1).abs().max()) <= 2.0 ** -24
    rel = {F32: 3 * 2.0 ** -24, BF16: 2.0 ** -8}
    off = (y.double().cpu() - want["y"]).abs()
    assert bool((off <= rel[types[0]] * want["y"].abs()).all())
    # the largest of the terms that a row's gradient adds
    w, dy, n = d["weight"].double(), d["dy"].double(), want["s"].double() * want["rstd"][:, None]
    terms = want["rstd"][:, None] * ((w * dy).abs() + n.abs() * (w * dy * n).abs().mean(1, keepdim=True))
    if d["ds"] is not None:
        terms = terms + d["ds"].double().abs()
    for got in (dx, dres):
        off = (got.double().cpu() - want["dx"]).abs()
        bound = 8 * 2.0 ** -24 * terms.amax(1, keepdim=True)
        if got.dtype is BF16:
            bound = bound + 2.0 ** -8 * want["dx"].abs()
        assert got.shape == dx.shape and bool((off <= bound).all())
    assert dres.dtype is (types[1] or types[0])
    off = (dw.double().cpu() - want["dweight"]).abs()
    assert bool((off <= 64 * 2.0 ** -24 * (dy * n).abs().sum(0)).all())


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("types", TYPES, ids=str)
def test_codes(code, group, types):
    for size in ((1, 1), (3, 130), (2, 1024), (5, 333), (2, 4104), (1, 9000)):
        say("norm q8", code, group, types, size)
        d = make(*size, *types)
        d["x"][0, 0] = 0.0
        c = dev(d)
        codes, scales, s = ssm.ssm_rmsnorm_fwd_q8(c["x"], c["weight"], c["residual"], eps=EPS, code=code, group=group)
        want = ref.norm(d["x"], d["weight"], d["residual"], EPS)
        values, want_scales, _ = ref.coded(want["y"].numpy(), code, group)
        assert scales.shape == want_scales.shape and bitwise_equal(scales.cpu(), torch.from_numpy(want_scales))
        got = ssm.ssm_q8_values(codes, scales, group=group)
        exact = codes.float() * scales.repeat_interleave(group or size[1], 1)[:, :size[1]]
        assert bitwise_equal(got, exact)
        assert torch.equal(got.cpu(), torch.from_numpy(values).float())
        if s is not None:
            assert bitwise_equal(s.cpu(), want["s"])


def test_code_borders():
    """Values next to and on the borders of two codes: a row whose norm is 1 by construction."""
    table = torch.from_numpy(ref.e4m3_values())
    mid = (table[1:] + table[:-1]) / 2
    row = torch.cat([table, mid, -mid, mid * (1 + 2.0 ** -22), mid * (1 - 2.0 ** -22)]).float()
    row[0] = 448.0
    scale = 2.0 ** -7
    w = row * scale  # y = n w, and n = 1 where x is constant
    x = torch.ones(1, len(row))
    codes, scales, _ = ssm.ssm_rmsnorm_fwd_q8(x.cuda(), w.cuda(), eps=0.0, code="e4m3")
    values, want, _ = ref.coded(w.double()[None].numpy(), "e4m3", 0)
    assert float(scales) == float(want[0, 0])
    assert torch.equal(ssm.ssm_q8_values(codes, scales).cpu(), torch.from_numpy(values).float())


def test_extremes():
    x = torch.tensor([[0.0] * 16, [1e30] * 16, [1e-30] * 16, [3e38] * 8 + [0.0] * 8]).cuda()
    w = torch.ones(16).cuda()
    y, _, rstd = ssm.ssm_rmsnorm_fwd(x, w, eps=1e-6)
    want = ref.norm(x, w, None, 1e-6)
    assert float((y.double().cpu() - want["y"]).abs().max()) <= 4 * 2.0 ** -24 * math.sqrt(2)
    codes, scales, _ = ssm.ssm_rmsnorm_fwd_q8(x, w, code="int8")
    assert float(scales[0]) == 0 and bool((codes[0] == 0).all()) and bool((codes[1] == 127).all())
    for bad in (math.nan, math.inf):
        for code in ("e4m3", "int8"):
            z = torch.ones(2, 256).cuda()
            z[0, 3] = bad
            codes, scales, _ = ssm.ssm_rmsnorm_fwd_q8(z, torch.ones(256).cuda(), code=code)
            v = ssm.ssm_q8_values(codes, scales)
            assert not bool(torch.isfinite(v[0, 3])) and bool((v[1] - 1).abs().max() < 1e-5)


def test_residual_in_place_and_shapes():
    d = dev(make(6, 200, BF16, F32))
    y, s, _ = ssm.ssm_rmsnorm_fwd(d["x"], d["weight"], d["residual"])
    r = d["residual"].clone()
    y2, s2, _ = ssm.ssm_rmsnorm_fwd(d["x"].view(2, 3, 200), d["weight"], r.view(2, 3, 200), residual_out=r.view(2, 3, 200))
    assert bitwise_equal(s, r) and bitwise_equal(y, y2.view(6, 200)) and y2.shape == (2, 3, 200)
    e = torch.empty(0, 5, device="cuda")
    y, s, rstd = ssm.ssm_rmsnorm_fwd(e, torch.ones(5, device="cuda"))
    dx, dres, dw = ssm.ssm_rmsnorm_bwd(e, e, torch.ones(5, device="cuda"), rstd)
    assert y.shape == (0, 5) and dx.shape == (0, 5) and bool((dw == 0).all())


@pytest.mark.parametrize("types", TYPES, ids=str)
def test_unaligned(types):
    d = dev(make(5, 256, *types))

    def moved(t):
        if t is None:
            return None
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:].copy_(t.reshape(-1))
        return flat[1:].view(t.shape)
    m = {k: moved(t) for k, t in d.items()}
    a = ssm.ssm_rmsnorm_fwd(d["x"], d["weight"], d["residual"])
    b = ssm.ssm_rmsnorm_fwd(m["x"], m["weight"], m["residual"])
    for p, q in zip(a, b):
        assert (p is None) == (q is None) and (p is None or bitwise_equal(p, q))
    # a row's sums in 32 bits run in another order where its elements are read one by one, so gradients are
    # equal up to the two sides' own bound, 8 x 2^-24 of the terms (here at most about 10) each
    s = d["x"] if a[1] is None else a[1]
    for p, q in zip(ssm.ssm_rmsnorm_bwd(d["dy"], s, d["weight"], a[2], ds=d["ds"]),
                    ssm.ssm_rmsnorm_bwd(m["dy"], moved(s), m["weight"], moved(a[2]), ds=m["ds"])):
        off = (p.double() - q.double()).abs()
        assert bool((off <= 2 * 8 * 2.0 ** -24 * 10 + (2 * 2.0 ** -8 * p.double().abs() if p.dtype is BF16 else 0)).all())
    for p, q in zip(ssm.ssm_rmsnorm_fwd_q8(d["x"], d["weight"], d["residual"], group=64),
                    ssm.ssm_rmsnorm_fwd_q8(m["x"], m["weight"], m["residual"], group=64)):
        assert (p is None) == (q is None) and (p is None or torch.equal(p.float(), q.float()))


def test_autograd_and_differences():
    d = make(7, 60, F32, F32)
    c = {k: t.cuda().requires_grad_(k in ("x", "residual", "weight")) for k, t in d.items()}
    y, s = ssm.rms_norm(c["x"], c["weight"], c["residual"], eps=EPS)
    ((y * c["dy"]).sum() + (s * c["ds"]).sum()).backward()
    want = ref.norm(d["x"], d["weight"], d["residual"], EPS, d["dy"], d["ds"])
    for t in (c["x"].grad, c["residual"].grad):
        assert float((t.double().cpu() - want["dx"]).abs().max()) <= 8 * 2.0 ** -24 * 10
    assert c["x"].grad.data_ptr() != c["residual"].grad.data_ptr()
    # the 64-bit form's gradients against its own differences
    step = torch.randn(7, 60, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    base = d["x"].double() + d["residual"].double()

    def loss(s64):
        r = 1 / torch.sqrt((s64 * s64).mean(-1, keepdim=True) + EPS)
        return float((s64 * r * d["weight"].double() * d["dy"].double()).sum() + (s64 * d["ds"].double()).sum())
    slope = (loss(base + 1e-5 * step) - loss(base - 1e-5 * step)) / 2e-5
    assert abs(slope - float((want["dx"] * step).sum())) <= 1e-6 * float((want["dx"] * step).abs().sum())
    x = d["x"].to(BF16).cuda().requires_grad_()
    y = ssm.rms_norm(x, c["weight"])
    y.sum().backward()
    assert x.grad.dtype is BF16
