"""Linear attention on the GPU against the step-by-step form in 64 bits.

Tolerances, of the largest entry of what is compared: a float32 result is a sum of up to about 300
products in 32 bits (128 of a state's column, 64 of a chunk, the carried ones), each rounded by 2^-24
and summed, 300 x 2^-24 = 1.8e-5. An output of bfloat16 is rounded by 2^-9, and so are the scores and
the state that enter its products: 3 x 2^-9 = 5.9e-3 of the terms' size where these errors agree in
sign, and 2^-7 leaves a third for terms that are larger than their sum."""
import math

import pytest
import torch

import selective_state_space_49_amd as ssm
from tests import layers_ref as ref
from tests.gpu_util import bitwise_equal, say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
IO = {"f32": F32, "bf16": BF16}
TOL = {F32: 1.8e-5, BF16: 2.0 ** -7}


def make(b, L, H, Hk, K, V, io="f32", decay="token", cuts=0.0, h0=False, strong=False, seed=0):
    """Inputs on the CPU."""
    g = torch.Generator().manual_seed(seed + 7919 * L + 31 * K + V)
    dt = IO[io]
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = {"q": rn(b, L, Hk, K).to(dt), "k": (rn(b, L, Hk, K) / math.sqrt(K)).to(dt), "v": rn(b, L, H, V).to(dt)}
    if decay == "head":
        d["g"] = -torch.rand(H, generator=g) * 0.1
    else:
        d["g"] = -torch.rand(b, L, H, generator=g) * (40.0 if strong else 0.3)
        d["g"][torch.rand(b, L, H, generator=g) < cuts] = -math.inf
    d["h0"] = rn(b, H, K, V) if h0 else None
    d["do"], d["dh_final"] = rn(b, L, H, V).to(dt), rn(b, H, K, V) if h0 else None
    return d


def close(got, want, name, tol=None):
    assert got.shape == want.shape, (name, got.shape, want.shape)
    if got.numel() == 0:
        return
    err = float((got.double().cpu() - want).abs().max())
    top = float(want.abs().max())
    assert err <= (TOL[got.dtype] if tol is None else tol) * max(top, 1e-30), f"{name}: off by {err} of {top}"


def dev(d):
    return {k: None if t is None else t.cuda() for k, t in d.items()}


def run(d, scale=None):
    c = dev(d)
    o, h, states = ssm.ssm_linattn_fwd_save(c["q"], c["k"], c["v"], c["g"], c["h0"], scale=scale)
    grads = ssm.ssm_linattn_bwd(c["q"], c["k"], c["v"], c["g"], states, do=c["do"], dh_final=c["dh_final"], scale=scale)
    torch.cuda.synchronize()
    return {"o": o, "h_final": h, "states": states, **grads}


def against(d, scale=None):
    got = run(d, scale)
    want = ref.linattn(d["q"], d["k"], d["v"], d["g"], d["h0"], scale, d["do"], d["dh_final"])
    for name in ("o", "h_final", "dq", "dk", "dv", "dg", "dh0"):
        close(got[name], want[name], name)
    chunk = ssm.LINATTN_CHUNK[d["q"].dtype is BF16]
    close(got["states"], torch.stack(want["states"][::chunk], 2), "states")
    return got, want


CASES = [
    # b, L, H, Hk, K, V
    (1, 1, 1, 1, 1, 1), (2, 1, 3, 3, 16, 16), (1, 2, 2, 1, 8, 24), (2, 31, 2, 2, 33, 17), (1, 32, 4, 2, 64, 64),
    (1, 33, 2, 2, 64, 128), (2, 63, 2, 1, 128, 64), (1, 64, 1, 1, 128, 128), (3, 65, 2, 2, 100, 127),
    (1, 128, 6, 3, 48, 80), (1, 129, 3, 1, 127, 65), (2, 300, 4, 4, 32, 40),
]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", CASES, ids=str)
def test_forward_and_gradients(size, io):
    say("linattn", size, io)
    against(make(*size, io=io))
    against(make(*size, io=io, cuts=0.1, h0=True, seed=1))
    against(make(*size, io=io, decay="head", h0=True, seed=2), scale=0.7)


@pytest.mark.parametrize("io,L", [("f32", 700), ("bf16", 1500), ("bf16", 2113)])
def test_segments(io, L):
    """Long enough for several segments, whose states come from passes of their own."""
    size = (1, L, 2, 1, 40, 72)
    say("linattn segments", size, io)
    args = (size[0], L, size[2], size[3], size[4], size[5])
    assert ssm.ssm_linattn_fwd_workspace(*args, int(io == "bf16")) > 0
    against(make(*size, io=io, h0=True))
    against(make(*size, io=io, cuts=0.002, h0=True, seed=1))
    against(make(*size, io=io, decay="head", seed=2))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strong_decays(io):
    """Decays down to e^-40 a step, and below float32's range: dg stays right relative to the largest of
    its own position's neighbours, not only to the largest of all."""
    d = make(1, 200, 3, 3, 24, 24, io=io, strong=True, h0=True)
    d["g"][:, 50:60] = -200.0
    d["g"][:, 100] = -1e30
    got, want = against(d)
    assert bool((got["dg"][:, 50:60] == 0).all()) and bool((got["dg"][:, 100] == 0).all())
    # every dg is a sum of products that all carry its own decay: relative to that decay times what
    # 24 x 24 products of values of size 1 add up to
    size = torch.exp(d["g"].double().clamp(min=-104)) * float((want["dg"].abs() / torch.exp(d["g"].double().clamp(min=-104))).max())
    live = d["g"] >= -80
    err = (got["dg"].double().cpu() - want["dg"]).abs()
    assert bool((err[live] <= 1.8e-5 * size[live]).all()), float((err[live] / size[live]).max())


def test_cut_in_head_decay_and_growth():
    d = make(2, 70, 3, 3, 16, 16, decay="head", h0=True)
    d["g"] = torch.tensor([-math.inf, 0.0, 0.01])
    against(d)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_a_document_sees_nothing_of_another(io):
    """Changing one document changes no bit of the others, in the outputs and in the gradients."""
    d = make(1, 400, 2, 1, 32, 32, io=io)
    for t in (90, 215):
        d["g"][:, t] = -math.inf
    base = run(d)
    e = {k: None if t is None else t.clone() for k, t in d.items()}
    for k in ("q", "k", "v", "do"):
        e[k][:, 90:215] = e[k][:, 90:215].flip(1) * 1.5
    other = run(e)
    for name in ("o", "dq", "dk", "dv", "dg"):
        for part in (slice(0, 90), slice(215, 400)):
            assert bitwise_equal(base[name][:, part].contiguous(), other[name][:, part].contiguous()), name
    assert bitwise_equal(base["h_final"], other["h_final"])


def test_nothing_of_later_tokens():
    d = make(1, 150, 2, 2, 16, 48, io="bf16")
    c = dev(d)
    whole, _ = ssm.ssm_linattn_fwd(c["q"], c["k"], c["v"], c["g"])
    for n in (1, 40, 64, 100):
        part, _ = ssm.ssm_linattn_fwd(*(c[k][:, :n].contiguous() for k in ("q", "k", "v", "g")))
        assert bitwise_equal(part, whole[:, :n].contiguous()), n


def test_rows_behind_a_short_output_stay():
    """Nothing is written past the last token, whatever the chunk."""
    d = dev(make(2, 37, 2, 2, 20, 12, io="bf16"))
    room = torch.full((2 * 37 + 64, 2, 12), 7.0, dtype=BF16, device="cuda")
    o = room[:74].view(2, 37, 2, 12)
    ssm.ssm_linattn_fwd(d["q"], d["k"], d["v"], d["g"], o=o)
    assert bool((room[74:] == 7).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shift", [1, 3])
def test_unaligned(io, shift):
    """Tensors that start on any element give the aligned ones' bits."""
    d = dev(make(2, 77, 4, 2, 32, 64, io=io, h0=True))
    got = run(make(2, 77, 4, 2, 32, 64, io=io, h0=True))

    def moved(t):
        flat = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
        flat[shift:].copy_(t.reshape(-1))
        return flat[shift:].view(t.shape)
    m = {k: None if t is None else moved(t) for k, t in d.items()}
    o = moved(torch.empty_like(d["v"]))
    states = moved(got["states"])
    ssm.ssm_linattn_fwd(m["q"], m["k"], m["v"], m["g"], m["h0"], o=o, states=states)
    assert bitwise_equal(o, got["o"]) and bitwise_equal(states, got["states"])
    g = ssm.ssm_linattn_bwd(m["q"], m["k"], m["v"], m["g"], states, do=m["do"], dh_final=m["dh_final"])
    for name in ("dq", "dk", "dv", "dg", "dh0"):
        assert bitwise_equal(g[name], got[name]), name


def test_same_bits_again():
    d = make(2, 600, 4, 2, 64, 64, io="bf16", decay="head", h0=True)
    a, b = run(d), run(d)
    for name in a:
        assert bitwise_equal(a[name], b[name]), name


def test_empty():
    z = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    h0 = torch.randn(2, 3, 4, 5, device="cuda")
    q, v, g = z(2, 0, 3, 4), z(2, 0, 3, 5), -torch.ones(3, device="cuda")
    o, h, states = ssm.ssm_linattn_fwd_save(q, q, v, g, h0)
    assert o.numel() == 0 and torch.equal(h, h0)
    out = ssm.ssm_linattn_bwd(q, q, v, g, states, do=v, dh_final=h0)
    assert torch.equal(out["dh0"], h0) and bool((out["dg"] == 0).all())
    o, h = ssm.ssm_linattn_fwd(z(0, 5, 3, 4), z(0, 5, 3, 4), z(0, 5, 3, 5), g)
    assert o.numel() == 0 and h.numel() == 0
    out = ssm.ssm_linattn_bwd(z(0, 5, 3, 4), z(0, 5, 3, 4), z(0, 5, 3, 5), g, z(0, 3, 1, 4, 5), do=z(0, 5, 3, 5))
    assert bool((out["dg"] == 0).all())


def test_gradients_against_differences():
    """The result is linear in q, k, v and h0 each, so differences of the kernel's own values are the
    gradient up to rounding: 2 x 1.8e-5 of the loss's terms; g's from the 64-bit form."""
    d = make(1, 70, 2, 1, 12, 20, h0=True)
    c, got = dev(d), run(d)

    def loss(x):
        o, h = ssm.ssm_linattn_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"])
        return float((o.double() * c["do"].double()).sum() + (h.double() * c["dh_final"].double()).sum())
    gen = torch.Generator().manual_seed(5)
    for name in ("q", "k", "v", "h0"):
        step = torch.randn(d[name].shape, generator=gen).cuda()
        up, down = (loss({**c, name: c[name] + e * step}) for e in (1.0, -1.0))
        want = float((got["d" + name].double() * step.double()).sum())
        size = float((got["d" + name].double() * step.double()).abs().sum())
        assert abs((up - down) / 2 - want) <= 3.6e-5 * size, (name, up, down, want)
    step = torch.randn(d["g"].shape, generator=gen, dtype=torch.float64)

    def loss64(g):
        r = ref.linattn(d["q"], d["k"], d["v"], g, d["h0"])
        return float((r["o"] * ref.f64(d["do"])).sum() + (r["h_final"] * ref.f64(d["dh_final"])).sum())
    e = 1e-5
    slope = (loss64(d["g"].double() + e * step) - loss64(d["g"].double() - e * step)) / (2 * e)
    mine = got["dg"].double().cpu() * step
    assert abs(slope - float(mine.sum())) <= 1e-6 * abs(slope) + 1.8e-5 * float(mine.abs().sum())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 1, 1, 1, 1, 1), (2, 3, 4, 2, 128, 128), (1, 5, 3, 3, 33, 50), (3, 2, 2, 1, 64, 7)], ids=str)
def test_step(size, io):
    """Tokens one by one are the recurrence, state and all."""
    Ln, S, H, Hk, K, V = size
    for decay in ("token", "head"):
        say("linattn step", size, io, decay)
        d = [make(S, 3, H, Hk, K, V, io=io, cuts=0.1, seed=n) for n in range(Ln)]
        g = [x["g"] if decay == "token" else x["g"][0, 0].clone() for x in d]
        h = torch.stack([torch.randn(S, H, K, V, generator=torch.Generator().manual_seed(n)) for n in range(Ln)])
        want = [ref.linattn(x["q"], x["k"], x["v"], gg, h[n]) for n, (x, gg) in enumerate(zip(d, g))]
        hd = h.cuda()
        for t in range(3):
            at = lambda key: torch.stack([x[key][:, t] for x in d]).cuda()  # noqa: E731
            gt = torch.stack([gg[:, t] if decay == "token" else gg for gg in g]).cuda()
            o = ssm.ssm_linattn_step(hd, at("q"), at("k"), at("v"), gt)
            close(o, torch.stack([w["o"][:, t] for w in want]), "o")
        close(hd, torch.stack([w["h_final"] for w in want]), "h")


def test_step_follows_prefill():
    d = dev(make(2, 90, 4, 2, 64, 64, io="bf16"))
    whole, last = ssm.ssm_linattn_fwd(d["q"], d["k"], d["v"], d["g"])
    cut = lambda a, b: [d[k][:, a:b].contiguous() for k in ("q", "k", "v", "g")]  # noqa: E731
    _, h = ssm.ssm_linattn_fwd(*cut(0, 70))
    h = h[None].contiguous()
    for t in range(70, 90):
        o = ssm.ssm_linattn_step(h, *(x[:, 0][None] for x in cut(t, t + 1)))
        close(o[0], whole[:, t].double().cpu(), "o")
    close(h[0], last.double().cpu(), "h")


def test_autograd():
    d = make(2, 100, 4, 2, 32, 16, h0=True)
    c = {k: t.cuda().requires_grad_(k in ("q", "k", "v", "g", "h0")) for k, t in d.items()}
    o, h = ssm.linear_attention(c["q"], c["k"], c["v"], c["g"], c["h0"])
    ((o * c["do"]).sum() + (h * c["dh_final"]).sum()).backward()
    got = run(d)
    for name in ("q", "k", "v", "g", "h0"):
        assert bitwise_equal(c[name].grad, got["d" + name]), name
    o, h = ssm.linear_attention(c["q"], c["k"], c["v"], c["g"])
    grads = torch.autograd.grad(h.sum(), (c["k"], c["q"]), create_graph=False)
    assert bool((grads[1] == 0).all()) and bool((grads[0] != 0).any())
    o, _ = ssm.linear_attention(c["q"], c["k"], c["v"], c["g"])
    with pytest.raises(RuntimeError):
        gq, = torch.autograd.grad(o.sum(), c["q"], create_graph=True)
        gq.sum().backward()


ODD = [(2, 70, 2, 2, 8, 9), (1, 65, 2, 1, 9, 8), (1, 100, 3, 3, 17, 33), (2, 64, 2, 2, 31, 66), (1, 90, 2, 1, 67, 15),
       (1, 130, 2, 2, 70, 121), (1, 129, 4, 2, 12, 20), (1, 33, 2, 2, 7, 40), (1, 80, 2, 2, 100, 5), (1, 66, 1, 1, 113, 126)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", ODD, ids=str)
def test_odd_widths(size, io):
    """Rows that are no whole vectors, the last of which ends with the row; and rows shorter than one.
    What lies beside the outputs stays."""
    say("linattn odd", size, io)
    d = make(*size, io=io, cuts=0.05, h0=True)
    got, _ = against(d)
    c = dev(d)
    n = d["v"].numel()
    room = torch.full((n + 600,), 7.0, dtype=IO[io], device="cuda")
    at = 257
    ssm.ssm_linattn_fwd(c["q"], c["k"], c["v"], c["g"], c["h0"], o=room[at:at + n].view(d["v"].shape))
    assert bitwise_equal(room[at:at + n].view(d["v"].shape).clone(), got["o"])
    assert bool((room[:at] == 7).all()) and bool((room[at + n:] == 7).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(1, 390, 100, 50, 9, 11), (3, 260, 45, 45, 8, 70), (2, 700, 150, 10, 40, 8)], ids=str)
def test_segments_of_many_heads(size, io):
    """Several segments, and more blocks than the GPU takes at once."""
    say("linattn many heads", size, io)
    against(make(*size, io=io, cuts=0.01, h0=True))
