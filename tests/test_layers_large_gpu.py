"""The layer operators where offsets pass 32 bits, on samples that a 64-bit form can follow.
Tolerances as in the operators' own tests."""
import pytest
import torch

import selective_state_space_49_amd as ssm
from tests import layers_ref as ref
from tests.gpu_util import bitwise_equal, say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 27):
        part = flat[at:at + (1 << 27)]
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda").mul_(scale))
    return out


def test_linear_attention_256k():
    # 262144 x 65 heads of 127: 2^31.01 elements in v, o and their gradients, twice as many bytes; heads
    # are independent, and behind a cut so are documents: the last one of three heads, and its gradients
    L, H, K, V, last = 262144, 65, 16, 127, 200
    say("linear attention 256k", L, H, K, V)
    q, k = randn((1, L, 5, K), BF16, 1), randn((1, L, 5, K), BF16, 2, 0.25)
    v, do = randn((1, L, H, V), BF16, 3), randn((1, L, H, V), BF16, 4)
    g = randn((1, L, H), F32, 5).abs_().mul_(-0.1)
    g[:, L - last] = -torch.inf
    o, h, states = ssm.ssm_linattn_fwd_save(q, k, v, g)
    out = ssm.ssm_linattn_bwd(q, k, v, g, states, do=do)
    torch.cuda.synchronize()
    for heads in ([0], [31], [64]):
        cut = lambda t: t[:, L - last:].index_select(2, torch.tensor(heads, device="cuda")).cpu()  # noqa: E731
        group = lambda t: t[:, L - last:, [heads[0] // 13]].cpu()  # noqa: E731
        want = ref.linattn(group(q), group(k), cut(v), cut(g), None, None, cut(do))
        for name, got in (("o", cut(o)), ("dv", cut(out["dv"]))):
            assert float((got.double() - want[name]).abs().max()) <= 2.0 ** -7 * float(want[name].abs().max()), (heads, name)
        top = float(want["h_final"].abs().max())
        assert float((h[:, heads].double().cpu() - want["h_final"]).abs().max()) <= 2.0 ** -7 * top
    # a group's heads share q: its gradient is their sum
    heads = torch.arange(52, 65, device="cuda")
    cut = lambda t: t[:, L - last:].index_select(2, heads).cpu()  # noqa: E731
    want = ref.linattn(q[:, L - last:, 4:].cpu(), k[:, L - last:, 4:].cpu(), cut(v), cut(g), None, None, cut(do))
    for name in ("dq", "dk"):
        got = out[name][:, L - last:, 4:].double().cpu()
        assert float((got - want[name]).abs().max()) <= 2.0 ** -7 * float(want[name].abs().max()), name


def test_token_of_many_states():
    # 17000 x 8 states of 128 x 128 in float32: 2^31.05 elements
    S = 17000
    say("token of many states", S)
    h = randn((1, S, 8, 128, 128), F32, 1)
    q, k, v = (randn((1, S, 8, 128), F32, n) for n in (2, 3, 4))
    g = randn((1, S, 8), F32, 5).abs_().mul_(-1.0)
    pick = [0, 8191, 16383, S - 1]
    before = h[0, pick].double().cpu()
    o = ssm.ssm_linattn_step(h, q, k, v, g)
    torch.cuda.synchronize()
    at = lambda t: t[0, pick].double().cpu()  # noqa: E731
    want = torch.exp(at(g))[..., None, None] * before + at(k)[..., None] * at(v)[..., None, :]
    assert float((at(h) - want).abs().max()) <= 4 * 2.0 ** -24 * float(want.abs().max())
    out = (at(q)[..., None] * want).sum(2) * 128 ** -0.5
    assert float((at(o) - out).abs().max()) <= 1.8e-5 * float(out.abs().max())


def test_norm_of_many_rows():
    # 2^31.02 elements in rows of 8225, and 2^25 rows of 65
    for rows, dim in ((264000, 8225), (1 << 25, 65)):
        say("norm of many rows", rows, dim)
        x, w = randn((rows, dim), BF16, 1), randn((dim,), F32, 2)
        y, _, rstd = ssm.ssm_rmsnorm_fwd(x, w)
        pick = torch.tensor([0, 1, rows // 2, rows - 2, rows - 1], device="cuda")
        want = ref.norm(x[pick], w)
        off = (y[pick].double().cpu() - want["y"]).abs()
        assert bool((off <= 2.0 ** -8 * want["y"].abs()).all())
        dy = randn((rows, dim), BF16, 3)
        dx, _, dw = ssm.ssm_rmsnorm_bwd(dy, x, w, rstd)
        part = ssm.ssm_rmsnorm_bwd(dy[pick], x[pick], w, rstd[pick])[0]
        assert bitwise_equal(dx[pick], part) and bool(torch.isfinite(dw).all())
        codes, scales, _ = ssm.ssm_rmsnorm_fwd_q8(x, w, group=32)
        some = ssm.ssm_rmsnorm_fwd_q8(x[pick], w, group=32)
        assert bitwise_equal(scales[pick], some[1]) and torch.equal(codes[pick].view(torch.int8), some[0].view(torch.int8))
        del dy, dx, y
        values = ssm.ssm_q8_values(codes, scales, group=32)
        assert bitwise_equal(values[pick], ssm.ssm_q8_values(some[0], some[1], group=32))


def test_sampling_over_many_logits():
    # 65535 x 32771: 2^31.0003 logits
    rows, vocab = 65535, 32771
    say("sampling over many logits", rows, vocab)
    logits = randn((rows, vocab), BF16, 1, 3.0)
    u = torch.rand(rows, generator=torch.Generator().manual_seed(2)).cuda()
    tokens = ssm.ssm_sample(logits, u, top_k=50, top_p=0.9)
    for r in (0, 32768, 65533, 65534):
        assert int(tokens[r]) == ref.sample(logits[r].cpu(), float(u[r]), top_k=50, top_p=0.9)[0]
