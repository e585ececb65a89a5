"""Calls whose tiles are more than one launch may have (2^32 work-items): the gated recurrence over
very many rows, steps or channels, and the values of very many 8-bit moments."""
import pytest
import torch

import selective_state_space_49_amd as ssm
from tests import train_ref
from tests.gpu_util import bitwise_equal, say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def need(gigabytes):
    free = torch.cuda.mem_get_info()[0]
    if free < gigabytes * 1e9:
        pytest.skip(f"{gigabytes} GB of device memory are needed, {free / 1e9:.0f} are free")


def randn(shape, seed, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        part = flat[at:at + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda"))
    return out


def test_many_rows():
    # 65535 x 16384 / 64 tiles of one step: two launches in each direction
    b, D = 65535, 16384
    need(60)
    say("gated rows", b, D)
    x, r, i, dy = (randn((b, 1, D), k) for k in range(4))
    decay, h0 = randn((D,), 5) - 3, None
    y, hf, st = ssm.ssm_gated_fwd_save(x, r, i, decay, h0)
    g = ssm.ssm_gated_bwd(x, r, i, decay, st, dy=dy, want_dh0=False)
    torch.cuda.synchronize()
    for rows in (slice(0, 8), slice(32764, 32772), slice(b - 8, b)):
        part = [t[rows].contiguous() for t in (x, r, i)]
        y1, hf1, st1 = ssm.ssm_gated_fwd_save(*part, decay)
        g1 = ssm.ssm_gated_bwd(*part, decay, st1, dy=dy[rows].contiguous(), want_dh0=False)
        assert bitwise_equal(y[rows], y1) and bitwise_equal(hf[rows], hf1)
        for k in ("dx", "dr", "di"):
            assert bitwise_equal(g[k][rows], g1[k]), k
    # ddecay against sums over fewer rows: its own rounding, 2e-5 of the root of the sum of squares
    total, squares = torch.zeros(D, dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
    for at in range(0, b, 8192):
        rows = slice(at, min(b, at + 8192))
        part = [t[rows].contiguous() for t in (x, r, i)]
        _, _, st1 = ssm.ssm_gated_fwd_save(*part, decay)
        g1 = ssm.ssm_gated_bwd(*part, decay, st1, dy=dy[rows].contiguous(), want_dh0=False)
        total += g1["ddecay"].double()
        squares += g1["ddecay"].double() ** 2
    assert bool(((g["ddecay"].double() - total).abs() <= 2e-5 * squares.sqrt()).all())


def test_many_steps():
    # 2^30 steps of one channel: 2^23 tiles forwards, 2^24 backwards; fast decays, so that a stretch
    # of 2000 steps forgets what lies 1000 steps away
    L = 1 << 30
    need(30)
    say("gated steps", L)
    x, r, i, dy = (randn((1, L, 1), k, torch.bfloat16) for k in range(4))
    decay = torch.full((1,), 1.0, device="cuda")
    y, hf, st = ssm.ssm_gated_fwd_save(x, r, i, decay)
    g = ssm.ssm_gated_bwd(x, r, i, decay, st, dy=dy, want_dh0=False)
    torch.cuda.synchronize()
    for at in (0, L // 2 - 1500, L - 3000):
        part = [t[:, at:at + 3000].cpu() for t in (x, r, i)]
        ref = train_ref.gated(*part, decay, dy=dy[:, at:at + 3000].cpu())
        inner = slice(0 if at == 0 else 1000, 3000 if at == L - 3000 else 2000)
        for k, t in (("y", y), ("dx", g["dx"]), ("dr", g["dr"]), ("di", g["di"])):
            top = float(ref[k].abs().max())
            got = t[:, at:at + 3000][:, inner].double().cpu()
            assert float((got - ref[k][:, inner]).abs().max()) <= 2.0 ** -8 * top, (k, at)
    assert float((hf.double().cpu() - ref["h_final"]).abs().max()) <= 2e-5 * float(ref["y"].abs().max())


def test_many_channels():
    # 2^28 channels of one step: the sums of ddecay take two launches
    D = 1 << 28
    need(20)
    say("gated channels", D)
    x, r, i, dy = (randn((1, 1, D), k, torch.bfloat16) for k in range(4))
    decay = randn((D,), 5) - 3
    y, hf, st = ssm.ssm_gated_fwd_save(x, r, i, decay)
    g = ssm.ssm_gated_bwd(x, r, i, decay, st, dy=dy, want_dh0=False)
    torch.cuda.synchronize()
    for at in (0, (1 << 26) * 4 - 400 - (1 << 27), (0xffffffff // 1024) * 64 - 200, D - 400):
        part = [t[..., at:at + 400].cpu() for t in (x, r, i)]
        ref = train_ref.gated(*part, decay[at:at + 400], dy=dy[..., at:at + 400].cpu())
        for k, t in (("y", y), ("dx", g["dx"]), ("ddecay", g["ddecay"])):
            tol = 2e-5 if k == "ddecay" else 2.0 ** -8
            assert float((t[..., at:at + 400].double().cpu() - ref[k]).abs().max()) <= tol * float(ref[k].abs().max()), (k, at)


def test_many_moments():
    # 2^34 codes and a block: 2^32 work-items of four values
    n = (1 << 34) + 256
    need(190)
    say("adamw values", n)
    m = torch.zeros(n, dtype=torch.int8, device="cuda")
    v = torch.zeros(n, dtype=torch.uint8, device="cuda")
    ms, vs = torch.ones(n // 256, device="cuda"), torch.ones(n // 256, device="cuda")
    spots = [0, (1 << 33) - 256, 1 << 33, (1 << 34) - 256, 1 << 34]
    for k, at in enumerate(spots):
        m[at:at + 256] = torch.arange(-128, 128, device="cuda").clamp(min=-127) // (k + 1)
        v[at:at + 256] = torch.arange(256, device="cuda") // (k + 1)
    mo, vo = ssm.ssm_adamw_values(m, v, ms, vs)
    torch.cuda.synchronize()
    for at in spots:
        s = slice(at, at + 256)
        want = train_ref.adam_values(*(t.cpu().numpy() for t in (m[s], v[s], ms[:1], vs[:1])))
        assert torch.equal(mo[s].cpu(), torch.from_numpy(want[0])) and torch.equal(vo[s].cpu(), torch.from_numpy(want[1]))
