"""The norm where its kernels change: rows that start on any element, whose gradients have the aligned ones' bits
too, and more rows of a block than one launch has."""
import pytest
import torch

import selective_state_space_49_amd as ssm
from tests import layers_ref as ref
from tests.gpu_util import bitwise_equal, say
from tests.test_rmsnorm_gpu import TYPES, dev, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [100, 256, 333, 1001, 1500, 5003, 9001])
@pytest.mark.parametrize("types", TYPES, ids=str)
def test_any_start(types, dim):
    """One order of sums for every alignment."""
    say("norm unaligned", types, dim)
    d = dev(make(7, dim, *types))

    def moved(t):
        if t is None:
            return None
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:].copy_(t.reshape(-1))
        return flat[1:].view(t.shape)

    def run(c):
        y, s, rstd = ssm.ssm_rmsnorm_fwd(c["x"], c["weight"], c["residual"])
        s = c["x"] if s is None else s
        back = ssm.ssm_rmsnorm_bwd(c["dy"], s, c["weight"], rstd, ds=c["ds"])
        return (y, s, rstd, *back)
    for a, b in zip(run(d), run({k: moved(t) for k, t in d.items()})):
        assert bitwise_equal(a, b)


def test_more_rows_than_a_launch():
    """2^21 rows are a launch where a block has one: the rows behind them come in a second."""
    rows, dim = (1 << 21) + 3, 1026
    say("norm of several launches", rows, dim)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(rows, dim, dtype=torch.bfloat16, device="cuda")
    for part in x.split(1 << 18):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    w = 1 + 0.2 * torch.randn(dim, generator=g, device="cuda")
    residual = x.float()
    pick = torch.tensor([0, 1, (1 << 21) - 1, 1 << 21, (1 << 21) + 2], device="cuda")
    want = ref.norm(x[pick], w, residual[pick])
    y, s, rstd = ssm.ssm_rmsnorm_fwd(x, w, residual, residual_out=residual)
    off = (y[pick].double().cpu() - want["y"]).abs()
    assert bool((off <= 2.0 ** -8 * want["y"].abs()).all())
    assert bitwise_equal(s[pick].cpu(), want["s"]) and s.data_ptr() == residual.data_ptr()
    assert float((rstd[pick].double().cpu() / want["rstd"] - 1).abs().max()) <= 2.0 ** -24
    del y, s, residual
    for group in (0, 128):
        codes, scales, _ = ssm.ssm_rmsnorm_fwd_q8(x, w, code="int8", group=group)
        some = ssm.ssm_rmsnorm_fwd_q8(x[pick], w, code="int8", group=group)
        assert torch.equal(codes[pick], some[0]) and bitwise_equal(scales[pick], some[1])


def test_sampling_takes_no_workspace():
    """Whatever the shape: one that is given is left as it is."""
    for shape in ((1, 1), (9, 5003), (65535, 1 << 24)):
        assert ssm.ssm_sample_workspace(*shape) == 0
    given = torch.full((256,), 7, dtype=torch.uint8, device="cuda")
    logits = torch.randn(9, 5003, device="cuda")
    ssm.ssm_sample(logits, torch.full((9,), 0.5, device="cuda"), top_k=50, top_p=0.9, workspace=given)
    assert bool((given == 7).all())
