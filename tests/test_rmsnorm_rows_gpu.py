"""dweight of many rows: a sum of positive terms keeps float32's bits however many there are. The bound is that of
few rows, 64 x 2^-24 of the sum of magnitudes; sums of 1024 rows in 32 bits were off by 160 x 2^-24, of 8192 rows
by more."""
import pytest
import torch

import selective_state_space_49_amd as ssm
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
# 1024 rows (the last: 256) for every sum that a lane or a block kept
SIZES = [(1 << 23, 24), (1 << 22, 160), (1 << 21, 520), (1 << 19, 1100), (1 << 19, 4200), (1 << 19, 8200), (1 << 17, 20000)]


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_terms_of_one_sign(size):
    rows, dim = size
    say("norm of many rows", size)
    x, w = torch.ones(rows, dim, dtype=torch.bfloat16, device="cuda"), torch.ones(dim, device="cuda")
    eps = 2e-4
    _, _, rstd = ssm.ssm_rmsnorm_fwd(x, w, eps=eps)
    dx, _, dw = ssm.ssm_rmsnorm_bwd(x, x, w, rstd)
    want = rows / (1 + eps) ** 0.5
    assert float((dw.double() - want).abs().max()) <= 64 * 2.0 ** -24 * want
    # a term that is not like the others arrives
    x[rows // 2 + 1, dim - 1] = 4096.0
    _, _, rstd = ssm.ssm_rmsnorm_fwd(x, w, eps=eps)
    dw = ssm.ssm_rmsnorm_bwd(x, x, w, rstd)[2]
    r = (1 + eps) ** -0.5
    own = ((dim - 1 + 4096.0 ** 2) / dim + eps) ** -0.5
    for at, term in ((dim - 1, 4096.0 ** 2 * own), (0, own)):
        want = (rows - 1) * r + term
        assert abs(float(dw[at]) - want) <= 64 * 2.0 ** -24 * want, (at, float(dw[at]), want)
