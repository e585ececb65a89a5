"""Quotients in the middle of two codes go to the even one, whatever the scale: y / scale, not y times a
reciprocal, which puts 73.5 / 49 below 1.5."""
import pytest
import torch

import selective_state_space_49_amd as ssm
from tests import layers_ref as ref
from tests.gpu_util import bitwise_equal, say

pytestmark = pytest.mark.gpu
# odd ones of up to 12 bits: their products with 9-bit quotients are float32 numbers
SCALES = [1.0, 3.0, 5.0, 7.0, 10.0, 49.0, 0.046875, 197.0, 1021.0, 4093.0, 49 * 2.0 ** -20, 2047 * 2.0 ** 30]


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
def test_middles(code, group):
    """A row of equal values has the norm 1, so y is the weight."""
    if code == "e4m3":
        table = torch.from_numpy(ref.e4m3_values())
    else:
        table = torch.arange(128.0, dtype=torch.float64)
    mid = (table[1:] + table[:-1]) / 2
    u = torch.cat([mid, -mid, table, mid * (1 + 2.0 ** -11), mid * (1 - 2.0 ** -11)])
    size = group or len(u) + 1
    most = float(table[-1])
    u = torch.cat([torch.cat([torch.tensor([most], dtype=torch.float64), part]) for part in u.split(size - 1)])
    for scale in SCALES:
        say("ties", code, group, scale)
        w = (u * scale).float()
        x = torch.ones(2, len(w), device="cuda")
        codes, scales, _ = ssm.ssm_rmsnorm_fwd_q8(x, w.cuda(), eps=0.0, code=code, group=group)
        values, want, _ = ref.coded(w.double()[None].numpy(), code, group)
        assert bitwise_equal(scales.cpu(), torch.from_numpy(want).expand(2, -1).contiguous())
        assert bool((scales == scale).all())
        got = ssm.ssm_q8_values(codes, scales, group=group).cpu()
        assert torch.equal(got, torch.from_numpy(values).float().expand(2, -1)), (scale, int((got[0] != torch.from_numpy(values).float()[0]).sum()))
