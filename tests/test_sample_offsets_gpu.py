"""Rows whose kept tokens end among thousands of equal or nearly equal logits: what a list in LDS does not hold.
bfloat16 logits around 20 lie 1/8 apart. Tokens are those of the sorted list, as everywhere (see
test_sample_gpu.py), and the time is not that of a row for every bit of a place."""
import math

import pytest
import torch

import selective_state_space_49_amd as ssm
from tests.gpu_util import say
from tests.test_sample_gpu import check

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U = torch.tensor([0.03, 0.5, 0.97])


def around(rows, vocab, io, mean, spread, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, vocab, generator=g) * spread + mean).to(io)


@pytest.mark.parametrize("case", [(20.0, 2.0, {"top_p": 0.9}), (20.0, 2.5, {"top_p": 0.95, "temperature": 1.3}),
                                  (-10.0, 1.5, {"top_p": 0.95}), (20.0, 2.0, {"top_k": 20000}),
                                  (-20.0, 2.0, {"top_k": 30000, "top_p": 0.7}), (100.0, 4.0, {"top_k": 60000, "top_p": 0.99, "min_p": 1e-4})],
                         ids=str)
def test_bfloat16_away_from_0(case):
    mean, spread, settings = case
    say("offset", case)
    check(around(2, 131072, BF16, mean, spread), U[1:], **settings)


@pytest.mark.parametrize("io", [F32, BF16], ids=str)
@pytest.mark.parametrize("vocab", [2049, 4096, 5000, 65537])
def test_plateaus(io, vocab):
    """All equal, two plateaus, and one below a few that are ahead, above and below 0."""
    for settings in ({"top_p": 0.37}, {"top_k": vocab - 7}, {"top_k": vocab // 2 + 1, "top_p": 0.61}, {"top_p": 0.999999}):
        for high in (3.0, -3.0):
            say("plateau", io, vocab, settings, high)
            x = torch.full((3, vocab), high)
            x[1, 1::2] = high - 0.5
            x[2, 100::1000] = high + 4
            check(x.to(io), U, **settings)


def test_many_nearly_equal():
    """float32 logits that are all different, thousands of them in a step."""
    for vocab in (5000, 100001):
        for settings in ({"top_p": 0.5}, {"top_k": 3000}, {"top_k": 4000, "top_p": 0.9}):
            say("nearly equal", vocab, settings)
            x = around(3, vocab, F32, 1.0, 1e-6)
            x[:, 7] = -30.0  # so that the steps are wide
            check(x, U, **settings)


def test_infinities_with_limits():
    x = around(3, 6000, F32, 0.0, 1.0)
    x[0, ::2] = math.inf
    x[1, 5] = math.inf
    x[2, 1000:] = -math.inf
    for io in (F32, BF16):
        for settings in ({"top_k": 2999}, {"top_p": 0.3}, {"top_k": 1500, "top_p": 0.5}, {"top_k": 3500}):
            say("infinities", io, settings)
            check(x.to(io), U, **settings)


def test_time():
    """Not more than 6 times as long as the same logits around 0 (a pass for every bit: 25 times)."""
    def time(mean):
        logits, u = around(64, 131072, BF16, mean, 2.0).cuda(), torch.rand(64, generator=torch.Generator().manual_seed(1)).cuda()
        call = lambda: ssm.ssm_sample(logits, u, top_p=0.9)  # noqa: E731
        times = []
        for _ in range(7):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            call()
            end.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(end))
        return sorted(times)[3]
    near, far = time(0.0), time(20.0)
    assert far <= 6 * near, (near, far)


def test_distances_past_float32():
    """A temperature so high that logits keep their mass over a distance that float32 does not hold."""
    x = torch.tensor([3e38, -3e38, 2e38, -1e38, 1e38, -2e38, 0.0, -math.inf]).repeat(4, 3)
    u = torch.tensor([0.05, 0.4, 0.8, 0.99])
    for t in (1e37, 1e38, 3e38):
        for settings in ({}, {"top_p": 0.97}, {"top_k": 20}, {"top_k": 19, "top_p": 0.9}, {"min_p": 0.01, "top_p": 0.999}):
            say("distances", t, settings)
            check(x, u, temperature=t, **settings)
