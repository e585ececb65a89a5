"""Resets of the gated recurrence with a gate, an input or a state that is NaN or infinite, on
either side of a boundary, wherever waves and tiles meet; and no reset without one."""
import pytest
import torch

import selective_state_space_49_amd as ssm
from tests import train_ref
from tests.gpu_util import bitwise_equal, say
from tests.test_gated_gpu import call, dev, make

pytestmark = pytest.mark.gpu

L = 400
# steps of a wave are 16 forwards and 8 backwards, of a tile 128 and 64
CUTS = (1, 5, 8, 9, 17, 64, 65, 128, 130, 300, L - 1)


def same(a, b):
    return bool((a.isnan() == b.isnan()).all()) and bitwise_equal(a.nan_to_num(), b.nan_to_num())


def with_reset(cut, seed, io=torch.float32):
    d = make(2, L, 70, io, seed=seed, h0=True)
    d["reset"] = torch.zeros(2, L, dtype=torch.bool)
    d["reset"][0, cut] = True
    return d


@pytest.mark.parametrize("name", ["r", "i", "x"])
@pytest.mark.parametrize("cut", CUTS)
def test_nan_before_a_reset(cut, name):
    # one step, or many, before the boundary: nothing of it after the boundary
    for back in {1, 2, min(cut, 20), min(cut, 140), cut}:
        if back > cut:
            continue
        d = with_reset(cut, cut)
        clean = call(dev(d))
        d[name][0, cut - back] = float("nan")
        say("gated nan before", name, cut, back)
        got = call(dev(d))
        for k in ("y", "dx", "dr", "di"):
            assert bitwise_equal(got[k][0, cut:], clean[k][0, cut:]), k
            assert bitwise_equal(got[k][1], clean[k][1]), k
        assert bool(got["y"][0, cut - back:cut].isnan().all())
        assert bitwise_equal(got["h_final"], clean["h_final"])
        after = -(-(cut + 1) // ssm.GATED_STATE_EVERY)  # stored states that enter a step after the reset
        assert bitwise_equal(got["states"][0, after:], clean["states"][0, after:])


@pytest.mark.parametrize("name", ["r", "i", "x", "dy"])
@pytest.mark.parametrize("cut", CUTS)
def test_nan_after_a_reset(cut, name):
    # in the gradients nothing of the later document reaches the earlier one
    for ahead in {0, 1, min(L - 1 - cut, 20), min(L - 1 - cut, 140), L - 1 - cut}:
        if cut + ahead >= L:
            continue
        d = with_reset(cut, cut)
        clean = call(dev(d))
        d[name][0, cut + ahead] = float("nan")
        say("gated nan after", name, cut, ahead)
        got = call(dev(d))
        for k in ("y", "dx", "dr", "di"):
            assert bitwise_equal(got[k][0, :cut], clean[k][0, :cut]), k
            assert bitwise_equal(got[k][1], clean[k][1]), k
        assert bitwise_equal(got["dh0"], clean["dh0"])
        assert bool(got["di"][0, cut + ahead].isnan().all())


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("b,D", [(2, 70), (2, 64), (40, 64), (40, 65)])
@pytest.mark.parametrize("name", [None, "x", "h0", "dy", "dh_final", "r"])
def test_no_reset_is_no_reset(b, D, name, io):
    # fast decays, whose products underflow within a tile: a reset array without a reset gives the
    # same bits as none, and a NaN stays to the end of its document
    say("gated no reset", b, D, name, io)
    d = make(b, L, D, io, seed=D, h0=True)
    d["decay"] = torch.linspace(-4, 3, D)
    if name in ("x", "r"):
        d[name][0, 10, :] = float("nan")
    elif name == "dy":
        d[name][0, L - 10, :] = float("nan")
    elif name:
        d[name][0] = float("nan")
    want = call(dev(d))
    d["reset"] = torch.zeros(b, L, dtype=torch.bool)
    got = call(dev(d))
    for k in want:
        assert same(got[k], want[k]), k
    if name in ("x", "r", "h0"):
        assert bool(got["y"][0, 10:].isnan().all()) and bool(got["h_final"][0].isnan().all())
        assert not bool(got["y"][1:].isnan().any())
    if name in ("dy", "dh_final"):
        assert bool(got["dx"][0, :L - 10].isnan().all()) and bool(got["dh0"][0].isnan().all())


def test_many_resets_against_64_bits():
    # documents of one step and more, whole tiles of resets
    d = make(2, 700, 66, torch.float32, seed=21, h0=True)
    d["reset"] = torch.rand((2, 700), generator=torch.Generator().manual_seed(3)) < 0.5
    d["reset"][0, 100:400] = True
    ref, got = train_ref.gated(**d), call(dev(d))
    for k in ("y", "dx", "dr", "di", "h_final", "dh0"):
        top = max(float(ref[k].abs().max()), 1e-30)
        assert float((got[k].double().cpu() - ref[k]).abs().max()) <= 2e-5 * top, k
