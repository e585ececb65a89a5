"""Cross entropies whose tiles are more than a launch may have are refused on the host, before
anything is enqueued (no GPU is touched; the addresses are never used)."""
import ctypes

import pytest

import selective_state_space_49_amd as ssm

OK, SHAPE, WS, MB = 0, 2, 6, 1 << 20
p = lambda v: ctypes.c_void_p(v << 40)  # noqa: E731  (a terabyte apart)


def fwd(T, K, V, io):
    return ssm.load_library().ssm_xent_fwd(p(1), p(2), p(3), -100, p(4), p(5), p(6), T, K, V, io, None, 0, None)


def bwd(T, K, V, io):
    return ssm.load_library().ssm_xent_bwd(p(1), p(2), p(3), -100, p(4), p(5), None, p(6), p(7), p(8), T, K, V, io, None,
                                           0, None)


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("T,K,V", [(8 << 20, 64, 128000), (1 << 29, 64, 64), (1 << 30, 64, 1000), (4 << 20, 64, 1 << 17)])
def test_too_many_tiles(T, K, V, io):
    assert fwd(T, K, V, io) == SHAPE and ssm.ssm_xent_fwd_workspace(T, K, V, io) == 0


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("T,K,V", [(1 << 30, 64, 1000), (1 << 29, 4096, 64)])
def test_too_many_tiles_of_gradients(T, K, V, io):
    assert bwd(T, K, V, io) == SHAPE and ssm.ssm_xent_bwd_workspace(T, K, V, io) == 0


@pytest.mark.parametrize("io", [0, 1])
@pytest.mark.parametrize("T,K,V", [((4 << 20) - 256, 64, 1 << 17), (1 << 20, 64, 1 << 18), ((1 << 29) - 64, 64, 64), (8, 4096, 1 << 24)])
def test_just_enough(T, K, V, io):
    # up to the missing workspace, which is looked at last
    assert fwd(T, K, V, io) == WS and ssm.ssm_xent_fwd_workspace(T, K, V, io) > 0
    assert bwd(T, K, V, io) == WS and ssm.ssm_xent_bwd_workspace(T, K, V, io) > 0
