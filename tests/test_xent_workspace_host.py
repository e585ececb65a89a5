"""The cross entropy's workspace on the host: what a call of given pointers needs, against what any
call of its sizes may, and against the logits that it does without."""
import ctypes

import pytest

import selective_state_space_49_amd as ssm

WS, F32, BF16 = 6, 0, 1
SIZES = [(8192, 4096, 32000), (2048, 4096, 128000), (8, 4096, 32000), (100, 256, 1000), (1000, 1000, 16001),
         (30, 1777, 40001), (1, 64, 300), (300, 65, 70001)]
p = lambda v: None if v is None else ctypes.c_void_p(v)  # noqa: E731
ALIGNED, ODD = 1 << 40, (1 << 40) + 4


def needs(T, K, V, io, at, each):
    lib = ssm.load_library()
    return (lib.ssm_xent_fwd_workspace_for(p(at), p(at), T, K, V, io),
            lib.ssm_xent_bwd_workspace_for(p(at), p(at), p(ALIGNED if each else None), T, K, V, io))


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("T,K,V", SIZES)
def test_bounds(T, K, V, io):
    fwd, bwd = ssm.ssm_xent_fwd_workspace(T, K, V, io), ssm.ssm_xent_bwd_workspace(T, K, V, io)
    # a piece of dlogits and one of weight's copy; two copies of hidden in up to three parts of 16 bits
    # (padded to 64); dhidden in float32; the partial sums of few tiles; pairs for every 64 logits
    piece, rows = 1 << 28, -(-T // 64) * 64 * -(-K // 64) * 64
    most = 3 * piece + 2 * rows * 6 + T * K * 4 + (64 << 20) + 4096
    assert bwd <= most and fwd <= 2 * piece + rows * 6 + T * V // 8 + 64 * T + 16 * V + 4096
    for at in (ALIGNED, ODD):
        for each in (False, True):
            f, b = needs(T, K, V, io, at, each)
            assert 0 < f <= fwd and 0 < b <= bwd


def test_aligned_bfloat16_needs_no_copies():
    # less than the float32 logits of many tokens, and little for few
    for T, K, V in SIZES[:2]:
        fwd, bwd = needs(T, K, V, BF16, ALIGNED, False)
        assert fwd < 0.02 * 4 * T * V and bwd < 0.5 * 4 * T * V
    fwd, bwd = needs(8, 4096, 32000, BF16, ALIGNED, False)
    assert fwd < 1 << 20 and bwd < 16 << 20
    assert needs(8, 4096, 32000, BF16, ODD, False)[1] > 200 << 20  # weight has to be copied


@pytest.mark.parametrize("io,at", [(F32, ALIGNED), (BF16, ALIGNED), (BF16, ODD)])
def test_a_byte_less_is_refused(io, at):
    lib, (T, K, V) = ssm.load_library(), (100, 256, 1000)
    MB = 1 << 20
    for each in (False, True):
        fwd, bwd = needs(T, K, V, io, at, each)
        assert lib.ssm_xent_fwd(p(at), p(at + 8 * MB), p(MB), -100, p(2 * MB), p(3 * MB), p(4 * MB), T, K, V, io,
                                p(64 * MB), fwd - 1, None) == WS
        assert lib.ssm_xent_bwd(p(at), p(at + 8 * MB), p(MB), -100, p(2 * MB), p(3 * MB), p(ALIGNED + 64 * MB) if each else None,
                                p(4 * MB), p(5 * MB), p(6 * MB), T, K, V, io, p(64 * MB), bwd - 1, None) == WS
