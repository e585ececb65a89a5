"""The layer operators' binding, on the host: what is not on a GPU, or of another shape or type, is refused
before the library is called."""
import pytest
import torch

import selective_state_space_49_amd as ssm

F32 = torch.float32


def tensors():
    q = torch.zeros(1, 5, 2, 8)
    v = torch.zeros(1, 5, 4, 6)
    return q, q.clone(), v, torch.zeros(1, 5, 4)


CALLS = {
    "linattn_fwd": lambda: ssm.ssm_linattn_fwd(*tensors()),
    "linattn_fwd_save": lambda: ssm.ssm_linattn_fwd_save(*tensors()),
    "linear_attention": lambda: ssm.linear_attention(*(t.requires_grad_() for t in tensors())),
    "linattn_bwd": lambda: ssm.ssm_linattn_bwd(*tensors(), torch.zeros(1, 4, 1, 8, 6), do=torch.zeros(1, 5, 4, 6)),
    "linattn_step": lambda: ssm.ssm_linattn_step(torch.zeros(1, 5, 4, 8, 6), *tensors()),
    "rmsnorm_fwd": lambda: ssm.ssm_rmsnorm_fwd(torch.zeros(3, 8), torch.ones(8)),
    "rms_norm": lambda: ssm.rms_norm(torch.zeros(3, 8), torch.ones(8), torch.zeros(3, 8)),
    "rmsnorm_fwd_q8": lambda: ssm.ssm_rmsnorm_fwd_q8(torch.zeros(3, 8), torch.ones(8)),
    "q8_values": lambda: ssm.ssm_q8_values(torch.zeros(3, 8, dtype=torch.int8), torch.ones(3, 1)),
    "rmsnorm_bwd": lambda: ssm.ssm_rmsnorm_bwd(torch.zeros(3, 8), torch.zeros(3, 8), torch.ones(8), torch.ones(3)),
    "sample": lambda: ssm.ssm_sample(torch.zeros(3, 8), torch.zeros(3)),
}


@pytest.mark.parametrize("name", CALLS)
def test_not_on_a_gpu(name):
    with pytest.raises((TypeError, ValueError), match="(?i)gpu|cuda|device"):
        CALLS[name]()


def test_types():
    half = torch.zeros(3, 8, dtype=torch.float16)
    for call in (lambda: ssm.ssm_rmsnorm_fwd(half, torch.ones(8)), lambda: ssm.ssm_sample(half, torch.zeros(3)),
                 lambda: ssm.ssm_rmsnorm_fwd(torch.zeros(3, 8), torch.ones(8), half)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="residual_out"):
        ssm.ssm_rmsnorm_fwd(torch.zeros(3, 8), torch.ones(8), residual_out=torch.zeros(3, 8))
    with pytest.raises(ValueError, match="e4m3"):
        ssm.ssm_rmsnorm_fwd_q8(torch.zeros(3, 8), torch.ones(8), code="e5m2")
    with pytest.raises(TypeError, match="codes"):
        ssm.ssm_q8_values(torch.zeros(3, 8), torch.ones(3, 1))
    with pytest.raises(ValueError, match="group"):
        ssm.ssm_q8_values(torch.zeros(3, 8, dtype=torch.int8), torch.ones(3, 5))
    with pytest.raises(ValueError):
        ssm.ssm_linattn_fwd(torch.zeros(5, 2, 8), torch.zeros(5, 2, 8), torch.zeros(5, 4, 6), torch.zeros(5, 4))
    with pytest.raises(ValueError):
        ssm.ssm_linattn_step(torch.zeros(4, 8, 6), torch.zeros(2, 8), torch.zeros(2, 8), torch.zeros(4, 6), torch.zeros(4))


def test_workspaces():
    """Sizes that depend on nothing but the shape, 0 for one that is refused."""
    assert ssm.ssm_linattn_fwd_workspace(1, 64, 8, 8, 128, 128) == 0
    assert ssm.ssm_linattn_fwd_workspace(1, 4096, 8, 8, 128, 128) > 0
    assert ssm.ssm_linattn_fwd_workspace(1, 4096, 8, 3, 128, 128) == 0
    assert ssm.ssm_linattn_bwd_workspace(1, 4096, 8, 2, 128, 128) >= 2 * 4096 * 8 * 128 * 4  # dq and dk of every head
    assert ssm.ssm_linattn_states_bytes(2, 130, 3, 8, 6, ssm.SSM_BF16) == 2 * 3 * 3 * 8 * 6 * 4
    assert ssm.ssm_linattn_states_bytes(2, 130, 3, 8, 6, ssm.SSM_F32) == 2 * 3 * 5 * 8 * 6 * 4
    assert ssm.ssm_rmsnorm_bwd_workspace(1, 100) == 400 and ssm.ssm_rmsnorm_bwd_workspace(1 << 20, 4096) == 512 * 4096 * 4
    assert ssm.ssm_rmsnorm_bwd_workspace(5, 1 << 20) == 0 and ssm.ssm_sample_workspace(9, 5003) == 0
