"""Sizes past 32 bits are refused: cut to 32 bits, a group of 2^32 + 32 wrote a scale for every 32 values into an
array that had one for the row, and 2^32 + 8 columns were normed as 8."""
import pytest
import torch

import selective_state_space_49_amd as ssm

FAR = 2 ** 32


def wide(*shape, dtype=torch.float32):
    return torch.zeros((), dtype=dtype).expand(*shape)


CALLS = {
    "fwd_q8 group": lambda: ssm.ssm_rmsnorm_fwd_q8(torch.zeros(3, 64), torch.ones(64), group=FAR + 32),
    "fwd_q8 group below": lambda: ssm.ssm_rmsnorm_fwd_q8(torch.zeros(3, 64), torch.ones(64), group=32 - FAR),
    "q8_values group": lambda: ssm.ssm_q8_values(torch.zeros(3, 64, dtype=torch.int8), torch.ones(3, 1), group=FAR + 32),
    "fwd dim": lambda: ssm.ssm_rmsnorm_fwd(wide(1, FAR + 8), wide(FAR + 8)),
    "fwd_q8 dim": lambda: ssm.ssm_rmsnorm_fwd_q8(wide(1, FAR + 8), wide(FAR + 8)),
    "bwd dim": lambda: ssm.ssm_rmsnorm_bwd(wide(1, FAR + 8), wide(1, FAR + 8), wide(FAR + 8), torch.ones(1)),
    "bwd_workspace dim": lambda: ssm.ssm_rmsnorm_bwd_workspace(1, FAR + 8),
    "q8_values dim": lambda: ssm.ssm_q8_values(wide(1, FAR + 8, dtype=torch.int8), torch.ones(1, 1)),
    "linattn_fwd d_k": lambda: ssm.ssm_linattn_fwd(wide(1, 2, 1, FAR + 8), wide(1, 2, 1, FAR + 8), wide(1, 2, 1, 8), torch.zeros(1)),
    "linattn_fwd d_v": lambda: ssm.ssm_linattn_fwd(wide(1, 2, 1, 8), wide(1, 2, 1, 8), wide(1, 2, 1, FAR + 8), torch.zeros(1)),
    "linattn_bwd heads": lambda: ssm.ssm_linattn_bwd(wide(1, 2, 1, 8), wide(1, 2, 1, 8), wide(1, 2, FAR + 1, 8), torch.zeros(1),
                                                     torch.zeros(1), do=torch.zeros(1)),
    "linattn_step groups": lambda: ssm.ssm_linattn_step(torch.zeros(1), wide(1, 2, FAR + 1, 8), wide(1, 2, FAR + 1, 8), wide(1, 2, 1, 8),
                                                        torch.zeros(1)),
    "linattn_fwd_workspace": lambda: ssm.ssm_linattn_fwd_workspace(1, 64, FAR + 1, 1, 8, 8),
    "linattn_bwd_workspace": lambda: ssm.ssm_linattn_bwd_workspace(1, 64, 1, 1, FAR + 8, 8),
    "linattn_states_bytes": lambda: ssm.ssm_linattn_states_bytes(1, 64, 1, 8, FAR + 8),
}


@pytest.mark.parametrize("name", CALLS)
def test_refused(name):
    with pytest.raises(ValueError, match="32 bits"):
        CALLS[name]()
