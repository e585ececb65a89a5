"""The cross entropy in workspaces of exactly the size it asks for, and with a copy of weight that
goes in pieces. Tolerances as in the operator's own tests."""
import pytest
import torch

import selective_state_space_49_amd as ssm
from tests import train_ref
from tests.gpu_util import bitwise_equal, say
from tests.test_xent_gpu import call, check, make

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def exactly(n):
    """A workspace of n bytes, and what lies behind it."""
    buffer = torch.full((n + 4096,), 171, dtype=torch.uint8, device="cuda")
    return buffer[:n], buffer[n:]


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("T,K,V,shift", [(100, 256, 1000, 0), (100, 256, 1000, 1), (70, 65, 300, 0), (9, 128, 3001, 0),
                                         (3000, 64, 50, 0), (300, 136, 1111, 0)])
@pytest.mark.parametrize("each", [False, True])
def test_exact_size(T, K, V, shift, io, each):
    say("xent exact workspace", T, K, V, shift, io, each)
    hidden, weight, target = (t.cuda() for t in make(T, K, V, io, seed=T + V))
    if shift:
        flat = torch.empty(weight.numel() + 1, dtype=io, device="cuda")
        flat[1:] = weight.view(-1)
        weight = flat[1:].view(V, K)
    dloss = torch.rand(T, generator=torch.Generator().manual_seed(1)).cuda() if each else None
    dmean = torch.ones((), device="cuda")
    ws, behind = exactly(ssm.ssm_xent_fwd_workspace_for(hidden, weight))
    loss, lse, mean = ssm.ssm_xent_fwd(hidden, weight, target, workspace=ws)
    assert bool((behind == 171).all())
    ws, behind = exactly(ssm.ssm_xent_bwd_workspace_for(hidden, weight, dloss))
    dh, dw = ssm.ssm_xent_bwd(hidden, weight, target, lse, mean, dloss=dloss, dmean=dmean, workspace=ws)
    assert bool((behind == 171).all())
    want = call(hidden, weight, target, dloss, dmean)
    for k, t in {"loss": loss, "lse": lse, "mean": mean, "dhidden": dh, "dweight": dw}.items():
        assert bitwise_equal(t, want[k]), k


@pytest.mark.parametrize("T,K,V,io", [(90, 1000, 100001, F32), (20, 2000, 140001, BF16)])
def test_copies_in_pieces(T, K, V, io):
    say("xent copies in pieces", T, K, V, io)
    hidden, weight, target = make(T, K, V, io, seed=5)
    target[-3:] = torch.tensor([V - 1, V - 2, 87040])
    ref = train_ref.xent(hidden, weight, target, dmean=1.0)
    check(hidden, weight, target, ref, call(hidden, weight, target, None, torch.ones((), device="cuda")), io, 1)
