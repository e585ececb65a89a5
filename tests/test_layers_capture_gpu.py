"""Which captured backward passes are refused: those whose gradients come to a function or a leaf that works on the
default stream, however far behind the operator it is; and no others."""
import pytest
import torch

import selective_state_space_49_amd as ssm
from selective_state_space_49_amd import layers
from tests.gpu_util import bitwise_equal, say

pytestmark = pytest.mark.gpu
BEHIND = {
    "cast": lambda w: w.bfloat16().float(),
    "view": lambda w: w.view(5, 10).view(50),
    "product": lambda w: w * 2,
    "matmul": lambda w: torch.eye(50, device="cuda") @ w,
    "norm": lambda w: ssm.rms_norm(w[None], torch.ones(50, device="cuda"))[0],
}


@pytest.mark.parametrize("name", BEHIND)
def test_leaves_behind_other_functions_are_told(name):
    """Without a capture: what the refusal goes by."""
    say("leaf behind", name)
    elsewhere = layers._table_module().leaves_elsewhere
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    x, w = torch.randn(3, 50, device="cuda"), torch.ones(50, device="cuda", requires_grad=True)
    for keep in (True, False):
        first = w * 1 if keep else None
        side.wait_stream(here)
        with torch.cuda.stream(side):
            y = ssm.rms_norm(x, BEHIND[name](w))
        assert elsewhere(y.grad_fn.next_functions, side.stream_id) is keep
        assert elsewhere(y.grad_fn.next_functions, here.stream_id) is True  # the functions between are the side's
        torch.cuda.synchronize()
        del y, first


def test_refused_behind_a_cast():
    say("captured backward, a leaf behind a cast: refused")
    x, w = torch.randn(3, 50, device="cuda"), torch.ones(50, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    eager = ssm.rms_norm(x, w.float())
    dy = torch.randn_like(x)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="cannot be captured"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            torch.autograd.grad(ssm.rms_norm(x, w.float()), w, dy)
    torch.cuda.synchronize()
    assert bool(torch.autograd.grad(eager, w, dy)[0].isfinite().all())


def test_a_stream_of_the_capture_is_not_refused():
    """A leaf's gradient from a stream that the capture has forked into: both streams belong to it."""
    say("captured backward over a forked stream")
    x, w = torch.randn(30, 50, device="cuda", requires_grad=True), torch.ones(50, device="cuda", requires_grad=True)
    dy = [torch.randn(30, 50, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()

    def grads():
        here = torch.cuda.current_stream()
        first = ssm.rms_norm(x, w)
        side.wait_stream(here)
        with torch.cuda.stream(side):
            second = ssm.rms_norm(x, w, eps=0.5)
        here.wait_stream(side)
        return torch.autograd.grad((first, second), (x, w), dy)
    want = [t.clone() for t in grads()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = grads()
    for _ in range(3):
        for t in got:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(bitwise_equal(a, b) for a, b in zip(got, want))
        (torch.ones(100, device="cuda") * 2).sum()


@pytest.mark.parametrize("accumulate", [False, True])
def test_leaves_of_a_side_stream_are_not_refused(accumulate):
    """An eager graph of the same leaves that was built on a stream of its own, as in a warm-up: that stream becomes
    a part of the capture."""
    say("captured backward beside an eager graph of a side stream", accumulate)
    x, w = torch.randn(30, 50, device="cuda", requires_grad=True), torch.ones(50, device="cuda", requires_grad=True)
    dy = torch.randn(30, 50, device="cuda")
    want = [t.clone() for t in torch.autograd.grad(ssm.rms_norm(x, w), (x, w), dy)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = ssm.rms_norm(x, w)
    torch.cuda.synchronize()
    got = [torch.empty_like(t) for t in want]
    if accumulate:
        x.grad, w.grad = got
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if accumulate:
            ssm.rms_norm(x, w).backward(dy)
        else:
            got = torch.autograd.grad(ssm.rms_norm(x, w), (x, w), dy)
    for _ in range(3):
        for t in got:
            t.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(bitwise_equal(a, b) for a, b in zip(got, want))
        (torch.ones(100, device="cuda") * 2).sum()
    assert all(bitwise_equal(a, b) for a, b in zip(torch.autograd.grad(eager, (x, w), dy), want))
