"""Every differentiable function looks, before its gradients are made, whether they can be captured."""
import pytest
import torch

import selective_state_space_49_amd as ssm
from selective_state_space_49_amd import layers, training

FUNCTIONS = [ssm._SelectiveScan, ssm._SelectiveScanFused, training._GatedScan, training._LinearCrossEntropy, layers._LinearAttention,
             layers._RmsNorm]


@pytest.mark.parametrize("function", FUNCTIONS, ids=lambda f: f.__name__)
def test_looked_at_first(function, monkeypatch):
    class Table:
        def leaves_elsewhere(self, edges, stream):
            return (edges, stream) == ("edges", 3)

    class Node:
        next_functions = "edges"

    class Stream:
        stream_id = 3
    monkeypatch.setattr(layers, "_table_module", Table)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    backward = getattr(function.backward, "__wrapped__", function.backward)
    with pytest.raises(RuntimeError, match="cannot be captured"):
        backward(Node, None, None)


def test_the_default_stream_joins_no_capture(monkeypatch):
    capturing = [True]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    assert training._joins(35) and not training._joins(0)
    capturing[0] = False
    assert not training._joins(35)
