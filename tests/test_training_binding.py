"""The training operators' binding, where it decides on the host (no GPU is touched)."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from selective_state_space_49_amd import training


def test_a_workspace_has_to_be_on_the_tensors_gpu():
    gpu = torch.device("cuda", 0)
    for bad in (torch.empty(512, dtype=torch.uint8), torch.empty(512, dtype=torch.uint8, device="meta"),
                torch.empty(512, 2, dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError, match="workspace"):
            training._scratch(bad, 256, gpu)
    cpu = torch.device("cpu")
    with pytest.raises(ValueError, match="workspace"):  # not contiguous
        training._scratch(torch.empty(512, 2, dtype=torch.uint8)[:, 0], 256, cpu)
    good = torch.empty(100, dtype=torch.float32)
    assert training._scratch(good, 256, cpu) == (good, good.data_ptr(), 400)
    assert training._scratch(None, 0, gpu) == (None, None, 0)


def on(index, **more):
    """What the binding asks a tensor of GPU `index`."""
    return SimpleNamespace(**{**dict(shape=(3,), dtype=torch.float32, is_cuda=True, device=torch.device("cuda", index),
                                     is_contiguous=lambda: True, data_ptr=lambda: 4096), **more})


def test_tensors_have_to_be_on_one_gpu():
    args = ("r", (3,), torch.float32, torch.device("cuda", 0))
    assert training._need(on(0), *args) == 4096 and training._need(None, *args) is None
    with pytest.raises(ValueError, match="cuda:0"):
        training._need(on(1), *args)
    with pytest.raises(ValueError, match="GPU"):
        training._need(torch.zeros(3), *args)


def test_the_tensors_gpu_is_current_during_a_call(monkeypatch):
    current = [torch.device("cuda", 0)]

    @contextlib.contextmanager
    def device(d):
        current.append(d)
        yield
        current.pop()
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(training, "_stream", lambda t: (current[-1], "stream"))
    seen = []

    def entry(*args):
        seen.append((current[-1], args))
        return 0
    training._called(on(1), entry, 7, 8)
    gpu = torch.device("cuda", 1)
    assert seen == [(gpu, (7, 8, (gpu, "stream")))] and current == [torch.device("cuda", 0)]
