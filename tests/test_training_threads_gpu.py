"""The training operators from two threads at once, on streams of their own: the bits of one
thread, and errors that stay in the thread that made them."""
import threading

import pytest
import torch

import selective_state_space_49_amd as ssm
from tests.gpu_util import bitwise_equal, say

pytestmark = pytest.mark.gpu


def inputs(seed):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
    return {"x": rnd(2, 300, 70).bfloat16(), "r": rnd(2, 300, 70).bfloat16(), "i": rnd(2, 300, 70).bfloat16(),
            "dy": rnd(2, 300, 70).bfloat16(), "decay": rnd(70), "hidden": rnd(90, 64), "weight": rnd(300, 64),
            "target": torch.randint(0, 300, (90,), generator=g).cuda(), "p": rnd(5000), "g": rnd(5000)}


def work(d):
    y, hf, st = ssm.ssm_gated_fwd_save(d["x"], d["r"], d["i"], d["decay"])
    grads = ssm.ssm_gated_bwd(d["x"], d["r"], d["i"], d["decay"], st, dy=d["dy"], want_dh0=False)
    loss, lse, mean = ssm.ssm_xent_fwd(d["hidden"], d["weight"], d["target"])
    dh, dw = ssm.ssm_xent_bwd(d["hidden"], d["weight"], d["target"], lse, mean, dmean=mean[:1])
    p, m, v = d["p"].clone(), torch.zeros(5120, device="cuda"), torch.zeros(5120, device="cuda")
    ssm.ssm_adamw_step([p], [d["g"]], m, v, lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, step=1)
    return [y, hf, grads["dx"], grads["ddecay"], loss, lse, mean, dh, dw, p, m, v]


def test_two_threads():
    say("two threads")
    sets = [inputs(1), inputs(2)]
    want = [work(d) for d in sets]
    torch.cuda.synchronize()
    failures = []

    def run(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got = work(sets[k])
                    with pytest.raises(ssm.SsmError, match="c must be" if k else "step"):
                        if k:
                            ssm.ssm_gated_fwd(sets[k]["x"], sets[k]["r"], sets[k]["i"], sets[k]["decay"], c=-1.0)
                        else:
                            ssm.ssm_adamw_step([got[9]], [sets[k]["g"]], got[10], got[11], lr=1e-2, beta1=0.9, beta2=0.99,
                                               eps=1e-8, weight_decay=0.1, step=0)
                    stream.synchronize()
                    assert all(bitwise_equal(a, b) for a, b in zip(got, want[k])), k
        except BaseException as e:  # noqa: BLE001
            failures.append(e)
    threads = [threading.Thread(target=run, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures
