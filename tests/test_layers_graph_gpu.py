"""The layer operators in captured graphs, on other streams, from two threads and under autograd."""
import threading

import pytest
import torch

import selective_state_space_49_amd as ssm
from tests import layers_ref as ref
from tests.gpu_util import bitwise_equal, say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def linattn_inputs(seed, io, L=700, H=3, V=40):
    """Long enough for several segments and their workspace."""
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    d = {"q": rn(1, L, 1, 24).to(io), "k": rn(1, L, 1, 24).to(io), "v": rn(1, L, H, V).to(io), "g": -torch.rand((1, L, H), generator=g),
         "h0": rn(1, H, 24, V), "do": rn(1, L, H, V).to(io), "dh": rn(1, H, 24, V)}
    d["g"][:, ::97] = -torch.inf
    return d


def linattn(d, ws=(None, None)):
    o, h, states = ssm.ssm_linattn_fwd_save(d["q"], d["k"], d["v"], d["g"], d["h0"], workspace=ws[0])
    g = ssm.ssm_linattn_bwd(d["q"], d["k"], d["v"], d["g"], states, do=d["do"], dh_final=d["dh"], workspace=ws[1])
    return [o, h, states, *g.values()]


def head_decay_inputs(seed, io):
    return linattn_inputs(seed, io) | {"g": -torch.rand(3, generator=torch.Generator().manual_seed(seed))}


def step_inputs(seed, io):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return {"h": rn(2, 3, 4, 24, 40), "q": rn(2, 3, 2, 24).to(io), "k": rn(2, 3, 2, 24).to(io), "v": rn(2, 3, 4, 40).to(io),
            "g": -torch.rand((2, 3, 4), generator=g)}


def step(d):
    h = d["h"].clone()
    return [ssm.ssm_linattn_step(h, d["q"], d["k"], d["v"], d["g"]), h]


def norm_inputs(seed, io):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return {k: rn(70, 333).to(io) for k in ("x", "r", "dy", "ds")} | {"w": rn(333)}


def norm(d, ws=None):
    y, s, rstd = ssm.ssm_rmsnorm_fwd(d["x"], d["w"], d["r"])
    out = [y, s, rstd, *ssm.ssm_rmsnorm_bwd(d["dy"], s, d["w"], rstd, ds=d["ds"], workspace=ws)]
    for code in ("e4m3", "int8"):
        codes, scales, _ = ssm.ssm_rmsnorm_fwd_q8(d["x"], d["w"], code=code, group=64)
        out += [scales, ssm.ssm_q8_values(codes, scales, group=64)]
    return out


def sample_inputs(seed, io):
    g = torch.Generator().manual_seed(seed)
    return {"logits": (3 * torch.randn(9, 5003, generator=g)).to(io), "u": torch.rand(9, generator=g),
            "t": torch.rand(9, generator=g), "k": torch.randint(0, 900, (9,), generator=g, dtype=torch.int32)}


def sample(d, ws=None):
    t, p = ssm.ssm_sample(d["logits"], d["u"], temperature=d["t"], top_k=d["k"], top_p=0.9, min_p=0.001, want_logprob=True,
                          workspace=ws)
    return [t.to(torch.int32), p]


ALL = [(linattn_inputs, linattn), (head_decay_inputs, linattn), (step_inputs, step), (norm_inputs, norm), (sample_inputs, sample)]


def held_and_captured(make, run, io, **kw):
    held = {k: t.cuda() for k, t in make(0, io).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(held, **kw)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run(held, **kw)
    return held, graph, outs


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("make,run", ALL)
def test_replays(make, run, io):
    say("graph", make.__name__, io)
    held, graph, outs = held_and_captured(make, run, io)
    for seed in (1, 2, 3):
        new = {k: t.cuda() for k, t in make(seed, io).items()}
        for k, t in held.items():
            t.copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        want = run(new)
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(outs, want)):
            assert bitwise_equal(a, b), (seed, k)


def workspaces(make, run, io):
    d = make(0, io)
    space = lambda n: torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")  # noqa: E731
    if run is linattn:
        b, L, Hk, K = d["q"].shape
        H, V = d["v"].shape[2:]
        kind = ssm.SSM_BF16 if io is BF16 else ssm.SSM_F32
        return (space(ssm.ssm_linattn_fwd_workspace(b, L, H, Hk, K, V, kind)),
                space(ssm.ssm_linattn_bwd_workspace(b, L, H, Hk, K, V, d["g"].dim() == 3, kind)))
    return space(ssm.ssm_rmsnorm_bwd_workspace(70, 333) if run is norm else ssm.ssm_sample_workspace(9, 5003))


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("make,run", [ALL[0], ALL[1], ALL[3], ALL[4]])
def test_two_graphs_and_a_workspace(make, run, io):
    """Two graphs and eager calls that share a workspace, one after the other: nothing stays in it
    that a later call goes by, whatever it holds."""
    say("shared workspace", make.__name__, io)
    ws = workspaces(make, run, io)
    every = ws if isinstance(ws, tuple) else (ws,)
    graphs = [held_and_captured(make, run, io, ws=ws) for _ in range(2)]
    sets = [{k: t.cuda() for k, t in make(seed, io).items()} for seed in (1, 2)]
    wants = [run(d) for d in sets]
    for (held, _, _), d in zip(graphs, sets):
        for k, t in held.items():
            t.copy_(d[k])
    for turn in range(3):
        for w in every:
            w.fill_(255)  # NaN in any type
        for which in (0, 1, 1, 0):
            graphs[which][1].replay()
            torch.cuda.synchronize()
            assert all(bitwise_equal(a, b) for a, b in zip(graphs[which][2], wants[which])), (turn, which)
            eager = run(sets[1 - which], ws=ws)
            torch.cuda.synchronize()
            assert all(bitwise_equal(a, b) for a, b in zip(eager, wants[1 - which])), (turn, which)


def test_a_workspace_too_small_or_misplaced():
    for make, run in (ALL[0], ALL[3], ALL[4]):
        ws = workspaces(make, run, F32)
        d = {k: t.cuda() for k, t in make(0, F32).items()}
        pairs = ([(ws[0][:-1], ws[1]), (ws[0], ws[1][:-1]), (torch.empty_like(ws[0], device="cpu"), ws[1])] if run is linattn
                 else [ws[:-1], torch.empty_like(ws, device="cpu")])
        for bad in pairs:
            if run is sample and (not ws.numel() > 256):
                continue
            say("bad workspace", run.__name__)
            with pytest.raises((ssm.SsmError, TypeError, ValueError)):
                run(d, ws=bad)


def test_two_threads():
    say("two threads")
    sets = [[{k: t.cuda() for k, t in make(seed, BF16).items()} for make, _ in ALL] for seed in (1, 2)]
    work = lambda ds: [t for d, (_, run) in zip(ds, ALL) for t in run(d)]  # noqa: E731
    want = [work(ds) for ds in sets]
    torch.cuda.synchronize()
    failures = []

    def go(n):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got = work(sets[n])
                    with pytest.raises(ssm.SsmError, match="eps" if n else "scale"):
                        d = sets[n][3 if n else 0]
                        if n:
                            ssm.ssm_rmsnorm_fwd(d["x"], d["w"], eps=-1.0)
                        else:
                            ssm.ssm_linattn_fwd(d["q"], d["k"], d["v"], d["g"], scale=float("nan"))
                    stream.synchronize()
                    assert all(bitwise_equal(a, b) for a, b in zip(got, want[n])), n
        except BaseException as e:  # noqa: BLE001
            failures.append(e)
    threads = [threading.Thread(target=go, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures


def test_another_stream_waits_for_its_work():
    """A call runs on torch's current stream, behind what was put there before."""
    d = {k: t.cuda() for k, t in linattn_inputs(3, BF16).items()}
    want = linattn(d)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    a = torch.randn(4096, 4096, device="cuda")
    say("another stream")
    with torch.cuda.stream(stream):
        late = torch.zeros_like(d["v"])
        for _ in range(10):
            a = a @ a * 1e-2
        late.copy_(d["v"])
        got = linattn(d | {"v": late})
    torch.cuda.current_stream().wait_stream(stream)
    assert all(bitwise_equal(x, y) for x, y in zip(got, want))


# ------------------------------------------------------------------ autograd
def leaves(d, *names):
    return {k: (t.detach().cuda().requires_grad_() if k in names else t.cuda()) for k, t in d.items()}


def training_step(dtype):
    d = leaves(linattn_inputs(0, dtype), "q", "k", "v", "g", "h0")
    w = torch.ones(40, device="cuda", requires_grad=True)
    names = [d[k] for k in ("q", "k", "v", "g", "h0")] + [w]

    def loss():
        o, h = ssm.linear_attention(d["q"], d["k"], d["v"], d["g"], d["h0"])
        return (ssm.rms_norm(o, w).float() * d["do"].float()).mean() + (h * d["dh"]).mean()
    return names, loss


def test_captured_backward():
    say("captured backward")
    names, loss = training_step(BF16)
    want = [t.clone() for t in torch.autograd.grad(loss(), names)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(loss(), names)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(loss(), names)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(bitwise_equal(a, b) for a, b in zip(got, want))
        (torch.ones(100, device="cuda") * 2).sum()
    late = torch.autograd.grad(loss(), names)
    assert all(bitwise_equal(a, b) for a, b in zip(late, want))


def test_leaves_of_another_stream_are_told():
    """Without a capture: what the refusal below goes by."""
    from selective_state_space_49_amd import layers
    elsewhere = layers._table_module().leaves_elsewhere
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    x, w = torch.randn(3, 50, device="cuda", requires_grad=True), torch.ones(50, device="cuda", requires_grad=True)
    for keep in (True, False):
        first = ssm.rms_norm(x, w) if keep else None
        side.wait_stream(here)
        with torch.cuda.stream(side):
            y = ssm.rms_norm(x, w)
        assert elsewhere(y.grad_fn.next_functions, side.stream_id) is keep
        assert elsewhere(y.grad_fn.next_functions, here.stream_id) is not keep
        torch.cuda.synchronize()
        del y, first


def test_captured_backward_beside_an_eager_graph_is_refused():
    say("captured backward beside an eager graph: refused")
    names, loss = training_step(F32)
    want = [t.clone() for t in torch.autograd.grad(loss(), names)]
    eager = loss()
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="cannot be captured"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            torch.autograd.grad(loss(), names)
    torch.cuda.synchronize()
    assert all(bitwise_equal(a, b) for a, b in zip(torch.autograd.grad(eager, names), want))


def test_some_gradients_only():
    say("some gradients")
    inputs = linattn_inputs(4, F32)
    full = leaves(inputs, "q", "k", "v", "g", "h0")

    def grads(d):
        o, h = ssm.linear_attention(d["q"], d["k"], d["v"], d["g"], d["h0"])
        ((o * d["do"]).sum() + (h * d["dh"]).sum()).backward()
        return {k: t.grad for k, t in d.items() if t.grad is not None}
    want = grads(full)
    for k in ("q", "k", "v", "g", "h0"):
        got = grads(leaves(inputs, k))
        assert list(got) == [k] and bitwise_equal(got[k], want[k])
    # an output alone
    for which in (0, 1):
        d = leaves(inputs, "q", "k", "v", "g", "h0")
        out = ssm.linear_attention(d["q"], d["k"], d["v"], d["g"], d["h0"])[which]
        (out * d["do" if which == 0 else "dh"]).sum().backward()
        r = ref.linattn(*(inputs[k] for k in ("q", "k", "v", "g", "h0")), None, inputs["do"] * (which == 0),
                        inputs["dh"] * which)
        for k in ("k", "v", "g"):
            want_k = r["d" + k]
            assert float((d[k].grad.double().cpu() - want_k).abs().max()) <= 1.8e-5 * float(want_k.abs().max())
        # the state does not depend on q
        assert which == 0 or not d["q"].grad.any()
    # broadcast leaves: the gradient is summed over what was shared
    v = torch.randn(1, 700, 1, 40, device="cuda", requires_grad=True)
    d = leaves(inputs, "q")
    (ssm.linear_attention(d["q"], d["k"], v.expand(1, 700, 3, 40).contiguous(), d["g"], d["h0"])[0] * d["do"]).sum().backward()
    e = v.detach().expand(1, 700, 3, 40).contiguous().requires_grad_()
    (ssm.linear_attention(d["q"], d["k"], e, d["g"], d["h0"])[0] * d["do"]).sum().backward()
    assert bitwise_equal(v.grad, e.grad.sum(2, keepdim=True))


def test_no_second_derivative():
    say("second derivative")
    d = leaves(linattn_inputs(0, F32), "q", "v")
    o, _ = ssm.linear_attention(d["q"], d["k"], d["v"], d["g"])
    grad, = torch.autograd.grad((o * o).sum(), d["q"], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.sum().backward()
    x, w = torch.randn(3, 50, device="cuda", requires_grad=True), torch.ones(50, device="cuda", requires_grad=True)
    grad, = torch.autograd.grad((ssm.rms_norm(x, w) ** 2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.sum().backward()


def test_outputs_tell_that_they_were_written():
    say("versions")
    d = {k: t.cuda() for k, t in step_inputs(0, F32).items()}
    o = torch.empty_like(d["v"])
    before = d["h"]._version, o._version, d["q"]._version
    ssm.ssm_linattn_step(d["h"], d["q"], d["k"], d["v"], d["g"], o_t=o)
    assert d["h"]._version > before[0] and o._version > before[1] and d["q"]._version == before[2]
    # a step in place on a state that a backward saved is refused there
    p = torch.randn_like(d["h"], requires_grad=True)
    loss = (p * d["h"]).sum()
    ssm.ssm_linattn_step(d["h"], d["q"], d["k"], d["v"], d["g"])
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        loss.backward()
    n = {k: t.cuda() for k, t in norm_inputs(0, F32).items()}
    y, rstd = torch.empty_like(n["x"]), torch.empty(70, device="cuda")
    before = y._version, n["r"]._version, rstd._version
    ssm.ssm_rmsnorm_fwd(n["x"], n["w"], n["r"], y=y, residual_out=n["r"], rstd=rstd)
    assert y._version > before[0] and n["r"]._version > before[1] and rstd._version > before[2]
    s = {k: t.cuda() for k, t in sample_inputs(0, F32).items()}
    tokens, logprob = torch.empty(9, dtype=torch.int64, device="cuda"), torch.empty(9, device="cuda")
    for ws in (None, workspaces(sample_inputs, sample, F32)):
        before = tokens._version, logprob._version
        ssm.ssm_sample(s["logits"], s["u"], tokens=tokens, logprob=logprob, workspace=ws)
        assert tokens._version > before[0] and logprob._version > before[1]
    codes, scales, _ = ssm.ssm_rmsnorm_fwd_q8(n["x"], n["w"])
    out = torch.empty_like(n["x"])
    before = out._version, codes._version
    ssm.ssm_rmsnorm_fwd_q8(n["x"], n["w"], codes=codes, scales=scales)
    ssm.ssm_q8_values(codes, scales, out=out)
    assert out._version > before[0] and codes._version > before[1]


def test_inference_tensors():
    with torch.inference_mode():
        d = {k: t.cuda() for k, t in step_inputs(0, F32).items()}
        ssm.ssm_linattn_step(d["h"], d["q"], d["k"], d["v"], d["g"])
        n = {k: t.cuda() for k, t in norm_inputs(0, BF16).items()}
        ssm.rms_norm(n["x"], n["w"], n["r"])
        ssm.ssm_rmsnorm_fwd(n["x"], n["w"], n["r"], residual_out=n["r"])
        linattn({k: t.cuda() for k, t in linattn_inputs(0, BF16).items()})
        sample({k: t.cuda() for k, t in sample_inputs(0, BF16).items()})
    torch.cuda.synchronize()


def test_refusals():
    """Strides, shapes and types that the kernels do not read are errors, and leave the outputs as they were."""
    d = {k: t.cuda() for k, t in linattn_inputs(0, F32).items()}
    o = torch.full_like(d["v"], 7.0)
    args = lambda **c: [(d | c)[k] for k in ("q", "k", "v", "g", "h0")]  # noqa: E731
    strided = torch.empty(1, 3, 700, 40, device="cuda").transpose(1, 2)
    for bad in ({"v": strided}, {"q": d["q"].bfloat16()}, {"k": d["k"][:, :-1]}, {"g": d["g"].double()}, {"h0": d["h0"][..., :-1]},
                {"g": d["g"][0]}, {"h0": d["h0"].cpu()}, {"v": d["v"].expand(2, -1, -1, -1)}):
        with pytest.raises((TypeError, ValueError)):
            ssm.ssm_linattn_fwd(*args(**bad), o=o)
    with pytest.raises((TypeError, ValueError)):
        ssm.ssm_linattn_fwd(*args(), o=o.bfloat16())
    with pytest.raises(ssm.SsmError, match="overlap"):
        ssm.ssm_linattn_fwd(*args(v=o), o=o)
    ws = torch.empty(ssm.ssm_linattn_fwd_workspace(1, 700, 3, 1, 24, 40, ssm.SSM_F32) + 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(ssm.SsmError, match="256"):
        ssm.ssm_linattn_fwd(*args(), o=o, workspace=ws[16:])
    n = {k: t.cuda() for k, t in norm_inputs(0, F32).items()}
    y = torch.full_like(n["x"], 7.0)
    for bad in ((n["x"].t(), n["w"]), (n["x"], n["w"][1:]), (n["x"], n["w"].bfloat16()), (n["x"], n["w"], n["r"][1:]),
                (n["x"], n["w"], n["r"].bfloat16())):
        with pytest.raises((TypeError, ValueError)):
            ssm.ssm_rmsnorm_fwd(*bad, y=y)
    with pytest.raises(ssm.SsmError, match="overlap"):
        ssm.ssm_rmsnorm_fwd(y, n["w"], y=y)
    with pytest.raises(ssm.SsmError, match="group"):
        ssm.ssm_rmsnorm_fwd_q8(n["x"], n["w"], group=16)
    s = {k: t.cuda() for k, t in sample_inputs(0, F32).items()}
    tokens = torch.full((9,), 7, device="cuda")
    for bad in ({"top_k": s["k"].long()}, {"temperature": s["t"].double()}, {"top_p": s["t"][1:]}, {"min_p": s["t"].cpu()}):
        with pytest.raises((TypeError, ValueError)):
            ssm.ssm_sample(s["logits"], s["u"], tokens=tokens, **bad)
    with pytest.raises((TypeError, ValueError)):
        ssm.ssm_sample(s["logits"].t(), s["u"], tokens=tokens)
    with pytest.raises(ssm.SsmError, match="temperature"):
        ssm.ssm_sample(s["logits"], s["u"], temperature=-1.0, tokens=tokens)
    torch.cuda.synchronize()
    assert bool((o == 7).all()) and bool((y == 7).all()) and bool((tokens == 7).all())
