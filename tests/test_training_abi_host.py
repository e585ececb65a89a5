"""Refusals of the training operators: every bad argument gives its status on the host,
before anything is enqueued (no GPU is touched; the addresses are never used)."""
import ctypes

import pytest
import torch

import selective_state_space_49_amd as ssm

OK, NULL, SHAPE, DTYPE, ALIGN, UNSUP, WS = 0, 1, 2, 3, 4, 5, 6
p = lambda v: None if v is None else ctypes.c_void_p(v)  # noqa: E731
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return ssm.load_library()


def test_gated_forward(lib):
    def call(x=MB, r=2 * MB, i=3 * MB, decay=4 * MB, h0=None, reset=None, c=8.0, y=5 * MB, hf=None, st=None, b=2,
             L=100, D=30, io=0, ws=64 * MB, wsb=MB):
        return lib.ssm_gated_fwd(p(x), p(r), p(i), p(decay), p(h0), p(reset), c, p(y), p(hf), p(st), b, L, D, io,
                                 p(ws), wsb, None)
    assert call(io=2) == DTYPE and call(b=-1) == SHAPE and call(b=65536) == SHAPE and call(L=-1) == SHAPE
    assert call(D=0) == SHAPE and call(D=1 << 29) == SHAPE
    for c in (0.0, -1.0, float("inf"), float("nan")):
        assert call(c=c) == UNSUP
    for k in ("x", "r", "i", "decay", "y"):
        assert call(**{k: None}) == NULL, k
    assert call(x=MB + 2) == ALIGN and call(io=1, x=MB + 1) == ALIGN and call(h0=6 * MB + 2) == ALIGN
    # 2 * 100 * 30 floats are 24000 bytes
    assert call(y=MB + 16000) == UNSUP and "overlap" in ssm.ssm_last_error()
    assert call(hf=5 * MB) == UNSUP and call(st=4 * MB) == UNSUP
    need = ssm.ssm_gated_fwd_workspace(2, 1000, 30)
    if need:
        assert call(L=1000, ws=None) == WS and call(L=1000, wsb=need - 1) == WS and call(L=1000, ws=MB * 64 + 16) == ALIGN
    assert call(b=0) == OK
    assert ssm.ssm_gated_states_bytes(2, 65, 30) == 2 * 2 * 30 * 4 and ssm.ssm_gated_states_bytes(2, 0, 30) == 0
    assert ssm.ssm_gated_states_bytes(-1, 65, 30) == 0


def test_gated_backward(lib):
    def call(x=MB, r=2 * MB, i=3 * MB, decay=4 * MB, st=5 * MB, reset=None, c=8.0, dy=6 * MB, dhf=None, dx=7 * MB,
             dr=8 * MB, di=9 * MB, dd=10 * MB, dh0=None, b=2, L=100, D=30, io=0, ws=64 * MB, wsb=MB):
        return lib.ssm_gated_bwd(p(x), p(r), p(i), p(decay), p(st), p(reset), c, p(dy), p(dhf), p(dx), p(dr), p(di),
                                 p(dd), p(dh0), b, L, D, io, p(ws), wsb, None)
    assert call(io=3) == DTYPE and call(L=-1) == SHAPE and call(c=0.0) == UNSUP
    for k in ("x", "r", "i", "decay", "st", "dy", "dx", "dr", "di", "dd"):
        assert call(**{k: None}) == NULL, k
    assert call(dd=10 * MB + 2) == ALIGN and call(st=5 * MB + 1) == ALIGN
    assert call(dx=6 * MB) == UNSUP and call(dr=7 * MB) == UNSUP and call(dd=4 * MB) == UNSUP
    need = ssm.ssm_gated_bwd_workspace(2, 100, 30)
    assert need > 0 and call(ws=None) == WS and call(wsb=need - 1) == WS and call(ws=64 * MB + 128) == ALIGN


def test_gated_step(lib):
    def call(h=MB, x=2 * MB, r=3 * MB, i=4 * MB, decay=5 * MB, c=8.0, y=6 * MB, Ln=2, S=3, D=30, io=1):
        return lib.ssm_gated_step(p(h), p(x), p(r), p(i), p(decay), c, p(y), Ln, S, D, io, None)
    assert call(io=5) == DTYPE and call(Ln=-1) == SHAPE and call(Ln=65536) == SHAPE and call(S=65536) == SHAPE
    assert call(D=0) == SHAPE and call(c=-1.0) == UNSUP
    for k in ("h", "x", "r", "i", "decay", "y"):
        assert call(**{k: None}) == NULL, k
    assert call(h=MB + 2) == ALIGN and call(y=6 * MB + 1) == ALIGN and call(y=2 * MB + 100) == UNSUP
    assert call(Ln=0) == OK and call(S=0) == OK


def test_cross_entropy(lib):
    def fwd(h=MB, w=2 * MB, t=3 * MB, loss=4 * MB, lse=5 * MB, mean=6 * MB, T=20, K=30, V=40, io=0, ws=64 * MB, wsb=MB):
        return lib.ssm_xent_fwd(p(h), p(w), p(t), -100, p(loss), p(lse), p(mean), T, K, V, io, p(ws), wsb, None)
    assert fwd(io=2) == DTYPE and fwd(T=-1) == SHAPE and fwd(K=0) == SHAPE and fwd(V=0) == SHAPE
    assert fwd(V=(1 << 30) + 1) == SHAPE
    for k in ("h", "w", "t", "loss", "lse", "mean"):
        assert fwd(**{k: None}) == NULL, k
    assert fwd(t=3 * MB + 4) == ALIGN and fwd(h=MB + 2) == ALIGN and fwd(lse=5 * MB + 1) == ALIGN
    assert fwd(loss=MB) == UNSUP and fwd(lse=4 * MB) == UNSUP
    need = ssm.ssm_xent_fwd_workspace(20, 30, 40, 0)
    assert need > 0 and fwd(ws=None) == WS and fwd(wsb=need - 1) == WS and fwd(ws=64 * MB + 8) == ALIGN
    assert ssm.ssm_xent_fwd_workspace(20, 0, 40, 0) == 0 and ssm.ssm_xent_bwd_workspace(20, 30, 40, 7) == 0

    def bwd(h=MB, w=2 * MB, t=3 * MB, lse=5 * MB, mean=6 * MB, dl=None, dm=7 * MB, dh=8 * MB, dw=9 * MB, T=20, K=30,
            V=40, io=0, ws=64 * MB, wsb=64 * MB):
        return lib.ssm_xent_bwd(p(h), p(w), p(t), -100, p(lse), p(mean), p(dl), p(dm), p(dh), p(dw), T, K, V, io,
                                p(ws), wsb, None)
    assert bwd(io=2) == DTYPE and bwd(K=-1) == SHAPE
    for k in ("h", "w", "t", "lse", "mean"):
        assert bwd(**{k: None}) == NULL, k
    assert bwd(dm=7 * MB + 2) == ALIGN and bwd(dw=2 * MB) == UNSUP and bwd(dw=8 * MB + 4) == UNSUP
    need = ssm.ssm_xent_bwd_workspace(20, 30, 40, 0)
    assert need > 0 and bwd(ws=None) == WS and bwd(wsb=need - 1) == WS and bwd(ws=64 * MB + 8) == ALIGN
    assert bwd(dh=None, dw=None) == OK


def test_adamw(lib):
    def call(n=2, params=(MB, 2 * MB), grads=(3 * MB, 4 * MB), sizes=(100, 300), pio=(0, 1), gio=(0, 1), m=5 * MB,
             v=6 * MB, ms=None, vs=None, gs=None, lr=1e-3, b1=0.9, b2=0.95, eps=1e-8, wd=0.1, step=1):
        arr = lambda kind, a: None if a is None else (kind * len(a))(*a)  # noqa: E731
        return lib.ssm_adamw_step(n, arr(ctypes.c_void_p, params), arr(ctypes.c_void_p, grads),
                                  arr(ctypes.c_int64, sizes), arr(ctypes.c_int32, pio), arr(ctypes.c_int32, gio),
                                  p(m), p(v), p(ms), p(vs), p(gs), lr, b1, b2, eps, wd, step, None)
    assert call(n=-1) == SHAPE and call(sizes=(100, -1)) == SHAPE and call(pio=(0, 2)) == DTYPE
    assert call(params=None) == NULL and call(sizes=None) == NULL and call(params=(MB, None)) == NULL
    assert call(m=None) == NULL and call(v=None) == NULL and call(ms=7 * MB) == NULL
    assert call(b1=1.0) == UNSUP and call(b2=-0.1) == UNSUP and call(eps=-1.0) == UNSUP and call(step=0) == UNSUP
    assert call(lr=float("nan")) == UNSUP and call(wd=float("inf")) == UNSUP
    assert call(params=(MB + 2, 2 * MB)) == ALIGN and call(m=5 * MB + 8) == ALIGN and call(gs=8 * MB + 1) == ALIGN
    assert call(grads=(MB + 4, 4 * MB)) == UNSUP
    assert call(n=0) == OK and call(sizes=(0, 0)) == OK and call(grads=(None, None)) == OK
    assert ssm.ssm_adamw_state_size([1, 256, 257, 0]) == 256 + 256 + 512 and ssm.ssm_adamw_state_size([]) == 0
    assert ssm.ssm_adamw_state_size([-1]) == 0

    def values(m=MB, v=2 * MB, ms=3 * MB, vs=4 * MB, mo=5 * MB, vo=6 * MB, n=512):
        return lib.ssm_adamw_values(p(m), p(v), p(ms), p(vs), p(mo), p(vo), n, None)
    assert values(n=100) == SHAPE and values(n=-256) == SHAPE and values(mo=None) == NULL
    assert values(vo=6 * MB + 4) == ALIGN and values(vo=5 * MB) == UNSUP and values(n=0) == OK


def test_binding_refuses():
    cpu = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError):
        ssm.ssm_gated_fwd(cpu, cpu, cpu, torch.zeros(8))
    with pytest.raises(ValueError):
        ssm.ssm_xent_fwd(torch.zeros(4, 8), torch.zeros(10, 8), torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        ssm.ssm_adamw_step([torch.zeros(8)], [torch.zeros(8)], torch.zeros(256), torch.zeros(256), lr=1e-3, beta1=0.9,
                           beta2=0.95, eps=1e-8, weight_decay=0.0, step=1)
    with pytest.raises(ValueError):
        ssm.linear_cross_entropy(torch.zeros(4, 8), torch.zeros(10, 8), torch.zeros(4, dtype=torch.int64), reduction="sum")
    with pytest.raises(ValueError):
        ssm.AdamW([torch.zeros(8)], bits=16)
