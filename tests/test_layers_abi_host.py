"""Refusals of the layer operators: every bad argument gives its status on the host, before
anything is enqueued (no GPU is touched; the addresses are never used)."""
import ctypes

import pytest
import torch

import selective_state_space_49_amd as ssm

OK, NULL, SHAPE, DTYPE, ALIGN, UNSUP, WS = 0, 1, 2, 3, 4, 5, 6
p = lambda v: None if v is None else ctypes.c_void_p(v)  # noqa: E731
MB = 1 << 20
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return ssm.load_library()


SHAPES = [{"b": -1}, {"L": -1}, {"H": 0}, {"Hk": 0}, {"H": 3, "Hk": 2}, {"Hk": 8}, {"K": 0}, {"K": 129}, {"V": 0}, {"V": 129},
          {"b": 1 << 19}, {"L": 1 << 40}]


def test_linattn_forward(lib):
    def call(q=MB, k=2 * MB, v=3 * MB, g=4 * MB, per=1, h0=None, scale=1.0, o=5 * MB, hf=None, st=None, b=2, L=100, H=4, Hk=2, K=16,
             V=32, io=0, ws=64 * MB, wsb=MB):
        return lib.ssm_linattn_fwd(p(q), p(k), p(v), p(g), per, p(h0), scale, p(o), p(hf), p(st), b, L, H, Hk, K, V, io, p(ws), wsb, None)
    assert call(io=2) == DTYPE
    for bad in SHAPES:
        assert call(**bad) == SHAPE, bad
    assert call(scale=NAN) == UNSUP and call(scale=INF) == UNSUP
    for k in ("q", "k", "v", "g", "o"):
        assert call(**{k: None}) == NULL, k
    assert call(q=MB + 2) == ALIGN and call(io=1, v=3 * MB + 1) == ALIGN and call(h0=6 * MB + 2) == ALIGN and call(g=4 * MB + 2) == ALIGN
    # o is 2 x 100 x 4 x 32 floats, 102400 bytes; h_final 2 x 4 x 16 x 32, 16384
    assert call(o=3 * MB + 102000) == UNSUP and "overlap" in ssm.ssm_last_error()
    assert call(hf=5 * MB + 102000) == UNSUP and call(st=4 * MB) == UNSUP and call(h0=6 * MB, hf=6 * MB) == UNSUP
    need = ssm.ssm_linattn_fwd_workspace(2, 4000, 4, 2, 16, 32, 0)
    assert need > 0
    far = {"v": 32 * MB, "o": 48 * MB, "L": 4000, "k": 8 * MB, "g": 16 * MB}
    assert call(**far, ws=None) == WS and call(**far, wsb=need - 1) == WS and call(**far, ws=64 * MB + 16) == ALIGN
    assert call(b=0) == OK
    assert ssm.ssm_linattn_states_bytes(2, 65, 4, 16, 32, 1) == 2 * 4 * 2 * 16 * 32 * 4
    assert ssm.ssm_linattn_states_bytes(2, 65, 4, 16, 32, 0) == 2 * 4 * 3 * 16 * 32 * 4
    assert ssm.ssm_linattn_states_bytes(2, 65, 4, 16, 129, 0) == 0 and ssm.ssm_linattn_fwd_workspace(2, 65, 4, 3, 16, 16) == 0


def test_linattn_backward(lib):
    def call(q=MB, k=2 * MB, v=3 * MB, g=4 * MB, per=1, st=5 * MB, do=6 * MB, dhf=None, scale=1.0, dq=7 * MB, dk=8 * MB, dv=9 * MB,
             dg=10 * MB, dh0=None, b=2, L=100, H=4, Hk=2, K=16, V=32, io=0, ws=64 * MB, wsb=MB):
        return lib.ssm_linattn_bwd(p(q), p(k), p(v), p(g), per, p(st), p(do), p(dhf), scale, p(dq), p(dk), p(dv), p(dg), p(dh0), b, L,
                                   H, Hk, K, V, io, p(ws), wsb, None)
    assert call(io=-1) == DTYPE and call(scale=-INF) == UNSUP
    for bad in SHAPES:
        assert call(**bad) == SHAPE, bad
    for k in ("q", "k", "v", "g", "st", "do", "dq", "dk", "dv", "dg"):
        assert call(**{k: None}) == NULL, k
    assert call(b=0, per=0, dg=None) == NULL  # the sum over no tokens is written
    for k, at in (("dq", 7 * MB), ("st", 5 * MB), ("dg", 10 * MB), ("do", 6 * MB), ("dh0", 11 * MB)):
        assert call(**{k: at + 2}) == ALIGN, k
    assert call(dq=8 * MB) == UNSUP and call(dv=6 * MB) == UNSUP and call(dg=4 * MB) == UNSUP and call(dhf=12 * MB, dh0=12 * MB) == UNSUP
    # heads that share: dq and dk by head in float32, 2 x 2 x 100 x 4 x 16 x 4 bytes
    need = ssm.ssm_linattn_bwd_workspace(2, 100, 4, 2, 16, 32, True, 0)
    assert need >= 2 * 2 * 100 * 4 * 16 * 4
    assert call(ws=None) == WS and call(wsb=need - 1) == WS and call(ws=64 * MB + 128) == ALIGN
    assert ssm.ssm_linattn_bwd_workspace(2, 100, 4, 2, 16, 32, False, 0) > need


def test_linattn_step(lib):
    def call(h=MB, q=32 * MB, k=33 * MB, v=34 * MB, g=35 * MB, per=1, scale=1.0, o=36 * MB, Ln=2, S=3, H=4, Hk=2, K=16, V=32, io=1):
        return lib.ssm_linattn_step(p(h), p(q), p(k), p(v), p(g), per, scale, p(o), Ln, S, H, Hk, K, V, io, None)
    assert call(io=3) == DTYPE and call(Ln=-1) == SHAPE and call(S=-1) == SHAPE and call(Ln=1 << 21) == SHAPE
    assert call(S=1 << 19) == SHAPE and call(H=3) == SHAPE and call(K=200) == SHAPE and call(scale=NAN) == UNSUP
    for k in ("h", "q", "k", "v", "g", "o"):
        assert call(**{k: None}) == NULL, k
    assert call(h=MB + 2) == ALIGN and call(o=36 * MB + 1) == ALIGN
    assert call(o=34 * MB) == UNSUP and call(h=32 * MB) == UNSUP and call(Ln=0) == OK and call(S=0) == OK


def test_norm(lib):
    def call(x=MB, r=None, w=2 * MB, eps=1e-6, y=3 * MB, s=None, rstd=None, rows=10, dim=100, io=1, rio=1):
        return lib.ssm_rmsnorm_fwd(p(x), p(r), p(w), eps, p(y), p(s), p(rstd), rows, dim, io, rio, None)
    assert call(io=2) == DTYPE and call(rio=7) == DTYPE and call(io=0, rio=1) == DTYPE
    for bad in ({"rows": -1}, {"rows": 1 << 31}, {"dim": 0}, {"dim": 65537}):
        assert call(**bad) == SHAPE, bad
    for eps in (-1e-9, NAN, INF):
        assert call(eps=eps) == UNSUP
    for k in ("x", "w", "y"):
        assert call(**{k: None}) == NULL, k
    assert call(r=4 * MB) == NULL and call(s=4 * MB) == NULL
    assert call(x=MB + 1) == ALIGN and call(w=2 * MB + 2) == ALIGN and call(r=4 * MB + 2, s=5 * MB, rio=0) == ALIGN
    assert call(y=MB + 1998) == UNSUP and call(y=MB) == UNSUP and call(r=4 * MB, s=4 * MB + 2) == UNSUP and call(rstd=2 * MB) == UNSUP
    assert call(rows=0, x=None, y=None) == OK


def test_norm_codes(lib):
    def call(x=MB, r=None, w=2 * MB, eps=1e-6, c=3 * MB, sc=4 * MB, code=1, group=128, s=None, rows=10, dim=300, io=1, rio=1):
        return lib.ssm_rmsnorm_fwd_q8(p(x), p(r), p(w), eps, p(c), p(sc), code, group, p(s), rows, dim, io, rio, None)
    assert call(code=0) == DTYPE and call(code=3) == DTYPE and call(io=9) == DTYPE
    for group in (-1, 1, 8, 16, 100, 256):
        assert call(group=group) == UNSUP, group
    assert call(sc=None) == NULL and call(c=None) == NULL and call(sc=4 * MB + 2) == ALIGN
    assert call(sc=3 * MB + 2996) == UNSUP and call(c=MB) == UNSUP and call(rows=0) == OK

    def values(c=MB, sc=2 * MB, code=2, group=0, out=3 * MB, rows=10, dim=300):
        return lib.ssm_q8_values(p(c), p(sc), code, group, p(out), rows, dim, None)
    assert values(code=0) == DTYPE and values(group=5) == UNSUP and values(dim=0) == SHAPE and values(rows=-1) == SHAPE
    assert values(c=None) == NULL and values(out=None) == NULL and values(out=3 * MB + 1) == ALIGN and values(out=MB + 2000) == UNSUP
    assert values(rows=0) == OK


def test_norm_backward(lib):
    def call(dy=MB, s=2 * MB, ds=None, w=3 * MB, rstd=4 * MB, dx=5 * MB, dr=None, dw=6 * MB, rows=10, dim=100, io=1, rio=0, ws=8 * MB,
             wsb=MB):
        return lib.ssm_rmsnorm_bwd(p(dy), p(s), p(ds), p(w), p(rstd), p(dx), p(dr), p(dw), rows, dim, io, rio, p(ws), wsb, None)
    assert call(io=4) == DTYPE and call(io=0, rio=1) == DTYPE and call(dim=0) == SHAPE and call(rows=-1) == SHAPE
    for k in ("dy", "s", "w", "rstd", "dx", "dw"):
        assert call(**{k: None}) == NULL, k
    assert call(s=2 * MB + 2) == ALIGN and call(dw=6 * MB + 1) == ALIGN
    assert call(dx=MB) == UNSUP and call(dr=2 * MB) == UNSUP and call(dw=3 * MB) == UNSUP and call(ds=7 * MB, dr=7 * MB) == UNSUP
    need = ssm.ssm_rmsnorm_bwd_workspace(10, 100)
    assert need > 0 and call(ws=None) == WS and call(wsb=need - 1) == WS and call(ws=8 * MB + 64) == ALIGN


def test_sample(lib):
    def call(x=MB, u=2 * MB, t=None, t1=1.0, k=None, k1=0, pp=None, p1=1.0, m=None, m1=0.0, tok=3 * MB, lp=None, rows=4, V=1000, io=0):
        return lib.ssm_sample(p(x), p(u), p(t), t1, p(k), k1, p(pp), p1, p(m), m1, p(tok), p(lp), rows, V, io, p(8 * MB), MB, None)
    assert call(io=2) == DTYPE and call(rows=-1) == SHAPE and call(rows=65536) == SHAPE and call(V=0) == SHAPE and call(V=(1 << 24) + 1) == SHAPE
    assert call(t1=-0.1) == UNSUP and call(t1=NAN) == UNSUP
    for k in ("x", "u", "tok"):
        assert call(**{k: None}) == NULL, k
    assert call(x=MB + 2) == ALIGN and call(tok=3 * MB + 4) == ALIGN and call(lp=4 * MB + 2) == ALIGN and call(k=5 * MB + 1) == ALIGN
    assert call(tok=MB + 8) == UNSUP and call(lp=2 * MB) == UNSUP and call(lp=3 * MB) == UNSUP and call(t=4 * MB, lp=4 * MB) == UNSUP
    assert call(rows=0) == OK


def test_binding_refuses():
    """What the binding says itself: tensors that are not on a GPU, wrong ranks, names and types."""
    z = torch.zeros
    with pytest.raises(ValueError, match="GPU"):
        ssm.ssm_linattn_fwd(z(1, 2, 2, 4), z(1, 2, 2, 4), z(1, 2, 2, 4), z(2))
    with pytest.raises(ValueError, match="batch, L"):
        ssm.ssm_linattn_fwd(z(2, 2, 4), z(2, 2, 4), z(2, 2, 4), z(2))
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ssm.ssm_sample(z(2, 4, dtype=torch.float16), z(2))
    with pytest.raises(TypeError, match="residual"):
        ssm.ssm_rmsnorm_fwd(z(2, 4), z(4), z(2, 4, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="e4m3"):
        ssm.ssm_rmsnorm_fwd_q8(z(2, 4), z(4), code="e5m2")
    with pytest.raises(ValueError, match="residual"):
        ssm.ssm_rmsnorm_fwd(z(2, 4), z(4), residual_out=z(2, 4))
    with pytest.raises(TypeError, match="codes"):
        ssm.ssm_q8_values(z(2, 4), z(2, 1))
