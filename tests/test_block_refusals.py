"""The block calls' checks: the C entry points refuse before any launch, the Python ones before the C call."""
import ctypes

import pytest
import torch

import sparse_moe_layer_amd as lib
from sparse_moe_layer_amd import _lib

OK, NULL, SHAPE, DTYPE, ALIGN, WS, UNSUP = (_lib.MOE_OK, _lib.MOE_ERR_NULL, _lib.MOE_ERR_SHAPE, _lib.MOE_ERR_DTYPE,
                                            _lib.MOE_ERR_ALIGN, _lib.MOE_ERR_WORKSPACE, _lib.MOE_ERR_UNSUPPORTED)
L = _lib.LIB
FAKE = 1 << 20  # never dereferenced: validation fails first


def call(fn, p, args, **change):
    a = dict(args, **change)
    return fn(ctypes.byref(p) if p is not None else None, *a.values())


def sweep(fn, p, args, required, vec16, vec4):
    """Every required pointer left out, every pointer off its alignment."""
    for n in required:
        assert call(fn, p, args, **{n: None}) == NULL, n
    for n in vec16:
        assert call(fn, p, args, **{n: FAKE + 8}) == ALIGN, n
    for n in vec4:
        assert call(fn, p, args, **{n: FAKE + 2}) == ALIGN, n


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(_lib.moe_norm_problem) == 32 and ctypes.sizeof(_lib.moe_linear_problem) == 48


def test_permute_calls():
    p = lib.problem(64, 256, 16, 4, 128)
    a = dict(x=FAKE, pos=FAKE, w=FAKE, xs=FAKE, stream=None)
    sweep(L.moe_permute, p, a, ("x", "pos", "xs"), ("x", "xs"), ("pos", "w"))
    assert call(L.moe_permute, None, a) == NULL
    assert call(L.moe_permute, lib.problem(64, 252, 16, 4, 128), a) == UNSUP
    b = dict(dxs=FAKE, pos=FAKE, w=FAKE, x=FAKE, dx=FAKE, dw=FAKE, stream=None)
    sweep(L.moe_permute_backward, p, b, ("dxs", "pos", "x", "dx"), ("dxs", "x", "dx"), ("pos", "w", "dw"))
    c = dict(dout=FAKE, y=FAKE, pos=FAKE, w=FAKE, ysh=FAKE, s=FAKE, dy=FAKE, dw=FAKE, dysh=FAKE, ds=FAKE, stream=None)
    sweep(L.moe_combine_backward, p, c, ("dout", "y", "pos", "w", "ysh", "s", "dy", "dysh", "ds"),
          ("dout", "y", "ysh", "dy", "dysh"), ("pos", "w", "s", "dw", "ds"))
    p0 = lib.problem(0, 256, 16, 4, 128)
    for fn, n in ((L.moe_permute, 5), (L.moe_permute_backward, 7), (L.moe_combine_backward, 11)):
        assert fn(ctypes.byref(p0), *[None] * n) == OK
        assert fn(None, *[None] * n) == NULL


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(T=0), OK), (dict(T=-1), SHAPE), (dict(H=0), SHAPE), (dict(H=16392), SHAPE), (dict(H=252), UNSUP),
    (dict(H=252, dtype="f32"), OK), (dict(dtype="fp8"), DTYPE), (dict(T=1 << 24, H=256), SHAPE), (dict(T=2 ** 62), SHAPE),
    (dict(eps=0.0), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE),
    (dict(resid_scale=float("inf")), SHAPE), (dict(resid_scale=float("nan")), SHAPE), (dict(resid_scale=-2.0), OK)])
def test_norm_problems(kw, status):
    p = lib.norm_problem(**dict(dict(T=64, H=256, dtype="bf16"), **kw))
    a = [None] * 8
    assert L.moe_block_norm(ctypes.byref(p), *a) == (status if status != OK or p.T == 0 else NULL)
    assert (lib.moe_block_norm_workspace_bytes(p) > 0) == (status == OK)
    if status != OK:
        with pytest.raises(lib.MoEError):
            lib.norm_workspace(p, "cpu")
    for gate in (-1, 4):
        q = _lib.moe_norm_problem(64, 256, 1, gate, 1e-6, 1.0)
        assert L.moe_block_norm(ctypes.byref(q), *a) == SHAPE


@pytest.mark.parametrize("gate", ["token", "channel", "full"])
def test_norm_calls(gate):
    p = lib.norm_problem(64, 256, "bf16", gate)
    a = dict(f=FAKE, resid=FAKE, g_post=FAKE, gate=FAKE, g_pre=FAKE, out=FAKE, x=FAKE, stream=None)
    g16 = ("gate",) if gate != "token" else ()
    sweep(L.moe_block_norm, p, a, ("f", "resid", "gate", "g_pre", "x"), ("f", "resid", "g_post", "g_pre", "out", "x") + g16,
          () if g16 else ("gate",))
    assert call(L.moe_block_norm, p, a, out=None, x=None, g_pre=None) == NULL
    ws = lib.moe_block_norm_workspace_bytes(p)
    b = dict(dro=FAKE, dx=FAKE, f=FAKE, out=FAKE, g_post=FAKE, gate=FAKE, g_pre=FAKE, dresid=FAKE, df=FAKE, dg_post=FAKE,
             dgate=FAKE, dg_pre=FAKE, ws=FAKE, n=ws, stream=None)
    fn = L.moe_block_norm_backward
    sweep(fn, p, b, ("f", "out", "g_post", "gate", "g_pre", "df", "dx", "ws"),
          ("dro", "dx", "f", "out", "g_post", "g_pre", "dresid", "df", "ws") + (("dgate",) if gate == "full" else ()) + g16,
          ("dg_post", "dg_pre") + (("dgate",) if gate != "full" else ()))
    assert call(fn, p, b, dro=None, dx=None) == NULL
    assert call(fn, p, b, n=ws - 1) == WS
    none = lib.norm_problem(64, 256, "bf16", "none")
    assert call(L.moe_block_norm, none, a) == NULL  # a gate where the problem has none
    assert call(fn, none, b, gate=None) == NULL  # its gradient likewise
    assert call(fn, none, b, gate=None, dgate=None, f=None, df=None, g_post=None, dg_post=None, dresid=None) == NULL
    zero = lib.norm_problem(0, 256, "bf16", gate)
    assert fn(ctypes.byref(zero), *[None] * 13, 0, None) == OK


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(rows=0), OK), (dict(rows=-1), SHAPE), (dict(rows=1 << 24), SHAPE), (dict(K=0), SHAPE), (dict(N=0), SHAPE),
    (dict(K=(1 << 17) + 8), SHAPE), (dict(N=(1 << 17) + 8), SHAPE), (dict(K=1 << 15, N=1 << 15), SHAPE), (dict(groups=0), SHAPE),
    (dict(groups=1025), SHAPE), (dict(K=252), UNSUP), (dict(N=252), UNSUP), (dict(K=252, N=4, dtype="f32"), OK),
    (dict(dtype="mxfp4"), DTYPE), (dict(w_stride=-8), SHAPE), (dict(w_stride=64 * 256 - 8), SHAPE),
    (dict(w_stride=64 * 256 + 8), OK), (dict(w_stride=64 * 256 + 4), ALIGN), (dict(w_stride=1 << 41), SHAPE)])
def test_linear_problems(kw, status):
    p = lib.linear_problem(**dict(dict(rows=40, K=256, N=64, groups=3), **kw))
    assert L.moe_linear(ctypes.byref(p), *[None] * 9) == (status if status != OK or p.rows == 0 else NULL)
    assert (lib.moe_linear_workspace_bytes(p) > 0) == (status == OK)
    if status != OK:
        with pytest.raises(lib.MoEError):
            lib.linear_workspace(p, "cpu")
    for act in (-1, 3):
        q = _lib.moe_linear_problem(40, 256, 64, 3, 0, 1, act)
        assert L.moe_linear(ctypes.byref(q), *[None] * 9) == SHAPE


def test_linear_calls():
    p = lib.linear_problem(40, 256, 64, 3, "bf16", "silu")
    a = dict(x=FAKE, w=FAKE, bias=FAKE, off=FAKE, mul=FAKE, resid=FAKE, y=FAKE, z=FAKE, stream=None)
    sweep(L.moe_linear, p, a, ("x", "w", "off", "y"), ("x", "w", "bias", "mul", "resid", "y", "z"), ("off",))
    ws = lib.moe_linear_workspace_bytes(p)
    b = dict(dy=FAKE, x=FAKE, w=FAKE, off=FAKE, mul=FAKE, z=FAKE, dx=FAKE, dw=FAKE, db=FAKE, dmul=FAKE, ws=FAKE, n=ws, stream=None)
    fn = L.moe_linear_backward
    sweep(fn, p, b, ("dy", "x", "w", "off", "mul", "z", "ws"), ("dy", "x", "w", "mul", "z", "dx", "dw", "dmul", "ws"), ("off", "db"))
    assert call(fn, p, b, n=ws - 1) == WS
    none = lib.linear_problem(40, 256, 64, 3, "bf16", "none")
    assert call(fn, none, b, z=None) == NULL  # dmul needs it
    p0 = lib.linear_problem(0, 256, 64, 3)
    assert fn(ctypes.byref(p0), *[None] * 11, 0, None) == OK
    assert call(fn, p0, b, ws=None) == NULL  # dw has to be cleared, by a call with a workspace like any other
    assert call(fn, p0, b, dw=FAKE + 8) == ALIGN



def test_python_checks(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    p = lib.problem(4, 64, 8, 2, 8)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    pos, xs = torch.zeros((4, 2), dtype=torch.int32), bf(8, 64)
    with pytest.raises(ValueError, match="current CUDA device"):
        lib.moe_permute(p, bf(4, 64), pos, None, xs)
    with pytest.raises(ValueError, match="256 values"):
        lib.moe_permute(p, bf(4, 32), pos, None, xs)
    with pytest.raises(ValueError, match="bfloat16"):
        lib.moe_permute(p, torch.zeros(4, 64), pos, None, xs)
    with pytest.raises(ValueError, match="strided"):
        lib.moe_permute(p, bf(64, 4).T, pos, None, xs)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    with pytest.raises(ValueError, match="int32"):
        lib.moe_permute(p, bf(4, 64), pos.long(), None, xs)
    with pytest.raises(ValueError, match="float32"):
        lib.moe_permute(p, bf(4, 64), pos, bf(4, 2), xs)
    q = lib.norm_problem(4, 64, "bf16", "channel")
    with pytest.raises(ValueError, match="64 values"):
        lib.moe_block_norm(q, bf(4, 64), bf(4, 64), None, torch.zeros(4), bf(64), bf(4, 64), bf(4, 64))
    l = lib.linear_problem(4, 64, 32, 2, "bf16", "none", 2 * 32 * 64)
    with pytest.raises(ValueError, match="from one matrix to the next"):
        lib.moe_linear(l, bf(4, 64), bf(2, 32, 64), None, torch.zeros(3, dtype=torch.int32), None, None, bf(4, 32), None)
    for name in ("tanh", None):
        with pytest.raises(KeyError):
            lib.linear_problem(4, 64, 32, act=name)
