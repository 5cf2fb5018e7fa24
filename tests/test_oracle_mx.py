"""The MXFP4 oracle and generator against independent statements of the format (CPU)."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import sparse_moe_layer_amd as lib
from oracle import mx
from sparse_moe_layer_amd import _lib
from synthetic.gen import quantize_mxfp4_rows


def test_code_table_is_the_formats():
    want = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    got = mx.decode_e2m1(np.arange(16))
    assert got[:8].tolist() == want and got[8:].tolist() == [-v for v in want]
    assert np.signbit(got[8])  # minus zero


def test_packing_puts_the_even_value_in_the_low_bits():
    assert mx.unpack(np.array([[0x21, 0xF3]], np.uint8)).tolist() == [[1, 2, 3, 15]]


def test_values_of_the_format_survive_a_round_trip():
    # every signed grid value at every scale that a group with a 4 or a 6 can have
    vals = np.concatenate([mx.GRID, -mx.GRID, mx.GRID[::-1], -mx.GRID[::-1]])
    for e in range(-127, 126):
        w = (vals * 2.0 ** e)[None]
        codes, scales = mx.quantize(w)
        assert scales[0, 0] == e + 127
        assert np.array_equal(mx.dequant(codes, scales), w)


def test_rounding_is_nearest_with_ties_to_the_even_code():
    mid = [(a + b) / 2 for a, b in itertools.pairwise(mx.GRID)] if hasattr(itertools, "pairwise") else [
        (mx.GRID[i] + mx.GRID[i + 1]) / 2 for i in range(7)]
    w = np.zeros((1, 32))
    w[0, 0] = 4.0  # scale 1
    w[0, 1:8] = mid
    w[0, 8:15] = np.array(mid) * (1 + 1e-6)
    w[0, 15:22] = np.array(mid) * (1 - 1e-6)
    w[0, 22] = 7.9
    codes, scales = mx.quantize(w)
    n = mx.unpack(codes)[0]
    assert scales[0, 0] == 127
    assert n[1:8].tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert n[8:15].tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert n[15:22].tolist() == [0, 1, 2, 3, 4, 5, 6]
    assert n[22] == 7


def test_zeros_infinities_and_nan():
    w = np.zeros((4, 32))
    w[0, 3] = -0.0
    w[1, 5] = np.inf
    w[2, 6] = np.nan
    w[3, 0] = 2.0 ** -149
    codes, scales = mx.quantize(w)
    assert scales[:, 0].tolist() == [0, 255, 255, 0]
    assert mx.unpack(codes)[0].tolist() == [8 if i == 3 else 0 for i in range(32)]
    v = mx.dequant(codes, scales)
    assert np.isnan(v[1]).all() and np.isnan(v[2]).all() and (v[3] == 0).all()


def test_generator_and_oracle_agree():
    torch.manual_seed(3)
    for scale in (1.0, 0.02, 1e-30, 1e-38, 3e38):
        w = torch.randn(7, 96) * scale
        w = w.clamp(-3.4e38, 3.4e38)
        w[2, 32:64] = 0
        c, s = quantize_mxfp4_rows(w)
        oc, os_ = mx.quantize(w.double().numpy())
        assert np.array_equal(s.numpy(), os_) and np.array_equal(c.numpy(), oc)


@pytest.mark.parametrize("kw,status", [
    (dict(), _lib.MOE_OK),
    (dict(scale_block=128), _lib.MOE_ERR_UNSUPPORTED),
    (dict(H=272), _lib.MOE_ERR_UNSUPPORTED),
    (dict(I=48), _lib.MOE_ERR_UNSUPPORTED),
    (dict(H=32, I=32), _lib.MOE_OK),
    (dict(act="f32"), _lib.MOE_ERR_DTYPE),
    (dict(T=0), _lib.MOE_OK),
])
def test_mx_problem_validation(kw, status):
    base = dict(T=64, H=256, E=16, k=4, I=160, I_shared=0, act="bf16", wdt="mxfp4", scale_block=32, flags=0)
    base.update(kw)
    p = lib.problem(**base)
    assert lib.moe_validate(p) == status
    assert (lib.moe_workspace_bytes(p) > 0) == (status == _lib.MOE_OK)


def test_mx_weights_are_checked_before_any_launch():
    L = _lib.LIB
    fake = 1 << 20  # never dereferenced: validation fails first
    p = lib.problem(64, 256, 16, 4, 160, 0, "bf16", "mxfp4", 32)
    wsz = lib.moe_workspace_bytes(p)

    def ffn(strides=(0, 0, 0), scales=(fake, fake, fake)):
        w = _lib.moe_weights(fake, fake, fake, fake, *strides, *scales, None, None, None, None)
        return L.moe_expert_ffn(ctypes.byref(p), ctypes.byref(w), fake, fake, fake, fake, None, fake, wsz - 1, None)

    assert ffn(scales=(fake, None, fake)) == _lib.MOE_ERR_NULL
    assert ffn(scales=(fake, fake + 8, fake)) == _lib.MOE_ERR_ALIGN
    assert ffn(strides=(16, 0, 0)) == _lib.MOE_ERR_ALIGN  # strides count values: multiples of 32
    assert ffn(strides=(0, 0, -32)) == _lib.MOE_ERR_SHAPE
    assert ffn() == _lib.MOE_ERR_WORKSPACE


def test_mx_conversions_validate_before_any_launch():
    L = _lib.LIB
    fake = 1 << 20
    bf, f32 = _lib.MOE_BF16, _lib.MOE_F32
    Q, D = L.moe_mx_quantize, L.moe_mx_dequantize
    assert Q(fake, _lib.MOE_FP8_E4M3FN, 4, 64, 64, fake, fake, None) == _lib.MOE_ERR_DTYPE
    assert Q(fake, bf, -1, 64, 64, fake, fake, None) == _lib.MOE_ERR_SHAPE
    assert Q(fake, bf, 4, 0, 64, fake, fake, None) == _lib.MOE_ERR_SHAPE
    assert Q(fake, bf, 4, 64, 56, fake, fake, None) == _lib.MOE_ERR_SHAPE
    assert Q(fake, bf, 1 << 40, 64, 64, fake, fake, None) == _lib.MOE_ERR_SHAPE
    assert Q(fake, bf, 4, 48, 48, fake, fake, None) == _lib.MOE_ERR_UNSUPPORTED
    assert Q(fake, bf, 4, 64, 68, fake, fake, None) == _lib.MOE_ERR_ALIGN
    assert Q(fake, f32, 4, 64, 66, fake, fake, None) == _lib.MOE_ERR_ALIGN
    for a in range(3):
        args = [fake] * 3
        args[a] = None
        assert Q(args[0], bf, 4, 64, 64, args[1], args[2], None) == _lib.MOE_ERR_NULL
        assert D(args[1], args[2], 4, 64, args[0], 64, None) == _lib.MOE_ERR_NULL
    assert Q(fake + 8, bf, 4, 64, 64, fake, fake, None) == _lib.MOE_ERR_ALIGN
    assert D(fake + 8, fake, 4, 64, fake, 64, None) == _lib.MOE_ERR_ALIGN
    assert Q(None, bf, 0, 64, 64, None, None, None) == _lib.MOE_OK  # no rows: nothing read or written
    assert D(None, None, 0, 64, None, 64, None) == _lib.MOE_OK


def test_binding_refuses_wrong_tensors():
    w = torch.zeros(4, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(lib.MoEError):
        lib.moe_mx_quantize(w.half(), c, s)
    with pytest.raises(lib.MoEError):
        lib.moe_mx_dequantize(c, s, w.float())
    with pytest.raises(lib.MoEError):
        lib.mx_quantize(torch.zeros(4, 40, dtype=torch.bfloat16))
    for bad in ((c[:, :16], s), (c, s[:3]), (c.int(), s), (c, s.int())):
        with pytest.raises(ValueError):
            lib.moe_mx_quantize(w, *bad)
    with pytest.raises(ValueError):
        lib.moe_mx_quantize(torch.zeros(64, 4, dtype=torch.bfloat16).T, c, s)  # columns not contiguous
