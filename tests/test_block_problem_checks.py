"""What a problem as a whole has to be in the block calls: refused by the library, also where Python looks at tensors first."""
import ctypes

import pytest
import torch

import sparse_moe_layer_amd as lib
from sparse_moe_layer_amd import _lib

SHAPE, UNSUP, NULL = _lib.MOE_ERR_SHAPE, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_NULL


@pytest.mark.parametrize("kw,status", [
    (dict(), NULL), (dict(I=8), NULL), (dict(I=0), SHAPE), (dict(I=4), UNSUP), (dict(I=4, act="f32", wdt="f32"), NULL),
    (dict(T=1 << 20, k=8, I=256), UNSUP), (dict(T=1 << 20, k=8, I=248), NULL), (dict(T=1 << 28, k=8, H=8, I=8), SHAPE)])
def test_permute_problems_as_a_whole(kw, status):
    """The expert's hidden width counts although the calls do not read it: any small one will do."""
    p = lib.problem(**dict(dict(T=64, H=256, E=16, k=4, I=128), **kw))
    for fn, n in ((_lib.LIB.moe_permute, 5), (_lib.LIB.moe_permute_backward, 7), (_lib.LIB.moe_combine_backward, 11)):
        assert fn(ctypes.byref(p), *[None] * n) == status


def test_no_groups_of_strided_weights(monkeypatch):
    """groups == 0 is the library's to refuse, with weights at a stride as without."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    off = torch.zeros(1, dtype=torch.int32)
    for stride in (0, 2 * 32 * 64):
        p = lib.linear_problem(4, 64, 32, 0, "bf16", "none", stride)
        w = bf(0, 64, 64)[:, :32]
        with pytest.raises(lib.MoEError):
            lib.moe_linear(p, bf(4, 64), w, None, off, None, None, bf(4, 32), None, stream=1)
        with pytest.raises(lib.MoEError):
            lib.moe_linear_backward(p, bf(4, 32), bf(4, 64), w, off, None, None, bf(4, 64), w, None, None,
                                    torch.zeros(256, dtype=torch.uint8), stream=1)
