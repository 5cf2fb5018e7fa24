"""What a problem as a whole has to be in the block calls: refused by the library, also where Python looks at tensors first."""
import pytest
import torch

import sparse_moe_layer_amd as lib


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
