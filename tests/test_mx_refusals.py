"""What the MXFP4 conversions refuse before any launch (no GPU needed)."""
import pytest
import torch

import sparse_moe_layer_amd as lib


def test_tensors_off_the_current_device_are_refused():
    """The conversions launch on the current device's stream: host tensors never reach a kernel."""
    c, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    w = torch.zeros((4, 64), dtype=torch.bfloat16)
    for call in (lambda: lib.moe_mx_quantize(w, c, s), lambda: lib.moe_mx_dequantize(c, s, w),
                 lambda: lib.mx_quantize(w)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
    with pytest.raises(ValueError, match="device"):
        lib.moe_mx_quantize(w, c.to("meta"), s)
