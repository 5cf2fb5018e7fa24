"""The largest numbers of tokens that the norms take: T * H < 2^31 as the header has it, also where H does not divide it."""
import ctypes

import pytest

import sparse_moe_layer_amd as lib
from sparse_moe_layer_amd import _lib


@pytest.mark.parametrize("H,dtype", [(4, "f32"), (8, "bf16"), (24, "bf16"), (264, "f32"), (2560, "bf16"), (4096, "bf16"),
                                     (16376, "bf16"), (16384, "f32")])
def test_largest_number_of_tokens(H, dtype):
    last = (2 ** 31 - 1) // H
    for T, ok in ((last, True), (last + 1, False)):
        p = lib.norm_problem(T, H, dtype)
        assert (T * H < 2 ** 31) == ok
        assert (lib.moe_block_norm_workspace_bytes(p) > 0) == ok
        st = _lib.LIB.moe_block_norm(ctypes.byref(p), *[None] * 8)
        assert st == (_lib.MOE_ERR_NULL if ok else _lib.MOE_ERR_SHAPE)
