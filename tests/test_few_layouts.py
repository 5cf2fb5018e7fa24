"""moe_layer_forward_few on weights at a stride and on tensors that are 16-byte aligned and no more: the bits of the dense
call, and nothing written beside the outputs."""
import pytest
import torch

import sparse_moe_layer_amd as lib
import test_parity_few as tf
from sparse_moe_layer_amd.tensors import structs

pytestmark = pytest.mark.gpu
SHAPES = {"bf16": (5, 328, 20, 3, 200, 72), "fp8": (5, 384, 20, 3, 256, 72), "mxfp4": (5, 416, 20, 3, 352, 72)}


def bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("wdt", ["bf16", "fp8", "mxfp4"])
def test_fused_gate_up_and_experts_apart(wdt):
    p = tf.few_problem(*SHAPES[wdt], wdt, seed=1)
    c = p.cfg
    ref, _, _ = tf.run_few(p)
    fused = torch.cat([p.w_gate, p.w_up], dim=1).contiguous()
    # down matrices with a matrix of NaN patterns between them
    apart = torch.full((c.E, 2, *p.w_down.shape[1:]), 0x7F if p.w_down.dtype == torch.uint8 else float("nan"),
                       dtype=p.w_down.dtype, device="cuda")
    apart[:, 0] = p.w_down
    P, _ = structs(p)
    n = c.I * c.H
    W = lib.weights(p.w_router, fused, fused, apart, p.s_gate, p.s_up, p.s_down, p.sh_gate, p.sh_up, p.sh_down, p.sh_gate_w,
                    stride_gate=2 * n, stride_up=2 * n, stride_down=2 * n)
    W.w_up = fused.data_ptr() + p.w_gate[0].numel() * fused.element_size()
    out = torch.full_like(ref, float("nan"))
    lib.moe_layer_forward_few(P, W, p.x, out, None, None, lib.few_workspace(P))
    torch.cuda.synchronize()
    assert torch.equal(bits(out), bits(ref))


@pytest.mark.parametrize("wdt", ["bf16", "fp8", "mxfp4"])
def test_tensors_at_any_sixteen_bytes(wdt):
    p = tf.few_problem(*SHAPES[wdt], wdt, seed=2)
    ref, ids, w = tf.run_few(p)
    keep = []

    def moved(t):
        if t is None:
            return None
        n = t.numel() * t.element_size()
        b = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN before and behind it
        at = 16 * (1 + len(keep) % 3)
        b[at:at + n] = t.contiguous().view(torch.uint8).reshape(-1)
        keep.append(b)
        return b[at:at + n].view(t.dtype).view(t.shape)

    P, _ = structs(p)
    W = lib.weights(*(moved(t) for t in (p.w_router, p.w_gate, p.w_up, p.w_down, p.s_gate, p.s_up, p.s_down, p.sh_gate, p.sh_up,
                                         p.sh_down, p.sh_gate_w)))
    out, i2, w2 = moved(torch.zeros_like(ref)), moved(torch.zeros_like(ids)), moved(torch.zeros_like(w))
    lib.moe_layer_forward_few(P, W, moved(p.x), out, i2, w2, lib.few_workspace(P))
    torch.cuda.synchronize()
    assert torch.equal(bits(out), bits(ref)) and torch.equal(ids, i2) and torch.equal(w, w2)
    for t in (out, i2, w2):
        b = next(b for b in keep if b.data_ptr() <= t.data_ptr() < b.data_ptr() + b.numel())
        at, n = t.data_ptr() - b.data_ptr(), t.numel() * t.element_size()
        assert (b[:at] == 0xFF).all() and (b[at + n:] == 0xFF).all()
