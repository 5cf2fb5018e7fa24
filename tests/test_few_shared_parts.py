"""The shared expert's hidden values of moe_layer_forward_few keep 16 significant bits, two bf16 parts."""
import numpy as np
import pytest
import torch

import expert_bounds as eb
import few_bounds as fb
import test_parity_few as tf

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,Is,wdt", [(16, 64, 64, "bf16"), (1, 64, 16, "bf16"), (4, 384, 640, "bf16"), (16, 384, 640, "fp8"),
                                        (3, 128, 200, "fp8"), (7, 320, 640, "mxfp4"), (16, 1024, 2048, "mxfp4")])
def test_shared_hidden_values_keep_sixteen_bits(T, H, Is, wdt):
    """The routed experts' down weights are zeros, so out is the shared expert's alone."""
    I = 128
    p = tf.few_problem(T, H, 4, 2, I, Is, wdt, seed=2)
    x, sg, wg, wu, wd = fb.cancelling_shared(T, H, Is, Is)
    dev = lambda a: torch.from_numpy(a).bfloat16().cuda().contiguous()
    p.x, p.sh_gate_w, p.sh_gate, p.sh_up, p.sh_down = dev(x), dev(sg[None]), dev(wg), dev(wu), dev(wd)
    p.w_down.zero_()
    out, _, _ = tf.run_few(p)
    torch.cuda.synchronize()
    ref, dy = fb.shared_parts(x, sg, wg, wu, wd)
    over = np.abs(out.double().cpu().numpy() - ref) / eb.rounded(ref, dy)
    print(f"[parts] {wdt} T={T} H={H} Is={Is}: {over.max():.3f} of the bound", flush=True)
    assert over.max() <= 1.0
