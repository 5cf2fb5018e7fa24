"""moe_layer_forward_few at long rows, held to the root mean square of few_bounds.py."""
import numpy as np
import pytest
import torch

import few_bounds as fb
import test_parity_few as tf
from oracle import adapter

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wdt", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("T,H,E,k,I,Is", [(1, 8192, 4, 2, 2048, 256), (16, 8192, 4, 2, 2048, 0), (5, 2048, 3, 3, 8192, 2048),
                                          (16, 2560, 24, 10, 640, 640)])
def test_long_rows_in_the_root_mean_square(T, H, E, k, I, Is, wdt):
    p = tf.few_problem(T, H, E, k, I, Is, wdt, seed=T)
    out, ids, _ = tf.run_few(p)
    torch.cuda.synchronize()
    r = adapter.forward(p)
    assert np.array_equal(ids.cpu().numpy(), r["ids"])
    ratio = fb.rms_ratio(out.double().cpu().numpy(), fb.exact(p, r))
    print(f"[rms] {p.cfg.name}: {ratio.max():.5f} of {fb.RMS:.5f}", flush=True)
    assert (ratio <= fb.RMS).all()
