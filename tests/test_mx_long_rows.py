"""The expert products with MXFP4 weights at long rows, held to a root mean square that does not grow with K.

y is rounded to bf16 once and h once, each by at most 2^-8 of itself: sqrt(2) 2^-8 of a row's root mean square, the limit
2^-7 (few_bounds.py says why, and its CPU test that a lost step of K passes four times the limit)."""
import numpy as np
import pytest
import torch

import few_bounds as fb
from oracle import mx
from test_mx_ffn import FLAGS, Ffn, ids_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("flag", ["default", "gemm", "stream"])
@pytest.mark.parametrize("H,I", [(8192, 2048), (2048, 8192), (2592, 672)])
@pytest.mark.parametrize("sizes", [[1, 0], [17, 3], [129, 5]])
def test_rms_of_long_rows(sizes, H, I, flag):
    f = Ffn(sum(sizes), H, len(sizes), 1, I, ids_of(sizes), seed=H, flags=FLAGS[flag])
    y, srt, off = f.run()
    torch.cuda.synchronize()
    y, srt, off = y.double().cpu().numpy(), srt.cpu().numpy(), off.cpu().numpy()
    x = f.x.double().cpu().numpy()
    for e in range(f.E):
        if off[e] == off[e + 1]:
            continue
        wg, wu, wd = (mx.dequant(f.m[n][0][e].cpu().numpy(), f.m[n][1][e].cpu().numpy()) for n in ("gate", "up", "down"))
        rows = slice(off[e], off[e + 1])
        ratio = fb.rms_ratio(y[rows], fb.swiglu(x[srt[rows]], wg, wu) @ wd.T)
        print(f"[rms] H={H} I={I} {sizes} {flag}: {ratio.max():.5f} of {fb.RMS:.5f}", flush=True)
        assert (ratio <= fb.RMS).all(), f"expert {e}"
