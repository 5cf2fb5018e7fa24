"""The limits of few_bounds.py on the CPU: they pass the layer's arithmetic and reject what loses a part of it."""
import numpy as np
import pytest

import few_bounds as fb


def one_expert(H, I, seed=0):
    g = np.random.default_rng(seed)
    x = fb.bf16(g.normal(0, 1, (2, H)))
    wg, wu, wd = (fb.bf16(g.normal(0, 0.02, s)) for s in ((I, H), (I, H), (1024, I)))  # 1024 of the output columns
    return x, wg, wu, wd


@pytest.mark.parametrize("H,I", [(8192, 2048), (2560, 640)])
def test_rms_limit(H, I):
    x, wg, wu, wd = one_expert(H, I)
    ref = fb.swiglu(x, wg, wu) @ wd.T

    def ratio(x=x, wg=wg, wu=wu, wd=wd, lost=slice(0, 0), column=None):
        h = fb.bf16(fb.swiglu(x, wg, wu))
        h[:, lost] = 0
        out = fb.bf16(h @ wd.T)
        if column is not None:
            out[:, column] = 0
        return fb.rms_ratio(out, ref).max()

    assert ratio() <= fb.RMS
    short = wg.copy()
    short[:, -128:] = 0
    assert ratio(wg=short) > 4 * fb.RMS  # a K unit of the gate's sums
    short = wu.copy()
    short[:, 256:288] = 0
    assert ratio(wu=short) > 4 * fb.RMS  # one scale group of the up rows
    assert ratio(lost=slice(I - 128, I)) > 4 * fb.RMS  # a K unit of the down rows
    assert ratio(lost=slice(32, 64)) > 4 * fb.RMS  # one scale group of them
    twice = wd.copy()
    twice[:, :128] *= 2
    assert ratio(wd=twice) > 4 * fb.RMS  # a K unit counted twice
    assert ratio(x=x[::-1]) > 4 * fb.RMS  # another token's rows
    assert ratio(column=np.arange(512, 528)) > 4 * fb.RMS  # a block of output columns
