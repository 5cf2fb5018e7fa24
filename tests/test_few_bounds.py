"""The limits of few_bounds.py on the CPU: they pass the layer's arithmetic and reject what loses a part of it."""
import numpy as np
import pytest

import expert_bounds as eb
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


@pytest.mark.parametrize("T,H,Is", [(16, 64, 64), (4, 320, 640), (1, 32, 16)])
def test_second_part_of_the_shared_hidden_values(T, H, Is):
    x, sg, wg, wu, wd = fb.cancelling_shared(T, H, Is, Is)
    ref, dy = fb.shared_parts(x, sg, wg, wu, wd)
    s = 1 / (1 + np.exp(-(x @ sg)))[:, None]
    h = fb.swiglu(x, wg, wu)
    hi = fb.bf16(h)
    lo = fb.bf16(h - hi)

    def over(h):
        return np.max(np.abs(fb.bf16(s * (h @ wd.T)) - ref) / eb.rounded(ref, dy), axis=1)

    assert (over(hi + lo) <= 1).all()
    assert (over(hi) > 2).all()  # not there
    assert (over(hi - lo) > 2).all()  # subtracted
    if T > 1:
        assert (over(hi + np.roll(lo, 1, axis=0)) > 2).all()  # another token's
    if Is > 128:  # missing in one K unit of 128
        for k in range(0, Is, 128):
            part = lo.copy()
            part[:, k:k + 128] = 0
            assert (over(hi + part) > 2).all()
