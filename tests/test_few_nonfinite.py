"""Infinities and NaN in moe_layer_forward_few stay with their token, their expert and their column."""
import pytest
import torch

import test_parity_few as tf

pytestmark = pytest.mark.gpu


def all_experts(T, wdt, H=640, I=384, Is=104, seed=3):
    """Every token takes every expert, and the batch is one group per expert: what one token holds changes neither the
    groups nor the order of any other token's sums."""
    return tf.few_problem(T, H, 6, 6, I, Is, wdt, seed=seed)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("where", ["row", "last"])
@pytest.mark.parametrize("wdt,T", [("bf16", 16), ("fp8", 8), ("mxfp4", 4), ("bf16", 3)])
def test_bad_tokens_leave_the_others_alone(wdt, T, value, where):
    p = all_experts(T, wdt)
    ref, ids, w = tf.run_few(p)
    bad = [1, T - 1]
    if where == "row":
        p.x[bad] = value
    else:
        p.x[bad, -1] = value
    out, i2, w2 = tf.run_few(p)
    torch.cuda.synchronize()
    good = [t for t in range(T) if t not in bad]
    assert torch.equal(out[good].view(torch.int16), ref[good].view(torch.int16))
    assert torch.equal(ids[good], i2[good]) and torch.equal(w[good], w2[good])
    assert not torch.isfinite(out[bad]).any()
    assert ((i2 >= 0) & (i2 < p.cfg.E)).all()


def users(ids, e):
    return (ids == e).any(dim=1).cpu()


@pytest.mark.parametrize("H,I", [(640, 384), (160, 96)])
def test_nan_scales_mark_what_they_scale(H, I):
    """MXFP4: a NaN scale of a down row is one column of the tokens that use the expert, one of a gate or up row all
    of theirs; the last group of rows that end inside a run of loads."""
    p = tf.few_problem(7, H, 24, 4, I, 0, "mxfp4", seed=4)
    ref, ids, _ = tf.run_few(p)
    torch.cuda.synchronize()
    e = int(ids[2, 1])
    uses = users(ids, e)
    assert 0 < int(uses.sum()) < 7

    def run(scales, row):
        keep = scales[e, row, -1].item()
        scales[e, row, -1] = 255
        out, i2, _ = tf.run_few(p)
        torch.cuda.synchronize()
        scales[e, row, -1] = keep
        assert torch.equal(i2, ids)
        return out

    for row in (0, 33, H - 1):
        out = run(p.s_down, row)
        want = torch.zeros(7, H, dtype=torch.bool)
        want[uses, row] = True
        assert torch.equal(torch.isnan(out).cpu(), want)
        assert torch.equal(out.cpu()[~want].view(torch.int16), ref.cpu()[~want].view(torch.int16))
    for scales in (p.s_gate, p.s_up):
        for row in (0, I - 1):
            out = run(scales, row).cpu()
            assert torch.isnan(out[uses]).all()
            assert torch.equal(out[~uses].view(torch.int16), ref.cpu()[~uses].view(torch.int16))


@pytest.mark.parametrize("wdt", ["bf16", "fp8"])
def test_nan_weights_mark_what_they_weigh(wdt):
    H, I = 640, 384
    p = tf.few_problem(7, H, 24, 4, I, 0, wdt, seed=5)
    ref, ids, _ = tf.run_few(p)
    torch.cuda.synchronize()
    e = int(ids[0, 0])
    uses = users(ids, e)
    nan = 0x7F if wdt == "fp8" else float("nan")
    keep = p.w_down[e, 77, I - 1].clone()
    p.w_down[e, 77, I - 1] = nan
    out, _, _ = tf.run_few(p)
    torch.cuda.synchronize()
    want = torch.zeros(7, H, dtype=torch.bool)
    want[uses, 77] = True
    assert torch.equal(torch.isnan(out).cpu(), want)
    assert torch.equal(out.cpu()[~want].view(torch.int16), ref.cpu()[~want].view(torch.int16))
    p.w_down[e, 77, I - 1] = keep
    p.w_up[e, I - 1, H - 1] = nan
    out = tf.run_few(p)[0].cpu()
    assert torch.isnan(out[uses]).all()
    assert torch.equal(out[~uses].view(torch.int16), ref.cpu()[~uses].view(torch.int16))


@pytest.mark.parametrize("wdt", ["bf16", "mxfp4"])
def test_hidden_values_past_the_largest_number_are_infinite(wdt):
    """Finite inputs whose shared hidden value overflows: out is infinite with the down weight's sign, not NaN (an
    infinity has no second part), and where that weight is zero NaN, as infinity times zero is."""
    T, H, Is = 3, 256, 136
    p = tf.few_problem(T, H, 4, 2, 128, Is, wdt, seed=6)
    ref, _, _ = tf.run_few(p)
    p.x[1] = 0
    p.x[1, 5] = 2.0 ** 30
    p.sh_gate[9] = 0
    p.sh_up[9] = 0
    p.sh_gate[9, 5] = p.sh_up[9, 5] = 2.0 ** 36  # 2^66 each of token 1: the product is 2^132
    p.sh_gate_w.zero_()  # the gate is 1/2
    p.sh_down[40:, 9] = 0
    out, _, _ = tf.run_few(p)
    torch.cuda.synchronize()
    out, wd = out.float().cpu(), p.sh_down.float().cpu()[:, 9]
    assert torch.isfinite(out[[0, 2]]).all()
    at = wd[:40] != 0
    assert (out[1, :40][at] == torch.sign(wd[:40][at]) * float("inf")).all()
    assert torch.isnan(out[1, 40:]).all()
