"""The fp64 oracle of the block calls (oracle/block.py): its gradients against central differences of its forward
functions, special cases, and assignments and rows that belong nowhere."""
import numpy as np
import pytest

from oracle import block

RNG = np.random.default_rng


def differences(fn, args, wrt, dout, h=1e-6):
    """d<fn(*args), dout> / d args[wrt] by central differences."""
    base = args[wrt]
    out = np.zeros_like(base)
    for i in np.ndindex(*base.shape):
        v = []
        for s in (h, -h):
            a = list(args)
            a[wrt] = base.copy()
            a[wrt][i] += s
            v.append(sum((o * d).sum() for o, d in zip(fn(*a), dout) if d is not None))
        out[i] = (v[0] - v[1]) / (2 * h)
    return out


# central differences: a truncation of order h^2 and a rounding of order 2^-52 / h of sums around 10
TOL = 1e-7


def test_permute_and_combine_gradients():
    r = RNG(1)
    T, k, H = 3, 2, 4
    pos = np.array([[4, 0], [2, -1], [3, 99]])  # rows 1 and 5 unnamed, two assignments without a row
    x, w, s = r.normal(size=(T, H)), r.normal(size=(T, k)), r.normal(size=T)
    y, y_sh = r.normal(size=(T * k, H)), r.normal(size=(T, H))
    dxs, dout = r.normal(size=(T * k, H)), r.normal(size=(T, H))
    zero = np.zeros((T * k, H))
    dx, dw = block.permute_backward(dxs, pos, w, x)
    fwd = lambda x, w: (block.permute(x, pos, w, zero),)
    assert np.abs(dx - differences(fwd, [x, w], 0, [dxs])).max() < TOL
    assert np.abs(dw - differences(fwd, [x, w], 1, [dxs])).max() < TOL
    assert dw[1, 1] == 0 and dw[2, 1] == 0
    assert np.abs(block.permute_backward(dxs, pos, None)[0]
                  - differences(lambda x: (block.permute(x, pos, None, zero),), [x], 0, [dxs])).max() < TOL
    fwd = lambda y, w, y_sh, s: (block.combine(y, pos, w, y_sh, s),)
    got = block.combine_backward(dout, y, pos, w, zero, y_sh, s)
    for i, (g, name) in enumerate(zip(got, ("y", "w", "y_sh", "s"))):
        assert np.abs(g - differences(fwd, [y, w, y_sh, s], i, [dout])).max() < TOL, name
    keep = np.full((T * k, H), 7.0)
    assert (block.permute(x, pos, w, keep)[[1, 5]] == 7.0).all()


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
def test_block_norm_gradients(post, gate):
    r = RNG(2)
    T, H, eps, c = 3, 5, 1e-2, 0.75
    f, resid = r.normal(size=(T, H)), r.normal(size=(T, H))
    g_post = r.normal(size=H) if post else None
    g_pre = r.normal(size=H)
    gt = {"none": None, "token": r.normal(size=T), "channel": r.normal(size=(1, H)), "full": r.normal(size=(T, H))}[gate]
    dro, dx = r.normal(size=(T, H)), r.normal(size=(T, H))
    fwd = lambda f, resid, g_post, gate, g_pre: block.block_norm(f, resid, g_post, gate, g_pre, eps, c)
    args = [f, resid, g_post, gt, g_pre]
    got = block.block_norm_backward(dro, dx, f, fwd(*args)[0], g_post, gt, g_pre, eps, c)
    for i, name in enumerate(("df", "dresid", "dg_post", "dgate", "dg_pre")):
        if args[i] is not None:
            assert np.abs(got[name] - differences(fwd, args, i, [dro, dx]).reshape(got[name].shape)).max() < TOL, name
    # without dx, and without dresid_out
    only = block.block_norm_backward(dro, None, f, None, g_post, gt, None, eps, c)
    assert np.abs(only["df"] - differences(fwd, args, 0, [dro, None])).max() < TOL
    only = block.block_norm_backward(None, dx, f, fwd(*args)[0], g_post, gt, g_pre, eps, c)
    assert np.abs(only["dresid"] - differences(fwd, args, 1, [None, dx])).max() < TOL


def test_block_norm_of_a_constant_row():
    f, resid = np.full((1, 4), 3.0), np.full((1, 4), 1.0)
    r, x = block.block_norm(f, resid, np.full(4, 2.0), np.array([0.5]), np.ones(4), 0.0, 1.0)
    assert np.allclose(r, 2.0) and np.allclose(x, 1.0)  # 1 + 0.5 * 2 * 3/3, then its sign


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
@pytest.mark.parametrize("mul", [False, True])
def test_linear_gradients(name, mul):
    r = RNG(3)
    rows, K, N, G = 6, 3, 4, 3
    off = np.array([1, 3, 3, 5])  # rows 0 and 5 in no group, group 1 empty
    x, w, b = r.normal(size=(rows, K)), r.normal(size=(G, N, K)), r.normal(size=(G, N))
    m = r.normal(size=(rows, N)) if mul else None
    dy = r.normal(size=(rows, N))
    z = block.linear(x, w, b, off, m, None, name)[1]
    dx, dw, db, dmul = block.linear_backward(dy, x, w, off, m, np.nan_to_num(z), name)
    inside = block.group_of_rows(off, rows, G) >= 0
    fwd = lambda x, w, b, m: (np.nan_to_num(block.linear(x, w, b, off, m, None, name)[0]),)
    args = [x, w, b, m]
    assert np.abs(dx[inside] - differences(fwd, args, 0, [dy])[inside]).max() < TOL
    assert np.abs(dw - differences(fwd, args, 1, [dy])).max() < TOL
    assert np.abs(db - differences(fwd, args, 2, [dy])).max() < TOL
    if mul:
        assert np.abs(dmul[inside] - differences(fwd, args, 3, [dy])[inside]).max() < TOL
    assert np.isnan(dx[~inside]).all() and (dw[1] == 0).all() and (db[1] == 0).all()


def test_activations_closed_forms():
    z = np.array([0.0, 1.0, -1.0, 30.0, -30.0])
    assert np.allclose(block.act("silu", z), [0.0, 0.7310585786300049, -0.2689414213699951, 30.0, 0.0], atol=1e-11)
    assert np.allclose(block.act("gelu", z), [0.0, 0.8413447460685429, -0.15865525393145707, 30.0, 0.0], atol=1e-12)
    assert block.act_slope("silu", np.array([0.0]))[0] == 0.5 and block.act_slope("gelu", np.array([0.0]))[0] == 0.5
