"""moe_linear's activations at infinities, NaN and the ends of the finite range: z * sigmoid(z) and z * Phi(z) as their
limits from above have it, in both dtypes and in every kernel of the forward call and of dz."""
import numpy as np
import pytest
import torch

import sparse_moe_layer_amd as lib
from block_bounds import DT, half, np64
from oracle import block

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
# a large value of each sign, and the places where the tails end
VALUES = [INF, NAN, -INF, 3.0e38, -3.0e38, 1.0e20, -1.0e20, 30.0, -30.0, 0.0]


def pre_activations(rows, n, dt):
    """Each of VALUES in each row, at another column from row to row, among ordinary ones."""
    gen = torch.Generator().manual_seed(rows + n)
    z = torch.empty((rows, n)).normal_(0, 2, generator=gen)
    for r in range(rows):
        for i, v in enumerate(VALUES):
            z[r, (7 * r + 5 * i) % n] = v
    return z.to(DT[dt])


def expected(act, z):
    """z * sigmoid(z) or z * Phi(z): +inf at +inf, NaN at NaN and (infinity times zero) at -inf."""
    with np.errstate(invalid="ignore", over="ignore"):
        return block.act(act, z)


def same_kind(got, want, what):
    g = np64(got)
    assert np.array_equal(np.isnan(g), np.isnan(want)), f"{what}: NaN"
    assert np.array_equal(np.isposinf(g), np.isposinf(want)) and np.array_equal(np.isneginf(g), np.isneginf(want)), what
    return np.isfinite(want)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 3, 64, 300], ids=["few-1", "few-3", "tiles-64", "tiles-300"])
def test_forward(rows, dt, act):
    """z from the bias: x is zero, so z is the bias itself, one row of it a group."""
    n = 64
    print(f"[linear nonfinite] {rows} {dt} {act}", flush=True)
    z = pre_activations(rows, n, dt)
    p = lib.linear_problem(rows, n, n, rows, dt, act)
    x = torch.zeros((rows, n), dtype=DT[dt], device="cuda")
    w = torch.zeros((rows, n, n), dtype=DT[dt], device="cuda")
    off = torch.arange(rows + 1, dtype=torch.int32, device="cuda")
    y, zo = torch.empty_like(x), torch.empty_like(x)
    lib.moe_linear(p, x, w, z.cuda(), off, None, None, y, zo)
    v = np64(z)
    same_kind(zo, v, "z")
    want = expected(act, v)
    fin = same_kind(y, want, "y")
    # the tails' absolute part and the value's relative one as over the finite range
    err = (half(dt) + 16 * 2.0 ** -24) * np.abs(want) + 8 * 2.0 ** -24 * np.minimum(np.abs(v), 8)
    assert (np.abs(np64(y)[fin] - want[fin]) <= err[fin]).all()


@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gradients(rows, dt, act):
    """dmul = dy * act(z), and dz at large finite z: the slope is 1 or 0 there.  (At an infinite z the slope's formula has
    infinity times zero.)"""
    n = 64
    z = pre_activations(rows, n, dt)
    gen = torch.Generator().manual_seed(5)
    dy = torch.empty((rows, n)).uniform_(0.5, 1.5, generator=gen).to(DT[dt])
    mul = torch.ones((rows, n), dtype=DT[dt])
    p = lib.linear_problem(rows, n, n, 1, dt, act)
    eye = torch.eye(n, dtype=DT[dt], device="cuda")[None]
    dx, dmul = (torch.empty((rows, n), dtype=DT[dt], device="cuda") for _ in range(2))
    v, d = np64(z), np64(dy)
    lib.moe_linear_backward(p, dy.cuda(), None, eye, None, mul.cuda(), z.cuda(), None, None, None, dmul,
                            lib.linear_workspace(p))
    want = d * expected(act, v)
    big = np.abs(want) > 3.3e38  # rounds past the largest value of the dtype
    g = np64(dmul)
    assert np.array_equal(np.isnan(g), np.isnan(want)) and np.isposinf(g[np.isposinf(want)]).all()
    fin = np.isfinite(want) & ~big
    err = (half(dt) + 20 * 2.0 ** -24) * np.abs(want) + 8 * 2.0 ** -24 * np.minimum(np.abs(v), 8) * d
    assert (np.abs(g[fin] - want[fin]) <= err[fin]).all()
    finite_z = torch.where(torch.isfinite(z), z, torch.ones_like(z))
    lib.moe_linear_backward(p, dy.cuda(), None, eye, None, mul.cuda(), finite_z.cuda(), dx, None, None, None,
                            lib.linear_workspace(p))
    vz = np64(finite_z)
    with np.errstate(over="ignore"):
        want = d * block.act_slope(act, vz)
    err = (2 * half(dt) + 24 * 2.0 ** -24) * np.abs(want) + 16 * 2.0 ** -24 * np.minimum(1 + np.abs(vz), 8) * d
    assert (np.abs(np64(dx) - want) <= err).all()
