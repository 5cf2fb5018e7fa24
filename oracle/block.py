"""Plain fp64 CPU oracle of the calls around experts of the caller's own: rows to expert order and back, the norms
before and after a block with its gate and residual, products over groups of rows, and the gradients of all three.

TEST INFRASTRUCTURE ONLY.  Only the tests may import or run this module; the library path never calls it and shares
no code with it.  Everything is computed in fp64 from the stored values; nothing is rounded.  Formulas:

  permute     xs[pos[t,j]] = w[t,j] x[t]
  combine     out[t] = sum_j w[t,j] y[pos[t,j]] + sigmoid(s[t]) y_sh[t]
  block norm  n = f / rms(f) g_post,  r' = c r + gate n,  x = r' / rms(r') g_pre,  rms(v) = sqrt(mean v^2 + eps)
  linear      z = x W_g^T + b_g,  y = resid + act(z) mul

An assignment whose position is outside the rows has no row: nothing is written for it and it adds nothing.
"""
from __future__ import annotations

import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def sigmoid(z):
    return 0.5 * (1.0 + np.tanh(0.5 * z))


def _rows(pos, R):
    p = np.asarray(pos).reshape(-1)
    return p, (p >= 0) & (p < R)


def permute(x, pos, w, xs):
    """xs: [R, H] as it was, returned with the rows that the assignments name."""
    k = pos.shape[1]
    p, ok = _rows(pos, xs.shape[0])
    rows = np.repeat(x, k, axis=0) * (1.0 if w is None else w.reshape(-1, 1))
    out = xs.copy()
    out[p[ok]] = rows[ok]
    return out


def _gather(rows, pos):
    p, ok = _rows(pos, rows.shape[0])
    out = np.zeros((p.size, rows.shape[1]))
    out[ok] = rows[p[ok]]
    return out.reshape(*pos.shape, -1)


def permute_backward(dxs, pos, w, x=None):
    """dx, and dw where x is given."""
    d = _gather(dxs, pos)
    dx = (d if w is None else d * w[:, :, None]).sum(axis=1)
    return dx, None if x is None else np.einsum("tkh,th->tk", d, x)


def combine(y, pos, w, y_sh=None, s=None):
    out = (_gather(y, pos) * w[:, :, None]).sum(axis=1)
    return out if y_sh is None else out + sigmoid(s)[:, None] * y_sh


def combine_backward(dout, y, pos, w, dy, y_sh=None, s=None):
    """dy (the given rows as they were where no assignment names them), dw, dy_sh, ds."""
    dy = permute(dout, pos, w, dy)
    dw = np.einsum("tkh,th->tk", _gather(y, pos), dout)
    if y_sh is None:
        return dy, dw, None, None
    g = sigmoid(s)
    return dy, dw, g[:, None] * dout, g * sigmoid(-s) * (dout * y_sh).sum(axis=1)


def _rms(v, eps):
    return np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def _gate(gate):
    """[T] -> [T, 1]; [1, H] and [T, H] as they are; None -> 1."""
    return 1.0 if gate is None else gate[:, None] if gate.ndim == 1 else gate


def block_norm(f, resid, g_post, gate, g_pre, eps, scale):
    """gate: None, [T], [1, H] or [T, H]."""
    r = scale * resid
    if f is not None:
        n = f if g_post is None else f / _rms(f, eps) * g_post
        r = r + _gate(gate) * n
    return r, None if g_pre is None else r / _rms(r, eps) * g_pre


def _norm_backward(d, v, eps):
    q = _rms(v, eps)
    return d / q - v * (d * v).mean(axis=1, keepdims=True) / q**3


def block_norm_backward(dresid_out, dx, f, resid_out, g_post, gate, g_pre, eps, scale):
    out = {}
    dr = 0.0 if dresid_out is None else dresid_out
    if dx is not None:
        dr = dr + _norm_backward(dx * g_pre, resid_out, eps)
        out["dg_pre"] = (dx * resid_out / _rms(resid_out, eps)).sum(axis=0)
    out["dresid"] = scale * dr
    if f is None:
        return out
    n = f if g_post is None else f / _rms(f, eps) * g_post
    dn = _gate(gate) * dr
    if gate is not None:
        each = n * dr
        out["dgate"] = each.sum(axis=1) if gate.ndim == 1 else each.sum(axis=0) if gate.shape[0] == 1 != f.shape[0] else each
    if g_post is None:
        out["df"] = dn
    else:
        out["df"] = _norm_backward(dn * g_post, f, eps)
        out["dg_post"] = (dn * f / _rms(f, eps)).sum(axis=0)
    return out


def act(name, z):
    if name == "silu":
        return z * sigmoid(z)
    return z * 0.5 * _erfc(-z / math.sqrt(2.0)) if name == "gelu" else z


def act_slope(name, z):
    if name == "silu":
        return sigmoid(z) * (1.0 + z * sigmoid(-z))
    if name == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return np.ones_like(z)


def group_of_rows(offsets, rows, G):
    """Each row's group, -1 for none."""
    g = np.full(rows, -1)
    if offsets is None:
        g[:] = 0
        return g
    for i in range(G):
        g[max(int(offsets[i]), 0):max(min(int(offsets[i + 1]), rows), 0)] = i
    return g


def linear(x, w, bias, offsets, mul, resid, name):
    """y, z [rows, N]; rows of no group are NaN."""
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    z = y.copy()
    g = group_of_rows(offsets, x.shape[0], w.shape[0])
    for i in range(w.shape[0]):
        r = g == i
        z[r] = x[r] @ w[i].T + (0.0 if bias is None else bias[i])
        y[r] = act(name, z[r]) * (1.0 if mul is None else mul[r]) + (0.0 if resid is None else resid[r])
    return y, z


def linear_backward(dy, x, w, offsets, mul, z, name):
    """dx, dw, dbias, dmul; rows of no group are NaN in dx and dmul."""
    g = group_of_rows(offsets, x.shape[0], w.shape[0])
    m = 1.0 if mul is None else mul
    dz = dy * m * (1.0 if name == "none" else act_slope(name, z))
    dx, dw, db = np.full(x.shape, np.nan), np.zeros_like(w), np.zeros(w.shape[:2])
    dmul = None
    if mul is not None:
        dmul = dy * act(name, z)
        dmul[g < 0] = np.nan
    for i in range(w.shape[0]):
        r = g == i
        dx[r] = dz[r] @ w[i]
        dw[i] = dz[r].T @ x[r]
        db[i] = dz[r].sum(axis=0)
    return dx, dw, db, dmul
