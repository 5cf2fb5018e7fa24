"""Limits on the few-token layer's outputs that a lost part of a sum does not pass.

The element bounds of expert_bounds.py are worst cases: a sum of K terms may be off by K 2^-23 of its terms' sizes.  At K
of 8192 that is wider than what a lost K step changes.  Two more limits, which do not grow with K:

rms(out - exact) <= 2^-7 rms(exact) for every token.  What rounds to bf16 is h of each routed expert and out, each by at
most 2^-8 of itself.  The rounding errors of h have no part in how the down weights were drawn, so a row of out has the
ratio of h's error to h, at most 2^-8 in the root mean square over the columns, up to the few percent by which a mean
over a thousand columns differs from its expectation; out's own rounding adds at most 2^-8 of itself.  Together
sqrt(2) 2^-8 = 0.0055; the limit is 2^-7 = 0.0078.  The fp32 sums are off by about sqrt(K) 2^-24, 5e-6 at K = 8192.
A part n of K lost changes a sum of K independent terms by sqrt(n / K) of itself: 0.125 for 128 of 8192.

shared_parts: the exact value of a gated shared expert and its bound where h is kept in two bf16 parts.  A part is off by
2^-8 of what it rounds, so h by 2^-16 of itself; otherwise as expert_bounds.expert, with K the number of terms of a sum
that are not zero (adding a zero rounds nothing).
Nothing here runs the library.
"""
import numpy as np

import expert_bounds as eb

RMS = 2.0 ** -7


def rms_ratio(out, exact):
    """rms(out - exact) / rms(exact) of each row."""
    return np.sqrt(((out - exact) ** 2).mean(axis=1) / (exact ** 2).mean(axis=1))


def bf16(v):
    """fp64 -> the nearest bf16, ties to even (of normal numbers in bf16's range)."""
    b = np.asarray(v, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)


def swiglu(x, wg, wu):
    g = x @ wg.T
    return g / (1 + np.exp(-g)) * (x @ wu.T)


def exact(p, r):
    """The layer's value in 64 bits, out [T, H], from the oracle's routing r of problem p."""
    from oracle import adapter

    c = p.cfg
    x, _, shared, _ = adapter.dense_inputs(p)
    get = adapter.expert_weights_fn(p)
    out = np.zeros((c.T, c.H))
    for e in np.unique(r["ids"]):
        t, j = np.nonzero(r["ids"] == e)
        wg, wu, wd = get(e)
        out[t] += r["w"][t, j][:, None] * (swiglu(x[t], wg, wu) @ wd.T)
    if c.I_shared:
        out += r["gamma"][:, None] * (swiglu(x, *shared[:2]) @ shared[2].T)
    return out


def shared_parts(x, sg, wg, wu, wd):
    """(value, bound) [T, H] of sigmoid(x . sg) shared(x), before out is rounded."""
    u32 = eb.U32
    terms = lambda a, b: (a != 0).astype(float) @ (b != 0).astype(float).T
    s = 1 / (1 + np.exp(-(x @ sg)))[:, None]
    ds = (terms(x, sg[None]) * u32) * (np.abs(x) @ np.abs(sg))[:, None] / 4 + 2.0 ** -20 * s  # sigmoid' <= 1/4; its evaluation 2^-20
    g, u = x @ wg.T, x @ wu.T
    dg, du = terms(x, wg) * u32 * (np.abs(x) @ np.abs(wg).T), terms(x, wu) * u32 * (np.abs(x) @ np.abs(wu).T)
    a = g / (1 + np.exp(-g))
    h = a * u
    dh = 1.1 * dg * np.abs(u) + np.abs(a) * du + (2.0 ** -20 + 2.0 ** -16) * np.abs(h)
    y = h @ wd.T
    dy = dh @ np.abs(wd).T + terms(h, wd) * u32 * (np.abs(h) @ np.abs(wd).T)
    # eight waves' parts of the columns' sums, and their product with s
    return s * y, s * dy + ds * np.abs(y) + 9 * u32 * s * (np.abs(h) @ np.abs(wd).T)


def cancelling_shared(T, H, Is, seed):
    """x [T, H], sg [H], wg, wu [Is, H], wd [H, Is], bf16 values in fp64, of a shared expert whose output is what one bf16
    part of h cannot hold: hidden columns come in pairs that differ by about 2^-8 of themselves, and an output column is
    the difference of one pair (every pair has one if H >= Is / 2).  x is zero but in 16 places."""
    g = np.random.default_rng(seed)
    places = g.permutation(H)[:16]
    x, sg = np.zeros((T, H)), bf16(g.normal(0, 0.02, H))
    x[:, places] = bf16(g.normal(0, 1, (T, 16)))
    wg, wu = bf16(g.normal(0, 0.2, (Is, H))), bf16(g.normal(0, 0.2, (Is, H)))
    wg[1::2], wu[1::2] = wg[::2], wu[::2]
    at = g.choice(places, Is // 2)
    odd = np.arange(1, Is, 2)
    wu[odd, at] = bf16(wu[odd, at] * (1 + 2.0 ** -4))  # one of 16 weights that count
    wd, n = np.zeros((H, Is)), np.arange(H)
    pair = g.permutation(H) % (Is // 2)
    wd[n, 2 * pair] = bf16(g.normal(0, 0.2, H))
    wd[n, 2 * pair + 1] = -wd[n, 2 * pair]
    return x, sg, wg, wu, wd
