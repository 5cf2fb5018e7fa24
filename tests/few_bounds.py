"""Limits on the few-token layer's outputs that a lost part of a sum does not pass.

The element bounds of expert_bounds.py are worst cases: a sum of K terms may be off by K 2^-23 of its terms' sizes.  At K
of 8192 that is wider than what a lost K step changes.  A limit that does not grow with K:

rms(out - exact) <= 2^-7 rms(exact) for every token.  What rounds to bf16 is h of each routed expert and out, each by at
most 2^-8 of itself.  The rounding errors of h have no part in how the down weights were drawn, so a row of out has the
ratio of h's error to h, at most 2^-8 in the root mean square over the columns, up to the few percent by which a mean
over a thousand columns differs from its expectation; out's own rounding adds at most 2^-8 of itself.  Together
sqrt(2) 2^-8 = 0.0055; the limit is 2^-7 = 0.0078.  The fp32 sums are off by about sqrt(K) 2^-24, 5e-6 at K = 8192.
A part n of K lost changes a sum of K independent terms by sqrt(n / K) of itself: 0.125 for 128 of 8192.

Nothing here runs the library.
"""
import numpy as np

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
