"""fp64 experts with a bound on the error of an evaluation in the library's arithmetic.

The kernels form g = W_gate x and u = W_up x as fp32 sums of exact bf16 products, h = SiLU(g) u in fp32, rounded to
bf16, and y = W_down h as an fp32 sum.  First-order bounds, element by element:
  dg <= K 2^-23 |W_gate| |x|      a sum of K terms, each addition off by at most one unit in the last place
  dh <= 1.1 dg |u| + |SiLU(g)| du + 2^-20 |SiLU(g) u| + 2^-8 |h|
        (|SiLU'| <= 1.1; exp, reciprocal and two products in fp32, a few units each: 2^-20; bf16 rounding: 2^-8)
  dy <= |W_down| dh + K' 2^-23 |W_down| |h|
Nothing here runs the library.
"""
import numpy as np

BF16 = 2.0 ** -8  # half a step of bf16, relative
U32 = 2.0 ** -23


def expert(x, wg, wu, wd):
    """y [n, H] and the bound dy, before y is rounded; all fp64."""
    K, K2 = wg.shape[1], wd.shape[1]
    g, u = x @ wg.T, x @ wu.T
    dg, du = K * U32 * (np.abs(x) @ np.abs(wg).T), K * U32 * (np.abs(x) @ np.abs(wu).T)
    sg = g / (1 + np.exp(-g))
    h = sg * u
    dh = 1.1 * dg * np.abs(u) + np.abs(sg) * du + 2.0 ** -20 * np.abs(h) + BF16 * np.abs(h) + 2.0 ** -130
    ad = np.abs(wd).T
    return h @ wd.T, dh @ ad + K2 * U32 * (np.abs(h) @ ad)


def rounded(y, dy):
    """The bound after rounding to bf16."""
    return dy + BF16 * (np.abs(y) + dy)
