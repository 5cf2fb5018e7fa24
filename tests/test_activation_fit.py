"""The polynomial that bf16 GELU takes (x + 3) erfcx(x) from: the constants as the kernels have them, against the error
function of the standard library."""
import math
import os
import re

import numpy as np

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_moe_layer_amd", "csrc", "linear.hpp")


def constants():
    """Highest power first."""
    body = re.search(r"float erfcx_poly\(float t\) \{(.*?)\n\}", open(SRC).read(), re.S).group(1)
    c = [float(v) for v in re.findall(r"(-?\d\.\d+(?:e-?\d+)?)f", body)]
    assert len(c) == 10
    return c


def test_the_fit_over_its_range():
    c = constants()
    worst = rel = 0.0
    for x in np.linspace(0.0, 12.0, 24001):
        want = (x + 3.0) * math.exp(x * x) * math.erfc(x)
        err = abs(np.polyval(c, (x - 3.0) / (x + 3.0)) - want)
        worst, rel = max(worst, err), max(rel, err / want)
    # the figures that the comment at the constants states
    assert worst < 4.7e-8 and rel < 2.0e-8


def f32(v):
    return np.asarray(v, dtype=np.float32)


def test_phi_as_the_kernel_forms_it():
    """Phi(z) with every step in fp32 (the exponential and the reciprocal exact but for that rounding): 2e-7 absolute,
    2e-5 relative down to z = -12, and 0 or 1 at the infinities."""
    z = f32(np.concatenate([np.linspace(-12, 12, 200001), [np.inf, -np.inf, 3e38, -3e38]]))
    with np.errstate(over="ignore"):
        density = f32(np.exp2(f32(f32(f32(-0.5) * z * z) * f32(1.44269504)).astype(np.float64)))
    x = np.minimum(np.abs(z) * f32(0.70710678), f32(16.0))
    r = f32(1.0) / (x + f32(3.0))
    t = (x - f32(3.0)) * r
    p = np.zeros_like(t)
    for k in constants():
        p = f32(p.astype(np.float64) * t + np.float64(f32(k)))
    h = f32(0.5) * density * r * p
    got = np.where(z < 0, h, f32(1.0) - h).astype(np.float64)
    want = np.array([0.5 * math.erfc(-float(v) / math.sqrt(2.0)) for v in z])
    assert np.isfinite(got).all()
    assert np.abs(got - want).max() < 2e-7
    tail = (z < 0) & (z >= -12)
    assert (np.abs(got - want)[tail] / want[tail]).max() < 2e-5
    assert got[-4] == 1.0 and got[-3] == 0.0 and got[-2] == 1.0 and got[-1] == 0.0
