"""How far the block calls may be from their fp64 definitions, from the arithmetic they promise: fp32 sums and one
rounding to the output's dtype.

eps(t) / 2 is a rounding's largest relative error (bf16 2^-8, fp32 2^-24).  A sum of n fp32 terms in any order, with
products formed in fp32 or exactly, is off by at most (n + 1) 2^-24 of the sum of the terms' sizes; the row kernels
add at most DEPTH terms one after the other (the values of a thread, then the lanes, waves and workgroups).
"""
import numpy as np
import torch

F = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# values a thread adds on its own (16384 values over 512 threads, or 64 rows), 6 steps over lanes, 16 waves
DEPTH = 128


def half(dt):
    return torch.finfo(DT[dt]).eps / 2


def normal(gen, shape, dt, std=1.0, mean=0.0):
    return torch.empty(shape, dtype=DT[dt]).normal_(mean, std, generator=gen)


def np64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def dev(t):
    return None if t is None else t.cuda()


def close(got, want, bound, what):
    """|got - want| <= bound in every place."""
    g = np64(got)
    assert g.shape == want.shape, f"{what}: shape {g.shape} for {want.shape}"
    err = np.abs(g - want)
    bad = ~(err <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, err / np.maximum(bound, 1e-300), 0)), err.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, worst at {i}: {g[i]} for {want[i]}, bound "
                             f"{np.broadcast_to(bound, err.shape)[i]:.3e}")


def rms_close(got, want, dt, what, roundings=2):
    """Root mean square of the error against that of the values: `roundings` independent ones of at most half a step
    each stay below sqrt(roundings) half steps."""
    g = np64(got)
    ref = np.sqrt((want ** 2).mean())
    err = np.sqrt(((g - want) ** 2).mean())
    assert err <= np.sqrt(roundings) * half(dt) * ref, f"{what}: rms error {err / ref:.3e}"


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
