"""The two implementations of the top-k give the same choice: moe_route's and that of moe_layer_forward_few.

Activations and router weights are small whole numbers, so every logit is exact in fp32 in whatever order it is summed,
and equal logits are equal bits.  The expected ids are numpy's stable sort; a weight is off by at most 2^-20 of itself
(exp, k additions and a division in fp32: (64 + 8) 2^-24).
"""
import numpy as np
import pytest
import torch

import sparse_moe_layer_amd as lib

pytestmark = pytest.mark.gpu


def route_both(x, wr, k, flags=0):
    """(ids, weights) of moe_route and of moe_layer_forward_few; the experts are zeros."""
    (T, H), E = x.shape, wr.shape[0]
    P = lib.problem(T, H, E, k, 8, 0, flags=flags)
    x, wr = x.bfloat16().cuda(), wr.bfloat16().cuda()
    zero = torch.zeros(E * 8 * H, dtype=torch.bfloat16, device="cuda")
    W = lib.weights(wr, zero, zero, zero)
    res = []
    for call in ("route", "few"):
        ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
        w = torch.full((T, k), float("nan"), device="cuda")
        if call == "route":
            lib.moe_route(P, x, wr, None, ids, w, None, lib.workspace(P))
        else:
            out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
            lib.moe_layer_forward_few(P, W, x, out, ids, w, lib.few_workspace(P))
            torch.cuda.synchronize()
            assert (out == 0).all()
        torch.cuda.synchronize()
        res.append((ids.cpu().numpy(), w.double().cpu().numpy()))
    return res


def check(logits, k, flags=0):
    """logits [T, E] whole numbers of at most 2^8: row t of x is the unit t, so they stand in the router's columns."""
    T, E = logits.shape
    x = torch.zeros((T, 16))
    x[range(T), range(T)] = 1.0
    wr = torch.zeros((E, 16))
    wr[:, :T] = torch.from_numpy(logits.T.astype(np.float32))
    want = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    top = np.take_along_axis(logits, want, 1).astype(np.float64)
    w = np.exp(top - top[:, :1])
    w /= w.sum(axis=1, keepdims=True)
    page = flags & lib.MOE_FLAG_PAGE_ROUTING
    for name, (ids, got) in zip(("route", "few"), route_both(x, wr, k, flags)):
        assert np.array_equal(ids, want), f"{name}: other experts"
        # (page: rounded to bf16, half a step of 2^-8, from a value that is off as without)
        assert (np.abs(got - w) <= (2.0 ** -20 + (2.0 ** -8 if page else 0)) * w).all(), f"{name}: other weights"


@pytest.mark.parametrize("flags", [0, lib.MOE_FLAG_PAGE_ROUTING])
@pytest.mark.parametrize("E,k", [(1024, 64), (1024, 1), (512, 10), (65, 10), (64, 64), (63, 3), (5, 5), (1, 1)])
def test_all_logits_equal(E, k, flags):
    check(np.full((3, E), 7), k, flags)


@pytest.mark.parametrize("E,k", [(1024, 64), (512, 10), (300, 64), (129, 2), (70, 64), (33, 8)])
def test_few_distinct_values(E, k):
    """16 rows of logits with 1 to 16 distinct values: ties at every place, more than 64 of them at the k-th."""
    rng = np.random.default_rng(E)
    check(np.stack([rng.integers(-t, 1, E) for t in range(16)]), k)


@pytest.mark.parametrize("equal", [63, 64, 65, 66, 128])
def test_as_many_equal_logits_as_the_short_ranking_holds(equal):
    """`equal` logits share the k-th place, spread over the experts; above them three larger ones."""
    rng = np.random.default_rng(equal)
    rows = []
    for _ in range(8):
        r = np.full(512, -9)
        at = rng.permutation(512)
        r[at[:equal]] = 3
        r[at[equal:equal + 3]] = (4, 5, 5)
        rows.append(r)
    check(np.stack(rows), 10)


def test_ties_within_one_lane_only():
    """Experts 64 apart, which one lane holds, tie; each lane's largest differs."""
    r = np.tile(np.arange(64)[None, :], (8, 1)).reshape(1, 512)
    check(np.repeat(r, 4, axis=0), 20)


def test_zeros_of_both_signs_are_equal():
    x = torch.ones((2, 16))
    x[1] = -1.0
    wr = torch.zeros((40, 16))
    wr[::2] = -0.0
    for ids, w in route_both(x, wr, 12):
        assert np.array_equal(ids, np.tile(np.arange(12), (2, 1)))
        assert (np.abs(w - 1 / 12) <= 2.0 ** -20 / 12).all()
