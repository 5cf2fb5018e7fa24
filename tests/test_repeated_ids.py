"""The grouped expert products of a small batch whose ids repeat an expert within a token (moe_dispatch takes any ids):
a group then holds more rows than there are tokens, and more than the 16 of one streamed block.

Every routed row, and the shared expert's, is held element by element to the bound of expert_bounds.py (fp8 weights
convert exactly, their block scales multiply fp32 sums) plus the rounding of y to bf16; the rows behind the last one
stay as they were.
"""
import numpy as np
import pytest
import torch

import expert_bounds as eb
import sparse_moe_layer_amd as lib
from oracle import adapter
from sparse_moe_layer_amd.tensors import structs
from synthetic import CONFIGS, make_problem

pytestmark = pytest.mark.gpu
FLAGS = {"default": 0, "gemm": lib.MOE_FLAG_FORCE_GEMM, "stream": lib.MOE_FLAG_FORCE_STREAM}


def bits(t):
    return t.view(torch.int16)


def run(p, ids, flags=0, stream=None):
    """(y [R + 3, H] with three rows of guard, y_shared, offsets, sorted) of the caller's ids."""
    c = p.cfg
    P, W = structs(p, flags)
    ws = lib.workspace(P)
    R = c.T * c.k
    off = torch.empty(c.E + 1, dtype=torch.int32, device="cuda")
    srt, pos = (torch.empty(R, dtype=torch.int32, device="cuda") for _ in range(2))
    y = torch.full((R + 3, c.H), float("nan"), dtype=torch.bfloat16, device="cuda")
    y[R:] = -3.0
    ysh = torch.full((c.T, c.H), float("nan"), dtype=torch.bfloat16, device="cuda") if c.I_shared else None
    lib.moe_dispatch(P, ids, off, srt, pos, ws, stream)
    lib.moe_expert_ffn(P, W, p.x, off, srt, y, ysh, ws, stream)
    # the two phases as calls of their own
    h = torch.full((R, c.I), float("nan"), dtype=torch.bfloat16, device="cuda")
    hsh = torch.full((c.T, c.I_shared), float("nan"), dtype=torch.bfloat16, device="cuda") if c.I_shared else None
    y2 = torch.full((R, c.H), float("nan"), dtype=torch.bfloat16, device="cuda")
    ysh2 = torch.empty_like(ysh) if c.I_shared else None
    lib.moe_expert_gate_up(P, W, p.x, off, srt, h, hsh, ws, stream)
    lib.moe_expert_down(P, W, off, h, hsh, y2, ysh2, ws, stream)
    torch.cuda.synchronize()
    assert (y[R:] == -3.0).all()
    assert torch.equal(bits(y[:R]), bits(y2)), "the phases as separate calls differ"
    assert ysh is None or torch.equal(bits(ysh), bits(ysh2))
    return y[:R], ysh, off, srt


def check(p, ids, flags=0):
    c = p.cfg
    y, ysh, off, srt = run(p, ids, flags)
    y, off, srt = y.double().cpu().numpy(), off.cpu().numpy(), srt.cpu().numpy()
    flat = ids.reshape(-1).cpu().numpy()
    assert np.array_equal(srt, np.argsort(flat, kind="stable"))
    x, _, shared, _ = adapter.dense_inputs(p)
    get = adapter.expert_weights_fn(p)
    for e in range(c.E):
        rows = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        ref, dy = eb.expert(x[srt[rows] // c.k], *get(e))
        over = np.abs(y[rows] - ref) / eb.rounded(ref, dy)
        bad = np.nonzero(~(over <= 1.0).all(axis=1))[0]
        assert not len(bad), f"expert {e}: rows {bad[:8].tolist()} of {off[e + 1] - off[e]} are off"
    if c.I_shared:
        ref, dy = eb.expert(x, *shared)
        assert (np.abs(ysh.double().cpu().numpy() - ref) <= eb.rounded(ref, dy)).all()


def problem(wdt, T, k, E, Is, H=256, I=128, seed=0):
    cfg = CONFIGS["max_fp8" if wdt == "fp8" else "flash_prefill"].with_(
        name=f"repeated_{wdt}_{T}_{k}", T=T, H=H, E=E, k=k, I=I, I_shared=Is, wdt=wdt, zipf_s=0.0)
    print(f"[repeated] {wdt} T={T} k={k} E={E} Is={Is}", flush=True)
    return make_problem(cfg, seed, device="cuda")


def sizes_to_ids(sizes, T, k):
    """ids [T, k] with the given group sizes (their sum is T * k), spread over the tokens."""
    flat = np.repeat(np.arange(len(sizes)), sizes)
    assert len(flat) == T * k
    return torch.from_numpy(flat[np.random.default_rng(T * k).permutation(len(flat))].reshape(T, k).astype(np.int32)).cuda()


@pytest.mark.parametrize("wdt", ["bf16", "fp8"])
@pytest.mark.parametrize("flag", ["default", "gemm", "stream"])
@pytest.mark.parametrize("Is", [0, 128])
@pytest.mark.parametrize("T,k,sizes", [
    (16, 4, [0, 16, 17, 0, 31, 0]),          # around one block and two
    (9, 8, [33, 0, 1, 15, 23, 0, 0, 0]),     # three blocks, next to groups of one block
    (1, 20, [20] + [0] * 19),                # one token, one expert named 20 times
    (16, 64, [1024] + [0] * 63),             # the longest group there is
])
def test_groups_of_more_rows_than_tokens(T, k, sizes, Is, flag, wdt):
    check(problem(wdt, T, k, len(sizes), Is, seed=T), sizes_to_ids(sizes, T, k), FLAGS[flag])


@pytest.mark.parametrize("wdt", ["bf16", "fp8"])
def test_the_most_blocks_that_a_batch_can_have(wdt):
    """1024 experts, 16 tokens of 64 picks: 1023 groups of at most one row beside one of three blocks, and 64 of 16."""
    p = problem(wdt, 16, 64, 1024, 128, H=128, seed=3)
    check(p, sizes_to_ids([1] * 983 + [41] + [0] * 40, 16, 64))
    check(p, sizes_to_ids(([16] + [0] * 15) * 64, 16, 64))


@pytest.mark.parametrize("wdt", ["bf16", "fp8"])
def test_replays_with_other_ids(wdt):
    """Captured once; replays read the ids that are there, whatever sizes their groups have."""
    p = problem(wdt, 8, 6, 12, 128, seed=4)
    c = p.cfg
    P, W = structs(p)
    sets = [sizes_to_ids(s, 8, 6) for s in ([48] + [0] * 11, [4] * 12, [17, 0, 31] + [0] * 9)]
    for i in sets:
        check(p, i)
    refs = [run(p, i)[0].clone() for i in sets]
    ids, ws = sets[0].clone(), lib.workspace(P)
    off = torch.empty(c.E + 1, dtype=torch.int32, device="cuda")
    srt, pos = (torch.empty(48, dtype=torch.int32, device="cuda") for _ in range(2))
    y, ysh = torch.empty(48, c.H, dtype=torch.bfloat16, device="cuda"), torch.empty_like(p.x)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        lib.moe_dispatch(P, ids, off, srt, pos, ws, side)
        lib.moe_expert_ffn(P, W, p.x, off, srt, y, ysh, ws, side)
    for i in range(6):
        ids.copy_(sets[i % 3])
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(y), bits(refs[i % 3])), f"replay {i}"
