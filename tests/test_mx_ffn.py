"""The expert products with MXFP4 weights (moe_expert_ffn) where the kernels' tiles end: groups of every size around
16 and 128 rows, K that ends inside a step, repeated ids, one dense expert, values that must stay in their own row.

The outputs are held element by element to the bound of expert_bounds.py plus the rounding of y to bf16.
"""
import numpy as np
import pytest
import torch

import expert_bounds
import sparse_moe_layer_amd as lib
from oracle import mx

pytestmark = pytest.mark.gpu
FLAGS = {"default": 0, "gemm": lib.MOE_FLAG_FORCE_GEMM, "stream": lib.MOE_FLAG_FORCE_STREAM}


class Ffn:
    """Seeded MXFP4 experts and caller-given ids; run() -> y [R, H] in dispatch order, sorted, offsets."""

    def __init__(self, T, H, E, k, I, ids, seed=0, flags=0):
        g = torch.Generator().manual_seed(seed)
        self.x = torch.randn((T, H), generator=g).bfloat16().cuda()
        self.m = {}
        for name, shape in (("gate", (E, I, H)), ("up", (E, I, H)), ("down", (E, H, I))):
            codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, dtype=torch.uint8)
            scales = torch.randint(119, 123, (*shape[:-1], shape[-1] // 32), generator=g, dtype=torch.uint8)
            self.m[name] = [codes.cuda(), scales.cuda()]
        self.T, self.H, self.E, self.k, self.I = T, H, E, k, I
        self.ids = ids.int().cuda()
        self.p = lib.problem(T, H, E, k, I, 0, "bf16", "mxfp4", 32, flags)
        self.ws = lib.workspace(self.p)

    def run(self, stream=None, y=None):
        R = self.T * self.k
        off = torch.empty(self.E + 1, dtype=torch.int32, device="cuda")
        srt, pos = (torch.empty(R, dtype=torch.int32, device="cuda") for _ in range(2))
        (cg, sg), (cu, su), (cd, sd) = (self.m[n] for n in ("gate", "up", "down"))
        w = lib.weights(None, cg, cu, cd, sg, su, sd)
        y = torch.full((R, self.H), float("nan"), dtype=torch.bfloat16, device="cuda") if y is None else y
        lib.moe_dispatch(self.p, self.ids, off, srt, pos, self.ws, stream)
        lib.moe_expert_ffn(self.p, w, self.x, off, srt, y, None, self.ws, stream)
        return y, srt, off

    def check(self):
        y, srt, off = self.run()
        torch.cuda.synchronize()
        y, srt, off = y.double().cpu().numpy(), srt.cpu().numpy(), off.cpu().numpy()
        x = self.x.double().cpu().numpy()
        for e in range(self.E):
            rows = slice(off[e], off[e + 1])
            if off[e] == off[e + 1]:
                continue
            mats = [mx.dequant(self.m[n][0][e].cpu().numpy(), self.m[n][1][e].cpu().numpy())
                    for n in ("gate", "up", "down")]
            ref, dy = expert_bounds.expert(x[srt[rows] // self.k], *mats)
            err, tol = np.abs(y[rows] - ref), expert_bounds.rounded(ref, dy)
            assert (err <= tol).all(), f"expert {e}: {np.max(err / tol):.2f} of the bound"


def ids_of(sizes):
    """ids [T, 1] with the given group sizes, tokens interleaved over the groups."""
    left, ids = list(sizes), []
    while any(left):
        for e, n in enumerate(left):
            if n:
                ids.append(e)
                left[e] -= 1
    return torch.tensor(ids)[:, None]


@pytest.mark.parametrize("flag", ["default", "gemm", "stream"])
@pytest.mark.parametrize("H,I", [(96, 160), (288, 416), (640, 256)])
def test_group_sizes_around_every_block(H, I, flag):
    sizes = [0, 1, 15, 16, 17, 31, 33, 48, 64, 65, 80, 96, 97, 112, 113, 127, 128, 129, 0, 257, 5]
    Ffn(sum(sizes), H, len(sizes), 1, I, ids_of(sizes), seed=H, flags=FLAGS[flag]).check()


@pytest.mark.parametrize("T", [1, 2, 7, 16, 17, 32, 33, 40, 130, 300])
def test_one_dense_expert(T):
    Ffn(T, 1024, 1, 1, 512, torch.zeros((T, 1)), seed=T).check()


@pytest.mark.parametrize("steps", range(1, 10))
def test_k_of_every_number_of_steps(steps):
    """K of 1 to 9 steps of 128, less 32, 64 or 96: odd and even counts, every place in the scale bytes' period."""
    H, I = 128 * steps - 32 * (steps % 4), 128 * ((steps + 3) % 9 + 1) - 32 * ((steps + 1) % 4)
    sizes = [3, 40, 130]
    Ffn(173, H, 3, 1, I, ids_of(sizes), seed=steps).check()


@pytest.mark.parametrize("T,k", [(16, 4), (9, 6), (30, 4)])
def test_repeated_ids(T, k):
    """A token may name an expert more than once; then a group has more rows than there are tokens."""
    ids = torch.zeros((T, k))
    ids[:, -1] = torch.arange(T) % 5
    Ffn(T, 160, 6, k, 96, ids, seed=T).check()


@pytest.mark.parametrize("flag", ["gemm", "stream"])
def test_infinite_and_nan_rows_stay_their_own(flag):
    """K ends inside a step, so what follows a row in memory is another token's; its infinities must not be read in."""
    f = Ffn(50, 160, 2, 1, 96, ids_of([18, 32]), seed=3, flags=FLAGS[flag])
    ref, srt, _ = f.run()
    torch.cuda.synchronize()
    bad = torch.tensor([1, 8, 20, 49])
    f.x[bad[:2], :] = float("inf")
    f.x[bad[2:], :] = float("nan")
    y, _, _ = f.run()
    torch.cuda.synchronize()
    own = torch.isin(srt.long().cpu(), bad)
    assert torch.equal(y.cpu()[~own].view(torch.int16), ref.cpu()[~own].view(torch.int16))
    assert not torch.isfinite(y.cpu()[own]).any()


@pytest.mark.parametrize("flag", ["gemm", "stream"])
def test_nan_scale_marks_its_column_only(flag):
    """A NaN scale in the last group of a row that ends inside a step, also of the tensor's last row."""
    f = Ffn(40, 160, 2, 1, 96, ids_of([8, 32]), seed=4, flags=FLAGS[flag])
    f.m["down"][1][1, 31, 2] = 255
    f.m["down"][1][1, 159, 2] = 255
    y, srt, off = f.run()
    torch.cuda.synchronize()
    nan = torch.isnan(y.cpu())
    want = torch.zeros_like(nan)
    want[8:, [31, 159]] = True
    assert torch.equal(nan, want)


def test_writes_its_rows_and_no_more():
    f = Ffn(40, 160, 3, 1, 96, ids_of([5, 17, 18]), seed=5)
    big = torch.full((40 + 64, 160), -3.0, dtype=torch.bfloat16, device="cuda")
    f.run(y=big[:40])
    torch.cuda.synchronize()
    assert (big[40:] == -3.0).all() and torch.isfinite(big).all()


@pytest.mark.parametrize("T,E,k", [(300, 4, 2), (24, 64, 4), (5, 64, 4)])
def test_same_bits_every_time_and_in_a_graph(T, E, k):
    """Tiles are claimed in any order; no sum depends on it.  Replays with eager work between them."""
    g = torch.Generator().manual_seed(T)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    f = Ffn(T, 416, E, k, 160, ids, seed=T)
    ref = f.run()[0].clone()
    for _ in range(5):
        assert torch.equal(f.run()[0].view(torch.int16), ref.view(torch.int16))
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    y = torch.empty_like(ref)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        keep = f.run(side, y)
    for i in range(4):
        y.fill_(float("nan"))
        torch.randn(1 << 18, device="cuda").sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), ref.view(torch.int16)), f"replay {i}"
    del keep


def test_two_streams_with_workspaces_of_their_own():
    fs = [Ffn(T, 288, 6, 1, 160, ids_of([T // 6 + (i < T % 6) for i in range(6)]), seed=T) for T in (90, 200)]
    refs = [f.run()[0].clone() for f in fs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in fs]
    for _ in range(5):
        ys = []
        for f, s in zip(fs, streams):
            with torch.cuda.stream(s):
                ys.append(f.run(s)[0])
        torch.cuda.synchronize()
        for y, r in zip(ys, refs):
            assert torch.equal(y.view(torch.int16), r.view(torch.int16))


def test_layer_with_a_shared_expert_beside_the_tiles():
    """Enough rows per expert for the shared expert's launches to run on the second stream: eager, in a graph, and the
    call that forks none give the same bits."""
    T, H, E, k, I, Is = 200, 160, 4, 2, 96, 72
    g = torch.Generator().manual_seed(1)
    f = Ffn(T, H, E, k, I, torch.zeros((T, k)), seed=2)
    mk = lambda *s: (torch.randn(s, generator=g) * 0.05).bfloat16().cuda()
    wr, sh = mk(E, H), (mk(Is, H), mk(Is, H), mk(H, Is), mk(1, H))
    (cg, sg), (cu, su), (cd, sd) = (f.m[n] for n in ("gate", "up", "down"))
    P = lib.problem(T, H, E, k, I, Is, "bf16", "mxfp4", 32)
    W = lib.weights(wr, cg, cu, cd, sg, su, sd, *sh)
    ws = lib.workspace(P)
    ref, one = (torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lib.moe_layer_forward(P, W, f.x, ref, None, None, ws)
    lib.moe_layer_forward_noalloc(P, W, f.x, one, None, None)
    torch.cuda.synchronize()
    assert torch.isfinite(ref).all()
    assert torch.equal(one.view(torch.int16), ref.view(torch.int16))
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    out = torch.empty_like(ref)
    with torch.cuda.graph(graph, stream=side):
        lib.moe_layer_forward(P, W, f.x, out, None, None, ws, side)
    for i in range(4):
        out.fill_(float("nan"))
        lib.moe_layer_forward(P, W, f.x, one, None, None, lib.workspace(P))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16)), f"replay {i}"


def test_repeated_ids_beside_a_shared_expert():
    """24 tokens whose groups hold up to 72 rows: the routed rows are the same bits as without the shared expert."""
    T, H, E, k, I, Is = 24, 160, 5, 4, 96, 72
    ids = torch.zeros((T, k))
    ids[:, -1] = torch.arange(T) % 5
    f = Ffn(T, H, E, k, I, ids, seed=7)
    ref, srt, off = f.run()
    g = torch.Generator().manual_seed(8)
    sh = [(torch.randn(s, generator=g) * 0.05).bfloat16().cuda() for s in ((Is, H), (Is, H), (H, Is))]
    (cg, sg), (cu, su), (cd, sd) = (f.m[n] for n in ("gate", "up", "down"))
    P = lib.problem(T, H, E, k, I, Is, "bf16", "mxfp4", 32)
    W = lib.weights(None, cg, cu, cd, sg, su, sd, *sh)
    y = torch.full((T * k, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    ysh = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    lib.moe_expert_ffn(P, W, f.x, off, srt, y, ysh, lib.workspace(P))
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), ref.view(torch.int16))
    x, m = f.x.double().cpu().numpy(), [t.double().cpu().numpy() for t in sh]
    want, dy = expert_bounds.expert(x, *m)
    assert (np.abs(ysh.double().cpu().numpy() - want) <= expert_bounds.rounded(want, dy)).all()
