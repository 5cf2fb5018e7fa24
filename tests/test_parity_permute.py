"""moe_permute, moe_permute_backward and moe_combine_backward against the fp64 oracle (oracle/block.py)."""
import numpy as np
import pytest
import torch

import sparse_moe_layer_amd as lib
from block_bounds import DEPTH, DT, F, close, dev, half, normal, np64, same_bits
from oracle import block

pytestmark = pytest.mark.gpu

# (T, H, k, dtype): one token and many, one and more than 16 rows a token, rows that end inside a wave's or a
# workgroup's chunks
SHAPES = [(1, 8, 1, "bf16"), (1, 2560, 10, "bf16"), (3, 4, 2, "f32"), (33, 1100, 3, "f32"), (257, 136, 4, "bf16"),
          (19, 4104, 8, "bf16"), (7, 8224, 10, "bf16"), (5, 2052, 16, "f32"), (21, 72, 17, "bf16"), (9, 264, 64, "f32"),
          (130, 640, 1, "f32")]
IDS = ["x".join(map(str, s)) for s in SHAPES]


def setup(T, H, k, dt, dropped=False, seed=0):
    gen = torch.Generator().manual_seed(1000 * T + H + k + seed)
    pos = torch.randperm(T * k, generator=gen).int().view(T, k)
    if dropped:  # places outside the rows: assignments without a row
        bad = torch.rand((T, k), generator=gen) < 0.3
        far = torch.tensor([-1, T * k, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
        pos = torch.where(bad, far[torch.randint(0, 4, (T, k), generator=gen)], pos)
    p = lib.problem(T, H, max(k, 2), k, 8, 0, dt, dt)
    return gen, p, pos, torch.softmax(torch.randn((T, k), generator=gen), 1)


@pytest.mark.parametrize("dropped", [False, True], ids=["all", "dropped"])
@pytest.mark.parametrize("weighted", [False, True], ids=["plain", "weighted"])
@pytest.mark.parametrize("T,H,k,dt", SHAPES, ids=IDS)
def test_permute(T, H, k, dt, weighted, dropped):
    print(f"[permute] {T} {H} {k} {dt} {weighted} {dropped}", flush=True)
    gen, p, pos, w = setup(T, H, k, dt, dropped)
    x, keep = normal(gen, (T, H), dt), normal(gen, (T * k, H), dt)
    xs = dev(keep)
    lib.moe_permute(p, dev(x), dev(pos), dev(w) if weighted else None, xs)
    want = block.permute(np64(x), pos.numpy(), np64(w) if weighted else None, np64(keep))
    # a product rounded to fp32 and then to dt, or nothing rounded
    close(xs, want, (half(dt) + 2 * F) * np.abs(want) if weighted else 0.0, "xs")


@pytest.mark.parametrize("dropped", [False, True], ids=["all", "dropped"])
@pytest.mark.parametrize("weighted", [False, True], ids=["plain", "weighted"])
@pytest.mark.parametrize("T,H,k,dt", SHAPES, ids=IDS)
def test_permute_backward(T, H, k, dt, weighted, dropped):
    print(f"[permute_backward] {T} {H} {k} {dt} {weighted} {dropped}", flush=True)
    gen, p, pos, w = setup(T, H, k, dt, dropped, 1)
    dxs, x = normal(gen, (T * k, H), dt), normal(gen, (T, H), dt)
    a = (np64(dxs), pos.numpy(), np64(w) if weighted else None, np64(x))
    want, dw = block.permute_backward(*a)
    size, dw_size = block.permute_backward(np.abs(a[0]), a[1], a[2], np.abs(a[3]))
    outs = []
    for with_dw in (False, True):
        dx = torch.empty((T, H), dtype=DT[dt], device="cuda")
        got = torch.empty((T, k), device="cuda") if with_dw else None
        lib.moe_permute_backward(p, dev(dxs), dev(pos), dev(w) if weighted else None, dev(x) if with_dw else None, dx, got)
        close(dx, want, (k + 2) * F * size + half(dt) * np.abs(want), "dx")
        outs.append(dx)
    close(got, dw, DEPTH * F * dw_size + F * np.abs(dw), "dtopk_w")
    assert same_bits(*outs)


@pytest.mark.parametrize("dropped", [False, True], ids=["all", "dropped"])
@pytest.mark.parametrize("shared", [False, True], ids=["routed", "shared"])
@pytest.mark.parametrize("T,H,k,dt", SHAPES, ids=IDS)
def test_combine_backward(T, H, k, dt, shared, dropped):
    print(f"[combine_backward] {T} {H} {k} {dt} {shared} {dropped}", flush=True)
    gen, p, pos, w = setup(T, H, k, dt, dropped, 2)
    dout, y, keep = normal(gen, (T, H), dt), normal(gen, (T * k, H), dt), normal(gen, (T * k, H), dt)
    y_sh, s = (normal(gen, (T, H), dt), 4 * torch.randn(T, generator=gen)) if shared else (None, None)
    dy, dw = dev(keep), torch.empty((T, k), device="cuda")
    dy_sh, ds = (torch.empty((T, H), dtype=DT[dt], device="cuda"), torch.empty(T, device="cuda")) if shared else (None, None)
    lib.moe_combine_backward(p, dev(dout), dev(y), dev(pos), dev(w), dev(y_sh), dev(s), dy, dw, dy_sh, ds)
    want = block.combine_backward(np64(dout), np64(y), pos.numpy(), np64(w), np64(keep), np64(y_sh), np64(s))
    size = block.combine_backward(np.abs(np64(dout)), np.abs(np64(y)), pos.numpy(), np64(w), np64(keep),
                                  None if y_sh is None else np.abs(np64(y_sh)), np64(s))
    close(dy, want[0], (half(dt) + 2 * F) * np.abs(want[0]), "dy")
    close(dw, want[1], DEPTH * F * size[1], "dtopk_w")
    if shared:
        # sigmoid: e^-z to 2 units in the last place, a sum and a quotient
        close(dy_sh, want[2], (half(dt) + 8 * F) * np.abs(want[2]), "dy_shared")
        close(ds, want[3], (DEPTH + 16) * F * size[3], "dshared_logit")
    # without the weights' gradient y is not needed; and in place
    again = dev(keep)
    lib.moe_combine_backward(p, dev(dout), None, dev(pos), dev(w), None, None, again, None, None, None)
    assert same_bits(again, dy)
    in_place, sh_place = dev(y), dev(y_sh)
    dw2 = torch.empty_like(dw)
    lib.moe_combine_backward(p, dev(dout), in_place, dev(pos), dev(w), sh_place, dev(s), in_place, dw2, sh_place, ds)
    assert same_bits(dw, dw2)
    named = torch.zeros(T * k, dtype=torch.bool)
    named[pos[(pos >= 0) & (pos < T * k)].long()] = True
    assert same_bits(in_place[named.cuda()], dy[named.cuda()])
    assert same_bits(in_place[~named.cuda()], dev(y)[~named.cuda()])
    if shared:
        assert same_bits(sh_place, dy_sh)


def test_infinities_and_nan_stay_with_their_rows():
    T, H, k = 6, 264, 3
    gen, p, pos, w = setup(T, H, k, "bf16")
    pos[4, 1] = -1  # a token's missing row adds nothing, whatever row 0 holds
    dxs, x = normal(gen, (T * k, H), "bf16"), normal(gen, (T, H), "bf16")
    dxs[0] = float("nan")
    dxs[1, 5] = float("inf")
    x[2] = float("inf")
    dx, dw = torch.empty((T, H), dtype=torch.bfloat16, device="cuda"), torch.empty((T, k), device="cuda")
    lib.moe_permute_backward(p, dev(dxs), dev(pos), dev(w), dev(x), dx, dw)
    t0, t1 = ((pos == 0).nonzero().tolist() or [[-1, -1]])[0], ((pos == 1).nonzero().tolist() or [[-1, -1]])[0]
    bad = torch.zeros((T, H), dtype=torch.bool)
    if t0[0] >= 0:
        bad[t0[0]] = True
    if t1[0] >= 0:
        bad[t1[0], 5] = True
    assert torch.equal(~torch.isfinite(dx.cpu()), bad)
    badw = torch.zeros((T, k), dtype=torch.bool)
    badw[2] = True
    for t, j in (t0, t1):
        if t >= 0:
            badw[t, j] = True
    badw[4, 1] = False
    assert torch.equal(~torch.isfinite(dw.cpu()), badw) and dw[4, 1] == 0


def test_positions_from_the_dispatch_bring_rows_there_and_back():
    """route's ids -> moe_dispatch -> permute; permute_backward without weights sums each token's k copies."""
    T, H, E, k = 50, 128, 12, 4
    gen = torch.Generator().manual_seed(5)
    p = lib.problem(T, H, E, k, 64)
    ids = torch.topk(torch.randn((T, E), generator=gen), k, dim=1)[1].int().cuda()
    off, order = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(T * k, dtype=torch.int32, device="cuda")
    pos, ws = torch.empty((T, k), dtype=torch.int32, device="cuda"), lib.workspace(p)
    lib.moe_dispatch(p, ids, off, order, pos, ws)
    x = normal(gen, (T, H), "bf16").cuda()
    xs = torch.empty((T * k, H), dtype=torch.bfloat16, device="cuda")
    lib.moe_permute(p, x, pos, None, xs)
    assert same_bits(xs, x[(order // k).long()])
    back = torch.empty_like(x)
    lib.moe_permute_backward(p, xs, pos, None, None, back, None)
    assert same_bits(back, x * k)  # k is a power of two: exact
