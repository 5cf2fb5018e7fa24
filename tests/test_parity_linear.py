"""moe_linear and its gradients against the fp64 oracle (oracle/block.py)."""
import numpy as np
import pytest
import torch

import sparse_moe_layer_amd as lib
from block_bounds import DT, F, close, dev, half, normal, np64, rms_close, same_bits
from oracle import block

pytestmark = pytest.mark.gpu

# (rows, K, N, groups, dtype): single rows and few, groups of a row or none, sizes that end inside every tile in every
# direction, many groups, long contractions
SHAPES = [(1, 8, 8, 1, "bf16"), (1, 2560, 640, 1, "bf16"), (10, 2560, 136, 16, "bf16"), (16, 264, 2056, 1, "bf16"),
          (17, 8192, 72, 1, "bf16"), (40, 520, 264, 3, "bf16"), (100, 128, 1032, 1, "bf16"), (300, 264, 328, 1, "bf16"),
          (700, 136, 72, 5, "bf16"), (513, 1032, 520, 2, "bf16"), (1030, 320, 264, 1, "bf16"), (2500, 64, 96, 40, "bf16"),
          (30, 72, 64, 1024, "bf16"), (1300, 1416, 256, 1, "bf16"), (70, 4104, 512, 1, "bf16"),
          (10, 520, 808, 64, "bf16"), (40, 1288, 264, 40, "bf16"), (9, 260, 660, 20, "f32"),
          (1, 4, 4, 1, "f32"), (3, 1100, 36, 1, "f32"), (33, 36, 20, 3, "f32"), (300, 132, 260, 1, "f32"),
          (400, 68, 132, 7, "f32"), (129, 516, 128, 2, "f32")]
IDS = ["x".join(map(str, s)) for s in SHAPES]
EPILOGUES = [("none", False, False, False), ("silu", False, True, False), ("gelu", True, False, True),
             ("none", True, True, True), ("silu", True, False, False), ("gelu", False, True, True)]
EIDS = ["none", "silu-mul", "gelu-bias-resid", "bias-mul-resid", "silu-bias", "gelu-mul-resid"]


def groups(gen, rows, G, outside=True):
    """Offsets with empty groups; a few rows before the first and behind the last group belong to none."""
    if G == 1:
        return None
    lo, hi = (min(2, rows // 4), rows - min(3, rows // 4)) if outside else (0, rows)
    cut = torch.sort(torch.randint(lo, hi + 1, (G - 1,), generator=gen))[0]
    return torch.cat([torch.tensor([lo]), cut, torch.tensor([hi])]).int()


def setup(rows, K, N, G, dt, bias, mul, resid, seed=0):
    gen = torch.Generator().manual_seed(rows + 10 * K + N + G + seed)
    d = {"x": normal(gen, (rows, K), dt), "w": normal(gen, (G, N, K), dt, K ** -0.5), "off": groups(gen, rows, G),
         "bias": normal(gen, (G, N), dt, 0.3) if bias else None, "mul": normal(gen, (rows, N), dt) if mul else None,
         "resid": normal(gen, (rows, N), dt) if resid else None, "dy": normal(gen, (rows, N), dt),
         "z": normal(gen, (rows, N), dt, 2.0)}
    return d


def sizes(d, K):
    """sum |x w| + |bias| of every output: what its fp32 sum's error is measured against."""
    return block.linear(np.abs(np64(d["x"])), np.abs(np64(d["w"])), None if d["bias"] is None else np.abs(np64(d["bias"])),
                        None if d["off"] is None else d["off"].numpy(), None, None, "none")[0]


def nan_like(shape, dt):
    return torch.full(shape, float("nan"), dtype=DT[dt], device="cuda")


@pytest.mark.parametrize("act,bias,mul,resid", EPILOGUES, ids=EIDS)
@pytest.mark.parametrize("rows,K,N,G,dt", SHAPES, ids=IDS)
def test_linear(rows, K, N, G, dt, act, bias, mul, resid):
    print(f"[linear] {rows} {K} {N} {G} {dt} {act} {bias} {mul} {resid}", flush=True)
    d = setup(rows, K, N, G, dt, bias, mul, resid)
    p = lib.linear_problem(rows, K, N, G, dt, act)
    g = {n: dev(v) for n, v in d.items()}
    y, z = nan_like((rows, N), dt), nan_like((rows, N), dt)
    lib.moe_linear(p, g["x"], g["w"], g["bias"], g["off"], g["mul"], g["resid"], y, z)
    off = None if d["off"] is None else d["off"].numpy()
    want, want_z = block.linear(*(np64(d[n]) for n in ("x", "w", "bias")), off, np64(d["mul"]), np64(d["resid"]), act)
    inside = block.group_of_rows(off, rows, G) >= 0
    for t in (y, z):  # rows of no group: as they were
        assert torch.isnan(t[~torch.from_numpy(inside).cuda()]).all()
    size = sizes(d, K)
    z_err = (K + 2) * F * size
    close(z[inside], want_z[inside], (z_err + half(dt) * np.abs(want_z))[inside], "z")
    # the activations' slopes stay below 1.13; act itself in fp32: at most 16 steps of its size and 2^-22 |z| beside the tail
    m = 1.0 if d["mul"] is None else np.abs(np64(d["mul"]))
    a = np.abs(block.act(act, want_z))
    err = m * (1.13 * z_err + 16 * F * a + (4 * F * np.abs(want_z) if act == "gelu" else 0)) + half(dt) * np.abs(want) + 2 * F * np.abs(want)
    if d["resid"] is not None:
        err = err + 2 * F * (m * a + np.abs(np64(d["resid"])))
    close(y[inside], want[inside], err[inside], "y")
    if dt == "bf16" and want[inside].size >= 64:
        rms_close(y[inside], want[inside], dt, "y")
    # without z; over resid and over mul: the same bits
    y2 = nan_like((rows, N), dt)
    lib.moe_linear(p, g["x"], g["w"], g["bias"], g["off"], g["mul"], g["resid"], y2, None)
    assert same_bits(y2, y)
    for n in ("resid", "mul"):
        if g[n] is not None:
            o = {k: v.clone() if k == n else v for k, v in g.items()}
            lib.moe_linear(p, g["x"], g["w"], g["bias"], g["off"], o["mul"], o["resid"], o[n], None)
            sel = torch.from_numpy(inside).cuda()
            assert same_bits(o[n][sel], y[sel]) and same_bits(o[n][~sel], g[n][~sel]), n


@pytest.mark.parametrize("act,bias,mul", [("none", False, False), ("none", True, False), ("silu", True, True),
                                          ("gelu", True, False), ("none", False, True), ("silu", False, True)],
                         ids=["none", "bias", "silu-bias-mul", "gelu-bias", "mul", "silu-mul"])
@pytest.mark.parametrize("rows,K,N,G,dt", SHAPES, ids=IDS)
def test_linear_backward(rows, K, N, G, dt, act, bias, mul):
    print(f"[linear_backward] {rows} {K} {N} {G} {dt} {act} {bias} {mul}", flush=True)
    d = setup(rows, K, N, G, dt, bias, mul, False, 1)
    p = lib.linear_problem(rows, K, N, G, dt, act)
    g = {n: dev(v) for n, v in d.items()}
    ws = lib.linear_workspace(p)
    ws.fill_(255)
    dx, dw, dmul = nan_like((rows, K), dt), nan_like((G, N, K), dt), nan_like((rows, N), dt) if mul else None
    db = torch.full((G, N), float("nan"), device="cuda") if bias else None
    z = g["z"] if act != "none" or mul else None
    lib.moe_linear_backward(p, g["dy"], g["x"], g["w"], g["off"], g["mul"], z, dx, dw, db, dmul, ws)
    off = None if d["off"] is None else d["off"].numpy()
    n64 = {n: np64(v) for n, v in d.items() if n != "off"}
    want = block.linear_backward(n64["dy"], n64["x"], n64["w"], off, n64["mul"], n64["z"], act)
    gr = block.group_of_rows(off, rows, G)
    inside = gr >= 0
    sel = torch.from_numpy(inside).cuda()
    assert torch.isnan(dx[~sel]).all() and (dmul is None or torch.isnan(dmul[~sel]).all())
    # dz: the slope in fp32 to 16 steps of its terms' sizes (at most 1 + |z|), then rounded to dtype where it is not dy
    s = 1.0 if mul is False else np.abs(n64["mul"])
    slope = 1.0 if act == "none" else np.abs(block.act_slope(act, n64["z"]))
    terms = 1.0 if act == "none" else 1.0 + np.abs(n64["z"])
    dz = np.abs(n64["dy"]) * s * slope
    dz32 = np.abs(n64["dy"]) * s * terms * 16 * F if act != "none" or mul else 0.0 * dz
    dz_err = dz32 + (half(dt) * dz if act != "none" or mul else 0.0)
    ones = lambda v: np.abs(v)
    dx_err, dw_err, db_err = np.zeros((rows, K)), np.zeros((G, N, K)), np.zeros((G, N))
    for i in range(G):
        r = gr == i
        n = int(r.sum())
        dx_err[r] = (dz_err + (N + 2) * F * dz)[r] @ ones(n64["w"][i])
        dw_err[i] = (dz_err + (n + 2) * F * dz)[r].T @ ones(n64["x"][r])
        db_err[i] = (dz32 + (n + 2) * F * dz)[r].sum(0)
    close(dx[sel], want[0][inside], (dx_err + half(dt) * np.abs(np.nan_to_num(want[0])))[inside], "dx")
    close(dw, want[1], dw_err + half(dt) * np.abs(want[1]), "dw")
    if dt == "bf16":
        if want[0][inside].size >= 64:
            rms_close(dx[sel], want[0][inside], dt, "dx")
        if want[1].size >= 64 and want[1].any():
            rms_close(dw, want[1], dt, "dw")
    if bias:
        close(db, want[2], db_err + F * np.abs(want[2]), "dbias")
    if mul:
        a = np.abs(n64["dy"] * block.act(act, n64["z"]))
        close(dmul[sel], want[3][inside], (half(dt) * np.abs(np.nan_to_num(want[3])) + 20 * F * a
                                           + 4 * F * np.abs(n64["dy"] * n64["z"]))[inside], "dmul")
    # each output alone gives the same bits
    for n in range(4):
        o = [nan_like((rows, K), dt), nan_like((G, N, K), dt), torch.empty((G, N), device="cuda"),
             nan_like((rows, N), dt) if mul else None]
        ref = (dx, dw, db, dmul)[n]
        if ref is None:
            continue
        only = [t if i == n else None for i, t in enumerate(o)]
        lib.moe_linear_backward(p, g["dy"], g["x"] if n == 1 else None, g["w"] if n == 0 else None, g["off"], g["mul"], z, *only, ws)
        keep = sel if n in (0, 3) else slice(None)
        assert same_bits(only[n][keep], ref[keep]), n
    if mul:  # over mul itself
        m2 = g["mul"].clone()
        lib.moe_linear_backward(p, g["dy"], g["x"], g["w"], g["off"], m2, z, dx, dw, db, m2, ws)
        assert same_bits(m2[sel], dmul[sel]) and same_bits(m2[~sel], g["mul"][~sel])


@pytest.mark.parametrize("rows,N", [(5, 64), (300, 136)])
def test_halves_of_a_fused_tensor(rows, N):
    """w_stride: the gate and up halves of one [G, 2 N, K] tensor, and their gradients in the halves of another."""
    G, K = 3, 72
    gen = torch.Generator().manual_seed(9)
    fused = normal(gen, (G, 2 * N, K), "bf16", 0.1).cuda()
    x, off = normal(gen, (rows, K), "bf16").cuda(), groups(gen, rows, G, False).cuda()
    dy = normal(gen, (rows, N), "bf16").cuda()
    p = lib.linear_problem(rows, K, N, G, "bf16", "none", 2 * N * K)
    dense = lib.linear_problem(rows, K, N, G, "bf16", "none")
    ws = lib.linear_workspace(p)
    grad = torch.full_like(fused, 7.0)
    for part in (slice(0, N), slice(N, 2 * N)):
        y, ref = (torch.empty((rows, N), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lib.moe_linear(p, x, fused[:, part], None, off, None, None, y, None)
        lib.moe_linear(dense, x, fused[:, part].contiguous(), None, off, None, None, ref, None)
        assert same_bits(y, ref)
        dx, dx_ref = torch.empty_like(x), torch.empty_like(x)
        dw = torch.empty((G, N, K), dtype=torch.bfloat16, device="cuda")
        before = grad.clone()
        lib.moe_linear_backward(p, dy, x, fused[:, part], off, None, None, dx, grad[:, part], None, None, ws)
        lib.moe_linear_backward(dense, dy, x, fused[:, part].contiguous(), off, None, None, dx_ref, dw, None, None, ws)
        assert same_bits(dx, dx_ref) and same_bits(grad[:, part], dw)
        rest = slice(N, 2 * N) if part.start == 0 else slice(0, N)
        assert same_bits(grad[:, rest], before[:, rest])


def test_no_rows_and_groups_without_rows():
    G, K, N = 4, 64, 72
    p0 = lib.linear_problem(0, K, N, G, "bf16", "silu")
    e = torch.empty((0, N), dtype=torch.bfloat16, device="cuda")
    x0 = torch.empty((0, K), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((G, N, K), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    lib.moe_linear(p0, x0, w, None, off, None, None, e, None)
    dw, db = torch.full_like(w, 3.0), torch.full((G, N), 3.0, device="cuda")
    lib.moe_linear_backward(p0, e, x0, w, off, None, e, x0, dw, db, None, lib.linear_workspace(p0))
    assert not dw.any() and not db.any()
    # every group empty, with rows there
    p = lib.linear_problem(6, K, N, G, "bf16", "none")
    for at in (0, 3, 6, -5, 100):
        off.fill_(at)
        y = torch.full((6, N), 5.0, dtype=torch.bfloat16, device="cuda")
        x = torch.ones((6, K), dtype=torch.bfloat16, device="cuda")
        lib.moe_linear(p, x, w, None, off, None, None, y, None)
        assert (y == 5.0).all()
        dx = torch.full_like(x, 5.0)
        dw.fill_(3.0)
        db.fill_(3.0)
        lib.moe_linear_backward(p, y, x, w, off, None, None, dx, dw, db, None, lib.linear_workspace(p))
        assert (dx == 5.0).all() and not dw.any() and not db.any()


def test_offsets_outside_the_rows():
    """Offsets below 0 and above rows are taken as the ends."""
    rows, K, N, G = 40, 64, 64, 3
    gen = torch.Generator().manual_seed(11)
    x, w = normal(gen, (rows, K), "bf16").cuda(), normal(gen, (G, N, K), "bf16", 0.1).cuda()
    p = lib.linear_problem(rows, K, N, G)
    ys = []
    for off in ([0, 10, 25, 40], [-7, 10, 25, 2 ** 31 - 1]):
        y = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
        lib.moe_linear(p, x, w, None, torch.tensor(off, dtype=torch.int32, device="cuda"), None, None, y, None)
        ys.append(y)
    assert same_bits(*ys)


@pytest.mark.parametrize("rows,G", [(3, 4), (200, 2)])
def test_infinities_and_nan_stay_with_their_rows(rows, G):
    K, N = 72, 136
    gen = torch.Generator().manual_seed(13)
    off = torch.linspace(0, rows, G + 1).int()
    x, w = normal(gen, (rows, K), "bf16"), normal(gen, (G, N, K), "bf16")
    dy, mul, z = (normal(gen, (rows, N), "bf16") for _ in range(3))
    bad = rows // 2
    x[bad, 3] = float("nan")
    dy[bad, 5] = float("inf")
    p = lib.linear_problem(rows, K, N, G, "bf16", "silu")
    y = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    lib.moe_linear(p, dev(x), dev(w), None, dev(off), dev(mul), None, y, None)
    fin = torch.isfinite(y.cpu())
    assert not fin[bad].any() and fin[torch.arange(rows) != bad].all()
    dx, dw, db = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda"), torch.empty_like(dev(w)), torch.empty((G, N), device="cuda")
    lib.moe_linear_backward(p, dev(dy), dev(x), dev(w), dev(off), dev(mul), dev(z), dx, dw, db, None, lib.linear_workspace(p))
    fin = torch.isfinite(dx.cpu())
    assert not fin[bad].any() and fin[torch.arange(rows) != bad].all()
    g = int(torch.searchsorted(off, bad, right=True)) - 1
    want = torch.ones((G, N, K), dtype=torch.bool)
    want[g, 5, :] = False  # the row of dW that the infinite gradient adds to
    want[g, :, 3] = False  # the column that the NaN input adds to
    assert torch.equal(torch.isfinite(dw.cpu()), want)
    assert int((~torch.isfinite(db)).sum()) == 1


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_activations_over_their_range(act, dt):
    """act and act' through an identity matrix over z from -40 to 40: relative to the value also in the tail, as far as
    2^-21 |z| (the forms' absolute part)."""
    n = 64
    z = torch.linspace(-40, 40, n * n).view(n, n).to(DT[dt])
    w = torch.eye(n, dtype=DT[dt])[None]
    p = lib.linear_problem(n, n, n, 1, dt, act)
    y = torch.empty((n, n), dtype=DT[dt], device="cuda")
    lib.moe_linear(p, z.cuda(), w.cuda(), None, None, None, None, y, None)
    v = np64(z)
    want = block.act(act, v)
    close(y, want, (half(dt) + 16 * F) * np.abs(want) + 8 * F * np.minimum(np.abs(v), 8), act)
    dx = torch.empty_like(y)
    one = torch.ones((n, n), dtype=DT[dt], device="cuda")
    lib.moe_linear_backward(p, one, None, w.cuda(), None, None, z.cuda(), dx, None, None, None, lib.linear_workspace(p))
    want = block.act_slope(act, v)
    close(dx, want, (half(dt) + 16 * F) * np.abs(want) + 16 * F * np.minimum(1 + np.abs(v), 8), act + "'")
