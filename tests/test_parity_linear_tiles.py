"""moe_linear and its gradients at sizes that take every size of tile, in each direction and dtype, with the groups'
ends inside the tiles, against products in fp64."""
import pytest
import torch

import sparse_moe_layer_amd as lib
from block_bounds import DT, F, half, same_bits

pytestmark = pytest.mark.gpu

# (rows, K, N, groups, dtype), long in the product's two output sizes and short in its contraction
FORWARD = [(4090, 136, 3320, 1, "bf16"), (4000, 72, 2568, 5, "bf16"), (2990, 200, 1608, 1, "bf16"),
           (3900, 136, 1000, 40, "bf16"), (1490, 392, 1016, 1, "bf16"), (1000, 520, 600, 1, "bf16"),
           (600, 520, 1032, 200, "bf16"), (300, 1288, 520, 40, "bf16"), (10, 2560, 808, 64, "bf16"), (2500, 264, 1800, 60, "bf16"), (16300, 40, 520, 64, "bf16"),
           (4090, 68, 3300, 1, "f32"), (2000, 132, 1028, 1, "f32"), (900, 260, 516, 3, "f32"), (200, 516, 324, 1, "f32"),
           (3900, 68, 516, 40, "f32")]
DX = [(4090, 3320, 136, 1, "bf16"), (4000, 2568, 72, 5, "bf16"), (2990, 1608, 200, 1, "bf16"),
      (3900, 1000, 136, 40, "bf16"), (1490, 1016, 392, 1, "bf16"), (1000, 600, 520, 1, "bf16"), (90, 600, 520, 1, "bf16"),
      (4090, 3300, 68, 1, "f32"), (2000, 1028, 132, 1, "f32"), (900, 516, 260, 3, "f32"), (200, 324, 516, 1, "f32")]
DW = [(1100, 3320, 4088, 1, "bf16"), (300, 2184, 2056, 1, "bf16"), (380, 776, 648, 10, "bf16"), (1000, 776, 648, 10, "bf16"),
      (200, 1016, 1504, 1, "bf16"), (200, 600, 520, 1, "bf16"), (200, 200, 520, 1, "bf16"),
      (300, 2052, 2180, 1, "f32"), (400, 1028, 1028, 4, "f32"), (200, 1028, 1028, 5, "f32"), (150, 516, 520, 3, "f32"), (150, 132, 260, 1, "f32")]
BOTH = [(9, 200, 2480, 1, "bf16"), (2000, 512, 128, 1, "bf16"), (16, 1028, 2052, 1, "f32"), (2000, 516, 132, 1, "f32"),
        (600, 1024, 2560, 1, "bf16"), (1490, 1016, 1504, 1, "bf16"), (1000, 600, 520, 1, "bf16"), (90, 200, 264, 1, "bf16"), (500, 264, 520, 1, "f32"),
        (100, 132, 260, 1, "f32")]


def ids(shapes):
    return ["x".join(map(str, s)) for s in shapes]


def tensors(rows, K, N, G, dt):
    gen = torch.Generator(device="cuda").manual_seed(rows + K + N + G)
    r = lambda *s: torch.empty(s, dtype=DT[dt], device="cuda").normal_(generator=gen)
    off = None
    if G > 1:  # uneven groups, some empty, rows before the first and behind the last of no group
        cut = torch.sort(torch.randint(3, rows - 4, (G - 1,), generator=gen, device="cuda"))[0]
        off = torch.cat([cut.new_tensor([3]), cut, cut.new_tensor([rows - 5])]).int()
    return r(rows, K), (r(G, N, K).float() * K ** -0.5).to(DT[dt]), r(rows, N), off


def spans(off, rows):
    return [(0, rows)] if off is None else list(zip(off.tolist()[:-1], off.tolist()[1:]))


def check(got, want, size, n, dt, what):
    """size: the sum of the n terms' sizes."""
    bound = (n + 2) * F * size + half(dt) * want.abs()
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), f"{what}: {float((err / bound.clamp_min(1e-300)).max()):.2f} bounds off"


@pytest.mark.parametrize("rows,K,N,G,dt", FORWARD, ids=ids(FORWARD))
def test_forward(rows, K, N, G, dt):
    print(f"[forward] {rows} {K} {N} {G} {dt}", flush=True)
    x, w, y, off = tensors(rows, K, N, G, dt)
    y.fill_(float("nan"))
    lib.moe_linear(lib.linear_problem(rows, K, N, G, dt), x, w, None, off, None, None, y, None)
    inside = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for g, (a, b) in enumerate(spans(off, rows)):
        inside[a:b] = True
        if b > a:
            xd, wd = x[a:b].double(), w[g].double().T.contiguous()
            check(y[a:b], xd @ wd, xd.abs() @ wd.abs(), K, dt, f"group {g}")
    assert bool(torch.isnan(y[~inside]).all())


@pytest.mark.parametrize("rows,K,N,G,dt", FORWARD, ids=ids(FORWARD))
def test_epilogue(rows, K, N, G, dt):
    """bias, SiLU, factor and residual at the same sizes, over the factor's own tensor too."""
    print(f"[epilogue] {rows} {K} {N} {G} {dt}", flush=True)
    x, w, mul, off = tensors(rows, K, N, G, dt)
    resid, bias = mul.flip(1).contiguous(), torch.linspace(-1, 1, G * N, device="cuda").view(G, N).to(DT[dt])
    y, z = torch.full_like(mul, float("nan")), torch.full_like(mul, float("nan"))
    p = lib.linear_problem(rows, K, N, G, dt, "silu")
    lib.moe_linear(p, x, w, bias, off, mul, resid, y, z)
    inside = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for g, (a, b) in enumerate(spans(off, rows)):
        inside[a:b] = True
        if b == a:
            continue
        xd, wd, bd = x[a:b].double(), w[g].double().T.contiguous(), bias[g].double()
        m, r, want = mul[a:b].double(), resid[a:b].double(), xd @ wd + bd
        size = xd.abs() @ wd.abs() + bd.abs()
        check(z[a:b], want, size, K + 1, dt, f"z of group {g}")
        # SiLU's slope is at most 1.1; 16 steps in fp32 for it, two more for the product and the sum
        v = want * torch.sigmoid(want)
        bound = m.abs() * (1.1 * (K + 3) * F * size + 18 * F * v.abs()) + 2 * F * r.abs() + half(dt) * (r + v * m).abs()
        err = (y[a:b].double() - (r + v * m)).abs()
        assert bool((err <= bound).all()), f"y of group {g}: {float((err / bound.clamp_min(1e-300)).max()):.2f} bounds off"
    assert bool(torch.isnan(y[~inside]).all())
    before = mul.clone()
    lib.moe_linear(p, x, w, bias, off, mul, resid, mul, None)
    assert same_bits(mul[inside], y[inside]) and same_bits(mul[~inside], before[~inside])


@pytest.mark.parametrize("rows,K,N,G,dt", DX, ids=ids(DX))
def test_dx(rows, K, N, G, dt):
    print(f"[dx] {rows} {K} {N} {G} {dt}", flush=True)
    x, w, dy, off = tensors(rows, K, N, G, dt)
    p = lib.linear_problem(rows, K, N, G, dt)
    x.fill_(float("nan"))
    lib.moe_linear_backward(p, dy, None, w, off, None, None, x, None, None, None, lib.linear_workspace(p))
    for g, (a, b) in enumerate(spans(off, rows)):
        if b > a:
            dd, wd = dy[a:b].double(), w[g].double()
            check(x[a:b], dd @ wd, dd.abs() @ wd.abs(), N, dt, f"group {g}")


@pytest.mark.parametrize("rows,K,N,G,dt", DW, ids=ids(DW))
def test_dw(rows, K, N, G, dt):
    print(f"[dw] {rows} {K} {N} {G} {dt}", flush=True)
    x, w, dy, off = tensors(rows, K, N, G, dt)
    p = lib.linear_problem(rows, K, N, G, dt)
    w.fill_(float("nan"))
    lib.moe_linear_backward(p, dy, x, None, off, None, None, None, w, None, None, lib.linear_workspace(p))
    for g, (a, b) in enumerate(spans(off, rows)):
        dd, xd = dy[a:b].double().T.contiguous(), x[a:b].double()
        check(w[g], dd @ xd, dd.abs() @ xd.abs(), b - a, dt, f"group {g}")


@pytest.mark.parametrize("rows,K,N,G,dt", BOTH, ids=ids(BOTH))
def test_both_in_one_call(rows, K, N, G, dt):
    """Side by side in one launch, with the bias's sums: the bits of the calls for each alone."""
    print(f"[both] {rows} {K} {N} {G} {dt}", flush=True)
    x, w, dy, off = tensors(rows, K, N, G, dt)
    p = lib.linear_problem(rows, K, N, G, dt, "silu")
    z, ws = torch.randn((rows, N), device="cuda").to(DT[dt]), lib.linear_workspace(p)
    out = lambda: [torch.full_like(x, float("nan")), torch.full_like(w, float("nan")), torch.empty((G, N), device="cuda")]
    both = out()
    lib.moe_linear_backward(p, dy, x, w, off, None, z, *both, None, ws)
    for i in range(3):
        o = out()
        lib.moe_linear_backward(p, dy, x, w, off, None, z, *[t if i == n else None for n, t in enumerate(o)], None, ws)
        assert same_bits(o[i], both[i])
