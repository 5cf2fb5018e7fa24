"""Tensors that begin at any 16 bytes of a larger one, one group of some of the rows, and the neighbours of every
output left as they were."""
import pytest
import torch

import sparse_moe_layer_amd as lib
from block_bounds import DT, same_bits

pytestmark = pytest.mark.gpu

PAD = 64  # values before and behind


class Views:
    """Tensors in the middle of larger ones, `at` units of 16 bytes past an aligned place, and plain copies of them."""

    def __init__(self, at, seed):
        self.at, self.gen, self.held = at, torch.Generator(device="cuda").manual_seed(seed), []

    def __call__(self, *shape, dt, fill=None):
        d = DT.get(dt, dt)
        n, q = 1, 16 // torch.empty(0, dtype=d).element_size()
        for v in shape:
            n *= v
        whole = torch.empty(n + 2 * PAD, dtype=d, device="cuda").normal_(generator=self.gen)
        view = whole[PAD + self.at * q:PAD + self.at * q + n].view(shape)
        values = torch.empty(shape, dtype=d, device="cuda").normal_(generator=self.gen)  # the same at every place
        view.copy_(values) if fill is None else view.fill_(fill)
        self.held.append((whole, view, whole.clone(), PAD + self.at * q, n))
        return view

    def untouched(self):
        """What lies around the tensors is as it was."""
        return all(same_bits(w[:a], b[:a]) and same_bits(w[a + n:], b[a + n:]) for w, _, b, a, n in self.held)


@pytest.mark.parametrize("at", [0, 1, 3])
@pytest.mark.parametrize("rows,K,N,G,dt", [(3, 264, 72, 1, "bf16"), (10, 520, 136, 4, "bf16"), (300, 264, 328, 2, "bf16"),
                                           (1490, 136, 1016, 1, "bf16"), (70, 132, 68, 3, "f32"), (300, 516, 260, 1, "f32")])
def test_linear(rows, K, N, G, dt, at):
    results = []
    for a in (0, at):
        v = Views(a, 7)
        x, w, bias, mul, resid, dy = v(rows, K, dt=dt), v(G, N, K, dt=dt), v(G, N, dt=dt), *(v(rows, N, dt=dt) for _ in range(3))
        y, z, dx, dw, dmul = (v(*s, dt=dt, fill=0) for s in ((rows, N), (rows, N), (rows, K), (G, N, K), (rows, N)))
        off = torch.linspace(0, rows, G + 1).int().cuda()
        p = lib.linear_problem(rows, K, N, G, dt, "silu")
        db, ws = torch.empty((G, N), device="cuda"), lib.linear_workspace(p)
        lib.moe_linear(p, x, w, bias, off, mul, resid, y, z)
        lib.moe_linear_backward(p, dy, x, w, off, mul, z, dx, dw, db, dmul, ws)
        assert v.untouched()
        results.append([t.clone() for t in (y, z, dx, dw, db, dmul)])
    assert all(same_bits(*t) for t in zip(*results))


@pytest.mark.parametrize("rows", [9, 200, 1500])
def test_one_group_of_some_rows(rows):
    """Offsets of a single group: the rows before and behind stay, and the results are those of a call for its rows."""
    K, N, a, b = 136, 264, 2, rows - 3
    v = Views(1, 9)
    x, w, dy, z = v(rows, K, dt="bf16"), v(1, N, K, dt="bf16"), v(rows, N, dt="bf16"), v(rows, N, dt="bf16")
    off = torch.tensor([a, b], dtype=torch.int32, device="cuda")
    out = []
    for part in (False, True):
        s = slice(a, b) if part else slice(0, rows)
        n = b - a if part else rows
        p = lib.linear_problem(n, K, N, 1, "bf16", "gelu")
        t = [torch.full((rows, c), 3.0, dtype=torch.bfloat16, device="cuda") for c in (N, K)]
        dw, db = torch.empty_like(w), torch.empty((1, N), device="cuda")
        o = None if part else off
        lib.moe_linear(p, x[s], w, None, o, None, None, t[0][s], None)
        lib.moe_linear_backward(p, dy[s], x[s], w, o, None, z[s], t[1][s], dw, db, None, lib.linear_workspace(p))
        for q in t:
            assert bool((q[:a] == 3.0).all()) and bool((q[b:] == 3.0).all())
        out.append(([q[a:b] for q in t], dw, db))
    # the tiles may differ with the number of rows, and with them the order of the sums: each result is off by (n + 2)
    # fp32 steps of the sum of its terms' sizes (GELU and its slope at most 1.13 of theirs) and half a step of bf16
    xa, wa, da = x.float().abs(), w[0].float().abs(), 1.13 * dy.float().abs()
    sizes = ((K, 1.13 * xa @ wa.T.contiguous()), (N, da @ wa), (rows, da.T.contiguous() @ xa))
    for (n, size), q, r in zip(sizes, out[0][0] + [out[0][1][0]], out[1][0] + [out[1][1][0]]):
        assert torch.allclose(q.float(), r.float(), rtol=2.0 ** -7, atol=2 * (n + 2) * 2.0 ** -24 * float(size.max()))
    assert torch.allclose(out[0][2], out[1][2], rtol=0, atol=2 * (rows + 2) * 2.0 ** -24 * float(da.sum(0).max()))


@pytest.mark.parametrize("at", [0, 1, 2])
@pytest.mark.parametrize("T,H,dt", [(3, 264, "bf16"), (70, 2568, "bf16"), (33, 1284, "f32")])
@pytest.mark.parametrize("gate", ["channel", "full"])
def test_norm(T, H, dt, gate, at):
    results = []
    for a in (0, at):
        v = Views(a, 11)
        f, resid, dro, dx = (v(T, H, dt=dt) for _ in range(4))
        g_post, g_pre = v(H, dt=dt), v(H, dt=dt)
        g = v(H, dt=dt) if gate == "channel" else v(T, H, dt=dt)
        r, x, dresid, df = (v(T, H, dt=dt, fill=0) for _ in range(4))
        dg = v(H, dt="f32", fill=0) if gate == "channel" else v(T, H, dt=dt, fill=0)
        dpost, dpre = v(H, dt="f32", fill=0), v(H, dt="f32", fill=0)
        p = lib.norm_problem(T, H, dt, gate)
        lib.moe_block_norm(p, f, resid, g_post, g, g_pre, r, x)
        lib.moe_block_norm_backward(p, dro, dx, f, r, g_post, g, g_pre, dresid, df, dpost, dg, dpre, lib.norm_workspace(p))
        assert v.untouched()
        results.append([t.clone() for t in (r, x, dresid, df, dg, dpost, dpre)])
    assert all(same_bits(*t) for t in zip(*results))


@pytest.mark.parametrize("at", [0, 1, 2])
@pytest.mark.parametrize("T,H,k,dt", [(5, 72, 3, "bf16"), (40, 2568, 10, "bf16"), (9, 1100, 17, "f32")])
def test_rows(T, H, k, dt, at):
    results = []
    for a in (0, at):
        v = Views(a, 13)
        x, dxs, dout, y = v(T, H, dt=dt), v(T * k, H, dt=dt), v(T, H, dt=dt), v(T * k, H, dt=dt)
        w = v(T, k, dt="f32")
        pos = torch.randperm(T * k, generator=v.gen, device="cuda").int().view(T, k)
        xs, dx, dy, dw, dw2 = (v(*s, dt=d, fill=0) for s, d in (((T * k, H), dt), ((T, H), dt), ((T * k, H), dt), ((T, k), "f32"), ((T, k), "f32")))
        p = lib.problem(T, H, 64, k, 8, act=dt, wdt=dt)
        lib.moe_permute(p, x, pos, w, xs)
        lib.moe_permute_backward(p, dxs, pos, w, x, dx, dw)
        lib.moe_combine_backward(p, dout, y, pos, w, None, None, dy, dw2, None, None)
        assert v.untouched()
        results.append([t.clone() for t in (xs, dx, dw, dy, dw2)])
    assert all(same_bits(*t) for t in zip(*results))
