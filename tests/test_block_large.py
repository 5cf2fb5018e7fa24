"""More rows than one dimension of a grid has threads for, and rows past 2 GiB."""
import pytest
import torch

import sparse_moe_layer_amd as lib

pytestmark = pytest.mark.gpu


def parts(n, step=1 << 24):
    return ((a, min(a + step, n)) for a in range(0, n, step))


def test_norm_of_very_many_short_rows():
    T, H = (1 << 26) + 37, 8
    p = lib.norm_problem(T, H, "bf16", "none", 1e-6, 0.5)
    resid = torch.empty((T, H), dtype=torch.bfloat16, device="cuda").normal_()
    out = torch.zeros_like(resid)
    lib.moe_block_norm(p, None, resid, None, None, None, out, None)
    for a, b in parts(T):  # a half of a bf16 is exact
        assert torch.equal(out[a:b], resid[a:b] * 0.5)


def test_gradients_of_very_many_assignments():
    T, H, k = (1 << 22) + 3, 4, 64
    with pytest.raises(lib.MoEError):  # more than the layer's hidden rows may be
        lib.moe_combine_backward(lib.problem(T, 8, k, k, 8), *[None] * 10)
    p = lib.problem(T, H, k, k, 4, act="f32", wdt="f32")
    dout = torch.empty((T, H), device="cuda").normal_()
    y = torch.empty((T * k, H), device="cuda").normal_()
    pos = torch.arange(T * k, dtype=torch.int32, device="cuda").flip(0).view(T, k).contiguous()
    w = torch.full((T, k), 2.0, device="cuda")
    dy, dw = torch.zeros_like(y), torch.zeros((T, k), device="cuda")
    lib.moe_combine_backward(p, dout, y, pos, w, None, None, dy, dw, None, None)
    for a, b in parts(T, 1 << 18):
        rows = pos[a:b].view(-1).long()
        d = dout[a:b].repeat_interleave(k, 0)
        assert torch.equal(dy[rows], d * 2)
        want = (y[rows].double() * d.double())
        err = (dw[a:b].view(-1).double() - want.sum(1)).abs()
        assert bool((err <= 10 * 2.0 ** -24 * want.abs().sum(1)).all())


def test_permute_past_two_gib():
    """Rows of xs beyond 2^31 bytes and 2^31 values."""
    T, H, k = 40000, 8192, 10
    p = lib.problem(T, H, 64, k, 8)
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda").normal_()
    pos = torch.randperm(T * k, device="cuda").int().view(T, k)
    xs = torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda")
    lib.moe_permute(p, x, pos, None, xs)
    for a, b in parts(T, 4000):
        assert torch.equal(xs[pos[a:b].long()], x[a:b, None].expand(-1, k, -1))
    dx, dw = torch.empty_like(x), torch.empty((T, k), device="cuda")
    w = torch.zeros((T, k), device="cuda")
    w[:, 3] = 1.0
    lib.moe_permute_backward(p, xs, pos, w, x, dx, dw)
    assert torch.equal(dx, x)
    for a, b in parts(T, 4000):
        want = (x[a:b].double() ** 2).sum(1, keepdim=True)
        assert bool(((dw[a:b].double() - want).abs() <= 128 * 2.0 ** -24 * want).all())


def test_linear_past_two_gib():
    """Outputs and weights beyond 2^31 bytes: the last rows and matrices as in a call of their own."""
    rows, K, N, G = 300, 2048, 4096, 300
    w = torch.empty((G, N, K), dtype=torch.bfloat16, device="cuda").normal_(0, K ** -0.5)
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda").normal_()
    off = torch.arange(G + 1, dtype=torch.int32, device="cuda")
    y = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    lib.moe_linear(lib.linear_problem(rows, K, N, G), x, w, None, off, None, None, y, None)
    for g in (0, 127, 128, 255, 256, 299):
        xd, wd = x[g:g + 1].double(), w[g].double().T.contiguous()
        want = xd @ wd
        assert bool(((y[g:g + 1].double() - want).abs() <= (K + 2) * 2.0 ** -24 * (xd.abs() @ wd.abs())
                     + 2.0 ** -8 * want.abs()).all())
    p = lib.linear_problem(rows, K, N, G)
    ws = lib.linear_workspace(p)
    dx, dw = torch.empty_like(x), torch.full_like(w, float("nan"))
    lib.moe_linear_backward(p, y, x, w, off, None, None, dx, dw, None, None, ws)
    for g in (0, 127, 128, 255, 256, 299):  # one row: products rounded once
        assert torch.equal(dw[g], (y[g].float()[:, None] * x[g].float()[None]).bfloat16())
        yd, wd = y[g:g + 1].double(), w[g].double()
        want = yd @ wd
        assert bool(((dx[g:g + 1].double() - want).abs() <= (N + 2) * 2.0 ** -24 * (yd.abs() @ wd.abs())
                     + 2.0 ** -8 * want.abs()).all())
    del w, dw
    rows, K, N = 300000, 64, 4096
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.empty((1, N, K), dtype=torch.bfloat16, device="cuda").normal_()
    y = torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    lib.moe_linear(lib.linear_problem(rows, K, N), x, w, None, None, None, None, y, None)
    wd = w[0].double().T.contiguous()
    for a, b in parts(rows, 20000):
        xd = x[a:b].double()
        want = xd @ wd
        assert bool(((y[a:b].double() - want).abs() <= (K + 2) * 2.0 ** -24 * (xd.abs() @ wd.abs())
                     + 2.0 ** -8 * want.abs()).all())
