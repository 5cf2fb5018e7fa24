"""moe_block_norm and its gradients against the fp64 oracle (oracle/block.py)."""
import numpy as np
import pytest
import torch

import sparse_moe_layer_amd as lib
from block_bounds import DEPTH, DT, F, close, dev, half, normal, np64, same_bits
from oracle import block

pytestmark = pytest.mark.gpu

SHAPES = [(1, 8, "bf16"), (1, 8192, "bf16"), (3, 4, "f32"), (2, 16384, "f32"), (2, 16384, "bf16"), (37, 2560, "bf16"),
          (5, 8200, "bf16"), (130, 1284, "f32"), (1030, 72, "bf16"), (600, 264, "f32"), (9, 4104, "f32"), (3, 2056, "f32")]
IDS = ["x".join(map(str, s)) for s in SHAPES]
EPS = 1e-6


def setup(T, H, dt, gate, post, seed=0):
    gen = torch.Generator().manual_seed(100 * T + H + seed)
    d = {n: normal(gen, (T, H), dt, std) for n, std in (("f", 0.7), ("resid", 2.0), ("dro", 1.0), ("dx", 1.0))}
    d["g_post"] = normal(gen, (H,), dt, 0.1, 1.0) if post else None
    d["g_pre"] = normal(gen, (H,), dt, 0.1, 1.0)
    d["gate"] = {"none": lambda: None, "token": lambda: torch.randn(T, generator=gen),
                 "channel": lambda: normal(gen, (H,), dt), "full": lambda: normal(gen, (T, H), dt)}[gate]()
    return d


def oracle_gate(d, gate):
    g = np64(d["gate"])
    return g[None, :] if gate == "channel" else g


# fp32 steps of a row statistic: the sum (half of it after the square root), the mean, root, quotient and products
STEPS = DEPTH


@pytest.mark.parametrize("post", [False, True], ids=["plain", "post"])
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("T,H,dt", SHAPES, ids=IDS)
def test_block_norm(T, H, dt, gate, post):
    print(f"[block_norm] {T} {H} {dt} {gate} {post}", flush=True)
    d, c = setup(T, H, dt, gate, post), 0.75
    p = lib.norm_problem(T, H, dt, gate, EPS, c)
    out, x = (torch.empty((T, H), dtype=DT[dt], device="cuda") for _ in range(2))
    g = {n: dev(v) for n, v in d.items()}
    lib.moe_block_norm(p, g["f"], g["resid"], g["g_post"], g["gate"], g["g_pre"], out, x)
    a = [np64(d["f"]), np64(d["resid"]), np64(d["g_post"]), oracle_gate(d, gate), np64(d["g_pre"])]
    r, want = block.block_norm(*a, EPS, c)
    part = block.block_norm(*[None if v is None else np.abs(v) for v in a], EPS, c)[0]  # sizes of the two terms
    rms = np.sqrt((r * r).mean(1, keepdims=True) + EPS)
    r_err = STEPS * F * part
    close(out, r, r_err + half(dt) * np.abs(r), "resid_out")
    # x: the residual's error over its norm, and the norm's own relative error, which the row's errors move too
    rel = np.sqrt((r_err * r_err).mean(1, keepdims=True)) / rms + STEPS * F
    close(x, want, np.abs(a[4]) * r_err / rms + (rel + half(dt)) * np.abs(want), "x")
    # in place, over resid and over f; without x; without resid_out
    for n in ("resid", "f"):
        o = dict(g, **{n: g[n].clone()})
        x2 = torch.empty_like(x)
        lib.moe_block_norm(p, o["f"], o["resid"], g["g_post"], g["gate"], g["g_pre"], o[n], x2)
        assert same_bits(o[n], out) and same_bits(x2, x), n
    o = torch.empty_like(out)
    lib.moe_block_norm(p, g["f"], g["resid"], g["g_post"], g["gate"], None, o, None)
    assert same_bits(o, out)
    lib.moe_block_norm(p, g["f"], g["resid"], g["g_post"], g["gate"], g["g_pre"], None, o)
    assert same_bits(o, x)


def bounds_backward(a, dro, dx, resid_out, gate, c):
    """Sizes of the terms of every gradient, from the formulas with every term's size."""
    f, g_post, g, g_pre = a
    T = dro.shape[0]
    one = np.abs
    rms = lambda v: np.sqrt((v * v).mean(1, keepdims=True) + EPS)
    rr = 1 / rms(resid_out)
    u = one(dx * g_pre)
    M = one(dro) + rr * (u + one(resid_out) * rr ** 2 * (u * one(resid_out)).mean(1, keepdims=True))
    gt = 1.0 if g is None else one(g[:, None] if g.ndim == 1 else g)
    dn = gt * M
    out = {"dresid": c * M, "dg_pre": (one(dx * resid_out) * rr).sum(0)}
    if g_post is None:
        out["df"], n = dn, one(f)
    else:
        q = 1 / rms(f)
        v = dn * one(g_post)
        out["df"] = q * (v + one(f) * q ** 2 * (v * one(f)).mean(1, keepdims=True))
        out["dg_post"] = (dn * one(f) * q).sum(0)
        n = one(f) * q * one(g_post)
    each = n * M
    if gate != "none":
        out["dgate"] = {"token": each.sum(1), "channel": each.sum(0), "full": each}[gate]
    return out


@pytest.mark.parametrize("post", [False, True], ids=["plain", "post"])
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("T,H,dt", SHAPES, ids=IDS)
def test_block_norm_backward(T, H, dt, gate, post):
    print(f"[block_norm_backward] {T} {H} {dt} {gate} {post}", flush=True)
    d, c = setup(T, H, dt, gate, post, 1), 0.75
    p = lib.norm_problem(T, H, dt, gate, EPS, c)
    ws = lib.norm_workspace(p)
    g = {n: dev(v) for n, v in d.items()}

    def run(dro, dx, dresid=None):
        ws.fill_(255)  # NaN bits: whatever the call reads of it, it has written
        o = {n: torch.full((T, H), float("nan"), dtype=DT[dt], device="cuda") for n in ("dresid", "df")}
        if dresid is not None:
            o["dresid"] = dresid
        o["dg_pre"] = torch.empty(H, device="cuda") if dx is not None else None
        o["dg_post"] = torch.empty(H, device="cuda") if post else None
        o["dgate"] = {"none": lambda: None, "token": lambda: torch.empty(T, device="cuda"),
                      "channel": lambda: torch.empty(H, device="cuda"),
                      "full": lambda: torch.empty((T, H), dtype=DT[dt], device="cuda")}[gate]()
        lib.moe_block_norm_backward(p, dro, dx, g["f"], g["resid"] if dx is not None else None, g["g_post"], g["gate"],
                                    g["g_pre"] if dx is not None else None, o["dresid"], o["df"], o["dg_post"],
                                    o["dgate"], o["dg_pre"], ws)
        return o

    n64 = {n: np64(v) for n, v in d.items()}
    gt = oracle_gate(d, gate)
    zero = np.zeros((T, H))
    for dro, dx in ((True, True), (True, False), (False, True)):
        got = run(g["dro"] if dro else None, g["dx"] if dx else None)
        want = block.block_norm_backward(n64["dro"] if dro else None, n64["dx"] if dx else None, n64["f"], n64["resid"],
                                         n64["g_post"], gt, n64["g_pre"], EPS, c)
        size = bounds_backward((n64["f"], n64["g_post"], gt, n64["g_pre"]), n64["dro"] if dro else zero,
                               n64["dx"] if dx else zero, n64["resid"], gate, c)
        for n, v in got.items():
            if v is None:
                continue
            # two row statistics, one on the other's result; then the sums over rows or columns
            err = 4 * STEPS * F * size[n]
            if v.dtype == torch.float32 and n.startswith("dg"):
                err = err + F * np.abs(want[n].reshape(size[n].shape))
            else:
                err = err + half(dt) * np.abs(want[n])
            if n == "dgate":
                close(v, want[n].reshape(v.shape), err.reshape(v.shape), n)
            else:
                close(v, want[n], err, n)
    # in place over either incoming gradient, bit for bit
    ref = run(g["dro"], g["dx"])
    a, b = g["dro"].clone(), g["dx"].clone()
    over = run(a, g["dx"], dresid=a)
    assert all(v is None or same_bits(v, ref[n]) for n, v in over.items())
    over = run(g["dro"], b, dresid=b)
    assert all(v is None or same_bits(v, ref[n]) for n, v in over.items())


@pytest.mark.parametrize("T,H,dt", [(5, 264, "f32"), (1100, 136, "bf16")])
def test_the_norm_before_the_first_block(T, H, dt):
    """f None: the residual scaled and its norm, and back."""
    d, c = setup(T, H, dt, "none", False, 2), 0.5
    p = lib.norm_problem(T, H, dt, "none", EPS, c)
    x, out = (torch.empty((T, H), dtype=DT[dt], device="cuda") for _ in range(2))
    lib.moe_block_norm(p, None, dev(d["resid"]), None, None, dev(d["g_pre"]), out, x)
    r, want = block.block_norm(None, np64(d["resid"]), None, None, np64(d["g_pre"]), EPS, c)
    close(out, r, (half(dt) + F) * np.abs(r), "resid_out")
    close(x, want, (half(dt) + STEPS * F) * np.abs(want), "x")
    dresid, dg = torch.empty_like(x), torch.empty(H, device="cuda")
    ws = lib.norm_workspace(p)
    lib.moe_block_norm_backward(p, dev(d["dro"]), dev(d["dx"]), None, dev(d["resid"]), None, None, dev(d["g_pre"]), dresid,
                                None, None, None, dg, ws)
    want = block.block_norm_backward(np64(d["dro"]), np64(d["dx"]), None, np64(d["resid"]), None, None, np64(d["g_pre"]), EPS, c)
    size = bounds_backward((np.zeros((T, H)), None, None, np64(d["g_pre"])), np64(d["dro"]), np64(d["dx"]), np64(d["resid"]),
                           "none", c)
    close(dresid, want["dresid"], 4 * STEPS * F * size["dresid"] + half(dt) * np.abs(want["dresid"]), "dresid")
    close(dg, want["dg_pre"], 4 * STEPS * F * size["dg_pre"], "dg_pre")


def test_zero_rows_large_rows_and_nan_rows():
    """A row of zeros has the norm sqrt(eps); rows around 1e18 do not overflow fp32's squares; NaN stays in its row."""
    T, H = 5, 520
    d = setup(T, H, "f32", "none", True, 3)
    d["f"][0] = 0.0
    d["resid"][0] = 0.0
    d["f"][1] *= 1e17
    d["resid"][1] *= 1e17
    d["f"][3, 7] = float("nan")
    d["resid"][4, 519] = float("inf")
    p = lib.norm_problem(T, H, "f32", "none", EPS, 1.0)
    out, x = torch.empty((T, H), device="cuda"), torch.empty((T, H), device="cuda")
    lib.moe_block_norm(p, dev(d["f"]), dev(d["resid"]), dev(d["g_post"]), None, dev(d["g_pre"]), out, x)
    r, want = block.block_norm(
        np64(d["f"][:3]), np64(d["resid"][:3]), np64(d["g_post"]), None, np64(d["g_pre"]), EPS, 1.0)
    size = block.block_norm(np.abs(np64(d["f"][:3])), np.abs(np64(d["resid"][:3])), np.abs(np64(d["g_post"])), None, None,
                            EPS, 1.0)[0]
    close(out[:3], r, 2 * STEPS * F * size, "resid_out")
    assert torch.equal(x[0], torch.zeros(H, device="cuda"))
    close(x[:3], want, 8 * STEPS * F * np.abs(np64(d["g_pre"])) * size / np.sqrt((r * r).mean(1, keepdims=True) + EPS), "x")
    assert torch.isnan(x[3]).all() and not torch.isfinite(x[4]).all()
    assert torch.isfinite(out[4]).sum() == H - 1
