"""moe_block_norm_backward where a workgroup takes several rounds of rows (the next round's loads go out ahead, its sums go
to the other half of their place, groups of a last round may have no row), where it takes all rows in one or two rounds
without a second launch, and where the mixed sums over a row cancel."""
import numpy as np
import pytest
import torch

import sparse_moe_layer_amd as lib
from block_bounds import DT, F, close, dev, half, np64, same_bits
from oracle import block
from test_parity_norm import EPS, STEPS, bounds_backward, oracle_gate, setup

pytestmark = pytest.mark.gpu

# At most 256 workgroups of 1 to 16 rows at a time: 2 to 7 rounds, the last one not full.  Chunks a thread: one, two and
# four, in both dtypes.
ROUNDS = [(1700, 2568, "bf16"), (600, 4104, "bf16"), (300, 8200, "bf16"), (9000, 72, "bf16"), (4100, 264, "bf16"),
          (1001, 1284, "f32"), (700, 2052, "f32"), (520, 4100, "f32"), (259, 16384, "f32"), (8200, 36, "f32")]
# Rows that one or two workgroups take at a time
FEW = [(3, 2560, "bf16"), (4, 2560, "bf16"), (5, 2560, "bf16"), (6, 2560, "bf16"), (7, 2560, "bf16"), (2, 4104, "bf16"),
       (20, 264, "bf16"), (12, 264, "bf16"), (33, 264, "bf16"), (17, 136, "f32"), (4, 1284, "f32"), (2, 4100, "f32")]


def gradients(p, d, gate, post, dro=True, dx=True):
    """Every gradient of one call, and its workspace's bytes NaN before it."""
    T, H, dt = p.T, p.H, d["f"].dtype
    ws = lib.norm_workspace(p).fill_(255)
    g = {n: dev(v) for n, v in d.items()}
    o = {n: torch.full((T, H), float("nan"), dtype=dt, device="cuda") for n in ("dresid", "df")}
    o["dg_pre"] = torch.full((H,), float("nan"), device="cuda") if dx else None
    o["dg_post"] = torch.full((H,), float("nan"), device="cuda") if post else None
    o["dgate"] = {"none": None, "token": torch.full((T,), float("nan"), device="cuda"),
                  "channel": torch.full((H,), float("nan"), device="cuda"),
                  "full": torch.full((T, H), float("nan"), dtype=dt, device="cuda")}[gate]
    lib.moe_block_norm_backward(p, g["dro"] if dro else None, g["dx"] if dx else None, g["f"], g["resid"] if dx else None,
                                g["g_post"], g["gate"], g["g_pre"] if dx else None, o["dresid"], o["df"], o["dg_post"],
                                o["dgate"], o["dg_pre"], ws)
    return o


def check(got, d, dt, gate, c, steps=STEPS):
    """Against the formulas in 64 bits, with an fp32 sum's error for every term, as the parity tests have it."""
    n64 = {n: np64(v) for n, v in d.items()}
    gt = oracle_gate(d, gate)
    want = block.block_norm_backward(n64["dro"], n64["dx"], n64["f"], n64["resid"], n64["g_post"], gt, n64["g_pre"], EPS, c)
    size = bounds_backward((n64["f"], n64["g_post"], gt, n64["g_pre"]), n64["dro"], n64["dx"], n64["resid"], gate, c)
    for n, v in got.items():
        if v is None:
            continue
        ref, s = want[n].reshape(v.shape), size[n].reshape(v.shape)
        rounding = F if v.dtype == torch.float32 and n.startswith("dg") else half(dt)
        close(v, ref, 4 * steps * F * s + rounding * np.abs(ref), n)


@pytest.mark.parametrize("post", [False, True], ids=["plain", "post"])
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("T,H,dt", ROUNDS + FEW, ids=["x".join(map(str, s)) for s in ROUNDS + FEW])
def test_rounds_of_rows(T, H, dt, gate, post):
    print(f"[norm rounds] {T} {H} {dt} {gate} {post}", flush=True)
    d, c = setup(T, H, dt, gate, post, 7), 0.75
    p = lib.norm_problem(T, H, dt, gate, EPS, c)
    got = gradients(p, d, gate, post)
    check(got, d, dt, gate, c)
    again = gradients(p, d, gate, post)  # a fixed order of the sums
    assert all(v is None or same_bits(v, again[n]) for n, v in got.items())


@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("T,H", [(40, 8192), (600, 1284)])
def test_gradients_along_the_residual(T, H, gate):
    """dx, f and the residual along one another: what dx sends through the norm cancels to eps times it, and so do the
    mixed sums over a row.  Errors are counted against the terms that cancel.  A row statistic here: at most 16 values a
    thread, 6 steps over lanes, 8 waves and the steps of a root and quotient, below 40."""
    gen = torch.Generator().manual_seed(H)
    d, c = setup(T, H, "f32", gate, True, 9), 0.75
    d["f"] = d["resid"] * torch.empty((T, 1)).uniform_(0.2, 0.6, generator=gen)
    d["dx"] = d["resid"] * torch.empty((T, 1)).uniform_(0.5, 2.0, generator=gen)
    d["g_pre"], d["g_post"] = torch.ones(H), torch.ones(H)
    d["dro"] = 1e-3 * d["dro"]
    p = lib.norm_problem(T, H, "f32", gate, EPS, c)
    check(gradients(p, d, gate, True), d, "f32", gate, c, steps=40)
