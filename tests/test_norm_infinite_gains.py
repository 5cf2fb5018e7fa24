"""Gradients of the block norm with an infinite gain or gate: what the formulas have finite is finite, and the sums over
tokens have an infinity or NaN as the formulas do, also where the last workgroup has fewer rows than it takes at a time.

Within a row that the infinity reaches, an infinity may be NaN: mean(q dr) over the row is formed as s3 + rr (s4 - mr s5),
whose terms are infinite where one value of q is, and infinity minus infinity is NaN where the mean itself is infinite.
An infinite gain before the next block reaches every value of dr, so the sums over tokens too."""
import numpy as np
import pytest
import torch

import sparse_moe_layer_amd as lib
from block_bounds import DT, dev, np64
from oracle import block

pytestmark = pytest.mark.gpu

EPS, INF = 1e-6, float("inf")


def kinds(v):
    """0 for a finite value, 1 and -1 for the infinities, 2 for NaN."""
    v = np.asarray(v, dtype=np.float64)
    return np.where(np.isnan(v), 2, np.where(np.isinf(v), np.sign(v), 0))


@pytest.mark.parametrize("gate,where", [(g, w) for g in ("none", "channel", "full") for w in ("g_post", "gate", "g_pre")
                                        if (g, w) != ("none", "gate")])
@pytest.mark.parametrize("T,H,dt", [(1, 72, "bf16"), (37, 72, "bf16"), (9, 264, "f32"), (1030, 136, "bf16"), (5, 2560, "bf16")])
def test_one_infinite_column(T, H, dt, gate, where):
    print(f"[infinite gain] {T} {H} {dt} {gate} {where}", flush=True)
    gen = torch.Generator().manual_seed(T + H)
    # one sign throughout, so that no sum has infinities of both
    d = {n: torch.empty(s).uniform_(0.5, 1.5, generator=gen).to(DT[dt])
         for n, s in (("f", (T, H)), ("resid", (T, H)), ("dro", (T, H)), ("dx", (T, H)), ("g_post", (H,)), ("g_pre", (H,)))}
    d["gate"] = {"none": None, "channel": torch.ones(H, dtype=DT[dt]), "full": torch.ones((T, H), dtype=DT[dt])}[gate]
    d[where][..., 3] = INF
    p = lib.norm_problem(T, H, dt, gate, EPS, 1.0)
    g = {n: dev(v) for n, v in d.items()}
    o = {n: torch.zeros((T, H), dtype=DT[dt], device="cuda") for n in ("dresid", "df")}
    o["dg_post"], o["dg_pre"] = torch.zeros(H, device="cuda"), torch.zeros(H, device="cuda")
    o["dgate"] = {"none": None, "channel": torch.zeros(H, device="cuda"), "full": torch.zeros((T, H), dtype=DT[dt], device="cuda")}[gate]
    lib.moe_block_norm_backward(p, g["dro"], g["dx"], g["f"], g["resid"], g["g_post"], g["gate"], g["g_pre"], o["dresid"], o["df"],
                                o["dg_post"], o["dgate"], o["dg_pre"], lib.norm_workspace(p))
    n64 = {n: np64(v) for n, v in d.items()}
    gt = n64["gate"][None, :] if gate == "channel" else n64["gate"]
    with np.errstate(invalid="ignore"):
        want = block.block_norm_backward(n64["dro"], n64["dx"], n64["f"], n64["resid"], n64["g_post"], gt, n64["g_pre"], EPS, 1.0)
    for n, v in o.items():
        if v is None:
            continue
        got, ref = kinds(np64(v)), kinds(want[n].reshape(v.shape))
        assert not got[ref == 0].any(), n
        if n in ("dg_post", "dg_pre") or (n == "dgate" and gate == "channel"):
            assert got[ref != 0].all() if where == "g_pre" else np.array_equal(got, ref), n
