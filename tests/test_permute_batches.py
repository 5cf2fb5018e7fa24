"""permute's gradient for every number of assignments around the sizes of a batch of rows, some without a row."""
import numpy as np
import pytest
import torch

import sparse_moe_layer_amd as lib
from block_bounds import DT, F, close, half, normal, np64
from oracle import block

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("weighted", [False, True], ids=["plain", "weighted"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("k", list(range(1, 13)) + [15, 16, 17, 24, 25, 64])
def test_dx_alone(k, dt, weighted):
    T, H = 13, 136
    print(f"[permute batches] {k} {dt} {weighted}", flush=True)
    gen = torch.Generator().manual_seed(k)
    R = T * k
    pos = torch.randperm(R, generator=gen).int().view(T, k)
    pos[torch.rand(T, k, generator=gen) < 0.2] = R
    dxs = normal(gen, (R, H), dt)
    dxs[0] = float("nan")  # row 0 belongs to one token at most
    w = torch.rand(T, k, generator=gen) if weighted else None
    p = lib.problem(T, H, 64, k, 8, act=dt, wdt=dt)
    dx = torch.empty((T, H), dtype=DT[dt], device="cuda")
    lib.moe_permute_backward(p, dxs.cuda(), pos.cuda(), None if w is None else w.cuda(), None, dx, None)
    want = block.permute_backward(np64(dxs), pos.numpy(), None if w is None else np64(w))[0]
    size = block.permute_backward(np.abs(np64(dxs)), pos.numpy(), None if w is None else np64(w))[0]
    bad = np.isnan(want).any(1)
    assert bad.sum() <= 1 and np.array_equal(np.isnan(np64(dx)).all(1), bad)
    close(dx[torch.from_numpy(~bad).cuda()], want[~bad], ((k + 1) * F * size + half(dt) * np.abs(want))[~bad], "dx")
