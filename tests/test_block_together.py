"""The calls of a trained block one after the other, forward and backward, as a user's program runs them: the norm
behind the block before, routing and dispatch, rows to expert order, SwiGLU experts and a shared one from grouped and
dense products, the combine, the next norm.  Against the same chain in fp64, eagerly, on other streams, from two
threads and in captured graphs.

How far the results may be: the chain in fp64 runs again with every tensor that a call stores off by up to the
rounding of its dtype (and fp32's sums), at random; the root mean square deviation of a result over eight such runs
is what the roundings make of it, and four times that the bound.
"""
import threading

import numpy as np
import pytest
import torch

import sparse_moe_layer_amd as lib
from block_bounds import DT, F, half, normal, np64, same_bits
from oracle import block

EPS, SCALE = 1e-6, 0.5
# T, H, E, k, I, I_shared, dtype
CASES = [(1, 64, 8, 2, 32, 64, "bf16"), (37, 136, 6, 3, 72, 40, "bf16"), (700, 256, 16, 4, 128, 128, "bf16"),
         (5, 36, 4, 2, 20, 12, "f32"), (150, 132, 8, 2, 68, 36, "f32")]
IDS = ["x".join(map(str, c)) for c in CASES]
GRADS = ["resid", "f", "gate1", "g_post1", "g_pre1", "w_gate", "w_up", "w_down", "sh_gate", "sh_up", "sh_down", "topk_w",
         "logit", "g_post2", "g_pre2"]


def inputs(T, H, E, k, I, Is, dt, seed=0):
    gen = torch.Generator().manual_seed(T + H + seed)
    n = lambda *s, std=1.0, mean=0.0: normal(gen, s, dt, std, mean)
    return {"resid": n(T, H, std=2.0), "f": n(T, H), "gate1": torch.randn(T, generator=gen),
            "g_post1": n(H, std=0.1, mean=1.0), "g_pre1": n(H, std=0.1, mean=1.0), "w_router": n(E, H),
            "sh_gate_w": n(H, std=H ** -0.5), "w_gate": n(E, I, H, std=H ** -0.5), "w_up": n(E, I, H, std=H ** -0.5),
            "w_down": n(E, H, I, std=I ** -0.5), "sh_gate": n(1, Is, H, std=H ** -0.5),
            "sh_up": n(1, Is, H, std=H ** -0.5), "sh_down": n(1, H, Is, std=Is ** -0.5),
            "g_post2": n(H, std=0.1, mean=1.0), "g_pre2": n(H, std=0.1, mean=1.0), "dresid": n(T, H), "dx": n(T, H)}


def chain64(d, pos, off, rnd=lambda v: v):
    """Outputs and gradients in fp64 (the routing's weights and logits are inputs); rnd: what each store does."""
    T, H = d["resid"].shape
    R = pos.size
    row = lambda f, *a: tuple(rnd(v) for v in f(*a))
    r1, x = row(block.block_norm, d["f"], d["resid"], d["g_post1"], d["gate1"], d["g_pre1"], EPS, SCALE)
    xs = block.permute(x, pos, None, np.zeros((R, H)))
    up = rnd(block.linear(xs, d["w_up"], None, off, None, None, "none")[0])
    h, zg = row(block.linear, xs, d["w_gate"], None, off, up, None, "silu")
    y = rnd(block.linear(h, d["w_down"], None, off, None, None, "none")[0])
    s_up = rnd(block.linear(x, d["sh_up"], None, None, None, None, "none")[0])
    s_h, s_zg = row(block.linear, x, d["sh_gate"], None, None, s_up, None, "silu")
    s_y = rnd(block.linear(s_h, d["sh_down"], None, None, None, None, "none")[0])
    out = rnd(block.combine(y, pos, d["topk_w"], s_y, d["logit"]))
    r2, x2 = row(block.block_norm, out, r1, d["g_post2"], None, d["g_pre2"], EPS, SCALE)
    g = {}
    b = block.block_norm_backward(d["dresid"], d["dx"], out, r2, d["g_post2"], None, d["g_pre2"], EPS, SCALE)
    g["g_post2"], g["g_pre2"] = b["dg_post"], b["dg_pre"]
    dr1, dout = rnd(b["dresid"]), rnd(b["df"])
    dy, g["topk_w"], ds_y, g["logit"] = block.combine_backward(dout, y, pos, d["topk_w"], np.zeros((R, H)), s_y, d["logit"])
    dy, ds_y = rnd(dy), rnd(ds_y)

    def swiglu(dy, xs, off, up, h, zg, w_gate, w_up, w_down):
        dh, dwd, _, _ = block.linear_backward(dy, h, w_down, off, None, None, "none")
        dh = rnd(dh)
        dz = rnd(dh * up * block.act_slope("silu", zg))  # dz is stored too
        dxg, dwg, _, _ = block.linear_backward(dz, xs, w_gate, off, None, None, "none")
        dup = rnd(dh * block.act("silu", zg))
        dxu, dwu, _, _ = block.linear_backward(dup, xs, w_up, off, None, None, "none")
        return rnd(rnd(dxg) + rnd(dxu)), rnd(dwg), rnd(dwu), rnd(dwd)

    dxs, g["w_gate"], g["w_up"], g["w_down"] = swiglu(dy, xs, off, up, h, zg, d["w_gate"], d["w_up"], d["w_down"])
    ds_x, g["sh_gate"], g["sh_up"], g["sh_down"] = swiglu(ds_y, x, None, s_up, s_h, s_zg, d["sh_gate"], d["sh_up"], d["sh_down"])
    dx = rnd(rnd(block.permute_backward(dxs, pos, None)[0]) + ds_x)
    b = block.block_norm_backward(dr1, dx, d["f"], r1, d["g_post1"], d["gate1"], d["g_pre1"], EPS, SCALE)
    g["resid"], g["f"], g["gate1"] = rnd(b["dresid"]), rnd(b["df"]), b["dgate"]
    g["g_post1"], g["g_pre1"] = b["dg_post"], b["dg_pre"]
    return r2, x2, g


class Block:
    """The chain on the GPU: tensors, outputs and workspaces of one user."""

    def __init__(self, d, T, H, E, k, I, Is, dt):
        self.d = {n: v.cuda() for n, v in d.items()}
        self.dims, self.R = (T, H, E, k, I, Is, dt), T * k
        e = lambda *s: torch.empty(s, dtype=DT[dt], device="cuda")
        f = lambda *s: torch.empty(s, device="cuda")
        i = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
        R = T * k
        self.p = lib.problem(T, H, E, k, I, Is, dt, dt)
        self.n1 = lib.norm_problem(T, H, dt, "token", EPS, SCALE)
        self.n2 = lib.norm_problem(T, H, dt, "none", EPS, SCALE)
        self.t = {"r1": e(T, H), "x": e(T, H), "ids": i(T, k), "w": f(T, k), "logit": f(T), "off": i(E + 1), "order": i(R),
                  "pos": i(T, k), "xs": e(R, H), "out": e(T, H), "r2": e(T, H), "x2": e(T, H), "dr1": e(T, H),
                  "dout": e(T, H), "dy": e(R, H), "ds_y": e(T, H), "dx": e(T, H), "moe_ws": lib.workspace(self.p),
                  "ws1": lib.norm_workspace(self.n1), "ws2": lib.norm_workspace(self.n2)}
        self.ffn = []
        for rows, G, inner, off, names in ((R, E, I, self.t["off"], ("w_gate", "w_up", "w_down")),
                                           (T, 1, Is, None, ("sh_gate", "sh_up", "sh_down"))):
            q = {"pu": lib.linear_problem(rows, H, inner, G, dt), "pg": lib.linear_problem(rows, H, inner, G, dt, "silu"),
                 "pd": lib.linear_problem(rows, inner, H, G, dt), "off": off, "names": names, "up": e(rows, inner),
                 "h": e(rows, inner), "z": e(rows, inner), "y": e(rows, H), "dh": e(rows, inner), "dup": e(rows, inner),
                 "dxg": e(rows, H), "dxu": e(rows, H)}
            q["ws"] = torch.empty(max(lib.moe_linear_workspace_bytes(q[n]) for n in ("pu", "pg", "pd")), dtype=torch.uint8,
                                  device="cuda")
            self.ffn.append(q)
        self.g = {n: f(T) if n in ("gate1", "logit") else f(T, k) if n == "topk_w" else f(H) if n[:2] == "g_" else
                  torch.empty_like(self.d[n]) for n in GRADS}

    def forward(self, s=None):
        d, t = self.d, self.t
        lib.moe_block_norm(self.n1, d["f"], d["resid"], d["g_post1"], d["gate1"], d["g_pre1"], t["r1"], t["x"], s)
        lib.moe_route(self.p, t["x"], d["w_router"], d["sh_gate_w"], t["ids"], t["w"], t["logit"], t["moe_ws"], s)
        lib.moe_dispatch(self.p, t["ids"], t["off"], t["order"], t["pos"], t["moe_ws"], s)
        lib.moe_permute(self.p, t["x"], t["pos"], None, t["xs"], s)
        for q, x in zip(self.ffn, (t["xs"], t["x"])):
            gate, up, down = (d[n] for n in q["names"])
            lib.moe_linear(q["pu"], x, up, None, q["off"], None, None, q["up"], None, s)
            lib.moe_linear(q["pg"], x, gate, None, q["off"], q["up"], None, q["h"], q["z"], s)
            lib.moe_linear(q["pd"], q["h"], down, None, q["off"], None, None, q["y"], None, s)
        lib.moe_combine(self.p, self.ffn[0]["y"], t["pos"], t["w"], self.ffn[1]["y"], t["logit"], t["out"], s)
        lib.moe_block_norm(self.n2, t["out"], t["r1"], d["g_post2"], None, d["g_pre2"], t["r2"], t["x2"], s)

    def backward(self, s=None):
        d, t, g = self.d, self.t, self.g
        lib.moe_block_norm_backward(self.n2, d["dresid"], d["dx"], t["out"], t["r2"], d["g_post2"], None, d["g_pre2"],
                                    t["dr1"], t["dout"], g["g_post2"], None, g["g_pre2"], t["ws2"], s)
        lib.moe_combine_backward(self.p, t["dout"], self.ffn[0]["y"], t["pos"], t["w"], self.ffn[1]["y"], t["logit"],
                                 t["dy"], g["topk_w"], t["ds_y"], g["logit"], s)
        for q, x, dy in zip(self.ffn, (t["xs"], t["x"]), (t["dy"], t["ds_y"])):
            n, ws = q["names"], q["ws"]
            lib.moe_linear_backward(q["pd"], dy, q["h"], d[n[2]], q["off"], None, None, q["dh"], g[n[2]], None, None, ws, s)
            lib.moe_linear_backward(q["pg"], q["dh"], x, d[n[0]], q["off"], q["up"], q["z"], q["dxg"], g[n[0]], None,
                                    q["dup"], ws, s)
            lib.moe_linear_backward(q["pu"], q["dup"], x, d[n[1]], q["off"], None, None, q["dxu"], g[n[1]], None, None, ws, s)
            q["dxg"].add_(q["dxu"])
        lib.moe_permute_backward(self.p, self.ffn[0]["dxg"], t["pos"], None, None, t["dx"], None, s)
        t["dx"].add_(self.ffn[1]["dxg"])
        lib.moe_block_norm_backward(self.n1, t["dr1"], t["dx"], d["f"], t["r1"], d["g_post1"], d["gate1"], d["g_pre1"],
                                    g["resid"], g["f"], g["g_post1"], g["gate1"], g["g_pre1"], t["ws1"], s)

    def results(self):
        return [self.t["r2"], self.t["x2"], *(self.g[n] for n in GRADS)]

    def clear(self):
        for v in self.results():
            v.fill_(float("nan"))


def routing64(T, E, k, seed=3):
    """Positions of random choices, in the dispatch's order: [T, k], offsets [E + 1]."""
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    pos = np.empty(T * k, np.int64)
    pos[np.argsort(ids.reshape(-1), kind="stable")] = np.arange(T * k)
    return pos.reshape(T, k), np.concatenate([[0], np.cumsum(np.bincount(ids.reshape(-1), minlength=E))])


@pytest.mark.parametrize("case", [CASES[1], CASES[4]], ids=[IDS[1], IDS[4]])
def test_the_fp64_chains_gradients_by_differences(case):
    """CPU: the gradient of <r2, dresid> + <x2, dx> along a random direction of every input."""
    T, H, E, k, I, Is, dt = case
    rng = np.random.default_rng(1)
    d = {n: np64(v) for n, v in inputs(*case).items()}
    pos, off = routing64(T, E, k)
    d["topk_w"], d["logit"] = rng.random((T, k)), rng.standard_normal(T)
    g = chain64(d, pos, off)[2]

    def value(e):
        r2, x2, _ = chain64(e, pos, off)
        return (r2 * d["dresid"]).sum() + (x2 * d["dx"]).sum()

    for n in GRADS:
        u = rng.standard_normal(d[n].shape)
        h = 1e-5
        diff = (value({**d, n: d[n] + h * u}) - value({**d, n: d[n] - h * u})) / (2 * h)
        want = (g[n] * u).sum()
        # the third derivative's part is about h^2 of the value's scale, the rounding's 2^-53 / h
        assert abs(diff - want) <= 1e-6 * (abs(want) + np.abs(g[n] * u).sum()), (n, diff, want)


def deviations(d, pos, off, dt):
    """The chain's results and each one's bound on the root mean square error."""
    rng = np.random.default_rng(7)
    e = half(dt) + 16 * F  # a store's rounding, and fp32 sums of a few hundred terms
    exact = chain64(d, pos, off)
    flat = lambda c: [c[0], c[1], *(c[2][n] for n in GRADS)]
    ref = flat(exact)
    sq = [0.0] * len(ref)
    for _ in range(8):
        got = flat(chain64(d, pos, off, lambda v: v * (1 + e * rng.uniform(-1, 1, v.shape))))
        sq = [s + ((a - b) ** 2).mean() / 8 for s, a, b in zip(sq, got, ref)]
    # fp32 outputs of sums have their own roundings beside those of their terms
    return ref, [4 * np.sqrt(s) + 64 * F * np.sqrt((v * v).mean()) for s, v in zip(sq, ref)]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_block_forward_and_backward(case):
    print(f"[block] {case}", flush=True)
    T, H, E, k, I, Is, dt = case
    d = inputs(*case)
    b = Block(d, *case)
    b.clear()
    b.forward()
    b.backward()
    d64 = {n: np64(v) for n, v in d.items()}
    d64["topk_w"], d64["logit"] = np64(b.t["w"]), np64(b.t["logit"])
    pos, off = b.t["pos"].cpu().numpy(), b.t["off"].cpu().numpy()
    assert sorted(pos.reshape(-1)) == list(range(T * k))
    ref, bound = deviations(d64, pos, off, dt)
    for n, got, want, lim in zip(["r2", "x2", *GRADS], b.results(), ref, bound):
        err = np.sqrt(((np64(got).reshape(want.shape) - want) ** 2).mean())
        assert err <= lim, f"{n}: rms error {err:.3e}, bound {lim:.3e}, values {np.sqrt((want ** 2).mean()):.3e}"


@pytest.mark.gpu
def test_blocks_on_other_streams_and_from_two_threads():
    cases = [CASES[2], CASES[1]]
    blocks = [Block(inputs(*c, seed=5), *c) for c in cases]
    want = []
    for b in blocks:
        b.forward()
        b.backward()
        want.append([v.clone() for v in b.results()])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for named in (True, False):  # the stream as an argument, or as the current one
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                b.clear()
                for _ in range(3):
                    b.forward(s if named else None)
                    b.backward(s if named else None)
        torch.cuda.synchronize()
        for b, w in zip(blocks, want):
            assert all(same_bits(x, y) for x, y in zip(b.results(), w))
    failed = []

    def work(b, s):
        try:
            with torch.cuda.stream(s):
                b.clear()
                for _ in range(20):
                    b.forward()
                    b.backward()
                s.synchronize()
        except Exception as e:  # noqa: BLE001 - reported by the assertion below
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(blocks, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for b, w in zip(blocks, want):
        assert all(same_bits(x, y) for x, y in zip(b.results(), w))


@pytest.mark.gpu
def test_blocks_in_captured_graphs():
    """Two graphs, each with its own tensors and workspaces, replayed in turn with eager work of both between."""
    blocks = [Block(inputs(*c, seed=9), *c) for c in (CASES[2], CASES[1])]
    eager = [Block(inputs(*c, seed=9), *c) for c in (CASES[2], CASES[1])]
    graphs = []
    for b, e in zip(blocks, eager):
        b.forward()  # eagerly first, as any program does before it captures
        b.backward()
        e.forward()
        e.backward()
        torch.cuda.synchronize()
        g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=side):
            b.forward(side)
            b.backward(side)
        graphs.append(g)
    for i in range(4):
        for b, e in zip(blocks, eager):  # other inputs, at the same addresses
            for n in ("resid", "f", "dx", "w_gate", "gate1"):
                v = torch.randn_like(b.d[n].float()).to(b.d[n].dtype) * (0.1 if n == "w_gate" else 1.0)
                b.d[n].copy_(v)
                e.d[n].copy_(v)
            b.clear()
        for g in graphs:
            g.replay()
        for e in eager:
            e.forward()
            e.backward()
        torch.cuda.synchronize()
        for b, e in zip(blocks, eager):
            assert all(same_bits(x, y) for x, y in zip(b.results(), e.results())), f"replay {i}"
