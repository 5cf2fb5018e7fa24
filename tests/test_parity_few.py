"""GPU parity of the layer for a few tokens (moe_layer_forward_few) against the fp64 oracle.

Expert ids must equal the oracle's (inputs with margins, as in test_parity.py).  The output is held element by element:
each expert's bound from expert_bounds.py (fp8 and MXFP4 weights convert exactly, fp8 scales multiply fp32 sums), the
routing weights' error (logits: sums of H exact products in fp32, off by H 2^-23 |x||w| at most; a weight is off by twice
that relative, and 2^-20 for exp and division), fp32 sums over the groups, and one rounding of out to bf16.
"""
import ctypes

import numpy as np
import pytest
import torch

import expert_bounds as eb
import sparse_moe_layer_amd as lib
import test_parity as tp
from oracle import adapter
from sparse_moe_layer_amd.tensors import structs
from synthetic.gen import CONFIGS

U32 = eb.U32


# ---------------------------------------------------------------------------
# refusals (CPU: every call fails its checks before a launch)
# ---------------------------------------------------------------------------
def test_few_refuses_before_any_launch():
    L = lib.LIB
    fake = 1 << 20

    def call(T=4, act="bf16", wdt="bf16", ws=fake, short=0, x=fake, out=fake, router=fake, **kw):
        p = lib.problem(T, 256, 16, 4, 128, kw.get("Is", 0), act, wdt, 32 if wdt == "mxfp4" else 128)
        w = lib.moe_weights(router, fake, fake, fake, *kw.get("strides", (0, 0, 0)), *kw.get("scales", (fake,) * 3),
                            *kw.get("sh", (None,) * 4))
        n = lib.moe_few_workspace_bytes(p)
        return L.moe_layer_forward_few(ctypes.byref(p), ctypes.byref(w), x, out, None, None, ws, n - short if n else 0,
                                       None)

    assert call(T=17) == 6 and call(T=-1) == 2 and call(act="f32", wdt="f32") == 6  # UNSUPPORTED, SHAPE, UNSUPPORTED
    assert call(short=1) == 5 and call(ws=None) == 1 and call(ws=fake + 16) == 4
    assert call(x=None) == 1 and call(out=None) == 1 and call(router=None) == 1
    assert call(x=fake + 8) == 4 and call(out=fake + 2) == 4 and call(router=fake + 4) == 4
    assert call(Is=64) == 1  # a shared expert declared and not passed
    assert call(wdt="fp8", scales=(fake, None, fake)) == 1
    assert call(wdt="mxfp4", strides=(48, 0, 0)) == 4
    assert call(T=0, x=None, out=None, ws=None) == 0  # an empty batch: a no-op
    big = lib.problem(17, 256, 16, 4, 128)
    assert lib.moe_few_workspace_bytes(big) == 0
    with pytest.raises(lib.MoEError):
        lib.few_workspace(big)
    sizes = [lib.moe_few_workspace_bytes(lib.problem(T, 2560, 512, 10, 640, 640)) for T in (1, 8, 16)]
    assert sizes[0] < sizes[1] < sizes[2] and all(s % 256 == 0 for s in sizes)


# ---------------------------------------------------------------------------
# parity
# ---------------------------------------------------------------------------
def few_problem(T, H, E, k, I, Is, wdt, seed=0, page=False, **kw):
    cfg = CONFIGS["flash_prefill"].with_(name=f"few_{wdt}_{T}_{H}_{E}_{k}_{I}_{Is}", T=T, H=H, E=E, k=k, I=I,
                                         I_shared=Is, wdt=wdt, scale_block=32 if wdt == "mxfp4" else 128, **kw)
    return tp.gpu_problem(cfg, seed, page=page)


def run_few(p, flags=0, ws=None, stream=None, routing=True):
    c = p.cfg
    P, W = structs(p, flags)
    ws = lib.few_workspace(P) if ws is None else ws
    out = torch.full((c.T, c.H), float("nan"), dtype=torch.bfloat16, device="cuda")
    ids = torch.full((c.T, c.k), -1, dtype=torch.int32, device="cuda") if routing else None
    w = torch.full((c.T, c.k), float("nan"), device="cuda") if routing else None
    lib.moe_layer_forward_few(P, W, p.x, out, ids, w, ws, stream)
    return out, ids, w


def check_few(p, out, ids, w, page=False):
    c = p.cfg
    r = adapter.forward(p, page=page)
    x, wr, shared, sg = adapter.dense_inputs(p)
    assert np.array_equal(ids.cpu().numpy(), r["ids"]), "expert ids differ"
    dl = c.H * U32 * (np.abs(x) @ np.abs(wr).T)
    drel = 2 * np.take_along_axis(dl, r["ids"].astype(np.int64), 1).max(axis=1, keepdims=True) + 2.0 ** -20
    if page:
        drel = drel + 2 * eb.BF16  # the weights are rounded to bf16; two evaluations may round apart
    dw = drel * r["w"]
    assert (np.abs(w.cpu().numpy() - r["w"]) <= dw).all(), "routing weights differ"
    get = adapter.expert_weights_fn(p)
    ref, bound, size = np.zeros((c.T, c.H)), np.zeros((c.T, c.H)), np.zeros((c.T, c.H))
    for e in np.unique(r["ids"]):
        t, j = np.nonzero(r["ids"] == e)
        y, dy = eb.expert(x[t], *get(e))
        ref[t] += r["w"][t, j][:, None] * y
        size[t] += r["w"][t, j][:, None] * np.abs(y)
        bound[t] += r["w"][t, j][:, None] * dy + dw[t, j][:, None] * np.abs(y)
    if c.I_shared:
        y, dy = eb.expert(x, *shared)
        ds = c.H * U32 * (np.abs(x) @ np.abs(sg))
        s = r["gamma"][:, None]
        ref, size = ref + s * y, size + s * np.abs(y)
        bound += s * dy + (ds[:, None] + 2.0 ** -20) * np.abs(y)  # sigmoid' <= 1/4; its evaluation 2^-20
    # units of a group and groups are added in fp32: at most 4 parts per group (K ranges) and 8 waves
    bound += (4 * (c.k + 1) + 8) * U32 * 4 * size
    err = np.abs(out.float().cpu().numpy() - ref) / (eb.rounded(ref, bound) + 1e-30)
    print(f"[few] {c.name}: largest error {err.max():.3f} of its bound", flush=True)
    assert err.max() <= 1.0, f"an output is {err.max():.2f} times its bound off"


@pytest.mark.gpu
@pytest.mark.parametrize("wdt", ["bf16", "fp8", "mxfp4"])
@pytest.mark.parametrize("shape", [
    # T, H, E, k, I, I_shared
    (1, 128, 1, 1, 128, 0),        # one expert, one token
    (1, 256, 16, 4, 128, 64),
    (2, 384, 8, 8, 256, 8),        # every expert takes every token; a tiny shared expert
    (5, 640, 33, 3, 384, 104),
    (16, 256, 64, 8, 128, 64),
    (16, 896, 4, 2, 1152, 0),      # groups of 8 rows: K in several units
    (7, 128, 1024, 10, 128, 32),   # the most experts
    (16, 128, 70, 64, 128, 0),     # the most picks
])
def test_few_layer(shape, wdt):
    p = few_problem(*shape, wdt)
    check_few(p, *run_few(p))


@pytest.mark.gpu
@pytest.mark.parametrize("wdt,shape", [
    ("bf16", (3, 8, 4, 2, 8, 8)),            # the smallest widths of each type
    ("mxfp4", (3, 32, 4, 2, 32, 0)),
    ("bf16", (7, 1192, 12, 3, 344, 40)),     # nothing ends on a tile
    ("mxfp4", (7, 1184, 60, 4, 352, 0)),
    ("bf16", (1, 72, 130, 2, 1032, 0)),
    ("mxfp4", (9, 96, 300, 5, 2016, 24)),
])
def test_few_layer_odd_sizes(wdt, shape):
    p = few_problem(*shape, wdt, seed=3)
    check_few(p, *run_few(p))


@pytest.mark.gpu
@pytest.mark.parametrize("T", range(1, 17))
def test_every_batch_size(T):
    p = few_problem(T, 256, 24, 4, 160, 64, "mxfp4", seed=T)
    check_few(p, *run_few(p))


@pytest.mark.gpu
@pytest.mark.parametrize("wdt,T", [("bf16", 1), ("mxfp4", 1), ("fp8", 4), ("mxfp4", 16)])
def test_model_shape(wdt, T):
    """The Flash-Next widths and expert count; also against the layer call of five launches."""
    p = few_problem(T, 2560, 512, 10, 640, 640, wdt, seed=5)
    out, ids, w = run_few(p)
    check_few(p, out, ids, w)
    P, W = structs(p)
    ref = torch.empty_like(out)
    lib.moe_layer_forward(P, W, p.x, ref, None, None, lib.workspace(P))
    # the layer call rounds each y to bf16: k + 1 terms of at most the largest output's size, half a step each
    assert (out.float() - ref.float()).abs().max() <= 2 ** -6 * ref.float().abs().max()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 16])
def test_long_rows(T):
    """The 2.4T widths over few experts: rows of 8192 and 2048 values."""
    p = few_problem(T, 8192, 6, 2, 2048, 256, "mxfp4", seed=6)
    check_few(p, *run_few(p))


@pytest.mark.gpu
def test_page_routing():
    p = few_problem(11, 256, 40, 6, 128, 64, "bf16", seed=7, page=True)
    check_few(p, *run_few(p, lib.MOE_FLAG_PAGE_ROUTING), page=True)


@pytest.mark.gpu
def test_equal_logits_go_to_the_lower_id():
    p = few_problem(4, 256, 12, 3, 128, 0, "bf16", seed=8)
    p.w_router[7] = p.w_router[2]
    p.w_router[11] = p.w_router[2]
    p.x[:] = p.w_router[2] * 16  # experts 2, 7 and 11 tie at the top
    _, ids, w = run_few(p)
    assert ids.tolist() == [[2, 7, 11]] * 4 and torch.equal(w[:, 0], w[:, 2])


@pytest.mark.gpu
@pytest.mark.parametrize("wdt", ["bf16", "fp8", "mxfp4"])
def test_deterministic_whatever_is_in_the_workspace(wdt):
    p = few_problem(13, 512, 48, 6, 256, 128, wdt, seed=9)
    P, _ = structs(p)
    ws = lib.few_workspace(P)
    ref, ids, w = run_few(p, ws=ws)
    for fill in (0, 255, 127):
        ws.fill_(fill)
        out, i2, w2 = run_few(p, ws=ws)
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16)) and torch.equal(ids, i2) and torch.equal(w, w2)
    out, _, _ = run_few(p, ws=ws, routing=False)  # no routing outputs
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))


@pytest.mark.gpu
def test_rows_beyond_the_batch_and_the_guard_bytes_stay():
    """A call with T tokens writes T rows of each output and moe_few_workspace_bytes of scratch, nothing else."""
    p = few_problem(5, 264, 16, 4, 136, 40, "bf16", seed=10)
    c = p.cfg
    P, W = structs(p)
    n = lib.moe_few_workspace_bytes(P)
    ws = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full((c.T + 2, c.H), 3.0, dtype=torch.bfloat16, device="cuda")
    ids = torch.full((c.T + 2, c.k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((c.T + 2, c.k), -7.0, device="cuda")
    lib.moe_layer_forward_few(P, W, p.x, out, ids, w, ws[:n])
    torch.cuda.synchronize()
    assert (out[c.T:] == 3.0).all() and (ids[c.T:] == -7).all() and (w[c.T:] == -7.0).all()
    assert (ws[n:] == 0xA5).all()
    check_few(p, out[:c.T], ids[:c.T], w[:c.T])


@pytest.mark.gpu
def test_two_streams_with_their_own_workspaces():
    """Two layers in flight at once, repeatedly: each gives the bits it gives alone."""
    ps = [few_problem(16, 512, 64, 8, 256, 64, "bf16", seed=11), few_problem(3, 768, 32, 4, 384, 0, "mxfp4", seed=12)]
    wss = [lib.few_workspace(structs(p)[0]) for p in ps]
    refs = [run_few(p)[0] for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(20):
        for p, s, ws in zip(ps, streams, wss):
            with torch.cuda.stream(s):
                outs.append(run_few(p, ws=ws, stream=s)[0])
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o.view(torch.int16), refs[i % 2].view(torch.int16)), f"call {i}"


@pytest.mark.gpu
@pytest.mark.parametrize("wdt", ["bf16", "fp8", "mxfp4"])
def test_replays_in_a_graph(wdt):
    """Captured, replayed with new activations and eager calls on the same workspace between the replays."""
    p = few_problem(6, 384, 40, 5, 256, 64, wdt, seed=13)
    P, W = structs(p)
    ws = lib.few_workspace(P)
    xs = [p.x.clone(), (p.x * 0.5).clone(), p.x.flip(0).clone()]
    refs = []
    for x in xs:
        p.x.copy_(x)
        refs.append(run_few(p)[0])
    out = torch.zeros_like(refs[0])
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        lib.moe_layer_forward_few(P, W, p.x, out, None, None, ws, side)
    for i in range(6):
        out.fill_(float("nan"))
        p.x.copy_(xs[i % 3])
        torch.randn(1 << 20, device="cuda").sum()
        other = run_few(p, ws=ws)[0]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), refs[i % 3].view(torch.int16)), f"replay {i}"
        assert torch.equal(other.view(torch.int16), refs[i % 3].view(torch.int16))


@pytest.mark.gpu
def test_a_decode_step_around_the_layer():
    """As a served model runs them: experts quantised to MXFP4, the gated residual read, the few-token layer and the
    write, against the same steps through the layer call."""
    from synthetic.gen import make_gr_problem

    T, H, E, k, I = 4, 256, 32, 4, 128
    p = few_problem(T, H, E, k, I, 64, "mxfp4", seed=14)
    gr = make_gr_problem(T, H, 32, 5, "cuda")
    P, _ = structs(p)
    gates = [torch.stack([p.expert_fp32(e, n) for e in range(E)]).bfloat16() for n in ("gate", "up", "down")]
    (cg, sg), (cu, su), (cd, sd) = (lib.mx_quantize(t) for t in gates)
    W = lib.weights(p.w_router, cg, cu, cd, sg, su, sd, p.sh_gate, p.sh_up, p.sh_down, p.sh_gate_w)
    G = lib.gr_weights(gr.norm_w, gr.w_read, gr.w_up, 32)
    x, s = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, 4, device="cuda")
    lib.moe_gr_read(P, G, gr.resid, x, s, lib.gr_workspace(P, 32))
    res = []
    for call, ws in ((lib.moe_layer_forward_few, lib.few_workspace(P)), (lib.moe_layer_forward, lib.workspace(P))):
        f, r = torch.empty_like(x), torch.empty_like(gr.resid)
        call(P, W, x, f, None, None, ws)
        lib.moe_gr_write(P, gr.resid, s, f, r)
        res.append(r.float())
    # F differs by the roundings of y (k + 1 of half a bf16 step), the streams by theirs and one more rounding
    lim = 2 ** -6 * f.float().abs().max() * s.abs().max() + 2 ** -7 * res[1].abs()
    assert ((res[0] - res[1]).abs() <= lim).all()
