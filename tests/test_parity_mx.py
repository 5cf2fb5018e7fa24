"""GPU parity of the MXFP4 weights: the conversions bit for bit, and the expert products and the whole layer with
4-bit experts against the fp64 oracle.

The conversions are exact arithmetic, so codes, scales and values must equal the oracle's.  The expert outputs are held
element by element to the bound of expert_bounds.py (E2M1 times a power of two is exact in bf16, so the weights add no
error of their own); whole layers also to the suite's 2e-2 of the largest output.
"""
import numpy as np
import pytest
import torch

import expert_bounds
import sparse_moe_layer_amd as lib
import test_parity as tp
from oracle import adapter, mx
from sparse_moe_layer_amd.tensors import structs
from synthetic.gen import CONFIGS, make_problem

pytestmark = pytest.mark.gpu
U8 = torch.uint8


def quantized(w, **kw):
    codes = torch.full((*w.shape[:-1], w.shape[-1] // 2), 0xEE, dtype=U8, device="cuda")
    scales = torch.full((*w.shape[:-1], w.shape[-1] // 32), 0xEE, dtype=U8, device="cuda")
    lib.moe_mx_quantize(w, codes, scales, **kw)
    torch.cuda.synchronize()
    return codes.cpu().numpy(), scales.cpu().numpy()


def check_quantize(w):
    codes, scales = quantized(w)
    oc, os_ = mx.quantize(w.double().cpu().numpy())
    assert np.array_equal(scales, os_), "scales differ"
    bad = np.argwhere(codes != oc)
    assert bad.size == 0, f"{len(bad)} code bytes differ, first at {bad[:3].tolist()}"


# ---------------------------------------------------------------------------
# conversions
# ---------------------------------------------------------------------------
def test_quantize_every_bf16_pattern_beside_larger_values():
    """Each of the 65536 patterns in a group whose largest value is d binades above it (d = 0 .. 6), so every
    rounding boundary, saturation, subnormals, zeros, infinities and NaN occur."""
    bits = torch.arange(65536, dtype=torch.int32)
    for d in range(7):
        ex = ((bits >> 7) & 255)
        lead = torch.where(ex == 255, ex, (ex + d).clamp(max=254)) << 7  # a power of two (or infinity)
        w = torch.stack([bits, lead] + [bits * 0] * 30, dim=1)
        w[:, 2::2] = bits[:, None]
        w = w.to(torch.int16).view(torch.bfloat16).cuda()
        print(f"[mx] quantize every pattern, {d} binades below the group's largest", flush=True)
        check_quantize(w)


def test_quantize_fp32_rounds_once_from_the_fp32_value():
    g = torch.Generator().manual_seed(5)
    # values at, just below and just above every boundary, over scales from the smallest to the largest
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0])
    near = torch.cat([mid, torch.nextafter(mid, mid + 1), torch.nextafter(mid, mid - 1)])
    rows = []
    for e in list(range(-126, 126, 7)) + [-125, -124, 123, 124, 125]:
        r = torch.zeros(32)
        r[:27] = near
        r[27:] = torch.tensor([4.0, -0.25, -0.75, -2.5, -0.0])
        rows.append(r * 2.0 ** e if e < 120 else r.clamp(max=6.0) * 2.0 ** e)
    w = torch.cat([torch.stack(rows), torch.randn(301, 32, generator=g), torch.randn(40, 32, generator=g) * 1e-38,
                   torch.randn(40, 32, generator=g) * 1e-44, torch.randn(3, 32, generator=g) * 1e37])
    w[-1, 4], w[-2, 0], w[-3, 31] = float("nan"), float("inf"), -float("inf")
    check_quantize(w.cuda())


@pytest.mark.parametrize("rows,K", [(1, 32), (3, 32), (1, 8192), (37, 672), (255, 96), (1025, 32), (130, 2560)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_conversions_at_odd_sizes(rows, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows * K)
    w = (torch.randn(rows, K, generator=g, device="cuda") * 0.02).to(dtype)
    check_quantize(w)
    codes, scales = lib.mx_quantize(w)
    v = torch.full((rows, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    lib.moe_mx_dequantize(codes, scales, v)
    assert np.array_equal(v.double().cpu().numpy(), mx.dequant(codes.cpu().numpy(), scales.cpu().numpy()))


@pytest.mark.parametrize("dtype,pad", [(torch.bfloat16, 8), (torch.float32, 4), (torch.bfloat16, 160)])
def test_rows_apart_in_memory(dtype, pad):
    """Rows with a stride: the same codes; what lies between the rows is neither read into a group nor written."""
    rows, K = 19, 160
    g = torch.Generator(device="cuda").manual_seed(7)
    base = torch.full((rows, K + pad), float("nan"), dtype=dtype, device="cuda")
    base[:, :K] = (torch.randn(rows, K, generator=g, device="cuda") * 3).to(dtype)
    check_quantize(base[:, :K])
    codes, scales = lib.mx_quantize(base[:, :K].contiguous())
    out = torch.full((rows, K + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.moe_mx_dequantize(codes, scales, out[:, :K])
    torch.cuda.synchronize()
    assert (out[:, K:] == 7.0).all()
    assert np.array_equal(out[:, :K].double().cpu().numpy(), mx.dequant(codes.cpu().numpy(), scales.cpu().numpy()))


def test_dequantize_every_code_at_every_scale():
    codes = torch.arange(256, dtype=torch.int32).to(U8).repeat(256, 1)  # every byte at every scale
    codes = codes.reshape(256, 256).cuda()
    scales = torch.arange(256, dtype=torch.int32).to(U8)[:, None].repeat(1, 512 // 32).cuda()
    v = torch.zeros(256, 512, dtype=torch.bfloat16, device="cuda")
    lib.moe_mx_dequantize(codes, scales, v)
    torch.cuda.synchronize()
    got = v.double().cpu().numpy()
    want = mx.dequant(codes.cpu().numpy(), scales.cpu().numpy())
    assert np.array_equal(np.isnan(got), np.isnan(want)), "NaN at s = 255 and nowhere else"
    assert np.array_equal(got[2:253], want[2:253]), "exact"  # at s = 253, 4 * 2^126 is 2^128 already
    # s < 2: a value below bf16's smallest normal number may be zero
    small = np.abs(want[:2]) < 2.0 ** -126
    assert np.array_equal(got[:2][~small], want[:2][~small])
    assert ((got[:2] == want[:2]) | (got[:2] == 0)).all()
    # values of 2^128 and more are infinite
    big = np.where(np.abs(want[253:255]) >= 2.0 ** 128, np.sign(want[253:255]) * np.inf, want[253:255])
    assert np.array_equal(got[253:255], big)
    assert np.array_equal(np.signbit(got[:255]), np.signbit(want[:255]))


def test_conversions_replay_in_a_graph_on_another_stream():
    w = torch.randn(257, 96, device="cuda").bfloat16()
    codes = torch.empty(257, 48, dtype=U8, device="cuda")
    scales = torch.empty(257, 3, dtype=U8, device="cuda")
    v = torch.empty(257, 96, dtype=torch.bfloat16, device="cuda")
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        lib.moe_mx_quantize(w, codes, scales, side)
        lib.moe_mx_dequantize(codes, scales, v, side)
    for i in range(4):
        w.copy_(torch.randn(257, 96, device="cuda"))
        v.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        oc, os_ = mx.quantize(w.double().cpu().numpy())
        assert np.array_equal(v.double().cpu().numpy(), mx.dequant(oc, os_)), f"replay {i}"


# ---------------------------------------------------------------------------
# expert products and the layer
# ---------------------------------------------------------------------------
def mx_problem(T, H, E, k, I, Is, seed=0, zipf=0.0):
    cfg = CONFIGS["flash_prefill"].with_(name=f"mx_{T}_{H}_{E}_{k}_{I}_{Is}", T=T, H=H, E=E, k=k, I=I, I_shared=Is,
                                         wdt="mxfp4", scale_block=32, zipf_s=zipf)
    return tp.gpu_problem(cfg, seed)


def check_bounds(p, g):
    """Every routed and shared expert output within its own bound."""
    c = p.cfg
    x, _, shared, _ = adapter.dense_inputs(p)
    get = adapter.expert_weights_fn(p)
    off, so = g["offsets"], g["sorted"]
    worst = 0.0
    for e in range(c.E):
        if off[e + 1] == off[e]:
            continue
        rows = slice(off[e], off[e + 1])
        y, dy = expert_bounds.expert(x[so[rows] // c.k], *get(e))
        r = np.abs(g["y"][rows] - y) / expert_bounds.rounded(y, dy)
        worst = max(worst, r.max())
    if c.I_shared:
        y, dy = expert_bounds.expert(x, *shared)
        worst = max(worst, (np.abs(g["ysh"] - y) / expert_bounds.rounded(y, dy)).max())
    print(f"[mx] {c.name}: largest error {worst:.3f} of its bound", flush=True)
    assert worst <= 1.0, f"an expert output is {worst:.2f} times its bound off"


FORCE = {"default": 0, "gemm": lib.MOE_FLAG_FORCE_GEMM, "stream": lib.MOE_FLAG_FORCE_STREAM}


@pytest.mark.parametrize("flag", ["default", "gemm", "stream"])
@pytest.mark.parametrize("shape", [
    # T, H, E, k, I, I_shared
    (1, 32, 1, 1, 32, 0),        # the smallest
    (1, 256, 8, 2, 64, 0),       # one token
    (13, 160, 12, 3, 96, 40),    # K ends inside a 64-, 128- and 256-wide step in both phases
    (16, 288, 6, 6, 352, 0),     # every expert takes every token
    (37, 1184, 9, 2, 224, 72),
    (200, 672, 5, 2, 416, 0),    # groups of 60 to 100 rows: ragged tiles
    (300, 256, 40, 2, 128, 0),   # streamed and tiled groups together
])
def test_experts_and_layer(shape, flag):
    p = mx_problem(*shape)
    g = tp.run_stages(p, FORCE[flag])
    tp.check(p, g)
    check_bounds(p, g)


@pytest.mark.parametrize("T", [64, 1100])
def test_skewed_load(T):
    """Groups from empty to nearly all tokens (several m-tiles)."""
    p = mx_problem(T, 256, 24, 3, 160, 0, seed=4, zipf=1.1)
    g = tp.run_stages(p)
    tp.check(p, g)
    check_bounds(p, g)


def test_model_shape_experts():
    """The Flash-Next width, 48 tokens over 64 experts: long rows in both phases."""
    p = mx_problem(48, 2560, 64, 10, 640, 640, seed=2)
    g = tp.run_stages(p)
    tp.check(p, g)
    check_bounds(p, g)


def test_experts_at_a_stride_and_fused_gate_up():
    """A fused [E, 2I, H/2] gate_up tensor by strides gives the same bits as separate matrices."""
    p = mx_problem(21, 192, 7, 2, 96, 0, seed=9)
    c = p.cfg
    ref = tp.run_stages(p)
    fused = torch.full((c.E, 2 * c.I + 5, c.H // 2), 0xEE, dtype=U8, device="cuda")
    fused[:, :c.I], fused[:, c.I:2 * c.I] = p.w_gate, p.w_up
    P, _ = structs(p)
    up = fused.view(-1)[c.I * c.H // 2:]
    st = (2 * c.I + 5) * c.H
    W = lib.weights(p.w_router, fused, up, p.w_down, p.s_gate, p.s_up, p.s_down, stride_gate=st, stride_up=st)
    out = torch.empty((c.T, c.H), dtype=torch.bfloat16, device="cuda")
    lib.moe_layer_forward(P, W, p.x, out, None, None, lib.workspace(P))
    assert np.array_equal(out.float().cpu().numpy(), ref["out"])


def test_quantized_weights_run_through_the_layer():
    """bf16 experts, mx_quantize, layer_forward: the same bits as the generator's codes; the no-allocation call too."""
    p = mx_problem(40, 256, 16, 4, 128, 64, seed=6)
    w = [torch.stack([p.expert_fp32(e, n) for e in range(16)]).cuda() for n in ("gate", "up", "down")]
    (cg, sg), (cu, su), (cd, sd) = (lib.mx_quantize(t) for t in w)
    assert torch.equal(cg, p.w_gate) and torch.equal(sd, p.s_down)
    out, ids, tw = lib.layer_forward(p.x, 4, p.w_router, cg, cu, cd, sg, su, sd, p.sh_gate, p.sh_up, p.sh_down,
                                     p.sh_gate_w)
    ref = adapter.forward(p)
    assert np.array_equal(ids.cpu().numpy(), ref["ids"])
    assert tp.rel_err(out.float().cpu().numpy(), ref["out"]) <= 2e-2
    P, W = structs(p)
    out2 = torch.empty_like(out)
    lib.moe_layer_forward_noalloc(P, W, p.x, out2, None, None)
    assert torch.equal(out2.view(torch.int16), out.view(torch.int16))


def test_nan_scale_stays_in_its_expert():
    """A NaN scale byte in one expert reaches the rows of that expert and no other."""
    p = mx_problem(24, 256, 8, 2, 96, 0, seed=11)
    p.s_down[3, 17, 1] = 255
    P, W = structs(p)
    ws = lib.workspace(P)
    ids = torch.empty((24, 2), dtype=torch.int32, device="cuda")
    out = torch.empty((24, 256), dtype=torch.bfloat16, device="cuda")
    lib.moe_layer_forward(P, W, p.x, out, ids, None, ws)
    hit = (ids == 3).any(dim=1)
    nan = torch.isnan(out)
    assert hit.any() and not hit.all()
    assert nan[hit][:, 17].all() and nan.sum() == hit.sum()


def test_layer_replays_under_graph_capture_with_mx_weights():
    p = mx_problem(40, 256, 16, 4, 128, 64, seed=8)
    P, W = structs(p)
    ws = lib.workspace(P)
    ref = torch.empty((40, 256), dtype=torch.bfloat16, device="cuda")
    lib.moe_layer_forward(P, W, p.x, ref, None, None, ws)
    torch.cuda.synchronize()
    out = torch.zeros_like(ref)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        lib.moe_layer_forward(P, W, p.x, out, None, None, ws, side)
    for i in range(4):
        out.fill_(float("nan"))
        torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16)), f"replay {i}"
