"""What is measured of the 4-bit expert weights and of the layer for a few tokens.

Four operators, each in its plain form (elementary torch operations in 32 bits, logits in 64)
and, where `own` is true, through the package's entry points:

  few         moe_layer_forward_few: router, top-k, experts, gated shared expert and combine of a
              batch of at most 16 tokens, in two kernels; bf16, fp8 or MXFP4 routed weights
  ffn         moe_expert_ffn with MXFP4 weights (E2M1 codes, one E8M0 scale per 32 values along K):
              the grouped SwiGLU products, from one token to prefill chunks
  quantize    moe_mx_quantize, read back with moe_mx_dequantize: weights to MXFP4 and to the values
              the codes stand for
  dequantize  moe_mx_dequantize: MXFP4 to bf16

Layouts are the package's: w_gate, w_up [E, I, H], w_down [E, H, I]; fp8 codes one a byte with fp32
scales of 128 x 128 blocks; MXFP4 codes two a byte along K (the even k in the low four bits) with
E8M0 bytes [.., K/32].
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one user's decode step at the Flash-Next shape, weights as released: latency counts
        {"name": "few 1 token bf16", "op": "few", "wdt": "bf16", "T": 1, "H": 2560, "E": 512, "k": 10, "I": 640, "Is": 640},
        # the same step with 4-bit experts, the smallest call that a served model makes
        {"name": "few 1 token mxfp4", "op": "few", "wdt": "mxfp4", "T": 1, "H": 2560, "E": 512, "k": 10, "I": 640, "Is": 640},
        # a full decode batch of 16 with fp8 experts: about 139 experts are touched
        {"name": "few 16 tokens fp8", "op": "few", "wdt": "fp8", "T": 16, "H": 2560, "E": 512, "k": 10, "I": 640, "Is": 640},
        # a speculative step of 4 tokens of the 2.4T shape with 4-bit experts: long rows, many bytes
        {"name": "few 4 tokens 2.4T mxfp4", "op": "few", "wdt": "mxfp4", "T": 4, "H": 8192, "E": 512, "k": 10, "I": 2048, "Is": 2048},
        # a small layer with sizes that end inside every tile, no shared expert
        {"name": "few 7 tokens odd", "op": "few", "wdt": "mxfp4", "T": 7, "H": 1184, "E": 60, "k": 4, "I": 352, "Is": 0},
        # a dense 4-bit SwiGLU of the 2.4T width for one token: matrix-vector products
        {"name": "ffn 1 token dense", "op": "ffn", "T": 1, "H": 8192, "E": 1, "k": 1, "I": 2048, "Is": 0, "skew": 0.0},
        # a decode batch of 24: every touched expert holds a row or two, its weights are read once
        {"name": "ffn 24 tokens", "op": "ffn", "T": 24, "H": 2560, "E": 512, "k": 10, "I": 640, "Is": 0, "skew": 0.0},
        # a Flash-Next prefill chunk: about 80 rows an expert, with the bf16 shared expert
        {"name": "ffn 4096 tokens", "op": "ffn", "T": 4096, "H": 2560, "E": 512, "k": 10, "I": 640, "Is": 640, "skew": 0.0},
        # a skewed chunk of the 2.4T width: from groups of a few rows to one that holds nearly all tokens
        {"name": "ffn 1023 tokens skewed", "op": "ffn", "T": 1023, "H": 8192, "E": 64, "k": 10, "I": 2048, "Is": 0, "skew": 1.1},
        # a small odd fp32 matrix
        {"name": "quantize 37 rows f32", "op": "quantize", "rows": 37, "K": 672, "src": "f32"},
        # the gate matrices of a whole Flash-Next layer, as a checkpoint is converted
        {"name": "quantize layer bf16", "op": "quantize", "rows": 512 * 640, "K": 2560, "src": "bf16"},
        # the gate matrices of 64 experts of the 2.4T shape, read back for the weight audit
        {"name": "dequantize 64 experts", "op": "dequantize", "rows": 64 * 2048, "K": 8192},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("few", "few", "ffn", "ffn", "quantize", "dequantize"))
    if op in ("quantize", "dequantize"):
        K = 32 * log(1, 256)
        rows = max(1, min(log(1, 300000), 500_000_000 // K))
        return {"op": op, "rows": rows, "K": K, **({"src": rng.choice(("bf16", "f32"))} if op == "quantize" else {})}
    E = log(1, 512)
    k = rng.randint(1, min(E, 12))
    wdt = rng.choice(("bf16", "fp8", "mxfp4")) if op == "few" else "mxfp4"
    q = {"bf16": 8, "fp8": 128, "mxfp4": 32}[wdt]
    H, I = q * max(1, log(256, 4096) // q), q * max(1, log(128, 2048) // q)
    while E * H * I > 900_000_000:  # the weights of the listed layers at most
        E = max(k, E // 2)
    Is = rng.choice((0, 8 * log(8, 128)))
    if op == "few":
        return {"op": op, "wdt": wdt, "T": rng.randint(1, 16), "H": H, "E": E, "k": k, "I": I, "Is": Is}
    T = max(1, min(log(1, 4096), int(6e10 // (k * H * I))))
    return {"op": op, "T": T, "H": H, "E": E, "k": k, "I": I, "Is": Is, "skew": rng.choice((0.0, 0.7, 1.1))}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _mx_random(gen, shape):
    """MXFP4 codes and scales as quantised N(0, 0.02) weights have them: uniform bit patterns, scales 2^-8 .. 2^-5."""
    codes = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.randint(119, 123, (*shape[:-1], shape[-1] // 32), generator=gen, device="cuda", dtype=torch.uint8)
    return codes, scales


def _normal(gen, shape, std):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=gen)


def _experts(gen, wdt, shape):
    if wdt == "bf16":
        return _normal(gen, shape, 0.02), None
    if wdt == "fp8":
        # e4m3fn bit patterns up to 240 in size (no NaN), with scales that bring them to about 0.02
        c = torch.randint(0, 120, shape, generator=gen, device="cuda", dtype=torch.uint8)
        c |= torch.randint(0, 2, shape, generator=gen, device="cuda", dtype=torch.uint8) << 7
        s = torch.rand((shape[0], shape[1] // 128, shape[2] // 128), generator=gen, device="cuda") * 2e-4 + 2e-4
        return c, s
    return _mx_random(gen, shape)


def _rows_apart(gen, T, H, k, w_router):
    """x [T, H] whose top k + 1 logits are 1e-4 apart, so that no sum's order decides a choice."""
    x = _normal(gen, (4 * T + 16, H), 1.0)
    top = torch.sort(x.double() @ w_router.double().T, dim=1, descending=True)[0][:, : k + 1]
    near = (top[:, :-1] - top[:, 1:] < 1e-4).any(dim=1)
    return x[torch.sort(near.int(), stable=True)[1][:T]].contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case, "e2m1": torch.tensor(E2M1, device="cuda")}
    if case["op"] in ("quantize", "dequantize"):
        rows, K = case["rows"], case["K"]
        if case["op"] == "quantize":
            w = torch.empty((rows, K), dtype=torch.float32 if case["src"] == "f32" else torch.bfloat16, device="cuda")
            s["w"] = w.normal_(0.0, 0.02, generator=gen)
            s["codes"] = torch.empty((rows, K // 2), dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty((rows, K // 32), dtype=torch.uint8, device="cuda")
        else:
            s["codes"], s["scales"] = _mx_random(gen, (rows, K))
        s["values"] = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
        return s
    T, H, E, k, I, Is = (case[n] for n in ("T", "H", "E", "k", "I", "Is"))
    wdt = case.get("wdt", "mxfp4")
    s["w_gate"], s["s_gate"] = _experts(gen, wdt, (E, I, H))
    s["w_up"], s["s_up"] = _experts(gen, wdt, (E, I, H))
    s["w_down"], s["s_down"] = _experts(gen, wdt, (E, H, I))
    if Is:
        s["sh_gate"], s["sh_up"] = _normal(gen, (Is, H), 0.02), _normal(gen, (Is, H), 0.02)
        s["sh_down"], s["sh_gate_w"] = _normal(gen, (H, Is), 0.02), _normal(gen, (1, H), 0.02)
    s["w_router"] = _normal(gen, (E, H), H**-0.5)
    if case["op"] == "few":
        s["x"] = _rows_apart(gen, T, H, k, s["w_router"])
        s["out"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        s["ids"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        s["tw"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
        return s
    # ffn: the dispatch is in hand (stable order by expert); `skew` biases expert e by -skew ln(rank e)
    s["x"] = _normal(gen, (T, H), 1.0)
    rank = torch.randperm(E, generator=gen, device="cuda") + 1.0
    score = torch.randn((T, E), generator=gen, device="cuda") - case["skew"] * torch.log(rank)
    flat = torch.topk(score, k, dim=1)[1].reshape(-1)
    count = torch.bincount(flat, minlength=E)
    s["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).int()
    s["sorted"] = torch.sort(flat, stable=True)[1].int()
    s["most"] = int(count.max())  # rows of the largest group
    s["y"] = torch.empty((T * k, H), dtype=torch.bfloat16, device="cuda")
    s["y_shared"] = torch.empty((T, H), dtype=torch.bfloat16, device="cuda") if Is else None
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _mx_values(codes, scales, e2m1):
    """E2M1 code times two to the power of its group's E8M0 byte less 127."""
    v = e2m1[torch.stack((codes & 15, codes >> 4), dim=-1).int()].flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * (scales.int() << 23).view(torch.float32).unsqueeze(-1)).flatten(-2)


def _values(wdt, w, s, e2m1):
    if wdt == "bf16":
        return w.float()
    if wdt == "fp8":
        return w.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, -2).repeat_interleave(128, -1)
    return _mx_values(w, s, e2m1)


def _swiglu(x, wg, wu, wd):
    """x [.., n, K] by matrices [.., N, K]."""
    g, u = x @ wg.mT, x @ wu.mT
    return (g / (1 + torch.exp(-g)) * u) @ wd.mT


def _plain_few(s):
    c, x = s["case"], s["x"].float()
    logits = s["x"].double() @ s["w_router"].double().T
    best, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    best, ids = best[:, : c["k"]], ids[:, : c["k"]]
    tw = torch.exp(best - best[:, :1])
    tw = (tw / tw.sum(dim=1, keepdim=True)).float()
    w = [_values(c["wdt"], s["w_" + n][ids], None if s["s_" + n] is None else s["s_" + n][ids], s["e2m1"]) for n in ("gate", "up", "down")]
    out = (_swiglu(x[:, None, None, :], *w).squeeze(2) * tw[:, :, None]).sum(dim=1)
    if c["Is"]:
        gate = 1 / (1 + torch.exp(-(x @ s["sh_gate_w"].float().T)))
        out = out + gate * _swiglu(x, s["sh_gate"].float(), s["sh_up"].float(), s["sh_down"].float())
    return {"out": out.bfloat16(), "ids": ids.int(), "weights": tw}


def _plain_ffn(s):
    c, x, off = s["case"], s["x"].float(), s["offsets"].long()
    R = c["T"] * c["k"]
    # the rows of every group side by side, groups with fewer than the largest filled up with any row
    at = (off[:-1, None] + torch.arange(s["most"], device="cuda")).clamp(max=R - 1)
    y = _swiglu(x[s["sorted"].long()[at] // c["k"]], *(_mx_values(s["w_" + n], s["s_" + n], s["e2m1"]) for n in ("gate", "up", "down")))
    row = torch.arange(R, device="cuda")
    e = torch.searchsorted(off, row, right=True) - 1
    out = {"y": y[e, row - off[e]].bfloat16()}
    if c["Is"]:
        out["y_shared"] = _swiglu(x, s["sh_gate"].float(), s["sh_up"].float(), s["sh_down"].float()).bfloat16()
    return out


def _plain_quantize(s):
    w = s["w"].float().unflatten(-1, (-1, 32))
    # scale 2^(floor(log2 amax) - 2), at least 2^-127: the exponent field of amax less 2
    byte = ((w.abs().amax(dim=-1, keepdim=True).view(torch.int32) >> 23) - 2).clamp(min=0)
    v = w * ((254 - byte) << 23).view(torch.float32)
    a = v.abs()
    # round to nearest even on the E2M1 grid: steps of 0.5 below 2, of 1 below 4, of 2 above, at most 6
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.copysign((torch.round(a / step) * step).clamp(max=6.0), v)
    return (q * (byte << 23).view(torch.float32)).flatten(-2).bfloat16()


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _handle(s):
    """The problem, the weights' struct and the workspace, as a program keeps them beside its weights."""
    import sparse_moe_layer_amd as moe

    c = s["case"]
    wdt = c.get("wdt", "mxfp4")
    p = moe.problem(c["T"], c["H"], c["E"], c["k"], c["I"], c["Is"], "bf16", wdt, 32 if wdt == "mxfp4" else 128)
    names = ("w_router", "w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down", "sh_gate", "sh_up", "sh_down", "sh_gate_w")
    return moe, p, moe.weights(*(s.get(n) for n in names)), moe.few_workspace(p) if c["op"] == "few" else moe.workspace(p)


def _own(s):
    op = s["case"]["op"]
    if op in ("quantize", "dequantize"):
        import sparse_moe_layer_amd as moe

        if op == "quantize":
            moe.moe_mx_quantize(s["w"], s["codes"], s["scales"])
        moe.moe_mx_dequantize(s["codes"], s["scales"], s["values"])
        return s["values"]
    if "handle" not in s:
        s["handle"] = _handle(s)
    moe, p, w, ws = s["handle"]
    if op == "few":
        moe.moe_layer_forward_few(p, w, s["x"], s["out"], s["ids"], s["tw"], ws)
        return {"out": s["out"], "ids": s["ids"], "weights": s["tw"]}
    moe.moe_expert_ffn(p, w, s["x"], s["offsets"], s["sorted"], s["y"], s["y_shared"], ws)
    return {"y": s["y"], **({"y_shared": s["y_shared"]} if s["case"]["Is"] else {})}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "few":
        return _plain_few(state)
    if op == "ffn":
        return _plain_ffn(state)
    if op == "quantize":
        return _plain_quantize(state)
    return _mx_values(state["codes"], state["scales"], state["e2m1"]).bfloat16()


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _mx64(codes, scales):
    """Sign, two exponent bits and one mantissa bit, as the format defines them."""
    n = torch.empty((*codes.shape, 2), dtype=torch.uint8, device=codes.device)
    n[..., 0] = codes % 16
    n[..., 1] = codes // 16
    n = n.reshape(*codes.shape[:-1], -1).double()
    sign = torch.where(n >= 8, -1.0, 1.0).double()
    ex, man = torch.floor(n % 8 / 2), n % 2
    v = torch.where(ex == 0, man / 2, (1 + man / 2) * torch.pow(torch.full_like(ex, 2.0), ex - 1)) * sign
    return v * torch.pow(torch.tensor(2.0, dtype=torch.float64, device=codes.device), scales.double() - 127).repeat_interleave(32, dim=-1)


def _w64(wdt, w, s):
    if wdt == "mxfp4":
        return _mx64(w, s)
    if wdt == "fp8":
        N, K = w.shape
        return (w.view(torch.float8_e4m3fn).double().reshape(N // 128, 128, K // 128, 128) * s.double()[:, None, :, None]).reshape(N, K)
    return w.double()


def _expert64(x, wg, wu, wd):
    g = torch.matmul(x, wg.T)
    return torch.matmul(g * torch.sigmoid(g) * torch.matmul(x, wu.T), wd.T)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dequantize":
        parts = [_mx64(c, e).float() for c, e in zip(s["codes"].split(4096), s["scales"].split(4096))]
        return torch.cat(parts)  # every value is exact in 32 bits
    if case["op"] == "quantize":
        grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
        done = []
        for part in s["w"].split(16384):
            w = part.double().reshape(part.shape[0], -1, 32)
            amax = w.abs().amax(dim=-1, keepdim=True)
            scale = torch.pow(torch.full_like(amax, 2.0), (torch.frexp(amax)[1] - 3).clamp(min=-127).double())
            a = w.abs() / scale
            # the nearest of the eight values; halfway, the one whose last bit is 0 (an even place in the grid)
            lo = (torch.searchsorted(grid, a, right=True) - 1).clamp(max=6)
            down, up = a - grid[lo], grid[lo + 1] - a
            at = torch.where((up < down) | ((up == down) & (lo % 2 == 1)), lo + 1, lo)
            done.append((torch.copysign(grid[at], w) * scale).reshape(part.shape).float())
        return torch.cat(done)
    T, k, E, Is = case["T"], case["k"], case["E"], case["Is"]
    wdt = case.get("wdt", "mxfp4")
    x = s["x"].double()

    def expert(e):
        return (_w64(wdt, s["w_" + n][e], None if s["s_" + n] is None else s["s_" + n][e]) for n in ("gate", "up", "down"))

    shared = _expert64(x, s["sh_gate"].double(), s["sh_up"].double(), s["sh_down"].double()) if Is else None
    if case["op"] == "ffn":
        y = torch.empty((T * k, case["H"]), dtype=torch.float64, device="cuda")
        off = s["offsets"].tolist()
        for e in range(E):
            if off[e + 1] > off[e]:
                y[off[e]: off[e + 1]] = _expert64(x[s["sorted"][off[e]: off[e + 1]].long() // k], *expert(e))
        return {"y": y, **({"y_shared": shared} if Is else {})}
    p = torch.softmax(x @ s["w_router"].double().T, dim=1)
    top, ids = torch.topk(p, k, dim=1)
    top = top / top.sum(dim=1, keepdim=True)
    out = torch.zeros_like(x)
    for e in sorted(set(ids.flatten().tolist())):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        out[t] += top[t, j, None] * _expert64(x[t], *expert(e))
    if Is:
        out += torch.sigmoid(x @ s["sh_gate_w"].double().T) * shared
    return {"out": out, "ids": None, "weights": top}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] in ("quantize", "dequantize"):
        n = case["rows"] * case["K"]
        packed, values = n / 2 + n / 32, 2 * n
        if case["op"] == "dequantize":
            return {"bytes": packed + values, "flops": n}
        # codes and scales are written, and read back for the values
        return {"bytes": n * (4 if case["src"] == "f32" else 2) + 2 * packed + values, "flops": 3 * n}
    T, H, E, k, I, Is = (case[n] for n in ("T", "H", "E", "k", "I", "Is"))
    wdt = case.get("wdt", "mxfp4")
    size = {"bf16": 2.0, "fp8": 1.0 + 4 / 128**2, "mxfp4": 0.5 + 1 / 32}[wdt]
    touched = E * (1 - (1 - k / E) ** T)  # experts that hold a row, on average over uniform choices
    weights = touched * 3 * H * I * size + 3 * H * Is * 2
    flops = 6.0 * H * (T * k * I + T * Is)
    if case["op"] == "few":
        router = E * H * 2 + (H * 2 if Is else 0)
        return {"bytes": weights + router + 4 * T * H + 8 * T * k, "flops": flops + 2.0 * T * H * E}
    return {"bytes": weights + 2 * T * H + 2 * T * k * H + (2 * T * H if Is else 0) + 4 * (T * k + E + 1), "flops": flops}
