"""Routed Mixture-of-Experts FFN layer for AMD Instinct MI355X (gfx950).

Python face of the C ABI in include/moe_mi355x.h: the functions below have
the C entry points' names and arguments, take torch tensors (device memory)
and pass their pointers plus the current HIP stream to the library.  No
computation happens here.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._lib import (LIB, MOE_BF16, MOE_F32, MOE_FLAG_FORCE_GEMM, MOE_FLAG_FORCE_STREAM,  # noqa: F401
                   MOE_FLAG_GEMM_TILE_128, MOE_FLAG_GEMM_TILE_256, MOE_FLAG_PAGE_ROUTING, MOE_FP8_E4M3FN,
                   MOE_FEW_MAX_TOKENS, MOE_MXFP4, MOE_NOALLOC_SCRATCH_BYTES, MOE_OK, EXPORTS, moe_audit_stats,
                   moe_gr_weights, moe_problem,
                   moe_weights,
                   MOE_ACT_GELU, MOE_ACT_NONE, MOE_ACT_SILU, MOE_GATE_CHANNEL, MOE_GATE_FULL, MOE_GATE_NONE,
                   MOE_GATE_TOKEN, MOE_NORM_MAX_H, moe_linear_problem, moe_norm_problem)

_DT = {"f32": MOE_F32, "bf16": MOE_BF16, "fp8": MOE_FP8_E4M3FN, "mxfp4": MOE_MXFP4}


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {LIB.moe_status_str(status).decode()} (status {status})")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the MoE library must be contiguous")
    return t.data_ptr()


# The current stream's handle without a Stream object around it (2.8 -> 0.4 us of a call), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(st: int, where: str):
    if st != MOE_OK:
        raise MoEError(st, where)


def problem(T, H, E, k, I, I_shared=0, act="bf16", wdt="bf16", scale_block=128, flags=0) -> moe_problem:
    return moe_problem(T, H, E, k, I, I_shared, _DT[act], _DT[wdt], scale_block, flags)


def weights(w_router, w_gate, w_up, w_down, s_gate=None, s_up=None, s_down=None, sh_gate=None, sh_up=None,
            sh_down=None, sh_gate_w=None, stride_gate=0, stride_up=0, stride_down=0) -> moe_weights:
    return moe_weights(_ptr(w_router), _ptr(w_gate), _ptr(w_up), _ptr(w_down), stride_gate, stride_up,
                       stride_down, _ptr(s_gate), _ptr(s_up), _ptr(s_down), _ptr(sh_gate), _ptr(sh_up),
                       _ptr(sh_down), _ptr(sh_gate_w))


def moe_abi_version() -> int:
    return LIB.moe_abi_version()


def moe_validate(p: moe_problem) -> int:
    return LIB.moe_validate(ctypes.byref(p))


def moe_workspace_bytes(p: moe_problem) -> int:
    return LIB.moe_workspace_bytes(ctypes.byref(p))


def workspace(p: moe_problem, device="cuda") -> torch.Tensor:
    """A device buffer of moe_workspace_bytes(p) bytes (torch allocations are 256-byte aligned)."""
    n = moe_workspace_bytes(p)
    if n == 0:
        _check(moe_validate(p), "moe_workspace_bytes")
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def moe_route(p, x, w_router, sh_gate_w, topk_ids, topk_w, shared_logit, ws, stream=None):
    _check(LIB.moe_route(ctypes.byref(p), _ptr(x), _ptr(w_router), _ptr(sh_gate_w), _ptr(topk_ids), _ptr(topk_w),
                         _ptr(shared_logit), _ptr(ws), ws.numel(), _stream(stream)), "moe_route")


def moe_dispatch(p, topk_ids, expert_offsets, sorted_assign, assign_pos, ws, stream=None):
    _check(LIB.moe_dispatch(ctypes.byref(p), _ptr(topk_ids), _ptr(expert_offsets), _ptr(sorted_assign),
                            _ptr(assign_pos), _ptr(ws), ws.numel(), _stream(stream)), "moe_dispatch")


def moe_expert_ffn(p, w: moe_weights, x, expert_offsets, sorted_assign, y, y_shared, ws, stream=None):
    _check(LIB.moe_expert_ffn(ctypes.byref(p), ctypes.byref(w), _ptr(x), _ptr(expert_offsets), _ptr(sorted_assign),
                              _ptr(y), _ptr(y_shared), _ptr(ws), ws.numel(), _stream(stream)), "moe_expert_ffn")


def moe_expert_gate_up(p, w: moe_weights, x, expert_offsets, sorted_assign, h, h_shared, ws, stream=None):
    _check(LIB.moe_expert_gate_up(ctypes.byref(p), ctypes.byref(w), _ptr(x), _ptr(expert_offsets),
                                  _ptr(sorted_assign), _ptr(h), _ptr(h_shared), _ptr(ws), ws.numel(),
                                  _stream(stream)), "moe_expert_gate_up")


def moe_expert_down(p, w: moe_weights, expert_offsets, h, h_shared, y, y_shared, ws, stream=None):
    _check(LIB.moe_expert_down(ctypes.byref(p), ctypes.byref(w), _ptr(expert_offsets), _ptr(h), _ptr(h_shared),
                               _ptr(y), _ptr(y_shared), _ptr(ws), ws.numel(), _stream(stream)), "moe_expert_down")


def moe_combine(p, y, assign_pos, topk_w, y_shared, shared_logit, out, stream=None):
    _check(LIB.moe_combine(ctypes.byref(p), _ptr(y), _ptr(assign_pos), _ptr(topk_w), _ptr(y_shared),
                           _ptr(shared_logit), _ptr(out), _stream(stream)), "moe_combine")


def moe_layer_forward(p, w: moe_weights, x, out, topk_ids, topk_w, ws, stream=None):
    _check(LIB.moe_layer_forward(ctypes.byref(p), ctypes.byref(w), _ptr(x), _ptr(out), _ptr(topk_ids),
                                 _ptr(topk_w), _ptr(ws), ws.numel(), _stream(stream)), "moe_layer_forward")


def moe_hbm_read_probe(src, sink, stream=None):
    _check(LIB.moe_hbm_read_probe(_ptr(src), src.numel() * src.element_size(), _ptr(sink), _stream(stream)),
           "moe_hbm_read_probe")


def moe_mfma_pipe_probe(variant: int, steps: int, src, sink, stream=None):
    nbytes = 0 if src is None else src.numel() * src.element_size()
    _check(LIB.moe_mfma_pipe_probe(variant, steps, _ptr(src), nbytes, _ptr(sink), _stream(stream)),
           "moe_mfma_pipe_probe")


def moe_layer_forward_noalloc(p, w: moe_weights, x, out, topk_ids, topk_w, stream=None):
    _check(LIB.moe_layer_forward_noalloc(ctypes.byref(p), ctypes.byref(w), _ptr(x), _ptr(out), _ptr(topk_ids),
                                         _ptr(topk_w), _stream(stream)), "moe_layer_forward_noalloc")


def moe_few_workspace_bytes(p: moe_problem) -> int:
    return LIB.moe_few_workspace_bytes(ctypes.byref(p))


def few_workspace(p: moe_problem, device="cuda") -> torch.Tensor:
    """A device buffer of moe_few_workspace_bytes(p) bytes."""
    n = moe_few_workspace_bytes(p)
    if n == 0:
        st = moe_validate(p)
        raise MoEError(st if st != MOE_OK else 6, "moe_few_workspace_bytes")  # 6: MOE_ERR_UNSUPPORTED
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_layer_forward_few(p, w: moe_weights, x, out, topk_ids, topk_w, ws, stream=None):
    """The whole layer for at most MOE_FEW_MAX_TOKENS tokens; ws: few_workspace(p)."""
    _check(LIB.moe_layer_forward_few(ctypes.byref(p), ctypes.byref(w), _ptr(x), _ptr(out), _ptr(topk_ids),
                                     _ptr(topk_w), _ptr(ws), ws.numel(), _stream(stream)), "moe_layer_forward_few")


def gr_weights(norm_w, w_read, w_up, rank: int, eps: float = 1e-6) -> moe_gr_weights:
    return moe_gr_weights(_ptr(norm_w), _ptr(w_read), _ptr(w_up), rank, eps)


def moe_gr_workspace_bytes(p: moe_problem, rank: int) -> int:
    return LIB.moe_gr_workspace_bytes(ctypes.byref(p), rank)


def gr_workspace(p: moe_problem, rank: int, device="cuda") -> torch.Tensor:
    """A device buffer of moe_gr_workspace_bytes(p, rank) bytes."""
    n = moe_gr_workspace_bytes(p, rank)
    if n == 0:
        st = LIB.moe_validate(ctypes.byref(p))
        raise MoEError(st if st != MOE_OK else 6, "moe_gr_workspace_bytes")  # 6: MOE_ERR_UNSUPPORTED
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_gr_read(p, g: moe_gr_weights, resid, x, s, ws, stream=None):
    _check(LIB.moe_gr_read(ctypes.byref(p), ctypes.byref(g), _ptr(resid), _ptr(x), _ptr(s), _ptr(ws), ws.numel(),
                           _stream(stream)), "moe_gr_read")


def moe_gr_write(p, resid, s, f, resid_out, stream=None):
    _check(LIB.moe_gr_write(ctypes.byref(p), _ptr(resid), _ptr(s), _ptr(f), _ptr(resid_out), _stream(stream)),
           "moe_gr_write")


def moe_combine_gr_write(p, y, assign_pos, topk_w, y_shared, shared_logit, resid, s, out, resid_out, stream=None):
    _check(LIB.moe_combine_gr_write(ctypes.byref(p), _ptr(y), _ptr(assign_pos), _ptr(topk_w), _ptr(y_shared),
                                    _ptr(shared_logit), _ptr(resid), _ptr(s), _ptr(out), _ptr(resid_out),
                                    _stream(stream)), "moe_combine_gr_write")


# numpy dtype of one moe_audit_stats record (int64 n, n_zero, n_nan; float64 median, mad, sigma_rob)
AUDIT_STATS_FIELDS = ("n", "n_zero", "n_nan", "median", "mad", "sigma_rob")


def moe_audit_workspace_bytes(slices: int) -> int:
    return LIB.moe_audit_workspace_bytes(slices)


def audit_workspace(slices: int, device="cuda") -> torch.Tensor:
    n = moe_audit_workspace_bytes(slices)
    if n == 0:
        raise MoEError(2, "moe_audit_workspace_bytes")  # 2: MOE_ERR_SHAPE
    return torch.empty(n, dtype=torch.uint8, device=device)


def audit_stats_buffer(slices: int, device="cuda") -> torch.Tensor:
    """Device buffer for slices + 1 records (48 bytes each, 8-byte aligned)."""
    return torch.empty((slices + 1, 6), dtype=torch.float64, device=device)


def moe_weight_audit(w, slices: int, n: int, slice_stride: int, stats, ws, stream=None):
    """w: bf16 device tensor; stats: audit_stats_buffer(slices)."""
    if w.dtype != torch.bfloat16:
        raise MoEError(6, "moe_weight_audit")  # 6: MOE_ERR_UNSUPPORTED
    _check(LIB.moe_weight_audit(_ptr(w), MOE_BF16, slices, n, slice_stride, _ptr(stats), _ptr(ws), ws.numel(),
                                _stream(stream)), "moe_weight_audit")


def audit_records(stats: torch.Tensor) -> list:
    """Host dicts of the records in an audit_stats_buffer (after the stream is synchronised)."""
    host = stats.detach().cpu().contiguous()
    ints = host.view(torch.int64)
    return [{"n": int(ints[i, 0]), "n_zero": int(ints[i, 1]), "n_nan": int(ints[i, 2]),
             "median": float(host[i, 3]), "mad": float(host[i, 4]), "sigma_rob": float(host[i, 5])}
            for i in range(host.shape[0])]


def _mx_shape(values, codes, scales, where: str):
    """(rows, K, row stride) of a matrix of values [.., K] (the last dimension contiguous, the ones before it one
    run of rows) with packed codes [.., K/2] and scales [.., K/32]."""
    shape = values.shape
    K = shape[-1]
    lead = shape[:-1]
    if codes.shape != (*lead, K // 2) or scales.shape != (*lead, K // 32) or K % 32 or K < 32:
        raise ValueError(f"{where}: codes must be [.., K/2] and scales [.., K/32] for values [.., K], K a multiple "
                         "of 32")
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise ValueError(f"{where}: codes and scales are uint8 tensors")
    if values.get_device() != codes.get_device() or values.get_device() != scales.get_device():
        raise ValueError(f"{where}: tensors on different devices")
    rows = codes.numel() // (K // 2)
    if values.is_contiguous():
        stride = K
    elif values.dim() != 2 or values.stride(1) != 1 or values.stride(0) < K:
        raise ValueError(f"{where}: values must be contiguous, or 2-D with contiguous rows")
    else:
        stride = values.stride(0)
    _on_current_device(values, where)
    return rows, K, stride


def _on_current_device(t, where: str):
    """The entry points launch on the current device's stream, so their tensors lie there."""
    if not t.is_cuda or t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{where}: tensors must be on the current CUDA device")


def moe_mx_quantize(w, codes, scales, stream=None):
    """w [.., K] (bf16 or fp32) -> MXFP4 codes [.., K/2] and E8M0 scales [.., K/32] (uint8)."""
    if w.dtype not in (torch.bfloat16, torch.float32):
        raise MoEError(3, "moe_mx_quantize")  # 3: MOE_ERR_DTYPE
    rows, K, stride = _mx_shape(w, codes, scales, "moe_mx_quantize")
    _check(LIB.moe_mx_quantize(w.data_ptr(), MOE_F32 if w.dtype == torch.float32 else MOE_BF16, rows, K, stride,
                               _ptr(codes), _ptr(scales), _stream(stream)), "moe_mx_quantize")


def moe_mx_dequantize(codes, scales, w, stream=None):
    """MXFP4 codes [.., K/2] and scales [.., K/32] -> their values, w [.., K] bf16."""
    if w.dtype != torch.bfloat16:
        raise MoEError(3, "moe_mx_dequantize")  # 3: MOE_ERR_DTYPE
    rows, K, stride = _mx_shape(w, codes, scales, "moe_mx_dequantize")
    _check(LIB.moe_mx_dequantize(_ptr(codes), _ptr(scales), rows, K, w.data_ptr(), stride, _stream(stream)),
           "moe_mx_dequantize")


def mx_quantize(w, stream=None):
    """MXFP4 form of a weight tensor [.., K]: (codes [.., K/2], scales [.., K/32]), uint8, on w's device."""
    if w.shape[-1] % 32 or w.shape[-1] < 32:
        raise MoEError(6, "moe_mx_quantize")  # 6: MOE_ERR_UNSUPPORTED
    codes = torch.empty((*w.shape[:-1], w.shape[-1] // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((*w.shape[:-1], w.shape[-1] // 32), dtype=torch.uint8, device=w.device)
    moe_mx_quantize(w, codes, scales, stream)
    return codes, scales


# ---------------------------------------------------------------------------
# a block around experts of the caller's own, and its gradients
# ---------------------------------------------------------------------------
_GATES = {"none": MOE_GATE_NONE, "token": MOE_GATE_TOKEN, "channel": MOE_GATE_CHANNEL, "full": MOE_GATE_FULL}
_ACTS = {"none": MOE_ACT_NONE, "silu": MOE_ACT_SILU, "gelu": MOE_ACT_GELU}
_TORCH_DT = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16}


def norm_problem(T, H, dtype="bf16", gate="none", eps=1e-6, resid_scale=1.0) -> moe_norm_problem:
    return moe_norm_problem(T, H, _DT[dtype], _GATES[gate], eps, resid_scale)


def linear_problem(rows, K, N, groups=1, dtype="bf16", act="none", w_stride=0) -> moe_linear_problem:
    return moe_linear_problem(rows, K, N, groups, w_stride, _DT[dtype], _ACTS[act])


def _bad(where: str, t, n: int, dtype, dev: int):
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{where}: a contiguous tensor of {n} values of {dtype} is needed, not {tuple(t.shape)} of "
                         f"{t.dtype}{'' if t.is_contiguous() else ', strided'}")
    raise ValueError(f"{where}: tensors must be on the current CUDA device")


def _arg(where: str, t, n: int, dtype, dev: int):
    """Pointer of a call's tensor (or None): contiguous, n values of dtype, on the current device, where the library
    launches."""
    if t is None:
        return None
    if t.dtype is dtype and t.numel() == n and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    return _bad(where, t, n, dtype, dev)


def _ws_arg(where: str, t, dev: int):
    if t is None:
        return None, 0
    n = t.numel()
    return _arg(where, t, n, t.dtype, dev), n * t.element_size()


def _act_of(code: int):
    return _TORCH_DT.get(code, torch.bfloat16)  # another dtype is the library's to refuse


def _stream_on(where: str, stream, dev: int):
    if stream is None:
        return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream
    if getattr(stream, "device_index", dev) != dev:
        raise ValueError(f"{where}: the stream must be one of the current CUDA device")
    return _stream(stream)


_I32, _F32 = torch.int32, torch.float32


def moe_permute(p, x, assign_pos, topk_w, xs, stream=None):
    """x [T, H] -> xs [T*k, H]: xs[assign_pos[t*k+j]] = topk_w[t, j] * x[t] (topk_w None: x[t])."""
    f, d, dt, H, R = "moe_permute", torch.cuda.current_device(), _act_of(p.act_dtype), p.H, p.T * p.k
    _check(LIB.moe_permute(p, _arg(f, x, p.T * H, dt, d), _arg(f, assign_pos, R, _I32, d),
                           _arg(f, topk_w, R, _F32, d), _arg(f, xs, R * H, dt, d), _stream_on(f, stream, d)), f)


def moe_permute_backward(p, dxs, assign_pos, topk_w, x, dx, dtopk_w, stream=None):
    """Gradients of moe_permute: dx [T, H], and dtopk_w [T, k] where it is not None (x is read for it alone)."""
    f, d, dt, H, R = "moe_permute_backward", torch.cuda.current_device(), _act_of(p.act_dtype), p.H, p.T * p.k
    n = p.T * H
    _check(LIB.moe_permute_backward(p, _arg(f, dxs, R * H, dt, d), _arg(f, assign_pos, R, _I32, d),
                                    _arg(f, topk_w, R, _F32, d), _arg(f, x, n, dt, d), _arg(f, dx, n, dt, d),
                                    _arg(f, dtopk_w, R, _F32, d), _stream_on(f, stream, d)), f)


def moe_combine_backward(p, dout, y, assign_pos, topk_w, y_shared, shared_logit, dy, dtopk_w, dy_shared,
                         dshared_logit, stream=None):
    """Gradients of moe_combine: dy [T*k, H], dtopk_w [T, k] (or None), dy_shared [T, H], dshared_logit [T]."""
    f, d, dt, T, H = "moe_combine_backward", torch.cuda.current_device(), _act_of(p.act_dtype), p.T, p.H
    n, R = T * H, T * p.k
    _check(LIB.moe_combine_backward(p, _arg(f, dout, n, dt, d), _arg(f, y, R * H, dt, d),
                                    _arg(f, assign_pos, R, _I32, d), _arg(f, topk_w, R, _F32, d),
                                    _arg(f, y_shared, n, dt, d), _arg(f, shared_logit, T, _F32, d),
                                    _arg(f, dy, R * H, dt, d), _arg(f, dtopk_w, R, _F32, d),
                                    _arg(f, dy_shared, n, dt, d), _arg(f, dshared_logit, T, _F32, d),
                                    _stream_on(f, stream, d)), f)


def _gate_arg(f, p, t, dt, dev, summed: bool):
    """A gate ([T] fp32, [H], [T, H]), or its gradient, which is fp32 where it is summed over rows or columns."""
    if t is None:
        return None
    if p.gate == MOE_GATE_FULL:
        return _arg(f, t, p.T * p.H, dt, dev)
    if p.gate == MOE_GATE_CHANNEL:
        return _arg(f, t, p.H, _F32 if summed else dt, dev)
    return _arg(f, t, p.T, _F32, dev)


def moe_block_norm(p: moe_norm_problem, f, resid, g_post, gate, g_pre, resid_out, x, stream=None):
    """resid_out = resid_scale * resid + gate * RMSNorm(f) g_post, x = RMSNorm(resid_out) g_pre (None: left out)."""
    w, d, dt, H = "moe_block_norm", torch.cuda.current_device(), _act_of(p.dtype), p.H
    n = p.T * H
    _check(LIB.moe_block_norm(p, _arg(w, f, n, dt, d), _arg(w, resid, n, dt, d), _arg(w, g_post, H, dt, d),
                              _gate_arg(w, p, gate, dt, d, False), _arg(w, g_pre, H, dt, d),
                              _arg(w, resid_out, n, dt, d), _arg(w, x, n, dt, d), _stream_on(w, stream, d)), w)


def moe_block_norm_workspace_bytes(p: moe_norm_problem) -> int:
    return LIB.moe_block_norm_workspace_bytes(p)


def norm_workspace(p: moe_norm_problem, device="cuda") -> torch.Tensor:
    """A device buffer of moe_block_norm_workspace_bytes(p) bytes."""
    n = moe_block_norm_workspace_bytes(p)
    if n == 0:
        raise MoEError(2, "moe_block_norm_workspace_bytes")  # 2: MOE_ERR_SHAPE
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_block_norm_backward(p: moe_norm_problem, dresid_out, dx, f, resid_out, g_post, gate, g_pre, dresid, df,
                            dg_post, dgate, dg_pre, ws, stream=None):
    """Gradients of moe_block_norm; dg_post, dg_pre [H] fp32, dgate [T] or [H] fp32 or [T, H]; ws: norm_workspace(p)."""
    w, d, dt, H = "moe_block_norm_backward", torch.cuda.current_device(), _act_of(p.dtype), p.H
    n = p.T * H
    _check(LIB.moe_block_norm_backward(p, _arg(w, dresid_out, n, dt, d), _arg(w, dx, n, dt, d), _arg(w, f, n, dt, d),
                                       _arg(w, resid_out, n, dt, d), _arg(w, g_post, H, dt, d),
                                       _gate_arg(w, p, gate, dt, d, False), _arg(w, g_pre, H, dt, d),
                                       _arg(w, dresid, n, dt, d), _arg(w, df, n, dt, d), _arg(w, dg_post, H, _F32, d),
                                       _gate_arg(w, p, dgate, dt, d, True), _arg(w, dg_pre, H, _F32, d),
                                       *_ws_arg(w, ws, d), _stream_on(w, stream, d)), w)


def _weights_arg(f, p, w, dt, dev):
    """[groups, N, K] contiguous, or at p.w_stride from one contiguous matrix to the next (a slice of a fused
    [groups, 2 N, K] tensor)."""
    if w is None or p.w_stride in (0, p.N * p.K) or p.groups < 1:
        return _arg(f, w, p.groups * p.N * p.K, dt, dev)
    want = (p.groups, p.N, p.K)
    if tuple(w.shape) != want or (p.groups > 1 and w.stride(0) != p.w_stride):
        raise ValueError(f"{f}: weights must be {want} with {p.w_stride} values from one matrix to the next")
    return _arg(f, w[0], p.N * p.K, dt, dev)  # the first matrix's


def moe_linear(p: moe_linear_problem, x, w, bias, offsets, mul, resid, y, z, stream=None):
    """y[r] = resid[r] + act(x[r] W_g^T + bias_g) * mul[r] for the rows r of each group g (bias, mul, resid, z may be
    None; offsets [groups + 1] int32, None for one group); z receives the activation's argument."""
    f, d, dt, rows, G = "moe_linear", torch.cuda.current_device(), _act_of(p.dtype), p.rows, p.groups
    n = rows * p.N
    _check(LIB.moe_linear(p, _arg(f, x, rows * p.K, dt, d), _weights_arg(f, p, w, dt, d),
                          _arg(f, bias, G * p.N, dt, d), _arg(f, offsets, G + 1, _I32, d), _arg(f, mul, n, dt, d),
                          _arg(f, resid, n, dt, d), _arg(f, y, n, dt, d), _arg(f, z, n, dt, d),
                          _stream_on(f, stream, d)), f)


def moe_linear_workspace_bytes(p: moe_linear_problem) -> int:
    return LIB.moe_linear_workspace_bytes(p)


def linear_workspace(p: moe_linear_problem, device="cuda") -> torch.Tensor:
    """A device buffer of moe_linear_workspace_bytes(p) bytes."""
    n = moe_linear_workspace_bytes(p)
    if n == 0:
        raise MoEError(2, "moe_linear_workspace_bytes")  # 2: MOE_ERR_SHAPE
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_linear_backward(p: moe_linear_problem, dy, x, w, offsets, mul, z, dx, dw, dbias, dmul, ws, stream=None):
    """Gradients of moe_linear (each output may be None; dbias [groups, N] fp32); ws: linear_workspace(p)."""
    f, d, dt, rows, G = "moe_linear_backward", torch.cuda.current_device(), _act_of(p.dtype), p.rows, p.groups
    n, m = rows * p.N, rows * p.K
    _check(LIB.moe_linear_backward(p, _arg(f, dy, n, dt, d), _arg(f, x, m, dt, d), _weights_arg(f, p, w, dt, d),
                                   _arg(f, offsets, G + 1, _I32, d), _arg(f, mul, n, dt, d), _arg(f, z, n, dt, d),
                                   _arg(f, dx, m, dt, d), _weights_arg(f, p, dw, dt, d),
                                   _arg(f, dbias, G * p.N, _F32, d), _arg(f, dmul, n, dt, d), *_ws_arg(f, ws, d),
                                   _stream_on(f, stream, d)), f)


_DT_OF_TORCH = {torch.float32: "f32", torch.bfloat16: "bf16", torch.uint8: "fp8"}


def layer_forward(x, k: int, w_router, w_gate, w_up, w_down, s_gate=None, s_up=None, s_down=None, sh_gate=None,
                  sh_up=None, sh_down=None, sh_gate_w=None, flags: int = 0, stream=None):
    """The whole layer in one call: returns (out [T, H], ids [T, k] int32, w [T, k] fp32).

    Shapes come from the tensors: x [T, H] (bf16 or fp32), w_router [E, H], w_gate / w_up [E, I, H],
    w_down [E, H, I] (bf16, fp32, or uint8 e4m3fn codes with fp32 128 x 128 block scales s_*; or
    MXFP4: uint8 codes [E, I, H/2], [E, H, I/2] with uint8 scales s_*, as mx_quantize makes them), and
    the optional shared expert sh_gate / sh_up [I_s, H], sh_down [H, I_s], sh_gate_w [1, H].
    Outputs and the workspace are allocated on x's device; every computation runs in the library.
    """
    T, H = x.shape
    E, I = w_gate.shape[0], w_gate.shape[1]
    Is = sh_gate.shape[0] if sh_gate is not None else 0
    wdt = "mxfp4" if s_gate is not None and s_gate.dtype == torch.uint8 else _DT_OF_TORCH[w_gate.dtype]
    P = problem(T, H, E, k, I, Is, _DT_OF_TORCH[x.dtype], wdt, 32 if wdt == "mxfp4" else 128, flags)
    W = weights(w_router, w_gate, w_up, w_down, s_gate, s_up, s_down, sh_gate, sh_up, sh_down, sh_gate_w)
    ws = workspace(P, device=x.device)
    out = torch.empty((T, H), dtype=x.dtype, device=x.device)
    ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
    tw = torch.empty((T, k), dtype=torch.float32, device=x.device)
    moe_layer_forward(P, W, x, out, ids, tw, ws, stream)
    return out, ids, tw
