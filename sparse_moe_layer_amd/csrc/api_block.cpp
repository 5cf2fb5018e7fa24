// C ABI of the calls around experts of the caller's own: permute, block norms,
// linear, and their gradients.  Host-side validation, then stream-ordered
// launches; the contract of every entry point is in include/moe_mi355x.h.
#include "moe_mi355x.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "kernels.hpp"

namespace {

constexpr size_t kAlign = 256;
inline size_t up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
inline bool al(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }  // NULL is aligned
inline bool al16(const void* p) { return al(p, 16); }
inline bool al4(const void* p) { return al(p, 4); }
inline moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

moe_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return MOE_ERR_NULL;
  if (!al(ws, kAlign)) return MOE_ERR_ALIGN;
  return ws_bytes < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

moe_status check_norm(const moe_norm_problem* p) {
  if (!p) return MOE_ERR_NULL;
  if (p->dtype != MOE_F32 && p->dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (p->T < 0 || p->H < 1 || p->H > MOE_NORM_MAX_H || p->T > INT32_MAX / p->H) return MOE_ERR_SHAPE;
  if (p->gate < MOE_GATE_NONE || p->gate > MOE_GATE_FULL) return MOE_ERR_SHAPE;
  if (!(p->eps > 0.f) || !std::isfinite(p->eps) || !std::isfinite(p->resid_scale)) return MOE_ERR_SHAPE;
  return p->H % (p->dtype == MOE_F32 ? 4 : 8) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// The gate's pointer, of dtype or (per token) fp32.
bool al_gate(const moe_norm_problem* p, const void* gate) {
  return p->gate == MOE_GATE_TOKEN ? al4(gate) : al16(gate);
}

moe_status check_linear(const moe_linear_problem* p) {
  if (!p) return MOE_ERR_NULL;
  if (p->dtype != MOE_F32 && p->dtype != MOE_BF16) return MOE_ERR_DTYPE;
  const int64_t wide = 1 << 17;
  if (p->rows < 0 || p->rows >= (1 << 24) || p->K < 1 || p->K > wide || p->N < 1 || p->N > wide || p->groups < 1 ||
      p->groups > moe::kMaxExperts || p->N * p->K >= ((int64_t)1 << 30))
    return MOE_ERR_SHAPE;
  if (p->act < MOE_ACT_NONE || p->act > MOE_ACT_GELU) return MOE_ERR_SHAPE;
  const int64_t q = p->dtype == MOE_F32 ? 4 : 8;
  if (p->K % q || p->N % q) return MOE_ERR_UNSUPPORTED;
  if (p->w_stride != 0 && (p->w_stride < p->N * p->K || p->w_stride > ((int64_t)1 << 40))) return MOE_ERR_SHAPE;
  return p->w_stride % q ? MOE_ERR_ALIGN : MOE_OK;
}

size_t dz_bytes(const moe_linear_problem* p) { return up((size_t)p->rows * p->N * (p->dtype == MOE_F32 ? 4 : 2)); }

}  // namespace

extern "C" {

moe_status moe_permute(const moe_problem* p, const void* x, const int32_t* assign_pos, const float* topk_w, void* xs,
                       void* stream) {
  const moe_status st = moe_validate(p);
  if (st != MOE_OK || p->T == 0) return st;
  if (!x || !assign_pos || !xs) return MOE_ERR_NULL;
  if (!al16(x) || !al16(xs) || !al4(assign_pos) || !al4(topk_w)) return MOE_ERR_ALIGN;
  return hip_status(moe::launch_permute(x, assign_pos, topk_w, xs, (int)p->T, (int)p->H, (int)p->k,
                                        p->act_dtype == MOE_F32, (hipStream_t)stream));
}

moe_status moe_permute_backward(const moe_problem* p, const void* dxs, const int32_t* assign_pos, const float* topk_w,
                                const void* x, void* dx, float* dtopk_w, void* stream) {
  const moe_status st = moe_validate(p);
  if (st != MOE_OK || p->T == 0) return st;
  if (!dxs || !assign_pos || !dx || (dtopk_w && !x)) return MOE_ERR_NULL;
  if (!al16(dxs) || !al16(x) || !al16(dx) || !al4(assign_pos) || !al4(topk_w) || !al4(dtopk_w)) return MOE_ERR_ALIGN;
  return hip_status(moe::launch_permute_backward(dxs, assign_pos, topk_w, x, dx, dtopk_w, (int)p->T, (int)p->H,
                                                 (int)p->k, p->act_dtype == MOE_F32, (hipStream_t)stream));
}

moe_status moe_combine_backward(const moe_problem* p, const void* dout, const void* y, const int32_t* assign_pos,
                                const float* topk_w, const void* y_shared, const float* shared_logit, void* dy,
                                float* dtopk_w, void* dy_shared, float* dshared_logit, void* stream) {
  const moe_status st = moe_validate(p);
  if (st != MOE_OK || p->T == 0) return st;
  if (!dout || !assign_pos || !topk_w || !dy || (dtopk_w && !y)) return MOE_ERR_NULL;
  const bool sh = y_shared != nullptr;
  if ((shared_logit != nullptr) != sh || (dy_shared != nullptr) != sh || (dshared_logit != nullptr) != sh)
    return MOE_ERR_NULL;
  if (!al16(dout) || !al16(y) || !al16(dy) || !al16(y_shared) || !al16(dy_shared) || !al4(assign_pos) ||
      !al4(topk_w) || !al4(shared_logit) || !al4(dtopk_w) || !al4(dshared_logit))
    return MOE_ERR_ALIGN;
  return hip_status(moe::launch_combine_backward(dout, y, assign_pos, topk_w, y_shared, shared_logit, dy, dtopk_w,
                                                 dy_shared, dshared_logit, (int)p->T, (int)p->H, (int)p->k,
                                                 p->act_dtype == MOE_F32, (hipStream_t)stream));
}

moe_status moe_block_norm(const moe_norm_problem* p, const void* f, const void* resid, const void* g_post,
                          const void* gate, const void* g_pre, void* resid_out, void* x, void* stream) {
  const moe_status st = check_norm(p);
  if (st != MOE_OK || p->T == 0) return st;
  if (!resid || (!resid_out && !x) || (g_pre == nullptr) != (x == nullptr)) return MOE_ERR_NULL;
  if ((gate == nullptr) != (p->gate == MOE_GATE_NONE) || (!f && (g_post || gate))) return MOE_ERR_NULL;
  if (!al16(f) || !al16(resid) || !al16(g_post) || !al_gate(p, gate) || !al16(g_pre) || !al16(resid_out) || !al16(x))
    return MOE_ERR_ALIGN;
  moe::NormArgs a{f, resid, g_post, gate, g_pre, resid_out, x, 0, p->gate, 1.f / (float)p->H, p->eps, p->resid_scale};
  const bool f32 = p->dtype == MOE_F32;
  a.nch = (int)p->H / (f32 ? 4 : 8);
  return hip_status(moe::launch_norm(a, (int)p->T, f32, (hipStream_t)stream));
}

size_t moe_block_norm_workspace_bytes(const moe_norm_problem* p) {
  if (check_norm(p) != MOE_OK) return 0;
  return up(moe::norm_partial_floats(p->T, p->H) * 4) + kAlign;  // never 0 for a valid problem
}

moe_status moe_block_norm_backward(const moe_norm_problem* p, const void* dresid_out, const void* dx, const void* f,
                                   const void* resid_out, const void* g_post, const void* gate, const void* g_pre,
                                   void* dresid, void* df, float* dg_post, void* dgate, float* dg_pre, void* ws,
                                   size_t ws_bytes, void* stream) {
  moe_status st = check_norm(p);
  if (st != MOE_OK) return st;
  if (p->T == 0) {  // the sums over no tokens; the gradients with a row a token are empty
    float* sum = p->gate == MOE_GATE_CHANNEL ? static_cast<float*>(dgate) : nullptr;
    if (!al4(dg_post) || !al4(dg_pre) || !al4(sum)) return MOE_ERR_ALIGN;
    if (!dg_post && !dg_pre && !sum) return MOE_OK;
    return hip_status(moe::launch_norm_no_rows(dg_post, dg_pre, sum, (int)p->H, (hipStream_t)stream));
  }
  if (!dresid_out && !dx) return MOE_ERR_NULL;
  if (dx && (!resid_out || !g_pre)) return MOE_ERR_NULL;
  if ((f == nullptr) != (df == nullptr) || (!f && !dresid)) return MOE_ERR_NULL;
  if ((gate == nullptr) != (p->gate == MOE_GATE_NONE) || (!f && (g_post || gate))) return MOE_ERR_NULL;
  if ((dg_post && !g_post) || (dgate && !gate) || (dg_pre && !dx)) return MOE_ERR_NULL;
  if (!al16(dresid_out) || !al16(dx) || !al16(f) || !al16(resid_out) || !al16(g_post) || !al_gate(p, gate) ||
      !al16(g_pre) || !al16(dresid) || !al16(df) || !al4(dg_post) || !al4(dg_pre) ||
      !(p->gate == MOE_GATE_FULL ? al16(dgate) : al4(dgate)))
    return MOE_ERR_ALIGN;
  if ((st = check_ws(ws, ws_bytes, moe_block_norm_workspace_bytes(p))) != MOE_OK) return st;
  moe::NormBackArgs a{};
  a.dresid_out = dresid_out;
  a.dx = dx;
  a.f = f;
  a.resid_out = resid_out;
  a.g_post = g_post;
  a.gate = gate;
  a.g_pre = g_pre;
  a.dresid = dresid;
  a.df = df;
  a.dg_post = dg_post;
  a.dgate = dgate;
  a.dg_pre = dg_pre;
  a.partial = static_cast<float*>(ws);
  const bool f32 = p->dtype == MOE_F32;
  a.T = (int)p->T;
  a.nch = (int)p->H / (f32 ? 4 : 8);
  a.gate_kind = p->gate;
  a.inv_h = 1.f / (float)p->H;
  a.eps = p->eps;
  a.scale = p->resid_scale;
  return hip_status(moe::launch_norm_backward(a, f32, (hipStream_t)stream));
}

moe_status moe_linear(const moe_linear_problem* p, const void* x, const void* w, const void* bias,
                      const int32_t* offsets, const void* mul, const void* resid, void* y, void* z, void* stream) {
  const moe_status st = check_linear(p);
  if (st != MOE_OK || p->rows == 0) return st;
  if (!x || !w || !y || (!offsets && p->groups > 1)) return MOE_ERR_NULL;
  if (!al16(x) || !al16(w) || !al16(bias) || !al16(mul) || !al16(resid) || !al16(y) || !al16(z) || !al4(offsets))
    return MOE_ERR_ALIGN;
  const moe::LinearArgs a{x, w, bias, offsets, mul, resid, y, z, (int)p->rows, (int)p->K, (int)p->N, (int)p->groups,
                          p->w_stride ? p->w_stride : p->N * p->K, p->act};
  return hip_status(moe::launch_linear(a, p->dtype == MOE_F32, (hipStream_t)stream));
}

size_t moe_linear_workspace_bytes(const moe_linear_problem* p) {
  if (check_linear(p) != MOE_OK) return 0;
  return dz_bytes(p) + up(moe::linear_partial_floats(p->rows, p->N, p->groups, p->dtype == MOE_F32) * 4) + kAlign;
}

moe_status moe_linear_backward(const moe_linear_problem* p, const void* dy, const void* x, const void* w,
                               const int32_t* offsets, const void* mul, const void* z, void* dx, void* dw,
                               float* dbias, void* dmul, void* ws, size_t ws_bytes, void* stream) {
  moe_status st = check_linear(p);
  if (st != MOE_OK) return st;
  if (p->rows == 0 && !dw && !dbias) return MOE_OK;
  if (p->rows > 0) {
    if (!dy || (!offsets && p->groups > 1)) return MOE_ERR_NULL;
    if ((dx && !w) || (dw && !x) || (dmul && !mul) || ((p->act != MOE_ACT_NONE || dmul) && !z)) return MOE_ERR_NULL;
  }
  if (!al16(dy) || !al16(x) || !al16(w) || !al16(mul) || !al16(z) || !al16(dx) || !al16(dw) || !al16(dmul) ||
      !al4(offsets) || !al4(dbias))
    return MOE_ERR_ALIGN;
  if ((st = check_ws(ws, ws_bytes, moe_linear_workspace_bytes(p))) != MOE_OK) return st;
  moe::LinearBackArgs a{};
  a.dy = dy;
  a.x = x;
  a.w = w;
  a.offsets = p->rows ? offsets : nullptr;
  a.mul = mul;
  a.z = z;
  a.dx = dx;
  a.dw = dw;
  a.dbias = dbias;
  a.dmul = dmul;
  a.dz = ws;
  a.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + dz_bytes(p));
  a.rows = (int)p->rows;
  a.K = (int)p->K;
  a.N = (int)p->N;
  a.G = (int)p->groups;
  a.w_stride = p->w_stride ? p->w_stride : p->N * p->K;
  a.act = p->act;
  return hip_status(moe::launch_linear_backward(a, p->dtype == MOE_F32, (hipStream_t)stream));
}

}  // extern "C"
