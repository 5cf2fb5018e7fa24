// The norm behind a block, its gate, the scaled residual and the norm before
// the next block in one pass, and the gradients in one pass:
//   n  = f rstd(f) g_post (or f)         rstd(v) = 1 / sqrt(mean v^2 + eps)
//   r' = c r + gate n,   x = r' rstd(r') g_pre
//   dr = dr' + rstd(r') (g_pre dx - r' rstd(r')^2 mean(g_pre dx r'))
//   dresid = c dr,  dgate = n dr,  dn = gate dr
//   df = rstd(f) (g_post dn - f rstd(f)^2 mean(g_post dn f))
//   dg_post = sum_t dn f rstd(f),  dg_pre = sum_t dx r' rstd(r')
// HBM-bound: every [T, H] tensor is read or written once.  A row stays in its
// workgroup's registers (NCH 16-byte chunks a thread) between the sums over it.
// The sums over tokens (gains, channel gate) stay in registers over a
// workgroup's rows; its partial sums go to the workspace and a second kernel
// adds the workgroups', in a fixed order.
#include "kernels.hpp"
#include "vec.hpp"

namespace moe {
namespace {

constexpr int kMaxWaves = 16;

// Sums of P values over the workgroup, in every thread.  red: [kMaxWaves][P]
// (one use per barrier interval: callers alternate two).
template <int P>
__device__ __forceinline__ void block_sums(float (&a)[P], float* red, int lane, int wave, int nw) {
  const float s = wave_sums<P>(a, lane);
  constexpr int kStep = 64 / P;
  if (lane % kStep == 0) red[wave * P + lane / kStep] = s;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < P; ++i) a[i] = 0.f;
  for (int w = 0; w < nw; ++w)
#pragma unroll
    for (int i = 0; i < P; ++i) a[i] += red[w * P + i];
}

template <bool F32, int NCH>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a) {
  using V = Vec<F32>;
  __shared__ float red[2][kMaxWaves];
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
  const int64_t base = (int64_t)t * a.nch;
  const u32x4* f = static_cast<const u32x4*>(a.f);
  const u32x4* resid = static_cast<const u32x4*>(a.resid);
  const u32x4* gate = static_cast<const u32x4*>(a.gate);
  const u32x4* g_post = static_cast<const u32x4*>(a.g_post);
  const u32x4* g_pre = static_cast<const u32x4*>(a.g_pre);
  u32x4 vf[NCH] = {}, vr[NCH] = {}, vg[NCH] = {};
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = tid + i * blockDim.x;
    if (c >= a.nch) continue;
    vr[i] = ld16_nt(resid + base + c);
    if (f) vf[i] = ld16_nt(f + base + c);
    if (a.gate_kind == MOE_GATE_FULL) vg[i] = ld16_nt(gate + base + c);
    if (a.gate_kind == MOE_GATE_CHANNEL) vg[i] = ld16(gate + c);
  }
  float rf = 1.f;
  if (g_post) {
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      float v[V::N];
      V::unpack(vf[i], v);
#pragma unroll
      for (int e = 0; e < V::N; ++e) ss[0] = fmaf(v[e], v[e], ss[0]);
    }
    block_sums<1>(ss, red[0], lane, wave, nw);
    rf = 1.f / sqrtf(ss[0] * a.inv_h + a.eps);
  }
  const float gt = a.gate_kind == MOE_GATE_TOKEN ? static_cast<const float*>(a.gate)[t] : 1.f;
  float r[NCH][V::N];
  float ss[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = tid + i * blockDim.x;
    float n[V::N], g[V::N];
    V::unpack(vr[i], r[i]);
    V::unpack(vf[i], n);
    if (g_post) {
      V::unpack(c < a.nch ? ld16(g_post + c) : u32x4{}, g);
#pragma unroll
      for (int e = 0; e < V::N; ++e) n[e] = n[e] * rf * g[e];
    }
    if (a.gate_kind >= MOE_GATE_CHANNEL) {
      V::unpack(vg[i], g);
#pragma unroll
      for (int e = 0; e < V::N; ++e) n[e] *= g[e];
    }
#pragma unroll
    for (int e = 0; e < V::N; ++e) {
      r[i][e] = fmaf(gt, n[e], a.scale * r[i][e]);
      ss[0] = fmaf(r[i][e], r[i][e], ss[0]);
    }
    if (a.resid_out && c < a.nch) st16(static_cast<u32x4*>(a.resid_out) + base + c, V::pack(r[i]));
  }
  if (!a.x) return;
  block_sums<1>(ss, red[1], lane, wave, nw);
  const float rr = 1.f / sqrtf(ss[0] * a.inv_h + a.eps);
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = tid + i * blockDim.x;
    if (c >= a.nch) continue;
    float g[V::N];
    V::unpack(ld16(g_pre + c), g);
#pragma unroll
    for (int e = 0; e < V::N; ++e) r[i][e] = r[i][e] * rr * g[e];
    st16(static_cast<u32x4*>(a.x) + base + c, V::pack(r[i]));
  }
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ...: NCH chunks a thread as above.
template <bool F32, int NCH>
__global__ __launch_bounds__(1024) void norm_backward_kernel(NormBackArgs a) {
  using V = Vec<F32>;
  __shared__ float red[2][kMaxWaves * 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
  const u32x4* f = static_cast<const u32x4*>(a.f);
  const u32x4* gate = static_cast<const u32x4*>(a.gate);
  const u32x4* g_post = static_cast<const u32x4*>(a.g_post);
  const u32x4* g_pre = static_cast<const u32x4*>(a.g_pre);
  float s_post[NCH][V::N] = {}, s_pre[NCH][V::N] = {}, s_gate[NCH][V::N] = {};
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t base = (int64_t)t * a.nch;
    u32x4 vd[NCH] = {}, vx[NCH] = {}, vf[NCH] = {}, vr[NCH] = {}, vg[NCH] = {};
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = tid + i * blockDim.x;
      if (c >= a.nch) continue;
      if (a.dresid_out) vd[i] = ld16_nt(static_cast<const u32x4*>(a.dresid_out) + base + c);
      if (a.dx) {
        vx[i] = ld16_nt(static_cast<const u32x4*>(a.dx) + base + c);
        vr[i] = ld16_nt(static_cast<const u32x4*>(a.resid_out) + base + c);
      }
      if (f) vf[i] = ld16_nt(f + base + c);
      if (a.gate_kind == MOE_GATE_FULL) vg[i] = ld16_nt(gate + base + c);
      if (a.gate_kind == MOE_GATE_CHANNEL) vg[i] = ld16(gate + c);
    }
    // sums over the row: r'^2, g_pre dx r', f^2
    float ss[4] = {};
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = tid + i * blockDim.x;
      float x[V::N], r[V::N], fv[V::N], g[V::N] = {};
      V::unpack(vx[i], x);
      V::unpack(vr[i], r);
      V::unpack(vf[i], fv);
      if (a.dx && c < a.nch) V::unpack(ld16(g_pre + c), g);
#pragma unroll
      for (int e = 0; e < V::N; ++e) {
        ss[0] = fmaf(r[e], r[e], ss[0]);
        ss[1] = fmaf(g[e] * x[e], r[e], ss[1]);
        ss[2] = fmaf(fv[e], fv[e], ss[2]);
      }
    }
    block_sums<4>(ss, red[0], lane, wave, nw);
    const float rr = 1.f / sqrtf(ss[0] * a.inv_h + a.eps);
    const float mr = ss[1] * a.inv_h * rr * rr;
    const float rf = g_post ? 1.f / sqrtf(ss[2] * a.inv_h + a.eps) : 1.f;
    const float gt = a.gate_kind == MOE_GATE_TOKEN ? static_cast<const float*>(a.gate)[t] : 1.f;
    // dr, and the sums g_post dn f and n dr
    float dn[NCH][V::N];
    float s2[2] = {};
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = tid + i * blockDim.x;
      float dr[V::N], x[V::N], r[V::N], g[V::N] = {}, fv[V::N], gp[V::N];
      V::unpack(vd[i], dr);
      if (a.dx) {
        V::unpack(vx[i], x);
        V::unpack(vr[i], r);
        if (c < a.nch) V::unpack(ld16(g_pre + c), g);
#pragma unroll
        for (int e = 0; e < V::N; ++e) {
          dr[e] = fmaf(rr, fmaf(-r[e], mr, g[e] * x[e]), dr[e]);
          s_pre[i][e] = fmaf(x[e] * rr, r[e], s_pre[i][e]);
        }
      }
      if (a.dresid && c < a.nch) {
        float o[V::N];
#pragma unroll
        for (int e = 0; e < V::N; ++e) o[e] = a.scale * dr[e];
        st16(static_cast<u32x4*>(a.dresid) + base + c, V::pack(o));
      }
      if (!f) continue;
      V::unpack(vf[i], fv);
#pragma unroll
      for (int e = 0; e < V::N; ++e) gp[e] = 1.f;
      if (g_post && c < a.nch) V::unpack(ld16(g_post + c), gp);
      float n_dr[V::N];  // n dr: the gate's gradient
#pragma unroll
      for (int e = 0; e < V::N; ++e) {
        n_dr[e] = fv[e] * rf * gp[e] * dr[e];
        s2[1] += n_dr[e];
        dn[i][e] = gt * dr[e];
      }
      if (a.gate_kind >= MOE_GATE_CHANNEL) {
        V::unpack(vg[i], g);
#pragma unroll
        for (int e = 0; e < V::N; ++e) dn[i][e] *= g[e];
        if (a.gate_kind == MOE_GATE_FULL) {
          if (a.dgate && c < a.nch) st16(static_cast<u32x4*>(a.dgate) + base + c, V::pack(n_dr));
        } else {
#pragma unroll
          for (int e = 0; e < V::N; ++e) s_gate[i][e] += n_dr[e];
        }
      }
      if (g_post) {
#pragma unroll
        for (int e = 0; e < V::N; ++e) {
          s_post[i][e] = fmaf(dn[i][e] * rf, fv[e], s_post[i][e]);
          dn[i][e] *= gp[e];
          s2[0] = fmaf(dn[i][e], fv[e], s2[0]);
        }
      }
    }
    if (!f) {
      __syncthreads();  // red[0] is read before the next row's sums
      continue;
    }
    float mf = 0.f;
    if (g_post || (a.gate_kind == MOE_GATE_TOKEN && a.dgate)) {
      block_sums<2>(s2, red[1], lane, wave, nw);
      mf = s2[0] * a.inv_h * rf * rf;
      if (a.gate_kind == MOE_GATE_TOKEN && a.dgate && tid == 0) static_cast<float*>(a.dgate)[t] = s2[1];
    } else {
      __syncthreads();  // red[0] is read before the next row's sums
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = tid + i * blockDim.x;
      if (c >= a.nch) continue;
      if (g_post) {
        float fv[V::N];
        V::unpack(vf[i], fv);
#pragma unroll
        for (int e = 0; e < V::N; ++e) dn[i][e] = rf * fmaf(-fv[e], mf, dn[i][e]);
      }
      st16(static_cast<u32x4*>(a.df) + base + c, V::pack(dn[i]));
    }
  }
  // partial sums [gridDim.x][sums][H]: dg_post, dg_pre, dgate, as far as wanted
  const int H = a.nch * V::N;
  float* p = a.partial + (int64_t)blockIdx.x * a.sums * H;
  auto put = [&](const float (&s)[NCH][V::N]) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = tid + i * blockDim.x;
      if (c >= a.nch) continue;
#pragma unroll
      for (int e = 0; e < V::N; e += 4)
        *reinterpret_cast<f32x4*>(p + c * V::N + e) = f32x4{s[i][e], s[i][e + 1], s[i][e + 2], s[i][e + 3]};
    }
    p += H;
  };
  if (a.dg_post) put(s_post);
  if (a.dg_pre) put(s_pre);
  if (a.gate_kind == MOE_GATE_CHANNEL && a.dgate) put(s_gate);
}

// One thread per column of the sums: the workgroups' partial sums in order.
__global__ __launch_bounds__(256) void norm_sums_kernel(const float* __restrict__ partial, float* o0, float* o1,
                                                        float* o2, int wgs, int H, int sums) {
  __shared__ float red[16][17];
  const int col = blockIdx.x * 16 + (threadIdx.x & 15), part = threadIdx.x >> 4;
  const int n = sums * H;
  float v = 0.f;
  if (col < n)
    for (int i = part; i < wgs; i += 16) v += partial[(int64_t)i * n + col];
  red[part][threadIdx.x & 15] = v;
  __syncthreads();
  if (part == 0 && col < n) {
    v = 0.f;
    for (int i = 0; i < 16; ++i) v += red[i][threadIdx.x & 15];
    const int which = col / H;
    (which == 0 ? o0 : which == 1 ? o1 : o2)[col - which * H] = v;
  }
}

// Threads of a workgroup for nch chunks, NCH a thread.
int threads_of(int nch, int per) { return ((nch + per - 1) / per + 63) / 64 * 64; }

}  // namespace

constexpr int kNormMaxPartials = 512;

size_t norm_partial_floats(int64_t T, int64_t H) {
  return (size_t)(T < kNormMaxPartials ? T : kNormMaxPartials) * 3 * (size_t)H;
}

hipError_t launch_norm(const NormArgs& a, int T, bool f32, hipStream_t s) {
#define MOE_NORM(NCH)                                                                     \
  do {                                                                                    \
    if (f32) norm_kernel<true, NCH><<<T, threads_of(a.nch, NCH), 0, s>>>(a);              \
    else norm_kernel<false, NCH><<<T, threads_of(a.nch, NCH), 0, s>>>(a);                 \
  } while (0)
  if (a.nch <= 512) MOE_NORM(1);
  else if (a.nch <= 1024) MOE_NORM(2);
  else MOE_NORM(4);
#undef MOE_NORM
  return hipGetLastError();
}

hipError_t launch_norm_backward(NormBackArgs a, bool f32, hipStream_t s) {
  const int H = a.nch * (f32 ? 4 : 8);
  a.sums = (a.dg_post != nullptr) + (a.dg_pre != nullptr) + (a.gate_kind == MOE_GATE_CHANNEL && a.dgate);
  const int grid = a.T < kNormMaxPartials ? a.T : kNormMaxPartials;
#define MOE_NORM(NCH)                                                                              \
  do {                                                                                             \
    if (f32) norm_backward_kernel<true, NCH><<<grid, threads_of(a.nch, NCH), 0, s>>>(a);           \
    else norm_backward_kernel<false, NCH><<<grid, threads_of(a.nch, NCH), 0, s>>>(a);              \
  } while (0)
  if (a.nch <= 512) MOE_NORM(1);
  else if (a.nch <= 1024) MOE_NORM(2);
  else MOE_NORM(4);
#undef MOE_NORM
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.sums == 0) return e;
  float* out[3] = {};
  int n = 0;
  if (a.dg_post) out[n++] = a.dg_post;
  if (a.dg_pre) out[n++] = a.dg_pre;
  if (a.gate_kind == MOE_GATE_CHANNEL && a.dgate) out[n++] = static_cast<float*>(a.dgate);
  norm_sums_kernel<<<(a.sums * H + 15) / 16, 256, 0, s>>>(a.partial, out[0], out[1], out[2], grid, H, a.sums);
  return hipGetLastError();
}

}  // namespace moe
