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

// Sums of P values over the waves [first, first + nw) of the workgroup, in each of their
// threads.  red: [kMaxWaves][P] (one use per barrier interval: callers alternate two).
template <int P>
__device__ __forceinline__ void block_sums(float (&a)[P], float* red, int lane, int wave, int first, int nw) {
  const float s = wave_sums<P>(a, lane);
  constexpr int kStep = 64 / P;
  if (lane % kStep == 0) red[wave * P + lane / kStep] = s;
  __syncthreads();
  // lane l takes value l % P of the waves l / P, l / P + kStep ..; then over the lanes
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kMaxWaves; w += kStep) {
    const int at = w + lane / P;
    if (w < nw) v += at < nw ? red[(first + at) * P + lane % P] : 0.f;
  }
#pragma unroll
  for (int o = P; o < 64; o <<= 1) v += __shfl_xor(v, o, kWave);
#pragma unroll
  for (int i = 0; i < P; ++i) a[i] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), i));
}

// One row a workgroup: all of a row's loads are out before the first sum, and the rows of the
// other workgroups on the compute unit cover the two sums' waits (8192 x 8192 bf16 with a full
// gate, 0.67 GB: 116 us, 5.8 TB/s; 4096 x 2560: 20 us, 4.1 TB/s; one row of 8192: 4.2 us of
// latency).
template <bool F32, int NCH>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a, int T) {
  using V = Vec<F32>;
  __shared__ float red[2][kMaxWaves];
  const int64_t row = blockIdx.y * (int64_t)gridDim.x + blockIdx.x;
  if (row >= T) return;
  const int t = (int)row, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
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
    block_sums<1>(ss, red[0], lane, wave, 0, nw);
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
  block_sums<1>(ss, red[1], lane, wave, 0, nw);
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

// At most a workgroup per compute unit, so that few partial sums are left to add (4096 x 2560
// bf16, 0.13 GB: 27 us and 4 for the sums, 4.1 TB/s; 8192 x 8192, 0.81 GB: 192 us).
// A workgroup has blockDim.x / tpr rows at a time, tpr threads (whole waves) a row with
// NCH chunks each; the next rows' loads go out before the present ones' sums.
// GATE: MOE_GATE_NONE stands for the token's gate too (a factor that is 1 without one).
template <bool F32, int NCH, int NT, bool POST, int GATE>
__global__ __launch_bounds__(NT) void norm_backward_kernel(NormBackArgs a, int tpr) {
  using V = Vec<F32>;
  __shared__ float red[2][kMaxWaves * 8];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wpr = tpr >> 6, group = wave / wpr, groups = blockDim.x / tpr;
  const int me = tid - group * tpr;  // thread of the row
  const u32x4* f = static_cast<const u32x4*>(a.f);
  const u32x4* gate = static_cast<const u32x4*>(a.gate);
  const u32x4* g_post = static_cast<const u32x4*>(a.g_post);
  const u32x4* g_pre = static_cast<const u32x4*>(a.g_pre);
  // sums over a row's P values, in each of its threads
  auto row_sums = [&](auto& v, float* r) {
    constexpr int P = sizeof(v) / 4;
    if (wpr == 1) {
      const float s = wave_sums<P>(v, lane);
#pragma unroll
      for (int i = 0; i < P; ++i) v[i] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(s), i * (64 / P)));
    } else {
      block_sums<P>(v, r, lane, wave, group * wpr, wpr);
    }
  };
  struct Row {
    u32x4 d[NCH], x[NCH], f[NCH], r[NCH], g[GATE == MOE_GATE_FULL ? NCH : 1];
    float gt;  // the token's gate
  };
  auto load = [&](Row& v, int t) {
    v.gt = GATE == MOE_GATE_NONE && a.gate && t < a.T ? static_cast<const float*>(a.gate)[t] : 1.f;
    const int64_t base = (int64_t)t * a.nch;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = me + i * tpr;
      v.d[i] = v.x[i] = v.f[i] = v.r[i] = u32x4{};
      if constexpr (GATE == MOE_GATE_FULL) v.g[i] = u32x4{};
      if (t >= a.T || c >= a.nch) continue;
      if (a.dresid_out) v.d[i] = ld16_nt(static_cast<const u32x4*>(a.dresid_out) + base + c);
      if (a.dx) {
        v.x[i] = ld16_nt(static_cast<const u32x4*>(a.dx) + base + c);
        v.r[i] = ld16_nt(static_cast<const u32x4*>(a.resid_out) + base + c);
      }
      if (f) v.f[i] = ld16_nt(f + base + c);
      if constexpr (GATE == MOE_GATE_FULL) v.g[i] = ld16_nt(gate + base + c);
    }
  };
  float s_post[POST ? NCH : 1][V::N] = {}, s_pre[NCH][V::N] = {}, s_gate[GATE == MOE_GATE_CHANNEL ? NCH : 1][V::N] = {};
  // the columns' gains and gate stay in registers: a load of theirs in the loop would wait
  // for the next rows' ahead of it
  u32x4 k_pre[NCH], k_post[POST ? NCH : 1], k_gate[GATE == MOE_GATE_CHANNEL ? NCH : 1];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = me + i * tpr;
    k_pre[i] = a.dx && c < a.nch ? ld16(g_pre + c) : u32x4{};
    if constexpr (POST) k_post[i] = c < a.nch ? ld16(g_post + c) : u32x4{};
    if constexpr (GATE == MOE_GATE_CHANNEL) k_gate[i] = c < a.nch ? ld16(gate + c) : u32x4{};
  }
  const int step = gridDim.x * groups;
  constexpr bool AHEAD = NCH < 4;  // registers for two rows
  Row v;
  if constexpr (AHEAD) load(v, blockIdx.x * groups + group);
  // every group runs the same number of rounds: the sums have barriers
  int round = 0;  // two places for the sums, in turn
  for (int t0 = blockIdx.x * groups; t0 < a.T; t0 += step, ++round) {
    const int t = t0 + group;
    const bool live = t < a.T;
    const int64_t base = (int64_t)t * a.nch;
    Row next;
    if constexpr (AHEAD) load(next, t0 + step + group);
    else load(v, t);
    // Sums over the row: r'^2, u r' with u = g_pre dx, f^2, and with q = gate g_post f
    // (the token's gate left out) q dresid_out, q u, q r': the last three give
    // sum q dr = s3 + rr s4 - rr mr s5, so one round of sums serves both norms.
    float ss[8] = {};
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      float d[V::N], x[V::N], r[V::N], q[V::N], g[V::N];
      V::unpack(v.x[i], x);
      V::unpack(v.r[i], r);
      V::unpack(v.f[i], q);
      V::unpack(v.d[i], d);
      V::unpack(k_pre[i], g);
#pragma unroll
      for (int e = 0; e < V::N; ++e) {
        x[e] *= g[e];
        ss[0] = fmaf(r[e], r[e], ss[0]);
        ss[1] = fmaf(x[e], r[e], ss[1]);
        if constexpr (POST) ss[2] = fmaf(q[e], q[e], ss[2]);
      }
      if constexpr (POST) {
        V::unpack(k_post[i], g);
#pragma unroll
        for (int e = 0; e < V::N; ++e) q[e] *= g[e];
      }
      if constexpr (GATE != MOE_GATE_NONE && POST) {
        if constexpr (GATE == MOE_GATE_FULL) V::unpack(v.g[i], g);
        else V::unpack(k_gate[i], g);
#pragma unroll
        for (int e = 0; e < V::N; ++e) q[e] *= g[e];
      }
#pragma unroll
      for (int e = 0; e < V::N; ++e) {
        if constexpr (POST || GATE == MOE_GATE_NONE) {
          ss[3] = fmaf(q[e], d[e], ss[3]);
          ss[4] = fmaf(q[e], x[e], ss[4]);
          ss[5] = fmaf(q[e], r[e], ss[5]);
        }
      }
    }
    row_sums(ss, red[round & 1]);
    const float rr = 1.f / sqrtf(ss[0] * a.inv_h + a.eps);
    const float mr = ss[1] * a.inv_h * rr * rr;
    const float rf = POST ? 1.f / sqrtf(ss[2] * a.inv_h + a.eps) : 1.f;
    const float gt = v.gt;
    const float sq = fmaf(rr, fmaf(-mr, ss[5], ss[4]), ss[3]);
    const float mf = gt * sq * a.inv_h * rf * rf;
    if (GATE == MOE_GATE_NONE && a.dgate && live && me == 0) static_cast<float*>(a.dgate)[t] = rf * sq;
    // an idle group's zeros times an infinite gain or gate would be NaN in the sums over tokens
    if (live) {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int c = me + i * tpr;
        const bool in = c < a.nch;
        float dr[V::N], fv[V::N], g[V::N], o[V::N];
        V::unpack(v.d[i], dr);
        V::unpack(v.f[i], fv);
        if (a.dx) {
          float x[V::N], r[V::N];
          V::unpack(v.x[i], x);
          V::unpack(v.r[i], r);
          V::unpack(k_pre[i], g);
#pragma unroll
          for (int e = 0; e < V::N; ++e) {
            dr[e] = fmaf(rr, fmaf(-r[e], mr, g[e] * x[e]), dr[e]);
            s_pre[i][e] = fmaf(x[e] * rr, r[e], s_pre[i][e]);
          }
        }
        if (a.dresid && in) {
#pragma unroll
          for (int e = 0; e < V::N; ++e) o[e] = a.scale * dr[e];
          st16(static_cast<u32x4*>(a.dresid) + base + c, V::pack(o));
        }
        if (!f) continue;
        float dn[V::N], gp[V::N];
#pragma unroll
        for (int e = 0; e < V::N; ++e) {
          dn[e] = gt * dr[e];
          gp[e] = 1.f;
        }
        if constexpr (POST) V::unpack(k_post[i], gp);
        if constexpr (GATE != MOE_GATE_NONE) {
          if constexpr (GATE == MOE_GATE_FULL) V::unpack(v.g[i], g);
          else V::unpack(k_gate[i], g);
#pragma unroll
          for (int e = 0; e < V::N; ++e) {
            dn[e] *= g[e];
            o[e] = fv[e] * rf * gp[e] * dr[e];  // n dr: the gate's gradient
            if constexpr (GATE == MOE_GATE_CHANNEL) s_gate[i][e] += o[e];
          }
          if (GATE == MOE_GATE_FULL && a.dgate && in) st16(static_cast<u32x4*>(a.dgate) + base + c, V::pack(o));
        }
        if constexpr (POST) {
#pragma unroll
          for (int e = 0; e < V::N; ++e) {
            s_post[i][e] = fmaf(dn[e] * rf, fv[e], s_post[i][e]);
            dn[e] = rf * fmaf(-fv[e], mf, dn[e] * gp[e]);
          }
        }
        if (in) st16(static_cast<u32x4*>(a.df) + base + c, V::pack(dn));
      }
    }
    if constexpr (AHEAD) v = next;
  }
  // partial sums [gridDim.x][sums][H]: dg_post, dg_pre, dgate, as far as wanted; the
  // workgroup's groups are added first
  const int H = a.nch * V::N;
  float* p = a.partial + (int64_t)blockIdx.x * a.sums * H;
  __shared__ __attribute__((aligned(16))) float other[NCH == 1 ? NT * V::N : 4];
  auto put = [&](float (&s)[NCH][V::N], float* alone) {
    if constexpr (NCH == 1) {
      if (groups > 1) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V::N; ++e) other[tid * V::N + e] = s[0][e];
        __syncthreads();
        if (group == 0)
          for (int q = 1; q < groups; ++q)
#pragma unroll
            for (int e = 0; e < V::N; ++e) s[0][e] += other[(q * tpr + tid) * V::N + e];
      }
    }
    if (group == 0) {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int c = me + i * tpr;
        if (c >= a.nch) continue;
        if (gridDim.x == 1) {  // the sums themselves, at any 4 bytes
#pragma unroll
          for (int e = 0; e < V::N; ++e) alone[c * V::N + e] = s[i][e];
          continue;
        }
#pragma unroll
        for (int e = 0; e < V::N; e += 4)
          *reinterpret_cast<f32x4*>(p + c * V::N + e) = f32x4{s[i][e], s[i][e + 1], s[i][e + 2], s[i][e + 3]};
      }
    }
    p += H;
  };
  if constexpr (POST) {
    if (a.dg_post) put(s_post, a.dg_post);
  }
  if (a.dg_pre) put(s_pre, a.dg_pre);
  if constexpr (GATE == MOE_GATE_CHANNEL) {
    if (a.dgate) put(s_gate, static_cast<float*>(a.dgate));
  }
}

// The workgroups' partial sums in order: 32 columns a workgroup, 32 parts of the partials.
__global__ __launch_bounds__(1024) void norm_sums_kernel(const float* __restrict__ partial, float* o0, float* o1,
                                                         float* o2, int wgs, int H, int sums) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  const int n = sums * H;
  float v = 0.f;
  if (col < n) {
    const float* p = partial + col;
#pragma unroll 8
    for (int i = part; i < wgs; i += 32) v += p[(int64_t)i * n];
  }
  red[part][lane] = v;
  __syncthreads();
  if (part == 0 && col < n) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += red[i][lane];
    const int which = col / H;
    (which == 0 ? o0 : which == 1 ? o1 : o2)[col - which * H] = v;
  }
}

// The sums over no tokens.
__global__ __launch_bounds__(256) void norm_no_rows_kernel(float* o0, float* o1, float* o2, int H) {
  const int col = blockIdx.x * 256 + threadIdx.x;
  if (col >= H) return;
  if (o0) o0[col] = 0.f;
  if (o1) o1[col] = 0.f;
  if (o2) o2[col] = 0.f;
}

// Threads of a workgroup for nch chunks, NCH a thread.
int threads_of(int nch, int per) { return ((nch + per - 1) / per + 63) / 64 * 64; }

}  // namespace

constexpr int kNormMaxPartials = 256;  // workgroups: one a compute unit, fewer sums to add

size_t norm_partial_floats(int64_t T, int64_t H) {
  return (size_t)(T < kNormMaxPartials ? T : kNormMaxPartials) * 3 * (size_t)H;
}

hipError_t launch_norm(const NormArgs& a, int T, bool f32, hipStream_t s) {
  const dim3 grid = row_grid(T);
#define MOE_NORM(NCH)                                                                     \
  do {                                                                                    \
    if (f32) norm_kernel<true, NCH><<<grid, threads_of(a.nch, NCH), 0, s>>>(a, T);        \
    else norm_kernel<false, NCH><<<grid, threads_of(a.nch, NCH), 0, s>>>(a, T);           \
  } while (0)
  if (a.nch <= 512) MOE_NORM(1);
  else if (a.nch <= 1024) MOE_NORM(2);
  else MOE_NORM(4);
#undef MOE_NORM
  return hipGetLastError();
}

template <bool F32, int NCH, int NT, bool POST>
static void back_kernel(const NormBackArgs& a, int grid, int threads, int tpr, hipStream_t s) {
  if (a.gate_kind == MOE_GATE_FULL) norm_backward_kernel<F32, NCH, NT, POST, MOE_GATE_FULL><<<grid, threads, 0, s>>>(a, tpr);
  else if (a.gate_kind == MOE_GATE_CHANNEL)
    norm_backward_kernel<F32, NCH, NT, POST, MOE_GATE_CHANNEL><<<grid, threads, 0, s>>>(a, tpr);
  else norm_backward_kernel<F32, NCH, NT, POST, MOE_GATE_NONE><<<grid, threads, 0, s>>>(a, tpr);
}
template <bool F32, int NCH, int NT>
static void back_kernel(const NormBackArgs& a, int& grid, hipStream_t s) {
  // short rows: several at a time
  const int tpr = threads_of(a.nch, NCH), groups = NCH == 1 && tpr < NT ? NT / tpr : 1;
  grid = (a.T + groups - 1) / groups;
  grid = grid < kNormMaxPartials ? grid : kNormMaxPartials;
  if (grid == 2) grid = 1;  // a second round of rows takes less than a launch for the sums (6 x 2560 11.3 -> 9.7 us)
  if (a.g_post) back_kernel<F32, NCH, NT, true>(a, grid, groups * tpr, tpr, s);
  else back_kernel<F32, NCH, NT, false>(a, grid, groups * tpr, tpr, s);
}

hipError_t launch_norm_no_rows(float* dg_post, float* dg_pre, float* dgate, int H, hipStream_t s) {
  norm_no_rows_kernel<<<(H + 255) / 256, 256, 0, s>>>(dg_post, dg_pre, dgate, H);
  return hipGetLastError();
}

hipError_t launch_norm_backward(NormBackArgs a, bool f32, hipStream_t s) {
  const int H = a.nch * (f32 ? 4 : 8);
  a.sums = (a.dg_post != nullptr) + (a.dg_pre != nullptr) + (a.gate_kind == MOE_GATE_CHANNEL && a.dgate);
  int grid = 0;
  if (f32) {
    if (a.nch <= 448) back_kernel<true, 1, 1024>(a, grid, s);  // rows that leave no wave idle
    else if (a.nch <= 512) back_kernel<true, 1, 512>(a, grid, s);
    else if (a.nch <= 1024) back_kernel<true, 2, 512>(a, grid, s);
    else if (a.nch <= 2048) back_kernel<true, 4, 512>(a, grid, s);
    else back_kernel<true, 4, 1024>(a, grid, s);
  } else {
    // 1024 threads where their 128 registers hold the sums (4096 x 2560, token's gate: 31.5 us,
    // 512 threads 33.8; full gate behind a post norm: 51.4, 40.9; channel's 46.1, 38.5)
    const bool few = !a.g_post || a.gate_kind < MOE_GATE_CHANNEL;
    if (a.nch <= 448 && few) back_kernel<false, 1, 1024>(a, grid, s);
    else if (a.nch <= 512) back_kernel<false, 1, 512>(a, grid, s);
    else if (a.nch <= 1024) back_kernel<false, 2, 512>(a, grid, s);
    else back_kernel<false, 4, 512>(a, grid, s);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.sums == 0 || grid == 1) return e;
  float* out[3] = {};
  int n = 0;
  if (a.dg_post) out[n++] = a.dg_post;
  if (a.dg_pre) out[n++] = a.dg_pre;
  if (a.gate_kind == MOE_GATE_CHANNEL && a.dgate) out[n++] = static_cast<float*>(a.dgate);
  norm_sums_kernel<<<(a.sums * H + 31) / 32, 1024, 0, s>>>(a.partial, out[0], out[1], out[2], grid, H, a.sums);
  return hipGetLastError();
}

}  // namespace moe
