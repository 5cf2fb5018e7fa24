// The whole layer for a few tokens (T <= 16) in two kernels (Qwen3.8-Flash-Next
// study, MoE section: eq. expert(x) and eq. MoE(x) over its pipeline figure):
//   few_router_kernel  : logits[t, e] = x_t . W_r[e] and x_t . w_sg, complete in fp32
//   few_experts_kernel : top-k and weights, then h = SiLU(W_gate x) * (W_up x) of every
//                        (token, expert) pair and of the shared expert, then
//     out[t] = sum_j w[t,j] W_down[e_j] h[t,j] + sigmoid(s_t) S_down h_sh[t]
// A batch this small is bound by reading the touched experts' weights once,
// and below a few hundred MB by the latency of the steps between them, so the
// launches between the stages go: every workgroup does the top-k itself (a few
// KB of logits), and the one dependency between workgroups, h before the down
// products, is a counter in memory.
//
// Work order and why every wait ends: the gate/up items are claimed from a
// counter, and a workgroup goes on to its down columns only when the counter
// has run out.  Then every gate/up item is held by a workgroup that runs and
// waits for nothing, so the number of finished items reaches their total
// whatever else the GPU runs, however few workgroups of this grid are resident.
//
// Down products: a workgroup owns 16 output columns and goes over all groups,
// its waves taking (group, K range) units in turn; a fragment row is a token
// (zero where the token does not use the expert), so each unit's fp32 block is
// scaled by the routing weights and added in registers, the waves' sums are
// added in LDS in wave order, and out is rounded once.  No per-assignment
// output is stored or rounded, and no sum depends on timing.
#include "common.hpp"
#include "kernels.hpp"
#include "stream_item.hpp"
#include "topk.hpp"

namespace moe {
namespace {

using namespace streamk;

constexpr int FW = 8;                      // waves per workgroup of the experts kernel
constexpr int kFewRows = kSmallBatch * 64;  // (token, expert) pairs at most
static_assert(kSmallBatch == 16 && kMaxExperts < 2048, "a fragment row per token; packed list entries");

// Workgroup b: router rows 16 b .. 16 b + 15 (row E: the shared gate), K split
// over 16 waves whose blocks are added in wave order.  The first workgroup
// zeroes the counters of the kernel that follows.
constexpr int RWF = 16;
__global__ __launch_bounds__(RWF * 64) void few_router_kernel(const bf16* __restrict__ x, const bf16* __restrict__ wr,
                                                              const bf16* __restrict__ wsg,
                                                              float* __restrict__ logits, int T, int H, int E, int N,
                                                              int kchunk, int32_t* counters) {
  if (blockIdx.x == 0 && threadIdx.x < 2) counters[threadIdx.x * kFewCounterStride] = 0;
  __shared__ f32x4 part[RWF][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int m = lane & 15, kq = (lane >> 4) * 8;
  const int kbeg = w * kchunk;
  const int kend = kbeg + kchunk < H ? kbeg + kchunk : H;
  f32x4 acc[1] = {f32x4{0.f, 0.f, 0.f, 0.f}};
  if (kbeg < kend) {
    const bf16* a_row = m < T ? x + (int64_t)m * H : nullptr;
    int n = blockIdx.x * 16 + m;
    n = n < N ? n : N - 1;
    const bf16* b_row[1] = {n < E ? wr + (int64_t)n * H : wsg};
    stream_dot<1>(a_row, b_row, kbeg, kend, kq, acc);
  }
  part[w][lane] = acc[0];
  __syncthreads();
  if (w == 0) {
    f32x4 t = part[0][lane];
#pragma unroll
    for (int i = 1; i < RWF; ++i) t += part[i][lane];
    const int col = blockIdx.x * 16 + m;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = 4 * (lane >> 4) + i;
      if (tok < T && col < N) logits[(int64_t)tok * N + col] = t[i];
    }
  }
}

// Top-k of one token by one wave: lane j < k returns the j-th pick and its
// renormalised weight.
template <int PER_LANE>
__device__ __forceinline__ void pick(const float* row, int E, int k, int page, int lane, int* id, float* wj) {
  uint64_t key[PER_LANE];
#pragma unroll
  for (int i = 0; i < PER_LANE; ++i) {
    const int e = lane + 64 * i;
    float a = row[e < E ? e : E - 1];
    if (page) a = bf2f(f2bf(a));
    key[i] = make_key(e < E ? ord(a) : 0u, e);
  }
  const uint64_t sel = select_topk<PER_LANE>(key, k, lane);
  const uint32_t hi = (uint32_t)(sel >> 32);
  const float top = unord(__builtin_amdgcn_readlane(hi, 0));
  const float ex = lane < k ? expf(unord(hi) - top) : 0.f;
  const float v = ex / wave_sum(ex);
  *wj = page ? bf2f(f2bf(v)) : v;
  int e = (int)~(uint32_t)sel;
  *id = (unsigned)e < (unsigned)E ? e : E - 1;  // (out of range only for NaN logits)
}

// What a workgroup knows of the batch's routing.
struct FewRoute {
  uint32_t list[kFewRows + 1];  // touched experts ascending, then E for the shared one: expert | its tokens << 11
  uint16_t base[kFewRows + 1];  // its first row of h
  float w[kFewRows];         // per row of h: the routing weight
  float sg[kSmallBatch];     // sigmoid of the shared gate logit
  int wtot[FW], wrow[FW];
  int next;                  // claimed item, block-wide
};

// The blocks of a unit: part = H_rows [16 tokens, kbeg..kend) x W_down rows c0 .. c0 + 15.
template <int WT>
__device__ __forceinline__ f32x4 down_dot(const FfnArgs& f, int g, const bf16* a_row, const bf16* a_any, int c0, int K,
                                          int kbeg, int kend, int lane, char* lds) {
  const int m = lane & 15;
  const int left = f.H - c0;  // columns from c0 to the end
  const int nv[1] = {left};
  f32x4 acc[1] = {f32x4{0.f, 0.f, 0.f, 0.f}};
  if constexpr (WT == kWtPlain) {
    const bool shared = g >= f.E;
    const bf16* mat = shared ? reinterpret_cast<const bf16*>(f.shd)
                             : reinterpret_cast<const bf16*>(f.wd) + (int64_t)g * f.sd;
    const bf16* w0[1] = {mat + (int64_t)c0 * K};
    stream_dot_lds<1, false, 2>(a_row, a_any, w0, nv, K, kbeg, kend, lane, lds, acc);
  } else if constexpr (WT == kWtFp8) {
    const uint8_t* w0[1] = {reinterpret_cast<const uint8_t*>(f.wd) + (int64_t)g * f.sd + (int64_t)c0 * K};
    const int col = m < left ? c0 + m : f.H - 1;
    const int kb = K / 128;
    const float* s0[1] = {reinterpret_cast<const float*>(f.scd) + (int64_t)g * (f.H / 128) * kb + (col / 128) * kb};
    stream_dot_lds8<1>(a_row, a_any, w0, nv, K, s0, kbeg, kend, lane, lds, acc);
  } else {
    const int row = m < left ? c0 + m : f.H - 1;
    const uint8_t* w0[1] = {reinterpret_cast<const uint8_t*>(f.wd) + ((int64_t)g * f.sd + (int64_t)row * K) / 2};
    const uint8_t* s0[1] = {reinterpret_cast<const uint8_t*>(f.scd) + ((int64_t)g * f.H + row) * (K / 32)};
    stream_dot_mx<1>(a_row, a_any, w0, s0, kbeg, kend, lane, acc);
  }
  return acc[0];
}

// K range of a unit: multiples of 256 (a batch of every weight form), so that
// the groups' units number at least two per wave where K allows it.
constexpr int kUnitK = 256;

template <int WT>
__global__ __launch_bounds__(FW * 64, 2) void few_experts_kernel(FfnArgs f, FewArgs a) {
  constexpr int ROUTED = item_lds_bytes<WT, true>(), PLAIN = item_lds_bytes<kWtPlain, true>();
  constexpr int STAGE = ROUTED > PLAIN ? ROUTED : PLAIN;  // per wave
  __shared__ __attribute__((aligned(16))) char stage[FW * STAGE];
  __shared__ FewRoute r;
  static_assert(FW * STAGE >= (2 * kFewRows + kMaxExperts) * 4, "routing scratch in the stage");
  static_assert(FW * STAGE >= FW * 64 * 16, "the waves' sums in the stage");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int T = f.T, k = f.k, E = f.E, R = T * k;
  const bool shared = a.has_shared != 0;
  const int N = E + (shared ? 1 : 0);

  // ---- routing: every workgroup for itself ----
  int* ids = reinterpret_cast<int*>(stage);
  float* wts = reinterpret_cast<float*>(stage) + kFewRows;
  uint32_t* tmask = reinterpret_cast<uint32_t*>(stage) + 2 * kFewRows;
  for (int e = tid; e < E; e += FW * 64) tmask[e] = 0u;
  for (int t = wave; t < T; t += FW) {
    int id;
    float wj;
    const float* row = a.logits + (int64_t)t * N;
    if (E <= 64) pick<1>(row, E, k, a.page, lane, &id, &wj);
    else if (E <= 128) pick<2>(row, E, k, a.page, lane, &id, &wj);
    else if (E <= 256) pick<4>(row, E, k, a.page, lane, &id, &wj);
    else if (E <= 512) pick<8>(row, E, k, a.page, lane, &id, &wj);
    else pick<16>(row, E, k, a.page, lane, &id, &wj);
    if (lane < k) {
      ids[t * k + lane] = id;
      wts[t * k + lane] = wj;
      if (blockIdx.x == 0 && a.ids) a.ids[t * k + lane] = id;
      if (blockIdx.x == 0 && a.w) a.w[t * k + lane] = wj;
    }
    if (shared && lane == 0) r.sg[t] = sigmoid(row[E]);
  }
  __syncthreads();
  for (int i = tid; i < R; i += FW * 64) atomicOr(&tmask[ids[i]], 1u << (i / k));
  __syncthreads();
  // the touched experts in ascending order, with their first rows
  int ng = 0, rows = 0;
  for (int g0 = 0; g0 < E; g0 += FW * 64) {
    const int g = g0 + tid;
    const uint32_t mk = g < E ? tmask[g] : 0u;
    const uint64_t bal = __ballot(mk != 0u);
    int incl = __popc(mk);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(incl, o, 64);
      if (lane >= o) incl += u;
    }
    if (lane == 63) {
      r.wtot[wave] = __popcll(bal);
      r.wrow[wave] = incl;
    }
    __syncthreads();
    int off = ng, roff = rows;
    for (int w = 0; w < FW; ++w) {
      if (w < wave) {
        off += r.wtot[w];
        roff += r.wrow[w];
      }
      ng += r.wtot[w];
      rows += r.wrow[w];
    }
    if (mk) {
      const int at = off + __popcll(bal & ((1ull << lane) - 1ull));
      r.list[at] = (uint32_t)g | mk << 11;
      r.base[at] = (uint16_t)(roff + incl - __popc(mk));
      tmask[g] = mk | (uint32_t)at << 16;  // the expert's place in the list, for the next loop
    }
    __syncthreads();
  }
  if (tid == 0) {
    r.list[ng] = (uint32_t)E | ((1u << T) - 1u) << 11;
    r.base[ng] = 0;
  }
  for (int i = tid; i < R; i += FW * 64) {
    const uint32_t v = tmask[ids[i]];
    r.w[r.base[v >> 16] + __popc(v & ((1u << (i / k)) - 1u))] = wts[i];
  }
  // ---- gate/up: items of 8 hidden columns, a wave each, claimed 8 at a time ----
  const int slabs_sh = shared ? (f.Is + 7) / 8 : 0, slabs = (f.I + 7) / 8;
  const int total = slabs_sh + ng * slabs;  // the shared expert's first: bf16, the largest
  int done = 0;                             // items of this workgroup
  for (;;) {
    __syncthreads();  // (also: the routing scratch is read out before the stage is used)
    if (tid == 0) r.next = atomicAdd(a.counters, FW);
    __syncthreads();
    const int first = r.next;
    if (first >= total) break;
    done += total - first < FW ? total - first : FW;
    const int it = first + wave;
    if (it < slabs_sh) {
      stream_item<1, kWtPlain, true>(f, E, 0, 0, T, nullptr, it, lane, stage + wave * STAGE);
    } else if (it < total) {
      const int i = (it - slabs_sh) / slabs, slab = (it - slabs_sh) % slabs;
      const uint32_t mk = r.list[i] >> 11;
      stream_item<1, WT, true>(f, r.list[i] & 2047, 0, r.base[i], __popc(mk), nullptr, slab, lane,
                               stage + wave * STAGE, mk);
    }
  }
  // ---- every h is written before the first down product reads one ----
  // (every wave's stores have left before the barrier; the fence makes them
  // visible to the device before they are counted)
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (tid == 0) {
    if (done) {
      __threadfence();
      atomicAdd(a.counters + kFewCounterStride, done);
    }
    while (__hip_atomic_load(a.counters + kFewCounterStride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < total)
      __builtin_amdgcn_s_sleep(1);
    __threadfence();
  }
  __syncthreads();

  // ---- down and combine: 16 output columns over all groups ----
  const int q = lane >> 4, m = lane & 15;
  const int nslab = (f.H + 15) / 16;
  // units of the routed groups and of the shared expert
  auto split = [&](int K) {
    const int most = (K + kUnitK - 1) / kUnitK;
    const int want = (2 * FW + ng - 1) / ng;  // units per group for two per wave
    const int n = want < most ? want : most;
    const int len = ((K + n - 1) / n + kUnitK - 1) / kUnitK * kUnitK;
    return len;
  };
  const int len = split(f.I), per = (f.I + len - 1) / len;
  const int len_sh = WT == kWtPlain ? (shared ? split(f.Is) : kUnitK) : kUnitK;
  const int units_sh = shared ? (f.Is + len_sh - 1) / len_sh : 0;
  const int units = units_sh + ng * per;
  for (int s = blockIdx.x; s < nslab; s += gridDim.x) {
    const int c0 = s * 16;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    for (int u = wave; u < units; u += FW) {
      const bool sh = u < units_sh;
      const int i = sh ? ng : (u - units_sh) / per;
      const int kbeg = sh ? u * len_sh : ((u - units_sh) % per) * len;
      const int K = sh ? f.Is : f.I;
      const int kend = kbeg + (sh ? len_sh : len) < K ? kbeg + (sh ? len_sh : len) : K;
      const int mk = (int)(r.list[i] >> 11), base = r.base[i];
      const bf16* h = reinterpret_cast<const bf16*>(sh ? f.h_sh : f.h);
      const bool in = m < T && (mk >> m & 1);
      const bf16* a_row = in ? h + (int64_t)(base + __popc(mk & ((1 << m) - 1))) * K : nullptr;
      const f32x4 p = sh ? down_dot<kWtPlain>(f, E, a_row, h, c0, K, kbeg, kend, lane, stage + wave * STAGE)
                         : down_dot<WT>(f, r.list[i] & 2047, a_row, h, c0, K, kbeg, kend, lane, stage + wave * STAGE);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int t = 4 * q + v;
        if (mk >> t & 1) sum[v] = fmaf(sh ? r.sg[t] : r.w[base + __popc(mk & ((1 << t) - 1))], p[v], sum[v]);
      }
    }
    __syncthreads();
    f32x4* part = reinterpret_cast<f32x4*>(stage);
    part[wave * 64 + lane] = sum;
    __syncthreads();
    if (wave == 0) {
      f32x4 t = part[lane];
#pragma unroll
      for (int w = 1; w < FW; ++w) t += part[w * 64 + lane];
      bf16* out = reinterpret_cast<bf16*>(a.out);
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (4 * q + v < T && c0 + m < f.H) out[(int64_t)(4 * q + v) * f.H + c0 + m] = f2bf(t[v]);
    }
    __syncthreads();
  }
}

int few_cus() {
  static int cus = 0;
  if (!cus) {
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
      n = 256;
    cus = n;
  }
  return cus;
}

}  // namespace

hipError_t launch_layer_few(const FfnArgs& f, const void* w_router, const void* w_sg, const FewArgs& a, hipStream_t s) {
  if (f.T < 1 || f.T > kSmallBatch || f.E > kMaxExperts || f.k > 64) return hipErrorInvalidValue;
  const int N = f.E + (a.has_shared ? 1 : 0);
  const int kchunk = ((f.H + RWF - 1) / RWF + KSTEP - 1) / KSTEP * KSTEP;
  few_router_kernel<<<(N + 15) / 16, RWF * 64, 0, s>>>(
      reinterpret_cast<const bf16*>(f.x), reinterpret_cast<const bf16*>(w_router), reinterpret_cast<const bf16*>(w_sg),
      a.logits, f.T, f.H, f.E, N, kchunk, a.counters);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int grid = few_cus();
  if (f.wt == kWtFp8) few_experts_kernel<kWtFp8><<<grid, FW * 64, 0, s>>>(f, a);
  else if (f.wt == kWtMx) few_experts_kernel<kWtMx><<<grid, FW * 64, 0, s>>>(f, a);
  else few_experts_kernel<kWtPlain><<<grid, FW * 64, 0, s>>>(f, a);
  return hipGetLastError();
}

}  // namespace moe
