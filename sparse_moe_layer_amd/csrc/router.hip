// Router epilogue: the fp32 logits (sum of K-chunk partials, chunk order
// fixed), softmax, top-k and renormalisation, one wavefront per token
// (Qwen3.8-Flash-Next study, MoE section: the top-k stage of its pipeline
// figure, where the chosen experts' probabilities are renormalised to sum to
// one).
//
// Each lane holds E/64 logits as 64-bit keys: an order-preserving image of
// the fp32 value in the high word, the complement of the expert id in the low
// word, so one unsigned maximum ranks by value and sends equal values to the
// lower id.  k rounds of a wave-wide maximum (DPP within each 16-lane row,
// then the four row results through readlane) pick the experts in descending
// order; lane j keeps round j's winner.  The renormalised weight of the j-th
// pick is exp(l_j - l_0) / sum_{j'<k} exp(l_j' - l_0), which equals the
// selected softmax probabilities divided by their sum (the full softmax's
// normaliser cancels).  With the section's routing numerics for bf16 layers
// the logits are rounded to bf16 first (ties become common) and the weights
// are rounded to bf16 last.  Also the fp32 SIMT router used for fp32 layers.
#include "common.hpp"
#include "kernels.hpp"
#include "topk.hpp"

namespace moe {
namespace {

template <int PER_LANE>
__device__ __forceinline__ void token_topk(const float* __restrict__ partial, int nsplit, int ldl, int T, int E,
                                           int k, int has_sg, int page, int t, int lane, int32_t* __restrict__ ids,
                                           float* __restrict__ w, float* __restrict__ shared_logit, int* lds_ids) {
  // logits = sum of the K-chunk partials, chunk order fixed
  const int64_t cstride = (int64_t)T * ldl;
  const float* row = partial + (int64_t)t * ldl;
  uint64_t key[PER_LANE];
  float lg[PER_LANE];
#pragma unroll
  for (int i = 0; i < PER_LANE; ++i) lg[i] = 0.f;
  // four chunks at a time, every load unconditional (addresses clamped into
  // the row, padding lanes zeroed later), then added in chunk order
  for (int c0 = 0; c0 < nsplit; c0 += 4) {
    float v[4][PER_LANE];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = c0 + u < nsplit ? c0 + u : nsplit - 1;
#pragma unroll
      for (int i = 0; i < PER_LANE; ++i) {
        const int e = lane + 64 * i < E ? lane + 64 * i : E - 1;
        v[u][i] = row[c * cstride + e];
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (c0 + u < nsplit)
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) lg[i] += v[u][i];
  }
#pragma unroll
  for (int i = 0; i < PER_LANE; ++i) {
    const int e = lane + 64 * i;
    float a = lg[i];
    if (page) a = bf2f(f2bf(a));  // logits in the activation dtype (round to nearest even)
    key[i] = make_key(e < E ? ord(a) : 0u, e);
  }
  const uint64_t sel = select_topk<PER_LANE>(key, k, lane);
  const uint32_t sel_hi = (uint32_t)(sel >> 32), sel_lo = (uint32_t)sel;
  const float top = unord(__builtin_amdgcn_readlane(sel_hi, 0));
  const float ex = lane < k ? expf(unord(sel_hi) - top) : 0.f;
  const float sum = wave_sum(ex);
  if (lane < k) {
    const float wj = ex / sum;
    ids[(int64_t)t * k + lane] = (int32_t)~sel_lo;
    w[(int64_t)t * k + lane] = page ? bf2f(f2bf(wj)) : wj;  // mixing weight in the activation dtype
    if (lds_ids) lds_ids[t * k + lane] = (int)~sel_lo;
  }
  if (has_sg && lane == 0) {
    float a = 0.f;
    for (int c = 0; c < nsplit; ++c) a += row[c * cstride + E];
    shared_logit[t] = a;
  }
}

template <int PER_LANE>
__global__ __launch_bounds__(256) void topk_kernel(const float* __restrict__ partial, int nsplit, int ldl, int T,
                                                   int E, int k, int has_sg, int page, int32_t* __restrict__ ids,
                                                   float* __restrict__ w, float* __restrict__ shared_logit) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;  // whole wave
  token_topk<PER_LANE>(partial, nsplit, ldl, T, E, k, has_sg, page, t, threadIdx.x & 63, ids, w, shared_logit,
                       nullptr);
}

// Top-k and dispatch of a batch of at most kSmallBatch tokens in one kernel:
// workgroup t (one wave) picks token t's experts as topk_kernel does; the
// last workgroup to finish (a device-scope counter, zero at launch) then
// performs the dispatch of the section's pipeline figure for the whole
// batch: a bit mask per expert of the tokens that chose it (a token's k
// picks are distinct experts), an exclusive scan of the mask populations
// into expert_offsets, and each assignment a = t*k + j placed at its
// expert's offset plus the number of earlier tokens in the expert's mask,
// which is its rank among the expert's assignments in ascending a: the same
// stable order as the counting sort of the dispatch kernels.  The last
// workgroup leaves the counter at zero.
template <int PER_LANE>
__global__ __launch_bounds__(64) void topk_dispatch_small_kernel(
    const float* __restrict__ partial, int nsplit, int ldl, int T, int E, int k, int has_sg, int page,
    int32_t* __restrict__ ids, float* __restrict__ w, float* __restrict__ shared_logit, int32_t* __restrict__ offsets,
    int32_t* __restrict__ sorted, int32_t* __restrict__ pos, int32_t* counter) {
  __shared__ uint32_t mask[kMaxExperts];
  __shared__ int start[kMaxExperts];
  const int lane = threadIdx.x;
  token_topk<PER_LANE>(partial, nsplit, ldl, T, E, k, has_sg, page, blockIdx.x, lane, ids, w, shared_logit,
                       nullptr);
  __threadfence();  // this token's ids are visible device-wide before it is counted
  int last = 0;
  if (lane == 0) last = atomicAdd(counter, 1) == T - 1 ? 1 : 0;
  if (!__builtin_amdgcn_readfirstlane(last)) return;
  __threadfence();  // every token's ids are visible here
  const int R = T * k;
  for (int e = lane; e < E; e += 64) mask[e] = 0u;
  __syncthreads();
  for (int a = lane; a < R; a += 64) atomicOr(&mask[ids[a]], 1u << (a / k));
  __syncthreads();
  // exclusive scan of the populations: lane owns experts [lane*per, +per)
  const int per = (E + 63) / 64;
  const int e0 = lane * per;
  int local = 0;
  for (int i = 0; i < per; ++i) local += e0 + i < E ? __popc(mask[e0 + i]) : 0;
  int incl = local;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(incl, o, 64);
    if (lane >= o) incl += u;
  }
  int run = incl - local;
  for (int i = 0; i < per; ++i) {
    const int e = e0 + i;
    if (e < E) {
      offsets[e] = run;
      start[e] = run;
      run += __popc(mask[e]);
    }
  }
  if (lane == 63) offsets[E] = incl;
  __syncthreads();
  for (int a = lane; a < R; a += 64) {
    const int e = ids[a];
    const int t = a / k;
    const int p = start[e] + __popc(mask[e] & ((1u << t) - 1u));
    sorted[p] = a;
    pos[a] = p;
  }
  if (lane == 0) *counter = 0;
}

// fp32 logits for fp32 layers: one thread per (token, column), h ascending.
__global__ void router_f32_kernel(const float* __restrict__ x, const float* __restrict__ wr,
                                  const float* __restrict__ wsg, float* __restrict__ logits, int T, int H, int E,
                                  int N, int32_t* zero_word) {
  const int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (zero_word && idx == 0) *zero_word = 0;  // a word the next kernel needs at zero (or null)
  if (idx >= (int64_t)T * N) return;
  const int t = (int)(idx / N), n = (int)(idx % N);
  const float* a = x + (int64_t)t * H;
  const float* b = n < E ? wr + (int64_t)n * H : wsg;
  float s = 0.f;
  for (int h = 0; h < H; ++h) s = fmaf(a[h], b[h], s);
  logits[idx] = s;
}

}  // namespace

hipError_t launch_topk(const float* partial, int nsplit, int ldl, int T, int E, int k, int has_sg, bool page,
                       int32_t* ids, float* w, float* shared_logit, hipStream_t s) {
  const int grid = (T + 3) / 4;
  const int per = (E + 63) / 64;
#define MOE_TOPK(P) \
  topk_kernel<P><<<grid, 256, 0, s>>>(partial, nsplit, ldl, T, E, k, has_sg, page ? 1 : 0, ids, w, shared_logit)
  if (per <= 1) MOE_TOPK(1);
  else if (per <= 2) MOE_TOPK(2);
  else if (per <= 4) MOE_TOPK(4);
  else if (per <= 8) MOE_TOPK(8);
  else MOE_TOPK(16);
#undef MOE_TOPK
  return hipGetLastError();
}

hipError_t launch_topk_dispatch_small(const float* partial, int nsplit, int ldl, int T, int E, int k, int has_sg,
                                     bool page, int32_t* ids, float* w, float* shared_logit, int32_t* offsets,
                                     int32_t* sorted, int32_t* pos, int32_t* counter, hipStream_t s) {
  if (T < 1 || T > kSmallBatch || k > 64 || E > kMaxExperts || !counter) return hipErrorInvalidValue;
  const int per = (E + 63) / 64;
#define MOE_TOPK_DISPATCH(P)                                                                                    \
  topk_dispatch_small_kernel<P><<<T, 64, 0, s>>>(partial, nsplit, ldl, T, E, k, has_sg, page ? 1 : 0, ids, w, \
                                                 shared_logit, offsets, sorted, pos, counter)
  if (per <= 1) MOE_TOPK_DISPATCH(1);
  else if (per <= 2) MOE_TOPK_DISPATCH(2);
  else if (per <= 4) MOE_TOPK_DISPATCH(4);
  else if (per <= 8) MOE_TOPK_DISPATCH(8);
  else MOE_TOPK_DISPATCH(16);
#undef MOE_TOPK_DISPATCH
  return hipGetLastError();
}

hipError_t launch_router_logits_f32(const float* x, const float* w_router, const float* w_sg, float* logits, int T,
                                    int H, int E, hipStream_t s, int32_t* zero_word) {
  const int N = E + (w_sg ? 1 : 0);
  const int64_t n = (int64_t)T * N;
  router_f32_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(x, w_router, w_sg, logits, T, H, E, N, zero_word);
  return hipGetLastError();
}

}  // namespace moe
