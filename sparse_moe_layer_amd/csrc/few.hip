// The whole layer for a few tokens (T <= 16) in two kernels (Qwen3.8-Flash-Next
// study, MoE section: eq. expert(x) and eq. MoE(x) over its pipeline figure):
//   few_router_kernel  : logits[t, e] = x_t . W_r[e] and x_t . w_sg, complete in fp32, and the
//                        shared expert's hidden h_sh = SiLU(S_gate x) * (S_up x), which needs no routing
//   few_experts_kernel : top-k and weights, then h = SiLU(W_gate x) * (W_up x) of every
//                        (token, expert) pair, then
//     out[t] = sum_j w[t,j] W_down[e_j] h[t,j] + sigmoid(s_t) S_down h_sh[t]
// A batch this small is bound by reading the touched experts' weights once,
// and below a few hundred MB by the latency of the steps between them, so the
// launches between the stages go: every workgroup does the top-k itself (a few
// KB of logits), and the one dependency between workgroups, h before the down
// products, is counters in memory.
//
// Work order and why every wait ends: the gate/up chunks have owners, but an
// owner takes its chunk by a flag first.  A workgroup waits for h only when its
// own chunks are done, and while it waits it looks for chunks whose flag is
// free and does them.  So a chunk is held by a wave that runs and waits for
// nothing, or free for any waiting workgroup, and the number of finished slabs
// reaches its total whatever else the GPU runs, even with one workgroup of the
// grid resident.
//
// Gate/up: a slab is 16 hidden columns, a block of their gate rows and one of
// their up rows; when the slabs are fewer than the waves their K range is split over 2
// to 8 waves of a workgroup, added in LDS in K order.  Down: a workgroup owns
// up to 16 output columns and goes over all groups, each wave over an equal
// share of their K ranges; a fragment row is a token, so each group's fp32 block
// is scaled by the routing weights and added in registers, the waves' sums are
// added in LDS in wave order, and out is rounded once.  No per-assignment
// output is stored or rounded, and no sum depends on timing.  A wave asks for
// its first down weights before it waits for h, so the memory stays busy
// across the dependency.
//
// Measured (2560 x 640, 512 experts, 10 a token): one token 36 us with bf16
// experts (111 MB, 17.7 us at the rate of a read probe), 30 with MXFP4 (39 MB,
// 6.2); 16 tokens fp8 150 us (692 MB, 110).  bf16 at 12 tokens and more (1 GB)
// streams slower than the kernels of moe_layer_forward: 16 tokens 257 us against
// 249, the 2.4T shape 213 to 2202 against 202 to 2084 (1 to 16 tokens).
// One token is bound by the steps' latency, in us of the MXFP4 call: router and the
// gap after it 6.5, top-k 4.7, list and first loads 2.6, gate/up 7.4, the counters
// 3.9, down 5.3.  Sixteen waves of 128 registers instead of 8 of 256 spilled in the
// MXFP4 loop (43.9 us); two batches of down weights in flight were slower (31.8: the
// compiler waits for both).
#include <atomic>

#include "common.hpp"
#include "frag_dot.hpp"
#include "kernels.hpp"
#include "topk.hpp"

namespace moe {
namespace {

using fragdot::Job;
using fragdot::BaseRows;
using fragdot::NoGate;

constexpr int RW = 16;                       // waves per workgroup of the router kernel
constexpr int kLogFW = 3, FW = 1 << kLogFW;  // of the experts kernel, one workgroup per compute unit
constexpr int kSlab = 16;                    // hidden columns per slab: a block of gate rows and one of up rows
constexpr int kFewRows = kSmallBatch * 64;  // (token, expert) pairs at most
static_assert(kSmallBatch == 16 && kMaxExperts < 2048, "a fragment row per token; packed list entries");

// A hidden value of the shared expert as two bf16, its rounding and what that
// left, together 16 bits of significand.  The shared expert outweighs the routed ones
// (a gate of about 1/2 against weights of about 1 / k), so with its h rounded to
// one bf16 the error of out against 64 bits is up to 1.56 times that of rounding
// out alone.  The routed experts' h is one bf16, as in the other calls: in
// two parts it took 159.5 against 150.5 us (16 tokens fp8) and 226 against 207 (4
// tokens of the 2.4T shape).  An infinity or NaN has no second part.
__device__ __forceinline__ uint32_t split(float v) {
  const bf16 hi = f2bf(v);
  const float rest = v - bf2f(hi);
  const bf16 lo = f2bf(fabsf(bf2f(hi)) < __builtin_inff() ? rest : 0.f);
  return (uint32_t)__builtin_bit_cast(uint16_t, hi) | (uint32_t)__builtin_bit_cast(uint16_t, lo) << 16;
}

// Workgroups [0, nr): 16 router rows each; workgroup nr (shared expert only):
// its gate's logit; the rest: 8 of its hidden columns each (8 gate, 8 up rows).
// K is split over the waves, whose blocks are added in wave order.  The grid also
// zeroes the counters and claim flags of the kernel that follows.
__global__ __launch_bounds__(RW * 64) void few_router_kernel(const bf16* __restrict__ x, const bf16* __restrict__ wr,
                                                             const bf16* __restrict__ wsg, float* __restrict__ logits,
                                                             int T, int H, int E, int N, int nr,
                                                             const bf16* __restrict__ shg,
                                                             const bf16* __restrict__ shu, int Is,
                                                             bf16* __restrict__ h_sh, int kchunk, int32_t* counters,
                                                             int ncounters) {
  for (int i = blockIdx.x * (RW * 64) + threadIdx.x; i < ncounters; i += gridDim.x * (RW * 64)) counters[i] = 0;
  __shared__ f32x4 part[RW][64];
  __shared__ __attribute__((aligned(16))) char act[RW][fragdot::kLds];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int m = lane & 15;
  const int kbeg = w * kchunk;
  const int kend = kbeg + kchunk < H ? kbeg + kchunk : H;
  const bool route = (int)blockIdx.x <= nr;
  const int c0 = (int)blockIdx.x <= nr ? blockIdx.x * 16 : (blockIdx.x - nr - 1) * 8;
  Job<1> b{};
  int cols;
  if ((int)blockIdx.x < nr) {
    cols = E - c0 < 16 ? E - c0 : 16;
    b.w[0] = reinterpret_cast<const char*>(wr + (int64_t)c0 * H);
    b.w[1] = reinterpret_cast<const char*>(wr + (int64_t)(c0 + 8) * H);
    b.wrows[0] = cols < 8 ? cols : 8;
    b.wrows[1] = cols < 8 ? 0 : cols - 8;
  } else if (route) {
    cols = 1;
    b.w[0] = b.w[1] = reinterpret_cast<const char*>(wsg);
    b.wrows[0] = 1;
  } else {
    cols = Is - c0 < 8 ? Is - c0 : 8;
    b.w[0] = reinterpret_cast<const char*>(shg + (int64_t)c0 * H);
    b.w[1] = reinterpret_cast<const char*>(shu + (int64_t)c0 * H);
    b.wrows[0] = b.wrows[1] = cols;
  }
  b.rows = T;
  b.ar = m < T ? m : 0;
  b.k0 = kbeg;
  b.kend = kend;
  bool todo = kbeg < kend;
  part[w][lane] = f32x4{0.f, 0.f, 0.f, 0.f};
  fragdot::run<kWtPlain, 1, 0>(
      x, (uint32_t)T * (uint32_t)H * 2u, H, lane, act[w], BaseRows{},
      [&](Job<1>& j) {
        if (todo) j = b;
        const bool was = todo;
        todo = false;
        return was;
      },
      [&](int, const f32x4 (&acc)[1]) { part[w][lane] = acc[0]; }, NoGate{});
  __syncthreads();
  if (w == 0) {
    f32x4 t = part[0][lane];
#pragma unroll
    for (int i = 1; i < RW; ++i) t += part[i][lane];
    const int col = (int)blockIdx.x == nr ? E : c0 + m;  // logits column
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = 4 * (lane >> 4) + i;
      if (route) {
        if (tok < T && m < cols) logits[(int64_t)tok * N + col] = t[i];
      } else {
        const float up = __shfl_xor(t[i], 8, 64);  // the up row of lane m is lane m + 8's
        if (tok < T && m < cols) {
          const uint32_t h = split(silu(t[i]) * up);
          bf16* at = h_sh + (int64_t)(2 * tok) * Is + c0 + m;
          at[0] = __builtin_bit_cast(bf16, (uint16_t)h);
          at[Is] = __builtin_bit_cast(bf16, (uint16_t)(h >> 16));
        }
      }
    }
  }
}

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, ROWS, 0xf, false));
}
// Sum over the 64 lanes (wave-uniform), in a fixed order.
__device__ __forceinline__ float row_sum(float v) {
  v = dpp_add<0x111, 0xf>(v);  // row_shr:1, 2, 4, 8: lane 15 of each row has the row's
  v = dpp_add<0x112, 0xf>(v);
  v = dpp_add<0x114, 0xf>(v);
  v = dpp_add<0x118, 0xf>(v);
  v = dpp_add<0x142, 0xa>(v);  // row_bcast:15 into rows 1 and 3
  v = dpp_add<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// Top-k of one token by one wave, into ids[0..k) and wts[0..k) (LDS).  The
// k-th largest of the 64 lanes' own maxima bounds the answer from below, so
// only logits at least that large (about k of them) are ranked, each by
// counting the larger ones.  More than 64 candidates (many equal logits): k
// rounds of a wave-wide maximum.  keys: kMaxExperts of LDS.  The loops are
// rolled where that costs little: the code runs once, and its instructions
// arrive from memory.
__device__ __forceinline__ void pick(const float* row, int E, int k, int page, int lane, uint32_t* keys,
                                     uint64_t* cand, int* ids, float* wts) {
  uint32_t top = 0;
#pragma unroll 4
  for (int e = lane; e < E; e += 64) {
    float a = row[e];
    if (page) a = bf2f(f2bf(a));
    const uint32_t v = ord(a);
    keys[e] = v;
    top = v > top ? v : top;
  }
  // how many lanes' maxima rank before this lane's: all 64 read back from LDS
  uint32_t* const tops = reinterpret_cast<uint32_t*>(cand);
  tops[lane] = top;
  __builtin_amdgcn_wave_barrier();
  int above = 0;
#pragma unroll 4
  for (int j = 0; j < 64; j += 4) {
    const u32x4 o = *reinterpret_cast<const u32x4*>(tops + j);
#pragma unroll
    for (int i = 0; i < 4; ++i) above += o[i] > top || (o[i] == top && j + i < lane);
  }
  const uint32_t bound =
      (uint32_t)__builtin_amdgcn_readlane((int)top, __builtin_ctzll(__ballot(above == k - 1) | 1ull << 63));
  int n = 0;
#pragma unroll 4
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    const uint32_t v = e < E ? keys[e] : 0u;
    const bool in = e < E && v >= bound;
    const uint64_t bal = __ballot(in);
    const int at = n + __popcll(bal & ((1ull << lane) - 1ull));
    if (in && at < 64) cand[at] = make_key(v, e);
    n += __popcll(bal);
  }
  n = (int)uniform((uint32_t)n);
  __builtin_amdgcn_wave_barrier();
  uint64_t mine = 0;
  int rank = 64;
  if (n <= 64) {
    mine = lane < n ? cand[lane] : 0ull;
    cand[lane] = mine;  // (zeros behind the candidates)
    __builtin_amdgcn_wave_barrier();
    rank = lane < n ? 0 : 64;
#pragma unroll 1
    for (int j = 0; j < n; j += 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) rank += cand[j + i] > mine;
    }
  } else {
    for (int j = 0; j < k; ++j) {
      uint64_t best = 0;
      for (int e = lane; e < E; e += 64)
        if (keys[e]) best = key_max(best, make_key(keys[e], e));
      best = wave_key_max(best);
      if (lane == j) {
        mine = best;
        rank = j;
      }
      const uint32_t e = ~(uint32_t)best;
      if (lane == 0 && e < (uint32_t)E) keys[e] = 0u;  // taken
      __builtin_amdgcn_wave_barrier();
    }
  }
  const float l = unord((uint32_t)(mine >> 32));
  const float best = __uint_as_float((uint32_t)__builtin_amdgcn_readlane(
      (int)__float_as_uint(l), __builtin_ctzll(__ballot(rank == 0) | 1ull << 63)));
  const bool in = rank < k;
  const float ex = in ? expf(l - best) : 0.f;
  const float v = ex / row_sum(ex);
  if (lane < k) ids[lane] = E - 1;  // (NaN logits may leave places without a pick)
  if (lane < k) wts[lane] = 0.f;
  if (in) {
    const uint32_t e = ~(uint32_t)mine;
    ids[rank] = e < (uint32_t)E ? (int)e : E - 1;
    wts[rank] = page ? bf2f(f2bf(v)) : v;
  }
}

// What a workgroup knows of the batch's routing.
struct FewRoute {
  // groups: a touched expert and up to ROWS of its tokens, experts by first use; expert | tokens << 11
  uint32_t list[kFewRows];
  uint16_t base[kFewRows];       // its first row of h
  float w[kFewRows];             // per row of h: the routing weight
  uint8_t token[kFewRows];       // and the token
  float sg[kSmallBatch];         // sigmoid of the shared gate logit
  int groups;
  int claim;                     // whether the workgroup's next chunk is its own
  int left;                      // waves done with their gate/up work, their slabs << 8
  int ready;                     // every h is written
};

// Polls (about 0.3 us each) between looks for unclaimed chunks; after one that was
// found, at once (16 tokens, 128 fp8 experts of 1024 x 640, half of the grid there:
// 9.4 -> 0.97 ms, of which the first look is 0.6).
constexpr int kHelpAfter = 2048;
constexpr int kUnitK = 128;     // K values per unit of the shares of K

template <int WT>
__global__ __launch_bounds__(FW * 64, 2) void few_experts_kernel(FfnArgs f, FewArgs a) {
  using F = fragdot::Form<WT>;
  // per wave: the logits' keys and candidates, later activations; picks and expert tables; the waves' blocks
  __shared__ __attribute__((aligned(16))) char act[FW][fragdot::Form<kWtPlain, 2 * kSmallBatch>::LDS];
  __shared__ __attribute__((aligned(16))) uint64_t cand[FW][64];
  __shared__ int ids[kFewRows];
  __shared__ float wts[kFewRows];
  __shared__ uint32_t tmask[kMaxExperts];
  __shared__ int lead[kMaxExperts];
  __shared__ f32x4 part[FW][2][64];
  __shared__ FewRoute r;
  const int tid = threadIdx.x, lane = tid & 63, wave = (int)uniform(tid >> 6);
  const int T = f.T, k = f.k, E = f.E, R = T * k;
  const bool shared = a.has_shared != 0;
  const int N = E + (shared ? 1 : 0);
  const int grid = a.owners, waves = grid * FW;  // that own gate/up chunks
  const int gw = (int)blockIdx.x * FW + wave;
  int32_t* const claims = a.counters + (kFewDone + 1) * kFewCounterStride;

  // ---- routing: every workgroup for itself, a wave per token ----
  for (int t = wave; t < T; t += FW) {
    const float* row = a.logits + (int64_t)t * N;
    pick(row, E, k, a.page, lane, reinterpret_cast<uint32_t*>(act[wave]), cand[wave], ids + t * k, wts + t * k);
    if (shared && lane == 0) r.sg[t] = sigmoid(row[E]);
  }
  __syncthreads();
  // Wave 0 groups the assignments i = t * k + j by expert: an expert's token
  // mask, its first assignment (its place in the list is by first use), its
  // first row of h and its groups.  (An expert with more than ROWS tokens is
  // read once per group: with MXFP4, 512 experts and 16 tokens 2 in 1000 have more
  // than 4; with 8 experts and 2 picks a third do: 40.6 us against 32.2 of the
  // layer call's kernels, 4096 x 1024.)
  // LDS operations of one wave are executed in order.
  if (wave == 0) {
    for (int i = lane; i < R; i += 64) {
      tmask[ids[i]] = 0u;
      lead[ids[i]] = R;
    }
    __builtin_amdgcn_wave_barrier();
    for (int i = lane; i < R; i += 64) {
      atomicOr(&tmask[ids[i]], 1u << (i / k));
      atomicMin(&lead[ids[i]], i);
    }
    __builtin_amdgcn_wave_barrier();
    const uint64_t below = (1ull << lane) - 1ull;
    int ng = 0, rows = 0;
    for (int i0 = 0; i0 < R; i0 += 64) {
      const int i = i0 + lane;
      const int e = i < R ? ids[i] : 0;
      const bool first = i < R && lead[e] == i;
      const uint32_t mk = first ? tmask[e] : 0u;
      const uint32_t n = (uint32_t)__popc(mk);                 // 0 .. 16 rows
      const uint32_t parts = (n + F::ROWS - 1) / F::ROWS;      // groups
      int rb = rows, gb = ng;  // rows and groups of lower lanes, by bit planes
      for (int b = 0; b < 5; ++b) {
        const uint64_t pr = __ballot(n >> b & 1u), pg = __ballot(parts >> b & 1u);
        rb += __popcll(pr & below) << b;
        gb += __popcll(pg & below) << b;
        rows += __popcll(pr) << b;
        ng += __popcll(pg) << b;
      }
      if (first) {
        tmask[e] = mk | (uint32_t)rb << 16;  // for the weights
        uint32_t left = mk;
        for (int at = gb; left; ++at) {
          uint32_t sub = 0;
          for (int j = 0; j < F::ROWS && left; ++j) {
            sub |= left & -left;
            left &= left - 1u;
          }
          r.list[at] = (uint32_t)e | sub << 11;
          r.base[at] = (uint16_t)rb;
          rb += __popc(sub);
        }
      }
    }
    if (lane == 0) {
      r.groups = ng;
      r.ready = r.left = 0;
    }
    __builtin_amdgcn_wave_barrier();
    for (int i = lane; i < R; i += 64) {
      const uint32_t v = tmask[ids[i]], row = (v >> 16) + __popc(v & ((1u << (i / k)) - 1u));
      r.w[row] = wts[i];
      r.token[row] = (uint8_t)(i / k);
    }
  } else if (wave == 1 && blockIdx.x == 0) {
    for (int i = lane; i < R; i += 64) {
      if (a.ids) a.ids[i] = ids[i];
      if (a.w) a.w[i] = wts[i];
    }
  }
  __syncthreads();
  const int ng = r.groups;
  // ---- gate/up: slabs of 16 hidden columns ----
  // Chunk c is slab c, wave c mod waves.  With fewer slabs than waves, P waves of
  // a workgroup share a slab's K range: chunk c is then FW / P slabs, workgroup
  // c mod grid.
  const int slabs = a.slabs.d, total = ng * slabs, units = a.units, cols = a.cols;
  int lp = 0;  // P = 1 << lp
  while (1 << lp < FW && (total << (lp + 1)) <= waves + waves / 4 && 2 << lp <= units) ++lp;
  const int P = 1 << lp;
  const int lper = lp > 0 ? kLogFW - lp : 0;
  const int chunks = (total + (1 << lper) - 1) >> lper;
  // Finished slabs are counted in kFewDone counters, by the chunk's owner; the
  // one that completes a counter adds to the last counter, which is watched.
  const int l_own = lp > 0 ? 0 : kLogFW;  // chunk c counts in counter (c >> l_own) % kFewDone
  auto counted = [&](int i) {        // slabs of counter i
    const int all = chunks >> l_own, rest = chunks & ((1 << l_own) - 1);  // owners in full, chunks of the last
    int n = ((all + kFewDone - 1 - i) / kFewDone) << l_own;
    if (all % kFewDone == i) n += rest;
    n <<= lper;
    if (((chunks - 1) >> l_own) % kFewDone == i) n -= (chunks << lper) - total;
    return n;
  };
  const int owners = (chunks + (1 << l_own) - 1) >> l_own, counters = owners < kFewDone ? owners : kFewDone;
  int32_t* const last = a.counters + kFewDone * kFewCounterStride;
  auto count = [&](int i, int n) {  // n finished slabs of counter i (one lane)
    const int got = n + __hip_atomic_fetch_add(a.counters + i * kFewCounterStride, n, __ATOMIC_RELAXED,
                                               __HIP_MEMORY_SCOPE_AGENT);
    if (got == counted(i)) __hip_atomic_fetch_add(last, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  const int q = lane >> 4, m = lane & 15;
  auto finish = [&](int s, const f32x4& gate, const f32x4& up) {  // lane: column m, group rows 4 q + v
    int i, c0;
    a.slabs.divide(s, i, c0);
    const int rows = __popc(uniform(r.list[i]) >> 11), col = c0 * kSlab + m;
    uint16_t* h = reinterpret_cast<uint16_t*>(f.h) + (int64_t)uniform(r.base[i]) * f.I + col;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (col < f.I && 4 * q + v < rows)  // written through to the device's memory
        __hip_atomic_store(h + (int64_t)(4 * q + v) * f.I, __builtin_bit_cast(uint16_t, f2bf(silu(gate[v]) * up[v])),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  // a chunk that nobody has claimed (then this wave has), or -1: 64 flags at a
  // time, from a place of the workgroup's own on, so that few ask for the same
  auto find_open = [&] {
    const int stride = P > 1 ? FW : 1, sets = (chunks + 63) / 64, turn = (int)blockIdx.x;
    for (int i = 0; i < sets; ++i) {
      const int c0 = (i + turn) % sets * 64, here = c0 + ((lane + turn / sets) & 63);
      const bool open =
          here < chunks && __hip_atomic_load(claims + here * stride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == 0;
      for (uint64_t bal = __ballot(open); bal; bal &= bal - 1) {
        const int c = c0 + ((__builtin_ctzll(bal) + turn / sets) & 63);
        int got = 1;
        if (lane == 0)
          got = __hip_atomic_exchange(claims + c * stride, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (uniform((uint32_t)got) == 0u) return c;
      }
    }
    return -1;
  };
  // A wave's own chunks first, claimed up to 64 at a time.  Then it says so, and
  // wave 0 watches the last counter for its workgroup; every so often it looks
  // for a chunk that nobody has claimed (its owner may not be resident while this
  // workgroup holds its place) and does it alone, with the same arithmetic.
  bool own = true;
  int polls = 0, done = 0;  // done: slabs of this wave (P > 1: of this workgroup, in wave 0)
  int c = P > 1 ? (int)blockIdx.x : gw;
  for (;;) {
    // the next jobs: parts [p0, p1) of slabs s, s + step (P == 1: those of a mask), one for P > 1
    uint64_t todo = 1;
    int s, end, p0 = 0, p1 = P;
    if (own && c < chunks) {
      s = c << lper;
      end = total;
      if (P > 1) {
        // (a workgroup's chunk has the flag claims[c * FW])
        if (tid == 0)
          r.claim = __hip_atomic_exchange(claims + c * FW, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        const bool mine = uniform((uint32_t)r.claim) == 0u;
        __syncthreads();
        c += grid;
        if (!mine) continue;
        end = s + (1 << lper) < total ? s + (1 << lper) : total;
        if (wave == 0) done += end - s;
        s += wave >> lp;
        end = s < end ? s + 1 : s;
        p0 = wave & (P - 1);
        p1 = p0 + 1;
        if (s >= end) todo = 0;
      } else {
        const int at = c + lane * waves;
        int taken = 1;
        if (at < chunks)
          taken = __hip_atomic_exchange(claims + at, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        todo = __ballot(taken == 0);
        done += __popcll(todo);
        c += 64 * waves;
      }
    } else if (own) {
      // Stores of h are written through, and acknowledged before they are
      // counted; the workgroup's last wave adds its slabs to one of the counters
      // (one counter for 256 workgroups took 2.9 us, a fence that writes the L2
      // back 1.4 us).
      own = false;
      __builtin_amdgcn_s_waitcnt(0);
      __builtin_amdgcn_sched_barrier(0);
      if (lane == 0) {
        const int before =
            __hip_atomic_fetch_add(&r.left, done << 8 | 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_WORKGROUP);
        if ((before & 255) == FW - 1 && (before >> 8) + done > 0)
          count((int)blockIdx.x % kFewDone, (before >> 8) + done);
      }
      if (wave != 0 || (int)blockIdx.x * cols >= f.H) break;  // (no down columns: nothing to wait for)
      continue;
    } else {
      if (__hip_atomic_load(last, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) >= counters) break;
      int open = -1;
      if (++polls % kHelpAfter == 0) open = find_open();
      if (open < 0) {
        __builtin_amdgcn_s_sleep(1);
        continue;
      }
      polls = kHelpAfter - 1;  // where there was one there may be more: look again after it
      s = open << lper;
      end = s + (1 << lper) < total ? s + (1 << lper) : total;
    }
    const int first = s;
    int p = p0, parts = 0;
    f32x4 v[2] = {};
    fragdot::run<WT, 2, 0>(
        f.x, (uint32_t)T * (uint32_t)f.H * 2u, f.H, lane, act[wave],
        [&](const auto& j, int row) { return (int)r.token[j.base + row]; },
        [&](auto& j) {
          if (!todo) return false;
          int at = s;
          if (P == 1) {
            at += __builtin_ctzll(todo) * waves;
            todo &= todo - 1;
          }
          int i, c0;
          a.slabs.divide(at, i, c0);
          c0 *= kSlab;
          const uint32_t entry = uniform(r.list[i]);
          const int g = entry & 2047;
          const int left = f.I - c0 < kSlab ? f.I - c0 : kSlab;
          j.w[0] = static_cast<const char*>(f.wg) + fragdot::wbytes<WT>((int64_t)g * f.sg + (int64_t)c0 * f.H);
          j.w[2] = static_cast<const char*>(f.wu) + fragdot::wbytes<WT>((int64_t)g * f.su + (int64_t)c0 * f.H);
          j.w[1] = j.w[0] + fragdot::wbytes<WT>(8 * (int64_t)f.H);
          j.w[3] = j.w[2] + fragdot::wbytes<WT>(8 * (int64_t)f.H);
          j.wrows[0] = j.wrows[2] = left < 8 ? left : 8;
          j.wrows[1] = j.wrows[3] = left < 8 ? 0 : left - 8;
          if constexpr (WT != kWtPlain) {
            const int n = WT == kWtMx ? lane >> 2 : m;
            const int col = c0 + (n < left ? n : left - 1);
            const int64_t at = WT == kWtFp8 ? ((int64_t)g * (f.I / 128) + col / 128) * (f.H / 128) * 4
                                            : ((int64_t)g * f.I + col) * (f.H / 32);
            j.scale[0] = reinterpret_cast<const char*>(f.scg) + at;
            j.scale[1] = reinterpret_cast<const char*>(f.scu) + at;
          }
          j.base = (int)uniform(r.base[i]);
          j.rows = __popc(entry >> 11);
          j.ar = m < j.rows ? m : 0;
          j.k0 = ((p * units) >> lp) * kUnitK;
          const int ke = (((p + 1) * units) >> lp) * kUnitK;
          j.kend = ke < f.H ? ke : f.H;
          j.tag = at;
          if (P > 1 && ++p == p1) {
            p = p0;
            if (++s >= end) todo = 0;
          }
          return true;
        },
        [&](int at, const f32x4 (&acc)[2]) {
          v[0] += acc[0];  // (parts of one slab follow each other in K order)
          v[1] += acc[1];
          if ((P > 1 && own) || ++parts < P) return;
          parts = 0;
          finish(at, v[0], v[1]);
          v[0] = v[1] = f32x4{0.f, 0.f, 0.f, 0.f};
        },
        NoGate{});
    if (own && P > 1) {
      part[wave][0][lane] = v[0];  // added in K order
      part[wave][1][lane] = v[1];
      __syncthreads();
      if (first < end && p0 == 0) {
        for (int w = 1; w < P; ++w) {
          v[0] += part[wave + w][0][lane];
          v[1] += part[wave + w][1][lane];
        }
        finish(first, v[0], v[1]);
      }
      __syncthreads();
    }
    if (!own) {
      __builtin_amdgcn_s_waitcnt(0);
      if (lane == 0) count(((first >> lper) >> l_own) % kFewDone, end - first);
    }
  }
  // every h is written: wave 0 knows, the others ask before their first activations
  if (tid == 0) __hip_atomic_store(&r.ready, 1, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_WORKGROUP);
  auto gate = [&] {
    while (!__hip_atomic_load(&r.ready, __ATOMIC_ACQUIRE, __HIP_MEMORY_SCOPE_WORKGROUP)) __builtin_amdgcn_s_sleep(1);
  };

  // ---- down and combine: up to 16 output columns over all groups ----
  // units of 128 K values: the groups', then the shared expert's (bf16, weighed by their size)
  constexpr int kWeigh = WT == kWtMx ? 4 : WT == kWtFp8 ? 2 : 1;  // a bf16 unit in units of this type
  const int ud = a.down_units.d, u_sh = a.shared_units;
  const int u_r = ng * ud, u_all = u_r + u_sh * kWeigh;
  const int lo = (u_all * wave) >> kLogFW, hi = (u_all * (wave + 1)) >> kLogFW;
  for (int c0 = (int)blockIdx.x * cols; c0 < f.H; c0 += (int)gridDim.x * cols) {
    const int ncol = f.H - c0 < cols ? f.H - c0 : cols;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    auto add = [&](bool sh, uint32_t mask, int base, const f32x4& p) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int t = 4 * q + v;
        if (mask >> t & 1u) sum[v] = fmaf(sh ? r.sg[t] : r.w[base + __popc(mask & ((1u << t) - 1u))], p[v], sum[v]);
      }
    };
    auto rows_of = [&](auto& j) {  // w[0] is the first column's row
      j.wrows[0] = ncol < 8 ? ncol : 8;
      j.wrows[1] = ncol < 8 ? 0 : ncol - 8;
    };
    // the shared expert's part first: it waits for no h of this kernel, and wave 0,
    // which watches the counter, has none of it
    const int s_lo = lo > u_r ? (lo - u_r) / kWeigh : 0, s_hi = hi > u_r ? (hi - u_r) / kWeigh : 0;
    bool todo = s_lo < s_hi;
    fragdot::run<kWtPlain, 1, 0, 2 * kSmallBatch, 4, true>(  // (h_sh is the first kernel's)
        f.h_sh, (uint32_t)T * (uint32_t)f.Is * 4u, f.Is, lane, act[wave], BaseRows{},
        [&](auto& j) {
          if (!todo) return false;
          todo = false;
          j.w[0] = static_cast<const char*>(f.shd) + (int64_t)c0 * f.Is * 2;
          j.w[1] = j.w[0] + 16 * (int64_t)f.Is;
          rows_of(j);
          j.rows = 2 * T;
          j.ar = m < T ? 2 * m : 0;
          j.k0 = s_lo * kUnitK;
          j.kend = s_hi * kUnitK < f.Is ? s_hi * kUnitK : f.Is;
          return true;
        },
        [&](int, const f32x4 (&acc)[1]) { add(true, (1u << T) - 1u, 0, acc[0]); }, NoGate{});
    int u = lo;
    const int r_hi = hi < u_r ? hi : u_r;
    fragdot::run<WT, 1, fragdot::kSc1>(
        f.h, (uint32_t)R * (uint32_t)f.I * 2u, f.I, lane, act[wave], BaseRows{},
        [&](auto& j) {
          if (u >= r_hi) return false;
          int i, u0;
          a.down_units.divide(u, i, u0);
          const int u1 = r_hi - u + u0 < ud ? r_hi - u + u0 : ud;
          const uint32_t entry = uniform(r.list[i]);
          const int g = entry & 2047;
          j.w[0] = static_cast<const char*>(f.wd) + fragdot::wbytes<WT>((int64_t)g * f.sd + (int64_t)c0 * f.I);
          j.w[1] = j.w[0] + fragdot::wbytes<WT>(8 * (int64_t)f.I);
          rows_of(j);
          auto scale_row = [&](int n) {
            const int col = c0 + (n < ncol ? n : ncol - 1);
            return WT == kWtFp8 ? static_cast<const void*>(f.scd +
                                                           ((int64_t)g * (f.H / 128) + col / 128) * (f.I / 128))
                                : static_cast<const void*>(reinterpret_cast<const uint8_t*>(f.scd) +
                                                           ((int64_t)g * f.H + col) * (f.I / 32));
          };
          if constexpr (WT != kWtPlain) j.scale[0] = scale_row(WT == kWtMx ? lane >> 2 : m);
          // fragment row m is token m (a token without this expert reads some row of it; its sum is not used)
          const uint32_t mask = entry >> 11;
          const int rank = __popc(mask & ((1u << m) - 1u));
          j.base = (int)uniform(r.base[i]);
          j.rows = __popc(mask);
          j.ar = rank < j.rows ? rank : j.rows - 1;
          j.k0 = u0 * kUnitK;
          j.kend = u1 * kUnitK < f.I ? u1 * kUnitK : f.I;
          j.tag = i;
          u += u1 - u0;
          return true;
        },
        [&](int i, const f32x4 (&acc)[1]) { add(false, uniform(r.list[i]) >> 11, (int)uniform(r.base[i]), acc[0]); },
        gate);
    part[wave][0][lane] = sum;
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int w = 1; w < FW; ++w) sum += part[w][0][lane];
      bf16* out = reinterpret_cast<bf16*>(a.out);
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (4 * q + v < T && m < ncol) out[(int64_t)(4 * q + v) * f.H + c0 + m] = f2bf(sum[v]);
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

// For tests (not in the public header): launch at most this many workgroups of
// the experts kernel, while the gate/up chunks stay dealt to the whole grid, so
// that those of the absent ones have to be found (0: the whole grid).
std::atomic<int> g_few_present{0};
extern "C" void moe_test_few_present(int32_t workgroups) { g_few_present.store(workgroups); }

size_t few_counter_ints(int64_t T, int64_t k, int64_t I) {
  // done counters, then a claim flag per wave chunk: of one slab or more each,
  // or FW flags per workgroup chunk where those are fewer than the waves
  const int64_t slabs = T * k * ((I + kSlab - 1) / kSlab), least = (int64_t)2 * kFewMaxGrid * FW;
  return (size_t)((kFewDone + 1) * kFewCounterStride + (slabs > least ? slabs : least));
}

hipError_t launch_layer_few(const FfnArgs& f, const void* w_router, const void* w_sg, FewArgs a, hipStream_t s) {
  if (f.T < 1 || f.T > kSmallBatch || f.E > kMaxExperts || f.k > 64) return hipErrorInvalidValue;
  const int N = f.E + (a.has_shared ? 1 : 0);
  const int kchunk = ((f.H + RW - 1) / RW + 31) / 32 * 32;
  const int nr = (f.E + 15) / 16, nsh = a.has_shared ? 1 + (f.Is + 7) / 8 : 0;
  few_router_kernel<<<nr + nsh, RW * 64, 0, s>>>(
      reinterpret_cast<const bf16*>(f.x), reinterpret_cast<const bf16*>(w_router), reinterpret_cast<const bf16*>(w_sg),
      a.logits, f.T, f.H, f.E, N, nr, reinterpret_cast<const bf16*>(f.shg), reinterpret_cast<const bf16*>(f.shu), f.Is,
      reinterpret_cast<bf16*>(f.h_sh), kchunk, a.counters, (int)few_counter_ints(f.T, f.k, f.I));
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // a workgroup per compute unit, a multiple of kFewDone
  int grid = (few_cus() < kFewMaxGrid ? few_cus() : kFewMaxGrid) / kFewDone * kFewDone;
  grid = grid < kFewDone ? kFewDone : grid;
  a.owners = grid;
  const int present = g_few_present.load(std::memory_order_relaxed);
  grid = present > 0 && present < grid ? present : grid;
  a.slabs = Divisor((f.I + kSlab - 1) / kSlab);
  a.units = (f.H + kUnitK - 1) / kUnitK;
  a.cols = (f.H + grid - 1) / grid < 16 ? (f.H + grid - 1) / grid : 16;
  a.down_units = Divisor((f.I + kUnitK - 1) / kUnitK);
  a.shared_units = a.has_shared ? (f.Is + kUnitK - 1) / kUnitK : 0;
  if (f.wt == kWtFp8) few_experts_kernel<kWtFp8><<<grid, FW * 64, 0, s>>>(f, a);
  else if (f.wt == kWtMx) few_experts_kernel<kWtMx><<<grid, FW * 64, 0, s>>>(f, a);
  else few_experts_kernel<kWtPlain><<<grid, FW * 64, 0, s>>>(f, a);
  return hipGetLastError();
}

}  // namespace moe
