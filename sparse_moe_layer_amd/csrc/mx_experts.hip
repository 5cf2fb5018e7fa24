// Grouped SwiGLU products of experts with MXFP4 weights (Qwen3.8-Flash-Next
// study, MoE section, eq. expert(x)): h = SiLU(W_gate x) * (W_up x) and
// y = W_down h with W[n, k] = e2m1(code[n, k]) 2^(scale[n, k / 32] - 127).
// Every such value is a bf16 value, so codes become bf16 by one scaled
// conversion per pair, exactly, and the products are v_mfma_f32_16x16x32_bf16
// with fp32 sums, as with bf16 weights.
//
// The K order inside a matrix instruction is free as long as both operands use
// it.  A lane's 16-byte load of codes is 32 values of one row, one scale group
// and its share of four instructions: instruction s of a 128-wide K run takes
// the values 32 q + 8 s .. + 8 of lane group q = lane / 16, of weights and
// activations alike.
//
//   mx_stream_kernel: groups of at most 16 rows; bound by reading the codes once
//   mx_tiles_kernel : 128-row m-tiles; bound by the matrix rate
#include <type_traits>

#include "common.hpp"
#include "frag_dot.hpp"
#include "kernels.hpp"

namespace moe {
namespace {

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

int cu_count() {
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

// ---- groups of at most 16 rows ---------------------------------------------
// An item is SB blocks of 16 weight rows and all rows of a group's m-block: with 4
// blocks 32 gate rows and the 32 up rows of the same hidden columns, or 64 output
// columns; with one, 8 gate and 8 up rows, or 16 output columns.  A wave goes
// through its items in one stream of loads, 128 bytes of 8 rows each.  With fewer
// items than waves, P waves of a workgroup share an item's K range and add their
// blocks in LDS in K order.
//   4 blocks use each activation fragment four times, which a batch of 24 tokens
// needs (512 experts, 2560 x 640: 120.5 us; 2 blocks and 256-byte runs, whose K
// step of 512 also fits a K of 640 badly, 128.4; both with a plan kernel before).  One block is for the few items
// of a small group list, where 4 leave compute units idle even with K split 8 ways
// (one token, a dense 8192 x 2048: 22.2 us with 4, 17.4 with one).
//   Bound by the loads: 24 tokens take 68 us in gate/up and 47 in down, without the
// products 64 and 45.
constexpr int kLogSW = 3, SW = 1 << kLogSW;  // waves per workgroup, one workgroup per compute unit
using SF = fragdot::Form<kWtMx, kStreamBM, 2>;
static_assert(kMaxExperts <= 1024, "packed list entries");

template <int PHASE, int SB>
__device__ __forceinline__ void mx_stream_items(const FfnArgs& f, int self_plan, int nblocks, const Divisor& slabs,
                                                const int* glist, const uint8_t* tokens, char* act,
                                                f32x4 (*part)[4][64], int lane, int wave) {
  constexpr int COLS = (PHASE == 1 ? 8 : 16) * SB;  // output columns of an item
  const int K = PHASE == 1 ? f.H : f.I, N = PHASE == 1 ? f.I : f.H;
  const int grid = (int)gridDim.x, waves = grid * SW;
  const int total = nblocks * slabs.d, units = (K + 127) >> 7;
  int lp = 0;  // P = 1 << lp
  while (1 << lp < SW && (total << (lp + 1)) <= waves + waves / 4 && 2 << lp <= units) ++lp;
  const int P = 1 << lp, p = wave & (P - 1);
  const int q = lane >> 4, m = lane & 15;

  auto finish = [&](int item, const f32x4 (&v)[SB]) {  // lane: column m, rows 4 q + i
    int sb, slab;
    slabs.divide(item, sb, slab);
    int base, nrows;
    if (self_plan) {
      const int g = glist[sb] & 1023, r0 = (glist[sb] >> 10) * kStreamBM;
      base = f.offsets[g] + r0;
      nrows = f.offsets[g + 1] - base;
    } else {
      base = f.sb_base[sb] + f.sb_row0[sb];
      nrows = f.sb_nrows[sb];
    }
    const int ld = PHASE == 1 ? f.I : f.H;
    bf16* out = reinterpret_cast<bf16*>(PHASE == 1 ? f.h : f.y) + (int64_t)(base + 4 * q) * ld;
#pragma unroll
    for (int b = 0; b < (PHASE == 1 && SB > 1 ? SB / 2 : SB); ++b) {
      const int col = slab * COLS + 16 * b + m;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float o = v[b][i];
        if (PHASE == 1) o = silu(o) * (SB > 1 ? v[(b + SB / 2) % SB][i] : __shfl_xor(o, 8, 64));  // (lane m + 8's)
        if (4 * q + i < nrows && col < N && (PHASE != 1 || SB > 1 || m < 8)) out[(int64_t)i * ld + col] = f2bf(o);
      }
    }
  };
  // P > 1: the workgroup takes SW / P items at a time
  const int step = P > 1 ? grid * (SW >> lp) : waves;
  int item = P > 1 ? ((int)blockIdx.x << (kLogSW - lp)) + (wave >> lp) : (int)blockIdx.x * SW + wave;
  const int rounds = P > 1 ? (total - ((int)blockIdx.x << (kLogSW - lp)) + step - 1) / step : 1;
  for (int round = 0; round < rounds; ++round) {
    bool todo = item < total;
    const int first = item;
    f32x4 v[SB] = {};
    fragdot::run<kWtMx, SB, 0, kStreamBM, 2>(
        PHASE == 1 ? f.x : f.h, (uint32_t)(PHASE == 1 ? f.T : f.T * f.k) * (uint32_t)K * 2u, K, lane, act,
        [&](const auto& j, int r) {
          if (PHASE != 1) return j.base + r;
          return self_plan ? (int)tokens[j.base + r] : f.sb_tok[j.base + r];
        },
        [&](auto& j) {
          if (!todo) return false;
          int sb, slab, g;
          slabs.divide(item, sb, slab);
          if (self_plan) {
            g = uniform(glist[sb] & 1023);
            j.base = uniform(f.offsets[g] + (glist[sb] >> 10) * kStreamBM);
            j.rows = uniform(f.offsets[g + 1]) - j.base;
          } else {
            g = uniform(f.sb_group[sb]);
            j.base = PHASE == 1 ? sb * kStreamBM : uniform(f.sb_base[sb]) + uniform(f.sb_row0[sb]);
            j.rows = uniform(f.sb_nrows[sb]);
          }
          j.rows = j.rows < kStreamBM ? j.rows : kStreamBM;
          j.ar = m < j.rows ? m : 0;
          const int c0 = slab * COLS;
#pragma unroll
          for (int i = 0; i < 2 * SB; ++i) {  // half blocks of 8 rows
            const bool up = i >= SB;
            const void* w = PHASE != 1 ? f.wd : up ? f.wu : f.wg;
            const int64_t stride = PHASE != 1 ? f.sd : up ? f.su : f.sg;
            const int r0 = c0 + 8 * (PHASE == 1 ? i % SB : i), left = N - r0;
            j.w[i] = static_cast<const char*>(w) + ((int64_t)g * stride + (int64_t)(left > 0 ? r0 : 0) * K) / 2;
            j.wrows[i] = left < 8 ? (left > 0 ? left : 0) : 8;
          }
#pragma unroll
          for (int b = 0; b < SB; ++b) {  // of row lane / 4
            const int r = 16 * b + (lane >> 2);
            const bool up = r >= 8 * SB;
            const float* sc = PHASE != 1 ? f.scd : up ? f.scu : f.scg;
            const int n = c0 + (PHASE == 1 && up ? r - 8 * SB : r);
            j.scale[b] = reinterpret_cast<const uint8_t*>(sc) + ((int64_t)g * N + (n < N ? n : N - 1)) * (K / 32);
          }
          j.k0 = ((p * units) >> lp) * 128;
          const int ke = (((p + 1) * units) >> lp) * 128;
          j.kend = ke < K ? ke : K;
          j.tag = item;
          item += step;
          todo = P == 1 && item < total;
          return true;
        },
        [&](int at, const f32x4 (&acc)[SB]) {
          if (P == 1) {
            finish(at, acc);
          } else {
#pragma unroll
            for (int b = 0; b < SB; ++b) v[b] = acc[b];
          }
        },
        fragdot::NoGate{});
    if (P > 1) {
#pragma unroll
      for (int b = 0; b < SB; ++b) part[wave][b][lane] = v[b];  // added in K order
      __syncthreads();
      if (p == 0 && first < total) {
        for (int w = 1; w < P; ++w)
#pragma unroll
          for (int b = 0; b < SB; ++b) v[b] += part[wave + w][b][lane];
        finish(first, v);
      }
      __syncthreads();
      if (first >= total) item += step;  // (it had none this time)
    }
  }
}

template <int PHASE>
__global__ __launch_bounds__(SW * 64, 2) void mx_stream_kernel(FfnArgs f, int self_plan, Divisor wide,
                                                               Divisor narrow) {
  __shared__ __attribute__((aligned(16))) char act[SW][SF::LDS];
  __shared__ f32x4 part[SW][4][64];
  __shared__ int glist[kMaxExperts + kMxFewTokens * 64 / kStreamBM];  // self_plan: m-blocks, group | block << 10
  __shared__ uint8_t tokens[kMxFewTokens * 64];  // and the dispatched rows' tokens
  __shared__ int wtot[SW];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  int nblocks;
  if (self_plan) {
    if (PHASE == 1)
      for (int i = tid; i < f.T * f.k; i += SW * 64) {
        const int tok = f.sorted[i] / f.k;
        tokens[i] = (uint8_t)((unsigned)tok < (unsigned)f.T ? tok : f.T - 1);  // also clamps a negative index
      }
    nblocks = 0;
    for (int g0 = 0; g0 < f.E; g0 += SW * 64) {
      const int g = g0 + tid;
      const int n = g < f.E ? (f.offsets[g + 1] - f.offsets[g] + kStreamBM - 1) / kStreamBM : 0;
      int upto = n;  // inclusive scan over the wave
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(upto, o, 64);
        if (lane >= o) upto += u;
      }
      if (lane == 63) wtot[wave] = upto;
      __syncthreads();
      int off = nblocks + upto - n;
      for (int w = 0; w < SW; ++w) {
        if (w < wave) off += wtot[w];
        nblocks += wtot[w];
      }
      for (int i = 0; i < n; ++i) glist[off + i] = g | i << 10;
      __syncthreads();
    }
    nblocks = uniform(nblocks);
  } else {
    nblocks = uniform(f.plan[kPlanRoutedBlocks]);
  }
  // one block an item where items of 4 do not even give every workgroup one
  if (nblocks * wide.d >= (int)gridDim.x)
    mx_stream_items<PHASE, 4>(f, self_plan, nblocks, wide, glist, tokens, act[wave], part, lane, wave);
  else
    mx_stream_items<PHASE, 1>(f, self_plan, nblocks, narrow, glist, tokens, act[wave], part, lane, wave);
}

// ---- 128-row m-tiles ---------------------------------------------------------
// A workgroup of 4 waves computes up to 128 rows x 256 weight rows (gate/up: 128
// hidden columns); a wave 64 weight rows in four blocks of 16 (gate/up: 32
// columns, two gate and two up blocks) of all the tile's 16-row blocks that hold
// rows.  A step is 128 values of K: activations go to LDS by direct loads, one
// step ahead in the other of two buffers, chunk c (16 bytes) of row r at
// c ^ (r % 16) of its 256 bytes, so a fragment read's 16 rows lie in 16 bank
// groups.  Codes go to registers two steps at a time, whole 128-byte lines of 8
// rows a load, take their fragment order through 2 KB of LDS of the wave, and
// become bf16 in registers.  The scale bytes of 3 steps go to LDS by a direct load,
// 16 bytes of a row.
//   A skewed layer of 1023 tokens (8192 x 2048, 64 experts) took 1265 us with codes
// and scale bytes loaded in fragment order, a lane to a row, which kept the address
// unit busy; 1061 with 64-byte rows, which cross L2 in two halves; 1035 so.  Of
// those 690 remain without any load.
constexpr int TW = 4;          // waves
constexpr int TK = 128;        // K per step
constexpr int TN = 256;        // weight rows per tile
constexpr int TBUF = kGemmBM * TK * 2;
constexpr int kScaleSteps = 3;  // steps whose scale bytes lie in LDS: 12 bytes and up to 3 before them
constexpr uint32_t kOut = 0xFFFFFFF0u;  // an offset past any buffer: reads as zeros

struct MxTile {  // a tile's rows and columns
  int g, base, r0, nrows, nt;
  bool once;  // the group's only m-tile: its codes are read once
};

// Fragments of step kt from one buffer times the step's codes, while `fetch`
// asks for the next step's.
template <int NBLK, class Fetch>
__device__ __forceinline__ void mx_step(f32x4 (&acc)[NBLK][4], const char* buf, const u32x4 (&w)[4],
                                        const float (&sc)[4], const uint32_t (&aswz)[4], Fetch fetch) {
  constexpr int NF = 4 * NBLK;  // activation fragments of the step, in order of use
  constexpr int kAhead = NBLK < 8 ? 3 : 2;  // read so many ahead of their use (8 blocks: what the registers allow)
  auto decode = [&](int s, bf16x8 (&bf)[4]) {
#pragma unroll
    for (int b = 0; b < 4; ++b) bf[b] = fragdot::frag(mx8_to_bf16x8(w[b][s], sc[b]));
  };
  auto read = [&](int j) { return *reinterpret_cast<const bf16x8*>(buf + aswz[j / NBLK] + (j % NBLK) * 4096); };
  bf16x8 ring[kAhead + 1];
#pragma unroll
  for (int j = 0; j < kAhead && j < NF; ++j) ring[j] = read(j);
  fetch();
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    bf16x8 bf[4];
    decode(s, bf);
#pragma unroll
    for (int i = 0; i < NBLK; ++i) {
      const int j = s * NBLK + i;
      if (j + kAhead < NF) ring[(j + kAhead) % (kAhead + 1)] = read(j + kAhead);
#pragma unroll
      for (int b = 0; b < 4; ++b)
        acc[i][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ring[j % (kAhead + 1)], bf[b], acc[i][b], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < NBLK; ++i) {
      if (s * NBLK + i + kAhead < NF) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <int PHASE, int NBLK>
__device__ __forceinline__ void mx_tile(const FfnArgs& f, const MxTile& t, char* lds0, char* lds1, char* codes,
                                        char* scales, int lane, int wave) {
  const int K = PHASE == 1 ? f.H : f.I, N = PHASE == 1 ? f.I : f.H;
  asm volatile("" : "+v"(lane));  // (so that no address is computed ahead of the tile loop and held through it)
  int q = lane >> 4, m = lane & 15;
  const int groups = K >> 5, steps = (K + TK - 1) / TK;
  // activation rows: load i of wave w brings rows 16 i + 4 w .. + 4
  const __amdgpu_buffer_rsrc_t ares = fragdot::resource(
      PHASE == 1 ? f.x : f.h, (uint32_t)(PHASE == 1 ? f.T : f.T * f.k) * (uint32_t)K * 2u);
  const int rl = 4 * wave + q, ac = m ^ rl;  // row of a 16-row block, chunk of the step's 16
  uint32_t aoff[NBLK];
#pragma unroll
  for (int i = 0; i < NBLK; ++i) {
    int r = 16 * i + rl;
    r = r < t.nrows ? r : t.nrows - 1;  // rows past the group are computed, never stored
    int row = t.base + t.r0 + r;
    if (PHASE == 1) {
      row = f.sorted[row] / f.k;
      row = (unsigned)row < (unsigned)f.T ? row : f.T - 1;  // also clamps a negative index
    }
    aoff[i] = (uint32_t)row * (uint32_t)K * 2u + 16u * (uint32_t)ac;
  }
  // weight rows, each `groups` scale bytes and 16 times as many of codes in the
  // expert's (which are aligned); what lies past the matrix reads as zeros
  __amdgpu_buffer_rsrc_t wres[PHASE == 1 ? 2 : 1], sres[PHASE == 1 ? 2 : 1];
  const uint32_t n0 = PHASE == 1 ? t.nt * (TN / 2) + wave * 32 : t.nt * TN + wave * 64;
  const uint32_t block = 16u * (uint32_t)groups;  // scale bytes of a block's rows (a multiple of 4)
  // codes: row lane / 8, chunk lane % 8 of two steps; scales in LDS: of row m, chunk q
  const uint32_t wrow = (n0 + (lane >> 3)) * block + 16u * (lane & 7);
  const uint32_t soff = m * 16 + (((n0 + m) * (uint32_t)groups) & 3u) + q;
  // chunk c of row r lies at c ^ (r / 2 % 8): 16 rows of a chunk in 16 bank groups
  const int cput = (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 4)) << 4);
  const int cget = m * 128 + ((q ^ (m >> 1)) << 4);
  const uint32_t sbytes = (uint32_t)N * (uint32_t)groups;
#pragma unroll
  for (int j = 0; j < (PHASE == 1 ? 2 : 1); ++j) {
    const void* wm = PHASE != 1 ? f.wd : j ? f.wu : f.wg;
    const float* sm = PHASE != 1 ? f.scd : j ? f.scu : f.scg;
    const int64_t stride = PHASE != 1 ? f.sd : j ? f.su : f.sg;
    wres[j] = fragdot::resource(static_cast<const char*>(wm) + (int64_t)t.g * stride / 2, sbytes * 16u);
    sres[j] = fragdot::resource(reinterpret_cast<const char*>(sm) + (int64_t)t.g * sbytes, sbytes);
  }
  uint32_t aswz[4];  // this lane's fragment of instruction s
#pragma unroll
  for (int s = 0; s < 4; ++s) aswz[s] = m * 256 + (((4 * q + s) ^ m) << 4);

  f32x4 acc[NBLK][4];
#pragma unroll
  for (int i = 0; i < NBLK; ++i)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[i][b] = f32x4{0.f, 0.f, 0.f, 0.f};

  u32x4 wa[4], wb[4];  // codes of the next two steps: rows 0-7 and 8-15 of each block, then (wb) of the odd step
  auto load_scales = [&](int kt) {  // of steps kt .. + 2: 64 rows, 16 bytes a lane from an aligned place on
    const uint32_t r = n0 + (PHASE == 1 ? lane & 31 : lane);
    const uint32_t at = ((r * (uint32_t)groups) & ~3u) + kt * 4;
    auto* const to = (__attribute__((address_space(3))) void*)scales;
    if (PHASE == 1) {  // half the lanes from each matrix
      if (lane < 32) __builtin_amdgcn_raw_ptr_buffer_load_lds(sres[0], to, 16, at, 0, 0, 0);
      else __builtin_amdgcn_raw_ptr_buffer_load_lds(sres[PHASE == 1 ? 1 : 0], to, 16, at, 0, 0, 0);
    } else {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(sres[0], to, 16, at, 0, 0, 0);
    }
  };
  auto load_codes = [&](int kt) {  // of steps kt and kt + 1: 128 bytes of 8 rows a load
    const uint32_t k = (uint32_t)kt * TK;
    const bool in = (int)k + (lane & 7) * 32 < K;
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t at = in ? wrow + ((PHASE == 1 ? b & 1 : b) * 16 + 8 * j) * block + k / 2 : kOut;
        const __amdgpu_buffer_rsrc_t r = wres[PHASE == 1 ? b >> 1 : 0];
        (j ? wb : wa)[b] =
            __builtin_bit_cast(u32x4, t.once ? __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, fragdot::kNt)
                                             : __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
      }
  };
  auto load = [&](int kt, char* buf) {
    const uint32_t k = (uint32_t)kt * TK;
    const bool in = (int)k + ac * 8 < K;
#pragma unroll
    for (int i = 0; i < NBLK; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          ares, (__attribute__((address_space(3))) void*)(buf + i * 4096 + wave * 1024), 16,
          in ? aoff[i] + 2u * k : kOut, 0, 0, 0);
  };
  int sk = 0;  // the step's place among those whose scales lie in LDS
  auto step = [&](int kt, const char* here, char* there, auto odd) {
    __builtin_amdgcn_s_waitcnt(0xF70);  // vmcnt(0): this wave's loads of the step have arrived
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();  // every wave's have, and every wave is done with the other buffer
    asm volatile("" ::: "memory");
    u32x4 w[4];
    float sc[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      // (LDS operations of one wave are executed in order)
      if (odd) {
        w[b] = wb[b];
      } else {
        *reinterpret_cast<u32x4*>(codes + cput) = wa[b];
        *reinterpret_cast<u32x4*>(codes + 1024 + (cput ^ 64)) = wb[b];
        w[b] = *reinterpret_cast<const u32x4*>(codes + cget);
        wb[b] = *reinterpret_cast<const u32x4*>(codes + (cget ^ 64));
      }
      const uint32_t s = *reinterpret_cast<const uint8_t*>(scales + soff + b * 256 + 4 * sk);
      sc[b] = e8m0(kt * TK + q * 32 < K ? s : 0u);  // (what lies behind a row's scales is not one of them)
    }
    mx_step<NBLK>(acc, here, w, sc, aswz, [&] {
      if (++sk == kScaleSteps && kt + 1 < steps) {
        sk = 0;
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this step's scales have been read
        asm volatile("" ::: "memory");
        load_scales(kt + 1);
      }
      if (kt + 1 < steps) load(kt + 1, there);
      if (odd && kt + 1 < steps) load_codes(kt + 1);
    });
  };
  load_scales(0);
  load_codes(0);
  load(0, lds0);
#pragma unroll 1
  for (int kt = 0; kt < steps; kt += 2) {
    step(kt, lds0, lds1, std::false_type{});
    if (kt + 1 < steps) step(kt + 1, lds1, lds0, std::true_type{});
  }
  asm volatile("" : "+v"(lane));
  q = lane >> 4, m = lane & 15;
  // Through LDS to whole 16-byte row chunks, 64 rows at a time in each buffer:
  // chunk c of row r at c ^ 2 ((r / 4) % 4), so that the four lane groups' rows lie in
  // different banks.
  __syncthreads();
  constexpr int CC = PHASE == 1 ? TN / 2 : TN;  // output columns
  constexpr int RB = TBUF / (2 * CC);           // rows per buffer
#pragma unroll
  for (int b = 0; b < (PHASE == 1 ? 2 : 4); ++b) {
    const int chunk = (wave * (CC / 32) + 2 * b + (m >> 3)) ^ (2 * q);
    const uint32_t at = (uint32_t)(4 * q * CC + chunk * 8 + (m & 7)) * 2u;
#pragma unroll
    for (int i = 0; i < NBLK; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float o = PHASE == 1 ? silu(acc[i][b][v]) * acc[i][(b + 2) & 3][v] : acc[i][b][v];
        char* const p = 16 * i < RB ? lds0 : lds1;
        *reinterpret_cast<bf16*>(p + at + (16 * i % RB + v) * CC * 2) = f2bf(o);
      }
  }
  __syncthreads();
  constexpr int RP = TW * 64 / (CC / 8);  // rows per pass
  const int tid = wave * 64 + lane, c = tid % (CC / 8), col = t.nt * CC + c * 8;
  bf16* out = reinterpret_cast<bf16*>(PHASE == 1 ? f.h : f.y) + (int64_t)(t.base + t.r0) * N + col;
#pragma unroll 2
  for (int r = tid / (CC / 8); r < t.nrows; r += RP) {
    const char* p = (r < RB ? lds0 : lds1) + (r % RB * CC + ((c ^ (((r >> 2) & 3) << 1)) << 3)) * 2;
    if (col < N) st16_nt(out + (int64_t)r * N, ld16(p));
  }
  __syncthreads();  // LDS is read out before the next tile fills it
}

template <int PHASE>
__global__ __launch_bounds__(TW * 64, 2) void mx_tiles_kernel(FfnArgs f, Divisor ntn, int32_t* counters) {
  __shared__ __attribute__((aligned(1024))) char lds0[TBUF];
  __shared__ __attribute__((aligned(1024))) char lds1[TBUF];  // (apart: a read of one waits for no load to the other)
  __shared__ __attribute__((aligned(16))) char wcodes[TW][2048];  // per wave: a block's codes of two steps
  __shared__ __attribute__((aligned(16))) char wscales[TW][64 * 16];  // and its 64 rows' scale bytes
  __shared__ int claim;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int mts = uniform(f.plan[kPlanRoutedTiles]);
  // Each XCD (workgroup i runs on XCD i % 8) has every eighth m-tile with all its
  // n-tiles, n fastest, so that an m-tile's activations are read into one L2; its
  // workgroups claim them one by one, then help the XCD that has most left.  (Sets of
  // 4 consecutive m-tiles to an XCD, for a large group's codes, measured the same.)
  auto tiles_of = [&](int x) { return ((mts - x + 7) >> 3) * ntn.d; };
  bool own = true;
  for (;;) {
    if (wave == 0) {
      int at = -1;
      if (own) {
        const int x = blockIdx.x & 7;
        int c = 0;
        if (lane == 0 && tiles_of(x) > 0) c = atomicAdd(&counters[x], 1);
        c = uniform(c);
        if (c < tiles_of(x)) at = c * 8 + x;
        else own = false;
      }
      while (at < 0) {
        int left = lane < 8 ? tiles_of(lane) - __hip_atomic_load(&counters[lane], __ATOMIC_RELAXED,
                                                                 __HIP_MEMORY_SCOPE_AGENT) : 0;
        int most = left, x = lane;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
          const int ol = __shfl_xor(most, o, 64), ox = __shfl_xor(x, o, 64);
          if (ol > most || (ol == most && ox < x)) most = ol, x = ox;
        }
        most = uniform(most);
        x = uniform(x);
        if (most <= 0) break;
        int c = 0;
        if (lane == 0) c = atomicAdd(&counters[x], 1);
        c = uniform(c);
        if (c < tiles_of(x)) at = c * 8 + x;
      }
      if (lane == 0) claim = at;
    }
    __syncthreads();
    const int at = uniform(claim);
    __syncthreads();
    if (at < 0) break;
    int mt;
    MxTile t;
    ntn.divide(at >> 3, mt, t.nt);
    mt = mt * 8 + (at & 7);
    t.g = uniform(f.mt_group[mt]);
    t.r0 = uniform(f.mt_row0[mt]);
    t.base = uniform(f.offsets[t.g]);
    t.nrows = uniform(f.offsets[t.g + 1]) - t.base - t.r0;
    t.once = t.r0 == 0 && t.nrows <= kGemmBM;
    t.nrows = t.nrows < kGemmBM ? t.nrows : kGemmBM;
    switch ((t.nrows + 15) >> 4) {
      case 1: mx_tile<PHASE, 1>(f, t, lds0, lds1, wcodes[wave], wscales[wave], lane, wave); break;
      case 2: mx_tile<PHASE, 2>(f, t, lds0, lds1, wcodes[wave], wscales[wave], lane, wave); break;
      case 3: mx_tile<PHASE, 3>(f, t, lds0, lds1, wcodes[wave], wscales[wave], lane, wave); break;
      case 4: mx_tile<PHASE, 4>(f, t, lds0, lds1, wcodes[wave], wscales[wave], lane, wave); break;
      case 5: mx_tile<PHASE, 5>(f, t, lds0, lds1, wcodes[wave], wscales[wave], lane, wave); break;
      case 6: mx_tile<PHASE, 6>(f, t, lds0, lds1, wcodes[wave], wscales[wave], lane, wave); break;
      case 7: mx_tile<PHASE, 7>(f, t, lds0, lds1, wcodes[wave], wscales[wave], lane, wave); break;
      default: mx_tile<PHASE, 8>(f, t, lds0, lds1, wcodes[wave], wscales[wave], lane, wave); break;
    }
  }
}

}  // namespace

hipError_t launch_mx_stream(const FfnArgs& a, int phase, hipStream_t s, bool self_plan) {
  const int grid = cu_count(), sp = self_plan ? 1 : 0;
  if (phase == 1)
    mx_stream_kernel<1><<<grid, SW * 64, 0, s>>>(a, sp, Divisor((a.I + 31) / 32), Divisor((a.I + 7) / 8));
  else
    mx_stream_kernel<2><<<grid, SW * 64, 0, s>>>(a, sp, Divisor((a.H + 63) / 64), Divisor((a.H + 15) / 16));
  return hipGetLastError();
}

hipError_t launch_mx_tiles(const FfnArgs& a, int phase, hipStream_t s) {
  const int grid = cu_count() * 2;
  int32_t* counters = const_cast<int32_t*>(a.plan) + kPlanCounters + (phase - 1) * 8;
  if (phase == 1) mx_tiles_kernel<1><<<grid, TW * 64, 0, s>>>(a, Divisor((a.I + TN / 2 - 1) / (TN / 2)), counters);
  else mx_tiles_kernel<2><<<grid, TW * 64, 0, s>>>(a, Divisor((a.H + TN - 1) / TN), counters);
  return hipGetLastError();
}

}  // namespace moe
