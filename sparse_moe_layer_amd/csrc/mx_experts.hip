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
// An item is 32 weight rows (gate/up: 16 gate rows and the 16 up rows of the same
// hidden columns; down: 32 output columns) and all rows of a group's m-block; a
// wave goes through its items in one stream of loads.  With fewer items than
// waves, P waves of a workgroup share an item's K range and add their blocks in
// LDS in K order.
constexpr int kLogSW = 3, SW = 1 << kLogSW;  // waves per workgroup, one workgroup per compute unit
using SF = fragdot::Form<kWtMx, kStreamBM>;

template <int PHASE>
__global__ __launch_bounds__(SW * 64, 2) void mx_stream_kernel(FfnArgs f, int self_plan, Divisor slabs) {
  __shared__ __attribute__((aligned(16))) char act[SW][SF::LDS];
  __shared__ f32x4 part[SW][2][64];
  __shared__ int glist[kMaxExperts];  // self_plan: the touched groups, ascending
  __shared__ int wtot[SW];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int K = PHASE == 1 ? f.H : f.I, N = PHASE == 1 ? f.I : f.H;
  int nblocks;
  if (self_plan) {
    nblocks = 0;
    for (int g0 = 0; g0 < f.E; g0 += SW * 64) {
      const int g = g0 + tid;
      const bool t = g < f.E && f.offsets[g + 1] > f.offsets[g];
      const uint64_t bal = __ballot(t);
      if (lane == 0) wtot[wave] = __popcll(bal);
      __syncthreads();
      int off = nblocks;
      for (int w = 0; w < SW; ++w) {
        if (w < wave) off += wtot[w];
        nblocks += wtot[w];
      }
      if (t) glist[off + __popcll(bal & ((1ull << lane) - 1ull))] = g;
      __syncthreads();
    }
    nblocks = uniform(nblocks);
  } else {
    nblocks = uniform(f.plan[kPlanRoutedBlocks]);
  }
  const int grid = (int)gridDim.x, waves = grid * SW;
  const int total = nblocks * slabs.d, units = (K + 127) >> 7;
  int lp = 0;  // P = 1 << lp
  while (1 << lp < SW && (total << (lp + 1)) <= waves + waves / 4 && 2 << lp <= units) ++lp;
  const int P = 1 << lp, p = wave & (P - 1);
  const int q = lane >> 4, m = lane & 15;

  auto finish = [&](int item, const f32x4& v0, const f32x4& v1) {  // lane: column m, rows 4 q + i
    int sb, slab;
    slabs.divide(item, sb, slab);
    int base, nrows;
    if (self_plan) {
      const int g = glist[sb];
      base = f.offsets[g];
      nrows = f.offsets[g + 1] - base;
    } else {
      base = f.sb_base[sb] + f.sb_row0[sb];
      nrows = f.sb_nrows[sb];
    }
    if (PHASE == 1) {
      const int col = slab * 16 + m;
      bf16* h = reinterpret_cast<bf16*>(f.h) + (int64_t)base * f.I + col;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * q + i < nrows && col < f.I) h[(int64_t)(4 * q + i) * f.I] = f2bf(silu(v0[i]) * v1[i]);
    } else {
      const int col = slab * 32 + m;
      bf16* y = reinterpret_cast<bf16*>(f.y) + (int64_t)base * f.H + col;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (4 * q + i < nrows && col < f.H) y[(int64_t)(4 * q + i) * f.H] = f2bf(v0[i]);
        if (4 * q + i < nrows && col + 16 < f.H) y[(int64_t)(4 * q + i) * f.H + 16] = f2bf(v1[i]);
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
    f32x4 v[2] = {};
    fragdot::run<kWtMx, 2, 0, kStreamBM>(
        PHASE == 1 ? f.x : f.h, (uint32_t)(PHASE == 1 ? f.T : f.T * f.k) * (uint32_t)K * 2u, K, lane, act[wave],
        [&](const auto& j, int r) {
          if (PHASE != 1) return j.base + r;
          int tok = self_plan ? f.sorted[j.base + r] / f.k : f.sb_tok[j.base + r];
          return (unsigned)tok < (unsigned)f.T ? tok : f.T - 1;  // also clamps a negative index
        },
        [&](auto& j) {
          if (!todo) return false;
          int sb, slab, g;
          slabs.divide(item, sb, slab);
          if (self_plan) {
            g = uniform(glist[sb]);
            j.base = uniform(f.offsets[g]);
            j.rows = uniform(f.offsets[g + 1]) - j.base;
          } else {
            g = uniform(f.sb_group[sb]);
            j.base = PHASE == 1 ? sb * kStreamBM : uniform(f.sb_base[sb]) + uniform(f.sb_row0[sb]);
            j.rows = uniform(f.sb_nrows[sb]);
          }
          j.rows = j.rows < kStreamBM ? j.rows : kStreamBM;
          j.ar = m < j.rows ? m : 0;
          const int c0 = slab * (PHASE == 1 ? 16 : 32);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const void* w = PHASE != 1 ? f.wd : b ? f.wu : f.wg;
            const float* sc = PHASE != 1 ? f.scd : b ? f.scu : f.scg;
            const int64_t stride = PHASE != 1 ? f.sd : b ? f.su : f.sg;
            const int r0 = PHASE == 1 ? c0 : c0 + 16 * b;
            const int left = N - r0 < 16 ? (N > r0 ? N - r0 : 0) : 16;
            j.w[2 * b] = static_cast<const char*>(w) + ((int64_t)g * stride + (int64_t)(left ? r0 : 0) * K) / 2;
            j.w[2 * b + 1] = j.w[2 * b] + 4 * (int64_t)K;
            j.wrows[2 * b] = left < 8 ? left : 8;
            j.wrows[2 * b + 1] = left < 8 ? 0 : left - 8;
            const int n = r0 + (lane >> 2);
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
        [&](int at, const f32x4 (&acc)[2]) {
          if (P == 1) {
            finish(at, acc[0], acc[1]);
          } else {
            v[0] = acc[0];
            v[1] = acc[1];
          }
        },
        fragdot::NoGate{});
    if (P > 1) {
      part[wave][0][lane] = v[0];  // added in K order
      part[wave][1][lane] = v[1];
      __syncthreads();
      if (p == 0 && first < total) {
        for (int w = 1; w < P; ++w) {
          v[0] += part[wave + w][0][lane];
          v[1] += part[wave + w][1][lane];
        }
        finish(first, v[0], v[1]);
      }
      __syncthreads();
      if (first >= total) item += step;  // (not taken in this round)
    }
  }
}

// ---- 128-row m-tiles ---------------------------------------------------------
// A workgroup of 4 waves computes up to 128 rows x 256 weight rows (gate/up: 128
// hidden columns); a wave 64 weight rows in four blocks of 16 (gate/up: 32
// columns, two gate and two up blocks) of all the tile's 16-row blocks that hold
// rows.  A step is 128 values of K: activations go to LDS by direct loads, one
// step ahead in the other of two buffers, chunk c (16 bytes) of row r at
// c ^ (r % 16) of its 256 bytes, so a fragment read's 16 rows lie in 16 bank
// groups.  Codes go to registers, also a step ahead, 64 bytes of 16 rows a load
// with four consecutive lanes to a row, take their fragment order through 1 KB of
// LDS of the wave, and become bf16 in registers (loaded in fragment order, a lane
// to a row, they cost the address unit a quarter of the kernel's time; a skewed
// layer of 1023 tokens took 1265 us with scale bytes loaded so as well, 857
// without the codes' loads, 980 without the scales').  The scale bytes of 7 steps
// go to LDS by direct loads, 32 bytes of a row.
constexpr int TW = 4;          // waves
constexpr int TK = 128;        // K per step
constexpr int TN = 256;        // weight rows per tile
constexpr int TBUF = kGemmBM * TK * 2;
constexpr int kAhead = 3;      // activation fragments read ahead of their use
constexpr int kScaleSteps = 7;  // steps whose scale bytes lie in LDS: 28 bytes and up to 3 before them
constexpr uint32_t kOut = 0xFFFFFFF0u;  // an offset past any buffer: reads as zeros

struct MxTile {  // a tile's rows and columns
  int g, base, r0, nrows, nt;
};

// Fragments of step kt from one buffer times the step's codes, while `fetch`
// asks for the next step's.
template <int NBLK, class Fetch>
__device__ __forceinline__ void mx_step(f32x4 (&acc)[NBLK][4], const char* buf, const u32x4 (&w)[4],
                                        const float (&sc)[4], const uint32_t (&aswz)[4], Fetch fetch) {
  constexpr int NF = 4 * NBLK;  // activation fragments of the step, in order of use
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
  // weight rows; columns past the matrix are computed, never stored
  __amdgpu_buffer_rsrc_t wres[PHASE == 1 ? 2 : 1], sres[PHASE == 1 ? 2 : 1];
  auto row_of = [&](int b, int r) {  // of block b: its first scale byte, in the expert's (which are aligned)
    const int n = (PHASE == 1 ? t.nt * (TN / 2) + wave * 32 + (b & 1) * 16 : t.nt * TN + wave * 64 + b * 16) + r;
    return (uint32_t)(n < N ? n : N - 1) * (uint32_t)groups;
  };
  uint32_t wrow[4], soff[4];  // codes: row lane / 4, chunk lane % 4 of a step; scales in LDS: of row m, chunk q
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    wrow[b] = row_of(b, lane >> 2) * 16u + 16u * (lane & 3);
    soff[b] = (b * 16 + m) * 32 + (row_of(b, m) & 3u) + q;
  }
  char* const cput = codes + (lane >> 2) * 64 + (((lane & 3) ^ (lane >> 4)) << 4);  // 16 rows of a chunk in 16 bank groups
  const char* const cget = codes + m * 64 + ((q ^ (m >> 2)) << 4);
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

  u32x4 wn[4];
  auto load_scales = [&](int kt) {  // of steps kt .. + 6: 32 rows a load, 16 bytes a lane from an aligned place on
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t at = (row_of(2 * j + (lane >> 5), (lane >> 1) & 15) & ~3u) + kt * 4 + 16 * (lane & 1);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(sres[PHASE == 1 ? j : 0],
                                               (__attribute__((address_space(3))) void*)(scales + j * 1024), 16, at, 0, 0,
                                               0);
    }
  };
  auto load = [&](int kt, char* buf) {
    const uint32_t k = (uint32_t)kt * TK;
    const bool win = (int)k + (lane & 3) * 32 < K, in = (int)k + ac * 8 < K;
#pragma unroll
    for (int b = 0; b < 4; ++b)
      wn[b] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wres[PHASE == 1 ? b >> 1 : 0],
                                                                              win ? wrow[b] + k / 2 : kOut, 0, 0));
#pragma unroll
    for (int i = 0; i < NBLK; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          ares, (__attribute__((address_space(3))) void*)(buf + i * 4096 + wave * 1024), 16,
          in ? aoff[i] + 2u * k : kOut, 0, 0, 0);
  };
  int sk = 0;  // the step's place among those whose scales lie in LDS
  auto step = [&](int kt, const char* here, char* there) {
    __builtin_amdgcn_s_waitcnt(0xF70);  // vmcnt(0): this wave's loads of the step have arrived
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();  // every wave's have, and every wave is done with the other buffer
    asm volatile("" ::: "memory");
    u32x4 w[4];
    float sc[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      // (LDS operations of one wave are executed in order)
      *reinterpret_cast<u32x4*>(cput) = wn[b];
      w[b] = *reinterpret_cast<const u32x4*>(cget);
      const uint32_t s = *reinterpret_cast<const uint8_t*>(scales + soff[b] + 4 * sk);
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
    });
  };
  load_scales(0);
  load(0, lds0);
#pragma unroll 1
  for (int kt = 0; kt < steps; kt += 2) {
    step(kt, lds0, lds1);
    if (kt + 1 < steps) step(kt + 1, lds1, lds0);
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
  __shared__ __attribute__((aligned(16))) char wcodes[TW][1024];  // per wave: a block's codes
  __shared__ __attribute__((aligned(16))) char wscales[TW][64 * 32];  // and its 64 rows' scale bytes
  __shared__ int claim;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int mts = uniform(f.plan[kPlanRoutedTiles]);
  // Each XCD (workgroup i runs on XCD i % 8) has every eighth m-tile with all its
  // n-tiles, n fastest, so that an m-tile's activations are read into one L2; its
  // workgroups claim them one by one, then help the XCD that has most left.
  auto tiles_of = [&](int x) { return (mts - x + 7) / 8 * ntn.d; };
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
  const int grid = cu_count();
  if (phase == 1) mx_stream_kernel<1><<<grid, SW * 64, 0, s>>>(a, self_plan ? 1 : 0, Divisor((a.I + 15) / 16));
  else mx_stream_kernel<2><<<grid, SW * 64, 0, s>>>(a, self_plan ? 1 : 0, Divisor((a.H + 31) / 32));
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
