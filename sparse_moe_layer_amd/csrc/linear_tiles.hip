// bf16 products over groups of rows on v_mfma_f32_32x32x16_bf16 tiles:
//   forward  z = x W_g^T     A = x  [r][k],  B = W [n][k]     (contracted along rows of both)
//   dx       dz W_g          A = dz [r][n],  B = W [n][k]     (B contracted along its columns)
//   dw       dz^T x          A = dz [r][n],  B = x [r][k]     (both contracted along their columns)
#include "linear.hpp"

namespace moe {
namespace {

template <int BM_, int BN_, int WM_, int WN_, int S_, int BK_, int WG_PER_CU_, bool W_ONCE_ = false>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_, BK = BK_;
  static constexpr bool W_ONCE = W_ONCE_;  // each weight is read by one tile
  static constexpr int KS = BK / 16;                              // matrix instructions deep
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int MI = BM / (32 * WM), NJ = BN / (32 * WN);  // 32 x 32 blocks of a wave
  static constexpr int LA = BM * BK / 512 / NW, LB = BN * BK / 512 / NW;  // 1 KB direct loads a wave and stage
  static constexpr int L = LA + LB;
  static constexpr int STAGE = (BM + BN) * BK;  // elements
  static constexpr int WG_PER_CU = WG_PER_CU_;
  static_assert(NT == 256, "the search for tiles takes 256 threads");
  static_assert(WM == 2 && BM == BN && (BK == 32 || BK == 64), "tiling");
  static_assert(MI >= 1 && NJ >= 1 && LA >= 1 && LB >= 1 && L * (S - 1) < 64, "tiling");
  static_assert(S * STAGE * 2 * WG_PER_CU <= 160 * 1024, "LDS");
};

constexpr int vmcnt_imm(int n) { return 0xF70 | (n & 15) | (((n >> 4) & 3) << 14); }
constexpr int vmcnt_lgkm0_imm(int n) { return vmcnt_imm(n) & ~0xF00; }

constexpr int kBufferFlags = 0x00020000;  // raw 32-bit buffer access
constexpr uint32_t kNowhere = 0xFFFFFFF0u;  // past every buffer: the load writes zeros to LDS

__device__ __forceinline__ void block_sync() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A 16-byte direct load from base + voff + soff to LDS (voff the lane's, soff the
// wave's); past `records` bytes it writes zeros.  once: non-temporal.
__device__ __forceinline__ void dma16(const char* base, uint32_t records, uint32_t voff, uint32_t soff, bf16* l,
                                      bool once) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, records, kBufferFlags);
  if (once) __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)l, 16, voff, soff, 0, 2);
  else __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)l, 16, voff, soff, 0, 0);
}

// One operand's tile of R rows (or, contracted along its columns, R columns) as
// the direct loads see it.  T: contracted along its columns.
//  !T: a stage holds [R][BK]; 16-byte chunk c of row r at c ^ ((r >> 2) & 3) for
//      64-byte rows, c ^ ((r >> 1) & 7) for 128-byte rows: 16 rows' fragment reads
//      of one chunk cover all banks.
//   T: a stage holds [BK][R], the 64-byte block b of contraction row k at
//      b ^ (k & 3), or b ^ ((k >> 1) & 1) for rows of two blocks: the transposing
//      reads of four rows cover all banks.
template <int BK>
__device__ __forceinline__ int swz(int r) { return BK == 32 ? (r >> 2) & 3 : (r >> 1) & 7; }

template <int R>
__device__ __forceinline__ int swz_t(int k) { return R == 64 ? (k >> 1) & 1 : k & 3; }

template <class C, int R, bool T>
struct Operand {
  static constexpr int LOADS = R * C::BK / 512 / C::NW;
  const char* base;    // the tile's first element
  int64_t bytes;       // from there to the tensor's (the contraction's) end
  int64_t ld;          // bytes from row to row
  uint32_t off[LOADS];
  int chunk[2];        // !T: the lane's first k within a stage, of even and odd pieces

  __device__ __forceinline__ Operand(const void* p, int64_t ld_elems, int64_t bytes_, int lane, int wave)
      : base(static_cast<const char*>(p)), bytes(bytes_), ld(ld_elems * 2) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int q = C::NW * i + wave;  // the 1 KB piece of the stage
      if constexpr (!T) {
        constexpr int LPR = C::BK / 8;  // lanes a row
        const int row = q * (64 / LPR) + lane / LPR;
        const int k = ((lane % LPR) ^ swz<C::BK>(row)) * 8;
        chunk[i & 1] = k;  // the swizzle repeats after 16 rows, which NW pieces make up
        off[i] = (uint32_t)(row * ld) + k * 2;
      } else {
        constexpr int LPR = R / 8;  // lanes a row
        const int row = q * (64 / LPR) + lane / LPR, pos = lane % LPR;
        off[i] = (uint32_t)(row * ld) + ((((pos >> 2) ^ swz_t<R>(row)) << 2) | (pos & 3)) * 16;
      }
    }
  }

  // The loads of the BK contraction steps from k0 on; steps past kn give zeros.
  __device__ __forceinline__ void issue(bf16* st, int k0, int kn, int wave, bool once = false) const {
    const char* b = base;
    int64_t left = bytes;
    if constexpr (T) {
      b += k0 * ld;
      left -= k0 * ld;
    }
    const uint32_t records = left <= 0 ? 0u : left < (int64_t)kNowhere ? (uint32_t)left : kNowhere;
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      dma16(b, records, !T && k0 + chunk[i & 1] >= kn ? kNowhere : off[i], T ? 0 : k0 * 2, st + (C::NW * i + wave) * 512, once);
  }
};

// Within each 16 lanes, lane i gives the address of values 4 (i & 3) .. + 4 of row
// i >> 2 and gets value i of the four rows.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ s16x4 read_tr(const bf16* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
}

// A lane's fragment reads of one operand: block b (of 32 rows or columns), K
// sub-step ks of 16.  first: the wave's first block; step: blocks apart.
template <int BK, int R, bool T, int NB, int STEP>
struct Frags {
  int o[T ? NB : BK / 16];
  __device__ __forceinline__ Frags(int first, int lane) {
    if constexpr (!T) {
#pragma unroll
      for (int ks = 0; ks < BK / 16; ++ks) {
        const int row = first * 32 + (lane & 31);
        o[ks] = row * BK + (((ks * 2 + (lane >> 5)) ^ swz<BK>(row)) << 3);
      }
    } else {
      const int k = 8 * (lane >> 5) + ((lane & 15) >> 2);
#pragma unroll
      for (int i = 0; i < NB; ++i)
        o[i] = k * R + (((first + i * STEP) ^ swz_t<R>(k)) << 5) + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    }
  }
  __device__ __forceinline__ void load(const bf16* st, int ks, bf16x8* f) const {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if constexpr (!T) {
        f[i] = *reinterpret_cast<const bf16x8*>(st + o[ks] + i * STEP * 32 * BK);
      } else {
        const bf16* p = st + o[i] + ks * 16 * R;
        f[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(read_tr(p), read_tr(p + 4 * R), 0, 1, 2, 3, 4, 5, 6, 7));
      }
    }
  }
};

template <class C>
__device__ __forceinline__ void mfma_sub(f32x16 (&acc)[C::MI][C::NJ], const bf16x8* a, const bf16x8* b) {
#pragma unroll
  for (int i = 0; i < C::MI; ++i)
#pragma unroll
    for (int j = 0; j < C::NJ; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[j], a[i], acc[i][j], 0, 0, 0);  // columns by rows
}

// The order of a stage's instructions, from matrix instruction I on: each comes
// after its share of the next sub-step's NR fragment reads and of the direct
// loads, which go out one by one (issued together they hold up the wave for as
// long as the address unit takes for all of them).
template <class C, int NR, int I>
__device__ __forceinline__ void spread() {
  constexpr int NM = C::MI * C::NJ, ALL = C::KS * NM / 2;
  if constexpr (I < C::KS * NM) {
    if constexpr (I % NM < NR) __builtin_amdgcn_sched_group_barrier(0x100, (NR + NM - 1) / NM, 0);
    if constexpr (I < ALL && (I + 1) * C::L / ALL > I * C::L / ALL)
      __builtin_amdgcn_sched_group_barrier(0x010, (I + 1) * C::L / ALL - I * C::L / ALL, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    spread<C, NR, I + 1>();
  }
}

template <int MODE, class C>
__global__ __launch_bounds__(C::NT, C::NW * C::WG_PER_CU / 4) void linear_tiles_kernel(LinearArgs a, const bf16* p,
                                                                                       const bf16* q, bf16* out) {
  constexpr bool TA = MODE == kLinDw, TB = MODE != kLinForward;
  // separate arrays: a read of one stage does not wait for loads into another
  __shared__ __attribute__((aligned(1024))) bf16 s0[C::STAGE];
  __shared__ __attribute__((aligned(1024))) bf16 s1[C::STAGE];
  __shared__ __attribute__((aligned(1024))) bf16 s2[C::S > 2 ? C::STAGE : 8];
  __shared__ __attribute__((aligned(1024))) bf16 s3[C::S > 3 ? C::STAGE : 8];
  bf16* stg[4];
  stg[0] = s0, stg[1] = s1, stg[2] = s2, stg[3] = s3;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;

  // ---- which tile: XCD x (workgroup i runs on XCD i % 8) takes a run of
  // consecutive tiles, so that its L2 holds what they share ----
  const int nn = MODE == kLinForward ? a.N : a.K;  // columns of the output
  const int tn = (nn + C::BN - 1) / C::BN;
  const TileMap map(MODE == kLinDw ? nullptr : a.offsets, a.G, a.rows, C::BM);
  const int tm = MODE == kLinDw ? a.G * ((a.N + C::BM - 1) / C::BM) : map.total;
  const int total = tm * tn;
  const int bid = blockIdx.x;
  if (bid >= total) return;
  const int x = bid & 7, per = total >> 3, rem = total & 7;
  const int t = x * per + min(x, rem) + (bid >> 3);
  // runs of kSuper m-tiles by all n-tiles, m first
  constexpr int kSuper = C::BM == 256 ? 4 : 1;
  const int sb = t / (kSuper * tn) * kSuper, in = t - sb * tn;
  const int deep = min(tm - sb, kSuper);
  const int mt = sb + in % deep, nt = in / deep;

  int g, m0, m1, kn;
  int64_t r0 = 0;  // first row of the contraction (dw)
  if constexpr (MODE == kLinDw) {
    const int tg = (a.N + C::BM - 1) / C::BM;
    g = mt / tg;
    m0 = (mt - g * tg) * C::BM;
    m1 = a.N;
    const int2 rr = group_rows(a.offsets, g, a.rows);
    r0 = rr.x;
    kn = rr.y - rr.x;
  } else {
    const MTile m = map.find(mt);
    g = m.g;
    m0 = m.row;
    m1 = m.end;
    kn = MODE == kLinForward ? a.K : a.N;
  }
  const int n0 = nt * C::BN;

  const int64_t K = a.K, N = a.N;
  const bf16 *pa, *pb;
  int64_t la, lb, ba, bb;  // row lengths, elements left
  if constexpr (MODE == kLinForward) {
    pa = p + m0 * K, la = K, ba = (m1 - m0) * K;
    pb = q + g * a.w_stride + n0 * K, lb = K, bb = (N - n0) * K;
  } else if constexpr (MODE == kLinDx) {
    pa = p + m0 * N, la = N, ba = (m1 - m0) * N;
    pb = q + g * a.w_stride + n0, lb = K, bb = N * K - n0;
  } else {
    pa = p + r0 * N + m0, la = N, ba = kn * N - m0;
    pb = q + r0 * K + n0, lb = K, bb = kn * K - n0;
  }
  const Operand<C, C::BM, TA> oa(pa, la, ba * 2, lane, wave);
  const Operand<C, C::BN, TB> ob(pb, lb, bb * 2, lane, wave);
  const Frags<C::BK, C::BM, TA, C::MI, C::WM> fa(wm, lane);  // M-blocks wm, wm + WM, ..
  const Frags<C::BK, C::BN, TB, C::NJ, 1> fb(wn * C::NJ, lane);
  const int nk = (kn + C::BK - 1) / C::BK;
  auto issue = [&](bf16* st, int step) {
    oa.issue(st, step * C::BK, kn, wave);
    ob.issue(st + C::BM * C::BK, step * C::BK, kn, wave, C::W_ONCE);
  };

  f32x16 acc[C::MI][C::NJ];
#pragma unroll
  for (int i = 0; i < C::MI; ++i)
#pragma unroll
    for (int j = 0; j < C::NJ; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  bf16x8 ca[C::MI] = {}, cb[C::NJ] = {};  // the stage's second sub-step, multiplied after the next barrier

#pragma unroll
  for (int s = 0; s < C::S - 1; ++s) issue(stg[s], s);
  auto step = [&](int s, const bf16* st, bf16* next) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm((C::S - 2) * C::L));
    block_sync();
    __builtin_amdgcn_sched_barrier(0);
    issue(next, s + C::S - 1);
    bf16x8 af[C::KS][C::MI], bf[C::KS][C::NJ];
#pragma unroll
    for (int ks = 0; ks < C::KS; ++ks) {
      fa.load(st, ks, af[ks]);
      fb.load(st + C::BM * C::BK, ks, bf[ks]);
      if (ks == 0) mfma_sub<C>(acc, ca, cb);
      else mfma_sub<C>(acc, af[ks - 1], bf[ks - 1]);
    }
#pragma unroll
    for (int i = 0; i < C::MI; ++i) ca[i] = af[C::KS - 1][i];
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) cb[j] = bf[C::KS - 1][j];
    constexpr int NR = (TA ? 2 : 1) * C::MI + (TB ? 2 : 1) * C::NJ;
    spread<C, NR, 0>();
  };
  int s = 0;
  for (; s + C::S <= nk; s += C::S) {
#pragma unroll
    for (int b = 0; b < C::S; ++b) step(s + b, stg[b], stg[(b + C::S - 1) % C::S]);
  }
#pragma unroll
  for (int b = 0; b < C::S - 1; ++b)
    if (s + b < nk) step(s + b, stg[b], stg[(b + C::S - 1) % C::S]);
  mfma_sub<C>(acc, ca, cb);
  __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(0));  // loads past the end have landed
  block_sync();

  // ---- epilogue: blocks of 32 rows go through LDS (forward: as fp32, so that z is
  // rounded once; the gradients as bf16), so that a thread has 8 values side by side.
  // A lane holds row lane % 32 of a block and columns 8 q + 4 (lane / 32) .. + 4; 16-byte
  // chunk c of row r sits at c ^ (r & 15) (& 7 in a row of 8), so 16 rows' writes cover
  // the banks. ----
  constexpr bool F = MODE == kLinForward;
  constexpr int ROW = C::BN * (F ? 4 : 2), PER = C::STAGE * 2 / (32 * ROW);  // bytes of a row, blocks a stage holds
  constexpr int BPP = C::BM / 32 < C::S * PER ? C::BM / 32 : C::S * PER;     // blocks of a pass
  static_assert(C::BM / 32 % BPP == 0 && BPP % C::WM == 0, "whole passes");
  constexpr int CPR = C::BN / 8;  // threads a row
  constexpr int SWZ = ROW >= 256 ? 15 : 7;
  auto block = [&](int b) { return reinterpret_cast<char*>(stg[b / PER]) + b % PER * 32 * ROW; };
#pragma unroll
  for (int pass = 0; pass < C::BM / 32 / BPP; ++pass) {
    if (pass) block_sync();
#pragma unroll
    for (int i = 0; i < BPP / C::WM; ++i) {
      const int ii = pass * (BPP / C::WM) + i, r = lane & 31;
      char* f = (wm ? block(i * C::WM + 1) : block(i * C::WM)) + r * ROW;
#pragma unroll
      for (int j = 0; j < C::NJ; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const f32x16& d = acc[ii][j];
          const int u = (wn * C::NJ + j) * 8 + 2 * v + (lane >> 5);  // four columns
          if constexpr (F) {
            *reinterpret_cast<f32x4*>(f + ((u ^ (r & SWZ)) << 4)) =
                f32x4{d[4 * v], d[4 * v + 1], d[4 * v + 2], d[4 * v + 3]};
          } else {
            *reinterpret_cast<bf16x4*>(f + (((u >> 1) ^ (r & SWZ)) << 4) + ((u & 1) << 3)) =
                bf16x4{f2bf(d[4 * v]), f2bf(d[4 * v + 1]), f2bf(d[4 * v + 2]), f2bf(d[4 * v + 3])};
          }
        }
    }
    block_sync();
#pragma unroll
    for (int b = 0; b < BPP; ++b) {
      const char* f = block(b);
      for (int e = tid; e < 32 * CPR; e += C::NT) {
        const int r = e / CPR, c = e % CPR * 8;
        const int row = m0 + (pass * BPP + b) * 32 + r, col = n0 + c;
        if (row >= m1 || col >= nn) continue;
        const char* fr = f + r * ROW;
        using V = Vec<false>;
        if constexpr (MODE == kLinDw) {
          st16_nt(out + g * a.w_stride + row * K + col, ld16(fr + (((c >> 3) ^ (r & SWZ)) << 4)));
        } else if constexpr (MODE == kLinDx) {
          st16(out + row * K + col, ld16(fr + (((c >> 3) ^ (r & SWZ)) << 4)));
        } else {
          const f32x4 v0 = *reinterpret_cast<const f32x4*>(fr + (((c >> 2) ^ (r & SWZ)) << 4));
          const f32x4 v1 = *reinterpret_cast<const f32x4*>(fr + ((((c >> 2) + 1) ^ (r & SWZ)) << 4));
          float z[8] = {v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
          const int64_t at = row * N + col;
          float o[8];
          if (a.bias) {
            V::unpack(ld16(static_cast<const bf16*>(a.bias) + g * N + col), o);
#pragma unroll
            for (int k = 0; k < 8; ++k) z[k] += o[k];
          }
          if (a.z) st16(static_cast<bf16*>(a.z) + at, V::pack(z));
          activate<true>(a.act, z);
          if (a.mul) {
            V::unpack(ld16(static_cast<const bf16*>(a.mul) + at), o);
#pragma unroll
            for (int k = 0; k < 8; ++k) z[k] *= o[k];
          }
          if (a.resid) {
            V::unpack(ld16(static_cast<const bf16*>(a.resid) + at), o);
#pragma unroll
            for (int k = 0; k < 8; ++k) z[k] += o[k];
          }
          st16(out + at, V::pack(z));
        }
      }
    }
  }
}

using Big = Tile<256, 256, 2, 2, 2, 64, 1>;
using Mid = Tile<128, 128, 2, 2, 2, 64, 2>;
using MidOnce = Tile<128, 128, 2, 2, 2, 64, 2, true>;
using Deep = Tile<128, 128, 2, 2, 4, 64, 1>;
using Short = Tile<128, 128, 2, 2, 2, 32, 4>;
using Small = Tile<64, 64, 2, 2, 4, 64, 2>;
using SmallOnce = Tile<64, 64, 2, 2, 4, 64, 2, true>;

template <class C>
hipError_t launch(LinearMode mode, const LinearArgs& a, const bf16* p, const bf16* q, bf16* out, hipStream_t s) {
  const int64_t tn = ((mode == kLinForward ? a.N : a.K) + C::BN - 1) / C::BN;
  const int64_t tm = mode == kLinDw ? (int64_t)a.G * ((a.N + C::BM - 1) / C::BM) : max_tiles(a.rows, a.G, C::BM);
  const dim3 grid((uint32_t)(tm * tn));
  if (mode == kLinForward) linear_tiles_kernel<kLinForward, C><<<grid, C::NT, 0, s>>>(a, p, q, out);
  else if (mode == kLinDx) linear_tiles_kernel<kLinDx, C><<<grid, C::NT, 0, s>>>(a, p, q, out);
  else linear_tiles_kernel<kLinDw, C><<<grid, C::NT, 0, s>>>(a, p, q, out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_tiles(LinearMode mode, const LinearArgs& a, const void* p, const void* q, void* out,
                               hipStream_t s) {
  const bf16 *pp = static_cast<const bf16*>(p), *qq = static_cast<const bf16*>(q);
  bf16* o = static_cast<bf16*>(out);
  const int64_t r = a.rows / a.G, touched = a.rows < a.G ? a.rows : a.G;
  const int64_t cols = mode == kLinForward ? a.N : a.K;
  auto tiles = [&](int b) {
    const int64_t m = mode == kLinDw ? (int64_t)a.G * ((a.N + b - 1) / b) : touched * ((r + b - 1) / b > 1 ? (r + b - 1) / b : 1);
    return m * ((cols + b - 1) / b);
  };
  // us, forward unless named, of one side and the other:
  // 256-row tiles once they fill three quarters of the chip (8192 x 2560 x 8192: 283; 128-row 391), dw
  // also with a contraction long enough for their pipeline (512 experts of 80 rows: 645, short 497);
  if (r >= (mode == kLinDw ? 1024 : 192) && tiles(256) >= 192) return launch<Big>(mode, a, pp, qq, o, s);
  // 64-row tiles where 128-row ones would leave most of the chip idle (256 x 4096 x 4096: 21.6; 25.7),
  // or groups of a few rows, whose weights they stream in more and smaller pieces (512 groups of 4:
  // 278; 291.  dx, whose rows of W they read in 128-byte pieces, only as long as there are few:
  // 38 groups of a row 24.8; 28.3, 139 groups 100; 87), weights that no cache holds anyway
  // non-temporally (365 groups of a row or two 185; 202, 38 groups 25.1; 21.7);
  if (mode == kLinForward && r <= 64 && touched * a.N * a.K > 100000000) return launch<SmallOnce>(mode, a, pp, qq, o, s);
  if (tiles(128) < 96 || (mode == kLinForward && r <= 64) || (mode == kLinDx && r <= 64 && tiles(128) <= 1024))
    return launch<Small>(mode, a, pp, qq, o, s);
  // a round of 128-row tiles with four stages (2000 x 2048 x 2048: 19.6; two workgroups of two stages 26.3);
  if (tiles(128) <= 256) return launch<Deep>(mode, a, pp, qq, o, s);
  // dw of short groups, which is loads, a few steps and stores: four workgroups a compute
  // unit overlap them (512 groups of 80 rows 497; two 554);
  if (mode == kLinDw && r <= 256) return launch<Short>(mode, a, pp, qq, o, s);
  // groups of one tile read their weights once (512 groups of 80 rows 393; 404), others share them.
  if (mode != kLinDw && r <= 128) return launch<MidOnce>(mode, a, pp, qq, o, s);
  return launch<Mid>(mode, a, pp, qq, o, s);
}

}  // namespace moe
