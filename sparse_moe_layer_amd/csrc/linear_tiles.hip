// Products over groups of rows on matrix-instruction tiles (bf16: v_mfma_f32_32x32x16_bf16,
// fp32: v_mfma_f32_32x32x2_f32, four of them with K 8 j + e and 8 j + 4 + e a sub-step, so
// that a lane's operands are one 16-byte chunk of a row along K):
//   forward  z = x W_g^T     A = x  [r][k],  B = W [n][k]     (contracted along rows of both)
//   dx       dz W_g          A = dz [r][n],  B = W [n][k]     (B contracted along its columns)
//   dw       dz^T x          A = dz [r][n],  B = x [r][k]     (both contracted along their columns)
// Stages of both operands arrive in LDS by direct loads, S - 1 of them ahead; fragments are
// read a sub-step ahead of the matrix instructions, whose last sub-step is carried past the
// barrier.  Bound by the matrix rate at the clock that the power limit leaves (8192 x 8192 x
// 2048 bf16: 208 to 233 us, 1.2 to 1.3 PFLOP/s, the library's product 200 to 205; fp32
// 4096 x 4096 x 4096 918 us, 0.150 PFLOP/s, the library 0.154 at 8192) or, for groups of few
// rows, by reading or writing each weight once (512 groups of 80 rows of 2560 x 640, 1.94 GB:
// forward 338 us, dx 420, dw 500).
#include "dma.hpp"
#include "linear.hpp"

#include <type_traits>

namespace moe {
namespace {

// F32_: fp32 tensors.  KB: bytes of a row's K step in a stage.  WK: waves that share
// a step's sub-steps (each has a sum of the whole tile) instead of the tile.
template <bool F32_, int BM_, int BN_, int WM_, int WN_, int S_, int KB_, int WG_PER_CU_, bool W_ONCE_ = false,
          int WK_ = 1>
struct Tile {
  static constexpr int WK = WK_;
  static constexpr bool F32 = F32_;
  using T = typename std::conditional<F32, float, bf16>::type;
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_, KB = KB_;
  static constexpr int BK = KB / (int)sizeof(T);                   // K step
  static constexpr int CE = 16 / (int)sizeof(T);                   // values of a 16-byte chunk
  static constexpr int KS = KB / 32 / WK;                          // a wave's sub-steps, of two chunks a row
  static constexpr int PER_SUB = F32 ? 4 : 1;                      // matrix instructions of a block and sub-step
  static constexpr bool W_ONCE = W_ONCE_;                          // each weight is read by one tile
  static constexpr int NW = WM * WN * WK, NT = 64 * NW;
  static constexpr int MI = BM / (32 * WM), NJ = BN / (32 * WN);   // 32 x 32 blocks of a wave
  static constexpr int LA = BM * KB / 1024 / NW, LB = BN * KB / 1024 / NW;  // 1 KB direct loads a wave and stage
  static constexpr int L = LA + LB;
  static constexpr int STAGE = (BM + BN) * KB;                     // bytes
  static constexpr int WG_PER_CU = WG_PER_CU_;
  static_assert(NT == 256, "the search for tiles takes 256 threads");
  static_assert((WM == 2 || WM == 1) && BM == BN && (KB == 64 || KB == 128), "tiling");
  static_assert(WK == 1 || (WM * WN == 1 && MI * NJ == 1 && KS == 1), "K over the waves: one block");
  static_assert(MI >= 1 && NJ >= 1 && LA >= 1 && LB >= 1 && L * (S - 1) < 64, "tiling");
  static_assert(S * STAGE * WG_PER_CU <= 160 * 1024, "LDS");
};

// Where 16-byte chunk c of an operand's row lies within the row of a stage: c ^ swz.
//  Rows along K (KB bytes): 16 rows' fragment reads of one chunk cover all banks.
template <int KB>
__device__ __forceinline__ int swz(int r) { return KB == 64 ? (r >> 2) & 3 : (r >> 1) & 7; }
//  Rows across K (R values): bf16, the transposing reads of four rows k .. k + 3 take 64
//  bytes each; fp32, a wave reads 128 bytes of rows k and k + 4.  (A row of 32 values
//  has no other place for them.)
template <bool F32, int R>
__device__ __forceinline__ int swz_t(int k) {
  return R == 32 ? 0 : F32 ? (k & 4) << 1 : R == 64 ? (k & 2) << 1 : (k & 3) << 2;
}

// One operand's tile of R rows (or, contracted along its columns, R columns) as
// the direct loads see it.  T: contracted along its columns; a stage then holds
// [BK][R] values, else [R][BK].
template <class C, int R, bool T>
struct Operand {
  static constexpr int LOADS = R * C::KB / 1024 / C::NW;
  const char* base;    // the tile's first element
  int64_t bytes;       // from there to the tensor's (the contraction's) end
  int64_t ld;          // bytes from row to row
  uint32_t off[LOADS];
  int chunk[2];        // !T: the lane's first k within a stage, of even and odd pieces

  __device__ __forceinline__ Operand(const typename C::T* p, int64_t ld_, int64_t left, int lane, int wave)
      : base(reinterpret_cast<const char*>(p)), bytes(left * (int)sizeof(*p)), ld(ld_ * (int)sizeof(*p)) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int q = C::NW * i + wave;  // the 1 KB piece of the stage
      constexpr int LPR = T ? R / C::CE : C::KB / 16;  // lanes a row
      const int row = q * (64 / LPR) + lane / LPR;
      const int c = (lane % LPR) ^ (T ? swz_t<C::F32, R>(row) : swz<C::KB>(row));
      if constexpr (!T) chunk[i & 1] = c * C::CE;  // the swizzle repeats after 16 rows, at most two pieces of NW
      off[i] = (uint32_t)(row * ld) + c * 16;
    }
  }

  // The loads of the BK contraction steps from k0 on; steps past kn give zeros.
  __device__ __forceinline__ void issue(char* st, int k0, int kn, int wave, bool once = false) const {
    const char* b = base;
    int64_t left = bytes;
    if constexpr (T) {
      b += k0 * ld;
      left -= k0 * ld;
    }
    const uint32_t records = left <= 0 ? 0u : left < (int64_t)kNowhere ? (uint32_t)left : kNowhere;
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      dma16(b, records, !T && k0 + chunk[i & 1] >= kn ? kNowhere : off[i], T ? 0 : k0 * (16 / C::CE),
            st + (C::NW * i + wave) * 1024, once);
  }
};

// Within each 16 lanes, lane i gives the address of values 4 (i & 3) .. + 4 of row
// i >> 2 and gets value i of the four rows.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ s16x4 read_tr(const char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
}

// A lane's fragments of one operand: block b (of 32 rows or columns), sub-step ks;
// row lane % 32, chunk 2 ks + lane / 32 of the stage's K.  first: the wave's first
// block; STEP: blocks apart.
template <class C, int R, bool T, int NB, int STEP>
struct Frags {
  using F = typename std::conditional<C::F32, f32x4, bf16x8>::type;
  int o[T ? NB : C::KS];
  // ks0: the wave's first sub-step
  __device__ __forceinline__ Frags(int first, int ks0, int lane) {
    if constexpr (!T) {
#pragma unroll
      for (int ks = 0; ks < C::KS; ++ks) {
        const int row = first * 32 + (lane & 31);
        o[ks] = row * C::KB + ((((ks0 + ks) * 2 + (lane >> 5)) ^ swz<C::KB>(row)) << 4);
      }
    } else if constexpr (C::F32) {
      const int k = 8 * ks0 + 4 * (lane >> 5);  // the swizzle is that of k & 7
#pragma unroll
      for (int i = 0; i < NB; ++i)
        o[i] = k * R * 4 + ((((first + i * STEP) * 8 + ((lane & 31) >> 2)) ^ swz_t<true, R>(k)) << 4) + 4 * (lane & 3);
    } else {
      const int k = 16 * ks0 + 8 * (lane >> 5) + ((lane & 15) >> 2);  // and k + 4, of the same swizzle
#pragma unroll
      for (int i = 0; i < NB; ++i)
        o[i] = k * R * 2 + ((((first + i * STEP) * 4 + ((lane & 31) >> 4) * 2 + ((lane & 3) >> 1)) ^ swz_t<false, R>(k)) << 4) +
               8 * (lane & 1);
    }
  }
  __device__ __forceinline__ void load(const char* st, int ks, F* f) const {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      if constexpr (!T) {
        f[i] = *reinterpret_cast<const F*>(st + o[ks] + i * STEP * 32 * C::KB);
      } else if constexpr (C::F32) {
        const char* p = st + o[i] + ks * 8 * R * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) f[i][e] = *reinterpret_cast<const float*>(p + e * R * 4);
      } else {
        const char* p = st + o[i] + ks * 16 * R * 2;
        f[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(read_tr(p), read_tr(p + 4 * R * 2), 0, 1, 2, 3, 4, 5, 6, 7));
      }
    }
  }
};

// Columns by rows, so that a lane has four columns of a row side by side.
template <class C, class F>
__device__ __forceinline__ void mfma_sub(f32x16 (&acc)[C::MI][C::NJ], const F* a, const F* b) {
#pragma unroll
  for (int e = 0; e < C::PER_SUB; ++e)
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
      for (int j = 0; j < C::NJ; ++j) {
        if constexpr (C::F32) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(b[j][e], a[i][e], acc[i][j], 0, 0, 0);
        else acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[j], a[i], acc[i][j], 0, 0, 0);
      }
}

// The order of a stage's instructions, from matrix instruction I on: each comes
// after its share of the next sub-step's NR fragment reads and of the direct
// loads, which go out one by one (issued together they hold up the wave for as
// long as the address unit takes for all of them).
template <class C, int NR, int I>
__device__ __forceinline__ void spread() {
  constexpr int NM = C::MI * C::NJ * C::PER_SUB, ALL = C::KS * NM / 2;
  if constexpr (I < C::KS * NM) {
    if constexpr (I % NM < NR) __builtin_amdgcn_sched_group_barrier(0x100, (NR + NM - 1) / NM, 0);
    if constexpr (I < ALL && (I + 1) * C::L / ALL > I * C::L / ALL)
      __builtin_amdgcn_sched_group_barrier(0x010, (I + 1) * C::L / ALL - I * C::L / ALL, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    spread<C, NR, I + 1>();
  }
}

// A thread's places in the epilogue: one 16-byte chunk of IT rows of each block of 32, so that
// a wave's accesses are whole lines (fp32 with two chunks a thread: dw of 379 groups of 464 x
// 180 84 us; 42).  And what the forward epilogue reads there beside the products: bias,
// factors and residual.  Places past the tile's rows or columns give values that nothing uses.
template <class C>
struct Epilogue {
  static constexpr int W = C::CE, CPR = C::BN / W, IT = (32 * CPR + C::NT - 1) / C::NT;  // threads a row
  struct Block {
    u32x4 mul[IT], resid[IT];
  };
  using T = typename C::T;
  const T *mul, *resid;
  u32x4 bias;
  int row0, last, nn, col;
  __device__ __forceinline__ Epilogue(const LinearArgs& a, int g, int m0, int m1, int n0, int tid)
      : mul(static_cast<const T*>(a.mul)), resid(static_cast<const T*>(a.resid)), row0(m0 + tid / CPR), last(m1 - 1),
        nn(a.N), col(min(n0 + tid % CPR * W, a.N - W)) {  // the same column in every row: CPR divides the threads
    if (a.bias) bias = ld16(static_cast<const T*>(a.bias) + (int64_t)g * nn + col);
  }
  __device__ __forceinline__ void load(Block& b, int block) const {
    if (mul) get(mul, b.mul, block);
    if (resid) get(resid, b.resid, block);
  }
  __device__ __forceinline__ void get(const T* p, u32x4 (&v)[IT], int block) const {
#pragma unroll
    for (int it = 0; it < IT; ++it)
      v[it] = ld16(p + (int64_t)min(row0 + block * 32 + it * (C::NT / CPR), last) * nn + col);
  }
};

// One tile, the bid-th: stg the stages.
template <int MODE, class C>
__device__ __forceinline__ void run_tile(const LinearArgs& a, const typename C::T* p, const typename C::T* q,
                                         typename C::T* out, int super, int bid, char* const (&stg)[4]) {
  using T = typename C::T;
  constexpr bool TA = MODE == kLinDw, TB = MODE != kLinForward;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = C::WK > 1 ? wave : 0, wm = C::WK > 1 ? 0 : wave / C::WN, wn = C::WK > 1 ? 0 : wave % C::WN;

  // ---- which tile: XCD x (workgroup i runs on XCD i % 8) takes a run of
  // consecutive tiles, so that its L2 holds what they share ----
  const int nn = MODE == kLinForward ? a.N : a.K;  // columns of the output
  const int tn = (nn + C::BN - 1) / C::BN;
  const TileMap map(MODE == kLinDw ? nullptr : a.offsets, a.G, a.rows, C::BM);
  const int tm = MODE == kLinDw ? a.G * ((a.N + C::BM - 1) / C::BM) : map.total;
  const int total = tm * tn;
  if (bid >= total) return;
  const int x = bid & 7, per = total >> 3, rem = total & 7;
  const int t = x * per + min(x, rem) + (bid >> 3);
  // runs of `super` m-tiles by all n-tiles, m first
  const int sb = t / (super * tn) * super, in = t - sb * tn;
  const int deep = min(tm - sb, super);
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
  const T *pa, *pb;
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
  const Operand<C, C::BM, TA> oa(pa, la, ba, lane, wave);
  const Operand<C, C::BN, TB> ob(pb, lb, bb, lane, wave);
  const Frags<C, C::BM, TA, C::MI, C::WM> fa(wm, wk * C::KS, lane);  // M-blocks wm, wm + WM, ..
  const Frags<C, C::BN, TB, C::NJ, 1> fb(wn * C::NJ, wk * C::KS, lane);
  const int nk = (kn + C::BK - 1) / C::BK;
  auto issue = [&](char* st, int step) {
    oa.issue(st, step * C::BK, kn, wave);
    ob.issue(st + C::BM * C::KB, step * C::BK, kn, wave, C::W_ONCE);
  };

  // The epilogue's reads go out a block ahead of their use, small tiles' first block ahead
  // of everything (8192 x 8192 x 2048 with bias and residual 244 -> 227 us, 512 groups of 80
  // rows of 640 x 2560 520 -> 474).
  using EX = Epilogue<C>;
  constexpr bool EARLY = C::BM <= 64;
  typename EX::Block extra[2];
  LinearArgs ea = a;
  if constexpr (MODE != kLinForward) ea.bias = ea.mul = ea.resid = nullptr;
  const EX ex(ea, g, m0, m1, n0, tid);
  if constexpr (EARLY) ex.load(extra[0], 0);

  f32x16 acc[C::MI][C::NJ];
#pragma unroll
  for (int i = 0; i < C::MI; ++i)
#pragma unroll
    for (int j = 0; j < C::NJ; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  using F = typename std::conditional<C::F32, f32x4, bf16x8>::type;
  F ca[C::MI] = {}, cb[C::NJ] = {};  // the stage's second sub-step, multiplied after the next barrier

#pragma unroll
  for (int s = 0; s < C::S - 1; ++s) issue(stg[s], s);
  auto step = [&](int s, const char* st, char* next) {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm((C::S - 2) * C::L));
    block_sync();
    __builtin_amdgcn_sched_barrier(0);
    issue(next, s + C::S - 1);
    F af[C::KS][C::MI], bf[C::KS][C::NJ];
#pragma unroll
    for (int ks = 0; ks < C::KS; ++ks) {
      fa.load(st, ks, af[ks]);
      fb.load(st + C::BM * C::KB, ks, bf[ks]);
      if (ks == 0) mfma_sub<C>(acc, ca, cb);
      else mfma_sub<C>(acc, af[ks - 1], bf[ks - 1]);
    }
#pragma unroll
    for (int i = 0; i < C::MI; ++i) ca[i] = af[C::KS - 1][i];
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) cb[j] = bf[C::KS - 1][j];
    constexpr int TR = C::F32 ? 4 : 2, NR = (TA ? TR : 1) * C::MI + (TB ? TR : 1) * C::NJ;
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

  // ---- epilogue: blocks of 32 rows go through LDS (bf16 gradients as bf16, the rest as
  // fp32, so that z is rounded once), so that a thread has 16 bytes of a row side by side.  A lane
  // holds row lane % 32 of a block and columns 8 q + 4 (lane / 32) .. + 4; 16-byte chunk c
  // of row r sits at c ^ (r & 15) (& 7 in a row of 8), so 16 rows' writes cover the banks. ----
  constexpr bool WIDE = MODE == kLinForward || C::F32 || C::WK > 1;
  constexpr int ROW = C::BN * (WIDE ? 4 : 2), PER = C::STAGE / (32 * ROW);  // bytes of a row, blocks a stage holds
  constexpr int BPP = C::BM / 32 < C::S * PER ? C::BM / 32 : C::S * PER;    // blocks of a pass
  static_assert(C::BM / 32 % BPP == 0 && BPP % C::WM == 0 && C::WK <= 2 * PER, "whole passes");
  constexpr int SWZ = ROW >= 256 ? 15 : 7;
  auto block = [&](int b) { return stg[b / PER] + b % PER * 32 * ROW; };
  if constexpr (!EARLY) ex.load(extra[0], 0);
#pragma unroll
  for (int pass = 0; pass < C::BM / 32 / BPP; ++pass) {
    if (pass) lds_sync();
#pragma unroll
    for (int i = 0; i < BPP / C::WM; ++i) {
      const int ii = pass * (BPP / C::WM) + i, r = lane & 31;
      char* f = (C::WK > 1 ? (wk < PER ? stg[0] : stg[1]) + wk % PER * 32 * ROW : wm ? block(i * C::WM + C::WM - 1) : block(i * C::WM)) + r * ROW;
#pragma unroll
      for (int j = 0; j < C::NJ; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const f32x16& d = acc[ii][j];
          const int u = (wn * C::NJ + j) * 8 + 2 * v + (lane >> 5);  // four columns
          if constexpr (WIDE) {
            *reinterpret_cast<f32x4*>(f + ((u ^ (r & SWZ)) << 4)) =
                f32x4{d[4 * v], d[4 * v + 1], d[4 * v + 2], d[4 * v + 3]};
          } else {
            *reinterpret_cast<bf16x4*>(f + (((u >> 1) ^ (r & SWZ)) << 4) + ((u & 1) << 3)) =
                bf16x4{f2bf(d[4 * v]), f2bf(d[4 * v + 1]), f2bf(d[4 * v + 2]), f2bf(d[4 * v + 3])};
          }
        }
    }
    lds_sync();
#pragma unroll
    for (int b = 0; b < BPP; ++b) {
      const char* f = block(b);
      const int bb = pass * BPP + b;
      if (bb + 1 < C::BM / 32) ex.load(extra[(bb + 1) & 1], bb + 1);
#pragma unroll
      for (int it = 0; it < EX::IT; ++it) {
        const int e = it * C::NT + tid, r = e / EX::CPR, c = e % EX::CPR * EX::W;
        const int row = m0 + bb * 32 + r, col = n0 + c;
        if (e >= 32 * EX::CPR || row >= m1 || col >= nn) continue;
        const char* fr = f + r * ROW;
        T* o = out + (MODE == kLinDw ? g * a.w_stride : 0) + (int64_t)row * nn + col;
        u32x4 v;
        if constexpr (!WIDE) {
          v = ld16(fr + (((c >> 3) ^ (r & SWZ)) << 4));
        } else {
          using V = Vec<C::F32>;
          float z[EX::W];
#pragma unroll
          for (int k = 0; k < EX::W; k += 4) {
            const int at = (((c + k) >> 2) ^ (r & SWZ)) << 4;
            f32x4 q = *reinterpret_cast<const f32x4*>(fr + at);
#pragma unroll
            for (int w = 1; w < C::WK; ++w) q += *reinterpret_cast<const f32x4*>(block(w) + r * ROW + at);
#pragma unroll
            for (int l = 0; l < 4; ++l) z[k + l] = q[l];
          }
          if constexpr (MODE == kLinForward) {
            float x[EX::W];
            if (a.bias) {
              V::unpack(ex.bias, x);
#pragma unroll
              for (int k = 0; k < EX::W; ++k) z[k] += x[k];
            }
            if (a.z) st16(static_cast<T*>(a.z) + (int64_t)row * nn + col, V::pack(z));
            activate<!C::F32>(a.act, z);
            if (a.mul) {
              V::unpack(extra[bb & 1].mul[it], x);
#pragma unroll
              for (int k = 0; k < EX::W; ++k) z[k] *= x[k];
            }
            if (a.resid) {
              V::unpack(extra[bb & 1].resid[it], x);
#pragma unroll
              for (int k = 0; k < EX::W; ++k) z[k] += x[k];
            }
          }
          v = V::pack(z);
        }
        if constexpr (MODE == kLinDw) st16_nt(o, v);
        else st16(o, v);
      }
    }
  }
}

// A launch's work: sums of the dbias partials (workgroups [0, sums)), then the tiles
// of one product, then those of another.
struct Job {
  LinearArgs a;
  const void *p, *q[2];
  void* out[2];
  int super[2];
  int first, second;  // first workgroups of the two products
  LinearSums sums;
};

// M1, M2: the products' modes (M2 < 0: one product), C1, C2 their tiles.
template <int M1, int M2, class C1, class C2 = C1>
__global__ __launch_bounds__(C1::NT, C1::NW * (C1::WG_PER_CU < C2::WG_PER_CU ? C1::WG_PER_CU : C2::WG_PER_CU) / 4)
void linear_tiles_kernel(Job j) {
  using T = typename C1::T;
  constexpr int STAGE = C1::STAGE > C2::STAGE ? C1::STAGE : C2::STAGE, S = C1::S > C2::S ? C1::S : C2::S;
  // separate arrays: a read of one stage does not wait for loads into another
  __shared__ __attribute__((aligned(1024))) char s0[STAGE];
  __shared__ __attribute__((aligned(1024))) char s1[STAGE];
  __shared__ __attribute__((aligned(1024))) char s2[S > 2 ? STAGE : 16];
  __shared__ __attribute__((aligned(1024))) char s3[S > 3 ? STAGE : 16];
  char* stg[4];
  stg[0] = s0, stg[1] = s1, stg[2] = s2, stg[3] = s3;
  const int bid = blockIdx.x;
  if constexpr (M1 != kLinForward) {
    if (bid < j.first) {
      add_partials(j.sums, bid);
      return;
    }
  }
  const T* p = static_cast<const T*>(j.p);
  if (M2 < 0 || bid < j.second)
    run_tile<M1, C1>(j.a, p, static_cast<const T*>(j.q[0]), static_cast<T*>(j.out[0]), j.super[0], bid - j.first, stg);
  else if constexpr (M2 >= 0)
    run_tile<M2, C2>(j.a, p, static_cast<const T*>(j.q[1]), static_cast<T*>(j.out[1]), j.super[1], bid - j.second, stg);
}

template <bool F32>
struct Tiles {
  using Big = Tile<F32, 256, 256, 2, 2, 2, 128, 1>;
  using Mid = Tile<F32, 128, 128, 2, 2, 2, 128, 2>;
  using MidOnce = Tile<F32, 128, 128, 2, 2, 2, 128, 2, true>;
  using Deep = Tile<F32, 128, 128, 2, 2, 4, 128, 1>;
  using Short = Tile<F32, 128, 128, 2, 2, 2, 64, 4>;
  using Short3 = Tile<F32, 128, 128, 2, 2, 3, 64, 3>;
  using Small = Tile<F32, 64, 64, 2, 2, 4, 128, 2>;
  using SmallOnce = Tile<F32, 64, 64, 2, 2, 4, 128, 2, true>;
  using Tiny = Tile<F32, 32, 32, 1, 1, 4, 128, 4, false, 4>;
};
enum Choice { kBig, kMid, kMidOnce, kDeep, kShort, kShort3, kSmall, kSmallOnce, kTiny };

// Rows of a group on average, and the tiles of edge b that a product takes about.
int64_t group_mean(const LinearArgs& a) { return a.rows / a.G; }
int64_t tiles_about(LinearMode mode, const LinearArgs& a, int b) {
  const int64_t touched = a.rows < a.G ? a.rows : a.G, deep = (group_mean(a) + b - 1) / b;
  const int64_t m = mode == kLinDw ? (int64_t)a.G * ((a.N + b - 1) / b) : touched * (deep > 1 ? deep : 1);
  return m * (((mode == kLinForward ? a.N : a.K) + b - 1) / b);
}

Choice choose(LinearMode mode, const LinearArgs& a, bool f32) {
  const int64_t r = group_mean(a), touched = a.rows < a.G ? a.rows : a.G;
  const int64_t t128 = tiles_about(mode, a, 128);
  if (f32) {
    // The matrix rate bounds every size of tile, so the least work of the busiest compute
    // unit decides, the smaller tiles' overhead counted in (forward, us, tiles of 32, 64 and
    // 128 rows: 300 x 1024 x 1024 11.9, 19.2, 63; 2000 x 2048 x 1024 76.9, 69.6, 123;
    // 8000 x 512 x 1024 84.9, 71.5, 69.0; the library's product 20.5, 64.2, 66.6.  256 rows
    // give nothing: 4096 x 4096 x 4096 923, 128 rows 918).
    struct Size {
      int b;
      double cost;
      Choice c;
    };
    const Size sizes[] = {{32, 1.2, kTiny}, {64, 1.05, kSmall}, {128, 1.0, kMid}};
    // But dw of short groups is mostly stores, of the longest rows in 128-row tiles (17 groups of
    // three rows of 968 x 2400: 47.7; 64 rows 59.0, 30 groups of 33 rows of 512 x 1024: 25.8; 30.4),
    // or of a few tiles that run beside dx (16 x 2048 x 2048 with dx: 16.9; 22.8).
    const bool stores = mode == kLinDw && r <= 64;
    if (stores && t128 > 256) return kMid;
    Choice best = kTiny;
    double least = 1e30;
    for (const Size& z : sizes) {
      if (stores && z.c == kMid) continue;
      const double work = (double)((tiles_about(mode, a, z.b) + 255) / 256) * z.b * z.b * z.cost;
      if (work < least) least = work, best = z.c;
    }
    return best;
  }
  // us, forward unless named, of one side and the other:
  // 256-row tiles, one a compute unit at a time, where they take fewer rounds than the four times
  // as many 128-row ones, two at a time: in one round if those need two (2304 x 4096 x 4096: 78; 97,
  // but 2048 x 4096 x 4096: 87; 70), in more if the last round leaves at most a quarter of them out
  // (6656 x 4096 x 4096: 188; 210, 8192 x 4096 x 2560: 177; 159); not for groups of less than a tile
  // nor dw of contractions too short for their pipeline (512 groups of 80 rows: 514; 363);
  const int64_t t256 = tiles_about(mode, a, 256), rounds = (t256 + 255) / 256;
  if (r >= (mode == kLinDw ? 1024 : 192) && (rounds == 1 ? t128 > 512 : 4 * t256 >= 3 * 256 * rounds)) return kBig;
  // 32-row tiles with K over the waves where even 64-row ones are few (100 x 8192 x 512: 11.9; 19.7)
  // or, as long as caches may hold the weights, groups are of at most 16 rows (16 x 4096 x 6400:
  // 11.9; 13.5, 30 groups of 2560 x 640: 20.1; 23.7, but ten of 640 x 2560: 10.3; 9.5);
  // 64-row tiles where 128-row ones would leave most of the chip idle (256 x 4096 x 4096: 21.6; 25.7),
  // or groups of a few rows, whose weights they stream in more and smaller pieces (512 groups of 4:
  // 278; 291.  dx, whose rows of W they read in 128-byte pieces, only as long as there are few:
  // 38 groups of a row 24.8; 28.3, 139 groups 100; 87), weights that no cache holds anyway
  // non-temporally (365 groups of a row or two 185; 202, 38 groups 25.1; 21.7);
  if (tiles_about(mode, a, 64) <= 64) return kTiny;
  if (mode == kLinForward && r <= 64 && touched * a.N * a.K > 100000000) return kSmallOnce;
  if (mode == kLinForward && r <= 16 && a.K >= 1280) return kTiny;
  if (t128 < 96 || (mode == kLinForward && r <= 64) || (mode == kLinDx && r <= 64 && t128 <= 1024)) return kSmall;
  // a round of 128-row tiles with four stages (2000 x 2048 x 2048: 19.6; two workgroups of two stages 26.3);
  if (t128 <= 256) return kDeep;
  // dw of short groups, which is loads, a few steps and stores: four workgroups a compute
  // unit overlap them, for more than a step or two three of one more stage (512 groups of
  // 80 rows with their dz 502, of 39 rows 332; four workgroups 542 and 305; two 553 of 80);
  if (mode == kLinDw && r <= 256) return r <= 44 ? kShort : kShort3;
  // groups of one tile read their weights once (512 groups of 80 rows 393; 404), others share them.
  return mode != kLinDw && r <= 128 ? kMidOnce : kMid;
}

// Workgroups of a product and, an XCD's share of the tiles that run at a time being
// `super` m-tiles deep, as square as it goes, so that its L2 takes in the fewest rows of
// both operands (256 x 4096 x 4096 21.8 -> 14.3 us against rows of tiles), 4 at most
// (8192^3: 5 822-869, 4 784-824); groups do not share their weights, and dw of
// short groups is all stores, of whole rows (512 groups of 80 rows: 5 567, 1 542).
template <class C>
int64_t grid_of(LinearMode mode, const LinearArgs& a, int& super) {
  const int64_t tn = ((mode == kLinForward ? a.N : a.K) + C::BN - 1) / C::BN;
  const int64_t tm = mode == kLinDw ? (int64_t)a.G * ((a.N + C::BM - 1) / C::BM) : max_tiles(a.rows, a.G, C::BM);
  const int64_t at_once = tm * tn < 256 * C::WG_PER_CU ? tm * tn : 256 * C::WG_PER_CU;
  const int64_t of_group = mode == kLinDw ? (a.N + C::BM - 1) / C::BM : (group_mean(a) + C::BM - 1) / C::BM;
  super = 1;
  while (super < 4 && super < of_group && 8 * (super + 1) * (super + 1) <= at_once) ++super;
  if (mode == kLinDw && group_mean(a) <= 256 && a.G > 1) super = 1;
  return tm * tn;
}

template <int MODE, class C>
hipError_t launch_as(Job j, hipStream_t s) {
  const dim3 grid((uint32_t)(j.first + grid_of<C>((LinearMode)MODE, j.a, j.super[0])));
  linear_tiles_kernel<MODE, -1, C><<<grid, C::NT, 0, s>>>(j);
  return hipGetLastError();
}

template <class C>
hipError_t launch(LinearMode mode, const Job& j, hipStream_t s) {
  return mode == kLinForward ? launch_as<kLinForward, C>(j, s)
         : mode == kLinDx    ? launch_as<kLinDx, C>(j, s)
                             : launch_as<kLinDw, C>(j, s);
}

// dx and dw of a small product side by side, in tiles X and W, dx first or dw.
template <class X, class W>
hipError_t launch_both(bool x_first, Job j, hipStream_t s) {
  const int64_t x = grid_of<X>(kLinDx, j.a, j.super[!x_first]), w = grid_of<W>(kLinDw, j.a, j.super[x_first]);
  j.second = (int)((j.first + (x_first ? x : w) + 7) / 8 * 8);  // its first workgroup on XCD 0 too
  const dim3 grid((uint32_t)(j.second + (x_first ? w : x)));
  if (x_first) linear_tiles_kernel<kLinDx, kLinDw, X, W><<<grid, X::NT, 0, s>>>(j);
  else linear_tiles_kernel<kLinDw, kLinDx, W, X><<<grid, X::NT, 0, s>>>(j);
  return hipGetLastError();
}

template <bool F32>
hipError_t launch_one(LinearMode mode, const Job& j, hipStream_t s) {
  using X = Tiles<F32>;
  const Choice c = choose(mode, j.a, F32);
  if constexpr (!F32) {  // fp32 takes the others alone
    if (c == kMidOnce)
      return mode == kLinDx ? launch_as<kLinDx, typename X::MidOnce>(j, s) : launch_as<kLinForward, typename X::MidOnce>(j, s);
    if (c == kDeep) return launch<typename X::Deep>(mode, j, s);
    if (c == kShort) return launch_as<kLinDw, typename X::Short>(j, s);
    if (c == kShort3) return launch_as<kLinDw, typename X::Short3>(j, s);
    if (c == kSmallOnce) return launch_as<kLinForward, typename X::SmallOnce>(j, s);
    if (c == kBig) return launch<typename X::Big>(mode, j, s);
  }
  if (c == kMid) return launch<typename X::Mid>(mode, j, s);
  if (c == kSmall) return launch<typename X::Small>(mode, j, s);
  return launch<typename X::Tiny>(mode, j, s);
}

template <bool F32>
hipError_t launch_back(const LinearArgs& a, const void* dz, const void* w, const void* x, void* dx, void* dw,
                       const LinearSums& sums, hipStream_t s) {
  Job j{};
  j.a = a;
  j.p = dz;
  j.sums = sums;
  j.first = sums.n ? (sums.workgroups() + 7) / 8 * 8 : 0;  // the first tile on XCD 0
  // Small products side by side in one launch (1000 x 1416 x 2056 with its dz: 54.0 -> 34.5
  // us, 9 x 200 x 2480 12.1 -> 8.5), where only one would take 128-row tiles both with smaller
  // ones (8192 x 512 x 1024: 57.2 -> 48.0).  The results are those of each alone:
  // 64 and 128 rows take K in the same steps.
  if (dx && dw) {
    using X = Tiles<F32>;
    Choice cx = choose(kLinDx, a, F32), cw = choose(kLinDw, a, F32);
    if (cx != kDeep && cw == kDeep) cw = kSmall;
    if (cx == kDeep && cw != kDeep) cx = kSmall;
    const bool x_first = a.N >= group_mean(a);  // the longer contraction first
    j.q[0] = x_first ? w : x;
    j.q[1] = x_first ? x : w;
    j.out[0] = x_first ? dx : dw;
    j.out[1] = x_first ? dw : dx;
    if (cx == kTiny && cw == kTiny) return launch_both<typename X::Tiny, typename X::Tiny>(x_first, j, s);
    if (cx == kTiny && cw == kSmall) return launch_both<typename X::Tiny, typename X::Small>(x_first, j, s);
    if (cx == kSmall && cw == kTiny) return launch_both<typename X::Small, typename X::Tiny>(x_first, j, s);
    if (cx == kSmall && cw == kSmall) return launch_both<typename X::Small, typename X::Small>(x_first, j, s);
    if constexpr (!F32)
      if (cx == kDeep && cw == kDeep) return launch_both<typename X::Deep, typename X::Deep>(x_first, j, s);
  }
  hipError_t e = hipSuccess;
  if (dx) {
    j.q[0] = w;
    j.out[0] = dx;
    e = launch_one<F32>(kLinDx, j, s);
    j.first = 0;
  }
  if (dw && e == hipSuccess) {
    j.q[0] = x;
    j.out[0] = dw;
    e = launch_one<F32>(kLinDw, j, s);
  }
  return e;
}

}  // namespace

hipError_t launch_linear_tiles(const LinearArgs& a, bool f32, hipStream_t s) {
  Job j{};
  j.a = a;
  j.p = a.x;
  j.q[0] = a.w;
  j.out[0] = a.y;
  return f32 ? launch_one<true>(kLinForward, j, s) : launch_one<false>(kLinForward, j, s);
}

hipError_t launch_linear_back_tiles(const LinearArgs& a, bool f32, const void* dz, const void* w, const void* x,
                                    void* dx, void* dw, const LinearSums& sums, hipStream_t s) {
  return f32 ? launch_back<true>(a, dz, w, x, dx, dw, sums, s) : launch_back<false>(a, dz, w, x, dx, dw, sums, s);
}

}  // namespace moe
