// The forward product for groups of few rows (single tokens, decode batches):
//   z[r][n] = sum_k x[r][k] W_g[n][k]
// bound by reading W_g once.  A workgroup has 16 rows of W (columns of y) and up to
// 16 rows of x; its waves take every WAVES-th 128 bytes of K, so that all of them
// stream, and add their sums through LDS.  Both operands come by direct loads (8 rows
// x 128 bytes each: whole lines, where fragments loaded straight into registers take
// 16 half lines a load) into LDS that only the wave itself uses, kAhead pieces in flight.
// A row of 8192 x 2048 (34 MB): 7.9 us, 4.3 TB/s with the launch; ten groups of 2560 x 640
// (33 MB): 9.8 us, of which 2 the launch and 1 the search for the groups.
#include "dma.hpp"
#include "linear.hpp"

#include <type_traits>

namespace moe {
namespace {

constexpr int kAhead = 4;
constexpr int kPiece = 16 * 128;  // bytes of an operand's piece

template <bool F32, int WAVES>
__global__ __launch_bounds__(WAVES * 64, 2) void linear_few_kernel(LinearArgs a) {
  using T = typename std::conditional<F32, float, bf16>::type;
  constexpr int ESZ = sizeof(T), CE = 16 / ESZ, BK = 128 / ESZ;  // values of a chunk, of a row's piece
  // separate arrays: a read of one does not wait for loads into another
  __shared__ __attribute__((aligned(1024))) char r0[WAVES * 2 * kPiece];
  __shared__ __attribute__((aligned(1024))) char r1[WAVES * 2 * kPiece];
  __shared__ __attribute__((aligned(1024))) char r2[WAVES * 2 * kPiece];
  __shared__ __attribute__((aligned(1024))) char r3[WAVES * 2 * kPiece];
  static_assert(kAhead == 4, "four arrays");
  __shared__ float red[WAVES][16][17];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tn = (a.N + 15) / 16;
  const TileMap map(a.offsets, a.G, a.rows, 16);
  const int mt = blockIdx.x / tn, n0 = (blockIdx.x - mt * tn) * 16;
  if (mt >= map.total) return;
  const MTile t = map.find(mt);
  const int64_t K = a.K;
  const int rows = min(t.end - t.row, 16), cols = min(a.N - n0, 16);
  const T* w = static_cast<const T*>(a.w) + t.g * a.w_stride + n0 * K;
  const T* x = static_cast<const T*>(a.x) + t.row * K;
  const uint32_t wb = (uint32_t)(cols * K * ESZ), xb = (uint32_t)(rows * K * ESZ);  // K <= 2^17
  // load h of a piece: rows 8 h .. + 8, chunk c of row r at c ^ ((r >> 1) & 7)
  int kc[2];
  uint32_t at[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = 8 * h + (lane >> 3);
    kc[h] = ((lane & 7) ^ ((r >> 1) & 7)) * CE;
    at[h] = (uint32_t)(r * K + kc[h]) * ESZ;
  }
  auto load = [&](char* l, int p) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t off = p * BK + kc[h] < a.K ? at[h] + p * 128 : kNowhere;
      dma16(w, wb, off, 0, l + h * 1024, true);
      dma16(x, xb, off, 0, l + kPiece + h * 1024);
    }
  };
  // the epilogue's reads go out first (thread: row tid / 16, column tid % 16)
  const int er = (tid >> 4) & 15, ec = tid & 15;
  const int64_t at_y = (int64_t)(t.row + min(er, rows - 1)) * a.N + n0 + min(ec, cols - 1);
  T e_bias{}, e_mul{}, e_resid{};
  if (a.bias) e_bias = static_cast<const T*>(a.bias)[(int64_t)t.g * a.N + n0 + min(ec, cols - 1)];
  if (a.mul) e_mul = static_cast<const T*>(a.mul)[at_y];
  if (a.resid) e_resid = static_cast<const T*>(a.resid)[at_y];
  const int fr = lane & 15;
  const int o0 = fr * 128 + (((lane >> 4) ^ ((fr >> 1) & 7)) << 4), o1 = fr * 128 + (((4 + (lane >> 4)) ^ ((fr >> 1) & 7)) << 4);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  const int mine = wave * 2 * kPiece, pieces = (a.K + BK - 1) / BK;
  load(r0 + mine, wave);
  load(r1 + mine, wave + WAVES);
  load(r2 + mine, wave + 2 * WAVES);
  load(r3 + mine, wave + 3 * WAVES);
  auto step = [&](char* l, int next) {
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(4 * (kAhead - 1)));  // this piece's four loads have landed
    asm volatile("" ::: "memory");
    using F = typename std::conditional<F32, f32x4, bf16x8>::type;
    const F f0 = *reinterpret_cast<const F*>(l + o0), g0 = *reinterpret_cast<const F*>(l + kPiece + o0);
    const F f1 = *reinterpret_cast<const F*>(l + o1), g1 = *reinterpret_cast<const F*>(l + kPiece + o1);
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(63));  // and are read, before the next ones overwrite them
    asm volatile("" ::: "memory");
    load(l, next);
    if constexpr (F32) {  // K 16 j + 4 h + e over the four h of a wave, for e in 0 .. 3
#pragma unroll
      for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(f0[e], g0[e], acc, 0, 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(f1[e], g1[e], acc, 0, 0, 0);
    } else {
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f0, g0, acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f1, g1, acc, 0, 0, 0);
    }
  };
  for (int p = wave; p < pieces; p += kAhead * WAVES) {
    step(r0 + mine, p + kAhead * WAVES);
    step(r1 + mine, p + (kAhead + 1) * WAVES);
    step(r2 + mine, p + (kAhead + 2) * WAVES);
    step(r3 + mine, p + (kAhead + 3) * WAVES);
  }
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // the loads past the end have landed too
  // rows 4 (lane / 16) .. + 4 of W, row lane % 16 of x
#pragma unroll
  for (int v = 0; v < 4; ++v) red[wave][lane & 15][4 * (lane >> 4) + v] = acc[v];
  __syncthreads();
  if (tid >= 256 || er >= rows || ec >= cols) return;
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) z += red[i][er][ec];
  if (a.bias) z += (float)e_bias;
  if (a.z) static_cast<T*>(a.z)[at_y] = (T)z;
  float y[1] = {z};
  activate<!F32>(a.act, y);
  if (a.mul) y[0] *= (float)e_mul;
  if (a.resid) y[0] += (float)e_resid;
  static_cast<T*>(a.y)[at_y] = (T)y[0];
}

}  // namespace

hipError_t launch_linear_few(const LinearArgs& a, int waves, bool f32, hipStream_t s) {
  const dim3 grid((uint32_t)((int64_t)max_tiles(a.rows, a.G, 16) * ((a.N + 15) / 16)));
  if (waves == 4) {
    if (f32) linear_few_kernel<true, 4><<<grid, 256, 0, s>>>(a);
    else linear_few_kernel<false, 4><<<grid, 256, 0, s>>>(a);
  } else {
    if (f32) linear_few_kernel<true, 8><<<grid, 512, 0, s>>>(a);
    else linear_few_kernel<false, 8><<<grid, 512, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace moe
