// Token rows to expert order, and the gradients of that and of the combine:
//   permute            xs[pos[t,j]] = w[t,j] x[t]
//   permute_backward   dx[t] = sum_j w[t,j] dxs[pos[t,j]],   dw[t,j] = <x[t], dxs[pos[t,j]]>
//   combine_backward   dy[pos[t,j]] = w[t,j] dout[t],        dw[t,j] = <dout[t], y[pos[t,j]]>
//                      dy_sh[t] = g dout[t],  ds[t] = g (1 - g) <dout[t], y_sh[t]>,  g = sigmoid(s[t])
// HBM-bound.  All of them go by token: a token's own row is read once for its k
// assignments, and each assignment's row is read or written once.
// A position outside [0, T k) stands for an assignment without a row.
#include "kernels.hpp"
#include "vec.hpp"

namespace moe {
namespace {

// One thread per 16 bytes of x, its k stores one after the other: bound by the writes, whole
// lines of a row next to each other (4096 x 2560 x 10 bf16, 0.23 GB: 45 us, 5.1 TB/s; the
// copy of a large tensor reaches 4.9).  n = T * (chunks of a row).
template <bool F32, bool W>
__global__ __launch_bounds__(256) void permute_kernel(const char* __restrict__ x, const int32_t* __restrict__ pos,
                                                      const float* __restrict__ w, char* __restrict__ xs, int n,
                                                      Divisor chunks, int k, int R) {
  using V = Vec<F32>;
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  int t, c;
  chunks.divide(i, t, c);
  const u32x4 v = ld16(x + (int64_t)i * 16);
  const int32_t* pt = pos + (int64_t)t * k;
  float f[V::N];
  if constexpr (W) V::unpack(v, f);
  for (int j = 0; j < k; ++j) {
    const int p = pt[j];
    if ((unsigned)p >= (unsigned)R) continue;
    u32x4 o = v;
    if constexpr (W) {
      const float wj = w[(int64_t)t * k + j];
      float g[V::N];
#pragma unroll
      for (int e = 0; e < V::N; ++e) g[e] = wj * f[e];
      o = V::pack(g);
    }
    st16(xs + ((int64_t)p * chunks.d + c) * 16, o);
  }
}

// dx alone: one thread per 16 bytes of dx, KB rows' loads in flight and summed in order
// (4096 x 2560 x 10, 0.23 GB read and 0.02 written: 44 us, 5.3 TB/s).  A batch's places past k
// load row 0, so KB is the least of 4, 8 and 10 that takes k at once (k = 8: 34.0 us in a batch of
// 8, 36.6 in one of 10; k = 5 27.2 and 29.0), and 8 at a time for more.
template <bool F32, bool W, int KB>
__global__ __launch_bounds__(256) void unpermute_kernel(const char* __restrict__ dxs, const int32_t* __restrict__ pos,
                                                        const float* __restrict__ w, char* __restrict__ dx, int n,
                                                        Divisor chunks, int k, int R) {
  using V = Vec<F32>;
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  int t, c;
  chunks.divide(i, t, c);
  const int64_t a0 = (int64_t)t * k;
  float acc[V::N] = {};
  for (int j0 = 0; j0 < k; j0 += KB) {
    u32x4 v[KB];
    bool ok[KB];
    float wj[KB];
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const int j = j0 + b < k ? j0 + b : k - 1;
      const int p = pos[a0 + j];
      ok[b] = j0 + b < k && (unsigned)p < (unsigned)R;
      wj[b] = W ? w[a0 + j] : 1.f;
      v[b] = ld16_nt(dxs + ((int64_t)(ok[b] ? p : 0) * chunks.d + c) * 16);
    }
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      float f[V::N];
      V::unpack(v[b], f);
#pragma unroll
      for (int e = 0; e < V::N; ++e) acc[e] = ok[b] ? fmaf(wj[b], f[e], acc[e]) : acc[e];
    }
  }
  st16(dx + (int64_t)i * 16, V::pack(acc));
}

// 1 / (1 + e^-z) to fp32's precision (a scalar per token, on fp32 outputs)
__device__ __forceinline__ float sigmoid_f32(float z) { return 1.f / (1.f + expf(-z)); }

// The combine's gradient, a row per assignment and, with a shared expert, one more per
// token: out = w * dout[t], dot = <dout[t], in>.  A wave has ROWS rows (short ones several
// at a time).  A token's rows follow each other, so dout comes from the caches for all
// but the first; nothing is shared between waves (4096 x 2560 x 10: 80 us; a workgroup per
// token with its rows in registers 146; with the shared expert 100 us, 0.48 GB, half of it
// writes, at 4.8 TB/s).  Without dy only the products (x and dxs of
// permute's gradient).
struct RowArgs {
  const char *dout, *y;
  const int32_t* pos;
  const float* w;
  const char* y_sh;
  const float* sl;
  char* dy;
  float* dw;
  char* dy_sh;
  float* dsl;
  int nch, k, R;  // 16-byte chunks of a row
  int64_t n;      // rows in all
  int per;        // rows a token
  int first;      // k: the shared expert's rows alone
};

// U: 16-byte pieces of each row that a lane has in flight.
template <bool F32, int ROWS, int U>
__global__ __launch_bounds__(256) void rows_kernel(RowArgs a) {
  using V = Vec<F32>;
  const int lane = threadIdx.x & 63;
  const int64_t wg = blockIdx.y * (int64_t)gridDim.x + blockIdx.x;
  const int64_t i0 = (wg * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * ROWS;
  const int64_t row = (int64_t)a.nch * 16;
  const char *d[ROWS], *in[ROWS];
  char* out[ROWS];
  float w[ROWS], dot[4] = {};
  bool ok[ROWS], shared[ROWS];
  int64_t at[ROWS];
#pragma unroll
  for (int q = 0; q < ROWS; ++q) {
    const int64_t i = i0 + q < a.n ? i0 + q : a.n - 1;
    const int t = (int)(i / a.per), j = (int)(i - (int64_t)t * a.per) + a.first;
    shared[q] = j == a.k;
    at[q] = shared[q] ? t : (int64_t)t * a.k + j;
    int p = shared[q] ? t : a.pos[at[q]];
    ok[q] = shared[q] || (unsigned)p < (unsigned)a.R;
    if (!ok[q]) p = 0;
    w[q] = shared[q] ? sigmoid_f32(a.sl[t]) : a.w ? a.w[at[q]] : 1.f;
    d[q] = a.dout + t * row;
    in[q] = (shared[q] ? a.y_sh : a.y) + p * row;
    out[q] = (shared[q] ? a.dy_sh : a.dy) + p * row;
    ok[q] = ok[q] && i0 + q < a.n;
  }
  for (int c0 = lane; c0 < a.nch; c0 += 64 * U) {
    u32x4 vd[ROWS * U], vi[ROWS * U];
#pragma unroll
    for (int u = 0; u < ROWS * U; ++u) {
      const int q = u / U, c = c0 + 64 * (u % U) < a.nch ? c0 + 64 * (u % U) : c0;
      vd[u] = ld16(d[q] + (int64_t)c * 16);
      vi[u] = ld16_nt(in[q] + (int64_t)c * 16);
    }
#pragma unroll
    for (int u = 0; u < ROWS * U; ++u) {
      const int q = u / U, c = c0 + 64 * (u % U);
      if (!ok[q] || c >= a.nch) continue;
      float x[V::N], y[V::N];
      V::unpack(vd[u], x);
      V::unpack(vi[u], y);
#pragma unroll
      for (int e = 0; e < V::N; ++e) {
        dot[u & 3] = fmaf(x[e], y[e], dot[u & 3]);  // a row's are next to each other
        x[e] *= w[q];
      }
      if (a.dy) st16(out[q] + (int64_t)c * 16, V::pack(x));
    }
  }
  const float s = wave_sums<4>(dot, lane);
#pragma unroll
  for (int q = 0; q < ROWS; ++q) {
    float v = __shfl(s, q * (64 / ROWS), kWave);
#pragma unroll
    for (int u = 1; u < 4 / ROWS; ++u) v += __shfl(s, q * (64 / ROWS) + u * 16, kWave);
    if (lane || i0 + q >= a.n) continue;
    if (shared[q]) a.dsl[at[q]] = w[q] * sigmoid_f32(-a.sl[at[q]]) * v;
    else a.dw[at[q]] = ok[q] ? v : 0.f;
  }
}

hipError_t launch_rows(RowArgs a, int T, int per, bool f32, hipStream_t s) {
  a.n = (int64_t)T * per;
  a.per = per;
  const int rows = a.nch <= 64 ? 4 : a.nch <= 128 ? 2 : 1;  // a wave: rows of one piece a lane, of two
  const int64_t waves = (a.n + rows - 1) / rows;
  const dim3 grid = row_grid((waves + 3) / 4);
#define MOE_ROWS(ROWS, U)                                              \
  do {                                                                 \
    if (f32) rows_kernel<true, ROWS, U><<<grid, 256, 0, s>>>(a);       \
    else rows_kernel<false, ROWS, U><<<grid, 256, 0, s>>>(a);          \
  } while (0)
  // a row that takes little more than one round of 4 pieces a lane in one of 5 (1500 x 1280 x 4
  // fp32 15.2 -> 13.9 us, 4096 x 2560 x 10 102.9 -> 100.9; longer ones in one of 8: the same)
  // (6550 x 552 x 18, one row a wave: 84 us; two 64)
  if (rows == 4) MOE_ROWS(4, 1);
  else if (rows == 2) MOE_ROWS(2, 2);
  else if (a.nch > 256 && a.nch <= 320) MOE_ROWS(1, 5);
  else MOE_ROWS(1, 4);
#undef MOE_ROWS
  return hipGetLastError();
}

// permute's gradient with dw for at most KB assignments a token: the token's waves over
// the row's 16-byte chunks, a sum in a register for each assignment.
struct TokenArgs {
  const char* x;
  const char* dxs;
  const int32_t* pos;
  const float* w;  // null: 1
  char* dx;
  float* dw;
  int T, nch, k, R;  // nch: 16-byte chunks of a row
};

constexpr int kTokenThreads = 512;

template <bool F32, int KB>
__global__ __launch_bounds__(kTokenThreads, 2) void token_kernel(TokenArgs a) {
  using V = Vec<F32>;
  constexpr int P = KB <= 4 ? 4 : KB <= 8 ? 8 : KB <= 16 ? 16 : 32;
  __shared__ float red[kTokenThreads / 64][P];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
  const int nch = a.nch;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t a0 = (int64_t)t * a.k;
    const char* x = a.x + (int64_t)t * nch * 16;
    float acc[P] = {};
    int64_t row[KB];
    bool ok[KB];
    float wj[KB];
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const int j = b < a.k ? b : a.k - 1;
      const int p = a.pos[a0 + j];
      ok[b] = b < a.k && (unsigned)p < (unsigned)a.R;
      row[b] = (int64_t)(ok[b] ? p : 0) * nch * 16;
      wj[b] = a.w ? a.w[a0 + j] : 1.f;
    }
    for (int c = tid; c < nch; c += blockDim.x) {
      u32x4 v[KB];
      const u32x4 vx = ld16(x + (int64_t)c * 16);
#pragma unroll
      for (int b = 0; b < KB; ++b) v[b] = ld16_nt(a.dxs + row[b] + (int64_t)c * 16);
      float d[V::N], dx[V::N] = {};
      V::unpack(vx, d);
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        float f[V::N];
        V::unpack(v[b], f);
        float s[2] = {};
#pragma unroll
        for (int e = 0; e < V::N; ++e) {
          s[e & 1] = fmaf(d[e], f[e], s[e & 1]);
          dx[e] = ok[b] ? fmaf(wj[b], f[e], dx[e]) : dx[e];
        }
        acc[b] += s[0] + s[1];
      }
      st16(a.dx + ((int64_t)t * nch + c) * 16, V::pack(dx));
    }
    const float s = wave_sums<P>(acc, lane);
    constexpr int kStep = 64 / P;
    __syncthreads();  // the token before has read its sums
    if (lane % kStep == 0) red[wave][lane / kStep] = s;
    __syncthreads();
    if (tid < KB && tid < a.k) {
      float v = 0.f;
      for (int i = 0; i < nw; ++i) v += red[i][tid];
      const int p = a.pos[a0 + tid];
      a.dw[a0 + tid] = (unsigned)p < (unsigned)a.R ? v : 0.f;
    }
  }
}

template <bool F32>
hipError_t launch_token(const TokenArgs& a, hipStream_t s) {
  // Waves a token: one, or as many as it takes to have about 16 a compute unit, but no
  // more than the row has work for (4096 x 2560 x 10: 58 us; five waves a token 138).
  int nw = 1;
  while (nw < kTokenThreads / 64 && (int64_t)a.T * nw < 4096 && nw * 64 < a.nch) nw *= 2;
  const int nt = nw * 64, grid = a.T < (1 << 22) ? a.T : 1 << 22;
  if (a.k <= 4) token_kernel<F32, 4><<<grid, nt, 0, s>>>(a);
  else if (a.k <= 8) token_kernel<F32, 8><<<grid, nt, 0, s>>>(a);
  else if (a.k <= 10) token_kernel<F32, 10><<<grid, nt, 0, s>>>(a);
  else if (a.k <= 16) token_kernel<F32, 16><<<grid, nt, 0, s>>>(a);
  else token_kernel<F32, 20><<<grid, nt, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_permute(const void* x, const int32_t* pos, const float* w, void* xs, int T, int H, int k, int f32,
                          hipStream_t s) {
  const Divisor chunks(H / (f32 ? 4 : 8));
  const int n = T * chunks.d, grid = (n + 255) / 256;
  const char* xb = static_cast<const char*>(x);
  char* o = static_cast<char*>(xs);
  if (f32 && w) permute_kernel<true, true><<<grid, 256, 0, s>>>(xb, pos, w, o, n, chunks, k, T * k);
  else if (w) permute_kernel<false, true><<<grid, 256, 0, s>>>(xb, pos, w, o, n, chunks, k, T * k);
  else permute_kernel<false, false><<<grid, 256, 0, s>>>(xb, pos, w, o, n, chunks, k, T * k);  // bytes alone
  return hipGetLastError();
}

hipError_t launch_permute_backward(const void* dxs, const int32_t* pos, const float* w, const void* x, void* dx,
                                   float* dw, int T, int H, int k, int f32, hipStream_t s) {
  const Divisor chunks(H / (f32 ? 4 : 8));
  const char* d = static_cast<const char*>(dxs);
  char* o = static_cast<char*>(dx);
  // (6550 x 552 x 18: 46 us, the products and then dx 81)
  if (dw && k <= 20) {
    const TokenArgs a{static_cast<const char*>(x), d, pos, w, o, dw, T, chunks.d, k, T * k};
    return f32 ? launch_token<true>(a, s) : launch_token<false>(a, s);
  }
  if (dw) {  // more rows than registers hold: the products, then dx
    RowArgs a{};
    a.dout = static_cast<const char*>(x);
    a.y = d;
    a.pos = pos;
    a.dw = dw;
    a.nch = chunks.d;
    a.k = k;
    a.R = T * k;
    const hipError_t e = launch_rows(a, T, k, f32, s);
    if (e != hipSuccess) return e;
  }
  const int n = T * chunks.d, grid = (n + 255) / 256;
#define MOE_UNPERMUTE(F32, W)                                                                                         \
  do {                                                                                                                \
    if (k <= 4) unpermute_kernel<F32, W, 4><<<grid, 256, 0, s>>>(d, pos, w, o, n, chunks, k, T * k);                  \
    else if (k == 9 || k == 10) unpermute_kernel<F32, W, 10><<<grid, 256, 0, s>>>(d, pos, w, o, n, chunks, k, T * k); \
    else unpermute_kernel<F32, W, 8><<<grid, 256, 0, s>>>(d, pos, w, o, n, chunks, k, T * k);                         \
  } while (0)
  if (f32 && w) MOE_UNPERMUTE(true, true);
  else if (f32) MOE_UNPERMUTE(true, false);
  else if (w) MOE_UNPERMUTE(false, true);
  else MOE_UNPERMUTE(false, false);
#undef MOE_UNPERMUTE
  return hipGetLastError();
}

hipError_t launch_combine_backward(const void* dout, const void* y, const int32_t* pos, const float* w,
                                   const void* y_sh, const float* sl, void* dy, float* dw, void* dy_sh, float* dsl,
                                   int T, int H, int k, int f32, hipStream_t s) {
  RowArgs a{static_cast<const char*>(dout), static_cast<const char*>(y), pos, w, static_cast<const char*>(y_sh), sl,
            static_cast<char*>(dy), dw, static_cast<char*>(dy_sh), dsl, H / (f32 ? 4 : 8), k, T * k};
  if (dw) return launch_rows(a, T, k + (y_sh ? 1 : 0), f32, s);
  // without the weights' gradient dy is dout permuted
  const hipError_t e = launch_permute(dout, pos, w, dy, T, H, k, f32, s);
  if (e != hipSuccess || !y_sh) return e;
  a.first = k;
  return launch_rows(a, T, 1, f32, s);
}

}  // namespace moe
