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

// One thread per 16 bytes of x; n = T * (chunks of a row).
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

// dx alone: one thread per 16 bytes of dx.
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

// With products over H: one workgroup per token, its threads over the row's
// 16-byte chunks, KB assignments at a time, each with a sum in a register.
// GRAD_Y: combine_backward, else permute_backward.
struct TokenArgs {
  const char* own;    // dout, or x
  const char* rows;   // y, or dxs (y may be null)
  const int32_t* pos;
  const float* w;     // null: 1
  const char* y_sh;
  const float* sl;
  char* out;          // dy, or dx (null, or k <= KB: a thread has all of a token's rows)
  float* dw;
  char* dy_sh;
  float* dsl;
  int nch, k, R;      // 16-byte chunks of a row
};

constexpr int kTokenThreads = 512;

template <bool F32, bool GRAD_Y, int KB>
__global__ __launch_bounds__(kTokenThreads) void token_kernel(TokenArgs a) {
  using V = Vec<F32>;
  constexpr int P = KB <= 4 ? 4 : KB <= 8 ? 8 : 16;
  __shared__ float red[kTokenThreads / 64][P];
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
  const int nch = a.nch;
  const int64_t a0 = (int64_t)t * a.k;
  const char* own = a.own + (int64_t)t * nch * 16;
  const bool sums = a.dw != nullptr;
  const bool shared = GRAD_Y && a.y_sh != nullptr;
  const float g = shared ? sigmoid_f32(a.sl[t]) : 0.f;
  float dots = 0.f;
  for (int j0 = 0; j0 < a.k; j0 += KB) {
    float acc[P] = {};
    int64_t row[KB];
    bool ok[KB];
    float wj[KB];
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const int j = j0 + b < a.k ? j0 + b : a.k - 1;
      const int p = a.pos[a0 + j];
      ok[b] = j0 + b < a.k && (unsigned)p < (unsigned)a.R;
      row[b] = (int64_t)(ok[b] ? p : 0) * nch * 16;
      wj[b] = a.w ? a.w[a0 + j] : 1.f;
    }
    for (int c = tid; c < nch; c += blockDim.x) {
      u32x4 v[KB], vs = {};
      const u32x4 vo = ld16(own + (int64_t)c * 16);
      if (!GRAD_Y || sums) {
#pragma unroll
        for (int b = 0; b < KB; ++b) v[b] = ld16_nt(a.rows + row[b] + (int64_t)c * 16);
      }
      const bool sh = shared && j0 == 0;
      if (sh) vs = ld16_nt(a.y_sh + ((int64_t)t * nch + c) * 16);
      float d[V::N], dx[V::N] = {};
      V::unpack(vo, d);
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        float f[V::N];
        if (!GRAD_Y || sums) {
          V::unpack(v[b], f);
#pragma unroll
          for (int e = 0; e < V::N; ++e) acc[b] = fmaf(d[e], f[e], acc[b]);
        }
        if constexpr (GRAD_Y) {
          if (ok[b]) {
#pragma unroll
            for (int e = 0; e < V::N; ++e) f[e] = wj[b] * d[e];
            st16(a.out + row[b] + (int64_t)c * 16, V::pack(f));
          }
        } else {
#pragma unroll
          for (int e = 0; e < V::N; ++e) dx[e] = ok[b] ? fmaf(wj[b], f[e], dx[e]) : dx[e];
        }
      }
      if constexpr (!GRAD_Y) {
        if (a.out) st16(a.out + ((int64_t)t * nch + c) * 16, V::pack(dx));
      }
      if (sh) {
        float f[V::N];
        V::unpack(vs, f);
#pragma unroll
        for (int e = 0; e < V::N; ++e) {
          dots = fmaf(d[e], f[e], dots);
          f[e] = g * d[e];
        }
        st16(a.dy_sh + ((int64_t)t * nch + c) * 16, V::pack(f));
      }
    }
    if (sums) {
      const float s = wave_sums<P>(acc, lane);
      constexpr int kStep = 64 / P;
      __syncthreads();  // the values of the batch before are read
      if (lane % kStep == 0) red[wave][lane / kStep] = s;
      __syncthreads();
      if (tid < KB && j0 + tid < a.k) {
        float v = 0.f;
        for (int i = 0; i < nw; ++i) v += red[i][tid];
        const int p = a.pos[a0 + j0 + tid];
        a.dw[a0 + j0 + tid] = (unsigned)p < (unsigned)a.R ? v : 0.f;
      }
    }
  }
  if (shared) {
    dots = wave_sum(dots);
    __syncthreads();
    if (lane == 0) red[wave][0] = dots;
    __syncthreads();
    if (tid == 0) {
      float v = 0.f;
      for (int i = 0; i < nw; ++i) v += red[i][0];
      a.dsl[t] = g * sigmoid_f32(-a.sl[t]) * v;
    }
  }
}

template <bool F32, bool GRAD_Y>
hipError_t launch_token(const TokenArgs& a, int T, hipStream_t s) {
  const int rounds = (a.nch + kTokenThreads - 1) / kTokenThreads;
  const int nt = ((a.nch + rounds - 1) / rounds + 63) / 64 * 64;
  if (a.k <= 4) token_kernel<F32, GRAD_Y, 4><<<T, nt, 0, s>>>(a);
  else if (a.k <= 8) token_kernel<F32, GRAD_Y, 8><<<T, nt, 0, s>>>(a);
  else if (a.k <= 10) token_kernel<F32, GRAD_Y, 10><<<T, nt, 0, s>>>(a);
  else token_kernel<F32, GRAD_Y, 16><<<T, nt, 0, s>>>(a);
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
  if (dw) {
    const TokenArgs a{static_cast<const char*>(x), d, pos, w, nullptr, nullptr, k <= 16 ? o : nullptr, dw, nullptr,
                      nullptr, chunks.d, k, T * k};
    const hipError_t e = f32 ? launch_token<true, false>(a, T, s) : launch_token<false, false>(a, T, s);
    if (a.out || e != hipSuccess) return e;  // more than 16 a token: dx by the kernel below
  }
  const int n = T * chunks.d, grid = (n + 255) / 256;
#define MOE_UNPERMUTE(F32, W)                                                                               \
  do {                                                                                                      \
    if (k <= 4) unpermute_kernel<F32, W, 4><<<grid, 256, 0, s>>>(d, pos, w, o, n, chunks, k, T * k);        \
    else if (k <= 10) unpermute_kernel<F32, W, 10><<<grid, 256, 0, s>>>(d, pos, w, o, n, chunks, k, T * k); \
    else unpermute_kernel<F32, W, 8><<<grid, 256, 0, s>>>(d, pos, w, o, n, chunks, k, T * k);               \
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
  const TokenArgs a{static_cast<const char*>(dout), static_cast<const char*>(y), pos, w,
                    static_cast<const char*>(y_sh), sl, static_cast<char*>(dy), dw, static_cast<char*>(dy_sh), dsl,
                    H / (f32 ? 4 : 8), k, T * k};
  return f32 ? launch_token<true, true>(a, T, s) : launch_token<false, true>(a, T, s);
}

}  // namespace moe
