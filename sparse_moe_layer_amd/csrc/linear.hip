// Products over groups of rows, and their gradients:
//   forward  z = x W_g^T + b_g,  y = resid + act(z) mul
//   backward dz = dy mul act'(z), dmul = dy act(z), db_g = sum dz;  dx = dz W_g;  dW_g = dz^T x
// The rows of group g are [offsets[g], offsets[g+1]), known to the device only.
#include "linear.hpp"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// fp32 matrix instructions on 64 x 64 tiles, any dtype
// ---------------------------------------------------------------------------
// MODE 0: rows x [r][K] by W [n][K].  MODE 1: rows dz [r][N] by W, contracted over
// its rows.  MODE 2: dz and x contracted over the group's rows.
// Both operands are staged as fp32 [k][64], so a lane's fragment values lie side
// by side across the lanes.
constexpr int kSB = 64, kSK = 16, kSP = kSB + 1;

template <bool F32>
__device__ __forceinline__ float elem(const void* p, int64_t i) {
  if constexpr (F32) return static_cast<const float*>(p)[i];
  else return bf2f(static_cast<const bf16*>(p)[i]);
}
template <bool F32>
__device__ __forceinline__ void put(void* p, int64_t i, float v) {
  if constexpr (F32) static_cast<float*>(p)[i] = v;
  else static_cast<bf16*>(p)[i] = f2bf(v);
}

// Stages [kSK][64] of an operand: element (row, k) at base + row * srow + k * sk
// (one stride is 1); rows from nrow and k from nk on are zeros.
template <bool F32, bool K_LAST>
__device__ __forceinline__ void stage(float* lds, const void* base, int64_t ld, int nrow, int nk, int tid) {
#pragma unroll
  for (int i = 0; i < kSB * kSK / 256; ++i) {
    const int q = tid + i * 256;
    const int k = K_LAST ? q % kSK : q / kSB, r = K_LAST ? q / kSK : q % kSB;
    const bool in = r < nrow && k < nk;
    lds[k * kSP + r] = in ? elem<F32>(base, K_LAST ? r * ld + k : k * ld + r) : 0.f;
  }
}

template <bool F32, int MODE>
__global__ __launch_bounds__(256) void linear_simple_kernel(LinearArgs a, const void* p, const void* q, void* out) {
  __shared__ float sa[kSK * kSP], sb[kSK * kSP];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int ESZ = F32 ? 4 : 2;
  int g, m0, m1, k0 = 0, kn, n0, nn;
  if constexpr (MODE == 2) {
    g = blockIdx.z;
    const int2 rr = group_rows(a.offsets, g, a.rows);
    k0 = rr.x;
    kn = rr.y - rr.x;
    m0 = blockIdx.y * kSB;
    m1 = a.N;
    n0 = blockIdx.x * kSB;
    nn = a.K;
  } else {
    const TileMap map(a.offsets, a.G, a.rows, kSB);
    if ((int)blockIdx.x >= map.total) return;
    const MTile t = map.find(blockIdx.x);
    g = t.g;
    m0 = t.row;
    m1 = t.end;
    kn = MODE == 0 ? a.K : a.N;
    n0 = blockIdx.y * kSB;
    nn = MODE == 0 ? a.N : a.K;
  }
  const char* pa = static_cast<const char*>(p);
  const char* pb = static_cast<const char*>(q);
  if constexpr (MODE == 0) {
    pa += (int64_t)m0 * a.K * ESZ;
    pb += (g * a.w_stride + (int64_t)n0 * a.K) * ESZ;
  } else if constexpr (MODE == 1) {
    pa += (int64_t)m0 * a.N * ESZ;
    pb += (g * a.w_stride + n0) * ESZ;
  } else {
    pa += ((int64_t)k0 * a.N + m0) * ESZ;
    pb += ((int64_t)k0 * a.K + n0) * ESZ;
  }
  f32x16 acc = {};
  const int wm = wave >> 1, wn = wave & 1;
  for (int k = 0; k < kn; k += kSK) {
    const int left = kn - k;
    if constexpr (MODE == 2) {
      stage<F32, false>(sa, pa + (int64_t)k * a.N * ESZ, a.N, m1 - m0, left, tid);
      stage<F32, false>(sb, pb + (int64_t)k * a.K * ESZ, a.K, nn - n0, left, tid);
    } else {
      stage<F32, true>(sa, pa + (int64_t)k * ESZ, MODE == 0 ? a.K : a.N, m1 - m0, left, tid);
      if constexpr (MODE == 0) stage<F32, true>(sb, pb + (int64_t)k * ESZ, a.K, nn - n0, left, tid);
      else stage<F32, false>(sb, pb + (int64_t)k * a.K * ESZ, a.K, nn - n0, left, tid);
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kSK; kk += 2) {
      const int o = (kk + (lane >> 5)) * kSP + (lane & 31);
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(sa[o + wm * 32], sb[o + wn * 32], acc, 0, 0, 0);
    }
    __syncthreads();
  }
  const int col = n0 + wn * 32 + (lane & 31);
  if (col >= nn) return;
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const int row = m0 + wm * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
    if (row >= m1) continue;
    if constexpr (MODE == 2) {
      put<F32>(out, g * a.w_stride + (int64_t)row * a.K + col, acc[v]);
    } else if constexpr (MODE == 1) {
      put<F32>(out, (int64_t)row * a.K + col, acc[v]);
    } else {
      const int64_t i = (int64_t)row * a.N + col;
      float z = acc[v];
      if (a.bias) z += elem<F32>(a.bias, (int64_t)g * a.N + col);
      if (a.z) put<F32>(a.z, i, z);
      float v[1] = {z};
      activate<false>(a.act, v);
      float y = v[0];
      if (a.mul) y *= elem<F32>(a.mul, i);
      if (a.resid) y += elem<F32>(a.resid, i);
      put<F32>(out, i, y);
    }
  }
}

// ---------------------------------------------------------------------------
// dz, dmul and the sums over a group's rows of dz
// ---------------------------------------------------------------------------
// Workgroup: 32 threads across 16-byte chunks, 8 rows at a time, of split
// blockIdx.x of group blockIdx.z's rows (without sums: of all groups' rows).
template <bool F32>
__global__ __launch_bounds__(256) void linear_dz_kernel(LinearBackArgs a, int splits, bool sums, bool store) {
  using V = Vec<F32>;
  __shared__ float red[8][32][V::N + 1];
  const int c = blockIdx.y * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  const int nch = a.N / V::N, g = blockIdx.z;
  int2 rr = group_rows(a.offsets, g, a.rows);
  if (!sums) rr.y = max(rr.x, group_rows(a.offsets, a.G - 1, a.rows).y);
  const int64_t n = rr.y - rr.x;
  const int r0 = rr.x + (int)(n * blockIdx.x / splits), r1 = rr.x + (int)(n * (blockIdx.x + 1) / splits);
  float s[V::N] = {};
  if (c < nch)
    for (int r = r0 + part; r < r1; r += 8) {
      const int64_t i = ((int64_t)r * nch + c) * 16;
      float d[V::N];
      V::unpack(ld16(static_cast<const char*>(a.dy) + i), d);
      if (store) {
        float z[V::N] = {}, m[V::N], dm[V::N];
        if (a.z) V::unpack(ld16(static_cast<const char*>(a.z) + i), z);
        if (a.mul) V::unpack(ld16(static_cast<const char*>(a.mul) + i), m);
#pragma unroll
        for (int e = 0; e < V::N; ++e) {
          float slope;
          const float v = activate_d<!F32>(a.act, z[e], slope);
          dm[e] = d[e] * v;
          d[e] = d[e] * (a.mul ? m[e] : 1.f) * slope;
        }
        if (a.dmul) st16(static_cast<char*>(a.dmul) + i, V::pack(dm));
        if (a.dz) st16(static_cast<char*>(a.dz) + i, V::pack(d));
      }
#pragma unroll
      for (int e = 0; e < V::N; ++e) s[e] += d[e];
    }
  if (!sums) return;
#pragma unroll
  for (int e = 0; e < V::N; ++e) red[part][threadIdx.x & 31][e] = s[e];
  __syncthreads();
  float* o = splits == 1 ? a.dbias : a.partial + (int64_t)blockIdx.x * a.G * a.N;
  for (int i = threadIdx.x; i < 32 * V::N; i += 256) {
    const int col = blockIdx.y * 32 * V::N + i;
    if (col >= a.N) break;
    float v = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) v += red[q][i / V::N][i % V::N];
    o[(int64_t)g * a.N + col] = v;
  }
}

__global__ __launch_bounds__(256) void linear_sums_kernel(const float* __restrict__ partial, float* __restrict__ out,
                                                          int n, int splits) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v = 0.f;
  for (int s = 0; s < splits; ++s) v += partial[(int64_t)s * n + i];
  out[i] = v;
}

// Parts of each group's rows for the sums: about 64 rows each
int sum_splits(int64_t rows, int64_t G) {
  const int64_t s = rows / G / 64;
  return s < 1 ? 1 : s > 64 ? 64 : (int)s;
}

}  // namespace

size_t linear_partial_floats(int64_t rows, int64_t N, int64_t G) {
  const int s = sum_splits(rows, G);
  return s > 1 ? (size_t)s * G * N : 0;
}

hipError_t launch_linear(const LinearArgs& a, bool f32, hipStream_t s) {
  const int64_t few = (int64_t)(a.G < a.rows ? a.G : a.rows) * ((a.N + 15) / 16);
  if (!f32 && a.rows <= 16 * (int64_t)a.G && few <= 256) return launch_linear_few(a, s);
  if (!f32) return launch_linear_tiles(kLinForward, a, a.x, a.w, a.y, s);
  const dim3 grid(max_tiles(a.rows, a.G, kSB), (a.N + kSB - 1) / kSB);
  linear_simple_kernel<true, 0><<<grid, 256, 0, s>>>(a, a.x, a.w, a.y);
  return hipGetLastError();
}

hipError_t launch_linear_backward(const LinearBackArgs& b, bool f32, hipStream_t s) {
  LinearBackArgs a = b;
  const bool store = a.act != MOE_ACT_NONE || a.mul || a.dmul;
  if (!(a.act != MOE_ACT_NONE || a.mul)) a.dz = nullptr;  // dz is dy
  const int vec = f32 ? 4 : 8;
  const int cols = (a.N / vec + 31) / 32;
  if (a.rows > 0 || a.dbias) {
    if (a.dbias) {
      const int splits = sum_splits(a.rows, a.G);
      const dim3 grid(splits, cols, a.G);
      if (f32) linear_dz_kernel<true><<<grid, 256, 0, s>>>(a, splits, true, store);
      else linear_dz_kernel<false><<<grid, 256, 0, s>>>(a, splits, true, store);
      if (splits > 1)
        linear_sums_kernel<<<(a.G * a.N + 255) / 256, 256, 0, s>>>(a.partial, a.dbias, a.G * a.N, splits);
    } else if (store) {
      const int splits = (a.rows + 31) / 32;
      const dim3 grid(splits, cols, 1);
      if (f32) linear_dz_kernel<true><<<grid, 256, 0, s>>>(a, splits, false, true);
      else linear_dz_kernel<false><<<grid, 256, 0, s>>>(a, splits, false, true);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const void* dz = a.dz ? a.dz : a.dy;
  LinearArgs l{};
  l.offsets = a.offsets;
  l.rows = a.rows;
  l.K = a.K;
  l.N = a.N;
  l.G = a.G;
  l.w_stride = a.w_stride;
  if (!f32) {
    hipError_t e = hipSuccess;
    if (a.dx && a.rows > 0) e = launch_linear_tiles(kLinDx, l, dz, a.w, a.dx, s);
    if (a.dw && e == hipSuccess) e = launch_linear_tiles(kLinDw, l, dz, a.x, a.dw, s);
    return e;
  }
  if (a.dx && a.rows > 0) {
    const dim3 grid(max_tiles(a.rows, a.G, kSB), (a.K + kSB - 1) / kSB);
    linear_simple_kernel<true, 1><<<grid, 256, 0, s>>>(l, dz, a.w, a.dx);
  }
  if (a.dw) {
    const dim3 grid((a.K + kSB - 1) / kSB, (a.N + kSB - 1) / kSB, a.G);
    linear_simple_kernel<true, 2><<<grid, 256, 0, s>>>(l, dz, a.x, a.dw);
  }
  return hipGetLastError();
}

}  // namespace moe
