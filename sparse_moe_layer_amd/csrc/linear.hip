// Products over groups of rows, and their gradients:
//   forward  z = x W_g^T + b_g,  y = resid + act(z) mul
//   backward dz = dy mul act'(z), dmul = dy act(z), db_g = sum dz;  dx = dz W_g;  dW_g = dz^T x
// The rows of group g are [offsets[g], offsets[g+1]), known to the device only.
#include "linear.hpp"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// dz, dmul and the sums over a group's rows of dz
// ---------------------------------------------------------------------------
// One pass over dy, z and mul, bound by HBM (40960 x 640 bf16 with SiLU and a factor, 0.26 GB:
// 43 us, 6 TB/s).  Workgroup: 32 threads across 16-byte chunks, 8 rows at a time, of split
// blockIdx.x of group blockIdx.z's rows (without sums: of all groups' rows).
// bf16 dz is rounded once here, as the operand of both products that bf16 matrix instructions
// take: dx and dw are then 2.35e-3 (root mean square) from the exact gradients, of which the
// rounding of dx and dw themselves is 1.66e-3.  Kept in two bf16 parts it would double both
// products' matrix instructions and dz's bytes; in fp32 they run at a ninth of the rate.  dbias
// adds the unrounded values, and without activation and factor dz is dy, not rounded at all.
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
  constexpr int U = 4;  // rows a thread has in flight
  if (c < nch)
    for (int r = r0 + part; r < r1; r += 8 * U) {
      u32x4 vd[U], vz[U], vm[U];
      int64_t at[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r + 8 * u >= r1) break;
        at[u] = ((int64_t)(r + 8 * u) * nch + c) * 16;
        vd[u] = ld16(static_cast<const char*>(a.dy) + at[u]);
        if (store && a.z) vz[u] = ld16(static_cast<const char*>(a.z) + at[u]);
        if (store && a.mul) vm[u] = ld16(static_cast<const char*>(a.mul) + at[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (r + 8 * u >= r1) break;
        float d[V::N];
        V::unpack(vd[u], d);
        if (store) {
          float z[V::N] = {}, m[V::N], dm[V::N];
          if (a.z) V::unpack(vz[u], z);
          if (a.mul) V::unpack(vm[u], m);
#pragma unroll
          for (int e = 0; e < V::N; ++e) {
            float slope;
            const float v = activate_d<!F32>(a.act, z[e], slope);
            dm[e] = d[e] * v;
            d[e] = d[e] * (a.mul ? m[e] : 1.f) * slope;
          }
          if (a.dmul) st16(static_cast<char*>(a.dmul) + at[u], V::pack(dm));
          if (a.dz) st16(static_cast<char*>(a.dz) + at[u], V::pack(d));
        }
#pragma unroll
        for (int e = 0; e < V::N; ++e) s[e] += d[e];
      }
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

__global__ __launch_bounds__(256) void linear_sums_kernel(LinearSums s) {
  add_partials(s, blockIdx.x);
}

// Rows of a part of a group of n rows, in `cols` columns of workgroups: 32, what a workgroup's
// threads have in flight, or 16 or 8 where those would be few workgroups (1000 x 2056 with
// GELU and db 11.6 us; parts of 32 rows 12.9).
int64_t part_rows(int64_t n, int64_t cols) {
  int64_t part = 32;
  while (part > 8 && (n + part - 1) / part * cols < 1024) part /= 2;
  return part;
}
int64_t chunk_columns(int64_t N, bool f32) { return (N / (f32 ? 4 : 8) + 31) / 32; }
// Parts of each group's rows for the sums
int sum_splits(int64_t rows, int64_t N, int64_t G, bool f32) {
  const int64_t n = rows / G, part = part_rows(n, chunk_columns(N, f32) * G), s = (n + part - 1) / part;
  return s < 1 ? 1 : s > 256 ? 256 : (int)s;
}

}  // namespace

size_t linear_partial_floats(int64_t rows, int64_t N, int64_t G, bool f32) {
  const int s = sum_splits(rows, N, G, f32);
  return s > 1 ? (size_t)s * G * N : 0;
}

hipError_t launch_linear(const LinearArgs& a, bool f32, hipStream_t s) {
  // Groups of at most 16 rows with few columns: 16 rows of W a workgroup and K over its 8
  // waves (a row of 8192 x 2048: 7.9 us, 64-row tiles 20.1).  Twice as many workgroups still
  // run at once with 4 waves each, better than tiles where those waves are done in a few
  // pieces and need little of x (ten groups of a row of 2560 x 640: 9.8; 10.3, fp32 14.4;
  // 17.2, but 8 groups of 4096 x 1024 14.2; 13.4 and with 16 rows each 17.0; 13.4).
  const int64_t touched = a.G < a.rows ? a.G : a.rows, few = touched * ((a.N + 15) / 16);
  if (a.rows <= 16 * (int64_t)a.G && few <= 256) return launch_linear_few(a, 8, f32, s);
  if (a.rows <= 2 * touched && few <= 512 && a.K <= 2560) return launch_linear_few(a, 4, f32, s);
  return launch_linear_tiles(a, f32, s);
}

hipError_t launch_linear_backward(const LinearBackArgs& b, bool f32, hipStream_t s) {
  LinearBackArgs a = b;
  const bool factor = a.act != MOE_ACT_NONE || a.mul;  // else dz is dy
  const bool store = factor || a.dmul;
  if (!factor) a.dz = nullptr;
  const int cols = (int)chunk_columns(a.N, f32);
  LinearSums sums{};
  if (a.dbias || (store && a.rows > 0)) {
    const int64_t part = part_rows(a.rows, cols);  // without the sums the groups do not matter
    const int splits = a.dbias ? sum_splits(a.rows, a.N, a.G, f32) : (int)((a.rows + part - 1) / part);
    const dim3 grid(splits, cols, a.dbias ? a.G : 1);
    if (f32) linear_dz_kernel<true><<<grid, 256, 0, s>>>(a, splits, a.dbias != nullptr, store);
    else linear_dz_kernel<false><<<grid, 256, 0, s>>>(a, splits, a.dbias != nullptr, store);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.dbias && splits > 1) sums = {a.partial, a.dbias, a.G * a.N, splits};
  }
  void* dx = a.rows > 0 ? a.dx : nullptr;
  if (!dx && !a.dw) {
    if (sums.n) linear_sums_kernel<<<sums.workgroups(), 256, 0, s>>>(sums);
    return hipGetLastError();
  }
  LinearArgs l{};
  l.offsets = a.offsets;
  l.rows = a.rows;
  l.K = a.K;
  l.N = a.N;
  l.G = a.G;
  l.w_stride = a.w_stride;
  return launch_linear_back_tiles(l, f32, a.dz ? a.dz : a.dy, a.w, a.x, dx, a.dw, sums, s);
}

}  // namespace moe
