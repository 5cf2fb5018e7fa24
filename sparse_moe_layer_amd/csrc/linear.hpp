// What the kernels of the grouped products share: activations, groups' rows and
// the search for the group that a tile of rows belongs to.
#pragma once
#include "kernels.hpp"
#include "vec.hpp"

namespace moe {

// (x + 3) erfcx(x) for x >= 0, erfcx(x) = e^(x^2) erfc(x), as a polynomial in
// t = (x - 3) / (x + 3): a least-maximum fit over x in [0, 12], off by at most 4.7e-8 (near
// x = 0.1; 2e-8 relative).
__device__ __forceinline__ float erfcx_poly(float t) {
  float p = -3.14715813e-4f;
  p = fmaf(p, t, -4.63499426e-4f);
  p = fmaf(p, t, 3.08281556e-3f);
  p = fmaf(p, t, -1.23808580e-3f);
  p = fmaf(p, t, -2.68434100e-2f);
  p = fmaf(p, t, 1.19531333e-1f);
  p = fmaf(p, t, -3.10465366e-1f);
  p = fmaf(p, t, 5.90228140e-1f);
  p = fmaf(p, t, -8.83394539e-1f);
  return fmaf(p, t, 1.07400692f);
}

// The activations.  FAST (bf16 tensors): e^x and 1/x by the hardware's, the normal
// distribution's integral by the fit above, 2e-7 absolute and 2e-5 relative down to
// z = -12 (8192 x 2560 x 2048 with GELU 99 -> 84 us); else the exact functions.
template <bool FAST>
__device__ __forceinline__ float exp_of(float x) {
  if constexpr (FAST) return __builtin_amdgcn_exp2f(x * 1.44269504f);
  else return expf(x);
}
template <bool FAST>
__device__ __forceinline__ float logistic(float z) {
  if constexpr (FAST) return __builtin_amdgcn_rcpf(1.f + exp_of<true>(-z));
  else return 1.f / (1.f + expf(-z));
}
// Phi(z); density: e^(-z^2 / 2)
template <bool FAST>
__device__ __forceinline__ float normal_cdf(float z, float& density) {
  density = exp_of<FAST>(-0.5f * z * z);
  if constexpr (FAST) {
    // past x = 16 the density is 0 in fp32; an infinite x would make the fit's argument inf * 0
    const float x = fminf(fabsf(z) * 0.70710678f, 16.f), r = __builtin_amdgcn_rcpf(x + 3.f);
    const float h = 0.5f * density * r * erfcx_poly((x - 3.f) * r);
    return z < 0.f ? h : 1.f - h;
  } else {
    return 0.5f * erfcf(-0.70710678f * z);
  }
}

// n values through act
template <bool FAST, int n>
__device__ __forceinline__ void activate(int act, float (&z)[n]) {
  if (act == MOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < n; ++i) z[i] *= logistic<FAST>(z[i]);
  } else if (act == MOE_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      float e;
      z[i] *= normal_cdf<FAST>(z[i], e);
    }
  }
}
// act(z) and its derivative
template <bool FAST>
__device__ __forceinline__ float activate_d(int act, float z, float& d) {
  if (act == MOE_ACT_SILU) {
    const float g = logistic<FAST>(z);
    d = g * fmaf(z, 1.f - g, 1.f);
    return z * g;
  }
  if (act == MOE_ACT_GELU) {
    float e;
    const float c = normal_cdf<FAST>(z, e);
    d = fmaf(z * 0.39894228f, e, c);
    return z * c;
  }
  d = 1.f;
  return z;
}

// First and last row of group g; offsets outside [0, rows] and decreasing ones
// are brought into range, so that no access leaves the tensors.
__device__ __forceinline__ int2 group_rows(const int32_t* offsets, int g, int rows) {
  if (!offsets) return {0, rows};
  const int lo = min(max(offsets[g], 0), rows);
  return {lo, min(max(offsets[g + 1], lo), rows)};
}

enum LinearMode { kLinForward = 0, kLinDx = 1, kLinDw = 2 };

struct MTile {
  int g, row, end;  // group, first row, end of the group
};

// The groups' rows cut into tiles of `bm` rows, counted in order.  Every thread
// of a workgroup of 256 or 512 builds it (groups <= 1024: four a thread), then
// looks a tile up; without offsets there is nothing to search.
struct TileMap {
  const int32_t* offsets;
  int rows, bm, total;
  int first, n[4];
  int2 rr[4];
  __device__ __forceinline__ TileMap(const int32_t* off, int G, int rows_, int bm_)
      : offsets(off), rows(rows_), bm(bm_) {
    if (!offsets) {
      total = (rows + bm - 1) / bm;
      return;
    }
    __shared__ int wave_total[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int g = tid * 4 + i;
      rr[i] = g < G ? group_rows(offsets, g, rows) : int2{0, 0};
      n[i] = (rr[i].y - rr[i].x + bm - 1) / bm;
      sum += n[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o, kWave);
      if (lane >= o) incl += v;
    }
    if (lane == 63) wave_total[wave] = incl;
    __syncthreads();
    first = incl - sum;
    total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {  // the first 256 threads have all groups
      if (w < wave) first += wave_total[w];
      total += wave_total[w];
    }
    total = __builtin_amdgcn_readfirstlane(total);
  }
  // Tile idx in [0, total).  At most one call per kernel.
  __device__ __forceinline__ MTile find(int idx) const {
    if (!offsets) return {0, idx * bm, rows};
    __shared__ MTile found;
    int f = first;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (idx >= f && idx < f + n[i]) found = {(int)threadIdx.x * 4 + i, rr[i].x + (idx - f) * bm, rr[i].y};
      f += n[i];
    }
    __syncthreads();
    return {__builtin_amdgcn_readfirstlane(found.g), __builtin_amdgcn_readfirstlane(found.row),
            __builtin_amdgcn_readfirstlane(found.end)};
  }
};

// m-tiles of bm rows over all groups, at most
inline int max_tiles(int rows, int G, int bm) { return rows / bm + (G < rows ? G : rows); }

// Forward for groups of at most 16 rows.
hipError_t launch_linear_few(const LinearArgs& a, int waves, bool f32, hipStream_t s);

// Sums of the dbias partials: n columns, `splits` each; n == 0: none.  A workgroup of 256
// threads has 256 columns or, of many splits, 32 with 8 threads each, whose loads are a
// chain otherwise (4096 x 1024 with GELU, dz with 128 splits: 13 us; 38).
struct LinearSums {
  const float* partial;
  float* dbias;
  int n, splits;
  __host__ __device__ int parts() const { return splits > 16 ? 8 : 1; }
  int workgroups() const { return (n + 256 / parts() - 1) / (256 / parts()); }
};
__device__ __forceinline__ void add_partials(const LinearSums& a, int block) {
  __shared__ float red[256];
  const int parts = a.parts(), cols = 256 / parts, part = threadIdx.x / cols;
  const int i = block * cols + threadIdx.x % cols;
  float v = 0.f;
  if (i < a.n) {
    const float* p = a.partial + i;
#pragma unroll 4
    for (int s = part; s < a.splits; s += parts) v += p[(int64_t)s * a.n];
  }
  red[threadIdx.x] = v;
  __syncthreads();
  if (part || i >= a.n) return;
  for (int q = 1; q < parts; ++q) v += red[threadIdx.x + q * cols];
  a.dbias[i] = v;
}

// Products by matrix-instruction tiles: forward (a.x, a.w, a.y), or dx and dw (either may
// be null) from dz, with the sums of the partials beside them.
hipError_t launch_linear_tiles(const LinearArgs& a, bool f32, hipStream_t s);
hipError_t launch_linear_back_tiles(const LinearArgs& a, bool f32, const void* dz, const void* w, const void* x,
                                    void* dx, void* dw, const LinearSums& sums, hipStream_t s);

}  // namespace moe
