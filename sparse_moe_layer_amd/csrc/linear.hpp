// What the kernels of the grouped products share: activations, groups' rows and
// the search for the group that a tile of rows belongs to.
#pragma once
#include "kernels.hpp"
#include "vec.hpp"

namespace moe {

__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(-0.70710678f * z); }

// act(z), and its derivative in d
__device__ __forceinline__ float activate(int act, float z) {
  if (act == MOE_ACT_SILU) return z / (1.f + expf(-z));
  if (act == MOE_ACT_GELU) return z * normal_cdf(z);
  return z;
}
__device__ __forceinline__ float activate_d(int act, float z, float& d) {
  if (act == MOE_ACT_SILU) {
    const float g = 1.f / (1.f + expf(-z));
    d = g * fmaf(z, 1.f - g, 1.f);
    return z * g;
  }
  if (act == MOE_ACT_GELU) {
    const float c = normal_cdf(z);
    d = fmaf(z * 0.39894228f, expf(-0.5f * z * z), c);
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

struct MTile {
  int g, row, end;  // group, first row, end of the group
};

// The groups' rows cut into tiles of `bm` rows, counted in order.  Every thread
// of a 256-thread workgroup builds it (groups <= 1024: four a thread), then
// looks tiles up; without offsets there is nothing to search.
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
    __shared__ int wave_total[4];
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
    for (int w = 0; w < 4; ++w) {
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

// The bf16 kernels: 1 forward, dx or dw by matrix-instruction tiles
// (p, q: the operands; out: y, dx or dw).
enum LinearMode { kLinForward = 0, kLinDx = 1, kLinDw = 2 };
hipError_t launch_linear_tiles(LinearMode mode, const LinearArgs& a, const void* p, const void* q, void* out,
                               hipStream_t s);

}  // namespace moe
