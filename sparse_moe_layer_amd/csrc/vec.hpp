// 16-byte vectors of act dtype as fp32 values, and sums over waves and
// workgroups, for the row kernels (permute, block norms, linear epilogues).
#pragma once
#include "common.hpp"

namespace moe {

// Vec<F32>::N values in 16 bytes: 4 fp32 or 8 bf16
template <bool F32>
struct Vec {
  static constexpr int N = F32 ? 4 : 8;
  static constexpr int ESZ = F32 ? 4 : 2;
  __device__ static __forceinline__ void unpack(u32x4 v, float* f) {
    if constexpr (F32) {
      const f32x4 a = __builtin_bit_cast(f32x4, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = a[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // bf16 is the high half of the fp32 word
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
      }
    }
  }
  __device__ static __forceinline__ u32x4 pack(const float* f) {
    if constexpr (F32) {
      return __builtin_bit_cast(u32x4, f32x4{f[0], f[1], f[2], f[3]});
    } else {
      bf16x8 b;
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = f2bf(f[i]);
      return __builtin_bit_cast(u32x4, b);
    }
  }
};

// Sums of P values (a power of two up to 64) over a wave's lanes.  A step over
// lanes o apart keeps one half of the values in the lanes with bit o set and
// the other half in the rest, so P values take P - 1 + 6 - log2(P) exchanges
// instead of 6 P.  Lane l returns the sum of value l >> (6 - log2(P)).
template <int P>
__device__ __forceinline__ float wave_sums(float (&a)[P], int lane) {
  int o = 32;
#pragma unroll
  for (int n = P; n > 1; n >>= 1, o >>= 1) {
    // (masks, not selects: those of two array elements become a run-time index)
    const uint32_t up = lane & o ? 0xFFFFFFFFu : 0u;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const uint32_t lo = __float_as_uint(a[i]), hi = __float_as_uint(a[i + n / 2]);
      const float send = __uint_as_float((lo & up) | (hi & ~up)), keep = __uint_as_float((hi & up) | (lo & ~up));
      a[i] = keep + __shfl_xor(send, o, kWave);
    }
  }
  for (; o > 0; o >>= 1) a[0] += __shfl_xor(a[0], o, kWave);
  return a[0];
}

// log2 of a power of two
constexpr int log2_of(int p) { return p <= 1 ? 0 : 1 + log2_of(p / 2); }

// A grid of at least n workgroups of up to 1024 threads, in rows: a dimension holds less
// than 2^32 threads.
inline dim3 row_grid(int64_t n) {
  const int64_t x = n < (1 << 21) ? n : 1 << 21;
  return dim3((uint32_t)x, (uint32_t)((n + x - 1) / x));
}

}  // namespace moe
