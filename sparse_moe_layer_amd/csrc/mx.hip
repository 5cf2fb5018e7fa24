// MXFP4 weights: rows of bf16 or fp32 values to E2M1 codes with one E8M0 scale
// per 32 values, and back to bf16.
//   s    = max(exponent field of amax - 2, 0)      (2^(s-127) = 2^(floor(log2 amax) - 2), at least 2^-127)
//   code = w / 2^(s-127) rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code
// Both directions stream: a lane handles 8 consecutive values (16 B of bf16, 4 B
// of codes), a quad of lanes one group, so its largest magnitude takes two
// in-quad exchanges and every access of a wave is one contiguous run.
#include "common.hpp"
#include "kernels.hpp"

namespace moe {
namespace {

constexpr int MX_NT = 256;
constexpr int MX_U = 4;  // chunks of 8 values per thread, MX_NT apart: their loads in flight together

// Maximum over the four lanes of a quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0xb1, 0xf, 0xf, false);  // quad_perm [1,0,3,2]
  v = o > v ? o : v;
  o = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x4e, 0xf, 0xf, false);  // quad_perm [2,3,0,1]
  return o > v ? o : v;
}

// E2M1 code of v: the number of rounding boundaries at or below |v| (a value on
// a boundary goes to the even one of its two codes), and the sign.
__device__ __forceinline__ uint32_t e2m1_code(float v) {
  const float a = fabsf(v);
  const uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
  return c | (__float_as_uint(v) >> 31 << 3);
}

// Chunk index -> element offset of its first value in rows `stride` apart.
template <bool DENSE>
__device__ __forceinline__ int64_t chunk_offset(int64_t c, int cpr, int64_t stride) {
  if constexpr (DENSE) return c * 8;
  const int64_t r = c / cpr;
  return r * stride + (c - r * cpr) * 8;
}

// n: chunks of 8 values; cpr: chunks per row.  n is a multiple of 4, so a
// group's four lanes are in or out together.
template <bool F32, bool DENSE>
__global__ __launch_bounds__(MX_NT) void mx_quantize_kernel(const void* __restrict__ w, int64_t n, int cpr,
                                                            int64_t stride, uint32_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
  const int64_t c0 = (int64_t)blockIdx.x * (MX_NT * MX_U) + threadIdx.x;
  u32x4 v[MX_U][F32 ? 2 : 1];
#pragma unroll
  for (int u = 0; u < MX_U; ++u) {
    const int64_t c = c0 + u * MX_NT;
    const int64_t o = chunk_offset<DENSE>(c < n ? c : n - 1, cpr, stride);
    const char* p = reinterpret_cast<const char*>(w) + o * (F32 ? 4 : 2);
    v[u][0] = ld16_nt(p);
    if constexpr (F32) v[u][1] = ld16_nt(p + 16);
  }
#pragma unroll
  for (int u = 0; u < MX_U; ++u) {
    const int64_t c = c0 + u * MX_NT;
    // the largest magnitude's bits, as fp32: magnitudes order as their bits do
    uint32_t m = 0;
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t a = v[u][i >> 2][i & 3] & 0x7fffffffu;
        m = a > m ? a : m;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t hi = v[u][0][i] & 0x7fff0000u, lo = (v[u][0][i] << 16) & 0x7fff0000u;
        m = hi > m ? hi : m;
        m = lo > m ? lo : m;
      }
    }
    m = quad_max(m);
    const uint32_t ex = m >> 23;
    const uint32_t s = ex == 255u ? 255u : (ex > 2u ? ex - 2u : 0u);
    uint32_t q = 0;
    if (s - 1u < 254u) {  // 1 .. 254: the scaled conversion rounds to nearest even and saturates at 6
      const float sc = e8m0(s);
      if constexpr (F32) {
        const f32x4 a = __builtin_bit_cast(f32x4, v[u][0]), b = __builtin_bit_cast(f32x4, v[u][1]);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, a[0], a[1], sc, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, a[2], a[3], sc, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, b[0], b[1], sc, 2);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, b[2], b[3], sc, 3);
      } else {
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, (uint32_t)v[u][0][0]), sc, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, (uint32_t)v[u][0][1]), sc, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, (uint32_t)v[u][0][2]), sc, 2);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, (uint32_t)v[u][0][3]), sc, 3);
      }
    } else if (s == 0u) {  // magnitudes below 2^-124: scaled by 2^127 first (also zeros, whose signs are kept)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float f;
        if constexpr (F32) f = __uint_as_float(v[u][i >> 2][i & 3]);
        else f = __uint_as_float(i & 1 ? v[u][0][i >> 1] & 0xffff0000u : v[u][0][i >> 1] << 16);
        q |= e2m1_code(f * 0x1p127f) << (4 * i);
      }
    }  // 255 (an infinity or a NaN in the group): codes 0, the scale says NaN
    if (c < n) {
      codes[c] = q;
      if ((threadIdx.x & 3) == 0) scales[c >> 2] = (uint8_t)s;
    }
  }
}

template <bool DENSE>
__global__ __launch_bounds__(MX_NT) void mx_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, int64_t n, int cpr,
                                                              int64_t stride, bf16* __restrict__ w) {
  const int64_t c0 = (int64_t)blockIdx.x * (MX_NT * MX_U) + threadIdx.x;
  uint32_t q[MX_U], s[MX_U];
#pragma unroll
  for (int u = 0; u < MX_U; ++u) {
    int64_t c = c0 + u * MX_NT;
    c = c < n ? c : n - 1;
    q[u] = __builtin_nontemporal_load(codes + c);
    s[u] = scales[c >> 2];
  }
#pragma unroll
  for (int u = 0; u < MX_U; ++u) {
    const int64_t c = c0 + u * MX_NT;
    if (c < n) st16_nt(w + chunk_offset<DENSE>(c, cpr, stride), mx8_to_bf16x8(q[u], e8m0(s[u])));
  }
}

inline unsigned mx_grid(int64_t n) { return (unsigned)((n + MX_NT * MX_U - 1) / (MX_NT * MX_U)); }

}  // namespace

hipError_t launch_mx_quantize(const void* w, bool f32, int64_t rows, int64_t K, int64_t row_stride, void* codes,
                              void* scales, hipStream_t s) {
  const int64_t n = rows * (K / 8);
  const bool dense = row_stride == K || rows == 1;
  uint32_t* c = static_cast<uint32_t*>(codes);
  uint8_t* e = static_cast<uint8_t*>(scales);
  const int cpr = (int)(K / 8);
  if (f32 && dense) mx_quantize_kernel<true, true><<<mx_grid(n), MX_NT, 0, s>>>(w, n, cpr, row_stride, c, e);
  else if (f32) mx_quantize_kernel<true, false><<<mx_grid(n), MX_NT, 0, s>>>(w, n, cpr, row_stride, c, e);
  else if (dense) mx_quantize_kernel<false, true><<<mx_grid(n), MX_NT, 0, s>>>(w, n, cpr, row_stride, c, e);
  else mx_quantize_kernel<false, false><<<mx_grid(n), MX_NT, 0, s>>>(w, n, cpr, row_stride, c, e);
  return hipGetLastError();
}

hipError_t launch_mx_dequantize(const void* codes, const void* scales, int64_t rows, int64_t K, void* w,
                                int64_t row_stride, hipStream_t s) {
  const int64_t n = rows * (K / 8);
  const bool dense = row_stride == K || rows == 1;
  const uint32_t* c = static_cast<const uint32_t*>(codes);
  const uint8_t* e = static_cast<const uint8_t*>(scales);
  bf16* o = static_cast<bf16*>(w);
  const int cpr = (int)(K / 8);
  if (dense) mx_dequantize_kernel<true><<<mx_grid(n), MX_NT, 0, s>>>(c, e, n, cpr, row_stride, o);
  else mx_dequantize_kernel<false><<<mx_grid(n), MX_NT, 0, s>>>(c, e, n, cpr, row_stride, o);
  return hipGetLastError();
}

}  // namespace moe
