// Order of logits (descending, equal ones by ascending expert id) as unsigned
// keys, which every routing kernel uses, and the top-k of one wave's keys
// (gfx950, 64 lanes).  The few-token layer picks from the same keys in a way of
// its own (few.hip), which ranks only the logits that can be among the k.
#pragma once
#include "common.hpp"

namespace moe {

// Monotone map fp32 -> u32 (a < b as floats <=> ord(a) < ord(b) unsigned),
// with -0 folded onto +0 so that equal values compare equal.  Every real
// logit maps above 0, which marks padding and taken entries.
__device__ __forceinline__ uint32_t ord(float v) {
  const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unord(uint32_t m) { return __uint_as_float((m >> 31) ? (m & 0x7fffffffu) : ~m); }

// Keys: the order-preserving image of the logit in the high word, the
// complement of the expert id in the low word; one unsigned 64-bit maximum
// ranks by value and sends equal values to the lower id.
__device__ __forceinline__ uint64_t make_key(uint32_t ordv, int e) { return ((uint64_t)ordv << 32) | (uint32_t)~e; }
__device__ __forceinline__ uint64_t key_max(uint64_t a, uint64_t b) { return b > a ? b : a; }

template <int CTRL>
__device__ __forceinline__ uint64_t dpp_max(uint64_t k) {
  const uint32_t hi = (uint32_t)(k >> 32), lo = (uint32_t)k;
  const uint32_t ohi = (uint32_t)__builtin_amdgcn_update_dpp((int)hi, (int)hi, CTRL, 0xf, 0xf, false);
  const uint32_t olo = (uint32_t)__builtin_amdgcn_update_dpp((int)lo, (int)lo, CTRL, 0xf, 0xf, false);
  return key_max(k, ((uint64_t)ohi << 32) | olo);
}

// Maximum key over the 64 lanes (wave-uniform result).
__device__ __forceinline__ uint64_t wave_key_max(uint64_t k) {
  k = dpp_max<0xb1>(k);   // quad_perm [1,0,3,2]
  k = dpp_max<0x4e>(k);   // quad_perm [2,3,0,1]: quad maximum in every lane
  k = dpp_max<0x141>(k);  // row_half_mirror: 8-lane maximum
  k = dpp_max<0x140>(k);  // row_mirror: 16-lane (row) maximum
  const uint32_t hi = (uint32_t)(k >> 32), lo = (uint32_t)k;
  uint64_t b = make_key(0, 0);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    // (readlane returns int: widen through uint32_t, not by sign extension)
    const uint64_t o = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane(hi, 16 * r) << 32) |
                       (uint32_t)__builtin_amdgcn_readlane(lo, 16 * r);
    b = r == 0 ? o : key_max(b, o);
  }
  return b;
}

// The k largest of the wave's 64 * PER_LANE keys (unique but for zeros, which
// mark padding), in descending order: lane j returns the j-th, lanes past k
// zero.  The keys are consumed.
template <int PER_LANE>
__device__ __forceinline__ uint64_t select_topk(uint64_t (&key)[PER_LANE], int k, int lane) {
  // each lane's keys in descending order (odd-even transposition sort), so
  // a round only compares the 64 lane heads and pops the winner's head
#pragma unroll
  for (int r = 0; r < PER_LANE; ++r)
#pragma unroll
    for (int i = r & 1; i + 1 < PER_LANE; i += 2) {
      const uint64_t a = key[i], b = key[i + 1];
      key[i] = key_max(a, b);
      key[i + 1] = b > a ? a : b;
    }
  uint64_t sel = 0;
  for (int j = 0; j < k; ++j) {
    const uint64_t b = wave_key_max(key[0]);
    // the winner (one lane: keys are unique) pops its head; a bit mask
    // rather than a select, which the compiler would turn into an indexed
    // read of the key array
    const uint64_t m = key[0] == b ? ~0ull : 0ull;
#pragma unroll
    for (int i = 0; i + 1 < PER_LANE; ++i) key[i] = (key[i + 1] & m) | (key[i] & ~m);
    key[PER_LANE - 1] &= ~m;
    if (lane == j) sel = b;
  }
  return sel;
}

}  // namespace moe
