// Dot products of 16 weight rows with at most 16 activation rows by one wave
// (v_mfma_f32_16x16x32_bf16; gfx950), for the few-token layer and the streamed
// MXFP4 experts.
//
// A batch is a 256-byte run of each weight row, 128 bf16, 256 e4m3fn or 512
// E2M1 values along K.  A load brings four rows' runs, 1 KB; the runs go to a
// wave-private LDS buffer and come back as fragments: A row
// m = lane % 16 is an activation row, B column n = lane % 16 a weight row, and
// lane group q = lane / 16 takes chunk 4 u + q (16 bytes) of the run for step u.
// The K order inside a step is free as long as both operands use it, so a chunk
// is 8 bf16, 16 e4m3fn or 32 E2M1 values (one scale group) and the matching
// activations.  Loads in fragment shape, 64 bytes of each of 16 rows, need no
// LDS but are half lines: 10 experts' gate and up rows at the Flash-Next shape
// took 6.7 us against 5.2 (MXFP4) and 15.9 against 12.2 us (bf16).
//
// Activation rows pass through the same buffer, which holds 16, 8 or 4 of them (a
// job has no more): one load brings 1 KB of them.  Loaded as fragments they would
// cost the address unit as much as a weight load, for 16 bytes of each of a few
// rows (MXFP4: four such loads per weight load, which bounded the kernel).
//
// One loop takes a wave through all its jobs (a job: 16 rows over a K range):
// each turn stages the batch that has arrived, asks for the next one, whichever
// job it belongs to, and multiplies.  So a compute unit's waves keep 64 KB in
// flight, and the code is small: where a wave runs a few KB, its time
// is that of the code around the loads (a three-slot ring of direct loads to LDS
// was ten times the code and slower).
#pragma once
#include "common.hpp"
#include "kernels.hpp"

namespace moe {
namespace fragdot {

constexpr int kSc1 = 16;             // cache policy: coherent across the device's L2 caches
constexpr int kNt = 2;               // non-temporal
constexpr int kLds = 16 * 256 + 256;  // a wave's buffer: runs of 16 rows, and their scale bytes (MXFP4)

// AROWS: the most activation rows of a job; 0: as many as fit a run of 16 weight
// rows.  U_: 16-byte chunks per lane and 16 rows, 4 (runs of 256 bytes) or 2 (of 128).
template <int WT, int AROWS = 0, int U_ = 4>
struct Form {
  static constexpr int G = WT == kWtMx ? 32 : WT == kWtFp8 ? 16 : 8;  // values per 16-byte chunk
  static constexpr int U = U_;
  static constexpr int KB = 4 * G * U;                                // K values per batch; U = 4: 128, 256, 512
  static constexpr int RUN = 64 * U;                                  // bytes of a weight row's run
  static constexpr int CPR = 4 * U;                                   // chunks of it
  static constexpr int WPL = 64 / CPR;                                // weight rows per load: 4 or 8
  static constexpr int NW = 16 / WPL;                                 // loads of 16 weight rows
  static constexpr int ROWS = AROWS ? AROWS : 16 * RUN / (2 * KB);    // 0: 16, 8, 4
  static constexpr int RPL = 512 / KB;                                // activation rows per load; U = 4: 4, 2, 1
  static constexpr int NL = ROWS / RPL;                               // loads of all of them
  static constexpr int BUF = 2 * KB * ROWS;                           // bytes of them
  static constexpr int LDS = BUF + 256;
  static constexpr int NS = WT == kWtMx ? 2 : KB / 128;               // scale registers of a batch
  static_assert(U == 4 || (U == 2 && WT == kWtMx), "half runs: MXFP4");
  static_assert(BUF >= 16 * RUN, "the weights pass through the same buffer");
  // Chunk c of row r lies at c ^ swizzle(r): the 16 rows of a chunk in 16 bank groups.
  static __device__ __forceinline__ int swizzle(int r) { return U == 4 ? r : (r >> 1) & 7; }
};


// bytes of n weights along K
template <int WT>
__device__ __forceinline__ int64_t wbytes(int64_t n) {
  return WT == kWtPlain ? n * 2 : WT == kWtFp8 ? n : n / 2;
}

__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00020000);
}

struct NoGate {
  __device__ void operator()() const {}
};
struct BaseRows {
  template <class J>
  __device__ int operator()(const J& j, int r) const { return j.base + r; }
};

// NB blocks of 16 weight rows of K values over [k0, kend): rows 0-7 of block b
// from w[2 b] on, rows 8-15 from w[2 b + 1] on, of which there are wrows[2 b + h]
// in each half (the others read as zeros).  scale[b]: MXFP4, the scale bytes of
// row lane / 4 (of a row there is); fp8, the scales of this lane's fragment row
// lane % 16, by K / 128.
// Activations: `rows` <= ROWS rows; this lane's fragment row is row ar < rows of
// them (results of rows that mean nothing are not used).
template <int NB>
struct Job {
  const char* w[2 * NB];
  int wrows[2 * NB];
  const void* scale[NB];
  int base, rows, ar;  // base: for the caller's row_of
  int k0, kend;
  int tag;  // for the caller
};

// Runs the jobs that next(Job&) gives until it returns false, and after(tag,
// acc) with each one's products A [16 rows] x W [16 rows]^T, NB blocks.  abase: the
// activation rows, K values each, `abytes` in all; row_of(job, r) is the index of
// a job's row r < rows.  k0 is a multiple of 128 (fp8, MXFP4: whole scale blocks and
// aligned scale bytes) or of 8 (bf16), K of 128 (fp8), 32 (MXFP4) or 8.
// lds: the wave's Form::LDS bytes.  gate(): called once if there is a job, after
// the first weights have been asked for and before any activation is.
// PAIR: a product's activation row is the sum of the rows ar and ar + 1 (a value in two
// bf16 parts).
template <int WT, int NB, int AUXA, int AROWS = 0, int U_ = 4, bool PAIR = false, class Rows, class Next, class After, class Gate>
__device__ __forceinline__ void run(const void* abase, uint32_t abytes, int K, int lane, char* lds, Rows row_of,
                                    Next next, After after, Gate gate) {
  using F = Form<WT, AROWS, U_>;
  constexpr int G = F::G, U = F::U;
  constexpr uint32_t kNone = 0x80000000u;  // past any weight rows: reads as zeros, fetches nothing
  constexpr uint32_t kOut = 0xFFFFFFF0u;   // past any activations
  constexpr int LPR = 64 / F::RPL;         // lanes per activation row
  const int q = lane >> 4, n = lane & 15;
  const uint32_t rowb = (uint32_t)wbytes<WT>(K);
  const __amdgpu_buffer_rsrc_t ares = resource(abase, abytes);
  const int wr = lane / F::CPR, wc = lane % F::CPR;  // this lane's row and chunk of a weight load
  Job<NB> job{};
  bool have = true, fresh = true, pending = false, first = true;  // fresh: a new job is due
  int kb = 0;
  // the batch in flight
  u32x4 t[NB][F::NW], at[F::NL];
  uint32_t sd[NB][F::NS], shift[NB];
  uint32_t aoff[F::NL];
  // the batch being multiplied
  int c_rows = 0, c_ar = 0, c_kb = 0, c_tag = 0;
  bool c_last = false;
  f32x4 acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (;;) {
    u32x4 wv[NB][U];
    uint32_t sv[NB][U];
    if (pending) {
      // through LDS (one wave's LDS operations are executed in order)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int i = 0; i < F::NW; ++i)
          *reinterpret_cast<u32x4*>(lds + (i * F::WPL + wr) * F::RUN + ((wc ^ F::swizzle(i * F::WPL + wr)) << 4)) =
              t[b][i];
#pragma unroll
        for (int u = 0; u < U; ++u)
          wv[b][u] = *reinterpret_cast<const u32x4*>(lds + n * F::RUN + (((4 * u + q) ^ F::swizzle(n)) << 4));
        if constexpr (WT == kWtMx) {
          *reinterpret_cast<uint32_t*>(lds + F::BUF + (lane >> 2) * 4 * U + (lane & (U - 1)) * 4) =
              __builtin_amdgcn_alignbyte(sd[b][1], sd[b][0], shift[b]);
#pragma unroll
          for (int u = 0; u < U; ++u)
            sv[b][u] = (*reinterpret_cast<const uint32_t*>(lds + F::BUF + n * 4 * U + 4 * u) >> (8 * q)) & 255u;
          if (c_kb + F::KB > K) {  // what lies behind the row's scales is not one of them
#pragma unroll
            for (int u = 0; u < U; ++u) sv[b][u] = c_kb + 4 * G * u + G * q < K ? sv[b][u] : 0u;
          }
        } else if constexpr (WT == kWtFp8) {
#pragma unroll
          for (int h = 0; h < F::NS; ++h) sv[b][h] = sd[b][h];
        }
      }
#pragma unroll
      for (int i = 0; i < F::NL; ++i)
        if (i * F::RPL < c_rows) *reinterpret_cast<u32x4*>(lds + i * 1024 + lane * 16) = at[i];
    }
    // ask for the next batch
    if (fresh) {
      have = next(job);
      kb = job.k0;
    }
    const bool issued = have;
    auto offsets = [&] {  // of a new job's activation rows
#pragma unroll
      for (int i = 0; i < F::NL; ++i)
        if (i * F::RPL < job.rows) {
          const int r = i * F::RPL + lane / LPR;
          const int at = r < job.rows ? r : 0;
          aoff[i] = r < job.rows ? (uint32_t)row_of(job, at) * (uint32_t)K * 2u + 16u * (uint32_t)(lane % LPR)
                                 : kNone;  // (some place or none: its results are not used)
        }
    };
    // Before the weights where a row's index may come from memory (the callers with
    // half runs): its wait is for every load before it.
    if (U == 2 && have && fresh) offsets();
    int n_rows = 0, n_ar = 0, n_kb = 0, n_tag = 0;
    bool n_last = false;
    if (have) {
      const uint32_t k0 = (uint32_t)wbytes<WT>(kb) + (uint32_t)wc * 16u, k1 = (uint32_t)wbytes<WT>(job.kend);
      const uint32_t v = k0 < k1 ? (uint32_t)wr * rowb + k0 : kNone;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const __amdgpu_buffer_rsrc_t w0 = resource(job.w[2 * b], (uint32_t)job.wrows[2 * b] * rowb);
        const __amdgpu_buffer_rsrc_t w1 = resource(job.w[2 * b + 1], (uint32_t)job.wrows[2 * b + 1] * rowb);
#pragma unroll
        for (int i = 0; i < F::NW; ++i)
          t[b][i] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(i < F::NW / 2 ? w0 : w1,
                                                           v + (uint32_t)(i % (F::NW / 2) * F::WPL) * rowb, 0, kNt));
      }
      if constexpr (WT == kWtMx) {
        // The 4 scale bytes of chunks 4 (lane % U) .. + 3 of a run: a dword, or, with
        // rows that are no multiple of 4 scales, its parts in two aligned dwords
        // (each holding a byte of the row, so that none lies outside the tensor).
        const int groups = K >> 5;
        int i = (kb >> 5) + 4 * (lane & (U - 1));
        i = i < groups ? i : 0;
        const int e = i + 3 < groups ? i + 3 : groups - 1;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uintptr_t row = reinterpret_cast<uintptr_t>(job.scale[b]);
          shift[b] = (uint32_t)row & 3u;
          sd[b][0] = *reinterpret_cast<const uint32_t*>((row + i) & ~(uintptr_t)3);
          sd[b][1] = 0;
          if (groups & 3) sd[b][1] = *reinterpret_cast<const uint32_t*>((row + e) & ~(uintptr_t)3);
        }
      }
      if constexpr (WT == kWtFp8) {  // two 128-wide blocks
        const int last = K / 128 - 1, i = kb / 128;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int h = 0; h < F::NS; ++h)
            sd[b][h] = static_cast<const uint32_t*>(job.scale[b])[i + h < last ? i + h : last];
      }
      if (first) gate();
      first = false;
      if (U != 2 && fresh) offsets();
#pragma unroll
      for (int i = 0; i < F::NL; ++i)
        if (i * F::RPL < job.rows)
          at[i] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                         ares, kb + (lane % LPR) * 8 < job.kend ? aoff[i] + 2u * (uint32_t)kb : kOut, 0, AUXA));
      n_rows = job.rows, n_ar = job.ar, n_kb = kb, n_tag = job.tag;
      kb += F::KB;
      fresh = n_last = kb >= job.kend;
    }
    if (pending) {
      const char* const arow = lds + 2 * (c_ar * F::KB + G * q);
      constexpr int NP = PAIR ? 2 : 1;
      auto act = [&](int k, int p) { return frag(*reinterpret_cast<const u32x4*>(arow + 2 * (k + p * F::KB))); };
      if constexpr (WT == kWtPlain) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const bf16x8 x = act(4 * G * u, p);
#pragma unroll
            for (int b = 0; b < NB; ++b)
              acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, frag(wv[b][u]), acc[b], 0, 0, 0);
          }
      } else if constexpr (WT == kWtFp8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f32x4 part[NB];
#pragma unroll
          for (int b = 0; b < NB; ++b) part[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int u = 2 * h; u < 2 * h + 2; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              bf16x8 w[NB];
#pragma unroll
              for (int b = 0; b < NB; ++b)
                w[b] = frag(fp8x8_to_bf16x8_exact(u32x2{wv[b][u][2 * j], wv[b][u][2 * j + 1]}));
#pragma unroll
              for (int p = 0; p < NP; ++p) {
                const bf16x8 x = act(4 * G * u + 8 * j, p);
#pragma unroll
                for (int b = 0; b < NB; ++b)
                  part[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w[b], part[b], 0, 0, 0);
              }
            }
#pragma unroll
          for (int b = 0; b < NB; ++b) acc[b] += __uint_as_float(sv[b][h]) * part[b];
        }
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (U == 2 && u > 0 && c_kb + 4 * G * u >= K) break;  // (nothing behind the rows' ends)
          float f[NB];
#pragma unroll
          for (int b = 0; b < NB; ++b) f[b] = e8m0(sv[b][u]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            bf16x8 w[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) w[b] = frag(mx8_to_bf16x8(wv[b][u][j], f[b]));
#pragma unroll
            for (int p = 0; p < NP; ++p) {
              const bf16x8 x = act(4 * G * u + 8 * j, p);
#pragma unroll
              for (int b = 0; b < NB; ++b) acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w[b], acc[b], 0, 0, 0);
            }
          }
        }
      }
      if (c_last) {
        after(c_tag, acc);
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
    }
    if (!issued) break;
    pending = true;
    c_rows = n_rows, c_ar = n_ar, c_kb = n_kb, c_tag = n_tag, c_last = n_last;
  }
}

}  // namespace fragdot
}  // namespace moe
