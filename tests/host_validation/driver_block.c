/* Host-side validation of the calls around experts of the caller's own, built
 * and run as driver.c is.  A seeded sweep of problems, pointers and workspaces;
 * then, only where no device is visible, every valid problem's calls with valid
 * arguments: the launches fail, and the host code before them (the choice of
 * tiles, grids, workspace sizes) runs under the sanitizers and the call returns
 * MOE_ERR_HIP. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "moe_mi355x.h"

int hipGetDeviceCount(int* count); /* the HIP runtime that the library is linked with */

static int failures = 0;
#define EXPECT(cond, ...)                                   \
  do {                                                      \
    if (!(cond)) {                                          \
      if (failures < 20) {                                  \
        fprintf(stderr, "line %d: ", __LINE__);             \
        fprintf(stderr, __VA_ARGS__);                       \
        fprintf(stderr, "\n");                              \
      }                                                     \
      ++failures;                                           \
    }                                                       \
  } while (0)

/* splitmix64 (Steele, Lea and Flood, "Fast splittable pseudorandom number
 * generators", 2014) */
static uint64_t rng_state = 0x9b1a615d3fa1c0deull;
static uint64_t next_u64(void) {
  uint64_t z = (rng_state += 0x9e3779b97f4a7c15ull);
  z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ull;
  z = (z ^ (z >> 27)) * 0x94d049bb133111ebull;
  return z ^ (z >> 31);
}
static int64_t pick(const int64_t* v, int n) { return v[next_u64() % (uint64_t)n]; }
#define PICK(arr) pick(arr, (int)(sizeof(arr) / sizeof(arr[0])))
#define FIELD(edge, good) (next_u64() % 16 == 0 ? PICK(edge) : PICK(good))

static const int64_t edge[] = {INT64_MIN, -1, 0, 3, (1 << 17) + 8, 1 << 24, INT32_MAX, (int64_t)1 << 40, INT64_MAX};
static const int64_t rows[] = {0, 1, 2, 16, 17, 100, 777, 4096, 40960, (1 << 24) - 1};
static const int64_t widths[] = {8, 64, 520, 640, 1416, 2560, 8192, 16384, 1 << 17};
static const int64_t groups[] = {1, 1, 2, 60, 512, 1024};
static const int64_t tokens[] = {0, 1, 3, 64, 777, 4096, 8192, 1 << 27};
static const int64_t small[] = {-1, 0, 1, 2, 3, 4, 5, 1000};
static const int64_t strides[] = {-8, 0, 0, 4, 8, 64, 1 << 20, (1 << 20) + 4, (int64_t)1 << 30, (int64_t)1 << 40,
                                  ((int64_t)1 << 40) + 8, INT64_MAX};

static _Alignas(256) unsigned char buf[4096];
static void* const P = buf;
static int no_device;
static long calls;

/* A call that passed its checks: with no device the launch fails. */
static void launched(moe_status st, const char* what) {
  ++calls;
  EXPECT(st == MOE_ERR_HIP, "%s: %d", what, st);
}

static void norms(void) {
  moe_norm_problem p;
  memset(&p, 0, sizeof(p));
  p.T = FIELD(edge, tokens);
  p.H = FIELD(edge, widths);
  p.dtype = next_u64() % 16 == 0 ? (int32_t)PICK(small) : next_u64() % 2 ? MOE_BF16 : MOE_F32;
  p.gate = next_u64() % 16 == 0 ? (int32_t)PICK(small) : (int32_t)(next_u64() % 4);
  p.eps = next_u64() % 32 == 0 ? (next_u64() % 2 ? -1.f : NAN) : 1e-6f;
  p.resid_scale = next_u64() % 32 == 0 ? INFINITY : 0.5f;
  const size_t ws = moe_block_norm_workspace_bytes(&p);
  const moe_status st = moe_block_norm(&p, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL);
  if (ws == 0) {
    EXPECT(st != MOE_OK && st != MOE_ERR_NULL && st != MOE_ERR_HIP, "norm of an invalid problem: %d", st);
    return;
  }
  EXPECT(st == (p.T == 0 ? MOE_OK : MOE_ERR_NULL), "norm without tensors: %d", st);
  EXPECT(ws % 256 == 0 && ws <= ((size_t)256 * 3 * 16384 * 4 + 256), "norm workspace %zu", ws);
  if (p.T == 0 || !no_device) return;
  void* gate = p.gate == MOE_GATE_NONE ? NULL : P;
  const int post = next_u64() % 2;
  launched(moe_block_norm(&p, P, P, post ? P : NULL, gate, P, P, P, NULL), "norm");
  launched(moe_block_norm_backward(&p, P, P, P, P, post ? P : NULL, gate, P, P, P, post ? P : NULL, gate, P, P, ws, NULL),
           "norm gradients");
  EXPECT(moe_block_norm_backward(&p, P, P, P, P, NULL, gate, P, P, P, NULL, gate, P, P, ws - 1, NULL) == MOE_ERR_WORKSPACE,
         "short workspace");
  EXPECT(moe_block_norm_backward(&p, P, P, P, P, NULL, gate, P, P, P, NULL, gate, P, buf + 16, ws, NULL) == MOE_ERR_ALIGN,
         "workspace's alignment");
  EXPECT(moe_block_norm_backward(&p, P, P, P, P, NULL, gate, P, P, P, NULL, gate, P, NULL, ws, NULL) == MOE_ERR_NULL,
         "no workspace");
}

static void linears(void) {
  moe_linear_problem p;
  memset(&p, 0, sizeof(p));
  p.rows = FIELD(edge, rows);
  p.K = FIELD(edge, widths);
  p.N = FIELD(edge, widths);
  p.groups = FIELD(edge, groups);
  p.w_stride = next_u64() % 4 == 0 ? PICK(strides) : 0;
  p.dtype = next_u64() % 16 == 0 ? (int32_t)PICK(small) : next_u64() % 2 ? MOE_BF16 : MOE_F32;
  p.act = next_u64() % 16 == 0 ? (int32_t)PICK(small) : (int32_t)(next_u64() % 3);
  const size_t ws = moe_linear_workspace_bytes(&p);
  const moe_status st = moe_linear(&p, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL);
  if (ws == 0) {
    EXPECT(st != MOE_OK && st != MOE_ERR_NULL && st != MOE_ERR_HIP, "linear of an invalid problem: %d", st);
    return;
  }
  EXPECT(st == (p.rows == 0 ? MOE_OK : MOE_ERR_NULL), "linear without tensors: %d", st);
  EXPECT(ws >= (size_t)p.rows * p.N * (p.dtype == MOE_F32 ? 4 : 2) && ws % 256 == 0, "linear workspace %zu", ws);
  if (!no_device) return;
  if (p.rows) {
    launched(moe_linear(&p, P, P, P, P, P, P, P, P, NULL), "linear");
    if (p.groups > 1)
      EXPECT(moe_linear(&p, P, P, P, NULL, P, P, P, P, NULL) == MOE_ERR_NULL, "groups without offsets");
    else
      launched(moe_linear(&p, P, P, NULL, NULL, NULL, NULL, P, NULL, NULL), "dense linear");
  }
  for (int what = 1; what < 16; ++what) {
    if (p.rows == 0 && !(what & 6)) continue;
    launched(moe_linear_backward(&p, P, P, P, P, P, P, what & 1 ? P : NULL, what & 2 ? P : NULL, what & 4 ? P : NULL,
                                 what & 8 ? P : NULL, P, ws, NULL), "linear gradients");
  }
  if (p.rows)
    EXPECT(moe_linear_backward(&p, P, P, P, P, P, P, P, P, P, P, P, ws - 1, NULL) == MOE_ERR_WORKSPACE, "short workspace");
}

static void permutes(void) {
  static const int64_t ks[] = {1, 2, 4, 8, 10, 16, 17, 64};
  moe_problem p;
  memset(&p, 0, sizeof(p));
  p.T = FIELD(edge, tokens);
  p.H = FIELD(edge, widths);
  p.E = 64;
  p.k = PICK(ks);
  p.I = 8;
  p.act_dtype = next_u64() % 2 ? MOE_BF16 : MOE_F32;
  p.w_dtype = p.act_dtype;
  const moe_status v = moe_validate(&p), st = moe_permute(&p, NULL, NULL, NULL, NULL, NULL);
  EXPECT(st == (v != MOE_OK || p.T == 0 ? v : MOE_ERR_NULL), "permute without tensors: %d", st);
  EXPECT(moe_permute_backward(&p, NULL, NULL, NULL, NULL, NULL, NULL, NULL) == st, "permute's gradient");
  EXPECT(moe_combine_backward(&p, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL) == st, "combine's");
  if (v != MOE_OK || p.T == 0 || !no_device) return;
  launched(moe_permute(&p, P, P, next_u64() % 2 ? P : NULL, P, NULL), "permute");
  launched(moe_permute_backward(&p, P, P, P, P, P, next_u64() % 2 ? P : NULL, NULL), "permute's gradient");
  const int shared = next_u64() % 2;
  void* s = shared ? P : NULL;
  launched(moe_combine_backward(&p, P, P, P, P, s, s, P, next_u64() % 2 ? P : NULL, s, s, NULL), "combine's gradient");
}

int main(void) {
  int devices = 0;
  const int status = hipGetDeviceCount(&devices);
  no_device = status != 0 || devices == 0;
  EXPECT(moe_block_norm_workspace_bytes(NULL) == 0 && moe_linear_workspace_bytes(NULL) == 0, "workspaces of NULL");
  for (int it = 0; it < 30000; ++it) {
    norms();
    linears();
    permutes();
  }
  EXPECT(!no_device || calls > 100000, "%ld calls", calls);
  printf("calls without a device %ld failures %d\n", calls, failures);
  return failures ? 1 : 0;
}
