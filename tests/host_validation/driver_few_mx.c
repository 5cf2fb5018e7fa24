/* Host-side validation of the few-token layer, the MXFP4 conversions and the
 * MXFP4 problems of every entry point that takes expert weights, built and run
 * as driver.c is.  Checks: a seeded sweep of shapes, dtypes, flags, pointers and
 * strides; then, only where no device is visible, whole calls with valid
 * arguments, whose launches fail: the host code between the checks and the
 * launches (work lists' sizes, grids, the choice of kernels) runs under the
 * sanitizers and every such call returns MOE_ERR_HIP. */
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
static uint64_t rng_state = 0x2545f4914f6cdd1dull;
static uint64_t next_u64(void) {
  uint64_t z = (rng_state += 0x9e3779b97f4a7c15ull);
  z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ull;
  z = (z ^ (z >> 27)) * 0x94d049bb133111ebull;
  return z ^ (z >> 31);
}
static int64_t pick(const int64_t* v, int n) { return v[next_u64() % (uint64_t)n]; }
#define PICK(arr) pick(arr, (int)(sizeof(arr) / sizeof(arr[0])))
#define FIELD(edge, good) (next_u64() % 8 == 0 ? PICK(edge) : PICK(good))

static const int64_t eTs[] = {-1, 0, 15, 16, 17, 31, 32, 33, 1 << 20, ((int64_t)1 << 31) - 1, INT64_MAX, INT64_MIN};
static const int64_t gTs[] = {0, 1, 2, 7, 12, 16, 17, 24, 32, 33, 300, 4096, 65536};
static const int64_t eHs[] = {-32, 0, 8, 32, 40, 96, 1184, 8224, 1 << 24, (1 << 24) + 32, INT64_MAX};
static const int64_t gHs[] = {32, 96, 128, 1184, 2560, 8192};
static const int64_t eEs[] = {-1, 0, 1, 1023, 1024, 1025, INT64_MAX};
static const int64_t gEs[] = {1, 12, 60, 64, 512, 1024};
static const int64_t eks[] = {-1, 0, 1, 63, 64, 65, INT64_MAX};
static const int64_t gks[] = {1, 2, 8, 10, 64};
static const int64_t eIs[] = {-32, 0, 32, 72, 416, 1 << 24, INT64_MAX};
static const int64_t gIs[] = {32, 128, 352, 640, 2048};
static const int64_t eIss[] = {-8, 0, 8, 40, 1 << 24, INT64_MAX};
static const int64_t gIss[] = {0, 0, 72, 640, 2048};
static const int64_t dts[] = {-1, 0, 1, 2, 3, 4, 1000};
static const int64_t sbs[] = {0, 16, 32, 64, 128, -32};

static _Alignas(256) unsigned char buf[4096];

static void random_problem(moe_problem* p) {
  memset(p, 0, sizeof(*p));
  p->T = FIELD(eTs, gTs);
  p->H = FIELD(eHs, gHs);
  p->E = FIELD(eEs, gEs);
  p->k = FIELD(eks, gks);
  p->I = FIELD(eIs, gIs);
  p->I_shared = FIELD(eIss, gIss);
  p->act_dtype = (int32_t)(next_u64() % 16 == 0 ? PICK(dts) : MOE_BF16);
  p->w_dtype = (int32_t)(next_u64() % 8 == 0 ? PICK(dts) : 1 + (int32_t)(next_u64() % 3));
  if (next_u64() % 2) p->w_dtype = MOE_MXFP4;
  p->scale_block = (int32_t)(next_u64() % 8 == 0 ? PICK(sbs) : p->w_dtype == MOE_MXFP4 ? 32 : 128);
  p->flags = (uint32_t)(next_u64() % 8 == 0 ? next_u64() : next_u64() & 0x1f);
}

/* every pointer at buf + off, every stride the given one */
static void all_weights(moe_weights* w, int off, int64_t stride) {
  memset(w, 0, sizeof(*w));
  w->w_router = w->w_gate = w->w_up = w->w_down = buf + off;
  w->s_gate = w->s_up = w->s_down = buf + off;
  w->sh_gate = w->sh_up = w->sh_down = w->sh_gate_w = buf + off;
  w->stride_gate = w->stride_up = w->stride_down = stride;
}

static moe_status few(const moe_problem* p, const moe_weights* w, void* x, void* out, void* ws, size_t n) {
  return moe_layer_forward_few(p, w, x, out, NULL, NULL, ws, n, NULL);
}

static void few_checks(const moe_problem* p) {
  const moe_status v = moe_validate(p);
  const size_t n = moe_few_workspace_bytes(p);
  const int takes = v == MOE_OK && p->act_dtype == MOE_BF16 && p->T <= MOE_FEW_MAX_TOKENS;
  EXPECT((n > 0) == takes && n % 256 == 0, "few workspace %zu", n);
  moe_weights w;
  all_weights(&w, 0, 0);
  if (!takes) {
    const moe_status st = few(p, &w, buf, buf, buf, SIZE_MAX);
    EXPECT(st == (v != MOE_OK ? v : MOE_ERR_UNSUPPORTED), "few: status %d of a problem that it does not take", (int)st);
    return;
  }
  moe_problem q = *p;
  q.T = p->T / 2;
  EXPECT(moe_few_workspace_bytes(&q) <= n, "few workspace not monotone in T");
  if (p->T == 0) {
    EXPECT(few(p, NULL, NULL, NULL, NULL, 0) == MOE_OK, "few: an empty batch");
    return;
  }
  EXPECT(few(p, NULL, buf, buf, buf, n) == MOE_ERR_NULL, "few: no weights");
  EXPECT(few(p, &w, NULL, buf, buf, n) == MOE_ERR_NULL, "few: no x");
  EXPECT(few(p, &w, buf, NULL, buf, n) == MOE_ERR_NULL, "few: no out");
  EXPECT(few(p, &w, buf, buf, NULL, n) == MOE_ERR_NULL, "few: no workspace");
  EXPECT(few(p, &w, buf, buf, buf, n - 1) == MOE_ERR_WORKSPACE, "few: short workspace");
  EXPECT(few(p, &w, buf, buf, buf + 16, n) == MOE_ERR_ALIGN, "few: workspace alignment");
  EXPECT(few(p, &w, buf + 8, buf, buf, n) == MOE_ERR_ALIGN, "few: x alignment");
  EXPECT(few(p, &w, buf, buf + 2, buf, n) == MOE_ERR_ALIGN, "few: out alignment");
  all_weights(&w, 1 + (int)(next_u64() % 15), 0);
  EXPECT(few(p, &w, buf, buf, buf, n) == MOE_ERR_ALIGN, "few: weights' alignment");
  all_weights(&w, 0, -32);
  EXPECT(few(p, &w, buf, buf, buf, n) == MOE_ERR_SHAPE, "few: negative stride");
}

/* MXFP4 strides and scales, through every call that takes expert weights */
static void mx_checks(const moe_problem* p) {
  if (moe_validate(p) != MOE_OK || p->w_dtype != MOE_MXFP4 || p->T == 0) return;
  const size_t n = moe_workspace_bytes(p);
  const int32_t* idx = (const int32_t*)buf;
  moe_weights w;
  moe_status want = MOE_ERR_NULL;
  switch (next_u64() % 4) {
    case 0: all_weights(&w, 0, 16 + 32 * (int64_t)(next_u64() % 1000)); want = MOE_ERR_ALIGN; break;
    case 1: all_weights(&w, 0, -32); want = MOE_ERR_SHAPE; break;
    case 2: all_weights(&w, 0, 0); w.s_down = NULL; break;
    default: all_weights(&w, 0, 0); w.s_gate = buf + 1 + next_u64() % 15; want = MOE_ERR_ALIGN; break;
  }
  EXPECT(moe_expert_ffn(p, &w, buf, idx, idx, buf, NULL, buf, n, NULL) == want, "mx expert_ffn");
  EXPECT(moe_expert_gate_up(p, &w, buf, idx, idx, buf, NULL, buf, n, NULL) == want, "mx gate_up");
  EXPECT(moe_expert_down(p, &w, idx, buf, NULL, buf, NULL, buf, n, NULL) == want, "mx down");
  EXPECT(moe_layer_forward(p, &w, buf, buf, NULL, NULL, buf, n, NULL) == want, "mx layer");
  EXPECT(moe_layer_forward_noalloc(p, &w, buf, buf, NULL, NULL, NULL) == want, "mx noalloc");
  all_weights(&w, 0, 32);
  EXPECT(moe_expert_ffn(p, &w, buf, idx, idx, buf, NULL, buf, n - 1, NULL) == MOE_ERR_WORKSPACE, "mx workspace");
}

static void conversion_checks(void) {
  static const int64_t rows[] = {-1, 0, 1, 37, 1 << 20, (int64_t)1 << 42, INT64_MAX, INT64_MIN};
  static const int64_t Ks[] = {INT64_MIN, -32, 0, 1, 16, 32, 48, 672, 8192, (int64_t)1 << 31, (int64_t)1 << 42, INT64_MAX};
  static const int64_t strides[] = {-1, 0, 32, 36, 40, 680, 8192, ((int64_t)1 << 31) - 32, (int64_t)1 << 31, INT64_MAX};
  for (int it = 0; it < 100000; ++it) {
    const int64_t r = PICK(rows), K = PICK(Ks);
    const int64_t s = next_u64() % 2 ? K : PICK(strides);
    const int32_t dt = (int32_t)PICK(dts);
    const int bytes = dt == MOE_F32 ? 4 : 2;
    const int shape = r >= 0 && K >= 1 && s >= K && s < (int64_t)1 << 31 && r < (int64_t)1 << 42 &&
                      (r == 0 || K <= ((int64_t)1 << 42) / r);
    moe_status want = !shape ? MOE_ERR_SHAPE : K % 32 ? MOE_ERR_UNSUPPORTED : s * bytes % 16 ? MOE_ERR_ALIGN : MOE_OK;
    const int types = dt == MOE_F32 || dt == MOE_BF16;
    /* (with sizes that are right: no pointers, or one that is misaligned) */
    if (want == MOE_OK && r > 0) want = MOE_ERR_NULL;
    EXPECT(moe_mx_quantize(NULL, dt, r, K, s, buf, buf, NULL) == (types ? want : MOE_ERR_DTYPE), "quantize %lld %lld %lld",
           (long long)r, (long long)K, (long long)s);
    if (types && want == MOE_ERR_NULL) {
      EXPECT(moe_mx_quantize(buf + 2, dt, r, K, s, buf, buf, NULL) == MOE_ERR_ALIGN, "quantize: w");
      EXPECT(moe_mx_quantize(buf, dt, r, K, s, buf + 8, buf, NULL) == MOE_ERR_ALIGN, "quantize: codes");
      EXPECT(moe_mx_quantize(buf, dt, r, K, s, buf, NULL, NULL) == MOE_ERR_NULL, "quantize: scales");
    }
    if (dt != MOE_F32) {
      EXPECT(moe_mx_dequantize(buf, buf, r, K, NULL, s, NULL) == want, "dequantize %lld %lld %lld", (long long)r,
             (long long)K, (long long)s);
      if (want == MOE_ERR_NULL) {
        EXPECT(moe_mx_dequantize(buf, buf, r, K, buf + 2, s, NULL) == MOE_ERR_ALIGN, "dequantize: w");
        EXPECT(moe_mx_dequantize(buf + 4, buf, r, K, buf, s, NULL) == MOE_ERR_ALIGN, "dequantize: codes");
        EXPECT(moe_mx_dequantize(NULL, buf, r, K, buf, s, NULL) == MOE_ERR_NULL, "dequantize: no codes");
      }
    }
  }
}

/* Valid calls without a device: up to the launches, which fail. */
static long launches(void) {
  static const uint32_t flags[] = {0, MOE_FLAG_FORCE_GEMM, MOE_FLAG_FORCE_STREAM, MOE_FLAG_GEMM_TILE_256,
                                   MOE_FLAG_PAGE_ROUTING};
  long calls = 0;
  for (int it = 0; it < 400; ++it) {
    moe_problem p;
    do random_problem(&p);
    while (moe_validate(&p) != MOE_OK || p.T == 0 || p.act_dtype != MOE_BF16);
    p.flags = flags[next_u64() % 5];
    moe_weights w;
    all_weights(&w, 0, 0);
    const size_t n = moe_workspace_bytes(&p);
    const int32_t* idx = (const int32_t*)buf;
    void* ysh = next_u64() % 2 ? buf : NULL;
    moe_status st[6];
    st[0] = moe_expert_ffn(&p, &w, buf, idx, idx, buf, ysh, buf, n, NULL);
    st[1] = moe_expert_gate_up(&p, &w, buf, idx, idx, buf, ysh, buf, n, NULL);
    st[2] = moe_expert_down(&p, &w, idx, buf, ysh, buf, ysh, buf, n, NULL);
    st[3] = moe_layer_forward(&p, &w, buf, buf, NULL, NULL, buf, n, NULL);
    st[4] = p.T <= MOE_FEW_MAX_TOKENS ? few(&p, &w, buf, buf, buf, moe_few_workspace_bytes(&p)) : MOE_ERR_HIP;
    st[5] = moe_mx_dequantize(buf, buf, p.E * p.I, p.H / 32 * 32 + 32, buf, p.H / 32 * 32 + 32, NULL);
    for (int i = 0; i < 6; ++i, ++calls) EXPECT(st[i] == MOE_ERR_HIP, "call %d without a device: status %d", i, (int)st[i]);
  }
  return calls;
}

int main(void) {
  EXPECT(moe_few_workspace_bytes(NULL) == 0, "few_workspace_bytes(NULL)");
  EXPECT(few(NULL, NULL, NULL, NULL, NULL, 0) == MOE_ERR_NULL, "few(NULL)");
  long valid = 0, mx = 0, small = 0;
  for (int it = 0; it < 100000; ++it) {
    moe_problem p;
    random_problem(&p);
    const int ok = moe_validate(&p) == MOE_OK;
    valid += ok;
    mx += ok && p.w_dtype == MOE_MXFP4;
    small += moe_few_workspace_bytes(&p) > 0;
    few_checks(&p);
    mx_checks(&p);
  }
  EXPECT(mx > 1000 && small > 1000, "the sweep hit %ld MXFP4 problems and %ld of few tokens", mx, small);
  conversion_checks();
  int devices = 0;
  const int status = hipGetDeviceCount(&devices);
  const long calls = status != 0 || devices == 0 ? launches() : 0;
  printf("valid %ld mxfp4 %ld few %ld calls without a device %ld failures %d\n", valid, mx, small, calls, failures);
  return failures ? 1 : 0;
}
