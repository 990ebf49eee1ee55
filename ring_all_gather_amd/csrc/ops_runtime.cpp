// Entry points of the block operators (ringag.h): argument checks, workspace and the choice of
// kernel, tile and split.  Each call enqueues one to five kernels on the caller's stream.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "context.hpp"
#include "ops.hpp"
#include "ringag.h"

using namespace ringag;

namespace {

constexpr int kMaxRows = 1 << 24;            // T
constexpr int kMaxCols = 1 << 19;            // M, F, K: tile counts stay below 2^31
constexpr int kMaxNormCols = 1 << 24;        // H
constexpr long long kMaxRowBytes = 1 << 22;  // GEMM operand rows: a tile's offsets fit 32 bits
constexpr long long kLastLevelCache = 256ll << 20;

// Pointers of a call: checked for device memory, and outputs for overlaps.
struct Buf {
  const void* p;
  size_t bytes;
  const char* name;
};

template <size_t NI, size_t NO>
int check_buffers(rag_ctx* c, const char* fn, const Buf (&in)[NI], const Buf (&out)[NO]) {
  HIPCHK(hipSetDevice(c->device));
  auto dev = [&](const Buf& b) { return !b.p || b.bytes == 0 || on_device(b.p, c->device); };
  for (const Buf& b : in)
    if (!dev(b))
      return fail(RAG_EINVAL, "%s: %s is not device memory of device %d", fn, b.name, c->device);
  for (size_t i = 0; i < NO; ++i) {
    if (!dev(out[i]))
      return fail(RAG_EINVAL, "%s: %s is not device memory of device %d", fn, out[i].name,
                  c->device);
    if (out[i].p && misaligned(out[i].p))
      return fail(RAG_EINVAL, "%s: %s must be 16-byte aligned", fn, out[i].name);
    for (const Buf& b : in)
      if (overlaps(out[i].p, out[i].bytes, b.p, b.bytes))
        return fail(RAG_EINVAL, "%s: %s must not overlap %s", fn, out[i].name, b.name);
    for (size_t j = 0; j < i; ++j)
      if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
        return fail(RAG_EINVAL, "%s: %s must not overlap %s", fn, out[i].name, out[j].name);
  }
  return RAG_OK;
}

// Bytes from the first to the last element of a [rows, cols] matrix with row stride ld.
size_t span(long long rows, long long cols, long long ld, int esz) {
  return rows > 0 ? (size_t)((rows - 1) * ld + cols) * esz : 0;
}

// At least `need` bytes in c->opsbuf.
int workspace(rag_ctx* c, size_t need) {
  if (c->opsbuf_bytes >= need) return RAG_OK;
  if (c->opsbuf && c->opsbuf_olds == rag_ctx::kOpsOld)
    return fail(RAG_ENOMEM, "the operator workspace cannot grow again (to %zu bytes)", need);
  size_t bytes = std::max({need, 2 * c->opsbuf_bytes, (size_t)1 << 20});
  void* p = nullptr;
  hipError_t e = hipMalloc(&p, bytes);
  if (e != hipSuccess && bytes > need) {
    (void)hipGetLastError();
    bytes = need;
    e = hipMalloc(&p, bytes);
  }
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return fail(RAG_ENOMEM, "cannot allocate the operator workspace (%zu bytes): %s", need,
                hipGetErrorString(e));
  }
  if (c->opsbuf) c->opsbuf_old[c->opsbuf_olds++] = c->opsbuf;
  c->opsbuf = p;
  c->opsbuf_bytes = bytes;
  return RAG_OK;
}

int check_sizes(const char* fn, int T, int N, const char* nname, int K, bool fp8) {
  const int kmul = fp8 ? 128 : 64;
  if (T < 0 || T > kMaxRows) return fail(RAG_EINVAL, "%s: T=%d outside [0, %d]", fn, T, kMaxRows);
  if (N < 1 || N > kMaxCols)
    return fail(RAG_EINVAL, "%s: %s=%d outside [1, %d]", fn, nname, N, kMaxCols);
  if (K < 1 || K > kMaxCols) return fail(RAG_EINVAL, "%s: K=%d outside [1, %d]", fn, K, kMaxCols);
  if (K % kmul)
    return fail(RAG_EINVAL, "%s: K=%d must be a multiple of %d for %s", fn, K, kmul,
                fp8 ? "fp8" : "bf16");
  return RAG_OK;
}

// The GEMM operand X: alignment and row stride.  A single row has no second one for the stride to
// lead to: whatever it is, *ldx becomes K.
int check_x(const char* fn, const void* X, long long* ldx, int T, int K, int esz) {
  if (T == 0) return RAG_OK;
  if (!X) return fail(RAG_EINVAL, "%s: X must not be NULL", fn);
  if (misaligned(X)) return fail(RAG_EINVAL, "%s: X must be 16-byte aligned", fn);
  if (T == 1) *ldx = K;
  if (*ldx < K || *ldx > kMaxRowBytes / esz || (*ldx * esz) % 16)
    return fail(RAG_EINVAL, "%s: ldx=%lld must be >= K=%d, a multiple of %d and at most %lld", fn,
                *ldx, K, 16 / esz, kMaxRowBytes / esz);
  return RAG_OK;
}

// An elementwise input [T, N]: not NULL, element-aligned, row stride at least its width (a single
// row's becomes that).
int check_rows(const char* fn, const char* name, const char* ldname, const void* p, long long* ld,
               int T, int N, int esz) {
  if (T == 0) return RAG_OK;
  if (!p) return fail(RAG_EINVAL, "%s: %s must not be NULL", fn, name);
  if (reinterpret_cast<uintptr_t>(p) % esz)
    return fail(RAG_EINVAL, "%s: %s is not aligned to its elements", fn, name);
  if (T == 1) *ld = N;
  if (*ld < N || *ld > (1ll << 31))
    return fail(RAG_EINVAL, "%s: %s=%lld must be >= %d and at most 2^31", fn, ldname, *ld, N);
  return RAG_OK;
}

int check_act(const char* fn, int act) {
  if (act < RAG_ACT_NONE || act > RAG_ACT_SILU)
    return fail(RAG_EINVAL, "%s: unknown activation %d", fn, act);
  return RAG_OK;
}

int check_scales(const char* fn, bool fp8, const float* const* s, int n) {
  for (int i = 0; i < n; ++i) {
    if (fp8 && !s[i]) return fail(RAG_EINVAL, "%s: fp8 needs a scale for every operand", fn);
    if (!fp8 && s[i])
      return fail(RAG_EINVAL, "%s: scales are only meaningful for fp8; pass NULL for bf16", fn);
    if (s[i] && (reinterpret_cast<uintptr_t>(s[i]) & 3u))
      return fail(RAG_EINVAL, "%s: scales must be 4-byte aligned", fn);
  }
  return RAG_OK;
}

#define RAG_TRY(call)         \
  do {                        \
    const int rc_ = (call);   \
    if (rc_ != RAG_OK) return rc_; \
  } while (0)

size_t align_up(size_t n) { return (n + 255) & ~(size_t)255; }
int ceil_div(int a, int b) { return (int)(((long long)a + b - 1) / b); }

// Tile and K splits of the products of one launch.  A 256x256 workgroup has a compute unit to
// itself, as has one of the four-stage 128x128 form; two of the two-stage 128x128 form share one.
struct Shape {
  int rows, cols, batches, ksteps, planes;   // planes of split sums: batches, or 2 for gate and up
  bool gated;
};
struct Plan {
  int tile = kOps256;
  int splits[2] = {1, 1}, blocks[2] = {0, 0}, whole[2] = {0, 0};
  int first = 0;                             // the product whose tiles go first
  size_t part_bytes[2] = {0, 0};
};

// Microseconds of one K stage (128 bytes of K per row), by tile, as measured at a full chip with
// the tile forced: 8192 x 8192 x 8192 on 256 x 256 tiles 772 us, four rounds of 128 stages; on two
// 128 x 128 ones per compute unit each of a pair takes 0.95 us, on one of four stages 0.50.
// Measured on bf16; fp8 plans take the same times, a stage there being twice the products at about
// twice the rate and the same bytes (3001 x 2500 x 8192: 64 stages of a half tile are 60 us by
// these, 62 measured).
constexpr double kStageUs[kOpsTiles] = {1.40, 0.95, 0.50};
constexpr double kHalfStageUs = 0.85;        // half a 256 x 256 tile, which reads 3/4 of its bytes
constexpr double kTileUs = 6.0;              // a workgroup's start and epilogue

// The time of nA workgroups of a microseconds each, then nB of b, on `slots` places that take them
// in order; *cut: how many of the nB remain for a last turn that is at most half full (they may run
// as halves of h microseconds), or 0.
double makespan(long long slots, long long nA, double a, long long nB, double b, double h,
                long long* cut) {
  *cut = 0;
  const long long fa = nA / slots, ra = nA % slots;
  double t[2] = {fa * a, (fa + 1) * a};
  const long long c[2] = {slots - ra, ra};
  while (nB > 0) {
    const int g = c[1] > 0 && t[1] < t[0] ? 1 : 0;
    if (h > 0 && 2 * nB <= c[g]) {
      *cut = nB;
      t[g] += h;
      break;
    }
    nB -= std::min(nB, c[g]);
    t[g] += b;
  }
  return c[1] > 0 ? std::max(t[0], t[1]) : t[0];
}

// `fixed`: the K splits to take, or null for the best ones.
Plan plan_gemm(const rag_ctx* c, const Shape* s, int n, const int* fixed = nullptr) {
  Plan best;
  double best_us = 1e30;
  for (int tile = 0; tile < kOpsTiles; ++tile) {
    int bi, bj;
    ops_tile_dims(tile, &bi, &bj);
    const long long slots = (long long)c->num_cus * (tile == kOps128 ? 2 : 1);
    Plan p;
    p.tile = tile;
    for (int s0 = 1; s0 <= 32; s0 *= 2)
      for (int s1 = 1; s1 <= (n > 1 ? 32 : 1); s1 *= 2) {
        const int splits[2] = {s0, s1};
        if (fixed && (s0 != fixed[0] || (n > 1 && s1 != fixed[1]))) continue;
        long long wgs[2] = {0, 0};
        double us[2] = {0, 0}, half[2] = {0, 0}, join = 0;
        bool ok = true;
        for (int i = 0; i < n; ++i) {
          ok = ok && splits[i] <= std::max(1, s[i].ksteps);
          const int cols = s[i].gated ? bj / 2 : bj;
          wgs[i] = (long long)ceil_div(s[i].rows, bi) * ceil_div(s[i].cols, cols) * s[i].batches *
                   splits[i];
          const int stages = ceil_div(s[i].ksteps, splits[i]);
          us[i] = stages * kStageUs[tile] + kTileUs;
          if (tile == kOps256) half[i] = stages * kHalfStageUs + kTileUs;
          p.part_bytes[i] = 0;
          if (splits[i] > 1) {
            const size_t part = (size_t)s[i].rows * ((s[i].cols + 3) & ~3) * s[i].planes * 4;
            p.part_bytes[i] = part * splits[i];
            join += 4.0 + 2.0 * p.part_bytes[i] / 4e6;
          }
        }
        if (!ok) continue;
        const int f = n > 1 && us[1] > us[0] ? 1 : 0;   // longest first
        const int l = n > 1 ? 1 - f : 0;
        long long cut = 0;
        const double total =
            join + (n > 1 ? makespan(slots, wgs[f], us[f], wgs[l], us[l], half[l], &cut)
                          : makespan(slots, 0, 0, wgs[0], us[0], half[0], &cut));
        if (total >= best_us) continue;
        best_us = total;
        for (int i = 0; i < 2; ++i) {
          p.splits[i] = splits[i];
          p.whole[i] = (int)(wgs[i] - (i == l ? cut : 0));
          p.blocks[i] = (int)(wgs[i] + (i == l ? cut : 0));
        }
        p.first = f;
        best = p;
      }
  }
  return best;
}

// Fills in the planned launch of product i.
void set_plan(const Plan& p, int i, const Shape& s, void* part, GemmArgs* a) {
  int bi, bj;
  ops_tile_dims(p.tile, &bi, &bj);
  if (s.gated) bj /= 2;
  a->tiles_i = ceil_div(s.rows, bi);
  a->tiles_j = ceil_div(s.cols, bj);
  a->batches = s.batches;
  a->splits = p.splits[i];
  a->blocks = p.blocks[i];
  a->whole = p.whole[i];
  a->part = (float*)part;
  a->ldp = (s.cols + 3) & ~3;
}

// The joins of the split ones among a launch's products.
int run_join(rag_ctx* c, const GemmArgs* const* a, int n, bool gated, hipStream_t stream) {
  JoinPair p = {};
  int used = 0;
  for (int i = 0; i < n; ++i) {
    if (!a[i]->blocks || a[i]->splits <= 1) continue;
    JoinArgs& j = p.part[used++];
    j.part = a[i]->part;
    j.ldp = a[i]->ldp;
    j.splits = a[i]->splits;
    j.batches = a[i]->batches;
    j.gated = gated;
    j.e = a[i]->e;
  }
  if (used) HIPCHK(launch_join(c->device, p, stream));
  return RAG_OK;
}

// Both products of a backward pass; sx.rows or sw.rows is 0 for one that is not asked for.
Plan plan_backward(const rag_ctx* c, const Shape& sx, const Shape& sw) {
  const Shape both[2] = {sx, sw};
  if (sx.rows && sw.rows) {
    // each product's splits are its own, so that its bits do not depend on whether the other one
    // is asked for (the tile does not change them: every tile adds along K in the same order)
    const int splits[2] = {plan_gemm(c, &sx, 1).splits[0], plan_gemm(c, &sw, 1).splits[0]};
    return plan_gemm(c, both, 2, splits);
  }
  const int i = sx.rows ? 0 : 1;
  Plan p = plan_gemm(c, &both[i], 1);
  if (i == 1) {
    std::swap(p.splits[0], p.splits[1]);
    std::swap(p.blocks[0], p.blocks[1]);
    std::swap(p.whole[0], p.whole[1]);
    std::swap(p.part_bytes[0], p.part_bytes[1]);
  }
  return p;
}

int run_backward(rag_ctx* c, const Plan& p, const Shape& sx, const Shape& sw, GemmArgs ax,
                 GemmArgs aw, char* parts, hipStream_t stream) {
  BackwardArgs b = {};
  set_plan(p, 0, sx, parts, &ax);
  set_plan(p, 1, sw, parts + align_up(p.part_bytes[0]), &aw);
  b.dx = ax;
  b.dw = aw;
  b.dx_first = p.first == 0;
  if (ax.blocks + aw.blocks == 0) return RAG_OK;
  HIPCHK(launch_backward_gemm(c->device, p.tile, b, stream));
  const GemmArgs* both[] = {&ax, &aw};
  return run_join(c, both, 2, false, stream);
}

constexpr long long kSmallWeight = 16 << 20;   // bytes

// The form for few rows that a forward product takes, or -1 for tiles.
int few_form(const rag_ctx* c, bool gated, bool fp8, int T, int N, int K) {
  // Few rows stream the weight (8192 x 8192 bf16: 16 rows 33 us against 40 on tiles, 32 rows 51
  // against 41), up to 32 of them where the weight is small and tiles leave most of the chip idle
  // (2048 x 2048: 8.3 us against 11.8).
  const long long w_bytes = (long long)N * K * (fp8 ? 1 : 2) * (gated ? 2 : 1);
  if (T > 32 || (T > 16 && w_bytes > kSmallWeight)) return -1;
  // Two blocks of weight rows to a workgroup, which share the tokens' loads, where the tokens are
  // many and one block each makes more workgroups than compute units.  16 rows, 8192 deep: 5120
  // columns 30.5 us, shared 24.0; 4096 columns 17.6 and 23.6 (too few workgroups); 8 rows, 8192
  // columns 30.2 and 32.6.  Gated, 8 rows: 2560 columns 25.4 and 21.4, 2048 columns 14.6 and 21.0;
  // 4 rows, 3584 columns 25.6 and 26.5.
  const bool twice = T > (gated ? 4 : 8) && N > (gated ? 8 : 16) * c->num_cus;
  return T > 16 ? kFew32 : twice ? kFew16x2 : kFew16;
}

// The products of a call, by their operands' K.
Shape forward_shape(bool gated, bool fp8, int T, int N, int K) {
  return {T, N, 1, K * (fp8 ? 1 : 2) / 128, gated ? 2 : 1, gated};
}
Shape dx_shape(bool gated, int T, int N, int K) {
  const int stages = ceil_div(N, 64);
  return {T, K, 1, gated ? 2 * stages : stages, 1, false};
}
Shape dw_shape(bool gated, int T, int N, int K) {
  return {N, K, gated ? 2 : 1, ceil_div(T, 64), gated ? 2 : 1, false};
}

int forward_kind(bool gated, bool fp8) {
  return gated ? (fp8 ? kGemmGated8 : kGemmGated) : (fp8 ? kGemmLin8 : kGemmLin);
}

int forward_product(rag_ctx* c, bool gated, bool fp8, const void* X, long long ldx, int T, int K,
                    const void* const* W, const EpiArgs& e, hipStream_t stream) {
  const int esz = fp8 ? 1 : 2;
  const int form = few_form(c, gated, fp8, T, e.cols, K);
  if (form >= 0) {
    SkinnyArgs s = {};
    s.x = X;
    s.w[0] = W[0];
    s.w[1] = gated ? W[1] : nullptr;
    s.ldx = ldx * esz;
    s.ldw = (long long)K * esz;
    s.kblocks = K * esz / 128;
    s.e = e;
    HIPCHK(launch_skinny(c->device, gated, fp8, form, s, stream));
    return RAG_OK;
  }
  GemmArgs a = {};
  a.x[0] = a.x[1] = X;
  a.y[0] = W[0];
  a.y[1] = gated ? W[1] : nullptr;
  a.ldx = ldx * esz;
  a.ldy = (long long)K * esz;
  a.ksteps = a.kseg = K * esz / 128;
  a.e = e;
  const Shape shape = forward_shape(gated, fp8, T, e.cols, K);
  const Plan plan = plan_gemm(c, &shape, 1);
  if (plan.part_bytes[0])
    RAG_TRY(workspace(c, plan.part_bytes[0]));
  set_plan(plan, 0, shape, c->opsbuf, &a);
  HIPCHK(launch_ops_gemm(c->device, forward_kind(gated, fp8), plan.tile, a, stream));
  const GemmArgs* one[] = {&a};
  return run_join(c, one, 1, gated, stream);
}

// The elementwise gradient kernel's threads across the columns and rows per slab.  A slab is at
// least what a workgroup has in flight, one row per thread or with column sums two.  There are no
// more slabs than fill the chip several times: 32 workgroups per compute unit, with column sums 4
// (8192 x 8192: 65 us, with 3 or 6 of them 76, with 8 67).  With column sums up to 256 rows are one
// slab, whose sums are the result, and 8 threads across, so that 32 rows are under way at once (256
// x 1024: 7.7 us in one launch, 9.4 in two; 512 x 1024: 13.2 and 9.4).
void grad_shape(const rag_ctx* c, bool sums, ActGradArgs* g) {
  const bool one = sums && g->rows <= 256;
  g->tx = 8;
  while (!one && g->tx < 64 && g->tx * 8 < g->cols_pad) g->tx *= 2;
  const int flight = (sums ? 2 : 1) * (256 / g->tx);
  const int across = ceil_div(g->cols_pad, g->tx * 8);
  const int want = one ? 1 : std::max(1, c->num_cus * (sums ? 4 : 32) / across);
  g->slab_rows = std::max(ceil_div(ceil_div(g->rows, want), flight), 1) * flight;
  g->slabs = ceil_div(g->rows, g->slab_rows);
}

// Thread count, register form and grid of a norm over H columns.  Forward, few rows: as many
// threads on a row as it has vectors, so that one round of loads covers it; else about 256, whose
// rows follow each other in a workgroup.  8192 columns bf16: 1 row 2.97 us of GPU time with a
// vector per thread, with four 3.63; 500 rows 5.75 and 6.45, 1000 rows 9.6 and 9.05.  16 waves per
// compute unit (16384 rows: 96.8 us, with 12 102.9, with 24 108.3); backward, whose rows take more
// registers, 8 (16384 x 1024: 24.9 us, with 4 33.6, with 16 26.5).  `narrow`: bf16 rows; the
// others' vectors take twice the registers, so they get more threads instead of more vectors.
void norm_shape(const rag_ctx* c, int H, int T, bool backward, bool narrow, int* form,
                int* threads, int* grid) {
  const int need = ceil_div(H, 8);
  int nv;
  if (backward)
    nv = need <= (narrow ? 512 : 1024) ? 1 : narrow && need > 1024 ? 4 : 2;
  else if (T < 2 * c->num_cus)
    nv = need <= 1024 ? 1 : 2;
  else
    nv = need <= 256 ? 1 : need <= 512 || !narrow ? 2 : 4;
  if (need > 2048) nv = 0;
  *form = nv == 0 ? kNorm0 : nv == 1 ? kNorm1 : nv == 2 ? kNorm2 : kNorm4;
  *threads = nv == 0 ? 1024 : (ceil_div(need, nv) + 63) & ~63;
  const int waves = backward ? 8 : 16;   // per compute unit
  *grid = std::min(T, c->num_cus * std::max(1, waves * 64 / *threads));
  // backward: a workgroup's rows follow each other, and every workgroup has column sums to write
  // and to join, so that both take equally long at rows ~ sqrt(T / 32), up to eight: of 1, 2, 3, 4
  // and 8 rows of 8192 bf16, T = 16 takes 6.6, 7.4, 8.5, 9.6, 14.0 us of GPU time, T = 143 11.8,
  // 10.1, 10.3, 10.9, 14.8, T = 400 16.3, 15.3, 14.4, 14.2, 16.6 (4096 x 1024: eight rows 13.9 us,
  // sixteen 18.4).  Whole rounds of compute units from one on (1777 x 1001 fp32: 254 workgroups
  // 13.6 us, 256 12.1; 3000 x 1001: 375 14.6, 512 13.5).  Up to four short rows go to one
  // workgroup, which then writes the sums itself (calls of 4 x 8192: 8.3 us, in two launches 10.8;
  // 8 x 8192: 11.7 and 10.8)
  if (backward && T <= 4 && need <= 1024) *grid = std::min(T, 1);
  else if (backward) {
    const int rows = std::clamp((int)std::lround(std::sqrt(T / 32.0)), 1, 8);
    const int step = ceil_div(T, rows) > c->num_cus ? c->num_cus : 8;
    *grid = std::min(*grid, ceil_div(ceil_div(T, rows), step) * step);
  }
}

int size_of(rag_dtype t) { return t == RAG_F32 ? 4 : 2; }

int norm_type(rag_dtype x, rag_dtype y, rag_dtype w) {
  const int f = w == RAG_F32 ? kNormWF : 0;
  if (x == RAG_BF16 && y == RAG_BF16) return kNormBB + f;
  if (x == RAG_F32 && y == RAG_F32) return kNormFF + f;
  if (x == RAG_F32 && y == RAG_BF16) return kNormFB + f;
  return -1;
}

int check_norm(const char* fn, int T, int H, rag_dtype x_dt, rag_dtype y_dt, rag_dtype w_dt) {
  if (T < 0 || T > kMaxRows) return fail(RAG_EINVAL, "%s: T=%d outside [0, %d]", fn, T, kMaxRows);
  if (H < 1 || H > kMaxNormCols)
    return fail(RAG_EINVAL, "%s: H=%d outside [1, %d]", fn, H, kMaxNormCols);
  if (norm_type(x_dt, y_dt, w_dt) < 0)
    return fail(RAG_EINVAL, "%s: x_dt=%d with y_dt=%d: both bf16, both fp32, or fp32 with bf16", fn,
                x_dt, y_dt);
  if (w_dt != RAG_BF16 && w_dt != RAG_F32)
    return fail(RAG_EINVAL, "%s: w_dt=%d must be RAG_BF16 or RAG_F32", fn, w_dt);
  return RAG_OK;
}

// Whether every row of H elements starts and ends at a multiple of 4 bytes.
bool word_rows(const void* p, long long ld, int H, int esz) {
  return (reinterpret_cast<uintptr_t>(p) & 3u) == 0 && (ld * esz) % 4 == 0 && (H * esz) % 4 == 0;
}

// How a norm that touches `bytes` of rows accesses them.
int norm_rows(bool words, int form, long long bytes) {
  if (!words) return kRowsOdd;
  return form != kNorm0 && bytes > kLastLevelCache ? kRowsStream : kRowsWords;
}

// Whether the products can read rows as they lie: 16-byte multiples.
bool vec_rows(const void* p, long long ld, int esz) {
  return !misaligned(p) && (ld * esz) % 16 == 0;
}

}  // namespace

extern "C" {

int layer_norm(rag_ctx* c, const void* x, long long ldx, rag_dtype x_dt, int T, int H,
               const void* weight, const void* bias, rag_dtype w_dt, float eps, void* y,
               rag_dtype y_dt, float* mean, float* rstd, void* stream) {
  const char* fn = "layer_norm";
  if (!c) return fail(RAG_EINVAL, "%s: ctx is NULL", fn);
  RAG_TRY(check_norm(fn, T, H, x_dt, y_dt, w_dt));
  if (!(eps > 0.0f)) return fail(RAG_EINVAL, "%s: eps=%g must be > 0", fn, (double)eps);
  const int ex = size_of(x_dt), ey = size_of(y_dt), ew = size_of(w_dt);
  RAG_TRY(check_rows(fn, "x", "ldx", x, &ldx, T, H, ex));
  if (!weight || (T > 0 && !y)) return fail(RAG_EINVAL, "%s: weight and y must not be NULL", fn);
  if (misaligned(weight) || misaligned(bias))
    return fail(RAG_EINVAL, "%s: weight and bias must be 16-byte aligned", fn);
  const size_t stat = (size_t)T * 4;
  const Buf in[] = {{x, span(T, H, ldx, ex), "x"},
                    {weight, (size_t)H * ew, "weight"},
                    {bias, (size_t)H * ew, "bias"}};
  const Buf out[] = {{y, (size_t)T * H * ey, "y"}, {mean, stat, "mean"}, {rstd, stat, "rstd"}};
  RAG_TRY(check_buffers(c, fn, in, out));
  if (T == 0) return RAG_OK;
  NormArgs a = {};
  a.x = x;
  a.w = weight;
  a.b = bias;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.ld_x = ldx;
  a.T = T;
  a.H = H;
  a.eps = eps;
  int form, threads, grid;
  const bool words = word_rows(x, ldx, H, ex) && word_rows(y, H, H, ey) &&
                     word_rows(weight, H, H, ew);
  norm_shape(c, H, T, false, x_dt == RAG_BF16, &form, &threads, &grid);
  HIPCHK(launch_norm(c->device, false, norm_type(x_dt, y_dt, w_dt), form,
                     norm_rows(words, form, (long long)T * H * (ex + ey)), threads, grid, a,
                     (hipStream_t)stream));
  return RAG_OK;
}

int layer_norm_backward(rag_ctx* c, const void* dy, long long lddy, rag_dtype y_dt, const void* x,
                        long long ldx, rag_dtype x_dt, int T, int H, const void* weight,
                        rag_dtype w_dt, const float* mean, const float* rstd, void* dx,
                        float* dweight, float* dbias, void* stream_v) {
  const char* fn = "layer_norm_backward";
  if (!c) return fail(RAG_EINVAL, "%s: ctx is NULL", fn);
  RAG_TRY(check_norm(fn, T, H, x_dt, y_dt, w_dt));
  const int ex = size_of(x_dt), ey = size_of(y_dt), ew = size_of(w_dt);
  RAG_TRY(check_rows(fn, "dy", "lddy", dy, &lddy, T, H, ey));
  RAG_TRY(check_rows(fn, "x", "ldx", x, &ldx, T, H, ex));
  if (!weight || !dweight || (T > 0 && (!mean || !rstd || !dx)))
    return fail(RAG_EINVAL, "%s: weight, mean, rstd, dx and dweight must not be NULL", fn);
  if (misaligned(weight)) return fail(RAG_EINVAL, "%s: weight must be 16-byte aligned", fn);
  if ((reinterpret_cast<uintptr_t>(mean) | reinterpret_cast<uintptr_t>(rstd)) & 3u)
    return fail(RAG_EINVAL, "%s: mean and rstd must be 4-byte aligned", fn);
  const Buf in[] = {{dy, span(T, H, lddy, ey), "dy"},
                    {x, span(T, H, ldx, ex), "x"},
                    {weight, (size_t)H * ew, "weight"},
                    {mean, (size_t)T * 4, "mean"},
                    {rstd, (size_t)T * 4, "rstd"}};
  const Buf out[] = {{dx, (size_t)T * H * ex, "dx"},
                     {dweight, (size_t)H * 4, "dweight"},
                     {dbias, (size_t)H * 4, "dbias"}};
  RAG_TRY(check_buffers(c, fn, in, out));
  hipStream_t stream = (hipStream_t)stream_v;
  int form, threads, grid;
  const bool words = word_rows(x, ldx, H, ex) && word_rows(dx, H, H, ex) &&
                     word_rows(dy, lddy, H, ey) && word_rows(weight, H, H, ew);
  norm_shape(c, H, T, true, x_dt == RAG_BF16, &form, &threads, &grid);
  if (T > 0) {
    RAG_TRY(workspace(c, (size_t)grid * 2 * H * 4));
    NormArgs a = {};
    a.x = x;
    a.dy = dy;
    a.w = weight;
    a.y = dx;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    // one workgroup: its sums are the result
    a.part = grid == 1 ? dweight : (float*)c->opsbuf;
    a.part_db = grid == 1 && dbias ? dbias : (float*)c->opsbuf + H;
    a.ld_x = ldx;
    a.ld_dy = lddy;
    a.T = T;
    a.H = H;
    HIPCHK(launch_norm(c->device, true, norm_type(x_dt, y_dt, w_dt), form,
                       norm_rows(words, form, (long long)T * H * (2 * ex + ey)), threads, grid, a,
                       stream));
  }
  if (grid == 1) return RAG_OK;
  ColSumArgs s = {};
  s.part = (const float*)c->opsbuf;
  s.ld = 2ll * H;
  s.slabs = grid;
  s.n0 = H;
  s.n1 = dbias ? H : 0;
  s.out0 = dweight;
  s.out1 = dbias;
  HIPCHK(launch_colsum(c->device, s, stream));
  return RAG_OK;
}

int fused_linear(rag_ctx* c, const void* X, long long ldx, int T, int K, const void* W, int M,
                 rag_dtype dt, const float* scale_X, const float* scale_W, const void* bias,
                 int act, const void* residual, long long ldr, void* Z, void* Y, void* stream) {
  const char* fn = "fused_linear";
  if (!c) return fail(RAG_EINVAL, "%s: ctx is NULL", fn);
  if (dt != RAG_BF16 && dt != RAG_FP8_E4M3) return fail(RAG_EINVAL, "%s: unknown dtype %d", fn, dt);
  const bool fp8 = dt == RAG_FP8_E4M3;
  const int esz = fp8 ? 1 : 2;
  RAG_TRY(check_sizes(fn, T, M, "M", K, fp8));
  RAG_TRY(check_act(fn, act));
  RAG_TRY(check_x(fn, X, &ldx, T, K, esz));
  if (!W || (T > 0 && !Y)) return fail(RAG_EINVAL, "%s: W and Y must not be NULL", fn);
  const float* scales[] = {scale_X, scale_W};
  RAG_TRY(check_scales(fn, fp8, scales, 2));
  if (misaligned(W) || misaligned(bias))
    return fail(RAG_EINVAL, "%s: W and bias must be 16-byte aligned", fn);
  if (residual) RAG_TRY(check_rows(fn, "residual", "ldr", residual, &ldr, T, M, 2));
  if (residual && T > 0 && ldr > kMaxRowBytes / 2)   // a tile's offsets fit 32 bits
    return fail(RAG_EINVAL, "%s: ldr=%lld must be at most %lld", fn, ldr, kMaxRowBytes / 2);
  const size_t out_bytes = (size_t)T * M * 2;
  // in place: every element of the residual is read by the thread that then writes it
  const bool in_place = residual && residual == Y && ldr == M;
  const Buf in[] = {{X, span(T, K, ldx, esz), "X"},
                    {W, (size_t)M * K * esz, "W"},
                    {bias, (size_t)M * 2, "bias"},
                    {in_place ? nullptr : residual, span(T, M, ldr, 2), "residual"},
                    {scale_X, 4, "scale_X"},
                    {scale_W, 4, "scale_W"}};
  const Buf out[] = {{Y, out_bytes, "Y"}, {Z, out_bytes, "Z"}};
  RAG_TRY(check_buffers(c, fn, in, out));
  if (T == 0) return RAG_OK;
  EpiArgs e = {};
  e.scale_x = scale_X;
  e.scale_w[0] = scale_W;
  e.bias = bias;
  e.residual = residual;
  e.z[0] = Z;
  e.out[0] = e.out[1] = Y;
  e.ld_res = ldr;
  e.ld_out = M;
  e.act = act;
  e.rows = T;
  e.cols = M;
  const void* w[] = {W};
  return forward_product(c, false, fp8, X, ldx, T, K, w, e, (hipStream_t)stream);
}

int gated_ffn(rag_ctx* c, const void* X, long long ldx, int T, int K, const void* Wg,
              const void* Wu, int F, rag_dtype dt, const float* scale_X, const float* scale_Wg,
              const float* scale_Wu, int act, void* G, void* U, void* H, void* stream) {
  const char* fn = "gated_ffn";
  if (!c) return fail(RAG_EINVAL, "%s: ctx is NULL", fn);
  if (dt != RAG_BF16 && dt != RAG_FP8_E4M3) return fail(RAG_EINVAL, "%s: unknown dtype %d", fn, dt);
  const bool fp8 = dt == RAG_FP8_E4M3;
  const int esz = fp8 ? 1 : 2;
  RAG_TRY(check_sizes(fn, T, F, "F", K, fp8));
  RAG_TRY(check_act(fn, act));
  RAG_TRY(check_x(fn, X, &ldx, T, K, esz));
  if (!Wg || !Wu || (T > 0 && !H)) return fail(RAG_EINVAL, "%s: Wg, Wu and H must not be NULL", fn);
  if (T > 0 && !G != !U) return fail(RAG_EINVAL, "%s: G and U must both be given or both NULL", fn);
  const float* scales[] = {scale_X, scale_Wg, scale_Wu};
  RAG_TRY(check_scales(fn, fp8, scales, 3));
  if (misaligned(Wg) || misaligned(Wu))
    return fail(RAG_EINVAL, "%s: Wg and Wu must be 16-byte aligned", fn);
  const size_t w_bytes = (size_t)F * K * esz, out_bytes = (size_t)T * F * 2;
  const Buf in[] = {{X, span(T, K, ldx, esz), "X"}, {Wg, w_bytes, "Wg"},
                    {Wu, w_bytes, "Wu"},            {scale_X, 4, "scale_X"},
                    {scale_Wg, 4, "scale_Wg"},      {scale_Wu, 4, "scale_Wu"}};
  const Buf out[] = {{H, out_bytes, "H"}, {G, out_bytes, "G"}, {U, out_bytes, "U"}};
  RAG_TRY(check_buffers(c, fn, in, out));
  if (T == 0) return RAG_OK;
  EpiArgs e = {};
  e.scale_x = scale_X;
  e.scale_w[0] = scale_Wg;
  e.scale_w[1] = scale_Wu;
  e.z[0] = G;
  e.z[1] = U;
  e.out[0] = e.out[1] = H;
  e.ld_out = F;
  e.act = act;
  e.rows = T;
  e.cols = F;
  const void* w[] = {Wg, Wu};
  return forward_product(c, true, fp8, X, ldx, T, K, w, e, (hipStream_t)stream);
}

int fused_linear_backward(rag_ctx* c, const void* dY, long long lddy, int T, int M, const void* X,
                          long long ldx, int K, const void* W, int act, const void* Z, void* dX,
                          void* dW, rag_dtype dw_dt, float* dbias, void* stream_v) {
  const char* fn = "fused_linear_backward";
  if (!c) return fail(RAG_EINVAL, "%s: ctx is NULL", fn);
  RAG_TRY(check_sizes(fn, T, M, "M", K, false));
  RAG_TRY(check_act(fn, act));
  RAG_TRY(check_rows(fn, "dY", "lddy", dY, &lddy, T, M, 2));
  RAG_TRY(check_x(fn, X, &ldx, T, K, 2));
  if (!dX && !dW && !dbias) return fail(RAG_EINVAL, "%s: no output is given", fn);
  if (!W) return fail(RAG_EINVAL, "%s: W must not be NULL", fn);
  if (act != RAG_ACT_NONE && T > 0 && !Z)
    return fail(RAG_EINVAL, "%s: Z must not be NULL with an activation", fn);
  if (dw_dt != RAG_BF16 && dw_dt != RAG_F32)
    return fail(RAG_EINVAL, "%s: dw_dt=%d must be RAG_BF16 or RAG_F32", fn, dw_dt);
  if (misaligned(W) || misaligned(Z))
    return fail(RAG_EINVAL, "%s: W and Z must be 16-byte aligned", fn);
  const int ew = dw_dt == RAG_F32 ? 4 : 2;
  const Buf in[] = {{dY, span(T, M, lddy, 2), "dY"},
                    {X, span(T, K, ldx, 2), "X"},
                    {W, (size_t)M * K * 2, "W"},
                    {Z, (size_t)T * M * 2, "Z"}};
  const Buf out[] = {{dX, (size_t)T * K * 2, "dX"},
                     {dW, (size_t)M * K * ew, "dW"},
                     {dbias, (size_t)M * 4, "dbias"}};
  RAG_TRY(check_buffers(c, fn, in, out));
  hipStream_t stream = (hipStream_t)stream_v;
  const int Mp = (M + 63) & ~63;
  const bool products = (dX && T > 0) || dW;
  // dY serves as dZ where there is no activation and the products can read it as it lies
  const bool direct = act == RAG_ACT_NONE && M % 64 == 0 && vec_rows(dY, lddy, 2) &&
                      lddy * 2 <= kMaxRowBytes;
  const bool make_dz = products && !direct && T > 0;
  ActGradArgs g = {};
  g.rows = T;
  g.cols = M;
  g.cols_pad = Mp;
  grad_shape(c, dbias != nullptr, &g);
  const int slabs = g.slabs;
  Shape sx = dx_shape(false, T, M, K), sw = dw_shape(false, T, M, K);
  if (!dX) sx.rows = 0;
  if (!dW) sw.rows = 0;
  const Plan plan = plan_backward(c, sx, sw);
  const size_t dz_bytes = make_dz ? align_up((size_t)T * Mp * 2) : 0;
  const size_t sum_bytes = dbias ? align_up((size_t)slabs * M * 4) : 0;
  const size_t part = align_up(plan.part_bytes[0]) + plan.part_bytes[1];
  if (dz_bytes + sum_bytes + part)
    RAG_TRY(workspace(c, dz_bytes + sum_bytes + part));
  char* ws = (char*)c->opsbuf;
  float* sums = (float*)(ws + dz_bytes);
  char* parts = ws + dz_bytes + sum_bytes;
  if (make_dz || (dbias && T > 0)) {
    g.dy = dY;
    g.z = Z;
    g.dz = make_dz ? ws : nullptr;
    g.colsum = dbias ? (slabs == 1 ? dbias : sums) : nullptr;
    g.ld_dy = lddy;
    g.ld_z = M;
    g.ld_dz = Mp;
    g.stream = (long long)T * M * 6 > kLastLevelCache;
    g.act = act;
    HIPCHK(launch_act_grad(c->device, g, stream));
  }
  if (dbias && slabs != 1) {
    ColSumArgs s = {};
    s.part = sums;
    s.ld = M;
    s.slabs = slabs;
    s.n0 = M;
    s.out0 = dbias;
    HIPCHK(launch_colsum(c->device, s, stream));
  }
  const void* dz = make_dz ? ws : dY;
  const long long lddz = (make_dz ? (long long)Mp : lddy) * 2;
  GemmArgs ax = {}, aw = {};
  ax.x[0] = ax.x[1] = dz;
  ax.ldx = lddz;
  ax.y[0] = W;
  ax.ldy = (long long)K * 2;
  ax.yk = M;
  ax.ycols = K;
  ax.ksteps = ax.kseg = sx.ksteps;
  ax.e.out[0] = ax.e.out[1] = dX;
  ax.e.ld_out = K;
  ax.e.rows = T;
  ax.e.cols = K;
  aw.x[0] = aw.x[1] = dz;
  aw.ldx = lddz;
  aw.xk = T;
  aw.xcols = Mp;
  aw.y[0] = X;
  aw.ldy = ldx * 2;
  aw.yk = T;
  aw.ycols = K;
  aw.ksteps = aw.kseg = sw.ksteps;
  aw.e.out[0] = aw.e.out[1] = dW;
  aw.e.ld_out = K;
  aw.e.out_f32 = dw_dt == RAG_F32;
  aw.e.rows = M;
  aw.e.cols = K;
  return run_backward(c, plan, sx, sw, ax, aw, parts, stream);
}

int gated_ffn_backward(rag_ctx* c, const void* dH, long long lddh, int T, int F, const void* X,
                       long long ldx, int K, const void* Wg, const void* Wu, int act,
                       const void* G, const void* U, void* dX, void* dWg, void* dWu,
                       rag_dtype dw_dt, void* stream_v) {
  const char* fn = "gated_ffn_backward";
  if (!c) return fail(RAG_EINVAL, "%s: ctx is NULL", fn);
  RAG_TRY(check_sizes(fn, T, F, "F", K, false));
  RAG_TRY(check_act(fn, act));
  RAG_TRY(check_rows(fn, "dH", "lddh", dH, &lddh, T, F, 2));
  RAG_TRY(check_x(fn, X, &ldx, T, K, 2));
  if (!dX && !dWg && !dWu) return fail(RAG_EINVAL, "%s: no output is given", fn);
  if (!dWg != !dWu) return fail(RAG_EINVAL, "%s: dWg and dWu must both be given or both NULL", fn);
  if (!Wg || !Wu || (T > 0 && (!G || !U)))
    return fail(RAG_EINVAL, "%s: Wg, Wu, G and U must not be NULL", fn);
  if (dw_dt != RAG_BF16 && dw_dt != RAG_F32)
    return fail(RAG_EINVAL, "%s: dw_dt=%d must be RAG_BF16 or RAG_F32", fn, dw_dt);
  if (misaligned(Wg) || misaligned(Wu) || misaligned(G) || misaligned(U))
    return fail(RAG_EINVAL, "%s: Wg, Wu, G and U must be 16-byte aligned", fn);
  const int ew = dw_dt == RAG_F32 ? 4 : 2;
  const size_t w_bytes = (size_t)F * K, a_bytes = (size_t)T * F * 2;
  const Buf in[] = {{dH, span(T, F, lddh, 2), "dH"}, {X, span(T, K, ldx, 2), "X"},
                    {Wg, w_bytes * 2, "Wg"},         {Wu, w_bytes * 2, "Wu"},
                    {G, a_bytes, "G"},               {U, a_bytes, "U"}};
  const Buf out[] = {{dX, (size_t)T * K * 2, "dX"},
                     {dWg, w_bytes * ew, "dWg"},
                     {dWu, w_bytes * ew, "dWu"}};
  RAG_TRY(check_buffers(c, fn, in, out));
  hipStream_t stream = (hipStream_t)stream_v;
  const int Fp = (F + 63) & ~63;
  Shape sx = dx_shape(true, T, F, K), sw = dw_shape(true, T, F, K);
  if (!dX) sx.rows = 0;
  if (!dWg) sw.rows = 0;
  const Plan plan = plan_backward(c, sx, sw);
  // [dG | dU], a row of 2 Fp each: one K-contiguous operand of dX, two K-strided ones of dW
  const size_t dz_bytes = align_up((size_t)T * 2 * Fp * 2);
  const size_t part = align_up(plan.part_bytes[0]) + plan.part_bytes[1];
  if (dz_bytes + part)
    RAG_TRY(workspace(c, dz_bytes + part));
  char* ws = (char*)c->opsbuf;
  char* parts = ws + dz_bytes;
  if (T > 0) {
    ActGradArgs g = {};
    g.dy = dH;
    g.z = G;
    g.u = U;
    g.dz = ws;
    g.ld_dy = lddh;
    g.ld_z = F;
    g.ld_dz = 2ll * Fp;
    g.rows = T;
    g.cols = F;
    g.cols_pad = Fp;
    g.stream = (long long)T * F * 10 > kLastLevelCache;
    g.act = act;
    g.gated = 1;
    grad_shape(c, false, &g);
    HIPCHK(launch_act_grad(c->device, g, stream));
  }
  GemmArgs ax = {}, aw = {};
  ax.x[0] = ax.x[1] = ws;
  ax.ldx = 4ll * Fp;
  ax.y[0] = Wg;
  ax.y[1] = Wu;
  ax.ldy = (long long)K * 2;
  ax.yk = F;
  ax.ycols = K;
  ax.ksteps = sx.ksteps;
  ax.kseg = Fp / 64;
  ax.e.out[0] = ax.e.out[1] = dX;
  ax.e.ld_out = K;
  ax.e.rows = T;
  ax.e.cols = K;
  aw.x[0] = ws;
  aw.x[1] = ws + 2ll * Fp;
  aw.ldx = 4ll * Fp;
  aw.xk = T;
  aw.xcols = Fp;
  aw.y[0] = X;
  aw.ldy = ldx * 2;
  aw.yk = T;
  aw.ycols = K;
  aw.ksteps = aw.kseg = sw.ksteps;
  aw.e.out[0] = dWg;
  aw.e.out[1] = dWu;
  aw.e.ld_out = K;
  aw.e.out_f32 = dw_dt == RAG_F32;
  aw.e.rows = F;
  aw.e.cols = K;
  return run_backward(c, plan, sx, sw, ax, aw, parts, stream);
}

int rag_ops_kernel_name(rag_ctx* c, int op, int T, int N, int K, rag_dtype dt, char* buf, int len) {
  const char* fn = "rag_ops_kernel_name";
  if (!c || !buf || len < 1) return fail(RAG_EINVAL, "%s: bad arguments", fn);
  const bool back = op == RAG_OP_FUSED_LINEAR_BACKWARD || op == RAG_OP_GATED_FFN_BACKWARD;
  const bool gated = op == RAG_OP_GATED_FFN || op == RAG_OP_GATED_FFN_BACKWARD;
  const bool fp8 = dt == RAG_FP8_E4M3;
  if (op < RAG_OP_FUSED_LINEAR || op > RAG_OP_GATED_FFN_BACKWARD || T < 1 ||
      (dt != RAG_BF16 && (!fp8 || back)))
    return fail(RAG_EINVAL, "%s: op=%d T=%d dt=%d", fn, op, T, dt);
  RAG_TRY(check_sizes(fn, T, N, "N", K, fp8));
  char name[96];
  if (back) {
    const Plan p = plan_backward(c, dx_shape(gated, T, N, K), dw_shape(gated, T, N, K));
    snprintf(buf, len, "%s dx %d/%d/%d dw %d/%d/%d",
             ops_gemm_name(kGemmBackward, p.tile, name, sizeof name), p.whole[0],
             p.blocks[0] - p.whole[0], p.splits[0], p.whole[1], p.blocks[1] - p.whole[1],
             p.splits[1]);
    return RAG_OK;
  }
  const int form = few_form(c, gated, fp8, T, N, K);
  if (form >= 0) {
    snprintf(buf, len, "%s", ops_few_name(gated, fp8, form, name, sizeof name));
    return RAG_OK;
  }
  const Shape s = forward_shape(gated, fp8, T, N, K);
  const Plan p = plan_gemm(c, &s, 1);
  snprintf(buf, len, "%s %d/%d/%d",
           ops_gemm_name(forward_kind(gated, fp8), p.tile, name, sizeof name), p.whole[0],
           p.blocks[0] - p.whole[0], p.splits[0]);
  return RAG_OK;
}

}  // extern "C"
