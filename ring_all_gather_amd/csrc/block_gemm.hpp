// The products of the block operators on the tile engine of gemm_core.hpp:
//     out[i][j] = sum_k X[i][k] Y[j][k]
// with each operand either K-contiguous (row i, then k: activations and weights of a forward pass)
// or K-strided (row k, then i: the weight of dX = dZ W, both operands of dW = dZ^T X).
//
// A K-contiguous operand is staged and read as in gemm_core.hpp.  A K-strided one is staged as it
// lies in memory, 64 rows of K by the tile's columns, and transposed on its way into the registers:
// ds_read_b64_tr_b16 gives each of 16 lanes one column of a 4 (k) x 16 block, so two of them make
// the 8 consecutive k of a 16x16x32 MFMA operand.  Nothing is transposed through memory.
//   LDS layout of a K-strided stage: row k of 2 B(columns) bytes, its 32-byte units (16 columns)
//   permuted inside each group of 8 by the key (k & 3) | ((k >> 3) & 1) << 2.  The half-wave that
//   the LDS serves at a time reads rows {0..3, 8..11} + const of one unit column, which the key
//   spreads over all 64 banks; rows of 256 or 512 bytes would otherwise share 8 of them.
//   Rows past the end of K come back as zero through the stage's descriptor, which covers exactly
//   the rows that exist, so K-strided operands have no granularity in K.
//
// What bounds it: the matrix cores under the chip's power limit, in whole rounds of tiles.
//   gated forward 8192 x 3584 (x 2) x 8192 bf16   680 to 693 us, 1390 to 1414 TFLOP/s: 896 tiles on
//                                                 256 compute units are 3.5 rounds, whose last one
//                                                 runs as half tiles (whole ones: 4 rounds)
//   gated backward 4096 x 3584 x 8192             700 us for the four products (1375 TFLOP/s) in
//                                                 one launch; two would leave two last rounds
//   linear 4096 x 4096 x 4096, GELU, Z, residual  111 us; the product alone 98.  The tiles are one
//                                                 round, so nothing runs beside its epilogue
//   fp8 3001 x 2500 x 8192                        61 us, 2000 TFLOP/s: 120 tiles, fewer than half
//                                                 the compute units, so all of them run as halves
// The backward products, whose operands are transposed on the way from LDS, run at the forward
// ones' rate.
#pragma once

#include "epilogue.hpp"
#include "gemm_core.hpp"
#include "ops.hpp"

namespace ringag {

using OpsTile256 = Tile256x256w8;                       // 8 waves of 128x64
using OpsTile256Half = TileShape<256, 128, 4, 2, 128, 3>;   // 8 waves of 64x64; a third stage fits
using OpsTile128 = TileShape<128, 128, 4, 2, 128, 2>;   // 8 waves of 32x64, two workgroups per CU
using OpsTile128Deep = TileShape<128, 128, 4, 2, 128, 4>;   // the same with four stages, one per CU

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// LDS of a workgroup: the K loop's stages, or the epilogue's pieces (each_row4).
template <class S>
constexpr int ops_lds() {
  const int pieces = S::NW * 32 * (S::TN + 4) * 4;
  return S::LDS > pieces ? S::LDS : pieces;
}

// The workgroup's tile.  The first a.whole workgroups run whole tiles; the rest, where there are
// any, run the tiles after those as two halves of the columns each, so that a last round that is at
// most half full still gives every compute unit work.  XCD x (workgroup index mod 8) takes one
// contiguous run of the tile order, which goes through bands of 8 tile rows column by column, so
// the tiles of an XCD share panels of both operands in its L2.
struct TileAt {
  int split, batch, ti, tj, half;   // half: -1 whole, else which
};
__device__ inline TileAt tile_at(const GemmArgs& a, int block) {
  const bool cut = block >= a.whole;
  const int w = cut ? block - a.whole : block;
  const int n = cut ? a.blocks - a.whole : a.whole;
  const int x = w & 7, lo = n >> 3, rest = n & 7;
  int t = x * lo + min(x, rest) + (w >> 3);
  TileAt r;
  r.half = cut ? t & 1 : -1;
  if (cut) t = a.whole + (t >> 1);
  const int per = a.tiles_i * a.tiles_j;
  const int sb = t / per;
  t -= sb * per;
  r.split = sb / a.batches;
  r.batch = sb - r.split * a.batches;
  const int band = t / (8 * a.tiles_j);
  const int in = t - band * 8 * a.tiles_j;
  const int h = min(8, a.tiles_i - band * 8);
  r.tj = in / h;
  r.ti = band * 8 + in - r.tj * h;
  return r;
}

// One operand of the K loop: B tile rows (output rows or columns), Q DMA instructions per wave and
// stage.  next() describes the following stage; issue() starts DMA instruction q of it.
template <class S, int B, int Q, bool STRIDED>
struct Operand;

template <class S, int B, int Q>
struct Operand<S, B, Q, false> {
  i32x4 r;
  uint32_t off[Q];
  uint32_t kb;
  int left;
  // `first`: row 0 of the tile at the first K stage; rows past `rows` read as zero
  __device__ void init(const char* first, long long ld, int rows, int stages, int wave, int lane) {
    const int n = min(rows, B);
    r = make_rsrc(first, (uint32_t)(n - 1) * (uint32_t)ld + (uint32_t)stages * S::BKB);
    tile_offsets<S, Q>(off, 0, n, (uint32_t)ld, wave, lane);
    kb = 0u - S::BKB;
    left = stages;
  }
  // The gated form's Y: tile rows in turns of 32 of the gate and 32 of the up weight, so that a
  // wave's 64 columns hold both products of 32 outputs.  A wave's DMA rows (8 at 64 q + 8 wave) are
  // all of one weight, the one `first` belongs to.
  static __device__ int pair_weight(int wave) { return (wave >> 2) & 1; }
  __device__ void init_pair(const char* first, long long ld, int rows, int stages, int wave,
                            int lane) {
    static_assert(S::NW == 8 && S::RPI == 8, "a wave stages rows of one weight only");
    const int n = min(rows, B / 2);
    init(first, ld, n, stages, wave, lane);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int lr = (q * S::NW + wave) * S::RPI + lane / S::SEGS;
      const int c = (lr >> 6) * 32 + (lr & 31);
      const int logical = (lane % S::SEGS) ^ swz<S::BKB>(lr);
      off[q] = c < n ? (uint32_t)c * (uint32_t)ld + (uint32_t)logical * 16u : kOOB;
    }
  }
  __device__ void next() {
    kb = left > 0 ? kb + S::BKB : kOOB;
    --left;
  }
  __device__ void issue(uint32_t lds, int q, int wave) const {
    dma16(r, lds + (uint32_t)((q * S::NW + wave) * 1024), off[q] + kb);
  }
  static __device__ bf16x8 frag(const char* tile, int row, int kk, int lane) {
    return frag16_bf16<S::BKB>(tile + row * S::BKB, kk * 4 + (lane >> 4), lane);
  }
};

template <class S, int B, int Q>
struct Operand<S, B, Q, true> {
  static constexpr int ROWB = 2 * B;              // bytes of a K row in the tile
  static constexpr int SEG = ROWB / 16;           // 16-byte segments per row
  static constexpr int RPI = 1024 / ROWB;         // K rows per DMA instruction
  static constexpr int KR = S::BKB / 2;           // K rows per stage
  i32x4 r;
  uint32_t off[Q];
  const char* p;
  const char* p_next;                             // the second K segment (or null)
  long long ld;
  uint32_t width;                                 // bytes of a row inside the operand
  int rows, rows_next, seg, left;
  static __device__ int key(int k) { return (k & 3) | (((k >> 3) & 1) << 2); }
  // `first`: column 0 of the tile at row 0 of the first segment (and of the second one); k0: first
  // stage; `cols`: columns from there that exist
  __device__ void init(const char* first, const char* second, long long ld_, int krows, int cols,
                       int k0, int kseg, int stages, int wave, int lane) {
    ld = ld_;
    width = 2u * (uint32_t)min(cols, B);
    left = stages;
    const bool one = k0 < kseg;
    const int k = one ? k0 : k0 - kseg;
    p = (one ? first : second) + (long long)k * KR * ld;
    rows = krows - k * KR;
    seg = one ? kseg - k0 : 0x7fffffff;
    p_next = second;
    rows_next = krows;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int kr = (q * S::NW + wave) * RPI + lane / SEG;
      const int s = lane % SEG;
      const uint32_t col = (uint32_t)((((s >> 1) ^ key(kr)) << 5) + ((s & 1) << 4));
      off[q] = col < width ? (uint32_t)kr * (uint32_t)ld + col : kOOB;
    }
    r = make_rsrc(p, 0);
  }
  __device__ void next() {
    const int n = left > 0 ? min(rows, KR) : 0;
    r = make_rsrc(p, n > 0 ? (uint32_t)(n - 1) * (uint32_t)ld + width : 0u);
    p += KR * ld;
    rows -= KR;
    --left;
    if (--seg == 0) {
      p = p_next;
      rows = rows_next;
    }
  }
  __device__ void issue(uint32_t lds, int q, int wave) const {
    dma16(r, lds + (uint32_t)((q * S::NW + wave) * 1024), off[q]);
  }
  // rows [row, row + 16) of the tile (columns of the stage), 32-deep k-step kk
  static __device__ bf16x8 frag(const char* tile, int row, int kk, int lane) {
    const int k = kk * 32 + (lane >> 4) * 8 + ((lane >> 2) & 3);
    const int ky = ((lane >> 2) & 3) | (((lane >> 4) & 1) << 2);
    const char* q = tile + k * ROWB + (((row >> 4) ^ ky) << 5) + (lane & 3) * 8;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)q);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(q + 4 * ROWB));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// The K loop of tile_kloop_bf16 (gemm_core.hpp, which explains the schedule) over two such
// operands, with NS stages in flight: same 16x16x32 MFMAs, handover and priorities.
template <class S, class OX, class OY>
__device__ inline void kloop_any(OX& ox, OY& oy, int ksteps, char* lds, int wave, int lane,
                                 f32x16 (&acc)[S::FI][S::FJ]) {
  static_assert(S::BKB == 128 && (S::NS - 1) * S::LOADS <= 63, "128-byte rows, countable loads");
  constexpr int GI = 2 * S::FI, GJ = 2 * S::FJ;
  constexpr int NM = GI * GJ, NR = GI + GJ, HB = NM / 4, NA = NM - HB;
  constexpr int R0 = 2 * NR < NM ? 2 * NR : NM;
  constexpr int R1 = 2 * NR < NA ? 2 * NR : NA;
  constexpr int L = S::LOADS;
  const int wi = wave / S::WJ, wj = wave % S::WJ;
  const uint32_t base = lds_addr(lds);
#pragma unroll
  for (int i = 0; i < S::FI; ++i)
#pragma unroll
    for (int j = 0; j < S::FJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  auto dma = [&](int buf, int q0, int q1) {
#pragma unroll
    for (int q = q0; q < q1; ++q) {
      if (q < S::XQ) ox.issue(base + buf, q, wave);
      else oy.issue(base + buf + S::BI * S::BKB, q - S::XQ, wave);
    }
  };
#pragma unroll
  for (int st = 0; st < S::NS; ++st) {
    ox.next();
    oy.next();
    dma(st * S::STAGE, 0, L);
  }
  wait_vmem<(S::NS - 1) * L>();
  __syncthreads();
  bf16x8 a[2][GI], b[2][GJ];
  auto rd = [&](int set, int st, int n, int kk) {
    const char* xs = lds + st;
    const char* ys = xs + S::BI * S::BKB;
    if (n == 0) a[set][0] = OX::frag(xs, wi * S::TM, kk, lane);
    else if (n <= GJ) b[set][n - 1] = OY::frag(ys, wj * S::TN + (n - 1) * 16, kk, lane);
    else a[set][n - GJ] = OX::frag(xs, wi * S::TM + (n - GJ) * 16, kk, lane);
  };
#pragma unroll
  for (int n = 0; n < NR; ++n) rd(0, 0, n, 0);
  int cur = 0;
  for (int kt = 0; kt < ksteps; ++kt) {
    const int nxt = cur + S::STAGE == S::NS * S::STAGE ? 0 : cur + S::STAGE;
    __builtin_amdgcn_s_setprio(0);
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      mma16_bf16(acc, m / GJ, m % GJ, a[0][m / GJ], b[0][m % GJ]);
      __builtin_amdgcn_sched_barrier(0);
      if (m < R0) {
#pragma unroll
        for (int n = m * NR / R0; n < (m + 1) * NR / R0; ++n) rd(1, cur, n, 1);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int m = 0; m < HB; ++m) mma16_bf16(acc, m / GJ, m % GJ, a[1][m / GJ], b[1][m % GJ]);
    __builtin_amdgcn_sched_barrier(0);
    stage_handover<(S::NS - 2) * L>();
    __builtin_amdgcn_s_setprio(1);
    ox.next();
    oy.next();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = HB; m < NM; ++m) {
      mma16_bf16(acc, m / GJ, m % GJ, a[1][m / GJ], b[1][m % GJ]);
      __builtin_amdgcn_sched_barrier(0);
      const int r = m - HB;
      if (r < R1) {
#pragma unroll
        for (int n = r * NR / R1; n < (r + 1) * NR / R1; ++n) rd(0, nxt, n, 0);
      }
      dma(cur, r * L / NA, (r + 1) * L / NA);
      __builtin_amdgcn_sched_barrier(0);
    }
    cur = nxt;
  }
  __builtin_amdgcn_s_setprio(0);
  wait_vmem<0>();
  __syncthreads();
}

// The same for fp8: the K loop of tile_kloop_2s_fp8 (32x32x64 MFMAs, Y fragments double-buffered, X
// fragments rotating in place), with NS stages in flight.
template <class S, class OX, class OY>
__device__ inline void kloop_fp8(OX& ox, OY& oy, int ksteps, char* lds, int wave, int lane,
                                 f32x16 (&acc)[S::FI][S::FJ]) {
  constexpr int NK = S::SEGS / 4, L = S::LOADS;
  static_assert(S::BKB == 128 && NK == 2 && (S::NS - 1) * L <= 63, "two k-steps per stage");
  const int wi = wave / S::WJ, wj = wave % S::WJ;
  const int h2 = (lane >> 5) * 2;
  const uint32_t base = lds_addr(lds);
#pragma unroll
  for (int i = 0; i < S::FI; ++i)
#pragma unroll
    for (int j = 0; j < S::FJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  auto dma = [&](int buf, int q0, int q1) {
#pragma unroll
    for (int q = q0; q < q1; ++q) {
      if (q < S::XQ) ox.issue(base + buf, q, wave);
      else oy.issue(base + buf + S::BI * S::BKB, q - S::XQ, wave);
    }
  };
#pragma unroll
  for (int st = 0; st < S::NS; ++st) {
    ox.next();
    oy.next();
    dma(st * S::STAGE, 0, L);
  }
  wait_vmem<(S::NS - 1) * L>();
  __syncthreads();
  const int xrow = wi * S::TM * S::BKB, yrow = (S::BI + wj * S::TN) * S::BKB;
  auto xfrag = [&](int st, int f, int kk) {
    return frag_fp8<S::BKB>(lds + st + xrow + f * 32 * S::BKB, kk * 4 + h2, lane);
  };
  auto yfrag = [&](int st, int f, int kk) {
    return frag_fp8<S::BKB>(lds + st + yrow + f * 32 * S::BKB, kk * 4 + h2, lane);
  };
  auto mma = [](const i32x8& x, const i32x8& y, const f32x16& c) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 0, 0, 0, 127, 0, 127);
  };
  i32x8 a[S::FI], b[2][S::FJ];
#pragma unroll
  for (int f = 0; f < S::FI; ++f) a[f] = xfrag(0, f, 0);
#pragma unroll
  for (int f = 0; f < S::FJ; ++f) b[0][f] = yfrag(0, f, 0);
  int cur = 0;
  for (int kt = 0; kt < ksteps; ++kt) {
    const int nxt = cur + S::STAGE == S::NS * S::STAGE ? 0 : cur + S::STAGE;
    __builtin_amdgcn_s_setprio(0);
#pragma unroll
    for (int f = 0; f < S::FJ; ++f) b[1][f] = yfrag(cur, f, 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < S::FI; ++i) {
#pragma unroll
      for (int j = 0; j < S::FJ; ++j) acc[i][j] = mma(a[i], b[0][j], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
      a[i] = xfrag(cur, i, 1);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < S::FJ; ++j) acc[0][j] = mma(a[0], b[1][j], acc[0][j]);
    __builtin_amdgcn_sched_barrier(0);
    stage_handover<(S::NS - 2) * L>();
    __builtin_amdgcn_s_setprio(1);
    ox.next();
    oy.next();
#pragma unroll
    for (int f = 0; f < S::FJ; ++f) b[0][f] = yfrag(nxt, f, 0);
#pragma unroll
    for (int i = 0; i < S::FI; ++i) {
      if (i > 0) {
#pragma unroll
        for (int j = 0; j < S::FJ; ++j) acc[i][j] = mma(a[i], b[1][j], acc[i][j]);
      }
      __builtin_amdgcn_sched_barrier(0);
      a[i] = xfrag(nxt, i, 0);
      dma(cur, i * L / S::FI, (i + 1) * L / S::FI);
      __builtin_amdgcn_sched_barrier(0);
    }
    cur = nxt;
  }
  __builtin_amdgcn_s_setprio(0);
  wait_vmem<0>();
  __syncthreads();
}

// Orders this wave's LDS accesses with each other across lanes.
__device__ inline void wave_lds_fence() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// One 32-row block of the wave's accumulators, row by row, through a piece of LDS of the wave's own
// in fp32: no barrier is needed and the epilogue sees unrounded sums.  A lane gets W neighbouring
// columns (of both products in the gated form, whose 64 columns are 32 of the gate and the same 32
// of the up product).  The row stride of TN + 4 floats puts the four row groups of one accumulator
// write 16 banks apart.
template <class S, int MB, bool PAIR, int W>
struct RowBlock {
  static_assert(!PAIR || S::TN == 64, "one gate block and one up block per wave");
  static constexpr int LD = S::TN + 4;
  static constexpr int CG = (PAIR ? S::TN / 2 : S::TN) / W;   // lanes per row
  static constexpr int RK = 64 / CG;                          // rows per step
  static constexpr int STEPS = 32 / RK;
  float* mine;
  int lane;
  __device__ RowBlock(char* lds, int wave, int lane_)
      : mine((float*)lds + wave * 32 * LD), lane(lane_) {}
  __device__ int row() const { return lane / CG; }         // in step 0
  __device__ int col() const { return (lane % CG) * W; }   // in the wave's columns
  __device__ void put(const f32x16 (&acc)[S::FJ]) {
    wave_lds_fence();
#pragma unroll
    for (int j = 0; j < S::FJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        mine[acc_row<MB>(0, e, lane) * LD + acc_col<MB>(j, e, lane)] = acc[j][e];
    wave_lds_fence();
  }
  // the lane's columns of step k, or four of them; product p of a pair
  __device__ f32x4 get4(int k, int h, int p = 0) const {
    return *(const f32x4*)(mine + (k * RK + row()) * LD + col() + 4 * h + 32 * p);
  }
  __device__ void get(float (&v)[W], int k, int p = 0) const {
    const float* q = mine + (k * RK + row()) * LD + col() + 32 * p;
#pragma unroll
    for (int h = 0; h < W / 4; ++h) {
      const f32x4 t = *(const f32x4*)(q + 4 * h);
#pragma unroll
      for (int c = 0; c < 4; ++c) v[4 * h + c] = t[c];
    }
  }
};

// A matrix of the epilogue, seen from the wave's first row and column, a lane's 8 columns at a time.
//   ALIGNED    (even widths: rows at 4-byte multiples, which is what buffer accesses need) through a
//              descriptor that ends with the output: rows past it read as zero and are not stored;
//              in one access where the width is a multiple of 8, else in pieces of `piece` columns,
//              each of which is inside or outside
//   otherwise  through pointers, at any element's address, with branches; a lane with fewer than 8
//              columns goes through Epilogue (epilogue_rows)
template <bool ALIGNED>
struct EpiMatrix {
  __amdgpu_buffer_rsrc_t r;
  char* p;
  int ld, piece;   // piece: 8, 4 or 2
  // cols: the output's width; nr, nc: rows and columns of the output from here on; lane_row,
  // lane_col: this lane's
  __device__ void init(const void* m, long long ld_, int esz, int cols, int row, int col, int nr,
                       int nc, int lane_row, int lane_col) {
    ld = (int)ld_;
    piece = (cols & 7) == 0 ? 8 : (cols & 3) == 0 ? 4 : 2;
    char* first = (char*)m + ((size_t)row * ld_ + col) * esz;
    if constexpr (ALIGNED)
      r = __builtin_amdgcn_make_buffer_rsrc(first, 0, ((nr - 1) * ld + nc) * esz, 0x00020000);
    else p = first + ((long long)lane_row * ld + lane_col) * esz;
  }
};

// Where this lane's part of the tile lies.
struct EpiLane {
  int row, col;   // in step 0, in the wave's columns
  int nr, nc;     // rows and columns of the output from the wave's first on
  __device__ bool full() const { return nc - col >= 8; }
  __device__ bool has_col(int c) const { return col + c < nc; }
  __device__ bool has(int step) const { return row + step < nr; }
};

struct Raw16 {
  uint32_t r[4];
  __device__ float get(int c) const {
    return __uint_as_float((c & 1) ? r[c >> 1] & 0xffff0000u : r[c >> 1] << 16);
  }
};

// 8 bf16 at `step` rows below the lane's first (zero outside), read once: non-temporal.
template <bool ALIGNED>
__device__ inline void epi_load(Raw16& v, const EpiMatrix<ALIGNED>& m, const EpiLane& l, int step) {
  if constexpr (ALIGNED) {
    const int off = ((l.row + step) * m.ld + l.col) * 2;
    if (m.piece == 8) {
      const u32x4 t =
          __builtin_amdgcn_raw_buffer_load_b128(m.r, l.has_col(0) ? off : (int)kOOB, 0, 2);
#pragma unroll
      for (int c = 0; c < 4; ++c) v.r[c] = t[c];
    } else if (m.piece == 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x2 t = __builtin_amdgcn_raw_buffer_load_b64(
            m.r, l.has_col(4 * h) ? off + 8 * h : (int)kOOB, 0, 0);
        v.r[2 * h] = t[0];
        v.r[2 * h + 1] = t[1];
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        v.r[c] = __builtin_amdgcn_raw_buffer_load_b32(
            m.r, l.has_col(2 * c) ? off + 4 * c : (int)kOOB, 0, 0);
    }
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) v.r[c] = 0;
    if (l.full() && l.has(step)) {
      const u32x4_u t = *(const u32x4_u*)(m.p + (long long)step * m.ld * 2);
#pragma unroll
      for (int c = 0; c < 4; ++c) v.r[c] = t[c];
    }
  }
}

// 8 values to memory, rounded to bf16 or as they are.  The outputs are written once and not read
// here: nt keeps the operands in the caches (4096^3 with GELU, residual and Z: 111 us, with the
// default policy 125).  The scalar offset is the constant 0: a 16-byte buffer store whose scalar
// offset is a register still reads its data when the next instruction may already overwrite it, and
// the compiler leaves a gap only where that offset is a constant (seen as single words 0 or 1 in the
// output, the result of the v_cndmask right behind the store).
template <bool ALIGNED>
__device__ inline void epi_store(const float (&v)[8], const EpiMatrix<ALIGNED>& m, const EpiLane& l,
                                 int step, bool f32) {
  u32x4 o;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const f32x2 p = {v[2 * c], v[2 * c + 1]};
    o[c] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
  }
  if constexpr (ALIGNED) {
    const f32x4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
    const int at = (l.row + step) * m.ld + l.col;
    if (f32) {   // (gradients only, whose width is a multiple of 64, so they are aligned)
      const int off = l.has_col(0) ? at * 4 : (int)kOOB;
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, lo), m.r, off, 0, 2);
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, hi), m.r, off + 16, 0, 2);
    } else if (m.piece == 8) {
      __builtin_amdgcn_raw_buffer_store_b128(o, m.r, l.has_col(0) ? at * 2 : (int)kOOB, 0, 2);
    } else if (m.piece == 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        __builtin_amdgcn_raw_buffer_store_b64((u32x2){o[2 * h], o[2 * h + 1]}, m.r,
                                              l.has_col(4 * h) ? at * 2 + 8 * h : (int)kOOB, 0, 2);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        __builtin_amdgcn_raw_buffer_store_b32(o[c], m.r,
                                              l.has_col(2 * c) ? at * 2 + 4 * c : (int)kOOB, 0, 2);
    }
  } else {
    if (!l.full() || !l.has(step)) return;
    *(u32x4_u*)(m.p + (long long)step * m.ld * 2) = o;
  }
}

// The epilogue of the wave's part of a tile, from row `row` and column `col` of the output on.
// Aligned: the residual of the whole tile is requested at once (the registers of the K loop's
// fragments are free by then); else of a 32-row block.
template <class S, int MB, bool PAIR, bool PLAIN, bool ALIGNED>
__device__ inline void epilogue_rows(const f32x16 (&acc)[S::FI][S::FJ], char* lds, int wave,
                                     int lane, const Epilogue& ep, int row, int col) {
  typedef RowBlock<S, MB, PAIR, 8> RB;
  RB rb(lds, wave, lane);
  const EpiArgs& e = ep.e;
  const EpiLane l = {rb.row(), rb.col(), min(e.rows - row, S::TM), e.cols - col};
  if (l.nr <= 0 || l.nc <= 0) return;
  auto open = [&](EpiMatrix<ALIGNED>& m, const void* p, long long ld, int esz) {
    m.init(p, ld, esz, e.cols, row, col, l.nr, l.nc, l.row, l.col);
  };
  constexpr bool RES = !PAIR && !PLAIN;
  constexpr int RI = RES && ALIGNED ? S::FI : 1;
  EpiMatrix<ALIGNED> mo, mz0, mz1, mr;
  Raw16 res[RI][RB::STEPS];
  float bias[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) bias[c] = 0.0f;
  open(mo, ep.out, e.ld_out, e.out_f32 ? 4 : 2);
  if constexpr (!PLAIN) open(mz0, e.z[0], e.cols, 2);
  if constexpr (PAIR) open(mz1, e.z[1], e.cols, 2);
  if constexpr (RES) {
    open(mr, e.residual, e.ld_res, 2);
    if (ALIGNED && e.residual)
#pragma unroll
      for (int i = 0; i < RI; ++i)
#pragma unroll
        for (int k = 0; k < RB::STEPS; ++k)
          epi_load<ALIGNED>(res[i][k], mr, l, i * 32 + k * RB::RK);
    if (e.bias) {
      if constexpr (ALIGNED) {
        const u32x4 t = __builtin_amdgcn_raw_buffer_load_b128(
            __builtin_amdgcn_make_buffer_rsrc((char*)e.bias, 0, e.cols * 2, 0x00020000),
            (col + l.col) * 2, 0, 0);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          bias[c] = __uint_as_float((c & 1) ? t[c >> 1] & 0xffff0000u : t[c >> 1] << 16);
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (l.col + c < l.nc) bias[c] = (float)((const __bf16*)e.bias)[col + l.col + c];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < S::FI; ++i) {
    if constexpr (RES && !ALIGNED) {
      if (e.residual)
#pragma unroll
        for (int k = 0; k < RB::STEPS; ++k)
          epi_load<ALIGNED>(res[0][k], mr, l, i * 32 + k * RB::RK);
    }
    rb.put(acc[i]);
    act_switch<PLAIN>(e.act, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
#pragma unroll
      for (int k = 0; k < RB::STEPS; ++k) {
        const int step = i * 32 + k * RB::RK;
        float v[8], u[8];
        rb.get(v, k);
        if constexpr (PLAIN) {
          epi_store<ALIGNED>(v, mo, l, step, e.out_f32);
          continue;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = v[c] * ep.s0 + bias[c];
        if constexpr (PAIR) {
          rb.get(u, k, 1);
#pragma unroll
          for (int c = 0; c < 8; ++c) u[c] *= ep.s1;
        }
        if (e.z[0]) {
          epi_store<ALIGNED>(v, mz0, l, step, false);
          if constexpr (PAIR) epi_store<ALIGNED>(u, mz1, l, step, false);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          v[c] = act_value<ACT>(v[c]);
          if constexpr (PAIR) v[c] *= u[c];
        }
        if constexpr (RES) {
          if (e.residual)
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] += res[RI > 1 ? i : 0][k].get(c);
        }
        epi_store<ALIGNED>(v, mo, l, step, false);
      }
    });
    if constexpr (!ALIGNED) {
      // the output's last columns, fewer than 8
      if (l.full() || l.col >= l.nc) continue;
#pragma unroll 1
      for (int n = 0; n < 2 * RB::STEPS; ++n) {
        const int r = i * 32 + (n >> 1) * RB::RK + l.row, c = l.col + (n & 1) * 4;
        if (r >= l.nr || c >= l.nc) continue;
        act_switch<PLAIN>(e.act, [&](auto act) {
          constexpr int ACT = decltype(act)::value;
          if constexpr (PAIR)
            ep.template gated<ACT>(row + r, col + c, rb.get4(n >> 1, n & 1),
                                   rb.get4(n >> 1, n & 1, 1));
          else ep.template linear<ACT>(row + r, col + c, rb.get4(n >> 1, n & 1));
        });
      }
    }
  }
}

// One tile: the K loop over this split's stages, then the epilogue or the split's fp32 sums.
template <class S, int KIND>
__device__ __forceinline__ void block_gemm_tile(const GemmArgs& a, const TileAt& t, char* lds) {
  constexpr bool kGated = KIND == kGemmGated || KIND == kGemmGated8;
  constexpr bool kFp8 = KIND == kGemmLin8 || KIND == kGemmGated8;
  constexpr bool kXS = KIND == kGemmDw, kYS = KIND == kGemmDx || KIND == kGemmDw;
  constexpr int MB = acc_block<S, kFp8>();
  constexpr int BC = kGated ? S::BJ / 2 : S::BJ;   // output columns of a tile
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int k0 = (int)((long long)a.ksteps * t.split / a.splits);
  const int k1 = (int)((long long)a.ksteps * (t.split + 1) / a.splits);
  const int row0 = t.ti * S::BI, col0 = t.half < 0 ? t.tj * BC : (t.tj * 2 + t.half) * BC;
  if (col0 >= a.e.cols) return;   // a right half wholly past the last column
  const char* x = (const char*)(t.batch ? a.x[1] : a.x[0]);
  const char* xk = x + (long long)row0 * a.ldx + (long long)k0 * S::BKB;   // K-contiguous X
  const int nx = min(a.e.rows - row0, S::BI), ny = min(a.e.cols - col0, BC);
  const int weight = kGated ? Operand<S, S::BJ, S::YQ, false>::pair_weight(wave) : 0;
  const char* yk = (const char*)(weight ? a.y[1] : a.y[0]) + (long long)col0 * a.ldy +
                   (long long)k0 * S::BKB;                                  // K-contiguous Y
  f32x16 acc[S::FI][S::FJ];
  Operand<S, S::BI, S::XQ, kXS> ox;
  Operand<S, S::BJ, S::YQ, kYS> oy;
  if constexpr (kXS)
    ox.init(x + 2ll * row0, nullptr, a.ldx, a.xk, a.xcols - row0, k0, a.ksteps, k1 - k0, wave,
            lane);
  else
    ox.init(xk, a.ldx, nx, k1 - k0, wave, lane);
  if constexpr (kYS)
    oy.init((const char*)a.y[0] + 2ll * col0, (const char*)a.y[1] + 2ll * col0, a.ldy, a.yk,
            a.ycols - col0, k0, a.kseg, k1 - k0, wave, lane);
  else if constexpr (kGated)
    oy.init_pair(yk, a.ldy, ny, k1 - k0, wave, lane);
  else
    oy.init(yk, a.ldy, ny, k1 - k0, wave, lane);
  if constexpr (kFp8) kloop_fp8<S>(ox, oy, k1 - k0, lds, wave, lane, acc);
  else kloop_any<S>(ox, oy, k1 - k0, lds, wave, lane, acc);

  const int wrow = row0 + wave / S::WJ * S::TM;
  const int wcol = col0 + (wave % S::WJ) * (kGated ? S::TN / 2 : S::TN);
  if (a.splits > 1) {
    typedef RowBlock<S, MB, kGated, 4> RB;
    RB rb(lds, wave, lane);
    const size_t plane = (size_t)a.e.rows * a.ldp;
    float* p = a.part + (size_t)(t.split * (kGated ? 2 : a.batches) + t.batch) * plane;
    const int c = wcol + rb.col();
#pragma unroll
    for (int i = 0; i < S::FI; ++i) {
      rb.put(acc[i]);
#pragma unroll
      for (int k = 0; k < RB::STEPS; ++k) {
        const int r = wrow + i * 32 + k * RB::RK + rb.row();
        if (r >= a.e.rows || c >= a.e.cols) continue;
        float* q = p + (size_t)r * a.ldp + c;
        float v[4];
        rb.get(v, k);
        *(f32x4*)q = (f32x4){v[0], v[1], v[2], v[3]};
        if constexpr (kGated) {
          rb.get(v, k, 1);
          *(f32x4*)(q + plane) = (f32x4){v[0], v[1], v[2], v[3]};
        }
      }
    }
    return;
  }
  const Epilogue ep(a.e, t.batch);
  constexpr bool kPlain = kXS || kYS;   // gradients: contiguous, K (a multiple of 64) wide
  if (kPlain || ep.aligned)
    epilogue_rows<S, MB, kGated, kPlain, true>(acc, lds, wave, lane, ep, wrow, wcol);
  else if constexpr (!kPlain)
    epilogue_rows<S, MB, kGated, false, false>(acc, lds, wave, lane, ep, wrow, wcol);
}

// S: the tile; H: its half (or S again where a launch has none).
template <class S, class H, int KIND>
__device__ inline void block_gemm_part(const GemmArgs& a, int block, char* lds) {
  const TileAt t = tile_at(a, block);
  if constexpr (!std::is_same<S, H>::value) {
    if (t.half >= 0) {
      block_gemm_tile<H, KIND>(a, t, lds);
      return;
    }
  }
  block_gemm_tile<S, KIND>(a, t, lds);
}

template <class S, class H>
constexpr int part_lds() {
  return ops_lds<S>() > ops_lds<H>() ? ops_lds<S>() : ops_lds<H>();
}

template <class S, class H, int KIND>
__device__ inline void block_gemm_body(const GemmArgs& a) {
  __shared__ __attribute__((aligned(1024))) char lds[part_lds<S, H>()];
  block_gemm_part<S, H, KIND>(a, (int)blockIdx.x, lds);
}

// The two products of a backward pass in one launch, so that neither leaves compute units idle in a
// last round of its own: the tiles of the one with the longer K loop first.
template <class S, class H>
__device__ inline void backward_gemm_body(const BackwardArgs& a) {
  __shared__ __attribute__((aligned(1024))) char lds[part_lds<S, H>()];
  const int b = (int)blockIdx.x;
  const int first = a.dx_first ? a.dx.blocks : a.dw.blocks;
  if ((b < first) == (a.dx_first != 0))
    block_gemm_part<S, H, kGemmDx>(a.dx, b - (a.dx_first ? 0 : first), lds);
  else
    block_gemm_part<S, H, kGemmDw>(a.dw, b - (a.dx_first ? first : 0), lds);
}

}  // namespace ringag
