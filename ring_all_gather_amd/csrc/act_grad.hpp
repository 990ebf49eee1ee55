// The elementwise half of the backward passes, and the column sums of bias and norm gradients.
//
// dZ = dY act'(Z) (gated: dG = dH U act'(G), dU = dH act(G)) is written once in bf16, because each
// of the two products reads it many times, over tiles; recomputing it from dY and Z on the way
// into a product would double that operand's loads and put the activation's slope between them and
// the MFMAs.  bf16 because that is what the MFMA takes beside the bf16 weight or input: dZ as a
// sum of two bf16 would double the products.  It costs accuracy in dX and dW, also where dW is
// fp32: their relative error against 64 bits is 0.0023, where products of unrounded dZ, rounded at
// the end, have 0.0017.  The column sums take dZ before that rounding.
//
// Bound by memory: 8192 x 8192 (two reads, one write of 134 MB) 65 to 77 us, 5.2 to 6.2 TB/s; gated
// 4096 x 3584 (147 MB, mostly still in the last-level cache) 25 us.
#pragma once

#include "epilogue.hpp"

namespace ringag {

// 8 neighbouring bf16 of row r, as one load without branches around it, so that all of a thread's
// are in flight together: the last columns' come from the row's last 8, and tail8 moves them into
// place (9225 x 2237: 27.4 us; with the last columns element by element 48.4).  STREAM: loaded
// non-temporally, for calls that touch more than the last-level cache holds (linear backward of
// 8192 x 8192 x 1024: 290.5 us with the default policy, 281.5 with this; gated backward of 1537 x
// 1000 x 2048, whose inputs are still cached: 36.3 us with the default, 38.0).
template <bool STREAM>
__device__ inline bf16x8 load8(const void* p, long long ld, int r, int c, int cols) {
  const __bf16* row = (const __bf16*)p + (size_t)r * ld;
  if (cols < 8) {
    bf16x8 x;
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = row[min(c + k, cols - 1)];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c + k >= cols) x[k] = (__bf16)0.0f;
    return x;
  }
  const bf16x8_u* at = (const bf16x8_u*)(row + min(c, cols - 8));
  if constexpr (STREAM) return __builtin_nontemporal_load(at);
  else return *at;
}

// The 8 elements moved down by n >= 0 places, zeros behind them.
__device__ inline bf16x8 tail8(bf16x8 x, int n) {
  if (n == 0) return x;
  typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
  u64x2 v = __builtin_bit_cast(u64x2, x);
  if (n >= 4) {
    v[0] = v[1];
    v[1] = 0;
  }
  if (n >= 8) v[0] = 0;
  const int bits = (n & 3) * 16;
  if (bits) {
    v[0] = v[0] >> bits | v[1] << (64 - bits);
    v[1] >>= bits;
  }
  return __builtin_bit_cast(bf16x8, v);
}

// dZ (or dG and dU) of the rows of one slab, bound by memory.  A workgroup is a.tx threads of 8
// columns by 256 / a.tx rows; a thread keeps its columns over the slab, two rows' loads at a time,
// so the bias gradient's partial sums stay in registers; the row groups are added in LDS in a fixed
// order.
template <int ACT, bool GATED, bool STREAM>
__device__ inline void act_grad_rows(const ActGradArgs& a) {
  __shared__ float red[2048];   // [row group][column]
  constexpr int N = 2;          // rows in flight (4: no faster, and a fifth slower gated)
  constexpr bool kZ = ACT != RAG_ACT_NONE || GATED;
  const int tx = threadIdx.x & (a.tx - 1), ty = threadIdx.x / a.tx, groups = 256 / a.tx;
  const int c = (blockIdx.x * a.tx + tx) * 8;
  const int r0 = (int)blockIdx.y * a.slab_rows, r1 = min(a.rows, r0 + a.slab_rows);
  const int past = a.cols < 8 ? 0 : max(0, c + 8 - a.cols);   // columns past the last one
  float sum[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) sum[k] = 0.0f;
  if (c < a.cols_pad) {
    for (int r = r0 + ty; r < r1; r += N * groups) {
      bf16x8 d[N], z[N], u[N];
#pragma unroll
      for (int h = 0; h < N; ++h) {
        const int rr = min(r + groups * h, r1 - 1);   // (past the slab: a row that exists, unused)
        d[h] = load8<STREAM>(a.dy, a.ld_dy, rr, c, a.cols);
        if constexpr (kZ) z[h] = load8<STREAM>(a.z, a.ld_z, rr, c, a.cols);
        if constexpr (GATED) u[h] = load8<STREAM>(a.u, a.ld_z, rr, c, a.cols);
      }
#pragma unroll
      for (int h = 0; h < N; ++h) {
        if (r + groups * h >= r1) break;
        d[h] = tail8(d[h], past);
        if constexpr (kZ) z[h] = tail8(z[h], past);
        if constexpr (GATED) u[h] = tail8(u[h], past);
        bf16x8 out, out_u;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float value, o;
          if constexpr (GATED) {
            const float dv = (float)d[h][k];
            o = dv * (float)u[h][k] * act_slope<ACT>((float)z[h][k], &value);
            out_u[k] = (__bf16)(dv * value);
          } else {
            o = (float)d[h][k];
            if constexpr (kZ) o *= act_slope<ACT>((float)z[h][k], &value);
            sum[k] += o;
          }
          out[k] = (__bf16)o;
        }
        if (!a.dz) continue;
        // the padding columns get exact zeros whatever act'(0) * 0 would be
        if (c + 8 > a.cols) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (c + k >= a.cols) {
              out[k] = (__bf16)0.0f;
              if constexpr (GATED) out_u[k] = (__bf16)0.0f;
            }
        }
        __bf16* q = (__bf16*)a.dz + (size_t)(r + groups * h) * a.ld_dz + c;
        *(bf16x8*)q = out;
        if constexpr (GATED) *(bf16x8*)(q + a.cols_pad) = out_u;
      }
    }
  }
  if (GATED || !a.colsum) return;
  const int width = a.tx * 8;
#pragma unroll
  for (int k = 0; k < 8; ++k) red[ty * width + tx * 8 + k] = sum[k];
  __syncthreads();
  for (int i = threadIdx.x; i < width; i += 256) {
    const int col = blockIdx.x * width + i;
    if (col >= a.cols) continue;
    float v = 0.0f;
    for (int g = 0; g < groups; ++g) v += red[g * width + i];
    a.colsum[(size_t)blockIdx.y * a.cols + col] = v;
  }
}

template <bool GATED, bool STREAM>
__device__ inline void act_grad_body(const ActGradArgs& a) {
  act_switch(a.act, [&](auto act) {
    act_grad_rows<decltype(act)::value, GATED, STREAM>(a);
  });
}

// Sums of the columns of a [slabs][n] array: 32 columns (a 128-byte line) per workgroup, 32 row
// groups whose sums are added in a fixed order.  A launch of its own: 4 to 5 us, most of it the
// launch and one round of loads (256 slabs of 2 x 8192: 16.8 MB in 4.7 us).  Float atomics in the
// launch before it would change the sums from run to run; an integer count by which the last
// workgroup to arrive adds the slabs in the same order would not, and has not been measured.
constexpr int kSumCols = 32;
__device__ inline void colsum_body(const ColSumArgs& a) {
  __shared__ float red[32][kSumCols + 1];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int n = blockIdx.x * kSumCols + tx;
  float s = 0.0f;
  if (n < a.n0 + a.n1) {
    const float* p = a.part + n;
#pragma unroll 8
    for (int i = ty; i < a.slabs; i += 32) s += p[(size_t)i * a.ld];
  }
  red[ty][tx] = s;
  __syncthreads();
  if (ty != 0 || n >= a.n0 + a.n1) return;
  float v = 0.0f;
#pragma unroll
  for (int k = 0; k < 32; ++k) v += red[k][tx];
  if (n < a.n0) a.out0[n] = v;
  else if (a.out1) a.out1[n - a.n0] = v;
}

}  // namespace ringag
