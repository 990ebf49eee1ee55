// Layer norm over rows of H, forward and backward, one workgroup per row at a time.
//   forward   y = (x - mean) rstd w + b
//   backward  g = dy w, xh = (x - mean) rstd:  dx = rstd (g - mean(g) - xh mean(g xh)),
//             dw = sum over rows of dy xh, db = sum over rows of dy
// Statistics are fp32: the row stays in registers (NV vectors of 8 columns per thread), so the
// variance is summed from the differences to the mean, with no second read and no cancellation.
// NV = 0 takes any width and reads the row again for each step.
//
// Bound by memory.  A workgroup goes through rows gridDim apart with the weight (and bias) in
// registers and the next row's loads under way before this row's reductions, so that a row's
// latency and its two reductions hide under the loads of the others.  Accesses go through a buffer
// descriptor of the row: columns past H read as zero and are not stored, without branches that
// would make each load wait for the last.
// Forward 16384 x 8192 bf16: 94 to 97 us, 5.5 to 5.7 TB/s (a large copy reaches 4.96).  Backward
// 8192 x 8192 bf16: 70 us and 4.7 for the column sums, 5.4 TB/s.  One row of 8192: 3.0 us, one
// round trip to memory and two reductions, in a call of 6.3 to 7.8.  1777 x 1001 fp32 backward:
// 11.9 us for both launches (21 MB, much of it still cached; seven rows to a workgroup, one after
// the other).  Two forms hold more than their registers: forward with four vectors keeps 3 to 6
// values in scratch (odd rows with an fp32 weight 56) and reads them back once a row, at the rate
// above all the same; backward of fp32 rows of more than 8192 columns 14 to 22 (odd ones up to
// 86), stored and read back in every row, which shows: 2048 x 16384 112.6 us against 81 for its
// bytes, where 2048 x 8192, one vector per thread and nothing in scratch, takes 46.7 against 41.
#pragma once

#include "gemm_core.hpp"
#include "ops.hpp"

namespace ringag {

typedef uint32_t u32x4n __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4n_u __attribute__((ext_vector_type(4), aligned(2)));

// Column k of vector j of this thread: 8 neighbouring ones.
__device__ inline int norm_col(int j, int k, int nt) { return (j * nt + (int)threadIdx.x) * 8 + k; }

// One row of H elements.  BUF: through a descriptor, whose range check is by 4 bytes: the row's
// start and length must be multiples of 4.  Else (odd bf16 rows) through pointers: 16-byte accesses
// at any element's address, the row's last few elements one by one.
template <class T, bool BUF>
struct Row {
  __amdgpu_buffer_rsrc_t r;
  T* p;
  int H;
  __device__ Row(const T* row, int H_) {
    if constexpr (BUF)
      r = __builtin_amdgcn_make_buffer_rsrc((void*)row, 0, H_ * (int)sizeof(T), 0x00020000);
    else {
      p = (T*)row;
      H = H_;
    }
  }
};

// Cache policy (the buffer instructions' nt bit) of the rows of x, dy, y and dx.  A call that
// touches more than the last-level cache holds streams them: forward 16384 x 8192 bf16 101.2 us
// with the default policy, 94.9 streamed; backward 8192 x 8192 79.3 and 75.5.  One whose rows
// another kernel has just left there finds them with the default (backward 1777 x 1001 fp32 12.6
// us, streamed 13.4).
constexpr int kCached = 0, kStream = 2;

// Eight elements as they lie in memory; those past the row's end are zero.
template <class T>
struct Raw8 {
  static constexpr int N = sizeof(T) * 2;   // registers
  uint32_t r[N];
  template <int POLICY, bool BUF>
  __device__ void load(const Row<T, BUF>& row, int j, int nt) {
    const int c = norm_col(j, 0, nt);
    if constexpr (BUF) {
#pragma unroll
      for (int h = 0; h < N / 4; ++h) {
        const u32x4n v =
            __builtin_amdgcn_raw_buffer_load_b128(row.r, c * (int)sizeof(T) + 16 * h, 0, POLICY);
#pragma unroll
        for (int k = 0; k < 4; ++k) r[4 * h + k] = v[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) r[k] = 0;
      if (c + 8 <= row.H) {
#pragma unroll
        for (int h = 0; h < N / 4; ++h) {
          const u32x4n v = *(const u32x4n_u*)((const char*)(row.p + c) + 16 * h);
#pragma unroll
          for (int k = 0; k < 4; ++k) r[4 * h + k] = v[k];
        }
      } else if (c < row.H) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (c + k >= row.H) continue;
          if constexpr (sizeof(T) == 4) r[k] = __float_as_uint(row.p[c + k]);
          else
            r[k >> 1] |= (uint32_t)__builtin_bit_cast(unsigned short, row.p[c + k])
                         << (16 * (k & 1));
        }
      }
    }
  }
  __device__ float get(int k) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(r[k]);
    else return __uint_as_float((k & 1) ? r[k >> 1] & 0xffff0000u : r[k >> 1] << 16);
  }
};

template <int POLICY, class T, bool BUF>
__device__ inline void norm_store(const float (&v)[8], const Row<T, BUF>& row, int j, int nt) {
  const int c = norm_col(j, 0, nt);
  u32x4n o[sizeof(T) / 2];
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const f32x2 p = {v[2 * k], v[2 * k + 1]};
      o[0][k] = __builtin_bit_cast(uint32_t, __builtin_convertvector(p, bf16x2));
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k >> 2][k & 3] = __float_as_uint(v[k]);
  }
  if constexpr (BUF) {
#pragma unroll
    for (int h = 0; h < (int)sizeof(T) / 2; ++h)
      __builtin_amdgcn_raw_buffer_store_b128(o[h], row.r, c * (int)sizeof(T) + 16 * h, 0,
                                             POLICY);
  } else if (c + 8 <= row.H) {
#pragma unroll
    for (int h = 0; h < (int)sizeof(T) / 2; ++h)
      *(u32x4n_u*)((char*)(row.p + c) + 16 * h) = o[h];
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (c + k < row.H) row.p[c + k] = (T)v[k];
  }
}

template <int CTRL>
__device__ inline float dpp_move(float v) {
  return __uint_as_float(
      (uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CTRL, 0xF, 0xF, true));
}

// Sum over the 64 lanes, the same bits in each: pairs, quads, eights and sixteens through DPP
// (quad_perm, row_half_mirror, row_mirror), then gfx950's row swaps.  No LDS round trips.
__device__ inline float wave_sum(float v) {
  v += dpp_move<0xB1>(v);
  v += dpp_move<0x4E>(v);
  v += dpp_move<0x141>(v);
  v += dpp_move<0x140>(v);
  uint32_t u = __float_as_uint(v);
  const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  u = __float_as_uint(v);
  const auto q = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// Sums N values over the workgroup, in an order that does not change from run to run; every thread
// gets them all.  `red`: one [N][16] array; two calls in a row need different ones (or a barrier).
template <int N>
__device__ inline void norm_sum(float (&v)[N], float (*red)[16]) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
  const int nw = (int)blockDim.x >> 6;
  if (nw == 1) return;
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int n = 0; n < N; ++n) red[n][threadIdx.x >> 6] = v[n];
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    v[n] = 0.0f;
    for (int i = 0; i < nw; ++i) v[n] += red[n][i];
  }
}

// mean, then the sum of squared differences, each of fp32 values v (zero past H)
template <class XT, class YT, class WT, int NV, bool BUF, int POLICY>
__device__ inline void norm_fwd_body(const NormArgs& a) {
  __shared__ float red[2][16];   // mean, variance: the other one's barrier lies between two uses
  const int nt = blockDim.x, H = a.H;
  const float inv = 1.0f / (float)H;
  if constexpr (NV > 0) {
    Raw8<XT> next[NV];
    const XT* x = (const XT*)a.x;
    auto fetch = [&](int r) {
      const Row<XT, BUF> row(x + (size_t)r * a.ld_x, H);
#pragma unroll
      for (int j = 0; j < NV; ++j) next[j].template load<POLICY>(row, j, nt);
    };
    fetch(blockIdx.x);
    // (without a bias its row has no columns and reads as zero)
    const Row<WT, BUF> rw((const WT*)a.w, H);
    const Row<WT, BUF> rb((const WT*)a.b, a.b ? H : 0);
    Raw8<WT> w[NV], b[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      w[j].template load<kCached>(rw, j, nt);
      b[j].template load<kCached>(rb, j, nt);
    }
    for (int r = blockIdx.x; r < a.T; r += gridDim.x) {
      float v[NV][8], s[1] = {0.0f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[j][k] = next[j].get(k);
          s[0] += v[j][k];
        }
      const int rn = r + (int)gridDim.x;
      if (rn < a.T) fetch(rn);
      norm_sum<1>(s, red);
      const float mean = s[0] * inv;
      float q[1] = {0.0f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[j][k] -= mean;
          q[0] += norm_col(j, k, nt) < H ? v[j][k] * v[j][k] : 0.0f;
        }
      norm_sum<1>(q, red + 1);
      const float rstd = 1.0f / sqrtf(q[0] * inv + a.eps);
      if (threadIdx.x == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
      }
      const Row<YT, BUF> y((const YT*)a.y + (size_t)r * H, H);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] = v[j][k] * rstd * w[j].get(k) + b[j].get(k);
        norm_store<POLICY>(v[j], y, j, nt);
      }
    }
  } else {
    const int nv = (H + 8 * nt - 1) / (8 * nt);
    for (int r = blockIdx.x; r < a.T; r += gridDim.x) {
      const Row<XT, BUF> x((const XT*)a.x + (size_t)r * a.ld_x, H);
      const Row<YT, BUF> y((const YT*)a.y + (size_t)r * H, H);
      Raw8<XT> t;
      float s[1] = {0.0f}, q[1] = {0.0f};
      for (int j = 0; j < nv; ++j) {
        t.template load<kCached>(x, j, nt);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[0] += t.get(k);
      }
      norm_sum<1>(s, red);
      const float mean = s[0] * inv;
      for (int j = 0; j < nv; ++j) {
        t.template load<kCached>(x, j, nt);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float d = t.get(k) - mean;
          q[0] += norm_col(j, k, nt) < H ? d * d : 0.0f;
        }
      }
      norm_sum<1>(q, red + 1);
      const float rstd = 1.0f / sqrtf(q[0] * inv + a.eps);
      if (threadIdx.x == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = rstd;
      }
      for (int j = 0; j < nv; ++j) {
        t.template load<kCached>(x, j, nt);
        Raw8<WT> w, b;
        w.template load<kCached>(Row<WT, BUF>((const WT*)a.w, H), j, nt);
        b.template load<kCached>(Row<WT, BUF>((const WT*)a.b, a.b ? H : 0), j, nt);
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = (t.get(k) - mean) * rstd * w.get(k) + b.get(k);
        norm_store<kCached>(o, y, j, nt);
      }
    }
  }
}

// A workgroup takes every gridDim-th row and keeps its column sums of dw and db in registers (NV =
// 0: in its own row of the partial sums); they are joined over workgroups by the column-sum kernel.
template <class XT, class YT, class WT, int NV, bool BUF, int POLICY>
__device__ inline void norm_bwd_body(const NormArgs& a) {
  __shared__ float red[2][2][16];   // by turns, so that one barrier per row is enough
  const int nt = blockDim.x, H = a.H;
  const float inv = 1.0f / (float)H;
  float* const pdw = a.part + (size_t)blockIdx.x * 2 * H;
  float* const pdb = a.part_db + (size_t)blockIdx.x * 2 * H;
  int turn = 0;
  if constexpr (NV > 0) {
    const XT* x = (const XT*)a.x;
    const YT* dy = (const YT*)a.dy;
    Raw8<XT> nx[NV];
    Raw8<YT> ny[NV];
    float dw[NV][8], db[NV][8];
    Raw8<WT> w[NV];
    auto fetch = [&](int r) {
      const Row<XT, BUF> rx(x + (size_t)r * a.ld_x, H);
      const Row<YT, BUF> ry(dy + (size_t)r * a.ld_dy, H);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        nx[j].template load<POLICY>(rx, j, nt);
        ny[j].template load<POLICY>(ry, j, nt);
      }
    };
    fetch(blockIdx.x);
    float mean = a.mean[blockIdx.x], rstd = a.rstd[blockIdx.x];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      w[j].template load<kCached>(Row<WT, BUF>((const WT*)a.w, H), j, nt);
#pragma unroll
      for (int k = 0; k < 8; ++k) dw[j][k] = db[j][k] = 0.0f;
    }
    for (int r = blockIdx.x; r < a.T; r += gridDim.x, turn ^= 1) {
      float xh[NV][8], g[NV][8], s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float d = ny[j].get(k);
          // (dy reads as zero past H; a row whose x is not finite there would not)
          xh[j][k] = norm_col(j, k, nt) < H ? (nx[j].get(k) - mean) * rstd : 0.0f;
          g[j][k] = d * w[j].get(k);
          dw[j][k] += d * xh[j][k];
          db[j][k] += d;
          s[0] += g[j][k];
          s[1] += g[j][k] * xh[j][k];
        }
      const float scale = rstd;
      const int rn = r + (int)gridDim.x;
      if (rn < a.T) {
        fetch(rn);
        mean = a.mean[rn];
        rstd = a.rstd[rn];
      }
      norm_sum<2>(s, red[turn]);
      s[0] *= inv;
      s[1] *= inv;
      const Row<XT, BUF> dx((const XT*)a.y + (size_t)r * H, H);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int k = 0; k < 8; ++k) g[j][k] = scale * (g[j][k] - s[0] - xh[j][k] * s[1]);
        norm_store<POLICY>(g[j], dx, j, nt);
      }
    }
    const Row<float, true> pw(pdw, H), pb(pdb, H);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      norm_store<kCached>(dw[j], pw, j, nt);
      norm_store<kCached>(db[j], pb, j, nt);
    }
  } else {
    const int nv = (H + 8 * nt - 1) / (8 * nt);
    for (int j = 0; j < nv; ++j)   // each thread clears the columns that it adds to
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = norm_col(j, k, nt);
        if (c < H) pdw[c] = pdb[c] = 0.0f;
      }
    for (int r = blockIdx.x; r < a.T; r += gridDim.x, turn ^= 1) {
      const Row<XT, BUF> x((const XT*)a.x + (size_t)r * a.ld_x, H);
      const Row<YT, BUF> dy((const YT*)a.dy + (size_t)r * a.ld_dy, H);
      const Row<XT, BUF> dx((const XT*)a.y + (size_t)r * H, H);
      const float mean = a.mean[r], rstd = a.rstd[r];
      Raw8<XT> tx;
      Raw8<YT> ty;
      Raw8<WT> w;
      float s[2] = {0.0f, 0.0f};
      for (int j = 0; j < nv; ++j) {
        tx.template load<kCached>(x, j, nt);
        ty.template load<kCached>(dy, j, nt);
        w.template load<kCached>(Row<WT, BUF>((const WT*)a.w, H), j, nt);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int c = norm_col(j, k, nt);
          if (c >= H) continue;
          const float xh = (tx.get(k) - mean) * rstd, d = ty.get(k);
          s[0] += d * w.get(k);
          s[1] += d * w.get(k) * xh;
          pdw[c] += d * xh;
          pdb[c] += d;
        }
      }
      norm_sum<2>(s, red[turn]);
      for (int j = 0; j < nv; ++j) {
        tx.template load<kCached>(x, j, nt);
        ty.template load<kCached>(dy, j, nt);
        w.template load<kCached>(Row<WT, BUF>((const WT*)a.w, H), j, nt);
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          o[k] = rstd * (ty.get(k) * w.get(k) - s[0] * inv -
                         (tx.get(k) - mean) * rstd * (s[1] * inv));
        norm_store<kCached>(o, dx, j, nt);
      }
    }
  }
}

}  // namespace ringag
