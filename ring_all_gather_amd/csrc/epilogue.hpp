// Epilogues of the block operators: what is done with four neighbouring columns of a finished row
// of sums.  All arithmetic is fp32; each output is rounded to bf16 once, as it is stored.
#pragma once

#include "act.hpp"
#include "gemm_core.hpp"
#include "ops.hpp"

namespace ringag {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
// Vectors at any element's address: global loads and stores take them in one instruction, so odd
// row lengths cost the crossed lines and no more.
typedef __bf16 bf16x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef __bf16 bf16x8_u __attribute__((ext_vector_type(8), aligned(2)));

__device__ inline f32x4 to_f32(const bf16x4& v) { return __builtin_convertvector(v, f32x4); }
__device__ inline bf16x4 to_bf16(const f32x4& v) { return __builtin_convertvector(v, bf16x4); }

// Columns [c, c + 4) of row r of a bf16 matrix; columns at or past `cols` are not touched (they
// read as zero).
__device__ inline f32x4 load4(const void* p, long long ld, int r, int c, int cols) {
  const __bf16* q = (const __bf16*)p + (size_t)r * ld + c;
  if (c + 4 <= cols) {
    const bf16x4 t = *(const bf16x4_u*)q;
    return to_f32(t);
  }
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (c + k < cols) v[k] = (float)q[k];
  return v;
}
__device__ inline void store4(void* p, long long ld, int r, int c, int cols, const f32x4& v) {
  __bf16* q = (__bf16*)p + (size_t)r * ld + c;
  const bf16x4 o = to_bf16(v);
  if (c + 4 <= cols) {
    *(bf16x4_u*)q = o;
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (c + k < cols) q[k] = o[k];
}
// (fp32 outputs are weight gradients, K wide: all four columns are inside)
__device__ inline void store4_f32(void* p, long long ld, int r, int c, const f32x4& v) {
  *(f32x4*)((float*)p + (size_t)r * ld + c) = v;
}

// The epilogue of an output matrix, set up once per workgroup: uniform flags and scales.
struct Epilogue {
  const EpiArgs& e;
  void* out;
  float s0, s1;
  bool aligned;   // every row of every matrix starts at a 4-byte multiple
  __device__ Epilogue(const EpiArgs& args, int batch) : e(args) {
    out = batch ? e.out[1] : e.out[0];   // (an index would put the arguments in memory)
    const float sx = e.scale_x ? e.scale_x[0] : 1.0f;
    s0 = e.scale_w[0] ? sx * e.scale_w[0][0] : sx;
    s1 = e.scale_w[1] ? sx * e.scale_w[1][0] : sx;
    // (the outputs, Z, G and U are contiguous from a 16-byte multiple on)
    aligned = ((e.cols | e.ld_out) & 1) == 0 &&
              (!e.residual || ((e.ld_res & 1) == 0 && ((uintptr_t)e.residual & 3) == 0));
  }
  // ACT: the activation; v: the sums of columns [c, c + 4) of row r, both inside the output
  template <int ACT>
  __device__ void linear(int r, int c, f32x4 v) const {
    v *= s0;
    if (e.bias) v += load4(e.bias, 0, 0, c, e.cols);
    if (e.z[0]) store4(e.z[0], e.cols, r, c, e.cols, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = act_value<ACT>(v[k]);
    if (e.residual) v += load4(e.residual, e.ld_res, r, c, e.cols);
    if (e.out_f32) store4_f32(out, e.ld_out, r, c, v);
    else store4(out, e.ld_out, r, c, e.cols, v);
  }
  template <int ACT>
  __device__ void gated(int r, int c, f32x4 g, f32x4 u) const {
    g *= s0;
    u *= s1;
    if (e.z[0]) {
      store4(e.z[0], e.cols, r, c, e.cols, g);
      store4(e.z[1], e.cols, r, c, e.cols, u);
    }
    f32x4 h;
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = act_value<ACT>(g[k]) * u[k];
    store4(out, e.ld_out, r, c, e.cols, h);
  }
};

// One product's split sums joined in split order (so the result does not depend on which
// workgroup finished first), then its epilogue: a thread per four columns.  `block` of `blocks`
// workgroups.
__device__ inline void join_part(const JoinArgs& a, int block, int blocks) {
  const int cg = (a.e.cols + 3) >> 2;
  const long long total = (long long)a.e.rows * cg * a.batches;
  const size_t plane = (size_t)a.e.rows * a.ldp;
  const int planes = a.gated ? 2 : a.batches;
  for (long long i = (long long)block * blockDim.x + threadIdx.x; i < total;
       i += (long long)blocks * blockDim.x) {
    const int c = (int)(i % cg) * 4;
    const long long rr = i / cg;
    const int r = (int)(rr % a.e.rows), b = (int)(rr / a.e.rows);
    const float* p = a.part + (size_t)b * plane + (size_t)r * a.ldp + c;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f}, u = v;
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
      const float* q = p + (size_t)s * planes * plane;
      v += *(const f32x4*)q;
      if (a.gated) u += *(const f32x4*)(q + plane);
    }
    const Epilogue ep(a.e, b);
    act_switch(a.e.act, [&](auto act) {
      if (a.gated) ep.gated<decltype(act)::value>(r, c, v, u);
      else ep.linear<decltype(act)::value>(r, c, v);
    });
  }
}

__device__ inline void join_body(const JoinPair& a) {
  const int b = (int)blockIdx.x, first = a.part[0].blocks;
  if (b < first) join_part(a.part[0], b, first);
  else join_part(a.part[1], b - first, a.part[1].blocks);
}

}  // namespace ringag
