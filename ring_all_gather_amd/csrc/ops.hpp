// Internal interface of the block operators (layer norm, fused linear, gated feed-forward) between
// the host runtime (ops_runtime.cpp, ops_launch.cpp) and their device code (ops_kernels.hip):
// kernel argument structs and launchers.  Nothing here is part of the public ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace ringag {

// What an epilogue does with the finished sums of one product (or of the gate and up products):
//   linear  z = v * scale + bias[c];  Z = z;  out = act(z) + residual       (out bf16 or fp32)
//   gated   g, u = the two products;  G = g, U = u;  out = act(g) * u
// Every pointer but `out` may be null.  Row strides are in elements.
struct EpiArgs {
  const float* scale_x;        // fp8 inputs: dequantisation factors (device scalars)
  const float* scale_w[2];
  const void* bias;            // [cols] bf16
  const void* residual;        // [rows, cols] bf16, row stride ld_res
  void* z[2];                  // [rows, cols] bf16: pre-activation, or G and U
  void* out[2];                // [rows, cols] with row stride ld_out; by batch
  long long ld_res, ld_out;
  int act;
  int out_f32;
  int rows, cols;
};

// One (batched, split) product out[i][j] = sum_k X[i][k] Y[j][k].  Operands are K-contiguous
// (row i or j, then k) or K-strided (row k, then i or j); ldx / ldy are row strides in bytes.
struct GemmArgs {
  const void* x[2];            // by batch
  const void* y[2];            // K-contiguous: the weight, or the gate and up weights of the gated
                               // form; K-strided: by K segment
  long long ldx, ldy;
  int xk, yk;                  // K-strided operands: rows of K that exist (per segment)
  int xcols, ycols;            // K-strided operands: columns that exist (a multiple of 8)
  int ksteps;                  // K stages of the whole product
  int kseg;                    // K stages of the first K segment of Y (ksteps if there is one)
  int tiles_i, tiles_j, batches, splits;
  int blocks;                  // workgroups
  int whole;                   // the first ones run a whole tile each; two share each later tile
  float* part;                 // splits > 1: [split][batch or gate/up][rows][ldp] fp32 sums
  long long ldp;
  EpiArgs e;
};

// dX and dW in one launch; either may have no workgroups.
struct BackwardArgs {
  GemmArgs dx, dw;
  int dx_first;
};

// Joins the split sums of a product in split order and runs its epilogue.
struct JoinArgs {
  const float* part;
  long long ldp;
  int splits, batches, gated;
  int blocks;                  // workgroups (set by the launcher)
  EpiArgs e;
};
struct JoinPair {
  JoinArgs part[2];            // the second may have no rows
};

// A product with at most 32 rows of X: streams the weight once.  Forms: 16 rows of X at most, the
// same with twice the weight rows per workgroup, and 32 rows.
enum OpsFew { kFew16 = 0, kFew16x2, kFew32, kFewForms };
struct SkinnyArgs {
  const void* x;
  const void* w[2];
  long long ldx, ldw;          // bytes
  int kblocks;                 // 128-byte blocks of K
  EpiArgs e;
};

// dZ = dY * act'(Z) (linear) or dG = dH U act'(G), dU = dH act(G) (gated), rounded to bf16 with
// the columns past `cols` up to cols_pad zero, and the column sums of the unrounded dZ by slab.
struct ActGradArgs {
  const void* dy;              // [rows, cols] bf16, row stride ld_dy
  const void* z;               // Z, or G
  const void* u;               // U (gated) or null
  void* dz;                    // [rows, ld_dz] bf16 or null
  float* colsum;               // [slabs][cols] or null
  long long ld_dy, ld_z, ld_dz;
  int rows, cols, cols_pad, slab_rows, slabs;
  int tx;                      // threads across the columns: 8, 16, 32 or 64
  int act, gated;
  int stream;                  // 1 = more data than the last-level cache holds
};

struct NormArgs {
  const void* x;
  const void* dy;              // backward
  const void* w;
  const void* b;               // or null
  void* y;                     // y, or dx
  float* mean;                 // forward: written when not null; backward: read
  float* rstd;
  float* part;                 // backward: column sums of dw by workgroup, 2 H apart
  float* part_db;              // ... of db
  long long ld_x, ld_dy;
  int T, H;
  float eps;
};

// out0[n] = sum over s of part[s][n] for n < n0, out1[n - n0] for n0 <= n < n0 + n1.
struct ColSumArgs {
  const float* part;
  long long ld;
  int slabs, n0, n1;
  float* out0;
  float* out1;                 // or null: those columns are not stored
};

enum OpsTile { kOps256 = 0, kOps128, kOps128Deep, kOpsTiles };
inline void ops_tile_dims(int tile, int* bi, int* bj) { *bi = *bj = tile == kOps256 ? 256 : 128; }

// GEMM forms: forward linear (bf16, fp8), forward gated (bf16, fp8), dX (X K-contiguous, Y
// K-strided), dW (both K-strided); the last two share the kernels of kGemmBackward.
enum OpsGemm { kGemmLin = 0, kGemmLin8, kGemmGated, kGemmGated8, kGemmBackward, kOpsGemms,
               kGemmDx, kGemmDw };
// Norm element types: x / y of bf16 / bf16, fp32 / fp32, fp32 / bf16; with an fp32 weight + kNormWF.
enum OpsNormType { kNormBB = 0, kNormFF, kNormFB, kNormWF, kNormTypes = 2 * kNormWF };
// Norm forms: 8-column vectors a thread holds (0 = any width, rows read again).
enum OpsNormForm { kNorm0 = 0, kNorm1, kNorm2, kNorm4, kNormForms };
// Rows: whole 4-byte words, the same streamed past the caches (not kNorm0), odd bf16 ones.
enum OpsNormRows { kRowsWords = 0, kRowsStream, kRowsOdd, kNormRows };

// Names of the products' entry points, written to buf.
const char* ops_gemm_name(int kind, int tile, char* buf, size_t len);
const char* ops_few_name(bool gated, bool fp8, int form, char* buf, size_t len);

hipError_t load_ops_kernels(int device);
hipError_t launch_ops_gemm(int device, int kind, int tile, const GemmArgs& a, hipStream_t s);
hipError_t launch_backward_gemm(int device, int tile, const BackwardArgs& a, hipStream_t s);
hipError_t launch_join(int device, const JoinPair& a, hipStream_t s);
hipError_t launch_skinny(int device, bool gated, bool fp8, int form, const SkinnyArgs& a,
                         hipStream_t s);
hipError_t launch_act_grad(int device, const ActGradArgs& a, hipStream_t s);
hipError_t launch_colsum(int device, const ColSumArgs& a, hipStream_t s);
hipError_t launch_norm(int device, bool backward, int type, int form, int rows, int threads,
                       int grid, const NormArgs& a, hipStream_t s);

}  // namespace ringag
