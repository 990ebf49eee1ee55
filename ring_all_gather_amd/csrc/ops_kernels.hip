// GPU code of the block operators (layer norm, fused linear, gated feed-forward), compiled on its
// own into a second gfx950 code object, so that the ring kernels' object does not change with it.
//
// Entry points:
//   rag_lin_<bf16|fp8>_<tile>, rag_ffn_<bf16|fp8>_<tile>   forward products with their epilogues
//                                                          (tiles t256, t128, t128d)
//   rag_backward_<tile>                                    both products of a backward pass
//   rag_join                                               split sums and their epilogue
//   rag_lin_<bf16|fp8>_few<16|16x2|32>, rag_ffn_...        products with at most 32 rows of X
//   rag_act_grad[_s], rag_ffn_grad[_s]                     the elementwise half of the backward
//   rag_colsum                                             column sums of bias and norm gradients
//   rag_ln_<fwd|bwd>_<x, y, weight type: b or f>_<v0|v1|v2|v4>[_s|_u]
//                                                          layer norm (_s: streamed rows, _u: odd
//                                                          bf16 rows)
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ops.hpp"
#include "ringag.h"

// Everything is inlined into its kernel: accumulators passed to a call would live in memory, and
// the K loop's descriptors have to stay in scalar registers.
#pragma clang attribute push(__attribute__((always_inline)), apply_to = function)
#include "act_grad.hpp"
#include "block_gemm.hpp"
#include "norm_kernel.hpp"
#include "skinny_gemm.hpp"
#pragma clang attribute pop

using namespace ringag;

// 256x256 and four-stage 128x128: one workgroup per compute unit (two waves per SIMD); two-stage
// 128x128: two (four waves per SIMD)
#define RAG_GEMM_ENTRY(NAME, ARGS, BODY256, BODY128, BODY128D)                                  \
  extern "C" __global__ void __launch_bounds__(512, 2) NAME##_t256(ARGS a) { BODY256(a); }      \
  extern "C" __global__ void __launch_bounds__(512, 4) NAME##_t128(ARGS a) { BODY128(a); }      \
  extern "C" __global__ void __launch_bounds__(512, 2) NAME##_t128d(ARGS a) { BODY128D(a); }
#define RAG_FORWARD_ENTRY(NAME, KIND)                                                           \
  RAG_GEMM_ENTRY(NAME, GemmArgs, (block_gemm_body<OpsTile256, OpsTile256Half, KIND>),           \
                 (block_gemm_body<OpsTile128, OpsTile128, KIND>),                               \
                 (block_gemm_body<OpsTile128Deep, OpsTile128Deep, KIND>))
RAG_FORWARD_ENTRY(rag_lin_bf16, kGemmLin)
RAG_FORWARD_ENTRY(rag_lin_fp8, kGemmLin8)
RAG_FORWARD_ENTRY(rag_ffn_bf16, kGemmGated)
RAG_FORWARD_ENTRY(rag_ffn_fp8, kGemmGated8)
RAG_GEMM_ENTRY(rag_backward, BackwardArgs, (backward_gemm_body<OpsTile256, OpsTile256Half>),
               (backward_gemm_body<OpsTile128, OpsTile128>),
               (backward_gemm_body<OpsTile128Deep, OpsTile128Deep>))

extern "C" __global__ void __launch_bounds__(256) rag_join(JoinPair a) { join_body(a); }

#define RAG_FEW_ENTRY1(NAME, GATED, FP8, SUFFIX, TB, RB)                                        \
  extern "C" __global__ void __launch_bounds__(skinny_waves<GATED>() * 64) NAME##_##SUFFIX(     \
      SkinnyArgs a) {                                                                           \
    skinny_body<GATED, FP8, TB, RB>(a);                                                         \
  }
#define RAG_FEW_ENTRY(NAME, GATED, FP8)                \
  RAG_FEW_ENTRY1(NAME, GATED, FP8, few16, 1, 1)        \
  RAG_FEW_ENTRY1(NAME, GATED, FP8, few16x2, 1, 2)      \
  RAG_FEW_ENTRY1(NAME, GATED, FP8, few32, 2, 1)
RAG_FEW_ENTRY(rag_lin_bf16, false, false)
RAG_FEW_ENTRY(rag_lin_fp8, false, true)
RAG_FEW_ENTRY(rag_ffn_bf16, true, false)
RAG_FEW_ENTRY(rag_ffn_fp8, true, true)

#define RAG_GRAD_ENTRY(NAME, GATED, STREAM)                                       \
  extern "C" __global__ void __launch_bounds__(256) NAME(ActGradArgs a) {         \
    act_grad_body<GATED, STREAM>(a);                                              \
  }
RAG_GRAD_ENTRY(rag_act_grad, false, false)
RAG_GRAD_ENTRY(rag_act_grad_s, false, true)
RAG_GRAD_ENTRY(rag_ffn_grad, true, false)
RAG_GRAD_ENTRY(rag_ffn_grad_s, true, true)
extern "C" __global__ void __launch_bounds__(1024) rag_colsum(ColSumArgs a) { colsum_body(a); }

// Threads per row at most: forward 1024 (four vectors per thread: 512); backward 1024, for bf16
// rows 512 with two or four vectors (the only ones that have four).
template <class XT>
constexpr int norm_bwd_threads(int nv) {
  return sizeof(XT) == 2 && nv > 1 ? 512 : 1024;
}
#define RAG_LN_ENTRY1(TYPES, XT, YT, WT, V, NV, SUFFIX, BUF, POLICY)                               \
  extern "C" __global__ void __launch_bounds__(NV > 2 ? 512 : 1024, 4)                           \
      rag_ln_fwd_##TYPES##_##V##SUFFIX(NormArgs a) {                                             \
    norm_fwd_body<XT, YT, WT, NV, BUF, POLICY>(a);                                                 \
  }                                                                                              \
  extern "C" __global__ void                                                                     \
      __launch_bounds__((norm_bwd_threads<XT>(NV))) rag_ln_bwd_##TYPES##_##V##SUFFIX(NormArgs a) { \
    norm_bwd_body<XT, YT, WT, NV, BUF, POLICY>(a);                                                 \
  }
#define RAG_LN_ENTRY(TYPES, XT, YT, WT, SUFFIX, BUF, POLICY)       \
  RAG_LN_ENTRY1(TYPES, XT, YT, WT, v1, 1, SUFFIX, BUF, POLICY)     \
  RAG_LN_ENTRY1(TYPES, XT, YT, WT, v2, 2, SUFFIX, BUF, POLICY)
#define RAG_LN_WORDS(TYPES, XT, YT, WT)                            \
  RAG_LN_ENTRY1(TYPES, XT, YT, WT, v0, 0, , true, kCached)         \
  RAG_LN_ENTRY(TYPES, XT, YT, WT, , true, kCached)                 \
  RAG_LN_ENTRY(TYPES, XT, YT, WT, _s, true, kStream)
#define RAG_LN_ODD(TYPES, XT, YT, WT)                              \
  RAG_LN_ENTRY1(TYPES, XT, YT, WT, v0, 0, _u, false, kCached)      \
  RAG_LN_ENTRY(TYPES, XT, YT, WT, _u, false, kCached)
RAG_LN_WORDS(bbb, __bf16, __bf16, __bf16)
RAG_LN_WORDS(ffb, float, float, __bf16)
RAG_LN_WORDS(fbb, float, __bf16, __bf16)
RAG_LN_WORDS(bbf, __bf16, __bf16, float)
RAG_LN_WORDS(fff, float, float, float)
RAG_LN_WORDS(fbf, float, __bf16, float)
RAG_LN_ENTRY1(bbb, __bf16, __bf16, __bf16, v4, 4, , true, kCached)
RAG_LN_ENTRY1(bbf, __bf16, __bf16, float, v4, 4, , true, kCached)
RAG_LN_ENTRY1(bbb, __bf16, __bf16, __bf16, v4, 4, _s, true, kStream)
RAG_LN_ENTRY1(bbf, __bf16, __bf16, float, v4, 4, _s, true, kStream)
RAG_LN_ODD(bbb, __bf16, __bf16, __bf16)
RAG_LN_ODD(ffb, float, float, __bf16)
RAG_LN_ODD(fbb, float, __bf16, __bf16)
RAG_LN_ODD(bbf, __bf16, __bf16, float)
RAG_LN_ODD(fbf, float, __bf16, float)
RAG_LN_ENTRY1(bbb, __bf16, __bf16, __bf16, v4, 4, _u, false, kCached)
RAG_LN_ENTRY1(bbf, __bf16, __bf16, float, v4, 4, _u, false, kCached)
