// Loading and launching the block operators' kernels (ops_kernels.hip): a code object of their own,
// embedded and loaded like the ring kernels' (launch.cpp).
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cstdio>
#include <mutex>

#include "ops.hpp"

extern "C" const unsigned char ringag_ops_co[];

namespace ringag {
namespace {

constexpr int kMaxDevices = 64;

const char* const kGemmName[kOpsGemms] = {"rag_lin_bf16", "rag_lin_fp8", "rag_ffn_bf16",
                                          "rag_ffn_fp8", "rag_backward"};
const char* const kFewName[kFewForms] = {"few16", "few16x2", "few32"};
const char* const kNormType[kNormTypes] = {"bbb", "ffb", "fbb", "bbf", "fff", "fbf"};
const char* const kNormForm[kNormForms] = {"v0", "v1", "v2", "v4"};
const char* const kNormRowsName[kNormRows] = {"", "_s", "_u"};

struct OpsKernels {
  bool loaded = false;
  hipModule_t module = nullptr;
  hipFunction_t gemm[kOpsGemms][kOpsTiles] = {};
  hipFunction_t few[2][2][kFewForms] = {};                        // [gated][fp8][form]
  hipFunction_t norm[2][kNormTypes][kNormForms][kNormRows] = {};  // [backward][types][form][rows]
  hipFunction_t act_grad[2] = {}, ffn_grad[2] = {};               // [streamed]
  hipFunction_t join = nullptr, colsum = nullptr;
};

OpsKernels g_ops[kMaxDevices];
std::mutex g_ops_mu;

OpsKernels* ready(int device) {
  return device >= 0 && device < kMaxDevices && g_ops[device].loaded ? &g_ops[device] : nullptr;
}

template <class A>
hipError_t launch(hipFunction_t f, dim3 grid, int threads, const A& a, hipStream_t s) {
  if (!f) return hipErrorInvalidDeviceFunction;
  A copy = a;
  void* params[] = {&copy};
  return hipModuleLaunchKernel(f, grid.x, grid.y, 1, threads, 1, 1, 0, s, params, nullptr);
}

}  // namespace

const char* ops_gemm_name(int kind, int tile, char* buf, size_t len) {
  snprintf(buf, len, "%s_%s", kGemmName[kind],
           tile == kOps256 ? "t256" : tile == kOps128 ? "t128" : "t128d");
  return buf;
}

const char* ops_few_name(bool gated, bool fp8, int form, char* buf, size_t len) {
  snprintf(buf, len, "rag_%s_%s_%s", gated ? "ffn" : "lin", fp8 ? "fp8" : "bf16", kFewName[form]);
  return buf;
}

hipError_t load_ops_kernels(int device) {
  if (device < 0 || device >= kMaxDevices) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_ops_mu);
  OpsKernels& d = g_ops[device];
  if (d.loaded) return hipSuccess;
  hipError_t e = hipSetDevice(device);
  if (e != hipSuccess) return e;
  hipModule_t m = nullptr;
  if ((e = hipModuleLoadData(&m, ringag_ops_co)) != hipSuccess) return e;
  char name[96];
  auto get = [&](hipFunction_t* f) { return hipModuleGetFunction(f, m, name); };
  for (int k = 0; k < kOpsGemms; ++k)
    for (int t = 0; t < kOpsTiles; ++t) {
      ops_gemm_name(k, t, name, sizeof name);
      if ((e = get(&d.gemm[k][t])) != hipSuccess) return e;
    }
  for (int g = 0; g < 2; ++g)
    for (int f = 0; f < 2; ++f)
      for (int t = 0; t < kFewForms; ++t) {
        ops_few_name(g, f, t, name, sizeof name);
        if ((e = get(&d.few[g][f][t])) != hipSuccess) return e;
      }
  for (int b = 0; b < 2; ++b)
    for (int t = 0; t < kNormTypes; ++t)
      for (int f = 0; f < kNormForms; ++f)
        for (int r = 0; r < kNormRows; ++r) {
          // not built: four vectors of fp32 rows, streamed rows read again, odd fp32 rows
          if ((f == kNorm4 && t % kNormWF != kNormBB) || (f == kNorm0 && r == kRowsStream) ||
              (t == kNormFF + kNormWF && r == kRowsOdd))
            continue;
          snprintf(name, sizeof name, "rag_ln_%s_%s_%s%s", b ? "bwd" : "fwd", kNormType[t],
                   kNormForm[f], kNormRowsName[r]);
          if ((e = get(&d.norm[b][t][f][r])) != hipSuccess) return e;
        }
  for (int st = 0; st < 2; ++st) {
    snprintf(name, sizeof name, "rag_act_grad%s", st ? "_s" : "");
    if ((e = get(&d.act_grad[st])) != hipSuccess) return e;
    snprintf(name, sizeof name, "rag_ffn_grad%s", st ? "_s" : "");
    if ((e = get(&d.ffn_grad[st])) != hipSuccess) return e;
  }
  if ((e = hipModuleGetFunction(&d.join, m, "rag_join")) != hipSuccess) return e;
  if ((e = hipModuleGetFunction(&d.colsum, m, "rag_colsum")) != hipSuccess) return e;
  d.module = m;
  d.loaded = true;
  return hipSuccess;
}

hipError_t launch_ops_gemm(int device, int kind, int tile, const GemmArgs& a, hipStream_t s) {
  OpsKernels* d = ready(device);
  if (!d || kind < 0 || kind >= kGemmBackward || tile < 0 || tile >= kOpsTiles)
    return hipErrorInvalidValue;
  return launch(d->gemm[kind][tile], dim3(a.blocks), 512, a, s);
}

hipError_t launch_backward_gemm(int device, int tile, const BackwardArgs& a, hipStream_t s) {
  OpsKernels* d = ready(device);
  if (!d || tile < 0 || tile >= kOpsTiles) return hipErrorInvalidValue;
  return launch(d->gemm[kGemmBackward][tile], dim3(a.dx.blocks + a.dw.blocks), 512, a, s);
}

hipError_t launch_join(int device, const JoinPair& a, hipStream_t s) {
  OpsKernels* d = ready(device);
  if (!d) return hipErrorInvalidValue;
  JoinPair p = a;
  int grid = 0;
  for (JoinArgs& j : p.part) {
    const long long n = (long long)j.e.rows * ((j.e.cols + 3) / 4) * j.batches;
    j.blocks = (int)std::min<long long>((n + 255) / 256, 1 << 15);
    grid += j.blocks;
  }
  return launch(d->join, dim3(grid), 256, p, s);
}

hipError_t launch_skinny(int device, bool gated, bool fp8, int form, const SkinnyArgs& a,
                         hipStream_t s) {
  OpsKernels* d = ready(device);
  if (!d || form < 0 || form >= kFewForms || a.e.rows < 1 || a.e.rows > (form == kFew32 ? 32 : 16))
    return hipErrorInvalidValue;
  const int cols = (gated ? 8 : 16) * (form == kFew16x2 ? 2 : 1);   // of a workgroup
  return launch(d->few[gated][fp8][form], dim3((a.e.cols + cols - 1) / cols), gated ? 512 : 1024, a,
                s);
}

hipError_t launch_act_grad(int device, const ActGradArgs& a, hipStream_t s) {
  OpsKernels* d = ready(device);
  if (!d) return hipErrorInvalidValue;
  if (a.tx < 8 || a.tx > 64 || (a.tx & (a.tx - 1))) return hipErrorInvalidValue;
  const int width = a.tx * 8;
  return launch(a.gated ? d->ffn_grad[a.stream != 0] : d->act_grad[a.stream != 0],
                dim3((a.cols_pad + width - 1) / width, a.slabs), 256, a, s);
}

hipError_t launch_colsum(int device, const ColSumArgs& a, hipStream_t s) {
  OpsKernels* d = ready(device);
  if (!d) return hipErrorInvalidValue;
  return launch(d->colsum, dim3((a.n0 + a.n1 + 31) / 32), 1024, a, s);
}

hipError_t launch_norm(int device, bool backward, int type, int form, int rows, int threads,
                       int grid, const NormArgs& a, hipStream_t s) {
  OpsKernels* d = ready(device);
  if (!d || type < 0 || type >= kNormTypes || form < 0 || form >= kNormForms ||
      rows < 0 || rows >= kNormRows)
    return hipErrorInvalidValue;
  return launch(d->norm[backward][type][form][rows], dim3(grid), threads, a, s);
}

}  // namespace ringag
