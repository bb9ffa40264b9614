// The host side of the layer operators without a GPU: linked with the library's objects, the CUDA runtime's calls
// replaced by these.  A launch succeeds or, the `fail`-th of a call, does not; another call's error is pending
// throughout.  Prints for a case (argv[1]) and fail = -1, 0, 1, ...: the call's status, then its launches as
// x,y,z grids.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <string>

#include <cuda.h>

#include "kernels.h"

static int g_fail = -1, g_launches = 0;
static std::string g_grids;

extern "C" {
cudaError_t __wrap_cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void*, void**) {
  char text[64];
  snprintf(text, sizeof text, " %u,%u,%u", c->gridDim.x, c->gridDim.y, c->gridDim.z);
  g_grids += text;
  return g_launches++ == g_fail ? cudaErrorMemoryAllocation : cudaSuccess;
}
cudaError_t __wrap_cudaGetDevice(int* d) {
  *d = 0;
  return cudaSuccess;
}
cudaError_t __wrap_cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t __wrap_cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
  const unsigned ctas = c->gridDim.x;
  *n = ctas == 2 ? 76 : ctas == 4 ? 36 : 15;
  return cudaSuccess;
}
cudaError_t __wrap_cudaGetLastError() { return cudaErrorUnknown; }
static CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                       const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                       CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
cudaError_t __wrap_cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long,
                                                    cudaDriverEntryPointQueryResult* q) {
  *p = reinterpret_cast<void*>(encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
}

using namespace ozemu;

static void* at(size_t p) { return reinterpret_cast<void*>(p); }

// m n k, or rows cols; leading dimensions odd where `odd`.
static cudaError_t call(const char* what, int a, int b, int c, int odd) {
  void *p = at(0x100000), *ws = at(0x200000);
  if (!strcmp(what, "linear")) {
    const LinearCall l = {a, b, c, 0, p, c + odd, p, c + odd, nullptr, nullptr, b, 0, nullptr, b, p, b, ws, nullptr};
    return launch_linear(l, nullptr);
  }
  if (!strcmp(what, "linear_backward")) {
    const LinearGradCall l = {a, b, c, 0, p, b + odd, p, c + odd, p, c + odd, 2, p, b, p, c, p, c, p, ws, nullptr};
    return launch_linear_backward(l, nullptr);
  }
  if (!strcmp(what, "norm")) {
    const NormCall n = {a, b, 0, 0, p, b + odd, nullptr, nullptr, 0.f, p, b, nullptr, nullptr, nullptr};
    return launch_layer_norm(n, nullptr);
  }
  const NormGradCall n = {a, b, 0, 0, p, b + odd, p, b + odd, nullptr, nullptr, nullptr, nullptr, b, p, b, p, p, ws,
                          nullptr};
  return launch_layer_norm_backward(n, nullptr);
}

int main(int, char** v) {
  int launches = 0;  // of the call that nothing fails in
  for (g_fail = -1; g_fail < launches; ++g_fail) {
    g_launches = 0;
    g_grids.clear();
    const cudaError_t e = call(v[1], atoi(v[2]), atoi(v[3]), atoi(v[4]), atoi(v[5]));
    printf("%d%s\n", static_cast<int>(e), g_grids.c_str());
    if (g_fail < 0) launches = g_launches;
  }
}
