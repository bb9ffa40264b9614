// Linear layer with a fused epilogue, and its gradients.
//
//   z = x w^T + b,  y = act(z) + r
//   dz = dy act'(pre),  dx = dz w,  dw = dz^T x,  db = sum over rows of dz
#include "kernels.h"
#include "layer.cuh"

namespace ozemu {

namespace {

constexpr int kTile = 64, kDepth = 16, kThreads = 256;

// D(i, j) = sum_p A(i, p) B(j, p), element (i, p) of an operand at
// i * outer + p * inner.
struct Operand {
  const void* p;
  long long outer, inner;
};
struct ProductArgs {
  int m, n, k;
  Operand a, b;
  const void* bias;
  const void* res;
  long long ldr;
  void* pre;
  long long ldpre;
  void* out;
  long long ldo;
  int act;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) product_kernel(const ProductArgs g) {
  __shared__ float sa[kDepth][kTile + 1], sb[kDepth][kTile + 1];
  const int i0 = blockIdx.y * kTile, j0 = blockIdx.x * kTile;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int p0 = 0; p0 < g.k; p0 += kDepth) {
    for (int e = threadIdx.x; e < kTile * kDepth; e += kThreads) {
      const int i = e / kDepth, p = e % kDepth;
      const bool in = p0 + p < g.k;
      sa[p][i] = in && i0 + i < g.m
                     ? to_float(static_cast<const T*>(g.a.p)[(i0 + i) * g.a.outer + (p0 + p) * g.a.inner])
                     : 0.f;
      sb[p][i] = in && j0 + i < g.n
                     ? to_float(static_cast<const T*>(g.b.p)[(j0 + i) * g.b.outer + (p0 + p) * g.b.inner])
                     : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < kDepth; ++p)
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[u][v] += sa[p][ty + 16 * u] * sb[p][tx + 16 * v];
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int i = i0 + ty + 16 * u, j = j0 + tx + 16 * v;
      if (i >= g.m || j >= g.n) continue;
      float z = acc[u][v];
      if (g.bias) z += to_float(static_cast<const T*>(g.bias)[j]);
      if (g.pre) static_cast<T*>(g.pre)[i * g.ldpre + j] = from_float<T>(z);
      float y = activate(z, g.act);
      if (g.res) y += to_float(static_cast<const T*>(g.res)[i * g.ldr + j]);
      static_cast<T*>(g.out)[i * g.ldo + j] = from_float<T>(y);
    }
}

// dz = dy act'(pre) into a dense m x n array, one thread per column so that
// db sums the unrounded values in row order.
template <typename T>
__global__ void __launch_bounds__(kThreads) slope_kernel(const LinearGradCall c, T* dz) {
  const int j = blockIdx.x * kThreads + threadIdx.x;
  if (j >= c.n) return;
  float s = 0.f;
  for (long long i = 0; i < c.m; ++i) {
    float v = to_float(static_cast<const T*>(c.dy)[i * c.lddy + j]);
    if (c.act != kActNone) v *= activation_slope(to_float(static_cast<const T*>(c.pre)[i * c.ldpre + j]), c.act);
    s += v;
    dz[i * c.n + j] = from_float<T>(v);
  }
  if (c.db) static_cast<T*>(c.db)[j] = from_float<T>(s);
}

template <typename T>
void run_product(const ProductArgs& g, cudaStream_t stream) {
  product_kernel<T><<<dim3((g.n + kTile - 1) / kTile, (g.m + kTile - 1) / kTile), kThreads, 0, stream>>>(g);
}

template <typename T>
cudaError_t linear_t(const LinearCall& c, cudaStream_t stream) {
  ProductArgs g = {c.m, c.n, c.k, {c.x, c.ldx, 1}, {c.w, c.ldw, 1}, c.bias, c.res, c.ldr, c.pre, c.ldpre,
                   c.y, c.ldy, c.act};
  run_product<T>(g, stream);
  return cudaGetLastError();
}

template <typename T>
cudaError_t linear_backward_t(const LinearGradCall& c, cudaStream_t stream) {
  T* dz = static_cast<T*>(c.ws);
  if (c.n > 0) slope_kernel<T><<<(c.n + kThreads - 1) / kThreads, kThreads, 0, stream>>>(c, dz);
  if (c.dx && c.m > 0 && c.k > 0) {
    ProductArgs g = {c.m, c.k, c.n, {dz, c.n, 1}, {c.w, 1, c.ldw}, nullptr, nullptr, 0, nullptr, 0,
                     c.dx, c.lddx, kActNone};
    run_product<T>(g, stream);
  }
  if (c.dw && c.n > 0 && c.k > 0) {
    ProductArgs g = {c.n, c.k, c.m, {dz, 1, c.n}, {c.x, 1, c.ldx}, nullptr, nullptr, 0, nullptr, 0,
                     c.dw, c.lddw, kActNone};
    run_product<T>(g, stream);
  }
  return cudaGetLastError();
}

}  // namespace

size_t linear_workspace(const LinearCall&) { return 0; }

cudaError_t launch_linear(const LinearCall& c, cudaStream_t stream) {
  return c.type == kF16 ? linear_t<__half>(c, stream) : linear_t<__nv_bfloat16>(c, stream);
}

size_t linear_backward_workspace(const LinearGradCall& c) { return static_cast<size_t>(c.m) * c.n * 2; }

cudaError_t launch_linear_backward(const LinearGradCall& c, cudaStream_t stream) {
  return c.type == kF16 ? linear_backward_t<__half>(c, stream) : linear_backward_t<__nv_bfloat16>(c, stream);
}

}  // namespace ozemu
