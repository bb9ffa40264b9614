// Layer norm, forward and backward.
//
//   y  = (x - mean) rstd w + b,  mean = 1/H sum x,  rstd = (1/H sum (x - mean)^2 + eps)^(-1/2)
//   dx = rstd (g - mean(g) - xhat mean(g xhat)) + dr,  g = dy w,  xhat = (x - mean) rstd
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
//
// All sums and statistics are fp32.
#include "kernels.h"
#include "layer.cuh"

namespace ozemu {

namespace {

constexpr int kThreads = 256;

// Sum over the CTA, returned to every thread; `red` holds one word per warp.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < kThreads / 32; ++w) s += red[w];
  return s;
}

template <typename T, typename W>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(const NormCall c) {
  __shared__ float red[kThreads / 32];
  const float inv = 1.f / static_cast<float>(c.cols);
  for (int row = blockIdx.x; row < c.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(c.x) + row * c.ldx;
    T* y = static_cast<T*>(c.y) + row * c.ldy;
    float s = 0.f;
    for (int j = threadIdx.x; j < c.cols; j += kThreads) s += to_float(x[j]);
    const float mean = block_sum(s, red) * inv;
    s = 0.f;
    for (int j = threadIdx.x; j < c.cols; j += kThreads) {
      const float d = to_float(x[j]) - mean;
      s += d * d;
    }
    const float rstd = 1.f / sqrtf(block_sum(s, red) * inv + c.eps);
    for (int j = threadIdx.x; j < c.cols; j += kThreads) {
      float v = (to_float(x[j]) - mean) * rstd;
      if (c.weight) v *= to_float(static_cast<const W*>(c.weight)[j]);
      if (c.bias) v += to_float(static_cast<const W*>(c.bias)[j]);
      y[j] = from_float<T>(v);
    }
    if (threadIdx.x == 0) {
      if (c.mean) c.mean[row] = mean;
      if (c.rstd) c.rstd[row] = rstd;
    }
  }
}

template <typename T, typename W>
__global__ void __launch_bounds__(kThreads) norm_backward_rows_kernel(const NormGradCall c) {
  __shared__ float red[kThreads / 32];
  const float inv = 1.f / static_cast<float>(c.cols);
  for (int row = blockIdx.x; row < c.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(c.x) + row * c.ldx;
    const T* dy = static_cast<const T*>(c.dy) + row * c.lddy;
    const T* dr = c.dr ? static_cast<const T*>(c.dr) + row * c.lddr : nullptr;
    T* dx = static_cast<T*>(c.dx) + row * c.lddx;
    const float mean = c.mean[row], rstd = c.rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int j = threadIdx.x; j < c.cols; j += kThreads) {
      const float g = to_float(dy[j]) * (c.weight ? to_float(static_cast<const W*>(c.weight)[j]) : 1.f);
      s1 += g;
      s2 += g * ((to_float(x[j]) - mean) * rstd);
    }
    s1 = block_sum(s1, red) * inv;
    s2 = block_sum(s2, red) * inv;
    for (int j = threadIdx.x; j < c.cols; j += kThreads) {
      const float g = to_float(dy[j]) * (c.weight ? to_float(static_cast<const W*>(c.weight)[j]) : 1.f);
      float v = rstd * (g - s1 - (to_float(x[j]) - mean) * rstd * s2);
      if (dr) v += to_float(dr[j]);
      dx[j] = from_float<T>(v);
    }
  }
}

// One thread per column, rows in order.
template <typename T, typename W>
__global__ void __launch_bounds__(kThreads) norm_backward_cols_kernel(const NormGradCall c) {
  const int j = blockIdx.x * kThreads + threadIdx.x;
  if (j >= c.cols) return;
  float sw = 0.f, sb = 0.f;
  for (int row = 0; row < c.rows; ++row) {
    const float dy = to_float(static_cast<const T*>(c.dy)[row * c.lddy + j]);
    sb += dy;
    sw += dy * ((to_float(static_cast<const T*>(c.x)[row * c.ldx + j]) - c.mean[row]) * c.rstd[row]);
  }
  if (c.dweight) static_cast<W*>(c.dweight)[j] = from_float<W>(sw);
  if (c.dbias) static_cast<W*>(c.dbias)[j] = from_float<W>(sb);
}

template <typename F>
cudaError_t with_types(int type, int param_type, F f) {
  if (type == kBf16) return param_type == kF32 ? f(__nv_bfloat16{}, float{}) : f(__nv_bfloat16{}, __nv_bfloat16{});
  if (type == kF16) return param_type == kF32 ? f(__half{}, float{}) : f(__half{}, __half{});
  return f(float{}, float{});
}

}  // namespace

cudaError_t launch_layer_norm(const NormCall& c, cudaStream_t stream) {
  return with_types(c.type, c.param_type, [&](auto t, auto w) {
    norm_forward_kernel<decltype(t), decltype(w)><<<c.rows < 65536 ? c.rows : 65536, kThreads, 0, stream>>>(c);
    return cudaGetLastError();
  });
}

size_t layer_norm_backward_workspace(int, int) { return 0; }

cudaError_t launch_layer_norm_backward(const NormGradCall& c, cudaStream_t stream) {
  return with_types(c.type, c.param_type, [&](auto t, auto w) {
    // The columns first: dx may be dy itself.
    if (c.dweight || c.dbias)
      norm_backward_cols_kernel<decltype(t), decltype(w)>
          <<<(c.cols + kThreads - 1) / kThreads, kThreads, 0, stream>>>(c);
    if (c.rows > 0)
      norm_backward_rows_kernel<decltype(t), decltype(w)>
          <<<c.rows < 65536 ? c.rows : 65536, kThreads, 0, stream>>>(c);
    return cudaGetLastError();
  });
}

}  // namespace ozemu
