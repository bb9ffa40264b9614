// Element types, activations and small reductions of the layer operators
// (linear.cu, layernorm.cu).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace ozemu {

// Element types and activations, numbered as in the C ABI.
enum LayerType { kBf16 = 0, kF16 = 1, kF32 = 2 };
enum Activation { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

inline int type_bytes(int type) { return type == kF32 ? 4 : 2; }

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __half from_float<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// act(z).  NaN passes through every activation (relu by its comparison); the
// tanh form is written with 1/2 (1 + tanh u) = 1 / (1 + e^(-2u)).
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case kActRelu:
      return z < 0.f ? 0.f : z;
    case kActGelu:
      return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    case kActGeluTanh:
      return z / (1.f + expf(-2.f * kGeluC * z * (1.f + kGeluA * z * z)));
    case kActSilu:
      return z / (1.f + expf(-z));
    default:
      return z;
  }
}

// act'(z).  The factors that multiply an already vanished exponential take z
// limited to +-64 (where it has vanished), so that a large z gives the limit
// 0 or 1 and not 0 * inf.
__device__ __forceinline__ float activation_slope(float z, int act) {
  const float zc = fminf(fmaxf(z, -64.f), 64.f);
  switch (act) {
    case kActRelu:
      return z > 0.f ? 1.f : 0.f;
    case kActGelu:
      return 0.5f * (1.f + erff(z * 0.70710678118654752f)) + zc * expf(-0.5f * zc * zc) * 0.3989422804014327f;
    case kActGeluTanh: {
      const float s = 1.f / (1.f + expf(-2.f * kGeluC * z * (1.f + kGeluA * z * z)));
      return s + zc * s * (1.f - s) * 2.f * kGeluC * (1.f + 3.f * kGeluA * zc * zc);
    }
    case kActSilu: {
      const float s = 1.f / (1.f + expf(-z));
      return s * (1.f + zc * (1.f - s));
    }
    default:
      return 1.f;
  }
}

}  // namespace ozemu
