// Element types, activations and small reductions of the layer operators
// (linear.cu, layernorm.cu).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"

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

// Two 16-bit elements in one word (the lower address in the low half).
template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  static constexpr bool kBf16 = true;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t v) {  // bf16 is the upper half of an fp32
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  }
};
template <>
struct Pair<__half> {
  static constexpr bool kBf16 = false;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
};

// Arithmetic on two fp32 at once (each rounded as its scalar form).
__device__ __forceinline__ unsigned long long f2_bits(float2 a) {
  return static_cast<unsigned long long>(__float_as_uint(a.x)) |
         (static_cast<unsigned long long>(__float_as_uint(a.y)) << 32);
}
__device__ __forceinline__ float2 f2_of(unsigned long long v) {
  return make_float2(__uint_as_float(static_cast<uint32_t>(v)), __uint_as_float(static_cast<uint32_t>(v >> 32)));
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return f2_of(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
  return f2_of(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
  return f2_of(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// A 16-byte vector of elements and its floats, as pairs of consecutive ones.
template <typename T>
__device__ __forceinline__ void unpack16(const uint4& u, float2* v) {
  if constexpr (sizeof(T) == 4) {
    v[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    v[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  } else {
    v[0] = Pair<T>::unpack(u.x);
    v[1] = Pair<T>::unpack(u.y);
    v[2] = Pair<T>::unpack(u.z);
    v[3] = Pair<T>::unpack(u.w);
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack16(const float2* v) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                      __float_as_uint(v[1].y));
  else
    return make_uint4(Pair<T>::pack(v[0].x, v[0].y), Pair<T>::pack(v[1].x, v[1].y), Pair<T>::pack(v[2].x, v[2].y),
                      Pair<T>::pack(v[3].x, v[3].y));
}

// A 16-byte vector of elements and its floats.
template <typename T>
__device__ __forceinline__ void unpack16(const uint4& u, float* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      v[i] = __uint_as_float(w[i]);
    } else {
      const float2 f = Pair<T>::unpack(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack16(const float* v) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  else
    return make_uint4(Pair<T>::pack(v[0], v[1]), Pair<T>::pack(v[2], v[3]), Pair<T>::pack(v[4], v[5]),
                      Pair<T>::pack(v[6], v[7]));
}

constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// The normal distribution's tail Phi(-a) = e^(-a^2/2) t P(t), t = 1 / (1 + p a),
// for a >= 0: the form of 7.1.26 of Abramowitz and Stegun's Handbook with two
// more coefficients, fitted by linear programming so that the largest error
// relative to Phi(-a) over 0 <= a <= 14.5 is least: 6.0e-7 (2^-20.6).  (Their
// five coefficients keep the absolute error below 1.5e-7, which is 5e-4 of the
// tail at a = 4 and 4e-3 at 6: more than the rounding to 16 bits.)  The fp32
// evaluation adds some 1e-6, the exponential a^2 2^-24.  The two more steps cost
// the pass over the slopes (8192 x 16384) 4 us of 159, the product 8192 x 4096 ->
// 16384 2 of 573.
constexpr float kTailP = 0.265f;
__device__ __forceinline__ constexpr float tail_coefficient(int i) {
  constexpr float c[7] = {0.105598755f,   0.107850529f, 0.0828776509f, 0.142668769f,
                          -0.0666030422f, 0.195441261f, -0.0678342208f};
  return c[i];
}

// The normal distribution function Phi(z) = 1/2 (1 + erf(z / sqrt 2)).  On the
// negative side the tail itself is formed, without cancellation.
__device__ __forceinline__ float normal_cdf(float z) {
  const float t = __fdividef(1.f, fmaf(kTailP, fabsf(z), 1.f));
  float q = tail_coefficient(6);
#pragma unroll
  for (int i = 5; i >= 0; --i) q = fmaf(t, q, tail_coefficient(i));
  q *= t * __expf(-0.5f * z * z);
  return z < 0.f ? q : 1.f - q;
}

// act(z).  NaN passes through every activation (relu by its comparison).
// gelu_tanh is written with 1/2 (1 + tanh u) = 1 / (1 + e^(-2u)).  Where the
// exponential's argument is a, the fast exponential, the quotient and gelu's tail
// are together within 2^-19 + (1 + |a|) 2^-22 of the result, relative to it,
// against the 2^-9 and 2^-12 that its 16-bit rounding takes.  (A quotient by more
// than 2^126 is 0: silu and gelu_tanh where they are below 2^-119.)
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case kActRelu:
      return z < 0.f ? 0.f : z;
    case kActGelu:
      return z * normal_cdf(z);
    case kActGeluTanh:
      return __fdividef(z, 1.f + __expf(-2.f * kGeluC * z * fmaf(kGeluA * z, z, 1.f)));
    case kActSilu:
      return __fdividef(z, 1.f + __expf(-z));
    default:
      return z;
  }
}

__device__ __forceinline__ float2 exp2_2(float2 v) {
  float2 r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(v.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 reciprocal2(float2 v) {
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(v.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(v.y));
  return r;
}

// act'(z) of two values at once: a pass over the gradients is bound by the
// instructions of this.  The factors that multiply an already vanished
// exponential take z limited to +-64 (where it has vanished), so that a large
// or infinite z gives the limit 0 or 1 and not 0 * inf; a NaN stays one through
// the other factors.
template <int kAct>
__device__ __forceinline__ float2 activation_slope2(float2 z) {
  const float2 one = both(1.f);
  const float2 zc = make_float2(fminf(fmaxf(z.x, -64.f), 64.f), fminf(fmaxf(z.y, -64.f), 64.f));
  if constexpr (kAct == kActRelu) {
    return make_float2(z.x > 0.f ? 1.f : 0.f, z.y > 0.f ? 1.f : 0.f);
  } else if constexpr (kAct == kActGelu) {  // Phi(z) + z phi(z); one exponential serves both
    const float2 a = make_float2(fabsf(z.x), fabsf(z.y));
    const float2 t = reciprocal2(fma2(a, both(kTailP), one));
    float2 q = both(tail_coefficient(6));
#pragma unroll
    for (int i = 5; i >= 0; --i) q = fma2(t, q, both(tail_coefficient(i)));
    const float2 e = exp2_2(mul2(mul2(z, z), both(-0.5f * 1.4426950408889634f)));
    q = mul2(mul2(q, t), e);
    const float2 p = make_float2(z.x < 0.f ? q.x : 1.f - q.x, z.y < 0.f ? q.y : 1.f - q.y);
    return fma2(mul2(zc, both(0.3989422804014327f)), e, p);
  } else if constexpr (kAct == kActGeluTanh) {  // s + z s (1 - s) 2 u'(z), s = 1 / (1 + e^(-2u))
    const float2 zz = mul2(z, z);
    const float2 u = mul2(mul2(z, both(-2.f * kGeluC * 1.4426950408889634f)), fma2(zz, both(kGeluA), one));
    const float2 s = reciprocal2(add2(exp2_2(u), one));
    const float2 du = fma2(mul2(zc, zc), both(6.f * kGeluC * kGeluA), both(2.f * kGeluC));
    return fma2(mul2(mul2(zc, s), fma2(s, both(-1.f), one)), du, s);
  } else if constexpr (kAct == kActSilu) {  // s (1 + z (1 - s)), s = 1 / (1 + e^(-z))
    const float2 s = reciprocal2(add2(exp2_2(mul2(z, both(-1.4426950408889634f))), one));
    return mul2(s, fma2(zc, fma2(s, both(-1.f), one), one));
  } else {
    return one;
  }
}

// out[s][j] = sum over the `used` parts of part[s][.][j], s = blockIdx.y: 32
// columns a CTA, 32 threads to a column, each taking every 32nd part in order.
// A NULL output is not wanted.
template <typename W>
static __global__ void __launch_bounds__(1024) join_parts_kernel(const float* part, int used, int parts, int cols, W* out0,
                                                          W* out1) {
  __shared__ float red[32][33];
  chain_next();
  chain_wait();
  W* out = blockIdx.y == 0 ? out0 : out1;
  if (!out) return;
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, j = blockIdx.x * 32 + tx;
  const float* p = part + static_cast<long long>(blockIdx.y) * parts * cols + j;
  float s = 0.f;
  if (j < cols) {
#pragma unroll 4
    for (int k = ty; k < used; k += 32) s += p[static_cast<long long>(k) * cols];
  }
  red[ty][tx] = s;
  __syncthreads();
  s = red[tx][ty];  // column ty of the CTA, its 32 partial sums across a warp
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (tx == 0 && blockIdx.x * 32 + ty < cols) out[blockIdx.x * 32 + ty] = from_float<W>(s);
}

}  // namespace ozemu
