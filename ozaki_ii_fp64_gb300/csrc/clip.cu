// Gradients of many tensors, clipped by their global norm:
//
//   N = sqrt(sum over all tensors of g^2),  g <- g min(1, max_norm / (N + eps))
//
// Two launches: the sums of squares, a partial one for each CTA, then the
// scaling, before which every CTA adds the partial sums up in the same order.
// No atomics: the same gradients give the same bits.  Squares and a thread's sum
// of 64 or fewer of them are fp32, everything after that is fp64 (one addition
// for 64 elements).  Bound by HBM: each gradient is read twice, the second time in
// the reverse order, so that what L2 still holds of the first pass (up to 129 MB)
// is read from there, and written once.
#include <algorithm>
#include <cstdint>

#include "kernels.h"
#include "layer.cuh"

namespace ozemu {

namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 152 * 4;
constexpr int kVectors = 8;                        // 16-byte vectors of a thread in a chunk
constexpr long long kChunk = kThreads * kVectors;  // vectors of a chunk

// A tensor's memory is taken in 16-byte vectors from the boundary at or below its
// first byte; of the first and the last vector a part may belong to others.
struct Tensor {
  const uint8_t* g;
  uint8_t* out;
  unsigned long long bytes;
  unsigned int first;  // chunk of the group
  int type;
};
template <int N>
struct Group {
  int count;
  unsigned int chunks;
  Tensor t[N];
};

// The tensor of a chunk: the last whose first chunk is not past it.
template <int N>
__device__ __forceinline__ int tensor_of(const Group<N>& g, unsigned int chunk) {
  int lo = 0, hi = g.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.t[mid].first <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Runs f<T> for a tensor's type.
template <typename F>
__device__ __forceinline__ void with_type(int type, F f) {
  switch (type) {
    case kBf16: f(__nv_bfloat16()); break;
    case kF16: f(__half()); break;
    default: f(float()); break;
  }
}

// The vectors of a chunk of a tensor, kThreads of them apart for a thread.
constexpr long long kStep = kThreads * 16;
struct Span {
  const uint8_t* first;  // the thread's first vector
  const uint8_t *begin, *end;
  bool inside;  // all of the chunk's vectors are the tensor's
  __device__ __forceinline__ Span(const Tensor& t, unsigned int chunk) : begin(t.g), end(t.g + t.bytes) {
    const uint8_t* from =
        reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(t.g) & ~uintptr_t(15)) + chunk * (kChunk * 16);
    inside = from >= begin && from + kChunk * 16 <= end;
    first = from + threadIdx.x * 16;
  }
};

template <int N>
__global__ void __launch_bounds__(kThreads, 4) squares_kernel(const __grid_constant__ Group<N> g, double* partial) {
  __shared__ double red[kThreads / 32];
  chain_next();
  chain_wait();
  double sum = 0.0;
  for (unsigned int c = blockIdx.x; c < g.chunks; c += gridDim.x) {
    const Tensor& t = g.t[tensor_of(g, c)];
    const Span span(t, c - t.first);
    with_type(t.type, [&](auto type) {
      using T = decltype(type);
      constexpr int kPairs = 8 / sizeof(T);
      float2 s[2] = {};
      auto add = [&](const uint4& v) {
        float2 f[kPairs];
        unpack16<T>(v, f);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) s[i & 1] = fma2(f[i], f[i], s[i & 1]);
      };
      if (span.inside) {
        uint4 v[kVectors];
#pragma unroll
        for (int j = 0; j < kVectors; ++j) v[j] = __ldg(reinterpret_cast<const uint4*>(span.first + j * kStep));
#pragma unroll
        for (int j = 0; j < kVectors; ++j) add(v[j]);
      } else {
#pragma unroll 1
        for (int j = 0; j < kVectors; ++j) {
          const uint8_t* p = span.first + j * kStep;
          if (p >= span.end) break;
          if (p >= span.begin && p + 16 <= span.end) {
            add(__ldg(reinterpret_cast<const uint4*>(p)));
          } else {
            const uint8_t* to = p + 16 < span.end ? p + 16 : span.end;
            for (const uint8_t* q = p < span.begin ? span.begin : p; q < to; q += sizeof(T)) {
              const float f = to_float(*reinterpret_cast<const T*>(q));
              s[0].x = fmaf(f, f, s[0].x);
            }
          }
        }
      }
      sum += static_cast<double>((s[0].x + s[1].x) + (s[0].y + s[1].y));
    });
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) sum += red[i];
    partial[blockIdx.x] = sum;
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, 4)
    scale_kernel(const __grid_constant__ Group<N> g, const double* partial, int parts, float max_norm, float eps,
                 float* norm) {
  __shared__ double red[kThreads / 32];
  chain_next();
  chain_wait();
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) sum += partial[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) sum += red[i];
  const float length = static_cast<float>(sqrt(sum));
  float factor = max_norm / (length + eps);
  if (factor > 1.f) factor = 1.f;  // (a NaN stays one)
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = length;
  const unsigned int mine = g.chunks > blockIdx.x ? (g.chunks - 1 - blockIdx.x) / gridDim.x : 0;
  if (blockIdx.x >= g.chunks) return;
  for (unsigned int i = mine + 1; i-- > 0;) {
    const unsigned int c = blockIdx.x + i * gridDim.x;
    const Tensor& t = g.t[tensor_of(g, c)];
    if (factor == 1.f && t.out == t.g) continue;
    const Span span(t, c - t.first);
    const long long to = t.out - t.g;
    const bool same = (to & 15) == 0;  // the output's vectors start on boundaries, too
    with_type(t.type, [&](auto type) {
      using T = decltype(type);
      constexpr int kPairs = 8 / sizeof(T);
      auto scaled = [&](const uint4& v) {
        float2 f[kPairs];
        unpack16<T>(v, f);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) f[i] = mul2(f[i], both(factor));
        return pack16<T>(f);
      };
      if (span.inside && same) {
        uint4 v[kVectors];
#pragma unroll
        for (int j = 0; j < kVectors; ++j) v[j] = *reinterpret_cast<const uint4*>(span.first + j * kStep);
#pragma unroll
        for (int j = 0; j < kVectors; ++j)
          *reinterpret_cast<uint4*>(const_cast<uint8_t*>(span.first + j * kStep + to)) = scaled(v[j]);
      } else {
#pragma unroll 1
        for (int j = 0; j < kVectors; ++j) {
          const uint8_t* p = span.first + j * kStep;
          if (p >= span.end) break;
          if (same && p >= span.begin && p + 16 <= span.end) {
            *reinterpret_cast<uint4*>(const_cast<uint8_t*>(p + to)) = scaled(*reinterpret_cast<const uint4*>(p));
          } else {
            const uint8_t* stop = p + 16 < span.end ? p + 16 : span.end;
            for (const uint8_t* q = p < span.begin ? span.begin : p; q < stop; q += sizeof(T))
              *reinterpret_cast<T*>(const_cast<uint8_t*>(q + to)) =
                  from_float<T>(to_float(*reinterpret_cast<const T*>(q)) * factor);
          }
        }
      }
    });
  }
}

// A launch's parameters hold up to so many tensors (they may take 32764 bytes);
// short lists take the short form, which is less to send.
constexpr int kFewTensors = 48, kTensors = 960;

int groups(int count) { return std::max(1, (count + kTensors - 1) / kTensors); }

template <int N>
cudaError_t run(const ClipCall& c, cudaStream_t stream) {
  double* partial = static_cast<double*>(c.ws);
  const int parts = groups(c.count) * kCtas;
  Group<N> g;
  for (int pass = 0; pass < 2; ++pass)
    for (int k = 0; k < groups(c.count); ++k) {
      g.count = 0;
      unsigned long long chunks = 0;
      const int end = std::min(c.count, (k + 1) * kTensors);
      for (int i = k * kTensors; i < end; ++i) {
        if (c.sizes[i] == 0) continue;
        Tensor& t = g.t[g.count++];
        t.g = static_cast<const uint8_t*>(c.grads[i]);
        t.out = static_cast<uint8_t*>(c.outs[i]);
        t.bytes = static_cast<unsigned long long>(c.sizes[i]) * type_bytes(c.types[i]);
        t.first = static_cast<unsigned int>(chunks);
        t.type = c.types[i];
        const unsigned long long vectors = ((reinterpret_cast<uintptr_t>(t.g) & 15) + t.bytes + 15) / 16;
        chunks += (vectors + kChunk - 1) / kChunk;
        if (chunks > INT32_MAX) return cudaErrorInvalidValue;
      }
      g.chunks = static_cast<unsigned int>(chunks);
      const cudaError_t s =
          pass == 0 ? launch_chained(squares_kernel<N>, dim3(kCtas), kThreads, 0, stream, 0, g, partial + k * kCtas)
                    : launch_chained(scale_kernel<N>, dim3(kCtas), kThreads, 0, stream, 0, g, partial, parts, c.max_norm,
                                     c.eps, k == 0 ? c.norm : nullptr);
      if (s != cudaSuccess) return s;
    }
  return cudaSuccess;
}

}  // namespace

size_t clip_workspace(int count) { return static_cast<size_t>(groups(count)) * kCtas * sizeof(double); }

cudaError_t launch_clip_grad_norm(const ClipCall& c, cudaStream_t stream) {
  return c.count <= kFewTensors ? run<kFewTensors>(c, stream) : run<kTensors>(c, stream);
}

}  // namespace ozemu
