// Gradients of many tensors, clipped by their global norm:
//
//   N = sqrt(sum over all tensors of g^2),  g <- g min(1, max_norm / (N + eps))
//
// Two launches: the sums of squares, a partial one for each CTA, then the
// scaling, before which every CTA adds the partial sums up in the same order; one
// for short lists of little memory.  No atomics: the same gradients give the same
// bits.  Squares and a warp's sum of 2048 of them are fp32 (a chain of 40 roundings
// at most; scaled where they leave its range), everything after that is fp64, whose
// rate is two additions a clock and SM.  Bound by HBM: each gradient is read twice,
// the second time in the reverse order, so that what L2 still holds of the first
// pass is read from there, and written once: 2.15 GB in 48 tensors 1000 us, 6.4 TB/s
// over the three; 100 MB in aligned tensors 45 us, packed without gaps 50.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

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

// A chunk of a tensor: which of its vectors are whole, and the elements of the
// tensor's first and last vector where that is not, which one thread takes.
struct Span {
  long long at;                // of the chunk's first vector, in bytes from the tensor's first element
  int whole_begin, whole_end;  // vectors of the chunk
  int head, tail;              // bytes of the parts, 0 for threads that take none
  int thread;                  // of the chunk's kThreads
  __device__ __forceinline__ Span(const Tensor& t, unsigned int chunk, int thread) : thread(thread) {
    const int past = static_cast<int>(reinterpret_cast<uintptr_t>(t.g) & 15);  // the first vector's bytes before the tensor
    const long long first = chunk * kChunk, bytes = past + static_cast<long long>(t.bytes), vectors = bytes / 16;
    at = first * 16 - past;
    whole_begin = first == 0 && past ? 1 : 0;
    whole_end = static_cast<int>(min(kChunk, max(0LL, vectors - first)));
    // (A tensor within one vector is all head.)
    const bool one = past && bytes < 16;
    head = first == 0 && past && thread == 0 ? min(16 - past, static_cast<int>(t.bytes)) : 0;
    const bool last = !one && vectors >= first && vectors < first + kChunk &&
                      (static_cast<int>(vectors - first) % kThreads) == thread;
    tail = last ? static_cast<int>(bytes & 15) : 0;
  }
  // Whether the thread's vector j is.
  __device__ __forceinline__ bool whole(int j) const {
    const int v = thread + j * kThreads;
    return v >= whole_begin && v < whole_end;
  }
  __device__ __forceinline__ bool all_whole() const { return whole_begin == 0 && whole_end == kChunk; }
  // f(byte from the tensor's first) for the elements of the parts.
  template <typename T, typename F>
  __device__ __forceinline__ void parts(const Tensor& t, F f) const {
#pragma unroll 1
    for (int i = 0; i < head; i += sizeof(T)) f(i);
#pragma unroll 1
    for (int i = tail; i > 0; i -= sizeof(T)) f(static_cast<long long>(t.bytes) - i);
  }
};

// Adds a warp's share of a chunk's sum of squares to its first lane's `sum`.  A
// share that overflows fp32, or is below 2^-110, where its 2048 squares can lose
// 2^-139 below the normal range, is formed again from elements times a power of
// two: of 2^-80 the largest are below 2^48; of 2^100 those that are all below 2^-55
// lie between 2^-49 and 2^45.  (Zeros come here, too.  An infinity or a NaN stays.)
__device__ __forceinline__ void add_chunk_squares(const Tensor& t, unsigned int chunk, int thread, double& sum) {
  const Span span(t, chunk, thread);
  const uint4* from = reinterpret_cast<const uint4*>(t.g + span.at) + thread;
  uint4 v[kVectors];
  if (span.all_whole()) {
#pragma unroll
    for (int j = 0; j < kVectors; ++j) v[j] = from[j * kThreads];
  } else {
#pragma unroll
    for (int j = 0; j < kVectors; ++j) v[j] = span.whole(j) ? from[j * kThreads] : make_uint4(0, 0, 0, 0);
  }
  auto squares = [&](auto times, float power) {  // in every lane
    float2 s[2] = {};
    with_type(t.type, [&](auto type) {
      using T = decltype(type);
      constexpr int kPairs = 8 / sizeof(T);
#pragma unroll
      for (int j = 0; j < kVectors; ++j) {
        float2 f[kPairs];
        unpack16<T>(v[j], f);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          if constexpr (decltype(times)::value) f[i] = mul2(f[i], both(power));
          s[i & 1] = fma2(f[i], f[i], s[i & 1]);
        }
      }
      span.template parts<T>(t, [&](long long at) {
        float f = to_float(*reinterpret_cast<const T*>(t.g + at));
        if constexpr (decltype(times)::value) f *= power;
        s[0].x = fmaf(f, f, s[0].x);
      });
    });
    float all = (s[0].x + s[1].x) + (s[0].y + s[1].y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
    return all;
  };
  const float once = squares(std::false_type(), 1.f);
  const bool first = (threadIdx.x & 31) == 0;
  if (once >= 0x1p-110f && once <= 0x1.fffffep127f) {
    if (first) sum += static_cast<double>(once);
    return;
  }
  const bool small = once < 1.f;
  const float again = squares(std::true_type(), small ? 0x1p100f : 0x1p-80f);
  if (first) sum += static_cast<double>(again) * (small ? 0x1p-200 : 0x1p160);
}

// out = g factor on a chunk.
__device__ __forceinline__ void chunk_scale(const Tensor& t, unsigned int chunk, int thread, float factor) {
  const Span span(t, chunk, thread);
  const bool same = ((t.out - t.g) & 15) == 0;  // the output's vectors start on boundaries, too
  uint4 v[kVectors];
  const uint4* from = reinterpret_cast<const uint4*>(t.g + span.at) + thread;
  uint4* to = reinterpret_cast<uint4*>(t.out + span.at) + thread;
  const bool all = same && span.all_whole();
  if (all) {
#pragma unroll
    for (int j = 0; j < kVectors; ++j) v[j] = from[j * kThreads];
  } else {
#pragma unroll
    for (int j = 0; j < kVectors; ++j) v[j] = same && span.whole(j) ? from[j * kThreads] : make_uint4(0, 0, 0, 0);
  }
  with_type(t.type, [&](auto type) {
    using T = decltype(type);
    constexpr int kPairs = 8 / sizeof(T);
#pragma unroll
    for (int j = 0; j < kVectors; ++j) {
      float2 f[kPairs];
      unpack16<T>(v[j], f);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) f[i] = mul2(f[i], both(factor));
      v[j] = pack16<T>(f);
    }
    auto scale = [&](long long at) {
      *reinterpret_cast<T*>(t.out + at) = from_float<T>(to_float(*reinterpret_cast<const T*>(t.g + at)) * factor);
    };
    if (!same) {  // the elements of the whole vectors, side by side over the threads
      constexpr int kOf = 16 / sizeof(T);
#pragma unroll 1
      for (int i = span.whole_begin * kOf + thread; i < span.whole_end * kOf; i += kThreads)
        scale(span.at + i * static_cast<long long>(sizeof(T)));
    }
    span.template parts<T>(t, scale);
  });
  if (all) {
#pragma unroll
    for (int j = 0; j < kVectors; ++j) to[j * kThreads] = v[j];
  } else if (same) {
#pragma unroll
    for (int j = 0; j < kVectors; ++j)
      if (span.whole(j)) to[j * kThreads] = v[j];
  }
}

// The sum of values in `red`, by one warp; in lane 0.
template <int kValues>
__device__ __forceinline__ double warp_sum(const double* red) {
  const int lane = threadIdx.x & 31;
  double v = 0.0;
#pragma unroll
  for (int i = 0; i < kValues; i += 32) v += kValues >= 32 || lane < kValues ? red[i + lane] : 0.0;
#pragma unroll
  for (int o = kValues < 32 ? kValues / 2 : 16; o > 0; o >>= 1) v += __shfl_down_sync(0xFFFFFFFFu, v, o);
  return v;
}

__device__ __forceinline__ float clip_factor(float norm, float max_norm, float eps) {
  const float factor = max_norm / (norm + eps);
  return factor > 1.f ? 1.f : factor;  // (a NaN stays one)
}

template <int N>
__global__ void __launch_bounds__(kThreads, 4) squares_kernel(const __grid_constant__ Group<N> g, double* partial) {
  __shared__ double red[kThreads / 32];
  chain_next();
  chain_wait();
  double sum = 0.0;
  for (unsigned int c = blockIdx.x; c < g.chunks; c += gridDim.x) {
    const Tensor& t = g.t[tensor_of(g, c)];
    add_chunk_squares(t, c - t.first, threadIdx.x, sum);
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x < 32) {
    sum = warp_sum<kThreads / 32>(red);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, 4)
    scale_kernel(const __grid_constant__ Group<N> g, const double* partial, int parts, float max_norm, float eps,
                 float* norm) {
  __shared__ double red[kThreads];
  __shared__ float length;
  chain_next();
  chain_wait();
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) sum += partial[i];
  red[threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.x < 32) {
    sum = warp_sum<kThreads>(red);
    if (threadIdx.x == 0) length = static_cast<float>(sqrt(sum));
  }
  __syncthreads();
  const float factor = clip_factor(length, max_norm, eps);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = length;
  if (blockIdx.x >= g.chunks) return;
  for (unsigned int i = (g.chunks - 1 - blockIdx.x) / gridDim.x + 1; i-- > 0;) {
    const unsigned int c = blockIdx.x + i * gridDim.x;
    const Tensor& t = g.t[tensor_of(g, c)];
    if (factor != 1.f || t.out != t.g) chunk_scale(t, c - t.first, threadIdx.x, factor);
  }
}

// Both in one launch, for short lists of little memory: a cluster of 16 CTAs,
// each with groups of kThreads that take a chunk; the CTAs' sums meet through
// distributed shared memory.  6 tensors of 1.1 MB in all: 6.8 us and 4 of the host,
// 7.3 and 9.5 by two launches.  (With twice the chunks, in turn, 4 MB take 10.9 us,
// 6.8 by two launches.)
constexpr int kClusterCtas = 16, kClusterGroups = 4;
constexpr int kClusterThreads = kClusterGroups * kThreads;
template <int N>
__global__ void __launch_bounds__(kClusterThreads, 1)
    clip_cluster_kernel(const __grid_constant__ Group<N> g, float max_norm, float eps, float* norm) {
  __shared__ double red[kClusterThreads / 32];
  __shared__ double mine;
  __shared__ float length;
  chain_next();
  chain_wait();
  const int thread = threadIdx.x % kThreads;
  const unsigned int first = cluster_rank() + kClusterCtas * (threadIdx.x / kThreads);
  constexpr unsigned int kTurn = kClusterCtas * kClusterGroups;
  double sum = 0.0;
#pragma unroll 1
  for (unsigned int c = first; c < g.chunks; c += kTurn) {
    const Tensor& t = g.t[tensor_of(g, c)];
    add_chunk_squares(t, c - t.first, thread, sum);
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x < 32) {
    sum = warp_sum<kClusterThreads / 32>(red);
    if (threadIdx.x == 0) mine = sum;
  }
  cluster_sync();
  if (threadIdx.x < 32) {
    static_assert(kClusterCtas == 16, "");
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(sum) : "r"(mapa_shared(&mine, threadIdx.x % 16)));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_down_sync(0xFFFFFFFFu, sum, o);
    if (threadIdx.x == 0) length = static_cast<float>(sqrt(sum));
  }
  cluster_sync();  // the norm is there, and the others have read this CTA's sum
  const float factor = clip_factor(length, max_norm, eps);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = length;
#pragma unroll 1
  for (unsigned int c = first; c < g.chunks; c += kTurn) {
    const Tensor& t = g.t[tensor_of(g, c)];
    if (factor != 1.f || t.out != t.g) chunk_scale(t, c - t.first, thread, factor);
  }
}

// A launch's parameters hold up to so many tensors (they may take 32764 bytes);
// short lists take a shorter form, which is less to send (60 tensors in two
// launches: 23 us of the host with parameters for 960, 14 with those for 64).
constexpr int kFewTensors = 64, kMoreTensors = 256, kTensors = 960;

int groups(int count) { return std::max(1, (count + kTensors - 1) / kTensors); }

// Tensors `begin` to `end` - 1 as a group.
template <int N>
bool make_group(const ClipCall& c, int begin, int end, Group<N>* g) {
  g->count = 0;
  unsigned long long chunks = 0;
  for (int i = begin; i < end; ++i) {
    if (c.sizes[i] == 0) continue;
    Tensor& t = g->t[g->count++];
    t.g = static_cast<const uint8_t*>(c.grads[i]);
    t.out = c.outs ? static_cast<uint8_t*>(c.outs[i]) : nullptr;  // (not looked at for the workspace's size)
    t.bytes = static_cast<unsigned long long>(c.sizes[i]) * type_bytes(c.types[i]);
    t.first = static_cast<unsigned int>(chunks);
    t.type = c.types[i];
    const unsigned long long vectors = ((reinterpret_cast<uintptr_t>(t.g) & 15) + t.bytes + 15) / 16;
    chunks += (vectors + kChunk - 1) / kChunk;
    if (chunks > INT32_MAX) return false;
  }
  g->chunks = static_cast<unsigned int>(chunks);
  return true;
}

template <int N>
cudaError_t run(const ClipCall& c, cudaStream_t stream) {
  double* partial = static_cast<double*>(c.ws);
  int parts = 0;
  Group<N> g;
  for (int pass = 0; pass < 2; ++pass)
    for (int k = 0; k < groups(c.count); ++k) {
      if ((pass == 0 || groups(c.count) > 1) && !make_group(c, k * kTensors, std::min(c.count, (k + 1) * kTensors), &g))
        return cudaErrorInvalidValue;
      // As many CTAs as chunks, where those are few; at least one to leave a sum.
      const int ctas = std::max(1, static_cast<int>(std::min<unsigned int>(g.chunks, kCtas)));
      if (pass == 0) parts += ctas;
      const cudaError_t s =
          pass == 0 ? launch_chained(squares_kernel<N>, dim3(ctas), kThreads, 0, stream, 0, g, partial + parts - ctas)
                    : launch_chained(scale_kernel<N>, dim3(ctas), kThreads, 0, stream, 0, g, partial, parts, c.max_norm,
                                     c.eps, k == 0 ? c.norm : nullptr);
      if (s != cudaSuccess) return s;
    }
  return cudaSuccess;
}

// Chunks that one cluster takes: 2 MB.
constexpr unsigned int kClusterChunks = kClusterCtas * kClusterGroups;
bool one_launch(const ClipCall& c, Group<kFewTensors>* g) {
  return c.count <= kFewTensors && make_group(c, 0, c.count, g) && g->chunks <= kClusterChunks;
}

cudaError_t run_cluster(const ClipCall& c, const Group<kFewTensors>& g, cudaStream_t stream) {
  auto kern = clip_cluster_kernel<kFewTensors>;
  constexpr int kMaxDev = 64;
  static std::atomic<bool> ready[kMaxDev];
  int dev = 0;
  cudaError_t s = cudaGetDevice(&dev);
  if (s != cudaSuccess) return s;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    s = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (s != cudaSuccess) return s;
    ready[dev] = true;
  }
  return launch_chained(kern, dim3(kClusterCtas), kClusterThreads, 0, stream, kClusterCtas, g, c.max_norm, c.eps, c.norm);
}

}  // namespace

size_t clip_workspace(const ClipCall& c) {
  Group<kFewTensors> g;
  return one_launch(c, &g) ? 0 : static_cast<size_t>(groups(c.count)) * kCtas * sizeof(double);
}

cudaError_t launch_clip_grad_norm(const ClipCall& c, cudaStream_t stream) {
  Group<kFewTensors> g;
  if (one_launch(c, &g)) return run_cluster(c, g, stream);
  return c.count <= kFewTensors    ? run<kFewTensors>(c, stream)
         : c.count <= kMoreTensors ? run<kMoreTensors>(c, stream)
                                   : run<kTensors>(c, stream);
}

}  // namespace ozemu
