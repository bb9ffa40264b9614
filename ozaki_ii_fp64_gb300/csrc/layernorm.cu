// Layer norm, forward and backward.
//
//   y  = (x - mean) rstd w + b,  mean = 1/H sum x,  rstd = (1/H sum (x - mean)^2 + eps)^(-1/2)
//   dx = rstd (g - mean(g) - xhat mean(g xhat)) + dr,  g = dy w,  xhat = (x - mean) rstd
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
//
// All sums and statistics are fp32.  A row stays in registers from its one
// read to its write, so that the variance is summed round the mean; rows too
// long for that are read again from L2.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "layer.cuh"

namespace ozemu {

namespace {

// VEC consecutive elements at p, of which `left` exist (the others read as 0):
// 16 bytes, or one element where rows do not start on 16-byte boundaries.
// Rows pass once: they take no room in L1, which keeps the parameters.
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, int left, float (&v)[VEC]) {
  if constexpr (VEC > 1) {
    static_assert(VEC * sizeof(T) == 16, "16-byte vectors");
    if (left >= VEC) {
      uint4 u;
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                   : "l"(p));
      unpack16<T>(u, v);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = i < left ? to_float(p[i]) : 0.f;
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC], int left) {
  if constexpr (VEC > 1) {
    if (left >= VEC) {
      *reinterpret_cast<uint4*>(p) = pack16<T>(v);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    if (i < left) p[i] = from_float<T>(v[i]);
}

// VEC parameters from column j on, in the rows' type T or fp32.
template <typename T, int VEC>
__device__ __forceinline__ void load_params(const void* base, bool f32, bool vec, int j, int left, float (&v)[VEC]) {
  if (vec && left >= VEC) {
    if (f32) {
      const float* p = static_cast<const float*>(base) + j;
      if constexpr (VEC >= 4) {
#pragma unroll
        for (int q = 0; q < VEC; q += 4) {
          const float4 f = __ldg(reinterpret_cast<const float4*>(p + q));
          v[q] = f.x;
          v[q + 1] = f.y;
          v[q + 2] = f.z;
          v[q + 3] = f.w;
        }
      } else {
        v[0] = __ldg(p);
      }
    } else if constexpr (VEC > 1) {
      unpack16<T>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(base) + j)), v);
    } else {
      v[0] = to_float(static_cast<const T*>(base)[j]);
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < VEC; ++q)
    v[q] = q >= left ? 0.f : (f32 ? static_cast<const float*>(base)[j + q] : to_float(static_cast<const T*>(base)[j + q]));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sum over the TPR threads of a row.  TPR = 32: one warp, no barrier.  Else
// the whole CTA; `red` (one word per warp) is not used again before another
// barrier.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < TPR / 32; w += 4) {
      const float4 t = *reinterpret_cast<const float4*>(red + w);
      s = add2(s, add2(make_float2(t.x, t.y), make_float2(t.z, t.w)));
    }
    v = s.x + s.y;
  }
  return v;
}

// s / n without a division: inv is 1 / n rounded, the remainder's correction
// makes the quotient of an exact multiple exact.
__device__ __forceinline__ float mean_of(float s, float n, float inv) {
  const float m = s * inv;
  return fabsf(m) <= 3.4e38f ? fmaf(fmaf(-m, n, s), inv, m) : m;  // an infinite sum stays one
}

constexpr int cta_threads(int tpr) { return tpr < 128 ? 128 : tpr; }

// One row per TPR threads, NV vectors each.
template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(cta_threads(TPR)) norm_forward_kernel(const NormCall c, int vec) {
  __shared__ __align__(16) float red[2][32];
  constexpr int kRows = cta_threads(TPR) / TPR;
  const int tid = threadIdx.x % TPR;
  const long long row = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / TPR;
  if (row >= c.rows) return;  // TPR = 32 only: whole warps
  const T* x = static_cast<const T*>(c.x) + row * c.ldx;
  T* y = static_cast<T*>(c.y) + row * c.ldy;
  float d[NV][VEC];
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    const int j = (q * TPR + tid) * VEC;
    load_vec<T, VEC>(x + j, c.cols - j, d[q]);
  }
#pragma unroll
  for (int q = 0; q < NV; ++q)
#pragma unroll
    for (int i = 0; i < VEC; ++i) s += d[q][i];
  const float mean = row_sum<TPR>(s, red[0]) / static_cast<float>(c.cols);
  s = 0.f;
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    const int j = (q * TPR + tid) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      d[q][i] -= mean;
      s += j + i < c.cols ? d[q][i] * d[q][i] : 0.f;
    }
  }
  const float rstd = 1.f / sqrtf(row_sum<TPR>(s, red[1]) / static_cast<float>(c.cols) + c.eps);
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    const int j = (q * TPR + tid) * VEC, left = c.cols - j;
    if (left <= 0) break;
    float w[VEC], b[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      w[i] = 1.f;
      b[i] = 0.f;
    }
    if (c.weight) load_params<T, VEC>(c.weight, c.param_type == kF32, vec & 1, j, left, w);
    if (c.bias) load_params<T, VEC>(c.bias, c.param_type == kF32, vec & 2, j, left, b);
#pragma unroll
    for (int i = 0; i < VEC; ++i) w[i] = fmaf(d[q][i] * rstd, w[i], b[i]);
    store_vec<T, VEC>(y + j, w, left);
  }
  if (tid == 0) {
    if (c.mean) c.mean[row] = mean;
    if (c.rstd) c.rstd[row] = rstd;
  }
}

// ---------------------------------------------------------------------------
// Rows through a ring in shared memory.  A group of TPR threads (a warp, or the
// CTA) takes every step-th row; bulk copies bring its next `stages` rows while
// it works on one, so that memory stays busy through the two sums and the
// barriers of a row.  A slot is free again once every thread holds its part of
// the row in registers, which the first sum's barrier says.
// ---------------------------------------------------------------------------
template <int TPR, int EPT, bool kBackward>
struct RingCfg {
  static constexpr int kThreads = TPR < 128 ? 256 : TPR;
  static constexpr int kGroups = kThreads / TPR;
  // Threads an SM holds: by the registers that a thread's EPT elements (and,
  // backward, their column sums) take.
  static constexpr int kResident = kBackward ? (EPT > 8 ? 512 : 1024) : (EPT > 16 ? 768 : 1024);
  static constexpr int kPerSm = kThreads >= kResident ? 1 : kResident / kThreads;
  static constexpr int kBytes = 200 * 1024 / kPerSm / 128 * 128;  // shared memory of a CTA's ring
};
constexpr int kMaxStages = 4;

// The 2 EPT parameters of one 16-byte vector, in the rows' type T or fp32.
template <typename T, typename W>
__device__ __forceinline__ void load_params16(const void* base, int j, float2* v) {
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const W*>(base) + j);
  unpack16<W>(__ldg(p), v);
  if constexpr (sizeof(W) > sizeof(T)) unpack16<W>(__ldg(p + 1), v + 2);
}

// Waits for a slot.  False: give up (this thread leaves the kernel; the thread
// that issues the group's copies first lets those in flight land).
template <int TPR>
__device__ __forceinline__ bool ring_wait(uint64_t* full, int turn, int slot, int stages, int issued,
                                          volatile int* abort_word, uint32_t* flags) {
  if (mbar_wait(&full[slot], (turn / stages) & 1, abort_word, flags)) return true;
  if (threadIdx.x % TPR == 0) {
    for (int i = turn; i < issued; ++i) {
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(&full[i % stages], (i / stages) & 1) && globaltimer() - t0 < kWaitLimitNs) {
      }
    }
  }
  return false;
}

template <typename T, typename W, int TPR, int EPT>
__global__ void __launch_bounds__(RingCfg<TPR, EPT, false>::kThreads, RingCfg<TPR, EPT, false>::kPerSm)
    norm_forward_ring_kernel(const NormCall c, int stages, float inv) {
  constexpr int VEC = 16 / sizeof(T), NV = EPT / VEC, H = VEC / 2;
  using R = RingCfg<TPR, EPT, false>;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) float red[2][32];
  __shared__ uint64_t bars[R::kGroups][kMaxStages];
  __shared__ int abort_word;
  const int tid = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const uint32_t bytes = static_cast<uint32_t>(c.cols) * sizeof(T);
  const float n = static_cast<float>(c.cols);
  uint8_t* slots = ring + static_cast<size_t>(group) * stages * bytes;
  uint64_t* full = bars[group];
  const int step = gridDim.x * R::kGroups, first = blockIdx.x * R::kGroups + group;
  const T* x = static_cast<const T*>(c.x);
  int issued = 0;
  if (threadIdx.x == 0) abort_word = 0;
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
    for (long long row = first; issued < stages && row < c.rows; ++issued, row += step) {
      mbar_arrive_expect_tx_relaxed(&full[issued], bytes);
      bulk_load(slots + issued * bytes, x + row * c.ldx, bytes, &full[issued]);
    }
  }
  __syncthreads();
  int slot = 0, turn = 0;
  for (long long row = first; row < c.rows; row += step, ++turn) {
    if (!ring_wait<TPR>(full, turn, slot, stages, issued, &abort_word, c.flags)) return;
    const uint8_t* in = slots + slot * bytes + tid * 16;
    float2 d[NV][H];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int q = 0; q < NV; ++q)
      if ((q * TPR + tid) * VEC < c.cols) {
        unpack16<T>(*reinterpret_cast<const uint4*>(in + q * TPR * 16), d[q]);
#pragma unroll
        for (int i = 0; i < H; ++i) s = add2(s, d[q][i]);
      }
    const float mean = mean_of(row_sum<TPR>(s.x + s.y, red[0]), n, inv);
    __syncwarp();
    if (tid == 0) {
      const long long later = row + static_cast<long long>(stages) * step;
      if (later < c.rows) {
        mbar_arrive_expect_tx_relaxed(&full[slot], bytes);
        bulk_load(slots + slot * bytes, x + later * c.ldx, bytes, &full[slot]);
        ++issued;
      }
    }
    if (++slot == stages) slot = 0;
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int q = 0; q < NV; ++q)
      if ((q * TPR + tid) * VEC < c.cols)
#pragma unroll
        for (int i = 0; i < H; ++i) {
          d[q][i] = add2(d[q][i], both(-mean));
          s = fma2(d[q][i], d[q][i], s);
        }
    const float rstd = 1.f / sqrtf(mean_of(row_sum<TPR>(s.x + s.y, red[1]), n, inv) + c.eps);
    T* y = static_cast<T*>(c.y) + row * c.ldy + tid * VEC;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int j = (q * TPR + tid) * VEC;
      if (j >= c.cols) break;
#pragma unroll
      for (int i = 0; i < H; ++i) d[q][i] = mul2(d[q][i], both(rstd));
      float2 p[H];
      if (c.weight) {
        load_params16<T, W>(c.weight, j, p);
#pragma unroll
        for (int i = 0; i < H; ++i) d[q][i] = mul2(d[q][i], p[i]);
      }
      if (c.bias) {
        load_params16<T, W>(c.bias, j, p);
#pragma unroll
        for (int i = 0; i < H; ++i) d[q][i] = add2(d[q][i], p[i]);
      }
      *reinterpret_cast<uint4*>(y + q * TPR * VEC) = pack16<T>(d[q]);
    }
    if (tid == 0) {
      if (c.mean) c.mean[row] = mean;
      if (c.rstd) c.rstd[row] = rstd;
    }
  }
}

// Rows of any length, read three times (from L2 after the first).
constexpr int kLong = 1024;
template <typename T>
__global__ void __launch_bounds__(kLong) norm_forward_long_kernel(const NormCall c) {
  __shared__ __align__(16) float red[2][32];
  const bool f32 = c.param_type == kF32;
  for (long long row = blockIdx.x; row < c.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(c.x) + row * c.ldx;
    T* y = static_cast<T*>(c.y) + row * c.ldy;
    float s = 0.f;
    for (int j = threadIdx.x; j < c.cols; j += kLong) s += to_float(x[j]);
    const float mean = row_sum<kLong>(s, red[0]) / static_cast<float>(c.cols);
    s = 0.f;
    for (int j = threadIdx.x; j < c.cols; j += kLong) {
      const float d = to_float(x[j]) - mean;
      s += d * d;
    }
    const float rstd = 1.f / sqrtf(row_sum<kLong>(s, red[1]) / static_cast<float>(c.cols) + c.eps);
    for (int j = threadIdx.x; j < c.cols; j += kLong) {
      float w[1] = {1.f}, b[1] = {0.f};
      if (c.weight) load_params<T, 1>(c.weight, f32, false, j, 1, w);
      if (c.bias) load_params<T, 1>(c.bias, f32, false, j, 1, b);
      y[j] = from_float<T>(fmaf((to_float(x[j]) - mean) * rstd, w[0], b[0]));
    }
    if (threadIdx.x == 0) {
      if (c.mean) c.mean[row] = mean;
      if (c.rstd) c.rstd[row] = rstd;
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  One pass over x and dy gives dx and, per CTA, the column sums of
// dy xhat and dy over the rows it took; a second kernel joins the CTAs' sums
// in order.  A thread keeps the same columns for every row, its sums in
// registers, or in shared memory (kShared) where a row takes up the
// registers.
// ---------------------------------------------------------------------------

// CTAs that leave partial sums, at most: what fits the GPU at once, fewer for
// long rows, whose CTAs are large.
int max_parts(int cols) { return cols <= 2048 ? 608 : (cols <= 4096 ? 304 : 152); }

// The sums of one row: (sum g, sum g xhat) over its TPR threads.
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float2 s, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    s = add2(s, make_float2(__shfl_xor_sync(0xFFFFFFFFu, s.x, o), __shfl_xor_sync(0xFFFFFFFFu, s.y, o)));
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < TPR / 32; w += 2) {
      const float4 t = *reinterpret_cast<const float4*>(red + w);
      s = add2(s, add2(make_float2(t.x, t.y), make_float2(t.z, t.w)));
    }
  }
  return s;
}

// A thread's column sums and what happens to them.  Element i of vector q
// stands for column (q TPR + tid) VEC + i.
template <int VEC, int TPR, int NV, int kGroups, bool kShared>
struct ColumnSums {
  static constexpr int kWidth = NV * TPR * VEC;
  static constexpr int kBytes = kShared ? 2 * kWidth * 4 : (kGroups > 1 ? 2 * kGroups * kWidth * 4 : 0);
  alignas(8) float w[kShared ? 1 : NV][VEC];
  alignas(8) float b[kShared ? 1 : NV][VEC];
  float* mem;
  int tid;

  __device__ __forceinline__ ColumnSums(float* shared, int t) : mem(shared), tid(t) {
#pragma unroll
    for (int q = 0; q < (kShared ? 1 : NV); ++q)
#pragma unroll
      for (int i = 0; i < VEC; ++i) w[q][i] = b[q][i] = 0.f;
    if constexpr (kShared) {
      // Each thread clears and keeps its own words.
#pragma unroll
      for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int i = 0; i < VEC; ++i) mem[(q * TPR + tid) * VEC + i] = mem[kWidth + (q * TPR + tid) * VEC + i] = 0.f;
    }
  }
  // One element's dy xhat and dy.
  __device__ __forceinline__ void add(int q, float xh, float dy) {
    if constexpr (kShared) {
      float* p = mem + (q * TPR + tid) * VEC;
      p[0] += dy * xh;
      p[kWidth] += dy;
    } else {
      w[q][0] += dy * xh;
      b[q][0] += dy;
    }
  }
  // The same for a vector.
  __device__ __forceinline__ void add(int q, const float2* xh, const float2* dy) {
    float2* pw = kShared ? reinterpret_cast<float2*>(mem + (q * TPR + tid) * VEC)
                         : reinterpret_cast<float2*>(w[kShared ? 0 : q]);
    float2* pb = kShared ? pw + kWidth / 2 : reinterpret_cast<float2*>(b[kShared ? 0 : q]);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      pw[i] = fma2(dy[i], xh[i], pw[i]);
      pb[i] = add2(pb[i], dy[i]);
    }
  }
  // Writes the CTA's sums: part[0][cta][.] of dw, part[1][cta][.] of db.
  __device__ __forceinline__ void leave(float* part, int parts, int cols, int group) {
    float* pw = part + static_cast<long long>(blockIdx.x) * cols;
    float* pb = pw + static_cast<long long>(parts) * cols;
    if constexpr (kGroups > 1) {
#pragma unroll
      for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          mem[(2 * group) * kWidth + (q * TPR + tid) * VEC + i] = w[q][i];
          mem[(2 * group + 1) * kWidth + (q * TPR + tid) * VEC + i] = b[q][i];
        }
      __syncthreads();
      for (int j = threadIdx.x; j < cols; j += kGroups * TPR) {
        float a = 0.f, d = 0.f;
#pragma unroll
        for (int r = 0; r < kGroups; ++r) {
          a += mem[(2 * r) * kWidth + j];
          d += mem[(2 * r + 1) * kWidth + j];
        }
        pw[j] = a;
        pb[j] = d;
      }
    } else {
#pragma unroll
      for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const int at = (q * TPR + tid) * VEC + i;
          if (at >= cols) continue;
          pw[at] = kShared ? mem[at] : w[kShared ? 0 : q][i];
          pb[at] = kShared ? mem[kWidth + at] : b[kShared ? 0 : q][i];
        }
    }
  }
};

// Rows through the ring (16-byte rows): a slot holds x, dy and, where given,
// dr of one row.
template <typename T, typename W, int TPR, int EPT, bool kShared>
__global__ void __launch_bounds__(RingCfg<TPR, EPT, true>::kThreads, RingCfg<TPR, EPT, true>::kPerSm)
    norm_backward_ring_kernel(const NormGradCall c, float* part, int parts, int stages, float inv) {
  constexpr int VEC = 16 / sizeof(T), NV = EPT / VEC, H = VEC / 2;
  using R = RingCfg<TPR, EPT, true>;
  using Sums = ColumnSums<VEC, TPR, NV, R::kGroups, kShared>;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) float2 red[2][32];
  __shared__ uint64_t bars[R::kGroups][kMaxStages];
  __shared__ int abort_word;
  const int tid = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const uint32_t bytes = static_cast<uint32_t>(c.cols) * sizeof(T), slot_bytes = bytes * (c.dr ? 3 : 2);
  const float n = static_cast<float>(c.cols);
  uint8_t* slots = ring + Sums::kBytes + static_cast<size_t>(group) * stages * slot_bytes;
  uint64_t* full = bars[group];
  const int step = gridDim.x * R::kGroups, first = blockIdx.x * R::kGroups + group;
  Sums sums(reinterpret_cast<float*>(ring), tid);
  int issued = 0;
  auto issue = [&](long long row, int slot) {
    uint8_t* to = slots + slot * slot_bytes;
    mbar_arrive_expect_tx_relaxed(&full[slot], slot_bytes);
    bulk_load(to, static_cast<const T*>(c.x) + row * c.ldx, bytes, &full[slot]);
    bulk_load(to + bytes, static_cast<const T*>(c.dy) + row * c.lddy, bytes, &full[slot]);
    if (c.dr) bulk_load(to + 2 * bytes, static_cast<const T*>(c.dr) + row * c.lddr, bytes, &full[slot]);
    ++issued;
  };
  if (threadIdx.x == 0) abort_word = 0;
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
    for (long long row = first; issued < stages && row < c.rows; row += step) issue(row, issued);
  }
  __syncthreads();
  int slot = 0, turn = 0;
  float mean = 0.f, rstd = 0.f;
  if (first < c.rows) {
    mean = c.mean[first];
    rstd = c.rstd[first];
  }
  for (long long row = first; row < c.rows; row += step, ++turn) {
    float next_mean = 0.f, next_rstd = 0.f;
    if (row + step < c.rows) {
      next_mean = c.mean[row + step];
      next_rstd = c.rstd[row + step];
    }
    if (!ring_wait<TPR>(full, turn, slot, stages, issued, &abort_word, c.flags)) return;
    const uint8_t* in = slots + slot * slot_bytes + tid * 16;
    float2 xh[NV][H], g[NV][H];
    uint4 dr[NV];
    float2 s1 = make_float2(0.f, 0.f), s2 = s1;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int j = (q * TPR + tid) * VEC;
      if (j >= c.cols) break;
      unpack16<T>(*reinterpret_cast<const uint4*>(in + q * TPR * 16), xh[q]);
      unpack16<T>(*reinterpret_cast<const uint4*>(in + bytes + q * TPR * 16), g[q]);
      if (c.dr) dr[q] = *reinterpret_cast<const uint4*>(in + 2 * bytes + q * TPR * 16);
#pragma unroll
      for (int i = 0; i < H; ++i) xh[q][i] = mul2(add2(xh[q][i], both(-mean)), both(rstd));
      sums.add(q, xh[q], g[q]);
      if (c.weight) {
        float2 w[H];
        load_params16<T, W>(c.weight, j, w);
#pragma unroll
        for (int i = 0; i < H; ++i) g[q][i] = mul2(g[q][i], w[i]);
      }
#pragma unroll
      for (int i = 0; i < H; ++i) {
        s1 = add2(s1, g[q][i]);
        s2 = fma2(g[q][i], xh[q][i], s2);
      }
    }
    const float2 s = row_sum2<TPR>(make_float2(s1.x + s1.y, s2.x + s2.y), red[turn & 1]);
    __syncwarp();
    if (tid == 0) {
      const long long later = row + static_cast<long long>(stages) * step;
      if (later < c.rows) issue(later, slot);
    }
    if (++slot == stages) slot = 0;
    const float c1 = mean_of(s.x, n, inv), c2 = mean_of(s.y, n, inv);
    T* dx = static_cast<T*>(c.dx) + row * c.lddx + tid * VEC;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      if ((q * TPR + tid) * VEC >= c.cols) break;
      float2 extra[H];
#pragma unroll
      for (int i = 0; i < H; ++i) extra[i] = make_float2(0.f, 0.f);
      if (c.dr) unpack16<T>(dr[q], extra);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float2 v = fma2(xh[q][i], both(-c2), add2(g[q][i], both(-c1)));
        extra[i] = fma2(v, both(rstd), extra[i]);
      }
      *reinterpret_cast<uint4*>(dx + q * TPR * VEC) = pack16<T>(extra);
    }
    mean = next_mean;
    rstd = next_rstd;
  }
  sums.leave(part, parts, c.cols, group);
}

// The same on rows that no 16-byte access fits, element by element; the next
// row is loaded before this row's sums meet.
template <typename T, int TPR, int NV, bool kShared>
__global__ void __launch_bounds__(cta_threads(TPR), TPR * NV > 4096 ? 1 : 1024 / cta_threads(TPR))
    norm_backward_kernel(const NormGradCall c, float* part, int parts) {
  constexpr int kRows = cta_threads(TPR) / TPR;
  using Sums = ColumnSums<1, TPR, NV, kRows, kShared>;
  __shared__ __align__(16) float2 red[2][32];
  extern __shared__ float shared_sums[];
  const int tid = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const bool f32 = c.param_type == kF32;
  Sums sums(shared_sums, tid);
  const long long step = static_cast<long long>(gridDim.x) * kRows;
  long long row = static_cast<long long>(blockIdx.x) * kRows + sub;
  T x[NV], dy[NV];
  auto load = [&](long long at) {
    const T* px = static_cast<const T*>(c.x) + at * c.ldx;
    const T* pd = static_cast<const T*>(c.dy) + at * c.lddy;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int j = q * TPR + tid;
      if (j < c.cols) {
        x[q] = px[j];
        dy[q] = pd[j];
      }
    }
  };
  if (row < c.rows) load(row);
  for (int turn = 0; row < c.rows; row += step, turn ^= 1) {
    const float mean = c.mean[row], rstd = c.rstd[row];
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int j = q * TPR + tid;
      if (j >= c.cols) break;
      float w[1] = {1.f};
      if (c.weight) load_params<T, 1>(c.weight, f32, true, j, 1, w);
      const float d = to_float(dy[q]), xh = (to_float(x[q]) - mean) * rstd, g = d * w[0];
      s.x += g;
      s.y += g * xh;
      sums.add(q, xh, d);
    }
    s = row_sum2<TPR>(s, red[turn]);
    const float c1 = s.x / static_cast<float>(c.cols), c2 = s.y / static_cast<float>(c.cols);
    T* dx = static_cast<T*>(c.dx) + row * c.lddx;
    const T* dr = c.dr ? static_cast<const T*>(c.dr) + row * c.lddr : nullptr;
    T o[NV];
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      const int j = q * TPR + tid;
      if (j >= c.cols) break;
      float w[1] = {1.f};
      if (c.weight) load_params<T, 1>(c.weight, f32, true, j, 1, w);
      float v = rstd * (to_float(dy[q]) * w[0] - c1 - (to_float(x[q]) - mean) * rstd * c2);
      if (dr) v += to_float(dr[j]);
      o[q] = from_float<T>(v);
    }
    if (row + step < c.rows) load(row + step);
#pragma unroll
    for (int q = 0; q < NV; ++q)
      if (q * TPR + tid < c.cols) dx[q * TPR + tid] = o[q];
  }
  sums.leave(part, parts, c.cols, sub);
}

// Rows of any length: dx with a CTA per row, reading the row twice.
template <typename T>
__global__ void __launch_bounds__(kLong) norm_backward_long_kernel(const NormGradCall c) {
  __shared__ __align__(16) float red[2][32];
  const bool f32 = c.param_type == kF32;
  for (long long row = blockIdx.x; row < c.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(c.x) + row * c.ldx;
    const T* dy = static_cast<const T*>(c.dy) + row * c.lddy;
    const T* dr = c.dr ? static_cast<const T*>(c.dr) + row * c.lddr : nullptr;
    T* dx = static_cast<T*>(c.dx) + row * c.lddx;
    const float mean = c.mean[row], rstd = c.rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int j = threadIdx.x; j < c.cols; j += kLong) {
      float w[1] = {1.f};
      if (c.weight) load_params<T, 1>(c.weight, f32, false, j, 1, w);
      const float g = to_float(dy[j]) * w[0];
      s1 += g;
      s2 += g * ((to_float(x[j]) - mean) * rstd);
    }
    s1 = row_sum<kLong>(s1, red[0]) / static_cast<float>(c.cols);
    s2 = row_sum<kLong>(s2, red[1]) / static_cast<float>(c.cols);
    for (int j = threadIdx.x; j < c.cols; j += kLong) {
      float w[1] = {1.f};
      if (c.weight) load_params<T, 1>(c.weight, f32, false, j, 1, w);
      float v = rstd * (to_float(dy[j]) * w[0] - s1 - (to_float(x[j]) - mean) * rstd * s2);
      if (dr) v += to_float(dr[j]);
      dx[j] = from_float<T>(v);
    }
  }
}

// Column sums over `chunk` rows, one column a thread, for those rows.
template <typename T>
__global__ void __launch_bounds__(256) norm_columns_long_kernel(const NormGradCall c, float* part, int parts,
                                                                int chunk) {
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= c.cols) return;
  float sw = 0.f, sb = 0.f;
  const long long end = min(static_cast<long long>(c.rows), (blockIdx.y + 1LL) * chunk);
  for (long long row = static_cast<long long>(blockIdx.y) * chunk; row < end; ++row) {
    const float dy = to_float(static_cast<const T*>(c.dy)[row * c.lddy + j]);
    sb += dy;
    sw += dy * ((to_float(static_cast<const T*>(c.x)[row * c.ldx + j]) - c.mean[row]) * c.rstd[row]);
  }
  part[static_cast<long long>(blockIdx.y) * c.cols + j] = sw;
  part[(static_cast<long long>(parts) + blockIdx.y) * c.cols + j] = sb;
}

// ------------------------------------------------------------------- host

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool rows_aligned16(const void* p, long long ld, int rows, int size) {
  return !p || (aligned16(p) && (rows <= 1 || (ld * size) % 16 == 0));
}

template <typename F>
cudaError_t with_type(int type, F f) {
  if (type == kBf16) return f(__nv_bfloat16{});
  if (type == kF16) return f(__half{});
  return f(float{});
}

constexpr int kSms = 152;

template <typename T, int VEC, int NV>
cudaError_t forward_vec(const NormCall& c, cudaStream_t stream) {
  const int vec = (aligned16(c.weight) ? 1 : 0) | (aligned16(c.bias) ? 2 : 0);
  const int span = VEC * NV;  // elements per thread
  if (c.cols <= 32 * span)
    norm_forward_kernel<T, VEC, 32, NV><<<(c.rows + 3) / 4, 128, 0, stream>>>(c, vec);
  else if (c.cols <= 128 * span)
    norm_forward_kernel<T, VEC, 128, NV><<<c.rows, 128, 0, stream>>>(c, vec);
  else if (c.cols <= 256 * span)
    norm_forward_kernel<T, VEC, 256, NV><<<c.rows, 256, 0, stream>>>(c, vec);
  else if (c.cols <= 512 * span)
    norm_forward_kernel<T, VEC, 512, NV><<<c.rows, 512, 0, stream>>>(c, vec);
  else if (c.cols <= 1024 * span)
    norm_forward_kernel<T, VEC, 1024, NV><<<c.rows, 1024, 0, stream>>>(c, vec);
  else
    norm_forward_long_kernel<T><<<std::min(c.rows, 65536), kLong, 0, stream>>>(c);
  return cudaGetLastError();
}

// Slots that a ring of `bytes` holds for each of its groups, and so whether it
// is worth running.
int ring_stages(int bytes, int groups, int slot_bytes) {
  return std::min(kMaxStages, bytes / (groups * std::max(slot_bytes, 16)));
}

struct ForwardLaunch {
  const NormCall& c;
  cudaStream_t stream;
  cudaError_t error = cudaSuccess;

  // Launches the ring for rows of at most TPR * EPT columns, if there are
  // enough rows to go round.
  template <typename T, typename W, int TPR, int EPT>
  bool fits() {
    if (c.cols > TPR * EPT) return false;
    using R = RingCfg<TPR, EPT, false>;
    const int bytes = c.cols * static_cast<int>(sizeof(T)), stages = ring_stages(R::kBytes, R::kGroups, bytes);
    const int ctas = R::kPerSm * kSms;
    if (stages < 2 || c.rows <= ctas * R::kGroups) return false;
    auto kern = norm_forward_ring_kernel<T, W, TPR, EPT>;
    error = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kBytes);
    if (error != cudaSuccess) return true;
    kern<<<ctas, R::kThreads, R::kGroups * stages * bytes, stream>>>(c, stages, 1.f / static_cast<float>(c.cols));
    error = cudaGetLastError();
    return true;
  }
  template <typename T, typename W>
  bool any() {
    return fits<T, W, 32, 32>() || fits<T, W, 128, 32>() || fits<T, W, 256, 32>() || fits<T, W, 512, 32>() ||
           fits<T, W, 1024, 32>();
  }
};

struct BackwardLaunch {
  const NormGradCall& c;
  cudaStream_t stream;
  int parts;     // room for partial sums
  int used = 0;  // of which this many are written
  cudaError_t error = cudaSuccess;

  template <typename T, typename W, int TPR, int EPT, bool kShared>
  bool ring() {
    if (c.cols > TPR * EPT) return false;
    using R = RingCfg<TPR, EPT, true>;
    constexpr int VEC = 16 / sizeof(T);
    constexpr int kSums = ColumnSums<VEC, TPR, EPT / VEC, R::kGroups, kShared>::kBytes;
    const int slot = c.cols * static_cast<int>(sizeof(T)) * (c.dr ? 3 : 2);
    const int stages = ring_stages(R::kBytes - kSums, R::kGroups, slot);
    if (stages < 1) return false;
    auto kern = norm_backward_ring_kernel<T, W, TPR, EPT, kShared>;
    error = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kBytes);
    if (error != cudaSuccess) return true;
    used = std::min({(c.rows + R::kGroups - 1) / R::kGroups, R::kPerSm * kSms, parts});
    kern<<<used, R::kThreads, kSums + R::kGroups * stages * slot, stream>>>(
        c, static_cast<float*>(c.ws), parts, stages, 1.f / static_cast<float>(c.cols));
    error = cudaGetLastError();
    return true;
  }
  template <typename T, typename W>
  bool any() {
    return ring<T, W, 32, 8, false>() || ring<T, W, 128, 16, false>() || ring<T, W, 256, 16, false>() ||
           ring<T, W, 512, 16, false>() || ring<T, W, 1024, 16, true>();
  }
  template <typename T, int TPR, int NV, bool kShared>
  bool plain() {
    if (c.cols > TPR * NV) return false;
    constexpr int kRows = cta_threads(TPR) / TPR;
    constexpr int kSums = ColumnSums<1, TPR, NV, kRows, kShared>::kBytes;
    auto kern = norm_backward_kernel<T, TPR, NV, kShared>;
    if (kSums > 48 * 1024) error = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSums);
    if (error != cudaSuccess) return true;
    used = std::min({(c.rows + kRows - 1) / kRows, (TPR * NV > 4096 ? 1 : 1024 / cta_threads(TPR)) * kSms, parts});
    kern<<<used, cta_threads(TPR), kSums, stream>>>(c, static_cast<float*>(c.ws), parts);
    error = cudaGetLastError();
    return true;
  }
  template <typename T>
  void any_length() {
    const int chunk = (c.rows + parts - 1) / parts;
    used = (c.rows + chunk - 1) / chunk;
    // The columns first: dx may be dy itself.
    norm_columns_long_kernel<T><<<dim3((c.cols + 255) / 256, used), 256, 0, stream>>>(
        c, static_cast<float*>(c.ws), parts, chunk);
    norm_backward_long_kernel<T><<<std::min(c.rows, 65536), kLong, 0, stream>>>(c);
    error = cudaGetLastError();
  }
};

}  // namespace

cudaError_t launch_layer_norm(const NormCall& c, cudaStream_t stream) {
  const int size = type_bytes(c.type);
  const bool vec = rows_aligned16(c.x, c.ldx, c.rows, size) && rows_aligned16(c.y, c.ldy, c.rows, size);
  const bool ring = vec && static_cast<long long>(c.cols) * size % 16 == 0 && aligned16(c.weight) && aligned16(c.bias);
  ForwardLaunch l{c, stream};
  return with_type(c.type, [&](auto t) {
    using T = decltype(t);
    if (!vec) return forward_vec<T, 1, 16>(c, stream);
    if (ring && (c.param_type == kF32 ? l.any<T, float>() : l.any<T, T>())) return l.error;
    return forward_vec<T, 16 / sizeof(T), 4>(c, stream);
  });
}

size_t layer_norm_backward_workspace(int, int cols) { return static_cast<size_t>(2 * max_parts(cols)) * cols * 4; }

cudaError_t launch_layer_norm_backward(const NormGradCall& c, cudaStream_t stream) {
  BackwardLaunch l{c, stream, max_parts(c.cols)};
  if (c.rows > 0) {
    const int size = type_bytes(c.type);
    const bool vec = static_cast<long long>(c.cols) * size % 16 == 0 && rows_aligned16(c.x, c.ldx, c.rows, size) &&
                     rows_aligned16(c.dy, c.lddy, c.rows, size) && rows_aligned16(c.dr, c.lddr, c.rows, size) &&
                     rows_aligned16(c.dx, c.lddx, c.rows, size) && aligned16(c.weight);
    with_type(c.type, [&](auto t) {
      using T = decltype(t);
      if (!(vec && (c.param_type == kF32 ? l.any<T, float>() : l.any<T, T>())) &&
          !(l.plain<T, 32, 8, false>() || l.plain<T, 128, 8, false>() || l.plain<T, 256, 8, false>() ||
            l.plain<T, 512, 8, false>() || l.plain<T, 512, 16, false>() || l.plain<T, 1024, 16, true>()))
        l.any_length<T>();
      return l.error;
    });
    if (l.error != cudaSuccess) return l.error;
  }
  if (c.dweight || c.dbias) {
    const dim3 grid((c.cols + 31) / 32, 2);
    with_type(c.param_type, [&](auto w) {
      using W = decltype(w);
      join_parts_kernel<W><<<grid, 1024, 0, stream>>>(static_cast<const float*>(c.ws), l.used, l.parts, c.cols,
                                                      static_cast<W*>(c.dweight), static_cast<W*>(c.dbias));
      return cudaSuccess;
    });
  }
  return cudaGetLastError();
}

}  // namespace ozemu
