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
#include "slot_wait.cuh"

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
// through `red` (one word per warp of the group), which is not used again
// before another barrier.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x % TPR >> 5] = v;
    row_barrier<TPR>();
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

// One row per TPR threads, NV vectors each, straight to registers: for fewer
// rows than the ring's groups, where a row's latency is the time (1 x 4096
// bf16: 4.0 us a call, the launch and two sums).
template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(cta_threads(TPR)) norm_forward_kernel(const NormCall c, int vec) {
  __shared__ __align__(16) float red[2][32];
  chain_next();
  chain_wait();
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
// Rows through a ring in shared memory.  A CTA fills an SM with groups of TPR
// threads (a warp, or several with a barrier of their own); each group takes
// every step-th row, and bulk copies bring its next `stages` rows while it
// works on one, so that memory stays busy through the two sums and the
// barriers of a row.  A slot is free again once every thread holds its part of
// the row in registers, which the first sum's barrier says.  The parameters
// lie in shared memory too, once for all groups: read through L1, what the
// ring leaves of it did not hold them (16384 x 8192 bf16: 107 us, 84 % of the
// stalls on those loads).  Bound by HBM: 16384 x 8192 bf16 88 us, 6.1 TB/s,
// 0.90 of the copy rate; 1021 x 5003 f32 in rows of no alignment 15.5 us, bound
// by its element-by-element loads and stores.
// ---------------------------------------------------------------------------
template <int TPR, int EPT, bool kBackward>
struct RingCfg {
  // Threads an SM holds: by the registers that a thread's EPT elements (and,
  // backward, their column sums) take.
  static constexpr int kResident = kBackward ? (EPT > 8 ? 512 : 1024) : (EPT > 16 ? 768 : 1024);
  static constexpr int kGroups = kResident > TPR ? kResident / TPR : 1;
  static constexpr int kThreads = kGroups * TPR;
};
constexpr int kRingBytes = 216 * 1024;  // shared memory of a CTA: parameters, kFront, the slots
constexpr int kMaxStages = 4;
constexpr int kFront = 128;  // bytes before the first slot: a row's start may lie up to 15 before its slot

// Copies n parameters to shared memory.
template <typename W, bool kAligned>
__device__ __forceinline__ void keep_params(W* to, const void* from, int n) {
  if constexpr (kAligned) {
    const int pieces = n * static_cast<int>(sizeof(W)) / 16;
#pragma unroll 4
    for (int j = threadIdx.x; j < pieces; j += blockDim.x)
      reinterpret_cast<uint4*>(to)[j] = static_cast<const uint4*>(from)[j];
  } else {
#pragma unroll 8
    for (int j = threadIdx.x; j < n; j += blockDim.x) to[j] = static_cast<const W*>(from)[j];
  }
}
// Bytes that n parameters of type W take there.
template <typename W>
__host__ __device__ __forceinline__ int param_bytes(int n) {
  return (n * static_cast<int>(sizeof(W)) + 127) & ~127;
}

// The 2 EPT parameters of one 16-byte vector, in the rows' type T or fp32.
template <typename T, typename W>
__device__ __forceinline__ void load_params16(const void* base, int j, float2* v) {
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const W*>(base) + j);
  unpack16<W>(p[0], v);
  if constexpr (sizeof(W) > sizeof(T)) unpack16<W>(p[1], v + 2);
}

// The ring's rows: any start, 16-byte rows, and 16-byte rows of exactly TPR EPT
// columns, which need no comparison for each vector (backward at 16384 x 4096
// bf16: 100 -> 92 us; forward it made no difference and is not built).
enum RowMode { kAnyRow, kAlignedRow, kExactRow };

// How a thread's EPT elements of a row are laid out.  Aligned rows: NV 16-byte
// vectors, vector q at (q TPR + tid) VEC.  Rows that start anywhere: element i
// of "vector" q is (q VEC + i) TPR + tid, so that a warp still reads and writes
// consecutive elements.
template <typename T, int TPR, int EPT, int kMode>
struct Row {
  static constexpr int VEC = 16 / sizeof(T), NV = EPT / VEC, H = VEC / 2;
  static __device__ __forceinline__ int column(int tid, int q, int i) {
    return kMode != kAnyRow ? (q * TPR + tid) * VEC + i : (q * VEC + i) * TPR + tid;
  }
};

// The bulk copy of one row: 16-byte pieces that hold it, taken whole where
// they lie within the matrix.  The first row's start and the last row's end
// may lie in pieces that do not: those elements are read by themselves.
struct RowCopy {
  uintptr_t from;
  uint32_t bytes;
  int shift;  // byte of the slot where the row starts (negative: not copied)
};
template <typename T>
__device__ __forceinline__ RowCopy row_copy(const void* base, long long ld, long long row, int rows, int cols) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(static_cast<const T*>(base) + row * ld);
  const uintptr_t end = at + static_cast<uintptr_t>(cols) * sizeof(T);
  const uintptr_t a = row > 0 ? at & ~uintptr_t(15) : (at + 15) & ~uintptr_t(15);
  const uintptr_t b = row < rows - 1 ? (end + 15) & ~uintptr_t(15) : end & ~uintptr_t(15);
  return {a, static_cast<uint32_t>(b - a), static_cast<int>(static_cast<intptr_t>(at - a))};
}
// Bytes of a slot for a row of `cols` elements.
template <typename T, int kMode>
__host__ __device__ __forceinline__ uint32_t slot_bytes_of(int cols) {
  const uint32_t bytes = static_cast<uint32_t>(cols) * sizeof(T);
  return kMode != kAnyRow ? bytes : (bytes + 30) & ~15u;
}

// Starts the copy of a row to its slot.
template <typename T, int kMode>
__device__ __forceinline__ uint32_t start_row(uint8_t* slot, const void* base, long long ld, long long row, int rows,
                                              int cols, uint64_t* bar, bool go) {
  if constexpr (kMode != kAnyRow) {
    const uint32_t bytes = static_cast<uint32_t>(cols) * sizeof(T);
    if (go) bulk_load(slot, static_cast<const T*>(base) + row * ld, bytes, bar);
    return bytes;
  } else {
    const RowCopy c = row_copy<T>(base, ld, row, rows, cols);
    if (go) bulk_load(slot, reinterpret_cast<const void*>(c.from), c.bytes, bar);
    return c.bytes;
  }
}

// A thread's elements of the row in a slot, NQ vectors from vector q0 on; 0
// past the row's end.
template <typename T, int TPR, int EPT, int kMode, int NQ = EPT / (16 / sizeof(T))>
__device__ __forceinline__ void take_row(const uint8_t* slot, const void* base, long long ld, long long row, int rows,
                                         int cols, int tid, float2 (&v)[NQ][8 / sizeof(T)], int q0 = 0) {
  using L = Row<T, TPR, EPT, kMode>;
  if constexpr (kMode != kAnyRow) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      if (kMode == kExactRow || L::column(tid, q0 + q, 0) < cols) {
        unpack16<T>(*reinterpret_cast<const uint4*>(slot + ((q0 + q) * TPR + tid) * 16), v[q]);
      } else {
#pragma unroll
        for (int i = 0; i < L::H; ++i) v[q][i] = make_float2(0.f, 0.f);
      }
    }
  } else {
    // Every element from the slot, those of the matrix's first and last bytes
    // again from memory.
    const RowCopy c = row_copy<T>(base, ld, row, rows, cols);
    const uint8_t* mine = slot + c.shift + tid * static_cast<int>(sizeof(T));
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int i = 0; i < L::VEC; ++i) {
        const int j = L::column(tid, q0 + q, i);
        const float f = j < cols ? to_float(*reinterpret_cast<const T*>(mine + ((q0 + q) * L::VEC + i) * TPR * sizeof(T))) : 0.f;
        (i & 1 ? v[q][i / 2].y : v[q][i / 2].x) = f;
      }
    if (row == 0 || row == rows - 1) {
      const T* whole = static_cast<const T*>(base) + row * ld;
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int i = 0; i < L::VEC; ++i) {
          const int j = L::column(tid, q0 + q, i), off = c.shift + j * static_cast<int>(sizeof(T));
          if (j < cols && (off < 0 || off + static_cast<int>(sizeof(T)) > static_cast<int>(c.bytes)))
            (i & 1 ? v[q][i / 2].y : v[q][i / 2].x) = to_float(whole[j]);
        }
    }
  }
}

// A thread's parameters of vector q, and its store of one.
template <typename T, typename W, int TPR, int EPT, int kMode>
__device__ __forceinline__ void take_params(const void* base, int cols, int tid, int q, float2 (&v)[8 / sizeof(T)]) {
  using L = Row<T, TPR, EPT, kMode>;
  if constexpr (kMode != kAnyRow) {
    load_params16<T, W>(base, L::column(tid, q, 0), v);
  } else {
#pragma unroll
    for (int i = 0; i < L::VEC; ++i) {
      const int j = L::column(tid, q, i);
      (i & 1 ? v[i / 2].y : v[i / 2].x) = j < cols ? to_float(static_cast<const W*>(base)[j]) : 0.f;
    }
  }
}
template <typename T, int TPR, int EPT, int kMode>
__device__ __forceinline__ void put_row(T* out, int cols, int tid, int q, const float2 (&v)[8 / sizeof(T)]) {
  using L = Row<T, TPR, EPT, kMode>;
  if constexpr (kMode != kAnyRow) {
    *reinterpret_cast<uint4*>(out + L::column(tid, q, 0)) = pack16<T>(v);
  } else {
#pragma unroll
    for (int i = 0; i < L::VEC; ++i) {
      const int j = L::column(tid, q, i);
      if (j < cols) out[j] = from_float<T>(i & 1 ? v[i / 2].y : v[i / 2].x);
    }
  }
}

template <typename T, typename W, int TPR, int EPT, int kMode>
__global__ void __launch_bounds__(RingCfg<TPR, EPT, false>::kThreads, 1)
    norm_forward_ring_kernel(const NormCall c, int stages, float inv) {
  using L = Row<T, TPR, EPT, kMode>;
  using R = RingCfg<TPR, EPT, false>;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) float red_all[R::kGroups][2][TPR < 128 ? 4 : TPR / 32];
  __shared__ uint64_t bars[R::kGroups][kMaxStages];
  __shared__ int gave_up[R::kGroups][2], abort_word;
  const int tid = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const uint32_t bytes = slot_bytes_of<T, kMode>(c.cols);
  const float n = static_cast<float>(c.cols);
  W* weight = reinterpret_cast<W*>(ring);
  W* bias = reinterpret_cast<W*>(ring + (c.weight ? param_bytes<W>(c.cols) : 0));
  uint8_t* slots = reinterpret_cast<uint8_t*>(bias) + (c.bias ? param_bytes<W>(c.cols) : 0) + kFront +
                   static_cast<size_t>(group) * stages * bytes;
  uint64_t* full = bars[group];
  float(*red)[TPR < 128 ? 4 : TPR / 32] = red_all[group];
  // The CTAs' first groups take the first rows, so that few rows spread.
  const int step = gridDim.x * R::kGroups, first = group * gridDim.x + blockIdx.x;
  int issued = 0;
  auto issue = [&](long long row, int slot) {
    uint64_t* bar = &full[slot];
    mbar_arrive_expect_tx_relaxed(bar, start_row<T, kMode>(nullptr, c.x, c.ldx, row, c.rows, c.cols, bar, false));
    start_row<T, kMode>(slots + slot * bytes, c.x, c.ldx, row, c.rows, c.cols, bar, true);
    ++issued;
  };
  if (threadIdx.x == 0) abort_word = 0;
  if (tid < 2) gave_up[group][tid] = 0;
  chain_next();
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
    chain_wait();
    for (long long row = first; issued < stages && row < c.rows; row += step) issue(row, issued);
  }
  chain_wait();
  if (c.weight) keep_params<W, kMode != kAnyRow>(weight, c.weight, c.cols);
  if (c.bias) keep_params<W, kMode != kAnyRow>(bias, c.bias, c.cols);
  __syncthreads();
  int slot = 0, turn = 0;
  for (long long row = first; row < c.rows; row += step, ++turn) {
    if (!slot_wait<TPR>(&full[slot], (turn / stages) & 1, &gave_up[group][turn & 1], &abort_word, c.flags)) break;
    float2 d[L::NV][L::H];
    take_row<T, TPR, EPT, kMode>(slots + slot * bytes, c.x, c.ldx, row, c.rows, c.cols, tid, d);
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int q = 0; q < L::NV; ++q)
#pragma unroll
      for (int i = 0; i < L::H; ++i) s = add2(s, d[q][i]);
    const float mean = mean_of(row_sum<TPR>(s.x + s.y, red[0]), n, inv);
    if (!group_goes_on<TPR>(&gave_up[group][turn & 1])) break;
    __syncwarp();
    if (tid == 0) {
      const long long later = row + static_cast<long long>(stages) * step;
      if (later < c.rows) issue(later, slot);
    }
    if (++slot == stages) slot = 0;
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int q = 0; q < L::NV; ++q)
#pragma unroll
      for (int i = 0; i < L::H; ++i) {
        d[q][i] = add2(d[q][i], both(-mean));
        if constexpr (kMode != kAnyRow) {
          if (kMode != kExactRow && L::column(tid, q, 0) >= c.cols) break;
        } else {
          if (L::column(tid, q, 2 * i) >= c.cols) d[q][i].x = 0.f;
          if (L::column(tid, q, 2 * i + 1) >= c.cols) d[q][i].y = 0.f;
        }
        s = fma2(d[q][i], d[q][i], s);
      }
    const float rstd = 1.f / sqrtf(mean_of(row_sum<TPR>(s.x + s.y, red[1]), n, inv) + c.eps);
    T* y = static_cast<T*>(c.y) + row * c.ldy;
#pragma unroll
    for (int q = 0; q < L::NV; ++q) {
      if (kMode != kExactRow && L::column(tid, q, 0) >= c.cols) break;
#pragma unroll
      for (int i = 0; i < L::H; ++i) d[q][i] = mul2(d[q][i], both(rstd));
      float2 p[L::H];
      if (c.weight) {
        take_params<T, W, TPR, EPT, kMode>(weight, c.cols, tid, q, p);
#pragma unroll
        for (int i = 0; i < L::H; ++i) d[q][i] = mul2(d[q][i], p[i]);
      }
      if (c.bias) {
        take_params<T, W, TPR, EPT, kMode>(bias, c.cols, tid, q, p);
#pragma unroll
        for (int i = 0; i < L::H; ++i) d[q][i] = add2(d[q][i], p[i]);
      }
      put_row<T, TPR, EPT, kMode>(y, c.cols, tid, q, d[q]);
    }
    if (tid == 0) {
      if (c.mean) c.mean[row] = mean;
      if (c.rstd) c.rstd[row] = rstd;
    }
  }
  if (tid == 0) let_copies_land(full, turn, stages, issued);  // none, unless the group gave up
}

// Rows of more than 32,768 columns, or too long for two slots: read three times
// (from L2 after the first).
constexpr int kLong = 1024;
template <typename T>
__global__ void __launch_bounds__(kLong) norm_forward_long_kernel(const NormCall c) {
  __shared__ __align__(16) float red[2][32];
  chain_next();
  chain_wait();
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
// in order.  A thread keeps the same columns for every row, their sums in
// registers.
// ---------------------------------------------------------------------------

// CTAs that leave partial sums, at most: one to an SM.
constexpr int kMaxParts = 152;

// The sums of one row: (sum g, sum g xhat) over its TPR threads.
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float2 s, float2* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    s = add2(s, make_float2(__shfl_xor_sync(0xFFFFFFFFu, s.x, o), __shfl_xor_sync(0xFFFFFFFFu, s.y, o)));
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x % TPR >> 5] = s;
    row_barrier<TPR>();
    s = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < TPR / 32; w += 2) {
      const float4 t = *reinterpret_cast<const float4*>(red + w);
      s = add2(s, add2(make_float2(t.x, t.y), make_float2(t.z, t.w)));
    }
  }
  return s;
}

// Rows through the ring: a slot holds x, dy and, where given, dr of one row.
// Up to 8192 columns a thread keeps its 16 elements of x and dy from the sums
// to dx; with 32 (and their 64 column sums) it takes them from the slot twice,
// and the slot is free after dx.  16384 x 4096 bf16 with dr: 92.1 us, 0.86 of
// the copy rate (its 512 threads, all that the column sums leave registers for,
// wait for shared memory); 8192 x 16384 bf16: 150 us where the two passes below
// took 413; with dr and fp32 weights, room for one slot, 292; 777 x 2051 f16, odd rows: 12.8 (5 rows an SM, each
// its latency; element by element).
template <typename T, typename W, int TPR, int EPT, int kMode>
__global__ void __launch_bounds__(RingCfg<TPR, EPT, true>::kThreads, 1)
    norm_backward_ring_kernel(const NormGradCall c, float* part, int parts, int stages, float inv) {
  using L = Row<T, TPR, EPT, kMode>;
  using R = RingCfg<TPR, EPT, true>;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) float2 red_all[R::kGroups][2][TPR < 128 ? 4 : TPR / 32];
  __shared__ uint64_t bars[R::kGroups][kMaxStages];
  __shared__ int gave_up[R::kGroups][2], abort_word;
  const int tid = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const uint32_t bytes = slot_bytes_of<T, kMode>(c.cols), slot_bytes = bytes * (c.dr ? 3 : 2);
  const float n = static_cast<float>(c.cols);
  W* weight = reinterpret_cast<W*>(ring);
  uint8_t* slots =
      ring + (c.weight ? param_bytes<W>(c.cols) : 0) + kFront + static_cast<size_t>(group) * stages * slot_bytes;
  uint64_t* full = bars[group];
  float2(*red)[TPR < 128 ? 4 : TPR / 32] = red_all[group];
  const int step = gridDim.x * R::kGroups, first = group * gridDim.x + blockIdx.x;
  constexpr bool kTwice = EPT > 16;
  constexpr int NQ = kTwice ? 1 : L::NV;  // vectors held at a time
  auto past = [&](int q) { return kMode != kExactRow && L::column(tid, q, 0) >= c.cols; };
  float2 sw[L::NV][L::H], sb[L::NV][L::H];
#pragma unroll
  for (int q = 0; q < L::NV; ++q)
#pragma unroll
    for (int i = 0; i < L::H; ++i) sw[q][i] = sb[q][i] = make_float2(0.f, 0.f);
  int issued = 0;
  auto issue = [&](long long row, int slot) {
    uint8_t* to = slots + slot * slot_bytes;
    uint64_t* bar = &full[slot];
    uint32_t all = start_row<T, kMode>(nullptr, c.x, c.ldx, row, c.rows, c.cols, bar, false) +
                   start_row<T, kMode>(nullptr, c.dy, c.lddy, row, c.rows, c.cols, bar, false);
    if (c.dr) all += start_row<T, kMode>(nullptr, c.dr, c.lddr, row, c.rows, c.cols, bar, false);
    mbar_arrive_expect_tx_relaxed(bar, all);
    start_row<T, kMode>(to, c.x, c.ldx, row, c.rows, c.cols, bar, true);
    start_row<T, kMode>(to + bytes, c.dy, c.lddy, row, c.rows, c.cols, bar, true);
    if (c.dr) start_row<T, kMode>(to + 2 * bytes, c.dr, c.lddr, row, c.rows, c.cols, bar, true);
    ++issued;
  };
  if (threadIdx.x == 0) abort_word = 0;
  if (tid < 2) gave_up[group][tid] = 0;
  chain_next();
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
    chain_wait();
    for (long long row = first; issued < stages && row < c.rows; row += step) issue(row, issued);
  }
  chain_wait();
  if (c.weight) keep_params<W, kMode != kAnyRow>(weight, c.weight, c.cols);
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
    if (!slot_wait<TPR>(&full[slot], (turn / stages) & 1, &gave_up[group][turn & 1], &abort_word, c.flags)) break;
    const uint8_t* in = slots + slot * slot_bytes;
    float2 xh[NQ][L::H], g[NQ][L::H], dr[NQ][L::H];
    auto take = [&](int q0) {
      take_row<T, TPR, EPT, kMode, NQ>(in, c.x, c.ldx, row, c.rows, c.cols, tid, xh, q0);
      take_row<T, TPR, EPT, kMode, NQ>(in + bytes, c.dy, c.lddy, row, c.rows, c.cols, tid, g, q0);
    };
    auto normalise = [&](float2(&v)[L::H]) {
#pragma unroll
      for (int i = 0; i < L::H; ++i) v[i] = mul2(add2(v[i], both(-mean)), both(rstd));
    };
    auto weigh = [&](int q, float2(&v)[L::H]) {
      if (!c.weight) return;
      float2 w[L::H];
      take_params<T, W, TPR, EPT, kMode>(weight, c.cols, tid, q, w);
#pragma unroll
      for (int i = 0; i < L::H; ++i) v[i] = mul2(v[i], w[i]);
    };
    float2 s1 = make_float2(0.f, 0.f), s2 = s1;
#pragma unroll
    for (int q0 = 0; q0 < L::NV; q0 += NQ) {
      take(q0);
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        if (past(q0 + q)) break;  // dy is 0 there, and so are the sums
        normalise(xh[q]);
#pragma unroll
        for (int i = 0; i < L::H; ++i) {
          sw[q0 + q][i] = fma2(g[q][i], xh[q][i], sw[q0 + q][i]);
          sb[q0 + q][i] = add2(sb[q0 + q][i], g[q][i]);
        }
        weigh(q0 + q, g[q]);
#pragma unroll
        for (int i = 0; i < L::H; ++i) {
          s1 = add2(s1, g[q][i]);
          s2 = fma2(g[q][i], xh[q][i], s2);
        }
      }
    }
    auto take_dr = [&](int q0) {
      if (c.dr) take_row<T, TPR, EPT, kMode, NQ>(in + 2 * bytes, c.dr, c.lddr, row, c.rows, c.cols, tid, dr, q0);
    };
    if (!kTwice) take_dr(0);
    const float2 s = row_sum2<TPR>(make_float2(s1.x + s1.y, s2.x + s2.y), red[turn & 1]);
    // A group that gives up still writes this row, of whatever its slot holds
    // (the status tells), and leaves at its end: a way out from here took the
    // rows of any start 76 bytes of spilled registers (777 x 2051 f16 13.4 us, 12.8 without).
    const bool on = group_goes_on<TPR>(&gave_up[group][turn & 1]);
    auto release = [&] {
      if (tid == 0 && on) {
        const long long later = row + static_cast<long long>(stages) * step;
        if (later < c.rows) issue(later, slot);
      }
      if (++slot == stages) slot = 0;
    };
    if (!kTwice) {
      __syncwarp();
      release();
    }
    const float c1 = mean_of(s.x, n, inv), c2 = mean_of(s.y, n, inv);
    T* dx = static_cast<T*>(c.dx) + row * c.lddx;
#pragma unroll
    for (int q0 = 0; q0 < L::NV; q0 += NQ) {
      if (kTwice) {
        take(q0);
        take_dr(q0);
      }
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        if (past(q0 + q)) break;
        if (kTwice) {
          normalise(xh[q]);
          weigh(q0 + q, g[q]);
        }
#pragma unroll
        for (int i = 0; i < L::H; ++i) {
          const float2 v = fma2(xh[q][i], both(-c2), add2(g[q][i], both(-c1)));
          g[q][i] = c.dr ? fma2(v, both(rstd), dr[q][i]) : mul2(v, both(rstd));
        }
        put_row<T, TPR, EPT, kMode>(dx, c.cols, tid, q0 + q, g[q]);
      }
    }
    if (kTwice) {
      row_barrier<TPR>();
      release();
    }
    if (!on) break;
    mean = next_mean;
    rstd = next_rstd;
  }
  if (tid == 0) let_copies_land(full, turn, stages, issued);  // none, unless the group gave up

  // This CTA's sums: part[0][cta][.] of dw, part[1][cta][.] of db.
  float* pw = part + static_cast<long long>(blockIdx.x) * c.cols;
  float* pb = pw + static_cast<long long>(parts) * c.cols;
  if constexpr (R::kGroups > 1) {  // the groups' sums first, in order, in the ring's memory
    constexpr int kWidth = TPR * EPT;
    float* mem = reinterpret_cast<float*>(ring);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < L::NV; ++q)
#pragma unroll
      for (int i = 0; i < L::H; ++i) {
        float* a = mem + (2 * group) * kWidth;
        const int j = L::column(tid, q, 2 * i), k = L::column(tid, q, 2 * i + 1);
        a[j] = sw[q][i].x;
        a[k] = sw[q][i].y;
        a[kWidth + j] = sb[q][i].x;
        a[kWidth + k] = sb[q][i].y;
      }
    __syncthreads();
    for (int j = threadIdx.x; j < c.cols; j += R::kThreads) {
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int r = 0; r < R::kGroups; ++r) {
        a += mem[(2 * r) * kWidth + j];
        b += mem[(2 * r + 1) * kWidth + j];
      }
      pw[j] = a;
      pb[j] = b;
    }
  } else {
#pragma unroll
    for (int q = 0; q < L::NV; ++q)
#pragma unroll
      for (int i = 0; i < L::H; ++i) {
        const int j = L::column(tid, q, 2 * i), k = L::column(tid, q, 2 * i + 1);
        if (j < c.cols) {
          pw[j] = sw[q][i].x;
          pb[j] = sb[q][i].x;
        }
        if (k < c.cols) {
          pw[k] = sw[q][i].y;
          pb[k] = sb[q][i].y;
        }
      }
  }
}

// Rows too long for a slot (above 16384 columns; fp32 with dr above 13,000 or
// so), and those below 64 bytes, in two passes: the row's mean(g) and mean(g xhat), a CTA
// a row; then dx and the column sums, a CTA 256 columns of a chunk of rows.
// The second reading of x and dy is the price of rows that no CTA can hold.
template <typename T>
__global__ void __launch_bounds__(512) norm_backward_means_kernel(const NormGradCall c, float2* means, bool vec,
                                                                  bool weight_vec) {
  constexpr int VEC = 16 / sizeof(T);
  __shared__ __align__(16) float2 red[2][32];
  chain_next();
  chain_wait();
  const bool f32 = c.param_type == kF32;
  int turn = 0;
  for (long long row = blockIdx.x; row < c.rows; row += gridDim.x, turn ^= 1) {
    const T* x = static_cast<const T*>(c.x) + row * c.ldx;
    const T* dy = static_cast<const T*>(c.dy) + row * c.lddy;
    const float mean = c.mean[row], rstd = c.rstd[row];
    float2 s = make_float2(0.f, 0.f);
    auto add = [&](float d, float xv, float w) {
      const float g = d * w;
      s.x += g;
      s.y += g * ((xv - mean) * rstd);
    };
    if (vec) {
      for (int j = threadIdx.x * VEC; j < c.cols; j += 512 * VEC) {
        const int left = c.cols - j;
        float a[VEC], d[VEC], w[VEC];
        load_vec<T, VEC>(x + j, left, a);
        load_vec<T, VEC>(dy + j, left, d);
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[i] = 1.f;
        if (c.weight) load_params<T, VEC>(c.weight, f32, weight_vec, j, left, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (i < left) add(d[i], a[i], w[i]);
      }
    } else {
      for (int j = threadIdx.x; j < c.cols; j += 512) {
        float w[1] = {1.f};
        if (c.weight) load_params<T, 1>(c.weight, f32, true, j, 1, w);
        add(to_float(dy[j]), to_float(x[j]), w[0]);
      }
    }
    s = row_sum2<512>(s, red[turn]);
    if (threadIdx.x == 0) means[row] = make_float2(s.x / static_cast<float>(c.cols), s.y / static_cast<float>(c.cols));
  }
}

template <typename T, bool kAligned>
__global__ void __launch_bounds__(256) norm_backward_columns_kernel(const NormGradCall c, const float2* means,
                                                                    float* part, int parts, int chunk) {
  // Eight columns a thread, eight rows at a time.
  __shared__ float red[2][8][264];
  chain_next();
  chain_wait();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, col0 = blockIdx.x * 256;
  const bool f32 = c.param_type == kF32;
  float w[8], sw[8] = {}, sb[8] = {};
  auto column = [&](int i) { return col0 + (kAligned ? tx * 8 + i : i * 32 + tx); };
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = 1.f;
    if (c.weight && column(i) < c.cols) {
      float v[1];
      load_params<T, 1>(c.weight, f32, true, column(i), 1, v);
      w[i] = v[0];
    }
  }
  auto take = [&](const void* base, long long ld, long long row, float (&v)[8]) {
    const T* p = static_cast<const T*>(base) + row * ld;
    constexpr int VEC = 16 / sizeof(T);
    if constexpr (kAligned) {
#pragma unroll
      for (int q = 0; q < 8; q += VEC)
        load_vec<T, VEC>(p + column(q), c.cols - column(q), reinterpret_cast<float(&)[VEC]>(v[q]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = column(i) < c.cols ? to_float(p[column(i)]) : 0.f;
    }
  };
  const long long end = min(static_cast<long long>(c.rows), (blockIdx.y + 1LL) * chunk);
#pragma unroll 2
  for (long long row = static_cast<long long>(blockIdx.y) * chunk + ty; row < end; row += 8) {
    float x[8], dy[8], dr[8];
    take(c.x, c.ldx, row, x);
    take(c.dy, c.lddy, row, dy);
    if (c.dr) take(c.dr, c.lddr, row, dr);
    const float mean = c.mean[row], rstd = c.rstd[row];
    const float2 m = means[row];
    T* out = static_cast<T*>(c.dx) + row * c.lddx;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float xh = (x[i] - mean) * rstd;
      if (column(i) < c.cols) {
        sw[i] += dy[i] * xh;
        sb[i] += dy[i];
      }
      x[i] = rstd * (dy[i] * w[i] - m.x - xh * m.y) + (c.dr ? dr[i] : 0.f);
    }
    constexpr int VEC = 16 / sizeof(T);
    if constexpr (kAligned) {
#pragma unroll
      for (int q = 0; q < 8; q += VEC)
        store_vec<T, VEC>(out + column(q), reinterpret_cast<float(&)[VEC]>(x[q]), c.cols - column(q));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (column(i) < c.cols) out[column(i)] = from_float<T>(x[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    red[0][ty][column(i) - col0] = sw[i];
    red[1][ty][column(i) - col0] = sb[i];
  }
  __syncthreads();
  const int j = col0 + threadIdx.x;
  if (j < c.cols) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      a += red[0][y][threadIdx.x];
      b += red[1][y][threadIdx.x];
    }
    part[static_cast<long long>(blockIdx.y) * c.cols + j] = a;
    part[(static_cast<long long>(parts) + blockIdx.y) * c.cols + j] = b;
  }
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
    return launch_chained(norm_forward_kernel<T, VEC, 32, NV>, dim3((c.rows + 3) / 4), 128, 0, stream, 0, c, vec);
  if (c.cols <= 128 * span)
    return launch_chained(norm_forward_kernel<T, VEC, 128, NV>, dim3(c.rows), 128, 0, stream, 0, c, vec);
  if (c.cols <= 256 * span)
    return launch_chained(norm_forward_kernel<T, VEC, 256, NV>, dim3(c.rows), 256, 0, stream, 0, c, vec);
  if (c.cols <= 512 * span)
    return launch_chained(norm_forward_kernel<T, VEC, 512, NV>, dim3(c.rows), 512, 0, stream, 0, c, vec);
  if (c.cols <= 1024 * span)
    return launch_chained(norm_forward_kernel<T, VEC, 1024, NV>, dim3(c.rows), 1024, 0, stream, 0, c, vec);
  return launch_chained(norm_forward_long_kernel<T>, dim3(std::min(c.rows, 65536)), kLong, 0, stream, 0, c);
}

// Slots of each of a ring's groups, with `params` bytes of parameters before
// them.
int ring_stages(int params, int groups, int slot_bytes) {
  const int room = kRingBytes - params - kFront;
  return room <= 0 ? 0 : std::min(kMaxStages, room / (groups * std::max(slot_bytes, 16)));
}

struct ForwardLaunch {
  const NormCall& c;
  cudaStream_t stream;
  cudaError_t error = cudaSuccess;

  // Launches the ring for rows of at most TPR * EPT columns, if there are
  // enough rows to go round.  Fewer rows go to wider groups, of which fewer
  // fit, but not to groups of which a row fills an eighth or less (a sixteenth
  // where it goes element by element): norm_forward_kernel is quicker there,
  // by its narrower groups and its lack of a start.  us, the wider ring and it,
  // bf16 unless named: 300 x 256 4.2, 2.2; 2000 x 256 5.9, 3.2; 456 x 1024 f32
  // 5.5, 3.0; 456 x 2048 5.5, 4.0; 950 x 63 5.9, 2.6.  Above those shares the
  // ring is: 700 x 2048 5.1, 6.8; 2000 x 1024 f32 7.6, 9.0; 300 x 2047 6.6, 8.4.
  template <typename T, typename W, int TPR, int EPT, int kMode>
  bool fits() {
    if (c.cols > TPR * EPT) return false;
    if (TPR > 32 && c.cols * (kMode == kAnyRow ? 16 : 8) <= TPR * EPT) return false;
    using R = RingCfg<TPR, EPT, false>;
    const int bytes = static_cast<int>(slot_bytes_of<T, kMode>(c.cols));
    const int params = param_bytes<W>(c.cols) * ((c.weight ? 1 : 0) + (c.bias ? 1 : 0));
    const int stages = ring_stages(params, R::kGroups, bytes);
    if (stages < 2 || c.rows <= kSms * R::kGroups) return false;
    auto kern = norm_forward_ring_kernel<T, W, TPR, EPT, kMode>;
    error = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (error != cudaSuccess) return true;
    error = launch_chained(kern, dim3(kSms), R::kThreads, params + kFront + R::kGroups * stages * bytes, stream, 0, c,
                           stages, 1.f / static_cast<float>(c.cols));
    return true;
  }
  template <typename T, typename W, int kMode>
  bool any() {
    if constexpr (kMode == kAnyRow)
      // Element by element: up to 2048 columns more threads of fewer elements
      // are quicker (65536 x 131 bf16 34 against 48 us, 16384 x 1025 f32 39
      // against 55), above it fewer of more (16384 x 4099 bf16 142 against 158).
      return fits<T, W, 32, 16, kMode>() || fits<T, W, 128, 16, kMode>() || fits<T, W, 128, 32, kMode>() ||
             fits<T, W, 256, 32, kMode>() || fits<T, W, 512, 32, kMode>() || fits<T, W, 1024, 32, kMode>();
    else
      return fits<T, W, 32, 32, kMode>() || fits<T, W, 128, 32, kMode>() || fits<T, W, 256, 32, kMode>() ||
             fits<T, W, 512, 32, kMode>() || fits<T, W, 1024, 32, kMode>();
  }
};

struct BackwardLaunch {
  const NormGradCall& c;
  cudaStream_t stream;
  int used = 0;  // parts written, of kMaxParts
  cudaError_t error = cudaSuccess;

  template <typename T, typename W, int TPR, int EPT, int kMode>
  bool ring() {
    if (c.cols > TPR * EPT) return false;
    if constexpr (kMode == kAlignedRow && TPR > 32)
      if (c.cols == TPR * EPT) return ring<T, W, TPR, EPT, kExactRow>();
    using R = RingCfg<TPR, EPT, true>;
    const int slot = static_cast<int>(slot_bytes_of<T, kMode>(c.cols)) * (c.dr ? 3 : 2);
    const int params = c.weight ? param_bytes<W>(c.cols) : 0;
    const int stages = ring_stages(params, R::kGroups, slot);
    if (stages < 1) return false;
    auto kern = norm_backward_ring_kernel<T, W, TPR, EPT, kMode>;
    error = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (error != cudaSuccess) return true;
    used = std::min(c.rows, kMaxParts);
    // The groups' column sums meet in the ring's memory.
    const int smem = std::max(params + kFront + R::kGroups * stages * slot, R::kGroups > 1 ? R::kThreads * EPT * 8 : 0);
    error = launch_chained(kern, dim3(used), R::kThreads, smem, stream, 0, c, static_cast<float*>(c.ws), kMaxParts,
                           stages, 1.f / static_cast<float>(c.cols));
    return true;
  }
  template <typename T, typename W, int kMode>
  bool any() {
    return ring<T, W, 32, 8, kMode>() || ring<T, W, 128, 16, kMode>() || ring<T, W, 256, 16, kMode>() ||
           ring<T, W, 512, 16, kMode>() || ring<T, W, 512, 32, kMode>();
  }
  template <typename T>
  void two_passes(bool vec) {
    float2* means = reinterpret_cast<float2*>(static_cast<float*>(c.ws) + 2LL * kMaxParts * c.cols);
    error = launch_chained(norm_backward_means_kernel<T>, dim3(std::min(c.rows, 65536)), 512, 0, stream, 0, c, means, vec,
                           aligned16(c.weight));
    if (error != cudaSuccess) return;
    const int across = (c.cols + 255) / 256;
    const int chunks = std::max(1, std::min({kMaxParts, 1216 / across, (c.rows + 7) / 8}));
    const int chunk = (c.rows + chunks - 1) / chunks;
    used = (c.rows - 1) / chunk + 1;  // rows + chunk may pass 2^31
    auto kern = vec ? norm_backward_columns_kernel<T, true> : norm_backward_columns_kernel<T, false>;
    error = launch_chained(kern, dim3(across, used), 256, 0, stream, 0, c, means, static_cast<float*>(c.ws), kMaxParts,
                           chunk);
  }
};

}  // namespace

cudaError_t launch_layer_norm(const NormCall& c, cudaStream_t stream) {
  const int size = type_bytes(c.type);
  const long long bytes = static_cast<long long>(c.cols) * size;
  const bool rows_vec = rows_aligned16(c.x, c.ldx, c.rows, size) && rows_aligned16(c.y, c.ldy, c.rows, size);
  const bool whole = rows_vec && bytes % 16 == 0 && aligned16(c.weight) && aligned16(c.bias);
  ForwardLaunch l{c, stream};
  return with_type(c.type, [&](auto t) {
    using T = decltype(t);
    const bool p32 = c.param_type == kF32;
    if (whole ? (p32 ? l.any<T, float, kAlignedRow>() : l.any<T, T, kAlignedRow>())
              : bytes >= 64 && (p32 ? l.any<T, float, kAnyRow>() : l.any<T, T, kAnyRow>()))
      return l.error;
    return rows_vec ? forward_vec<T, 16 / sizeof(T), 4>(c, stream) : forward_vec<T, 1, 16>(c, stream);
  });
}

size_t layer_norm_backward_workspace(int rows, int cols) {
  return static_cast<size_t>(2 * kMaxParts) * cols * 4 + static_cast<size_t>(rows) * 8;
}

cudaError_t launch_layer_norm_backward(const NormGradCall& c, cudaStream_t stream) {
  BackwardLaunch l{c, stream};
  if (c.rows > 0) {
    const int size = type_bytes(c.type);
    const long long bytes = static_cast<long long>(c.cols) * size;
    const bool vec = rows_aligned16(c.x, c.ldx, c.rows, size) && rows_aligned16(c.dy, c.lddy, c.rows, size) &&
                     rows_aligned16(c.dr, c.lddr, c.rows, size) && rows_aligned16(c.dx, c.lddx, c.rows, size);
    const bool whole = vec && bytes % 16 == 0 && aligned16(c.weight);
    with_type(c.type, [&](auto t) {
      using T = decltype(t);
      const bool p32 = c.param_type == kF32;
      if (!(whole ? (p32 ? l.any<T, float, kAlignedRow>() : l.any<T, T, kAlignedRow>())
                  : bytes >= 64 && (p32 ? l.any<T, float, kAnyRow>() : l.any<T, T, kAnyRow>())))
        l.two_passes<T>(vec);
      return l.error;
    });
    if (l.error != cudaSuccess) return l.error;
  }
  if (c.dweight || c.dbias) {
    const dim3 grid((c.cols + 31) / 32, 2);
    return with_type(c.param_type, [&](auto w) {
      using W = decltype(w);
      return launch_chained(join_parts_kernel<W>, grid, 1024, 0, stream, 0, static_cast<const float*>(c.ws), l.used,
                            kMaxParts, c.cols, static_cast<W*>(c.dweight), static_cast<W*>(c.dbias));
    });
  }
  return cudaSuccess;
}

}  // namespace ozemu
