// What the products on the tensor cores share (linear.cu, mx.cu): waits of
// whole warps, the way of accumulators through the epilogue into rows of any
// alignment, the order of tiles, and the host's helpers.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "layer.cuh"

namespace ozemu {

namespace {

constexpr int kEpiWarps = 16;

// What happens to an accumulator on its way out.
struct Epilogue {
  const void* bias;
  const void* res;
  long long ldr;
  void* pre;
  long long ldpre;
  void* out;
  long long ldo;
  int act;
  // Bits: 1 bias, 2 res, 4 pre, 8 out rows start on 16-byte boundaries.  Gated: 16
  // bias's, 32 pre's second half do; 4-bit product: 16 res and out rows on 32 bytes.
  int vec;
  bool times;  // res multiplies act(z) (kTimes epilogues) instead of being added
  const float* scale;  // of the sums: a number in memory (NULL: 1), in plain epilogues
};

// That number, which a launch before this one wrote (by L2: a line in L1 may be
// older than it).
__device__ __forceinline__ float sums_scale(const Epilogue& e) { return __ldcg(e.scale); }

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_word,
                                          uint32_t* flags) {
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, abort_word, flags) ? 1 : 0;
  return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}

// The loops that issue loads and MMAs are run by a whole warp, so that their
// addresses and descriptors stay in uniform registers, which these
// instructions take; one elected lane, always the same, issues.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ bool all_wait(uint64_t* bar, uint32_t parity, volatile int* abort_word, uint32_t* flags) {
  const bool ok = mbar_wait(bar, parity, abort_word, flags);
  return __all_sync(0xFFFFFFFFu, ok);
}

// Bounded wait that ignores the abort word (used while draining).
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, uint32_t* flags) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer() - t0 > kWaitLimitNs) {
      atomicOr(flags, kFlagTimeout);
      return;
    }
  }
}

// After an abort, gives copies already issued time to land.
__device__ __forceinline__ void settle_after_abort() {
  const uint64_t t0 = globaltimer();
  while (globaltimer() - t0 < 50000ull) {
  }
}

// Four elements, by plain loads (the memory may be the output's).
template <typename T>
__device__ __forceinline__ void load4(const T* p, int left, bool vec, float (&v)[4]) {
  if (vec && left >= 4) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = Pair<T>::unpack(u.x), b = Pair<T>::unpack(u.y);
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < left ? to_float(p[i]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&v)[4], int left, bool vec) {
  if (vec && left >= 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(Pair<T>::pack(v[0], v[1]), Pair<T>::pack(v[2], v[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) p[i] = from_float<T>(v[i]);
  }
}

template <int kAct, int N>
__device__ __forceinline__ void activate_each(float (&z)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) z[i] = activate(z[i], kAct);
}
template <int N>
__device__ __forceinline__ void activate_all(float (&z)[N], int act) {
  switch (act) {
    case kActRelu: activate_each<kActRelu>(z); break;
    case kActGelu: activate_each<kActGelu>(z); break;
    case kActGeluTanh: activate_each<kActGeluTanh>(z); break;
    case kActSilu: activate_each<kActSilu>(z); break;
    default: break;
  }
}

// The same of pairs of values, by packed arithmetic.
template <int kAct, int N>
__device__ __forceinline__ void activate_pairs(float2 (&z)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float2 a, slope;
    activation_and_slope2<kAct>(z[i], a, slope);
    z[i] = a;
  }
}
template <int N>
__device__ __forceinline__ void activate_all(float2 (&z)[N], int act) {
  switch (act) {
    case kActRelu: activate_pairs<kActRelu>(z); break;
    case kActGelu: activate_pairs<kActGelu>(z); break;
    case kActGeluTanh: activate_pairs<kActGeluTanh>(z); break;
    case kActSilu: activate_pairs<kActSilu>(z); break;
    default: break;
  }
}

// The 16 bytes that lie `off` bytes (even, under 16) into lo and hi together;
// without a branch, for lanes whose off differ.
__device__ __forceinline__ uint4 shifted16(const uint4& lo, const uint4& hi, uint32_t off) {
  uint32_t w[7] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z};
  const bool two = (off & 8) != 0, one = (off & 4) != 0;
  const uint32_t past = two ? hi.w : hi.z;
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = two ? w[i + 2] : w[i];
  w[5] = two ? past : w[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = one ? w[i + 1] : w[i];
  const uint32_t bits = (off & 2) * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A warp's 32 rows x 32 columns of 16-bit elements pass through its 2 KB of
// shared memory (row r at byte 64 r, its 16-byte piece c at piece
// c ^ (r / 2 % 4): no bank conflicts by rows or by pieces), so that a row moves
// as one 64-byte run.  A lane's share on the way: piece lane % 4 of rows
// 8 i + lane / 4, in global memory between two aligned pieces where rows do not
// start on 16-byte boundaries; or, of columns that the matrix ends within, word
// lane % 16 of rows 2 i + lane / 16, element by element.
__device__ __forceinline__ uint4* stage_piece(uint8_t* stage, int r, int c) {
  return reinterpret_cast<uint4*>(stage + r * 64) + (c ^ (r >> 1 & 3));
}
__device__ __forceinline__ uint32_t* stage_word(uint8_t* stage, int r, int w) {
  return reinterpret_cast<uint32_t*>(stage_piece(stage, r, w >> 2)) + (w & 3);
}

template <typename T>
__device__ __forceinline__ void read_rows(uint4 (&v)[4], const T* in, long long ld, int row0, int col0, int m, int n,
                                          bool vec) {
  const int lane = threadIdx.x & 31;
  if (col0 + 32 <= n) {
    // The memory that a vector may be read from: the matrix's.
    const uintptr_t begin = reinterpret_cast<uintptr_t>(in), end = reinterpret_cast<uintptr_t>(in + (m - 1LL) * ld + n);
    const int rows = m - row0, l4 = lane >> 2;
    const T* p = in + (row0 + l4) * ld + col0 + 8 * (lane & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i, p += 8 * ld) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (l4 + 8 * i >= rows) continue;
      if (vec) {
        v[i] = *reinterpret_cast<const uint4*>(p);
        continue;
      }
      const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
      const uintptr_t from = reinterpret_cast<uintptr_t>(p) - off;
      if (from >= begin && from + 32 <= end) {
        v[i] = shifted16(*reinterpret_cast<const uint4*>(from), *reinterpret_cast<const uint4*>(from + 16), off);
      } else {
        uint32_t* w = reinterpret_cast<uint32_t*>(&v[i]);
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = q[2 * k] | (static_cast<uint32_t>(q[2 * k + 1]) << 16);
      }
    }
    return;
  }
  uint32_t* w = reinterpret_cast<uint32_t*>(v);
  const uint16_t* p = reinterpret_cast<const uint16_t*>(in) + row0 * ld + col0;
  const int word = lane & 15;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = 2 * i + (lane >> 4);
    const uint16_t* q = p + r * ld + 2 * word;
    const uint32_t a = row0 + r < m && col0 + 2 * word < n ? q[0] : 0;
    const uint32_t b = row0 + r < m && col0 + 2 * word + 1 < n ? q[1] : 0;
    w[i] = a | (b << 16);
  }
}

__device__ __forceinline__ void stage_rows(const uint4 (&v)[4], uint8_t* stage, int col0, int n) {
  const int lane = threadIdx.x & 31;
  if (col0 + 32 <= n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) *stage_piece(stage, 8 * i + (lane >> 2), lane & 3) = v[i];
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
    for (int i = 0; i < 16; ++i) *stage_word(stage, 2 * i + (lane >> 4), lane & 15) = w[i];
  }
}

template <typename T>
__device__ __forceinline__ void write_rows(uint8_t* stage, T* out, long long ldo, int row0, int col0, int m, int n,
                                           bool vec) {
  const int lane = threadIdx.x & 31;
  if (vec && col0 + 32 <= n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2);
      if (row0 + r < m)
        *reinterpret_cast<uint4*>(out + (row0 + r) * ldo + col0 + 8 * (lane & 3)) = *stage_piece(stage, r, lane & 3);
    }
    return;
  }
  uint16_t* p = reinterpret_cast<uint16_t*>(out) + row0 * ldo + col0;
  if (col0 + 32 <= n) {
    // The whole 16-byte pieces of a row's run, `to` bytes in: three, or four of a
    // row that starts on a boundary.  Bound by instructions, so their addresses are
    // stepped: the places of a lane's rows, eight or four apart, differ by a
    // constant (the pieces' order comes from bits 1 and 2 of the row).
    const int rows = m - row0, l4 = lane >> 2, slot = lane & 3;
    uint16_t* q = p + l4 * ldo;
    const uint4 *a = stage_piece(stage, l4, slot), *b = stage_piece(stage, l4, (slot + 1) & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i, q += 8 * ldo) {
      const uint32_t to = (0u - static_cast<uint32_t>(reinterpret_cast<uintptr_t>(q))) & 15u;
      const uint4 v = shifted16(a[32 * i], b[32 * i], to);
      if (l4 + 8 * i < rows && (to == 0 || slot < 3)) *reinterpret_cast<uint4*>(q + to / 2 + 8 * slot) = v;
    }
    // And the eight elements before and after them, of piece 0 or 3 each, by eight
    // lanes a row.
    const int l8 = lane >> 3, k = lane & 7;
    q = p + l8 * ldo;
    const uint8_t* row = stage + l8 * 64 + 2 * k;
#pragma unroll
    for (int i = 0; i < 8; ++i, q += 4 * ldo) {
      const int head = static_cast<int>(((0u - static_cast<uint32_t>(reinterpret_cast<uintptr_t>(q))) & 15u) / 2);
      const int order = 2 * (i & 1) + (l8 >> 1);
      const uint16_t v = *reinterpret_cast<const uint16_t*>(row + 256 * i + 16 * (k < head ? order : order ^ 3));
      if (l8 + 4 * i < rows && head != 0) q[k < head ? k : 24 + k] = v;
    }
    return;
  }
  const int word = lane & 15;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int r = 2 * i + (lane >> 4);
    const uint32_t a = *stage_word(stage, r, word);
    uint16_t* q = p + r * ldo;
    const bool in_m = row0 + r < m;
    if (in_m && col0 + 2 * word < n) q[2 * word] = static_cast<uint16_t>(a);
    if (in_m && col0 + 2 * word + 1 < n) q[2 * word + 1] = static_cast<uint16_t>(a >> 16);
  }
}

// The four warps that hold the same 32 rows of a tile (a lane quarter of TMEM),
// 128 columns together.  Where rows start on no 16-byte boundaries they write
// them as one, in runs of 256 bytes: a run's first and last sector go out in part,
// and a part of a sector takes the way to L2 that a whole one takes.  (8192 x 192
// -> 9449 gated, the pre-activations kept, by runs of 64 bytes: 884 MB on that way
// for 464 written.  15075 rows of it: 578 us, 380 by these.)
struct Quarter {
  uint8_t* staging;  // of its first warp; the next one's is kQuarterStride on
  int id, group;     // quarter, and which of its warps
};
constexpr int kQuarterStride = 4 * 2048;
__device__ __forceinline__ void quarter_sync(const Quarter& q) {
  asm volatile("bar.sync %0, 128;" ::"r"(q.id + 1) : "memory");
}
// Whether all four say so: they give up a wait together or not at all, since
// each would be missing from the others' barriers.
__device__ __forceinline__ bool quarter_all(const Quarter& q, bool ok) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.and.pred p, %2, 128, q;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u), "r"(q.id + 1)
      : "memory");
  return all != 0;
}

// Rows row0 .. row0 + 31 of the quarter's columns from col0 on, up to 128 and
// below `end`, staged by its warps, to memory of any alignment: eight rows a warp,
// half a warp a row.
template <typename T>
__device__ __forceinline__ void write_together(const Quarter& q, T* out, long long ldo, int row0, int col0, int m, int end) {
  const int lane = threadIdx.x & 31, slot = lane & 15, cols = min(128, end - col0);
  const int first = q.group * 8 + (lane >> 4), rows = m - row0 - first, next = min(slot + 1, 15);
  uint16_t* p = reinterpret_cast<uint16_t*>(out) + (row0 + first) * ldo + col0;
  const uint8_t* at0 = q.staging + first * 64;  // rows go by two, whose pieces' order is i
  const uint8_t *a = at0 + (slot >> 2) * kQuarterStride, *b = at0 + (next >> 2) * kQuarterStride;
#pragma unroll
  for (int i = 0; i < 4; ++i, p += 2 * ldo) {
    // Elements to the first boundary, whole pieces after it, and the rest.
    const int head = static_cast<int>(((0u - static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p))) & 15u) / 2);
    const int whole = max(cols - head, 0) / 8;
    const uint4 v = shifted16(*reinterpret_cast<const uint4*>(a + 128 * i + 16 * ((slot & 3) ^ i)),
                              *reinterpret_cast<const uint4*>(b + 128 * i + 16 * ((next & 3) ^ i)), 2 * head);
    if (2 * i < rows && slot < whole) *reinterpret_cast<uint4*>(p + head + 8 * slot) = v;
    const int at = slot < 8 ? slot : head + 8 * whole + slot - 8, stop = slot < 8 ? min(head, cols) : cols;
    const int piece = (at >> 3) & 15;
    const uint16_t one = *reinterpret_cast<const uint16_t*>(at0 + (piece >> 2) * kQuarterStride + 128 * i +
                                                            16 * ((piece & 3) ^ i) + 2 * (at & 7));
    if (2 * i < rows && at < stop) p[at] = one;
  }
}

constexpr int kGroupM = 8;  // tile rows swept together, for reuse of B's columns in L2

// A grid of tiles and the reciprocal that gives a tile's turn.
struct Raster {
  int m, n;
  uint32_t group_inverse, group_shift;  // of kGroupM n
  __host__ __device__ int count() const { return m * n; }
};
inline Raster raster(int m, int n) {
  // ceil(2^(32 + shift) / d) with 2^shift >= d gives t / d for t < 2^31; with
  // the shift one less the multiplier fits 32 bits, for t < 2^31 still.
  Raster r = {m, n, 0, 0};
  const uint64_t d = static_cast<uint64_t>(kGroupM) * n;
  while ((2ull << r.group_shift) < d) ++r.group_shift;
  r.group_inverse = static_cast<uint32_t>(((1ull << (32 + r.group_shift)) + d - 1) / d);
  return r;
}

__device__ __forceinline__ void tile_of(int t, const Raster& p, int& tm, int& tn) {
  // t / (kGroupM n) by the reciprocal that the host rounded up: exact
  // for the product's tiles.
  const int turn = static_cast<int>(__umulhi(static_cast<uint32_t>(t), p.group_inverse) >> p.group_shift);
  const int first = turn * kGroupM, rest = t - turn * kGroupM * p.n;
  const int gm = min(kGroupM, p.m - first);
  if (gm == kGroupM) {
    tn = rest / kGroupM;
    tm = first + rest % kGroupM;
  } else {
    tn = rest / gm;
    tm = first + rest % gm;
  }
}

// 16 bytes of shared memory of a CTA of the cluster.
__device__ __forceinline__ float4 load_cluster16(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// act(z) and the residual, or the factor, of its place.
template <bool kTimes>
__device__ __forceinline__ float with_res(float z, float r, const Epilogue& e) {
  return kTimes && e.times ? z * r : z + r;
}

// One warp's 32 rows x 32 columns of accumulators, a row a lane, from
// source(last, z) through the epilogue; the source is asked for the last time
// with last = true.
template <typename T, bool kTimes, typename F>
__device__ __forceinline__ void finish_rows(F source, const uint4 (&res)[4], const Epilogue& e, uint8_t* stage,
                                            const uint4* bias, int row0, int col0, int m, int n) {
  const int lane = threadIdx.x & 31;
  float z[32];
  auto take = [&](bool last) {
    source(last, z);
    if (!kTimes && e.scale) {
      const float f = sums_scale(e);
#pragma unroll
      for (int i = 0; i < 32; ++i) z[i] *= f;
    }
    if (e.bias) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float b[8];
        unpack16<T>(bias[q], b);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[8 * q + i] += b[i];
      }
    }
  };
  if (e.pre) {
    take(false);
#pragma unroll
    for (int c = 0; c < 4; ++c) *stage_piece(stage, lane, c) = pack16<T>(z + 8 * c);
    __syncwarp();
    write_rows(stage, static_cast<T*>(e.pre), e.ldpre, row0, col0, m, n, (e.vec & 4) != 0);
    __syncwarp();
  }
  if (e.res) {
    stage_rows(res, stage, col0, n);
    __syncwarp();
  }
  take(true);
  activate_all(z, e.act);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint4* at = stage_piece(stage, lane, c);
    if (e.res) {
      float r[8];
      unpack16<T>(*at, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[8 * c + i] = with_res<kTimes>(z[8 * c + i], r[i], e);
    }
    *at = pack16<T>(z + 8 * c);
  }
  __syncwarp();
  write_rows(stage, static_cast<T*>(e.out), e.ldo, row0, col0, m, n, (e.vec & 8) != 0);
  __syncwarp();
}

// The join of a kernel for few rows: a cluster's CTAs hold the fp32 sums of 128
// rows of the wide operand and each token, [token][128], in shared memory; this
// CTA takes its share of the columns, kCols / split of them, every token, four
// columns of a token at a time.  kCols = 64: a gated layer's, the gate in the
// first 64 sums and up in the others.  kScaled: the sums have a scale (asked for
// here, 128 rows of 4096 -> 4096 take 13.9 us without one, 13.5 by a kernel of its own).
template <typename T, int kCols, bool kTimes, bool kScaled>
__device__ __forceinline__ void join_few(const uint8_t* smem, const Epilogue& e, int split, int rank, int j0, int i0,
                                         int rows, int n, int threads) {
  const int width = kCols / 4 / split;
  for (int at = threadIdx.x; at < rows * width; at += threads) {
    const int i = at / width, jj = (rank * width + at % width) * 4, j = j0 + jj, left = n - j;
    if (left <= 0) continue;
    const float* mine = reinterpret_cast<const float*>(smem) + i * 128 + jj;
    auto joined = [&](const float* at, float(&z)[4]) {
      for (int s0 = 0; s0 < split; s0 += 8) {
        float4 u[8];  // all loads before the first sum
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s0 + s < split) u[s] = load_cluster16(mapa_shared(at, s0 + s));
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s0 + s < split) {
            z[0] += u[s].x;
            z[1] += u[s].y;
            z[2] += u[s].z;
            z[3] += u[s].w;
          }
      }
    };
    float z[4] = {};
    joined(mine, z);
    const long long row = i0 + i;
    float v[4];
    if constexpr (kCols == 64) {
      float u[4] = {};
      joined(mine + 64, u);
      if (e.bias) {
        load4(static_cast<const T*>(e.bias) + j, left, e.vec & 1, v);
#pragma unroll
        for (int q = 0; q < 4; ++q) z[q] += v[q];
        load4(static_cast<const T*>(e.bias) + n + j, left, (e.vec & 16) != 0, v);
#pragma unroll
        for (int q = 0; q < 4; ++q) u[q] += v[q];
      }
      if (e.pre) {
        store4(static_cast<T*>(e.pre) + row * e.ldpre + j, z, left, (e.vec & 4) != 0);
        store4(static_cast<T*>(e.pre) + row * e.ldpre + n + j, u, left, (e.vec & 32) != 0);
      }
      activate_all(z, e.act);
#pragma unroll
      for (int q = 0; q < 4; ++q) z[q] *= u[q];
      store4(static_cast<T*>(e.out) + row * e.ldo + j, z, left, (e.vec & 8) != 0);
      continue;
    }
    if constexpr (kScaled) {
      const float f = sums_scale(e);
#pragma unroll
      for (int q = 0; q < 4; ++q) z[q] *= f;
    }
    if (e.bias) {
      load4(static_cast<const T*>(e.bias) + j, left, e.vec & 1, v);
#pragma unroll
      for (int q = 0; q < 4; ++q) z[q] += v[q];
    }
    if (e.pre) store4(static_cast<T*>(e.pre) + row * e.ldpre + j, z, left, (e.vec & 4) != 0);
    activate_all(z, e.act);
    if (e.res) {
      load4(static_cast<const T*>(e.res) + row * e.ldr + j, left, (e.vec & 2) != 0, v);
#pragma unroll
      for (int q = 0; q < 4; ++q) z[q] = with_res<kTimes>(z[q], v[q], e);
    }
    store4(static_cast<T*>(e.out) + row * e.ldo + j, z, left, (e.vec & 8) != 0);
  }
}

// ------------------------------------------------------------------- host

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

int pad8(int x) { return (x + 7) & ~7; }

bool rows_aligned(const void* p, long long ld, int rows) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows <= 1 || (ld & 7) == 0);
}

constexpr int kMaxDev = 64;

}  // namespace

}  // namespace ozemu
