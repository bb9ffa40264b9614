// Microscaled 4-bit matrices (MXFP4) and their product.
//
//   s = 2^max(floor(log2 max|x|) - 2, -127) over 32 consecutive columns,
//   q = x / s rounded to e2m1 (half to even, 6 beyond),  x ~ s q
//   y = act(x w^T + b) + r  or  act(x w^T + b) r  of two such matrices
//
// Every step of the quantisation is exact but the one rounding: s is a power of
// two, so x / s is, and the conversion instruction rounds it.  The product runs
// on tcgen05 kind::mxf4, whose operands are the codes and whose scales are the
// bytes as they lie in memory, with fp32 accumulators in TMEM.
//
// A matrix of `rows` x k:
//   codes   [rows][ceil(k / 32) * 16] bytes, element j of a row in byte j / 2,
//           the low half for even j; 0 past column k
//   scales  [ceil(rows / 128)][ceil(k / 256)][1024] bytes: of 128 rows and 256
//           columns, the exponent byte (127 + log2 s) of row r and columns
//           32 b .. 32 b + 31 at (b / 4) 512 + (r % 32) 16 + (r / 32) 4 + b % 4;
//           127 past the last row or column.  512 bytes are what one tcgen05.cp
//           brings to TMEM as the MMA reads them (32 lanes of 16 bytes), so a
//           stage's scales are one contiguous copy.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <mutex>

#include "kernels.h"
#include "product.cuh"

namespace ozemu {

namespace {

constexpr int kTileRows = 128, kTileCols = 256;  // of a 1024-byte tile of scales

// Eight consecutive elements of a row, raw: one or two 16-byte vectors.
template <typename T>
struct Eight {
  static constexpr int kVectors = sizeof(T) / 2;
  uint4 u[kVectors];
  __device__ __forceinline__ void unpack(float2 (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < kVectors; ++i) unpack16<T>(u[i], v + 4 / kVectors * i);
  }
};

// Eight values already divided by their scale to eight codes, the first lowest.
__device__ __forceinline__ uint32_t to_codes(const float2 (&v)[4]) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(r)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
  return r;
}

// The values of eight codes.
__device__ __forceinline__ void from_codes(uint32_t w, float2 (&v)[4]) {
  uint32_t h[4];
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = Pair<__half>::unpack(h[i]);
}

// Place of the scale of a tile's row r and 32-column block b.
__device__ __forceinline__ int scale_at(int r, int b) { return (b >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (b & 3); }

// A CTA's tile, or quarter of one.
struct TilePart {
  int tile, kt, quarter;
  int r0, rows;  // the first row, and how many exist
  __device__ __forceinline__ TilePart(int ktiles, int quarters, int all) {
    tile = quarters ? blockIdx.x >> 2 : blockIdx.x;
    quarter = quarters ? blockIdx.x & 3 : 0;
    kt = tile % ktiles;
    r0 = tile / ktiles * kTileRows + quarter * 32;
    rows = min(quarters ? 32 : kTileRows, all - r0);
  }
};

// One CTA to a tile of scales, 128 rows of 256 columns, or, where those are few
// (1021 x 5003 fp32 has 160 of them: 12.8 us, by quarters 5.6), to a quarter of
// one, the 32 rows of one byte column of its words.  A warp takes a row, a
// lane eight columns of it, four lanes a block; the next rows of a warp (64
// bytes a lane) are on their way while it works on as many.  kVec: rows start on
// 16-byte boundaries; else their elements come one by one, a warp's side by side,
// and pass through shared memory to the lanes that take eight.  A block with an
// infinity or a NaN takes the scale NaN (255).  Bound by HBM: 16384 x 8192 bf16, 268
// MB in and 71 out, 55 us, 6.2 TB/s (93 without rows ahead).
template <typename T, bool kVec>
__global__ void __launch_bounds__(256, 4) mx_quantize_kernel(const T* x, long long ldx, int rows, int k, uint8_t* codes,
                                                             uint8_t* scales, int ktiles, int quarters) {
  constexpr int kRows = 4 / Eight<T>::kVectors;  // of a warp at a time
  __shared__ uint4 tile[64];
  __shared__ uint4 through[kVec ? 1 : 8 * 128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < 64) tile[threadIdx.x] = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
  chain_next();
  chain_wait();
  __syncthreads();
  const TilePart part(ktiles, quarters, rows);
  const int kt = part.kt, r0 = part.r0, here = part.rows;
  const int col = kt * kTileCols + lane * 8, left = k - col;
  const long long row_bytes = (k + 31LL) / 32 * 16;
  const bool stored = col < (k + 31) / 32 * 32;
  const T* from = x + static_cast<long long>(r0) * ldx;

  auto load = [&](Eight<T>(&e)[kRows], int i0) {
    if constexpr (kVec) {
#pragma unroll
      for (int q = 0; q < kRows; ++q) {
        const int r = i0 + 8 * q;
        const T* p = from + r * ldx + col;
#pragma unroll
        for (int i = 0; i < Eight<T>::kVectors; ++i) {
          const int exist = left - i * static_cast<int>(16 / sizeof(T));
          e[q].u[i] = make_uint4(0, 0, 0, 0);
          if (r < here && exist >= static_cast<int>(16 / sizeof(T))) {
            e[q].u[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
          } else if (r < here && exist > 0) {
            T* at = reinterpret_cast<T*>(&e[q].u[i]);
#pragma unroll
            for (int c = 0; c < static_cast<int>(16 / sizeof(T)); ++c)
              if (c < exist) at[c] = p[i * (16 / sizeof(T)) + c];
          }
        }
      }
    } else {
      T one[kRows][8];
#pragma unroll
      for (int q = 0; q < kRows; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i0 + 8 * q, c = kt * kTileCols + 32 * i + lane;
          one[q][i] = r < here && c < k ? from[r * ldx + c] : from_float<T>(0.f);
        }
      uint4* mine = through + warp * 128;
      __syncwarp();
#pragma unroll
      for (int q = 0; q < kRows; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) reinterpret_cast<T*>(mine + q * 32 * Eight<T>::kVectors)[32 * i + lane] = one[q][i];
      __syncwarp();
#pragma unroll
      for (int q = 0; q < kRows; ++q)
#pragma unroll
        for (int i = 0; i < Eight<T>::kVectors; ++i) e[q].u[i] = mine[(q * 32 + lane) * Eight<T>::kVectors + i];
    }
  };
  auto finish = [&](const Eight<T>& e, int r) {
    float2 v[4];
    e.unpack(v);
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      most = max(most, max(__float_as_uint(v[i].x) & 0x7FFFFFFFu, __float_as_uint(v[i].y) & 0x7FFFFFFFu));
    most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
    most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
    const int exponent = static_cast<int>(most >> 23), byte = exponent == 255 ? 255 : max(exponent - 2, 0);
    const float2 inverse = both(__uint_as_float(static_cast<uint32_t>(254 - byte) << 23));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], inverse);
    const uint32_t w = byte == 255 ? 0 : to_codes(v);
    if (r < here && stored) {
      *reinterpret_cast<uint32_t*>(codes + (r0 + r) * row_bytes + col / 2) = w;
      if ((lane & 3) == 0) reinterpret_cast<uint8_t*>(tile)[scale_at(r, lane >> 2)] = static_cast<uint8_t>(byte);
    }
  };

  Eight<T> next[kRows];
  load(next, warp);
#pragma unroll 1
  for (int i0 = warp; i0 < here; i0 += 8 * kRows) {
    Eight<T> now[kRows];
#pragma unroll
    for (int q = 0; q < kRows; ++q) now[q] = next[q];
    if (i0 + 8 * kRows < here) load(next, i0 + 8 * kRows);
#pragma unroll
    for (int q = 0; q < kRows; ++q) finish(now[q], i0 + 8 * q);
  }
  __syncthreads();
  if (threadIdx.x >= 64) return;
  uint4* to = reinterpret_cast<uint4*>(scales + part.tile * 1024LL) + threadIdx.x;
  if (quarters)  // rows r of the quarter stood where a whole tile's first 32 rows do
    reinterpret_cast<uint32_t*>(to)[part.quarter] = tile[threadIdx.x].x;
  else
    *to = tile[threadIdx.x];
}

// The values that codes and scales stand for: the same tiles and lanes, and
// through shared memory where rows start on no 16-byte boundaries.  16384 x 8192
// bf16, 71 MB in and 268 out, 54 us.
template <typename T, bool kVec>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const uint8_t* codes, const uint8_t* scales, int ktiles,
                                                            int quarters, T* y, long long ldy, int rows, int k) {
  __shared__ uint4 through[kVec ? 1 : 8 * 4 * 32 * Eight<T>::kVectors];
  chain_next();
  chain_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const TilePart part(ktiles, quarters, rows);
  const int kt = part.kt, r0 = part.r0, here = part.rows;
  const int col = kt * kTileCols + lane * 8, left = k - col;
  const long long row_bytes = (k + 31LL) / 32 * 16;
  const uint8_t* tile = scales + part.tile * 1024LL + part.quarter * 4;  // (a quarter's rows count from 0)
#pragma unroll 1
  for (int i0 = warp; i0 < here; i0 += 32) {
    uint32_t w[4], byte[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = i0 + 8 * q;
      w[q] = byte[q] = 0;
      if (r < here && left > 0) {
        w[q] = __ldg(reinterpret_cast<const uint32_t*>(codes + (r0 + r) * row_bytes + col / 2));
        byte[q] = __ldg(tile + scale_at(r, lane >> 2));
      }
    }
    uint4* mine = through + warp * 4 * 32 * Eight<T>::kVectors;
    if constexpr (!kVec) __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = i0 + 8 * q;
      const float s = __uint_as_float(byte[q] == 255 ? 0x7FC00000u : byte[q] == 0 ? 0x00400000u : byte[q] << 23);
      float2 v[4];
      from_codes(w[q], v);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = mul2(v[i], both(s));
      T* p = y + static_cast<long long>(r0 + r) * ldy + col;
#pragma unroll
      for (int i = 0; i < Eight<T>::kVectors; ++i) {
        const uint4 u = pack16<T>(v + 4 / Eight<T>::kVectors * i);
        const int exist = left - i * static_cast<int>(16 / sizeof(T));
        if constexpr (!kVec) {
          mine[(q * 32 + lane) * Eight<T>::kVectors + i] = u;
        } else if (r < here && exist >= static_cast<int>(16 / sizeof(T))) {
          reinterpret_cast<uint4*>(p)[i] = u;
        } else if (r < here && exist > 0) {
          const T* at = reinterpret_cast<const T*>(&u);
#pragma unroll
          for (int c = 0; c < static_cast<int>(16 / sizeof(T)); ++c)
            if (c < exist) p[i * (16 / sizeof(T)) + c] = at[c];
        }
      }
    }
    if constexpr (!kVec) {
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i0 + 8 * q, c = kt * kTileCols + 32 * i + lane;
          if (r < here && c < k)
            y[static_cast<long long>(r0 + r) * ldy + c] =
                reinterpret_cast<const T*>(mine + q * 32 * Eight<T>::kVectors)[32 * i + lane];
        }
    }
  }
}

// ---------------------------------------------------------------------------
// Large products: 256 x BN tiles on CTA pairs, BN = 256 or 128.
//
// As the pair kernel of linear.cu: each CTA of a cluster of two stages its 128
// rows of A and BN / 2 rows of B, 256 of the reduction (128 bytes) a stage,
// with the scales of its rows of A and of all the tile's rows of B; a warp loads
// A, one B, one brings the scales to TMEM and issues the MMAs (4 of K = 64 a
// stage), and sixteen take finished accumulators out.  Scales take 24 columns a
// stage, two stages in turn.  That leaves 448 columns for accumulators: two of
// 256 that share 64, the end of one and the start of the other.  The epilogue
// takes the half with the shared columns first, and the next tile's MMAs start
// once that half is in registers.
//
// Bound by shared memory (operands in and out), 560 clocks a stage against the
// MMAs' 512, by the wait between a tile's last MMA and the next one's first (14 us
// at 16 stages a tile, when the whole took 186) and by the outputs' way out: 8192 x
// 4096 -> 16384 bf16 160 us (6.9 PFLOP/s), with gelu_tanh 170, with a residual 186;
// 8192 x 256 -> 8192 31, 45 and 76; 8192 x 16384 -> 4096 144 (7.6),
// in a short burst; a second of the first runs at 180, the power cap's clocks.
// ---------------------------------------------------------------------------
constexpr int kMxThreads = 32 * (3 + kEpiWarps);
constexpr int kCodes = 128 * 128;                        // bytes of 128 rows of 256 codes
constexpr int kMxStage = 2 * kCodes + 3 * 1024;          // A, B, scales of A's 128 rows and of B's 256
constexpr int kMxStages = 5;
constexpr int kMxSmem = 1024 + kMxStages * kMxStage + kEpiWarps * (2048 + 64) + 256;
constexpr uint32_t kScaleColumns = 448, kScaleTurn = 32;
constexpr uint32_t kSecondAccumulator = 192;  // of two of 256 columns

struct MxProduct {
  int m, n, kt;  // kt: 256-element stages of the reduction
  int bn;
  Raster tiles;
  Epilogue e;
};

template <int kGroup>
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                       uint32_t accumulate) {
  if constexpr (kGroup == 2)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}

// 512 bytes of scales (32 lanes of 16 bytes, no swizzle) to four columns of
// TMEM, the same for each of its four lane quarters.
template <int kGroup>
__device__ __forceinline__ void copy_scales(uint32_t columns, uint32_t saddr) {
  const uint64_t desc = ((saddr & 0x3FFFFu) >> 4) | (1u << 16) | (static_cast<uint64_t>((128u >> 4) | (1u << 14)) << 32);
  if constexpr (kGroup == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(columns), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(columns), "l"(desc) : "memory");
}

// Instruction descriptor: e2m1 operands, K-major, exponent-byte scales, of which
// a 32-bit word of TMEM holds four for a row: this MMA takes those of byte
// 2 half and the next.
__device__ __forceinline__ uint32_t idesc_mx(int m, int n, int half) {
  return (static_cast<uint32_t>(2 * half) << 4)    // B's scales
         | (1u << 7)                               // A format: e2m1
         | (1u << 10)                              // B format: e2m1
         | (static_cast<uint32_t>(n >> 3) << 17)   // N / 8
         | (1u << 23)                              // scale type: exponent byte
         | (static_cast<uint32_t>(m >> 7) << 27)   // M / 128
         | (static_cast<uint32_t>(2 * half) << 29);  // A's scales
}

// The copies and MMAs of one stage: codes at a and b, scales of A's 128 rows and
// of B's (b_tiles tiles of 128 rows) to 8 + 8 b_tiles columns of TMEM.
template <int kGroup>
__device__ __forceinline__ void stage_mmas(uint32_t d, uint32_t a, uint32_t b, uint32_t scales_a, uint32_t scales_b,
                                           int b_tiles, uint32_t columns, int m, int n, bool first) {
  const uint32_t sa = columns, sb = columns + 8, b_step = 4 * b_tiles;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    copy_scales<kGroup>(sa + 4 * q, scales_a + 512 * q);
    copy_scales<kGroup>(sb + b_step * q, scales_b + 512 * q);
    if (b_tiles > 1) copy_scales<kGroup>(sb + b_step * q + 4, scales_b + 1024 + 512 * q);
  }
  const uint32_t a_lo = smem_desc_sw128_lo(a, false), b_lo = smem_desc_sw128_lo(b, false);
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
    mma_mx<kGroup>(d, smem_desc_sw128(a_lo + 2 * ks), smem_desc_sw128(b_lo + 2 * ks), idesc_mx(m, n, ks & 1),
                   sa + 4 * (ks >> 1), sb + b_step * (ks >> 1), first && ks == 0 ? 0u : 1u);
}

// 32 bytes of global memory.
__device__ __forceinline__ void load32(const void* p, uint32_t (&v)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "l"(p)
               : "memory");
}
// Without a place in L1, which nothing reads it from again: 8192 x 4096 -> 16384
// 180 us -> 171, before other steps.
__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// A warp's 32 rows x 32 columns of accumulators, a row a lane, where rows start
// on 16-byte boundaries: straight from registers in pieces of 32 bytes, or of 16
// where some row starts on no 32-byte boundary.  (The MMAs and the copies that
// feed them take all of shared memory's bandwidth, 67 KB in the 512 clocks of a
// stage; without the outputs' way through it 8192 x 4096 -> 16384 went from 186 to
// 180 us, before other steps.)
template <typename T>
__device__ __forceinline__ void finish_direct(const uint32_t (&u)[32], const Epilogue& e, const uint4* bias,
                                              long long row, int col0, int m) {
  if (row >= m) return;
  float2 z[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
  if (e.bias) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float2 b[4];
      unpack16<T>(bias[q], b);
#pragma unroll
      for (int i = 0; i < 4; ++i) z[4 * q + i] = add2(z[4 * q + i], b[i]);
    }
  }
  activate_all(z, e.act);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    alignas(16) uint32_t w[8];
    if (e.res) {
      const T* p = static_cast<const T*>(e.res) + row * e.ldr + col0 + 16 * h;
      if (e.vec & 16) {
        load32(p, w);
      } else {
        *reinterpret_cast<uint4*>(w) = reinterpret_cast<const uint4*>(p)[0];
        *reinterpret_cast<uint4*>(w + 4) = reinterpret_cast<const uint4*>(p)[1];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 r = Pair<T>::unpack(w[i]);
        z[8 * h + i] = e.times ? mul2(z[8 * h + i], r) : add2(z[8 * h + i], r);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = Pair<T>::pack(z[8 * h + i].x, z[8 * h + i].y);
    T* to = static_cast<T*>(e.out) + row * e.ldo + col0 + 16 * h;
    if (e.vec & 16) {
      store32(to, w);
    } else {
      reinterpret_cast<uint4*>(to)[0] = *reinterpret_cast<const uint4*>(w);
      reinterpret_cast<uint4*>(to)[1] = *reinterpret_cast<const uint4*>(w + 4);
    }
  }
}

// The same where the output's rows start on no 16-byte boundaries, from source(z),
// by a quarter's warps together (`some`: whether this one's columns exist).
template <typename T, typename F>
__device__ __forceinline__ void finish_together(F source, bool some, const uint4 (&res)[4], const Epilogue& e,
                                                uint8_t* stage, const uint4* bias, const Quarter& q, int row0, int col0,
                                                int m, int n) {
  const int lane = threadIdx.x & 31;
  if (some && e.res) {
    stage_rows(res, stage, col0, n);
    __syncwarp();
  }
  float2 z[16];
  source(z);
  if (some) {
    if (e.bias) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float2 b[4];
        unpack16<T>(bias[k], b);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[4 * k + i] = add2(z[4 * k + i], b[i]);
      }
    }
    activate_all(z, e.act);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint4* at = stage_piece(stage, lane, c);
      if (e.res) {
        float2 r[4];
        unpack16<T>(*at, r);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          z[4 * c + i] = e.times ? mul2(z[4 * c + i], r[i]) : add2(z[4 * c + i], r[i]);
      }
      *at = pack16<T>(z + 4 * c);
    }
  }
  quarter_sync(q);
  write_together(q, static_cast<T*>(e.out), e.ldo, row0, col0 - 32 * q.group, m, n);
  quarter_sync(q);
}

template <typename T>
__global__ void __launch_bounds__(kMxThreads, 1)
    mx_pair_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                   const __grid_constant__ CUtensorMap msa, const __grid_constant__ CUtensorMap msb,
                   const __grid_constant__ MxProduct p, uint32_t* flags) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + kMxStages * kMxStage;
  uint8_t* biases = staging + kEpiWarps * 2048;
  uint64_t* full = reinterpret_cast<uint64_t*>(biases + kEpiWarps * 64);
  uint64_t* empty = full + kMxStages;
  uint64_t* tfull = empty + kMxStages;
  uint64_t* taken = tfull + 2;
  uint64_t* mma_done = taken + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_word = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1, total = p.tiles.count();
  const bool wide = p.bn == 256;
  const uint32_t second = wide ? kSecondAccumulator : 128;

  cluster_arrive();
  if (warp == 0 && lane == 0) {
    for (int s = 0; s < kMxStages; ++s) {
      mbar_init(&full[s], 1);   // armed by the first CTA with both CTAs' bytes
      mbar_init(&empty[s], 1);  // one commit from the pair's MMA issuer
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&taken[b], 2 * kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *abort_word = 0;
    fence_mbar_init();
    tma_prefetch_desc(&ma);
    tma_prefetch_desc(&mb);
    tma_prefetch_desc(&msa);
    tma_prefetch_desc(&msb);
  }
  __syncwarp();
  cluster_wait();  // both CTAs run
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  chain_next();
  chain_wait();

  if (warp == 0 || warp == 2 + kEpiWarps) {
    const bool loads_a = warp == 0;
    const uint32_t bar0 = mapa_shared(&full[0], 0);
    const uint32_t bytes = 2 * (kCodes + p.bn / 2 * 128 + 1024 + p.bn / 128 * 1024);  // of both CTAs
    int s = 0;
    uint32_t phase = 1;
    bool ok = true;
    for (int t = pair; t < total && ok; t += npairs) {
      int tm, tn;
      tile_of(t, p.tiles, tm, tn);
      const int at = loads_a ? tm * 256 + rank * 128 : tn * p.bn + rank * (p.bn / 2);
      const int block = loads_a ? tm * 2 + rank : tn * p.bn / 128;  // of 128 rows, the scales'
      for (int kt = 0; kt < p.kt; ++kt) {
        if (!all_wait(&empty[s], phase, abort_word, flags)) {
          ok = false;
          break;
        }
        uint8_t* st = smem + s * kMxStage;
        const uint32_t bar = bar0 + s * 8;
        if (elect_one()) {
          if (loads_a) {
            if (rank == 0) mbar_arrive_expect_tx_relaxed(&full[s], bytes);
            tma_load_2d_pair(st, &ma, bar, kt * 128, at);
            tma_load_2d_pair(st + 2 * kCodes, &msa, bar, kt * 256, block);
          } else {
            tma_load_2d_pair(st + kCodes, &mb, bar, kt * 128, at);
            tma_load_2d_pair(st + 2 * kCodes + 1024, &msb, bar, kt * 256, block);
            if (wide) tma_load_2d_pair(st + 2 * kCodes + 2048, &msb, bar, kt * 256, block + 1);
          }
        }
        __syncwarp();
        if (++s == kMxStages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) settle_after_abort();
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      int s = 0, n_tiles = 0, turn = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = pair; t < total && ok; t += npairs, ++n_tiles) {
        const int buf = n_tiles & 1;
        // Its columns are free: of two wide accumulators, once the tile before
        // has left the shared ones, else once the tile before that has.
        const int before = n_tiles - (wide ? 1 : 2);
        if (before >= 0 && !all_wait(&taken[before & 1], (before >> 1) & 1, abort_word, flags)) break;
        tc_fence_after();
        const uint32_t d = tbase + (buf ? second : 0);
        for (int kt = 0; kt < p.kt; ++kt, turn ^= 1) {
          if (!all_wait(&full[s], phase, abort_word, flags)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_u32(smem) + s * kMxStage;
          if (elect_one()) {
            stage_mmas<2>(d, st, st + kCodes, st + 2 * kCodes, st + 2 * kCodes + 1024, p.bn / 128,
                          tbase + kScaleColumns + turn * kScaleTurn, 256, p.bn, kt == 0);
            tc_commit_pair_multicast(&empty[s], 0x3);
          }
          __syncwarp();
          if (++s == kMxStages) {
            s = 0;
            phase ^= 1;
          }
        }
        if (ok && elect_one()) tc_commit_pair_multicast(&tfull[buf], 0x3);
        __syncwarp();
      }
      if (elect_one()) {
        tc_commit_pair_multicast(mma_done, 0x1);
        drain_wait(mma_done, 0, flags);
        if (!ok) settle_after_abort();
      }
    }
    __syncwarp();
  } else {
    const int ew = warp - 2, quarter = warp & 3, group = ew >> 2;
    uint8_t *stage = staging + ew * 2048, *bias = biases + ew * 64;
    const Epilogue& e = p.e;
    const bool rows16 = (e.vec & 8) && (!e.res || (e.vec & 2)), together = (e.vec & 8) == 0;
    const Quarter q = {staging + (ew & 3) * 2048, quarter, group};
    int n_tiles = 0;
    bool live = true;
    for (int t = pair; t < total && live; t += npairs, ++n_tiles) {
      int tm, tn;
      tile_of(t, p.tiles, tm, tn);
      const int buf = n_tiles & 1, use = n_tiles >> 1;
      const int row0 = tm * 256 + rank * 128 + quarter * 32;
      const int cols = row0 < p.m ? min(p.bn, p.n - tn * p.bn) : 0;
      const uint32_t tcol = tbase + (static_cast<uint32_t>(quarter * 32) << 16) + (buf ? second : 0);
      // The half with the shared columns (the upper one of the first
      // accumulator), then the other; what is left of this is nothing to take.
      const int first = wide && !buf ? 128 : 0;
      bool waited = false;
#pragma unroll 1
      for (int h = 0; h < p.bn; h += 128) {
        const int c = (first ^ h) + group * 32;
        const int col0 = tn * p.bn + c;
        const bool direct = rows16 && c + 32 <= cols;
        uint4 res[4];
        if (c < cols) {
          if (e.res && !direct)
            read_rows(res, static_cast<const T*>(e.res), e.ldr, row0, col0, p.m, p.n, (e.vec & 2) != 0);
          if (e.bias) {  // the chunk's 32 values, for every lane
            const uint16_t b = col0 + lane < p.n ? static_cast<const uint16_t*>(e.bias)[col0 + lane] : 0;
            __syncwarp();
            reinterpret_cast<uint16_t*>(bias)[lane] = b;
            __syncwarp();
          }
        }
        if (!waited) {
          live = warp_wait(&tfull[buf], use & 1, abort_word, flags);
          if (together) live = quarter_all(q, live);
          if (!live) break;
          tc_fence_after();
          waited = true;
        }
        // The warp's sums of this half are in registers: of the first half (of BN =
        // 128 the whole tile) the MMAs wait for that.
        auto release = [&] {
          if (h != 0) return;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(&taken[buf], 0));
        };
        uint32_t u[32];
        if (direct) {
          tmem_ld32(tcol + c, u);
          tmem_wait_ld();
          release();
          finish_direct<T>(u, e, reinterpret_cast<const uint4*>(bias), row0 + lane, col0, p.m);
          __syncwarp();  // lanes past the last row are back for the next read of TMEM, a warp's
        } else if (together && (first ^ h) < cols) {
          finish_together<T>(
              [&](float2(&z)[16]) {
                tmem_ld32(tcol + c, u);
                tmem_wait_ld();
                release();
#pragma unroll
                for (int i = 0; i < 16; ++i) z[i] = make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
              },
              c < cols, res, e, stage, reinterpret_cast<const uint4*>(bias), q, row0, col0, p.m, p.n);
        } else if (c < cols) {
          finish_rows<T, true>(
              [&](bool, float(&z)[32]) {
                tmem_ld32(tcol + c, u);
                tmem_wait_ld();
                release();
#pragma unroll
                for (int i = 0; i < 32; ++i) z[i] = __uint_as_float(u[i]);
              },
              res, e, stage, reinterpret_cast<const uint4*>(bias), row0, col0, p.m, p.n);
        } else {
          release();
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's MMAs, commits and remote signals are all done
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, 512);
  }
}

// ---------------------------------------------------------------------------
// Few rows (tokens being decoded): the weights are all the traffic.
//
// As the kernel for few rows of linear.cu: the weights take the MMA's 128 rows,
// the tokens its N = NT columns, a cluster of up to 16 CTAs shares the
// reduction of 128 columns of D, and joins its fp32 sums in rank order.  Bound by
// HBM and the start and end of a launch: 1 x 4096 -> 16384, 35.7 MB, 8.4 us from
// HBM, 6.6 from L2.
// ---------------------------------------------------------------------------
template <int NT>
struct MxFewCfg {
  static constexpr int kStage = kCodes + NT * 128 + 2048;
  static constexpr int kStages = 108 * 1024 / kStage;
  static constexpr int kSmem = 1024 + kStages * kStage + 256;
  static constexpr int kScales = NT < 32 ? 32 : NT;        // columns of TMEM: NT sums, then 16 of scales a stage,
  static constexpr int kTmemCols = kScales < 64 ? 64 : 2 * NT;  // two stages in turn; a power of two
  static_assert(kScales + 32 <= kTmemCols, "");
  static_assert(NT * 512 <= kStages * kStage, "the partial sums take the ring's memory");
  static_assert(kStage % 1024 == 0, "tiles on the swizzle's boundaries");
};
constexpr int kMxFewThreads = 192;

struct MxFewProduct {
  int m, n, kt, split;
  const uint8_t *wscales, *xscales;
  Epilogue e;
};

template <typename T, int NT>
__global__ void __launch_bounds__(kMxFewThreads, 2)
    mx_few_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                  const __grid_constant__ MxFewProduct p, uint32_t* flags) {
  using C = MxFewCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStage);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(tfull + 1);
  volatile int* abort_word = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int block = blockIdx.x / p.split, j0 = block * 128, i0 = blockIdx.y * NT;
  const int per = (p.kt + p.split - 1) / p.split;
  const int kt0 = min(rank * per, p.kt), kt1 = min(kt0 + per, p.kt);

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    *abort_word = 0;
    fence_mbar_init();
    tma_prefetch_desc(&mw);
    tma_prefetch_desc(&mx);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  chain_next();
  chain_wait();

  if (warp == 0) {
    int s = 0;
    uint32_t phase = 1;
    bool ok = true;
    for (int kt = kt0; kt < kt1; ++kt) {
      if (!all_wait(&empty[s], phase, abort_word, flags)) {
        ok = false;
        break;
      }
      uint8_t* st = smem + s * C::kStage;
      if (elect_one()) {
        mbar_arrive_expect_tx_relaxed(&full[s], C::kStage);
        tma_load_2d(st, &mw, &full[s], kt * 128, j0);
        tma_load_2d(st + kCodes, &mx, &full[s], kt * 128, i0);
        bulk_load(st + kCodes + NT * 128, p.wscales + (static_cast<long long>(block) * p.kt + kt) * 1024, 1024, &full[s]);
        bulk_load(st + kCodes + NT * 128 + 1024, p.xscales + (static_cast<long long>(i0 / 128) * p.kt + kt) * 1024, 1024,
                  &full[s]);
      }
      __syncwarp();
      if (++s == C::kStages) {
        s = 0;
        phase ^= 1;
      }
    }
    if (!ok) settle_after_abort();
    __syncwarp();
  } else if (warp == 1) {
    int s = 0, turn = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int kt = kt0; kt < kt1; ++kt, turn ^= 1) {
      if (!all_wait(&full[s], phase, abort_word, flags)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t st = smem_u32(smem) + s * C::kStage;
      if (elect_one()) {
        stage_mmas<1>(tbase, st, st + kCodes, st + kCodes + NT * 128, st + kCodes + NT * 128 + 1024, 1,
                      tbase + C::kScales + turn * 16, 128, NT, kt == kt0);
        tc_commit(&empty[s]);
      }
      __syncwarp();
      if (++s == C::kStages) {
        s = 0;
        phase ^= 1;
      }
    }
    if (elect_one()) {
      tc_commit(tfull);  // also when giving up: the MMAs issued are waited for below
      if (!ok) settle_after_abort();
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3;
    float* part = reinterpret_cast<float*>(smem);
    if (kt0 == kt1) {
      for (int i = 0; i < NT; ++i) part[i * 128 + quarter * 32 + lane] = 0.f;
    } else if (warp_wait(tfull, 0, abort_word, flags)) {
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < NT; i += 16) {
        uint32_t v[16];
        tmem_ld16(tbase + (static_cast<uint32_t>(quarter * 32) << 16) + i, v);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 16; ++q) part[(i + q) * 128 + quarter * 32 + lane] = __uint_as_float(v[q]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  join_few<T, 128, true, false>(smem, p.e, p.split, rank, j0, i0, min(NT, p.m - i0), p.n, kMxFewThreads);
  cluster_sync();  // peers have read this CTA's sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, C::kTmemCols);
  }
}

// ------------------------------------------------------------------- host

long long row_bytes(int k) { return (k + 31LL) / 32 * 16; }
int k_tiles(int k) { return static_cast<int>((k + 255LL) / 256); }

bool code_map(CUtensorMap* map, const void* codes, int rows, int k, int box) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(row_bytes(k)), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes(k))};
  const cuuint32_t shape[2] = {128, static_cast<cuuint32_t>(box)}, ones[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, shape, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Tiles of scales, 256 words each (past the last one: zeros, which stand for
// 2^-127 and meet codes of 0 only).
bool scale_map(CUtensorMap* map, const void* scales, int rows, int k) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k_tiles(k)) * 256, static_cast<cuuint64_t>((rows + 127) / 128)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(k_tiles(k)) * 1024};
  const cuuint32_t shape[2] = {256, 1}, ones[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(scales), dims, strides, shape, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs of a pass over a matrix: its tiles, or their quarters where those do not
// give every SM four (bf16, us, quantised and read back, whole / quarters: 1024 x
// 4096 6.8 + 4.9 / 3.5 + 3.8, 4096 x 4096 9.3 + 10.9 / 9.0 + 7.5, 8192 x 4096 15.0 +
// 15.1 / 17.3 + 13.9, 16384 x 8192 55.6 + 53.3 / 70.2 + 54.9).
long long tile_ctas(int rows, int k, int* quarters) {
  const long long tiles = static_cast<long long>((rows + 127) / 128) * k_tiles(k);
  *quarters = tiles < 152 * 4;
  return *quarters ? 4 * tiles : tiles;
}

template <typename T>
cudaError_t quantize_t(const MxQuantCall& c, cudaStream_t stream) {
  int quarters;
  const long long ctas = tile_ctas(c.rows, c.k, &quarters);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  const bool vec = rows_aligned(c.x, c.ldx * static_cast<long long>(sizeof(T)) / 2, c.rows);
  return launch_chained(vec ? mx_quantize_kernel<T, true> : mx_quantize_kernel<T, false>,
                        dim3(static_cast<unsigned>(ctas)), 256, 0, stream, 0, static_cast<const T*>(c.x), c.ldx, c.rows,
                        c.k, c.codes, c.scales, k_tiles(c.k), quarters);
}

template <typename T>
cudaError_t dequantize_t(const MxDequantCall& c, cudaStream_t stream) {
  int quarters;
  const long long ctas = tile_ctas(c.rows, c.k, &quarters);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  const bool vec = rows_aligned(c.y, c.ldy * static_cast<long long>(sizeof(T)) / 2, c.rows);
  return launch_chained(vec ? mx_dequantize_kernel<T, true> : mx_dequantize_kernel<T, false>,
                        dim3(static_cast<unsigned>(ctas)), 256, 0, stream, 0, c.codes, c.scales, k_tiles(c.k),
                        quarters, static_cast<T*>(c.y), c.ldy, c.rows, c.k);
}

// CTA pairs that are resident at once (a persistent grid must not exceed
// them); sets the kernel's shared-memory size on the way.
template <typename T>
cudaError_t resident_pairs(int* out) {
  static int known[kMaxDev];
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (known[dev] == 0) {
    auto kern = mx_pair_kernel<T>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMxSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(kMxThreads, 1, 1);
    cfg.dynamicSmemBytes = kMxSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    known[dev] = n;
  }
  *out = known[dev];
  return cudaSuccess;
}

template <typename T, int NT>
cudaError_t launch_mx_few(const MxLinearCall& c, const Epilogue& e, cudaStream_t stream) {
  CUtensorMap mw, mx;
  if (!code_map(&mw, c.wcodes, c.n, c.k, 128) || !code_map(&mx, c.xcodes, c.m, c.k, NT)) return cudaErrorInvalidValue;
  auto kern = mx_few_kernel<T, NT>;
  static std::atomic<bool> ready[kMaxDev];
  int dev = 0;
  cudaError_t s = cudaGetDevice(&dev);
  if (s != cudaSuccess) return s;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    s = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, MxFewCfg<NT>::kSmem);
    if (s == cudaSuccess) s = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (s != cudaSuccess) return s;
    ready[dev] = true;
  }
  const int across = (c.n + 127) / 128, down = (c.m + NT - 1) / NT;
  MxFewProduct p = {c.m, c.n, k_tiles(c.k), 1, c.wscales, c.xscales, e};
  // Two CTAs on each SM, and at least two stages of the reduction for each.
  while (p.split < (NT > 32 ? 8 : 16) && 2LL * p.split * across * down <= 304 && p.kt >= 4 * p.split) p.split *= 2;
  return launch_chained(kern, dim3(across * p.split, down, 1), kMxFewThreads, MxFewCfg<NT>::kSmem, stream, p.split, mw,
                        mx, p, c.flags);
}

// The product of an empty reduction: act(bias), and the residual or factor.
template <typename T>
__global__ void __launch_bounds__(256) mx_empty_kernel(int m, int n, const Epilogue e) {
  chain_next();
  chain_wait();
  const long long all = static_cast<long long>(m) * n;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < all; i += gridDim.x * 256LL) {
    const long long row = i / n;
    const int col = static_cast<int>(i % n);
    float y = activate(e.bias ? to_float(static_cast<const T*>(e.bias)[col]) : 0.f, e.act);
    if (e.res) y = with_res<true>(y, to_float(static_cast<const T*>(e.res)[row * e.ldr + col]), e);
    static_cast<T*>(e.out)[row * e.ldo + col] = from_float<T>(y);
  }
}

// Whether the kernel for few rows takes a product.  The pairs' time is that of
// their stages, 0.26 us each, whatever the rows up to 256; this one's shares the
// stages over a cluster but grows with its rows.  Weights of 4096 rows from HBM,
// us, few rows / pairs: 32 rows of 1024 columns 5.7 / 4.5, of 2048 5.8 / 5.7, of
// 4096 6.6 / 8.0; 64 rows of 4096 8.4 / 8.1, of 8192 9.9 / 12.6; 128 rows of 4096
// 11.2 / 8.3, of 8192 13.0 / 12.9, of 16384 15.4 / 21.9.  Above 128 rows its 128 x
// 128 tiles have to leave SMs for a shared reduction (256 rows of 16384: 16.7 /
// 22.0).
bool few_rows(int m, int n, int kt) {
  if (m <= 16) return true;
  if (m <= 64) return kt >= (m <= 32 ? 8 : 17);
  const long long squares = static_cast<long long>((m + 127) / 128) * ((n + 127) / 128);
  return kt >= 32 && (m <= 128 || squares <= 76);
}

template <typename T>
cudaError_t mx_linear_t(const MxLinearCall& c, cudaStream_t stream) {
  Epilogue e = {c.bias, c.res, c.ldr, nullptr, 0, c.y, c.ldy, c.act, 0, c.times};
  e.vec = (e.bias && rows_aligned(e.bias, 0, 1) ? 1 : 0) | (e.res && rows_aligned(e.res, e.ldr, c.m) ? 2 : 0) |
          (rows_aligned(e.out, e.ldo, c.m) ? 8 : 0);
  // Rows of the output and the residual on 32-byte boundaries.
  const auto wide = [&](const void* p, long long ld) {
    return (reinterpret_cast<uintptr_t>(p) & 31u) == 0 && (c.m <= 1 || (ld & 15) == 0);
  };
  if (wide(e.out, e.ldo) && (!e.res || wide(e.res, e.ldr))) e.vec |= 16;
  if (c.k == 0) {
    const long long all = static_cast<long long>(c.m) * c.n;
    return launch_chained(mx_empty_kernel<T>, dim3(static_cast<unsigned>(std::min<long long>((all + 255) / 256, 4096))),
                          256, 0, stream, 0, c.m, c.n, e);
  }
  if (few_rows(c.m, c.n, k_tiles(c.k)))
    return c.m <= 16   ? launch_mx_few<T, 16>(c, e, stream)
           : c.m <= 32 ? launch_mx_few<T, 32>(c, e, stream)
           : c.m <= 64 ? launch_mx_few<T, 64>(c, e, stream)
                       : launch_mx_few<T, 128>(c, e, stream);
  int pairs = 0;
  const cudaError_t s = resident_pairs<T>(&pairs);
  if (s != cudaSuccess) return s;
  MxProduct p = {c.m, c.n, k_tiles(c.k), 256, {}, e};
  auto tiles = [&](int bn) { return static_cast<long long>((c.m + 255) / 256) * ((c.n + bn - 1) / bn); };
  // Narrow tiles where every one of them has a pair of its own (1024 x 4096 -> 2048:
  // 8.6 us, 9.0 by half as many wide ones); in two rounds they lose (1024 x 4096 ->
  // 4096: 13.8, 11.1 by one round of wide ones).
  if (tiles(128) <= pairs) p.bn = 128;
  p.tiles = raster((c.m + 255) / 256, (c.n + p.bn - 1) / p.bn);
  CUtensorMap ma, mb, msa, msb;
  if (!code_map(&ma, c.xcodes, c.m, c.k, 128) || !code_map(&mb, c.wcodes, c.n, c.k, p.bn / 2) ||
      !scale_map(&msa, c.xscales, c.m, c.k) || !scale_map(&msb, c.wscales, c.n, c.k))
    return cudaErrorInvalidValue;
  return launch_chained(mx_pair_kernel<T>, dim3(2 * static_cast<unsigned>(std::min<long long>(tiles(p.bn), pairs))),
                        kMxThreads, kMxSmem, stream, 2, ma, mb, msa, msb, p, c.flags);
}

}  // namespace

size_t mx_code_bytes(int rows, int k) { return static_cast<size_t>(rows) * row_bytes(k); }
size_t mx_scale_bytes(int rows, int k) { return static_cast<size_t>((rows + 127) / 128) * k_tiles(k) * 1024; }

cudaError_t launch_mx_quantize(const MxQuantCall& c, cudaStream_t stream) {
  return c.type == kF32   ? quantize_t<float>(c, stream)
         : c.type == kF16 ? quantize_t<__half>(c, stream)
                          : quantize_t<__nv_bfloat16>(c, stream);
}

cudaError_t launch_mx_dequantize(const MxDequantCall& c, cudaStream_t stream) {
  return c.type == kF32   ? dequantize_t<float>(c, stream)
         : c.type == kF16 ? dequantize_t<__half>(c, stream)
                          : dequantize_t<__nv_bfloat16>(c, stream);
}

cudaError_t launch_mx_linear(const MxLinearCall& c, cudaStream_t stream) {
  return c.type == kF16 ? mx_linear_t<__half>(c, stream) : mx_linear_t<__nv_bfloat16>(c, stream);
}

}  // namespace ozemu
