// Linear layer with a fused epilogue, and its gradients, on tcgen05 kind::f16.
//
//   z = x w^T + b,  y = act(z) + r
//   dz = dy act'(pre),  dx = dz w,  dw = dz^T x,  db = sum over rows of dz
//
// Each product D(i, j) = sum_p A(i, p) B(j, p) runs on bf16 or f16 operands
// with fp32 accumulators in TMEM.  The operands of the three products are the
// same three matrices, read with the reduction along a row (K-major: x and w
// in the forward product, dz in dx) or down the rows (MN-major: w in dx, dz
// and x in dw); TMA brings both in the same 64 x 64 blocks, and the matrix
// descriptors say which way the reduction runs, so no operand is transposed
// in memory.
#include <algorithm>
#include <cstdint>
#include <cuda.h>

#include "kernels.h"
#include "layer.cuh"

namespace ozemu {

namespace {

constexpr int kBlock = 64;               // elements of an operand block: 64 rows of 64 (128 bytes)
constexpr int kBlockBytes = 64 * 128;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);

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
  int vec;  // bits: 1 bias, 2 res, 4 pre, 8 out rows start on 16-byte boundaries
};

struct Product {
  int m, n;        // rows and columns of D
  int kb;          // 64-element blocks of the reduction
  int a_mn, b_mn;  // the operand's reduction runs down its rows
  int tiles_m, tiles_n;
  Epilogue e;
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_word,
                                          uint32_t* flags) {
  int ok = 0;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, abort_word, flags) ? 1 : 0;
  return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
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

// Eight consecutive elements p[0..7] of which `left` exist, as floats (0 past
// the end); one 16-byte load where the address allows.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int left, bool vec, float (&v)[8]) {
  if (vec && left >= 8) {
    unpack16<T>(__ldg(reinterpret_cast<const uint4*>(p)), v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? to_float(p[i]) : 0.f;
  }
}

template <int kAct>
__device__ __forceinline__ void activate_all(float (&z)[64]) {
#pragma unroll
  for (int i = 0; i < 64; ++i) z[i] = activate(z[i], kAct);
}

// A warp writes its 32 rows x 64 columns (one row a lane, in v) to rows
// row0.. and columns col0.. of an m x n matrix, through its 4 KB of shared
// memory so that each row leaves in 16-byte pieces of one 128-byte run.  The
// 16-byte pieces of row i are stored at piece ^ (i % 8): neither side has
// bank conflicts.
template <typename T>
__device__ __forceinline__ void store_rows(const float (&v)[64], uint8_t* stage, T* out, long long ldo, int row0,
                                           int col0, int m, int n, bool vec) {
  const int lane = threadIdx.x & 31;
  uint4* mine = reinterpret_cast<uint4*>(stage + lane * 128);
#pragma unroll
  for (int c = 0; c < 8; ++c)
    mine[c ^ (lane & 7)] = pack16<T>(v + 8 * c);
  __syncwarp();
  if (vec && col0 + 64 <= n) {
    const int c = lane & 7;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      if (row0 + r < m)
        *reinterpret_cast<uint4*>(out + (row0 + r) * ldo + col0 + 8 * c) =
            reinterpret_cast<const uint4*>(stage + r * 128)[c ^ (r & 7)];
    }
  } else {
    const int rows = m - row0 < 32 ? m - row0 : 32;
    for (int r = 0; r < rows; ++r) {
      T* o = out + (row0 + r) * ldo + col0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = 32 * h + lane;
        if (col0 + j < n)
          o[j] = reinterpret_cast<const T*>(stage + r * 128 + (((j >> 3) ^ (r & 7)) << 4))[j & 7];
      }
    }
  }
  __syncwarp();
}

// ---------------------------------------------------------------------------
// 256 x BN tiles on CTA pairs.
//
// Two CTAs of a cluster form one tile with the 2-SM MMA (M = 256): each stages
// its 128 rows of A and BN / 2 rows of B, so an operand byte in shared memory
// serves twice the multiplications of a single-CTA tile.  Persistent: each
// pair walks the tiles.  Warp 0 issues the TMA loads, one thread of warp 1 the
// MMAs (4 of K = 16 per 64-element stage), warps 2-9 take finished
// accumulators out of TMEM; two accumulators of BN columns alternate, so the
// next tile's MMAs run under this tile's epilogue.
// ---------------------------------------------------------------------------
template <int BN>
struct PairCfg {
  static constexpr int kABytes = 2 * kBlockBytes;          // 128 rows
  static constexpr int kBBlocks = BN / 2 / kBlock;         // 64-row blocks of B per CTA
  static constexpr int kStage = kABytes + kBBlocks * kBlockBytes;
  static constexpr int kStages = 192 * 1024 / kStage;
  static constexpr int kSmem = 1024 + kStages * kStage + kEpiWarps * 4096 + 256;
};
constexpr int kGroupM = 8;  // tile rows swept together, for reuse of B's columns in L2

__device__ __forceinline__ void tile_of(int t, const Product& p, int& tm, int& tn) {
  const int group = kGroupM * p.tiles_n;
  const int first = t / group * kGroupM;
  const int gm = min(kGroupM, p.tiles_m - first);
  tm = first + (t % group) % gm;
  tn = (t % group) / gm;
}

template <typename T, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product_pair_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                        const __grid_constant__ Product p, uint32_t* flags) {
  using C = PairCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + C::kStages * C::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kEpiWarps * 4096);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_word = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int total = p.tiles_m * p.tiles_n;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);   // armed by the first CTA with both CTAs' bytes
      mbar_init(&empty[s], 1);  // one commit from the pair's MMA issuer
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *abort_word = 0;
    fence_mbar_init();
    tma_prefetch_desc(&ma);
    tma_prefetch_desc(&mb);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int t = pair; t < total && ok; t += npairs) {
        int tm, tn;
        tile_of(t, p, tm, tn);
        const int i0 = tm * 256 + rank * 128, j0 = tn * BN + rank * (BN / 2);
        for (int kb = 0; kb < p.kb; ++kb, ++it) {
          const int s = it % C::kStages;
          if (!mbar_wait(&empty[s], ((it / C::kStages) & 1) ^ 1, abort_word, flags)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + s * C::kStage;
          const uint32_t bar = mapa_shared(&full[s], 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::kStage);
          const int k0 = kb * kBlock;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int i = i0 + q * kBlock;
            tma_load_2d_pair(st + q * kBlockBytes, &ma, bar, p.a_mn ? i : k0, p.a_mn ? k0 : i);
          }
#pragma unroll
          for (int q = 0; q < C::kBBlocks; ++q) {
            const int j = j0 + q * kBlock;
            tma_load_2d_pair(st + C::kABytes + q * kBlockBytes, &mb, bar, p.b_mn ? j : k0, p.b_mn ? k0 : j);
          }
        }
      }
      if (!ok) settle_after_abort();
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_f16(256, BN, Pair<T>::kBf16, p.a_mn != 0, p.b_mn != 0);
      // One MMA takes 16 of the reduction: 32 bytes along a K-major row, 16
      // rows of 128 bytes down an MN-major block.
      const uint32_t a_step = p.a_mn ? 2048 : 32, b_step = p.b_mn ? 2048 : 32;
      int it = 0, g = 0;
      bool ok = true;
      for (int t = pair; t < total && ok; t += npairs, ++g) {
        const int buf = g & 1, use = g >> 1;
        if (use > 0 && !mbar_wait(&tempty[buf], (use - 1) & 1, abort_word, flags)) break;
        tc_fence_after();
        const uint32_t d = tbase + static_cast<uint32_t>(buf * BN);
        for (int kb = 0; kb < p.kb; ++kb, ++it) {
          const int s = it % C::kStages;
          if (!mbar_wait(&full[s], (it / C::kStages) & 1, abort_word, flags)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_u32(smem + s * C::kStage);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_f16_pair(d, smem_desc_sw128(st + ks * a_step, p.a_mn != 0),
                         smem_desc_sw128(st + C::kABytes + ks * b_step, p.b_mn != 0), idesc,
                         (kb | ks) != 0 ? 1u : 0u);
          tc_commit_pair_multicast(&empty[s], 0x3);
        }
        if (ok) tc_commit_pair_multicast(&tfull[buf], 0x3);
      }
      tc_commit_pair_multicast(mma_done, 0x1);
      drain_wait(mma_done, 0, flags);
      if (!ok) settle_after_abort();
    }
    __syncwarp();
  } else {
    const int ew = warp - 2, quarter = warp & 3, half = ew >> 2;
    uint8_t* stage = staging + ew * 4096;
    const Epilogue& e = p.e;
    int g = 0;
    for (int t = pair; t < total; t += npairs, ++g) {
      int tm, tn;
      tile_of(t, p, tm, tn);
      const int buf = g & 1, use = g >> 1;
      if (!warp_wait(&tfull[buf], use & 1, abort_word, flags)) break;
      tc_fence_after();
      const int row0 = tm * 256 + rank * 128 + quarter * 32, row = row0 + lane;
      const uint32_t tcol = tbase + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(buf * BN);
#pragma unroll 1
      for (int c = half * (BN / 2); c < (half + 1) * (BN / 2); c += 64) {
        const int col0 = tn * BN + c;
        const bool last = c + 64 == (half + 1) * (BN / 2);
        if (row0 < p.m && col0 < p.n) {
          float z[64];
          {
            uint32_t u[32], v[32];
            tmem_ld32(tcol + c, u);
            tmem_ld32(tcol + c + 32, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              z[i] = __uint_as_float(u[i]);
              z[32 + i] = __uint_as_float(v[i]);
            }
          }
          if (last) {  // all of this warp's columns are in registers
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(&tempty[buf], 0));
          }
          if (e.bias) {
#pragma unroll
            for (int q = 0; q < 64; q += 8) {
              float b[8];
              load8(static_cast<const T*>(e.bias) + col0 + q, p.n - col0 - q, e.vec & 1, b);
#pragma unroll
              for (int i = 0; i < 8; ++i) z[q + i] += b[i];
            }
          }
          if (e.pre)
            store_rows(z, stage, static_cast<T*>(e.pre), e.ldpre, row0, col0, p.m, p.n, (e.vec & 4) != 0);
          switch (e.act) {
            case kActRelu: activate_all<kActRelu>(z); break;
            case kActGelu: activate_all<kActGelu>(z); break;
            case kActGeluTanh: activate_all<kActGeluTanh>(z); break;
            case kActSilu: activate_all<kActSilu>(z); break;
            default: break;
          }
          if (e.res && row < p.m) {
            const T* r = static_cast<const T*>(e.res) + row * e.ldr + col0;
#pragma unroll
            for (int q = 0; q < 64; q += 8) {
              float b[8];
              load8(r + q, p.n - col0 - q, (e.vec & 2) != 0, b);
#pragma unroll
              for (int i = 0; i < 8; ++i) z[q + i] += b[i];
            }
          }
          __syncwarp();  // every lane has read its part of r, which may be out
          store_rows(z, stage, static_cast<T*>(e.out), e.ldo, row0, col0, p.m, p.n, (e.vec & 8) != 0);
        } else if (last) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(&tempty[buf], 0));
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
// Elementwise and copying passes.
// ---------------------------------------------------------------------------

// out = act(bias) + r: the product of an empty reduction.
template <typename T>
__global__ void __launch_bounds__(256) empty_product_kernel(const Product p) {
  const Epilogue& e = p.e;
  const long long all = static_cast<long long>(p.m) * p.n;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < all; i += gridDim.x * 256LL) {
    const long long row = i / p.n;
    const int col = static_cast<int>(i % p.n);
    const float z = e.bias ? to_float(static_cast<const T*>(e.bias)[col]) : 0.f;
    if (e.pre) static_cast<T*>(e.pre)[row * e.ldpre + col] = from_float<T>(z);
    float y = activate(z, e.act);
    if (e.res) y += to_float(static_cast<const T*>(e.res)[row * e.ldr + col]);
    static_cast<T*>(e.out)[row * e.ldo + col] = from_float<T>(y);
  }
}

// Rows of 16-bit elements copied to rows on 16-byte boundaries.
__global__ void __launch_bounds__(256) align_rows_kernel(const uint16_t* in, long long ldi, uint16_t* out,
                                                         long long ldo, int rows, int cols) {
  for (int r = blockIdx.y; r < rows; r += gridDim.y)
    for (int j = blockIdx.x * 256 + threadIdx.x; j < cols; j += gridDim.x * 256)
      out[r * ldo + j] = in[r * ldi + j];
}

// dz = dy act'(pre) (where dz is given) and, per chunk of rows, the column
// sums of the unrounded dz (where part is given).  A CTA takes 256 columns,
// eight to a thread, and `chunk` rows, eight at a time; the eight partial
// sums of a column are joined in shared memory in a fixed order.
template <typename T>
__global__ void __launch_bounds__(256) slope_kernel(const T* dy, long long lddy, const T* pre, long long ldpre, T* dz,
                                                    long long lddz, float* part, int m, int n, int chunk, int act,
                                                    int vec) {
  __shared__ float red[8][264];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int col = blockIdx.x * 256 + tx * 8, left = n - col;
  float s[8] = {};
  const long long end = min(static_cast<long long>(m), (blockIdx.y + 1LL) * chunk);
  if (left > 0) {
    for (long long i = static_cast<long long>(blockIdx.y) * chunk + ty; i < end; i += 8) {
      float v[8];
      load8(dy + i * lddy + col, left, vec & 1, v);
      if (act != kActNone) {
        float z[8];
        load8(pre + i * ldpre + col, left, vec & 2, z);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] *= activation_slope(z[q], act);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] += v[q];
      if (dz) {  // rows of dz start on 16-byte boundaries and are padded to 8
        *reinterpret_cast<uint4*>(dz + i * lddz + col) = pack16<T>(v);
      }
    }
  }
  if (!part) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) red[ty][tx * 8 + q] = s[q];
  __syncthreads();
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j < n) {
    float sum = 0.f;
#pragma unroll
    for (int y = 0; y < 8; ++y) sum += red[y][threadIdx.x];
    part[static_cast<long long>(blockIdx.y) * n + j] = sum;
  }
}

// out[j] = sum over the chunks of part[., j], in order.
template <typename T>
__global__ void __launch_bounds__(256) column_sum_kernel(const float* part, int chunks, int n, T* out) {
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= n) return;
  float s = 0.f;
  for (int c = 0; c < chunks; ++c) s += part[static_cast<long long>(c) * n + j];
  out[j] = from_float<T>(s);
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

struct Matrix {
  const void* p;
  long long ld;
  int rows, cols;
};

int pad8(int x) { return (x + 7) & ~7; }

bool rows_aligned(const void* p, long long ld, int rows) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows <= 1 || (ld & 7) == 0);
}
bool rows_aligned(const Matrix& x) { return rows_aligned(x.p, x.ld, x.rows); }

// Bytes of a copy of x with rows on 16-byte boundaries; 0 where x's are.
size_t aligned_copy_bytes(const Matrix& x) {
  if (rows_aligned(x)) return 0;
  return (static_cast<size_t>(x.rows) * pad8(x.cols) * 2 + 255) & ~static_cast<size_t>(255);
}

// Takes that copy (where one is needed) at *ws and moves *ws past it.
Matrix aligned_copy(const Matrix& x, uint8_t** ws, cudaStream_t stream) {
  const size_t bytes = aligned_copy_bytes(x);
  if (bytes == 0) return x;
  const Matrix y = {*ws, pad8(x.cols), x.rows, x.cols};
  *ws += bytes;
  const dim3 grid(std::min((x.cols + 255) / 256, 64), std::min(x.rows, 2048));
  align_rows_kernel<<<grid, 256, 0, stream>>>(static_cast<const uint16_t*>(x.p), x.ld,
                                              reinterpret_cast<uint16_t*>(const_cast<void*>(y.p)), y.ld, x.rows,
                                              x.cols);
  return y;
}

// Map of an operand read in blocks of `box` rows of 64 elements; what lies
// outside the matrix reads as 0.
bool make_map(CUtensorMap* map, const Matrix& x, bool bf16, int box) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(x.cols), static_cast<cuuint64_t>(x.rows)};
  // A single row's leading dimension is never used, but has to be encodable.
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(x.rows > 1 ? x.ld : pad8(x.cols)) * 2};
  const cuuint32_t shape[2] = {kBlock, static_cast<cuuint32_t>(box)}, ones[2] = {1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
            const_cast<void*>(x.p), dims, strides, shape, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDev = 64;

// CTA pairs that can be resident at once (a persistent grid must not exceed
// them); sets the kernel's shared-memory size on the way.
template <typename T, int BN>
cudaError_t resident_pairs(int* pairs) {
  static int known[kMaxDev] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  if (known[dev] == 0) {
    auto kern = product_pair_kernel<T, BN>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PairCfg<BN>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = PairCfg<BN>::kSmem;
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
  *pairs = known[dev];
  return cudaSuccess;
}

template <typename T, int BN>
cudaError_t launch_pairs(const CUtensorMap& ma, const CUtensorMap& mb, Product p, uint32_t* flags,
                         cudaStream_t stream) {
  int pairs = 0;
  const cudaError_t e = resident_pairs<T, BN>(&pairs);
  if (e != cudaSuccess) return e;
  p.tiles_m = (p.m + 255) / 256;
  p.tiles_n = (p.n + BN - 1) / BN;
  const int tiles = p.tiles_m * p.tiles_n;
  product_pair_kernel<T, BN>
      <<<2 * std::min(tiles, pairs), kThreads, PairCfg<BN>::kSmem, stream>>>(ma, mb, p, flags);
  return cudaGetLastError();
}

// D = A B^T over `depth`, with the epilogue e.  a: m x depth (or depth x m
// where a_mn), b likewise; rows on 16-byte boundaries.
template <typename T>
cudaError_t run_product(int m, int n, int depth, const Matrix& a, bool a_mn, const Matrix& b, bool b_mn, Epilogue e,
                        uint32_t* flags, cudaStream_t stream) {
  e.vec = (e.bias && rows_aligned(e.bias, 0, 1) ? 1 : 0) | (e.res && rows_aligned(e.res, e.ldr, m) ? 2 : 0) |
          (e.pre && rows_aligned(e.pre, e.ldpre, m) ? 4 : 0) | (rows_aligned(e.out, e.ldo, m) ? 8 : 0);
  Product p = {m, n, (depth + kBlock - 1) / kBlock, a_mn, b_mn, 0, 0, e};
  if (depth == 0) {
    const long long all = static_cast<long long>(m) * n;
    empty_product_kernel<T><<<static_cast<int>(std::min<long long>((all + 255) / 256, 4096)), 256, 0, stream>>>(p);
    return cudaGetLastError();
  }
  CUtensorMap ma, mb;
  if (!make_map(&ma, a, Pair<T>::kBf16, kBlock) || !make_map(&mb, b, Pair<T>::kBf16, kBlock))
    return cudaErrorInvalidValue;
  return n > 128 ? launch_pairs<T, 256>(ma, mb, p, flags, stream) : launch_pairs<T, 128>(ma, mb, p, flags, stream);
}

template <typename T>
cudaError_t linear_t(const LinearCall& c, cudaStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(c.ws);
  Matrix x = {c.x, c.ldx, c.m, c.k}, w = {c.w, c.ldw, c.n, c.k};
  if (c.k > 0) {
    x = aligned_copy(x, &ws, stream);
    w = aligned_copy(w, &ws, stream);
  }
  const Epilogue e = {c.bias, c.res, c.ldr, c.pre, c.ldpre, c.y, c.ldy, c.act, 0};
  return run_product<T>(c.m, c.n, c.k, x, false, w, false, e, c.flags, stream);
}

// Row chunks of the slope pass: enough CTAs to fill the GPU, at most 64 sums
// to join per column.
int slope_chunk(int m, int n) {
  const int across = (n + 255) / 256;
  const int chunks = std::max(1, std::min(64, 1216 / across));
  return std::max(8, ((m + chunks - 1) / chunks + 7) / 8 * 8);
}

struct BackwardPlan {
  bool own_dz;  // dz is written to the workspace (else it is dy itself)
  size_t dz, part, x, w;
};
BackwardPlan backward_plan(const LinearGradCall& c) {
  BackwardPlan p;
  p.own_dz = c.act != kActNone || !rows_aligned(c.dy, c.lddy, c.m);
  const size_t up = 255;
  p.dz = p.own_dz ? (static_cast<size_t>(c.m) * pad8(c.n) * 2 + up) & ~up : 0;
  const int chunk = slope_chunk(c.m, c.n);
  p.part = (static_cast<size_t>((c.m + chunk - 1) / chunk) * c.n * 4 + up) & ~up;
  p.x = aligned_copy_bytes({c.x, c.ldx, c.m, c.k});
  p.w = aligned_copy_bytes({c.w, c.ldw, c.n, c.k});
  return p;
}

template <typename T>
cudaError_t linear_backward_t(const LinearGradCall& c, cudaStream_t stream) {
  const Epilogue none = {nullptr, nullptr, 0, nullptr, 0, nullptr, 0, kActNone, 0};
  Matrix dz = {c.dy, c.lddy, c.m, c.n};
  uint8_t* ws = static_cast<uint8_t*>(c.ws);
  if (c.m > 0 && c.n > 0) {
    const BackwardPlan plan = backward_plan(c);
    T* own = nullptr;
    if (plan.own_dz && (c.dx || c.dw)) {
      own = reinterpret_cast<T*>(ws);
      dz = {own, pad8(c.n), c.m, c.n};
    }
    ws += plan.dz;
    float* part = reinterpret_cast<float*>(ws);
    ws += plan.part;
    if (own || c.db) {
      const int chunk = slope_chunk(c.m, c.n), chunks = (c.m + chunk - 1) / chunk;
      const int vec = (rows_aligned(c.dy, c.lddy, c.m) ? 1 : 0) |
                      (c.act != kActNone && rows_aligned(c.pre, c.ldpre, c.m) ? 2 : 0);
      slope_kernel<T><<<dim3((c.n + 255) / 256, chunks), 256, 0, stream>>>(
          static_cast<const T*>(c.dy), c.lddy, static_cast<const T*>(c.pre), c.ldpre, own, pad8(c.n),
          c.db ? part : nullptr, c.m, c.n, chunk, c.act, vec);
      if (c.db)
        column_sum_kernel<T><<<(c.n + 255) / 256, 256, 0, stream>>>(part, chunks, c.n, static_cast<T*>(c.db));
    }
  } else if (c.db && c.n > 0) {
    column_sum_kernel<T><<<(c.n + 255) / 256, 256, 0, stream>>>(nullptr, 0, c.n, static_cast<T*>(c.db));
  }
  cudaError_t s = cudaGetLastError();
  if (s == cudaSuccess && c.dx && c.m > 0 && c.k > 0) {
    Matrix w = {c.w, c.ldw, c.n, c.k};
    if (c.n > 0) w = aligned_copy(w, &ws, stream);
    Epilogue e = none;
    e.out = c.dx;
    e.ldo = c.lddx;
    s = run_product<T>(c.m, c.k, c.n, dz, false, w, true, e, c.flags, stream);
  }
  if (s == cudaSuccess && c.dw && c.n > 0 && c.k > 0) {
    Matrix x = {c.x, c.ldx, c.m, c.k};
    if (c.m > 0) x = aligned_copy(x, &ws, stream);
    Epilogue e = none;
    e.out = c.dw;
    e.ldo = c.lddw;
    s = run_product<T>(c.n, c.k, c.m, dz, true, x, true, e, c.flags, stream);
  }
  return s;
}

}  // namespace

size_t linear_workspace(const LinearCall& c) {
  return aligned_copy_bytes({c.x, c.ldx, c.m, c.k}) + aligned_copy_bytes({c.w, c.ldw, c.n, c.k});
}

cudaError_t launch_linear(const LinearCall& c, cudaStream_t stream) {
  return c.type == kF16 ? linear_t<__half>(c, stream) : linear_t<__nv_bfloat16>(c, stream);
}

size_t linear_backward_workspace(const LinearGradCall& c) {
  const BackwardPlan p = backward_plan(c);
  return p.dz + p.part + p.x + p.w;
}

cudaError_t launch_linear_backward(const LinearGradCall& c, cudaStream_t stream) {
  return c.type == kF16 ? linear_backward_t<__half>(c, stream) : linear_backward_t<__nv_bfloat16>(c, stream);
}

}  // namespace ozemu
