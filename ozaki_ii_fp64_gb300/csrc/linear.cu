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
//
// dz is rounded to the operands' type for dx and dw, as the tensor cores take
// it; db sums it unrounded.  That is one more rounding than products of fp32
// values would have: where dz has one (an activation other than none and relu),
// the error of dx and dw against 64 bits, relative in 2-norm, goes from 1.7e-3
// to 2.3e-3 in bf16 (8192 x 4096 -> 16384, gelu) and from 2.1e-4 to 2.9e-4 in
// f16, and an f16 dz beyond 65504 is infinite.  Two 16-bit parts of dz would
// avoid it for twice the MMAs of both products.  Sums in the tensor cores
// differ from sums of fp32 roundings in the last bits: the forward product's
// outputs by 1.4e-4 of them, bf16 roundings that fall the other way, at the
// same error against 64 bits.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <mutex>
#include <utility>

#include "kernels.h"
#include "layer.cuh"

namespace ozemu {

namespace {

constexpr int kBlock = 64;               // elements of an operand block: 64 rows of 64 (128 bytes)
constexpr int kBlockBytes = 64 * 128;
constexpr int kEpiWarps = 16;
constexpr int kThreads = 32 * (3 + kEpiWarps);

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

// Eight consecutive elements p[0..7] of which `left` exist, as floats (0 past
// the end); one 16-byte load where the address allows.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int left, bool vec, float2 (&v)[4]) {
  if (vec && left >= 8) {
    unpack16<T>(__ldg(reinterpret_cast<const uint4*>(p)), v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = make_float2(2 * i < left ? to_float(p[2 * i]) : 0.f, 2 * i + 1 < left ? to_float(p[2 * i + 1]) : 0.f);
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

// A warp's 32 rows x 32 columns of 16-bit elements pass through its 2 KB of
// shared memory (row r at byte 64 r, its 16-byte piece c at piece
// c ^ (r / 2 % 4): no bank conflicts by rows or by pieces), so that a row moves
// as one 64-byte run.  A lane's share on the way: piece lane % 4 of rows
// 8 i + lane / 4; or, where rows do not start on 16-byte boundaries, word
// lane % 16 of rows 2 i + lane / 16, between words where the row starts on an
// odd element.
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
  if (vec && col0 + 32 <= n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row0 + 8 * i + (lane >> 2);
      v[i] = r < m ? *reinterpret_cast<const uint4*>(in + r * ld + col0 + 8 * (lane & 3)) : make_uint4(0, 0, 0, 0);
    }
    return;
  }
  uint32_t* w = reinterpret_cast<uint32_t*>(v);
  const uint16_t* p = reinterpret_cast<const uint16_t*>(in) + row0 * ld + col0;
  const int word = lane & 15;
  if (col0 > 0 && col0 + 32 <= n) {  // the element before the run is the row's, too
    // All loads first: the words, and for row `lane` the last element, which a
    // row that starts on an odd element has in a 17th word.
    const uint32_t last = row0 + lane < m ? p[lane * ld + 31] : 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = 2 * i + (lane >> 4);
      const uintptr_t q = reinterpret_cast<uintptr_t>(p + r * ld) & ~uintptr_t(3);
      w[i] = row0 + r < m ? *(reinterpret_cast<const uint32_t*>(q) + word) : 0;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = 2 * i + (lane >> 4);
      const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, w[i], 1), tail = __shfl_sync(0xFFFFFFFFu, last, r);
      if (reinterpret_cast<uintptr_t>(p + r * ld) & 2u) w[i] = __funnelshift_r(w[i], word == 15 ? tail : next, 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = 2 * i + (lane >> 4);
      const uint16_t* q = p + r * ld + 2 * word;
      const uint32_t a = row0 + r < m && col0 + 2 * word < n ? q[0] : 0;
      const uint32_t b = row0 + r < m && col0 + 2 * word + 1 < n ? q[1] : 0;
      w[i] = a | (b << 16);
    }
  }
}

__device__ __forceinline__ void stage_rows(const uint4 (&v)[4], uint8_t* stage, int col0, int n, bool vec) {
  const int lane = threadIdx.x & 31;
  if (vec && col0 + 32 <= n) {
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
  const bool whole = col0 + 32 <= n;
  const int word = lane & 15;
#pragma unroll 1
  for (int i0 = 0; i0 < 16; i0 += 4) {
    uint32_t a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *stage_word(stage, 2 * (i0 + i) + (lane >> 4), word);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __shfl_down_sync(0xFFFFFFFFu, a[i], 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 2 * (i0 + i) + (lane >> 4);
      uint16_t* q = p + r * ldo;
      const bool odd = (reinterpret_cast<uintptr_t>(q) & 2u) != 0, in_m = row0 + r < m;
      if (whole) {  // from an odd start: words of elements 2 word + 1 and 2 word + 2, and the two ends
        const uint32_t both = odd ? __funnelshift_r(a[i], b[i], 16) : a[i];
        if (in_m && !(odd && word == 15)) *reinterpret_cast<uint32_t*>(q + 2 * word + (odd ? 1 : 0)) = both;
        if (in_m && odd && word == 15) q[31] = static_cast<uint16_t>(a[i] >> 16);
        if (in_m && odd && word == 0) q[0] = static_cast<uint16_t>(a[i]);
      } else {
        if (in_m && col0 + 2 * word < n) q[2 * word] = static_cast<uint16_t>(a[i]);
        if (in_m && col0 + 2 * word + 1 < n) q[2 * word + 1] = static_cast<uint16_t>(a[i] >> 16);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// 256 x BN tiles on CTA pairs, BN = 64, 128, 192 or 256.
//
// Two CTAs of a cluster form one tile with the 2-SM MMA (M = 256): each stages
// its 128 rows of A and BN / 2 rows of B, so an operand byte in shared memory
// serves twice the multiplications of a single-CTA tile.  Persistent: each
// pair walks the tiles.  A warp issues the TMA loads of A, another those of B,
// another the MMAs (4 of K = 16 per 64-element stage), and sixteen take finished
// accumulators out of TMEM; two accumulators of 256 columns, or four of 128,
// alternate, so the next tiles' MMAs run under this tile's epilogue.
//
// Few tiles with a long reduction: `split` (2 or 4) pairs of a cluster share a
// tile, each with a part of the reduction.  Each CTA leaves its fp32 sums in
// the ring's shared memory, and the pairs take alternate 64-column chunks,
// adding the parts up through distributed shared memory in order.
//
// Bound by the MMAs (256 columns) or a CTA's loads (128): 8192 x 4096 -> 16384
// bf16 with gelu_tanh, pre kept: 575 us in a short burst (1.91 PFLOP/s), 694 at
// the clocks that the power cap leaves after seconds of it.  A launch costs 4 to
// 6.5 us beyond its rounds, and rows of no alignment another 8 at 1000 x 2049 ->
// 4099, f16 with a residual (35 us).
// ---------------------------------------------------------------------------
constexpr int kRing = 192 * 1024;  // stages of two blocks of A and one or two of B: 8 or 6
constexpr int kMaxStages = 8;
constexpr int kPairSmem = 1024 + kRing + kEpiWarps * (2048 + 64) + 256;  // staging, a chunk's bias, barriers
constexpr int kGroupM = 8;  // tile rows swept together, for reuse of B's columns in L2

struct Product {
  int m, n;        // rows and columns of D
  int kb;          // 64-element blocks of the reduction
  int a_mn, b_mn;  // the operand's reduction runs down its rows
  int bn;          // columns of a tile
  int split;       // pairs that share a tile's reduction
  int share;       // blocks of it for each
  int tiles_m, tiles_n;
  uint32_t group_inverse, group_shift;  // of kGroupM tiles_n
  Epilogue e;
};

// One product, or two whose tiles follow each other in one launch (the
// gradients dx and dw).
struct Products {
  Product p[2];
  int count;
  int stage_bytes;
  int bufs;  // accumulators in TMEM: 4 of 128 columns or 2 of 256
};

__device__ __forceinline__ void tile_of(int t, const Product& p, int& tm, int& tn) {
  // t / (kGroupM tiles_n) by the reciprocal that the host rounded up: exact
  // for the product's tiles.
  const int turn = static_cast<int>(__umulhi(static_cast<uint32_t>(t), p.group_inverse) >> p.group_shift);
  const int first = turn * kGroupM, rest = t - turn * kGroupM * p.tiles_n;
  const int gm = min(kGroupM, p.tiles_m - first);
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

// The sums that a pair of a split tile leaves: 128 rows of up to 256 fp32, the
// 16-byte piece c of row r at piece c ^ (r % 32), so that a warp's rows meet
// in no bank.
__device__ __forceinline__ uint32_t part_piece(int r, int c) {
  return static_cast<uint32_t>(r * 1024 + ((c ^ (r & 31)) << 4));
}

// One warp's 32 rows x 32 columns of accumulators, a row a lane, from
// source(last, z) through the epilogue; the source is asked for the last time
// with last = true.
template <typename T, typename F>
__device__ __forceinline__ void finish_rows(F source, const uint4 (&res)[4], const Epilogue& e, uint8_t* stage,
                                            const uint4* bias, int row0, int col0, int m, int n) {
  const int lane = threadIdx.x & 31;
  float z[32];
  auto take = [&](bool last) {
    source(last, z);
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
    stage_rows(res, stage, col0, n, (e.vec & 2) != 0);
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
      for (int i = 0; i < 8; ++i) z[8 * c + i] += r[i];
    }
    *at = pack16<T>(z + 8 * c);
  }
  __syncwarp();
  write_rows(stage, static_cast<T*>(e.out), e.ldo, row0, col0, m, n, (e.vec & 8) != 0);
  __syncwarp();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    product_pair_kernel(const __grid_constant__ CUtensorMap ma0, const __grid_constant__ CUtensorMap mb0,
                        const __grid_constant__ CUtensorMap ma1, const __grid_constant__ CUtensorMap mb1,
                        const __grid_constant__ Products g, uint32_t* flags) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + kRing;
  uint8_t* biases = staging + kEpiWarps * 2048;
  uint64_t* full = reinterpret_cast<uint64_t*>(biases + kEpiWarps * 64);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 4;
  uint64_t* mma_done = tempty + 4;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_word = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int place = static_cast<int>(cluster_rank()), rank = place & 1, lead = place & ~1;
  const uint16_t both_ctas = static_cast<uint16_t>(0x3 << lead);
  const int first = g.p[0].tiles_m * g.p[0].tiles_n;  // tiles of the first product
  const int total = first + (g.count > 1 ? g.p[1].tiles_m * g.p[1].tiles_n : 0);
  // A pair walks the tiles, or takes its part of one tile's reduction (of one
  // product).
  const int split = g.p[0].split;
  const int pair = blockIdx.x / (2 * split), npairs = split > 1 ? total : gridDim.x >> 1;
  const int stage_bytes = g.stage_bytes, stages = kRing / stage_bytes;
  const int buf_shift = g.bufs == 4 ? 2 : 1, buf_columns = 512 >> buf_shift;
  // This pair's blocks of a product's reduction.
  auto part = [&](const Product& p, int& kb0, int& kb1) {
    kb0 = min((place >> 1) * p.share, p.kb);
    kb1 = min(kb0 + p.share, p.kb);
  };

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);   // armed by the first CTA with both CTAs' bytes
      mbar_init(&empty[s], 1);  // one commit from the pair's MMA issuer
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *abort_word = 0;
    fence_mbar_init();
    tma_prefetch_desc(&ma0);
    tma_prefetch_desc(&mb0);
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
  chain_next();
  chain_wait();

  if (warp == 0 || warp == 2 + kEpiWarps) {
    // One thread loads A, one B: a stage's loads, issued by one thread, took
    // longer than its MMAs.
    const bool loads_a = warp == 0;
    const uint32_t bar0 = mapa_shared(&full[0], lead);
    int s = 0;
    uint32_t phase = 1;
    bool ok = true;
    for (int t = pair; t < total && ok; t += npairs) {
      const bool second = t >= first;
      const Product& p = g.p[second];
      const CUtensorMap* map = loads_a ? (second ? &ma1 : &ma0) : (second ? &mb1 : &mb0);
      int tm, tn, kb0, kb1;
      tile_of(second ? t - first : t, p, tm, tn);
      part(p, kb0, kb1);
      // B's BN / 2 rows of this CTA come in whole blocks (a part block's last
      // rows are loaded and not used).
      const int b_blocks = p.bn > 128 ? 2 : 1;
      const uint32_t bytes = 2 * (2 + b_blocks) * kBlockBytes;
      const bool arms = loads_a && rank == 0;  // for both CTAs and operands
      const bool down = loads_a ? p.a_mn != 0 : p.b_mn != 0;
      const bool two = down && (loads_a || b_blocks == 2);
      const int at = loads_a ? tm * 256 + rank * 128 : tn * p.bn + rank * (p.bn / 2);
      const uint32_t to = loads_a ? 0 : 2 * kBlockBytes;
      for (int k = kb0 * kBlock; k < kb1 * kBlock; k += kBlock) {
        if (!all_wait(&empty[s], phase, abort_word, flags)) {
          ok = false;
          break;
        }
        uint8_t* st = smem + s * stage_bytes + to;
        const uint32_t bar = bar0 + s * 8;
        if (elect_one()) {
          if (arms) mbar_arrive_expect_tx_relaxed(&full[s], bytes);
          tma_load_2d_pair(st, map, bar, down ? at : k, down ? k : at);
          if (two) tma_load_2d_pair(st + kBlockBytes, map, bar, at + kBlock, k);
        }
        __syncwarp();
        if (++s == stages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) settle_after_abort();
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      int s = 0, n_tiles = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = pair; t < total && ok; t += npairs, ++n_tiles) {
        const Product& p = g.p[t >= first];
        const uint32_t idesc = idesc_f16(256, p.bn, Pair<T>::kBf16, p.a_mn != 0, p.b_mn != 0);
        // One MMA takes 16 of the reduction: 32 bytes along a K-major row, 16
        // rows of 128 bytes down an MN-major block (descriptors count 16 bytes).
        const uint32_t a_step = p.a_mn ? 128 : 2, b_step = p.b_mn ? 128 : 2;
        const uint32_t a_lo = smem_desc_sw128_lo(smem_u32(smem), p.a_mn != 0);
        const uint32_t b_lo = smem_desc_sw128_lo(smem_u32(smem) + 2 * kBlockBytes, p.b_mn != 0);
        int kb0, kb1;
        part(p, kb0, kb1);
        const int buf = n_tiles & (g.bufs - 1), use = n_tiles >> buf_shift;
        if (use > 0 && !all_wait(&tempty[buf], (use - 1) & 1, abort_word, flags)) break;
        tc_fence_after();
        const uint32_t d = tbase + static_cast<uint32_t>(buf * buf_columns);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!all_wait(&full[s], phase, abort_word, flags)) {
            ok = false;
            break;
          }
          const uint32_t at = s * (stage_bytes / 16);
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_f16_pair(d, smem_desc_sw128(a_lo + at + ks * a_step), smem_desc_sw128(b_lo + at + ks * b_step), idesc,
                           ks != 0 ? 1u : (kb != kb0 ? 1u : 0u));
            tc_commit_pair_multicast(&empty[s], both_ctas);
          }
          __syncwarp();
          if (++s == stages) {
            s = 0;
            phase ^= 1;
          }
        }
        if (ok && elect_one()) tc_commit_pair_multicast(&tfull[buf], both_ctas);
        __syncwarp();
      }
      if (elect_one()) {
        tc_commit_pair_multicast(mma_done, static_cast<uint16_t>(1 << lead));
        drain_wait(mma_done, 0, flags);
        if (!ok) settle_after_abort();
      }
    }
    __syncwarp();
  } else {
    // Lane quarter warp % 4; the quarter's four warps take 32-column chunks in
    // turn.  (Eight warps of 64-column chunks left each scheduler two warps to
    // hide an epilogue's latencies with.)
    const int ew = warp - 2, quarter = warp & 3, group = ew >> 2;
    uint8_t *stage = staging + ew * 2048, *bias = biases + ew * 64;
    int n_tiles = 0;
    for (int t = pair; t < total; t += npairs, ++n_tiles) {
      const bool second = t >= first;
      const Product& p = g.p[second];
      const Epilogue& e = p.e;
      int tm, tn;
      tile_of(second ? t - first : t, p, tm, tn);
      const int buf = n_tiles & (g.bufs - 1), use = n_tiles >> buf_shift;
      const int row0 = tm * 256 + rank * 128 + quarter * 32;
      // Columns of the tile that this warp has to take: none past D's edge.
      const int cols = row0 < p.m ? min(p.bn, p.n - tn * p.bn) : 0;
      const uint32_t tcol = tbase + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(buf * buf_columns);
      if (split > 1) {  // leave the sums; the cluster joins them below
        int kb0, kb1;
        part(p, kb0, kb1);
        if (!warp_wait(&tfull[buf], use & 1, abort_word, flags)) break;
        tc_fence_after();
        const int r = quarter * 32 + lane;
        for (int c = group * 32; c < cols; c += 128) {
          uint32_t u[32];
          if (kb0 < kb1) {
            tmem_ld32(tcol + c, u);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = 0;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(smem + part_piece(r, c / 4 + i)) =
                make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
        }
        break;  // one tile
      }
      bool waited = false, live = true;
#pragma unroll 1
      for (int c = group * 32; c < cols; c += 128) {
        const int col0 = tn * p.bn + c;
        uint4 res[4];
        if (e.res)
          read_rows(res, static_cast<const T*>(e.res), e.ldr, row0, col0, p.m, p.n, (e.vec & 2) != 0);
        if (e.bias) {  // the chunk's 32 values, for every lane
          const uint16_t b = col0 + lane < p.n ? static_cast<const uint16_t*>(e.bias)[col0 + lane] : 0;
          __syncwarp();
          reinterpret_cast<uint16_t*>(bias)[lane] = b;
          __syncwarp();
        }
        if (!waited) {
          live = warp_wait(&tfull[buf], use & 1, abort_word, flags);
          if (!live) break;
          tc_fence_after();
          waited = true;
        }
        finish_rows<T>(
            [&](bool last, float(&z)[32]) {
              uint32_t u[32];
              tmem_ld32(tcol + c, u);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) z[i] = __uint_as_float(u[i]);
              if (last && c + 128 >= cols) {  // this warp's last columns of the tile
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(&tempty[buf], lead));
              }
            },
            res, e, stage, reinterpret_cast<const uint4*>(bias), row0, col0, p.m, p.n);
      }
      if (!live) break;
      if (group * 32 >= cols) {  // nothing to take: still let the buffer go, after the tile is done
        if (!warp_wait(&tfull[buf], use & 1, abort_word, flags)) break;
        if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(&tempty[buf], lead));
      }
    }
  }

  if (split > 1) {
    const Product& p = g.p[0];
    __syncthreads();
    cluster_sync();  // every pair's sums are in its shared memory
    if (warp >= 2 && warp < 2 + kEpiWarps) {
      // Eight rows a warp, a row's 64 columns to half a warp: shared memory of
      // another CTA is read in contiguous runs, and so is global memory.
      const Epilogue& e = p.e;
      int tm, tn;
      tile_of(pair, p, tm, tn);
      const int r0 = (warp - 2) * 8 + (lane >> 4), cols = min(p.bn, p.n - tn * p.bn);
      const long long grow0 = tm * 256 + rank * 128;
      for (int c = (place >> 1) * 64; c < cols; c += 64 * split) {
        const int piece = c / 4 + (lane & 15), col = tn * p.bn + c + (lane & 15) * 4, left = p.n - col;
        if (left <= 0) continue;
        float b[4] = {0.f, 0.f, 0.f, 0.f};
        if (e.bias) load4(static_cast<const T*>(e.bias) + col, left, e.vec & 1, b);
        {
          float z[4][4] = {};
          for (int q = 0; q < split; q += 2) {
            float4 v[2][4];  // all loads before the first sum
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                v[k][i] = load_cluster16(mapa_shared(smem, 2 * (q + k) + rank) + part_piece(r0 + 2 * i, piece));
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                z[i][0] += v[k][i].x;
                z[i][1] += v[k][i].y;
                z[i][2] += v[k][i].z;
                z[i][3] += v[k][i].w;
              }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const long long row = grow0 + r0 + 2 * i;
            if (row >= p.m) continue;
#pragma unroll
            for (int k = 0; k < 4; ++k) z[i][k] += b[k];
            if (e.pre) store4(static_cast<T*>(e.pre) + row * e.ldpre + col, z[i], left, (e.vec & 4) != 0);
            activate_all(z[i], e.act);
            if (e.res) {
              float r[4];
              load4(static_cast<const T*>(e.res) + row * e.ldr + col, left, (e.vec & 2) != 0, r);
#pragma unroll
              for (int k = 0; k < 4; ++k) z[i][k] += r[k];
            }
            store4(static_cast<T*>(e.out) + row * e.ldo + col, z[i], left, (e.vec & 8) != 0);
          }
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
// Few rows (tokens being decoded): the other operand is all the traffic.
//
// The wide operand takes the MMA's 128 rows and the tokens its N = NT columns,
// so every byte of a tile is one of the weights.  A cluster of S CTAs shares
// the 128 columns of D: each takes a part of the reduction, leaves its fp32
// sums in shared memory, and then adds up its share of the columns over the
// cluster, in rank order, with the epilogue.  Two CTAs fit an SM, so one's
// loads run under the other's start and end.  Bound by HBM: 1 x 4096 -> 16384
// bf16 24.9 us, 5.4 TB/s, 0.80 of the copy rate; the rest is the start and the
// cluster's join.  13 x 16384 -> 4096 f16 25.6 us; 128 x 4096 -> 4096 15.3.
// ---------------------------------------------------------------------------
template <int NT>
struct FewCfg {
  static constexpr int kStage = 2 * kBlockBytes + NT * 128;
  static constexpr int kStages = 108 * 1024 / kStage;
  static constexpr int kSmem = 1024 + kStages * kStage + 256;
  static constexpr int kTmemCols = NT < 32 ? 32 : NT;
  static_assert(NT * 512 <= kStages * kStage, "the partial sums take the ring's memory");
};
constexpr int kFewThreads = 192;
constexpr int kMaxSplit = 16;

struct FewProduct {
  int m, n;  // D: tokens x columns
  int kb;
  int w_mn;  // the wide operand's reduction runs down its rows
  int split;
  Epilogue e;
};

template <typename T, int NT>
__global__ void __launch_bounds__(kFewThreads, 2)
    product_few_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                       const __grid_constant__ FewProduct p, uint32_t* flags) {
  using C = FewCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStage);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(tfull + 1);
  volatile int* abort_word = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int j0 = blockIdx.x / p.split * 128, i0 = blockIdx.y * NT;
  const int per = (p.kb + p.split - 1) / p.split;
  const int kb0 = min(rank * per, p.kb), kb1 = min(kb0 + per, p.kb);

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
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!all_wait(&empty[s], phase, abort_word, flags)) {
        ok = false;
        break;
      }
      uint8_t* st = smem + s * C::kStage;
      const int k0 = kb * kBlock;
      if (elect_one()) {
        mbar_arrive_expect_tx_relaxed(&full[s], C::kStage);
        if (p.w_mn) {
          tma_load_2d(st, &mw, &full[s], j0, k0);
          tma_load_2d(st + kBlockBytes, &mw, &full[s], j0 + kBlock, k0);
        } else {
          tma_load_2d(st, &mw, &full[s], k0, j0);
        }
        tma_load_2d(st + 2 * kBlockBytes, &mx, &full[s], k0, i0);
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
    const uint32_t idesc = idesc_f16(128, NT, Pair<T>::kBf16, p.w_mn != 0, false);
    const uint32_t w_step = p.w_mn ? 128 : 2;
    const uint32_t w_lo = smem_desc_sw128_lo(smem_u32(smem), p.w_mn != 0);
    const uint32_t x_lo = smem_desc_sw128_lo(smem_u32(smem) + 2 * kBlockBytes, false);
    int s = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!all_wait(&full[s], phase, abort_word, flags)) {
        ok = false;
        break;
      }
      const uint32_t at = s * (C::kStage / 16);
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_f16(tbase, smem_desc_sw128(w_lo + at + ks * w_step), smem_desc_sw128(x_lo + at + ks * 2), idesc,
                  ks != 0 ? 1u : (kb != kb0 ? 1u : 0u));
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
    if (kb0 == kb1) {
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

  // This CTA's share of the columns: 128 / split of them, every token, four
  // columns of a token at a time.
  const Epilogue& e = p.e;
  const int width = 32 / p.split, rows = min(NT, p.m - i0);
  for (int at = threadIdx.x; at < rows * width; at += kFewThreads) {
    const int i = at / width, jj = (rank * width + at % width) * 4, j = j0 + jj, left = p.n - j;
    if (left <= 0) continue;
    const float* mine = reinterpret_cast<const float*>(smem) + i * 128 + jj;
    float z[4] = {};
    for (int s0 = 0; s0 < p.split; s0 += 8) {
      float4 u[8];  // all loads before the first sum
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s0 + s < p.split) u[s] = load_cluster16(mapa_shared(mine, s0 + s));
#pragma unroll
      for (int s = 0; s < 8; ++s)
        if (s0 + s < p.split) {
          z[0] += u[s].x;
          z[1] += u[s].y;
          z[2] += u[s].z;
          z[3] += u[s].w;
        }
    }
    const long long row = i0 + i;
    float v[4];
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
      for (int q = 0; q < 4; ++q) z[q] += v[q];
    }
    store4(static_cast<T*>(e.out) + row * e.ldo + j, z, left, (e.vec & 8) != 0);
  }
  cluster_sync();  // peers have read this CTA's sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, C::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Elementwise and copying passes.
// ---------------------------------------------------------------------------

// out = act(bias) + r: the product of an empty reduction.
template <typename T>
__global__ void __launch_bounds__(256) empty_product_kernel(const Product p) {
  chain_next();
  chain_wait();
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

// Copies of matrices of 16-bit elements with rows on 16-byte boundaries.  A
// thread makes 16-byte pieces: each from the two aligned pieces of the source
// that its elements lie in, moved by the bytes that the row starts past a
// boundary; element by element where those reach beyond the matrix.  (TMA takes
// rows on 16-byte boundaries only.)  Bound by L2 and the launch: 1000 x 2049 and
// 4099 x 2049, 21 MB read and 21 written, 8.5 us.
struct AlignArgs {
  const uint16_t* in;
  uint16_t* out;
  long long ldi, ldo;
  int rows, cols;
};
struct AlignPair {
  AlignArgs a[2];
};
__global__ void __launch_bounds__(256) align_rows_kernel(const __grid_constant__ AlignPair both) {
  chain_next();
  chain_wait();
  const AlignArgs& a = both.a[blockIdx.z];
  const int pieces = (a.cols + 7) / 8;
  const uintptr_t begin = reinterpret_cast<uintptr_t>(a.in);
  const uintptr_t end = reinterpret_cast<uintptr_t>(a.in + (a.rows - 1) * a.ldi + a.cols);
  const int across = (pieces + 31) / 32;  // 32 pieces of a row to a warp
  const long long all = static_cast<long long>(a.rows) * across;
  for (long long at = blockIdx.x * 8LL + (threadIdx.x >> 5); at < all; at += gridDim.x * 8LL) {
    const long long r = at / across;
    const int j = (static_cast<int>(at % across) * 32 + (threadIdx.x & 31)) * 8, left = a.cols - j;
    if (left <= 0) continue;
    const uint16_t* p = a.in + r * a.ldi + j;
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
    const uintptr_t from = reinterpret_cast<uintptr_t>(p) - off;
    uint32_t w[4];
    if (from >= begin && from + 32 <= end) {
      const uint4 lo = *reinterpret_cast<const uint4*>(from), hi = *reinterpret_cast<const uint4*>(from + 16);
      uint32_t u[5];
      switch (off >> 2) {  // the same for the whole warp
        case 0: u[0] = lo.x, u[1] = lo.y, u[2] = lo.z, u[3] = lo.w, u[4] = hi.x; break;
        case 1: u[0] = lo.y, u[1] = lo.z, u[2] = lo.w, u[3] = hi.x, u[4] = hi.y; break;
        case 2: u[0] = lo.z, u[1] = lo.w, u[2] = hi.x, u[3] = hi.y, u[4] = hi.z; break;
        default: u[0] = lo.w, u[1] = hi.x, u[2] = hi.y, u[3] = hi.z, u[4] = hi.w; break;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = (off & 2) ? __funnelshift_r(u[i], u[i + 1], 16) : u[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = 2 * i < left ? p[2 * i] : 0, hi = 2 * i + 1 < left ? p[2 * i + 1] : 0;
        w[i] = lo | (hi << 16);
      }
    }
    *reinterpret_cast<uint4*>(a.out + r * a.ldo + j) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// dz = dy act'(pre), rounded (where dz is given) and, per chunk of rows, the column
// sums of the unrounded dz (to part, or to db where there is one chunk).  A
// CTA takes 8 TX columns, eight to a thread, and `chunk` rows, 256 / TX at a
// time; the partial sums of a column are joined in shared memory in a fixed
// order.  TX = 4 for few rows (64 at a time, so that one or two turns read
// them all), else 32.  Bound by HBM and the slopes' instructions: 8192 x 16384
// bf16 gelu, 805 MB, 159 us (5.1 TB/s).
template <typename T, int kAct, int TX>
__global__ void __launch_bounds__(256, 4) slope_kernel(const T* dy, long long lddy, const T* pre, long long ldpre,
                                                       T* dz, long long lddz, float* part, T* db, int m, int n,
                                                       int chunk, int vec) {
  constexpr int TY = 256 / TX, kCols = 8 * TX;
  __shared__ float red[TY][kCols + 8];
  chain_next();
  chain_wait();
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
  const int col = blockIdx.x * kCols + tx * 8, left = n - col;
  float2 s[4] = {};
  const long long end = min(static_cast<long long>(m), (blockIdx.y + 1LL) * chunk);
  if (left > 0) {
#pragma unroll 2
    for (long long i = static_cast<long long>(blockIdx.y) * chunk + ty; i < end; i += TY) {
      float2 v[4];
      load8(dy + i * lddy + col, left, vec & 1, v);
      if constexpr (kAct != kActNone) {
        float2 z[4];
        load8(pre + i * ldpre + col, left, vec & 2, z);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = mul2(v[q], activation_slope2<kAct>(z[q]));
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) s[q] = add2(s[q], v[q]);
      if (dz) {  // rows of dz start on 16-byte boundaries and are padded to 8
        *reinterpret_cast<uint4*>(dz + i * lddz + col) = pack16<T>(v);
      }
    }
  }
  if (!part && !db) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    red[ty][tx * 8 + 2 * q] = s[q].x;
    red[ty][tx * 8 + 2 * q + 1] = s[q].y;
  }
  __syncthreads();
  const int j = blockIdx.x * kCols + threadIdx.x;
  if (threadIdx.x < kCols && j < n) {
    float sum = 0.f;
#pragma unroll 8
    for (int y = 0; y < TY; ++y) sum += red[y][threadIdx.x];
    if (db)  // one chunk: the sum is whole
      db[j] = from_float<T>(sum);
    else
      part[static_cast<long long>(blockIdx.y) * n + j] = sum;
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

// Makes those copies (where they are needed) of x and y at ws, in one launch,
// and points x and y at them.
cudaError_t align_operands(Matrix* x, Matrix* y, uint8_t* ws, cudaStream_t stream) {
  AlignPair both;
  int count = 0;
  long long most = 0;
  for (Matrix* m : {x, y}) {
    const size_t bytes = aligned_copy_bytes(*m);
    if (bytes == 0 || m->rows == 0 || m->cols == 0) continue;
    both.a[count++] = {static_cast<const uint16_t*>(m->p), reinterpret_cast<uint16_t*>(ws), m->ld, pad8(m->cols),
                       m->rows, m->cols};
    most = std::max(most, static_cast<long long>(m->rows) * ((m->cols + 255) / 256));
    m->p = ws;
    m->ld = pad8(m->cols);
    ws += bytes;
  }
  if (count == 0) return cudaSuccess;
  return launch_chained(align_rows_kernel, dim3(static_cast<unsigned>(std::min<long long>((most + 7) / 8, 152 * 16)), 1, count),
                        256, 0, stream, 0, both);
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

// Tiles that can be worked on at once by clusters of one, two or four CTA
// pairs (a persistent grid must not exceed the first; the GPCs leave some SMs
// out of the larger clusters: 76, 36 and 15 on this GPU); sets the kernel's
// shared-memory size on the way.
struct Resident {
  int tiles[3] = {0, 0, 0};
};
template <typename T>
cudaError_t resident_clusters(Resident* out) {
  static Resident known[kMaxDev];
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (known[dev].tiles[0] == 0) {
    auto kern = product_pair_kernel<T>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
    if (e != cudaSuccess) return e;
    Resident r;
    for (int i = 2; i >= 0; --i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2 << i, 1, 1);
      cfg.blockDim = dim3(kThreads, 1, 1);
      cfg.dynamicSmemBytes = kPairSmem;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = 2 << i;
      attr.val.clusterDim.y = 1;
      attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&r.tiles[i], kern, &cfg);
      if (e != cudaSuccess) return e;
    }
    if (r.tiles[0] < 1) return cudaErrorInvalidConfiguration;
    known[dev] = r;
  }
  *out = known[dev];
  return cudaSuccess;
}

// The tiling of a product: the columns of a tile, and the pairs that share a
// tile's reduction, whose estimated time in clocks is least.  Measured at
// 2 GHz on 256-row tiles: a 64-element block of the reduction takes 0.263 us
// at 256 columns (its MMAs 0.256), 0.21 at 192, 0.187 at 128 and 64 (a CTA's
// loads); a round of short reductions 3 us at 256 columns and 1.66 at 128 (its
// epilogue); joining a split tile's sums 5.2 us at 256 columns and 4 at 192.
// 2560 x 8192 -> 512: 40 us by one pair a tile of 256, 29 by two, 33 and 25.6
// at 192, 29 by one at 128; 512 x 4096 -> 4096: 23.5, 21.3, 20.7, 35.9, 18.4.
// An MN-major B comes in whole blocks of 64 columns for each CTA.
struct Tiling {
  int bn, split;
  long long cost;
};
// A round of tiles: their blocks of the reduction, or the epilogue of the
// round before where that takes longer.
long long round_cost(int kb, int bn) {
  const int block = bn == 256 ? 530 : bn == 192 ? 430 : 375;
  return std::max<long long>(static_cast<long long>(kb) * block, 2000 + 16 * bn);
}
long long tiles_of(int m, int n, int bn) { return static_cast<long long>((m + 255) / 256) * ((n + bn - 1) / bn); }

Tiling tiling(const Product& p, const Resident& resident) {
  Tiling t = {256, 1, -1};
  for (int bn = 256; bn >= 64; bn -= p.b_mn ? 128 : 64)
    for (int i = 0; i < 3 && (64 << i) <= bn && resident.tiles[i] > 0; ++i) {
      const int split = 1 << i;
      const long long rounds = (tiles_of(p.m, p.n, bn) + resident.tiles[i] - 1) / resident.tiles[i];
      const long long cost =
          rounds * (round_cost((p.kb + split - 1) / split, bn) + (split > 1 ? 4000 + 25 * bn : 0)) + 16 * bn;
      if (t.cost < 0 || cost < t.cost) t = {bn, split, cost};
    }
  return t;
}

// The widths of two products whose tiles the pairs walk in one launch (pair i
// takes tiles i, i + pairs, ...), and the longest pair's time.
constexpr int kLaunch = 8000;  // clocks that a launch of its own costs
struct TwoTilings {
  int bn[2];
  long long cost;
};
TwoTilings together(const Product& a, const Product& b, int pairs) {
  TwoTilings best = {{256, 256}, -1};
  for (int x = 256; x >= 128; x -= 128)
    for (int y = 256; y >= 128; y -= 128) {
      const long long na = tiles_of(a.m, a.n, x), nb = tiles_of(b.m, b.n, y);
      const long long ca = round_cost(a.kb, x), cb = round_cost(b.kb, y);
      long long longest = 0;
      for (int p = 0; p < pairs; ++p) {
        const long long mine_a = na > p ? (na - p + pairs - 1) / pairs : 0;
        const long long all = na + nb > p ? (na + nb - p + pairs - 1) / pairs : 0;
        longest = std::max(longest, mine_a * ca + (all - mine_a) * cb);
      }
      if (best.cost < 0 || longest < best.cost) best = {{x, y}, longest};
    }
  best.cost += 16 * 256;
  return best;
}

// A product and its operands' maps, ready to launch.
struct Ready {
  Product p;
  Matrix a, b;
};
template <typename T>
bool make_maps(const Ready& r, CUtensorMap* ma, CUtensorMap* mb) {
  // Operand tiles of 128 rows come as one box where the reduction runs along
  // them, as boxes of 64 x 64 where it runs down.
  return make_map(ma, r.a, Pair<T>::kBf16, r.p.a_mn ? kBlock : 2 * kBlock) &&
         make_map(mb, r.b, Pair<T>::kBf16, r.p.b_mn || r.p.bn <= 128 ? kBlock : 2 * kBlock);
}
template <typename T>
cudaError_t launch_pairs(Ready* r, int count, int pairs, uint32_t* flags, cudaStream_t stream) {
  CUtensorMap m[4];
  Products g;
  g.count = count;
  g.stage_bytes = 3 * kBlockBytes;
  g.bufs = 4;
  int tiles = 0;
  for (int i = 0; i < count; ++i) {
    Product& p = r[i].p;
    p.tiles_m = (p.m + 255) / 256;
    p.tiles_n = (p.n + p.bn - 1) / p.bn;
    p.share = (p.kb + p.split - 1) / p.split;
    // ceil(2^(32 + shift) / d) with 2^shift >= d gives t / d for t < 2^31; with
    // the shift one less the multiplier fits 32 bits, for t < 2^31 still.
    const uint64_t d = static_cast<uint64_t>(kGroupM) * p.tiles_n;
    p.group_shift = 0;
    while ((2ull << p.group_shift) < d) ++p.group_shift;
    p.group_inverse = static_cast<uint32_t>(((1ull << (32 + p.group_shift)) + d - 1) / d);
    tiles += p.tiles_m * p.tiles_n;
    if (p.bn > 128) {
      g.stage_bytes = 4 * kBlockBytes;
      g.bufs = 2;
    }
    if (!make_maps<T>(r[i], &m[2 * i], &m[2 * i + 1])) return cudaErrorInvalidValue;
    g.p[i] = p;
  }
  if (count == 1) {
    g.p[1] = g.p[0];
    m[2] = m[0];
    m[3] = m[1];
  }
  const int split = g.p[0].split;
  return launch_chained(product_pair_kernel<T>, dim3(2 * (split > 1 ? tiles * split : std::min(tiles, pairs))), kThreads,
                        kPairSmem, stream, 2 * split, m[0], m[1], m[2], m[3], g, flags);
}

template <typename T, int NT>
cudaError_t launch_few(const Matrix& w, bool w_mn, const Matrix& x, FewProduct p, uint32_t* flags,
                       cudaStream_t stream) {
  CUtensorMap mw, mx;
  if (!make_map(&mw, w, Pair<T>::kBf16, w_mn ? kBlock : 2 * kBlock) || !make_map(&mx, x, Pair<T>::kBf16, NT))
    return cudaErrorInvalidValue;
  auto kern = product_few_kernel<T, NT>;
  static std::atomic<bool> ready[kMaxDev];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, FewCfg<NT>::kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  const int across = (p.n + 127) / 128, down = (p.m + NT - 1) / NT;
  p.w_mn = w_mn;
  // Two CTAs on each SM, and at least four blocks of the reduction for each.
  p.split = 1;
  while (p.split < (NT > 32 ? kMaxSplit / 2 : kMaxSplit) && 2 * p.split * across * down <= 304 && p.kb >= 8 * p.split)
    p.split *= 2;
  return launch_chained(kern, dim3(across * p.split, down, 1), kFewThreads, FewCfg<NT>::kSmem, stream, p.split, mw, mx,
                        p, flags);
}

// The product D = A B^T over `depth`, with the epilogue e.  a: m x depth (or
// depth x m where a_mn), b likewise; rows on 16-byte boundaries.
Ready ready(int m, int n, int depth, const Matrix& a, bool a_mn, const Matrix& b, bool b_mn, Epilogue e) {
  e.vec = (e.bias && rows_aligned(e.bias, 0, 1) ? 1 : 0) | (e.res && rows_aligned(e.res, e.ldr, m) ? 2 : 0) |
          (e.pre && rows_aligned(e.pre, e.ldpre, m) ? 4 : 0) | (rows_aligned(e.out, e.ldo, m) ? 8 : 0);
  Product p = {};
  p.m = m;
  p.n = n;
  p.kb = (depth + kBlock - 1) / kBlock;
  p.a_mn = a_mn;
  p.b_mn = b_mn;
  p.bn = 256;
  p.split = 1;
  p.e = e;
  return {p, a, b};
}

// Whether the kernel for few rows takes a product: up to 128 rows, and up to
// 76 tiles of 128 x 128 with a reduction worth sharing.  128 rows of 4096 ->
// 4096 take it 15.5 us (pairs 18), 256 rows of 8192 -> 1024 15.7 (19.5); but
// 256 rows of 4096 -> 16384 41.7 (30).
bool few_rows(const Product& p) {
  const long long squares = static_cast<long long>((p.m + 127) / 128) * ((p.n + 127) / 128);
  return !p.a_mn && (p.m <= 128 || (squares <= 76 && p.kb >= 32));
}

template <typename T>
cudaError_t run_product(Ready r, uint32_t* flags, cudaStream_t stream) {
  Product& p = r.p;
  if (p.kb == 0) {
    const long long all = static_cast<long long>(p.m) * p.n;
    return launch_chained(empty_product_kernel<T>,
                          dim3(static_cast<unsigned>(std::min<long long>((all + 255) / 256, 4096))), 256, 0, stream, 0, p);
  }
  if (few_rows(p)) {
    const FewProduct f = {p.m, p.n, p.kb, 0, 1, p.e};
    return p.m <= 16   ? launch_few<T, 16>(r.b, p.b_mn, r.a, f, flags, stream)
           : p.m <= 32 ? launch_few<T, 32>(r.b, p.b_mn, r.a, f, flags, stream)
           : p.m <= 64 ? launch_few<T, 64>(r.b, p.b_mn, r.a, f, flags, stream)
                       : launch_few<T, 128>(r.b, p.b_mn, r.a, f, flags, stream);
  }
  Resident resident;
  const cudaError_t s = resident_clusters<T>(&resident);
  if (s != cudaSuccess) return s;
  const Tiling t = tiling(p, resident);
  p.bn = t.bn;
  p.split = t.split;
  return launch_pairs<T>(&r, 1, resident.tiles[0], flags, stream);
}

// Two products, in one launch where that is quicker: their tiles together fill
// the pairs better.  (1328 x 2048 -> 1024, dx and dw: 15.4 us, 21.7 apart.)
template <typename T>
cudaError_t run_products(Ready a, Ready b, uint32_t* flags, cudaStream_t stream) {
  if (a.p.kb > 0 && b.p.kb > 0 && !few_rows(a.p) && !few_rows(b.p)) {
    Resident resident;
    const cudaError_t s = resident_clusters<T>(&resident);
    if (s != cudaSuccess) return s;
    if (a.p.kb < b.p.kb) std::swap(a, b);  // the longer tiles first
    const TwoTilings t = together(a.p, b.p, resident.tiles[0]);
    if (t.cost < tiling(a.p, resident).cost + tiling(b.p, resident).cost + kLaunch) {
      a.p.bn = t.bn[0];
      b.p.bn = t.bn[1];
      Ready both[2] = {a, b};
      return launch_pairs<T>(both, 2, resident.tiles[0], flags, stream);
    }
  }
  const cudaError_t s = run_product<T>(a, flags, stream);
  return s != cudaSuccess ? s : run_product<T>(b, flags, stream);
}

template <typename T>
cudaError_t linear_t(const LinearCall& c, cudaStream_t stream) {
  Matrix x = {c.x, c.ldx, c.m, c.k}, w = {c.w, c.ldw, c.n, c.k};
  const cudaError_t s = align_operands(&x, &w, static_cast<uint8_t*>(c.ws), stream);
  if (s != cudaSuccess) return s;
  const Epilogue e = {c.bias, c.res, c.ldr, c.pre, c.ldpre, c.y, c.ldy, c.act, 0};
  return run_product<T>(ready(c.m, c.n, c.k, x, false, w, false, e), c.flags, stream);
}

// Row chunks of the slope pass: one where that is quick, else enough CTAs to
// fill the GPU.
constexpr int kFewSlopeRows = 256;
int slope_chunk(int m, int n) {
  if (m <= kFewSlopeRows) return kFewSlopeRows;
  const int across = (n + 255) / 256;
  const int chunks = std::max(1, std::min(256, 608 / across));
  return std::max(32, ((m + chunks - 1) / chunks + 7) / 8 * 8);
}

struct BackwardPlan {
  bool own_dz;  // dz is written to the workspace (else it is dy itself)
  int chunk, chunks;
  size_t dz, part, x, w;
};
BackwardPlan backward_plan(const LinearGradCall& c) {
  BackwardPlan p;
  p.own_dz = c.act != kActNone || !rows_aligned(c.dy, c.lddy, c.m);
  const size_t up = 255;
  p.dz = p.own_dz ? (static_cast<size_t>(c.m) * pad8(c.n) * 2 + up) & ~up : 0;
  p.chunk = slope_chunk(c.m, c.n);
  p.chunks = (c.m + p.chunk - 1) / p.chunk;
  p.part = p.chunks > 1 ? (static_cast<size_t>(p.chunks) * c.n * 4 + up) & ~up : 0;
  p.x = aligned_copy_bytes({c.x, c.ldx, c.m, c.k});
  p.w = aligned_copy_bytes({c.w, c.ldw, c.n, c.k});
  return p;
}

template <typename T, int kAct>
cudaError_t run_slope(const LinearGradCall& c, const BackwardPlan& p, T* dz, float* part, cudaStream_t stream) {
  const int vec = (rows_aligned(c.dy, c.lddy, c.m) ? 1 : 0) |
                  (kAct != kActNone && rows_aligned(c.pre, c.ldpre, c.m) ? 2 : 0);
  T* db = static_cast<T*>(c.db);
  const bool whole = p.chunks == 1;
  const int tx = c.m <= kFewSlopeRows ? 4 : 32;
  const cudaError_t s = launch_chained(
      tx == 4 ? slope_kernel<T, kAct, 4> : slope_kernel<T, kAct, 32>, dim3((c.n + 8 * tx - 1) / (8 * tx), p.chunks), 256,
      0, stream, 0, static_cast<const T*>(c.dy), c.lddy, static_cast<const T*>(c.pre), c.ldpre, dz, pad8(c.n),
      db && !whole ? part : nullptr, whole ? db : nullptr, c.m, c.n, p.chunk, vec);
  if (s != cudaSuccess || !db || whole) return s;
  return launch_chained(join_parts_kernel<T>, dim3((c.n + 31) / 32), 1024, 0, stream, 0, part, p.chunks, p.chunks, c.n,
                        db, nullptr);
}

template <typename T>
cudaError_t linear_backward_t(const LinearGradCall& c, cudaStream_t stream) {
  Matrix dz = {c.dy, c.lddy, c.m, c.n}, x = {c.x, c.ldx, c.m, c.k}, w = {c.w, c.ldw, c.n, c.k};
  cudaError_t s = cudaSuccess;
  if (c.m > 0 && c.n > 0) {
    const BackwardPlan plan = backward_plan(c);
    uint8_t* ws = static_cast<uint8_t*>(c.ws);
    T* own = nullptr;
    if (plan.own_dz && (c.dx || c.dw)) {
      own = reinterpret_cast<T*>(ws);
      dz = {own, pad8(c.n), c.m, c.n};
    }
    float* part = reinterpret_cast<float*>(ws + plan.dz);
    if (own || c.db) {
      switch (c.act) {
        case kActRelu: s = run_slope<T, kActRelu>(c, plan, own, part, stream); break;
        case kActGelu: s = run_slope<T, kActGelu>(c, plan, own, part, stream); break;
        case kActGeluTanh: s = run_slope<T, kActGeluTanh>(c, plan, own, part, stream); break;
        case kActSilu: s = run_slope<T, kActSilu>(c, plan, own, part, stream); break;
        default: s = run_slope<T, kActNone>(c, plan, own, part, stream); break;
      }
    }
    Matrix none = {nullptr, 0, 0, 0};
    if (s == cudaSuccess) s = align_operands(c.dw ? &x : &none, c.dx ? &w : &none, ws + plan.dz + plan.part, stream);
  } else if (c.db && c.n > 0) {
    s = launch_chained(join_parts_kernel<T>, dim3((c.n + 31) / 32), 1024, 0, stream, 0, nullptr, 0, 0, c.n,
                       static_cast<T*>(c.db), nullptr);
  }
  if (s != cudaSuccess) return s;
  Epilogue to_dx = {nullptr, nullptr, 0, nullptr, 0, c.dx, c.lddx, kActNone, 0}, to_dw = to_dx;
  to_dw.out = c.dw;
  to_dw.ldo = c.lddw;
  const bool want_dx = c.dx && c.m > 0 && c.k > 0, want_dw = c.dw && c.n > 0 && c.k > 0;
  const Ready dx = ready(c.m, c.k, c.n, dz, false, w, true, to_dx), dw = ready(c.n, c.k, c.m, dz, true, x, true, to_dw);
  if (want_dx && want_dw) return run_products<T>(dx, dw, c.flags, stream);
  if (want_dx) return run_product<T>(dx, c.flags, stream);
  if (want_dw) return run_product<T>(dw, c.flags, stream);
  return cudaSuccess;
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
