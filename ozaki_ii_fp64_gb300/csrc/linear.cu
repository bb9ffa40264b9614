// Linear layer with a fused epilogue, and its gradients, on tcgen05 kind::f16.
//
//   z = x w^T + b,  y = act(z) + r
//   dz = dy act'(pre),  dx = dz w,  dw = dz^T x,  db = sum over rows of dz
//
// and its gated form, whose w holds the rows of two layers, gate and up:
//
//   [g u] = x w^T + b,  h = act(g) u
//   dz = [dh u act'(g)  dh act(g)],  dx, dw, db as above
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
// f16.  Two 16-bit parts of dz would avoid it for twice the MMAs of both
// products.  In f16 dz can leave the type's range where the gradients do not.
// The gated layer's, products of three, are rounded times a power of two that
// brings the largest of them to 2^14 .. 2^15, and dx and dw have it taken out of
// their fp32 sums.  The plain layer's, dy times a slope, are rounded as they are:
// beyond 65504 (a slope is up to 1.13) they are infinite, below 2^-14 they keep
// 2^-25 absolutely, as dy itself does.  Sums in the tensor cores
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
#include "product.cuh"

namespace ozemu {

namespace {

constexpr int kBlock = 64;               // elements of an operand block: 64 rows of 64 (128 bytes)
constexpr int kBlockBytes = 64 * 128;
constexpr int kThreads = 32 * (3 + kEpiWarps);

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
// 6.5 us beyond its rounds; at 1000 x 2049 -> 4099, f16 with a residual (34 us),
// the copies of both odd operands cost 8 and the odd rows of y and the residual 2.
// ---------------------------------------------------------------------------
constexpr int kRing = 192 * 1024;  // stages of two blocks of A and one or two of B: 8 or 6
constexpr int kMaxStages = 8;
constexpr int kPairSmem = 1024 + kRing + kEpiWarps * (2048 + 64) + 256;  // staging, a chunk's bias, barriers
struct Product {
  int m, n;        // rows and columns of D
  int kb;          // 64-element blocks of the reduction
  int a_mn, b_mn;  // the operand's reduction runs down its rows
  int bn;          // columns of a tile
  int split;       // pairs that share a tile's reduction
  int share;       // blocks of it for each
  Raster tiles;
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

// The sums that a pair of a split tile leaves: 128 rows of up to 256 fp32, the
// 16-byte piece c of row r at piece c ^ (r % 32), so that a warp's rows meet
// in no bank.
__device__ __forceinline__ uint32_t part_piece(int r, int c) {
  return static_cast<uint32_t>(r * 1024 + ((c ^ (r & 31)) << 4));
}

// Whether a gated tile has an output whose rows have no alignment.
__device__ __forceinline__ bool gated_together(const Epilogue& e) {
  return (e.vec & 8) == 0 || (e.pre && (e.vec & 36) != 36);
}

// The same for a gated tile, from source(half, v): the gate's accumulators, half
// 0, and the up projection's.  One half's 32 values live at a time but for the
// product, so that writing rows has registers left.  `some`: whether this warp's
// columns exist (a quarter's warps come together); the tile's end at `end`.
template <typename T, typename F>
__device__ __forceinline__ void finish_gated(F source, bool some, const Epilogue& e, uint8_t* stage, uint8_t* bias,
                                             const Quarter& quarter, int row0, int col0, int m, int n, int end) {
  const int lane = threadIdx.x & 31;
  auto take = [&](float2 (&v)[16], int half) {
    source(half, v);
    if (e.bias) {  // the chunk's 32 values, for every lane
      const uint16_t b = col0 + lane < n ? static_cast<const uint16_t*>(e.bias)[half * n + col0 + lane] : 0;
      __syncwarp();
      reinterpret_cast<uint16_t*>(bias)[lane] = b;
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float2 f[4];
        unpack16<T>(reinterpret_cast<const uint4*>(bias)[q], f);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * q + i] = add2(v[4 * q + i], f[i]);
      }
    }
  };
  auto put = [&](const float2 (&v)[16]) {
    if (!some) return;
#pragma unroll
    for (int c = 0; c < 4; ++c) *stage_piece(stage, lane, c) = pack16<T>(v + 4 * c);
  };
  auto write = [&](void* to, long long ld, int at, int aligned) {
    if (e.vec & aligned) {
      __syncwarp();
      if (some) write_rows(stage, static_cast<T*>(to) + at, ld, row0, col0, m, n, true);
      __syncwarp();
    } else {
      quarter_sync(quarter);
      write_together(quarter, static_cast<T*>(to) + at, ld, row0, col0 - 32 * quarter.group, m, end);
      quarter_sync(quarter);
    }
  };
  float2 z[16];
  take(z, 0);
  if (e.pre) {
    put(z);
    write(e.pre, e.ldpre, 0, 4);
  }
  activate_all(z, e.act);
  {
    float2 u[16];
    take(u, 1);
    if (e.pre) put(u);
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = mul2(z[i], u[i]);
  }
  if (e.pre) write(e.pre, e.ldpre, n, 32);
  put(z);
  write(e.out, e.ldo, 0, 8);
}

// kGated: B holds the rows of two layers, gate (n of them) and up (n more), and
// D is m x n.  One CTA of a pair stages a tile's gate rows, the other as many
// up rows, so the accumulators of an output's two halves lie BN / 2 columns
// apart in the same TMEM lane and meet in one thread's registers: the gate and
// up products are never written unless they are kept for the backward pass.
template <typename T, bool kGated>
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
  const int first = g.p[0].tiles.count();  // tiles of the first product
  const int total = first + (g.count > 1 ? g.p[1].tiles.count() : 0);
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

  cluster_arrive();
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
      tile_of(second ? t - first : t, p.tiles, tm, tn);
      part(p, kb0, kb1);
      // B's BN / 2 rows of this CTA come in whole blocks (a part block's last
      // rows are loaded and not used).
      const int b_blocks = p.bn > 128 ? 2 : 1;
      const uint32_t bytes = 2 * (2 + b_blocks) * kBlockBytes;
      const bool arms = loads_a && rank == 0;  // for both CTAs and operands
      const bool down = loads_a ? p.a_mn != 0 : p.b_mn != 0;
      const bool two = down && (loads_a || b_blocks == 2);
      const int at = loads_a  ? tm * 256 + rank * 128
                     : kGated ? tn * (p.bn / 2) + rank * p.n
                              : tn * p.bn + rank * (p.bn / 2);
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
      tile_of(second ? t - first : t, p.tiles, tm, tn);
      const int buf = n_tiles & (g.bufs - 1), use = n_tiles >> buf_shift;
      const int row0 = tm * 256 + rank * 128 + quarter * 32;
      // Columns of the tile that this warp has to take: none past D's edge.
      const int width = kGated ? p.bn / 2 : p.bn;  // of the tile in D
      const int cols = row0 < p.m ? min(width, p.n - tn * width) : 0;
      const uint32_t tcol = tbase + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(buf * buf_columns);
      if (split > 1) {  // leave the sums; the cluster joins them below
        int kb0, kb1;
        part(p, kb0, kb1);
        if (!warp_wait(&tfull[buf], use & 1, abort_word, flags)) break;
        tc_fence_after();
        const int r = quarter * 32 + lane;
        const int sums = kGated && cols > 0 ? p.bn : cols;
        for (int c = group * 32; c < sums; c += 128) {
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
      if constexpr (kGated) {  // 128 columns or fewer: a chunk a warp
        const int c = group * 32;
        const bool some = c < cols, together = gated_together(e);
        const Quarter q = {staging + (ew & 3) * 2048, quarter, group};
        live = warp_wait(&tfull[buf], use & 1, abort_word, flags);
        if (together) live = quarter_all(q, live);
        if (!live) break;
        tc_fence_after();
        auto release = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(&tempty[buf], lead));
        };
        if (some || (together && cols > 0))
          finish_gated<T>(
              [&](int half, float2(&v)[16]) {
                uint32_t a[32];
                tmem_ld32(tcol + (half ? width : 0) + (some ? c : 0), a);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = make_float2(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1]));
                if (half) release();
              },
              some, e, stage, bias, q, row0, tn * width + c, p.m, p.n, min(p.n, (tn + 1) * width));
        else
          release();
        continue;
      }
#pragma unroll 1
      for (int c = group * 32; c < cols; c += 128) {
        const int col0 = tn * width + c;
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
        finish_rows<T, false>(
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
      tile_of(pair, p.tiles, tm, tn);
      const int width = kGated ? p.bn / 2 : p.bn;
      const int r0 = (warp - 2) * 8 + (lane >> 4), cols = min(width, p.n - tn * width);
      const long long grow0 = tm * 256 + rank * 128;
      for (int c = (place >> 1) * 64; c < cols; c += 64 * split) {
        const int piece = c / 4 + (lane & 15), col = tn * width + c + (lane & 15) * 4, left = p.n - col;
        if (left <= 0) continue;
        float b[4] = {0.f, 0.f, 0.f, 0.f};
        if (e.bias) load4(static_cast<const T*>(e.bias) + col, left, e.vec & 1, b);
        // The pairs' sums of a piece of four rows, in order.
        auto joined = [&](int piece, float(&z)[4][4]) {
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
        };
        float z[4][4] = {};
        joined(piece, z);
        if constexpr (kGated) {
          float u[4][4] = {}, bu[4] = {0.f, 0.f, 0.f, 0.f};
          joined(piece + width / 4, u);
          if (e.bias) load4(static_cast<const T*>(e.bias) + p.n + col, left, (e.vec & 16) != 0, bu);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const long long row = grow0 + r0 + 2 * i;
            if (row >= p.m) continue;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              z[i][k] += b[k];
              u[i][k] += bu[k];
            }
            if (e.pre) {
              store4(static_cast<T*>(e.pre) + row * e.ldpre + col, z[i], left, (e.vec & 4) != 0);
              store4(static_cast<T*>(e.pre) + row * e.ldpre + p.n + col, u[i], left, (e.vec & 32) != 0);
            }
            activate_all(z[i], e.act);
#pragma unroll
            for (int k = 0; k < 4; ++k) z[i][k] *= u[i][k];
            store4(static_cast<T*>(e.out) + row * e.ldo + col, z[i], left, (e.vec & 8) != 0);
          }
        } else {
          const float f = e.scale ? sums_scale(e) : 1.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const long long row = grow0 + r0 + 2 * i;
            if (row >= p.m) continue;
#pragma unroll
            for (int k = 0; k < 4; ++k) z[i][k] = z[i][k] * f + b[k];
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

// kGated: the MMA's 128 rows are 64 gate rows of the wide operand and the 64 up
// rows that belong to the same outputs, so a CTA's sums hold both halves.
template <typename T, int NT, bool kGated, bool kScaled>
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
  constexpr int kCols = kGated ? 64 : 128;  // of D
  const int j0 = blockIdx.x / p.split * kCols, i0 = blockIdx.y * NT;
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
        if (kGated) {
          tma_load_2d(st, &mw, &full[s], k0, j0);
          tma_load_2d(st + kBlockBytes, &mw, &full[s], k0, p.n + j0);
        } else if (p.w_mn) {
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

  join_few<T, kCols, false, kScaled>(smem, p.e, p.split, rank, j0, i0, min(NT, p.m - i0), p.n, kFewThreads);
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

// The same of a gated layer: out = act(bias of the gate) bias of up.
template <typename T>
__global__ void __launch_bounds__(256) empty_gated_kernel(const Product p) {
  chain_next();
  chain_wait();
  const Epilogue& e = p.e;
  const long long all = static_cast<long long>(p.m) * p.n;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < all; i += gridDim.x * 256LL) {
    const long long row = i / p.n;
    const int col = static_cast<int>(i % p.n);
    const T* b = static_cast<const T*>(e.bias);
    const float z = b ? to_float(b[col]) : 0.f, u = b ? to_float(b[p.n + col]) : 0.f;
    if (e.pre) {
      T* pre = static_cast<T*>(e.pre) + row * e.ldpre + col;
      pre[0] = from_float<T>(z);
      pre[p.n] = from_float<T>(u);
    }
    static_cast<T*>(e.out)[row * e.ldo + col] = from_float<T>(activate(z, e.act) * u);
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

// The aligned 16 bytes at `from`, of a matrix that lies from begin to end: what is
// not its memory is not read.
__device__ __forceinline__ uint4 load_aligned(uintptr_t from, uintptr_t begin, uintptr_t end) {
  if (from >= begin && from + 16 <= end) return __ldg(reinterpret_cast<const uint4*>(from));
  uint4 v = make_uint4(0, 0, 0, 0);
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uintptr_t at = from + 2 * i;
    if (at >= begin && at < end) w[i / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(at)) << (16 * (i & 1));
  }
  return v;
}
__device__ __forceinline__ uint4 from_next_lane(const uint4& v) {
  return make_uint4(__shfl_down_sync(0xFFFFFFFFu, v.x, 1), __shfl_down_sync(0xFFFFFFFFu, v.y, 1),
                    __shfl_down_sync(0xFFFFFFFFu, v.z, 1), __shfl_down_sync(0xFFFFFFFFu, v.w, 1));
}

// Stores eight consecutive elements of which `left` exist.  A warp whose first
// kRow lanes' elements follow each other stores vectors from the first boundary
// on, made of a lane's elements and the next one's, where p is on none; all of its
// lanes call this.
template <typename T, int kRow>
__device__ __forceinline__ void store8(T* p, int left, bool vec, const float2 (&v)[4]) {
  const uint4 mine = pack16<T>(v);
  if (vec) {
    if (left >= 8) {
      *reinterpret_cast<uint4*>(p) = mine;
      return;
    }
  } else if constexpr (kRow > 0) {
    const int lane = threadIdx.x & 31;
    const uint32_t off = 16 - static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);  // to the boundary
    const uint4 next = from_next_lane(mine);
    const int head = static_cast<int>(off) / 2;
    const bool joins = lane < kRow - 1 && left >= 16;
    if (joins) *reinterpret_cast<uint4*>(p + head) = shifted16(mine, next, off);
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // a head that the lane before does not take, a tail that does not join
      const float f = i & 1 ? v[i / 2].y : v[i / 2].x;
      if (i < left && (i < head ? lane == 0 || left < 8 : !joins)) p[i] = from_float<T>(f);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (2 * i < left) p[2 * i] = from_float<T>(v[i].x);
    if (2 * i + 1 < left) p[2 * i + 1] = from_float<T>(v[i].y);
  }
}

// The largest magnitude of dz = [dh u act'(g)  dh act(g)], of its finite values,
// for its scale: largest[CTA] of the grid's.  float16 only: the other type has
// fp32's range.  A CTA takes a strip of columns (every gridDim.x-th), a warp a row
// at a time, eight columns a lane: kVec, where rows start on 16-byte boundaries, 256
// of them, as they are; else 248, as in gated_slope_kernel.  Bound by HBM: 8192 x
// 8192 silu, 403 MB, 78 us (112 a row at a time); 8192 x 5330, rows of no alignment, 73.
constexpr int kLargestCtas = 152 * 4;
template <typename T, int kAct, bool kVec>
__global__ void __launch_bounds__(256, 4) gated_largest_kernel(const T* dh, long long lddh, const T* pre, long long ldpre,
                                                               float* largest, int m, int n) {
  constexpr int kOwn = kVec ? 32 : 31;
  __shared__ uint32_t red[8];
  chain_next();
  chain_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uintptr_t begin[2] = {reinterpret_cast<uintptr_t>(dh), reinterpret_cast<uintptr_t>(pre)};
  const uintptr_t stop[2] = {reinterpret_cast<uintptr_t>(dh + (m - 1) * lddh + n),
                             reinterpret_cast<uintptr_t>(pre + (m - 1) * ldpre + 2 * n)};
  const int step = 8 * gridDim.y;
  uint32_t most = 0;
  for (long long col0 = blockIdx.x * 8LL * kOwn; col0 < n; col0 += gridDim.x * 8LL * kOwn) {
    const int col = static_cast<int>(col0) + lane * 8, left = lane < kOwn ? n - col : 0;
    const T* at[3] = {dh + col, pre + col, pre + n + col};
#pragma unroll 1
    for (int row = blockIdx.y * 8 + warp; row < m; row += 2 * step) {
      uint4 u[2][3];  // two rows' loads before the first of them is needed
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int a = 0; a < 3; ++a) {
          const T* p = at[a] + (row + static_cast<long long>(r) * step) * (a == 0 ? lddh : ldpre);
          u[r][a] = make_uint4(0, 0, 0, 0);
          if (row + static_cast<long long>(r) * step >= m) continue;
          if constexpr (kVec) {  // (n is a multiple of 8)
            if (left > 0) u[r][a] = __ldg(reinterpret_cast<const uint4*>(p));
          } else {
            u[r][a] = load_aligned(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15), begin[a != 0], stop[a != 0]);
          }
        }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float2 v[3][4];
#pragma unroll
        for (int a = 0; a < 3; ++a) {
          if constexpr (!kVec) {
            const T* p = at[a] + (row + static_cast<long long>(r) * step) * (a == 0 ? lddh : ldpre);
            u[r][a] = shifted16(u[r][a], from_next_lane(u[r][a]), static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u);
          }
          unpack16<T>(u[r][a], v[a]);
        }
        auto take = [&](float f, bool some) {
          const uint32_t bits = __float_as_uint(f) & 0x7FFFFFFFu;
          if (some && bits < 0x7F800000u) most = max(most, bits);
        };
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float2 a, slope;
          activation_and_slope2<kAct>(v[1][q], a, slope);
          slope = mul2(mul2(v[0][q], v[2][q]), slope);
          a = mul2(v[0][q], a);
          take(slope.x, kVec || 2 * q < left);
          take(a.x, kVec || 2 * q < left);
          take(slope.y, kVec || 2 * q + 1 < left);
          take(a.y, kVec || 2 * q + 1 < left);
        }
      }
    }
  }
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (lane == 0) red[warp] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, red[i]);
    largest[blockIdx.y * gridDim.x + blockIdx.x] = __uint_as_float(most);
  }
}

// The power of two that brings the largest of those (parts of them) to 2^14 ..
// 2^15, the same for every thread of a CTA; 1 where all are 0.  The first CTA
// leaves its inverse.
__device__ __forceinline__ float gated_scale(const float* largest, int parts, float* inverse) {
  __shared__ uint32_t red[8];
  uint32_t most = 0;
  for (int i = threadIdx.x; i < parts; i += 256) most = max(most, __float_as_uint(__ldcg(largest + i)));
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = most;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) most = max(most, red[i]);
  // 2^s with s = 14 - floor(log2 most), within what has an inverse.
  const int exponent = most == 0 ? 127 : min(max(268 - static_cast<int>(most >> 23), 1), 253);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    *inverse = __uint_as_float(static_cast<uint32_t>(254 - exponent) << 23);
  return __uint_as_float(static_cast<uint32_t>(exponent) << 23);
}

// dz = [dh u act'(g)  dh act(g)] of the gated layer, rounded (where dz is given;
// rows of 2 n elements, lddz apart; float16 times gated_scale), and its column
// sums per chunk of rows as slope_kernel forms them: to part ([chunk][2 n]) or db.
// vec: bits 1 dh, 2 g, 4 u start on 16-byte boundaries, 8 so does dz's second
// half.  Rows of a warp's length (TX = 32) are a row ahead on their way: kWhole, where all of those do, as
// they are; else as the aligned vectors that they lie in, one a lane, whose
// elements a lane takes from its own and the next lane's, 31 lanes of them.
// Bound by HBM, three matrices read and two written: 8192 x 8192 bf16 silu 102 us,
// 6.6 TB/s (two rows ahead: 122, three: 140, in spilled registers); 11431 x 5330,
// rows of no alignment, 302 us by two vectors a lane as they are needed, 186 by
// the next lane's (which spills 8 to 44 bytes at the 80 registers of three CTAs an
// SM, 64 with float16's scale).
template <typename T, int kAct, int TX, bool kWhole>
__global__ void __launch_bounds__(256, 3) gated_slope_kernel(const T* dh, long long lddh, const T* pre, long long ldpre,
                                                             T* dz, long long lddz, float* part, T* db, int m, int n,
                                                             int chunk, int vec, const float* largest, int parts,
                                                             float* inverse) {
  constexpr bool kShifted = TX == 32 && !kWhole;
  constexpr bool kScaled = !Pair<T>::kBf16;
  constexpr int TY = 256 / TX, kOwn = kShifted ? 31 : TX, kCols = 8 * kOwn;
  __shared__ float red[TY][8 * TX + 8];
  chain_next();
  chain_wait();
  float scale = 1.f;
  auto find_scale = [&] {
    if (kScaled && dz) scale = gated_scale(largest, parts, inverse);
  };
  const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
  const int col = blockIdx.x * kCols + tx * 8, left = tx < kOwn ? n - col : 0;
  float2 sums[2][4] = {};
  const long long end = min(static_cast<long long>(m), (blockIdx.y + 1LL) * chunk);
  const long long first = static_cast<long long>(blockIdx.y) * chunk + ty;
  auto row = [&](long long i, float2(&d)[4], const float2(&g)[4], float2(&u)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float2 a, slope;
      activation_and_slope2<kAct>(g[q], a, slope);
      u[q] = mul2(mul2(d[q], u[q]), slope);
      d[q] = mul2(d[q], a);
      sums[0][q] = add2(sums[0][q], u[q]);
      sums[1][q] = add2(sums[1][q], d[q]);
    }
    if (dz) {
      if constexpr (kScaled) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          u[q] = mul2(u[q], both(scale));
          d[q] = mul2(d[q], both(scale));
        }
      }
      constexpr int kRow = TX == 32 ? kOwn : 0;
      store8<T, kRow>(dz + i * lddz + col, left, true, u);  // rows start on 16-byte boundaries
      store8<T, kRow>(dz + i * lddz + n + col, left, kWhole || (vec & 8), d);
    }
  };
  if constexpr (TX != 32) {
    find_scale();
    if (left > 0)
      for (long long i = first; i < end; i += TY) {
        float2 d[4], g[4], u[4];
        load8(dh + i * lddh + col, left, vec & 1, d);
        load8(pre + i * ldpre + col, left, vec & 2, g);
        load8(pre + i * ldpre + n + col, left, vec & 4, u);
        row(i, d, g, u);
      }
  } else {
    const T* at[3] = {dh + col, pre + col, pre + n + col};
    const uintptr_t begin[2] = {reinterpret_cast<uintptr_t>(dh), reinterpret_cast<uintptr_t>(pre)};
    const uintptr_t stop[2] = {reinterpret_cast<uintptr_t>(dh + (m - 1) * lddh + n),
                               reinterpret_cast<uintptr_t>(pre + (m - 1) * ldpre + 2 * n)};
    uint4 next[3];
    auto fetch = [&](long long i) {
      if (i >= end || (kWhole && left < 8)) return;  // (n is a multiple of 8 then)
#pragma unroll
      for (int a = 0; a < 3; ++a) {
        const T* p = at[a] + i * (a == 0 ? lddh : ldpre);
        if constexpr (kWhole)
          next[a] = __ldg(reinterpret_cast<const uint4*>(p));
        else
          next[a] = load_aligned(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15), begin[a != 0], stop[a != 0]);
      }
    };
    fetch(first);
    find_scale();
    for (long long i = first; i < end; i += TY) {
      float2 v[3][4];
#pragma unroll
      for (int a = 0; a < 3; ++a) {
        uint4 mine = next[a];
        if constexpr (!kWhole) {
          const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at[a] + i * (a == 0 ? lddh : ldpre))) & 15u;
          mine = shifted16(mine, from_next_lane(mine), off);
        }
        unpack16<T>(mine, v[a]);
      }
      fetch(i + TY);
      if (!kWhole || left >= 8) row(i, v[0], v[1], v[2]);
    }
  }
  if (!part && !db) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      red[ty][tx * 8 + 2 * q] = sums[h][q].x;
      red[ty][tx * 8 + 2 * q + 1] = sums[h][q].y;
    }
    __syncthreads();
    const int j = blockIdx.x * kCols + threadIdx.x;
    if (threadIdx.x < kCols && j < n) {
      float sum = 0.f;
#pragma unroll 8
      for (int y = 0; y < TY; ++y) sum += red[y][threadIdx.x];
      if (db)  // one chunk: the sum is whole
        db[static_cast<long long>(h) * n + j] = from_float<T>(sum);
      else
        part[(2LL * blockIdx.y + h) * n + j] = sum;
    }
  }
}

// ------------------------------------------------------------------- host

struct Matrix {
  const void* p;
  long long ld;
  int rows, cols;
};

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

// Tiles that can be worked on at once by clusters of one, two or four CTA
// pairs (a persistent grid must not exceed the first; the GPCs leave some SMs
// out of the larger clusters: 76, 36 and 15 on this GPU); sets the kernel's
// shared-memory size on the way.
struct Resident {
  int tiles[3] = {0, 0, 0};
};
template <typename T, bool kGated>
cudaError_t resident_clusters(Resident* out) {
  static Resident known[kMaxDev];
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (known[dev].tiles[0] == 0) {
    auto kern = product_pair_kernel<T, kGated>;
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
long long tiles_of(int m, long long n, int bn) { return static_cast<long long>((m + 255) / 256) * ((n + bn - 1) / bn); }

// A gated product's tiles have n / (bn / 2) columns, of 256 or 128: whole
// 64-column chunks of each half.
Tiling tiling(const Product& p, const Resident& resident, bool gated = false) {
  Tiling t = {256, 1, -1};
  for (int bn = 256; bn >= (gated ? 128 : 64); bn -= p.b_mn || gated ? 128 : 64)
    for (int i = 0; i < 3 && (64 << i) <= bn && resident.tiles[i] > 0; ++i) {
      const int split = 1 << i;
      const long long rounds =
          (tiles_of(p.m, gated ? 2LL * p.n : p.n, bn) + resident.tiles[i] - 1) / resident.tiles[i];
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
template <typename T, bool kGated>
cudaError_t launch_pairs(Ready* r, int count, int pairs, uint32_t* flags, cudaStream_t stream) {
  CUtensorMap m[4];
  Products g;
  g.count = count;
  g.stage_bytes = 3 * kBlockBytes;
  g.bufs = 4;
  int tiles = 0;
  for (int i = 0; i < count; ++i) {
    Product& p = r[i].p;
    const int width = kGated ? p.bn / 2 : p.bn;
    p.tiles = raster((p.m + 255) / 256, (p.n + width - 1) / width);
    p.share = (p.kb + p.split - 1) / p.split;
    tiles += p.tiles.count();
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
  return launch_chained(product_pair_kernel<T, kGated>, dim3(2 * (split > 1 ? tiles * split : std::min(tiles, pairs))), kThreads,
                        kPairSmem, stream, 2 * split, m[0], m[1], m[2], m[3], g, flags);
}

template <typename T, int NT, bool kGated>
cudaError_t launch_few(const Matrix& w, bool w_mn, const Matrix& x, FewProduct p, uint32_t* flags,
                       cudaStream_t stream) {
  CUtensorMap mw, mx;
  if (!make_map(&mw, w, Pair<T>::kBf16, w_mn || kGated ? kBlock : 2 * kBlock) || !make_map(&mx, x, Pair<T>::kBf16, NT))
    return cudaErrorInvalidValue;
  auto kern = product_few_kernel<T, NT, kGated, false>;
  if constexpr (!Pair<T>::kBf16 && !kGated)
    if (p.e.scale) kern = product_few_kernel<T, NT, kGated, true>;
  static std::atomic<bool> known[2][kMaxDev];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
  std::atomic<bool>& ready = known[p.e.scale != nullptr][dev];
  if (!ready) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, FewCfg<NT>::kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    ready = true;
  }
  const int across = kGated ? (p.n + 63) / 64 : (p.n + 127) / 128, down = (p.m + NT - 1) / NT;
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
  // A gated product's second halves start n elements on.
  const bool half = (n & 7) == 0;
  e.vec = (half && e.bias && rows_aligned(e.bias, 0, 1) ? 16 : 0) |
          (half && e.pre && rows_aligned(e.pre, e.ldpre, m) ? 32 : 0) |
          (e.bias && rows_aligned(e.bias, 0, 1) ? 1 : 0) | (e.res && rows_aligned(e.res, e.ldr, m) ? 2 : 0) |
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
// Of a gated layer up to 64 rows, whose sums it joins twice: 128 rows of 1024 -> 2 x
// 2048 from HBM 10.4 us (pairs 8.2), of 4096 -> 2 x 8192 32 (30), 64 rows 8.1 (8.0)
// and 28.4 (29.6).
bool few_rows(const Product& p, bool gated = false) {
  const long long squares =
      static_cast<long long>((p.m + 127) / 128) * (gated ? (p.n + 63) / 64 : (p.n + 127) / 128);
  return !p.a_mn && (p.m <= (gated ? 64 : 128) || (squares <= 76 && p.kb >= 32));
}

template <typename T, bool kGated = false>
cudaError_t run_product(Ready r, uint32_t* flags, cudaStream_t stream) {
  Product& p = r.p;
  if (p.kb == 0) {
    const long long all = static_cast<long long>(p.m) * p.n;
    return launch_chained(kGated ? empty_gated_kernel<T> : empty_product_kernel<T>,
                          dim3(static_cast<unsigned>(std::min<long long>((all + 255) / 256, 4096))), 256, 0, stream, 0, p);
  }
  if (few_rows(p, kGated)) {
    const FewProduct f = {p.m, p.n, p.kb, 0, 1, p.e};
    return p.m <= 16   ? launch_few<T, 16, kGated>(r.b, p.b_mn, r.a, f, flags, stream)
           : p.m <= 32 ? launch_few<T, 32, kGated>(r.b, p.b_mn, r.a, f, flags, stream)
           : p.m <= 64 ? launch_few<T, 64, kGated>(r.b, p.b_mn, r.a, f, flags, stream)
                       : launch_few<T, 128, kGated>(r.b, p.b_mn, r.a, f, flags, stream);
  }
  Resident resident;
  const cudaError_t s = resident_clusters<T, kGated>(&resident);
  if (s != cudaSuccess) return s;
  const Tiling t = tiling(p, resident, kGated);
  p.bn = t.bn;
  p.split = t.split;
  return launch_pairs<T, kGated>(&r, 1, resident.tiles[0], flags, stream);
}

// Two products, in one launch where that is quicker: their tiles together fill
// the pairs better.  (1328 x 2048 -> 1024, dx and dw: 15.4 us, 21.7 apart.)
template <typename T>
cudaError_t run_products(Ready a, Ready b, uint32_t* flags, cudaStream_t stream) {
  if (a.p.kb > 0 && b.p.kb > 0 && !few_rows(a.p) && !few_rows(b.p)) {
    Resident resident;
    const cudaError_t s = resident_clusters<T, false>(&resident);
    if (s != cudaSuccess) return s;
    if (a.p.kb < b.p.kb) std::swap(a, b);  // the longer tiles first
    const TwoTilings t = together(a.p, b.p, resident.tiles[0]);
    if (t.cost < tiling(a.p, resident).cost + tiling(b.p, resident).cost + kLaunch) {
      a.p.bn = t.bn[0];
      b.p.bn = t.bn[1];
      Ready both[2] = {a, b};
      return launch_pairs<T, false>(both, 2, resident.tiles[0], flags, stream);
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
int slope_chunk(int m, int n, int ctas, int least) {
  if (m <= kFewSlopeRows) return kFewSlopeRows;
  const int across = (n + 255) / 256;
  const int chunks = std::max(1, std::min(256, ctas / across));
  return std::max(least, ((m + chunks - 1) / chunks + 7) / 8 * 8);
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
  p.chunk = slope_chunk(c.m, c.n, 152 * 4, 32);
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

// dx = dz w and dw = dz^T x, with dz of n columns, times a number in memory (NULL: 1).
template <typename T>
cudaError_t grad_products(const LinearGradCall& c, int n, const Matrix& dz, const Matrix& x, const Matrix& w,
                          const float* scale, cudaStream_t stream) {
  Epilogue to_dx = {nullptr, nullptr, 0, nullptr, 0, c.dx, c.lddx, kActNone, 0, false, scale}, to_dw = to_dx;
  to_dw.out = c.dw;
  to_dw.ldo = c.lddw;
  const bool want_dx = c.dx && c.m > 0 && c.k > 0, want_dw = c.dw && n > 0 && c.k > 0;
  const Ready dx = ready(c.m, c.k, n, dz, false, w, true, to_dx), dw = ready(n, c.k, c.m, dz, true, x, true, to_dw);
  if (want_dx && want_dw) return run_products<T>(dx, dw, c.flags, stream);
  if (want_dx) return run_product<T>(dx, c.flags, stream);
  if (want_dw) return run_product<T>(dw, c.flags, stream);
  return cudaSuccess;
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
  return s == cudaSuccess ? grad_products<T>(c, c.n, dz, x, w, nullptr, stream) : s;
}

// ------------------------------------------------------- the gated layer's

template <typename T>
cudaError_t gated_t(const LinearCall& c, cudaStream_t stream) {
  Matrix x = {c.x, c.ldx, c.m, c.k}, w = {c.w, c.ldw, 2 * c.n, c.k};
  const cudaError_t s = align_operands(&x, &w, static_cast<uint8_t*>(c.ws), stream);
  if (s != cudaSuccess) return s;
  const Epilogue e = {c.bias, nullptr, 0, c.pre, c.ldpre, c.y, c.ldy, c.act, 0};
  return run_product<T, true>(ready(c.m, c.n, c.k, x, false, w, false, e), c.flags, stream);
}

struct GatedPlan {
  int chunk, chunks;
  size_t dz, part, x, w;
};
// What the CTAs find largest, and, in a line of its own, the scale's inverse.
constexpr size_t kScaleBytes = (kLargestCtas * sizeof(float) + 255) / 256 * 256 + 256;
GatedPlan gated_plan(const LinearGradCall& c) {
  GatedPlan p;
  const size_t up = 255;
  p.dz = (static_cast<size_t>(c.m) * pad8(2 * c.n) * 2 + up) & ~up;
  p.chunk = slope_chunk(c.m, c.n, 152 * 3, 16);
  p.chunks = (c.m + p.chunk - 1) / p.chunk;
  p.part = p.chunks > 1 ? (static_cast<size_t>(p.chunks) * 2 * c.n * 4 + up) & ~up : 0;
  p.x = aligned_copy_bytes({c.x, c.ldx, c.m, c.k});
  p.w = aligned_copy_bytes({c.w, c.ldw, 2 * c.n, c.k});
  return p;
}

template <typename T, int kAct>
cudaError_t run_gated_slope(const LinearGradCall& c, const GatedPlan& p, T* dz, float* part, float* largest, float* inverse,
                            cudaStream_t stream) {
  const bool half = (c.n & 7) == 0, pre = rows_aligned(c.pre, c.ldpre, c.m);
  const int vec = (rows_aligned(c.dy, c.lddy, c.m) ? 1 : 0) | (pre ? 2 : 0) | (pre && half ? 4 : 0) | (half ? 8 : 0);
  T* db = static_cast<T*>(c.db);
  const bool whole = p.chunks == 1;
  const int tx = c.m <= kFewSlopeRows ? 4 : 32, cols = tx == 4 ? 32 : vec == 15 ? 256 : 248;
  int parts = 0;
  if constexpr (!Pair<T>::kBf16) {
    if (dz) {
      const bool whole_rows = (vec & 7) == 7;
      const int across = std::min(kLargestCtas, (c.n - 1) / (whole_rows ? 256 : 248) + 1);
      const int down = std::max(1, std::min(kLargestCtas / across, (c.m - 1) / 8 + 1));
      parts = across * down;
      const cudaError_t s = launch_chained(
          whole_rows ? gated_largest_kernel<T, kAct, true> : gated_largest_kernel<T, kAct, false>, dim3(across, down), 256,
          0, stream, 0, static_cast<const T*>(c.dy), c.lddy, static_cast<const T*>(c.pre), c.ldpre, largest, c.m, c.n);
      if (s != cudaSuccess) return s;
    }
  }
  const cudaError_t s = launch_chained(
      tx == 4     ? gated_slope_kernel<T, kAct, 4, false>
      : vec == 15 ? gated_slope_kernel<T, kAct, 32, true>
                  : gated_slope_kernel<T, kAct, 32, false>,
      dim3((c.n + cols - 1) / cols, p.chunks), 256, 0, stream, 0, static_cast<const T*>(c.dy), c.lddy,
      static_cast<const T*>(c.pre), c.ldpre, dz, pad8(2 * c.n), db && !whole ? part : nullptr, whole ? db : nullptr, c.m,
      c.n, p.chunk, vec, static_cast<const float*>(largest), parts, inverse);
  if (s != cudaSuccess || !db || whole) return s;
  return launch_chained(join_parts_kernel<T>, dim3((2 * c.n + 31) / 32), 1024, 0, stream, 0, part, p.chunks, p.chunks,
                        2 * c.n, db, nullptr);
}

template <typename T>
cudaError_t gated_backward_t(const LinearGradCall& c, cudaStream_t stream) {
  Matrix dz = {nullptr, pad8(2 * c.n), c.m, 2 * c.n}, x = {c.x, c.ldx, c.m, c.k}, w = {c.w, c.ldw, 2 * c.n, c.k};
  float* inverse = nullptr;
  cudaError_t s = cudaSuccess;
  if (c.m > 0 && c.n > 0) {
    const GatedPlan plan = gated_plan(c);
    uint8_t* ws = static_cast<uint8_t*>(c.ws);
    T* own = c.dx || c.dw ? reinterpret_cast<T*>(ws) : nullptr;
    dz.p = own;
    float* part = reinterpret_cast<float*>(ws + plan.dz);
    float* largest = reinterpret_cast<float*>(ws + plan.dz + plan.part + plan.x + plan.w);
    if (!Pair<T>::kBf16 && own) inverse = largest + (kScaleBytes - 256) / sizeof(float);
    switch (c.act) {
      case kActRelu: s = run_gated_slope<T, kActRelu>(c, plan, own, part, largest, inverse, stream); break;
      case kActGelu: s = run_gated_slope<T, kActGelu>(c, plan, own, part, largest, inverse, stream); break;
      case kActGeluTanh: s = run_gated_slope<T, kActGeluTanh>(c, plan, own, part, largest, inverse, stream); break;
      case kActSilu: s = run_gated_slope<T, kActSilu>(c, plan, own, part, largest, inverse, stream); break;
      default: s = run_gated_slope<T, kActNone>(c, plan, own, part, largest, inverse, stream); break;
    }
    Matrix none = {nullptr, 0, 0, 0};
    if (s == cudaSuccess) s = align_operands(c.dw ? &x : &none, c.dx ? &w : &none, ws + plan.dz + plan.part, stream);
  } else if (c.db && c.n > 0) {
    s = launch_chained(join_parts_kernel<T>, dim3((2 * c.n + 31) / 32), 1024, 0, stream, 0, nullptr, 0, 0, 2 * c.n,
                       static_cast<T*>(c.db), nullptr);
  }
  return s == cudaSuccess ? grad_products<T>(c, 2 * c.n, dz, x, w, inverse, stream) : s;
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

size_t gated_linear_workspace(const LinearCall& c) {
  return aligned_copy_bytes({c.x, c.ldx, c.m, c.k}) + aligned_copy_bytes({c.w, c.ldw, 2 * c.n, c.k});
}

cudaError_t launch_gated_linear(const LinearCall& c, cudaStream_t stream) {
  return c.type == kF16 ? gated_t<__half>(c, stream) : gated_t<__nv_bfloat16>(c, stream);
}

size_t gated_linear_backward_workspace(const LinearGradCall& c) {
  const GatedPlan p = gated_plan(c);
  return p.dz + p.part + p.x + p.w + kScaleBytes;
}

cudaError_t launch_gated_linear_backward(const LinearGradCall& c, cudaStream_t stream) {
  return c.type == kF16 ? gated_backward_t<__half>(c, stream) : gated_backward_t<__nv_bfloat16>(c, stream);
}

}  // namespace ozemu
