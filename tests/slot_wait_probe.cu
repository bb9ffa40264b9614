// Groups of threads that wait for a slot, some threads of them on one that is
// never filled (a wait of `limit_ns`).  Group 0's slot is filled; in group 1
// the threads with (threadIdx.x & mask) == value wait for the empty one.
// out: per group, the threads that left and those that went on, their sums
// over the group, and the flag word.
#include <cstdint>
#include <cuda_runtime.h>

#include "slot_wait.cuh"

using namespace ozemu;

template <int TPR>
__global__ void __launch_bounds__(2 * TPR) probe_kernel(int mask, int value, unsigned long long limit_ns, int* out,
                                                        uint32_t* flags) {
  __shared__ uint64_t bars[2];
  __shared__ int gave_up[2][2], abort_word, sums[2][32];
  const int tid = threadIdx.x % TPR, group = threadIdx.x / TPR;
  if (threadIdx.x == 0) {
    mbar_init(&bars[0], 1);
    mbar_init(&bars[1], 1);
    fence_mbar_init();
    mbar_arrive(&bars[0]);
    abort_word = 0;
  }
  if (tid < 2) gave_up[group][tid] = 0;
  __syncthreads();
  const bool empty = group == 1 && (tid & mask) == value;
  bool on = slot_wait<TPR>(&bars[empty ? 1 : 0], 0, &gave_up[group][0], &abort_word, flags, limit_ns);
  int sum = 0;
  if (on) {  // what a row does next: shuffles and, for several warps, a barrier
    int v = 1;
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (TPR > 32) {
      if ((threadIdx.x & 31) == 0) sums[group][tid >> 5] = v;
      row_barrier<TPR>();
      v = 0;
      for (int w = 0; w < TPR / 32; ++w) v += sums[group][w];
    }
    sum = v;
    on = group_goes_on<TPR>(&gave_up[group][0]);
  }
  atomicAdd(&out[2 * group + (on ? 1 : 0)], 1);
  if (on && tid == 0) out[4 + group] = sum;
}

extern "C" int probe(int tpr, int mask, int value, unsigned long long limit_ns, int* result) {
  int* out = nullptr;  // 6 counters and the flag word
  cudaError_t e = cudaMalloc(&out, 32);
  if (e == cudaSuccess) e = cudaMemset(out, 0, 32);
  if (e == cudaSuccess) {
    uint32_t* flags = reinterpret_cast<uint32_t*>(out + 6);
    switch (tpr) {
      case 32: probe_kernel<32><<<1, 64>>>(mask, value, limit_ns, out, flags); break;
      case 128: probe_kernel<128><<<1, 256>>>(mask, value, limit_ns, out, flags); break;
      default: probe_kernel<512><<<1, 1024>>>(mask, value, limit_ns, out, flags); break;
    }
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = cudaMemcpy(result, out, 28, cudaMemcpyDeviceToHost);
  cudaFree(out);
  return static_cast<int>(e);
}
