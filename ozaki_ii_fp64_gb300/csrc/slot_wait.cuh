// Waits of a group of threads for the slots of its ring in shared memory
// (layernorm.cu).
#pragma once

#include <cstdint>

#include "common.cuh"

namespace ozemu {

// Barrier of a group of TPR threads, one of the CTA's groups of that many.
template <int TPR>
__device__ __forceinline__ void row_barrier() {
  asm volatile("bar.sync %0, %1;" ::"r"(static_cast<int>(threadIdx.x) / TPR + 1), "n"(TPR) : "memory");
}

// Waits for a slot.  Each thread's wait gives up by itself (its limit, or the
// time-out of another CTA, may fall between the polls of two threads), but a
// group leaves its loop together or not at all: a thread that left alone would
// be missing from the others' shuffles and barriers.  One warp votes here.  A
// larger group notes the failure in `gave_up` and goes on, every thread of it,
// to its next barrier, after which group_goes_on tells all of them; that costs
// no barrier of its own.  The caller alternates two words for `gave_up`, zero
// at the start: a thread may be at the next turn's wait while another still
// reads this turn's.
template <int TPR>
__device__ __forceinline__ bool slot_wait(uint64_t* bar, uint32_t parity, volatile int* gave_up,
                                          volatile int* abort_word, uint32_t* flags,
                                          uint64_t limit_ns = kWaitLimitNs) {
  const bool ok = mbar_wait(bar, parity, abort_word, flags, limit_ns);
  if constexpr (TPR == 32) {
    return __all_sync(0xFFFFFFFFu, ok);
  } else {
    if (!ok) *gave_up = 1;
    return true;
  }
}

// Past the first barrier of the group's TPR threads after slot_wait: whether
// none of them gave up.
template <int TPR>
__device__ __forceinline__ bool group_goes_on(const volatile int* gave_up) {
  return TPR == 32 || *gave_up == 0;
}

// By the thread that issues a group's copies, when the group gives up: lets
// those in flight, of turns `turn` to issued - 1, land.
__device__ __forceinline__ void let_copies_land(uint64_t* full, int turn, int stages, int issued) {
  for (int i = turn; i < issued; ++i) {
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(&full[i % stages], (i / stages) & 1) && globaltimer() - t0 < kWaitLimitNs) {
    }
  }
}

}  // namespace ozemu
