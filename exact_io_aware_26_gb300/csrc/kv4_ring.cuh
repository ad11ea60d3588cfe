// kv4_ring.cuh -- a warp's ring of bulk copies: which stage's copy is the coming one, with
// which parity its barrier completes, and, after a wait that gave up, which stages still have
// a copy under way.  Also compiled for the host, where a test runs it through every order of
// copies, consumed units and waits that give up.
#pragma once
#include <cstdint>

#ifndef __CUDACC__
#define __host__
#define __device__
#endif

namespace fa {

// A stage's word: bit h for a block h of its unit that is not read, or kStageIdle alone where
// no copy is under way and none has landed that is still to be consumed.
constexpr uint32_t kStageIdle = 4;

template <int S>
struct Ring {
  int stage = 0;        // of the coming unit
  uint32_t parity = 0;  // of the phase in which its copy lands
  // the coming unit has been consumed
  __host__ __device__ inline void next() {
    if (++stage == S) {
      stage = 0;
      parity ^= 1u;
    }
  }
  // Calls f(stage, parity) for each stage with a copy under way, in the order of their arming.
  template <class F>
  __host__ __device__ inline void each_armed(const volatile uint32_t* words, F f) const {
    for (int k = 0; k < S; ++k) {
      const bool around = stage + k >= S;
      const int s = around ? stage + k - S : stage + k;
      if (!(words[s] & kStageIdle)) f(s, around ? parity ^ 1u : parity);
    }
  }
};

}  // namespace fa
