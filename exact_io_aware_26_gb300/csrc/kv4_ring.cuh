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

// A stage's word: bit h for a block h of its unit that is not read, or kStageIdle where there was
// no unit left to copy.
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
  // Units that have a copy, of those that the stages were last filled for.
  __host__ __device__ inline int armed(const uint32_t* words) const {
    int n = 0;
    while (n < S && !(words[(stage + n) % S] & kStageIdle)) ++n;
    return n;
  }
  // Calls f(stage, parity) for the coming n units, n <= S.
  template <class F>
  __host__ __device__ inline void each(int n, F f) const {
    for (int k = 0; k < n; ++k) {
      const bool around = stage + k >= S;
      f(around ? stage + k - S : stage + k, around ? parity ^ 1u : parity);
    }
  }
};

}  // namespace fa
