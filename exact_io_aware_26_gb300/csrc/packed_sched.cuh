// packed_sched.cuh -- which tiles of packed sequences there are, what each has to visit, and how
// long ones are cut: the arithmetic of the work list of packed attention (packed_plan.cu).
// Also compiled for the host, where a test runs it over small problems.
//
// A sequence has n queries (rows q0 .. of q) over m keys (rows k0 .. of k and v); with the causal
// rule query i sees the keys j <= i + m - n.  Query tiles hold `tpt` tokens (all the query heads
// of a key head: tpt * G <= 128 rows), key tiles 128 keys.  A unit of the forward pass is a query
// tile, whose steps are the key tiles that some row of it sees; a unit of the backward pass is a
// key tile, whose steps are the query tiles that see some key of it.
#pragma once
#include <cstdint>

#ifndef __CUDACC__
#define __host__
#define __device__
#endif

namespace fa {

constexpr int kPackedKeys = 128;  // keys of a key tile

struct PackedSeq {
  int q0, n, k0, m;
};

// A CTA's work, for each key head: steps [s0, s1) of a unit; slot < 0 where these are all of the
// unit's, else the place of its partial result.  In the list of cut units s0 is the first slot
// and s1 the number of slots.
struct PackedItem {
  PackedSeq seq;
  int tile, s0, s1, slot;
};

__host__ __device__ inline int packed_units(const PackedSeq& s, int tpt, bool bwd) {
  return bwd ? (int)(((long long)s.m + kPackedKeys - 1) / kPackedKeys) : (int)(((long long)s.n + tpt - 1) / tpt);
}

// Steps [s0, s1) of unit `tile`; none (s0 = s1) where no query of it sees a key.
__host__ __device__ inline void packed_steps(const PackedSeq& s, int tile, int tpt, bool causal, bool bwd, int& s0,
                                             int& s1) {
  const long long ahead = (long long)s.m - s.n;  // keys before the first query's own
  if (!bwd) {
    long long end = s.m;  // keys that the tile's last row sees
    if (causal) {
      const long long last = (long long)(tile + 1) * tpt < s.n ? (long long)(tile + 1) * tpt : s.n;
      end = ahead + last;
    }
    s0 = 0;
    s1 = end <= 0 ? 0 : (int)((end + kPackedKeys - 1) / kPackedKeys);
    return;
  }
  s1 = (int)(((long long)s.n + tpt - 1) / tpt);
  s0 = 0;
  if (causal) {
    const long long first = (long long)tile * kPackedKeys - ahead;  // first query that sees the tile's first key
    if (first > 0) s0 = first >= s.n ? s1 : (int)(first / tpt);
  }
}

// Steps of a slice, so that `target` CTAs have even shares of `steps` steps of each of `heads` key
// heads, but at least `least`.  Units with more steps are cut: into c = ceil(w / P) < 2 w / P
// slices, so that all of them take fewer than 2 target / heads slots.
__host__ __device__ inline long long packed_slice(long long steps, int heads, int target, long long least) {
  const long long even = (steps * heads + target - 1) / target;
  return even > least ? even : least;
}
__host__ __device__ inline int packed_slots(int heads, int target) { return 2 * target / heads + 1; }
__host__ __device__ inline int packed_cuts(int w, long long slice) { return w <= slice ? 1 : (int)((w + slice - 1) / slice); }
// Slice i of w steps cut into c: first step and end.
__host__ __device__ inline void packed_cut(int w, int c, int i, int& a, int& b) {
  const int base = w / c, more = w % c;
  a = i * base + (i < more ? i : more);
  b = a + base + (i < more ? 1 : 0);
}

}  // namespace fa
