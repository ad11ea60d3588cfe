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
// unit's, else the place of its partial result, one of `parts` from slot `first` on of the unit that was
// cut as the `cut`-th.  r: which sequence.
struct alignas(16) PackedItem {
  PackedSeq seq;
  int tile, s0, s1, slot;
  int first, parts, cut, r;
};

// n, m and tile * tpt are at most 2^30, so that all of this fits an int.
__host__ __device__ inline int packed_units(const PackedSeq& s, int tpt, bool bwd) {
  return bwd ? (s.m + kPackedKeys - 1) / kPackedKeys : (s.n + tpt - 1) / tpt;
}

// Steps [s0, s1) of unit `tile`; none (s0 = s1) where no query of it sees a key.
__host__ __device__ inline void packed_steps(const PackedSeq& s, int tile, int tpt, bool causal, bool bwd, int& s0,
                                             int& s1) {
  const int ahead = s.m - s.n;  // keys before the first query's own
  s0 = 0;
  if (!bwd) {
    int end = s.m;  // keys that the tile's last row sees
    if (causal) end = ahead + ((tile + 1) * tpt < s.n ? (tile + 1) * tpt : s.n);
    s1 = end <= 0 ? 0 : (int)(((unsigned)end + kPackedKeys - 1) / kPackedKeys);
    return;
  }
  s1 = (s.n + tpt - 1) / tpt;
  if (causal) {
    const int first = tile * kPackedKeys - ahead;  // first query that sees the tile's first key
    if (first > 0) s0 = first >= s.n ? s1 : first / tpt;
  }
}

// How long a slice is.  `even` is what each of `target` CTAs would have of all units' steps, times the
// key heads.  A launch takes about as long as its longest slice and its start where all slices
// run at once (a few more stand behind the shortest of them), and otherwise as an even share of
// the steps and of the slices' starts, and half of the longest one behind it; parts of cut units
// cost their fp32 sums, and their join.  Candidates from 3/4 of `even` on are weighed (and the
// longest unit's steps: nothing cut), the longer of equals first.  The constants, in steps, are from
// sweeps: 8 requests of up to 512 rows over up to 8192 keys take 65 us cut at 30 or 33 steps, 73 at 27,
// 84 at 18 and 22, 70 at 38 and 89 uncut; 4 causal sequences of up to 2048 30 uncut and 34, 35 and 39
// cut at 13, 12 and 10 of 14 steps.
constexpr int kPackedCandidates = 32;
constexpr float kPackedStart = 4.f, kPackedJoin = 2.f, kPackedPart = 1.5f;
__host__ __device__ inline float packed_even(long long steps, int heads, int target) {
  return (float)steps * (float)heads / (float)target;
}
__host__ __device__ inline int packed_candidate(int k, float even, int least, int longest) {
  if (k == 0) return longest;
  const float p = even * (float)(kPackedCandidates - 1 - k + 12) * (1.f / 16.f);  // 2.6 to 3/4 of it
  const int up = p < (float)longest ? (int)p + 1 : longest;
  const int floor_ = least < longest ? least : longest;
  return up < floor_ ? floor_ : up > longest ? longest : up;
}
__host__ __device__ inline int packed_cuts(int w, int slice) { return w <= slice ? 1 : (w + slice - 1) / slice; }
// share: key heads for each of the target's CTAs, so that slices * share is the slices that each has.
__host__ __device__ inline float packed_time(int slice, int slices, int parts, float even, float share) {
  const float join = parts > 0 ? kPackedJoin + (float)parts * share * kPackedPart : 0.f;
  if ((float)slices * share <= 1.1f) return (float)slice + kPackedStart + join;
  return even + (float)slices * share * kPackedStart + 0.5f * (float)slice + join;
}
// A unit that is cut into c = ceil(w / P) slices has w > P, so that c < 2 w / P; with P at least 3/4 of
// the even share all cut units take fewer than 8/3 target / heads slots.
__host__ __device__ inline int packed_slots(int heads, int target) { return 8 * target / (3 * heads) + 1; }
// Slice i of w steps cut into c: first step and end.
__host__ __device__ inline void packed_cut(int w, int c, int i, int& a, int& b) {
  const int base = w / c, more = w % c;
  a = i * base + (i < more ? i : more);
  b = a + base + (i < more ? 1 : 0);
}

}  // namespace fa
