// Checks the work list's arithmetic of packed attention (packed_sched.cuh) on the CPU: every
// unit's steps against the pairs that a causal or full mask leaves, slices that divide them, and
// the bounds that the workspace's sizes rest on.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "../exact_io_aware_26_gb300/csrc/packed_sched.cuh"

using namespace fa;

static void fail(const char* what, const PackedSeq& s, int tile, int tpt) {
  std::printf("%s: n %d m %d tile %d tpt %d\n", what, s.n, s.m, tile, tpt);
  std::exit(1);
}

static bool sees(const PackedSeq& s, bool causal, int i, int j) { return !causal || j <= i + s.m - s.n; }

int main() {
  const int kTpt[] = {128, 64, 42, 25, 16, 1};
  long long checked = 0;
  for (int tpt : kTpt)
    for (int n : {0, 1, 2, 15, 16, 17, 64, 127, 128, 129, 200, 300})
      for (int m : {0, 1, 2, 100, 127, 128, 129, 256, 300, 513})
        for (int causal = 0; causal < 2; ++causal) {
          const PackedSeq s{0, n, 0, m};
          const int nq = packed_units(s, tpt, false), nk = packed_units(s, tpt, true);
          if (nq != (n + tpt - 1) / tpt || nk != (m + 127) / 128) fail("units", s, -1, tpt);
          std::vector<char> seen(nq * nk + 1, 0);
          for (int i = 0; i < n; ++i)
            for (int j = 0; j < m; ++j)
              if (sees(s, causal, i, j)) seen[i / tpt * nk + j / 128] = 1;
          for (int bwd = 0; bwd < 2; ++bwd)
            for (int t = 0; t < (bwd ? nk : nq); ++t) {
              int a, b;
              packed_steps(s, t, tpt, causal, bwd, a, b);
              if (a < 0 || a > b || b > (bwd ? nq : nk)) fail("range", s, t, tpt);
              for (int u = 0; u < (bwd ? nq : nk); ++u)
                if ((bool)seen[bwd ? u * nk + t : t * nk + u] != (u >= a && u < b)) fail(bwd ? "key tile" : "query tile", s, t, tpt);
              ++checked;
            }
        }
  // slices, and what the workspace has to hold
  std::mt19937 rng(1);
  for (int round = 0; round < 20000; ++round) {
    const int R = 1 + rng() % 20, heads = 1 + rng() % (round % 5 == 0 ? 700 : 16), target = 1 + rng() % 320;
    const int tpt = kTpt[rng() % 6];
    const bool bwd = rng() % 2, causal = rng() % 2;
    const int least = 1 + rng() % 6;
    std::vector<int> work;
    long long all = 0, rows = 0;
    for (int r = 0; r < R; ++r) {
      const PackedSeq s{0, (int)(rng() % 3000), 0, (int)(rng() % 5000)};
      rows += bwd ? s.m : s.n;
      for (int t = 0; t < packed_units(s, tpt, bwd); ++t) {
        int a, b;
        packed_steps(s, t, tpt, causal, bwd, a, b);
        work.push_back(b - a);
        all += b - a;
      }
    }
    int longest = 0;
    for (int w : work) longest = w > longest ? w : longest;
    const float even = packed_even(all, heads, target);
    for (int k = 0; k < kPackedCandidates; ++k) {
      // a call weighs the candidates only where some unit is longer than the shortest of them
      if (k > 0 && !(longest > least && (float)longest > 0.75f * even)) break;
      const int slice = packed_candidate(k, even, least, longest);
      if (slice > longest || (slice < least && slice < longest)) fail("candidate", PackedSeq{}, slice, longest);
      long long slots = 0, items = 0, cut = 0;
      for (int w : work) {
        const int c = packed_cuts(w, slice);
        int at = 0;
        for (int i = 0; i < c; ++i) {
          int a, b;
          packed_cut(w, c, i, a, b);
          const int want = c == 1 ? w : i < w % c ? w / c + 1 : w / c;
          if (a != at || b - a > slice || b - a != want || (w > 0 && b <= a)) fail("slice", PackedSeq{}, w, c);
          at = b;
        }
        if (at != w) fail("slices", PackedSeq{}, w, c);
        items += c;
        if (c > 1) slots += c, ++cut;
      }
      const long long most = packed_slots(heads, target);
      if (slots > most || cut > most / 2 || items > rows / (bwd ? 128 : tpt) + R + most) fail("capacity", PackedSeq{}, R, target);
      if (!(packed_time(slice, (int)items, (int)slots, even, packed_even(1, heads, target)) > 0.f)) fail("time", PackedSeq{}, slice, longest);
    }
    ++checked;
  }
  std::printf("ok %lld\n", checked);
  return 0;
}
