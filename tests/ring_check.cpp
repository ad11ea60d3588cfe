// Checks the ring of bulk copies of a warp of the cache's attention (kv4_ring.cuh) on the
// CPU against a model of its barriers: random tiles and rings, with a wait that gives up at
// every unit in turn.  The order of arming, consuming, keeping a stage for the join and giving
// up is that of the kernel's unit loop.  Held: a stage is armed only when its last copy has
// been consumed; every wait names the phase that the stage's copy completes; a stage that is
// written for the join has no copy under way; after a wait that gave up nothing is armed, and
// the drain names every stage with a copy under way once, with its phase, and no other (it
// would wait for a copy that nobody issued); a run without one ends with nothing under way.
// Usage: ring_check   (exit status 0 when every check holds)
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "kv4_ring.cuh"

using namespace fa;

#define CHECK(c)                                                           \
  do {                                                                     \
    if (!(c)) {                                                            \
      std::fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #c); \
      std::exit(1);                                                        \
    }                                                                      \
  } while (0)

// A barrier with one arrival: its phase completes when the copy that was armed lands.
struct Barrier {
  int phase = 0;
  bool armed = false;
  void arm() {
    CHECK(!armed);
    armed = true;
  }
  void land() {
    CHECK(armed);
    armed = false;
    ++phase;
  }
  bool done(uint32_t parity) const { return (uint32_t)(phase & 1) != parity; }
};

// One warp over its units of each tile; `across`: copies of the next tile go on during the
// join.  give_up: the unit whose wait gives up, or -1.  warp_fails: the wait is this warp's, or
// else another warp's in the same tile (it learns of it at the tile's end).
template <int S>
int run(const std::vector<int>& tiles, bool across, int give_up, bool warp_fails, std::mt19937& rng) {
  uint32_t words[S];
  for (auto& w : words) w = (uint32_t)(rng() % 8);  // whatever shared memory holds
  Barrier bars[S];
  std::vector<int> in(S, -1);  // unit of a stage: armed or landed, -1 when consumed
  Ring<S> at;
  int left = 0, issued = 0, consumed = 0, left_of_tile = 0;
  for (int n : tiles) left += n;
  bool stopped = false;
  auto land_some = [&] {
    // copies land in any order
    for (int s = 0; s < S; ++s)
      if (bars[s].armed && rng() % 2) bars[s].land();
  };
  auto produce = [&](int s) {
    CHECK(!stopped);
    if (across ? left == 0 : left_of_tile == 0) {
      if (across) words[s] = kStageIdle;
      return;
    }
    CHECK(in[s] == -1);
    bars[s].arm();
    in[s] = issued++;
    words[s] = (uint32_t)(rng() % 4);
    --left;
    --left_of_tile;
  };
  auto drain = [&](int n) {
    stopped = true;
    CHECK(n <= S);
    std::vector<int> named(S, 0);
    int before = -1;
    at.each(n, [&](int s, uint32_t p) {
      CHECK(!named[s]++);
      CHECK(in[s] != -1 && in[s] > before);  // in the order of their arming
      before = in[s];
      if (bars[s].armed) CHECK(!bars[s].done(p));
      if (bars[s].armed) bars[s].land();
      CHECK(bars[s].done(p));
    });
    for (int s = 0; s < S; ++s) {
      CHECK(!bars[s].armed);
      CHECK(named[s] == (in[s] != -1));
      in[s] = -1;  // given up
    }
  };
  if (across) {
    left_of_tile = 1 << 30;
    for (int s = 0; s < S; ++s) produce(s);
  }
  for (int n : tiles) {
    bool given_up = false;
    if (!across) {
      left_of_tile = n;
      for (int s = 0; s < S && s < n; ++s) produce((at.stage + s) % S);
    }
    int held = -1;
    for (int u = 0; u < n; ++u) {
      const int s = at.stage;
      land_some();
      if (consumed == give_up) {
        given_up = true;
        if (warp_fails) {
          drain(across ? at.armed(words) : n - u < S ? n - u : S);
          held = s;
          break;
        }
      }
      CHECK(in[s] == consumed && (!across || !(words[s] & kStageIdle)));
      if (bars[s].armed) {
        CHECK(!bars[s].done(at.parity));
        bars[s].land();
      }
      CHECK(bars[s].done(at.parity));
      in[s] = -1;
      ++consumed;
      if (across ? u + 1 < n : u + S < n) {
        produce(s);
      } else {
        held = s;
      }
      at.next();
    }
    // the join writes to `held` (across), or to the whole ring
    if (across) {
      if (held >= 0) CHECK(!bars[held].armed);
    } else {
      for (auto& b : bars) CHECK(!b.armed);
    }
    if (given_up) {
      if (across) {
        if (held >= 0) words[held] = kStageIdle;
        drain(at.armed(words));
      }
      return 1;
    }
    if (across && held >= 0) produce(held);
  }
  if (across) CHECK(at.armed(words) == 0);
  for (auto& b : bars) CHECK(!b.armed);
  return 0;
}

template <int S>
void all(std::mt19937& rng) {
  for (int turn = 0; turn < 400; ++turn) {
    std::vector<int> tiles(1 + rng() % 6);
    int units = 0;
    for (auto& n : tiles) units += n = (int)(rng() % (turn % 2 ? 3 : 12));
    for (bool across : {false, true}) {
      CHECK(run<S>(tiles, across, -1, false, rng) == 0);
      for (int u = 0; u < units; ++u)
        for (bool mine : {false, true}) CHECK(run<S>(tiles, across, u, mine, rng) == 1);
    }
  }
}

int main() {
  std::mt19937 rng(1);
  all<2>(rng);
  all<3>(rng);
  all<4>(rng);
  return 0;
}
