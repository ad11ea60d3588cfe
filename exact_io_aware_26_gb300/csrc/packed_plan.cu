// packed_plan.cu -- the work list of packed attention, from the sequences' offsets on the GPU.
//
// One CTA: prefix maxima of the offsets (so that any offsets give sequences that lie in the
// tensors, one behind the other), prefix sums of the units, the steps of every unit, how long a
// slice is, and the slices in order of their steps, the longest first, by counting (many units
// sequence by sequence).  The main kernel's CTAs take the list in order, so that what is left at
// the end is short.  Where in its class of lengths an item stands, and which slots a cut unit has,
// is left to the order of atomics: results do not depend on it.  Bound by latency (three
// prompts of up to 32 tokens take 10.7 us with the list, 6.1 without), of which the main kernel's
// launch hides a part, and by the fetching of instructions: loops that hardly any call enters twice
// stay rolled (unrolled by four, 4 sequences of up to 2048 tokens take 30.4 us and not 29.4, their
// backward pass 71.9 and not 69.9).
#include "packed.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32, kClasses = kThreads, kNear = 1024, kWeighed = 4096;
// Units, times key heads, for each CTA that runs at a time, from which on the list goes sequence by
// sequence, for the sake of L2.  In this order and by steps alone: 12 sequences up to 16384 tokens, 32
// and 8 heads, d = 128, forward 7.33 and 7.70 ms, of up to 8192 backward 6.58 and 7.00; 20 up to
// 4096, 12 and 4 heads, d = 64, backward (10 units for each CTA) 0.728 and 0.713.
constexpr float kGrouped = 12.f;
static_assert(kPackedCandidates == kWarps, "a warp weighs a candidate");

// Inclusive scans of N values per thread over the CTA; `total` gets the last.
template <int N, class Op>
__device__ __forceinline__ void block_scan(int (&v)[N], int (*warp_s)[kWarps], int (&total)[N], Op op) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, v[i], off);
      if (lane >= off) v[i] = op(up, v[i]);
    }
    if (lane == 31) warp_s[i][warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    int w = warp_s[i][lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w = op(up, w);
    }
    total[i] = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    if (warp) v[i] = op(before, v[i]);
  }
}

// FEW: at most 32 sequences, which each warp has in its lanes, of at most kThreads units, one a thread's, and
// fewer than kGrouped asks for: half of the barriers and of the instructions (4 sequences of up to 2048
// tokens 28.4 us and 29.8 without it, their backward pass 68.4 and 70.2, 8 pieces over a cached prefix
// 63.2 and 65.3).
template <bool FEW>
__global__ void __launch_bounds__(kThreads) packed_plan_kernel(const PackedPlanArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // they wait for this grid's end
  __shared__ int near_s[4][kNear + 1];
  __shared__ int scan_s[4][kWarps];
  __shared__ long long steps_s[kWarps];
  __shared__ int longest_s[kWarps];
  __shared__ int class_s[kClasses];
  __shared__ int work_s[kWeighed];
  __shared__ float time_s[kWarps];
  __shared__ int end_s[2][kThreads];
  __shared__ int slot_s, cut_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = a.R;
  int *first_q = a.list.starts, *first_k = first_q + R + 1, *first_u = first_k + R + 1, *place_u = first_u + R + 1;
  if (R <= kNear) {
    first_q = near_s[0];
    first_k = near_s[1];
    first_u = near_s[2];
    place_u = near_s[3];
  }
  class_s[tid] = 0;
  if (tid == 0) slot_s = cut_s = 0;
  if (a.most)
    for (long long i = tid; i < (long long)R * a.Hk; i += kThreads) a.most[i] = make_float4(0.f, 0.f, 0.f, 0.f);

  // ---- the sequences: each begins where the furthest offset up to its own lies
  const int per = (R + kThreads) / kThreads, my0 = min(R + 1, tid * per), my1 = min(R + 1, my0 + per);
  auto sequence = [&](int r) {
    return PackedSeq{first_q[r], first_q[r + 1] - first_q[r], first_k[r], first_k[r + 1] - first_k[r]};
  };
  PackedItem own;  // this thread's first unit
  own.s0 = own.s1 = 0;
  int units, rows0, rows1;  // units; query rows that are a sequence's
  if constexpr (FEW) {
    bool wrong;
    const PackedSeq s = packed_lane_sequence(a, packed_lane_offsets(a), wrong);
    if (warp == 0 && wrong) atomicCAS(&a.st->code, 0, (int)FA_ERR_INDEX);
    if (a.most && warp == 0 && lane < R) {
      int *const q = a.list.starts + lane, *const k = q + R + 1;
      *q = s.q0;
      *k = s.k0;
      if (lane == R - 1) {
        q[1] = s.q0 + s.n;
        k[1] = s.k0 + s.m;
      }
    }
    const int mine = lane < R ? packed_units(s, a.tpt, a.bwd) : 0, end = packed_lane_end(mine);
    units = __shfl_sync(0xffffffffu, end, 31);
    rows0 = __shfl_sync(0xffffffffu, s.q0, 0);
    rows1 = __shfl_sync(0xffffffffu, s.q0 + s.n, 31);
    int of = 0;  // the sequence of unit tid: those before it end at it at most
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      if (__shfl_sync(0xffffffffu, end, of + off - 1) <= tid) of += off;
    own.seq.q0 = __shfl_sync(0xffffffffu, s.q0, of);
    own.seq.n = __shfl_sync(0xffffffffu, s.n, of);
    own.seq.k0 = __shfl_sync(0xffffffffu, s.k0, of);
    own.seq.m = __shfl_sync(0xffffffffu, s.m, of);
    own.tile = tid - __shfl_sync(0xffffffffu, end - mine, of);
    own.r = of;
    if (tid < units) packed_steps(own.seq, own.tile, a.tpt, a.causal, a.bwd, own.s0, own.s1);
  } else {
    auto offset = [&](const int* cu, int T, int r) { return min(max(__ldg(cu + r), 0), T); };
    auto larger = [](int x, int y) { return max(x, y); };
    int most[2] = {0, 0}, last[2];
#pragma unroll 1
    for (int r = my0; r < my1; ++r) {
      most[0] = max(most[0], offset(a.cu_q, a.Tq, r));
      most[1] = max(most[1], offset(a.cu_k, a.Tk, r));
    }
    block_scan(most, scan_s, last, larger);
    end_s[0][tid] = most[0];
    end_s[1][tid] = most[1];
    __syncthreads();
    int run_q = tid ? end_s[0][tid - 1] : 0, run_k = tid ? end_s[1][tid - 1] : 0;
    bool bad = false;
#pragma unroll 1
    for (int r = my0; r < my1; ++r) {
      run_q = max(run_q, offset(a.cu_q, a.Tq, r));
      run_k = max(run_k, offset(a.cu_k, a.Tk, r));
      bad |= run_q != __ldg(a.cu_q + r) || run_k != __ldg(a.cu_k + r);
      first_q[r] = run_q;
      first_k[r] = run_k;
      if (a.most) {
        a.list.starts[r] = run_q;
        a.list.starts[R + 1 + r] = run_k;
      }
    }
    if (bad) atomicCAS(&a.st->code, 0, (int)FA_ERR_INDEX);
    __syncthreads();
    int mine[1] = {0}, all[1];
#pragma unroll 1
    for (int r = my0; r < min(my1, R); ++r) mine[0] += packed_units(sequence(r), a.tpt, a.bwd);
    int at = -mine[0];
    block_scan(mine, scan_s + 2, all, [](int x, int y) { return x + y; });
    units = all[0];
    at += mine[0];
#pragma unroll 1
    for (int r = my0; r < my1; ++r) {
      first_u[r] = at;
      if (r < R) at += packed_units(sequence(r), a.tpt, a.bwd);
    }
    __syncthreads();
    rows0 = first_q[0];
    rows1 = first_q[R];
  }

  // ---- a unit's sequence, tile and steps
  auto unit = [&](int u, PackedItem& x) {
    int lo = 0, hi = R;  // the last sequence whose first unit is not behind u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first_u[mid] <= u) lo = mid; else hi = mid;
    }
    x.seq = sequence(lo);
    x.tile = u - first_u[lo];
    x.r = lo;
    packed_steps(x.seq, x.tile, a.tpt, a.causal, a.bwd, x.s0, x.s1);
  };
  if (!FEW && tid < units) unit(tid, own);
  auto with_units = [&](auto f) {  // f(unit) of every unit of this thread
    if constexpr (FEW) {
      if (tid < units) f(tid, own);
      return;
    }
    PackedItem x = own;
#pragma unroll 1
    for (int u = tid; u < units; u += kThreads) {
      if (u != tid) unit(u, x);
      f(u, x);
    }
  };
  long long steps = 0;
  int longest = 0;
  with_units([&](int u, const PackedItem& x) {
    const int w = x.s1 - x.s0;
    steps += w;
    longest = max(longest, w);
    if (FEW || u < kWeighed) work_s[u] = w;
  });
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) steps += __shfl_xor_sync(0xffffffffu, steps, off);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) {
    steps_s[warp] = steps;
    longest_s[warp] = longest;
  }
  __syncthreads();
  steps = steps_s[lane];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) steps += __shfl_xor_sync(0xffffffffu, steps, off);
  longest = __reduce_max_sync(0xffffffffu, longest_s[lane]);

  // ---- how long a slice is: each warp weighs a candidate.  Not where no unit is longer than the
  // shortest of them; and of more units than are kept only an even share is tried
  const float even = packed_even(steps, a.Hk, a.target);
  int slice = longest;
  if (a.slots > 0 && longest > a.least && (float)longest > 0.75f * even) {
    if (FEW || units <= kWeighed) {
      const int mine_slice = packed_candidate(warp, even, a.least, longest);
      int n = 0, cut = 0;
      for (int u = lane; u < units; u += 32) {
        const int c = packed_cuts(work_s[u], mine_slice);
        n += c;
        cut += c > 1 ? c : 0;
      }
      n = __reduce_add_sync(0xffffffffu, n);
      cut = __reduce_add_sync(0xffffffffu, cut);
      if (lane == 0) time_s[warp] = packed_time(mine_slice, n, cut, even, packed_even(1, a.Hk, a.target));
      __syncthreads();
      float best = time_s[lane];
      int which = lane;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        const float t = __shfl_xor_sync(0xffffffffu, best, off);
        const int k = __shfl_xor_sync(0xffffffffu, which, off);
        if (t < best || (t == best && k < which)) {
          best = t;
          which = k;
        }
      }
      slice = packed_candidate(which, even, a.least, longest);
    } else {
      slice = min(longest, max(a.least, (int)even + 1));
    }
  }
  float per_step = (float)(kClasses - 1) / (float)max(slice, 1);
  auto class_of = [&](int w) { return min(kClasses - 1, max(0, (int)((float)(slice - w) * per_step))); };

  // ---- many whole units: the sequences by their longest units' steps, and the units of each behind one
  // another, the longest first, so that the CTAs that run at a time read the same sequence
  if (!FEW && slice == longest && (float)units * (float)a.Hk >= kGrouped * (float)a.target) {
    auto seq_class = [&](int r, const PackedSeq& q, int n) {
      int s0, s1;
      packed_steps(q, a.bwd ? 0 : n - 1, a.tpt, a.causal, a.bwd, s0, s1);
      return class_of(s1 - s0);
    };
#pragma unroll 1
    for (int r = my0; r < min(my1, R); ++r) {
      const PackedSeq q = sequence(r);
      const int n = packed_units(q, a.tpt, a.bwd);
      if (n > 0) atomicAdd(&class_s[seq_class(r, q, n)], n);
    }
    __syncthreads();
    int of[1] = {class_s[tid]}, total[1];
    const int had = of[0];
    block_scan(of, scan_s + 3, total, [](int x, int y) { return x + y; });
    class_s[tid] = of[0] - had;
    __syncthreads();
#pragma unroll 1
    for (int r = my0; r < min(my1, R); ++r) {
      const PackedSeq q = sequence(r);
      const int n = packed_units(q, a.tpt, a.bwd);
      if (n > 0) place_u[r] = atomicAdd(&class_s[seq_class(r, q, n)], n);
    }
    __syncthreads();
    with_units([&](int u, const PackedItem& unit_x) {
      PackedItem x = unit_x;
      const int n = packed_units(x.seq, a.tpt, a.bwd);
      x.slot = -1;
      x.first = x.parts = x.cut = 0;
      a.list.items[place_u[x.r] + (a.bwd ? x.tile : n - 1 - x.tile)] = x;
    });
    if (tid == 0) {
      a.list.head[0] = units;
      a.list.head[1] = 0;
      a.list.head[2] = rows0;
      a.list.head[3] = rows1;
      a.list.head[4] = 0;
    }
    return;
  }

  // ---- else the slices, counted and placed by their lengths
  for (;;) {
    with_units([&](int, const PackedItem& x) {
      const int w = x.s1 - x.s0, c = packed_cuts(w, slice);
      if (c == 1) {
        atomicAdd(&class_s[class_of(w)], 1);
      } else {  // the first w % c of one length, the others of one less
        if (w % c) atomicAdd(&class_s[class_of(w / c + 1)], w % c);
        atomicAdd(&class_s[class_of(w / c)], c - w % c);
        atomicAdd(&slot_s, c);
      }
    });
    __syncthreads();
    if (slot_s <= a.slots) break;
    // more parts than there is room for (packed_slots rules it out): nothing is cut
    __syncthreads();
    slice = longest;
    per_step = (float)(kClasses - 1) / (float)max(slice, 1);
    class_s[tid] = 0;
    if (tid == 0) slot_s = 0;
    __syncthreads();
  }
  __syncthreads();
  if (tid == 0) slot_s = 0;
  int in_class[1] = {class_s[tid]}, items[1];
  const int had = in_class[0];
  block_scan(in_class, scan_s + 3, items, [](int x, int y) { return x + y; });
  class_s[tid] = in_class[0] - had;
  __syncthreads();
  with_units([&](int, const PackedItem& unit_x) {
    PackedItem x = unit_x;
    const int s0 = x.s0, w = x.s1 - x.s0, c = packed_cuts(w, slice);
    x.slot = -1;
    x.first = x.parts = x.cut = 0;
    if (c > 1) {
      x.first = atomicAdd(&slot_s, c);
      x.parts = c;
      x.cut = atomicAdd(&cut_s, 1);
      a.list.cuts[x.cut] = x;
      for (int h = 0; h < a.Hk && !a.bwd; ++h) a.list.left[x.cut * a.Hk + h] = 0;
    }
    for (int i = 0; i < c; ++i) {
      int b, e;
      packed_cut(w, c, i, b, e);
      x.s0 = s0 + b;
      x.s1 = s0 + e;
      x.slot = c > 1 ? x.first + i : -1;
      a.list.items[atomicAdd(&class_s[class_of(e - b)], 1)] = x;
    }
  });
  __syncthreads();
  if (tid == 0) {
    a.list.head[0] = items[0];
    a.list.head[1] = cut_s;
    a.list.head[2] = rows0;
    a.list.head[3] = rows1;
    a.list.head[4] = 0;
  }
}

}  // namespace

cudaError_t launch_packed_plan(const PackedPlanArgs& a, cudaStream_t s) {
  const bool few = a.R <= kPackedFew && a.units <= kThreads && (float)a.units * (float)a.Hk < kGrouped * (float)a.target;
  if (few)
    packed_plan_kernel<true><<<1, kThreads, 0, s>>>(a);
  else
    packed_plan_kernel<false><<<1, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
