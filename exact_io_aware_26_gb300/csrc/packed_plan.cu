// packed_plan.cu -- the work list of packed attention, from the sequences' offsets on the GPU.
//
// One CTA: prefix maxima of the offsets (so that any offsets give sequences that lie in the
// tensors, one behind the other), prefix sums of the units, the steps of every unit, how long a
// slice is, and the slices in order of their steps, the longest first, by counting.  The main
// kernel's CTAs take the list in order, so that what is left at the end is short.  Where in its
// class of lengths an item stands, and which slots a cut unit has, is left to the order of
// atomics: results do not depend on it.  Bound by latency: 3 us for a few sequences, of which the
// main kernel's launch hides a part.
#include "packed.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32, kClasses = kThreads, kNear = 1024;

// Inclusive scan of one value per thread over the CTA; `total` gets the last.
template <class T, class Op>
__device__ __forceinline__ T block_scan(T v, T* warp_s, T& total, Op op) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const T up = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v = op(up, v);
  }
  __syncthreads();  // warp_s read by a scan before
  if (lane == 31) warp_s[warp] = v;
  __syncthreads();
  T w = warp_s[lane];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const T up = __shfl_up_sync(0xffffffffu, w, off);
    if (lane >= off) w = op(up, w);
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const T before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return warp ? op(before, v) : v;
}

__global__ void __launch_bounds__(kThreads) packed_plan_kernel(const PackedPlanArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // they wait for this grid's end
  __shared__ int near_s[3][kNear + 1];
  __shared__ long long sum_s[kWarps];
  __shared__ int scan_s[kWarps];
  __shared__ int class_s[kClasses];
  __shared__ int slot_s, cut_s;
  const int tid = threadIdx.x, R = a.R;
  int *first_q = a.list.starts, *first_k = first_q + R + 1, *first_u = first_k + R + 1;
  if (R <= kNear) {
    first_q = near_s[0];
    first_k = near_s[1];
    first_u = near_s[2];
  }
  class_s[tid] = 0;
  if (tid == 0) slot_s = cut_s = 0;

  // ---- the sequences: each begins where the furthest offset up to its own lies
  const int per = (R + kThreads) / kThreads, my0 = min(R + 1, tid * per), my1 = min(R + 1, my0 + per);
  auto offset = [&](const int* cu, int T, int r) { return min(max(__ldg(cu + r), 0), T); };
  auto larger = [](int x, int y) { return max(x, y); };
  int most_q = 0, most_k = 0;
  for (int r = my0; r < my1; ++r) {
    most_q = max(most_q, offset(a.cu_q, a.Tq, r));
    most_k = max(most_k, offset(a.cu_k, a.Tk, r));
  }
  int last;
  const int up_q = block_scan(most_q, scan_s, last, larger), up_k = block_scan(most_k, scan_s, last, larger);
  // of the threads before this one
  __shared__ int end_s[2][kThreads];
  end_s[0][tid] = up_q;
  end_s[1][tid] = up_k;
  __syncthreads();
  int run_q = tid ? end_s[0][tid - 1] : 0, run_k = tid ? end_s[1][tid - 1] : 0;
  bool bad = false;
  for (int r = my0; r < my1; ++r) {
    run_q = max(run_q, offset(a.cu_q, a.Tq, r));
    run_k = max(run_k, offset(a.cu_k, a.Tk, r));
    bad |= run_q != __ldg(a.cu_q + r) || run_k != __ldg(a.cu_k + r);
    first_q[r] = run_q;
    first_k[r] = run_k;
  }
  if (bad) atomicCAS(&a.st->code, 0, (int)FA_ERR_INDEX);
  __syncthreads();
  auto sequence = [&](int r) {
    return PackedSeq{first_q[r], first_q[r + 1] - first_q[r], first_k[r], first_k[r + 1] - first_k[r]};
  };
  int mine = 0;
  for (int r = my0; r < min(my1, R); ++r) mine += packed_units(sequence(r), a.tpt, a.bwd);
  int units;
  int at = block_scan(mine, scan_s, units, [](int x, int y) { return x + y; }) - mine;
  for (int r = my0; r < my1; ++r) {
    first_u[r] = at;
    if (r < R) at += packed_units(sequence(r), a.tpt, a.bwd);
  }
  __syncthreads();

  // ---- a unit's sequence, tile and steps
  auto unit = [&](int u, PackedItem& x) {
    int lo = 0, hi = R;  // the last sequence whose first unit is not behind u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first_u[mid] <= u) lo = mid; else hi = mid;
    }
    x.seq = sequence(lo);
    x.tile = u - first_u[lo];
    packed_steps(x.seq, x.tile, a.tpt, a.causal, a.bwd, x.s0, x.s1);
    x.slot = -1;
  };
  long long steps = 0;
  int longest = 0;
  for (int u = tid; u < units; u += kThreads) {
    PackedItem x;
    unit(u, x);
    steps += x.s1 - x.s0;
    longest = max(longest, x.s1 - x.s0);
  }
  long long all;
  block_scan(steps, sum_s, all, [](long long x, long long y) { return x + y; });
  int most;
  block_scan(longest, scan_s, most, larger);
  const long long slice = packed_slice(all, a.Hk, a.target, a.least);
  most = (int)min((long long)most, slice);  // an upper bound of a slice's steps
  auto class_of = [&](int w) { return (int)((long long)(most - w) * (kClasses - 1) / max(most, 1)); };

  // ---- the slices, counted and placed by their lengths
  for (int u = tid; u < units; u += kThreads) {
    PackedItem x;
    unit(u, x);
    const int w = x.s1 - x.s0, c = packed_cuts(w, slice);
    for (int i = 0; i < c; ++i) {
      int b, e;
      packed_cut(w, c, i, b, e);
      atomicAdd(&class_s[class_of(e - b)], 1);
    }
  }
  __syncthreads();
  const int in_class = class_s[tid];
  int items;
  const int class_end = block_scan(in_class, scan_s, items, [](int x, int y) { return x + y; });
  class_s[tid] = class_end - in_class;
  __syncthreads();
  for (int u = tid; u < units; u += kThreads) {
    PackedItem x;
    unit(u, x);
    const int s0 = x.s0, w = x.s1 - x.s0, c = packed_cuts(w, slice);
    int slot = -1;
    if (c > 1) {
      slot = atomicAdd(&slot_s, c);
      PackedItem cut = x;
      cut.s0 = slot;
      cut.s1 = c;
      a.list.cuts[atomicAdd(&cut_s, 1)] = cut;
    }
    for (int i = 0; i < c; ++i) {
      int b, e;
      packed_cut(w, c, i, b, e);
      x.s0 = s0 + b;
      x.s1 = s0 + e;
      x.slot = c > 1 ? slot + i : -1;
      a.list.items[atomicAdd(&class_s[class_of(e - b)], 1)] = x;
    }
  }
  __syncthreads();
  if (tid == 0) {
    a.list.head[0] = items;
    a.list.head[1] = cut_s;
    a.list.head[2] = first_q[0];  // query and key rows that are a sequence's
    a.list.head[3] = first_q[R];
  }
}

}  // namespace

cudaError_t launch_packed_plan(const PackedPlanArgs& a, cudaStream_t s) {
  packed_plan_kernel<<<1, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
