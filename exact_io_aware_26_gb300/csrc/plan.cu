// plan.cu -- block tables and slot maps of a serving step from request lengths.
//
// Every CTA forms the prefix sums over all requests (new tokens, pages given back, pages
// needed) in its shared memory, and the CTAs write the step's tokens and table entries side
// by side: what one writes no other reads, except where kv_lens or counts lie over the
// inputs.  Then the CTAs are one cluster, which meets once all inputs have been read.
// Integers in a fixed order, no atomics.  Bound by latency (a step writes 8 bytes per
// token): the time goes into chains of searches and loads, so few tokens per thread.
// Measured: 256 requests of a token each 7.0 us, 96 requests with 65,536 tokens 7.2 us (as
// one cluster of 8 CTAs 15.3 us).
#include "ops.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kMaxThreads = 1024;

// Exclusive prefix sums over the CTA of N values per thread; `total` gets the sums.
template <int N>
__device__ __forceinline__ void block_scan(long long (&v)[N], long long (*warp_sums)[32], long long (&total)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  long long inc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    inc[i] = v[i];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, inc[i], off);
      if (lane >= off) inc[i] += up;
    }
    if (lane == 31) warp_sums[i][warp] = inc[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {  // every warp scans the warps' sums
    long long w = lane < warps ? warp_sums[i][lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += up;
    }
    total[i] = __shfl_sync(0xffffffffu, w, 31);
    const long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    v[i] = inc[i] - v[i] + (warp ? before : 0);
  }
}

// First index in [0, n) whose value is > x, of a non-decreasing array; n if none.
__device__ int upper_bound(const int* v, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ int clamp_int(long long v) { return v > 0x7FFFFFFFll ? 0x7FFFFFFF : (int)v; }

// What a request brings: tokens before the step, new ones (none where it has ended), pages
// given back, pages held and needed.  Pages are quotients of numbers below 2^32.
struct Request {
  int seq, fresh, freed, have, want;
  bool open;  // not ended, its pages fit its row of the table and its length an int
};
__device__ __forceinline__ Request request(const PlanArgs& a, int r) {
  Request q;
  q.seq = max(0, a.seq[r]);
  const int fresh = a.fresh[r];
  q.fresh = max(0, fresh);
  const uint32_t page = (uint32_t)a.page, up = page - 1;
  q.have = (int)(((uint32_t)q.seq + up) / page);
  q.freed = fresh < 0 ? min(q.have, a.width) : 0;
  const uint32_t after = ((uint32_t)q.seq + (uint32_t)q.fresh + up) / page;
  q.open = fresh >= 0 && (long long)q.seq + q.fresh <= 0x7FFFFFFFll && after <= (uint32_t)a.width;
  q.want = q.open ? (int)after - q.have : 0;
  return q;
}

__global__ void __launch_bounds__(kMaxThreads) paged_plan_kernel(const PlanArgs a) {
  extern __shared__ int smem[];
  __shared__ long long warp_sums[2][2][32];
  const int R = a.R, n_threads = blockDim.x;
  // per request: the ends (inclusive prefix sums) of its new tokens, its freed pages and its
  // needed pages; its tokens before the step; whether it is served
  int *tok_end = smem, *freed_end = smem + R, *need_end = smem + 2 * R, *seq_s = smem + 3 * R;
  uint8_t* served = reinterpret_cast<uint8_t*>(smem + 4 * R);
  const int per = (R + n_threads - 1) / n_threads;  // consecutive requests of a thread
  const int r0 = min(R, (int)threadIdx.x * per), r1 = min(R, r0 + per);
  const int top = max(0, min(*a.count, a.pages));
  Request mine;
  long long sums[2] = {0, 0}, totals[2];
  for (int r = r0; r < r1; ++r) {
    mine = request(a, r);
    sums[0] += mine.fresh;
    sums[1] += mine.freed;
  }
  block_scan<2>(sums, warp_sums[0], totals);
  const long long tok_total = totals[0];
  // pages on the stack once the ended requests' are back; more than it has entries for
  // would be pages given back twice, which are dropped
  const int there = (int)min((long long)top + totals[1], (long long)a.pages);
  long long need[1] = {0}, need_total[1];
  for (int r = r0; r < r1; ++r) {
    if (per > 1) mine = request(a, r);
    sums[0] += mine.fresh;
    sums[1] += mine.freed;
    const bool fits = mine.open && sums[0] <= a.T;
    tok_end[r] = clamp_int(sums[0]);
    freed_end[r] = clamp_int(sums[1]);
    seq_s[r] = mine.seq;
    served[r] = fits;
    need[0] += fits ? mine.want : 0;
  }
  block_scan<1>(need, warp_sums[1], need_total);
  int taken = 0;
  for (int r = r0; r < r1; ++r) {
    if (per > 1) mine = request(a, r);
    const int want = served[r] ? mine.want : 0;
    need[0] += want;
    need_end[r] = clamp_int(need[0]);
    if (served[r]) {
      served[r] = want == 0 || need[0] <= there;
      if (served[r] && want > 0) taken = (int)need[0];
    }
  }
  taken = __reduce_max_sync(0xffffffffu, taken);
  __shared__ int taken_s[32];
  if ((threadIdx.x & 31) == 0) taken_s[threadIdx.x >> 5] = taken;
  // shared arrays complete; with outputs over inputs, also the inputs read by every CTA
  if (a.aliased)
    cluster_sync();
  else
    __syncthreads();
  taken = (threadIdx.x & 31) < (n_threads >> 5) ? taken_s[threadIdx.x & 31] : 0;
  taken = __reduce_max_sync(0xffffffffu, taken);
  const int left = there - taken;
  // page v of the stack with the freed pages on top
  auto pool = [&](int v) -> int {
    if (v < top) return a.stack[v];
    const int f = v - top;
    const int r = upper_bound(freed_end, R, f);
    if (r >= R) return -1;
    return a.table[r * a.stride + f - (r ? freed_end[r - 1] : 0)];
  };
  const int t0 = blockIdx.x * n_threads + threadIdx.x, step = gridDim.x * n_threads;
  const uint32_t page = (uint32_t)a.page;
  auto held = [&](int seq) { return (int)(((uint32_t)seq + page - 1) / page); };

  // page i of a served request, after the step
  auto page_of = [&](int r, int i) {
    const int have = held(seq_s[r]);
    return i < have ? a.table[r * a.stride + i] : pool(there - 1 - ((r ? need_end[r - 1] : 0) + i - have));
  };
  // more tokens than threads: four neighbours a thread, one search and the next from there
  const int each = a.T > step ? 4 : 1;
  const bool wide = each == 4 && ((reinterpret_cast<uintptr_t>(a.pos) | reinterpret_cast<uintptr_t>(a.slots)) & 15) == 0;
  for (int first = each * t0; first < a.T; first += each * step) {
    int r = upper_bound(tok_end, R, first);
    int pos[4], slot[4];
    // the token's place in its request, its page there and its place in it, the page's number
    long long p = 0;
    int i = 0, in = -1, id = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= each) break;
      const int t = first + k;
      pos[k] = 0;
      slot[k] = -1;
      while (r < R && tok_end[r] <= t) {
        ++r;
        in = -1;
      }
      if (r >= R) continue;
      if (in < 0) {
        p = (long long)seq_s[r] + t - (r ? tok_end[r - 1] : 0);
        i = (int)((uint32_t)clamp_int(p) / page);
        in = (int)((uint32_t)clamp_int(p) - (uint32_t)i * page);
        id = served[r] ? page_of(r, i) : -1;
      }
      pos[k] = clamp_int(p);
      const long long sl = (long long)id * a.page + in;
      slot[k] = id < 0 || sl > 0x7FFFFFFFll ? -1 : (int)sl;
      ++p;
      if (++in == a.page) {
        in = 0;
        ++i;
        id = served[r] && t + 1 < tok_end[r] ? page_of(r, i) : -1;
      }
    }
    if (wide && first + 4 <= a.T) {
      *reinterpret_cast<int4*>(a.pos + first) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(a.slots + first) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < each && first + k < a.T) {
          a.pos[first + k] = pos[k];
          a.slots[first + k] = slot[k];
        }
    }
  }
  for (int r = t0; r < R; r += step) {
    const int fresh = tok_end[r] - (r ? tok_end[r - 1] : 0);
    const bool ended = freed_end[r] != (r ? freed_end[r - 1] : 0);
    a.kv[r] = ended ? 0 : seq_s[r] + (served[r] ? fresh : 0);
    a.cu[r + 1] = min(tok_end[r], a.T);
  }
  // the entries the taken pages go to: the k-th page needed is the k-th off the top
  for (int k = t0; k < taken; k += step) {
    const int r = upper_bound(need_end, R, k);
    a.table[r * a.stride + held(seq_s[r]) + k - (r ? need_end[r - 1] : 0)] = pool(there - 1 - k);
  }
  // what stays of the freed pages: stack entries from `top` on, never read above
  for (int v = top + t0; v < left; v += step) a.stack[v] = pool(v);
  if (t0 == 0) {
    a.cu[0] = 0;
    a.counts[0] = left;
    a.counts[1] = clamp_int(tok_total);
    a.counts[2] = clamp_int(max(0ll, need_total[0] - there));
  }
}

bool overlap(const int* a, int na, const int* b, int nb) { return a < b + nb && b < a + na; }

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t s) {
  const size_t smem = (size_t)a.R * 17;
  constexpr int kMost = FA_PLAN_MAX_REQUESTS * 17;
  static_assert(kMost + 4096 <= 227 * 1024, "a CTA's shared memory holds every request");
  if (smem > 40 * 1024) {  // beyond what every kernel may have: one limit for all calls, which may run at once
    const cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
  }
  // A token for each thread, and threads for the pages of ended requests besides (the step of
  // 256 single tokens: 8.4 us with as many threads as tokens).
  const bool few = a.T <= 256 && a.R <= 32;
  const int threads = few ? 256 : kMaxThreads;
  const long long want = ((long long)a.T + threads - 1) / threads;
  PlanArgs b = a;
  b.aliased = overlap(a.kv, a.R, a.seq, a.R) || overlap(a.kv, a.R, a.fresh, a.R) || overlap(a.kv, a.R, a.count, 1) ||
              overlap(a.counts, 3, a.count, 1) || overlap(a.counts, 3, a.seq, a.R) || overlap(a.counts, 3, a.fresh, a.R);
  const int ctas = (int)(want < 1 ? 1 : b.aliased ? (want < 8 ? want : 8) : (want < 128 ? want : 128));
  if (!b.aliased) {
    paged_plan_kernel<<<ctas, threads, smem, s>>>(b);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = ctas;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_plan_kernel, b);
}

}  // namespace fa
