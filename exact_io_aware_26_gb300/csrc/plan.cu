// plan.cu -- block tables and slot maps of a serving step from request lengths.
//
// One cluster of CTAs; every CTA forms the prefix sums over all requests (new
// tokens, pages given back, pages needed) in its shared memory, the cluster meets
// once -- every input that an output may alias has been read by then -- and the CTAs
// write the step's tokens and table entries side by side.  Integers in a fixed
// order, no atomics.  Bound by latency: a step writes 8 bytes per token.
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
  int n_ctas;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n_ctas));
  // inputs read everywhere, shared arrays complete here
  if (n_ctas > 1)
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
  const int t0 = cluster_rank() * n_threads + threadIdx.x, step = n_ctas * n_threads;
  const uint32_t page = (uint32_t)a.page;
  auto held = [&](int seq) { return (int)(((uint32_t)seq + page - 1) / page); };

  for (int t = t0; t < a.T; t += step) {
    const int r = upper_bound(tok_end, R, t);
    int pos = 0, slot = -1;
    if (r < R) {
      const int seq = seq_s[r];
      const long long p = (long long)seq + t - (r ? tok_end[r - 1] : 0);
      pos = clamp_int(p);
      if (served[r]) {
        const int i = (int)((uint32_t)pos / page), have = held(seq);
        const int id = i < have ? a.table[r * a.stride + i] : pool(there - 1 - ((r ? need_end[r - 1] : 0) + i - have));
        const long long sl = (long long)id * a.page + ((uint32_t)pos - (uint32_t)i * page);
        slot = id < 0 || sl > 0x7FFFFFFFll ? -1 : (int)sl;
      }
    }
    a.pos[t] = pos;
    a.slots[t] = slot;
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

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t s) {
  const size_t smem = (size_t)a.R * 17;
  static_assert(FA_PLAN_MAX_REQUESTS * 17 + 4096 <= 227 * 1024, "a CTA's shared memory holds every request");
  if (smem > 40 * 1024) {  // beyond what every kernel may have
    const cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  // A CTA of as many threads as there are tokens and requests to spread over it; a cluster
  // of eight where one CTA would write more than a few tokens a thread.
  const int most = a.T > a.R ? a.T : a.R;
  const int threads = most >= kMaxThreads ? kMaxThreads : (most + 127) / 128 * 128;
  const int ctas = a.T <= 4 * kMaxThreads ? 1 : 8;
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
  return cudaLaunchKernelEx(&cfg, paged_plan_kernel, a);
}

}  // namespace fa
