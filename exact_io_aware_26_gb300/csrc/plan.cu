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

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// Exclusive prefix sum over the CTA of one value per thread; `total` gets the sum.
__device__ long long block_scan(long long v, long long* warp_sums, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += up;
  }
  __syncthreads();  // warp_sums of an earlier scan have been read
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  long long before = 0, all = 0;
  for (int w = 0; w < kWarps; ++w) {
    const long long x = warp_sums[w];
    if (w < warp) before += x;
    all += x;
  }
  total = all;
  return before + inc - v;
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

// Shared memory, per request: the ends (inclusive prefix sums) of its new tokens, its
// freed pages and its needed pages; its tokens before the step; whether it is served.
struct Shared {
  int* tok_end;
  int* freed_end;
  int* need_end;
  int* seq;
  uint8_t* served;
};

__global__ void __launch_bounds__(kThreads) paged_plan_kernel(const PlanArgs a) {
  extern __shared__ int smem[];
  __shared__ long long warp_sums[kWarps];
  __shared__ int taken_s;
  const int R = a.R;
  Shared S{smem, smem + R, smem + 2 * R, smem + 3 * R, reinterpret_cast<uint8_t*>(smem + 4 * R)};
  const int per = (R + kThreads - 1) / kThreads;  // consecutive requests of a thread
  const int r0 = min(R, (int)threadIdx.x * per), r1 = min(R, r0 + per);
  const long long page = a.page;
  const int top = max(0, min(*a.count, a.pages));
  if (threadIdx.x == 0) taken_s = 0;

  long long tok = 0, freed = 0;
  for (int r = r0; r < r1; ++r) {
    const int seq = max(0, a.seq[r]), fresh = a.fresh[r];
    S.seq[r] = seq;
    tok += max(0, fresh);
    if (fresh < 0) freed += min((seq + page - 1) / page, (long long)a.width);
  }
  long long tok_total, freed_total, need_total;
  long long tok_at = block_scan(tok, warp_sums, tok_total);
  long long freed_at = block_scan(freed, warp_sums, freed_total);
  // pages on the stack once the ended requests' are back; more than it has entries
  // for would be pages given back twice, which are dropped
  const long long there = min((long long)top + freed_total, (long long)a.pages);
  long long need = 0;
  for (int r = r0; r < r1; ++r) {
    const int seq = S.seq[r], fresh = a.fresh[r];
    const long long have = (seq + page - 1) / page;
    if (fresh < 0) freed_at += min(have, (long long)a.width);
    tok_at += max(0, fresh);
    const long long after = ((long long)seq + max(0, fresh) + page - 1) / page;
    const bool fits = fresh >= 0 && after <= a.width && tok_at <= a.T && (long long)seq + fresh <= 0x7FFFFFFFll;
    S.tok_end[r] = clamp_int(tok_at);
    S.freed_end[r] = clamp_int(freed_at);
    S.served[r] = fits;
    need += fits ? after - have : 0;
  }
  long long need_at = block_scan(need, warp_sums, need_total);
  int taken = 0;
  for (int r = r0; r < r1; ++r) {
    const int seq = S.seq[r], fresh = a.fresh[r];
    const long long have = (seq + page - 1) / page;
    const long long want = S.served[r] ? ((long long)seq + fresh + page - 1) / page - have : 0;
    need_at += want;
    S.need_end[r] = clamp_int(need_at);
    if (S.served[r]) {
      S.served[r] = want == 0 || need_at <= there;
      if (S.served[r] && want > 0) taken = (int)need_at;
    }
  }
  atomicMax(&taken_s, taken);
  cluster_sync();  // inputs read everywhere, shared arrays complete here
  taken = taken_s;
  const int left = (int)(there - taken);
  // page v of the stack with the freed pages on top
  auto pool = [&](int v) -> int {
    if (v < top) return a.stack[v];
    const int f = v - top;
    const int r = upper_bound(S.freed_end, R, f);
    if (r >= R) return -1;
    const int off = f - (r ? S.freed_end[r - 1] : 0);
    return a.table[r * a.stride + off];
  };
  const int me = cluster_rank();
  int n_ctas;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n_ctas));
  const int t0 = me * kThreads + threadIdx.x, step = n_ctas * kThreads;

  for (int t = t0; t < a.T; t += step) {
    const int r = upper_bound(S.tok_end, R, t);
    int pos = 0, slot = -1;
    if (r < R) {
      const long long p = (long long)S.seq[r] + t - (r ? S.tok_end[r - 1] : 0);
      pos = clamp_int(p);
      if (S.served[r]) {
        const int i = (int)(p / page), have = (int)((S.seq[r] + page - 1) / page);
        const int id = i < have ? a.table[r * a.stride + i]
                                : pool((int)(there - 1 - ((r ? S.need_end[r - 1] : 0) + i - have)));
        const long long sl = (long long)id * page + p % page;
        slot = id < 0 || sl > 0x7FFFFFFFll ? -1 : (int)sl;
      }
    }
    a.pos[t] = pos;
    a.slots[t] = slot;
  }
  for (int r = t0; r < R; r += step) {
    const int fresh = S.tok_end[r] - (r ? S.tok_end[r - 1] : 0);
    const bool ended = S.freed_end[r] != (r ? S.freed_end[r - 1] : 0);
    a.kv[r] = ended ? 0 : S.seq[r] + (S.served[r] ? fresh : 0);
    a.cu[r + 1] = min(S.tok_end[r], a.T);
  }
  // the entries the taken pages go to: the k-th page needed is the k-th off the top
  for (int k = t0; k < taken; k += step) {
    const int r = upper_bound(S.need_end, R, k);
    const int have = (int)((S.seq[r] + page - 1) / page);
    a.table[r * a.stride + have + k - (r ? S.need_end[r - 1] : 0)] = pool((int)there - 1 - k);
  }
  // what stays of the freed pages: stack entries from `top` on, never read above
  for (int v = top + t0; v < left; v += step) a.stack[v] = pool(v);
  if (t0 == 0) {
    a.cu[0] = 0;
    a.counts[0] = left;
    a.counts[1] = clamp_int(tok_total);
    a.counts[2] = clamp_int(max(0ll, need_total - there));
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t s) {
  const size_t smem = (size_t)a.R * 17;
  static_assert(FA_PLAN_MAX_REQUESTS * 17 + 1024 <= 227 * 1024, "a CTA's shared memory holds every request");
  cudaError_t e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int ctas = a.T <= kThreads ? 1 : 8;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
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
