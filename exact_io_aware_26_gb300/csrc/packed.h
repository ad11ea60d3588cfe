// packed.h -- declarations shared by the entry points of packed attention (packed_api.cu) and
// its kernels.  Not part of the public interface.
#pragma once
#include "ops.h"
#include "packed_sched.cuh"

namespace fa {

// The list of a call's work, made on the GPU (packed_plan.cu), in the workspace.
struct PackedList {
  int* head;           // [0] items, [1] cut units, [2], [3] first query row and end, [4] items that CTAs took
                       // after their first
  PackedItem* items;
  PackedItem* cuts;    // the cut units (s0, s1: the whole unit's steps)
  int* left;           // of each cut unit and key head: the parts that are done (forward)
  int* starts;         // scratch: first query, key and unit of each sequence and behind the last; its place in the list
                       // (backward in fp16: the first two for the other kernels)
};

struct PackedPlanArgs {
  int R, Tq, Tk, Hk;
  int tpt, causal, bwd;
  int target;          // CTAs to share the steps among
  int slots, least;    // places for parts of cut units (0: none is cut); steps that a slice has at least
  int units;           // at most that many
  const int* cu_q;
  const int* cu_k;
  PackedList list;
  float4* most;        // backward in fp16: to be zeroed, else nullptr
  DevStatus* st;
};

struct PackedArgs {
  int R, Tq, Tk, Hq, Hk, G;
  FastDiv divG, divHk;
  FastDiv divRows, divTk;  // backward: by Tq * G and Tk
  int tpt, causal;
  float scale, scale_log2;
  PackedList list;
  int direct;          // forward: no list; each CTA finds its unit in the offsets
  const int *cu_q, *cu_k;
  const void* v;       // for values that are not finite
  long long vs[2];     // element strides {token, head}
  void* o;             // forward: result; backward: its values
  const void* dout;
  float* lse;
  void *dq, *dk, *dv;
  long long os[2], dos[2], dqs[2], dks[2], dvs[2];
  float* slots;        // partial results of cut units
  float *stat_lse, *stat_d;  // backward: [Hk][Tq * G] LSE (+inf: no key seen) and rowsum(dO O)
  float* dq_acc;       // backward: [Hk][Tq * G][d]
  int* seq_of;         // backward in fp16: [Tq] the sequence of a row, any for one of none
  float4* most;        // backward in fp16: [R][Hk] largest |dO|^2, |V|^2 and |D| of a sequence and key head
  Report rep;
};

constexpr int kPackedFew = 32;  // sequences that a warp's lanes hold, one each
#ifdef __CUDACC__
// At most 32 sequences from their offsets, lane r of a warp sequence r (and the last one in the lanes
// behind it): each begins where the furthest offset up to its own lies.  wrong: some offset of
// the lane's is outside the tensors or smaller than one before.
struct PackedOffsets {
  int q0, q1, k0, k1;
};
template <class Args>
__device__ __forceinline__ PackedOffsets packed_lane_offsets(const Args& a) {
  const int r = min((int)(threadIdx.x & 31), a.R - 1);
  return PackedOffsets{__ldg(a.cu_q + r), __ldg(a.cu_q + r + 1), __ldg(a.cu_k + r), __ldg(a.cu_k + r + 1)};
}
template <class Args>
__device__ __forceinline__ PackedSeq packed_lane_sequence(const Args& a, const PackedOffsets& cu, bool& wrong) {
  const int lane = threadIdx.x & 31, q0 = cu.q0, q1 = cu.q1, k0 = cu.k0, k1 = cu.k1;
  auto clamp = [](int v, int T) { return min(max(v, 0), T); };
  PackedSeq s{clamp(q0, a.Tq), 0, clamp(k0, a.Tk), 0};
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int uq = __shfl_up_sync(0xffffffffu, s.q0, off), uk = __shfl_up_sync(0xffffffffu, s.k0, off);
    if (lane >= off) {
      s.q0 = max(s.q0, uq);
      s.k0 = max(s.k0, uk);
    }
  }
  s.n = max(clamp(q1, a.Tq), s.q0) - s.q0;
  s.m = max(clamp(k1, a.Tk), s.k0) - s.k0;
  wrong = s.q0 != q0 || s.q0 + s.n != q1 || s.k0 != k0 || s.k0 + s.m != k1;
  return s;
}
// The units up to and including those of the lane's sequence, of which it has `mine`.
__device__ __forceinline__ int packed_lane_end(int mine) {
  const int lane = threadIdx.x & 31;
  int end = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, end, off);
    if (lane >= off) end += up;
  }
  return end;
}

// Without a list: unit `index` of at most 32 sequences; false: there is none.  Offsets that are wrong
// are recorded by the first CTA.
__device__ __forceinline__ bool packed_direct(const PackedArgs& a, const PackedOffsets& cu, int index, PackedItem& x) {
  const int lane = threadIdx.x & 31;
  bool wrong;
  const PackedSeq s = packed_lane_sequence(a, cu, wrong);
  if (blockIdx.x == 0 && wrong) atomicCAS(&a.rep.st->code, 0, (int)FA_ERR_INDEX);
  const int mine = lane < a.R ? packed_units(s, a.tpt, false) : 0, end = packed_lane_end(mine);
  const uint32_t here = __ballot_sync(0xffffffffu, index < end && index >= end - mine);
  if (here == 0u) return false;
  const int from = __ffs((int)here) - 1;
  x.seq.q0 = __shfl_sync(0xffffffffu, s.q0, from);
  x.seq.n = __shfl_sync(0xffffffffu, s.n, from);
  x.seq.k0 = __shfl_sync(0xffffffffu, s.k0, from);
  x.seq.m = __shfl_sync(0xffffffffu, s.m, from);
  x.tile = index - __shfl_sync(0xffffffffu, end - mine, from);
  packed_steps(x.seq, x.tile, a.tpt, a.causal, false, x.s0, x.s1);
  x.slot = -1;
  return true;
}
#endif

// fp32 words of a slot: forward (m, l) and O of 128 rows; backward dV and dK of 128 keys.
inline size_t packed_slot_words(int d, bool bwd) { return bwd ? (size_t)2 * 128 * d : (size_t)128 * (d + 2); }

cudaError_t launch_packed_plan(const PackedPlanArgs& a, cudaStream_t s);
// `items`, `cuts`: at most that many items and cut units of the list.  The CTAs stay and take item
// after item, an item's key heads next to each other.  (Key head after key head, 32 heads over 8 of 12
// sequences up to 16384 tokens take 7.8 ms instead of 7.3.)
cudaError_t launch_packed_fwd(const PackedArgs& a, int d, bool f16, const CUtensorMap* tm, int items, cudaStream_t s);
cudaError_t launch_packed_bwd_preprocess(const PackedArgs& a, int d, bool f16, cudaStream_t s);
cudaError_t launch_packed_bwd(const PackedArgs& a, int d, bool f16, const CUtensorMap* tm, int items, cudaStream_t s);
cudaError_t launch_packed_bwd_finalize(const PackedArgs& a, int d, bool f16, int cuts, cudaStream_t s);

}  // namespace fa
