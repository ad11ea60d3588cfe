// packed.h -- declarations shared by the entry points of packed attention (packed_api.cu) and
// its kernels.  Not part of the public interface.
#pragma once
#include "ops.h"
#include "packed_sched.cuh"

namespace fa {

// The list of a call's work, made on the GPU (packed_plan.cu), in the workspace.
struct PackedList {
  int* head;           // [0] items, [1] cut units
  PackedItem* items;
  PackedItem* cuts;
  int* starts;         // scratch: first query, key and unit of each sequence and behind the last; its place in the list
};

struct PackedPlanArgs {
  int R, Tq, Tk, Hk;
  int tpt, causal, bwd;
  int target;          // CTAs to share the steps among
  int cuttable, least; // whether units may be cut; steps that a slice has at least
  const int* cu_q;
  const int* cu_k;
  PackedList list;
  DevStatus* st;
};

struct PackedArgs {
  int R, Tq, Tk, Hq, Hk, G;
  FastDiv divG, divHk;
  int tpt, causal;
  float scale, scale_log2;
  PackedList list;
  const void* v;       // for values that are not finite
  long long vs[2];     // element strides {token, head}
  void* o;             // forward: result; backward: its values
  const void* dout;
  float* lse;
  void *dq, *dk, *dv;
  long long os[2], dos[2], dqs[2], dks[2], dvs[2];
  float* slots;        // partial results of cut units
  float *stat_lse, *stat_d;  // backward: [Hk][Tq * G] LSE log2 e (+inf: no key seen) and rowsum(dO O)
  float* dq_acc;       // backward: [Hk][Tq * G][d]
  Report rep;
};

#ifdef __CUDACC__
// A CTA's item of the list and its key head, an item's key heads next to each other; false: none is
// left for it.  (Key head after key head, 32 heads over 8 of 12 sequences up to 16384 tokens take 7.8 ms
// instead of 7.3.)
__device__ __forceinline__ bool packed_place(const PackedArgs& a, int& index, int& hk) {
  index = a.divHk.div((int)blockIdx.x);
  hk = (int)blockIdx.x - index * a.Hk;
  return index < a.list.head[0];
}
#endif

// fp32 words of a slot: forward (m, l) and O of 128 rows; backward dV and dK of 128 keys.
inline size_t packed_slot_words(int d, bool bwd) { return bwd ? (size_t)2 * 128 * d : (size_t)128 * (d + 2); }

cudaError_t launch_packed_plan(const PackedPlanArgs& a, cudaStream_t s);
// `items`: at most that many; `cuts`: at most that many cut units, 0 where none can be.
cudaError_t launch_packed_fwd(const PackedArgs& a, int d, bool f16, const CUtensorMap* tm, int items, int cuts,
                              cudaStream_t s);
cudaError_t launch_packed_bwd_preprocess(const PackedArgs& a, int d, bool f16, cudaStream_t s);
cudaError_t launch_packed_bwd(const PackedArgs& a, int d, bool f16, const CUtensorMap* tm, int items, cudaStream_t s);
cudaError_t launch_packed_bwd_finalize(const PackedArgs& a, int d, bool f16, int cuts, cudaStream_t s);

}  // namespace fa
