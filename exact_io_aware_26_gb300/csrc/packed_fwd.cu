// packed_fwd.cu -- attention forward of packed sequences with grouped heads (sm_103a).
//
// O = softmax(scale Q K^T) V and LSE for each sequence's queries over its own keys: the tiled
// recurrence of fwd_tc.cu ("L'algorithme Flash Attention", marketmaker.cc), with
//   - a query tile of tpt tokens times the G query heads of one key head, row = token * G + head,
//     which one TMA box {64 channels, G heads, tpt tokens} brings: a short prompt fills a tile's
//     128 rows with its heads, and K and V are read once for all of them;
//   - tiles taken from the list that packed_plan.cu makes of the offsets, longest first, by CTAs that
//     stay: the next tile's copies and first scores run beside the last one's results' way out
//     (1520 sequences of 512 tokens, one head, d = 128: 267 us with a CTA for each tile, 229 so);
//   - units longer than an even share of the steps cut along the keys, their parts (m, l, O in
//     fp32) joined by the CTA that is done last, so that few rows over many keys fill the GPU (8
//     requests of up to 512 rows over up to 8192 keys: 89 us uncut, 65 cut);
//   - keys and values behind a sequence's end, which belong to the next sequence or to none, and
//     those that only some rows of a tile see: scores are replaced by -inf, and values that are
//     not finite, which a weight of 0 would make NaN, are zeroed in shared memory and added
//     to the rows that see them at the end.
//
// Bound: the tensor core (4 d FLOPs a seen pair and query head) beside one exponential for each
// 4 d FLOPs; two CTAs an SM, so that one's exponentials run beside the other's products.  Measured,
// causal: a sequence of 30,000 tokens, 32 and 8 heads, d = 128, 1642 TFLOP/s; 12 of up to 16384
// 1500 to 1550; a sequence of 23,400, 12 heads, d = 64, where there are twice the exponentials, 1107.
//
// Warp roles (192 threads) as in fwd_tc.cu: warps 0-3 softmax (thread = row = TMEM lane), warp
// 4 TMA producer, warp 5 TMEM owner and MMA issuer.
#include <algorithm>

#include "fwd_common.cuh"
#include "packed.h"

namespace fa {
namespace {

constexpr float kRescaleThr = 8.f;  // the running maximum moves past 2^8 only
constexpr float kLargeScore = 65536.f;  // log2 units, from which on the maximum is taken off first
constexpr int kNone = 0x7FFFFFFF;

// A CTA's item as its warps use it.
struct alignas(16) Work {
  PackedItem x;
  int hk, rows, pos0, seen_by_all;  // key head; rows that are the sequence's; the first row's place among the keys
  int scrub;                        // first key tile some of whose values were zeroed
  int cuts, unused[2];              // parts of cut units that the CTA had before
  Work() = default;
  __device__ __forceinline__ Work(const PackedItem& item, int hk_, int cuts_, const PackedArgs& a) {
    x = item;
    hk = hk_;
    cuts = cuts_;
    const int t0 = x.tile * a.tpt;  // the tile's first token in its sequence
    rows = min(a.tpt, x.seq.n - t0) * a.G;
    pos0 = x.seq.m - x.seq.n + t0;
    seen_by_all = a.causal ? min(x.seq.m, pos0 + 1) : x.seq.m;
    scrub = kNone;
  }
};

template <int D>
struct Layout {
  static constexpr uint32_t TILE = kTile * D * 2;
  static constexpr int NS = D == 64 ? 2 : 1;  // K/V ring depth: two CTAs on an SM
  static constexpr uint32_t Q = 0;
  static constexpr uint32_t K0 = Q + TILE;
  static constexpr uint32_t V0 = K0 + NS * TILE;
  static constexpr uint32_t BAR = V0 + NS * TILE;
  // FwdBars, then item[2], item_free[2], o_free (O has been read), part (a cut unit's rows are out), last,
  // q_free (an item's last S has been computed)
  static constexpr uint32_t MORE = BAR + FwdBars<NS>::kCount * 8;
  static constexpr uint32_t TSLOT = MORE + 8 * 8;
  static constexpr uint32_t ABORT = TSLOT + 4;
  static constexpr uint32_t LAST = ABORT + 4;  // whether this CTA joins the parts
  static constexpr uint32_t ITEM = (LAST + 4 + 15) & ~15u;  // two of Work
  static constexpr uint32_t BYTES = ITEM + 2 * sizeof(Work);
  static_assert(2 * (BYTES + 1024) <= 233472, "two CTAs an SM");
  // TMEM: S at [0, 128), O behind it; at d = 64 P~ has columns of its own, at d = 128 S's
  static constexpr uint32_t TMEM_COLS = 256;
  static constexpr bool PSEP = D == 64;
  static constexpr uint32_t T_S = 0, T_O = 128, T_P = PSEP ? 192 : 0;
};

template <bool F16>
__device__ __forceinline__ uint32_t times_zero(uint32_t x, uint32_t acc) {  // NaN where a value is not finite
  uint32_t y;
  if constexpr (F16)
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(0), "r"(acc));
  else
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(0), "r"(acc));
  return y;
}
// The halves of a word that are infinite or NaN, as all ones.
template <bool F16>
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  constexpr uint32_t e = F16 ? 0x7C00u : 0x7F80u;
  return ((x & e) == e ? 0xFFFFu : 0u) | ((x >> 16 & e) == e ? 0xFFFF0000u : 0u);
}

// Whether the 128 values rows of the tile at `tile` are all finite; those that are not become 0.
// 1: some were of its first `inside` rows.  A warp calls it.
template <int D, bool F16>
__device__ __forceinline__ bool scrub_tile(uint32_t tile, int inside) {
  const int lane = threadIdx.x & 31;
  constexpr int CHUNKS = kTile * D * 2 / 16;
  uint32_t acc[4] = {0u, 0u, 0u, 0u};
#pragma unroll 8
  for (int i = lane; i < CHUNKS; i += 32) {
    const uint4 v = ld_shared_v4(tile + 16u * (uint32_t)i);
    acc[0] = times_zero<F16>(v.x, acc[0]);
    acc[1] = times_zero<F16>(v.y, acc[1]);
    acc[2] = times_zero<F16>(v.z, acc[2]);
    acc[3] = times_zero<F16>(v.w, acc[3]);
  }
  const bool bad = (not_finite<F16>(acc[0]) | not_finite<F16>(acc[1]) | not_finite<F16>(acc[2]) | not_finite<F16>(acc[3])) != 0u;
  if (!__any_sync(0xffffffffu, bad)) return false;
  bool in = false;
#pragma unroll 1
  for (int i = lane; i < CHUNKS; i += 32) {
    const uint4 v = ld_shared_v4(tile + 16u * (uint32_t)i);
    const uint32_t m[4] = {not_finite<F16>(v.x), not_finite<F16>(v.y), not_finite<F16>(v.z), not_finite<F16>(v.w)};
    if ((m[0] | m[1] | m[2] | m[3]) != 0u) {
      st_shared_v4(tile + 16u * (uint32_t)i, v.x & ~m[0], v.y & ~m[1], v.z & ~m[2], v.w & ~m[3]);
      in |= i % (kTile * 8) / 8 < inside;  // 8 chunks a row of 64 channels
    }
  }
  fence_async_smem();
  return __any_sync(0xffffffffu, in);
}

// Joins the parts of a unit that was cut: with M = max m_s, L = sum l_s 2^((m_s - M) c2),
// O = sum O_s 2^((m_s - M) c2) / L, in the order of the parts.  128 threads, one for each row, of the CTA
// whose part was done last.
template <int D, bool F16>
__device__ __noinline__ void join_parts(const PackedArgs& a, const PackedItem& x, int hk, int r) {
  const int t0 = x.tile * a.tpt;
  if (r >= min(a.tpt, x.seq.n - t0) * a.G) return;
  constexpr size_t words = kTile * (D + 2);
  const size_t step = words * a.Hk;
  const float* base = a.slots + ((size_t)x.first * a.Hk + hk) * words;
  // four (m, l) at a time, so that their loads are on their way together; a part that saw no key, or
  // is none, weighs nothing
  constexpr int ML = 4;
  auto fetch = [&](int s0, float2 (&ml)[ML]) {
#pragma unroll
    for (int k = 0; k < ML; ++k)
      ml[k] = s0 + k < x.parts ? __ldcg(reinterpret_cast<const float2*>(base + (s0 + k) * step + 2 * r)) : make_float2(-INFINITY, 0.f);
  };
  float2 ml[ML];
  float top = -INFINITY, sum = 0.f;
#pragma unroll 1
  for (int s0 = 0; s0 < x.parts; s0 += ML) {
    fetch(s0, ml);
#pragma unroll
    for (int k = 0; k < ML; ++k)
      if (ml[k].y != 0.f) top = fmaxf(top, ml[k].x);
  }
  auto weight = [&](const float2& p) { return p.y == 0.f ? 0.f : p.x == top ? 1.f : ex2((p.x - top) * a.scale_log2); };
#pragma unroll 1
  for (int s0 = 0; s0 < x.parts; s0 += ML) {
    if (x.parts > ML) fetch(s0, ml);
#pragma unroll
    for (int k = 0; k < ML; ++k)
      if (ml[k].y != 0.f) sum = fmaf(weight(ml[k]), ml[k].y, sum);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int i = a.divG.div(r), token = x.seq.q0 + t0 + i, head = hk * a.G + r - i * a.G;
  if (!fa_bounds(a.rep.st, token < a.Tq && head < a.Hq)) return;
  a.lse[(long long)token * a.Hq + head] = sum == 0.f ? -INFINITY : fmaf(top, a.scale, __logf(sum));
  uint16_t* to = static_cast<uint16_t*>(a.o) + (long long)token * a.os[0] + head * a.os[1];
#pragma unroll 1
  for (int c0 = 0; c0 < D; c0 += 32) {
    float acc[32] = {};
#pragma unroll 1
    for (int s0 = 0; s0 < x.parts; s0 += ML) {
      if (x.parts > ML) fetch(s0, ml);
#pragma unroll
      for (int k = 0; k < ML; k += 2) {  // two parts at a time
        float4 v[2][8];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool there = ml[k + e].y != 0.f;
          const float4* from = reinterpret_cast<const float4*>(base + (s0 + k + e) * step + 2 * kTile) + c0 / 4 * kTile + r;
#pragma unroll
          for (int c = 0; c < 8; ++c) v[e][c] = there ? __ldcg(from + c * kTile) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float f = weight(ml[k + e]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            acc[4 * c] = fmaf(f, v[e][c].x, acc[4 * c]);
            acc[4 * c + 1] = fmaf(f, v[e][c].y, acc[4 * c + 1]);
            acc[4 * c + 2] = fmaf(f, v[e][c].z, acc[4 * c + 2]);
            acc[4 * c + 3] = fmaf(f, v[e][c].w, acc[4 * c + 3]);
          }
        }
      }
    }
#pragma unroll
    for (int c = 0; c < 32; c += 8)
      *reinterpret_cast<uint4*>(to + c0 + c) =
          make_uint4(pack2<F16>(acc[c] * inv, acc[c + 1] * inv), pack2<F16>(acc[c + 2] * inv, acc[c + 3] * inv),
                     pack2<F16>(acc[c + 4] * inv, acc[c + 5] * inv), pack2<F16>(acc[c + 6] * inv, acc[c + 7] * inv));
  }
}

// DIRECT: no list; each CTA has one item, which it finds in the offsets, and nothing is cut.
template <int D, bool F16, bool DIRECT>
__global__ void __launch_bounds__(192, 2)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const PackedArgs a) {
  using L = Layout<D>;
  constexpr int NS = L::NS;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (!DIRECT) asm volatile("griddepcontrol.wait;" ::: "memory");  // the list
  const FwdBars<NS> bars{sb + L::BAR};
  auto more = [&](int i) { return sb + L::MORE + 8u * (uint32_t)i; };
  auto bar_item = [&](int k) { return more(k & 1); };
  auto bar_item_free = [&](int k) { return more(2 + (k & 1)); };
  const uint32_t bar_o_free = more(4), bar_part = more(5), bar_last = more(6), bar_q_free = more(7);
  volatile int* abort_cta = reinterpret_cast<volatile int*>(smem + L::ABORT);
  const WaitCtx w{abort_cta, a.rep.st, a.rep.epoch, a.rep.wait_ns};
  if ((sb & 1023u) != 0) {  // the swizzled layouts need a 1024-byte aligned base
    if (threadIdx.x == 0) raise_error(w, FA_ERR_CUDA);
    return;
  }
  // The CTA's k-th item, which the producer puts into shared memory; tile < 0: there is none left.
  // Key tiles are counted through all items (`it`, for the phases of a tile's barriers), and so are
  // the items that have any (n: those of q, q_free and o_free).
  auto place = [&](int k) { return reinterpret_cast<Work*>(smem + L::ITEM) + (k & 1); };
  // producer: its item; K and V copies, items with copies, parts of cut units so far
  PackedItem x{};
  int hk = 0, it = 0, nv = 0, n = 0, cuts = 0, total = 0;
  auto publish = [&](int k) -> bool {  // false: a check of the debug build failed
    // debug build: the tile lies in its sequence, and that in the tensors
    if (x.tile >= 0 && !__all_sync(0xffffffffu, dbg_check(w, x.tile * a.tpt < x.seq.n && x.s0 >= 0 && x.s0 <= x.s1 &&
                                                                 x.s1 <= packed_units(x.seq, a.tpt, true) && x.seq.q0 >= 0 &&
                                                                 x.seq.q0 + x.seq.n <= a.Tq && x.seq.k0 >= 0 &&
                                                                 x.seq.k0 + x.seq.m <= a.Tk && hk < a.Hk)))
      return false;
    if (lane == 0) {
      *place(k) = Work(x, hk, cuts, a);
      mbar_arrive(bar_item(k));
    }
    if (x.tile >= 0 && x.slot >= 0) ++cuts;
    return true;
  };
  auto load_q = [&] {
    mbar_arrive_expect_tx(bars.q(), (uint32_t)(a.tpt * a.G) * D * 2u);
    for (int c = 0; c < D / 64; ++c)
      tma_load_3d(sb + L::Q + c * (kTile * 128), &tmQ, bars.q(), c * 64, hk * a.G, x.seq.q0 + x.tile * a.tpt);
  };
  auto load_tile = [&](const CUtensorMap* tm, uint32_t to, uint32_t on, int kt) {
    mbar_arrive_expect_tx(on, L::TILE);
    for (int c = 0; c < D / 64; ++c)
      tma_load_3d(to + c * (kTile * 128), tm, on, c * 64, hk, x.seq.k0 + kt * kTile);
  };
  bool go = true;
  if (warp == 4) {
    PackedOffsets cu{};
    if (DIRECT) cu = packed_lane_offsets(a);  // on their way beside the barriers' set-up
    if (lane == 0) {
      bars.init();
      for (int k = 0; k < 2; ++k) {
        mbar_init(bar_item(k), 1);
        mbar_init(bar_item_free(k), 5);
      }
      mbar_init(bar_o_free, 4);
      mbar_init(bar_part, 4);
      mbar_init(bar_last, 1);
      mbar_init(bar_q_free, 1);
      *abort_cta = 0;
      fence_barrier_init();
    }
    __syncwarp();
    // the first item is the CTA's own
    const int index = (int)blockIdx.x, at = a.divHk.div(index);
    hk = index - at * a.Hk;
    if (DIRECT) {
      if (!packed_direct(a, cu, at, x)) x.tile = -1;
    } else {  // there is room for it in the list: on its way beside the list's length
      total = a.list.head[0] * a.Hk;
      x = a.list.items[at];
      if (index >= total) x.tile = -1;
    }
    go = publish(0);
    // its copies that need no wait go beside the rest of the set-up
    if (go && x.tile >= 0 && x.s0 < x.s1) {
      n = 1;
      if (lane == 0) load_q();
      for (; it < NS && x.s0 + it < x.s1; ++it, ++nv)
        if (lane == 0) {
          load_tile(&tmK, sb + L::K0 + it * L::TILE, bars.kf(it), x.s0 + it);
          load_tile(&tmV, sb + L::V0 + it * L::TILE, bars.vf(it), x.s0 + it);
        }
    }
  }
  if (warp == 5) {
    tmem_alloc(sb + L::TSLOT, L::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::TSLOT);

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    for (int k = 0; go && x.tile >= 0; ) {
      if (x.s0 < x.s1) {  // some row sees a key
        if (k > 0) {
          if (n > 0 && !(go = warp_wait(w, bar_q_free, (n - 1) & 1))) break;
          if (lane == 0) load_q();
          ++n;
        }
        for (int kt = x.s0 + (k == 0 ? it : 0); kt < x.s1; ++kt) {
          const int st = it % NS;
          const uint32_t ph = ((it / NS) - 1) & 1;
          if (it >= NS && !(go = warp_wait(w, bars.ke(st), ph))) break;
          if (lane == 0) load_tile(&tmK, sb + L::K0 + st * L::TILE, bars.kf(st), kt);
          ++it;
          if (nv >= NS && !(go = warp_wait(w, bars.ve(st), ph))) break;
          if (lane == 0) load_tile(&tmV, sb + L::V0 + st * L::TILE, bars.vf(st), kt);
          ++nv;
        }
        if (!go) break;
      }
      if (DIRECT) break;
      // the next one: taken in order as CTAs come to need them
      ++k;
      int index = 0;
      if (lane == 0) index = (int)gridDim.x + atomicAdd(a.list.head + 4, 1);
      index = __shfl_sync(0xffffffffu, index, 0);
      if (k >= 2 && !(go = warp_wait(w, bar_item_free(k), ((k >> 1) - 1) & 1))) break;
      const int at = a.divHk.div(index);
      hk = index - at * a.Hk;
      x.tile = -1;
      if (index < total) x = a.list.items[at];
      if (!(go = publish(k))) break;
    }
    if (lane == 0) {  // every copy has landed before the CTA ends
      if (n > 0) mbar_drain(w, bars.q(), (n - 1) & 1);
      for (int st = 0; st < NS; ++st) {
        const int ck = (it - st + NS - 1) / NS, cv = (nv - st + NS - 1) / NS;  // copies into stage st
        if (ck > 0) mbar_drain(w, bars.kf(st), (ck - 1) & 1);
        if (cv > 0) mbar_drain(w, bars.vf(st), (cv - 1) & 1);
      }
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    // The schedule of fwd_common.cuh for each item: at d = 64 S_{j+1} as soon as S_j has been copied out,
    // at d = 128 after P~ V_j.  An item's first S goes beside the last one's way out.
    constexpr uint32_t idS = idesc_f16(F16, kTile, kTile, false, false);
    constexpr uint32_t idO = idesc_f16(F16, kTile, D, false, true);
    const uint32_t tS = tmem + L::T_S, tO = tmem + L::T_O;
    const uint64_t dQ = desc_kmajor_base(sb + L::Q);
    const uint64_t dK0 = desc_kmajor_base(sb + L::K0);
    const uint64_t dV0 = desc_mnmajor_base(sb + L::V0, kTile);
    auto s_tile = [&](int it, bool last) -> bool {  // S = Q K^T; last: of the item
      const int st = it % NS;
      if (!warp_wait(w, bars.kf(st), (it / NS) & 1)) return false;
      tc_fence_after();
      const uint64_t dK = desc_add(dK0, (uint32_t)st * L::TILE);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        tc_mma_ss_elect(tS, dQ + kmajor_step(kk, kTile), dK + kmajor_step(kk, kTile), idS, kk > 0 ? 1u : 0u);
      tc_commit_elect(bars.s());
      tc_commit_elect(bars.ke(st));
      if (last) tc_commit_elect(bar_q_free);
      return true;
    };
    bool ok = true;
    int it = 0, n = 0;
    for (int k = 0; ok; ++k) {
      if (!(ok = warp_wait(w, bar_item(k), (k >> 1) & 1))) break;
      Work* x = place(k);
      const int tile = x->x.tile, s0 = x->x.s0, s1 = x->x.s1, m = x->x.seq.m, seen_by_all = x->seen_by_all;
      if (tile >= 0 && s0 < s1) {
        if (!(ok = warp_wait(w, bars.q(), n & 1))) break;
        if (L::PSEP && it > 0 && !(ok = warp_wait(w, bars.sfree(), (it - 1) & 1))) break;
        if (!(ok = s_tile(it, s0 + 1 == s1))) break;
        for (int kt = s0; kt < s1; ++kt, ++it) {
          const int st = it % NS;
          const bool next = kt + 1 < s1;
          if (L::PSEP && next) {
            if (!(ok = warp_wait(w, bars.sfree(), it & 1))) break;
            if (!(ok = s_tile(it + 1, kt + 2 == s1))) break;
          }
          if (kt * kTile + kTile > seen_by_all) {  // some row does not see all of it: its values are looked over
            if (!(ok = warp_wait(w, bars.vf(st), (it / NS) & 1))) break;
            if (scrub_tile<D, F16>(sb + L::V0 + st * L::TILE, m - kt * kTile) && lane == 0 && x->scrub == kNone) {
              x->scrub = kt;
              __threadfence_block();
            }
            __syncwarp();
          }
          if (!(ok = warp_wait(w, bars.p(), it & 1))) break;
          if (!(ok = warp_wait(w, bars.vf(st), (it / NS) & 1))) break;
          if (kt == s0 && n > 0 && !(ok = warp_wait(w, bar_o_free, (n - 1) & 1))) break;
          tc_fence_after();
          const uint64_t dV = desc_add(dV0, (uint32_t)st * L::TILE);
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)  // O += P~ V
            tc_mma_ts_elect(tO, tmem + L::T_P + (uint32_t)kk * 8u, dV + mnmajor_step(kk), idO,
                            (kt > s0 || kk > 0) ? 1u : 0u);
          tc_commit_elect(bars.o());
          tc_commit_elect(bars.ve(st));
          if (!L::PSEP && next && !(ok = s_tile(it + 1, kt + 2 == s1))) break;
        }
        if (!ok) break;
        ++n;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_item_free(k));
      if (DIRECT || tile < 0) break;
    }
    tc_commit_elect(bars.fin());
    if (lane == 0) mbar_drain(w, bars.fin(), 0);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const int r = threadIdx.x;
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const uint32_t tS = tmem + L::T_S + lane_off, tO = tmem + L::T_O + lane_off;
    const float c2 = a.scale_log2;
    bool ok = true;
    int it = 0;
    for (int k = 0; ok; ++k) {
      if (!(ok = warp_wait(w, bar_item(k), (k >> 1) & 1))) break;
      // keys that the row sees (formed where it is wanted: the loop has no registers to spare)
      auto limit = [&](const Work* x) { return a.causal ? min(x->x.seq.m, x->pos0 + a.divG.div(r) + 1) : x->x.seq.m; };
      if (place(k)->x.tile < 0) break;
      const int first = it, end = it + place(k)->x.s1 - place(k)->x.s0;
      const int masked = it + (place(k)->seen_by_all >> 7) - place(k)->x.s0;  // tiles from here on hide a key from some row
      static_assert(kTile == 128, "of the shift");
      float m_use = -INFINITY;  // running maximum in use, of the products
      float l = 0.f;
      for (; it < end; ++it) {
        if (!(ok = warp_wait(w, bars.s(), it & 1))) break;
        tc_fence_after();
        float s[kTile];
        float m8[8];
        {
          uint32_t u[64], v[64];
          tmem_ld64(tS, u);
          tmem_ld64_nowait(tS + 64, v);
#pragma unroll
          for (int c = 0; c < 64; ++c) s[c] = __uint_as_float(u[c]);
#pragma unroll
          for (int j = 0; j < 4; ++j) m8[j] = max16(s, j);
          tmem_wait_ld64(v);
#pragma unroll
          for (int c = 0; c < 64; ++c) s[64 + c] = __uint_as_float(v[c]);
        }
        if (L::PSEP) {  // S_j is in registers: the MMA warp may compute S_{j+1}
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars.sfree());
        }
        if (it >= masked) {
          const Work* x = place(k);
          const int low = limit(x) - (x->x.s1 - (end - it)) * kTile;
#pragma unroll
          for (int c = 0; c < kTile; ++c)
            if (c >= low) s[c] = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; ++j) m8[j] = max16(s, j);
        }
#pragma unroll
        for (int j = 4; j < 8; ++j) m8[j] = max16(s, j);
        const float mx = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
        float alpha = 1.f;
        if ((mx - m_use) * c2 > kRescaleThr) {
          alpha = ex2((m_use - mx) * c2);  // 0 on the first tile that sees a key
          m_use = mx;
        }
        float mneg = m_use == -INFINITY ? 0.f : -m_use * c2;
        // (rows that are not the sequence's, of other sequences or of nobody, have no say in it: results
        // do not depend on what is there)
        if (__any_sync(0xffffffffu, fabsf(mneg) > kLargeScore) &&
            __any_sync(0xffffffffu, fabsf(mneg) > kLargeScore && r < place(k)->rows)) {
          // the rounded maximum would be off by more than 2^-8: the difference first, which is
          // exact near the maximum
          const float top = m_use == -INFINITY ? 0.f : m_use;
#pragma unroll
          for (int c = 0; c < kTile; ++c) s[c] -= top;
          mneg = 0.f;
        }
        const uint64_t c2p = f2pack(c2, c2), mp = f2pack(mneg, mneg);
        uint64_t acc[4] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f), f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
        // four chunks of 32 keys, each chunk's P~ stored as soon as it is formed; P~ is rounded to the
        // inputs' type (half a step of each weight), l adds the fp32 weights
        bool o_ready = !(L::PSEP && it > first);
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t pk[16];
#pragma unroll
          for (int pr = 0; pr < 16; ++pr) {
            const int c = 32 * ch + 2 * pr;
            float x0, x1;
            f2unpack(ffma2(f2pack(s[c], s[c + 1]), c2p, mp), x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            acc[pr & 3] = fadd2(acc[pr & 3], f2pack(p0, p1));
            pk[pr] = pack2<F16>(p0, p1);
          }
          if (!o_ready) {  // P~ V_{j-1} reads the P~ columns and writes O
            if (!(ok = warp_wait(w, bars.o(), (it - 1) & 1))) break;
            tc_fence_after();
            o_ready = true;
          }
          tmem_st16(tmem + L::T_P + lane_off + 16 * ch, pk);
        }
        if (!ok) break;
        // (before a row's first key its O is 0, or of the item before)
        if (__any_sync(0xffffffffu, alpha != 1.f && l != 0.f)) scale_o_row<D>(tO, alpha);
        l = l * alpha + sum_packed4(acc);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.p());
      }
      // ------------------------------------------------------------ the item's results
      const Work* x = place(k);
      const bool have_o = x->x.s0 < x->x.s1;
      if (!ok || (have_o && !(ok = warp_wait(w, bars.o(), (it - 1) & 1)))) break;
      tc_fence_after();
      const int i = a.divG.div(r), token = x->x.seq.q0 + x->x.tile * a.tpt + i, hk = x->hk, head = hk * a.G + r - i * a.G;
      const bool live = r < x->rows;
      const int slot = x->x.slot;
      const bool whole = DIRECT || slot < 0;
      const float inv_l = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;  // a NaN stays one
      float* part = whole ? nullptr : a.slots + ((long long)slot * a.Hk + hk) * (kTile * (D + 2));
      if (whole) {
        if (live) a.lse[(long long)token * a.Hq + head] = l == 0.f ? -INFINITY : fmaf(m_use, a.scale, __logf(l));
      } else {
        *reinterpret_cast<float2*>(part + 2 * r) = make_float2(m_use, l);
      }
      // values that were zeroed: added to the rows that see them
      const int from = *reinterpret_cast<const volatile int*>(&x->scrub);
      const bool patch = from != kNone;
      const uint16_t* vrow = static_cast<const uint16_t*>(a.v) + (long long)x->x.seq.k0 * a.vs[0] + hk * a.vs[1];
      const int last_key = min(limit(x), x->x.s1 * kTile);
      uint16_t* dst = static_cast<uint16_t*>(a.o) + (long long)token * a.os[0] + head * a.os[1];
      // (rolled: an item's end is bound by the fetching of its instructions; unrolled, 12 sequences of up to
      // 16384 tokens take 7.6 ms and not 7.3, 4 of up to 2048 28.0 us and not 27.7)
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        if (have_o) {
          tmem_ld32(tO + c0, o);
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = 0u;
        }
        if (!DIRECT && have_o && c0 + 32 == D) {  // all is in registers: the next item's O may go there
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_o_free);
        }
        if (patch && live) {
#pragma unroll 1
          for (int j = from * kTile; j < last_key; ++j)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const uint4 u = __ldg(reinterpret_cast<const uint4*>(vrow + j * a.vs[0] + c0) + v);
              const uint32_t h[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const float2 f = unpack2<F16>(h[c] & not_finite<F16>(h[c]));
                o[8 * v + 2 * c] = __float_as_uint(__uint_as_float(o[8 * v + 2 * c]) + f.x);
                o[8 * v + 2 * c + 1] = __float_as_uint(__uint_as_float(o[8 * v + 2 * c + 1]) + f.y);
              }
            }
        }
        if (whole && live) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint4 q;
            q.x = pack2<F16>(__uint_as_float(o[v * 8 + 0]) * inv_l, __uint_as_float(o[v * 8 + 1]) * inv_l);
            q.y = pack2<F16>(__uint_as_float(o[v * 8 + 2]) * inv_l, __uint_as_float(o[v * 8 + 3]) * inv_l);
            q.z = pack2<F16>(__uint_as_float(o[v * 8 + 4]) * inv_l, __uint_as_float(o[v * 8 + 5]) * inv_l);
            q.w = pack2<F16>(__uint_as_float(o[v * 8 + 6]) * inv_l, __uint_as_float(o[v * 8 + 7]) * inv_l);
            *reinterpret_cast<uint4*>(dst + c0 + v * 8) = q;
          }
        } else if (!whole) {
          // four channels of all rows side by side: a warp's stores are whole lines
          float* to = part + 2 * kTile + 4 * (c0 / 4 * kTile + r);
#pragma unroll
          for (int v = 0; v < 8; ++v)
            *reinterpret_cast<uint4*>(to + 4 * kTile * v) = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
        }
        __syncwarp();
      }
      if (!whole) {  // the last of the unit's parts to be done joins them
        // (the rows' stores are ordered before the count by the barrier within the CTA, which is one
        // lane's to see, and by that lane's fence)
        volatile int* last = reinterpret_cast<volatile int*>(smem + L::LAST);
        if (lane == 0) mbar_arrive(bar_part);
        if (warp == 0) {
          if (!(ok = warp_wait(w, bar_part, x->cuts & 1))) break;
          if (lane == 0) {
            __threadfence();
            const bool done = atomicAdd(a.list.left + x->x.cut * a.Hk + hk, 1) == x->x.parts - 1;
            __threadfence();
            *last = done;
            mbar_arrive(bar_last);
          }
          __syncwarp();
        }
        if (!(ok = warp_wait(w, bar_last, x->cuts & 1))) break;
        if (*last) join_parts<D, F16>(a, x->x, hk, r);
        __syncwarp();
      }
      if (DIRECT) break;
      if (lane == 0) mbar_arrive(bar_item_free(k));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

template <int D, bool F16, bool DIRECT>
cudaError_t launch_t(const PackedArgs& a, const CUtensorMap* tm, int items, cudaStream_t s) {
  using L = Layout<D>;
  const auto kern = packed_fwd_kernel<D, F16, DIRECT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::BYTES);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = DIRECT ? 0 : 1;
  cfg.stream = s;
  // CTAs that stay and take one item after the other; without a list an item each
  const long long all = (long long)items * a.Hk;
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cfg.gridDim = dim3((unsigned)(DIRECT ? all : std::min(all, 2ll * sms)));
  cfg.blockDim = dim3(192);
  cfg.dynamicSmemBytes = L::BYTES;
  return cudaLaunchKernelEx(&cfg, kern, tm[0], tm[1], tm[2], a);
}

template <int D, bool F16>
cudaError_t launch_any(const PackedArgs& a, const CUtensorMap* tm, int items, cudaStream_t s) {
  return a.direct ? launch_t<D, F16, true>(a, tm, items, s) : launch_t<D, F16, false>(a, tm, items, s);
}

}  // namespace

cudaError_t launch_packed_fwd(const PackedArgs& a, int d, bool f16, const CUtensorMap* tm, int items, cudaStream_t s) {
  if (d == 64) return f16 ? launch_any<64, true>(a, tm, items, s) : launch_any<64, false>(a, tm, items, s);
  return f16 ? launch_any<128, true>(a, tm, items, s) : launch_any<128, false>(a, tm, items, s);
}

}  // namespace fa
