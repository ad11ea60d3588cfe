// packed_bwd.cu -- attention backward of packed sequences with grouped heads: the main kernel.
//
// The tiled recomputation of bwd_tc.cu ("Passe arrière : recalculer au lieu de stocker",
// marketmaker.cc): one CTA holds a 128-key tile (K_j, V_j) of a sequence and key head, accumulates
// dK_j and dV_j in TMEM and walks the query tiles that see it,
//   S^T = K_j Q_i^T, P^T = exp(scale S^T - LSE_i), dP^T = V_j dO_i^T, dV += P^T dO_i,
//   dS^T = P^T (dP^T - D_i), dK += dS^T Q_i, dQ_i = dS K_j (added to an fp32 accumulator by TMA).
// A query tile is tpt tokens times the G query heads of the key head (row = token * G + head), so
// that the sum over a group's heads is part of the products' sums: dK and dV of shared heads
// need no pass of their own, and their order is fixed.  The CTAs stay and take the list that
// packed_plan.cu makes, key tiles by the query tiles they visit, the longest first: the next tile's
// copies and first products run beside the last one's results' way out (1520 sequences of 512
// tokens, one head, d = 64: 417 us with a CTA for each tile, 345 so, and 347 with the weights as below).  A tile longer than an even share is cut; its
// parts are fp32 sums that the last kernel adds.
//
// What lies behind a sequence's end in its last tiles is another sequence's or nobody's: rows of
// Q, dO and K there are zeroed in shared memory before the products read them, dS of hidden pairs
// is 0, and rows of dQ there are added as 0.
//
// In fp16 P^T and dS^T are kept where the type has all its bits, and below its largest number: P times
// 2^13, and dS, for a sequence and key head, times the power of two that its largest |dO|, |V| and |D|
// allow (|dP - D| <= |dO| |V| + |D|).  The gradients take both back, exactly, in fp32.  (Without them a
// weight over 2^16 keys has eight bits, and dS over 4096 keys of a dO of 2^-13 is 0.)  bf16 needs neither.
// It costs a pass over V, the maxima and their way to the tiles: 4 sequences up to 2048 tokens, 12 heads,
// d = 64, 72.4 us and 65.0 in bf16; 12 up to 8192, 32 and 8 heads, d = 128, 6.26 ms and 6.23.
//
// P is exp((scale S) - LSE), the product rounded as the forward rounds it into LSE, so that a key with all
// of the weight has exactly 1 however large the scores are (as 2^(scale log2 e S - log2 e LSE), one fma,
// 0.98 at a score of 10^6 and 0.80 at 2^24).  Three instructions for one cost 4 sequences up to 2048 tokens, d =
// 64, 1.8 us of 64, and two where scale is a power of two, whose products need no rounding, 0.8; at d = 128
// 12 up to 8192 5 to 20 us of 6220; looking for large scores and a way of their own cost 2.5 to 4 of the 64.
//
// Bound: the tensor core (five products, 10 d FLOPs a seen pair and query head) beside the
// exponentials and the elementwise steps; one CTA an SM.  Measured, causal, with the kernels before
// and behind it: 12 sequences of up to 8192 tokens, 32 and 8 heads, d = 128, 951 TFLOP/s (6.23 ms).
//
// Warp roles as in bwd_tc.cu: 4 NG compute warps in NG groups that split the 128 query
// columns of a tile (TMEM lane = key row); a producer warp; a warp that owns TMEM and issues the
// products; at d = 64 four warps that read dQ_i out of TMEM.
#include <algorithm>
#include <cmath>

#include "packed.h"
#include "ptx.cuh"
#include "tiles.cuh"

namespace fa {
namespace {

// fp16: log2 of the factor of P^T (P is at most 1, but for roundings of the scores), and its reciprocal.
constexpr float kPScale = 13.f, kPDown = 0x1p-13f;
constexpr float kLog2e = 1.4426950408889634f;
// fp16: the factor of dS of a sequence and key head, from its largest |dO|^2 < 2^(x + 1), |V|^2 < 2^(y + 1)
// and |D| < 2^(z + 1): |dP - D| < 2^((x + y + 2) / 2) + 2^(z + 1) <= 2^e, and 2^(1 - e) brings that to 2, so
// that 2^13 P |dP - D| stays below 2^14 and what is 2^-26 of that has all its bits.  (At most 2^60: the bound
// of numbers that are not 0 is 2^-48 at least, and no dP of fp16 numbers times that is infinite, also not in rows
// that have no say in it, whose P is 0.)
__device__ __forceinline__ float dS_up(const float4& most) {
  auto exponent = [](float f) { return (int)(__float_as_uint(f) >> 23) - 127; };  // -127 of 0
  const int e = max((exponent(most.x) + exponent(most.y) + 3) >> 1, exponent(most.z) + 1) + 1;
  return __uint_as_float((uint32_t)min(max(128 - e, 1), 187) << 23);
}
// Here and not where it is used, so that it is on its way beside other loads.
__device__ __forceinline__ float4 ld_early(const float4* p) {
  float4 v;
  asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}
// Of a power of two.
__device__ __forceinline__ float reciprocal(float x) { return __uint_as_float(0x7F000000u - __float_as_uint(x)); }

// A CTA's item as its warps use it.
struct alignas(16) Work {
  int tile, s0, s1, slot;
  int hk, key0, keys, first_key;  // the tile's first row of k; its keys; the query that is its first key's
  int q_last, last_rows, whole_from, q_row0;  // the last query tile and its rows; tiles from which on all see all
  Work() = default;
  __device__ __forceinline__ Work(const PackedItem& x, int hk_, const PackedArgs& a) {
    tile = x.tile;
    s0 = x.s0;
    s1 = x.s1;
    slot = x.slot;
    hk = hk_;
    if (tile < 0) return;
    const int at = tile * kTile, ahead = x.seq.m - x.seq.n;
    key0 = x.seq.k0 + at;
    keys = min(kTile, x.seq.m - at);
    first_key = at - ahead;
    q_last = (x.seq.n - 1) / a.tpt;
    last_rows = (x.seq.n - q_last * a.tpt) * a.G;
    // keys behind the sequence's end are seen by no query
    whole_from = keys < kTile ? 0x7FFFFFFF : !a.causal ? 0 : max(0, (first_key + keys - 1 + a.tpt - 1) / a.tpt);
    q_row0 = x.seq.q0 * a.G;
  }
};

template <int D>
struct Layout {
  static constexpr int NG = D == 64 ? 4 : 2;  // compute warpgroups (d = 128: a warp's dQ box is its own dS^T rows)
  static constexpr int CW = kTile / NG;       // query columns of a warpgroup
  static constexpr int KPG = CW / 16;
  static constexpr int NCW = 4 * NG;
  static constexpr bool QW = D == 64;         // warps of their own for dQ
  static constexpr int NQW = QW ? 4 : 0;
  static constexpr int NT = 32 * (NCW + 2 + NQW);
  static constexpr int DQG = D / NG;
  static constexpr int DQC = 32;              // columns of a dQ box of 32 rows
  static constexpr uint32_t BOXB = 32u * DQC * 4u;
  static constexpr int DQ_READERS = QW ? NQW : NCW;
  static constexpr uint32_t TILE = kTile * D * 2;
  static constexpr int NS = D == 64 ? 3 : 2;  // Q/dO ring depth
  static constexpr uint32_t K = 0;
  static constexpr uint32_t V = TILE;
  static constexpr uint32_t QS = 2 * TILE;    // stage s: Q at QS + 2 s TILE, dO behind it
  static constexpr int NDS = D == 64 ? 2 : 1;
  static constexpr uint32_t DSB = kTile * kTile * 2;
  static constexpr uint32_t DST = QS + NS * 2 * TILE;
  static constexpr uint32_t STAT = DST + NDS * DSB;  // per stage -LSE [128], -D [128]
  static constexpr bool STG_SEP = D == 64;           // dQ boxes: of their own, or over dS^T
  static constexpr uint32_t STG_BYTES = (QW ? NQW : NCW) * BOXB;
  static constexpr uint32_t STG = STG_SEP ? STAT + NS * 256 * 4 : DST;
  static_assert(STG_SEP || STG_BYTES == DSB, "staging size");
  static constexpr uint32_t BAR = STAT + NS * 256 * 4 + (STG_SEP ? STG_BYTES : 0);
  // 0 kv, 1 s_full, 2 dp_full, 3 dp_free, 4 p_full, 5 ds_full, 6 dq_full, 7 dq_free, 8 done,
  // 9 pt_free, 10 tail (copies of tiles whose rows are to be zeroed), 11 acc_free (dV and dK read),
  // 12.. item[2], item_free[2], q_full[NS], q_empty[NS], ds_free[NDS]
  static constexpr uint32_t NBAR = 16 + 2 * NS + NDS;
  static constexpr uint32_t TSLOT = BAR + NBAR * 8;
  static constexpr uint32_t ABORT = TSLOT + 4;
  static constexpr uint32_t ITEM = (ABORT + 4 + 15) & ~15u;  // two of Work
  static constexpr uint32_t UP = ITEM + 2 * sizeof(Work);  // fp16: their factors of dS, twice, there before the first tile's bar_qf
  static constexpr uint32_t BYTES = UP + 2 * 8;
  static_assert(BYTES <= 232448, "shared memory per CTA");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t T_S = 0, T_DP = 128, T_DV = 256, T_DK = 256 + D;
  static constexpr bool ALIAS = D == 128;  // dQ over dP^T, P^T over S^T
  static constexpr uint32_t T_DQ = ALIAS ? T_DP : 384;
  static constexpr uint32_t T_PT = ALIAS ? T_S : 448;
  __device__ static constexpr uint32_t pt_col(int kk) {
    return ALIAS ? (uint32_t)CW * (uint32_t)(kk / KPG) + 8u * (uint32_t)(kk % KPG) : T_PT + 8u * (uint32_t)kk;
  }
  __device__ static constexpr uint32_t pt_write_col(int g) {
    return ALIAS ? (uint32_t)CW * (uint32_t)g : T_PT + (uint32_t)(CW / 2) * (uint32_t)g;
  }
};

// Rows [from, 128) of a tile in shared memory become 0 (a warp's lanes, or `n` threads).
template <int D>
__device__ __forceinline__ void zero_rows(uint32_t tile, int from, int t, int n) {
  const int chunks = (kTile - from) * 8;  // 16-byte chunks of the rows of an atom of 64 channels
#pragma unroll
  for (int c = 0; c < D / 64; ++c)
    for (int i = t; i < chunks; i += n) st_shared_v4(tile + (uint32_t)(c * kTile * 128 + from * 128 + 16 * i), 0u, 0u, 0u, 0u);
}

// EXACT: scale is a power of two (1 / 8 at d = 64), so that no product with it is rounded.
template <int D, bool F16, bool EXACT>
__global__ void __launch_bounds__(Layout<D>::NT, 1)
    packed_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                      const __grid_constant__ CUtensorMap tmdQ, const PackedArgs a) {
  using L = Layout<D>;
  constexpr int NS = L::NS;
  constexpr int kProd = L::NCW, kMma = L::NCW + 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.wait;" ::: "memory");  // the list, the rows' statistics, the zeroed accumulator
  const int tpt = a.tpt, G = a.G, full = tpt * G;

  auto bar = [&](int i) { return sb + L::BAR + 8u * (uint32_t)i; };
  const uint32_t bar_kv = bar(0), bar_s_full = bar(1), bar_dp_full = bar(2), bar_dp_free = bar(3), bar_p_full = bar(4),
                 bar_ds_full = bar(5), bar_dq_full = bar(6), bar_dq_free = bar(7), bar_done = bar(8),
                 bar_pt_free = bar(9), bar_tail = bar(10), bar_acc_free = bar(11);
  auto bar_item = [&](int k) { return bar(12 + (k & 1)); };
  auto bar_item_free = [&](int k) { return bar(14 + (k & 1)); };
  auto bar_qf = [&](int s) { return bar(16 + s); };
  auto bar_qe = [&](int s) { return bar(16 + NS + s); };
  auto bar_ds_free = [&](int b) { return bar(16 + 2 * NS + b); };

  volatile int* abort_cta = reinterpret_cast<volatile int*>(smem + L::ABORT);
  const WaitCtx w{abort_cta, a.rep.st, a.rep.epoch, a.rep.wait_ns};
  if ((sb & 1023u) != 0) {
    if (threadIdx.x == 0) raise_error(w, FA_ERR_CUDA);
    return;
  }
  if (warp == kProd && lane == 0) {
    mbar_init(bar_kv, 2);
    mbar_init(bar_s_full, 1);
    mbar_init(bar_dp_full, 1);
    mbar_init(bar_dp_free, L::NCW);
    mbar_init(bar_p_full, L::NCW);
    mbar_init(bar_ds_full, L::NCW);
    for (int b = 0; b < L::NDS; ++b) mbar_init(bar_ds_free(b), 1);
    mbar_init(bar_dq_full, 1);
    mbar_init(bar_dq_free, L::DQ_READERS);
    mbar_init(bar_done, 1);
    mbar_init(bar_pt_free, 1);
    mbar_init(bar_tail, 1);
    mbar_init(bar_acc_free, L::NCW);
    for (int k = 0; k < 2; ++k) {
      mbar_init(bar_item(k), 1);
      mbar_init(bar_item_free(k), L::NCW + 1 + L::NQW);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar_qf(s), 1 + 32);  // the copies' arrival and every producer lane
      mbar_init(bar_qe(s), 1);
    }
    *abort_cta = 0;
    fence_barrier_init();
  }
  if (full < kTile) {  // rows that no copy writes
    for (int s = 0; s < 2 * NS; ++s) zero_rows<D>(sb + L::QS + (uint32_t)s * L::TILE, full, (int)threadIdx.x, L::NT);
    fence_async_smem();
  }
  if (warp == kMma) {
    tmem_alloc(sb + L::TSLOT, L::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::TSLOT);
  // The CTA's k-th item, which the producer puts into shared memory; tile < 0: there is none left.
  // Steps are counted through all items (`it`, for the phases of a step's barriers), and so are the
  // items that have steps (those of kv, done and acc_free); an item without any, whose results
  // are 0, passes no barrier but its own two.
  auto place = [&](int k) { return reinterpret_cast<Work*>(smem + L::ITEM) + (k & 1); };
  auto place_up = [&](int k) { return reinterpret_cast<float2*>(smem + L::UP) + (k & 1); };

  if (warp == kProd) {
    // ------------------------------------------------------------ producer
    int it = 0, tails = 0, loads = 0;  // stages copied; copies on bar_tail; K_j, V_j copied
    const int total = a.list.head[0] * a.Hk;
    bool go = true;
    for (int k = 0; go; ++k) {
      // the first item is the CTA's own, the others are taken in order as CTAs come to need them
      int index = 0;
      if (lane == 0) index = k == 0 ? (int)blockIdx.x : (int)gridDim.x + atomicAdd(a.list.head + 4, 1);
      index = __shfl_sync(0xffffffffu, index, 0);
      if (k >= 2 && !(go = warp_wait(w, bar_item_free(k), ((k >> 1) - 1) & 1))) break;
      const int at = a.divHk.div(index), hk = index - at * a.Hk;
      PackedItem x;
      x.tile = -1;
      if (k == 0 || index < total) x = a.list.items[at];  // (for the first there is room in the list)
      if (index >= total) x.tile = -1;
      // debug build: the tile lies in its sequence, and that in the tensors
      if (x.tile >= 0 && !__all_sync(0xffffffffu, dbg_check(w, x.tile * kTile < x.seq.m && x.s0 >= 0 && x.s0 <= x.s1 &&
                                                                   x.s1 <= packed_units(x.seq, tpt, false) && x.seq.q0 >= 0 &&
                                                                   x.seq.q0 + x.seq.n <= a.Tq && x.seq.k0 >= 0 &&
                                                                   x.seq.k0 + x.seq.m <= a.Tk && hk < a.Hk)))
        break;
      if (lane == 0) {
        *place(k) = Work(x, hk, a);
        mbar_arrive(bar_item(k));
      }
      if (x.tile < 0) break;
      if (x.s0 == x.s1) continue;  // no query sees the tile
      const int kt = x.tile, keys = min(kTile, x.seq.m - kt * kTile);
      const int q_last = (x.seq.n - 1) / tpt, last_rows = (x.seq.n - q_last * tpt) * G;
      const float* lse = a.stat_lse + (long long)hk * a.Tq * G;
      const float* dsum = a.stat_d + (long long)hk * a.Tq * G;
      const uint32_t q_bytes = (uint32_t)full * D * 2u;
      float up = 1.f;
      float4 most{};
      if (F16) most = ld_early(a.most + (long long)x.r * a.Hk + hk);
      // Q and dO of the first query tiles go ahead of K_j and V_j, whose places are free when the last
      // item's products are done; one stage is freed by those products only.  (A CTA's first K_j and V_j at
      // once: at d = 64 4 sequences of up to 2048 tokens 66.8 and 67.7 us; at d = 128 it gains nothing.)
      const int ahead = D == 64 && loads == 0 ? x.s0 : min(x.s0 + NS - 1, x.s1);
      for (int qt = x.s0; go && qt <= x.s1; ++qt) {
        if (qt == ahead) {
          if (loads > 0 && !(go = warp_wait(w, bar_done, (loads - 1) & 1))) break;
          const bool tail = keys < kTile;  // rows behind the sequence's end
          if (lane == 0) {
            mbar_arrive_expect_tx(bar_kv, (tail ? 1u : 2u) * L::TILE);
            if (tail) mbar_arrive_expect_tx(bar_tail, L::TILE);
            for (int c = 0; c < D / 64; ++c) {
              tma_load_3d(sb + L::K + c * (kTile * 128), &tmK, tail ? bar_tail : bar_kv, c * 64, hk, x.seq.k0 + kt * kTile);
              tma_load_3d(sb + L::V + c * (kTile * 128), &tmV, bar_kv, c * 64, hk, x.seq.k0 + kt * kTile);
            }
          }
          ++loads;
          if (tail) {
            if (!(go = warp_wait(w, bar_tail, tails++ & 1))) break;
            zero_rows<D>(sb + L::K, keys, lane, 32);
            fence_async_smem();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(bar_kv);
        }
        if (qt == x.s1) break;
        const int s = it % NS, rows = qt == q_last ? last_rows : full, token = x.seq.q0 + qt * tpt;
        // statistics, negated as the compute warps use them, loaded before the wait for the stage
        const long long row0 = (long long)token * G;
        float l4[4], d4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 4 * lane + i;
          l4[i] = r < rows ? -__ldg(lse + row0 + r) : -INFINITY;
          d4[i] = r < rows ? -__ldg(dsum + row0 + r) : 0.f;
        }
        if (it >= NS && !(go = warp_wait(w, bar_qe(s), ((it / NS) - 1) & 1))) break;
        const bool tail = rows < full;  // the sequence's last query tile
        const uint32_t dst = sb + L::QS + (uint32_t)s * 2u * L::TILE;
        if (lane == 0) {
          const uint32_t on = tail ? bar_tail : bar_qf(s);
          mbar_arrive_expect_tx(on, 2 * q_bytes);
          for (int c = 0; c < D / 64; ++c) {
            tma_load_3d(dst + c * (kTile * 128), &tmQ, on, c * 64, hk * G, token);
            tma_load_3d(dst + L::TILE + c * (kTile * 128), &tmdO, on, c * 64, hk * G, token);
          }
        }
        if (F16) {  // behind the copies, which need not wait for it
          if (qt == x.s0) {
            up = dS_up(most);
            if (lane == 0) *place_up(k) = make_float2(up, up);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) d4[i] *= up;
        }
        float* st = reinterpret_cast<float*>(smem + L::STAT) + s * 256;
        reinterpret_cast<float4*>(st)[lane] = make_float4(l4[0], l4[1], l4[2], l4[3]);
        reinterpret_cast<float4*>(st + 128)[lane] = make_float4(d4[0], d4[1], d4[2], d4[3]);
        if (tail) {
          if (!(go = warp_wait(w, bar_tail, tails++ & 1))) break;
          zero_rows<D>(dst, rows, lane, 32);
          zero_rows<D>(dst + L::TILE, rows, lane, 32);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_qf(s));
        }
        mbar_arrive(bar_qf(s));
        ++it;
      }
    }
    if (lane == 0) {  // every copy has landed before the CTA ends
      if (tails > 0) mbar_drain(w, bar_tail, (tails - 1) & 1);
      if (loads > 0) mbar_drain(w, bar_kv, (loads - 1) & 1);
      for (int s = 0; s < NS; ++s) {
        const int n = (it - s + NS - 1) / NS;
        if (n > 0) mbar_drain(w, bar_qf(s), (n - 1) & 1);
      }
    }
  } else if (warp == kMma) {
    // ------------------------------------------------------------ MMA issuer
    // Per query tile i, in the order of bwd_tc.cu:
    //   d = 64:  S^T_{i+1}, dV_i, dP^T_{i+1}, then dQ_i, dK_i
    //   d = 128: dV_i, S^T_{i+1} (over P^T), then dQ_i, dK_i, dP^T_{i+1} (over dQ_i)
    // and at an item's first tile S^T and dP^T by themselves, beside the results' way out.
    constexpr uint32_t idS = idesc_f16(F16, kTile, kTile, false, false);
    constexpr uint32_t idKV = idesc_f16(F16, kTile, D, false, true);
    constexpr uint32_t idQ = idesc_f16(F16, kTile, D, true, true);
    constexpr int KS = D / 16;
    const uint32_t tS = tmem + L::T_S, tDP = tmem + L::T_DP, tDV = tmem + L::T_DV, tDK = tmem + L::T_DK,
                   tDQ = tmem + L::T_DQ;
    const uint64_t dK_k = desc_kmajor_base(sb + L::K), dV_k = desc_kmajor_base(sb + L::V);
    const uint64_t dK_mn = desc_mnmajor_base(sb + L::K, kTile);
    const uint64_t dS_k = desc_kmajor_base(sb + L::DST);
    const uint64_t dS_mn = desc_mnmajor_base(sb + L::DST, kTile);
    auto ds_off = [&](int it) { return (uint32_t)(it % L::NDS) * L::DSB; };
    const uint64_t dQ_k0 = desc_kmajor_base(sb + L::QS), dQ_mn0 = desc_mnmajor_base(sb + L::QS, kTile);
    auto stage_off = [&](int it) { return (uint32_t)(it % NS) * 2u * L::TILE; };
    auto mma_s = [&](int it, int kk) {
      tc_mma_ss_elect(tS, dK_k + kmajor_step(kk, kTile), desc_add(dQ_k0, stage_off(it)) + kmajor_step(kk, kTile), idS,
                      kk > 0 ? 1u : 0u);
    };
    auto mma_dp = [&](int it, int kk) {
      tc_mma_ss_elect(tDP, dV_k + kmajor_step(kk, kTile),
                      desc_add(dQ_k0, stage_off(it) + L::TILE) + kmajor_step(kk, kTile), idS, kk > 0 ? 1u : 0u);
    };
    auto mma_dv = [&](int it, int kk, bool first) {
      tc_mma_ts_elect(tDV, tmem + L::pt_col(kk), desc_add(dQ_mn0, stage_off(it) + L::TILE) + mnmajor_step(kk), idKV,
                      (!first || kk > 0) ? 1u : 0u);
    };
    auto mma_dk = [&](int it, int kk, bool first) {
      tc_mma_ss_elect(tDK, desc_add(dS_k, ds_off(it)) + kmajor_step(kk, kTile),
                      desc_add(dQ_mn0, stage_off(it)) + mnmajor_step(kk), idKV, (!first || kk > 0) ? 1u : 0u);
    };
    auto mma_dq = [&](int it, int kk) {
      tc_mma_ss_elect(tDQ, desc_add(dS_mn, ds_off(it)) + mnmajor_step(kk), dK_mn + mnmajor_step(kk), idQ,
                      kk > 0 ? 1u : 0u);
    };
    bool ok = true;
    int it = 0, n = 0;  // steps, items with steps
    for (int k = 0; ok; ++k) {
      if (!(ok = warp_wait(w, bar_item(k), (k >> 1) & 1))) break;
      const int tile = place(k)->tile, steps = place(k)->s1 - place(k)->s0;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_item_free(k));
      if (tile < 0) break;
      if (steps == 0) continue;
      if (!(ok = warp_wait(w, bar_kv, n & 1))) break;
      if (!(ok = warp_wait(w, bar_qf(it % NS), (it / NS) & 1))) break;
      // dP^T goes where the last item's was, and at d = 128 its dQ
      if (it > 0 && !(ok = warp_wait(w, bar_dp_free, (it - 1) & 1))) break;
      if (L::ALIAS && it > 0 && !(ok = warp_wait(w, bar_dq_free, (it - 1) & 1))) break;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) mma_s(it, kk);
      tc_commit_elect(bar_s_full);
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) mma_dp(it, kk);
      tc_commit_elect(bar_dp_full);
      // dV and dK go where the last item's were
      if (n > 0 && !(ok = warp_wait(w, bar_acc_free, (n - 1) & 1))) break;
      for (int j = 0; j < steps; ++j, ++it) {
        const bool next = j + 1 < steps, first = j == 0;
        if (!(ok = warp_wait(w, bar_p_full, it & 1))) break;
        if (next && !(ok = warp_wait(w, bar_qf((it + 1) % NS), ((it + 1) / NS) & 1))) break;
        tc_fence_after();
        if (!L::ALIAS) {
          if (next) {
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) mma_s(it + 1, kk);
            tc_commit_elect(bar_s_full);
          }
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk) mma_dv(it, kk, first);
          tc_commit_elect(bar_pt_free);
          if (next) {
            if (!(ok = warp_wait(w, bar_dp_free, it & 1))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) mma_dp(it + 1, kk);
            tc_commit_elect(bar_dp_full);
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk) mma_dv(it, kk, first);
          if (next) {
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) mma_s(it + 1, kk);
            tc_commit_elect(bar_s_full);
          }
        }
        if (!(ok = warp_wait(w, bar_ds_full, it & 1))) break;
        if (!L::ALIAS && it > 0 && !(ok = warp_wait(w, bar_dq_free, (it - 1) & 1))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk) mma_dq(it, kk);
        if (L::STG_SEP) tc_commit_elect(bar_dq_full);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk) mma_dk(it, kk, first);
        if (!L::STG_SEP) tc_commit_elect(bar_dq_full);  // the boxes lie over the dS^T that dK_i reads
        tc_commit_elect(bar_ds_free(it % L::NDS));
        tc_commit_elect(bar_qe(it % NS));
        if (L::ALIAS && next) {  // dP^T_{i+1} goes over dQ_i
          if (!(ok = warp_wait(w, bar_dp_free, it & 1))) break;
          if (!(ok = warp_wait(w, bar_dq_free, it & 1))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < KS; ++kk) mma_dp(it + 1, kk);
          tc_commit_elect(bar_dp_full);
        }
      }
      if (!ok) break;
      tc_commit_elect(bar_done);
      ++n;
    }
    if (!ok) {  // a wait gave up: what is under way completes this phase
      tc_commit_elect(bar_done);
      ++n;
    }
    if (n > 0 && lane == 0) mbar_drain(w, bar_done, (n - 1) & 1);  // before TMEM is released
    __syncwarp();
  } else if (warp > kMma) {
    if constexpr (L::QW) {
      // ------------------------------------------------------------ dQ warps (d = 64)
      const int qd = warp & 3;
      const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
      const uint32_t stg = sb + L::STG + (uint32_t)qd * L::BOXB;
      bool pend = false, ok = true;  // pend: a reduce may still be reading the box
      int it = 0;
      for (int k = 0; ok; ++k) {
        if (!warp_wait(w, bar_item(k), (k >> 1) & 1)) break;
        const Work x = *place(k);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_item_free(k));
        if (x.tile < 0) break;
        for (int qt = x.s0; qt < x.s1; ++qt, ++it) {
          if (!(ok = warp_wait(w, bar_dq_full, it & 1))) break;
          tc_fence_after();
          const int rows = qt == x.q_last ? x.last_rows : full;
          const bool dead = 32 * qd + lane >= rows;  // a row of 0: of no query, or another sequence's
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += L::DQC) {
            uint32_t dq[L::DQC];
            tmem_ld_n<L::DQC>(tmem + L::T_DQ + lane_off + (uint32_t)c0, dq);
            if (c0 + L::DQC == D) {  // dQ_i is in registers: the next one may be computed
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar_dq_free);
            }
            if (32 * qd >= rows) continue;
            if (pend) {
              if (lane == 0) bulk_wait_group_read0();
              __syncwarp();
            }
            if (dead) {
#pragma unroll
              for (int i = 0; i < L::DQC; ++i) dq[i] = 0u;
            }
#pragma unroll
            for (int v = 0; v < L::DQC / 4; ++v)
              st_shared_v4(stg + (uint32_t)lane * 128u + (uint32_t)((v ^ (lane & 7)) * 16), dq[4 * v], dq[4 * v + 1],
                           dq[4 * v + 2], dq[4 * v + 3]);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_reduce_add_3d(&tmdQ, stg, c0, x.q_row0 + qt * full + qd * 32, x.hk);
              bulk_commit_group();
            }
            pend = true;
          }
        }
      }
      if (lane == 0) bulk_wait_group0();
    }
  } else {
    // ------------------------------------------------------------ compute warpgroups
    constexpr int CW = L::CW;
    const int g = warp >> 2;               // query columns [CW g, CW g + CW)
    const int r = (warp & 3) * 32 + lane;  // key row of the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint64_t scale2 = f2pack(a.scale, a.scale);
    // scale S - LSE, the product rounded: as an fma with 0, because a product and a sum of pairs become one
    // instruction, whatever their rounding says
    auto less_lse = [&](float x, float y, uint64_t nl) {
      return EXACT ? ffma2(f2pack(x, y), scale2, nl) : fadd2(ffma2(f2pack(x, y), scale2, 0ull), nl);
    };
    auto weight = [](float x) { return ex2(F16 ? fmaf(x, kLog2e, kPScale) : x * kLog2e); };
    const uint32_t stg = sb + L::STG + (uint32_t)warp * L::BOXB;
    bool pend = false;
    auto stg_acquire = [&]() {
      if (pend) {
        if (lane == 0) bulk_wait_group_read0();
        __syncwarp();
        pend = false;
      }
    };
    auto stat = [&](int it) { return reinterpret_cast<const float*>(smem + L::STAT) + (it % NS) * 256; };
    bool ok = true;
    int it = 0, n = 0;  // steps, items with steps
    for (int k = 0; ok; ++k) {
      if (!(ok = warp_wait(w, bar_item(k), (k >> 1) & 1))) break;
      const Work* x = place(k);
      if (x->tile < 0) break;
      const int s0 = x->s0, q_end = x->s1;
      // query tiles some row of which does not see some key of the tile; the first query that sees this key
      const int whole_from = x->whole_from, sees = r >= x->keys ? 1 << 30 : a.causal ? x->first_key + r : 0;
      // the first of the warpgroup's columns whose query sees this key
      auto first_col = [&](int qt) {
        const int i = sees - qt * tpt;
        return (i <= 0 ? 0 : i >= tpt ? kTile : i * G) - CW * g;
      };
      float p[CW];
      // S^T -> P^T: fp32 in p[] for dS, 16-bit into TMEM for dV
      auto p_phase = [&](int it, int qt) -> bool {
        if (!warp_wait(w, bar_qf(it % NS), (it / NS) & 1)) return false;
        if (!warp_wait(w, bar_s_full, it & 1)) return false;
        tc_fence_after();
        {
          uint32_t u[CW];
          tmem_ld_n<CW>(tmem + L::T_S + lane_off + CW * g, u);
#pragma unroll
          for (int c = 0; c < CW; ++c) p[c] = __uint_as_float(u[c]);
        }
        const float4* nl4 = reinterpret_cast<const float4*>(stat(it) + CW * g);  // -LSE
        uint32_t pk[CW / 2];
#pragma unroll
        for (int c = 0; c < CW; c += 4) {
          const float4 nl = nl4[c / 4];
          float x0, x1, x2, x3;
          f2unpack(less_lse(p[c], p[c + 1], f2pack(nl.x, nl.y)), x0, x1);
          f2unpack(less_lse(p[c + 2], p[c + 3], f2pack(nl.z, nl.w)), x2, x3);
          p[c] = weight(x0);
          p[c + 1] = weight(x1);
          p[c + 2] = weight(x2);
          p[c + 3] = weight(x3);
        }
        if (qt < whole_from) {
          const int first = first_col(qt);
#pragma unroll
          for (int c = 0; c < CW; ++c)
            if (c < first) p[c] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < CW; c += 2) pk[c / 2] = pack2<F16>(p[c], p[c + 1]);
        if constexpr (!L::ALIAS) {
          if (it > 0) {  // dV of the tile before has read its P^T
            if (!warp_wait(w, bar_pt_free, (it - 1) & 1)) return false;
            tc_fence_after();
          }
        }
        tmem_st_n<CW / 2>(tmem + L::pt_write_col(g) + lane_off, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p_full);
        return true;
      };
      if (s0 < q_end) ok = p_phase(it, s0);
      auto item_up = [&] { return *reinterpret_cast<const volatile uint64_t*>(place_up(k)); };
      uint64_t up2 = 0ull;
      if (F16 && D == 128 && s0 < q_end) up2 = item_up();
      for (int qt = s0; ok && qt < q_end; ++it, ++qt) {
        // ---- dS_i = P_i (dP_i - D)
        if (!(ok = warp_wait(w, bar_dp_full, it & 1))) break;
        tc_fence_after();
        uint32_t pk[CW / 2];
        const float4* nd4 = reinterpret_cast<const float4*>(stat(it) + 128 + CW * g);  // -D, in fp16 times the factor
        if (F16 && D == 64) up2 = item_up();  // (a register that it would spill: 16 bytes)
        auto ds = [&](uint32_t a0, uint32_t a1, float n0, float n1) {  // dP - D, the same
          const uint64_t dp = f2pack(__uint_as_float(a0), __uint_as_float(a1)), nd = f2pack(n0, n1);
          return F16 ? ffma2(dp, up2, nd) : fadd2(dp, nd);
        };
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          constexpr int HW = CW / 2;
          uint32_t u[HW];
          tmem_ld_n<HW>(tmem + L::T_DP + lane_off + CW * g + HW * hf, u);
          if (hf == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_dp_free);
          }
#pragma unroll
          for (int c = 0; c < HW; c += 4) {
            const int cc = HW * hf + c;
            const float4 nd = nd4[cc / 4];
            float y0, y1, y2, y3;
            f2unpack(fmul2(f2pack(p[cc], p[cc + 1]), ds(u[c], u[c + 1], nd.x, nd.y)), y0, y1);
            f2unpack(fmul2(f2pack(p[cc + 2], p[cc + 3]), ds(u[c + 2], u[c + 3], nd.z, nd.w)), y2, y3);
            pk[cc / 2] = pack2<F16>(y0, y1);
            pk[cc / 2 + 1] = pack2<F16>(y2, y3);
          }
        }
        if (qt < whole_from) {  // 0, whatever dP is there
          const int first = first_col(qt);
#pragma unroll
          for (int c = 0; c < CW; c += 2) {
            if (c < first) pk[c / 2] &= 0xFFFF0000u;
            if (c + 1 < first) pk[c / 2] &= 0x0000FFFFu;
          }
        }
        if (it >= L::NDS && !(ok = warp_wait(w, bar_ds_free(it % L::NDS), ((it / L::NDS) - 1) & 1))) break;
        if (!L::STG_SEP) stg_acquire();
#pragma unroll
        for (int ch = 0; ch < CW / 8; ++ch)
          st_shared_v4(sb + L::DST + (uint32_t)(it % L::NDS) * L::DSB + sw128_chunk_offset(r, (CW / 8) * g + ch, kTile),
                       pk[ch * 4 + 0], pk[ch * 4 + 1], pk[ch * 4 + 2], pk[ch * 4 + 3]);
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_ds_full);

        // ---- P of the next query tile, while dK_i, dQ_i, dP^T_{i+1} run
        if (qt + 1 < q_end && !(ok = p_phase(it + 1, qt + 1))) break;

        // ---- dQ_i -> the fp32 accumulator (d = 128; at d = 64 the dQ warps' job)
        if constexpr (!L::QW) {
          if (!(ok = warp_wait(w, bar_dq_full, it & 1))) break;
          tc_fence_after();
          const int rows = qt == x->q_last ? x->last_rows : full;
          uint32_t dq[L::DQG];
          tmem_ld_n<L::DQG>(tmem + L::T_DQ + lane_off + g * L::DQG, dq);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_dq_free);
          if (32 * (warp & 3) < rows) {
            if (r >= rows) {  // a row of 0: of no query, or another sequence's
#pragma unroll
              for (int i = 0; i < L::DQG; ++i) dq[i] = 0u;
            }
#pragma unroll
            for (int c0 = 0; c0 < L::DQG; c0 += L::DQC) {
              stg_acquire();
#pragma unroll
              for (int v = 0; v < L::DQC / 4; ++v)
                st_shared_v4(stg + (uint32_t)lane * 128u + (uint32_t)((v ^ (lane & 7)) * 16), dq[c0 + 4 * v],
                             dq[c0 + 4 * v + 1], dq[c0 + 4 * v + 2], dq[c0 + 4 * v + 3]);
              fence_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_reduce_add_3d(&tmdQ, stg, g * L::DQG + c0, x->q_row0 + qt * full + (warp & 3) * 32, x->hk);
                bulk_commit_group();
              }
              pend = true;
            }
          }
        }
      }
      // ------------------------------------------------------------ dK, dV of the item
      if (!ok) break;
      const bool have = q_end > s0;
      if (have && !(ok = warp_wait(w, bar_done, n++ & 1))) break;
      tc_fence_after();
      {
        const bool store = r < x->keys;
        const int hk = x->hk;
        float* part = x->slot < 0 ? nullptr
                                  : a.slots + ((long long)x->slot * a.Hk + hk) * (2 * kTile * D) + 4 * (g * L::DQG / 4 * kTile + r);
        constexpr int EC = L::DQG < 32 ? L::DQG : 32;
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
          const uint32_t col = (which == 0 ? L::T_DV : L::T_DK) + g * L::DQG;
          float mul = which == 0 ? 1.f : a.scale;
          if (F16) mul *= which == 0 ? kPDown : have ? kPDown * reciprocal(place_up(k)->x) : 1.f;
          const long long* st = which == 0 ? a.dvs : a.dks;
          constexpr int N = D == 64 ? 2 : 1;  // lanes that store a key's row
          uint16_t* dst = static_cast<uint16_t*>(which == 0 ? a.dv : a.dk) + (long long)(x->key0 + (r & -N)) * st[0] + hk * st[1] +
                          g * L::DQG + 8 * (r % N);
#pragma unroll
          for (int c0 = 0; c0 < L::DQG; c0 += EC) {
            uint32_t u[EC];
            if (have) {
              tmem_ld_n<EC>(tmem + col + lane_off + c0, u);
            } else {
#pragma unroll
              for (int i = 0; i < EC; ++i) u[i] = 0u;
            }
            if (have && which == 1 && c0 + EC == L::DQG) {  // all is in registers: the next item's dV and dK may go there
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar_acc_free);
            }
            if (part) {  // four channels of all keys side by side: a warp's stores are whole lines
#pragma unroll
              for (int v = 0; v < EC / 4; ++v)
                *reinterpret_cast<uint4*>(part + which * (kTile * D) + 4 * kTile * (c0 / 4 + v)) =
                    make_uint4(u[4 * v], u[4 * v + 1], u[4 * v + 2], u[4 * v + 3]);
            } else {
              uint4 q[EC / 8];
#pragma unroll
              for (int v = 0; v < EC / 8; ++v) {
                q[v].x = pack2<F16>(__uint_as_float(u[v * 8 + 0]) * mul, __uint_as_float(u[v * 8 + 1]) * mul);
                q[v].y = pack2<F16>(__uint_as_float(u[v * 8 + 2]) * mul, __uint_as_float(u[v * 8 + 3]) * mul);
                q[v].z = pack2<F16>(__uint_as_float(u[v * 8 + 4]) * mul, __uint_as_float(u[v * 8 + 5]) * mul);
                q[v].w = pack2<F16>(__uint_as_float(u[v * 8 + 6]) * mul, __uint_as_float(u[v * 8 + 7]) * mul);
              }
              if constexpr (D == 64) {
                // two lanes with 32 bytes of a key each exchange 16, so that they store side by side (4
                // sequences of up to 2048 tokens 64.2 us and not 66.8; four lanes with 64 bytes at d = 128
                // and in the forward pass were slower so)
                static_assert(EC == 16);
                const bool odd = lane & 1;
                uint4 t = odd ? q[0] : q[1];
                t.x = __shfl_xor_sync(0xffffffffu, t.x, 1);
                t.y = __shfl_xor_sync(0xffffffffu, t.y, 1);
                t.z = __shfl_xor_sync(0xffffffffu, t.z, 1);
                t.w = __shfl_xor_sync(0xffffffffu, t.w, 1);
                if (odd) q[0] = t; else q[1] = t;
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  if ((r & ~1) + j < x->keys) *reinterpret_cast<uint4*>(dst + j * st[0]) = q[j];
              } else if (store) {
#pragma unroll
                for (int v = 0; v < EC / 8; ++v) *reinterpret_cast<uint4*>(dst + c0 + v * 8) = q[v];
              }
            }
            __syncwarp();
          }
        }
      }
      if (lane == 0) mbar_arrive(bar_item_free(k));
    }
    if (lane == 0) bulk_wait_group0();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

// Before the main kernel: the rows' statistics in the order of the query tiles' rows, and the
// accumulator of dQ zeroed.  Streams O, dO and the accumulator; runs beside the list's making.
template <int D>
__global__ void __launch_bounds__(256) packed_rows_kernel(const PackedArgs a) {
  constexpr int TPR = D / 8;
  const long long total = (long long)a.Tq * a.Hq * TPR, n = (long long)gridDim.x * blockDim.x;
  for (long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x; t - (threadIdx.x & 31) < total; t += n) {
    const bool in = t < total;
    const long long row = (in ? t : 0) / TPR;
    const int c = (int)(t % TPR), token = (int)(row / a.Hq), head = (int)(row - (long long)token * a.Hq);
    const int hk = a.divG.div(head);
    const long long at = ((long long)hk * a.Tq + token) * a.G + (head - hk * a.G);  // [Hk][Tq][G]
    float acc = 0.f;
    if (in) {
      const uint4 o = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.o) + token * a.os[0] + head * a.os[1] + 8 * c);
      const uint4 g = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.dout) + token * a.dos[0] + head * a.dos[1] + 8 * c);
      const uint32_t ov[4] = {o.x, o.y, o.z, o.w}, gv[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 u = unpack2<false>(ov[i]), v = unpack2<false>(gv[i]);
        acc = fmaf(u.x, v.x, acc);
        acc = fmaf(u.y, v.y, acc);
      }
      float4* z = reinterpret_cast<float4*>(a.dq_acc + at * D + 8 * c);
      z[0] = z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int off = TPR / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (in && c == 0) {
      const float lse = a.lse[row];
      a.stat_d[at] = acc;
      a.stat_lse[at] = lse == -INFINITY ? INFINITY : lse;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // so that what waits for this grid finds the list too
}

// The last sequence that does not begin behind the token: r, and its first and end.  Of fewer than
// 32, each lane holds a first (`mine`), so that a search is no chain of loads; whole warps call it.
struct Place {
  int r = 0, begin = 0, end = 0;
};
__device__ __forceinline__ int lane_first(const int* first, int R) { return first[min((int)(threadIdx.x & 31), R)]; }
__device__ __forceinline__ Place place_of(const int* first, int mine, int R, int token) {
  Place p;
  if (R < 32) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const int at = __shfl_sync(0xffffffffu, mine, p.r + off);
      if (p.r + off < R && at <= token) p.r += off;
    }
    p.begin = __shfl_sync(0xffffffffu, mine, p.r);
    p.end = __shfl_sync(0xffffffffu, mine, p.r + 1);
    return p;
  }
  int hi = R;
  while (hi - p.r > 1) {
    const int mid = (p.r + hi) >> 1;
    if (first[mid] <= token) p.r = mid; else hi = mid;
  }
  p.begin = first[p.r];
  p.end = first[p.r + 1];
  return p;
}

// The same in fp16, and what dS's factors are formed from: the largest |dO|^2, |D| and |V|^2 of each
// sequence and key head.  Rows that have no part in the gradients, or are not finite, have no say in them.
// A block has a run of rows, and one of V's beside it, and its warps keep their own maxima until they are
// another sequence's or head's; those of warps that end alike are one atomic (an atomic a warp, all to
// the same few words, took 5 us of 4 sequences up to 2048 tokens).
constexpr int kRowsCtas = 5;  // an SM: 48 registers (6 spill: 13 us of 4 sequences up to 2048 tokens, and not 11.4; by now 10.4)
template <int D>
__global__ void __launch_bounds__(256, kRowsCtas) packed_rows_f16_kernel(const PackedArgs a) {
  constexpr int TPR = D / 8, PER = 32 / TPR;  // lanes of a row, rows of a warp's turn
  const int lane = threadIdx.x & 31, c = lane % TPR, sub = lane / TPR;
  struct Run {  // a block's warps take its rows in turn
    int at, left, turns;  // the warp's first row, the rows from there on, its turns
    __device__ __forceinline__ explicit Run(int all) {
      constexpr int TURN = 8 * PER;  // of a block
      const int per = (int)(((long long)all + TURN * gridDim.x - 1) / (TURN * gridDim.x));
      const long long first = (long long)blockIdx.x * per * TURN + (threadIdx.x >> 5) * PER;
      at = first < all ? (int)first : 0;
      left = first < all ? all - at : 0;
      turns = min(per, (int)(((long long)left + TURN - 1) / TURN));
    }
  };
  const Run rows(a.Tq * a.Hq), keys(a.Tk * a.Hk);
  const int span = a.Tq * a.G;
  const int *first_q = a.list.starts, *first_k = first_q + a.R + 1;
  auto add_up = [](float x) {  // over a row's lanes
#pragma unroll
    for (int off = TPR / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
  };
  // Maxima of a sequence and key head; unit: which, -1 at first and of rows that are no sequence's.
  struct Most {
    long long unit = -1;
    float x = 0.f, y = 0.f;
    Place of;  // the last row's sequence
  } of_q, of_k;
  auto warp_most = [](float x) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x))); };  // x >= 0
  auto raise = [&](long long unit, int which, float x) {
    if (x > 0.f) atomicMax(reinterpret_cast<int*>(a.most + unit) + which, __float_as_int(x));
  };
  auto flush = [&](const Most& m, int x_at, int y_at) {
    const float x = warp_most(m.x), y = warp_most(m.y);
    if (lane == 0 && m.unit >= 0) {
      raise(m.unit, x_at, x);
      if (y_at >= 0) raise(m.unit, y_at, y);
    }
  };
  int mine_q = 0, mine_k = 0;
  auto take = [&](Most& m, const int* first, int mine, bool in, int token, int hk, float x, float y, int x_at, int y_at) {
    if (__any_sync(0xffffffffu, in && (token < m.of.begin || token >= m.of.end))) m.of = place_of(first, mine, a.R, token);
    const long long unit = in && token >= m.of.begin && token < m.of.end ? (long long)m.of.r * a.Hk + hk : -1;
    if (!__all_sync(0xffffffffu, unit == m.unit)) {
      flush(m, x_at, y_at);
      m.x = m.y = 0.f;
      m.unit = __shfl_sync(0xffffffffu, unit, 31);
      if (unit != m.unit) {
        if (unit >= 0 && c == 0) {
          raise(unit, x_at, x);
          if (y_at >= 0) raise(unit, y_at, y);
        }
        return;
      }
    }
    m.x = fmaxf(m.x, x);
    m.y = fmaxf(m.y, y);
  };
  for (int j = 0; j < max(rows.turns, keys.turns); ++j) {
    const int ahead = j * 8 * PER + sub, at = rows.at + ahead, key = keys.at + ahead;
    const bool in = j < rows.turns && ahead < rows.left, key_in = j < keys.turns && ahead < keys.left;
    uint4 o = make_uint4(0u, 0u, 0u, 0u), g = o, v = o;
    int token = 0, hk = 0, key_token = 0, key_hk = 0;
    float lse = 0.f;
    if (in) {
      hk = a.divRows.div(at);
      const int rest = at - hk * span;
      token = a.divG.div(rest);
      const int head = hk * a.G + rest - token * a.G;
      o = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.o) + token * a.os[0] + head * a.os[1] + 8 * c);
      g = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.dout) + token * a.dos[0] + head * a.dos[1] + 8 * c);
      lse = a.lse[(long long)token * a.Hq + head];
    }
    if (key_in) {
      key_hk = a.divTk.div(key);
      key_token = key - key_hk * a.Tk;
      v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.v) + key_token * a.vs[0] + key_hk * a.vs[1] + 8 * c);
    }
    float dot = 0.f, square = 0.f, v_square = 0.f;
    const uint32_t ow[4] = {o.x, o.y, o.z, o.w}, gw[4] = {g.x, g.y, g.z, g.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack2<true>(ow[i]), y = unpack2<true>(gw[i]), z = unpack2<true>(vw[i]);
      dot = fmaf(x.y, y.y, fmaf(x.x, y.x, dot));
      square = fmaf(y.y, y.y, fmaf(y.x, y.x, square));
      v_square = fmaf(z.y, z.y, fmaf(z.x, z.x, v_square));
    }
    dot = add_up(dot);
    square = add_up(square);
    v_square = add_up(v_square);
    if (in) {
      float4* z = reinterpret_cast<float4*>(a.dq_acc + (long long)at * D + 8 * c);
      z[0] = z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c == 0) {
        a.stat_d[at] = dot;
        a.stat_lse[at] = lse == -INFINITY ? INFINITY : lse;
      }
    }
    if (j == 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");  // the sequences, and the maxima zeroed
      mine_q = lane_first(first_q, a.R);
      mine_k = lane_first(first_k, a.R);
    }
    const bool counts = in && lse != -INFINITY && square < INFINITY;
    if (j < rows.turns) take(of_q, first_q, mine_q, in, token, hk, counts ? square : 0.f, counts && fabsf(dot) < INFINITY ? fabsf(dot) : 0.f, 0, 2);
    if (in && c == 0 && at == token * a.G) a.seq_of[token] = of_q.of.r;  // once for each token
    if (j < keys.turns) take(of_k, first_k, mine_k, key_in, key_token, key_hk, v_square < INFINITY ? v_square : 0.f, 0.f, 1, -1);
  }
  // what is left: by the block
  __shared__ long long unit_s[2][8];
  __shared__ float most_s[3][8];
  const float x = warp_most(of_q.x), y = warp_most(of_k.x), z = warp_most(of_q.y);
  if (lane == 0) {
    const int i = threadIdx.x >> 5;
    most_s[0][i] = x;
    most_s[1][i] = y;
    most_s[2][i] = z;
    unit_s[0][i] = of_q.unit;
    unit_s[1][i] = of_k.unit;
  }
  __syncthreads();
  if (threadIdx.x < 24) {  // warp i's k-th maximum: joined with the others of the same unit by the first of them
    const int k = threadIdx.x / 8, i = threadIdx.x % 8, of = k & 1;
    const long long unit = unit_s[of][i];
    float x = most_s[k][i];
    bool first = unit >= 0;
    for (int j = 0; j < 8; ++j)
      if (unit_s[of][j] == unit) {
        x = fmaxf(x, most_s[k][j]);
        first &= j >= i;
      }
    if (first) raise(unit, k, x);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // so that what waits for this grid finds the list too
}

// After it: dQ = scale * accumulator, for rows that are a sequence's; and dK, dV of the cut key
// tiles from their parts, in order.  (fp16: less the factors of P and dS.)
constexpr int kSumParts = 8;
template <int D, bool F16>
__global__ void __launch_bounds__(256) packed_finish_kernel(const PackedArgs a, int dq_blocks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if ((int)blockIdx.x < dq_blocks) {
    constexpr int TPR = D / 8;
    const int first = a.list.head[2], end = a.list.head[3];
    const long long total = (long long)(end - first) * a.Hq * TPR, n = (long long)dq_blocks * blockDim.x;
    for (long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x; t < total; t += n) {
      const long long row = t / TPR;
      const int c = (int)(t % TPR), rel = (int)(row / a.Hq), head = (int)(row - (long long)rel * a.Hq), token = first + rel;
      const int hk = a.divG.div(head);
      const long long at = ((long long)hk * a.Tq + token) * a.G + (head - hk * a.G);
      const float4* src = reinterpret_cast<const float4*>(a.dq_acc + at * D + 8 * c);
      const float4 x = src[0], y = src[1];
      float mul = a.scale;
      if constexpr (F16) {
        mul *= kPDown * reciprocal(dS_up(a.most[(long long)a.seq_of[token] * a.Hk + hk]));
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dq) + token * a.dqs[0] + head * a.dqs[1] + 8 * c) =
          make_uint4(pack2<F16>(x.x * mul, x.y * mul), pack2<F16>(x.z * mul, x.w * mul),
                     pack2<F16>(y.x * mul, y.y * mul), pack2<F16>(y.z * mul, y.w * mul));
    }
    return;
  }
  const int k = (int)blockIdx.x - dq_blocks, unit = k / kSumParts, part = k % kSumParts;
  const int cut = a.divHk.div(unit), hk = unit - cut * a.Hk;
  if (cut >= a.list.head[1]) return;
  const PackedItem x = a.list.cuts[cut];
  // eight channels of a key a thread, keys side by side
  constexpr int PER = 2 * kTile * D / 8, PART = PER / kSumParts;
  constexpr size_t words = 2 * kTile * D;
  const float* base = a.slots + ((size_t)x.first * a.Hk + hk) * words;
  const int keys = min(kTile, x.seq.m - x.tile * kTile);
  const float up = F16 ? dS_up(a.most[(long long)x.r * a.Hk + hk]) : 1.f;
  for (int e = part * PART + (int)threadIdx.x; e < (part + 1) * PART; e += blockDim.x) {
    const int row = e % kTile, pair = e / kTile, which = pair / (D / 8), col = pair % (D / 8) * 8;
    if (row >= keys) continue;
    float acc[8] = {};
#pragma unroll 2
    for (int s = 0; s < x.parts; ++s) {
      const float4* from = reinterpret_cast<const float4*>(base + (size_t)s * a.Hk * words) + 2 * pair * kTile + row;
      const float4 u = from[0], v = from[kTile];
      acc[0] += u.x; acc[1] += u.y; acc[2] += u.z; acc[3] += u.w;
      acc[4] += v.x; acc[5] += v.y; acc[6] += v.z; acc[7] += v.w;
    }
    float mul = which == 0 ? 1.f : a.scale;
    if (F16) mul *= which == 0 ? kPDown : kPDown * reciprocal(up);
    const long long* st = which == 0 ? a.dvs : a.dks;
    uint16_t* dst = static_cast<uint16_t*>(which == 0 ? a.dv : a.dk) +
                    (long long)(x.seq.k0 + x.tile * kTile + row) * st[0] + hk * st[1] + col;
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack2<F16>(acc[0] * mul, acc[1] * mul), pack2<F16>(acc[2] * mul, acc[3] * mul),
                                                pack2<F16>(acc[4] * mul, acc[5] * mul), pack2<F16>(acc[6] * mul, acc[7] * mul));
  }
}

struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  Launch(long long grid, int threads, size_t smem, cudaStream_t s) {
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
  }
};

int sms() {
  int dev = 0, n = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}
int stream_blocks(long long threads) {
  const long long blocks = (threads + 255) / 256, most = (long long)sms() * 8;
  return (int)(blocks < 1 ? 1 : blocks < most ? blocks : most);
}

template <int D, bool F16, bool EXACT>
cudaError_t main_t(const PackedArgs& a, const CUtensorMap* tm, int items, cudaStream_t s) {
  using L = Layout<D>;
  const auto kern = packed_bwd_kernel<D, F16, EXACT>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::BYTES);
  if (e != cudaSuccess) return e;
  Launch l(std::min((long long)items * a.Hk, (long long)sms()), L::NT, L::BYTES, s);
  return cudaLaunchKernelEx(&l.cfg, kern, tm[0], tm[1], tm[2], tm[3], tm[4], a);
}
template <int D, bool F16>
cudaError_t rows_t(const PackedArgs& a, cudaStream_t s) {
  const long long rows = std::max((long long)a.Tq * a.Hq, F16 ? (long long)a.Tk * a.Hk : 0ll);
  const int blocks = stream_blocks(rows * (D / 8));
  Launch l(F16 ? std::min(blocks, kRowsCtas * sms()) : blocks, 256, 0, s);
  return cudaLaunchKernelEx(&l.cfg, F16 ? packed_rows_f16_kernel<D> : packed_rows_kernel<D>, a);
}
template <int D, bool F16>
cudaError_t finish_t(const PackedArgs& a, int cuts, cudaStream_t s) {
  const int dq_blocks = stream_blocks((long long)a.Tq * a.Hq * (D / 8));
  Launch l(dq_blocks + (long long)cuts * a.Hk * kSumParts, 256, 0, s);
  return cudaLaunchKernelEx(&l.cfg, packed_finish_kernel<D, F16>, a, dq_blocks);
}

}  // namespace

cudaError_t launch_packed_bwd_preprocess(const PackedArgs& a, int d, bool f16, cudaStream_t s) {
  if (d == 64) return f16 ? rows_t<64, true>(a, s) : rows_t<64, false>(a, s);
  return f16 ? rows_t<128, true>(a, s) : rows_t<128, false>(a, s);
}
cudaError_t launch_packed_bwd(const PackedArgs& a, int d, bool f16, const CUtensorMap* tm, int items, cudaStream_t s) {
  int e;
  if (d == 64 && std::frexp(a.scale, &e) == 0.5f)
    return f16 ? main_t<64, true, true>(a, tm, items, s) : main_t<64, false, true>(a, tm, items, s);
  if (d == 64) return f16 ? main_t<64, true, false>(a, tm, items, s) : main_t<64, false, false>(a, tm, items, s);
  return f16 ? main_t<128, true, false>(a, tm, items, s) : main_t<128, false, false>(a, tm, items, s);
}
cudaError_t launch_packed_bwd_finalize(const PackedArgs& a, int d, bool f16, int cuts, cudaStream_t s) {
  if (d == 64) return f16 ? finish_t<64, true>(a, cuts, s) : finish_t<64, false>(a, cuts, s);
  return f16 ? finish_t<128, true>(a, cuts, s) : finish_t<128, false>(a, cuts, s);
}

}  // namespace fa
