// kv_attn.cuh -- attention of each request's newest tokens over its 4-bit or 8-bit cache.
//
// Bound: HBM.  A token of one head is 160 bytes (d = 128; in 8 bits 257) for both its key and
// its value, and 8 query rows need 4 * 8 * d FLOPs of it: 26 (16) FLOPs a byte, far below
// what the tensor cores give.  What limits the kernel besides is turning codes into
// fp16 operands, so that is done once per token for all query heads of its key head,
// in registers, straight into tensor-core fragments.
//
// Products.  The cache is the A operand of mma.sync.m16n8k16 and the query rows are
// the 8 columns of B, so that one key head's few query rows waste nothing:
//     S^T [16 tokens x 8 rows] = K [16 x d] Q^T,   O^T [16 channels x 8 rows] += V^T P^T.
// (tcgen05.mma takes its A operand from shared or tensor memory with 64 or 128 rows;
// the fp16 values would have to be written there and read back, four times the bytes
// the codes have, for products that are not what bounds the kernel.)  A tile of more
// rows repeats the products on NT columns blocks; the fragments of K and V are reused.
//   - Which channel a fragment position stands for is free as long as K and Q agree, and
//     which token as long as S, P and V do.  A lane's position t = lane % 4 along the
//     contraction takes d / 4 neighbouring channels of a token: one 16-byte (d = 128)
//     load of codes, all of one (scale, base) pair.  Code pairs (p, p + 4) of a 32-bit
//     word lie 16 bits apart: a shift, one three-input logic operation (mask, set the
//     exponent) and one half2 fma make both values.
//   - V^T needs neighbouring tokens in one register: a byte permute of two tokens' words
//     does it for eight values at a time; the fma then takes the two tokens' scales.
//   - P^T as a B operand is the transpose of S^T as an accumulator: movmatrix.
// Softmax.  Rows lie across lanes with the same t, so the maximum moves only when some
// score of the block is above it by more than 2^8 (one vote); then it is reduced by
// shuffles and O and l are rescaled.  l is kept per lane and reduced at the end.
//
// Work.  A tile is a request's 8 NT query rows of one key head; its tokens are taken in
// units of 32.  Within a CTA the warps take the units in turn, each with its own ring of
// bulk copies and its own m, l, O, joined in shared memory at the end.  Across CTAs there
// are two ways:
//   - shares: all tiles lie one after the other, and each CTA takes an equal share of all
//     units, wherever it begins and ends, so that ragged lengths leave no SM idle.  A tile
//     that is cut leaves fp32 (O, m, l) per share, which a second kernel adds (launched with
//     the first, it waits for it on the GPU).
//   - clusters, for few tiles of few units: the CTAs of a cluster divide a tile evenly and
//     join through distributed shared memory; one launch, nothing in device memory.
// kv4_cluster (ops_api.cu) chooses, by the number of tiles and the units a warp would take.
//
// Measured (shares): 64 requests of up to 16384 tokens, 32 query and 8 key heads, d = 128:
// 145 us for 748 MB, 5.2 TB/s; the unit loop alone goes at 5.9 TB/s, with the integer pipe at
// 54% (codes to fp16) and four warps a scheduler, and about 13 us are start-up, uneven ends
// and the second kernel.  (Clusters): one request of 23,400 tokens, 12 heads, d = 64: 14.5 us.
// In 8 bits, 1202 MB of the same requests: 190 us, 6.3 TB/s; the day's one request 15.7 us.
#pragma once
#include <type_traits>

#include "kv4.cuh"
#include "kv8.cuh"
#include "kv4_ring.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr float kNoMax = -3e38f;     // running maximum before any token is seen
constexpr float kLeast = 1e-37f;     // of a score's factor: a hidden token's -inf times it stays -inf
constexpr int kUnit = 2 * kKvBlock;  // tokens a warp takes at a time
constexpr int kReqCache = 128;       // requests whose lengths a CTA keeps at hand

// CL: the CTAs are a cluster's.  A block of 8 bits has 1.6 times the bytes of one of 4, so that
// as many bytes are on their way with fewer stages or CTAs.
template <class Blk, int NT, bool CL>
struct Cfg {
  static constexpr int D = Blk::D;
  static constexpr bool wide = Blk::bits == 8;
  static constexpr int ROWS = 8 * NT;
  static constexpr int WARPS = CL ? 8 : 4, THREADS = 32 * WARPS;
  static constexpr int CTAS_PER_SM =
      CL ? (NT == 1 && !(wide && D == 128) ? 2 : 1) : kv_share_ctas(Blk::bits, ROWS, 1);
  static constexpr int LDO = D + 4;  // row pitch of the joined O, in floats
  static constexpr int stage = 2 * Blk::bytes;
  // For the join each warp's O goes into its ring.  Eight rows of a share take the stage of the
  // tile's last unit, and the copies of the next tile go on in the others; otherwise it is
  // the whole ring, which then holds one tile at a time.
  static constexpr bool across = NT == 1 && !CL;
  static constexpr int STAGES = wide ? (D == 64 || NT == 4 ? 3 : 2) : D == 64 || NT == 4 ? 4 : 2;
  static constexpr int ring = WARPS * STAGES * stage;
  static_assert(ROWS * LDO * 4 <= (across ? stage : STAGES * stage), "a warp's O fits");
  static constexpr int qfrag = NT == 4 ? NT * (D / 16) * 32 * 8 : 0;
  static constexpr int smem = ring + qfrag;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// 1 + c / 16 of codes P and P + 4 (bits 4 P and 16 + 4 P) of a word, as half2: a shift, and
// one (x & mask) | one -- written out, with both constants in registers, because as two
// operations with constants it would cost a third more of the integer pipe, which is
// what bounds the unit loop.
struct Magic {
  uint32_t mask, one;
  __device__ __forceinline__ Magic() {
    asm volatile("mov.u32 %0, 0x03C003C0;" : "=r"(mask));
    asm volatile("mov.u32 %0, 0x3C003C00;" : "=r"(one));
  }
};
template <int P>
__device__ __forceinline__ uint32_t code_pair(const Magic& k, uint32_t w) {
  const uint32_t x = P == 0 ? w << 6 : P == 1 ? w << 2 : P == 2 ? w >> 2 : w >> 6;
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(k.mask), "r"(k.one));
  return y;
}

// Four int8 codes as two half2: 1024 + (code + 128) is the fp16 number 0x6400 | (code + 128), and
// less 1152 it is the code.  One logic operation and a permute and a sum for each pair.
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ void codes4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  lo = hadd2(__byte_perm(u, 0x64646464u, 0x4140), 0xE480E480u);
  hi = hadd2(__byte_perm(u, 0x64646464u, 0x4342), 0xE480E480u);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// A request's place: its first query row, its query rows and its cached tokens.
struct Req {
  int q0, n, kv;
};
__device__ __forceinline__ Req load_req(const Kv4AttnArgs& a, int r) {
  Req x;
  if (a.cu_q) {
    x.q0 = min(max(__ldg(a.cu_q + r), 0), a.T);
    x.n = min(max(__ldg(a.cu_q + r + 1), x.q0), a.T) - x.q0;
  } else {
    x.q0 = min(r, a.T);
    x.n = r < a.T ? 1 : 0;
  }
  x.kv = max(__ldg(a.kv_lens + r), 0);
  const long long most = (long long)a.table_width << a.c.page_log;
  if (x.kv > most) {
    atomicCAS(&a.rep.st->code, 0, (int)FA_ERR_INDEX);
    x.kv = (int)most;
  }
  return x;
}

// The first token that the row at position pos sees (pos may be negative, and the window any:
// pos - window is formed only where it is not negative).
__device__ __forceinline__ int first_seen(const Kv4AttnArgs& a, int pos) {
  return a.window > 0 && pos >= a.window ? pos - a.window + 1 : 0;
}

// Bits 0 .. n - 1, for any n.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// Tile `t` of a request: rows [row0, row0 + ROWS) of its n * G, tokens [k0, k1) that some
// row of it sees, units from token u0 on, n_u of them (one, of hidden tokens, where no
// row sees any).
struct Tile {
  int row0, rows, k0, k1, u0, n_u;
};
template <int ROWS>
__device__ __forceinline__ int tiles_of(const Kv4AttnArgs& a, const Req& x) {
  return (int)(((long long)x.n * a.G.d + ROWS - 1) / ROWS);
}
template <int ROWS>
__device__ __forceinline__ Tile tile_of(const Kv4AttnArgs& a, const Req& x, int t) {
  Tile y;
  y.row0 = t * ROWS;
  y.rows = min(ROWS, x.n * (int)a.G.d - y.row0);
  const int i0 = a.G.div(y.row0), i1 = a.G.div(y.row0 + y.rows - 1);
  y.k1 = max(0, x.kv - x.n + i1 + 1);
  y.k0 = min(first_seen(a, x.kv - x.n + i0), y.k1);
  y.u0 = y.k0 & ~(kUnit - 1);
  y.n_u = max(1, (y.k1 - y.u0 + kUnit - 1) / kUnit);
  return y;
}

// Walks the tiles in order: request, tile, key head.
template <int ROWS>
struct Walk {
  int r, t, h;
  Req x;
  Tile y;
  __device__ __forceinline__ void at(const Kv4AttnArgs& a, const Req* cache, int cache_r0, int r_, int t_, int h_) {
    r = r_;
    t = t_;
    h = h_;
    fetch(a, cache, cache_r0);
    y = tile_of<ROWS>(a, x, t);
  }
  __device__ __forceinline__ void fetch(const Kv4AttnArgs& a, const Req* cache, int cache_r0) {
    const int i = r - cache_r0;
    x = i < kReqCache ? cache[i] : load_req(a, r);
  }
  __device__ __forceinline__ void next(const Kv4AttnArgs& a, const Req* cache, int cache_r0) {
    if (++h < a.c.Hk) return;
    h = 0;
    if (++t < tiles_of<ROWS>(a, x)) {
      y = tile_of<ROWS>(a, x, t);
      return;
    }
    t = 0;
    do {  // requests without new tokens have no tiles
      if (++r >= a.R) return;
      fetch(a, cache, cache_r0);
    } while (x.n == 0);
    y = tile_of<ROWS>(a, x, 0);
  }
};

// Where a warp's coming units lie, in shared memory: its copies' addresses are formed 32
// units at a time, one by each lane, off the path of the unit loop.
template <int ROWS>
struct Feed {
  Walk<ROWS> w;           // tile of the coming units
  long long tile0;        // its first unit
  int u, end;             // the warp's next unit of it, and the end of the share's part of it
  int ids_r, ids_tok;     // request and first token that `id` was read for
  int id[2][32];          // pages of the two blocks of each of the 32 units
  ulonglong2 src[32];     // addresses of the two blocks; 1 for one that is not to be read
  uint32_t hidden[8];     // per ring stage: bit h for block h not read, or kStageIdle (across)
};

// Fills src with the warp's next units of the share, at most 32, all of one tile; returns
// how many (0: none left).
template <class Blk, int ROWS, int kWarps>
__device__ __noinline__ int feed_refill(const Kv4AttnArgs& a, Feed<ROWS>& f, const Req* reqs, int reqs_r0, int warp,
                                        long long u1) {
  const int lane = threadIdx.x & 31, page_log = a.c.page_log;
  __syncwarp();
  Walk<ROWS> w = f.w;
  long long tile0 = f.tile0;
  int u = f.u, end = f.end;
  const bool moved = u >= end;
  while (u >= end) {
    if (tile0 + w.y.n_u >= u1) return 0;
    tile0 += w.y.n_u;
    w.next(a, reqs, reqs_r0);
    u = warp;
    end = (int)min((long long)w.y.n_u, u1 - tile0);
  }
  const int first = w.y.u0 + u * kUnit, tok = first + lane * kWarps * kUnit;
  int id0 = f.id[0][lane], id1 = f.id[1][lane];
  if (f.ids_r != w.r || f.ids_tok != first) {  // not another head of the same tokens
    const int pg0 = tok >> page_log, pg1 = (tok + kKvBlock) >> page_log;
    const int* row = a.table + w.r * a.table_stride;
    id0 = pg0 < a.table_width ? __ldg(row + pg0) : -1;
    id1 = pg1 == pg0 ? id0 : pg1 < a.table_width ? __ldg(row + pg1) : -1;
    f.id[0][lane] = id0;
    f.id[1][lane] = id1;
  }
  // blocks that some row sees a token of (the first one of a window may lie behind it, in a page
  // that is no longer the request's)
  const bool mine = u + lane * kWarps < end;
  const bool in0 = mine && tok < w.y.k1 && tok + kKvBlock > w.y.k0;
  const bool in1 = mine && tok + kKvBlock < w.y.k1 && tok + 2 * kKvBlock > w.y.k0;
  const bool ok0 = in0 && (unsigned)id0 < (unsigned)a.c.num_pages, ok1 = in1 && (unsigned)id1 < (unsigned)a.c.num_pages;
  if ((in0 && !ok0) || (in1 && !ok1)) atomicCAS(&a.rep.st->code, 0, (int)FA_ERR_INDEX);
  auto place = [&](int id, int t) {
    const int blk = (t & ((1 << page_log) - 1)) / kKvBlock;
    return reinterpret_cast<unsigned long long>(a.c.data) + id * a.c.page_stride +
           (((long long)w.h << (page_log - 4)) + blk) * Blk::bytes;
  };
  f.src[lane] = make_ulonglong2(ok0 ? place(id0, tok) : 1ull, ok1 ? place(id1, tok + kKvBlock) : 1ull);
  __syncwarp();  // every lane has read the old state
  const int n = min(32, (end - u + kWarps - 1) / kWarps);
  if (lane == 0) {
    f.ids_r = w.r;
    f.ids_tok = first;
    f.u = u + n * kWarps;
    if (moved) {
      f.w = w;
      f.tile0 = tile0;
      f.end = end;
    }
  }
  __syncwarp();
  return n;
}

// A wait gave up (which is recorded, and void what this launch writes): the warp's n copies
// under way must land, within one limit for all of them, before anything else is written over
// the ring or the CTA ends.  No more are issued and no unit is consumed from then on, but the
// CTA goes through its barriers to the end.  W: the context, by reference in shares and by value in
// clusters, which is what costs the unit loop least (decode_n16384 145.0 and 146.7 us, shares;
// decode_n2048 9.08 and 8.90, clusters).
template <int S, typename W>
__device__ __noinline__ void drain_ring(W wc, uint32_t bar0, Ring<S> at, int n) {
  const uint64_t since = globaltimer_ns();
  at.each(n, [&](int s, uint32_t p) { mbar_drain_since(wc, bar0 + 8 * s, p, since); });
  __syncwarp();
}

template <class Blk, int NT, bool F16, bool CL>
__global__ void __launch_bounds__(Cfg<Blk, NT, CL>::THREADS, Cfg<Blk, NT, CL>::CTAS_PER_SM) kv_attn_kernel(const Kv4AttnArgs a) {
  using C = Cfg<Blk, NT, CL>;
  constexpr int D = Blk::D;
  constexpr bool wide = C::wide;
  constexpr int kWarps = C::WARPS, kThreads = C::THREADS;
  constexpr int ROWS = C::ROWS, S = C::STAGES, KS = D / 16, MT = D / 16, WPT = D / 32 /* words per lane of K */;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][S];
  __shared__ long long warp_sums[kWarps];
  __shared__ int longest_s;  // units of the longest tile (shares)
  __shared__ Req reqs[kReqCache];
  __shared__ long long start_u;
  __shared__ int start_r, start_t, start_h;
  __shared__ float m_s[kWarps][ROWS], l_s[kWarps][ROWS];
  __shared__ __align__(16) float2 ml_s[CL ? ROWS : 1];  // of the CTA, for the cluster
  __shared__ int held_s[kWarps];
  __shared__ float up_s[NT == 4 ? ROWS : 1];
  static_assert(NT != 4 || kWarps >= 4, "a warp for every eight rows");
  __shared__ volatile int abort_s;
  __shared__ Feed<ROWS> feed_s[kWarps];
  __shared__ Walk<ROWS> tile_s[2];  // the current tile; the next one

  if constexpr (!CL) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge waits for this grid's end
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const uint32_t ring = smem_addr(smem) + warp * (S * C::stage);
  const uint32_t bar0 = smem_addr(&bars[warp][0]);
  uint2* qfrag = reinterpret_cast<uint2*>(smem + C::ring);
  (void)qfrag;

  // ---- prefix sums over all requests, of their units or (CL) their tiles
  if (tid == 0) abort_s = longest_s = 0;
  if (!CL) __syncthreads();
  if (lane == 0)
    for (int s = 0; s < S; ++s) mbar_init(bar0 + 8 * s, 1);
  fence_barrier_init();
  const int per = (a.R + kThreads - 1) / kThreads;
  const int my0 = min(a.R, tid * per), my1 = min(a.R, my0 + per);
  int longest = 0;
  auto count_of = [&](const Req& x) {
    const int nt = tiles_of<ROWS>(a, x);
    long long n = nt;
    if constexpr (!CL) {
      n = 0;
      for (int t = 0; t < nt; ++t) {
        const int n_u = tile_of<ROWS>(a, x, t).n_u;
        longest = max(longest, n_u);
        n += n_u;
      }
    }
    return n * a.c.Hk;
  };
  const bool cached = a.R <= min(kThreads, kReqCache);  // every request's lengths are at hand
  long long mine = 0;
  for (int r = my0; r < my1; ++r) {
    const Req x = load_req(a, r);
    if (cached) reqs[r] = x;
    mine += count_of(x);
  }
  long long end = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, end, off);
    if (lane >= off) end += up;
  }
  if (lane == 31) warp_sums[warp] = end;
  if constexpr (!CL) {
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) atomicMax(&longest_s, longest);
  }
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) end += warp_sums[w];
    total += warp_sums[w];
  }
  // shares: this CTA's units [u0, u1)
  long long share = 0, u0 = 0, u1 = 0;
  if constexpr (!CL) {
    share = (total + gridDim.x - 1) / gridDim.x;
    // a unit for each warp; where no tile has as many, enough that none need be cut (320 tiles
    // of one unit, 16 rows: 26.6 us with four of them to a CTA, 11.5 with one)
    share = longest_s >= kWarps ? (share + kWarps - 1) / kWarps * kWarps : max(share, (long long)longest_s);
    u0 = (long long)blockIdx.x * share;
    u1 = min(total, u0 + share);
    if (u0 >= total) {  // no share (the CTA's threads all leave)
      if (tid == 0) a.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
      return;
    }
    // the thread whose requests hold unit u0 finds its tile
    if (u0 < end && u0 >= end - mine) {
      long long u = end - mine;
      bool found = false;
      for (int r = my0; r < my1 && !found; ++r) {
        const Req x = cached ? reqs[r] : load_req(a, r);
        const int nt = tiles_of<ROWS>(a, x);
        for (int t = 0; t < nt && !found; ++t) {
          const long long n = tile_of<ROWS>(a, x, t).n_u;
          if (u0 < u + n * a.c.Hk) {
            const int h = (int)((u0 - u) / n);
            start_r = r;
            start_t = t;
            start_h = h;
            start_u = u + h * n;  // first unit of the tile
            found = true;
          } else {
            u += n * a.c.Hk;
          }
        }
      }
    }
    __syncthreads();
  }
  const int cache_r0 = CL || cached ? 0 : start_r;
  if (!CL && !cached) {
    for (int i = tid; i < kReqCache; i += kThreads)
      if (cache_r0 + i < a.R) reqs[i] = load_req(a, cache_r0 + i);
    __syncthreads();
  }

  const Magic magic;
  using Context = std::conditional_t<CL, WaitCtx, const WaitCtx&>;
  const WaitCtx wc{&abort_s, a.rep.st, a.rep.epoch, a.rep.wait_ns};

  Feed<ROWS>& feed = feed_s[warp];
  if (!CL && lane == 0) {
    feed.w.at(a, reqs, cache_r0, start_r, start_t, start_h);
    feed.tile0 = start_u;
    feed.u = (int)(u0 - start_u) + warp;
    feed.end = (int)min((long long)feed.w.y.n_u, u1 - start_u);
    feed.ids_r = -1;
    if (warp == 0) tile_s[0] = feed.w;
  }
  int turn = 0, ready = 0;  // of feed.src
  auto produce = [&](int stage) {  // the copies of this warp's next unit, if any is left
    if (turn == ready) {
      ready = feed_refill<Blk, ROWS, kWarps>(a, feed, reqs, cache_r0, warp, u1);
      turn = 0;
      if (ready == 0) {
        if (C::across && lane == 0) feed.hidden[stage] = kStageIdle;
        return;
      }
    }
    if (lane == 0) {
      const ulonglong2 src = feed.src[turn];
      const uint32_t bar = bar0 + 8 * stage, dst = ring + stage * C::stage;
      if (src.y == src.x + Blk::bytes) {
        mbar_arrive_expect_tx(bar, C::stage);
        bulk_load(dst, reinterpret_cast<const void*>(src.x), C::stage, bar);
        feed.hidden[stage] = 0;
      } else {
        const bool b0 = src.x == 1, b1 = src.y == 1;
        mbar_arrive_expect_tx(bar, (uint32_t)(2 - b0 - b1) * Blk::bytes);
        if (!b0) bulk_load(dst, reinterpret_cast<const void*>(src.x), Blk::bytes, bar);
        if (!b1) bulk_load(dst + Blk::bytes, reinterpret_cast<const void*>(src.y), Blk::bytes, bar);
        feed.hidden[stage] = (uint32_t)b0 | ((uint32_t)b1 << 1);
      }
    }
    ++turn;
  };
  if constexpr (C::across)
#pragma unroll 1
    for (int s = 0; s < S; ++s) produce(s);
  __syncthreads();  // tile_s

  // ---- the tiles of the share, or of the cluster
  Ring<S> ring_at;
  int4 meta = make_int4(-1, 0, 0, 0);
  int meta_q0 = 0, meta_c0 = 0;
  long long tile0 = CL ? 0 : start_u;
  uint32_t rank = 0, ctas = 1;
  long long index = 0;
  if constexpr (CL) {
    rank = cluster_rank();
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    index = blockIdx.x / ctas;
  }
#pragma unroll 1
  for (int which = 0; CL ? index < total : tile0 < u1; which ^= (CL ? 0 : 1)) {
    [[maybe_unused]] bool given_up = false;
    if constexpr (CL) {
      given_up = tile0 > 0 && abort_s != 0;  // in a tile before; no thread waits for a copy until the barrier below
      if (index < end && index >= end - mine) {
        long long u = end - mine;
        bool found = false;
        for (int r = my0; r < my1 && !found; ++r) {
          const Req x = cached ? reqs[r] : load_req(a, r);
          const long long n = count_of(x);
          if (index < u + n) {
            Walk<ROWS> w;
            w.r = r;
            w.t = (int)((uint32_t)(index - u) / (uint32_t)a.c.Hk);
            w.h = (int)((uint32_t)(index - u) - (uint32_t)w.t * (uint32_t)a.c.Hk);
            w.x = x;
            w.y = tile_of<ROWS>(a, x, w.t);
            tile_s[0] = w;
            found = true;
          }
          u += n;
        }
      }
      __syncthreads();
    }
    const Walk<ROWS>& cw = tile_s[which];
    const Tile y = cw.y;
    const Req x = cw.x;
    int first, last;
    bool alone = true;  // CL: the whole tile is this CTA's
    if constexpr (CL) {
      int part = (y.n_u + (int)ctas - 1) / (int)ctas;
      part = (part + kWarps - 1) / kWarps * kWarps;
      first = min(y.n_u, (int)rank * part);
      last = min(y.n_u, first + part);
      alone = part >= y.n_u;
      if (given_up) first = last = y.n_u;
      if (lane == 0) {
        feed.w = cw;
        feed.tile0 = 0;
        feed.u = first + warp;
        feed.end = last;
        feed.ids_r = -1;
      }
      turn = ready = 0;
    } else {
      first = (int)max(0ll, u0 - tile0);
      last = (int)min((long long)y.n_u, u1 - tile0);
    }
    // the lane's channels of the query rows that its warp prepares (32 rows: eight for each warp)
    constexpr int NQ = NT == 4 ? 1 : NT;
    uint4 raw[NQ][D / 32];
    auto load_q = [&] {
#pragma unroll
      for (int jj = 0; jj < NQ; ++jj) {
        const int n = g + 8 * (NT == 4 ? warp : jj);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) raw[jj][i] = make_uint4(0, 0, 0, 0);
        if (n < y.rows) {
          const int row = y.row0 + n, qi = a.G.div(row);
          const uint4* src = reinterpret_cast<const uint4*>(
              static_cast<const uint16_t*>(a.q) + (x.q0 + qi) * a.qs[0] +
              ((long long)cw.h * a.G.d + (row - qi * (int)a.G.d)) * a.qs[1]);
#pragma unroll
          for (int i = 0; i < D / 32; ++i)  // 8 bits: 16-channel chunks t4 and, of 128 channels, t4 + 4
            raw[jj][i] = __ldg(src + (wide ? (t4 + 4 * (i >> 1)) * 2 + (i & 1) : t4 * (D / 32) + i));
        }
      }
    };
    if constexpr (CL) load_q();  // on their way beside the first units (shares: no gain, more registers)
    if constexpr (!C::across) {
      for (int s = 0, u = first + warp; s < S && u < last; ++s, u += kWarps) produce((ring_at.stage + s) % S);
      __syncwarp();  // the stages' words, which lane 0 writes (of later copies: the unit loop's)
    }
    if constexpr (!CL) load_q();
    // query rows: column n = g + 8 j of the tile's rows, this lane's channels, as B fragments.
    // Each row is brought to a largest magnitude in [1, 2) by a power of two (exact),
    // which its score factor takes back: no 16-bit query leaves fp16's range.
    // (32 rows: each warp prepares eight of them for all, in shared memory.)
    uint32_t qf[NT == 4 ? 1 : NT][KS][2];
    float factor[NT][2];
#pragma unroll
    for (int jj = 0; jj < NQ; ++jj) {
      const int j = NT == 4 ? warp : jj;
      if (NT == 4 && warp >= 4) break;
      const int n = g + 8 * j;
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t w[4] = {raw[jj][i].x, raw[jj][i].y, raw[jj][i].z, raw[jj][i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = unpack2<F16>(w[k]);
          big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // 2^e <= big < 2^(e + 1): exponent bits; down, up are 2^-e, 2^e (1 for 0 and inf)
      uint32_t eb = __float_as_uint(big) >> 23;
      eb = eb == 0 || eb == 255 ? 127u : min(eb, 253u);
      const float down = __uint_as_float((254u - eb) << 23), up = __uint_as_float(eb << 23);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t w[4] = {raw[jj][i].x, raw[jj][i].y, raw[jj][i].z, raw[jj][i].w};
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = unpack2<F16>(w[k]);
          f[2 * k] = v.x * down;
          f[2 * k + 1] = v.y * down;
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t v = wide ? pack2<true>(f[2 * p], f[2 * p + 1]) : pack2<true>(f[p], f[p + 4]);
          if constexpr (NT == 4) {
            reinterpret_cast<uint32_t*>(qfrag)[((j * KS + 2 * i + (p >> 1)) * 32 + lane) * 2 + (p & 1)] = v;
          } else {
            qf[jj][2 * i + (p >> 1)][p & 1] = v;
          }
        }
      }
      if constexpr (NT == 4) {
        if (t4 == 0) up_s[n] = up;
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c) factor[jj][c] = fmaxf(__shfl_sync(0xffffffffu, up, 4 * (2 * t4 + c)) * a.scale_log2, kLeast);
      }
    }
    if constexpr (NT == 4) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) factor[j][c] = fmaxf(up_s[8 * j + 2 * t4 + c] * a.scale_log2, kLeast);
    }
    // tokens that every row sees: no comparisons in their units
    const int i0 = a.G.div(y.row0), i1 = a.G.div(y.row0 + y.rows - 1);
    const int all_hi = x.kv - x.n + i0 + 1;
    const int all_lo = first_seen(a, x.kv - x.n + i1);

    // m: less the running maximum of the raw products; a score is (product + m) * factor, the
    // difference first: it is exact near the maximum, so that the weight there is 1 however large
    // the products (a product with the factor is off by whole powers of two from 2^24 on)
    float m[NT][2], l[NT][2], o[MT][NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      m[j][0] = m[j][1] = -kNoMax;
      l[j][0] = l[j][1] = 0.f;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][j][c] = 0.f;
    }
    // token of fragment row g of a block, and how far that of row g + 8 is from it.  8 bits: rows 2 t,
    // 2 t + 1, 2 t + 8 and 2 t + 9 are tokens 4 t to 4 t + 3, a word of values.
    const int kr = wide ? 4 * (g >> 1) + (g & 1) : g ^ ((g >> 1) & 1);
    constexpr int kr_next = wide ? 2 : 8;
    // 8 bits: O stands for o * vref, 2^-7 times the scale of the values of late (before the first block far
    // above any, so that the first one's is taken, while o is 0)
    constexpr float kNoScale = 0x1p40f;
    [[maybe_unused]] float vref = kNoScale, inv_vref = 1.f / kNoScale;
    auto product_k = [&](float (&s)[NT][4], int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        uint2 q0;
        if constexpr (NT == 4) q0 = qfrag[(j * KS + i) * 32 + lane];
        else q0 = make_uint2(qf[j][i][0], qf[j][i][1]);
        mma16816(s[j], a0, a1, a2, a3, q0.x, q0.y);
      }
    };
    // S^T of a block: raw products
    auto scores = [&](uint32_t kb, float (&s)[NT][4]) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[j][c] = 0.f;
      if constexpr (wide) {
        const uint32_t ra = kb + kr * Blk::row + kv8_key_chunk<D>(kr, t4) * 16, rb = ra + kr_next * Blk::row;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {  // chunk t4 + 4 h: the other half of the row
          const int off = h == 0 ? 0 : (g & 1) ? -64 : 64;
          const uint4 u = ld_shared_v4(ra + off), v = ld_shared_v4(rb + off);
          const uint32_t wu[4] = {u.x, u.y, u.z, u.w}, wv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t a0, a1, a2, a3;
            codes4(wu[i], a0, a2);
            codes4(wv[i], a1, a3);
            product_k(s, 4 * h + i, a0, a1, a2, a3);
          }
        }
        return;
      } else {
        uint32_t wa[WPT], wb[WPT];
        const uint32_t ra = kb + kr * Blk::row + t4 * (D / 8), rb = ra + 8 * Blk::row;
        if constexpr (D == 128) {
          const uint4 u = ld_shared_v4(ra), v = ld_shared_v4(rb);
          wa[0] = u.x; wa[1] = u.y; wa[2] = u.z; wa[3] = u.w;
          wb[0] = v.x; wb[1] = v.y; wb[2] = v.z; wb[3] = v.w;
        } else {
          const uint2 u = lds64(ra), v = lds64(rb);
          wa[0] = u.x; wa[1] = u.y;
          wb[0] = v.x; wb[1] = v.y;
        }
        const uint32_t pa = kb + Blk::codes + (kr * Blk::groups + (D == 128 ? t4 : t4 >> 1)) * 4;
        const uint32_t xa = lds32(pa), xb = lds32(pa + 8 * Blk::groups * 4);
        const uint32_t sa = __byte_perm(xa, xa, 0x1010), ca = __byte_perm(xa, xa, 0x3232);
        const uint32_t sb = __byte_perm(xb, xb, 0x1010), cb = __byte_perm(xb, xb, 0x3232);
#pragma unroll
        for (int i = 0; i < WPT; ++i) {
          const uint32_t a0 = hfma2(code_pair<0>(magic, wa[i]), sa, ca), a1 = hfma2(code_pair<0>(magic, wb[i]), sb, cb);
          const uint32_t a2 = hfma2(code_pair<1>(magic, wa[i]), sa, ca), a3 = hfma2(code_pair<1>(magic, wb[i]), sb, cb);
          const uint32_t c0 = hfma2(code_pair<2>(magic, wa[i]), sa, ca), c1 = hfma2(code_pair<2>(magic, wb[i]), sb, cb);
          const uint32_t c2 = hfma2(code_pair<3>(magic, wa[i]), sa, ca), c3 = hfma2(code_pair<3>(magic, wb[i]), sb, cb);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            uint2 q0, q1;
            if constexpr (NT == 4) {
              q0 = qfrag[(j * KS + 2 * i) * 32 + lane];
              q1 = qfrag[(j * KS + 2 * i + 1) * 32 + lane];
            } else {
              q0 = make_uint2(qf[j][2 * i][0], qf[j][2 * i][1]);
              q1 = make_uint2(qf[j][2 * i + 1][0], qf[j][2 * i + 1][1]);
            }
            mma16816(s[j], a0, a1, a2, a3, q0.x, q0.y);
            mma16816(s[j], c0, c1, c2, c3, q1.x, q1.y);
          }
        }
      }
    };
    // O^T += V^T P^T of a block: this lane's tokens are those of fragment rows 2 t, 2 t + 1 and 8 more
    auto values = [&](uint32_t vb, const uint32_t (&p0)[NT], const uint32_t (&p1)[NT]) {
      if constexpr (wide) {
#pragma unroll
        for (int n = 0; n < D / 32; ++n) {
          const uint4 u = ld_shared_v4(vb + (8 * n + g) * 64 + t4 * 16);  // channels 4 (8 n + g) .., tokens 4 t4 ..
          const uint32_t wu[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t a0, a1, a2, a3;
            codes4(wu[2 * e], a0, a2);
            codes4(wu[2 * e + 1], a1, a3);
#pragma unroll
            for (int j = 0; j < NT; ++j) mma16816(o[2 * n + e][j], a0, a1, a2, a3, p0[j], p1[j]);
          }
        }
        return;
      } else {
        constexpr int WV = D / 64;  // words of codes of a token per lane (8 channels each)
        const int e0 = 2 * t4, e1 = 2 * t4 + 1;
        const int ke = e0 ^ ((e0 >> 1) & 1), kf = e1 ^ ((e1 >> 1) & 1);
        uint32_t w[4][WV], pr[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int key = (q & 1 ? kf : ke) + (q >> 1) * 8;
          const uint32_t at = vb + key * Blk::row + g * (D / 16);
          if constexpr (D == 128) {
            const uint2 u = lds64(at);
            w[q][0] = u.x;
            w[q][1] = u.y;
          } else {
            w[q][0] = lds32(at);
          }
          pr[q] = lds32(vb + Blk::codes + (key * Blk::groups + (D == 128 ? g >> 1 : g >> 2)) * 4);
        }
        const uint32_t sx = __byte_perm(pr[0], pr[1], 0x5410), cx = __byte_perm(pr[0], pr[1], 0x7632);
        const uint32_t sy = __byte_perm(pr[2], pr[3], 0x5410), cy = __byte_perm(pr[2], pr[3], 0x7632);
#pragma unroll
        for (int i = 0; i < WV; ++i) {
          const uint32_t xl = __byte_perm(w[0][i], w[1][i], 0x5410), xh = __byte_perm(w[0][i], w[1][i], 0x7632);
          const uint32_t yl = __byte_perm(w[2][i], w[3][i], 0x5410), yh = __byte_perm(w[2][i], w[3][i], 0x7632);
          auto product = [&](int mt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
            a0 = hfma2(a0, sx, cx);
            a1 = hfma2(a1, sx, cx);
            a2 = hfma2(a2, sy, cy);
            a3 = hfma2(a3, sy, cy);
#pragma unroll
            for (int j = 0; j < NT; ++j) mma16816(o[mt][j], a0, a1, a2, a3, p0[j], p1[j]);
          };
          product(4 * i + 0, code_pair<0>(magic, xl), code_pair<0>(magic, xh), code_pair<0>(magic, yl), code_pair<0>(magic, yh));
          product(4 * i + 1, code_pair<1>(magic, xl), code_pair<1>(magic, xh), code_pair<1>(magic, yl), code_pair<1>(magic, yh));
          product(4 * i + 2, code_pair<2>(magic, xl), code_pair<2>(magic, xh), code_pair<2>(magic, yl), code_pair<2>(magic, yh));
          product(4 * i + 3, code_pair<3>(magic, xl), code_pair<3>(magic, xh), code_pair<3>(magic, yl), code_pair<3>(magic, yh));
        }
      }
    };

    constexpr int kGaveUp = S;  // of `held`: and the copies under way
    int held = -1;  // stage of the tile's last unit, kept for the join (across)
#pragma unroll 1
    for (int u = first + warp; u < last; u += kWarps) {
      const int stage = ring_at.stage;
      if (!warp_wait(wc, bar0 + 8 * stage, ring_at.parity)) {
        held = kGaveUp + (C::across ? 0 : min(S, (last - u + kWarps - 1) / kWarps));
        break;
      }
      const uint32_t kb = ring + stage * C::stage;
      const int key0 = y.u0 + u * kUnit;
      const uint32_t hidden = feed.hidden[stage];
      bool masked = hidden || key0 + kUnit > all_hi || key0 < all_lo;
      // 8 bits: the blocks' scales, 0 for one that was not read (whose weights are 0), and marks
      [[maybe_unused]] float ks[2], vs[2];
      [[maybe_unused]] uint32_t k_nan = 0, v_nan = 0;
      if constexpr (wide) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 tail = ld_shared_v4(kb + h * Blk::bytes + Blk::tail);
          const bool read = !((hidden >> h) & 1u);
          ks[h] = read ? __uint_as_float(tail.x) : 0.f;
          vs[h] = read ? __uint_as_float(tail.y) : 0.f;
          k_nan |= read ? (tail.z & 0xFFFFu) << (16 * h) : 0u;
          v_nan |= read ? (tail.z >> 16) << (16 * h) : 0u;
        }
        masked |= (k_nan | v_nan) != 0u;
        if (v_nan != 0u) {  // a NaN value makes the sums NaN of the rows that see its token
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int pos = x.kv - x.n + a.G.div(y.row0 + 8 * j + 2 * t4 + c);
              const uint32_t behind = below(min(pos + 1, x.kv) - key0), before = below(first_seen(a, pos) - key0);
              const float add = v_nan & behind & ~before ? NAN : 0.f;
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[i][j][c] += add;
                o[i][j][c + 2] += add;
              }
            }
        }
      }
      if constexpr (!wide) if (masked) {
        // values that no row sees must not reach the product (0 x NaN), nor a NaN that only
        // some rows see: their pairs become 0, and a NaN one makes the sums NaN of the rows
        // that see its token, in its group's channels
        uint32_t nan_keys = 0;  // of group lane % groups
        for (int e = lane; e < kUnit * Blk::groups; e += 32) {
          const int key = e / Blk::groups;
          const uint32_t at = kb + (key / kKvBlock) * Blk::bytes + Blk::half + Blk::codes + (e % (kKvBlock * Blk::groups)) * 4;
          const uint32_t pair = lds32(at);
          const bool seen = !((hidden >> (key / kKvBlock)) & 1u) && key0 + key >= y.k0 && key0 + key < y.k1;
          const __half2 h = *reinterpret_cast<const __half2*>(&pair);
          const bool nan = __hisnan(__low2half(h)) || __hisnan(__high2half(h));
          if (!seen || nan) asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(0) : "memory");
          if (seen && nan) nan_keys |= 1u << key;
        }
        if (__any_sync(0xffffffffu, nan_keys)) {
#pragma unroll
          for (int off = Blk::groups; off < 32; off <<= 1) nan_keys |= __shfl_xor_sync(0xffffffffu, nan_keys, off);
          nan_keys = __shfl_sync(0xffffffffu, nan_keys, D == 128 ? g >> 1 : g >> 2);  // of this lane's channels
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int pos = x.kv - x.n + a.G.div(y.row0 + 8 * j + 2 * t4 + c);
              const uint32_t behind = below(min(pos + 1, x.kv) - key0), before = below(first_seen(a, pos) - key0);
              const float add = nan_keys & behind & ~before ? NAN : 0.f;
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[i][j][c] += add;
                o[i][j][c + 2] += add;
              }
            }
        }
        __syncwarp();
        fence_async_smem();  // these stores before the copy that reuses the stage
      }
      float s[2][NT][4];
      scores(kb, s[0]);
      scores(kb + Blk::bytes, s[1]);
      if constexpr (wide) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 4; c += 2)
              f2unpack(fmul2(f2pack(s[h][j][c], s[h][j][c + 1]), f2pack(ks[h], ks[h])), s[h][j][c], s[h][j][c + 1]);
      }
      if (masked) {  // hidden tokens
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int pos = x.kv - x.n + a.G.div(y.row0 + 8 * j + 2 * t4 + c);  // rows behind the last: of no consequence
            const int lim = min(pos + 1, x.kv) - key0, low = first_seen(a, pos) - key0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const int key = 16 * h + kr_next * q + kr;
                const bool seen = !((hidden >> h) & 1u) && key < lim && key >= low;
                float& v = s[h][j][2 * q + c];
                if (wide && (k_nan >> key) & 1u) v = NAN;
                v = seen ? v : -INFINITY;
              }
          }
      }
      // the running maximum, moved when a score is above it by more than 8 in log2 units
      float most[NT][2];
      bool grow = false;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          most[j][c] = fmax3(fmaxf(s[0][j][c], s[0][j][c + 2]), s[1][j][c], s[1][j][c + 2]);
          grow |= (most[j][c] + m[j][c]) * factor[j][c] > 8.f;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = fmaxf(most[j][c], -m[j][c]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float back = ex2((-m[j][c] - top) * factor[j][c]);
            m[j][c] = -top;
            l[j][c] *= back;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[i][j][c] *= back;
              o[i][j][c + 2] *= back;
            }
          }
      }
      // weights, and their transpose as the B operand: in fp16 (2^-11 of each, 2^-25 where
      // subnormal), the type of the values they are multiplied with; l adds them in fp32
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t p0[NT], p1[NT];
        [[maybe_unused]] float ratio = 1.f;
        if constexpr (wide) {
          // the weights, at most 2^8, take the scale of the block's values relative to vref: in [1, 2^7], so
          // that they stay below fp16's largest number and none is rounded to less than without it,
          // whatever the blocks before; where it is not O takes the block's.  (In [2^-8, 1] a weight of e^-12
          // behind a block of values 2^8 times as large would be 0.)
          ratio = vs[h] * inv_vref;
          if (!(ratio <= 0x1p7f && ratio >= 1.f) && vs[h] != 0.f) {
            const float to = vs[h] * 0x1p-7f;
            if (vref != kNoScale) {
              const float back = vref / to;
#pragma unroll
              for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                  for (int c = 0; c < 4; ++c) o[i][j][c] *= back;
            }
            vref = to;
            inv_vref = 1.f / to;
            ratio = 0x1p7f;
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
          for (int c = 0; c < 4; c += 2) {
            float x, y;
            f2unpack(fmul2(fadd2(f2pack(s[h][j][c], s[h][j][c + 1]), f2pack(m[j][0], m[j][1])), f2pack(factor[j][0], factor[j][1])), x, y);
            s[h][j][c] = ex2(x);
            s[h][j][c + 1] = ex2(y);
          }
          l[j][0] += s[h][j][0] + s[h][j][2];
          l[j][1] += s[h][j][1] + s[h][j][3];
          if constexpr (wide) {
#pragma unroll
            for (int c = 0; c < 4; c += 2)
              f2unpack(fmul2(f2pack(s[h][j][c], s[h][j][c + 1]), f2pack(ratio, ratio)), s[h][j][c], s[h][j][c + 1]);
          }
          p0[j] = transpose8x8(pack2<true>(s[h][j][0], s[h][j][1]));
          p1[j] = transpose8x8(pack2<true>(s[h][j][2], s[h][j][3]));
        }
        values(kb + h * Blk::bytes + Blk::half, p0, p1);
      }
      __syncwarp();  // every lane has read the stage
      if (C::across ? u + kWarps < last : u + S * kWarps < last)
        produce(stage);
      else
        held = stage;
      ring_at.next();
    }
    if (held >= kGaveUp) {
      __syncwarp();
      drain_ring<S, Context>(wc, bar0, ring_at, C::across ? ring_at.armed(feed.hidden) : held - kGaveUp);
      held = ring_at.stage;
    }

    // ---- join the warps that took units of the tile
    const int active = min(kWarps, last - first);
    auto joined = [&](int w) {  // warp w's O, [ROWS][LDO]
      return reinterpret_cast<float*>(smem + w * (S * C::stage) + (C::across ? held_s[w] * C::stage : 0));
    };
    if (warp < active) {
      if (lane == 0) held_s[warp] = held;
      __syncwarp();
      float* mine = joined(warp);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float v = l[j][c];
          v += __shfl_xor_sync(0xffffffffu, v, 4);
          v += __shfl_xor_sync(0xffffffffu, v, 8);
          v += __shfl_xor_sync(0xffffffffu, v, 16);
          const int row = 8 * j + 2 * t4 + c;
          if (g == 0) {
            m_s[warp][row] = m[j][c] == -kNoMax ? kNoMax : -m[j][c] * factor[j][c];
            l_s[warp][row] = v;
          }
          if constexpr (wide) {  // channels 4 (8 n + g) .. of m-tiles 2 n and 2 n + 1
#pragma unroll
            for (int n = 0; n < D / 32; ++n)
              *reinterpret_cast<float4*>(mine + row * C::LDO + 32 * n + 4 * g) =
                  make_float4(o[2 * n][j][c] * vref, o[2 * n][j][c + 2] * vref, o[2 * n + 1][j][c] * vref, o[2 * n + 1][j][c + 2] * vref);
            continue;
          }
          float* to = mine + row * C::LDO + g * (D / 8);
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            *reinterpret_cast<float4*>(to + 8 * i) =
                make_float4(o[4 * i][j][c], o[4 * i + 1][j][c], o[4 * i + 2][j][c], o[4 * i + 3][j][c]);
            *reinterpret_cast<float4*>(to + 8 * i + 4) =
                make_float4(o[4 * i][j][c + 2], o[4 * i + 1][j][c + 2], o[4 * i + 2][j][c + 2], o[4 * i + 3][j][c + 2]);
          }
        }
      }
      fence_async_smem();  // these stores before the copies that reuse the ring
    }
    __syncthreads();
    constexpr int TPR = D / 8;  // threads per row, 8 channels each
    // adds weight f's (l, O[8 channels])
    auto add8 = [](float f, float l, const float4& u, const float4& v, float& sum, float (&acc)[8]) {
      sum = fmaf(f, l, sum);
      acc[0] = fmaf(f, u.x, acc[0]); acc[1] = fmaf(f, u.y, acc[1]);
      acc[2] = fmaf(f, u.z, acc[2]); acc[3] = fmaf(f, u.w, acc[3]);
      acc[4] = fmaf(f, v.x, acc[4]); acc[5] = fmaf(f, v.y, acc[5]);
      acc[6] = fmaf(f, v.z, acc[6]); acc[7] = fmaf(f, v.w, acc[7]);
    };
    // the warps' sum at (row, channels ch .. ch + 7)
    auto join = [&](int row, int ch, float& top, float& sum, float (&acc)[8]) {
      top = kNoMax;
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.f;
      for (int w = 0; w < active; ++w) top = fmaxf(top, m_s[w][row]);
      for (int w = 0; w < active; ++w) {
        const float4* src = reinterpret_cast<const float4*>(joined(w) + row * C::LDO + ch);
        add8(ex2(m_s[w][row] - top), l_s[w][row], src[0], src[1], sum, acc);
      }
    };
    auto write = [&](int row, int ch, float top, float sum, const float (&acc)[8]) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int gr = y.row0 + row, qi = a.G.div(gr);
      const long long head = (long long)cw.h * a.G.d + (gr - qi * (int)a.G.d);
      uint16_t* to = static_cast<uint16_t*>(a.o) + (x.q0 + qi) * a.os[0] + head * a.os[1] + ch;
      if (fa_bounds(a.rep.st, x.q0 + qi < a.T && head < a.Hq)) {
        *reinterpret_cast<uint4*>(to) =
            make_uint4(pack2<F16>(acc[0] * inv, acc[1] * inv), pack2<F16>(acc[2] * inv, acc[3] * inv),
                       pack2<F16>(acc[4] * inv, acc[5] * inv), pack2<F16>(acc[6] * inv, acc[7] * inv));
        if (ch == 0 && a.lse)
          a.lse[(long long)(x.q0 + qi) * a.Hq + head] =
              sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
      }
    };
    if constexpr (CL) {
      constexpr int ITEMS = (ROWS * TPR + kThreads - 1) / kThreads;
      if (alone) {  // the first CTA's
        if (rank == 0)
          for (int e = tid; e < y.rows * TPR; e += kThreads) {
            float top, sum, acc[8];
            join(e / TPR, e % TPR * 8, top, sum, acc);
            write(e / TPR, e % TPR * 8, top, sum, acc);
          }
        __syncthreads();  // joined, m_s, l_s, tile_s read
      } else {
        float top[ITEMS], sum[ITEMS], acc[ITEMS][8];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          const int e = tid + i * kThreads;
          if (e < y.rows * TPR) join(e / TPR, e % TPR * 8, top[i], sum[i], acc[i]);
        }
        __syncthreads();  // joined read: the CTA's sum takes its place
        float* red = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          const int e = tid + i * kThreads, row = e / TPR, ch = e % TPR * 8;
          if (e < y.rows * TPR) {
            *reinterpret_cast<float4*>(red + row * C::LDO + ch) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
            *reinterpret_cast<float4*>(red + row * C::LDO + ch + 4) = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
            if (ch == 0) ml_s[row] = make_float2(top[i], sum[i]);
          }
        }
        fence_async_smem();
        cluster_sync();
        // the cluster's sum, its items spread over the CTAs
        for (int e = (int)rank * kThreads + tid; e < y.rows * TPR; e += (int)ctas * kThreads) {
          const int row = e / TPR, ch = e % TPR * 8;
          float t = kNoMax, l = 0.f, v[8] = {};
          const uint32_t ml = smem_addr(&ml_s[row]), at = smem_addr(red + row * C::LDO + ch);
          for (uint32_t c = 0; c < ctas; ++c) t = fmaxf(t, ld_cluster_f32x2(cluster_map(ml, c)).x);
          for (uint32_t c = 0; c < ctas; ++c) {
            const float2 p = ld_cluster_f32x2(cluster_map(ml, c));
            const uint32_t from = cluster_map(at, c);
            add8(ex2(p.x - t), p.y, ld_cluster_f32x4(from), ld_cluster_f32x4(from + 16), l, v);
          }
          write(row, ch, t, l, v);
        }
        cluster_sync();  // the CTAs' sums read
      }
      index += gridDim.x / ctas;
    } else {
      const bool from_before = first > 0, goes_on = tile0 + y.n_u > u1;
      given_up = abort_s != 0;  // no thread waits for a copy until the barrier below
      for (int e = tid; e < y.rows * TPR; e += kThreads) {
        const int row = e / TPR, ch = (e % TPR) * 8;
        float top, sum, acc[8];
        join(row, ch, top, sum, acc);
        if (from_before || goes_on) {
          float* to = a.part + ((size_t)(2 * blockIdx.x + (from_before ? 0 : 1)) * ROWS + row) * (D + 4);
          *reinterpret_cast<float4*>(to + 4 + ch) = make_float4(acc[0], acc[1], acc[2], acc[3]);
          *reinterpret_cast<float4*>(to + 8 + ch) = make_float4(acc[4], acc[5], acc[6], acc[7]);
          if (ch == 0) {
            to[0] = top;
            to[1] = sum;
          }
        } else {
          write(row, ch, top, sum, acc);
        }
      }
      if (tid == 0) {
        const long long tile_end = tile0 + y.n_u;
        if (goes_on) {  // this share's last tile
          meta = make_int4(y.row0, y.rows, cw.h, (int)((tile_end - 1) / share));
          meta_q0 = x.q0;
          meta_c0 = from_before ? (int)(tile0 / share) : (int)blockIdx.x;
        }
        if (tile_end < u1) {
          Walk<ROWS> w = cw;
          w.next(a, reqs, cache_r0);
          tile_s[which ^ 1] = w;
        }
      }
      __syncthreads();  // joined, m_s, l_s read; the next tile known
    }
    if constexpr (!CL) {
      if (given_up) {
        if constexpr (C::across) {  // what was fetched of the coming tiles
          if (held >= 0 && lane == 0) feed.hidden[held] = kStageIdle;  // consumed
          __syncwarp();
          drain_ring<S, Context>(wc, bar0, ring_at, ring_at.armed(feed.hidden));
        }
        break;
      }
    }
    if (C::across && held >= 0) produce(held);
    tile0 += y.n_u;
  }
  if (!CL && tid == 0) {
    a.meta[2 * blockIdx.x] = meta;
    a.meta[2 * blockIdx.x + 1] = make_int4(meta_q0, meta_c0, 0, 0);
  }
}

// Adds the shares of the tiles that were cut.  A tile cut into k shares has k - 1 blocks here,
// those of its shares but the last, and as many of them as it has rows divide the rows: a
// pair of shares is one block's, a tile of hundreds of shares (a long context among short
// ones) a block's for every row.  Few shares: a warp for each row; many: the block's warps
// divide a row's shares.  A lane has D / 32 channels.  Bound by the chain: the end of the
// first kernel, the tile's place, its sums (64 requests up to 16384 tokens: 146 us with the first
// kernel; with eight rows to a block and two passes 149).
constexpr int kMergeWarps = 8;
// Of shares c, c + step, ... to `last` of a row: the largest maximum, and l and O by it.
// AT_ONCE of them are on their way together.  (The first share's slot is its second one.)
template <int D, int ROWS, int AT_ONCE>
__device__ __forceinline__ void add_shares(const float* part, int row, int c0, int last, int c, int step, float& top,
                                           float& sum, float (&acc)[D / 32]) {
  constexpr int CPL = D / 32;
  const int lane = threadIdx.x & 31;
  top = kNoMax;
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < CPL; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (; c <= last; c += AT_ONCE * step) {
    float2 ml[AT_ONCE];
    float v[AT_ONCE][CPL];
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const int e = c + k * step;
      ml[k] = make_float2(kNoMax, 0.f);
#pragma unroll
      for (int i = 0; i < CPL; ++i) v[k][i] = 0.f;
      if (e <= last) {
        const float* s = part + ((size_t)(2 * e + (e == c0 ? 1 : 0)) * ROWS + row) * (D + 4);
        ml[k] = *reinterpret_cast<const float2*>(s);
        if constexpr (CPL == 4) {
          const float4 u = *reinterpret_cast<const float4*>(s + 4 + 4 * lane);
          v[k][0] = u.x; v[k][1] = u.y; v[k][2] = u.z; v[k][3] = u.w;
        } else {
          const float2 u = *reinterpret_cast<const float2*>(s + 4 + 2 * lane);
          v[k][0] = u.x; v[k][1] = u.y;
        }
      }
    }
    float t = top;
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) t = fmaxf(t, ml[k].x);
    const float f = ex2(top - t);
    top = t;
    sum *= f;
#pragma unroll
    for (int i = 0; i < CPL; ++i) acc[i] *= f;
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const float g = ex2(ml[k].x - t);
      sum = fmaf(g, ml[k].y, sum);
#pragma unroll
      for (int i = 0; i < CPL; ++i) acc[i] = fmaf(g, v[k][i], acc[i]);
    }
  }
}

template <int D, int NT, bool F16>
__global__ void __launch_bounds__(32 * kMergeWarps) kv_merge_kernel(const Kv4AttnArgs a) {
  constexpr int ROWS = 8 * NT, CPL = D / 32, FEW = 16;
  __shared__ float top_s[kMergeWarps], sum_s[kMergeWarps];
  __shared__ __align__(16) float acc_s[kMergeWarps][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 meta = a.meta[2 * blockIdx.x];  // first row, rows, key head, last share
  const int4 more = a.meta[2 * blockIdx.x + 1];
  const int q0 = more.x, c0 = more.y;  // the request's first query row, the tile's first share
  if (meta.x < 0) return;
  const int rows = meta.y, shares = meta.w - c0 + 1, blocks = min(rows, shares - 1), mine = (int)blockIdx.x - c0;
  if (mine >= blocks) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto write = [&](int row, float top, float sum, const float (&acc)[CPL]) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int gr = meta.x + row, qi = a.G.div(gr);
    const long long head = (long long)meta.z * a.G.d + (gr - qi * (int)a.G.d);
    if (!fa_bounds(a.rep.st, q0 + qi < a.T && head < a.Hq)) return;
    uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + (q0 + qi) * a.os[0] + head * a.os[1] + lane * CPL);
#pragma unroll
    for (int i = 0; i < CPL / 2; ++i) to[i] = pack2<F16>(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    if (lane == 0 && a.lse)
      a.lse[(long long)(q0 + qi) * a.Hq + head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
  };
  float top, sum, acc[CPL];
  if (shares <= FEW) {
    for (int row = mine + blocks * warp; row < rows; row += blocks * kMergeWarps) {
      add_shares<D, ROWS, 4>(a.part, row, c0, meta.w, c0, 1, top, sum, acc);
      write(row, top, sum, acc);
    }
    return;
  }
  for (int row = mine; row < rows; row += blocks) {
    add_shares<D, ROWS, 8>(a.part, row, c0, meta.w, c0 + warp, kMergeWarps, top, sum, acc);
    __syncthreads();  // the row before has been written
    if (lane == 0) {
      top_s[warp] = top;
      sum_s[warp] = sum;
    }
#pragma unroll
    for (int i = 0; i < CPL; ++i) acc_s[warp][lane * CPL + i] = acc[i];
    __syncthreads();
    if (warp == 0) {
      top = top_s[0];
#pragma unroll
      for (int w = 1; w < kMergeWarps; ++w) top = fmaxf(top, top_s[w]);
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < CPL; ++i) acc[i] = 0.f;
#pragma unroll
      for (int w = 0; w < kMergeWarps; ++w) {
        const float f = ex2(top_s[w] - top);
        sum = fmaf(f, sum_s[w], sum);
#pragma unroll
        for (int i = 0; i < CPL; ++i) acc[i] = fmaf(f, acc_s[w][lane * CPL + i], acc[i]);
      }
      write(row, top, sum, acc);
    }
  }
}

// ctas: of the launch; cluster: CTAs of a cluster, or 0 for shares.
template <class Blk, int NT, bool F16>
cudaError_t launch(const Kv4AttnArgs& a, int ctas, int cluster, cudaStream_t s) {
  using C = Cfg<Blk, NT, false>;
  using CC = Cfg<Blk, NT, true>;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cudaError_t e;
  if (cluster > 0) {
    const auto k = kv_attn_kernel<Blk, NT, F16, true>;
    if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, CC::smem)) != cudaSuccess) return e;
    if (cluster > 8 && (e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
      return e;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(CC::THREADS);
    cfg.dynamicSmemBytes = CC::smem;
    return cudaLaunchKernelEx(&cfg, k, a);
  }
  const auto k = kv_attn_kernel<Blk, NT, F16, false>;
  if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem)) != cudaSuccess) return e;
  k<<<ctas, C::THREADS, C::smem, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.gridDim = dim3(ctas);
  return cudaLaunchKernelEx(&cfg, kv_merge_kernel<Blk::D, NT, F16>, a);
}

}  // namespace

// Clusters of a size that the GPU holds at once: what its groups of SMs have room for, fewer
// than the CTAs alone would allow (of 16 CTAs, two to an SM: 14, not 19).
template <class Blk>
int kv_clusters_at_once(int rows, int cluster) {
  auto ask = [&](auto k, int threads, int smem) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    int n = 0;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    return n;
  };
  return rows == 8    ? ask(kv_attn_kernel<Blk, 1, false, true>, Cfg<Blk, 1, true>::THREADS, Cfg<Blk, 1, true>::smem)
         : rows == 16 ? ask(kv_attn_kernel<Blk, 2, false, true>, Cfg<Blk, 2, true>::THREADS, Cfg<Blk, 2, true>::smem)
                      : ask(kv_attn_kernel<Blk, 4, false, true>, Cfg<Blk, 4, true>::THREADS, Cfg<Blk, 4, true>::smem);
}

template <class Blk>
cudaError_t launch_kv_attention(const Kv4AttnArgs& a, bool f16, int rows, int ctas, int cluster, cudaStream_t s) {
  if (f16)
    return rows == 8    ? launch<Blk, 1, true>(a, ctas, cluster, s)
           : rows == 16 ? launch<Blk, 2, true>(a, ctas, cluster, s)
                        : launch<Blk, 4, true>(a, ctas, cluster, s);
  return rows == 8    ? launch<Blk, 1, false>(a, ctas, cluster, s)
         : rows == 16 ? launch<Blk, 2, false>(a, ctas, cluster, s)
                      : launch<Blk, 4, false>(a, ctas, cluster, s);
}

}  // namespace fa
