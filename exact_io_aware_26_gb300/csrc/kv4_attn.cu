// kv4_attn.cu -- attention of each request's newest tokens over its 4-bit cache.
//
// Bound: HBM.  A token of one head is 160 bytes (d = 128) for both its key and its
// value, and 8 query rows need 4 * 8 * d FLOPs of it: 26 FLOPs a byte, far below
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
// Work.  All tiles (request, 8 NT query rows, key head) lie one after the other as
// 16-token blocks; each CTA takes an equal share of all blocks, wherever it begins and
// ends, so that ragged lengths leave no SM idle.  A tile inside one share is finished
// there; one that is cut leaves fp32 (O, m, l) per share, which the second kernel adds.
// Within a CTA the warps take the blocks of a tile in turn, each with its own ring of
// bulk copies and its own m, l, O, joined in shared memory at the tile's end.
#include "kv4.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kNoMax = -1e30f;     // running maximum before any token is seen
constexpr int kMinShare = 32;        // blocks: shares are not cut finer (8 per warp)
constexpr int kReqCache = 128;       // requests whose lengths a CTA keeps at hand

template <int D, int NT>
struct Cfg {
  using Blk = KvBlock<D>;
  static constexpr int ROWS = 8 * NT;
  static constexpr int STAGES = D == 128 ? 3 : 6;
  static constexpr int CTAS_PER_SM = NT == 1 ? 4 : NT == 2 ? 3 : 2;
  static constexpr int LDO = D + 4;  // row pitch of the joined O, in floats
  static constexpr int ring = kWarps * STAGES * Blk::bytes;
  static constexpr int joined = kWarps * ROWS * LDO * 4;
  static constexpr int qfrag = NT == 4 ? NT * (D / 16) * 32 * 8 : 0;
  static constexpr int smem = ring + joined + qfrag;
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

// 1 + c / 16 of codes P and P + 4 (bits 4 P and 16 + 4 P) of a word, as half2.
template <int P>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  const uint32_t x = P == 0 ? w << 6 : P == 1 ? w << 2 : P == 2 ? w >> 2 : w >> 6;
  return (x & 0x03C003C0u) | 0x3C003C00u;
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

// Tile `t` of a request: rows [row0, row0 + ROWS) of its n * G, tokens [k0, k1) that some
// row of it sees, blocks [b0, b0 + nb) (one, of hidden tokens, where no row sees any).
struct Tile {
  int row0, rows, k0, k1, b0, nb;
};
template <int ROWS>
__device__ __forceinline__ int tiles_of(const Kv4AttnArgs& a, const Req& x) {
  return (int)(((long long)x.n * a.G + ROWS - 1) / ROWS);
}
template <int ROWS>
__device__ __forceinline__ Tile tile_of(const Kv4AttnArgs& a, const Req& x, int t) {
  Tile y;
  y.row0 = t * ROWS;
  y.rows = min(ROWS, x.n * a.G - y.row0);
  const int i0 = y.row0 / a.G, i1 = (y.row0 + y.rows - 1) / a.G;
  y.k1 = max(0, x.kv - x.n + i1 + 1);
  y.k0 = a.window > 0 ? max(0, x.kv - x.n + i0 - a.window + 1) : 0;
  y.k0 = min(y.k0, y.k1);
  y.b0 = y.k0 / kKvBlock;
  y.nb = max(1, (y.k1 + kKvBlock - 1) / kKvBlock - y.b0);
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

template <int D, int NT, bool F16>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::CTAS_PER_SM) kv4_attn_kernel(const Kv4AttnArgs a) {
  using C = Cfg<D, NT>;
  using Blk = KvBlock<D>;
  constexpr int ROWS = C::ROWS, S = C::STAGES, KS = D / 16, MT = D / 16, WPT = D / 32 /* words per lane of K */;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps][S];
  __shared__ long long thread_end[kThreads];
  __shared__ Req reqs[kReqCache];
  __shared__ long long start_s[2];
  __shared__ int start_r, start_t, start_h;
  __shared__ float m_s[kWarps][ROWS], l_s[kWarps][ROWS];
  __shared__ volatile int abort_s;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const uint32_t ring = smem_addr(smem) + warp * (S * Blk::bytes);
  float* joined = reinterpret_cast<float*>(smem + C::ring);
  uint2* qfrag = reinterpret_cast<uint2*>(smem + C::ring + C::joined);
  (void)qfrag;

  // ---- shares: prefix sums of the blocks of all requests
  if (tid == 0) abort_s = 0;
  if (lane == 0)
    for (int s = 0; s < S; ++s) mbar_init(smem_addr(&bars[warp][s]), 1);
  fence_barrier_init();
  const int per = (a.R + kThreads - 1) / kThreads;
  const int my0 = min(a.R, tid * per), my1 = min(a.R, my0 + per);
  long long units = 0;
  for (int r = my0; r < my1; ++r) {
    const Req x = load_req(a, r);
    const int nt = tiles_of<ROWS>(a, x);
    for (int t = 0; t < nt; ++t) units += (long long)tile_of<ROWS>(a, x, t).nb * a.c.Hk;
  }
  long long end = units;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, end, off);
    if (lane >= off) end += up;
  }
  thread_end[tid] = end;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    const long long x = thread_end[32 * w + 31];
    if (w < warp) before += x;
    total += x;
  }
  end += before;
  long long share = (total + gridDim.x - 1) / gridDim.x;
  share = max((share + kWarps - 1) / kWarps * kWarps, (long long)kMinShare);
  const long long u0 = (long long)blockIdx.x * share, u1 = min(total, u0 + share);
  if (u0 >= total) {  // no share (the CTA's threads all leave)
    if (tid == 0) a.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  // the thread whose requests hold block u0 finds its tile
  if (u0 < end && u0 >= end - units) {
    long long u = end - units;
    bool found = false;
    for (int r = my0; r < my1 && !found; ++r) {
      const Req x = load_req(a, r);
      const int nt = tiles_of<ROWS>(a, x);
      for (int t = 0; t < nt && !found; ++t) {
        const long long nb = tile_of<ROWS>(a, x, t).nb;
        if (u0 < u + nb * a.c.Hk) {
          const long long h = (u0 - u) / nb;
          start_r = r;
          start_t = t;
          start_h = (int)h;
          start_s[0] = u + h * nb;  // first block of the tile
          found = true;
        } else {
          u += nb * a.c.Hk;
        }
      }
    }
  }
  __syncthreads();
  const int cache_r0 = start_r;
  for (int i = tid; i < kReqCache; i += kThreads)
    if (cache_r0 + i < a.R) reqs[i] = load_req(a, cache_r0 + i);
  __syncthreads();

  const WaitCtx wc{&abort_s, a.rep.st, a.rep.epoch, a.rep.wait_ns};
  const int page_log = a.c.page_log - 4;  // blocks of a page, log2

  // ---- producer state of this warp: the tile its next copy belongs to, the block of
  // it, and the pages of its next 32 blocks (one per lane)
  Walk<ROWS> pw;
  pw.at(a, reqs, cache_r0, start_r, start_t, start_h);
  Walk<ROWS> cw = pw;
  long long p_tile0 = start_s[0];  // first block of the producer's tile, as a unit
  int p_b = (int)(u0 - p_tile0) + warp;
  int ids = -1, ids_r = -1, ids_b = 0;  // ... of request ids_r, from block ids_b on
  uint32_t bad = 0;  // stages whose page is outside the cache
  bool p_done = false;
  auto refill = [&]() {  // pages of blocks p_b + 4 i (i < 32) of the producer's tile
    const int b = p_b + lane * kWarps;
    const int pg = (pw.y.b0 + b) >> page_log;
    ids = pg < a.table_width ? __ldg(a.table + pw.r * a.table_stride + pg) : -1;
    ids_r = pw.r;
    ids_b = pw.y.b0 + p_b;
  };
  auto produce = [&](int stage) {  // the copy of this warp's next block, if any is left
    while (!p_done && (p_b >= pw.y.nb || p_tile0 + p_b >= u1)) {
      if (p_tile0 + pw.y.nb >= u1) {
        p_done = true;
        break;
      }
      p_tile0 += pw.y.nb;
      pw.next(a, reqs, cache_r0);
      p_b = warp;
    }
    if (p_done) return;
    const int ab = pw.y.b0 + p_b, i = (ab - ids_b) / kWarps;
    if (ids_r != pw.r || ab < ids_b || i >= 32 || (ab - ids_b) % kWarps != 0) refill();
    const int id = __shfl_sync(0xffffffffu, ids, (ab - ids_b) / kWarps);
    const bool ok = (unsigned)id < (unsigned)a.c.num_pages && pw.y.k1 > pw.y.k0;
    bad = (bad & ~(1u << stage)) | ((ok ? 0u : 1u) << stage);
    if (lane == 0) {
      const uint32_t bar = smem_addr(&bars[warp][stage]);
      if (ok) {
        const uint8_t* src = a.c.data + id * a.c.page_stride +
                             (((long long)pw.h << page_log) + (ab & ((1 << page_log) - 1))) * Blk::bytes;
        mbar_arrive_expect_tx(bar, Blk::bytes);
        bulk_load(ring + stage * Blk::bytes, src, Blk::bytes, bar);
      } else {
        if (pw.y.k1 > pw.y.k0) atomicCAS(&a.rep.st->code, 0, (int)FA_ERR_INDEX);
        mbar_arrive(bar);
      }
    }
    p_b += kWarps;
  };
#pragma unroll 1
  for (int s = 0; s < S; ++s) produce(s);

  // ---- the share's tiles
  int it = 0;  // blocks this warp has taken
  int4 meta = make_int4(-1, 0, 0, 0);
  long long tile0 = start_s[0];
  while (tile0 < u1) {
    const Tile y = cw.y;
    const Req x = cw.x;
    const int first = (int)max(0ll, u0 - tile0), last = (int)min((long long)y.nb, u1 - tile0);
    // query rows: column n = g + 8 j of the tile's rows, this lane's channels, as B fragments.
    // Each row is brought to a largest magnitude in [1, 2) by a power of two (exact),
    // which its score factor takes back: no 16-bit query leaves fp16's range.
    uint32_t qf[NT == 4 ? 1 : NT][KS][2];
    float factor[NT][2];
    int lim[NT][2], low[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int n = g + 8 * j;
      uint4 raw[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) raw[i] = make_uint4(0, 0, 0, 0);
      if (n < y.rows) {
        const int row = y.row0 + n, qi = row / a.G;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(a.q) + (x.q0 + qi) * a.qs[0] +
            ((long long)cw.h * a.G + row % a.G) * a.qs[1] + t4 * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) raw[i] = __ldg(src + i);
      }
      float big = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
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
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 v = unpack2<F16>(w[k]);
          f[2 * k] = v.x * down;
          f[2 * k + 1] = v.y * down;
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t v = pack2<true>(f[p], f[p + 4]);
          if constexpr (NT == 4) {
            if (warp == j) reinterpret_cast<uint32_t*>(qfrag)[((j * KS + 2 * i + (p >> 1)) * 32 + lane) * 2 + (p & 1)] = v;
          } else {
            qf[j][2 * i + (p >> 1)][p & 1] = v;
          }
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float u = __shfl_sync(0xffffffffu, up, 4 * (2 * t4 + c));
        factor[j][c] = u * a.scale_log2;
        const int row = y.row0 + 8 * j + 2 * t4 + c;
        const int pos = x.kv - x.n + row / a.G;  // rows behind the last: of no consequence
        lim[j][c] = min(pos + 1, x.kv);
        low[j][c] = a.window > 0 ? pos - a.window + 1 : 0;
      }
    }
    if constexpr (NT == 4) __syncthreads();
    // tokens that every row sees: no comparisons in their blocks
    const int i0 = y.row0 / a.G, i1 = (y.row0 + y.rows - 1) / a.G;
    const int all_hi = x.kv - x.n + i0 + 1;
    const int all_lo = a.window > 0 ? x.kv - x.n + i1 - a.window + 1 : 0;

    float m[NT][2], l[NT][2], o[MT][NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      m[j][0] = m[j][1] = kNoMax;
      l[j][0] = l[j][1] = 0.f;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][j][c] = 0.f;
    }

#pragma unroll 1
    for (int b = first + warp; b < last; b += kWarps) {
      const int stage = it % S;
      const uint32_t parity = (uint32_t)(it / S) & 1u;
      // a wait that gave up has recorded it; the copy must still land before the stage is left
      if (!warp_wait(wc, smem_addr(&bars[warp][stage]), parity)) mbar_drain(wc, smem_addr(&bars[warp][stage]), parity);
      const uint32_t kb = ring + stage * Blk::bytes, vb = kb + Blk::half;
      const int key0 = (y.b0 + b) * kKvBlock;
      const int kr = g ^ ((g >> 1) & 1);  // token of fragment row g (and kr + 8 of row g + 8)
      const bool hidden = (bad >> stage) & 1u;
      const bool masked = hidden || key0 + kKvBlock > all_hi || key0 < all_lo;
      uint32_t nan_keys = 0;
      if (masked) {
        // values that no row sees must not reach the product (0 x NaN), nor a NaN that only
        // some rows see: their pairs become 0, and a NaN one marks its token's scores
        for (int e = lane; e < kKvBlock * Blk::groups; e += 32) {
          const int key = e / Blk::groups;
          const uint32_t at = vb + Blk::codes + e * 4, pair = lds32(at);
          const bool seen = !hidden && key0 + key >= y.k0 && key0 + key < y.k1;
          const __half2 h = *reinterpret_cast<const __half2*>(&pair);
          const bool nan = __hisnan(__low2half(h)) || __hisnan(__high2half(h));
          if (!seen || nan) asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(0) : "memory");
          if (seen && nan) nan_keys |= 1u << key;
        }
        nan_keys = __reduce_or_sync(0xffffffffu, nan_keys);
        __syncwarp();
        fence_async_smem();  // these stores before the copy that reuses the stage
      }

      // S^T
      float s[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[j][c] = 0.f;
      {
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
          const uint32_t a0 = hfma2(code_pair<0>(wa[i]), sa, ca), a1 = hfma2(code_pair<0>(wb[i]), sb, cb);
          const uint32_t a2 = hfma2(code_pair<1>(wa[i]), sa, ca), a3 = hfma2(code_pair<1>(wb[i]), sb, cb);
          const uint32_t c0 = hfma2(code_pair<2>(wa[i]), sa, ca), c1 = hfma2(code_pair<2>(wb[i]), sb, cb);
          const uint32_t c2 = hfma2(code_pair<3>(wa[i]), sa, ca), c3 = hfma2(code_pair<3>(wb[i]), sb, cb);
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
      // scores in log2 units; hidden tokens
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[j][c] *= factor[j][c & 1];
      if (masked) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = kr + (c >= 2 ? 8 : 0);
            const bool seen = !hidden && key0 + key < lim[j][c & 1] && key0 + key >= low[j][c & 1];
            s[j][c] = !seen ? -INFINITY : (nan_keys >> key) & 1u ? NAN : s[j][c];
          }
      }
      // the running maximum, moved when a score is above it by more than 2^8
      bool grow = false;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) grow |= s[j][c] > m[j][c & 1] + 8.f;
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = fmaxf(s[j][c], s[j][c + 2]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            top = fmaxf(top, m[j][c]);
            const float back = ex2(m[j][c] - top);
            m[j][c] = top;
            l[j][c] *= back;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[i][j][c] *= back;
              o[i][j][c + 2] *= back;
            }
          }
      }
      // weights, and their transpose as the B operand
      uint32_t p0[NT], p1[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int c = 0; c < 4; ++c) s[j][c] = ex2(s[j][c] - m[j][c & 1]);
        l[j][0] += s[j][0] + s[j][2];
        l[j][1] += s[j][1] + s[j][3];
        p0[j] = transpose8x8(pack2<true>(s[j][0], s[j][1]));
        p1[j] = transpose8x8(pack2<true>(s[j][2], s[j][3]));
      }
      // O^T += V^T P^T: this lane's tokens are those of fragment rows 2 t, 2 t + 1 and 8 more
      {
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
          product(4 * i + 0, code_pair<0>(xl), code_pair<0>(xh), code_pair<0>(yl), code_pair<0>(yh));
          product(4 * i + 1, code_pair<1>(xl), code_pair<1>(xh), code_pair<1>(yl), code_pair<1>(yh));
          product(4 * i + 2, code_pair<2>(xl), code_pair<2>(xh), code_pair<2>(yl), code_pair<2>(yh));
          product(4 * i + 3, code_pair<3>(xl), code_pair<3>(xh), code_pair<3>(yl), code_pair<3>(yh));
        }
      }
      __syncwarp();  // every lane has read the stage
      produce(stage);
      ++it;
    }

    // ---- join the warps that took blocks of the tile
    const int active = min(kWarps, last - first);
    if (warp < active) {
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
            m_s[warp][row] = m[j][c];
            l_s[warp][row] = v;
          }
          float* to = joined + (warp * ROWS + row) * C::LDO + g * (D / 8);
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            *reinterpret_cast<float4*>(to + 8 * i) =
                make_float4(o[4 * i][j][c], o[4 * i + 1][j][c], o[4 * i + 2][j][c], o[4 * i + 3][j][c]);
            *reinterpret_cast<float4*>(to + 8 * i + 4) =
                make_float4(o[4 * i][j][c + 2], o[4 * i + 1][j][c + 2], o[4 * i + 2][j][c + 2], o[4 * i + 3][j][c + 2]);
          }
        }
      }
    }
    __syncthreads();
    const bool from_before = first > 0, goes_on = tile0 + y.nb > u1;
    constexpr int TPR = D / 8;  // threads per row, 8 channels each
    for (int e = tid; e < ROWS * TPR; e += kThreads) {
      const int row = e / TPR, ch = (e % TPR) * 8;
      if (row >= y.rows) continue;
      float top = m_s[0][row];
      for (int w = 1; w < active; ++w) top = fmaxf(top, m_s[w][row]);
      float sum = 0.f, acc[8] = {};
      for (int w = 0; w < active; ++w) {
        const float f = ex2(m_s[w][row] - top);
        sum = fmaf(f, l_s[w][row], sum);
        const float4* src = reinterpret_cast<const float4*>(joined + (w * ROWS + row) * C::LDO + ch);
        const float4 u = src[0], v = src[1];
        acc[0] = fmaf(f, u.x, acc[0]); acc[1] = fmaf(f, u.y, acc[1]);
        acc[2] = fmaf(f, u.z, acc[2]); acc[3] = fmaf(f, u.w, acc[3]);
        acc[4] = fmaf(f, v.x, acc[4]); acc[5] = fmaf(f, v.y, acc[5]);
        acc[6] = fmaf(f, v.z, acc[6]); acc[7] = fmaf(f, v.w, acc[7]);
      }
      if (from_before || goes_on) {
        float* to = a.part + ((size_t)(2 * blockIdx.x + (from_before ? 0 : 1)) * ROWS + row) * (D + 4);
        *reinterpret_cast<float4*>(to + 4 + ch) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        *reinterpret_cast<float4*>(to + 8 + ch) = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (ch == 0) {
          to[0] = top;
          to[1] = sum;
        }
      } else {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int gr = y.row0 + row, qi = gr / a.G;
        const long long head = (long long)cw.h * a.G + gr % a.G;
        uint16_t* to = static_cast<uint16_t*>(a.o) + (x.q0 + qi) * a.os[0] + head * a.os[1] + ch;
        if (fa_bounds(a.rep.st, x.q0 + qi < a.T && head < a.Hq)) {
          *reinterpret_cast<uint4*>(to) =
              make_uint4(pack2<F16>(acc[0] * inv, acc[1] * inv), pack2<F16>(acc[2] * inv, acc[3] * inv),
                         pack2<F16>(acc[4] * inv, acc[5] * inv), pack2<F16>(acc[6] * inv, acc[7] * inv));
          if (ch == 0 && a.lse)
            a.lse[(long long)(x.q0 + qi) * a.Hq + head] =
                sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
        }
      }
    }
    if (goes_on && !from_before) {
      const long long tile_end = tile0 + y.nb;
      meta = make_int4(cw.r, cw.t, cw.h, (int)((tile_end - 1) / share));
    }
    __syncthreads();  // joined, m_s, l_s read
    tile0 += y.nb;
    if (tile0 < u1) cw.next(a, reqs, cache_r0);
  }
  if (tid == 0) a.meta[blockIdx.x] = meta;
}

// Adds the shares of the tile that starts in share blockIdx.x and goes on, if any.
// One warp per row: the row's slots are read with 4 (d = 128) or 2 channels per lane.
template <int D, int NT, bool F16>
__global__ void __launch_bounds__(256) kv4_merge_kernel(const Kv4AttnArgs a) {
  constexpr int ROWS = 8 * NT, CPL = D / 32;
  const int4 meta = a.meta[blockIdx.x];
  if (meta.x < 0) return;
  const Req x = load_req(a, meta.x);
  const Tile y = tile_of<ROWS>(a, x, meta.y);
  const int lane = threadIdx.x & 31;
  const int c0 = blockIdx.x;
  for (int row = threadIdx.x >> 5; row < y.rows; row += 8) {
    auto slot = [&](int c) {  // the first share's slot is its second one
      return a.part + ((size_t)(2 * c + (c == c0 ? 1 : 0)) * ROWS + row) * (D + 4);
    };
    float top = kNoMax;
    for (int c = c0 + lane; c <= meta.w; c += 32) top = fmaxf(top, slot(c)[0]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    float sum = 0.f, acc[CPL] = {};
#pragma unroll 4
    for (int c = c0; c <= meta.w; ++c) {
      const float* s = slot(c);
      const float f = ex2(s[0] - top);
      sum = fmaf(f, s[1], sum);
#pragma unroll
      for (int i = 0; i < CPL; ++i) acc[i] = fmaf(f, s[4 + lane * CPL + i], acc[i]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int gr = y.row0 + row, qi = gr / a.G;
    const long long head = (long long)meta.z * a.G + gr % a.G;
    if (!fa_bounds(a.rep.st, x.q0 + qi < a.T && head < a.Hq)) continue;
    uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + (x.q0 + qi) * a.os[0] +
                                               head * a.os[1] + lane * CPL);
#pragma unroll
    for (int i = 0; i < CPL / 2; ++i) to[i] = pack2<F16>(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    if (lane == 0 && a.lse)
      a.lse[(long long)(x.q0 + qi) * a.Hq + head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
  }
}

template <int D, int NT, bool F16>
cudaError_t launch(const Kv4AttnArgs& a, int ctas, cudaStream_t s) {
  using C = Cfg<D, NT>;
  cudaError_t e = cudaFuncSetAttribute(kv4_attn_kernel<D, NT, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
  if (e != cudaSuccess) return e;
  kv4_attn_kernel<D, NT, F16><<<ctas, kThreads, C::smem, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  kv4_merge_kernel<D, NT, F16><<<ctas, 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <int D, bool F16>
cudaError_t launch_rows(const Kv4AttnArgs& a, int rows, int ctas, cudaStream_t s) {
  return rows == 8 ? launch<D, 1, F16>(a, ctas, s) : rows == 16 ? launch<D, 2, F16>(a, ctas, s) : launch<D, 4, F16>(a, ctas, s);
}

}  // namespace

int kv4_tile_rows(int G, int max_q_len) {
  const long long rows = (long long)G * max_q_len;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
}

int kv4_max_ctas(int d, int rows, int sms) {
  (void)d;
  return sms * (rows == 8 ? Cfg<128, 1>::CTAS_PER_SM : rows == 16 ? Cfg<128, 2>::CTAS_PER_SM : Cfg<128, 4>::CTAS_PER_SM);
}

cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, int d, bool f16, int rows, int ctas, cudaStream_t s) {
  if (d == 64) return f16 ? launch_rows<64, true>(a, rows, ctas, s) : launch_rows<64, false>(a, rows, ctas, s);
  return f16 ? launch_rows<128, true>(a, rows, ctas, s) : launch_rows<128, false>(a, rows, ctas, s);
}

}  // namespace fa
