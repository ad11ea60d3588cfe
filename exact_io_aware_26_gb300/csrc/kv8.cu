// kv8.cu -- writing tokens' keys and values into the 8-bit cache, and reading them back.
//
// A block of 16 tokens of a head has one scale for its keys and one for its values: the least
// power of two that brings the largest magnitude among them to 127.  Powers of two make every
// step exact but the roundings to codes: a kernel, and anyone who follows the steps, gets
// the same codes.  Tokens that join a block may raise its scale; the codes that are there are
// then rounded to the new one, which happens a few times at most while a block fills.
#include <algorithm>

#include "kv8.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256, kAppend = 128, kWarps = kAppend / 32;

constexpr float kRound = 12582912.f;  // 1.5 * 2^23: a number added to it is rounded to a whole one, its low byte the code

// Four neighbouring channels as they are in memory, their largest magnitude (as the bits of an
// fp32 number: a NaN is above all others), and their values.
template <int DT>
struct Quad {
  uint2 w;
  __device__ __forceinline__ void zero() { w = make_uint2(0u, 0u); }
  __device__ __forceinline__ void load(const void* base, long long at) {
    w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at));
  }
  __device__ __forceinline__ uint32_t most(uint32_t so_far) const {  // halves, joined by widest()
    return __vmaxu2(so_far, __vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu));
  }
  static __device__ __forceinline__ uint32_t widest(uint32_t m) {
    const float2 f = unpack2<DT == FA_F16>(m);
    return max(__float_as_uint(f.x), __float_as_uint(f.y));
  }
  __device__ __forceinline__ float4 values() const {
    const float2 a = unpack2<DT == FA_F16>(w.x), b = unpack2<DT == FA_F16>(w.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
};
template <>
struct Quad<FA_F32> {
  float4 v;
  __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const void* base, long long at) {
    v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + at));
  }
  __device__ __forceinline__ uint32_t most(uint32_t so_far) const {
    auto mag = [](float f) { return __float_as_uint(f) & 0x7FFFFFFFu; };
    return max(max(so_far, mag(v.x)), max(max(mag(v.y), mag(v.z)), mag(v.w)));
  }
  static __device__ __forceinline__ uint32_t widest(uint32_t m) { return m; }
  __device__ __forceinline__ float4 values() const { return v; }
};
template <int DT>
__device__ __forceinline__ void store4(void* base, long long at, const float4& v) {
  if constexpr (DT == FA_F32)
    *reinterpret_cast<float4*>(static_cast<float*>(base) + at) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + at) =
        make_uint2(pack2<DT == FA_F16>(v.x, v.y), pack2<DT == FA_F16>(v.z, v.w));
}

// The first byte of block `blk` (slot / 16) of a head; nullptr for one outside the cache.
__device__ __forceinline__ uint8_t* block_at(const Kv4Cache& c, int blk, int head, int bytes) {
  const int page = blk >> (c.page_log - 4);
  if (page >= c.num_pages) return nullptr;
  return const_cast<uint8_t*>(c.data) + page * c.page_stride +
         (long long)((head << (c.page_log - 4)) + (blk & ((1 << (c.page_log - 4)) - 1))) * bytes;
}

// The least power of two that brings magnitudes of up to `most` to 127: most = m 2^e with m in [1, 2),
// 127 2^x >= most from x = e - 6 on where m <= 127 / 64.  0 for 0.
__device__ __forceinline__ float scale_for(float most) {
  const uint32_t b = __float_as_uint(most);
  int e = (int)(b >> 23) - 127 - ((b & 0x7FFFFFu) <= 0x7E0000u ? 6 : 5);
  e = max(e, kKv8LeastExp);
  return most > 0.f ? __uint_as_float((uint32_t)(e + 127) << 23) : 0.f;
}

// Of a power of two; 0 for 0.
__device__ __forceinline__ float reciprocal(float scale) {
  return scale > 0.f ? __uint_as_float(0x7F000000u - __float_as_uint(scale)) : 0.f;
}

// Codes of four values: rint(x * inv), |x * inv| <= 127; the product is exact for a power of two.
__device__ __forceinline__ uint32_t codes_of(const float4& x, float inv) {
  const uint64_t inv2 = f2pack(inv, inv), up2 = f2pack(kRound, kRound);
  float a, b, c, d;
  f2unpack(ffma2(f2pack(x.x, x.y), inv2, up2), a, b);
  f2unpack(ffma2(f2pack(x.z, x.w), inv2, up2), c, d);
  return __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040),
                     __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040), 0x5410);
}
// A word's four codes times `ratio`, rounded.
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float ratio) {
  return codes_of(make_float4((float)(int8_t)w, (float)(int8_t)(w >> 8), (float)(int8_t)(w >> 16), (float)(int8_t)(w >> 24)), ratio);
}
// The words of four channels by four tokens, from words of four tokens by four channels.
__device__ __forceinline__ uint4 turned(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t ab = __byte_perm(a, b, 0x5140), cd = __byte_perm(c, d, 0x5140);  // a0 b0 a1 b1
  const uint32_t AB = __byte_perm(a, b, 0x7362), CD = __byte_perm(c, d, 0x7362);  // a2 b2 a3 b3
  return make_uint4(__byte_perm(ab, cd, 0x5410), __byte_perm(ab, cd, 0x7632), __byte_perm(AB, CD, 0x5410),
                    __byte_perm(AB, CD, 0x7632));
}

// A side's scale and marks of a block, written by one lane.
__device__ __forceinline__ void set_tail(uint8_t* tail_at, int side, float scale, uint32_t marks, bool fresh) {
  Kv8Tail* tail = reinterpret_cast<Kv8Tail*>(tail_at);
  if (side) {
    tail->vs = scale;
    tail->v_nan = (uint16_t)marks;
  } else {
    tail->ks = scale;
    tail->k_nan = (uint16_t)marks;
    if (fresh) tail->zero = 0u;
  }
}
__device__ __forceinline__ float saturated(float f, bool lost) { return lost ? 0.f : fminf(fmaxf(f, -kKvSaturate), kKvSaturate); }
__device__ __forceinline__ float4 saturated(const float4& v, bool lost) {
  return make_float4(saturated(v.x, lost), saturated(v.y, lost), saturated(v.z, lost), saturated(v.w, lost));
}
__device__ __forceinline__ bool has_nan(const float4& v) { return v.x != v.x || v.y != v.y || v.z != v.z || v.w != v.w; }
__device__ __forceinline__ uint32_t most4(const float4& v) {
  return __float_as_uint(fmaxf(fmax3(fabsf(v.x), fabsf(v.y), fabsf(v.z)), fabsf(v.w)));
}

// 16 rows from x0 on into the places of a block, of one side of a head, by a warp; all of them in
// registers.  A lane has four channels of every place (d = 64: half of the warp each of two of
// the four groups of four places).
template <int D>
constexpr int kGroups = D == 128 ? 4 : 2;  // of a lane
template <int D>
__device__ __forceinline__ int lane_place(int p) {  // of a lane's p-th quad
  return D == 128 ? p : (p >> 2) * 8 + (threadIdx.x >> 4 & 1) * 4 + (p & 3);
}
template <int D, int DT>
__device__ __forceinline__ void load_whole(Quad<DT> (&x)[4 * kGroups<D>], const char* x0, long long row_bytes) {
  const int l = threadIdx.x % (D / 4);
#pragma unroll
  for (int p = 0; p < 4 * kGroups<D>; ++p) x[p].load(x0 + lane_place<D>(p) * row_bytes, 4 * l);
}
template <int D, int DT>
__device__ __forceinline__ void append_whole(const Quad<DT> (&x)[4 * kGroups<D>], uint8_t* at, int side) {
  using Blk = Kv8Block<D>;
  constexpr int LPR = D / 4, GROUPS = kGroups<D>;  // lanes of a row
  const int lane = threadIdx.x & 31, l = lane % LPR, hw = lane / LPR;
  auto place = [](int p) { return lane_place<D>(p); };
  uint32_t bits = 0, nan = 0;
#pragma unroll
  for (int p = 0; p < 4 * GROUPS; ++p) bits = x[p].most(bits);
  bits = __reduce_max_sync(0xffffffffu, Quad<DT>::widest(bits));
  // values beyond the range, infinite or NaN among them: looked at one by one
  const bool odd = bits > __float_as_uint(kKvSaturate);
  if (odd) {
    bits = 0;
#pragma unroll
    for (int p = 0; p < 4 * GROUPS; ++p) {
      const bool mine = has_nan(x[p].values());
      const uint32_t half = D == 128 ? 0xffffffffu : 0xFFFFu << (16 * hw);
      const bool lost = (__ballot_sync(0xffffffffu, mine) & half) != 0u;
      if (lost) nan |= 1u << place(p);
      bits = max(bits, most4(saturated(x[p].values(), lost)));
    }
    bits = __reduce_max_sync(0xffffffffu, bits);
  }
  const float scale = scale_for(__uint_as_float(bits));
  const float inv = reciprocal(scale);
#pragma unroll
  for (int q = 0; q < GROUPS; ++q) {
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float4 v = x[4 * q + j].values();
      if (odd) v = saturated(v, nan >> place(4 * q + j) & 1u);
      c[j] = codes_of(v, inv);
    }
    if (side == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int o = place(4 * q + j);
        *reinterpret_cast<uint32_t*>(at + o * Blk::row + kv8_key_chunk<D>(j, l / 4) * 16 + (l % 4) * 4) = c[j];
      }
    } else {
      *reinterpret_cast<uint4*>(at + Blk::half + l * 64 + place(4 * q) * 4) = turned(c[0], c[1], c[2], c[3]);
    }
  }
  nan = __reduce_or_sync(0xffffffffu, nan);
  if (lane == 0) set_tail(at + Blk::tail, side, scale, nan, true);
}

// `run` rows, at most 16, into the places s % 16 of lanes 0 .. run - 1: a few at a time, read once for
// the scale and once more for the codes.
template <int D, int DT>
__device__ __forceinline__ void append_some(const char* x0, long long row_bytes, uint8_t* at, int side, int s, int run) {
  using Blk = Kv8Block<D>;
  constexpr int LPR = D / 4, HW = 32 / LPR, ROWS = 4;  // rows that a lane has at a time
  const int lane = threadIdx.x & 31, l = lane % LPR, hw = lane / LPR;
  const uint32_t written = __reduce_or_sync(0xffffffffu, lane < run ? 1u << (s & (kKvBlock - 1)) : 0u);
  const bool fresh = written & 1u;  // what was there is another request's
  float old = 0.f;
  uint32_t marks = 0;
  if (!fresh) {
    const uint4 u = *reinterpret_cast<const uint4*>(at + Blk::tail);
    old = __uint_as_float(side ? u.y : u.x);
    marks = (side ? u.z >> 16 : u.z & 0xFFFFu) & ~written;
  }
  Quad<DT> x[ROWS];
  auto fetch = [&](int j0) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int j = j0 + i * HW + hw;
      x[i].zero();
      if (j < run) x[i].load(x0 + j * row_bytes, 4 * l);
    }
  };
  uint32_t bits = 0;
#pragma unroll 1
  for (int j0 = 0; j0 < run; j0 += ROWS * HW) {
    fetch(j0);
    uint32_t some = 0;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) some = x[i].most(some);
    bits = max(bits, Quad<DT>::widest(some));
  }
  bits = __reduce_max_sync(0xffffffffu, bits);
  const uint32_t half = D == 128 ? 0xffffffffu : 0xFFFFu << (16 * hw);
  auto row_lost = [&](int i) { return (__ballot_sync(0xffffffffu, has_nan(x[i].values())) & half) != 0u; };
  const bool odd = bits > __float_as_uint(kKvSaturate);
  if (odd) {
    bits = 0;
#pragma unroll 1
    for (int j0 = 0; j0 < run; j0 += ROWS * HW) {
      if (run > ROWS * HW) fetch(j0);
#pragma unroll
      for (int i = 0; i < ROWS; ++i) bits = max(bits, most4(saturated(x[i].values(), row_lost(i))));
    }
    bits = __reduce_max_sync(0xffffffffu, bits);
  }
  const float scale = fmaxf(old, scale_for(__uint_as_float(bits)));
  const float inv = reciprocal(scale);
  if (old > 0.f && scale > old) {  // the codes that are there to the larger scale (those to be written, too)
    const float ratio = old * inv;
#pragma unroll 4
    for (int i = 0; i < kKvBlock / HW / 4; ++i) {
      uint4* to = reinterpret_cast<uint4*>(at + (side ? Blk::half : 0) + lane * 16 + i * 512);
      const uint4 u = *to;
      *to = make_uint4(rescaled(u.x, ratio), rescaled(u.y, ratio), rescaled(u.z, ratio), rescaled(u.w, ratio));
    }
    __syncwarp();
  }
#pragma unroll 1
  for (int j0 = 0; j0 < run; j0 += ROWS * HW) {
    if (run > ROWS * HW) fetch(j0);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int j = j0 + i * HW + hw, o = __shfl_sync(0xffffffffu, s, j & 31) & (kKvBlock - 1);
      bool lost = false;
      float4 v = x[i].values();
      if (odd) {
        lost = row_lost(i);
        v = saturated(v, lost);
      }
      if (j >= run) continue;
      if (lost) marks |= 1u << o;
      const uint32_t c = codes_of(v, inv);
      if (side == 0) {
        *reinterpret_cast<uint32_t*>(at + o * Blk::row + kv8_key_chunk<D>(o, l / 4) * 16 + (l % 4) * 4) = c;
      } else {
        uint8_t* to = at + Blk::half + l * 64 + o / 4 * 16 + o % 4;
#pragma unroll
        for (int k = 0; k < 4; ++k) to[4 * k] = (uint8_t)(c >> (8 * k));
      }
    }
  }
  marks = __reduce_or_sync(0xffffffffu, marks);
  if (lane == 0) set_tail(at + Blk::tail, side, scale, marks, fresh);
}

// A warp takes the blocks that begin (the first token of a run in one block) among `span` tokens,
// for one head and side; of long prompts with 64 16-bit channels for both sides, whose rows are on
// their way together (23,400 tokens of 12 heads: 20.3 us, one side a warp 28.8; with more bytes
// to a block it spills).
//
// Long prompts are bound by HBM and instructions (packed maxima of 16-bit values as they are, a
// packed fma that rounds, byte permutes), single tokens by a chain of loads: slots, then the tail and
// the row.  23,400 tokens of 12 heads, d = 64: bf16 20.3 us (108 MB, 5.3 TB/s), fp32 30.4 us (5.9);
// 16384 tokens of 8 heads, d = 128: fp16 18.0 us (5.6 TB/s); 256 single tokens of 8 heads 3.2 us.
template <int D, int DT>
constexpr bool kBoth = D == 64 && DT != FA_F32;
template <int D, int DT>
__global__ void __launch_bounds__(kAppend, D == 128 && DT == FA_F32 ? 4 : 8)
    kv8_append_kernel(const Kv4RowArgs a, int tokens, int span, int sides) {
  using Blk = Kv8Block<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = blockIdx.x * kWarps + warp, side0 = sides == 2 ? 0 : w & 1, row = sides == 2 ? w : w >> 1;
  const int chunk = a.heads.div(row), head = row - chunk * (int)a.heads.d;
  const int t0 = chunk * span;
  if (t0 >= tokens) return;  // the whole warp
  constexpr int E = DT == FA_F32 ? 4 : 2;
  long long row_bytes[2];
  const char* x0[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    row_bytes[i] = (long long)a.xs[i][0] * E;
    x0[i] = static_cast<const char*>(a.x[i]) + (long long)head * a.xs[i][1] * E;
  }
  // lane i has the slot of token t0 - 1 + i: those of the span, of the one before and of the runs' ends
  const int mine = t0 - 1 + lane;
  const int own = mine >= 0 && mine < tokens ? __ldg(a.slots + mine) : -1;
  const int before = __shfl_up_sync(0xffffffffu, own, 1);
  const bool leads = lane >= 1 && lane <= span && own >= 0 && !(before >= 0 && before / kKvBlock == own / kKvBlock);
  uint32_t rest = __ballot_sync(0xffffffffu, leads);
  while (rest) {
    const int lead = __ffs((int)rest) - 1, first = t0 - 1 + lead;
    rest &= rest - 1;
    // lane j gets the slot of the run's j-th token
    const int there = __shfl_sync(0xffffffffu, own, (lead + lane) & 31);
    const int s = lane < kKvBlock ? there : -1;
    const int blk = __shfl_sync(0xffffffffu, s, 0) / kKvBlock;
    uint8_t* at = block_at(a.c, blk, head, Blk::bytes);
    if (!at) {
      if (lane == 0) atomicCAS(&a.st->code, 0, (int)FA_ERR_INDEX);
      continue;
    }
    if (__all_sync(0xffffffffu, lane >= kKvBlock || s == blk * kKvBlock + lane)) {  // a whole block, in order
      Quad<DT> x[4 * kGroups<D>];
      load_whole<D, DT>(x, x0[side0] + first * row_bytes[side0], row_bytes[side0]);
      if (kBoth<D, DT> && sides == 2) {
        Quad<DT> y[4 * kGroups<D>];
        load_whole<D, DT>(y, x0[1] + first * row_bytes[1], row_bytes[1]);
        append_whole<D, DT>(x, at, 0);
        append_whole<D, DT>(y, at, 1);
      } else {
        append_whole<D, DT>(x, at, side0);
      }
    } else {
      const uint32_t same = __ballot_sync(0xffffffffu, s >= 0 && s / kKvBlock == blk);
      const int run = __ffs((int)~same) - 1;  // at most 16: the other lanes' slots are -1
#pragma unroll 1
      for (int side = side0; side < side0 + sides; ++side)
        append_some<D, DT>(x0[side] + first * row_bytes[side], row_bytes[side], at, side, s, run);
    }
  }
}

// Four codes times a scale: 2^23 + (code + 128) is the fp32 number 0x4B000000 | (code + 128).
__device__ __forceinline__ float4 values_of(uint32_t w, float scale) {
  const uint32_t u = w ^ 0x80808080u;
  auto one = [&](int sel) { return __uint_as_float(__byte_perm(u, 0x4B000000u, sel)); };
  const uint64_t off = f2pack(-8388736.f, -8388736.f), s = f2pack(scale, scale);
  float4 v;
  f2unpack(fmul2(fadd2(f2pack(one(0x7440), one(0x7441)), off), s), v.x, v.y);
  f2unpack(fmul2(fadd2(f2pack(one(0x7442), one(0x7443)), off), s), v.z, v.w);
  return v;
}

// A thread reads four channels of four tokens that stand one behind the other in the call.  Where
// these are a block's places 4 n to 4 n + 3 in order (prompts), one cell has their values; others
// are read one by one.  Groups of four tokens run along a block of a head, then its heads.  Bound by HBM:
// 23,400 tokens of 12 heads, d = 64, bf16: 15.5 us (108 MB, 7 TB/s, of which the cache's 36 MB mostly
// from L2; a token a thread 27.7 us).
constexpr int kGather = 4;
template <int D, int DT>
__global__ void __launch_bounds__(kThreads, 6) kv8_gather_kernel(const Kv4RowArgs a, int tokens) {
  using Blk = Kv8Block<D>;
  constexpr int LPR = D / 4, ROWS = kThreads / LPR, QUADS = kKvBlock / kGather;
  const int l = threadIdx.x % LPR;
  const long long r = (long long)blockIdx.x * ROWS + threadIdx.x / LPR;
  const int unit = (int)(r / QUADS), group = a.heads.div(unit), head = unit - group * (int)a.heads.d;
  const int tok = group * kKvBlock + (int)(r % QUADS) * kGather;
  if (tok >= tokens) return;
  int slot[kGather];
#pragma unroll
  for (int i = 0; i < kGather; ++i) slot[i] = tok + i < tokens ? __ldg(a.slots + tok + i) : -1;
  const long long to_k = (long long)tok * a.xs[0][0] + (long long)head * a.xs[0][1] + 4 * l;
  const long long to_v = (long long)tok * a.xs[1][0] + (long long)head * a.xs[1][1] + 4 * l;
  const uint8_t* at = slot[0] >= 0 ? block_at(a.c, slot[0] / kKvBlock, head, Blk::bytes) : nullptr;
  auto key = [&](const uint8_t* b, int o) {
    return __ldg(reinterpret_cast<const uint32_t*>(b + o * Blk::row + kv8_key_chunk<D>(o, l / 4) * 16 + (l % 4) * 4));
  };
  if (at && slot[0] % kGather == 0 && slot[1] == slot[0] + 1 && slot[2] == slot[0] + 2 && slot[3] == slot[0] + 3) {
    const int o = slot[0] % kKvBlock;
    uint32_t kw[kGather];
#pragma unroll
    for (int i = 0; i < kGather; ++i) kw[i] = key(at, o + i);
    const uint4 cell = __ldg(reinterpret_cast<const uint4*>(at + Blk::half + l * 64 + o * 4));
    const uint4 tail = __ldg(reinterpret_cast<const uint4*>(at + Blk::tail));
    const uint4 rows = turned(cell.x, cell.y, cell.z, cell.w);
    const uint32_t vw[kGather] = {rows.x, rows.y, rows.z, rows.w};
#pragma unroll
    for (int i = 0; i < kGather; ++i) {
      store4<DT>(a.x[0], to_k + (long long)i * a.xs[0][0], values_of(kw[i], tail.z >> (o + i) & 1u ? NAN : __uint_as_float(tail.x)));
      store4<DT>(a.x[1], to_v + (long long)i * a.xs[1][0],
                 values_of(vw[i], tail.z >> (16 + o + i) & 1u ? NAN : __uint_as_float(tail.y)));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kGather; ++i) {
    if (tok + i >= tokens) return;
    const int s = slot[i], o = s & (kKvBlock - 1);
    uint32_t kw = 0, vw = 0;
    float ks = 0.f, vs = 0.f;
    if (s >= 0) {
      at = block_at(a.c, s / kKvBlock, head, Blk::bytes);
      if (at) {
        kw = key(at, o);
        const uint4 cell = __ldg(reinterpret_cast<const uint4*>(at + Blk::half + l * 64 + (o / 4) * 16));
        const uint4 tail = __ldg(reinterpret_cast<const uint4*>(at + Blk::tail));
        const int sel = o % 4 * 0x11 + 0x40;  // the token's byte of two words
        vw = __byte_perm(__byte_perm(cell.x, cell.y, sel), __byte_perm(cell.z, cell.w, sel), 0x5410);
        ks = tail.z >> o & 1u ? NAN : __uint_as_float(tail.x);
        vs = tail.z >> (16 + o) & 1u ? NAN : __uint_as_float(tail.y);
      } else {
        atomicCAS(&a.st->code, 0, (int)FA_ERR_INDEX);
      }
    }
    store4<DT>(a.x[0], to_k + (long long)i * a.xs[0][0], values_of(kw, ks));
    store4<DT>(a.x[1], to_v + (long long)i * a.xs[1][0], values_of(vw, vs));
  }
}

template <int D, int DT>
cudaError_t launch(const Kv4RowArgs& a, bool gather, int sms, cudaStream_t s) {
  const int heads = (int)a.heads.d, tokens = a.rows / heads;
  if (gather) {
    const long long rows = (long long)(tokens + kKvBlock - 1) / kKvBlock * (kKvBlock / kGather) * heads, per = kThreads / (D / 4);
    kv8_gather_kernel<D, DT><<<(unsigned)((rows + per - 1) / per), kThreads, 0, s>>>(a, tokens);
  } else {
    // a token and side a warp where that gives the GPU no more than a few warps for each scheduler
    const long long most = (long long)sms * 64, span = std::min((long long)kKvBlock, std::max(1ll, 2ll * a.rows / most));
    const int sides = kBoth<D, DT> && span == kKvBlock ? 2 : 1;
    const long long warps = (3 - sides) * ((tokens + span - 1) / span) * heads;
    kv8_append_kernel<D, DT><<<(unsigned)((warps + kWarps - 1) / kWarps), kAppend, 0, s>>>(a, tokens, (int)span, sides);
  }
  return cudaGetLastError();
}

cudaError_t launch_any(const Kv4RowArgs& a, int d, int dtype, bool gather, int sms, cudaStream_t s) {
  if (d == 64)
    return dtype == FA_F32   ? launch<64, FA_F32>(a, gather, sms, s)
           : dtype == FA_F16 ? launch<64, FA_F16>(a, gather, sms, s)
                             : launch<64, FA_BF16>(a, gather, sms, s);
  return dtype == FA_F32   ? launch<128, FA_F32>(a, gather, sms, s)
         : dtype == FA_F16 ? launch<128, FA_F16>(a, gather, sms, s)
                           : launch<128, FA_BF16>(a, gather, sms, s);
}

}  // namespace

cudaError_t launch_kv8_append(const Kv4RowArgs& a, int d, int dtype, int sms, cudaStream_t s) {
  return launch_any(a, d, dtype, false, sms, s);
}
cudaError_t launch_kv8_gather(const Kv4RowArgs& a, int d, int dtype, cudaStream_t s) {
  return launch_any(a, d, dtype, true, 0, s);
}

}  // namespace fa
