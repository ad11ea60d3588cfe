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

constexpr int kThreads = 256, kWarps = kThreads / 32;

// Four neighbouring channels.
template <int DT>
__device__ __forceinline__ float4 load4(const void* base, long long at) {
  if constexpr (DT == FA_F32) {
    return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + at));
  } else {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at));
    const float2 a = unpack2<DT == FA_F16>(u.x), b = unpack2<DT == FA_F16>(u.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
}
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

__device__ __forceinline__ uint32_t code_of(float x, float inv) { return (uint32_t)__float2int_rn(x * inv) & 0xFFu; }
// A word's four codes times `ratio`, rounded.
__device__ __forceinline__ uint32_t rescaled(uint32_t w, float ratio) {
  uint32_t y = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) y |= code_of((float)(int8_t)(w >> (8 * k)), ratio) << (8 * k);
  return y;
}

// A warp takes the blocks that begin (the first token of a run in one block) among `span` tokens,
// for one head and side.  A lane has four channels of every place of the block (d = 64: half of
// the warp each of two of the four places' groups).
template <int D, int DT>
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(const Kv4RowArgs a, int tokens, int span) {
  using Blk = Kv8Block<D>;
  constexpr int LPR = D / 4, GROUPS = D == 128 ? 4 : 2;  // lanes of a row; groups of four places of a lane
  __shared__ int map_s[kWarps][kKvBlock];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % LPR, hw = lane / LPR;
  const int w = blockIdx.x * kWarps + warp, side = w & 1, row = w >> 1;
  const int chunk = a.heads.div(row), head = row - chunk * (int)a.heads.d;
  const int t0 = chunk * span;
  if (t0 >= tokens) return;  // the whole warp
  int* map = map_s[warp];
  // which of the span's tokens begin a run
  const int mine = t0 + lane;
  bool leads = false;
  if (lane < span && mine < tokens) {
    const int s = __ldg(a.slots + mine), before = mine > 0 ? __ldg(a.slots + mine - 1) : -1;
    leads = s >= 0 && !(before >= 0 && before / kKvBlock == s / kKvBlock);
  }
  uint32_t rest = __ballot_sync(0xffffffffu, leads);
  while (rest) {
    const int first = t0 + __ffs((int)rest) - 1;
    rest &= rest - 1;
    // the run: its places, and which token each gets
    const int s = lane < kKvBlock && first + lane < tokens ? __ldg(a.slots + first + lane) : -1;
    const int blk = __shfl_sync(0xffffffffu, s, 0) / kKvBlock;
    const uint32_t same = __ballot_sync(0xffffffffu, s >= 0 && s / kKvBlock == blk);
    const int run = __ffs((int)~same) - 1;  // at most 16: the other lanes' slots are -1
    if (lane < kKvBlock) map[lane] = -1;
    __syncwarp();
    if (lane < run) map[s % kKvBlock] = lane;
    __syncwarp();
    const uint32_t written = __ballot_sync(0xffffffffu, lane < kKvBlock && map[lane] >= 0);
    uint8_t* at = block_at(a.c, blk, head, Blk::bytes);
    if (!at) {
      if (lane == 0) atomicCAS(&a.st->code, 0, (int)FA_ERR_INDEX);
      __syncwarp();
      continue;
    }
    Kv8Tail* tail = reinterpret_cast<Kv8Tail*>(at + Blk::tail);
    const bool fresh = written & 1u;  // what was there is another request's
    const float old = fresh ? 0.f : side ? tail->vs : tail->ks;
    const uint32_t old_nan = fresh ? 0u : side ? tail->v_nan : tail->k_nan;
    float4 x[4 * GROUPS];
    float most = 0.f;
    uint32_t nan = 0;
#pragma unroll
    for (int p = 0; p < 4 * GROUPS; ++p) {
      const int o = D == 128 ? p : (p >> 2) * 8 + hw * 4 + (p & 3), j = map[o];
      x[p] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j >= 0) x[p] = load4<DT>(a.x[side], (long long)(first + j) * a.xs[side][0] + (long long)head * a.xs[side][1] + 4 * l);
    }
#pragma unroll
    for (int p = 0; p < 4 * GROUPS; ++p) {
      const int o = D == 128 ? p : (p >> 2) * 8 + hw * 4 + (p & 3);
      const float sum = x[p].x * 0.f + x[p].y * 0.f + x[p].z * 0.f + x[p].w * 0.f;  // NaN where one is not finite
      if (sum != 0.f) {
        const bool is_nan = x[p].x != x[p].x || x[p].y != x[p].y || x[p].z != x[p].z || x[p].w != x[p].w;
        if (is_nan) nan |= 1u << o;
      }
      float* v = &x[p].x;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = fminf(fmaxf(v[k], -kKvSaturate), kKvSaturate);
    }
    nan = __reduce_or_sync(0xffffffffu, nan);
#pragma unroll
    for (int p = 0; p < 4 * GROUPS; ++p) {
      const int o = D == 128 ? p : (p >> 2) * 8 + hw * 4 + (p & 3);
      if (nan >> o & 1u) x[p] = make_float4(0.f, 0.f, 0.f, 0.f);
      most = fmaxf(fmax3(most, fabsf(x[p].x), fabsf(x[p].y)), fmaxf(fabsf(x[p].z), fabsf(x[p].w)));
    }
    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
    const float scale = fmaxf(old, scale_for(most));
    const float inv = scale > 0.f ? 1.f / scale : 0.f;
    const bool grown = old > 0.f && scale > old;
    const float ratio = old * inv;
    const uint32_t kept = ~written & 0xFFFFu;
    if (side == 0) {
#pragma unroll
      for (int p = 0; p < 4 * GROUPS; ++p) {
        const int o = D == 128 ? p : (p >> 2) * 8 + hw * 4 + (p & 3);
        uint32_t* to = reinterpret_cast<uint32_t*>(at + o * Blk::row + kv8_key_chunk<D>(o, l / 4) * 16 + (l % 4) * 4);
        if (written >> o & 1u)
          *to = code_of(x[p].x, inv) | code_of(x[p].y, inv) << 8 | code_of(x[p].z, inv) << 16 | code_of(x[p].w, inv) << 24;
        else if (grown)
          *to = rescaled(*to, ratio);
      }
    } else {
#pragma unroll
      for (int q = 0; q < GROUPS; ++q) {
        const int group = D == 128 ? q : 2 * q + hw;
        const uint32_t here = written >> (4 * group) & 15u;
        if (here == 0 && !grown) continue;
        uint4* to = reinterpret_cast<uint4*>(at + Blk::half + l * 64 + group * 16);
        uint32_t c[4] = {0u, 0u, 0u, 0u};
        if (here != 15u) {
          const uint4 u = *to;
          c[0] = u.x; c[1] = u.y; c[2] = u.z; c[3] = u.w;
          if (grown)
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] = rescaled(c[k], ratio);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (here >> j & 1u) {
            const float4& v = x[4 * q + j];
            const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] = (c[k] & ~(0xFFu << (8 * j))) | code_of(f[k], inv) << (8 * j);
          }
        *to = make_uint4(c[0], c[1], c[2], c[3]);
      }
    }
    if (lane == 0) {
      const uint16_t marks = (uint16_t)((old_nan & kept) | (nan & written));
      if (side) {
        tail->vs = scale;
        tail->v_nan = marks;
      } else {
        tail->ks = scale;
        tail->k_nan = marks;
        if (fresh) tail->zero = 0u;
      }
    }
    __syncwarp();  // the map is read
  }
}

// D / 4 lanes a row, the rows of 16 tokens of a head one after the other: they mostly lie in one
// block, whose cells of values they share in L1.
template <int D, int DT>
__global__ void __launch_bounds__(kThreads) kv8_gather_kernel(const Kv4RowArgs a, int tokens) {
  using Blk = Kv8Block<D>;
  constexpr int LPR = D / 4, ROWS = kThreads / LPR;
  const int l = threadIdx.x % LPR;
  const long long r = (long long)blockIdx.x * ROWS + threadIdx.x / LPR;
  const int unit = (int)(r / kKvBlock), group = a.heads.div(unit), head = unit - group * (int)a.heads.d;
  const int tok = group * kKvBlock + (int)(r % kKvBlock);
  if (tok >= tokens) return;
  const int slot = __ldg(a.slots + tok);
  float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
  if (slot >= 0) {
    const uint8_t* at = block_at(a.c, slot / kKvBlock, head, Blk::bytes);
    if (at) {
      const int o = slot % kKvBlock;
      const uint32_t kw = *reinterpret_cast<const uint32_t*>(at + o * Blk::row + kv8_key_chunk<D>(o, l / 4) * 16 + (l % 4) * 4);
      const uint4 cell = *reinterpret_cast<const uint4*>(at + Blk::half + l * 64 + (o / 4) * 16);
      const uint4 tail = *reinterpret_cast<const uint4*>(at + Blk::tail);
      const int sh = 8 * (o % 4);
      const float ks = tail.z >> o & 1u ? NAN : __uint_as_float(tail.x);
      const float vs = tail.z >> (16 + o) & 1u ? NAN : __uint_as_float(tail.y);
      k = make_float4((float)(int8_t)kw * ks, (float)(int8_t)(kw >> 8) * ks, (float)(int8_t)(kw >> 16) * ks, (float)(int8_t)(kw >> 24) * ks);
      v = make_float4((float)(int8_t)(cell.x >> sh) * vs, (float)(int8_t)(cell.y >> sh) * vs, (float)(int8_t)(cell.z >> sh) * vs,
                      (float)(int8_t)(cell.w >> sh) * vs);
    } else {
      atomicCAS(&a.st->code, 0, (int)FA_ERR_INDEX);
    }
  }
  store4<DT>(a.x[0], (long long)tok * a.xs[0][0] + (long long)head * a.xs[0][1] + 4 * l, k);
  store4<DT>(a.x[1], (long long)tok * a.xs[1][0] + (long long)head * a.xs[1][1] + 4 * l, v);
}

template <int D, int DT>
cudaError_t launch(const Kv4RowArgs& a, bool gather, int sms, cudaStream_t s) {
  const int heads = (int)a.heads.d, tokens = a.rows / heads;
  if (gather) {
    const long long rows = (long long)(tokens + kKvBlock - 1) / kKvBlock * kKvBlock * heads, per = kThreads / (D / 4);
    kv8_gather_kernel<D, DT><<<(unsigned)((rows + per - 1) / per), kThreads, 0, s>>>(a, tokens);
  } else {
    // a token a warp where that gives the GPU no more than a few warps for each scheduler
    const long long most = (long long)sms * 64, span = std::min(16ll, std::max(1ll, 2ll * a.rows / most));
    const long long warps = 2 * ((tokens + span - 1) / span) * heads;
    kv8_append_kernel<D, DT><<<(unsigned)((warps + kWarps - 1) / kWarps), kThreads, 0, s>>>(a, tokens, (int)span);
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
