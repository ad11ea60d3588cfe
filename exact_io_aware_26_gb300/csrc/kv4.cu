// kv4.cu -- writing tokens' keys and values into the 4-bit cache, and reading them
// back.  Both are streams, of long prompts against HBM, of single tokens against latency.
// Eight channels per lane (a 16-byte load of a 16-bit type, one 4-byte word of codes),
// four lanes per pair, whose least and largest are two shuffles each.
#include "kv4.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256, kAppendThreads = 128;

template <int DT>
__device__ __forceinline__ void load8(const void* base, long long at, float (&v)[8]) {
  if constexpr (DT == FA_F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<DT == FA_F16>(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

// Byte address of a slot's block, and its row there; nullptr for a slot that is left
// out (negative) or outside the cache (recorded).
__device__ __forceinline__ uint8_t* slot_block(const Kv4RowArgs& a, int slot, int head, int block_bytes, int& row) {
  row = 0;
  if (slot < 0) return nullptr;
  const int page = slot >> a.c.page_log, in = slot & ((1 << a.c.page_log) - 1);
  if (page >= a.c.num_pages) {
    atomicCAS(&a.st->code, 0, (int)FA_ERR_INDEX);
    return nullptr;
  }
  row = in % kKvBlock;
  return const_cast<uint8_t*>(a.c.data) + page * a.c.page_stride +
         (long long)((head << (a.c.page_log - 4)) + in / kKvBlock) * block_bytes;
}

__device__ __forceinline__ long long row_at(const Kv4RowArgs& a, int side, int tok, int head) {
  return (long long)tok * a.xs[side][0] + (long long)head * a.xs[side][1];
}

// Least and largest of three, NaN if one is.
__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Writing prompts of 16-bit types is bound by its instructions (326 a warp for 512 values,
// 0.72 issued a cycle) before HBM; hence packed fp32 arithmetic, three-input minima, one pair
// per lane (the key's or the value's), and no division or clamping per value where neither
// can matter.  23,400 tokens of 12 heads, d = 64: bf16 27.3 us (94 MB, 3.4 TB/s; 25.3 with
// sixteen values of each tensor to a lane, where single tokens of 256 requests cost 3.3 us
// instead of 2.8), fp32 27.8 us (166 MB, 6.0 TB/s).

// Least and largest of a lane's eight values and those of its group of four lanes.
__device__ __forceinline__ void range8(const float (&v)[8], float& lo, float& hi) {
  lo = min3_nan(min3_nan(v[0], v[1], v[2]), min3_nan(v[3], v[4], v[5]), min3_nan(v[6], v[7], v[7]));
  hi = max3_nan(max3_nan(v[0], v[1], v[2]), max3_nan(v[3], v[4], v[5]), max3_nan(v[6], v[7], v[7]));
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) {
    const float l = __shfl_xor_sync(0xffffffffu, lo, off), h = __shfl_xor_sync(0xffffffffu, hi, off);
    lo = min3_nan(lo, l, l);
    hi = max3_nan(hi, h, h);
  }
}

// The pair of a group, and 16 / scale: negative where its codes need the documented steps
// one by one (codes8).
__device__ __forceinline__ void pair_of(float lo, float hi, uint32_t& pair, float& inv) {
  const bool nan = lo != lo;
  const float sat_lo = fminf(fmaxf(lo, -kKvSaturate), kKvSaturate), sat_hi = fminf(fmaxf(hi, -kKvSaturate), kKvSaturate);
  // the documented steps, each rounded once: plain fp32, no contraction
  const __half s = __float2half_rn(__fdiv_rn(__fmul_rn(__fsub_rn(sat_hi, sat_lo), 16.f), 15.f));
  const __half c = __float2half_rn(__fsub_rn(sat_lo, __half2float(s)));
  const float sf = __half2float(s), cf = __half2float(c);
  pair = nan ? 0x7E007E00u : (uint32_t)__half_as_ushort(s) | ((uint32_t)__half_as_ushort(c) << 16);
  inv = __fdividef(16.f, sf);
  // a scale of 0 or NaN, saturated values, or a least or largest value whose code is out of
  // range (fp16's rounding of a base far from 0)
  const float first = fmaf(lo - cf, inv, -16.f), last = fmaf(hi - cf, inv, -16.f);
  if (!(first > -0.5f && last < 15.5f && sat_lo == lo && sat_hi == hi && sf > 0.f)) inv = -1.f;
}

// Codes of a lane's eight values.  The quotient (x - base) * 16 / scale only decides between
// neighbouring codes: a product with the reciprocal is off by less than 2^-22 of it, below
// 2^-17, so its rounding is the quotient's unless it lies within 2^-16 of a half.
__device__ __forceinline__ uint32_t codes8(float (&v)[8], uint32_t pair, float inv) {
  const float cf = __half2float(__ushort_as_half((unsigned short)(pair >> 16)));
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number
  const uint64_t inv2 = f2pack(inv, inv), base2 = f2pack(-cf, -cf), off2 = f2pack(-16.f, -16.f);
  const uint64_t up2 = f2pack(kRound, kRound), down2 = f2pack(-kRound, -kRound), neg2 = f2pack(-1.f, -1.f);
  uint64_t code[4];
  float border = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t t = ffma2(fadd2(f2pack(v[2 * i], v[2 * i + 1]), base2), inv2, off2);
    code[i] = fadd2(fadd2(t, up2), down2);
    float x, y;
    f2unpack(ffma2(code[i], neg2, t), x, y);
    border = fmax3(border, fabsf(x), fabsf(y));
  }
  uint32_t word;
  if (border < 0.5f - 0x1p-16f && inv > 0.f) {
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // four codes: a whole number below 2^16, in the low bits of 2^23 more
      float even, odd;
      f2unpack(ffma2(code[2 * k + 1], f2pack(256.f, 256.f), code[2 * k]), even, odd);
      w[k] = __float_as_uint(fmaf(odd, 16.f, even) + 8388608.f);
    }
    word = __byte_perm(w[0], w[1], 0x5410);
  } else {
    const float sf = __half2float(__ushort_as_half((unsigned short)(pair & 0xFFFFu)));
    word = 0;
    if (sf > 0.f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = fminf(fmaxf(v[i], -kKvSaturate), kKvSaturate);
        const float t = __fsub_rn(__fdiv_rn(__fmul_rn(__fsub_rn(x, cf), 16.f), sf), 16.f);
        word |= (uint32_t)fminf(fmaxf(rintf(t), 0.f), 15.f) << (4 * i);
      }
    }
  }
  return word;
}

// A row is one head of one token: D / 8 lanes, which take its key and its value.
template <int D, int DT>
__global__ void __launch_bounds__(kAppendThreads) kv4_append_kernel(const Kv4RowArgs a) {
  using Blk = KvBlock<D>;
  constexpr int LPR = D / 8;
  const int j = threadIdx.x % LPR, r = blockIdx.x * (kAppendThreads / LPR) + threadIdx.x / LPR;
  const bool live = r < a.rows;
  const int tok = a.heads.div(r), head = r - tok * (int)a.heads.d;
  float k[8] = {}, v[8] = {};
  int row = 0;
  uint8_t* blk = nullptr;
  if (live) {
    load8<DT>(a.x[0], row_at(a, 0, tok, head) + 8 * j, k);
    load8<DT>(a.x[1], row_at(a, 1, tok, head) + 8 * j, v);
    blk = slot_block(a, __ldg(a.slots + tok), head, Blk::bytes, row);
  }
  float lo[2], hi[2];
  range8(k, lo[0], hi[0]);
  range8(v, lo[1], hi[1]);
  uint32_t pair;  // even lanes the key's, odd lanes the value's
  float inv;
  pair_of(j & 1 ? lo[1] : lo[0], j & 1 ? hi[1] : hi[0], pair, inv);
  const int lane = threadIdx.x & 31;
  const uint32_t pk = __shfl_sync(0xffffffffu, pair, lane & ~1), pv = __shfl_sync(0xffffffffu, pair, lane | 1);
  const float ik = __shfl_sync(0xffffffffu, inv, lane & ~1), iv = __shfl_sync(0xffffffffu, inv, lane | 1);
  const uint32_t wk = codes8(k, pk, ik), wv = codes8(v, pv, iv);
  if (!blk) return;
  uint8_t* at = blk + row * Blk::row + 4 * j;
  *reinterpret_cast<uint32_t*>(at) = wk;
  *reinterpret_cast<uint32_t*>(at + Blk::half) = wv;
  // the pairs of a group: its first lane stores the key's, its second the value's
  if ((j & 2) == 0) {
    at = blk + Blk::codes + (row * Blk::groups + (j >> 2)) * 4;
    *reinterpret_cast<uint32_t*>(at + (j & 1) * Blk::half) = j & 1 ? pv : pk;
  }
}

template <int DT>
__device__ __forceinline__ void store_values(void* x, long long to, bool live, uint32_t word, uint32_t pair) {
  // codes p and p + 4 of the word as half2, then neighbours side by side
  const __half2 p = *reinterpret_cast<const __half2*>(&pair);
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = ((i < 2 ? word << (6 - 4 * i) : word >> (4 * i - 6)) & 0x03C003C0u) | 0x3C003C00u;
    const __half2 h = __hfma2(*reinterpret_cast<const __half2*>(&m), __low2half2(p), __high2half2(p));
    q[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  uint32_t n[4] = {__byte_perm(q[0], q[1], 0x5410), __byte_perm(q[2], q[3], 0x5410),
                   __byte_perm(q[0], q[1], 0x7632), __byte_perm(q[2], q[3], 0x7632)};
  // fp32: two lanes swap halves, so that their stores lie side by side (whole sectors)
  const int odd = threadIdx.x & 1;
  if constexpr (DT == FA_F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? n[i] : n[2 + i], 1);
      n[i] = odd ? got : n[i];
      n[2 + i] = odd ? n[2 + i] : got;
    }
  }
  if (!live) return;
  if constexpr (DT == FA_F16) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(x) + to) = make_uint4(n[0], n[1], n[2], n[3]);
  } else {
    float2 f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = unpack2<true>(n[i]);
    if constexpr (DT == FA_F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(x) + to - 4 * odd);
      o[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
      o[2] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(x) + to) =
          make_uint4(pack2<false>(f[0].x, f[0].y), pack2<false>(f[1].x, f[1].y), pack2<false>(f[2].x, f[2].y),
                     pack2<false>(f[3].x, f[3].y));
    }
  }
}

// Two rows per lane, so that two chains of loads (slot, then codes) are in flight: what
// there is of latency bounds it.  23,400 tokens of 12 heads, d = 64: bf16 18.7 us (94 MB, 5.0
// TB/s), fp32 30.8 us (166 MB, 5.4 TB/s; 42.6 with each lane's 32 bytes in two stores).
template <int D, int DT>
__global__ void __launch_bounds__(kThreads) kv4_gather_kernel(const Kv4RowArgs a) {
  using Blk = KvBlock<D>;
  constexpr int LPR = D / 8, ROWS = kThreads / LPR;
  const int j = threadIdx.x % LPR, r0 = blockIdx.x * (2 * ROWS) + threadIdx.x / LPR;
  int tok[2], head[2];
  uint32_t wk[2] = {}, pk[2] = {}, wv[2] = {}, pv[2] = {};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = min(r0 + i * ROWS, a.rows - 1);
    tok[i] = a.heads.div(r);
    head[i] = r - tok[i] * (int)a.heads.d;
    int row;
    const uint8_t* blk = slot_block(a, __ldg(a.slots + tok[i]), head[i], Blk::bytes, row);
    if (blk) {
      const uint8_t* at = blk + row * Blk::row + 4 * j;
      wk[i] = *reinterpret_cast<const uint32_t*>(at);
      wv[i] = *reinterpret_cast<const uint32_t*>(at + Blk::half);
      at = blk + Blk::codes + (row * Blk::groups + (j >> 2)) * 4;
      pk[i] = *reinterpret_cast<const uint32_t*>(at);
      pv[i] = *reinterpret_cast<const uint32_t*>(at + Blk::half);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool live = r0 + i * ROWS < a.rows;
    store_values<DT>(a.x[0], row_at(a, 0, tok[i], head[i]) + 8 * j, live, wk[i], pk[i]);
    store_values<DT>(a.x[1], row_at(a, 1, tok[i], head[i]) + 8 * j, live, wv[i], pv[i]);
  }
}

template <int D, int DT>
cudaError_t launch(const Kv4RowArgs& a, bool gather, cudaStream_t s) {
  auto grid = [&](int rows) { return (a.rows + rows - 1) / rows; };
  if (gather) {
    kv4_gather_kernel<D, DT><<<grid(2 * kThreads / (D / 8)), kThreads, 0, s>>>(a);
  } else {
    kv4_append_kernel<D, DT><<<grid(kAppendThreads / (D / 8)), kAppendThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_any(const Kv4RowArgs& a, int d, int dtype, bool gather, cudaStream_t s) {
  if (d == 64)
    return dtype == FA_F32   ? launch<64, FA_F32>(a, gather, s)
           : dtype == FA_F16 ? launch<64, FA_F16>(a, gather, s)
                             : launch<64, FA_BF16>(a, gather, s);
  return dtype == FA_F32   ? launch<128, FA_F32>(a, gather, s)
         : dtype == FA_F16 ? launch<128, FA_F16>(a, gather, s)
                           : launch<128, FA_BF16>(a, gather, s);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4RowArgs& a, int d, int dtype, cudaStream_t s) {
  return launch_any(a, d, dtype, false, s);
}
cudaError_t launch_kv4_gather(const Kv4RowArgs& a, int d, int dtype, cudaStream_t s) {
  return launch_any(a, d, dtype, true, s);
}

}  // namespace fa
