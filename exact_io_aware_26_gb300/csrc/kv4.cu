// kv4.cu -- writing tokens' keys and values into the 4-bit cache, and reading them
// back.  Both are streams: bound by HBM for prompts, by latency for single tokens.
// Eight channels per lane (a 16-byte load of a 16-bit type, one 4-byte word of
// codes), four lanes per pair, whose least and largest are two shuffles each.
#include "kv4.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

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
         (((long long)head << (a.c.page_log - 4)) + in / kKvBlock) * block_bytes;
}

// Codes of a lane's eight values and the pair of its group of four lanes.
__device__ __forceinline__ void quantise8(float (&v)[8], uint32_t& word, uint32_t& pair) {
  float lo = kKvSaturate, hi = -kKvSaturate;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    nan |= v[i] != v[i];
    v[i] = fminf(fmaxf(v[i], -kKvSaturate), kKvSaturate);
    lo = fminf(lo, v[i]);
    hi = fmaxf(hi, v[i]);
  }
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    nan |= __shfl_xor_sync(0xffffffffu, (int)nan, off) != 0;
  }
  // the documented steps, each rounded once: plain fp32, no contraction
  const __half s = __float2half_rn(__fdiv_rn(__fmul_rn(__fsub_rn(hi, lo), 16.f), 15.f));
  const __half c = __float2half_rn(__fsub_rn(lo, __half2float(s)));
  const float sf = __half2float(s), cf = __half2float(c);
  word = 0;
  if (sf > 0.f && !nan) {
    // The quotient only decides between neighbouring codes: a product with the rounded
    // reciprocal is off by less than 2^-22 of it, at most 31 + a clamped rest, so that
    // its rounding is the quotient's unless it lies within 2^-16 of a half, where the
    // division itself is done (a fifth of the time of eight divisions).
    const float inv = 1.f / sf;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = __fmul_rn(__fsub_rn(v[i], cf), 16.f);
      float t = fminf(__fmul_rn(d, inv), 64.f) - 16.f;
      if (fabsf(fabsf(t - rintf(t)) - 0.5f) < 0x1p-16f) t = __fsub_rn(__fdiv_rn(d, sf), 16.f);
      word |= (uint32_t)fminf(fmaxf(rintf(t), 0.f), 15.f) << (4 * i);
    }
  }
  pair = nan ? 0x7E007E00u : (uint32_t)__half_as_ushort(s) | ((uint32_t)__half_as_ushort(c) << 16);
}

// A row is one head of one token: D / 8 lanes, which take its key and its value.
template <int D, int DT>
__global__ void __launch_bounds__(kThreads) kv4_append_kernel(const Kv4RowArgs a) {
  using Blk = KvBlock<D>;
  constexpr int LPR = D / 8;
  const int j = threadIdx.x % LPR, r = blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
  const bool live = r < a.rows;
  const int tok = a.heads.div(r), head = r - tok * (int)a.heads.d;
  float k[8] = {}, v[8] = {};
  int row = 0;
  uint8_t* blk = nullptr;
  if (live) {
    load8<DT>(a.x[0], tok * a.xs[0][0] + head * a.xs[0][1] + 8 * j, k);
    load8<DT>(a.x[1], tok * a.xs[1][0] + head * a.xs[1][1] + 8 * j, v);
    blk = slot_block(a, __ldg(a.slots + tok), head, Blk::bytes, row);
  }
  uint32_t wk, pk, wv, pv;
  quantise8(k, wk, pk);
  quantise8(v, wv, pv);
  if (!blk) return;
  uint8_t* at = blk + row * Blk::row + 4 * j;
  *reinterpret_cast<uint32_t*>(at) = wk;
  *reinterpret_cast<uint32_t*>(at + Blk::half) = wv;
  if ((j & 3) == 0) {
    at = blk + Blk::codes + (row * Blk::groups + (j >> 2)) * 4;
    *reinterpret_cast<uint32_t*>(at) = pk;
    *reinterpret_cast<uint32_t*>(at + Blk::half) = pv;
  }
}

template <int DT>
__device__ __forceinline__ void store_values(void* x, long long to, uint32_t word, uint32_t pair) {
  const __half2 p = *reinterpret_cast<const __half2*>(&pair);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half m = __ushort_as_half((unsigned short)(0x3C00u | (((word >> (4 * i)) & 15u) << 6)));
    v[i] = __half2float(__hfma(m, __low2half(p), __high2half(p)));
  }
  if constexpr (DT == FA_F32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(x) + to);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    constexpr bool F16 = DT == FA_F16;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(x) + to) =
        make_uint4(pack2<F16>(v[0], v[1]), pack2<F16>(v[2], v[3]), pack2<F16>(v[4], v[5]), pack2<F16>(v[6], v[7]));
  }
}

template <int D, int DT>
__global__ void __launch_bounds__(kThreads) kv4_gather_kernel(const Kv4RowArgs a) {
  using Blk = KvBlock<D>;
  constexpr int LPR = D / 8;
  const int j = threadIdx.x % LPR, r = blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
  if (r >= a.rows) return;
  const int tok = a.heads.div(r), head = r - tok * (int)a.heads.d;
  int row;
  const uint8_t* blk = slot_block(a, __ldg(a.slots + tok), head, Blk::bytes, row);
  uint32_t wk = 0, pk = 0, wv = 0, pv = 0;
  if (blk) {
    const uint8_t* at = blk + row * Blk::row + 4 * j;
    wk = *reinterpret_cast<const uint32_t*>(at);
    wv = *reinterpret_cast<const uint32_t*>(at + Blk::half);
    at = blk + Blk::codes + (row * Blk::groups + (j >> 2)) * 4;
    pk = *reinterpret_cast<const uint32_t*>(at);
    pv = *reinterpret_cast<const uint32_t*>(at + Blk::half);
  }
  store_values<DT>(a.x[0], tok * a.xs[0][0] + head * a.xs[0][1] + 8 * j, wk, pk);
  store_values<DT>(a.x[1], tok * a.xs[1][0] + head * a.xs[1][1] + 8 * j, wv, pv);
}

template <int D, int DT>
cudaError_t launch(const Kv4RowArgs& a, bool gather, cudaStream_t s) {
  const int per = kThreads / (D / 8), grid = (a.rows + per - 1) / per;
  if (gather)
    kv4_gather_kernel<D, DT><<<grid, kThreads, 0, s>>>(a);
  else
    kv4_append_kernel<D, DT><<<grid, kThreads, 0, s>>>(a);
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
