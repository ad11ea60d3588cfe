// qk_norm_rope.cu -- RMS norms of the query and key heads and the rotation by
// position in one pass, and the gradient.
//
//   n = x r w, r = 1 / sqrt(mean x^2 + eps);  (y_a, y_b) = R(t) (n_a, n_b) per pair
//   dz = R(-t) dy, dn = w dz, h = x r:  dx = r (dn - h mean(dn h)),  dw = sum dz h
//
// Every element is read once and written once, so both directions are bound by
// HBM.  A row (one head of one token) belongs to D / 16 lanes of 16 channels, two
// chunks of eight (16-byte loads for 16-bit types) chosen so that a lane holds both
// elements of its pairs: sums over the row are a few shuffles and the rotation none.
// A lane keeps one token of its tile and walks its heads, so that the angles of its
// eight pairs are formed once for all heads it visits.
//
// The angle is exact at any position: position * freqs[i] mod 2^64 is the phase in
// 2^-64 turns, of which the leading 32 bits, signed, are taken to fp32 (an error of
// at most 2^-25 of half a turn).
#include "ops.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

// Eight consecutive elements, as loaded and as fp32.  (Plain loads: the result may be the
// input itself.)
template <int DT>
struct Raw8 {
  uint4 u[DT == FA_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, long long at) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + at * (DT == FA_F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (DT == FA_F32 ? 2 : 1); ++i) u[i] = p[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (DT == FA_F32 ? 2 : 1); ++i) u[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (DT == FA_F32) {
      v[0] = __uint_as_float(u[0].x); v[1] = __uint_as_float(u[0].y);
      v[2] = __uint_as_float(u[0].z); v[3] = __uint_as_float(u[0].w);
      v[4] = __uint_as_float(u[1].x); v[5] = __uint_as_float(u[1].y);
      v[6] = __uint_as_float(u[1].z); v[7] = __uint_as_float(u[1].w);
    } else {
      const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<DT == FA_F16>(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
};
template <int DT>
__device__ __forceinline__ void store8(void* base, long long at, const float (&v)[8]) {
  if constexpr (DT == FA_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    constexpr bool F16 = DT == FA_F16;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) =
        make_uint4(pack2<F16>(v[0], v[1]), pack2<F16>(v[2], v[3]), pack2<F16>(v[4], v[5]),
                   pack2<F16>(v[6], v[7]));
  }
}
template <int DT>
__device__ __forceinline__ void load_w8(const void* w, bool w_f32, int at, float (&v)[8]) {
  if (w_f32) {
    Raw8<FA_F32> r;
    r.load(w, at);
    r.get(v);
  } else {
    Raw8<DT> r;
    r.load(w, at);
    r.get(v);
  }
}

__device__ __forceinline__ void angle(const QkArgs& a, int pair, int pos, float& c, float& s) {
  const unsigned long long ph = (unsigned long long)(long long)pos * __ldg(a.freqs + pair);
  // signed leading 32 bits: the phase in 2^-32 turns; in half turns for sincospi
  sincospif((float)(int)(ph >> 32) * 4.656612873077393e-10f, &s, &c);
}

// Which channels and pairs a lane holds.  `paired`: rot % 16 == 0 (or interleaved
// pairs): the lane's chunks lo, hi hold both elements of its pairs -- element e of lo
// with element e of hi, or, interleaved, neighbours within each chunk -- and `on` has
// a bit for each of its eight pairs that is rotated.
struct Lane {
  int lo, hi;    // first channel of each chunk
  uint32_t on;   // pairs rotated
  float c[8], s[8];
};

template <int D>
__device__ __forceinline__ void lane_channels(const QkArgs& a, int j, Lane& L) {
  const int q = a.rot / 16;  // chunks in the first elements of the rotated pairs
  if (a.interleaved) {
    L.lo = 8 * j;
    L.hi = D / 2 + 8 * j;
    L.on = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      L.on |= (uint32_t)(L.lo + 2 * i < a.rot) << i;
      L.on |= (uint32_t)(L.hi + 2 * i < a.rot) << (4 + i);
    }
  } else if (j < q) {
    L.lo = 8 * j;
    L.hi = 8 * (j + q);
    L.on = 0xFFu;
  } else {  // behind the rotated channels: two neighbouring chunks
    L.lo = 8 * (2 * j);
    L.hi = 8 * (2 * j + 1);
    L.on = 0;
  }
}

__device__ __forceinline__ void lane_angles(const QkArgs& a, int pos, Lane& L) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    L.c[i] = 1.f;
    L.s[i] = 0.f;
    if ((L.on >> i) & 1u) {
      const int pair = a.interleaved ? ((i < 4 ? L.lo : L.hi) >> 1) + (i & 3) : L.lo + i;
      angle(a, pair, pos, L.c[i], L.s[i]);
    }
  }
}

// Rotates the lane's pairs (back with sgn = -1).
__device__ __forceinline__ void rotate(const QkArgs& a, const Lane& L, float sgn, float (&lo)[8], float (&hi)[8]) {
  if (L.on == 0) return;
  if (a.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((L.on >> i) & 1u) {
        const float u = lo[2 * i], v = lo[2 * i + 1], s = sgn * L.s[i];
        lo[2 * i] = u * L.c[i] - v * s;
        lo[2 * i + 1] = u * s + v * L.c[i];
      }
      if ((L.on >> (4 + i)) & 1u) {
        const float u = hi[2 * i], v = hi[2 * i + 1], s = sgn * L.s[4 + i];
        hi[2 * i] = u * L.c[4 + i] - v * s;
        hi[2 * i + 1] = u * s + v * L.c[4 + i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = lo[i], v = hi[i], s = sgn * L.s[i];
      lo[i] = u * L.c[i] - v * s;
      hi[i] = u * s + v * L.c[i];
    }
  }
}

// A rotated range whose halves are no whole chunks (rot % 16 != 0, pairs i and
// i + rot / 2): the row goes through shared memory and every element finds its
// partner there; angles are formed on the spot.  All lanes of the row's group call it.
template <int D>
__device__ __forceinline__ void rotate_any(const QkArgs& a, float* row, int pos, float sgn, const Lane& L,
                                           float (&lo)[8], float (&hi)[8]) {
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    row[L.lo + i] = lo[i];
    row[L.hi + i] = hi[i];
  }
  __syncwarp();
  const int half = a.rot / 2;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int ch = (side ? L.hi : L.lo) + i;
      if (ch >= a.rot) continue;
      const int pair = ch < half ? ch : ch - half;
      float c, s;
      angle(a, pair, pos, c, s);
      s *= sgn;
      const float u = row[pair], v = row[pair + half];
      const float y = ch < half ? u * c - v * s : u * s + v * c;
      if (side)
        hi[i] = y;
      else
        lo[i] = y;
    }
  }
  // the loop above indexes lo, hi at run time only through its own counter: both
  // stay in local memory in this variant, which is for unusual rotation sizes
}

template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = D / 32; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// What a CTA does: its tensor (0: queries, 1: keys) and its place among that tensor's CTAs.
struct Part {
  int t, first, step;
};
__device__ __forceinline__ Part part_of(const QkArgs& a) {
  const int b = blockIdx.x;
  return b < a.ctas[0] ? Part{0, b, a.ctas[0]} : Part{1, b - a.ctas[0], a.ctas[1]};
}

// The kThreads / (D / 16) row slots of a CTA hold tok_tile tokens, each by as many slots as
// are left, which share its heads; the CTA walks the tiles (batch entry, tok_tile tokens)
// of its tensor.  The next row is loaded before this one is worked on.
template <int D, int DT, bool ANY>
__global__ void __launch_bounds__(kThreads, 3) qk_norm_rope_kernel(const QkArgs a, const bool w_f32) {
  constexpr int LPR = D / 16, ROWS = kThreads / LPR;
  __shared__ float rows_s[ANY ? ROWS * D : 1];
  const Part part = part_of(a);
  const int t = part.t, H = t ? a.Hk : a.Hq;
  const int j = threadIdx.x % LPR, slot = threadIdx.x / LPR;
  const int tok = slot & (a.tok_tile - 1), share = slot / a.tok_tile, shares = ROWS / a.tok_tile;
  Lane L;
  if constexpr (ANY) {
    L.lo = 8 * j;
    L.hi = D / 2 + 8 * j;
  } else {
    lane_channels<D>(a, j, L);
  }
  const long long xh = t ? a.xs[1][2] : a.xs[0][2], yh = t ? a.ys[1][2] : a.ys[0][2];
  const void* x = t ? a.x[1] : a.x[0];
  void* y = t ? a.y[1] : a.y[0];
  float wl[8], wh[8];
  load_w8<DT>(t ? a.w[1] : a.w[0], w_f32, L.lo, wl);
  load_w8<DT>(t ? a.w[1] : a.w[0], w_f32, L.hi, wh);
  for (int tile = part.first; tile < a.B * a.tiles; tile += part.step) {
    const int b = tile / a.tiles, n = (tile - b * a.tiles) * a.tok_tile + tok;
    const bool in = n < a.N;
    const long long xb = b * (t ? a.xs[1][0] : a.xs[0][0]) + (long long)n * (t ? a.xs[1][1] : a.xs[0][1]);
    const long long yb = b * (t ? a.ys[1][0] : a.ys[0][0]) + (long long)n * (t ? a.ys[1][1] : a.ys[0][1]);
    Raw8<DT> rl, rh;
    rl.zero();
    rh.zero();
    if (in && share < H) {
      rl.load(x, xb + share * xh + L.lo);
      rh.load(x, xb + share * xh + L.hi);
    }
    const int pos = !in ? 0 : a.pos ? __ldg(a.pos + b * a.pos_stride + n) : n;
    if constexpr (!ANY) lane_angles(a, pos, L);
    // every lane of a warp takes the same number of turns: the row sums are shuffles
    for (int h0 = 0; h0 < H; h0 += shares) {
      const int h = h0 + share;
      float lo[8], hi[8];
      rl.get(lo);
      rh.get(hi);
      if (in && h + shares < H) {
        rl.load(x, xb + (h + shares) * xh + L.lo);
        rh.load(x, xb + (h + shares) * xh + L.hi);
      }
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(lo[i], lo[i], fmaf(hi[i], hi[i], ss));
      const float r = rsqrtf(row_sum<D>(ss) * (1.f / D) + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo[i] *= r * wl[i];
        hi[i] *= r * wh[i];
      }
      if constexpr (ANY)
        rotate_any<D>(a, rows_s + slot * D, pos, 1.f, L, lo, hi);
      else
        rotate(a, L, 1.f, lo, hi);
      if (in && h < H) {
        store8<DT>(y, yb + h * yh + L.lo, lo);
        store8<DT>(y, yb + h * yh + L.hi, hi);
      }
    }
  }
}

// The gradient, in the same way; a lane adds up the weights' gradients of its channels, and
// each CTA leaves one partial sum.
template <int D, int DT, bool ANY>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_rope_bwd_kernel(const QkArgs a, const bool w_f32) {
  constexpr int LPR = D / 16, ROWS = kThreads / LPR, WARPS = kThreads / 32;
  __shared__ float rows_s[ANY ? ROWS * D : 1];
  __shared__ float red[WARPS][D];
  const Part part = part_of(a);
  const int t = part.t, H = t ? a.Hk : a.Hq;
  const int j = threadIdx.x % LPR, slot = threadIdx.x / LPR;
  const int tok = slot & (a.tok_tile - 1), share = slot / a.tok_tile, shares = ROWS / a.tok_tile;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Lane L;
  if constexpr (ANY) {
    L.lo = 8 * j;
    L.hi = D / 2 + 8 * j;
  } else {
    lane_channels<D>(a, j, L);
  }
  const long long xh = t ? a.xs[1][2] : a.xs[0][2], yh = t ? a.ys[1][2] : a.ys[0][2], dh = t ? a.ds[1][2] : a.ds[0][2];
  const void *x = t ? a.x[1] : a.x[0], *dy = t ? a.dy[1] : a.dy[0];
  void* y = t ? a.y[1] : a.y[0];
  float wl[8], wh[8];
  load_w8<DT>(t ? a.w[1] : a.w[0], w_f32, L.lo, wl);
  load_w8<DT>(t ? a.w[1] : a.w[0], w_f32, L.hi, wh);
  float acc[16] = {};
  for (int tile = part.first; tile < a.B * a.tiles; tile += part.step) {
    const int b = tile / a.tiles, n = (tile - b * a.tiles) * a.tok_tile + tok;
    const bool in = n < a.N;
    const long long xb = b * (t ? a.xs[1][0] : a.xs[0][0]) + (long long)n * (t ? a.xs[1][1] : a.xs[0][1]);
    const long long yb = b * (t ? a.ys[1][0] : a.ys[0][0]) + (long long)n * (t ? a.ys[1][1] : a.ys[0][1]);
    const long long db = b * (t ? a.ds[1][0] : a.ds[0][0]) + (long long)n * (t ? a.ds[1][1] : a.ds[0][1]);
    Raw8<DT> rl, rh, sl, sh;
    rl.zero();
    rh.zero();
    sl.zero();
    sh.zero();
    if (in && share < H) {
      rl.load(x, xb + share * xh + L.lo);
      rh.load(x, xb + share * xh + L.hi);
      sl.load(dy, db + share * dh + L.lo);
      sh.load(dy, db + share * dh + L.hi);
    }
    const int pos = !in ? 0 : a.pos ? __ldg(a.pos + b * a.pos_stride + n) : n;
    if constexpr (!ANY) lane_angles(a, pos, L);
    for (int h0 = 0; h0 < H; h0 += shares) {
      const int h = h0 + share;
      const bool live = in && h < H;
      float lo[8], hi[8], gl[8], gh[8];
      rl.get(lo);
      rh.get(hi);
      sl.get(gl);
      sh.get(gh);
      if (in && h + shares < H) {
        rl.load(x, xb + (h + shares) * xh + L.lo);
        rh.load(x, xb + (h + shares) * xh + L.hi);
        sl.load(dy, db + (h + shares) * dh + L.lo);
        sh.load(dy, db + (h + shares) * dh + L.hi);
      }
      if constexpr (ANY)
        rotate_any<D>(a, rows_s + slot * D, pos, -1.f, L, gl, gh);
      else
        rotate(a, L, -1.f, gl, gh);
      float ss = 0.f, sd = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(lo[i], lo[i], fmaf(hi[i], hi[i], ss));
        sd = fmaf(gl[i] * wl[i], lo[i], fmaf(gh[i] * wh[i], hi[i], sd));
      }
      const float r = rsqrtf(row_sum<D>(ss) * (1.f / D) + a.eps);
      const float m = row_sum<D>(sd) * (1.f / D) * r * r;  // mean(dn h) r: what x takes off dn
      const float in_sum = live ? r : 0.f;                 // rows of other lanes' turns add nothing
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[i] = fmaf(gl[i], lo[i] * in_sum, acc[i]);
        acc[8 + i] = fmaf(gh[i], hi[i] * in_sum, acc[8 + i]);
        lo[i] = r * (gl[i] * wl[i] - lo[i] * m);
        hi[i] = r * (gh[i] * wh[i] - hi[i] * m);
      }
      if (live) {
        store8<DT>(y, yb + h * yh + L.lo, lo);
        store8<DT>(y, yb + h * yh + L.hi, hi);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float v = acc[i];
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (lane < LPR) red[warp][(i < 8 ? L.lo : L.hi) + (i & 7)] = v;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v += red[w][threadIdx.x];
    a.part[(size_t)blockIdx.x * D + threadIdx.x] = v;
  }
}

// dw: the partial sums of a tensor's CTAs, in a fixed order.  One CTA per 32 channels.
__global__ void __launch_bounds__(1024) qk_dw_kernel(const QkArgs a, const int D) {
  __shared__ float red[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int t = blockIdx.x * 32 >= D, lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int ch = blockIdx.x * 32 - t * D + lane;
  const int c0 = t ? a.ctas[0] : 0, c1 = c0 + a.ctas[t];
  float v = 0.f;
#pragma unroll 8
  for (int c = c0 + row; c < c1; c += 32) v += a.part[(size_t)c * D + ch];
  red[row][lane] = v;
  __syncthreads();
  if (row == 0) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][lane];
    (t ? a.dw[1] : a.dw[0])[ch] = s;
  }
}

template <int D, int DT>
cudaError_t launch_d(const QkArgs& a, bool w_f32, bool bwd, cudaStream_t s) {
  const bool any = !a.interleaved && a.rot % 16 != 0;
  const int grid = a.ctas[0] + a.ctas[1];
  if (grid > 0) {
    if (bwd) {
      if (any)
        qk_norm_rope_bwd_kernel<D, DT, true><<<grid, kThreads, 0, s>>>(a, w_f32);
      else
        qk_norm_rope_bwd_kernel<D, DT, false><<<grid, kThreads, 0, s>>>(a, w_f32);
    } else {
      if (any)
        qk_norm_rope_kernel<D, DT, true><<<grid, kThreads, 0, s>>>(a, w_f32);
      else
        qk_norm_rope_kernel<D, DT, false><<<grid, kThreads, 0, s>>>(a, w_f32);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (bwd) {
    // launched with the first kernel, whose end it waits for on the GPU
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * D / 32);
    cfg.blockDim = dim3(1024);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = grid > 0 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, qk_dw_kernel, a, D);
  }
  return cudaSuccess;
}

cudaError_t launch(const QkArgs& a, int d, int dtype, bool w_f32, bool bwd, cudaStream_t s) {
  if (d == 64)
    return dtype == FA_F32   ? launch_d<64, FA_F32>(a, w_f32, bwd, s)
           : dtype == FA_F16 ? launch_d<64, FA_F16>(a, w_f32, bwd, s)
                             : launch_d<64, FA_BF16>(a, w_f32, bwd, s);
  return dtype == FA_F32   ? launch_d<128, FA_F32>(a, w_f32, bwd, s)
         : dtype == FA_F16 ? launch_d<128, FA_F16>(a, w_f32, bwd, s)
                           : launch_d<128, FA_BF16>(a, w_f32, bwd, s);
}

}  // namespace

int qk_rows_per_pass(int d) { return kThreads / (d / 16); }

cudaError_t launch_qk_norm_rope(const QkArgs& a, int d, int dtype, bool w_f32, cudaStream_t s) {
  return launch(a, d, dtype, w_f32, false, s);
}
cudaError_t launch_qk_norm_rope_bwd(const QkArgs& a, int d, int dtype, bool w_f32, cudaStream_t s) {
  return launch(a, d, dtype, w_f32, true, s);
}

}  // namespace fa
