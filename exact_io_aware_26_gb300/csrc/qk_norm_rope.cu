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
// Each CTA takes an equal run of tokens, a few per SM in flight, and walks their rows
// token by token (a token's heads lie side by side in the projection), the next row
// loaded before this one is worked on; the angles of a run's tokens are formed once, in
// shared memory, for all their heads.
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
constexpr int kChunk = 32;  // tokens whose angles a CTA holds at a time

// cos and sin of a chunk's tokens, [token][pair], in shared memory.
template <int D>
struct Angles {
  float c[kChunk][D / 2], s[kChunk][D / 2];
};
template <int D>
__device__ __forceinline__ void form_angles(const QkArgs& a, int token0, int n, Angles<D>& out) {
  const int pairs = a.rot / 2;
  for (int e = threadIdx.x; e < n * (D / 2); e += kThreads) {
    const int tok = e / (D / 2), pair = e % (D / 2);
    if (pair >= pairs) continue;
    const int t = token0 + tok, b = a.divN.div(t), i = t - b * a.N;
    const int pos = a.pos ? __ldg(a.pos + b * a.pos_stride + i) : i;
    const unsigned long long ph = (unsigned long long)(long long)pos * __ldg(a.freqs + pair);
    // signed leading 32 bits: the phase in 2^-32 turns; in half turns for sincospi
    sincospif((float)(int)(ph >> 32) * 4.656612873077393e-10f, &out.s[tok][pair], &out.c[tok][pair]);
  }
}

// Which channels and pairs a lane holds.  With rot % 16 == 0 (or interleaved pairs) the
// lane's chunks lo, hi hold both elements of its pairs -- element e of lo with element e of
// hi, or, interleaved, neighbours within each chunk -- and `on` has a bit for each of its
// eight pairs that is rotated; pl, ph are the first pairs of its chunks.
struct Lane {
  int lo, hi;  // first channel of each chunk
  int pl, ph;
  uint32_t on;
};

template <int D, bool ANY>
__device__ __forceinline__ Lane lane_channels(const QkArgs& a, int j) {
  Lane L;
  const int q = a.rot / 16;  // chunks in the first elements of the rotated pairs
  L.lo = 8 * j;
  L.hi = D / 2 + 8 * j;
  L.on = 0;
  if (ANY) {
    L.pl = L.ph = 0;
  } else if (a.interleaved) {
    L.pl = L.lo / 2;
    L.ph = L.hi / 2;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      L.on |= (uint32_t)(L.lo + 2 * i < a.rot) << i;
      L.on |= (uint32_t)(L.hi + 2 * i < a.rot) << (4 + i);
    }
  } else if (j < q) {
    L.hi = 8 * (j + q);
    L.pl = L.lo;
    L.ph = L.lo + 4;
    L.on = 0xFFu;
  } else {  // behind the rotated channels: two neighbouring chunks
    L.lo = 8 * (2 * j);
    L.hi = 8 * (2 * j + 1);
    L.pl = L.ph = 0;
  }
  return L;
}

// Rotates the lane's pairs (back with BACK).
template <int D, bool BACK>
__device__ __forceinline__ void rotate(const QkArgs& a, const Lane& L, const float* c_row, const float* s_row,
                                       float (&lo)[8], float (&hi)[8]) {
  if (L.on == 0) return;
  float c[8], s[8];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float4 u = *reinterpret_cast<const float4*>(c_row + (k ? L.ph : L.pl));
    const float4 v = *reinterpret_cast<const float4*>(s_row + (k ? L.ph : L.pl));
    c[4 * k] = u.x; c[4 * k + 1] = u.y; c[4 * k + 2] = u.z; c[4 * k + 3] = u.w;
    s[4 * k] = v.x; s[4 * k + 1] = v.y; s[4 * k + 2] = v.z; s[4 * k + 3] = v.w;
  }
  auto turn = [&](float& p, float& q, int i) {
    const float u = p, v = q, sn = BACK ? -s[i] : s[i];
    p = u * c[i] - v * sn;
    q = u * sn + v * c[i];
  };
  if (a.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((L.on >> i) & 1u) turn(lo[2 * i], lo[2 * i + 1], i);
      if ((L.on >> (4 + i)) & 1u) turn(hi[2 * i], hi[2 * i + 1], 4 + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(lo[i], hi[i], i);
  }
}

// A rotated range whose halves are no whole chunks (rot % 16 != 0, pairs i and
// i + rot / 2): the row goes through shared memory and every element finds its
// partner there.  All lanes of the row's group call it.
template <int D, bool BACK>
__device__ __forceinline__ void rotate_any(const QkArgs& a, float* row, const Lane& L, const float* c_row,
                                           const float* s_row, float (&lo)[8], float (&hi)[8]) {
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    row[L.lo + i] = lo[i];
    row[L.hi + i] = hi[i];
  }
  __syncwarp();
  const int half = a.rot / 2;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int ch = (side ? L.hi : L.lo) + i;
      if (ch < a.rot) {
        const int pair = ch < half ? ch : ch - half;
        const float c = c_row[pair], s = BACK ? -s_row[pair] : s_row[pair];
        const float u = row[pair], v = row[pair + half];
        (side ? hi : lo)[i] = ch < half ? u * c - v * s : u * s + v * c;
      }
    }
  }
}

// Sum over the lanes of a row.
template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = D / 32; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// One of the two tensors: its heads, strides and pointers.
struct Tensor {
  int H;
  FastDiv div;
  const char *x, *dy;
  char* y;
  long long xs[3], ys[3], ds[3];  // bytes
};
template <int DT>
__device__ __forceinline__ Tensor tensor_of(const QkArgs& a, int t) {
  constexpr long long E = DT == FA_F32 ? 4 : 2;
  Tensor r;
  r.H = t ? a.Hk : a.Hq;
  r.div = t ? a.divH[1] : a.divH[0];
  r.x = static_cast<const char*>(t ? a.x[1] : a.x[0]);
  r.dy = static_cast<const char*>(t ? a.dy[1] : a.dy[0]);
  r.y = static_cast<char*>(t ? a.y[1] : a.y[0]);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    r.xs[i] = E * (t ? a.xs[1][i] : a.xs[0][i]);
    r.ys[i] = E * (t ? a.ys[1][i] : a.ys[0][i]);
    r.ds[i] = E * (t ? a.ds[1][i] : a.ds[0][i]);
  }
  return r;
}
// A row of it: the token's place in the chunk, and batch, token, head.
struct Row {
  int tok, b, n, h;
};
__device__ __forceinline__ Row row_of(const QkArgs& a, const Tensor& t, int token0, int i) {
  Row r;
  r.tok = t.div.div(i);
  r.h = i - r.tok * t.H;
  r.b = a.divN.div(token0 + r.tok);
  r.n = token0 + r.tok - r.b * a.N;
  return r;
}
__device__ __forceinline__ long long at(const Row& r, const long long (&s)[3]) {
  return r.b * s[0] + r.n * s[1] + r.h * s[2];
}

template <int DT>
__device__ __forceinline__ void weights_to_shared(const QkArgs& a, bool w_f32, int D, float* out) {
  for (int e = threadIdx.x; e < 2 * D; e += kThreads) {
    const void* w = e < D ? a.w[0] : a.w[1];
    const int c = e < D ? e : e - D;
    if (w_f32 || DT == FA_F32)
      out[e] = static_cast<const float*>(w)[c];
    else if (DT == FA_F16)
      out[e] = __half2float(static_cast<const __half*>(w)[c]);
    else
      out[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c]);
  }
}
__device__ __forceinline__ void read8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Tokens [first, last) of the CTA, and chunks of equal size over them.
struct Run {
  int first, last, chunk;
};
__device__ __forceinline__ Run run_of(const QkArgs& a) {
  Run r;
  const long long T = (long long)a.B * a.N;
  r.first = (int)(T * blockIdx.x / gridDim.x);
  r.last = (int)(T * (blockIdx.x + 1) / gridDim.x);
  const int n = r.last - r.first, chunks = (n + kChunk - 1) / kChunk;
  r.chunk = chunks ? (n + chunks - 1) / chunks : 1;
  return r;
}

template <int D, int DT, bool ANY>
__global__ void __launch_bounds__(kThreads, 3) qk_norm_rope_kernel(const QkArgs a, const bool w_f32) {
  constexpr int LPR = D / 16, ROWS = kThreads / LPR;
  __shared__ __align__(16) Angles<D> ang;
  __shared__ __align__(16) float w_s[2 * D];
  __shared__ float rows_s[ANY ? ROWS * D : 1];
  const int slot = threadIdx.x / LPR;
  const Lane L = lane_channels<D, ANY>(a, threadIdx.x % LPR);
  weights_to_shared<DT>(a, w_f32, D, w_s);
  const Run run = run_of(a);
  for (int t0 = run.first; t0 < run.last; t0 += run.chunk) {
    const int nt = min(run.chunk, run.last - t0);
    __syncthreads();  // the angles before have been used
    form_angles<D>(a, t0, nt, ang);
    __syncthreads();
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      const Tensor X = tensor_of<DT>(a, t);
      const int rows = nt * X.H;
      Raw8<DT> rl, rh;
      rl.zero();
      rh.zero();
      Row next = row_of(a, X, t0, min(slot, rows - 1));
      if (slot < rows) {
        rl.load(X.x + at(next, X.xs), L.lo);
        rh.load(X.x + at(next, X.xs), L.hi);
      }
      // every lane of a warp takes the same number of turns: the row sums are shuffles
      for (int i0 = 0; i0 < rows; i0 += ROWS) {
        const Row r = next;
        const bool live = i0 + slot < rows;
        float lo[8], hi[8];
        rl.get(lo);
        rh.get(hi);
        if (i0 + ROWS + slot < rows) {
          next = row_of(a, X, t0, i0 + ROWS + slot);
          rl.load(X.x + at(next, X.xs), L.lo);
          rh.load(X.x + at(next, X.xs), L.hi);
        }
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(lo[i], lo[i], fmaf(hi[i], hi[i], ss));
        const float rn = rsqrtf(row_sum<D>(ss) * (1.f / D) + a.eps);
        float w[8];
        read8(w_s + t * D + L.lo, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) lo[i] *= rn * w[i];
        read8(w_s + t * D + L.hi, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) hi[i] *= rn * w[i];
        if constexpr (ANY)
          rotate_any<D, false>(a, rows_s + slot * D, L, ang.c[r.tok], ang.s[r.tok], lo, hi);
        else
          rotate<D, false>(a, L, ang.c[r.tok], ang.s[r.tok], lo, hi);
        if (live) {
          store8<DT>(X.y + at(r, X.ys), L.lo, lo);
          store8<DT>(X.y + at(r, X.ys), L.hi, hi);
        }
      }
    }
  }
}

// The gradient, in the same way, one tensor after the other: a lane adds up the weights'
// gradients of its channels, and each CTA leaves one partial sum for each tensor.
template <int D, int DT, bool ANY>
__global__ void __launch_bounds__(kThreads, 2) qk_norm_rope_bwd_kernel(const QkArgs a, const bool w_f32) {
  constexpr int LPR = D / 16, ROWS = kThreads / LPR, WARPS = kThreads / 32;
  __shared__ __align__(16) Angles<D> ang;
  __shared__ __align__(16) float w_s[2 * D];
  __shared__ float rows_s[ANY ? ROWS * D : 1];
  __shared__ float red[WARPS][D];
  const int slot = threadIdx.x / LPR, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Lane L = lane_channels<D, ANY>(a, threadIdx.x % LPR);
  weights_to_shared<DT>(a, w_f32, D, w_s);
  const Run run = run_of(a);
#pragma unroll 1
  for (int t = 0; t < 2; ++t) {
    const Tensor X = tensor_of<DT>(a, t);
    float acc[16] = {};
    for (int t0 = run.first; t0 < run.last; t0 += run.chunk) {
      const int nt = min(run.chunk, run.last - t0), rows = nt * X.H;
      Raw8<DT> rl, rh, sl, sh;
      rl.zero();
      rh.zero();
      sl.zero();
      sh.zero();
      Row next = row_of(a, X, t0, min(slot, rows - 1));
      auto load = [&]() {
        rl.load(X.x + at(next, X.xs), L.lo);
        rh.load(X.x + at(next, X.xs), L.hi);
        sl.load(X.dy + at(next, X.ds), L.lo);
        sh.load(X.dy + at(next, X.ds), L.hi);
      };
      if (slot < rows) load();
      __syncthreads();  // the angles before have been used
      form_angles<D>(a, t0, nt, ang);
      __syncthreads();
      for (int i0 = 0; i0 < rows; i0 += ROWS) {
        const Row r = next;
        const bool live = i0 + slot < rows;
        float lo[8], hi[8], gl[8], gh[8];
        rl.get(lo);
        rh.get(hi);
        sl.get(gl);
        sh.get(gh);
        if (i0 + ROWS + slot < rows) {
          next = row_of(a, X, t0, i0 + ROWS + slot);
          load();
        }
        if constexpr (ANY)
          rotate_any<D, true>(a, rows_s + slot * D, L, ang.c[r.tok], ang.s[r.tok], gl, gh);
        else
          rotate<D, true>(a, L, ang.c[r.tok], ang.s[r.tok], gl, gh);
        float ss = 0.f, sd = 0.f;
        float w[8];
        read8(w_s + t * D + L.lo, w);
        const float* wh = w_s + t * D + L.hi;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(lo[i], lo[i], fmaf(hi[i], hi[i], ss));
          sd = fmaf(gl[i] * w[i], lo[i], fmaf(gh[i] * wh[i], hi[i], sd));
        }
        const float rn = rsqrtf(row_sum<D>(ss) * (1.f / D) + a.eps);
        const float m = row_sum<D>(sd) * (1.f / D) * rn * rn;  // mean(dn h) r: what x takes off dn
        const float in_sum = live ? rn : 0.f;  // a slot without a row holds an earlier one's values
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[i] = fmaf(gl[i], lo[i] * in_sum, acc[i]);
          acc[8 + i] = fmaf(gh[i], hi[i] * in_sum, acc[8 + i]);
          lo[i] = rn * (gl[i] * w[i] - lo[i] * m);
          hi[i] = rn * (gh[i] * wh[i] - hi[i] * m);
        }
        if (live) {
          store8<DT>(X.y + at(r, X.ys), L.lo, lo);
          store8<DT>(X.y + at(r, X.ys), L.hi, hi);
        }
      }
    }
    __syncthreads();  // red of the tensor before has been read
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
      a.part[((size_t)blockIdx.x * 2 + t) * D + threadIdx.x] = v;
    }
  }
}

// dw: the partial sums of all CTAs, in a fixed order.  One CTA per 32 channels.
__global__ void __launch_bounds__(1024) qk_dw_kernel(const QkArgs a, const int ctas, const int D) {
  __shared__ float red[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float v = 0.f;
#pragma unroll 4
  for (int c = row; c < ctas; c += 32) v += a.part[(size_t)c * 2 * D + col];
  red[row][lane] = v;
  __syncthreads();
  if (row == 0) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][lane];
    (col < D ? a.dw[0] : a.dw[1])[col < D ? col : col - D] = s;
  }
}

template <int D, int DT>
cudaError_t launch_d(const QkArgs& a, bool w_f32, bool bwd, cudaStream_t s) {
  const bool any = !a.interleaved && a.rot % 16 != 0;
  if (a.ctas > 0) {
    if (bwd) {
      if (any)
        qk_norm_rope_bwd_kernel<D, DT, true><<<a.ctas, kThreads, 0, s>>>(a, w_f32);
      else
        qk_norm_rope_bwd_kernel<D, DT, false><<<a.ctas, kThreads, 0, s>>>(a, w_f32);
    } else {
      if (any)
        qk_norm_rope_kernel<D, DT, true><<<a.ctas, kThreads, 0, s>>>(a, w_f32);
      else
        qk_norm_rope_kernel<D, DT, false><<<a.ctas, kThreads, 0, s>>>(a, w_f32);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (!bwd) return cudaSuccess;
  // launched with the first kernel, whose end it waits for on the GPU
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * D / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.ctas > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, qk_dw_kernel, a, a.ctas, D);
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
