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
// Each CTA takes an equal run of rows (backward: of tokens), a few CTAs per SM, and walks them
// token by token (a token's heads lie side by side in the projection); the coming rows are
// on their way into shared memory, each lane's own chunks at its own place, so that no
// barrier is needed; the angles of a run's tokens are formed once for all their heads.
//
// The angle is exact at any position: position * freqs[i] mod 2^64 is the phase in
// 2^-64 turns, of which the leading 32 bits, signed, are taken to fp32 (an error of
// at most 2^-25 of half a turn).
#include "ops.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int align16(int n) { return (n + 15) / 16 * 16; }

// Eight elements, as loaded and as fp32; in fp32 two words `step` elements apart.
template <int DT>
struct Raw8 {
  uint4 u[DT == FA_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const char* at, int step) {
#pragma unroll
    for (int i = 0; i < (DT == FA_F32 ? 2 : 1); ++i) u[i] = *reinterpret_cast<const uint4*>(at + 4 * i * step);
  }
  // as four pairs for packed fp32 arithmetic
  __device__ __forceinline__ void get(uint64_t (&v)[4]) const {
    if constexpr (DT == FA_F32) {
      v[0] = f2pack(__uint_as_float(u[0].x), __uint_as_float(u[0].y));
      v[1] = f2pack(__uint_as_float(u[0].z), __uint_as_float(u[0].w));
      v[2] = f2pack(__uint_as_float(u[1].x), __uint_as_float(u[1].y));
      v[3] = f2pack(__uint_as_float(u[1].z), __uint_as_float(u[1].w));
    } else {
      const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<DT == FA_F16>(w[i]);
        v[i] = f2pack(f.x, f.y);
      }
    }
  }
};
template <int DT>
__device__ __forceinline__ void store8(char* p, int step, const uint64_t (&v)[4]) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2unpack(v[i], f[2 * i], f[2 * i + 1]);
  if constexpr (DT == FA_F32) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4 * step) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    constexpr bool F16 = DT == FA_F16;
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack2<F16>(f[0], f[1]), pack2<F16>(f[2], f[3]), pack2<F16>(f[4], f[5]), pack2<F16>(f[6], f[7]));
  }
}
__device__ __forceinline__ uint64_t fsub2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fdup(float x) { return f2pack(x, x); }
__device__ __forceinline__ float fsum2(uint64_t v) {
  float x, y;
  f2unpack(v, x, y);
  return x + y;
}

// cos and sin of a chunk's tokens, [token][pair], in shared memory; with ANY by channel,
// the sine with its sign, and (1, 0) behind the rotated channels.
template <int D, bool ANY>
struct Angles {
  static constexpr int W = ANY ? D : D / 2;
  float *c, *s;
  __device__ __forceinline__ Angles(char* smem, int chunk)
      : c(reinterpret_cast<float*>(smem)), s(reinterpret_cast<float*>(smem) + chunk * W) {}
  __device__ __forceinline__ const float* cos_of(int tok) const { return c + tok * W; }
  __device__ __forceinline__ const float* sin_of(int tok) const { return s + tok * W; }
};
template <int D, bool ANY>
__device__ __forceinline__ void form_angles(const QkArgs& a, int token0, int n, const Angles<D, ANY>& out) {
  const int pairs = a.rot / 2;
  for (int e = threadIdx.x; e < n * (D / 2); e += kThreads) {
    const int tok = e / (D / 2), pair = e % (D / 2);
    float *c = out.c + tok * out.W, *s = out.s + tok * out.W;
    if (pair >= pairs) {
      if constexpr (ANY) {
        c[2 * pair] = c[2 * pair + 1] = 1.f;
        s[2 * pair] = s[2 * pair + 1] = 0.f;
      }
      continue;
    }
    const int t = token0 + tok, b = a.divN.div(t), i = t - b * a.N;
    const int pos = a.pos ? __ldg(a.pos + b * a.pos_stride + i) : i;
    const unsigned long long ph = (unsigned long long)(long long)pos * __ldg(a.freqs + pair);
    // signed leading 32 bits: the phase in 2^-32 turns; in half turns for sincospi
    float sn, cs;
    sincospif((float)(int)(ph >> 32) * 4.656612873077393e-10f, &sn, &cs);
    c[pair] = cs;
    s[pair] = ANY ? -sn : sn;
    if constexpr (ANY) {
      c[pair + pairs] = cs;
      s[pair + pairs] = sn;
    }
  }
}

// Which channels a lane holds: eight from lo and eight from hi on (in fp32 two words of four
// each, `step` apart), so that every access of a row's lanes is to neighbouring words.  With
// rot % 16 == 0 the rotated channels and those behind them have lanes of their own, and
// element e of lo is paired with element e of hi; interleaved pairs are neighbours anyway,
// and `on` has a bit for each of the lane's eight pairs that is rotated.
struct Lane {
  int lo, hi, step;
  uint32_t on;
};

template <int D, int DT, bool ANY>
__device__ __forceinline__ Lane lane_channels(const QkArgs& a, int j) {
  constexpr int LPR = D / 16, WORD = DT == FA_F32 ? 4 : 8;
  const bool split = !ANY && !a.interleaved;
  const int q = split ? a.rot / 16 : LPR;  // lanes of the rotated channels
  const bool behind = j >= q;
  const int n = behind ? LPR - q : q;
  Lane L;
  L.lo = (behind ? 16 * q : 0) + WORD * (behind ? j - q : j);
  L.hi = L.lo + 8 * n;
  L.step = DT == FA_F32 ? 4 * n : 4;
  L.on = split && !behind ? 0xFFu : 0u;
  if (a.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ch = (i & 1) * 2 + (i >> 1) * L.step;
      L.on |= (uint32_t)(L.lo + ch < a.rot) << i;
      L.on |= (uint32_t)(L.hi + ch < a.rot) << (4 + i);
    }
  }
  return L;
}

// Rotates the lane's pairs (back with BACK).
template <bool BACK>
__device__ __forceinline__ void rotate(const QkArgs& a, const Lane& L, const float* c_row, const float* s_row,
                                       uint64_t (&lo)[4], uint64_t (&hi)[4]) {
  if (L.on == 0) return;
  uint64_t c[4], s[4];
  if (a.interleaved) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int pair = ((k < 2 ? L.lo : L.hi) + (k & 1) * L.step) / 2;
      c[k] = *reinterpret_cast<const uint64_t*>(c_row + pair);
      s[k] = *reinterpret_cast<const uint64_t*>(s_row + pair);
    }
    float cf[8], sf[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f2unpack(c[i], cf[2 * i], cf[2 * i + 1]);
      f2unpack(s[i], sf[2 * i], sf[2 * i + 1]);
    }
    auto turn = [&](uint64_t& x, int i) {
      float u, v;
      f2unpack(x, u, v);
      const float sn = BACK ? -sf[i] : sf[i];
      x = f2pack(u * cf[i] - v * sn, u * sn + v * cf[i]);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((L.on >> i) & 1u) turn(lo[i], i);
      if ((L.on >> (4 + i)) & 1u) turn(hi[i], 4 + i);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(c_row + L.lo + k * L.step);
      const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(s_row + L.lo + k * L.step);
      c[2 * k] = u.x;
      c[2 * k + 1] = u.y;
      s[2 * k] = v.x;
      s[2 * k + 1] = v.y;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t uc = fmul2(lo[i], c[i]), us = fmul2(lo[i], s[i]);
      lo[i] = BACK ? ffma2(hi[i], s[i], uc) : fsub2(uc, fmul2(hi[i], s[i]));
      hi[i] = BACK ? fsub2(fmul2(hi[i], c[i]), us) : ffma2(hi[i], c[i], us);
    }
  }
}

// A rotated range whose halves are no whole chunks (rot % 16 != 0, pairs i and
// i + rot / 2): the row goes through shared memory and every element finds its
// partner there.  Four words are left free after each 32 and one after each row, so that
// the lanes of a warp, 8 channels apart, meet different banks (with the rows packed the
// forward pass of 64 + 16 heads, N = 19735, d = 64 took 276 us, and 121 so).  All lanes of
// the row's group call it.
template <int D>
struct AnyRow {
  static constexpr int stride = D + D / 32 * 4 + 1;  // floats
  static __device__ __forceinline__ int at(int ch) { return ch + (ch >> 5) * 4; }
};
template <int D, bool BACK>
__device__ __forceinline__ void rotate_any(const QkArgs& a, float* row, const Lane& L, const float* c_row,
                                           const float* s_row, uint64_t (&lo)[4], uint64_t (&hi)[4]) {
  using R = AnyRow<D>;
  __syncwarp();
  const int half = a.rot / 2;
  auto channel = [&](int i) { return (i < 4 ? L.lo : L.hi) + (i & 1) * 2 + ((i >> 1) & 1) * L.step; };
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float* p = row + R::at(channel(i));
    f2unpack(i < 4 ? lo[i & 3] : hi[i & 3], p[0], p[1]);
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int ch = channel(2 * k);
    const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(c_row + ch);
    const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(s_row + ch);
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int x = ch + e, partner = x < half ? x + half : x - half;
      v[e] = x < a.rot ? row[R::at(partner)] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint64_t& x = (k < 2 ? lo : hi)[2 * (k & 1) + e];
      const uint64_t y = fmul2(f2pack(v[2 * e], v[2 * e + 1]), e ? s.y : s.x), z = fmul2(x, e ? c.y : c.x);
      x = BACK ? fsub2(z, y) : fadd2(z, y);
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

// A row: tensor (0: queries, 1: keys), the token's place in the chunk, batch, token, head.
struct Row {
  int t, tok, b, n, h;
};
// Row i of a chunk, token by token: queries' heads, then keys' (t < 0), or those of tensor t.
__device__ __forceinline__ Row row_of(const QkArgs& a, int t, int token0, int i) {
  Row r;
  if (t >= 0) {
    r.t = t;
    r.tok = (t ? a.divH[1] : a.divH[0]).div(i);
    r.h = i - r.tok * (t ? a.Hk : a.Hq);
  } else {
    r.tok = a.divAll.div(i);
    r.h = i - r.tok * (a.Hq + a.Hk);
    r.t = r.h >= a.Hq;
    if (r.t) r.h -= a.Hq;
  }
  r.b = a.divN.div(token0 + r.tok);
  r.n = token0 + r.tok - r.b * a.N;
  return r;
}
// Its address in a pair of tensors with byte strides {batch, token, head}.
template <typename P>
__device__ __forceinline__ P row_at(const Row& r, P const (&base)[2], const long long (&sb)[2], const int (&sn)[2],
                                    const int (&sh)[2]) {
  return (r.t ? base[1] : base[0]) + r.b * (r.t ? sb[1] : sb[0]) + (long long)r.n * (r.t ? sn[1] : sn[0]) +
         (long long)r.h * (r.t ? sh[1] : sh[0]);
}

// A lane's eight weights from channel c on, as pairs.
template <int DT>
__device__ __forceinline__ void weights8(const void* w, bool w_f32, int c, int step, uint64_t (&v)[4]) {
  if (w_f32) {
    Raw8<FA_F32> r;
    r.load(static_cast<const char*>(w) + 4 * c, step);
    r.get(v);
  } else {
    Raw8<DT> r;
    r.load(static_cast<const char*>(w) + (DT == FA_F32 ? 4 : 2) * c, step);
    r.get(v);
  }
}

// Tokens [first, last) of the CTA, and chunks over them: of equal size, whole turns of rows
// where a chunk may have as many tokens (which fills the turns of a single head, too).
struct Run {
  int first, last, chunk;
};
__device__ __forceinline__ Run run_of(int first, int last, int most, int turn) {
  Run r{first, last, 1};
  const int n = r.last - r.first, chunks = (n + most - 1) / most;
  if (chunks) r.chunk = (n + chunks - 1) / chunks;
  if (chunks > 1 && most >= turn) r.chunk = min(most / turn, (r.chunk + turn - 1) / turn) * turn;
  return r;
}

// Rows on their way: kAhead turns of N chunks of eight elements for each lane, 16 bytes of
// each lane side by side.
template <int DT, int N>
struct Feed {
  static constexpr int V = DT == FA_F32 ? 2 : 1;     // 16-byte words of a chunk
  static constexpr int kAhead = DT == FA_F32 ? 2 : 3;
  static constexpr int bytes = kAhead * N * V * kThreads * 16;
  uint32_t base;  // this lane's first word
  __device__ __forceinline__ explicit Feed(char* smem) : base(smem_addr(smem) + threadIdx.x * 16) {
    // a slot without a row works on zeros or an earlier row's values: never on garbage
    for (int i = 0; i < kAhead * N * V; ++i) st_shared_v4(base + i * kThreads * 16, 0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(int turn, int chunk, const char* src, int step) const {
#pragma unroll
    for (int v = 0; v < V; ++v)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(base + ((turn * N + chunk) * V + v) * kThreads * 16),
                   "l"(src + 4 * v * step)
                   : "memory");
  }
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // all but the last kAhead - 1 turns have arrived
  static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory"); }
  __device__ __forceinline__ void get(int turn, int chunk, uint64_t (&x)[4]) const {
    Raw8<DT> r;
#pragma unroll
    for (int v = 0; v < V; ++v) r.u[v] = ld_shared_v4(base + ((turn * N + chunk) * V + v) * kThreads * 16);
    r.get(x);
  }
};

template <bool ANY, bool BWD>
constexpr int kCtasPerSm = BWD ? 2 : ANY ? 3 : 4;

// Shared memory: the weights in fp32 (forward), rows for rotate_any, the feed, and the angles
// of as many tokens as the rest of a CTA's part of the SM holds, 64 at most (128 at d = 64).
template <int D, int DT, bool ANY, bool BWD>
struct Smem {
  static constexpr int ctas = kCtasPerSm<ANY, BWD>;
  static constexpr int rows = BWD ? 0 : 2 * D * 4;  // behind the weights
  static constexpr int feed = align16(rows + (ANY ? kThreads / (D / 16) * AnyRow<D>::stride * 4 : 0));
  static constexpr int angles = feed + Feed<DT, BWD ? 4 : 2>::bytes;
  static constexpr int token = 2 * Angles<D, ANY>::W * 4;
  static constexpr int room = (228 * 1024 / ctas - 1024 - (BWD ? 2 * (kThreads / 32) * D * 4 : 0) - angles) / token;
  static constexpr int most = 64 * 128 / D;
  static constexpr int chunk = room < most ? room : most;
  static constexpr int bytes = angles + chunk * token;
  static_assert(chunk >= 16, "angles of a chunk");
};

// The forward pass.  Measured: 23,400 tokens of 12 + 12 heads, d = 64, bf16 26.5 us (144 MB,
// 5.4 TB/s; three CTAs an SM 27.3 us), of which about 3 are the launch, the angles and the
// first rows; 19,735 tokens of 64 + 16 heads, d = 64, fp32 142 us (808 MB, 5.7
// TB/s; 137 with 34 of the channels rotated, which go through shared memory).
template <int D, int DT, bool ANY>
__global__ void __launch_bounds__(kThreads, Smem<D, DT, ANY, false>::ctas) qk_norm_rope_kernel(const QkArgs a, const bool w_f32) {
  constexpr int LPR = D / 16, ROWS = kThreads / LPR, E = DT == FA_F32 ? 4 : 2;
  using S = Smem<D, DT, ANY, false>;
  extern __shared__ __align__(16) char smem[];
  const Angles<D, ANY> ang(smem + S::angles, S::chunk);
  float* w_s = reinterpret_cast<float*>(smem);
  const Feed<DT, 2> feed(smem + S::feed);
  constexpr int AHEAD = Feed<DT, 2>::kAhead;
  const int slot = threadIdx.x / LPR;
  float* row_s = reinterpret_cast<float*>(smem + S::rows) + slot * AnyRow<D>::stride;
  Lane L = lane_channels<D, DT, ANY>(a, threadIdx.x % LPR);
  if (DT != FA_F32) L.step = 4;
  for (int e = threadIdx.x; e < 2 * D / 8; e += kThreads) {
    uint64_t v[4];
    weights8<DT>(e < D / 8 ? a.w[0] : a.w[1], w_f32, 8 * (e % (D / 8)), 4, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<uint64_t*>(w_s)[4 * e + i] = v[i];
  }
  // an equal share of all rows, which may begin and end inside a token: rows [skip, stop) from
  // its first token on
  const int H = a.Hq + a.Hk;
  const long long row0 = a.share * blockIdx.x + min((int)blockIdx.x, a.spare);
  const long long row1 = row0 + a.share + ((int)blockIdx.x < a.spare);
  auto token_of = [&](long long row) { return row < (1ll << 31) ? a.divAll.div((int)row) : (int)(row / H); };
  const Run run = run_of(token_of(row0), token_of(row1 - 1) + 1, S::chunk, ROWS);
  const int skip = (int)(row0 - (long long)run.first * H), stop = (int)(row1 - (long long)run.first * H);
  // the rows to load next, of the chunk that starts at token lt: they run ahead of the
  // chunk whose rows are worked on
  int lt = run.first, li = skip;
  auto load = [&](int place) {
    const int rows = min(run.chunk * H, stop - (lt - run.first) * H), i = li + slot;
    if (i < rows) {
      const char* p = row_at(row_of(a, -1, lt, i), a.x, a.xb, a.xn, a.xh);
      feed.load(place, 0, p + L.lo * E, L.step);
      feed.load(place, 1, p + L.hi * E, L.step);
    }
    feed.commit();
    li += ROWS;
    if (li >= rows) {
      li = 0;
      lt = min(lt + run.chunk, run.last);
    }
  };
#pragma unroll
  for (int k = 0; k < AHEAD - 1; ++k) load(k);
  int turn = 0;
  for (int t0 = run.first; t0 < run.last; t0 += run.chunk) {
    const int nt = min(run.chunk, run.last - t0), before = (t0 - run.first) * H, rows = min(nt * H, stop - before);
    __syncthreads();  // the angles before have been used
    form_angles(a, t0, nt, ang);
    __syncthreads();
    // every lane of a warp takes the same number of turns: the row sums are shuffles
    for (int i0 = max(skip - before, 0); i0 < rows; i0 += ROWS) {
      const bool live = i0 + slot < rows;
      const Row r = row_of(a, -1, t0, min(i0 + slot, rows - 1));
      load(turn == 0 ? AHEAD - 1 : turn - 1);
      feed.wait();
      uint64_t lo[4], hi[4];
      feed.get(turn, 0, lo);
      feed.get(turn, 1, hi);
      turn = turn + 1 == AHEAD ? 0 : turn + 1;
      uint64_t ss = fmul2(lo[0], lo[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) ss = ffma2(lo[i], lo[i], ss);
#pragma unroll
      for (int i = 0; i < 4; ++i) ss = ffma2(hi[i], hi[i], ss);
      const uint64_t rn = fdup(rsqrtf(row_sum<D>(fsum2(ss)) * (1.f / D) + a.eps));
      const float *wl = w_s + r.t * D + L.lo, *wh = w_s + r.t * D + L.hi;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(wl + i * L.step),
                         v = *reinterpret_cast<const ulonglong2*>(wh + i * L.step);
        lo[2 * i] = fmul2(fmul2(lo[2 * i], rn), u.x);
        lo[2 * i + 1] = fmul2(fmul2(lo[2 * i + 1], rn), u.y);
        hi[2 * i] = fmul2(fmul2(hi[2 * i], rn), v.x);
        hi[2 * i + 1] = fmul2(fmul2(hi[2 * i + 1], rn), v.y);
      }
      if constexpr (ANY)
        rotate_any<D, false>(a, row_s, L, ang.cos_of(r.tok), ang.sin_of(r.tok), lo, hi);
      else
        rotate<false>(a, L, ang.cos_of(r.tok), ang.sin_of(r.tok), lo, hi);
      if (live) {
        char* p = row_at(r, a.y, a.yb, a.yn, a.yh);
        store8<DT>(p + L.lo * E, L.step, lo);
        store8<DT>(p + L.hi * E, L.step, hi);
      }
    }
  }
}

// The gradient, in the same way; of a chunk first the queries' rows, then the keys' (both
// token by token in one loop, with the sums of both, measured 10% slower): a lane adds up the
// weights' gradients of its channels, its warp's sums are kept in shared memory from one
// change of tensor to the next, and each CTA leaves one partial sum for each tensor.
// Measured: 2 x 16384 tokens of 16 + 16 heads, d = 128, bf16 127 us (805 MB, 6.3 TB/s, 94% of a
// copy); 4 x 2048 of 12 + 12, d = 64, 20 us (75 MB), of which start-up, angles and the
// weights' sums are 8.
template <int D, int DT, bool ANY>
__global__ void __launch_bounds__(kThreads, Smem<D, DT, ANY, true>::ctas) qk_norm_rope_bwd_kernel(const QkArgs a, const bool w_f32) {
  constexpr int LPR = D / 16, ROWS = kThreads / LPR, WARPS = kThreads / 32, E = DT == FA_F32 ? 4 : 2;
  using S = Smem<D, DT, ANY, true>;
  extern __shared__ __align__(16) char smem[];
  __shared__ float red[2][WARPS][D];
  const Angles<D, ANY> ang(smem + S::angles, S::chunk);
  const Feed<DT, 4> feed(smem + S::feed);
  constexpr int AHEAD = Feed<DT, 4>::kAhead;
  const int slot = threadIdx.x / LPR, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row_s = reinterpret_cast<float*>(smem + S::rows) + slot * AnyRow<D>::stride;
  Lane L = lane_channels<D, DT, ANY>(a, threadIdx.x % LPR);
  if (DT != FA_F32) L.step = 4;
  const long long T = (long long)a.B * a.N;
  const Run run = run_of((int)(T * blockIdx.x / gridDim.x), (int)(T * (blockIdx.x + 1) / gridDim.x), S::chunk, ROWS);
  for (int e = lane; e < 2 * D; e += 32) red[e / D][warp][e % D] = 0.f;
  __syncwarp();
  // the rows to load next: of tensor ltn in the chunk that starts at token lt
  int lt = run.first, ltn = 0, li = 0;
  auto load = [&](int place) {
    const int rows = min(run.chunk, run.last - lt) * (ltn ? a.Hk : a.Hq), i = li + slot;
    if (i < rows) {
      const Row r = row_of(a, ltn, lt, i);
      const char *p = row_at(r, a.x, a.xb, a.xn, a.xh), *q = row_at(r, a.dy, a.db, a.dn, a.dh);
      feed.load(place, 0, p + L.lo * E, L.step);
      feed.load(place, 1, p + L.hi * E, L.step);
      feed.load(place, 2, q + L.lo * E, L.step);
      feed.load(place, 3, q + L.hi * E, L.step);
    }
    feed.commit();
    li += ROWS;
    if (li >= rows) {
      li = 0;
      if (ltn) lt = min(lt + run.chunk, run.last);
      ltn ^= 1;
    }
  };
#pragma unroll
  for (int k = 0; k < AHEAD - 1; ++k) load(k);
  int place = 0;
  for (int t0 = run.first; t0 < run.last; t0 += run.chunk) {
    const int nt = min(run.chunk, run.last - t0);
    __syncthreads();  // the angles before have been used
    form_angles(a, t0, nt, ang);
    __syncthreads();
    for (int t = 0; t < 2; ++t) {
      const int rows = nt * (t ? a.Hk : a.Hq);
      uint64_t wl[4], wh[4], acc[8];
      weights8<DT>(t ? a.w[1] : a.w[0], w_f32, L.lo, L.step, wl);
      weights8<DT>(t ? a.w[1] : a.w[0], w_f32, L.hi, L.step, wh);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = 0;
#pragma unroll 1
      for (int i0 = 0; i0 < rows; i0 += ROWS) {
        const bool live = i0 + slot < rows;
        const Row r = row_of(a, t, t0, min(i0 + slot, rows - 1));
        load(place == 0 ? AHEAD - 1 : place - 1);
        feed.wait();
        uint64_t lo[4], hi[4], gl[4], gh[4];
        feed.get(place, 0, lo);
        feed.get(place, 1, hi);
        feed.get(place, 2, gl);
        feed.get(place, 3, gh);
        place = place + 1 == AHEAD ? 0 : place + 1;
        if constexpr (ANY)
          rotate_any<D, true>(a, row_s, L, ang.cos_of(r.tok), ang.sin_of(r.tok), gl, gh);
        else
          rotate<true>(a, L, ang.cos_of(r.tok), ang.sin_of(r.tok), gl, gh);
        uint64_t ss = 0, sd = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          ss = ffma2(lo[k], lo[k], ffma2(hi[k], hi[k], ss));
          sd = ffma2(fmul2(gl[k], wl[k]), lo[k], ffma2(fmul2(gh[k], wh[k]), hi[k], sd));
        }
        const float rn = rsqrtf(row_sum<D>(fsum2(ss)) * (1.f / D) + a.eps);
        const float m = row_sum<D>(fsum2(sd)) * (1.f / D) * rn * rn;  // mean(dn h) r: what x takes off dn
        const uint64_t rn2 = fdup(rn), m2 = fdup(-m);
        if (live) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            acc[k] = ffma2(gl[k], fmul2(lo[k], rn2), acc[k]);
            acc[4 + k] = ffma2(gh[k], fmul2(hi[k], rn2), acc[4 + k]);
            lo[k] = fmul2(rn2, ffma2(lo[k], m2, fmul2(gl[k], wl[k])));
            hi[k] = fmul2(rn2, ffma2(hi[k], m2, fmul2(gh[k], wh[k])));
          }
          char* p = row_at(r, a.y, a.yb, a.yn, a.yh);
          store8<DT>(p + L.lo * E, L.step, lo);
          store8<DT>(p + L.hi * E, L.step, hi);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float v[2];
        f2unpack(acc[k], v[0], v[1]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int off = LPR; off < 32; off <<= 1) v[c] += __shfl_xor_sync(0xffffffffu, v[c], off);
          if (lane < LPR) red[t][warp][(k < 4 ? L.lo : L.hi) + ((k >> 1) & 1) * L.step + 2 * (k & 1) + c] += v[c];
        }
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < 2 * D) {
    const int t = threadIdx.x / D, ch = threadIdx.x % D;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v += red[t][w][ch];
    a.part[((size_t)blockIdx.x * 2 + t) * D + ch] = v;
  }
}

// dw: the partial sums of all CTAs, in a fixed order.  One CTA per 32 channels.  It is a
// dependent launch of the kernel before, but that one does not let it start early
// (griddepcontrol.launch_dependents): it starts at its end (5.8 us by itself).
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

template <typename K>
cudaError_t launch_one(K kernel, int smem, const QkArgs& a, bool w_f32, cudaStream_t s) {
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<a.ctas, kThreads, smem, s>>>(a, w_f32);
  return cudaGetLastError();
}

template <int D, int DT>
cudaError_t launch_d(const QkArgs& a, bool w_f32, bool bwd, cudaStream_t s) {
  const bool any = a.any;
  if (a.ctas > 0) {
    const cudaError_t e =
        bwd ? (any ? launch_one(qk_norm_rope_bwd_kernel<D, DT, true>, Smem<D, DT, true, true>::bytes, a, w_f32, s)
                   : launch_one(qk_norm_rope_bwd_kernel<D, DT, false>, Smem<D, DT, false, true>::bytes, a, w_f32, s))
            : (any ? launch_one(qk_norm_rope_kernel<D, DT, true>, Smem<D, DT, true, false>::bytes, a, w_f32, s)
                   : launch_one(qk_norm_rope_kernel<D, DT, false>, Smem<D, DT, false, false>::bytes, a, w_f32, s));
    if (e != cudaSuccess) return e;
  }
  if (!bwd) return cudaSuccess;
  // a dependent launch: it starts at the first kernel's end, and waits for it besides
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

int qk_ctas_per_sm(bool any, bool bwd) {
  return bwd ? kCtasPerSm<false, true> : any ? kCtasPerSm<true, false> : kCtasPerSm<false, false>;
}
int qk_rows_per_pass(int d) { return kThreads / (d / 16); }

cudaError_t launch_qk_norm_rope(const QkArgs& a, int d, int dtype, bool w_f32, cudaStream_t s) {
  return launch(a, d, dtype, w_f32, false, s);
}
cudaError_t launch_qk_norm_rope_bwd(const QkArgs& a, int d, int dtype, bool w_f32, cudaStream_t s) {
  return launch(a, d, dtype, w_f32, true, s);
}

}  // namespace fa
