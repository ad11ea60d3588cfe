// ops.h -- declarations shared by the entry points of the operators around the
// attention (ops_api.cu) and their kernels.  Not part of the public interface.
#pragma once
#include "internal.h"

namespace fa {

// Quotients by a fixed divisor of numbers below 2^31: a multiplication, an addition and a
// shift (with s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1).
struct FastDiv {
  uint32_t d, m, s;
  static FastDiv of(uint32_t d) {
    FastDiv f{d, 0, 0};
    while ((1ull << f.s) < d) ++f.s;
    f.m = (uint32_t)(((1ull << 32) * ((1ull << f.s) - d)) / d + 1);
    return f;
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int div(int n) const { return (int)((__umulhi((uint32_t)n, m) + (uint32_t)n) >> s); }
#endif
};

// Norm and rotation of query and key heads (qk_norm_rope.cu).
struct QkArgs {
  int B, N, Hq, Hk;
  int rot, interleaved;
  int any;  // rotate through shared memory
  float eps;
  const char* x[2];   // q, k
  const void* w[2];   // wq, wk
  char* y[2];         // forward: results; backward: gradients of q, k
  const char* dy[2];  // backward: gradients at the results
  // byte strides between batch entries, tokens and heads of x, y, dy
  long long xb[2], yb[2], db[2];
  int xn[2], xh[2], yn[2], yh[2], dn[2], dh[2];
  const unsigned long long* freqs;
  const int* pos;  // or nullptr
  long long pos_stride;
  FastDiv divN, divH[2], divAll;  // by N, Hq and Hk, their sum
  int ctas;
  long long share;  // forward: rows of a CTA; the first `spare` CTAs have one more
  int spare;
  float* part;    // backward: [CTA][2][d] partial weight gradients
  float* dw[2];
};
// CTAs on an SM, rows of a CTA's turn.
int qk_ctas_per_sm(bool any, bool bwd);
int qk_rows_per_pass(int d);
cudaError_t launch_qk_norm_rope(const QkArgs& a, int d, int dtype, bool w_f32, cudaStream_t s);
cudaError_t launch_qk_norm_rope_bwd(const QkArgs& a, int d, int dtype, bool w_f32, cudaStream_t s);

// The 4-bit cache (kv4.cuh has its block layout).
struct Kv4Cache {
  const uint8_t* data;
  long long page_stride;  // bytes
  int num_pages, page_log, Hk;  // tokens of a page: 1 << page_log
};
struct Kv4RowArgs {
  Kv4Cache c;
  int rows;       // tokens x heads
  FastDiv heads;
  const int* slots;
  void* x[2];              // keys, values
  int xs[2][2];            // element strides {token, head}
  DevStatus* st;
};
cudaError_t launch_kv4_append(const Kv4RowArgs& a, int d, int dtype, cudaStream_t s);
cudaError_t launch_kv4_gather(const Kv4RowArgs& a, int d, int dtype, cudaStream_t s);

struct Kv4AttnArgs {
  Kv4Cache c;
  int R, T, Hq;
  FastDiv G;  // query heads of a key head
  int window;
  int table_width;
  long long table_stride;
  const int* table;
  const int* kv_lens;
  const int* cu_q;  // or nullptr
  float scale_log2;
  const void* q;
  long long qs[2];  // element strides {token, head}
  void* o;
  long long os[2];
  float* lse;       // or nullptr
  float* part;      // 2 slots per CTA: rows x (d + 2) fp32 each
  int4* meta;       // two per CTA: the tile that starts in its share and goes on
  Report rep;
};
// Rows of a query tile: 8, 16 or 32 (kv4_attn.cuh).
inline int kv4_tile_rows(int G, int max_q_len) {
  const long long rows = (long long)G * max_q_len;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
}
// The CTAs of a launch in shares: one wave.
inline int kv4_share_ctas(int rows, int sms) { return sms * (rows == 8 ? 4 : rows == 16 ? 3 : 2); }
template <int D>
cudaError_t launch_kv4_attention_d(const Kv4AttnArgs& a, bool f16, int rows, int ctas, int cluster, cudaStream_t s);
template <int D>
int kv4_clusters_at_once(int rows, int cluster);

struct PlanArgs {
  int R, T, page, pages, width;
  long long stride;
  const int* seq;
  const int* fresh;
  int* table;
  int* stack;
  const int* count;
  int* kv;
  int* cu;
  int* pos;
  int* slots;
  int* counts;
  bool aliased;  // kv or counts lie over the inputs (set by the launch)
};
cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t s);

}  // namespace fa
