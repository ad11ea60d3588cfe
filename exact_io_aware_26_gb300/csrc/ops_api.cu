// ops_api.cu -- the C ABI of the operators around the attention (include/fa.h): norm
// and rotation of queries and keys, the 4-bit paged cache and its attention, block
// tables and slot maps.  Host code: argument checks, before any CUDA call, and the
// launches.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "kv4.cuh"
#include "ops.h"

#include <nvtx3/nvToolsExt.h>

using namespace fa;

namespace {

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

fa_status fail(fa_status s, const char* fmt, ...) {
  char text[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  set_error_text(text);
  return s;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
long long elem_bytes(int dtype) { return dtype == FA_F32 ? 4 : 2; }

fa_status need(const void* p, size_t align, const char* name) {
  if (!p) return fail(FA_ERR_INVALID, "%s is NULL", name);
  if (!aligned(p, align)) return fail(FA_ERR_INVALID, "%s is not %zu-byte aligned", name, align);
  return FA_OK;
}

// Strides (elements) of a tensor [size[0]][size[1]]...[inner]: whole 16-byte vectors,
// not negative; for a tensor that is written, no two elements in one place.
fa_status check_strides(const long long* stride, const long long* size, int n, long long inner, int dtype, bool written,
                        const char* name) {
  const long long vec = 16 / elem_bytes(dtype);
  int order[3] = {0, 1, 2};
  for (int i = 0; i < n; ++i)
    if (stride[i] < 0 || stride[i] % vec != 0)
      return fail(FA_ERR_INVALID, "%s: stride %lld is negative or no multiple of 16 bytes", name, stride[i]);
  if (!written) return FA_OK;
  for (int i = 0; i < n; ++i)
    if (size[i] == 0) return FA_OK;  // no element
  std::sort(order, order + n, [&](int x, int y) { return stride[x] < stride[y]; });
  long long extent = inner;
  for (int i = 0; i < n; ++i) {
    const int k = order[i];
    if (size[k] <= 1) continue;
    if (stride[k] < extent) return fail(FA_ERR_INVALID, "%s overlaps itself (stride %lld)", name, stride[k]);
    extent = stride[k] * (size[k] - 1) + extent;
  }
  return FA_OK;
}

// ------------------------------------------------------- norm and rotation

fa_status qk_check(const fa_qk_params* p, bool bwd) {
  if (!p) return fail(FA_ERR_INVALID, "params is NULL");
  if (p->B < 1 || p->N < 0 || p->Hq < 1 || p->Hk < 1)
    return fail(FA_ERR_INVALID, "B, Hq, Hk must be >= 1 and N >= 0 (got %d, %d, %d, %d)", p->B, p->Hq, p->Hk, p->N);
  if (p->d != 64 && p->d != 128) return fail(FA_ERR_UNSUPPORTED, "head size %d is not supported (64 or 128)", p->d);
  if (p->dtype != FA_F32 && p->dtype != FA_F16 && p->dtype != FA_BF16)
    return fail(FA_ERR_INVALID, "dtype %d is not an fa_dtype", p->dtype);
  if (p->weight_dtype != p->dtype && p->weight_dtype != FA_F32)
    return fail(FA_ERR_INVALID, "weight_dtype must be dtype or FA_F32");
  if (p->rot_dim < 0 || p->rot_dim > p->d || p->rot_dim % 2 != 0)
    return fail(FA_ERR_INVALID, "rot_dim %d must be even, from 0 to d", p->rot_dim);
  if (!(std::isfinite(p->eps) && p->eps > 0.f)) return fail(FA_ERR_INVALID, "eps must be positive and finite");
  if (p->pos_stride < 0) return fail(FA_ERR_INVALID, "pos_stride is negative");
  // tokens and rows of a chunk are counted in 32 bits
  if ((long long)p->B * p->N >= (1ll << 30) || (long long)p->Hq + p->Hk >= (1 << 24))
    return fail(FA_ERR_UNSUPPORTED, "B*N exceeds 2^30 - 1 or the heads 2^24 - 1");
  for (int i = 1; i < 3; ++i)
    for (const long long* st : {p->q_stride, p->k_stride, p->yq_stride, p->yk_stride, bwd ? p->dq_stride : p->q_stride,
                                bwd ? p->dk_stride : p->k_stride})
      if (st[i] * elem_bytes(p->dtype) > 0x7FFFFFFFll)
        return fail(FA_ERR_UNSUPPORTED, "a token or head stride exceeds 2^31 - 1 bytes");
  const long long sq[3] = {p->B, p->N, p->Hq}, sk[3] = {p->B, p->N, p->Hk};
  FA_TRY(check_strides(p->q_stride, sq, 3, p->d, p->dtype, false, "q"));
  FA_TRY(check_strides(p->k_stride, sk, 3, p->d, p->dtype, false, "k"));
  FA_TRY(check_strides(p->yq_stride, sq, 3, p->d, p->dtype, !bwd, bwd ? "dyq" : "yq"));
  FA_TRY(check_strides(p->yk_stride, sk, 3, p->d, p->dtype, !bwd, bwd ? "dyk" : "yk"));
  if (bwd) {
    FA_TRY(check_strides(p->dq_stride, sq, 3, p->d, p->dtype, true, "dq"));
    FA_TRY(check_strides(p->dk_stride, sk, 3, p->d, p->dtype, true, "dk"));
  }
  return FA_OK;
}

constexpr int kQkMaxSms = 160;

// Byte strides of a pair of tensors.
void qk_strides(const fa_qk_params* p, const long long* q, const long long* k, long long (&b)[2], int (&n)[2], int (&h)[2]) {
  const long long e = elem_bytes(p->dtype);
  for (int t = 0; t < 2; ++t) {
    const long long* s = t ? k : q;
    b[t] = s[0] * e;
    n[t] = (int)(s[1] * e);
    h[t] = (int)(s[2] * e);
  }
}

QkArgs qk_args(const fa_qk_params* p, const void* q, const void* k, const void* wq, const void* wk,
               const uint64_t* freqs, const int* positions, int sms, bool bwd) {
  QkArgs a;
  std::memset(&a, 0, sizeof(a));
  a.B = p->B;
  a.N = p->N;
  a.Hq = p->Hq;
  a.Hk = p->Hk;
  a.rot = p->rot_dim;
  a.interleaved = p->interleaved != 0;
  // Through shared memory where the rotated halves are no whole chunks; and a rotated part of a
  // 64-channel head where a row is read twice or is of 256 bytes, because the halves of the part
  // are read in pieces of 32 bytes then (80 heads, N = 19735, 32 of 64 channels, in registers
  // and through shared memory: bf16 forward 79 and 93 us, backward 122 and 104; fp32 forward
  // 150 and 137, backward 221 and 202.  128 channels, 24 heads, N = 26016: bf16 backward 84 and
  // 104, fp32 alike).
  a.any = !a.interleaved && (p->rot_dim % 16 != 0 || (p->d == 64 && p->rot_dim > 0 && p->rot_dim < 64 &&
                                                      (bwd || p->dtype == FA_F32)));
  a.eps = p->eps;
  a.x[0] = static_cast<const char*>(q);
  a.x[1] = static_cast<const char*>(k);
  a.w[0] = wq;
  a.w[1] = wk;
  a.freqs = reinterpret_cast<const unsigned long long*>(freqs);
  a.pos = positions;
  a.pos_stride = p->pos_stride;
  qk_strides(p, p->q_stride, p->k_stride, a.xb, a.xn, a.xh);
  a.divN = FastDiv::of((uint32_t)std::max(p->N, 1));
  a.divH[0] = FastDiv::of((uint32_t)p->Hq);
  a.divH[1] = FastDiv::of((uint32_t)p->Hk);
  a.divAll = FastDiv::of((uint32_t)(p->Hq + p->Hk));
  // one wave of CTAs, but no more than have a row for each of their row slots
  const long long T = (long long)p->B * p->N, slots = qk_rows_per_pass(p->d);
  const long long rows = T * (p->Hq + p->Hk), least = std::max(1ll, slots / (p->Hq + p->Hk));
  const long long wave = (long long)std::min(sms, kQkMaxSms) * qk_ctas_per_sm(a.any, bwd);
  a.ctas = (int)std::min(wave, bwd ? (T + least - 1) / least : (rows + slots - 1) / slots);
  if (a.ctas > 0) {
    a.share = rows / a.ctas;
    a.spare = (int)(rows % a.ctas);
  }
  return a;
}

fa_status qk_pointers(const fa_qk_params* p, const void* q, const void* k, const void* wq, const void* wk,
                      const uint64_t* freqs, const int* positions) {
  FA_TRY(need(q, 16, "q"));
  FA_TRY(need(k, 16, "k"));
  FA_TRY(need(wq, 16, "wq"));
  FA_TRY(need(wk, 16, "wk"));
  if (p->rot_dim > 0) FA_TRY(need(freqs, 8, "freqs"));
  if (positions && !aligned(positions, 4)) return fail(FA_ERR_INVALID, "positions is not 4-byte aligned");
  return FA_OK;
}

// A result over its own input: rows are read ahead, so every row must stay in its place.
fa_status qk_in_place(const void* x, const void* y, const long long* sx, const long long* sy, const char* name) {
  if (x == y && std::memcmp(sx, sy, 3 * sizeof(long long)) != 0)
    return fail(FA_ERR_INVALID, "%s lies over its input with other strides", name);
  return FA_OK;
}

// ------------------------------------------------------- 4-bit cache

fa_status cache_check(const fa_kv4_cache* c) {
  if (!c) return fail(FA_ERR_INVALID, "cache description is NULL");
  if (c->d != 64 && c->d != 128) return fail(FA_ERR_UNSUPPORTED, "head size %d is not supported (64 or 128)", c->d);
  if (c->num_pages < 1 || c->Hk < 1) return fail(FA_ERR_INVALID, "num_pages and Hk must be >= 1");
  if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)) != 0)
    return fail(FA_ERR_UNSUPPORTED, "page_size %d must be a power of two from 16 to 4096", c->page_size);
  if ((long long)c->num_pages * c->page_size > 0x7FFFFFFFll)
    return fail(FA_ERR_UNSUPPORTED, "num_pages * page_size exceeds 2^31 - 1 slots");
  const long long page = (long long)c->Hk * (c->page_size / 16) * fa_kv4_block_bytes(c->d);
  if (page > 0x7FFFFFFFll) return fail(FA_ERR_UNSUPPORTED, "a page of %lld bytes exceeds 2^31 - 1", page);
  if (c->page_stride < page || c->page_stride % 16 != 0)
    return fail(FA_ERR_INVALID, "page_stride %lld must be a multiple of 16, at least %lld", c->page_stride, page);
  return FA_OK;
}

Kv4Cache cache_args(const fa_kv4_cache* c, const void* data) {
  Kv4Cache k;
  k.data = static_cast<const uint8_t*>(data);
  k.page_stride = c->page_stride;
  k.num_pages = c->num_pages;
  k.page_log = 0;
  while ((1 << k.page_log) < c->page_size) ++k.page_log;
  k.Hk = c->Hk;
  return k;
}

fa_status kv4_rows_call(const fa_kv4_cache* c, const fa_kv4_rows* rows, const void* k, const void* v, const int* slots,
                        const void* cache, bool gather, void* stream) {
  FA_TRY(cache_check(c));
  if (!rows) return fail(FA_ERR_INVALID, "rows is NULL");
  if (rows->T < 0) return fail(FA_ERR_INVALID, "T is negative");
  if ((long long)rows->T * c->Hk >= (1ll << 30)) return fail(FA_ERR_UNSUPPORTED, "T*Hk exceeds 2^30 - 1");
  if (rows->dtype != FA_F32 && rows->dtype != FA_F16 && rows->dtype != FA_BF16)
    return fail(FA_ERR_INVALID, "dtype %d is not an fa_dtype", rows->dtype);
  const long long size[2] = {rows->T, c->Hk};
  for (int i = 0; i < 2; ++i)
    if (rows->k_stride[i] > 0x7FFFFFFFll || rows->v_stride[i] > 0x7FFFFFFFll)
      return fail(FA_ERR_UNSUPPORTED, "a stride of k or v exceeds 2^31 - 1 elements");
  FA_TRY(check_strides(rows->k_stride, size, 2, c->d, rows->dtype, gather, "k"));
  FA_TRY(check_strides(rows->v_stride, size, 2, c->d, rows->dtype, gather, "v"));
  if (rows->T > 0) {
    FA_TRY(need(k, 16, "k"));
    FA_TRY(need(v, 16, "v"));
    FA_TRY(need(slots, 4, "slots"));
  }
  FA_TRY(need(cache, 16, "cache"));
  Report rep;
  FA_TRY(api_device(&rep, nullptr));
  if (rows->T == 0) return FA_OK;
  Kv4RowArgs a;
  std::memset(&a, 0, sizeof(a));
  a.c = cache_args(c, cache);
  a.rows = rows->T * c->Hk;
  a.heads = FastDiv::of((uint32_t)c->Hk);
  a.slots = slots;
  a.x[0] = const_cast<void*>(k);
  a.x[1] = const_cast<void*>(v);
  for (int i = 0; i < 2; ++i) {
    a.xs[0][i] = (int)rows->k_stride[i];
    a.xs[1][i] = (int)rows->v_stride[i];
  }
  a.st = rep.st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = gather ? launch_kv4_gather(a, c->d, rows->dtype, s) : launch_kv4_append(a, c->d, rows->dtype, s);
  if (e != cudaSuccess) return api_cuda_fail(e, gather ? "cache gather launch" : "cache append launch");
  return FA_OK;
}

fa_status attn_check(const fa_kv4_cache* c, const fa_kv4_attn_params* p) {
  FA_TRY(cache_check(c));
  if (!p) return fail(FA_ERR_INVALID, "params is NULL");
  if (p->dtype != FA_F16 && p->dtype != FA_BF16)
    return fail(p->dtype == FA_F32 ? FA_ERR_UNSUPPORTED : FA_ERR_INVALID, "the cache's attention takes fp16 or bf16 queries");
  if (p->R < 1 || p->T < 0) return fail(FA_ERR_INVALID, "R must be >= 1 and T >= 0 (got %d, %d)", p->R, p->T);
  if (p->Hq < 1 || p->Hq % c->Hk != 0)
    return fail(FA_ERR_INVALID, "Hq = %d is no multiple of the cache's %d heads", p->Hq, c->Hk);
  if ((long long)p->T * p->Hq >= (1ll << 31)) return fail(FA_ERR_UNSUPPORTED, "T*Hq exceeds 2^31 - 1");
  if (p->max_q_len < 1) return fail(FA_ERR_INVALID, "max_q_len must be >= 1");
  if (p->window < 0) return fail(FA_ERR_INVALID, "window is negative");
  if (p->table_width < 1 || p->table_stride < p->table_width)
    return fail(FA_ERR_INVALID, "block_table needs at least one column and a row stride of at least its width");
  if ((long long)p->table_width * c->page_size > (1ll << 30))
    return fail(FA_ERR_UNSUPPORTED, "table_width * page_size exceeds 2^30 tokens");
  if (!(std::isfinite(p->scale) && p->scale > 0.f)) return fail(FA_ERR_INVALID, "scale must be positive and finite");
  const long long size[2] = {p->T, p->Hq};
  FA_TRY(check_strides(p->q_stride, size, 2, c->d, p->dtype, false, "q"));
  FA_TRY(check_strides(p->o_stride, size, 2, c->d, p->dtype, true, "o"));
  return FA_OK;
}

constexpr int kMaxSms = 160;

// Tiles of a launch whose requests all have max_q_len rows.
long long kv4_tiles(const fa_kv4_cache* c, const fa_kv4_attn_params* p, int rows) {
  const long long q_rows = (long long)std::min(p->max_q_len, std::max(p->T, 1)) * (p->Hq / c->Hk);
  return (long long)p->R * c->Hk * ((q_rows + rows - 1) / rows);
}

// How many clusters of 1 << log CTAs the current device `dev` holds at once, asked for once.
long long kv4_clusters(int dev, int d, int rows, int log) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][2][3][5];  // number + 1
  if (dev < 0 || dev >= kDevices) return 0;
  std::atomic<int>& k = known[dev][d == 128][rows == 8 ? 0 : rows == 16 ? 1 : 2][log];
  int n = k.load(std::memory_order_relaxed);
  if (n == 0) {
    n = 1 + (d == 64 ? kv4_clusters_at_once<64>(rows, 1 << log) : kv4_clusters_at_once<128>(rows, 1 << log));
    k.store(n, std::memory_order_relaxed);
  }
  return n - 1;
}

// CTAs of a cluster (8 warps each) for a tile, as many as lets one wave hold all tiles; 0 for
// the way in shares: with more tiles than that, or where even shares would save a warp more
// units of 32 tokens (for requests as long as the block table has room for) than the second
// launch costs, two of them at d = 64 and one at d = 128.  Measured, in clusters and in
// shares: d = 64, 12 tiles of 16384 tokens 12.7 and 15.0 us (4 units a warp and 3), of 24576
// 14.9 and 14.7 (6 and 4), of 49152 22.4 and 19.4 (12 and 8); d = 128, 8 tiles of 4096
// tokens 10.5 and 11.1 us (1 and 1), of 8192 12.5 and 12.2 (2 and 1), of 16384 16.6 and 14.4
// (4 and 2).
int kv4_cluster(const fa_kv4_cache* c, const fa_kv4_attn_params* p, int rows, int share_ctas) {
  const long long tiles = kv4_tiles(c, p, rows);
  long long tokens = (long long)p->table_width * c->page_size;
  if (p->window > 0) tokens = std::min(tokens, (long long)p->window + p->max_q_len + 31);
  const long long units = (tokens + 31) / 32;
  int dev = 0, log = 4;
  if (tiles > 2 * kMaxSms || cudaGetDevice(&dev) != cudaSuccess) return 0;
  while (tiles > kv4_clusters(dev, c->d, rows, log))
    if (--log < 0) return 0;
  const int cluster = 1 << log;
  const long long mine = (units + 8 * cluster - 1) / (8 * cluster);
  const long long share = (tiles * units + 4 * share_ctas - 1) / (4 * share_ctas);
  return (mine - share) * c->d > 128 ? 0 : cluster;
}

size_t attn_part_bytes(int ctas, int rows, int d) { return align256((size_t)2 * ctas * rows * (d + 4) * 4); }

}  // namespace

extern "C" {

fa_status fa_qk_norm_rope(const fa_qk_params* p, const void* q, const void* k, const void* wq, const void* wk,
                          const uint64_t* freqs, const int* positions, void* yq, void* yk, void* stream) {
  NvtxRange nvtx_range("fa_qk_norm_rope");
  FA_TRY(qk_check(p, false));
  if (p->N > 0) {
    FA_TRY(qk_pointers(p, q, k, wq, wk, freqs, positions));
    FA_TRY(need(yq, 16, "yq"));
    FA_TRY(need(yk, 16, "yk"));
    FA_TRY(qk_in_place(q, yq, p->q_stride, p->yq_stride, "yq"));
    FA_TRY(qk_in_place(k, yk, p->k_stride, p->yk_stride, "yk"));
  }
  Report rep;
  int sms = 0;
  FA_TRY(api_device(&rep, &sms));
  if (p->N == 0) return FA_OK;
  QkArgs a = qk_args(p, q, k, wq, wk, freqs, positions, sms, false);
  a.y[0] = static_cast<char*>(yq);
  a.y[1] = static_cast<char*>(yk);
  qk_strides(p, p->yq_stride, p->yk_stride, a.yb, a.yn, a.yh);
  const cudaError_t e =
      launch_qk_norm_rope(a, p->d, p->dtype, p->weight_dtype == FA_F32, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return api_cuda_fail(e, "norm and rotation launch");
  return FA_OK;
}

size_t fa_qk_norm_rope_bwd_workspace_size(const fa_qk_params* p) {
  if (qk_check(p, true) != FA_OK) return 0;
  return (size_t)kQkMaxSms * qk_ctas_per_sm(false, true) * 2 * p->d * 4;
}

fa_status fa_qk_norm_rope_bwd(const fa_qk_params* p, const void* q, const void* k, const void* dyq, const void* dyk,
                              const void* wq, const void* wk, const uint64_t* freqs, const int* positions, void* dq,
                              void* dk, float* dwq, float* dwk, void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("fa_qk_norm_rope_bwd");
  FA_TRY(qk_check(p, true));
  if (p->N > 0) {
    FA_TRY(qk_pointers(p, q, k, wq, wk, freqs, positions));
    FA_TRY(need(dyq, 16, "dyq"));
    FA_TRY(need(dyk, 16, "dyk"));
    FA_TRY(need(dq, 16, "dq"));
    FA_TRY(need(dk, 16, "dk"));
    FA_TRY(qk_in_place(q, dq, p->q_stride, p->dq_stride, "dq"));
    FA_TRY(qk_in_place(k, dk, p->k_stride, p->dk_stride, "dk"));
    FA_TRY(qk_in_place(dyq, dq, p->yq_stride, p->dq_stride, "dq"));
    FA_TRY(qk_in_place(dyk, dk, p->yk_stride, p->dk_stride, "dk"));
  }
  FA_TRY(need(dwq, 4, "dwq"));
  FA_TRY(need(dwk, 4, "dwk"));
  const size_t want = fa_qk_norm_rope_bwd_workspace_size(p);
  if (!workspace || workspace_bytes < want || !aligned(workspace, 256))
    return fail(FA_ERR_WORKSPACE, "workspace %p of %zu bytes; need %zu bytes, 256-byte aligned", workspace,
                workspace_bytes, want);
  Report rep;
  int sms = 0;
  FA_TRY(api_device(&rep, &sms));
  QkArgs a = qk_args(p, q, k, wq, wk, freqs, positions, sms, true);
  a.y[0] = static_cast<char*>(dq);
  a.y[1] = static_cast<char*>(dk);
  a.dy[0] = static_cast<const char*>(dyq);
  a.dy[1] = static_cast<const char*>(dyk);
  qk_strides(p, p->dq_stride, p->dk_stride, a.yb, a.yn, a.yh);
  qk_strides(p, p->yq_stride, p->yk_stride, a.db, a.dn, a.dh);
  a.part = static_cast<float*>(workspace);
  a.dw[0] = dwq;
  a.dw[1] = dwk;
  const cudaError_t e =
      launch_qk_norm_rope_bwd(a, p->d, p->dtype, p->weight_dtype == FA_F32, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return api_cuda_fail(e, "norm and rotation backward launch");
  return FA_OK;
}

int fa_kv4_block_bytes(int d) { return d == 128 ? KvBlock<128>::bytes : d == 64 ? KvBlock<64>::bytes : 0; }

fa_status fa_kv4_append(const fa_kv4_cache* c, const fa_kv4_rows* rows, const void* k, const void* v, const int* slots,
                        void* cache, void* stream) {
  NvtxRange nvtx_range("fa_kv4_append");
  return kv4_rows_call(c, rows, k, v, slots, cache, false, stream);
}

fa_status fa_kv4_gather(const fa_kv4_cache* c, const fa_kv4_rows* rows, const void* cache, const int* slots, void* k,
                        void* v, void* stream) {
  NvtxRange nvtx_range("fa_kv4_gather");
  return kv4_rows_call(c, rows, k, v, slots, cache, true, stream);
}

size_t fa_kv4_attention_workspace_size(const fa_kv4_cache* c, const fa_kv4_attn_params* p) {
  if (attn_check(c, p) != FA_OK) return 0;
  const int rows = kv4_tile_rows(p->Hq / c->Hk, p->max_q_len);
  const int ctas = kv4_share_ctas(rows, kMaxSms);
  return attn_part_bytes(ctas, rows, c->d) + align256((size_t)ctas * 32);
}

fa_status fa_kv4_attention(const fa_kv4_cache* c, const fa_kv4_attn_params* p, const void* q, const void* cache,
                           const int* block_table, const int* kv_lens, const int* cu_q, void* o, float* lse,
                           void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("fa_kv4_attention");
  FA_TRY(attn_check(c, p));
  if (p->T > 0) {
    FA_TRY(need(q, 16, "q"));
    FA_TRY(need(o, 16, "o"));
  }
  FA_TRY(need(cache, 16, "cache"));
  FA_TRY(need(block_table, 4, "block_table"));
  FA_TRY(need(kv_lens, 4, "kv_lens"));
  if (cu_q && !aligned(cu_q, 4)) return fail(FA_ERR_INVALID, "cu_q is not 4-byte aligned");
  if (lse && !aligned(lse, 4)) return fail(FA_ERR_INVALID, "lse is not 4-byte aligned");
  const size_t want = fa_kv4_attention_workspace_size(c, p);
  if (!workspace || workspace_bytes < want || !aligned(workspace, 256))
    return fail(FA_ERR_WORKSPACE, "workspace %p of %zu bytes; need %zu bytes, 256-byte aligned", workspace,
                workspace_bytes, want);
  // shares read a request's queries when another has already written its rows
  if (p->T > 0 && o == q) return fail(FA_ERR_INVALID, "o lies over q");
  Report rep;
  int sms = 0;
  FA_TRY(api_device(&rep, &sms));
  if (p->T == 0) return FA_OK;
  Kv4AttnArgs a;
  std::memset(&a, 0, sizeof(a));
  a.c = cache_args(c, cache);
  a.R = p->R;
  a.T = p->T;
  a.Hq = p->Hq;
  a.G = FastDiv::of((uint32_t)(p->Hq / c->Hk));
  a.window = p->window;
  a.table_width = p->table_width;
  a.table_stride = p->table_stride;
  a.table = block_table;
  a.kv_lens = kv_lens;
  a.cu_q = cu_q;
  a.scale_log2 = p->scale * 1.4426950408889634f;
  a.q = q;
  a.o = o;
  std::memcpy(a.qs, p->q_stride, sizeof(a.qs));
  std::memcpy(a.os, p->o_stride, sizeof(a.os));
  a.lse = lse;
  const int rows = kv4_tile_rows((int)a.G.d, p->max_q_len);
  int ctas = kv4_share_ctas(rows, std::min(sms, kMaxSms));
  a.part = static_cast<float*>(workspace);
  a.meta = reinterpret_cast<int4*>(static_cast<char*>(workspace) + attn_part_bytes(ctas, rows, c->d));
  const int cluster = kv4_cluster(c, p, rows, ctas);
  if (cluster > 0) ctas = (int)std::min<long long>(kv4_tiles(c, p, rows), (1 << 20)) * cluster;
  a.rep = rep;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f16 = p->dtype == FA_F16;
  const cudaError_t e = c->d == 64 ? launch_kv4_attention_d<64>(a, f16, rows, ctas, cluster, st)
                                   : launch_kv4_attention_d<128>(a, f16, rows, ctas, cluster, st);
  if (e != cudaSuccess) return api_cuda_fail(e, "cache attention launch");
  return FA_OK;
}

fa_status fa_paged_plan(const fa_plan_params* p, const int* seq_lens, const int* new_lens, int* block_table,
                        int* free_pages, const int* free_count, int* kv_lens, int* cu_q, int* positions, int* slots,
                        int* counts, void* stream) {
  NvtxRange nvtx_range("fa_paged_plan");
  if (!p) return fail(FA_ERR_INVALID, "params is NULL");
  if (p->R < 1 || p->T < 0 || p->page_size < 1 || p->num_pages < 1)
    return fail(FA_ERR_INVALID, "R, page_size and num_pages must be >= 1 and T >= 0");
  if (p->T > (1 << 30) || p->num_pages > (1 << 30)) return fail(FA_ERR_UNSUPPORTED, "T or num_pages exceeds 2^30");
  if (p->R > FA_PLAN_MAX_REQUESTS) return fail(FA_ERR_UNSUPPORTED, "R = %d exceeds %d", p->R, FA_PLAN_MAX_REQUESTS);
  if (p->table_width < 1 || p->table_stride < p->table_width)
    return fail(FA_ERR_INVALID, "block_table needs at least one column and a row stride of at least its width");
  const void* all[] = {seq_lens, new_lens, block_table, free_pages, free_count, kv_lens, cu_q, counts};
  const char* names[] = {"seq_lens", "new_lens", "block_table", "free_pages", "free_count", "kv_lens", "cu_q", "counts"};
  for (int i = 0; i < 8; ++i) FA_TRY(need(all[i], 4, names[i]));
  if (p->T > 0) {
    FA_TRY(need(positions, 4, "positions"));
    FA_TRY(need(slots, 4, "slots"));
  }
  Report rep;
  FA_TRY(api_device(&rep, nullptr));
  PlanArgs a;
  a.R = p->R;
  a.T = p->T;
  a.page = p->page_size;
  a.pages = p->num_pages;
  a.width = p->table_width;
  a.stride = p->table_stride;
  a.seq = seq_lens;
  a.fresh = new_lens;
  a.table = block_table;
  a.stack = free_pages;
  a.count = free_count;
  a.kv = kv_lens;
  a.cu = cu_q;
  a.pos = positions;
  a.slots = slots;
  a.counts = counts;
  a.aliased = false;
  const cudaError_t e = launch_paged_plan(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return api_cuda_fail(e, "plan launch");
  return FA_OK;
}

}  // extern "C"
