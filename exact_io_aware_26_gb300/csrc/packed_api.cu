// packed_api.cu -- the C ABI of packed attention (include/fa.h): argument checks, before any
// CUDA call, tensor maps and launches.
#include <cmath>
#include <cstring>

#include "api_checks.h"
#include "packed.h"

using namespace fa;

namespace {

constexpr int kMaxSms = 160;
constexpr int kMostGroup = 128;  // query heads of a key head: a tile's rows
// CTAs that the steps are shared among, for each SM, and the steps of a slice at least: below
// that a part's fp32 result costs more than the steps it takes off the others.
constexpr int kFwdCtas = 2, kBwdCtas = 1;
constexpr int kFwdLeast = 4, kBwdLeast = 2;

fa_status check(const fa_packed_params* p, bool bwd) {
  if (!p) return fail(FA_ERR_INVALID, "params is NULL");
  if (p->R < 1 || p->Tq < 0 || p->Tk < 0)
    return fail(FA_ERR_INVALID, "R must be >= 1, Tq and Tk >= 0 (got %d, %d, %d)", p->R, p->Tq, p->Tk);
  if (p->d != 64 && p->d != 128) return fail(FA_ERR_UNSUPPORTED, "head size %d is not supported (64 or 128)", p->d);
  if (p->dtype != FA_F16 && p->dtype != FA_BF16)
    return fail(p->dtype == FA_F32 ? FA_ERR_UNSUPPORTED : FA_ERR_INVALID, "packed attention takes fp16 or bf16");
  if (p->Hk < 1 || p->Hq < 1 || p->Hq % p->Hk != 0)
    return fail(FA_ERR_INVALID, "Hq = %d is no multiple of Hk = %d", p->Hq, p->Hk);
  if (p->Hq / p->Hk > kMostGroup)
    return fail(FA_ERR_UNSUPPORTED, "%d query heads to a key head exceed %d", p->Hq / p->Hk, kMostGroup);
  if (!(std::isfinite(p->scale) && p->scale > 0.f)) return fail(FA_ERR_INVALID, "scale must be positive and finite");
  if (p->R >= (1 << 24) || p->Tq > (1 << 30) || p->Tk > (1 << 30))
    return fail(FA_ERR_UNSUPPORTED, "R exceeds 2^24 - 1, or Tq or Tk 2^30");
  if ((long long)p->Tq * p->Hq >= (1ll << 31) || (long long)p->Tk * p->Hk >= (1ll << 31))
    return fail(FA_ERR_UNSUPPORTED, "Tq*Hq or Tk*Hk exceeds 2^31 - 1");
  const long long sq[2] = {p->Tq, p->Hq}, sk[2] = {p->Tk, p->Hk};
  const struct {
    const long long *stride, *size;
    bool written;
    const char* name;
  } all[] = {{p->q_stride, sq, false, "q"},   {p->k_stride, sk, false, "k"},   {p->v_stride, sk, false, "v"},
             {p->o_stride, sq, !bwd, "o"},    {p->do_stride, sq, false, "do"}, {p->dq_stride, sq, true, "dq"},
             {p->dk_stride, sk, true, "dk"},  {p->dv_stride, sk, true, "dv"}};
  for (int i = 0; i < (bwd ? 8 : 4); ++i) {
    FA_TRY(check_strides(all[i].stride, all[i].size, 2, p->d, p->dtype, all[i].written, all[i].name));
    for (int k = 0; k < 2; ++k) {
      if (all[i].size[k] > 1 && all[i].stride[k] == 0)
        return fail(FA_ERR_UNSUPPORTED, "%s: a stride of 0 (give each %s its own place)", all[i].name, k ? "head" : "token");
      if (all[i].stride[k] >= (1ll << 38)) return fail(FA_ERR_UNSUPPORTED, "%s: a stride exceeds 2^38 - 1", all[i].name);
    }
  }
  return FA_OK;
}

// The sizes of a call's work list and where it lies in the workspace.
struct Sizes {
  int tpt, target, least, slots, units, items, cuts;
  size_t items_at, cuts_at, left_at, starts_at, slots_at, stat_at, acc_at, most_at, seq_at, bytes;
  Sizes(const fa_packed_params* p, int sms, bool bwd) {
    const int G = p->Hq / p->Hk;
    tpt = 128 / G;
    target = std::min(sms, kMaxSms) * (bwd ? kBwdCtas : kFwdCtas);
    least = bwd ? kBwdLeast : kFwdLeast;
    // no unit has more steps than one over the whole of the other tensor
    const long long most = bwd ? ((long long)p->Tq + tpt - 1) / tpt : ((long long)p->Tk + 127) / 128;
    slots = most > least ? packed_slots(p->Hk, target) : 0;
    cuts = slots / 2;
    units = (int)((bwd ? p->Tk / 128 : p->Tq / tpt) + (long long)p->R);
    items = units + slots;
    size_t at = 256;
    auto place = [&](size_t n) {
      const size_t here = at;
      at += align256(n);
      return here;
    };
    items_at = place((size_t)items * sizeof(PackedItem));
    cuts_at = place((size_t)cuts * sizeof(PackedItem));
    left_at = place(bwd ? 0 : (size_t)cuts * p->Hk * sizeof(int));
    starts_at = place((size_t)4 * (p->R + 1) * sizeof(int));
    slots_at = place((size_t)slots * p->Hk * packed_slot_words(p->d, bwd) * 4);
    const size_t rows = (size_t)p->Tq * p->Hq;
    stat_at = bwd ? place(2 * rows * 4) : at;
    acc_at = bwd ? place(rows * p->d * 4) : at;
    const bool scaled = bwd && p->dtype == FA_F16;
    most_at = scaled ? place((size_t)p->R * p->Hk * sizeof(float4)) : 0;
    seq_at = scaled ? place((size_t)p->Tq * 4) : 0;
    bytes = at;
  }
};

fa_status workspace_check(const void* workspace, size_t bytes, size_t want) {
  if (!workspace || bytes < want || !aligned(workspace, 256))
    return fail(FA_ERR_WORKSPACE, "workspace %p of %zu bytes; need %zu bytes, 256-byte aligned", workspace, bytes, want);
  return FA_OK;
}

// [T][H][d] as {d, H, T}; boxes of 64 channels, `heads` heads and `tokens` tokens.
fa_status map_of(CUtensorMap* m, const fa_packed_params* p, const void* x, int T, int H, const long long* stride,
                 int heads, int tokens) {
  const uint64_t dims[3] = {(uint64_t)p->d, (uint64_t)H, (uint64_t)T};
  const uint64_t strides[2] = {H > 1 ? (uint64_t)stride[1] * 2 : (uint64_t)p->d * 2,
                               T > 1 ? (uint64_t)stride[0] * 2 : (uint64_t)p->d * H * 2};
  const uint32_t box[3] = {64, (uint32_t)heads, (uint32_t)tokens};
  return api_encode_3d(m, p->dtype == FA_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x,
                       dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

PackedArgs common_args(const fa_packed_params* p, const Sizes& z, void* workspace, const Report& rep) {
  PackedArgs a;
  std::memset(&a, 0, sizeof(a));
  a.R = p->R;
  a.Tq = p->Tq;
  a.Tk = p->Tk;
  a.Hq = p->Hq;
  a.Hk = p->Hk;
  a.G = p->Hq / p->Hk;
  a.divG = FastDiv::of((uint32_t)a.G);
  a.divHk = FastDiv::of((uint32_t)a.Hk);
  a.divRows = FastDiv::of((uint32_t)std::max(p->Tq * a.G, 1));
  a.divTk = FastDiv::of((uint32_t)std::max(p->Tk, 1));
  a.tpt = z.tpt;
  a.causal = p->causal != 0;
  a.scale = p->scale;
  a.scale_log2 = p->scale * 1.4426950408889634f;
  char* ws = static_cast<char*>(workspace);
  a.list.head = reinterpret_cast<int*>(ws);
  a.list.items = reinterpret_cast<PackedItem*>(ws + z.items_at);
  a.list.cuts = reinterpret_cast<PackedItem*>(ws + z.cuts_at);
  a.list.left = reinterpret_cast<int*>(ws + z.left_at);
  a.list.starts = reinterpret_cast<int*>(ws + z.starts_at);
  a.slots = reinterpret_cast<float*>(ws + z.slots_at);
  a.stat_lse = reinterpret_cast<float*>(ws + z.stat_at);
  a.stat_d = a.stat_lse + (size_t)p->Tq * p->Hq;
  a.dq_acc = reinterpret_cast<float*>(ws + z.acc_at);
  a.seq_of = reinterpret_cast<int*>(ws + z.seq_at);
  a.most = z.most_at ? reinterpret_cast<float4*>(ws + z.most_at) : nullptr;
  std::memcpy(a.vs, p->v_stride, sizeof(a.vs));
  std::memcpy(a.os, p->o_stride, sizeof(a.os));
  std::memcpy(a.dos, p->do_stride, sizeof(a.dos));
  std::memcpy(a.dqs, p->dq_stride, sizeof(a.dqs));
  std::memcpy(a.dks, p->dk_stride, sizeof(a.dks));
  std::memcpy(a.dvs, p->dv_stride, sizeof(a.dvs));
  a.rep = rep;
  return a;
}

PackedPlanArgs plan_args(const PackedArgs& a, const Sizes& z, const int* cu_q, const int* cu_k, bool bwd) {
  PackedPlanArgs q;
  q.R = a.R;
  q.Tq = a.Tq;
  q.Tk = a.Tk;
  q.Hk = a.Hk;
  q.tpt = a.tpt;
  q.causal = a.causal;
  q.bwd = bwd;
  q.target = z.target;
  q.slots = z.slots;
  q.least = z.least;
  q.units = z.units;
  q.cu_q = cu_q;
  q.cu_k = cu_k;
  q.list = a.list;
  q.most = a.most;
  q.st = a.rep.st;
  return q;
}

// Results are written while other CTAs still read the inputs (dq when all have been read).
fa_status forward_overlaps(const fa_packed_params* p, const void* q, const void* k, const void* v, const void* o,
                           const void* lse) {
  const long long sq[2] = {p->Tq, p->Hq}, sk[2] = {p->Tk, p->Hk}, dense[2] = {p->Hq, 1};
  const Extent in[3] = {{q, p->q_stride, sq, p->d, 2}, {k, p->k_stride, sk, p->d, 2}, {v, p->v_stride, sk, p->d, 2}};
  const Extent eo(o, p->o_stride, sq, p->d, 2), el(lse, dense, sq, 1, 4);
  for (const Extent& x : in) {
    if (!apart(eo, x)) return fail(FA_ERR_INVALID, "o lies over an input");
    if (!apart(el, x)) return fail(FA_ERR_INVALID, "lse lies over an input");
  }
  return apart(el, eo) ? FA_OK : fail(FA_ERR_INVALID, "o and lse lie over each other");
}

fa_status backward_overlaps(const fa_packed_params* p, const void* q, const void* k, const void* v, const void* dout,
                            const void* dq, const void* dk, const void* dv) {
  const long long sq[2] = {p->Tq, p->Hq}, sk[2] = {p->Tk, p->Hk};
  const Extent in[4] = {{q, p->q_stride, sq, p->d, 2}, {k, p->k_stride, sk, p->d, 2}, {v, p->v_stride, sk, p->d, 2},
                        {dout, p->do_stride, sq, p->d, 2}};
  const Extent eq(dq, p->dq_stride, sq, p->d, 2), ek(dk, p->dk_stride, sk, p->d, 2), ev(dv, p->dv_stride, sk, p->d, 2);
  for (const Extent& x : in)
    if (!apart(ek, x) || !apart(ev, x)) return fail(FA_ERR_INVALID, "dk or dv lies over an input");
  if (!apart(ek, ev) || !apart(eq, ek) || !apart(eq, ev)) return fail(FA_ERR_INVALID, "two gradients lie over each other");
  return FA_OK;
}

fa_status offsets_check(const fa_packed_params* p, const int* cu_q, const int*& cu_k) {
  FA_TRY(need(cu_q, 4, "cu_q"));
  if (!cu_k) {
    if (p->Tk != p->Tq) return fail(FA_ERR_INVALID, "cu_k is NULL where Tq = %d and Tk = %d differ", p->Tq, p->Tk);
    cu_k = cu_q;
  }
  return need(cu_k, 4, "cu_k");
}

}  // namespace

extern "C" {

size_t fa_fwd_packed_workspace_size(const fa_packed_params* p) {
  return check(p, false) != FA_OK ? 0 : Sizes(p, kMaxSms, false).bytes;
}

fa_status fa_fwd_packed(const fa_packed_params* p, const void* q, const void* k, const void* v, const int* cu_q,
                        const int* cu_k, void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("fa_fwd_packed");
  FA_TRY(check(p, false));
  FA_TRY(offsets_check(p, cu_q, cu_k));
  if (p->Tq > 0) {
    FA_TRY(need(q, 16, "q"));
    FA_TRY(need(o, 16, "o"));
    FA_TRY(need(lse, 4, "lse"));
  }
  if (p->Tk > 0) {
    FA_TRY(need(k, 16, "k"));
    FA_TRY(need(v, 16, "v"));
  }
  FA_TRY(forward_overlaps(p, q, k, v, o, lse));
  FA_TRY(workspace_check(workspace, workspace_bytes, fa_fwd_packed_workspace_size(p)));
  Report rep;
  int sms = 0;
  FA_TRY(api_device(&rep, &sms));
  if (p->Tq == 0) return FA_OK;
  const Sizes z(p, sms, false);
  if ((long long)z.items * p->Hk > 0x7FFFFFFFll) return fail(FA_ERR_UNSUPPORTED, "the tiles exceed 2^31 - 1");
  PackedArgs a = common_args(p, z, workspace, rep);
  a.v = v;
  a.o = o;
  a.lse = lse;
  CUtensorMap tm[3];
  const bool none = p->Tk == 0;  // no copy is made: any address
  FA_TRY(map_of(&tm[0], p, q, p->Tq, p->Hq, p->q_stride, a.G, a.tpt));
  FA_TRY(map_of(&tm[1], p, none ? q : k, none ? 1 : p->Tk, p->Hk, p->k_stride, 1, 128));
  FA_TRY(map_of(&tm[2], p, none ? q : v, none ? 1 : p->Tk, p->Hk, p->v_stride, 1, 128));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // a few sequences that no cut can shorten need no list (three prompts of up to 32 tokens: 10.7 us with it)
  a.direct = z.slots == 0 && p->R <= kPackedFew;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  cudaError_t e = cudaSuccess;
  if (!a.direct) e = launch_packed_plan(plan_args(a, z, cu_q, cu_k, false), s);
  if (e != cudaSuccess) return api_cuda_fail(e, "packed work list launch");
  e = launch_packed_fwd(a, p->d, p->dtype == FA_F16, tm, z.items, s);
  if (e != cudaSuccess) return api_cuda_fail(e, "packed forward launch");
  return FA_OK;
}

size_t fa_bwd_packed_workspace_size(const fa_packed_params* p) {
  return check(p, true) != FA_OK ? 0 : Sizes(p, kMaxSms, true).bytes;
}

fa_status fa_bwd_packed(const fa_packed_params* p, const void* q, const void* k, const void* v, const void* o,
                        const void* dout, const float* lse, const int* cu_q, const int* cu_k, void* dq, void* dk, void* dv,
                        void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("fa_bwd_packed");
  FA_TRY(check(p, true));
  FA_TRY(offsets_check(p, cu_q, cu_k));
  if (p->Tq > 0) {
    FA_TRY(need(q, 16, "q"));
    FA_TRY(need(o, 16, "o"));
    FA_TRY(need(dout, 16, "do"));
    FA_TRY(need(lse, 4, "lse"));
    FA_TRY(need(dq, 16, "dq"));
  }
  if (p->Tk > 0) {
    FA_TRY(need(k, 16, "k"));
    FA_TRY(need(v, 16, "v"));
    FA_TRY(need(dk, 16, "dk"));
    FA_TRY(need(dv, 16, "dv"));
  }
  FA_TRY(backward_overlaps(p, q, k, v, dout, dq, dk, dv));
  FA_TRY(workspace_check(workspace, workspace_bytes, fa_bwd_packed_workspace_size(p)));
  Report rep;
  int sms = 0;
  FA_TRY(api_device(&rep, &sms));
  if (p->Tq == 0 && p->Tk == 0) return FA_OK;
  const Sizes z(p, sms, true);
  if ((long long)z.items * p->Hk > 0x7FFFFFFFll) return fail(FA_ERR_UNSUPPORTED, "the tiles exceed 2^31 - 1");
  PackedArgs a = common_args(p, z, workspace, rep);
  a.v = v;
  a.o = const_cast<void*>(o);
  a.dout = dout;
  a.lse = const_cast<float*>(lse);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  const bool f16 = p->dtype == FA_F16;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  CUtensorMap tm[5];
  if (p->Tk > 0) {
    const bool none = p->Tq == 0;  // no copy is made: any address
    FA_TRY(map_of(&tm[0], p, none ? k : q, none ? 1 : p->Tq, p->Hq, p->q_stride, a.G, a.tpt));
    FA_TRY(map_of(&tm[1], p, k, p->Tk, p->Hk, p->k_stride, 1, 128));
    FA_TRY(map_of(&tm[2], p, v, p->Tk, p->Hk, p->v_stride, 1, 128));
    FA_TRY(map_of(&tm[3], p, none ? k : dout, none ? 1 : p->Tq, p->Hq, p->do_stride, a.G, a.tpt));
    const uint64_t rows = std::max<uint64_t>((uint64_t)p->Tq * a.G, 1);
    const uint64_t dims[3] = {(uint64_t)p->d, rows, (uint64_t)p->Hk};
    const uint64_t strides[2] = {(uint64_t)p->d * 4, rows * p->d * 4};
    const uint32_t box[3] = {32, 32, 1};
    FA_TRY(api_encode_3d(&tm[4], CU_TENSOR_MAP_DATA_TYPE_FLOAT32, none ? workspace : a.dq_acc, dims, strides, box,
                         CU_TENSOR_MAP_SWIZZLE_128B));
  }
  cudaError_t e = launch_packed_plan(plan_args(a, z, cu_q, cu_k, true), s);
  if (e != cudaSuccess) return api_cuda_fail(e, "packed work list launch");
  e = launch_packed_bwd_preprocess(a, p->d, f16, s);
  if (e != cudaSuccess) return api_cuda_fail(e, "packed backward rows launch");
  if (p->Tk > 0) {
    e = launch_packed_bwd(a, p->d, f16, tm, z.items, s);
    if (e != cudaSuccess) return api_cuda_fail(e, "packed backward launch");
  }
  e = launch_packed_bwd_finalize(a, p->d, f16, z.cuts, s);
  if (e != cudaSuccess) return api_cuda_fail(e, "packed backward finish launch");
  return FA_OK;
}

}  // extern "C"
