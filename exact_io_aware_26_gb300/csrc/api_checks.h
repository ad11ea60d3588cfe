// api_checks.h -- argument checks that the entry points of the operators share (host code).
#pragma once
#include <algorithm>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "internal.h"

#include <nvtx3/nvToolsExt.h>

namespace fa {
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

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline long long elem_bytes(int dtype) { return dtype == FA_F32 ? 4 : 2; }

inline fa_status need(const void* p, size_t align, const char* name) {
  if (!p) return fail(FA_ERR_INVALID, "%s is NULL", name);
  if (!aligned(p, align)) return fail(FA_ERR_INVALID, "%s is not %zu-byte aligned", name, align);
  return FA_OK;
}

// Strides (elements) of a tensor [size[0]][size[1]]...[inner]: whole 16-byte vectors,
// not negative; for a tensor that is written, no two elements in one place.
inline fa_status check_strides(const long long* stride, const long long* size, int n, long long inner, int dtype,
                               bool written, const char* name) {
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

// The memory of a tensor [size[0]][size[1]][inner], in bytes.
struct Extent {
  uintptr_t base;
  long long stride[2], size[2], inner;
  Extent(const void* p, const long long* element_stride, const long long* n, long long channels, long long e)
      : base(reinterpret_cast<uintptr_t>(p)), stride{element_stride[0] * e, element_stride[1] * e}, size{n[0], n[1]},
        inner(channels * e) {}
  // Bytes from the base on, of the dimensions whose stride is below `period`; negative where another one's is
  // no multiple of it, or they do not fit into it.
  long long within(long long period) const {
    long long n = inner;
    for (int i = 0; i < 2; ++i) {
      if (size[i] <= 1) continue;
      if (stride[i] < period)
        n += stride[i] * (size[i] - 1);
      else if (stride[i] % period != 0)
        return -1;
    }
    return n <= period ? n : -1;
  }
};
// Whether two tensors share no byte: one ends before the other begins, or they are rows (or heads) that take
// turns at the distance of a stride of either, such as the views of one packed projection.  Other
// layouts that take turns count as one over the other.
inline bool apart(const Extent& a, const Extent& b) {
  for (const Extent* x : {&a, &b})
    if (!x->base || x->size[0] == 0 || x->size[1] == 0) return true;
  constexpr long long kAll = 0x7FFFFFFFFFFFFFFFll;
  if (b.base >= a.base ? b.base - a.base >= (uintptr_t)a.within(kAll) : a.base - b.base >= (uintptr_t)b.within(kAll)) return true;
  for (const Extent* x : {&a, &b})
    for (int i = 0; i < 2; ++i) {
      const long long period = x->stride[i];
      if (x->size[i] <= 1 || period <= 0) continue;
      const long long na = a.within(period), nb = b.within(period);
      if (na < 0 || nb < 0) continue;
      const long long at = b.base >= a.base ? (long long)((b.base - a.base) % (uintptr_t)period)
                                            : (period - (long long)((a.base - b.base) % (uintptr_t)period)) % period;
      if (at >= na && at + nb <= period) return true;
    }
  return false;
}

}  // namespace
}  // namespace fa
