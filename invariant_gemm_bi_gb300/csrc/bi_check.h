// bi_check.h -- what the entry points of the serving operations check of their
// operands before any launch (bi_serve_abi.cu, bi_quant_abi.cu).
#pragma once

#include <stdint.h>

#include <algorithm>
#include <string>

#include "../../include/bi.h"

namespace bi {
namespace {

bool is_float(int dtype) { return dtype == BI_BF16 || dtype == BI_F16 || dtype == BI_F32; }
bool is_index(int dtype) { return dtype == BI_I32 || dtype == BI_I64; }
int bytes_of(int dtype) {
  return dtype == BI_I64 ? 8 : (dtype == BI_F32 || dtype == BI_I32) ? 4 : dtype == BI_E4M3 ? 1 : 2;
}
int kind_of(int dtype) { return dtype == BI_E4M3 ? 3 : dtype == BI_F32 ? 2 : (dtype == BI_F16 ? 1 : 0); }
bool on(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A check that fails keeps its status and reason; later checks are skipped.
// Reasons are put together only then: a decode step makes these calls by the
// hundred.
struct Check {
  bi_status st = BI_OK;
  std::string why;

  bool ok() const { return st == BI_OK; }
  // `name` (if any): `reason`
  void that(bool good, bi_status bad, const char* reason, const char* name = nullptr) {
    if (good || !ok()) return;
    st = bad;
    why = name ? std::string(name) + ": " + reason : std::string(reason);
  }
  static bool empty(const bi_tensor* t) {
    for (int i = 0; i < t->ndim; ++i)
      if (t->shape[i] <= 0) return true;
    return false;
  }
  enum Kind { kFloat, kIndex, kE4m3, kScale };  // bf16, fp16 or fp32; int32 or int64; e4m3; fp32
  void tensor(const bi_tensor* t, const char* name, int ndim, bool index) {
    operand(t, name, ndim, index ? kIndex : kFloat, true);
  }
  // rank, type class, extents, strides (the last one 1 if `unit`), element alignment
  void operand(const bi_tensor* t, const char* name, int ndim, Kind kind, bool unit) {
    if (!ok()) return;
    that(t != nullptr, BI_ERR_INVALID_ARG, "null tensor descriptor", name);
    if (!ok()) return;
    if (t->ndim != ndim) {
      st = BI_ERR_INVALID_ARG;
      why = std::string(name) + ": expected rank " + std::to_string(ndim) + ", got " + std::to_string(t->ndim);
      return;
    }
    that(kind == kFloat   ? is_float(t->dtype)
         : kind == kIndex ? is_index(t->dtype)
                          : t->dtype == (kind == kE4m3 ? BI_E4M3 : BI_F32),
         BI_ERR_UNSUPPORTED_DTYPE,
         kind == kFloat   ? "a bf16, fp16 or fp32 type is needed"
         : kind == kIndex ? "an integer type is needed"
         : kind == kE4m3  ? "e4m3 is needed"
                          : "fp32 is needed",
         name);
    for (int i = 0; i < ndim; ++i) {
      that(t->shape[i] >= 0 && t->shape[i] <= INT32_MAX, BI_ERR_INVALID_ARG, "an extent is out of range", name);
      that(t->stride[i] >= 0 && t->stride[i] <= (int64_t)1 << 44, BI_ERR_UNSUPPORTED_LAYOUT,
           "a stride is negative or out of range", name);
    }
    if (!ok()) return;
    if (!empty(t)) {
      double span = 1.0;
      for (int i = 0; i < ndim; ++i) span += (double)(t->shape[i] - 1) * (double)t->stride[i];
      that(span < 1125899906842624.0 /* 2^50 */, BI_ERR_UNSUPPORTED_LAYOUT, "spans more memory than there is", name);
      that(t->ptr != nullptr, BI_ERR_INVALID_ARG, "null data pointer", name);
      that(on(t->ptr, bytes_of(t->dtype)), BI_ERR_UNSUPPORTED_LAYOUT, "not aligned to its element size", name);
    }
    that(!unit || ndim == 0 || t->shape[ndim - 1] <= 1 || t->stride[ndim - 1] == 1, BI_ERR_UNSUPPORTED_LAYOUT,
         "unit stride on the last dimension required", name);
  }
  // a contiguous index vector of n elements of the given type
  void vec(const bi_tensor* t, const char* name, int64_t n, int dtype) {
    tensor(t, name, 1, true);
    if (!ok()) return;
    if (t->shape[0] != n) {
      st = BI_ERR_SHAPE_MISMATCH;
      why = std::string(name) + ": expected " + std::to_string(n) + " elements";
      return;
    }
    that(t->dtype == dtype, BI_ERR_UNSUPPORTED_DTYPE, dtype == BI_I64 ? "int64 is needed" : "int32 is needed", name);
  }
  // every element of an output has an address of its own
  void distinct(const bi_tensor* t, const char* name) {
    if (!ok() || empty(t)) return;
    // dimensions in the order of their strides: each must clear what the smaller ones span
    int order[4] = {0, 1, 2, 3};
    for (int i = 0; i < t->ndim; ++i)
      for (int j = i + 1; j < t->ndim; ++j)
        if (t->stride[order[j]] < t->stride[order[i]]) std::swap(order[i], order[j]);
    int64_t span = 0;
    for (int i = 0; i < t->ndim; ++i) {
      const int d = order[i];
      if (t->shape[d] == 1) continue;
      that(t->stride[d] > span, BI_ERR_UNSUPPORTED_LAYOUT, "elements of the output overlap", name);
      span += (t->shape[d] - 1) * t->stride[d];
    }
  }
  // memory that t spans, as [begin, end)
  static void range(const bi_tensor* t, uintptr_t* b, uintptr_t* e) {
    *b = reinterpret_cast<uintptr_t>(t->ptr);
    int64_t last = 0;
    for (int i = 0; i < t->ndim; ++i) last += (t->shape[i] - 1) * t->stride[i];
    *e = *b + (uintptr_t)((last + 1) * bytes_of(t->dtype));
  }
  void apart(const bi_tensor* out, const bi_tensor* in, const char* what) {
    if (!ok() || !out || !in || empty(out) || empty(in)) return;
    uintptr_t a0, a1, b0, b1;
    range(out, &a0, &a1);
    range(in, &b0, &b1);
    if (a1 <= b0 || b1 <= a0) return;
    that(interleaved(out, in), BI_ERR_INVALID_ARG, "an output overlaps another operand", what);
  }
  // Views of one buffer that interleave without touching (q, k and v of one
  // projection; keys, values and scales of one cache buffer): with some period s,
  // each view's dimensions either lie within one period or step by whole
  // periods, and the parts of the period they take are apart.
  static bool interleaved(const bi_tensor* x, const bi_tensor* y) {
    const int64_t d = reinterpret_cast<intptr_t>(y->ptr) - reinterpret_cast<intptr_t>(x->ptr);
    for (int i = 0; i < x->ndim; ++i) {
      const int64_t s = x->stride[i] * bytes_of(x->dtype);
      if (x->shape[i] < 2 || s < 1) continue;
      const int64_t xs = within(x, s), ys = within(y, s);
      if (xs <= 0 || ys <= 0) continue;
      const int64_t off = (d % s + s) % s;  // y starts this far into x's period
      if (off >= xs && off + ys <= s) return true;
    }
    return false;
  }
  // Bytes that t spans inside a period of s; 0 when a dimension fits neither way.
  static int64_t within(const bi_tensor* t, int64_t s) {
    int64_t span = bytes_of(t->dtype);
    for (int i = 0; i < t->ndim; ++i) {
      const int64_t step = t->stride[i] * bytes_of(t->dtype);
      if (t->shape[i] < 2 || step % s == 0) continue;
      if (step > s) return 0;
      span += (t->shape[i] - 1) * step;
    }
    return span <= s ? span : 0;
  }
};

constexpr int64_t kMaxRequests = 1 << 22;  // of a plan and an attention call
constexpr int64_t kMaxHeads = 1 << 30;     // head numbers of a token, and steps past them, fit 32 bits

int64_t stride_or(const bi_tensor* t, int d, int64_t alone) { return t->shape[d] > 1 ? t->stride[d] : alone; }

// Row and head strides (those that are walked) in whole 16-byte units.
bool rows_on_16(const bi_tensor* t) {
  const int e = bytes_of(t->dtype);
  for (int i = 0; i + 1 < t->ndim; ++i)
    if (t->shape[i] > 1 && (t->stride[i] * e) % 16 != 0) return false;
  return on(t->ptr, 16);
}

bool same_view(const bi_tensor* a, const bi_tensor* b) {
  return a->ptr == b->ptr && a->dtype == b->dtype && a->stride[0] == b->stride[0] && a->stride[1] == b->stride[1];
}

}  // namespace
}  // namespace bi
