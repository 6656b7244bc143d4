// buffers.h — the buffers of one call of the C ABI, checked as they are added:
// natural alignment on the way in, then (check) outputs against every other
// buffer and each one's residency.
#pragma once

#include "zs_internal.h"

namespace zs {

class Buffers {
 public:
  explicit Buffers(const char* fn) : fn_(fn) {}

  zs_status add(const char* name, const void* p, int64_t bytes, int align, bool output) {
    if ((uintptr_t)p % (unsigned)align)
      return zs::fail(ZS_ERR_ALIGN, "%s: %s is not %d-byte aligned", fn_, name, align);
    if (p) items_[n_++] = {name, (uintptr_t)p, (uintptr_t)p + (uint64_t)bytes, output};
    return ZS_OK;
  }
  zs_status need(const char* name, const void* p, int64_t bytes, int align, bool output) {
    if (!p) return zs::fail(ZS_ERR_INVAL, "%s: %s is NULL", fn_, name);
    return add(name, p, bytes, align, output);
  }
  // The output and the input of these names may be one and the same.
  void may_share(const char* out, const char* in) { shared_[n_shared_++] = {out, in}; }

  zs_status check() const {
    for (int a = 0; a < n_; ++a) {
      if (!items_[a].output) continue;
      for (int b = 0; b < n_; ++b) {
        if (a == b || items_[a].lo >= items_[b].hi || items_[b].lo >= items_[a].hi) continue;
        if (one_place(items_[a], items_[b])) continue;
        return zs::fail(ZS_ERR_INVAL, "%s: %s overlaps %s", fn_, items_[a].name, items_[b].name);
      }
    }
    for (int a = 0; a < n_; ++a)
      if (zs_status st = zs::check_device_array(
              (const void*)items_[a].lo, (int64_t)(items_[a].hi - items_[a].lo), fn_,
              items_[a].name))
        return st;
    return ZS_OK;
  }

 private:
  struct Item {
    const char* name;
    uintptr_t lo, hi;
    bool output;
  };
  bool one_place(const Item& a, const Item& b) const {
    if (a.lo != b.lo || a.hi != b.hi) return false;
    for (int s = 0; s < n_shared_; ++s)
      if (a.name == shared_[s].out && b.name == shared_[s].in) return true;
    return false;
  }
  const char* fn_;
  Item items_[20];
  struct {
    const char *out, *in;
  } shared_[4];
  int n_ = 0, n_shared_ = 0;
};

// The rows of one matrix: (rows - 1) * stride + cols elements, kMaxExtent at most
// (2^46 bytes of fp32, past any device's memory), so that no product of them wraps.
constexpr int64_t kMaxExtent = int64_t(1) << 44;
inline zs_status check_stride(const char* fn, const char* name, int64_t stride, int64_t rows,
                              int64_t cols, const char* cols_name) {
  if (stride < cols || stride > int64_t(1) << 40)
    return zs::fail(ZS_ERR_RANGE, "%s: %s %lld outside %s..2^40", fn, name, (long long)stride,
                    cols_name);
  if (rows > 1 && stride > (kMaxExtent - cols) / (rows - 1))
    return zs::fail(ZS_ERR_RANGE, "%s: %lld rows %s %lld apart are more than 2^44 elements", fn,
                    (long long)rows, name, (long long)stride);
  return ZS_OK;
}

inline zs_status launched(const char* fn, cudaError_t e) {
  if (e != cudaSuccess)
    return zs::fail(ZS_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return ZS_OK;
}

}  // namespace zs
