// layers_api.cpp — the C entry points of the operators around the layers: the
// embedding lookup and its gradient, layer norm and its gradient, and the norm
// and clipping of a list of gradients. Argument checks, then the launches; every
// check runs before anything is enqueued.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "buffers.h"
#include "zs_internal.h"

namespace {

zs_status check_dtype(const char* fn, const char* name, zs_dtype dt) {
  if (dt != ZS_BF16 && dt != ZS_FP32)
    return zs::fail(ZS_ERR_INVAL, "%s: %s %d is not bf16 or fp32", fn, name, (int)dt);
  return ZS_OK;
}

zs_status check_rows(const char* fn, int64_t rows, int64_t dim) {
  if (rows < 0 || rows > 0x7FFFFFFF)
    return zs::fail(ZS_ERR_RANGE, "%s: rows %lld outside 0..2^31-1", fn, (long long)rows);
  if (dim < 1 || dim > ZS_MAX_DIM)
    return zs::fail(ZS_ERR_RANGE, "%s: dim %lld outside 1..%d", fn, (long long)dim, ZS_MAX_DIM);
  return ZS_OK;
}

// Bytes that a matrix spans from its first element to its last.
int64_t extent(int64_t rows, int64_t stride, int64_t dim, zs_dtype dt) {
  return rows > 0 ? ((rows - 1) * stride + dim) * zs::elem_bytes(dt) : 0;
}

// The table's and the rows' sizes, types and strides; the scale.
zs_status check_embedding(const char* fn, const zs::EmbeddingLaunch& a, const char* stride_name) {
  if (zs_status st = check_dtype(fn, "table_dtype", a.table_dtype)) return st;
  if (zs_status st = check_dtype(fn, "dtype", a.dtype)) return st;
  if (zs_status st = check_rows(fn, a.rows, a.dim)) return st;
  if (a.vocab < 1 || a.vocab > ZS_MAX_VOCAB)
    return zs::fail(ZS_ERR_RANGE, "%s: vocab %lld outside 1..%d", fn, (long long)a.vocab,
                    ZS_MAX_VOCAB);
  if (zs_status st = zs::check_stride(fn, "table_stride", a.table_stride, a.vocab, a.dim, "dim"))
    return st;
  if (zs_status st = zs::check_stride(fn, stride_name, a.row_stride, a.rows, a.dim, "dim"))
    return st;
  if (!std::isfinite(a.scale) || std::fabs(a.scale) > 3e38)
    return zs::fail(ZS_ERR_INVAL, "%s: scale must be finite in fp32 (got %g)", fn, a.scale);
  return ZS_OK;
}

const char* const kX = "x";
const char* const kResidual = "residual";
const char* const kSum = "sum_out";
const char* const kY = "y";
const char* const kDY = "d_y";
const char* const kDX = "d_x";
const char* const kDSum = "d_sum";
const char* const kAdd = "add_to";
const char* const kDTable = "d_table";

// ---- lists of tensors -------------------------------------------------------------
struct Span {
  uintptr_t lo, hi;
  int32_t index;
};

// A list's addresses, lengths and residency.
zs_status check_list(const char* fn, const char* name, const void* const* p, const int64_t* numels,
                     int32_t n, zs_dtype dt) {
  const int es = zs::elem_bytes(dt);
  if (n > 0 && !p) return zs::fail(ZS_ERR_INVAL, "%s: %s is NULL", fn, name);
  for (int32_t i = 0; i < n; ++i) {
    if (numels[i] == 0) continue;
    if (!p[i]) return zs::fail(ZS_ERR_INVAL, "%s: %s[%d] is NULL", fn, name, i);
    if ((uintptr_t)p[i] % (unsigned)es)
      return zs::fail(ZS_ERR_ALIGN, "%s: %s[%d] is not %d-byte aligned", fn, name, i, es);
  }
  return ZS_OK;
}
zs_status check_lengths(const char* fn, const int64_t* numels, int32_t n) {
  if (n < 0 || n > ZS_MAX_TENSORS)
    return zs::fail(ZS_ERR_RANGE, "%s: %d tensors outside 0..%d", fn, n, ZS_MAX_TENSORS);
  if (n > 0 && !numels) return zs::fail(ZS_ERR_INVAL, "%s: numels is NULL", fn);
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (numels[i] < 0 || numels[i] > zs::kMaxExtent || (total += numels[i]) > zs::kMaxExtent)
      return zs::fail(ZS_ERR_RANGE, "%s: numels[%d] = %lld: lengths are 0..2^44, their sum too", fn,
                      i, (long long)numels[i]);
  }
  return ZS_OK;
}
zs_status check_resident(const char* fn, const char* name, const void* const* p,
                         const int64_t* numels, int32_t n, zs_dtype dt) {
  for (int32_t i = 0; i < n; ++i)
    if (zs_status st =
            zs::check_device_array(p[i], numels[i] * zs::elem_bytes(dt), fn, name))
      return st;
  return ZS_OK;
}

// Outputs lie apart from one another, from the fixed buffers, and from the
// inputs (but for tensor i in place of tensor i). A model's outputs come in
// ascending order mostly, so that sorting them is one look at each.
zs_status check_apart(const char* fn, const void* const* in, zs_dtype dt, void* const* out,
                      zs_dtype out_dt, const int64_t* numels, int32_t n, const Span* fixed,
                      int n_fixed) {
  std::vector<Span> outs;
  outs.reserve((size_t)n);
  for (int32_t i = 0; i < n; ++i)
    if (numels[i] > 0)
      outs.push_back({(uintptr_t)out[i],
                      (uintptr_t)out[i] + (uint64_t)numels[i] * zs::elem_bytes(out_dt), i});
  auto before = [](const Span& x, const Span& y) { return x.lo < y.lo; };
  if (!std::is_sorted(outs.begin(), outs.end(), before))
    std::sort(outs.begin(), outs.end(), before);
  for (size_t k = 1; k < outs.size(); ++k)
    if (outs[k].lo < outs[k - 1].hi)
      return zs::fail(ZS_ERR_INVAL, "%s: outs[%d] overlaps outs[%d]", fn, outs[k].index,
                      outs[k - 1].index);
  // the outputs are apart, so ends ascend too: the first that ends behind x.lo
  auto met = [&](const Span& x) {
    return std::partition_point(outs.begin(), outs.end(),
                                [&](const Span& o) { return o.hi <= x.lo; });
  };
  for (int32_t i = 0; i < n; ++i) {
    if (numels[i] == 0) continue;
    const Span x = {(uintptr_t)in[i],
                    (uintptr_t)in[i] + (uint64_t)numels[i] * zs::elem_bytes(dt), i};
    const auto o = met(x);
    if (o == outs.end() || o->lo >= x.hi) continue;
    if (o->index == i && o->lo == x.lo && o->hi == x.hi) continue;
    return zs::fail(ZS_ERR_INVAL, "%s: outs[%d] overlaps tensors[%d]", fn, o->index, i);
  }
  for (int k = 0; k < n_fixed; ++k) {
    const auto o = met(fixed[k]);
    if (o != outs.end() && o->lo < fixed[k].hi)
      return zs::fail(ZS_ERR_INVAL, "%s: outs[%d] overlaps another buffer of the call", fn,
                      o->index);
  }
  return ZS_OK;
}

// The call's small buffers, apart from one another and from the inputs they are
// not read from.
zs_status check_small(const char* fn, const zs::TensorsLaunch& a, int64_t workspace_bytes,
                      bool norm, std::vector<Span>* fixed) {
  zs::Buffers b(fn);
  if (norm) {
    if (zs_status st = b.need("workspace", a.workspace, zs::kNormWorkspaceBytes, 16, true))
      return st;
    if (workspace_bytes < zs::kNormWorkspaceBytes)
      return zs::fail(ZS_ERR_RANGE, "%s: workspace of %lld bytes, needs %lld", fn,
                      (long long)workspace_bytes, (long long)zs::kNormWorkspaceBytes);
    if (zs_status st = b.add("sqnorm_out", a.sqnorm, 8, 8, true)) return st;
    if (zs_status st = b.add("norm_out", a.norm, 4, 4, true)) return st;
    if (zs_status st = b.add("coef_out", a.coef_out, 4, 4, true)) return st;
    if (zs_status st = b.add("nonfinite_out", a.nonfinite_out, 4, 4, true)) return st;
  } else {
    if (zs_status st = b.add("coef", a.coef, 4, 4, false)) return st;
    if (zs_status st = b.add("skip", a.skip, 4, 4, false)) return st;
  }
  auto span = [&](const void* p, int64_t bytes) {
    if (p) fixed->push_back({(uintptr_t)p, (uintptr_t)p + (uint64_t)bytes, -1});
  };
  if (norm) {
    span(a.workspace, zs::kNormWorkspaceBytes);
    span(a.sqnorm, 8);
    span(a.norm, 4);
    span(a.coef_out, 4);
    span(a.nonfinite_out, 4);
    for (int64_t i = 0; i < a.count; ++i) {
      if (a.numels[i] == 0) continue;
      const uintptr_t lo = (uintptr_t)a.tensors[i];
      const uintptr_t hi = lo + (uint64_t)a.numels[i] * zs::elem_bytes(a.dtype);
      for (const Span& s : *fixed)
        if (s.lo < hi && lo < s.hi)
          return zs::fail(ZS_ERR_INVAL, "%s: an output or the workspace overlaps tensors[%d]", fn,
                          (int)i);
    }
  } else {
    span(a.coef, 4);
    span(a.skip, 4);
  }
  return b.check();
}

}  // namespace

// ---- embedding --------------------------------------------------------------------
extern "C" zs_status zs_embedding(const void* table, zs_dtype table_dtype, int64_t vocab,
                                  int64_t dim, int64_t table_stride, const int64_t* tokens,
                                  int64_t rows, double scale, void* out, zs_dtype out_dtype,
                                  int64_t out_stride, void* cuda_stream) {
  static const char* fn = "zs_embedding";
  const zs::CallRange range(fn);
  zs::clear_error();
  zs::EmbeddingLaunch a = {};
  a.table = table;
  a.table_dtype = table_dtype;
  a.vocab = vocab;
  a.dim = dim;
  a.table_stride = table_stride;
  a.tokens = tokens;
  a.rows = rows;
  a.scale = scale;
  a.rows_out = out;
  a.dtype = out_dtype;
  a.row_stride = out_stride;
  if (zs_status st = check_embedding(fn, a, "out_stride")) return st;
  if (rows == 0) return ZS_OK;
  const int ts = zs::elem_bytes(table_dtype), es = zs::elem_bytes(out_dtype);
  zs::Buffers b(fn);
  if (zs_status st =
          b.need("table", table, extent(vocab, table_stride, dim, table_dtype), ts, false))
    return st;
  if (zs_status st = b.need("tokens", tokens, rows * 8, 8, false)) return st;
  if (zs_status st = b.need("out", out, extent(rows, out_stride, dim, out_dtype), es, true))
    return st;
  if (zs_status st = b.check()) return st;
  return zs::launched(fn, zs::launch_embedding(a, static_cast<cudaStream_t>(cuda_stream)));
}

extern "C" int64_t zs_embedding_grad_workspace_bytes(int64_t rows, int64_t dim) {
  if (rows < 0 || rows > 0x7FFFFFFF || dim < 1 || dim > ZS_MAX_DIM) return -1;
  return zs::embedding_grad_workspace_bytes(rows, dim);
}

extern "C" zs_status zs_embedding_grad(const void* d_out, zs_dtype dtype, int64_t rows,
                                       int64_t dim, int64_t row_stride, const int64_t* tokens,
                                       int64_t vocab, double scale, const void* add_to,
                                       void* workspace, int64_t workspace_bytes, void* d_table,
                                       zs_dtype table_dtype, int64_t table_stride,
                                       void* cuda_stream) {
  static const char* fn = "zs_embedding_grad";
  const zs::CallRange range(fn);
  zs::clear_error();
  zs::EmbeddingLaunch a = {};
  a.table_dtype = table_dtype;
  a.vocab = vocab;
  a.dim = dim;
  a.table_stride = table_stride;
  a.tokens = tokens;
  a.rows = rows;
  a.scale = scale;
  a.rows_in = d_out;
  a.dtype = dtype;
  a.row_stride = row_stride;
  a.add = add_to;
  a.d_table = d_table;
  a.workspace = workspace;
  if (zs_status st = check_embedding(fn, a, "row_stride")) return st;
  const int ts = zs::elem_bytes(table_dtype), es = zs::elem_bytes(dtype);
  const int64_t table_bytes = extent(vocab, table_stride, dim, table_dtype);
  zs::Buffers b(fn);
  if (zs_status st = b.need(kDTable, d_table, table_bytes, ts, true)) return st;
  if (zs_status st = b.add(kAdd, add_to, table_bytes, ts, false)) return st;
  if (rows > 0) {
    const int64_t need = zs::embedding_grad_workspace_bytes(rows, dim);
    if (workspace_bytes < need)
      return zs::fail(ZS_ERR_RANGE, "%s: workspace of %lld bytes, needs %lld", fn,
                      (long long)workspace_bytes, (long long)need);
    if (zs_status st = b.need("d_out", d_out, extent(rows, row_stride, dim, dtype), es, false))
      return st;
    if (zs_status st = b.need("tokens", tokens, rows * 8, 8, false)) return st;
    if (zs_status st = b.need("workspace", workspace, need, 16, true)) return st;
  }
  b.may_share(kDTable, kAdd);
  if (zs_status st = b.check()) return st;
  return zs::launched(fn, zs::launch_embedding_grad(a, static_cast<cudaStream_t>(cuda_stream)));
}

// ---- layer norm -------------------------------------------------------------------
extern "C" zs_status zs_layer_norm(const void* x, zs_dtype dtype, int64_t rows, int64_t dim,
                                   int64_t row_stride, const void* residual, const void* weight,
                                   const void* bias, zs_dtype weight_dtype, double eps,
                                   void* sum_out, void* y, int64_t out_stride, float* mean,
                                   float* rstd, void* cuda_stream) {
  static const char* fn = "zs_layer_norm";
  const zs::CallRange range(fn);
  zs::clear_error();
  if (zs_status st = check_dtype(fn, "dtype", dtype)) return st;
  if (zs_status st = check_dtype(fn, "weight_dtype", weight_dtype)) return st;
  if (zs_status st = check_rows(fn, rows, dim)) return st;
  if (zs_status st = zs::check_stride(fn, "row_stride", row_stride, rows, dim, "dim")) return st;
  if (zs_status st = zs::check_stride(fn, "out_stride", out_stride, rows, dim, "dim")) return st;
  if (!(eps >= 1e-30 && eps <= 1e30))
    return zs::fail(ZS_ERR_INVAL, "%s: eps must be within 1e-30..1e30 (got %g)", fn, eps);
  if (sum_out && !residual)
    return zs::fail(ZS_ERR_INVAL, "%s: sum_out needs a residual", fn);
  if (rows == 0) return ZS_OK;
  const int es = zs::elem_bytes(dtype), ws = zs::elem_bytes(weight_dtype);
  const int64_t in_bytes = extent(rows, row_stride, dim, dtype),
                out_bytes = extent(rows, out_stride, dim, dtype);
  zs::Buffers b(fn);
  if (zs_status st = b.need(kX, x, in_bytes, es, false)) return st;
  if (zs_status st = b.add(kResidual, residual, in_bytes, es, false)) return st;
  if (zs_status st = b.add("weight", weight, dim * ws, ws, false)) return st;
  if (zs_status st = b.add("bias", bias, dim * ws, ws, false)) return st;
  if (zs_status st = b.add(kSum, sum_out, out_bytes, es, true)) return st;
  if (zs_status st = b.need(kY, y, out_bytes, es, true)) return st;
  if (zs_status st = b.add("mean", mean, rows * 4, 4, true)) return st;
  if (zs_status st = b.add("rstd", rstd, rows * 4, 4, true)) return st;
  if (row_stride == out_stride || rows == 1) {
    b.may_share(kY, kX);
    b.may_share(kSum, kX);
    b.may_share(kY, kResidual);
    b.may_share(kSum, kResidual);
  }
  if (zs_status st = b.check()) return st;
  zs::LayerNormLaunch a = {};
  a.x = x;
  a.residual = residual;
  a.dtype = dtype;
  a.rows = rows;
  a.dim = dim;
  a.row_stride = row_stride;
  a.out_stride = out_stride;
  a.weight = weight;
  a.bias = bias;
  a.weight_dtype = weight_dtype;
  a.eps = eps;
  a.sum = sum_out;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  return zs::launched(fn, zs::launch_layer_norm(a, static_cast<cudaStream_t>(cuda_stream)));
}

extern "C" int64_t zs_layer_norm_grad_workspace_bytes(int64_t rows, int64_t dim) {
  if (rows < 0 || rows > 0x7FFFFFFF || dim < 1 || dim > ZS_MAX_DIM) return -1;
  return zs::layer_norm_grad_workspace_bytes(rows, dim);
}

extern "C" zs_status zs_layer_norm_grad(const void* d_y, const void* x, zs_dtype dtype,
                                        int64_t rows, int64_t dim, int64_t grad_stride,
                                        int64_t row_stride, const void* weight,
                                        zs_dtype weight_dtype, const float* mean,
                                        const float* rstd, const void* d_sum, void* workspace,
                                        int64_t workspace_bytes, void* d_x, void* d_weight,
                                        void* d_bias, zs_dtype grad_dtype, void* cuda_stream) {
  static const char* fn = "zs_layer_norm_grad";
  const zs::CallRange range(fn);
  zs::clear_error();
  if (zs_status st = check_dtype(fn, "dtype", dtype)) return st;
  if (zs_status st = check_dtype(fn, "weight_dtype", weight_dtype)) return st;
  if (zs_status st = check_dtype(fn, "grad_dtype", grad_dtype)) return st;
  if (zs_status st = check_rows(fn, rows, dim)) return st;
  if (zs_status st = zs::check_stride(fn, "grad_stride", grad_stride, rows, dim, "dim")) return st;
  if (zs_status st = zs::check_stride(fn, "row_stride", row_stride, rows, dim, "dim")) return st;
  const int es = zs::elem_bytes(dtype), ws = zs::elem_bytes(weight_dtype),
            gs = zs::elem_bytes(grad_dtype);
  const bool sums = d_weight || d_bias;
  zs::Buffers b(fn);
  if (rows > 0) {
    const int64_t grad_bytes = extent(rows, grad_stride, dim, dtype);
    if (zs_status st = b.need(kDY, d_y, grad_bytes, es, false)) return st;
    if (zs_status st = b.need(kX, x, extent(rows, row_stride, dim, dtype), es, false)) return st;
    if (zs_status st = b.add("weight", weight, dim * ws, ws, false)) return st;
    if (zs_status st = b.need("mean", mean, rows * 4, 4, false)) return st;
    if (zs_status st = b.need("rstd", rstd, rows * 4, 4, false)) return st;
    if (zs_status st = b.add(kDSum, d_sum, grad_bytes, es, false)) return st;
    if (zs_status st = b.need(kDX, d_x, grad_bytes, es, true)) return st;
    if (sums) {
      const int64_t need = zs::layer_norm_grad_workspace_bytes(rows, dim);
      if (workspace_bytes < need)
        return zs::fail(ZS_ERR_RANGE, "%s: workspace of %lld bytes, needs %lld", fn,
                        (long long)workspace_bytes, (long long)need);
      if (zs_status st = b.need("workspace", workspace, need, 16, true)) return st;
    }
    b.may_share(kDX, kDY);
    b.may_share(kDX, kDSum);
  }
  if (zs_status st = b.add("d_weight", d_weight, dim * gs, gs, true)) return st;
  if (zs_status st = b.add("d_bias", d_bias, dim * gs, gs, true)) return st;
  if (zs_status st = b.check()) return st;
  zs::LayerNormLaunch a = {};
  a.x = x;
  a.dtype = dtype;
  a.rows = rows;
  a.dim = dim;
  a.row_stride = row_stride;
  a.grad_stride = grad_stride;
  a.weight = weight;
  a.weight_dtype = weight_dtype;
  a.grad_dtype = grad_dtype;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.d_y = d_y;
  a.d_sum = d_sum;
  a.d_x = d_x;
  a.d_weight = d_weight;
  a.d_bias = d_bias;
  a.workspace = workspace;
  return zs::launched(fn, zs::launch_layer_norm_grad(a, static_cast<cudaStream_t>(cuda_stream)));
}

// ---- lists of gradients -----------------------------------------------------------
namespace {

zs_status list_call(const char* fn, zs::TensorsLaunch a, int64_t workspace_bytes, bool norm,
                    bool scale, void* cuda_stream) try {
  zs::clear_error();
  if (zs_status st = check_dtype(fn, "dtype", a.dtype)) return st;
  if (scale)
    if (zs_status st = check_dtype(fn, "out_dtype", a.out_dtype)) return st;
  const int32_t n = (int32_t)a.count;
  if (zs_status st = check_lengths(fn, a.numels, n)) return st;
  if (zs_status st = check_list(fn, "tensors", a.tensors, a.numels, n, a.dtype)) return st;
  if (scale)
    if (zs_status st = check_list(fn, "outs", (const void* const*)a.outs, a.numels, n, a.out_dtype))
      return st;
  if (!norm && std::all_of(a.numels, a.numels + n, [](int64_t k) { return k == 0; }))
    return ZS_OK;  // nothing to scale
  std::vector<Span> fixed;
  if (zs_status st = check_small(fn, a, workspace_bytes, norm, &fixed)) return st;
  if (scale)
    if (zs_status st = check_apart(fn, a.tensors, a.dtype, a.outs, a.out_dtype, a.numels, n,
                                   fixed.data(), (int)fixed.size()))
      return st;
  if (zs_status st = check_resident(fn, "tensors", a.tensors, a.numels, n, a.dtype)) return st;
  if (scale)
    if (zs_status st =
            check_resident(fn, "outs", (const void* const*)a.outs, a.numels, n, a.out_dtype))
      return st;
  return zs::launched(
      fn, zs::launch_tensors(a, norm, scale, static_cast<cudaStream_t>(cuda_stream)));
} catch (const std::bad_alloc&) {
  return zs::fail(ZS_ERR_NOMEM, "%s: out of host memory", fn);
}

}  // namespace

extern "C" zs_status zs_tensors_sqnorm(const void* const* tensors, const int64_t* numels,
                                       int32_t n, zs_dtype dtype, void* workspace,
                                       int64_t workspace_bytes, double* sqnorm_out,
                                       void* cuda_stream) {
  static const char* fn = "zs_tensors_sqnorm";
  const zs::CallRange range(fn);
  zs::TensorsLaunch a = {};
  a.tensors = tensors;
  a.numels = numels;
  a.count = n;
  a.dtype = dtype;
  a.workspace = workspace;
  a.sqnorm = sqnorm_out;
  if (!sqnorm_out) {
    zs::clear_error();
    return zs::fail(ZS_ERR_INVAL, "%s: sqnorm_out is NULL", fn);
  }
  return list_call(fn, a, workspace_bytes, true, false, cuda_stream);
}

extern "C" zs_status zs_tensors_scale(const void* const* tensors, const int64_t* numels, int32_t n,
                                      zs_dtype dtype, const float* coef, const int32_t* skip,
                                      void* const* outs, zs_dtype out_dtype, void* cuda_stream) {
  static const char* fn = "zs_tensors_scale";
  const zs::CallRange range(fn);
  zs::TensorsLaunch a = {};
  a.tensors = tensors;
  a.numels = numels;
  a.count = n;
  a.dtype = dtype;
  a.outs = outs;
  a.out_dtype = out_dtype;
  a.coef = coef;
  a.skip = skip;
  if (!coef) {
    zs::clear_error();
    return zs::fail(ZS_ERR_INVAL, "%s: coef is NULL", fn);
  }
  return list_call(fn, a, 0, false, true, cuda_stream);
}

extern "C" zs_status zs_tensors_clip(const void* const* tensors, const int64_t* numels, int32_t n,
                                     zs_dtype dtype, double max_norm, void* const* outs,
                                     zs_dtype out_dtype, void* workspace, int64_t workspace_bytes,
                                     float* norm_out, float* coef_out, int32_t* nonfinite_out,
                                     void* cuda_stream) {
  static const char* fn = "zs_tensors_clip";
  const zs::CallRange range(fn);
  zs::TensorsLaunch a = {};
  a.tensors = tensors;
  a.numels = numels;
  a.count = n;
  a.dtype = dtype;
  a.outs = outs;
  a.out_dtype = out_dtype;
  a.workspace = workspace;
  a.max_norm = max_norm;
  a.norm = norm_out;
  a.coef = a.coef_out = coef_out;
  a.skip = a.nonfinite_out = nonfinite_out;
  zs::clear_error();
  if (!(std::isfinite(max_norm) && max_norm > 0))
    return zs::fail(ZS_ERR_INVAL, "%s: max_norm must be finite and > 0 (got %g)", fn, max_norm);
  if (!norm_out || !coef_out || !nonfinite_out)
    return zs::fail(ZS_ERR_INVAL, "%s: norm_out, coef_out or nonfinite_out is NULL", fn);
  return list_call(fn, a, workspace_bytes, true, true, cuda_stream);
}
