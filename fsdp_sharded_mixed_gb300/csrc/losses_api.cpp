// losses_api.cpp — the C entry points of the losses over vocabulary rows:
// argument checks, then one launch. As in api.cpp, every check runs before
// anything is enqueued.
#include <cuda_runtime.h>

#include "zs_internal.h"

namespace {

// The buffers of one call, checked as they are added: natural alignment here,
// then (check) outputs against every other buffer and each one's residency.
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
  // in_place: the buffers named so may be one and the same.
  zs_status check(const char* in_place_out, const char* in_place_in) const {
    for (int a = 0; a < n_; ++a) {
      if (!items_[a].output) continue;
      for (int b = 0; b < n_; ++b) {
        if (a == b || items_[a].lo >= items_[b].hi || items_[b].lo >= items_[a].hi) continue;
        if (items_[a].name == in_place_out && items_[b].name == in_place_in &&
            items_[a].lo == items_[b].lo && items_[a].hi == items_[b].hi)
          continue;
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
  const char* fn_;
  Item items_[20];
  int n_ = 0;
};

const char* const kLogits = "logits";
const char* const kGrad = "d_logits";

// The rows of one matrix: (rows - 1) * stride + vocab elements, kMaxExtent at most
// (2^46 bytes of fp32, past any device's memory), so that no product of them wraps.
constexpr int64_t kMaxExtent = int64_t(1) << 44;
zs_status check_stride(const char* fn, const char* name, int64_t stride,
                       const zs::VocabLaunch& a) {
  if (stride < a.vocab || stride > int64_t(1) << 40)
    return zs::fail(ZS_ERR_RANGE, "%s: %s %lld outside vocab..2^40", fn, name, (long long)stride);
  if (a.rows > 1 && stride > (kMaxExtent - a.vocab) / (a.rows - 1))
    return zs::fail(ZS_ERR_RANGE, "%s: %lld rows %s %lld apart are more than 2^44 elements", fn,
                    (long long)a.rows, name, (long long)stride);
  return ZS_OK;
}

// Sizes, dtype, stride and temperature.
zs_status check_rows(const char* fn, const zs::VocabLaunch& a) {
  if (a.dtype != ZS_BF16 && a.dtype != ZS_FP32)
    return zs::fail(ZS_ERR_INVAL, "%s: logits dtype %d is not bf16 or fp32", fn, (int)a.dtype);
  if (a.rows < 0 || a.rows > 0x7FFFFFFF)
    return zs::fail(ZS_ERR_RANGE, "%s: rows %lld outside 0..2^31-1", fn, (long long)a.rows);
  if (a.vocab < 1 || a.vocab > ZS_MAX_VOCAB)
    return zs::fail(ZS_ERR_RANGE, "%s: vocab %lld outside 1..%d", fn, (long long)a.vocab,
                    ZS_MAX_VOCAB);
  if (zs_status st = check_stride(fn, "row_stride", a.row_stride, a)) return st;
  if (a.d_logits)
    if (zs_status st = check_stride(fn, "grad_stride", a.grad_stride, a)) return st;
  // (log2(e)/T is finite in fp32 and 1/T normal, and so is T times an lse of flat rows)
  if (!(a.temperature >= 1e-38 && a.temperature <= 1e37))
    return zs::fail(ZS_ERR_INVAL, "%s: temperature must be within 1e-38..1e37 (got %g)", fn,
                    a.temperature);
  return ZS_OK;
}

// Every buffer the launch structure names, with the bytes the kernels touch.
zs_status check_buffers(const char* fn, const zs::VocabLaunch& a) {
  const int es = zs::elem_bytes(a.dtype);
  const int64_t R = a.rows;
  Buffers b(fn);
  if (zs_status st = b.need(kLogits, a.logits, ((R - 1) * a.row_stride + a.vocab) * es, es, false))
    return st;
  if (zs_status st = b.add("targets", a.targets, R * 8, 8, false)) return st;
  if (a.teacher_k > 0) {
    const int ts = zs::elem_bytes(a.teacher_dtype);
    if (zs_status st = b.need("teacher_ids", a.teacher_ids, R * a.teacher_k * 4, 4, false))
      return st;
    if (zs_status st =
            b.need("teacher_logits", a.teacher_logits, R * a.teacher_k * ts, ts, false))
      return st;
    if (zs_status st = b.add("teacher_lse", a.teacher_lse, R * 4, 4, false)) return st;
  }
  const struct {
    const char* name;
    const void* p;
    bool output;
  } per_row[] = {{"logprob", a.logprob, true},       {"entropy", a.entropy, true},
                 {"lse", a.lse, true},               {"loss", a.loss, true},
                 {"hard_lse", a.hard_lse, true},     {"lse", a.in_lse, false},
                 {"entropy", a.in_entropy, false},   {"hard_lse", a.in_hard_lse, false},
                 {"d_loss", a.d_loss, false},        {"d_logprob", a.d_logprob, false},
                 {"d_entropy", a.d_entropy, false}};
  for (const auto& x : per_row)
    if (zs_status st = b.add(x.name, x.p, R * 4, 4, x.output)) return st;
  if (a.top_k > 0) {
    if (zs_status st = b.need("top_ids", a.top_ids, R * a.top_k * 4, 4, true)) return st;
    if (zs_status st = b.need("top_logprobs", a.top_logprobs, R * a.top_k * 4, 4, true)) return st;
  }
  if (zs_status st = b.add(kGrad, a.d_logits, ((R - 1) * a.grad_stride + a.vocab) * es, es, true))
    return st;
  const bool in_place = a.d_logits && a.d_logits == a.logits && a.grad_stride == a.row_stride;
  return b.check(in_place ? kGrad : nullptr, kLogits);
}

zs_status check_teacher(const char* fn, const zs::VocabLaunch& a) {
  if (a.teacher_k < 0 || a.teacher_k > ZS_MAX_TEACHER)
    return zs::fail(ZS_ERR_RANGE, "%s: teacher_k %d outside 0..%d", fn, a.teacher_k,
                    ZS_MAX_TEACHER);
  if (a.teacher_k > 0 && a.teacher_dtype != ZS_BF16 && a.teacher_dtype != ZS_FP32)
    return zs::fail(ZS_ERR_INVAL, "%s: teacher dtype %d is not bf16 or fp32", fn,
                    (int)a.teacher_dtype);
  return ZS_OK;
}

zs_status launched(const char* fn, cudaError_t e) {
  if (e != cudaSuccess)
    return zs::fail(ZS_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  return ZS_OK;
}

zs::VocabLaunch rows_of(const void* logits, zs_dtype dtype, int64_t rows, int64_t vocab,
                        int64_t row_stride, const int64_t* targets, double temperature) {
  zs::VocabLaunch a = {};
  a.logits = logits;
  a.dtype = dtype;
  a.rows = rows;
  a.vocab = vocab;
  a.row_stride = row_stride;
  a.targets = targets;
  a.temperature = temperature;
  return a;
}

void set_teacher(zs::VocabLaunch* a, const int32_t* ids, const void* logits, zs_dtype dtype,
                 int32_t k, const float* lse) {
  a->distill = true;
  a->teacher_ids = ids;
  a->teacher_logits = logits;
  a->teacher_dtype = dtype;
  a->teacher_k = k;
  a->teacher_lse = lse;
}

}  // namespace

extern "C" zs_status zs_token_logprobs(const void* logits, zs_dtype dtype, int64_t rows,
                                       int64_t vocab, int64_t row_stride, const int64_t* targets,
                                       double temperature, float* logprob, float* entropy,
                                       float* lse, int32_t top_k, int32_t* top_ids,
                                       float* top_logprobs, void* cuda_stream) {
  static const char* fn = "zs_token_logprobs";
  const zs::CallRange range(fn);
  zs::clear_error();
  zs::VocabLaunch a = rows_of(logits, dtype, rows, vocab, row_stride, targets, temperature);
  a.logprob = logprob;
  a.entropy = entropy;
  a.lse = lse;
  a.top_k = top_k;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  if (zs_status st = check_rows(fn, a)) return st;
  if (top_k < 0 || top_k > ZS_MAX_TOP || top_k > vocab)
    return zs::fail(ZS_ERR_RANGE, "%s: top_k %d outside 0..min(vocab, %d)", fn, top_k, ZS_MAX_TOP);
  if (!logprob && !entropy && !lse && top_k == 0)
    return zs::fail(ZS_ERR_INVAL, "%s: no output", fn);
  if (rows == 0) return ZS_OK;
  if (logprob && !targets) return zs::fail(ZS_ERR_INVAL, "%s: logprob needs targets", fn);
  if (zs_status st = check_buffers(fn, a)) return st;
  return launched(fn, zs::launch_vocab_loss(a, static_cast<cudaStream_t>(cuda_stream)));
}

extern "C" zs_status zs_token_logprobs_grad(const void* logits, zs_dtype dtype, int64_t rows,
                                            int64_t vocab, int64_t row_stride,
                                            const int64_t* targets, double temperature,
                                            const float* lse, const float* entropy,
                                            const float* d_logprob, const float* d_entropy,
                                            void* d_logits, int64_t grad_stride,
                                            void* cuda_stream) {
  static const char* fn = "zs_token_logprobs_grad";
  const zs::CallRange range(fn);
  zs::clear_error();
  zs::VocabLaunch a = rows_of(logits, dtype, rows, vocab, row_stride, targets, temperature);
  a.in_lse = lse;
  a.in_entropy = entropy;
  a.d_logprob = d_logprob;
  a.d_entropy = d_entropy;
  a.d_logits = d_logits;
  a.grad_stride = grad_stride;
  if (zs_status st = check_rows(fn, a)) return st;
  if (rows == 0) return ZS_OK;
  if (!d_logits || !lse) return zs::fail(ZS_ERR_INVAL, "%s: NULL buffer", fn);
  if (!d_logprob && !d_entropy) return zs::fail(ZS_ERR_INVAL, "%s: no upstream gradient", fn);
  if (d_logprob && !targets) return zs::fail(ZS_ERR_INVAL, "%s: d_logprob needs targets", fn);
  if (d_entropy && !entropy) return zs::fail(ZS_ERR_INVAL, "%s: d_entropy needs entropy", fn);
  if (zs_status st = check_buffers(fn, a)) return st;
  return launched(fn, zs::launch_vocab_grad(a, static_cast<cudaStream_t>(cuda_stream)));
}

extern "C" zs_status zs_distill_loss(const void* logits, zs_dtype dtype, int64_t rows,
                                     int64_t vocab, int64_t row_stride,
                                     const int32_t* teacher_ids, const void* teacher_logits,
                                     zs_dtype teacher_dtype, int32_t teacher_k,
                                     const float* teacher_lse, double temperature,
                                     const int64_t* targets, float* loss, float* lse,
                                     float* logprob, float* hard_lse, void* cuda_stream) {
  static const char* fn = "zs_distill_loss";
  const zs::CallRange range(fn);
  zs::clear_error();
  zs::VocabLaunch a = rows_of(logits, dtype, rows, vocab, row_stride, targets, temperature);
  set_teacher(&a, teacher_ids, teacher_logits, teacher_dtype, teacher_k, teacher_lse);
  a.loss = loss;
  a.lse = lse;
  a.logprob = logprob;
  a.hard_lse = hard_lse;
  if (zs_status st = check_rows(fn, a)) return st;
  if (zs_status st = check_teacher(fn, a)) return st;
  if (!loss && !lse && !logprob && !hard_lse) return zs::fail(ZS_ERR_INVAL, "%s: no output", fn);
  if (loss && teacher_k == 0) return zs::fail(ZS_ERR_INVAL, "%s: loss needs a teacher", fn);
  if (rows == 0) return ZS_OK;
  if (logprob && !targets) return zs::fail(ZS_ERR_INVAL, "%s: logprob needs targets", fn);
  if (zs_status st = check_buffers(fn, a)) return st;
  return launched(fn, zs::launch_vocab_loss(a, static_cast<cudaStream_t>(cuda_stream)));
}

extern "C" zs_status zs_distill_grad(const void* logits, zs_dtype dtype, int64_t rows,
                                     int64_t vocab, int64_t row_stride,
                                     const int32_t* teacher_ids, const void* teacher_logits,
                                     zs_dtype teacher_dtype, int32_t teacher_k,
                                     const float* teacher_lse, double temperature,
                                     const int64_t* targets, const float* lse,
                                     const float* hard_lse, const float* d_loss,
                                     const float* d_logprob, void* d_logits, int64_t grad_stride,
                                     void* cuda_stream) {
  static const char* fn = "zs_distill_grad";
  const zs::CallRange range(fn);
  zs::clear_error();
  zs::VocabLaunch a = rows_of(logits, dtype, rows, vocab, row_stride, targets, temperature);
  set_teacher(&a, teacher_ids, teacher_logits, teacher_dtype, teacher_k, teacher_lse);
  a.in_lse = lse;
  a.in_hard_lse = hard_lse;
  a.d_loss = d_loss;
  a.d_logprob = d_logprob;
  a.d_logits = d_logits;
  a.grad_stride = grad_stride;
  if (zs_status st = check_rows(fn, a)) return st;
  if (zs_status st = check_teacher(fn, a)) return st;
  if (rows == 0) return ZS_OK;
  if (!d_logits) return zs::fail(ZS_ERR_INVAL, "%s: d_logits is NULL", fn);
  if (!d_loss && !d_logprob) return zs::fail(ZS_ERR_INVAL, "%s: no upstream gradient", fn);
  if (d_loss && (!lse || teacher_k == 0))
    return zs::fail(ZS_ERR_INVAL, "%s: d_loss needs a teacher and lse", fn);
  if (d_logprob && (!targets || !hard_lse))
    return zs::fail(ZS_ERR_INVAL, "%s: d_logprob needs targets and hard_lse", fn);
  if (zs_status st = check_buffers(fn, a)) return st;
  return launched(fn, zs::launch_vocab_grad(a, static_cast<cudaStream_t>(cuda_stream)));
}

extern "C" zs_status zs_distill_loss_grad(const void* logits, zs_dtype dtype, int64_t rows,
                                          int64_t vocab, int64_t row_stride,
                                          const int32_t* teacher_ids, const void* teacher_logits,
                                          zs_dtype teacher_dtype, int32_t teacher_k,
                                          const float* teacher_lse, double temperature,
                                          const int64_t* targets, const float* d_loss,
                                          const float* d_logprob, float* loss, float* lse,
                                          float* logprob, float* hard_lse, void* d_logits,
                                          int64_t grad_stride, void* cuda_stream) {
  static const char* fn = "zs_distill_loss_grad";
  const zs::CallRange range(fn);
  zs::clear_error();
  zs::VocabLaunch a = rows_of(logits, dtype, rows, vocab, row_stride, targets, temperature);
  set_teacher(&a, teacher_ids, teacher_logits, teacher_dtype, teacher_k, teacher_lse);
  a.loss = loss;
  a.lse = lse;
  a.logprob = logprob;
  a.hard_lse = hard_lse;
  a.d_loss = d_loss;
  a.d_logprob = d_logprob;
  a.d_logits = d_logits;
  a.grad_stride = grad_stride;
  if (zs_status st = check_rows(fn, a)) return st;
  if (zs_status st = check_teacher(fn, a)) return st;
  if (rows == 0) return ZS_OK;
  if (!d_logits) return zs::fail(ZS_ERR_INVAL, "%s: d_logits is NULL", fn);
  if (!d_loss && !d_logprob) return zs::fail(ZS_ERR_INVAL, "%s: no upstream gradient", fn);
  if ((d_loss || loss) && teacher_k == 0)
    return zs::fail(ZS_ERR_INVAL, "%s: loss and d_loss need a teacher", fn);
  if ((d_logprob || logprob) && !targets)
    return zs::fail(ZS_ERR_INVAL, "%s: logprob and d_logprob need targets", fn);
  if (zs_status st = check_buffers(fn, a)) return st;
  return launched(fn, zs::launch_vocab_loss(a, static_cast<cudaStream_t>(cuda_stream)));
}
