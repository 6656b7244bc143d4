// losses_api.cpp — the C entry points of the losses over vocabulary rows:
// argument checks, then one launch. As in api.cpp, every check runs before
// anything is enqueued.
#include <cuda_runtime.h>

#include "buffers.h"
#include "zs_internal.h"

namespace {

const char* const kLogits = "logits";
const char* const kGrad = "d_logits";

// Sizes, dtype, stride and temperature.
zs_status check_rows(const char* fn, const zs::VocabLaunch& a) {
  if (a.dtype != ZS_BF16 && a.dtype != ZS_FP32)
    return zs::fail(ZS_ERR_INVAL, "%s: logits dtype %d is not bf16 or fp32", fn, (int)a.dtype);
  if (a.rows < 0 || a.rows > 0x7FFFFFFF)
    return zs::fail(ZS_ERR_RANGE, "%s: rows %lld outside 0..2^31-1", fn, (long long)a.rows);
  if (a.vocab < 1 || a.vocab > ZS_MAX_VOCAB)
    return zs::fail(ZS_ERR_RANGE, "%s: vocab %lld outside 1..%d", fn, (long long)a.vocab,
                    ZS_MAX_VOCAB);
  if (zs_status st =
          zs::check_stride(fn, "row_stride", a.row_stride, a.rows, a.vocab, "vocab"))
    return st;
  if (a.d_logits)
    if (zs_status st =
            zs::check_stride(fn, "grad_stride", a.grad_stride, a.rows, a.vocab, "vocab"))
      return st;
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
  zs::Buffers b(fn);
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
  if (in_place) b.may_share(kGrad, kLogits);
  return b.check();
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
  return zs::launched(fn, zs::launch_vocab_loss(a, static_cast<cudaStream_t>(cuda_stream)));
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
  return zs::launched(fn, zs::launch_vocab_grad(a, static_cast<cudaStream_t>(cuda_stream)));
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
  return zs::launched(fn, zs::launch_vocab_loss(a, static_cast<cudaStream_t>(cuda_stream)));
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
  return zs::launched(fn, zs::launch_vocab_grad(a, static_cast<cudaStream_t>(cuda_stream)));
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
  return zs::launched(fn, zs::launch_vocab_loss(a, static_cast<cudaStream_t>(cuda_stream)));
}
