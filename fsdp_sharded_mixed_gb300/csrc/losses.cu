// losses.cu — losses over vocabulary rows and their gradients: the log
// probability of a given token with the row's entropy and top alternatives,
// and the distillation loss against a teacher's top logits.
//
// Mathematics, for one row z of V logits at temperature T, with y = z / T,
// M = max z and everything in fp32:
//   S   = sum_j exp(y_j - M/T)        lse = M/T + ln S
//   U   = sum_j e_j d_j,  e_j = exp(y_j - M/T) = 2^d_j
//   H   = ln S - ln 2 * U / S         (every term of U is <= 0: no cancellation)
//   ln p_t = (z_t - M)/T - ln S
//   loss = sum_k q_k (ln q_k - ln p_{id_k})
// Gradients are p_j times a row constant (plus, for the entropy, a multiple of
// p_j ln p_j), except at the few columns that are the target or a teacher's id.
//
// z - M is formed before the scaling: both may be the type's lowest value (a
// row masked with it), whose product with 1/T is no longer finite.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bounds.cuh"
#include "overlap.cuh"
#include "zs_internal.h"

namespace zs {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 256;

struct RowArgs {
  const void* logits;
  void* d_logits;
  int64_t row_stride, grad_stride;
  int32_t vocab, top_k, teacher_k;
  bool teacher_bf16;
  bool distill;   // targets are hard labels at T = 1
  bool hard_own;  // T != 1, and the hard labels' softmax is wanted as well
  float inv_t, scale;                 // 1/T, log2(e)/T
  const int64_t* targets;
  const int32_t* teacher_ids;
  const void* teacher_logits;
  const float *teacher_lse, *in_lse, *in_entropy, *in_hard_lse, *d_loss, *d_logprob, *d_entropy;
  float *logprob, *entropy, *lse, *loss, *hard_lse, *top_logprobs;
  int32_t* top_ids;
  unsigned int* err;
};

__device__ __forceinline__ float value_of(float x) { return x; }
__device__ __forceinline__ float value_of(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store(float* p, float x) { *p = x; }
// The gradient's one rounding to fewer bits: to nearest even.
__device__ __forceinline__ void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename F>
__device__ __forceinline__ float block_reduce(float x, float* sm, F f) {
  for (int off = 16; off > 0; off >>= 1) x = f(x, __shfl_xor_sync(0xFFFFFFFFu, x, off));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
  __syncthreads();
  x = sm[0];
  for (int w = 1; w < kThreads / 32; ++w) x = f(x, sm[w]);
  return x;
}

// Unique keys that order logits as the alternatives are ranked: NaN above all,
// then by value (-0 as +0), then the lowest column first.
__device__ __forceinline__ uint64_t rank_key(float z, int32_t column) {
  uint32_t u = __float_as_uint(z + 0.0f);
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  if (z != z) u = 0xFFFFFFFFu;
  return ((uint64_t)u << 32) | (uint32_t)~column;
}

__device__ __forceinline__ float teacher_logit(const RowArgs& a, int64_t i) {
  return a.teacher_bf16 ? value_of(static_cast<const __nv_bfloat16*>(a.teacher_logits)[i])
                        : static_cast<const float*>(a.teacher_logits)[i];
}

// One block per row. LOSS: statistics and losses from the logits; GRAD: the
// gradient, from them or from the forward call's normalisers.
template <typename T, bool LOSS, bool GRAD>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ RowArgs a) {
  overlap_wait();
  const int64_t r = blockIdx.x;
  const int V = a.vocab, K = a.teacher_k, tid = threadIdx.x;
  const T* z = static_cast<const T*>(a.logits) + r * a.row_stride;
  __shared__ float sm[kThreads / 32];
  __shared__ uint64_t sm_key[kThreads / 32];
  __shared__ int32_t s_id[ZS_MAX_TEACHER + 1];
  __shared__ float s_q[ZS_MAX_TEACHER], s_lnq[ZS_MAX_TEACHER], s_z[ZS_MAX_TEACHER + 1];
  auto fmax_ = [](float x, float y) { return fmaxf(x, y); };
  auto fadd_ = [](float x, float y) { return x + y; };

  // The target (-1: none) and the teacher's record with its softmax q.
  int32_t target = -1;
  bool bad_target = false;
  if (a.targets) {
    const int64_t t = a.targets[r];
    bad_target = t >= V;
    if (bad_target && tid == 0) atomicOr(a.err, 1u);
    target = t < 0 || bad_target ? -1 : (int32_t)t;
  }
  float Q = 0.0f;
  if (K > 0) {
    int32_t id = -1;
    float u = -INFINITY;
    if (tid < K) {
      id = a.teacher_ids[r * K + tid];
      if (id >= V) {
        atomicOr(a.err, 1u);
        id = -1;
      }
      if (id >= 0) u = teacher_logit(a, r * K + tid) * a.inv_t;
    }
    float lnq;
    if (a.teacher_lse) {
      lnq = u - a.teacher_lse[r];
    } else {
      float m = block_reduce(u, sm, fmax_);
      if (m == -INFINITY) m = 0.0f;
      const float s = block_reduce(id >= 0 ? expf(u - m) : 0.0f, sm, fadd_);
      lnq = u - m - logf(s);
    }
    const float q = id >= 0 && u != -INFINITY ? expf(lnq) : 0.0f;
    Q = block_reduce(q, sm, fadd_);
    if (tid < K) {
      s_id[tid] = id;
      s_q[tid] = q;
      s_lnq[tid] = lnq;
      s_z[tid] = id >= 0 ? value_of(z[id]) : 0.0f;
    }
  }
  const float z_target = target >= 0 ? value_of(z[target]) : 0.0f;
  if (GRAD && tid == 0) {
    s_id[K] = target;
    s_z[K] = z_target;
  }
  __syncthreads();

  // Statistics.
  float M = 0.0f, S = 1.0f, S1 = 1.0f, lse = 0.0f, lse1 = 0.0f;
  if (LOSS) {
    float m = -INFINITY;
    for (int j = tid; j < V; j += kThreads) m = fmaxf(m, value_of(z[j]));
    m = block_reduce(m, sm, fmax_);
    M = m == -INFINITY ? 0.0f : m;  // a row masked throughout: every e is 2^-inf = 0
    float s = 0.0f, u = 0.0f, s1 = 0.0f;
    for (int j = tid; j < V; j += kThreads) {
      const float x = value_of(z[j]) - M;
      const float d = x * a.scale, e = exp2f(d);
      s += e;
      u = fmaf(e, fmaxf(d, -1e4f), u);  // e is 0 below the clamp, and 0 * -inf is not
      if (a.hard_own) s1 += exp2f(x * kLog2e);
    }
    S = block_reduce(s, sm, fadd_);
    const float U = block_reduce(u, sm, fadd_);
    S1 = a.hard_own ? block_reduce(s1, sm, fadd_) : S;
    const bool empty = m == -INFINITY && S == 0.0f;
    const float ln_s = logf(S), ln_s1 = a.hard_own ? logf(S1) : ln_s;
    lse = empty ? -INFINITY : fmaf(M, a.inv_t, ln_s);
    lse1 = empty ? -INFINITY : M + ln_s1;
    if (tid == 0) {
      if (a.lse) a.lse[r] = lse;
      if (a.hard_lse) a.hard_lse[r] = lse1;
      if (a.entropy) a.entropy[r] = empty ? 0.0f : ln_s - kLn2 * (U / S);
      if (a.logprob) {
        const float t = a.distill ? 1.0f : a.inv_t;
        a.logprob[r] = bad_target       ? NAN
                       : target < 0     ? 0.0f
                       : empty          ? -INFINITY
                                        : (z_target - M) * t - (a.distill ? ln_s1 : ln_s);
      }
    }
    if (a.loss) {
      float l = 0.0f;
      if (tid < K && !(s_q[tid] == 0.0f))
        l = s_q[tid] * (s_lnq[tid] - (empty ? -INFINITY : (s_z[tid] - M) * a.inv_t - ln_s));
      l = block_reduce(l, sm, fadd_);
      if (tid == 0) a.loss[r] = l;
    }
    // The alternatives: the largest key below the last one, top_k times.
    uint64_t last = ~0ull;
    for (int k = 0; k < a.top_k; ++k) {
      uint64_t best = 0;
      for (int j = tid; j < V; j += kThreads) {
        const uint64_t key = rank_key(value_of(z[j]), j);
        if (key < last && key > best) best = key;
      }
      for (int off = 16; off > 0; off >>= 1) {
        const uint64_t o = __shfl_xor_sync(0xFFFFFFFFu, best, off);
        if (o > best) best = o;
      }
      __syncthreads();
      if ((tid & 31) == 0) sm_key[tid >> 5] = best;
      __syncthreads();
      best = sm_key[0];
      for (int w = 1; w < kThreads / 32; ++w)
        if (sm_key[w] > best) best = sm_key[w];
      last = best;
      if (tid == 0) {
        const int32_t id = (int32_t)~(uint32_t)best;
        a.top_ids[r * a.top_k + k] = id;
        a.top_logprobs[r * a.top_k + k] =
            empty ? -INFINITY : (value_of(z[id]) - M) * a.inv_t - ln_s;
      }
    }
  }

  if (GRAD) {
    // g_j = e_j (A + B d_j) [+ e1_j A1], e_j = 2^((z_j - M) scale).
    T* g = static_cast<T*>(a.d_logits) + r * a.grad_stride;
    const float al = a.d_logprob && target >= 0 ? a.d_logprob[r] : 0.0f;
    const float w = a.d_loss ? a.d_loss[r] : 0.0f, b = a.d_entropy ? a.d_entropy[r] : 0.0f;
    float A = 0.0f, B = 0.0f, A1 = 0.0f, M1 = M, at_target = 0.0f;
    bool zero;
    if (LOSS) {
      zero = lse == -INFINITY;
      A = w * a.inv_t * Q / S;
      if (a.hard_own)
        A1 = -al / S1;
      else
        A -= al / S;
      at_target = al;
    } else if (a.distill) {
      if (a.in_hard_lse) lse = lse1 = a.in_hard_lse[r];
      if (a.in_lse) lse = a.in_lse[r];
      zero = lse == -INFINITY;
      M = lse / a.inv_t;
      M1 = lse1;
      A = w * a.inv_t * Q;
      if (a.hard_own)
        A1 = -al;
      else
        A -= al;
      at_target = al;
    } else {
      lse = a.in_lse[r];
      zero = lse == -INFINITY;
      M = lse / a.inv_t;
      A = -(al + (b == 0.0f ? 0.0f : b * a.in_entropy[r])) * a.inv_t;
      B = -b * kLn2 * a.inv_t;
      at_target = al * a.inv_t;
    }
    zero = zero || (al == 0.0f && w == 0.0f && b == 0.0f);
    auto smooth = [&](float zj) {
      const float d = (zj - M) * a.scale;
      float x = 0.0f;
      if (A != 0.0f || B != 0.0f) x = exp2f(d) * fmaf(B, fmaxf(d, -1e4f), A);
      if (A1 != 0.0f) x = fmaf(exp2f((zj - M1) * kLog2e), A1, x);
      return x;
    };
    for (int j = tid; j < V; j += kThreads) store(g + j, zero ? 0.0f : smooth(value_of(z[j])));
    __syncthreads();
    // The columns of the target and the teacher's ids, from the logits kept
    // above (z may be overwritten by now). Equal ids all store the same value.
    for (int k = tid; k <= K; k += kThreads) {
      const int32_t id = s_id[k];
      if (id < 0 || zero) continue;
      float q = 0.0f;
      for (int i = 0; i < K; ++i)
        if (s_id[i] == id) q += s_q[i];
      float x = smooth(s_z[k]) - w * a.inv_t * q;
      if (id == target) x += at_target;
      store(g + id, x);
    }
  }
}

RowArgs row_args(const VocabLaunch& in) {
  RowArgs a = {};
  a.logits = in.logits;
  a.d_logits = in.d_logits;
  a.row_stride = in.row_stride;
  a.grad_stride = in.grad_stride;
  a.vocab = (int32_t)in.vocab;
  a.top_k = in.top_k;
  a.teacher_k = in.teacher_k;
  a.teacher_bf16 = in.teacher_dtype == ZS_BF16;
  a.distill = in.distill;
  a.hard_own = in.distill && in.temperature != 1.0 &&
               (in.logprob || in.hard_lse || in.d_logprob);
  a.inv_t = (float)(1.0 / in.temperature);
  a.scale = (float)(1.4426950408889634 / in.temperature);
  a.targets = in.targets;
  a.teacher_ids = in.teacher_ids;
  a.teacher_logits = in.teacher_logits;
  a.teacher_lse = in.teacher_lse;
  a.in_lse = in.in_lse;
  a.in_entropy = in.in_entropy;
  a.in_hard_lse = in.in_hard_lse;
  a.d_loss = in.d_loss;
  a.d_logprob = in.d_logprob;
  a.d_entropy = in.d_entropy;
  a.logprob = in.logprob;
  a.entropy = in.entropy;
  a.lse = in.lse;
  a.loss = in.loss;
  a.hard_lse = in.hard_lse;
  a.top_ids = in.top_ids;
  a.top_logprobs = in.top_logprobs;
  a.err = device_error_word();
  return a;
}

template <bool LOSS, bool GRAD>
cudaError_t launch(const VocabLaunch& in, cudaStream_t stream) {
  const RowArgs a = row_args(in);
  if (!a.err) return cudaErrorInvalidSymbol;
  const dim3 grid((unsigned)in.rows);
  return in.dtype == ZS_BF16
             ? launch_kernel(rows_kernel<__nv_bfloat16, LOSS, GRAD>, grid, dim3(kThreads), 0,
                             stream, a)
             : launch_kernel(rows_kernel<float, LOSS, GRAD>, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_vocab_loss(const VocabLaunch& a, cudaStream_t stream) {
  return a.d_logits ? launch<true, true>(a, stream) : launch<true, false>(a, stream);
}

cudaError_t launch_vocab_grad(const VocabLaunch& a, cudaStream_t stream) {
  return launch<false, true>(a, stream);
}

}  // namespace zs
