// tensors.cu — the global norm of a list of gradients, and clipping.
//
//   n = sqrt(sum_i sum_k g_ik^2),  c = min(1, max_norm / (n + 1e-6)),  out_ik = c g_ik
//
// The list's addresses and lengths are kernel parameters (no table in device
// memory, nothing to copy before the launch). Every tensor is cut into chunks of
// kChunk elements, and the blocks stride over the chunks of the whole list, so
// that the load is even however unequal the tensors are.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bounds.cuh"
#include "overlap.cuh"
#include "row_vec.cuh"
#include "zs_internal.h"

namespace zs {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;  // elements

template <int MAXN>
struct ListArgs {
  const void* in[MAXN];
  void* out[MAXN];
  int64_t numel[MAXN];
  int64_t first[MAXN + 1];  // chunks of the tensors before
  int32_t count;
  bool begins, ends;        // the launches of one list follow one another
  double* partials;         // [kNormPartials], then the ticket
  unsigned int* ticket;
  double* sqnorm;
  double max_norm;          // 0: no coefficient
  float *norm, *coef_out;
  int32_t* nonfinite_out;
  const float* coef;        // scaling
  const int32_t* skip;
  unsigned int* err;
};

template <int MAXN>
__device__ __forceinline__ int tensor_of(const ListArgs<MAXN>& a, int64_t chunk) {
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The sum of the squares of eight elements in fp32, unless it left fp32's range
// (or is so small that squares may have): then in double.
__device__ __forceinline__ double squares(const float* v) {
  float s = 0.0f, m = 0.0f;
#pragma unroll
  for (int k = 0; k < kLane; ++k) {
    s = __fmaf_rn(v[k], v[k], s);
    m = fmaxf(m, fabsf(v[k]));
  }
  if (s > 1e-25f && s < 1e37f) return s;
  if (m == 0.0f && s == 0.0f) return 0.0;
  double d = 0.0;
#pragma unroll
  for (int k = 0; k < kLane; ++k) d += (double)v[k] * (double)v[k];
  return d;
}

template <typename T, int MAXN>
__global__ void __launch_bounds__(kThreads) list_sqnorm_kernel(const __grid_constant__ ListArgs<MAXN> a) {
  overlap_wait();
  const int64_t chunks = a.first[a.count];
  double sum = 0.0;
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int t = tensor_of(a, c);
    const int64_t from = (c - a.first[t]) * kChunk;
    const int64_t left = a.numel[t] - from;
    const int n = (int)(left < kChunk ? left : kChunk);
    if (!within(from, from + n, 0, a.numel[t], a.err)) continue;
    const T* p = static_cast<const T*>(a.in[t]) + from;
    const bool vec = (uintptr_t)p % 16 == 0;
    const int lane = threadIdx.x & 31;
    for (int col0 = threadIdx.x / 32 * kSlab; col0 < n; col0 += kThreads / 32 * kSlab) {
      const Raw8<T> r = vec ? load8<T, kEight>(p, col0, lane, n) : load8<T, kOne>(p, col0, lane, n);
      float v[kLane];
#pragma unroll
      for (int k = 0; k < kLane; ++k) v[k] = raw_value(r, k);
      sum += squares(v);
    }
  }
  __shared__ double warp_sums[kThreads / 32];
  __shared__ bool last;
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_down_sync(0xFFFFFFFFu, sum, off);
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double b = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) b += warp_sums[w];
    if (within(blockIdx.x, blockIdx.x + 1, 0, kNormPartials, a.err)) a.partials[blockIdx.x] = b;
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  // The last block adds the partials in a fixed order.
  __threadfence();
  double t = 0.0;
  for (int b = threadIdx.x; b < (int)gridDim.x; b += kThreads) t += __ldcg(a.partials + b);
  for (int off = 16; off > 0; off >>= 1) t += __shfl_down_sync(0xFFFFFFFFu, t, off);
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = t;
  __syncthreads();
  if (threadIdx.x != 0) return;
  double total = a.begins ? 0.0 : *a.sqnorm;
  for (int w = 0; w < kThreads / 32; ++w) total += warp_sums[w];
  *a.sqnorm = total;
  *a.ticket = 0u;
  if (!a.ends || a.max_norm == 0.0) return;
  const double norm = sqrt(total);
  const bool bad = !isfinite(norm);
  const double c = a.max_norm / (norm + 1e-6);
  *a.norm = (float)norm;
  *a.nonfinite_out = bad ? 1 : 0;
  *a.coef_out = bad ? 1.0f : (float)(c < 1.0 ? c : 1.0);
}

template <typename T, typename OT, int MAXN>
__global__ void __launch_bounds__(kThreads) list_scale_kernel(const __grid_constant__ ListArgs<MAXN> a) {
  overlap_wait();
  if (a.skip && *a.skip) return;
  const float coef = *a.coef;
  const int64_t chunks = a.first[a.count];
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int t = tensor_of(a, c);
    if (coef == 1.0f && a.in[t] == a.out[t]) continue;  // in place: nothing changes
    const int64_t from = (c - a.first[t]) * kChunk;
    const int64_t left = a.numel[t] - from;
    const int n = (int)(left < kChunk ? left : kChunk);
    if (!within(from, from + n, 0, a.numel[t], a.err)) continue;
    const T* p = static_cast<const T*>(a.in[t]) + from;
    OT* q = static_cast<OT*>(a.out[t]) + from;
    const bool vec = ((uintptr_t)p | (uintptr_t)q) % 16 == 0;
    const int lane = threadIdx.x & 31;
    for (int col0 = threadIdx.x / 32 * kSlab; col0 < n; col0 += kThreads / 32 * kSlab) {
      const Raw8<T> r = vec ? load8<T, kEight>(p, col0, lane, n) : load8<T, kOne>(p, col0, lane, n);
      float v[kLane];
#pragma unroll
      for (int k = 0; k < kLane; ++k) v[k] = raw_value(r, k) * coef;
      if (vec)
        store8<OT, kEight>(q, col0, lane, n, v);
      else
        store8<OT, kOne>(q, col0, lane, n, v);
    }
  }
}

constexpr int kMostListed = 768;  // tensors of one launch

template <int MAXN>
cudaError_t launch_part(const TensorsLaunch& in, int64_t from, int n, cudaStream_t stream) {
  ListArgs<MAXN> a;
  a.count = 0;
  a.first[0] = 0;
  for (int64_t i = from; i < from + n; ++i) {
    if (in.numels[i] == 0) continue;
    const int k = a.count++;
    a.in[k] = in.tensors[i];
    a.out[k] = in.outs ? in.outs[i] : nullptr;
    a.numel[k] = in.numels[i];
    a.first[k + 1] = a.first[k] + (in.numels[i] + kChunk - 1) / kChunk;
  }
  a.begins = from == 0;
  a.ends = from + n >= in.count;
  a.partials = static_cast<double*>(in.workspace);
  a.ticket = reinterpret_cast<unsigned int*>(static_cast<unsigned char*>(in.workspace) +
                                             kNormTicketOffset);
  a.sqnorm = in.sqnorm;
  a.max_norm = in.max_norm;
  a.norm = in.norm;
  a.coef_out = in.coef_out;
  a.nonfinite_out = in.nonfinite_out;
  a.coef = in.coef;
  a.skip = in.skip;
  a.err = ZS_BOUNDS_CHECK ? device_error_word() : nullptr;
  if (ZS_BOUNDS_CHECK && !a.err) return cudaErrorInvalidSymbol;
  const int64_t chunks = a.first[a.count];
  const bool bf16 = in.dtype == ZS_BF16;
  if (!in.coef) {
    cudaError_t e = cudaMemsetAsync(a.ticket, 0, sizeof(unsigned int), stream);
    if (e != cudaSuccess) return e;
    const dim3 grid(kNormPartials);
    return bf16 ? launch_kernel(list_sqnorm_kernel<__nv_bfloat16, MAXN>, grid, dim3(kThreads), 0,
                                stream, a)
                : launch_kernel(list_sqnorm_kernel<float, MAXN>, grid, dim3(kThreads), 0, stream,
                                a);
  }
  if (chunks == 0) return cudaSuccess;
  const dim3 grid((unsigned)(chunks < kNormPartials ? chunks : kNormPartials));
  const bool to_bf16 = in.out_dtype == ZS_BF16;
  if (bf16)
    return to_bf16 ? launch_kernel(list_scale_kernel<__nv_bfloat16, __nv_bfloat16, MAXN>, grid,
                                   dim3(kThreads), 0, stream, a)
                   : launch_kernel(list_scale_kernel<__nv_bfloat16, float, MAXN>, grid,
                                   dim3(kThreads), 0, stream, a);
  return to_bf16 ? launch_kernel(list_scale_kernel<float, __nv_bfloat16, MAXN>, grid,
                                 dim3(kThreads), 0, stream, a)
                 : launch_kernel(list_scale_kernel<float, float, MAXN>, grid, dim3(kThreads), 0,
                                 stream, a);
}

cudaError_t launch_list(const TensorsLaunch& in, cudaStream_t stream) {
  int64_t from = 0;
  do {  // (an empty list still has a norm)
    const int n = (int)(in.count - from < kMostListed ? in.count - from : kMostListed);
    const cudaError_t e = n <= 64 ? launch_part<64>(in, from, n, stream)
                                  : launch_part<kMostListed>(in, from, n, stream);
    if (e != cudaSuccess) return e;
    from += n;
  } while (from < in.count);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_tensors(const TensorsLaunch& in, bool norm, bool scale, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (norm) {
    TensorsLaunch a = in;
    a.coef = nullptr;
    if (!a.sqnorm)  // behind the ticket
      a.sqnorm = reinterpret_cast<double*>(static_cast<unsigned char*>(in.workspace) +
                                           kNormTicketOffset + 8);
    e = launch_list(a, stream);
  }
  if (e != cudaSuccess || !scale) return e;
  return launch_list(in, stream);
}

}  // namespace zs
