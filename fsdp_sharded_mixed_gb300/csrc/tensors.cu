// tensors.cu — the global norm of a list of gradients, and clipping.
//
//   n = sqrt(sum_i sum_k g_ik^2),  c = min(1, max_norm / (n + 1e-6)),  out_ik = c g_ik
//
// The list's addresses and lengths are kernel parameters (no table in device
// memory, nothing to copy before the launch). Every tensor is cut into chunks of
// 32 KB, and a fixed number of blocks stride over the chunks of the whole list, so
// that the load is even however unequal the tensors are; a thread has four 32-byte
// loads of its chunk on their way at once.
//
// Each block leaves a partial sum (double) in scratch memory. The blocks of the
// scaling kernel add all partials up themselves, in the same fixed order, rather
// than wait for a last block of the norm's to do it: no ticket to clear, and no
// launch between the two. It walks the list from its end, where the norm's pass
// left what L2 still holds.
//
// Bound: HBM, with two readings of a list that L2 does not hold, as the norm has to be
// known before the first element is scaled: 3.09e9 bf16 in 650 tensors 2775 us (0.98
// of that floor), 152e6 fp32 to bf16 in 218 234 us (0.95). Few small tensors are two
// launches of latency: 38 in 11 us.
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
constexpr int kParts = 608;      // blocks: four to an SM of 152; fixed, so that sums are
constexpr int kUnitBytes = 32;   // of the list's tensors: a thread's access
constexpr int kAtOnce = 4;       // units of a thread's
constexpr int kChunkUnits = kAtOnce * kThreads;
static_assert(kParts <= kNormPartials, "the workspace is the flat norm's");

template <typename T>
constexpr int kPer = kUnitBytes / (int)sizeof(T);  // elements of a unit

// Tensor i has `lead` elements less than a whole first unit: its unit u holds
// elements [u * kPer - lead, (u + 1) * kPer - lead) that are in the tensor.
template <int MAXN>
struct List {
  const void* in[MAXN];
  int64_t numel[MAXN];
  uint32_t first[MAXN + 1];  // chunks of the tensors before
  uint16_t begin[kParts];    // the tensors that the blocks begin with
  uint8_t lead[MAXN];
  int32_t count;
};
template <int MAXN>
struct NormArgs {
  List<MAXN> list;
  bool begins;       // the first launch of a list's
  double* partials;  // [kParts]
  unsigned int* err;
};
template <int MAXN>
struct ScaleArgs {
  List<MAXN> list;
  void* out[MAXN];
  const float* coef;       // NULL: from the partials
  const int32_t* skip;     // with coef, or NULL
  const double* partials;
  double max_norm;
  float *norm_out, *coef_out;  // written by block 0, unless NULL
  int32_t* nonfinite_out;
  unsigned int* err;
};

// The tensor of a chunk, from tensor t on.
template <int MAXN>
__device__ __forceinline__ int tensor_of(const List<MAXN>& a, uint32_t chunk, int lo, int hi) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ void load32(uint32_t* w, const void* p) {
  asm volatile("ld.global.L1::no_allocate.v8.u32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                 "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ float2 pair_at(const uint32_t* w, int i, float) {
  return {__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])};
}
__device__ __forceinline__ float2 pair_at(const uint32_t* w, int i, __nv_bfloat16) {
  return {__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)};
}

// The sum of a unit's squares in fp32, in two chains.
template <typename T>
__device__ __forceinline__ float squares(const uint32_t* w) {
  float2 s = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kPer<T> / 2; ++i) {
    const float2 v = pair_at(w, i, T());
    s = __ffma2_rn(v, v, s);
  }
  return s.x + s.y;
}
// The same in double, for units whose squares leave fp32's range.
template <typename T>
__device__ __forceinline__ double squares_wide(const uint32_t* w) {
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < kPer<T> / 2; ++i) {
    const float2 v = pair_at(w, i, T());
    d += (double)v.x * (double)v.x;
    d += (double)v.y * (double)v.y;
  }
  return d;
}
// A chunk's units: 16 elements of fp32 or 32 of bf16 go from fp32 to double as one
// (double runs at a sixtieth of fp32's rate here: one conversion and addition a unit
// kept its pipe 75 % busy and the norm of fp32 lists at 5.7 TB/s), unless their sum
// is out of fp32's range, or so small that squares in it may have been: unit by unit.
template <typename T>
__device__ __forceinline__ double chunk_squares(const uint32_t (*w)[8]) {
  constexpr int kTogether = sizeof(T) == 4 ? kAtOnce : 2;
  double d = 0.0;
#pragma unroll
  for (int j = 0; j < kAtOnce; j += kTogether) {
    float s = squares<T>(w[j]) + squares<T>(w[j + 1]);
    if (kTogether == 4) s += squares<T>(w[j + 2]) + squares<T>(w[j + 3]);
    if (s > 1e-25f && s < 1e37f) {
      d += (double)s;
      continue;
    }
    uint32_t any = 0;
#pragma unroll
    for (int u = 0; u < kTogether; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        any |= w[j + u][i] & (sizeof(T) == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu);
    if (any == 0) continue;
#pragma unroll
    for (int u = 0; u < kTogether; ++u) d += squares_wide<T>(w[j + u]);
  }
  return d;
}

// The elements of a unit that lie within the tensor, the others 0.
template <typename T>
__device__ __forceinline__ void load_edge(uint32_t* w, const T* p, int64_t e, int64_t numel) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 0;
#pragma unroll
  for (int k = 0; k < kPer<T>; ++k) {
    if (e + k < 0 || e + k >= numel) continue;
    if (sizeof(T) == 4)
      w[k % 8] = reinterpret_cast<const uint32_t*>(p)[e + k];
    else
      w[k / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[e + k] << (k % 2 * 16);
  }
}

template <typename T, int MAXN>
__global__ void __launch_bounds__(kThreads, 4)
    list_sqnorm_kernel(const __grid_constant__ NormArgs<MAXN> a) {
  overlap_wait();
  const uint32_t chunks = a.list.first[a.list.count];
  double sum = 0.0;
  int t = a.list.begin[blockIdx.x];
  for (uint32_t c = blockIdx.x; c < chunks; c += kParts) {
    const int64_t numel = a.list.numel[t];
    const T* p = static_cast<const T*>(a.list.in[t]);
    const int64_t e0 = (int64_t)(c - a.list.first[t]) * kChunkUnits * kPer<T> - a.list.lead[t] +
                       threadIdx.x * kPer<T>;
    uint32_t w[kAtOnce][8];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int64_t e = e0 + j * (kThreads * kPer<T>);
      if (e >= 0 && e + kPer<T> <= numel) {
        if (within(e, e + kPer<T>, 0, numel, a.err)) load32(w[j], p + e);
      } else {
        load_edge(w[j], p, e, numel);
      }
    }
    // while they are on their way: the next chunk's tensor
    if (c + kParts < chunks) t = tensor_of(a.list, c + kParts, t, a.list.count - 1);
    sum += chunk_squares<T>(w);
  }
  __shared__ double warp_sums[kThreads / 32];
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_down_sync(0xFFFFFFFFu, sum, off);
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x != 0 || !within(blockIdx.x, blockIdx.x + 1, 0, kParts, a.err)) return;
  double b = a.begins ? 0.0 : a.partials[blockIdx.x];
  for (int w = 0; w < kThreads / 32; ++w) b += warp_sums[w];
  a.partials[blockIdx.x] = b;
}

// The partials' sum, in one order, by the first warp (whose lanes get it).
__device__ __forceinline__ double total_of(const double* partials) {
  constexpr int kEach = kParts / 32;
  static_assert(kParts % 32 == 0, "every lane takes as many");
  double t = 0.0, p[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) p[k] = __ldcg(partials + threadIdx.x % 32 + 32 * k);
#pragma unroll
  for (int k = 0; k < kEach; ++k) t += p[k];
  for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, off);
  return t;
}

__global__ void __launch_bounds__(32) join_norm_kernel(const double* partials, double* out) {
  overlap_wait();
  const double total = total_of(partials);
  if (threadIdx.x == 0) *out = total;
}

// A unit at any address: the two aligned ones that it lies in, shifted. off: its
// bytes behind the first one's start.
__device__ __forceinline__ void load_shifted(uint32_t* w, const unsigned char* p, int off) {
  if (off == 0) {
    load32(w, p);
    return;
  }
  uint32_t x[16];
  load32(x, p - off);
  load32(x + 8, p - off + 32);
  if (off & 16)
#pragma unroll
    for (int i = 0; i < 12; ++i) x[i] = x[i + 4];
  if (off & 8)
#pragma unroll
    for (int i = 0; i < 10; ++i) x[i] = x[i + 2];
  if (off & 4)
#pragma unroll
    for (int i = 0; i < 9; ++i) x[i] = x[i + 1];
  if (off & 2)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __funnelshift_r(x[i], x[i + 1], 16);
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = x[i];
}

// A unit's elements times the coefficient, as a whole (q on 16 bytes at least).
__device__ __forceinline__ void store_unit(float* q, const float2* v, int n) {
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    if (2 * i >= n) break;
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      w[2 * k] = __float_as_uint(v[i + k].x);
      w[2 * k + 1] = __float_as_uint(v[i + k].y);
    }
    store_words<8>(q + 2 * i, w);
  }
}
__device__ __forceinline__ void store_unit(__nv_bfloat16* q, const float2* v, int n) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (2 * i >= n) break;
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[i].x, v[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  if (n == 16)
    store_words<8>(q, w);
  else
    store_words<4>(q, w);
}

// The units here are those of the output: its addresses decide `lead`.
template <typename T, typename OT, int MAXN>
__global__ void __launch_bounds__(kThreads, 4)
    list_scale_kernel(const __grid_constant__ ScaleArgs<MAXN> a) {
  __shared__ float shared_coef;
  __shared__ bool shared_skip;
  overlap_wait();
  float coef = 1.0f;
  bool known = false;  // the coefficient: found out while the first loads are on their way
  const uint32_t chunks = a.list.first[a.list.count];
  int t = a.list.begin[blockIdx.x];
  for (uint32_t k = blockIdx.x; k < chunks || !known; k += gridDim.x) {
    const uint32_t c = chunks - 1 - k;
    const int64_t numel = k < chunks ? a.list.numel[t] : 0;
    const T* p = static_cast<const T*>(a.list.in[t]);
    OT* q = static_cast<OT*>(a.out[t]);
    const int64_t e0 = (int64_t)(c - a.list.first[t]) * kChunkUnits * kPer<T> - a.list.lead[t] +
                       threadIdx.x * kPer<T>;
    const int off = (int)((uintptr_t)(p + e0) % kUnitBytes);  // the same for all units
    uint32_t w[kAtOnce][8];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int64_t e = e0 + j * (kThreads * kPer<T>);
      // whole units, the aligned ones that they lie in within the tensor too
      if (e >= off / (int)sizeof(T) && e + (off ? 2 : 1) * kPer<T> <= numel) {
        if (within(e - off / (int)sizeof(T), e + kPer<T>, 0, numel, a.err))
          load_shifted(w[j], reinterpret_cast<const unsigned char*>(p + e), off);
      } else {
        load_edge(w[j], p, e, numel);
      }
    }
    const bool same = (const void*)p == (const void*)q;
    if (k + gridDim.x < chunks) t = tensor_of(a.list, c - gridDim.x, 0, t);
    if (!known) {
      known = true;
      if (a.coef) {
        if (a.skip && *a.skip) return;
        coef = *a.coef;
      } else {
        if (threadIdx.x < 32) {
          const double total = total_of(a.partials);
          if (threadIdx.x == 0) {
            const double norm = sqrt(total), c = a.max_norm / (norm + 1e-6);
            shared_skip = !isfinite(norm);
            shared_coef = shared_skip ? 1.0f : (float)(c < 1.0 ? c : 1.0);
            if (a.norm_out && blockIdx.x == 0) {
              *a.norm_out = (float)norm;
              *a.coef_out = shared_coef;
              *a.nonfinite_out = shared_skip ? 1 : 0;
            }
          }
        }
        __syncthreads();
        if (shared_skip) return;
        coef = shared_coef;
      }
    }
    if (coef == 1.0f && same) continue;  // in place: nothing changes
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int64_t e = e0 + j * (kThreads * kPer<T>);
      float2 v[8];
#pragma unroll
      for (int i = 0; i < kPer<T> / 2; ++i)
        v[i] = __fmul2_rn(pair_at(w[j], i, T()), make_float2(coef, coef));
      if (e >= 0 && e + kPer<T> <= numel) {
        if (within(e, e + kPer<T>, 0, numel, a.err)) store_unit(q + e, v, kPer<T>);
      } else {
#pragma unroll
        for (int i = 0; i < kPer<T>; ++i)
          if (e + i >= 0 && e + i < numel) put(q + e + i, i % 2 ? v[i / 2].y : v[i / 2].x);
      }
    }
  }
}

constexpr int kMostListed = 768;  // tensors of one launch

// Fills the list with tensors [from, from + n) of a call's that hold something.
// From the list's end (the scaling), block b of `blocks` begins with chunk b from there.
template <int MAXN>
void fill_list(List<MAXN>* l, const TensorsLaunch& in, int64_t from, int n, void** out) {
  const int es = in.dtype == ZS_BF16 ? 2 : 4, per = kUnitBytes / es;
  const int os = out ? (in.out_dtype == ZS_BF16 ? 2 : 4) : es;
  // a unit of an output is aligned to its own bytes, or to 32
  const int align = per * os < kUnitBytes ? per * os : kUnitBytes;
  l->count = 0;
  l->first[0] = 0;
  for (int64_t i = from; i < from + n; ++i) {
    if (in.numels[i] == 0) continue;
    const int k = l->count++;
    l->in[k] = in.tensors[i];
    l->numel[k] = in.numels[i];
    if (out) out[k] = in.outs[i];
    const uintptr_t at = (uintptr_t)(out ? out[k] : in.tensors[i]);
    l->lead[k] = (uint8_t)(at % align / os);
    const int64_t units = (l->lead[k] + in.numels[i] + per - 1) / per;
    l->first[k + 1] = l->first[k] + (uint32_t)((units + kChunkUnits - 1) / kChunkUnits);
  }
  const uint32_t chunks = l->first[l->count];
  int t = out && l->count > 0 ? l->count - 1 : 0;
  for (uint32_t b = 0; b < (uint32_t)kParts; ++b) {
    if (b < chunks && !out)
      while (l->first[t + 1] <= b) ++t;
    if (b < chunks && out)
      while (l->first[t] > chunks - 1 - b) --t;
    l->begin[b] = (uint16_t)t;
  }
}

template <int MAXN>
cudaError_t launch_norm_of(const TensorsLaunch& in, int64_t from, int n, cudaStream_t stream) {
  NormArgs<MAXN> a;
  fill_list(&a.list, in, from, n, nullptr);
  a.begins = from == 0;
  a.partials = static_cast<double*>(in.workspace);
  a.err = ZS_BOUNDS_CHECK ? device_error_word() : nullptr;
  if (ZS_BOUNDS_CHECK && !a.err) return cudaErrorInvalidSymbol;
  return in.dtype == ZS_BF16
             ? launch_kernel(list_sqnorm_kernel<__nv_bfloat16, MAXN>, dim3(kParts),
                             dim3(kThreads), 0, stream, a)
             : launch_kernel(list_sqnorm_kernel<float, MAXN>, dim3(kParts), dim3(kThreads), 0,
                             stream, a);
}

template <int MAXN>
cudaError_t launch_scale_of(const TensorsLaunch& in, int64_t from, int n, cudaStream_t stream) {
  ScaleArgs<MAXN> a;
  fill_list(&a.list, in, from, n, a.out);
  const bool clip = in.max_norm > 0;
  a.coef = clip ? nullptr : in.coef;
  a.skip = in.skip;
  a.partials = static_cast<const double*>(in.workspace);
  a.max_norm = in.max_norm;
  a.norm_out = clip && from == 0 ? in.norm : nullptr;
  a.coef_out = in.coef_out;
  a.nonfinite_out = in.nonfinite_out;
  a.err = ZS_BOUNDS_CHECK ? device_error_word() : nullptr;
  if (ZS_BOUNDS_CHECK && !a.err) return cudaErrorInvalidSymbol;
  const uint32_t chunks = a.list.first[a.list.count];
  if (chunks == 0 && !a.norm_out) return cudaSuccess;
  const dim3 grid(chunks < 1 ? 1 : chunks < kParts ? chunks : kParts), block(kThreads);
  if (in.dtype == ZS_BF16)
    return in.out_dtype == ZS_BF16
               ? launch_kernel(list_scale_kernel<__nv_bfloat16, __nv_bfloat16, MAXN>, grid, block,
                               0, stream, a)
               : launch_kernel(list_scale_kernel<__nv_bfloat16, float, MAXN>, grid, block, 0,
                               stream, a);
  return in.out_dtype == ZS_BF16
             ? launch_kernel(list_scale_kernel<float, __nv_bfloat16, MAXN>, grid, block, 0, stream,
                             a)
             : launch_kernel(list_scale_kernel<float, float, MAXN>, grid, block, 0, stream, a);
}

// Launches over kMostListed tensors at a time; few tensors take fewer parameters.
// (An empty list has a norm, too: one launch at least.)
template <typename Small, typename Middle, typename Large>
cudaError_t in_parts(const TensorsLaunch& in, Small small, Middle middle, Large large) {
  int64_t from = 0;
  do {
    const int n = (int)(in.count - from < kMostListed ? in.count - from : kMostListed);
    const cudaError_t e = n <= 64    ? small(from, n)
                          : n <= 256 ? middle(from, n)
                                     : large(from, n);
    if (e != cudaSuccess) return e;
    from += n;
  } while (from < in.count);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_tensors(const TensorsLaunch& in, bool norm, bool scale, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (norm)
    e = in_parts(in, [&](int64_t f, int n) { return launch_norm_of<64>(in, f, n, stream); },
                 [&](int64_t f, int n) { return launch_norm_of<256>(in, f, n, stream); },
                 [&](int64_t f, int n) { return launch_norm_of<kMostListed>(in, f, n, stream); });
  if (e == cudaSuccess && norm && in.sqnorm)
    e = launch_kernel(join_norm_kernel, dim3(1), dim3(32), 0, stream,
                      static_cast<const double*>(in.workspace), in.sqnorm);
  if (e != cudaSuccess || !scale) return e;
  return in_parts(in, [&](int64_t f, int n) { return launch_scale_of<64>(in, f, n, stream); },
                  [&](int64_t f, int n) { return launch_scale_of<256>(in, f, n, stream); },
                  [&](int64_t f, int n) {
                    return launch_scale_of<kMostListed>(in, f, n, stream);
                  });
}

}  // namespace zs
