// layer_norm.cu — layer norm behind an optional residual sum, and its backward
// pass with the sums over the rows that make the weight's and bias's gradients.
//
//   h  = x + residual, rounded to the rows' type      (h = x without a residual)
//   mu = mean h,  r = 1 / sqrt(mean (h - mu)^2 + eps)
//   y  = (h - mu) r w + b
//   xh = (x - mu) r,  g = dy w
//   dx = r (g - mean g - xh mean(g xh)) + d_sum
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// A row is read once and stays in the registers of its warps (a slab of 256
// columns is eight elements a lane, up to four slabs a warp). The mean is taken
// twice: what the first sum loses shows in the mean of the deviations from it,
// which costs no pass, as it is summed with their squares. h is rounded before
// it is normalised because the backward pass sees the stored h alone.
// Statistics and sums are fp32. The backward pass keeps each warp's columns of
// dw and db in registers over its rows; blocks leave partial sums in scratch
// memory, and a second launch adds them in a fixed order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bounds.cuh"
#include "overlap.cuh"
#include "row_vec.cuh"
#include "zs_internal.h"

namespace zs {
namespace {

constexpr int kWarps = 8;       // of a block, where rows leave the choice
constexpr int kMaxSlabs = 4;    // of a warp
constexpr int kMaxRowWarps = 32;
static_assert(ZS_MAX_DIM == kMaxRowWarps * kMaxSlabs * kSlab, "the widest row is one block's");

struct NormArgs {
  const void *x, *residual, *weight, *bias;
  void *sum, *y;
  float *mean, *rstd;  // outputs of the forward pass, inputs of the backward pass
  const void *d_y, *d_sum;
  void* d_x;
  float* parts;        // [blocks][dw, db][dim]
  int64_t rows, row_stride, out_stride, grad_stride;
  int32_t dim, row_warps;  // warps of a row
  bool weight_bf16, want_weight, want_bias;
  float eps;
  unsigned int* err;
};

// Eight weights of a lane, in either type.
template <bool VEC>
__device__ __forceinline__ void weights8(const void* w, bool bf16, int col0, int lane, int D,
                                         float* v) {
  if (bf16) {
    const Raw8<__nv_bfloat16> r =
        load8<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(w), col0, lane, D);
#pragma unroll
    for (int k = 0; k < kLane; ++k) v[k] = raw_value(r, k);
  } else {
    const Raw8<float> r = load8<float, VEC>(static_cast<const float*>(w), col0, lane, D);
#pragma unroll
    for (int k = 0; k < kLane; ++k) v[k] = raw_value(r, k);
  }
}

__device__ __forceinline__ float2 warp_sum(float2 s) {
  for (int off = 16; off > 0; off >>= 1) {
    s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, off);
    s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, off);
  }
  return s;
}

// The sums over a row's warps, in a fixed order; every lane gets them. `turn`
// alternates between calls, so that one barrier a call is enough.
struct RowSums {
  float2 of_warp[2][kMaxRowWarps];
  __device__ __forceinline__ float2 operator()(float2 s, int row_warps, int turn) {
    s = warp_sum(s);
    if (row_warps == 1) return s;
    const int warp = threadIdx.x / 32, first = warp / row_warps * row_warps;
    if ((threadIdx.x & 31) == 0) of_warp[turn][warp] = s;
    __syncthreads();
    float2 t = {0.0f, 0.0f};
    for (int w = first; w < first + row_warps; ++w) {
      t.x += of_warp[turn][w].x;
      t.y += of_warp[turn][w].y;
    }
    return t;
  }
};

// ---- forward ---------------------------------------------------------------------
// THREADS: the most of a block (256, or 1024 for rows past 8192 columns).
template <typename T, bool VEC, int SLABS, int THREADS>
__global__ void __launch_bounds__(THREADS) layer_norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ RowSums sums;
  overlap_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int at = warp % a.row_warps * SLABS * kSlab, D = a.dim;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / 32 / a.row_warps) + warp / a.row_warps;
  const bool on = row < a.rows && within(row, row + 1, 0, a.rows, a.err);
  float h[SLABS][kLane];
  {
    Raw8<T> x[SLABS], res[SLABS];
    const T* from = static_cast<const T*>(a.x) + row * a.row_stride;
    const T* more = a.residual ? static_cast<const T*>(a.residual) + row * a.row_stride : nullptr;
#pragma unroll
    for (int s = 0; s < SLABS; ++s)
      if (on) x[s] = load8<T, VEC>(from, at + s * kSlab, lane, D);
#pragma unroll
    for (int s = 0; s < SLABS; ++s)
      if (on && more) res[s] = load8<T, VEC>(more, at + s * kSlab, lane, D);
#pragma unroll
    for (int s = 0; s < SLABS; ++s)
#pragma unroll
      for (int k = 0; k < kLane; ++k) {
        h[s][k] = on ? raw_value(x[s], k) : 0.0f;
        if (on && more) h[s][k] = rounded(h[s][k] + raw_value(res[s], k), T());
      }
    if (on && a.sum) {
      T* to = static_cast<T*>(a.sum) + row * a.out_stride;
#pragma unroll
      for (int s = 0; s < SLABS; ++s) store8<T, VEC>(to, at + s * kSlab, lane, D, h[s]);
    }
  }
  const float per = 1.0f / (float)D;
  float2 t = {0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < SLABS; ++s)
#pragma unroll
    for (int k = 0; k < kLane; ++k) t.x += h[s][k];  // columns past the end are 0
  float mean = sums(t, a.row_warps, 0).x * per;
  t = {0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < SLABS; ++s)
#pragma unroll
    for (int k = 0; k < kLane; ++k) {
      h[s][k] = column<VEC>(at + s * kSlab, lane, k) < D ? h[s][k] - mean : 0.0f;
      t.x += h[s][k];
      t.y = __fmaf_rn(h[s][k], h[s][k], t.y);
    }
  t = sums(t, a.row_warps, 1);
  const float off = t.x * per;
  mean += off;
  const float var = fmaxf(__fmaf_rn(-off, off, t.y * per), 0.0f);
  // (fmaxf drops a NaN; the deviations still hold it)
  const float rstd = 1.0f / sqrtf(var + a.eps);
  if (!on) return;
  if (lane == 0 && warp % a.row_warps == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = t.y != t.y ? t.y : rstd;
  }
  T* to = static_cast<T*>(a.y) + row * a.out_stride;
#pragma unroll
  for (int s = 0; s < SLABS; ++s) {
    float w[kLane], b[kLane];
    if (a.weight) weights8<VEC>(a.weight, a.weight_bf16, at + s * kSlab, lane, D, w);
    if (a.bias) weights8<VEC>(a.bias, a.weight_bf16, at + s * kSlab, lane, D, b);
#pragma unroll
    for (int k = 0; k < kLane; ++k) {
      float v = (h[s][k] - off) * rstd;
      if (a.weight) v *= w[k];
      if (a.bias) v += b[k];
      h[s][k] = v;
    }
    store8<T, VEC>(to, at + s * kSlab, lane, D, h[s]);
  }
}

// ---- backward --------------------------------------------------------------------
constexpr int kGradBlocks = 304;  // two to an SM of 152; fixed, so that sums are

// Rows of a block's groups of warps: group g of G takes rows g, g + G, ...
template <typename T, bool VEC, int SLABS, int THREADS>
__global__ void __launch_bounds__(THREADS) layer_norm_grad_kernel(const __grid_constant__ NormArgs a) {
  __shared__ RowSums sums;
  extern __shared__ float columns[];  // [groups of the block][dim]
  overlap_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int at = warp % a.row_warps * SLABS * kSlab, D = a.dim;
  const int groups = blockDim.x / 32 / a.row_warps, group = warp / a.row_warps;
  float w[SLABS][kLane], dw[SLABS][kLane], db[SLABS][kLane];
#pragma unroll
  for (int s = 0; s < SLABS; ++s) {
#pragma unroll
    for (int k = 0; k < kLane; ++k) {
      w[s][k] = 1.0f;
      dw[s][k] = db[s][k] = 0.0f;
    }
    if (a.weight) weights8<VEC>(a.weight, a.weight_bf16, at + s * kSlab, lane, D, w[s]);
  }
  const float per = 1.0f / (float)D;
  const int64_t stride = (int64_t)gridDim.x * groups;
  int turn = 0;
  // a block's groups go round together, for the barriers
  for (int64_t row0 = (int64_t)blockIdx.x * groups; row0 < a.rows; row0 += stride) {
    const int64_t row = row0 + group;
    const bool on = row < a.rows && within(row, row + 1, 0, a.rows, a.err);
    Raw8<T> x[SLABS], dy[SLABS];
    float mean = 0.0f, rstd = 0.0f;
    if (on) {
      const T* xp = static_cast<const T*>(a.x) + row * a.row_stride;
      const T* dp = static_cast<const T*>(a.d_y) + row * a.grad_stride;
#pragma unroll
      for (int s = 0; s < SLABS; ++s) {
        x[s] = load8<T, VEC>(xp, at + s * kSlab, lane, D);
        dy[s] = load8<T, VEC>(dp, at + s * kSlab, lane, D);
      }
      mean = a.mean[row];
      rstd = a.rstd[row];
    }
    float2 t = {0.0f, 0.0f};
    if (on) {
#pragma unroll
      for (int s = 0; s < SLABS; ++s)
#pragma unroll
        for (int k = 0; k < kLane; ++k) {
          // (past the row's end dy is 0, and so is all that it multiplies)
          const float xh = column<VEC>(at + s * kSlab, lane, k) < D
                               ? (raw_value(x[s], k) - mean) * rstd
                               : 0.0f;
          const float d = raw_value(dy[s], k), g = d * w[s][k];
          t.x += g;
          t.y = __fmaf_rn(g, xh, t.y);
          dw[s][k] = __fmaf_rn(d, xh, dw[s][k]);
          db[s][k] += d;
        }
    }
    t = sums(t, a.row_warps, turn);
    turn ^= 1;
    if (!on) continue;
    const float c1 = t.x * per, c2 = t.y * per;
    T* to = static_cast<T*>(a.d_x) + row * a.grad_stride;
    const T* past = a.d_sum ? static_cast<const T*>(a.d_sum) + row * a.grad_stride : nullptr;
#pragma unroll
    for (int s = 0; s < SLABS; ++s) {
      Raw8<T> more;
      if (past) more = load8<T, VEC>(past, at + s * kSlab, lane, D);
      float v[kLane];
#pragma unroll
      for (int k = 0; k < kLane; ++k) {
        const float xh = (raw_value(x[s], k) - mean) * rstd;
        const float g = raw_value(dy[s], k) * w[s][k];
        v[k] = rstd * (g - c1 - xh * c2);
        if (past) v[k] += raw_value(more, k);
      }
      store8<T, VEC>(to, at + s * kSlab, lane, D, v);
    }
  }
  // The block's sums of its columns, then to scratch memory.
  for (int which = 0; which < 2; ++which) {
    if (!(which ? a.want_bias : a.want_weight)) continue;
    float* to = a.parts + ((int64_t)blockIdx.x * 2 + which) * D;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < SLABS; ++s)
#pragma unroll
      for (int k = 0; k < kLane; ++k) {
        const int c = column<VEC>(at + s * kSlab, lane, k);
        if (c < D) columns[group * D + c] = which ? db[s][k] : dw[s][k];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
      float v = 0.0f;
      for (int g = 0; g < groups; ++g) v += columns[g * D + c];
      to[c] = v;
    }
  }
}

// The blocks' sums joined: 32 columns a block, its warps take every 8th part.
struct JoinArgs {
  const float* parts;
  void *d_weight, *d_bias;
  int32_t dim, blocks;
  bool bf16;
};
__global__ void __launch_bounds__(256) join_columns_kernel(const __grid_constant__ JoinArgs a) {
  __shared__ float part[8][32];
  overlap_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  for (int which = 0; which < 2; ++which) {
    void* out = which ? a.d_bias : a.d_weight;
    if (!out) continue;
    float v = 0.0f;
    if (c < a.dim)
#pragma unroll 4
      for (int b = warp; b < a.blocks; b += 8) v += a.parts[((int64_t)b * 2 + which) * a.dim + c];
    part[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < a.dim) {
      v = 0.0f;
      for (int w = 0; w < 8; ++w) v += part[w][lane];
      if (a.bf16)
        put(static_cast<__nv_bfloat16*>(out) + c, v);
      else
        put(static_cast<float*>(out) + c, v);
    }
    __syncthreads();
  }
}

// How a row of `dim` columns is laid over warps.
struct Shape {
  int row_warps, slabs, threads, groups;  // groups: rows of a block at a time
};
Shape shape_of(int64_t dim) {
  Shape s;
  const int slabs = (int)((dim + kSlab - 1) / kSlab);
  s.row_warps = 1;
  while (s.row_warps * kMaxSlabs < slabs) s.row_warps *= 2;
  s.slabs = (slabs + s.row_warps - 1) / s.row_warps;
  s.threads = 32 * (s.row_warps > kWarps ? s.row_warps : kWarps);
  s.groups = s.threads / 32 / s.row_warps;
  return s;
}

int grad_blocks(int64_t rows, int64_t dim) {
  const int64_t groups = shape_of(dim).groups, blocks = (rows + groups - 1) / groups;
  return (int)(blocks < kGradBlocks ? blocks : kGradBlocks);
}

template <typename T, bool VEC, int SLABS, int THREADS>
cudaError_t launch_one(const NormArgs& a, const Shape& s, bool grad, int smem,
                       cudaStream_t stream) {
  if (!grad)
    return launch_kernel(layer_norm_kernel<T, VEC, SLABS, THREADS>,
                         dim3((unsigned)((a.rows + s.groups - 1) / s.groups)), dim3(s.threads), 0,
                         stream, a);
  cudaError_t e = cudaFuncSetAttribute(layer_norm_grad_kernel<T, VEC, SLABS, THREADS>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, 160 << 10);
  if (e != cudaSuccess) return e;
  return launch_kernel(layer_norm_grad_kernel<T, VEC, SLABS, THREADS>,
                       dim3((unsigned)grad_blocks(a.rows, a.dim)), dim3(s.threads), smem, stream,
                       a);
}

template <typename T, bool VEC>
cudaError_t launch_slabs(const NormArgs& a, const Shape& s, bool grad, cudaStream_t stream) {
  const int smem = s.groups * a.dim * (int)sizeof(float);
  if (s.threads > 256)
    return s.slabs == 3 ? launch_one<T, VEC, 3, 1024>(a, s, grad, smem, stream)
                        : launch_one<T, VEC, 4, 1024>(a, s, grad, smem, stream);
  switch (s.slabs) {
    case 1: return launch_one<T, VEC, 1, 256>(a, s, grad, smem, stream);
    case 2: return launch_one<T, VEC, 2, 256>(a, s, grad, smem, stream);
    case 3: return launch_one<T, VEC, 3, 256>(a, s, grad, smem, stream);
    default: return launch_one<T, VEC, 4, 256>(a, s, grad, smem, stream);
  }
}

cudaError_t launch_norm(const NormArgs& a, bool bf16, bool vec, bool grad, cudaStream_t stream) {
  const Shape s = shape_of(a.dim);
  if (bf16)
    return vec ? launch_slabs<__nv_bfloat16, true>(a, s, grad, stream)
               : launch_slabs<__nv_bfloat16, false>(a, s, grad, stream);
  return vec ? launch_slabs<float, true>(a, s, grad, stream)
             : launch_slabs<float, false>(a, s, grad, stream);
}

}  // namespace

int64_t layer_norm_grad_workspace_bytes(int64_t rows, int64_t dim) {
  return 2 * (int64_t)sizeof(float) * grad_blocks(rows, dim) * dim;
}

namespace {

cudaError_t launch_rows(const LayerNormLaunch& in, bool grad, cudaStream_t stream) {
  NormArgs a = {};
  a.x = in.x;
  a.residual = in.residual;
  a.weight = in.weight;
  a.bias = in.bias;
  a.sum = in.sum;
  a.y = in.y;
  a.mean = in.mean;
  a.rstd = in.rstd;
  a.d_y = in.d_y;
  a.d_sum = in.d_sum;
  a.d_x = in.d_x;
  a.parts = static_cast<float*>(in.workspace);
  a.rows = in.rows;
  a.row_stride = in.row_stride;
  a.out_stride = in.out_stride;
  a.grad_stride = in.grad_stride;
  a.dim = (int32_t)in.dim;
  a.row_warps = shape_of(in.dim).row_warps;
  a.weight_bf16 = in.weight_dtype == ZS_BF16;
  a.want_weight = in.d_weight != nullptr;
  a.want_bias = in.d_bias != nullptr;
  a.eps = (float)in.eps;
  a.err = ZS_BOUNDS_CHECK ? device_error_word() : nullptr;
  if (ZS_BOUNDS_CHECK && !a.err) return cudaErrorInvalidSymbol;
  const bool bf16 = in.dtype == ZS_BF16;
  const int es = bf16 ? 2 : 4, ws = a.weight_bf16 ? 2 : 4;
  const bool vec = rows_aligned(a.x, a.row_stride, es) &&
                   rows_aligned(a.residual, a.row_stride, es) &&
                   rows_aligned(a.sum, a.out_stride, es) && rows_aligned(a.y, a.out_stride, es) &&
                   rows_aligned(a.d_y, a.grad_stride, es) &&
                   rows_aligned(a.d_sum, a.grad_stride, es) &&
                   rows_aligned(a.d_x, a.grad_stride, es) && rows_aligned(a.weight, 16, ws) &&
                   rows_aligned(a.bias, 16, ws);
  return launch_norm(a, bf16, vec, grad, stream);
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormLaunch& in, cudaStream_t stream) {
  return launch_rows(in, false, stream);
}

cudaError_t launch_layer_norm_grad(const LayerNormLaunch& in, cudaStream_t stream) {
  if (in.rows > 0) {
    const cudaError_t e = launch_rows(in, true, stream);
    if (e != cudaSuccess) return e;
  }
  if (!in.d_weight && !in.d_bias) return cudaSuccess;
  JoinArgs j;
  j.parts = static_cast<const float*>(in.workspace);
  j.d_weight = in.d_weight;
  j.d_bias = in.d_bias;
  j.dim = (int32_t)in.dim;
  j.blocks = in.rows > 0 ? grad_blocks(in.rows, in.dim) : 0;
  j.bf16 = in.grad_dtype == ZS_BF16;
  return launch_kernel(join_columns_kernel, dim3((unsigned)((j.dim + 31) / 32)), dim3(256), 0,
                       stream, j);
}

}  // namespace zs
