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
// columns is eight elements a lane, one to four slabs a warp). The mean is taken
// twice: what the first sum loses shows in the mean of the deviations from it,
// which costs no pass, as it is summed with their squares. h is rounded before
// it is normalised because the backward pass sees the stored h alone.
// Statistics and sums are fp32. The backward pass keeps each warp's columns of
// dw and db in registers over its rows; blocks leave partial sums in scratch
// memory, and a second launch adds them in a fixed order.
//
// Bound: HBM, and instructions an element close behind it: packed arithmetic and
// two slabs a warp, which halve the shuffles and addresses an element, are what
// brought 16384 x 4096 bf16 from 170 us forward and 274 backward to 86.5 and 87
// (0.91 of the measured copy rate, 46 and 52 % of the issue slots). 8192 x 768:
// 12.4 (0.60) and 17.2 (0.43), of which the join is 3.5; 8192 x 8192 0.95 and 0.85.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bounds.cuh"
#include "overlap.cuh"
#include "row_vec.cuh"
#include "zs_internal.h"

namespace zs {
namespace {

constexpr int kMaxRowWarps = 32;
constexpr int kMaxSlabs = 4;   // of a warp
constexpr int kHeldSlabs = 2;  // whose weights stay in registers
constexpr int kMostStages = 4;
constexpr int kPairs = kLane / 2;
static_assert(ZS_MAX_DIM == kMaxRowWarps * kMaxSlabs * kSlab, "the widest row is one block's");

struct NormArgs {
  const void *x, *residual, *weight, *bias;
  void *sum, *y;
  float *mean, *rstd;  // outputs of the forward pass, inputs of the backward pass
  const void *d_y, *d_sum;
  void* d_x;
  float* parts;        // [blocks][dw, db][dim]
  int64_t rows, row_stride, out_stride, grad_stride;
  int32_t dim, row_warps, groups;  // a row's warps, a block's rows at a time
  bool weight_bf16, want_weight, want_bias;
  float eps;
  unsigned int* err;
};

// Eight weights of a lane, of either type (kept in L1: every row asks for them).
template <typename W, Lay LAY>
__device__ __forceinline__ void weights_of(float2* v, const W* p, int col0, int lane, int D) {
  Raw8<W> r;
  constexpr int kParts = LAY == kFour ? 2 : 1, kWords = kLane * (int)sizeof(W) / 4 / kParts;
  if (LAY != kOne && column<LAY>(col0, lane, kLane - 1) < D) {
#pragma unroll
    for (int part = 0; part < kParts; ++part) {
      const W* q = p + column<LAY>(col0, lane, part * 4);
      if (kWords % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(q) + i);
          uint32_t* w = r.w + part * kWords + 4 * i;
          w[0] = u.x;
          w[1] = u.y;
          w[2] = u.z;
          w[3] = u.w;
        }
      } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(q));
        r.w[part * kWords] = u.x;
        r.w[part * kWords + 1] = u.y;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < kLane; ++k) {
      const int c = column<LAY>(col0, lane, k);
      set_raw(r, k, c < D ? p[c] : W(0.0f));
    }
  }
#pragma unroll
  for (int i = 0; i < kPairs; ++i) v[i] = pair_of(r, i);
}
template <Lay LAY>
__device__ __forceinline__ void weights8(float2* v, const void* p, bool bf16, int col0, int lane,
                                         int D) {
  if (bf16)
    weights_of<__nv_bfloat16, LAY>(v, static_cast<const __nv_bfloat16*>(p), col0, lane, D);
  else
    weights_of<float, LAY>(v, static_cast<const float*>(p), col0, lane, D);
}

__device__ __forceinline__ float2 both(float x) { return {x, x}; }

// Sums over a row's warps, of one value or two, in a fixed order; every lane gets
// them. Rows of one block meet at barriers of their own. `turn` alternates between
// calls, so that one barrier a call is enough.
__device__ __forceinline__ float sum_lanes(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
  return x;
}
__device__ __forceinline__ float2 sum_lanes(float2 x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    x = __fadd2_rn(x, {__shfl_xor_sync(0xFFFFFFFFu, x.x, off),
                       __shfl_xor_sync(0xFFFFFFFFu, x.y, off)});
  return x;
}
struct RowSums {
  float2 of_warp[2][kMaxRowWarps];
  template <typename V>
  __device__ __forceinline__ V operator()(V s, int row_warps, int group, int turn) {
    s = sum_lanes(s);
    if (row_warps == 1) return s;
    V* mine = reinterpret_cast<V*>(of_warp[turn]);
    const int lane = threadIdx.x & 31;
    if (lane == 0) mine[threadIdx.x / 32] = s;
    // (barrier 0 is the whole block's: groups that are through wait there for the others)
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(32 * row_warps) : "memory");
    V t = {};
    if (lane < row_warps) t = mine[group * row_warps + lane];
    return sum_lanes(t);
  }
};

// ---- rows on their way -----------------------------------------------------------
// A ring of rows in shared memory, private to each thread: it asks (cp.async) for
// its own eight elements a slab of the rows to come, and reads what it asked for,
// so that no barrier is needed. ARRAYS matrices; each row is one group of copies.
// STAGES rows, the one at work among them. A unit is what one copy brings: 16 bytes,
// or one fp32 of a row that starts anywhere.
template <typename T, Lay LAY, int SLABS, int ARRAYS, int STAGES>
struct RowRing {
  static constexpr int kUnit = LAY == kOne ? 4 : 16;  // bytes
  static constexpr int kUnits = kLane * (int)sizeof(T) / kUnit;
  static constexpr int kBytes = STAGES * ARRAYS * SLABS * kUnits * kUnit;  // a thread
  static constexpr int kApart = kSlab / kUnits;  // columns (kEight: one unit a slab)
  uint32_t base, step;      // the thread's first unit, and from a unit to the next
  uint32_t asked, at_work;  // the stages' first units
  int left;                 // the lane's elements up to the row's end, from its first

  __device__ __forceinline__ RowRing(void* smem, int elements)
      : base((uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * kUnit),
        step(blockDim.x * kUnit), asked(base), at_work(base), left(elements) {
    if (left < SLABS * kSlab)  // what ask() leaves out is 0
      for (int i = 0; i < kBytes / kUnit; ++i) {
        if (kUnit == 16)
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(base + i * step), "r"(0)
                       : "memory");
        else
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(base + i * step), "r"(0) : "memory");
      }
  }
  __device__ __forceinline__ uint32_t next(uint32_t stage) const {
    stage += ARRAYS * SLABS * kUnits * step;
    return stage == base + STAGES * ARRAYS * SLABS * kUnits * step ? base : stage;
  }
  // Asks for the lane's elements of a row, from its first one.
  __device__ __forceinline__ void ask(int array, const T* from) {
#pragma unroll
    for (int s = 0; s < SLABS; ++s)
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int c = s * kSlab + u * kApart;
        const uint32_t to = asked + ((array * SLABS + s) * kUnits + u) * step;
        if (kUnit == 16) {
          const int bytes = min(16, max(0, (left - c) * (int)sizeof(T)));
          if (bytes == 0) continue;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from + c),
                       "r"(bytes)
                       : "memory");
        } else if (c < left) {
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from + c)
                       : "memory");
        }
      }
  }
  __device__ __forceinline__ void close() {
    asm volatile("cp.async.commit_group;" ::: "memory");
    asked = next(asked);
  }
  // The row to work on is there.
  __device__ __forceinline__ void wait() const {
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES > 0 ? STAGES - 1 : 0) : "memory");
  }
  __device__ __forceinline__ Raw8<T> take(int array, int s) const {
    Raw8<T> r;
    const uint32_t from = at_work + (array * SLABS + s) * kUnits * step;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      if (kUnit == 16)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.w[4 * u % (kLane * sizeof(T) / 4)]),
                       "=r"(r.w[(4 * u + 1) % (kLane * sizeof(T) / 4)]),
                       "=r"(r.w[(4 * u + 2) % (kLane * sizeof(T) / 4)]),
                       "=r"(r.w[(4 * u + 3) % (kLane * sizeof(T) / 4)])
                     : "r"(from + u * step));
      else
        asm volatile("ld.shared.u32 %0, [%1];"
                     : "=r"(r.w[u % (kLane * sizeof(T) / 4)])
                     : "r"(from + u * step));
    }
    return r;
  }
  __device__ __forceinline__ void done() { at_work = next(at_work); }
};
// The threads that an SM holds of a kernel, by the most of its blocks: rows of one
// slab a warp in blocks of 384, two of them with 80 registers; of two slabs one block
// of 512 with 128 (two of 256: 94.5 us against 86.5 for 16384 x 4096 forward; one slab
// a warp, 1024 threads with 64 registers: 90, and 131 backward, which spills); rows of
// more than 16 warps one block of up to 1024.
template <int THREADS, int SLABS>
constexpr int kOfSm = THREADS > 512 ? 1024 : SLABS > 1 ? 512 : THREADS == 512 ? 1024 : 768;
// Rows in the ring: what those threads hold in 200 KB. 0: rows too wide for one, and
// bf16 rows that start anywhere (cp.async has no copy of two bytes), whose values
// are loaded as they are needed.
template <typename T, Lay LAY, int SLABS, int ARRAYS, int THREADS>
constexpr int kRowsThatFit =
    (200 << 10) / kOfSm<THREADS, SLABS> / (ARRAYS * SLABS * (int)sizeof(T) * kLane);
template <typename T, Lay LAY, int SLABS, int ARRAYS, int THREADS>
constexpr int kStagesOf =
    LAY == kOne && sizeof(T) == 2 ? 0
    : kRowsThatFit<T, LAY, SLABS, ARRAYS, THREADS> < kMostStages
        ? kRowsThatFit<T, LAY, SLABS, ARRAYS, THREADS>
        : kMostStages;

// ---- forward ---------------------------------------------------------------------
// Group g of G takes rows g, g + G, ...
template <typename T, Lay LAY, int SLABS, int THREADS>
__global__ void __launch_bounds__(THREADS, kOfSm<THREADS, SLABS> / THREADS)
    layer_norm_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kStages = kStagesOf<T, LAY, SLABS, 2, THREADS>;
  __shared__ RowSums sums;
  extern __shared__ __align__(16) unsigned char smem[];
  overlap_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int group = warp / a.row_warps, D = a.dim;
  const int at = warp % a.row_warps * SLABS * kSlab, c0 = column<LAY>(at, lane, 0);
  const uint32_t stride = gridDim.x * a.groups, rows = (uint32_t)a.rows;
  uint32_t row = blockIdx.x * a.groups + group;
  const int64_t in_step = stride * a.row_stride, out_step = stride * a.out_stride;
  // where the row at work lies, and the next one to ask for
  const T* x = static_cast<const T*>(a.x) + row * a.row_stride;
  const T* residual = static_cast<const T*>(a.residual) + row * a.row_stride;
  T* sum = static_cast<T*>(a.sum) + row * a.out_stride;
  T* y = static_cast<T*>(a.y) + row * a.out_stride;
  RowRing<T, LAY, SLABS, 2, kStages> ring(smem, D - c0);
  const T *x_ahead = x + c0, *residual_ahead = residual + c0;
  uint32_t row_ahead = row;
  auto ask = [&] {
    if (row_ahead < rows && within(row_ahead, (int64_t)row_ahead + 1, 0, rows, a.err)) {
      ring.ask(0, x_ahead);
      if (a.residual) ring.ask(1, residual_ahead);
    }
    ring.close();
    row_ahead += stride;
    x_ahead += in_step;
    residual_ahead += in_step;
  };
  if (kStages > 0)
    for (int i = 0; i < kStages - 1; ++i) ask();
  // (the weights of wider rows stay in L1)
  constexpr int kHeld = SLABS <= kHeldSlabs ? SLABS : 1;
  float2 w[kHeld][kPairs], b[kHeld][kPairs];
  auto weights = [&](int s) {
    if (a.weight) weights8<LAY>(w[s % kHeld], a.weight, a.weight_bf16, at + s * kSlab, lane, D);
    if (a.bias) weights8<LAY>(b[s % kHeld], a.bias, a.weight_bf16, at + s * kSlab, lane, D);
  };
  if (SLABS == kHeld)
#pragma unroll
    for (int s = 0; s < SLABS; ++s) weights(s);
  const float per = 1.0f / (float)D;
  for (; row < rows; row += stride) {
    const bool in = within(row, (int64_t)row + 1, 0, rows, a.err);
    float2 h[SLABS][kPairs], one = both(0.0f);
    if (kStages > 0) {
      ask();
      ring.wait();
    }
#pragma unroll
    for (int s = 0; s < SLABS; ++s) {
      Raw8<T> r = {};
      if (kStages > 0)
        r = ring.take(0, s);
      else if (in)
        r = load8<T, LAY>(x, at + s * kSlab, lane, D);
      if (a.residual) {
        Raw8<T> more = {};
        if (kStages > 0)
          more = ring.take(1, s);
        else if (in)
          more = load8<T, LAY>(residual, at + s * kSlab, lane, D);
        r = sum_of(r, more);
        if (a.sum && in) store_raw8<T, LAY>(sum, at + s * kSlab, lane, D, r);
      }
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        h[s][i] = pair_of(r, i);
        one = __fadd2_rn(one, h[s][i]);  // columns past the end are 0
      }
    }
    float mean = sums(one.x + one.y, a.row_warps, group, 0) * per;
    float2 dev = both(0.0f), square = both(0.0f);
#pragma unroll
    for (int s = 0; s < SLABS; ++s) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) h[s][i] = __fadd2_rn(h[s][i], both(-mean));
      if (at + (s + 1) * kSlab > D) {  // the slab that the row ends in, or one past it
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          if (column<LAY>(at + s * kSlab, lane, 2 * i) >= D) h[s][i].x = 0.0f;
          if (column<LAY>(at + s * kSlab, lane, 2 * i + 1) >= D) h[s][i].y = 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        dev = __fadd2_rn(dev, h[s][i]);
        square = __ffma2_rn(h[s][i], h[s][i], square);
      }
    }
    const float2 t = sums(make_float2(dev.x + dev.y, square.x + square.y), a.row_warps, group, 1);
    const float off = t.x * per;
    mean += off;
    const float var = fmaxf(__fmaf_rn(-off, off, t.y * per), 0.0f);
    // (fmaxf drops a NaN; the deviations still hold it)
    const float rstd = rsqrtf(var + a.eps);  // to 2 units in the last place
    if (in) {
      if (lane == 0 && at == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = t.y != t.y ? t.y : rstd;
      }
      const float2 scale = both(rstd), shift = both(-off * rstd);
#pragma unroll
      for (int s = 0; s < SLABS; ++s) {
        if (SLABS > kHeld) weights(s);
        Raw8<T> r;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          float2 v = __ffma2_rn(h[s][i], scale, shift);
          if (a.weight) v = __fmul2_rn(v, w[s % kHeld][i]);
          if (a.bias) v = __fadd2_rn(v, b[s % kHeld][i]);
          set_pair(r, i, v);
        }
        store_raw8<T, LAY>(y, at + s * kSlab, lane, D, r);
      }
    }
    ring.done();
    x += in_step;
    residual += in_step;
    sum += out_step;
    y += out_step;
  }
}

// ---- backward --------------------------------------------------------------------
// Group g of G takes rows g, g + G, ...
template <typename T, Lay LAY, int SLABS, int THREADS>
__global__ void __launch_bounds__(THREADS, kOfSm<THREADS, SLABS> / THREADS)
    layer_norm_grad_kernel(const __grid_constant__ NormArgs a) {
  constexpr int kStages = kStagesOf<T, LAY, SLABS, 3, THREADS>;
  __shared__ RowSums sums;
  extern __shared__ __align__(16) unsigned char smem[];  // the ring, then [groups][dim]
  overlap_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int group = warp / a.row_warps, D = a.dim;
  const int at = warp % a.row_warps * SLABS * kSlab, c0 = column<LAY>(at, lane, 0);
  const uint32_t stride = gridDim.x * a.groups, rows = (uint32_t)a.rows;
  uint32_t row = blockIdx.x * a.groups + group;
  const int64_t x_step = stride * a.row_stride, grad_step = stride * a.grad_stride;
  // where the row at work lies, and the next one to ask for
  const T *x = static_cast<const T*>(a.x) + row * a.row_stride,
          *d_y = static_cast<const T*>(a.d_y) + row * a.grad_stride,
          *d_sum = static_cast<const T*>(a.d_sum) + row * a.grad_stride;
  T* d_x = static_cast<T*>(a.d_x) + row * a.grad_stride;
  RowRing<T, LAY, SLABS, 3, kStages> ring(smem, D - c0);
  const T *x_ahead = x + c0, *d_y_ahead = d_y + c0, *d_sum_ahead = d_sum + c0;
  uint32_t row_ahead = row;
  auto ask = [&] {
    if (row_ahead < rows && within(row_ahead, (int64_t)row_ahead + 1, 0, rows, a.err)) {
      ring.ask(0, x_ahead);
      ring.ask(1, d_y_ahead);
      if (a.d_sum) ring.ask(2, d_sum_ahead);
    }
    ring.close();
    row_ahead += stride;
    x_ahead += x_step;
    d_y_ahead += grad_step;
    d_sum_ahead += grad_step;
  };
  if (kStages > 0)
    for (int i = 0; i < kStages - 1; ++i) ask();
  constexpr int kHeld = SLABS <= kHeldSlabs ? SLABS : 1;
  float2 dw[SLABS][kPairs], db[SLABS][kPairs], w[kHeld][kPairs];
#pragma unroll
  for (int s = 0; s < SLABS; ++s)
#pragma unroll
    for (int i = 0; i < kPairs; ++i) dw[s][i] = db[s][i] = both(0.0f);
  auto weights = [&](int s) {
    if (a.weight)
      weights8<LAY>(w[s % kHeld], a.weight, a.weight_bf16, at + s * kSlab, lane, D);
    else
#pragma unroll
      for (int i = 0; i < kPairs; ++i) w[s % kHeld][i] = both(1.0f);
  };
  if (SLABS == kHeld)
#pragma unroll
    for (int s = 0; s < SLABS; ++s) weights(s);
  const float per = 1.0f / (float)D;
  float mean = 0.0f, rstd = 0.0f, mean_next = 0.0f, rstd_next = 0.0f;
  if (row < rows) {
    mean_next = a.mean[row];
    rstd_next = a.rstd[row];
  }
  for (int turn = 0; row < rows; row += stride, turn ^= 1) {
    const bool in = within(row, (int64_t)row + 1, 0, rows, a.err);
    mean = mean_next;
    rstd = rstd_next;
    if (row + stride < rows) {
      mean_next = a.mean[row + stride];
      rstd_next = a.rstd[row + stride];
    }
    Raw8<T> xs[SLABS] = {}, dy[SLABS] = {};
    if (kStages > 0) {
      ask();
      ring.wait();
    }
#pragma unroll
    for (int s = 0; s < SLABS; ++s) {
      if (kStages > 0) {
        xs[s] = ring.take(0, s);
        dy[s] = ring.take(1, s);
      } else if (in) {
        xs[s] = load8<T, LAY>(x, at + s * kSlab, lane, D);
        dy[s] = load8<T, LAY>(d_y, at + s * kSlab, lane, D);
      }
    }
    float2 sum_g = both(0.0f), sum_gx = both(0.0f);
#pragma unroll
    for (int s = 0; s < SLABS; ++s) {
      if (SLABS > kHeld) weights(s);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        // (past the row's end dy is 0, and so is all that it multiplies)
        const float2 xh = __fmul2_rn(__fadd2_rn(pair_of(xs[s], i), both(-mean)), both(rstd));
        const float2 d = pair_of(dy[s], i), g = __fmul2_rn(d, w[s % kHeld][i]);
        sum_g = __fadd2_rn(sum_g, g);
        sum_gx = __ffma2_rn(g, xh, sum_gx);
        dw[s][i] = __ffma2_rn(d, xh, dw[s][i]);
        db[s][i] = __fadd2_rn(db[s][i], d);
      }
    }
    const float2 t =
        sums(make_float2(sum_g.x + sum_g.y, sum_gx.x + sum_gx.y), a.row_warps, group, turn);
    const float2 c1 = both(-t.x * per), c2 = both(-t.y * per);
    if (in) {
#pragma unroll
      for (int s = 0; s < SLABS; ++s) {
        if (kStages > 0) {  // (read again: registers are few)
          xs[s] = ring.take(0, s);
          dy[s] = ring.take(1, s);
        }
        Raw8<T> past = {}, r;
        if (a.d_sum)
          past = kStages > 0 ? ring.take(2, s) : load8<T, LAY>(d_sum, at + s * kSlab, lane, D);
        if (SLABS > kHeld) weights(s);
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const float2 xh = __fmul2_rn(__fadd2_rn(pair_of(xs[s], i), both(-mean)), both(rstd));
          const float2 g = __fmul2_rn(pair_of(dy[s], i), w[s % kHeld][i]);
          const float2 v = __fadd2_rn(__ffma2_rn(xh, c2, g), c1);
          set_pair(r, i, __ffma2_rn(v, both(rstd), pair_of(past, i)));
        }
        store_raw8<T, LAY>(d_x, at + s * kSlab, lane, D, r);
      }
    }
    ring.done();
    x += x_step;
    d_y += grad_step;
    d_sum += grad_step;
    d_x += grad_step;
  }
  // The block's sums of its columns, then to scratch memory.
  float* columns = reinterpret_cast<float*>(smem);
  if (kStages > 0) asm volatile("cp.async.wait_all;" ::: "memory");
  for (int which = 0; which < 2; ++which) {
    if (!(which ? a.want_bias : a.want_weight)) continue;
    float* to = a.parts + ((int64_t)blockIdx.x * 2 + which) * D;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < SLABS; ++s)
#pragma unroll
      for (int k = 0; k < kLane; ++k) {
        const int c = column<LAY>(at + s * kSlab, lane, k);
        const float2 v = which ? db[s][k / 2] : dw[s][k / 2];
        if (c < D) columns[group * D + c] = k % 2 ? v.y : v.x;
      }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
      float v = 0.0f;
      for (int g = 0; g < a.groups; ++g) v += columns[g * D + c];
      to[c] = v;
    }
  }
}

// The blocks' sums joined: 32 columns a block, each warp takes every 32nd part.
constexpr int kJoinWarps = 32;
struct JoinArgs {
  const float* parts;
  void *d_weight, *d_bias;
  int32_t dim, blocks;
  bool bf16;
};
__global__ void __launch_bounds__(32 * kJoinWarps)
    join_columns_kernel(const __grid_constant__ JoinArgs a) {
  __shared__ float part[2][kJoinWarps][32];
  overlap_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  float v[2] = {0.0f, 0.0f};
  if (c < a.dim)
#pragma unroll 4
    for (int b = warp; b < a.blocks; b += kJoinWarps) {
      const float* p = a.parts + (int64_t)b * 2 * a.dim + c;
      if (a.d_weight) v[0] += p[0];
      if (a.d_bias) v[1] += p[a.dim];
    }
  part[0][warp][lane] = v[0];
  part[1][warp][lane] = v[1];
  __syncthreads();
  if (warp > 1 || c >= a.dim) return;
  void* out = warp ? a.d_bias : a.d_weight;
  if (!out) return;
  float sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) sum += part[warp][w][lane];
  if (a.bf16)
    put(static_cast<__nv_bfloat16*>(out) + c, sum);
  else
    put(static_cast<float*>(out) + c, sum);
}

// How a row of `dim` columns is laid over warps, and how many rows share a block.
struct Shape {
  int row_warps, slabs, groups, block;  // block: the most threads of its kernel
  int threads() const { return 32 * row_warps * groups; }
};
constexpr int kSMs = 152;  // (fixed, so that the backward pass's sums are)

// One slab a warp up to 1024 columns (8192 x 768 forward 12.4 us, three slabs a warp
// 16.3) and for rows that start anywhere up to 8192, whose single elements want
// threads (8191 x 1023 24.9 against 34.1); two up to 8192, three up to
// 12288 (4096 x 12288 backward 104 us against 134 with four, whose warps are fewer), four
// beyond.
Shape shape_of(int64_t rows, int64_t dim, bool one) {
  const int n = (int)((dim + kSlab - 1) / kSlab);
  Shape s;
  s.slabs = n <= 4 || (one && n <= 32) ? 1 : n <= 32 ? 2 : n <= 48 ? 3 : 4;
  s.row_warps = (n + s.slabs - 1) / s.slabs;
  s.block = s.row_warps > 16 ? 1024 : s.slabs > 1 || s.row_warps > 12 ? 512 : 384;
  // few rows are spread over the SMs before they share blocks
  const int64_t each = (rows + 2 * kSMs - 1) / (2 * kSMs);
  const int64_t most = s.block / 32 / s.row_warps;
  s.groups = (int)(each < 1 ? 1 : each < most ? each : most);
  return s;
}

int blocks_of(const Shape& s, int64_t rows) {
  const int64_t blocks = (rows + s.groups - 1) / s.groups;
  const int64_t most =
      kSMs * (s.block > 512 || s.slabs > 1 ? 1 : 2);
  return (int)(blocks < most ? blocks : most);
}

constexpr int kMostSmem = 208 << 10;  // dynamic shared memory of any of these kernels
template <typename K>
cudaError_t launch_rows_kernel(K* kernel, const NormArgs& a, const Shape& s, int smem,
                               cudaStream_t stream) {
  if (smem > 40 << 10) {  // (beside what the kernels declare)
    // the same for every call: another thread's must not lower it before this one's launch
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(kernel, dim3((unsigned)blocks_of(s, a.rows)), dim3(s.threads()), smem,
                       stream, a);
}

template <typename T, Lay LAY, int SLABS, int THREADS>
cudaError_t launch_as(const NormArgs& a, const Shape& s, bool grad, cudaStream_t stream) {
  if (!grad) {
    constexpr int kRing = RowRing<T, LAY, SLABS, 2, kStagesOf<T, LAY, SLABS, 2, THREADS>>::kBytes;
    return launch_rows_kernel(layer_norm_kernel<T, LAY, SLABS, THREADS>, a, s,
                              kRing * s.threads(), stream);
  }
  constexpr int kRing = RowRing<T, LAY, SLABS, 3, kStagesOf<T, LAY, SLABS, 3, THREADS>>::kBytes;
  const int ring = kRing * s.threads(), columns = s.groups * a.dim * 4;
  return launch_rows_kernel(layer_norm_grad_kernel<T, LAY, SLABS, THREADS>, a, s,
                            ring > columns ? ring : columns, stream);
}

template <typename T, Lay LAY>
cudaError_t launch_shape(NormArgs a, bool grad, cudaStream_t stream) {
  const Shape s = shape_of(a.rows, a.dim, LAY == kOne);
  a.row_warps = s.row_warps;
  a.groups = s.groups;
  if (s.slabs == 4)
    return s.block == 512 ? launch_as<T, LAY, 4, 512>(a, s, grad, stream)
                          : launch_as<T, LAY, 4, 1024>(a, s, grad, stream);
  if (s.slabs == 3) return launch_as<T, LAY, 3, 512>(a, s, grad, stream);
  if (s.slabs == 2) return launch_as<T, LAY, 2, 512>(a, s, grad, stream);
  return s.block == 384   ? launch_as<T, LAY, 1, 384>(a, s, grad, stream)
         : s.block == 512 ? launch_as<T, LAY, 1, 512>(a, s, grad, stream)
                          : launch_as<T, LAY, 1, 1024>(a, s, grad, stream);
}

// Whether every row (and weight) may be read in 16-byte accesses.
bool aligned(const LayerNormLaunch& in, bool grad) {
  const int es = in.dtype == ZS_BF16 ? 2 : 4, ws = in.weight_dtype == ZS_BF16 ? 2 : 4;
  if (!rows_aligned(in.x, in.row_stride, es) || !rows_aligned(in.weight, 16, ws)) return false;
  if (grad)
    return rows_aligned(in.d_y, in.grad_stride, es) && rows_aligned(in.d_x, in.grad_stride, es) &&
           rows_aligned(in.d_sum, in.grad_stride, es);
  return rows_aligned(in.residual, in.row_stride, es) && rows_aligned(in.y, in.out_stride, es) &&
         rows_aligned(in.sum, in.out_stride, es) && rows_aligned(in.bias, 16, ws);
}

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
  a.weight_bf16 = in.weight_dtype == ZS_BF16;
  a.want_weight = in.d_weight != nullptr;
  a.want_bias = in.d_bias != nullptr;
  a.eps = (float)in.eps;
  a.err = ZS_BOUNDS_CHECK ? device_error_word() : nullptr;
  if (ZS_BOUNDS_CHECK && !a.err) return cudaErrorInvalidSymbol;
  const bool vec = aligned(in, grad);
  if (in.dtype == ZS_BF16)
    return vec ? launch_shape<__nv_bfloat16, kEight>(a, grad, stream)
               : launch_shape<__nv_bfloat16, kOne>(a, grad, stream);
  return vec ? launch_shape<float, kFour>(a, grad, stream)
             : launch_shape<float, kOne>(a, grad, stream);
}

int parts_of(const LayerNormLaunch& in) {
  const bool one = !aligned(in, true);
  return blocks_of(shape_of(in.rows, in.dim, one), in.rows);
}

}  // namespace

int64_t layer_norm_grad_workspace_bytes(int64_t rows, int64_t dim) {
  const int one = blocks_of(shape_of(rows, dim, true), rows),
            vec = blocks_of(shape_of(rows, dim, false), rows);
  return 2 * (int64_t)sizeof(float) * (one > vec ? one : vec) * dim;
}

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
  j.blocks = in.rows > 0 ? parts_of(in) : 0;
  j.bf16 = in.grad_dtype == ZS_BF16;
  return launch_kernel(join_columns_kernel, dim3((unsigned)((j.dim + 31) / 32)),
                       dim3(32 * kJoinWarps), 0, stream, j);
}

}  // namespace zs
