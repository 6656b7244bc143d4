// row_vec.cuh — rows of bf16 or fp32 elements in slabs of 256 columns, eight
// elements a lane, for the kernels that hold a row (or a part of one) in a
// warp's registers. Included by the library's .cu files only.
//
// VEC: rows start on 16-byte boundaries, and a lane's eight elements are
// neighbours (one 16-byte access of bf16, two of fp32). Otherwise rows start at
// any element, and a lane's elements are 32 columns apart, so that a warp's
// accesses still cover whole sectors. Columns past the row's end are not
// touched and read as 0.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bounds.cuh"

namespace zs {

constexpr int kSlab = 256;  // columns
constexpr int kLane = 8;    // elements of a lane in a slab

__device__ __forceinline__ float value_of(float x) { return x; }
__device__ __forceinline__ float value_of(__nv_bfloat16 x) { return __bfloat162float(x); }
// The one rounding of a result to its type: to nearest even.
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
// x rounded to T.
__device__ __forceinline__ float rounded(float x, float) { return x; }
__device__ __forceinline__ float rounded(float x, __nv_bfloat16) {
  return __bfloat162float(__float2bfloat16_rn(x));
}

// A lane's eight elements as stored.
template <typename T>
struct Raw8 {
  uint32_t w[kLane * sizeof(T) / 4];
};

template <bool VEC>
__device__ __forceinline__ int column(int col0, int lane, int k) {
  return VEC ? col0 + lane * kLane + k : col0 + k * 32 + lane;
}

__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ void store16(void* p, uint4 v) {
  asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

__device__ __forceinline__ void set_raw(Raw8<float>& r, int k, float x) {
  r.w[k] = __float_as_uint(x);
}
__device__ __forceinline__ void set_raw(Raw8<__nv_bfloat16>& r, int k, __nv_bfloat16 x) {
  const uint32_t bits = __bfloat16_as_ushort(x);
  r.w[k / 2] = k % 2 ? (r.w[k / 2] & 0xFFFFu) | bits << 16 : bits;
}
__device__ __forceinline__ float raw_value(const Raw8<float>& r, int k) {
  return __uint_as_float(r.w[k]);
}
__device__ __forceinline__ float raw_value(const Raw8<__nv_bfloat16>& r, int k) {
  return __uint_as_float(k % 2 ? r.w[k / 2] & 0xFFFF0000u : r.w[k / 2] << 16);
}

// The lane's elements of the slab at col0 of a row of D columns.
template <typename T, bool VEC>
__device__ __forceinline__ Raw8<T> load8(const T* row, int col0, int lane, int D) {
  Raw8<T> r;
  if (VEC && col0 + lane * kLane + kLane <= D) {
    const T* p = row + col0 + lane * kLane;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      const uint4 v = load16(reinterpret_cast<const uint4*>(p) + i);
      r.w[4 * i] = v.x;
      r.w[4 * i + 1] = v.y;
      r.w[4 * i + 2] = v.z;
      r.w[4 * i + 3] = v.w;
    }
    return r;
  }
#pragma unroll
  for (int k = 0; k < kLane; ++k) {
    const int c = column<VEC>(col0, lane, k);
    set_raw(r, k, c < D ? row[c] : T(0.0f));
  }
  return r;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* row, int col0, int lane, int D, const float* v) {
  if (VEC && col0 + lane * kLane + kLane <= D) {
    Raw8<T> r;
#pragma unroll
    for (int k = 0; k < kLane; ++k) {
      T x;
      put(&x, v[k]);
      set_raw(r, k, x);
    }
    T* p = row + col0 + lane * kLane;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      store16(reinterpret_cast<uint4*>(p) + i,
              make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]));
    return;
  }
#pragma unroll
  for (int k = 0; k < kLane; ++k) {
    const int c = column<VEC>(col0, lane, k);
    if (c < D) put(row + c, v[k]);
  }
}

// Rows at p, `stride` elements apart, that load8 and store8 may take as VEC.
inline bool rows_aligned(const void* p, int64_t stride, int elem_bytes) {
  return p == nullptr || ((uintptr_t)p % 16 == 0 && stride * elem_bytes % 16 == 0);
}

}  // namespace zs
