// row_vec.cuh — rows of bf16 or fp32 elements in slabs of 256 columns, eight
// elements a lane, for the kernels that hold a row (or a part of one) in a
// warp's registers. Included by the library's .cu files only.
//
// A lane's eight elements lie in one of three ways:
//   kEight  side by side: one 16-byte access of bf16, 32 bytes of fp32
//   kFour   twice four side by side, 128 columns apart: two 16-byte accesses of
//           fp32 whose warps cover whole sectors each (cp.async has no wider one)
//   kOne    32 columns apart each, for rows that start at any element
// The first two want rows that start on 16-byte boundaries. Columns past the row's
// end are not touched and read as 0.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bounds.cuh"

namespace zs {

constexpr int kSlab = 256;  // columns
constexpr int kLane = 8;    // elements of a lane in a slab

// The one rounding of a result to its type: to nearest even.
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// A lane's eight elements as stored.
template <typename T>
struct Raw8 {
  uint32_t w[kLane * sizeof(T) / 4];
};

enum Lay { kOne, kFour, kEight };

template <Lay LAY>
__device__ __forceinline__ int column(int col0, int lane, int k) {
  return LAY == kEight  ? col0 + lane * 8 + k
         : LAY == kFour ? col0 + k / 4 * 128 + lane * 4 + k % 4
                        : col0 + k * 32 + lane;
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

// N words at p, in accesses of 16 bytes, of 32 where p allows.
template <int N>
__device__ __forceinline__ void load_words(uint32_t* w, const void* p) {
  if (N == 8 && (uintptr_t)p % 32 == 0) {
    asm volatile("ld.global.L1::no_allocate.v8.u32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[N - 4]), "=r"(w[N - 3]),
                   "=r"(w[N - 2]), "=r"(w[N - 1])
                 : "l"(p));
    return;
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint4 v = load16(static_cast<const uint4*>(p) + i);
    w[4 * i] = v.x;
    w[4 * i + 1] = v.y;
    w[4 * i + 2] = v.z;
    w[4 * i + 3] = v.w;
  }
}
template <int N>
__device__ __forceinline__ void store_words(void* p, const uint32_t* w, bool once = false) {
  if (once) {  // L2 is told to let it go first
    if (N == 8 && (uintptr_t)p % 32 == 0) {
      asm volatile("st.global.L2::evict_first.v8.u32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
                   "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[N - 4]), "r"(w[N - 3]),
                   "r"(w[N - 2]), "r"(w[N - 1])
                   : "memory");
      return;
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      asm volatile("st.global.cs.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(static_cast<uint4*>(p) + i),
                   "r"(w[4 * i]), "r"(w[4 * i + 1]), "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                   : "memory");
    return;
  }
  if (N == 8 && (uintptr_t)p % 32 == 0) {
    asm volatile("st.global.v8.u32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[N - 4]), "r"(w[N - 3]), "r"(w[N - 2]),
                 "r"(w[N - 1])
                 : "memory");
    return;
  }
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    store16(static_cast<uint4*>(p) + i,
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
}

// The lane's elements of the slab at col0 of a row of D columns. (kFour: fp32 alone.)
template <typename T, Lay LAY>
__device__ __forceinline__ Raw8<T> load8(const T* row, int col0, int lane, int D) {
  static_assert(LAY != kFour || sizeof(T) == 4, "bf16 rows lie as kEight");
  Raw8<T> r;
  constexpr int kWords = kLane * (int)sizeof(T) / 4;
  if (LAY == kEight && col0 + lane * 8 + 8 <= D) {
    load_words<kWords>(r.w, row + col0 + lane * 8);
    return r;
  }
  if (LAY == kFour && col0 + 128 + lane * 4 + 4 <= D) {
    load_words<4>(r.w, row + col0 + lane * 4);
    load_words<4>(r.w + kWords - 4, row + col0 + 128 + lane * 4);
    return r;
  }
#pragma unroll
  for (int k = 0; k < kLane; ++k) {
    const int c = column<LAY>(col0, lane, k);
    set_raw(r, k, c < D ? row[c] : T(0.0f));
  }
  return r;
}

template <typename T, Lay LAY>
__device__ __forceinline__ void store_raw8(T* row, int col0, int lane, int D, const Raw8<T>& r,
                                           bool once = false) {
  constexpr int kWords = kLane * (int)sizeof(T) / 4;
  if (LAY == kEight && col0 + lane * 8 + 8 <= D) {
    store_words<kWords>(row + col0 + lane * 8, r.w, once);
    return;
  }
  if (LAY == kFour && col0 + 128 + lane * 4 + 4 <= D) {
    store_words<4>(row + col0 + lane * 4, r.w);
    store_words<4>(row + col0 + 128 + lane * 4, r.w + kWords - 4);
    return;
  }
#pragma unroll
  for (int k = 0; k < kLane; ++k) {
    const int c = column<LAY>(col0, lane, k);
    if (c < D) put(row + c, raw_value(r, k));  // exact: the value has the type already
  }
}

template <typename T, Lay LAY>
__device__ __forceinline__ void store8(T* row, int col0, int lane, int D, const float* v,
                                       bool once = false) {
  Raw8<T> r;
#pragma unroll
  for (int k = 0; k < kLane; ++k) {
    T x;
    put(&x, v[k]);
    set_raw(r, k, x);
  }
  store_raw8<T, LAY>(row, col0, lane, D, r, once);
}

// A lane's elements two by two, for the packed fp32 arithmetic.
__device__ __forceinline__ float2 pair_of(const Raw8<float>& r, int i) {
  return {__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1])};
}
__device__ __forceinline__ float2 pair_of(const Raw8<__nv_bfloat16>& r, int i) {
  return {__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xFFFF0000u)};
}
__device__ __forceinline__ void set_pair(Raw8<float>& r, int i, float2 v) {
  r.w[2 * i] = __float_as_uint(v.x);
  r.w[2 * i + 1] = __float_as_uint(v.y);
}
__device__ __forceinline__ void set_pair(Raw8<__nv_bfloat16>& r, int i, float2 v) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
  r.w[i] = *reinterpret_cast<const uint32_t*>(&b);
}
// a + b, rounded once.
__device__ __forceinline__ Raw8<float> sum_of(const Raw8<float>& a, const Raw8<float>& b) {
  Raw8<float> r;
#pragma unroll
  for (int i = 0; i < kLane / 2; ++i) set_pair(r, i, __fadd2_rn(pair_of(a, i), pair_of(b, i)));
  return r;
}
__device__ __forceinline__ Raw8<__nv_bfloat16> sum_of(const Raw8<__nv_bfloat16>& a,
                                                      const Raw8<__nv_bfloat16>& b) {
  Raw8<__nv_bfloat16> r;
#pragma unroll
  for (int i = 0; i < kLane / 2; ++i) {
    const __nv_bfloat162 v = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162*>(&a.w[i]),
                                        *reinterpret_cast<const __nv_bfloat162*>(&b.w[i]));
    r.w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return r;
}

// Rows at p, `stride` elements apart, that load8 and store8 may take as kEight or kFour.
inline bool rows_aligned(const void* p, int64_t stride, int elem_bytes) {
  return p == nullptr || ((uintptr_t)p % 16 == 0 && stride * elem_bytes % 16 == 0);
}

}  // namespace zs
