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
//
// Bound: HBM. A call reads its logits once (V * 2 or 4 bytes a row) and, with
// a gradient, writes as much; 6 to 15 flops and one or two exponentials an
// element. On GB300, as a share of the measured copy bandwidth (6779 GB/s):
// scoring 4096 x 151936 bf16 180 us = 1.02; evaluating 8192 x 32000 bf16, T = 2
// with hard labels, 85.3 us = 0.91; the gradient alone of 8192 x 50257 bf16 237 us
// = 0.99; loss and gradient in one call 0.87 (4095 x 32000, 89.3 us) and 0.77
// (8192 x 151936, 954 us), where a block's reading and writing take turns; 64
// alternatives of 8191 x 32000 fp32 220 us = 0.71, the search coming after the
// stream. Short rows are bound by what a row takes beside its bytes (16384 x 1000
// bf16: 17.4 us = 0.28, with 20 alternatives 62 us = 0.09). Small calls take 3 to
// 8 us of GPU time, less than a call from Python.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "bounds.cuh"
#include "overlap.cuh"
#include "zs_internal.h"

namespace zs {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxThreads = 256;         // of a row's block (32, 64, 128 or 256)
constexpr int kResident = 1024;          // threads of an SM: 64 registers each
constexpr int kSMs = 152;
constexpr int kMaxSplit = 8;             // blocks of a row: the portable cluster size
constexpr int64_t kRowsInL2 = 96 << 20;  // bytes of rows in flight that L2 (129 MB) keeps
constexpr int64_t kTableBytes = 40 << 10;
constexpr int kMaxSmem = 200 * 1024;     // dynamic shared memory of a block

struct RowArgs {
  const void* logits;
  void* d_logits;
  int64_t row_stride, grad_stride;
  int32_t vocab, shift, top_k, teacher_k;  // a row has 2^shift blocks
  bool teacher_bf16;
  bool distill;   // targets are hard labels at T = 1
  float inv_t, scale;  // 1/T, log2(e)/T
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

// ---- the row in 32-byte chunks -------------------------------------------------
// A chunk is one thread's widest load, aligned in memory: 16 bf16 or 8 fp32
// logits. Rows start at any element (an odd vocabulary's do), so a row is a
// head of single elements up to the first boundary, whole chunks, and a tail.
constexpr int kChunkBytes = 32;
constexpr int kWords = kChunkBytes / 4;
template <typename T>
constexpr int kPer = kChunkBytes / (int)sizeof(T);

// A block's part of a row: part `rank` of 2^shift takes its share of the body;
// the first one the head as well, the last one the tail.
struct Part {
  int lo, hi;            // its elements
  int head, body, tail;  // elements, chunks, elements
  int chunk0;            // its first chunk's place in the whole row's body
};
template <typename T>
__device__ __forceinline__ Part part_of(const T* z, int V, int rank, int shift) {
  const int head = min(V, (int)((0 - (uintptr_t)z) % kChunkBytes / sizeof(T)));
  const int body = (V - head) / kPer<T>;
  const int c0 = body * rank >> shift, c1 = body * (rank + 1) >> shift;  // below 2^21
  Part p;
  p.chunk0 = c0;
  p.body = c1 - c0;
  p.head = rank == 0 ? head : 0;
  p.lo = rank == 0 ? 0 : head + c0 * kPer<T>;
  p.tail = rank + 1 == 1 << shift ? V - head - body * kPer<T> : 0;
  p.hi = head + c1 * kPer<T> + p.tail;
  return p;
}

// How long L2 should hold what a load brings: as ever; until it is read again
// (a row whose gradient follows its sums); no longer.
enum Hold { kUsual, kUntilRead, kOnce };
template <Hold HOLD>
__device__ __forceinline__ void load_chunk(uint32_t* w, const void* p) {
#define ZS_LOAD_CHUNK(hold)                                                                    \
  asm volatile("ld.global.L1::no_allocate" hold                                                \
               ".v8.u32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"                               \
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),       \
                 "=r"(w[6]), "=r"(w[7])                                                        \
               : "l"(p)                                                                        \
               : "memory")
  if (HOLD == kUsual)
    ZS_LOAD_CHUNK("");
  else if (HOLD == kUntilRead)
    ZS_LOAD_CHUNK(".L2::evict_last");
  else
    ZS_LOAD_CHUNK(".L2::evict_first");
#undef ZS_LOAD_CHUNK
}
// Elements 2i and 2i+1 of a chunk.
__device__ __forceinline__ float2 pair_of(const uint32_t* w, int i, __nv_bfloat16) {
  return {__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)};
}
__device__ __forceinline__ float2 pair_of(const uint32_t* w, int i, float) {
  return {__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])};
}
// The chunk's maximum (NaN if it holds one); bf16 maxima two at a time.
__device__ __forceinline__ float max_of(const uint32_t* w, __nv_bfloat16) {
  __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(w);
#pragma unroll
  for (int i = 1; i < kWords; ++i)
    m = __hmax2_nan(m, *reinterpret_cast<const __nv_bfloat162*>(w + i));
  return __bfloat162float(__hmax_nan(m.x, m.y));
}
__device__ __forceinline__ float max_nan(float x, float y) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(x), "f"(y));
  return m;
}
__device__ __forceinline__ float max_of(const uint32_t* w, float) {
  float m = __uint_as_float(w[0]);
#pragma unroll
  for (int i = 1; i < kWords; ++i) m = max_nan(m, __uint_as_float(w[i]));
  return m;
}

// The largest of the warp's (those that are NaN do not count).
__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

// 2^x to 2 units in the last place; results below the normal range become 0.
__device__ __forceinline__ float exp2_fast(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
  return e;
}
// A log2 weight that is 2^-10000 = 0 rather than 2^-inf: 0 * -inf is not 0.
__device__ __forceinline__ float clamped(float d) { return fmaxf(d, -1e4f); }

// ---- one pass over the row ------------------------------------------------------
// S and U (and S1, the sum at T = 1) relative to the largest logit m that the
// warp has met: no e exceeds 1, and no term of U is above 0. m = -inf until a
// finite logit was seen (ref is 0 meanwhile). The warp's threads move together: on
// its own each would rise with every record of its few dozen chunks, at another
// step than the others (8192 x 32000 bf16, T = 2 with hard labels: 88.9 us; with the
// warp 85.3; sums left up to 2^8 above the reference, whose U cancels, 85.5).
template <bool ENTROPY, bool OWN>
struct Stats {
  float m = -INFINITY, ref = 0.0f;
  float2 s = {0.0f, 0.0f}, u = {0.0f, 0.0f}, s1 = {0.0f, 0.0f};

  __device__ __forceinline__ void move_to(float to, float scale) {
    const float delta = m == -INFINITY ? -1e4f : clamped((ref - to) * scale);
    const float f = exp2_fast(delta);
    if (ENTROPY) {
      u.x = f * fmaf(s.x, delta, u.x);
      u.y = f * fmaf(s.y, delta, u.y);
    }
    s.x *= f;
    s.y *= f;
    if (OWN) {
      const float f1 = m == -INFINITY ? 0.0f : exp2_fast((ref - to) * kLog2e);
      s1.x *= f1;
      s1.y *= f1;
    }
    m = ref = to;
  }
  __device__ __forceinline__ void add(float2 z, float scale) {
    const float2 x = __fadd2_rn(z, {-ref, -ref});
    const float2 d = __fmul2_rn(x, {scale, scale});
    const float2 e = {exp2_fast(d.x), exp2_fast(d.y)};
    s = __fadd2_rn(s, e);
    if (ENTROPY) u = __ffma2_rn(e, {clamped(d.x), clamped(d.y)}, u);
    if (OWN) {
      const float2 d1 = __fmul2_rn(x, {kLog2e, kLog2e});
      s1 = __fadd2_rn(s1, {exp2_fast(d1.x), exp2_fast(d1.y)});
    }
  }
  template <typename T>
  __device__ __forceinline__ void add_chunk(const uint32_t* w, float scale) {
#pragma unroll
    for (int i = 0; i < kPer<T> / 2; ++i) add(pair_of(w, i, T()), scale);
  }
  __device__ __forceinline__ void add_one(float z, float scale) {
    if (z > m) move_to(z, scale);
    add({z, -INFINITY}, scale);
  }
};

// What a group of threads knows of a row: m and the sums relative to it
// (m = -inf: no finite logit, sums 0 or NaN).
struct Sums {
  float m, s, u, s1;
};
// The factor's exponent from reference m to the group's M.
__device__ __forceinline__ float toward(float m, float M, float scale) {
  return M == -INFINITY ? 0.0f : clamped((m - M) * scale);
}
template <bool OWN>
__device__ __forceinline__ Sums moved(const Sums& a, float M, float scale) {
  const float delta = toward(a.m, M, scale), f = exp2_fast(delta);
  const float f1 = OWN ? exp2_fast(toward(a.m, M, kLog2e)) : 0.0f;
  return {M, f * a.s, f * fmaf(a.s, delta, a.u), f1 * a.s1};
}

// What a block's warps share to join their sums and their largest u.
struct BlockSums {
  Sums sums[kMaxThreads / 32];
  float u[kMaxThreads / 32];
};
// The sums of groups of n lanes (a power of two), in a fixed order.
template <bool ENTROPY, bool OWN>
__device__ __forceinline__ Sums lane_sums(Sums t, int n, float scale) {
  float M = t.m;
  for (int off = n / 2; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
  t = moved<OWN>(t, M, scale);
  for (int off = n / 2; off > 0; off >>= 1) {
    t.s += __shfl_xor_sync(0xFFFFFFFFu, t.s, off);
    if (ENTROPY) t.u += __shfl_xor_sync(0xFFFFFFFFu, t.u, off);
    if (OWN) t.s1 += __shfl_xor_sync(0xFFFFFFFFu, t.s1, off);
  }
  return t;
}
__device__ __forceinline__ float lane_max(float x, int n) {
  for (int off = n / 2; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, off));
  return x;
}
// The block's sums, in a fixed order, and its largest u; every thread gets them.
template <int THREADS, bool ENTROPY, bool OWN>
__device__ __forceinline__ Sums block_sums(Sums t, float scale, float* u, BlockSums& sm) {
  constexpr int kWarps = THREADS / 32;
  t = lane_sums<ENTROPY, OWN>(t, 32, scale);
  *u = lane_max(*u, 32);
  if ((threadIdx.x & 31) == 0) {
    sm.sums[threadIdx.x >> 5] = t;
    sm.u[threadIdx.x >> 5] = *u;
  }
  __syncthreads();
  if (THREADS == 32) return t;
  *u = lane_max(sm.u[threadIdx.x % kWarps], kWarps);
  return lane_sums<ENTROPY, OWN>(sm.sums[threadIdx.x % kWarps], kWarps, scale);
}

// ---- the top alternatives -------------------------------------------------------
// Unique keys that order logits as the alternatives are ranked: NaN above all,
// then by value (-0 as +0), then the lowest position first. 0 is below them all.
// The value takes the upper half; of a bf16's only the upper 16 bits count.
template <typename T>
__device__ __forceinline__ uint64_t rank_key(float z, int32_t position) {
  uint32_t u = __float_as_uint(z + 0.0f);
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  if (z != z) u = 0xFFFFFFFFu;
  if (sizeof(T) == 2) u &= 0xFFFF0000u;
  return ((uint64_t)u << 32) | (uint32_t)~position;
}

// The value of a key (NaN for a NaN's and for key 0).
template <typename T>
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t u = (uint32_t)(key >> 32);
  const uint32_t bits = (u & 0x80000000u) ? u ^ 0x80000000u : ~u;
  return __uint_as_float(sizeof(T) == 2 ? bits & 0xFFFF0000u : bits);
}

// The pass over the row leaves every chunk's maximum in shared memory, and each
// thread knows the best of its own chunks. A chunk is ranked by its maximum,
// equal ones by position. If k chunks reach a bound, the row's top k elements
// do, each taken at its chunk's position: an element below the bound is beaten
// by the maxima of all k. So a bound that about k of the threads' best chunks
// reach leaves few chunks to read again and few elements to rank.
// Table entry p: body chunk p; then the tail and the head (whose position comes
// first). An end without elements has key 0. Entry p belongs to thread p modulo
// the block.

// Elements that may be ranked: those of k chunks at least, and enough for the
// sorted lists of a row's blocks.
__host__ __device__ __forceinline__ int list_capacity(int k) { return 16 * (k < 16 ? 16 : k); }
constexpr int kFound = 512;    // chunks that are read again; ZS_MAX_TOP at least
struct TopShared {
  uint64_t best[ZS_MAX_TOP];
  int found[kFound];
  int count, total;
  int capacity;    // of the list
  uint64_t* list;  // after this, then the table
};
// A bound that at least k of the keys reach, and at most `most` where unique
// keys allow it: bit by bit from the top, count(bound) being how many keys of
// the block are >= bound (called by all its threads).
template <typename T, typename F>
__device__ __forceinline__ uint64_t bound_of(int k, int most, F count) {
  uint64_t bound = 0;
  for (int bit = 63; bit >= 0; --bit) {
    if (sizeof(T) == 2 && bit >= 32 && bit < 48) continue;  // 0 in every key
    const uint64_t tried = bound | (uint64_t(1) << bit);
    const int n = count(tried);
    if (n < k) continue;
    bound = tried;
    if (n <= most) break;
  }
  return bound;
}

template <typename T>
struct Chunks {  // the table of a block's part
  Part sp;
  const T* maxima;
  __device__ __forceinline__ int count() const { return sp.body + 2; }
  __device__ __forceinline__ int position(int p) const {
    return p == sp.body + 1 ? 0 : sp.chunk0 + p + 1;
  }
  __device__ __forceinline__ uint64_t key(int p) const {
    if ((p == sp.body && sp.tail == 0) || (p == sp.body + 1 && sp.head == 0)) return 0;
    return rank_key<T>(value_of(maxima[p]), position(p));
  }
  __device__ __forceinline__ void elements(int p, int* lo, int* hi) const {
    *lo = p == sp.body + 1 ? 0 : sp.lo + sp.head + p * kPer<T>;
    *hi = p == sp.body + 1 ? sp.head : min(sp.hi, *lo + kPer<T>);
  }
};

// Ranks the part's top k into sh.best (keys, best first; position = column; 0
// where the part has no more).
// `mine`: the best key of the thread's body chunks.
template <typename T, int THREADS>
__device__ __forceinline__ void select_top(const T* z, const Chunks<T>& ch, int k, uint64_t mine,
                                           TopShared& sh, unsigned int* err) {
  const int tid = threadIdx.x;
  for (int p = ch.sp.body; p < ch.count(); ++p)
    if (p % THREADS == tid) mine = max(mine, ch.key(p));
  for (int i = tid; i < k; i += THREADS) sh.best[i] = 0;
  auto total_of = [&](int n) {
    __syncthreads();
    if (tid == 0) sh.total = 0;
    __syncthreads();
    if (n) atomicAdd(&sh.total, n);
    __syncthreads();
    return sh.total;
  };
  // Lists the elements at or above the bound: first the chunks that reach it,
  // then their elements, read again by all threads, so that these loads are in
  // flight together. More than fit are counted, not listed.
  auto list_from = [&](uint64_t bound, bool look) {
    __syncthreads();  // total_of's last answer has been read
    if (tid == 0) sh.count = sh.total = 0;
    __syncthreads();
    // Most chunks are decided by their maximum alone. Where it is the bound's value,
    // or either of them is a NaN (the bound may be 0 or a NaN's key), the key decides.
    const float at_least = key_value<T>(bound);
    for (int p0 = tid; look && p0 < ch.count(); p0 += 32 * THREADS) {
      uint32_t reach = 0;
#pragma unroll 4
      for (int i = 0; i < 32; ++i) {
        const int p = p0 + i * THREADS;
        if (p >= ch.count()) break;
        const float most = value_of(ch.maxima[p]);
        if (most < at_least) continue;
        if (!(most > at_least) || p >= ch.sp.body) {
          const uint64_t key = ch.key(p);
          if (key < bound || key == 0) continue;
        }
        reach |= 1u << i;
      }
      if (reach == 0) continue;
      int at = atomicAdd(&sh.total, __popc(reach));
      for (; reach != 0 && at < kFound; reach &= reach - 1, ++at)
        sh.found[at] = p0 + (__ffs(reach) - 1) * THREADS;
    }
    __syncthreads();
    if (sh.total > kFound) return sh.capacity + 1;
    // An element a thread, four of them on their way at once.
    const int found = sh.total * kPer<T>;
    for (int i0 = tid; i0 < found; i0 += 4 * THREADS) {
      float x[4];
      int place[4], column[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int i = i0 + f * THREADS;
        column[f] = -1;
        if (i >= found) continue;
        const int p = sh.found[i / kPer<T>];
        int lo, hi;
        ch.elements(p, &lo, &hi);
        const int j = lo + i % kPer<T>;
        if (j >= hi || !within(j, j + 1, ch.sp.lo, ch.sp.hi, err)) continue;
        x[f] = value_of(z[j]);
        place[f] = ch.position(p);
        column[f] = j;
      }
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        if (column[f] < 0 || rank_key<T>(x[f], place[f]) < bound) continue;
        const int at = atomicAdd(&sh.count, 1);
        if (at < sh.capacity) sh.list[at] = rank_key<T>(x[f], column[f]);
      }
    }
    __syncthreads();
    return sh.count;
  };
  uint64_t bound =
      bound_of<T>(k, k + k / 4 + 2, [&](uint64_t b) { return __syncthreads_count(mine >= b); });
  int n = list_from(bound, mine >= bound);
  if (n > sh.capacity) {
    // Very many in a few threads' chunks: the exact k-th best chunk leaves k chunks
    // at most (keys are unique), whose elements the list holds.
    bound = bound_of<T>(k, k, [&](uint64_t b) {
      int reach = 0;
      for (int p = tid; p < ch.count(); p += THREADS) reach += ch.key(p) >= b;
      return total_of(reach);
    });
    n = list_from(bound, true);
  }
  bound = 0;
  if (n > 512)  // ranking is quadratic: first the exact k-th best
    bound = bound_of<T>(k, k, [&](uint64_t b) {
      int reach = 0;
      for (int i = tid; i < n; i += THREADS) reach += sh.list[i] >= b;
      return total_of(reach);
    });
  // The list's order is that of its atomics; the ranks are not.
  for (int i = tid; i < n; i += THREADS) {
    const uint64_t key = sh.list[i];
    if (key < bound) continue;
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank += sh.list[j] > key;
    if (rank < k) sh.best[rank] = key;
  }
  __syncthreads();
}

// The sums of a block's part of a row: each thread keeps kFlight chunks in
// flight ahead of those that it works on, two sets of buffers taking turns (one
// copied to the other: 92 instead of 89 us for loss and gradient of 4095 x 32000
// bf16; four single ones in turn, the same registers: 238 instead of 180 us for
// 4096 x 151936 bf16). TOP: the table, and the thread's best chunk.
constexpr int kFlight = 2;
// labels: its read() asks for a row's labels once the first chunks are on their
// way, gather() for the logits that they name after the first of them were used,
// finish() puts all in place and gives the thread's u.
template <typename T, int THREADS, bool ENTROPY, bool OWN, bool TOP, Hold HOLD, typename L>
__device__ __forceinline__ Sums part_sums(const T* z, const Part& sp, float scale, BlockSums& sm,
                                          T* maxima, uint64_t* best, float* u, unsigned int* err,
                                          L& labels) {
  const int tid = threadIdx.x;
  const T* body = z + sp.lo + sp.head;
  Stats<ENTROPY, OWN> st;
  uint32_t now[kFlight][kWords], next[kFlight][kWords];
  auto load = [&](uint32_t(*w)[kWords], int q0) {
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int q = q0 + f * THREADS + tid;
      const int64_t at = (int64_t)q * kPer<T>;
      if (q < sp.body && within(sp.lo + sp.head + at, sp.lo + sp.head + at + kPer<T>, sp.lo,
                                sp.hi, err))
        load_chunk<HOLD>(w[f], body + at);
    }
  };
  load(now, 0);
  labels.read();
  if (tid < sp.head) st.add_one(value_of(z[tid]), scale);
  if (tid < sp.tail) st.add_one(value_of(z[sp.hi - sp.tail + tid]), scale);
  if (TOP && tid < 32) {
    float h = tid < sp.head ? value_of(z[tid]) : -INFINITY;
    float t = tid < sp.tail ? value_of(z[sp.hi - sp.tail + tid]) : -INFINITY;
    for (int off = 16; off > 0; off >>= 1) {
      h = max_nan(h, __shfl_xor_sync(0xFFFFFFFFu, h, off));
      t = max_nan(t, __shfl_xor_sync(0xFFFFFFFFu, t, off));
    }
    if (tid == 0) {
      store(maxima + sp.body, t);
      store(maxima + sp.body + 1, h);
    }
  }
  auto use = [&](uint32_t(*w)[kWords], int q0) {
    float most[kFlight], all = -INFINITY;
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      most[f] = q0 + f * THREADS + tid < sp.body ? max_of(w[f], T()) : -INFINITY;
      all = fmaxf(all, most[f]);
    }
    all = warp_max(all);  // (every thread of the block is here: q0 is the block's)
    if (all > st.m) st.move_to(all, scale);
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int q = q0 + f * THREADS + tid;
      if (q >= sp.body) continue;
      st.template add_chunk<T>(w[f], scale);
      if (TOP) {
        store(maxima + q, most[f]);
        *best = max(*best, rank_key<T>(most[f], sp.chunk0 + q + 1));
      }
    }
  };
  constexpr int kStep = kFlight * THREADS;
  for (int q0 = 0; q0 < sp.body; q0 += 2 * kStep) {
    load(next, q0 + kStep);
    use(now, q0);
    if (q0 == 0) labels.gather();
    if (q0 + kStep >= sp.body) break;
    load(now, q0 + 2 * kStep);
    use(next, q0 + kStep);
  }
  if (sp.body == 0) labels.gather();
  *u = labels.finish();
  return block_sums<THREADS, ENTROPY, OWN>(
      {st.m, st.s.x + st.s.y, st.u.x + st.u.y, st.s1.x + st.s1.y}, scale, u, sm);
}

// ---- the blocks of a row ----------------------------------------------------------
// A row split over a cluster: each block's sums and best keys, read by the
// others through the cluster's shared memory.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* p, int rank) {
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(at)
      : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return at;
}
__device__ __forceinline__ Sums remote_sums(const Sums* p, int rank) {
  Sums x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.m), "=f"(x.s), "=f"(x.u), "=f"(x.s1)
               : "r"(remote(p, rank))
               : "memory");
  return x;
}
__device__ __forceinline__ uint64_t remote_key(const uint64_t* p, int rank) {
  uint64_t x;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(remote(p, rank)) : "memory");
  return x;
}

// The row's sums from its blocks': lane i of every warp reads block i's.
template <bool ENTROPY, bool OWN>
__device__ __forceinline__ Sums cluster_sums(const Sums* mine, int split, float scale) {
  return lane_sums<ENTROPY, OWN>(remote_sums(mine, threadIdx.x & (split - 1)), split, scale);
}

// The row's top k from its blocks' sorted lists, into sh.best of this block: a
// key's rank is its place in its own list plus, for each other list, the number
// of keys there above it (a binary search in each, all at once).
template <int THREADS>
__device__ __forceinline__ void cluster_top(TopShared& sh, int k, int split) {
  const int tid = threadIdx.x;
  const int lane = tid & 31;
  for (int own = tid >> 5; own < split; own += THREADS / 32)  // a warp for each block's list
    for (int i = lane; i < k; i += 32) sh.list[own * k + i] = remote_key(sh.best + i, own);
  __syncthreads();
  for (int own = tid >> 5; own < split; own += THREADS / 32) {
    for (int i = lane; i < k; i += 32) {
      const uint64_t key = sh.list[own * k + i];
      int above[kMaxSplit] = {};
      for (int step = 128; step > 0; step /= 2) {
#pragma unroll
        for (int l = 0; l < kMaxSplit; ++l) {
          const int at = above[l] + step;
          if (l < split && at <= k && sh.list[l * k + at - 1] > key) above[l] = at;
        }
      }
      int rank = 0;  // (its own list's part is its place there)
#pragma unroll
      for (int l = 0; l < kMaxSplit; ++l) rank += above[l];
      if (key != 0 && rank < k) sh.best[rank] = key;
    }
  }
  __syncthreads();
}

// ---- the gradient's smooth part -------------------------------------------------
// g_j = 2^d (A + B d) + 2^d1 A1 with d = (z_j - M) scale, d1 = (z_j - M1) log2(e):
// the row's constants. zero: the whole row's gradient is 0.
struct GradRow {
  float A, B, A1, M, M1, scale;
  bool zero;
};
template <bool ENTROPY, bool OWN>
__device__ __forceinline__ float2 smooth(const GradRow& r, float2 z) {
  const float2 d = __fmul2_rn(__fadd2_rn(z, {-r.M, -r.M}), {r.scale, r.scale});
  const float2 e = {exp2_fast(d.x), exp2_fast(d.y)};
  float2 c = {r.A, r.A};
  if (ENTROPY) c = __ffma2_rn({r.B, r.B}, {clamped(d.x), clamped(d.y)}, c);
  float2 g = __fmul2_rn(e, c);
  if (OWN) {
    const float2 d1 = __fmul2_rn(__fadd2_rn(z, {-r.M1, -r.M1}), {kLog2e, kLog2e});
    g = __ffma2_rn({exp2_fast(d1.x), exp2_fast(d1.y)}, {r.A1, r.A1}, g);
  }
  return g;
}
__device__ __forceinline__ void put_pair(uint32_t* w, int i, float2 g, __nv_bfloat16) {
  const __nv_bfloat162 b = __float22bfloat162_rn(g);
  w[i] = *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void put_pair(uint32_t* w, int i, float2 g, float) {
  w[2 * i] = __float_as_uint(g.x);
  w[2 * i + 1] = __float_as_uint(g.y);
}
// (a gradient is not read again soon)
__device__ __forceinline__ void store_chunk(void* p, const uint32_t* w) {
  asm volatile("st.global.L2::evict_first.v8.u32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
               "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]),
               "r"(w[7])
               : "memory");
}

// The chunks of a part that start at the q0-th, kFlight of them a thread.
template <typename T, int THREADS>
__device__ __forceinline__ void load_ahead(uint32_t (&w)[kFlight][kWords], const T* z,
                                           const Part& sp, int q0, unsigned int* err) {
#pragma unroll
  for (int f = 0; f < kFlight; ++f) {
    const int q = q0 + f * THREADS + threadIdx.x;
    const int64_t at = sp.lo + sp.head + (int64_t)q * kPer<T>;
    if (q < sp.body && within(at, at + kPer<T>, sp.lo, sp.hi, err)) load_chunk<kOnce>(w[f], z + at);
  }
}
// Writes the smooth part of the gradient of a block's part of a row, whose first
// chunks load_ahead has asked for. Each
// element is read and written by one thread, so g may be z. Rows of z and g
// that sit differently in their 32-byte chunks (other strides or bases) go
// element by element.
template <typename T, int THREADS, bool ENTROPY, bool OWN>
__device__ __forceinline__ void write_part(uint32_t (&now)[kFlight][kWords], const T* z, T* g,
                                           const Part& sp, const GradRow& r, unsigned int* err) {
  const int tid = threadIdx.x;
  if (((uintptr_t)z ^ (uintptr_t)g) % kChunkBytes != 0) {
#pragma unroll 4
    for (int j = sp.lo + tid; j < sp.hi; j += THREADS)
      store(g + j, r.zero ? 0.0f : smooth<ENTROPY, OWN>(r, {value_of(z[j]), 0.0f}).x);
    return;
  }
  auto one = [&](int j) {
    store(g + j, r.zero ? 0.0f : smooth<ENTROPY, OWN>(r, {value_of(z[j]), 0.0f}).x);
  };
  if (tid < sp.head) one(tid);
  if (tid < sp.tail) one(sp.hi - sp.tail + tid);
  T* gb = g + sp.lo + sp.head;
  auto in_row = [&](int q) {
    const int64_t at = sp.lo + sp.head + (int64_t)q * kPer<T>;
    return q < sp.body && within(at, at + kPer<T>, sp.lo, sp.hi, err);
  };
  uint32_t next[kFlight][kWords];
  if (r.zero) {  // what load_ahead brought is not used: the row may hold anything
#pragma unroll
    for (int i = 0; i < kWords; ++i) next[0][i] = 0;
    for (int q = tid; q < sp.body; q += THREADS)
      if (in_row(q)) store_chunk(gb + (int64_t)q * kPer<T>, next[0]);
    return;
  }
  auto put = [&](uint32_t(*w)[kWords], int q0) {
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int q = q0 + f * THREADS + tid;
      if (!in_row(q)) continue;
#pragma unroll
      for (int i = 0; i < kPer<T> / 2; ++i)
        put_pair(w[f], i, smooth<ENTROPY, OWN>(r, pair_of(w[f], i, T())), T());
      store_chunk(gb + (int64_t)q * kPer<T>, w[f]);
    }
  };
  constexpr int kStep = kFlight * THREADS;
  for (int q0 = 0; q0 < sp.body; q0 += 2 * kStep) {
    load_ahead<T, THREADS>(next, z, sp, q0 + kStep, err);
    put(now, q0);
    if (q0 + kStep >= sp.body) break;
    load_ahead<T, THREADS>(now, z, sp, q0 + 2 * kStep, err);
    put(next, q0 + kStep);
  }
}

// The block's sums of x and y; every thread gets them.
template <int THREADS>
__device__ __forceinline__ float2 block_add(float x, float y, float2* sm) {
  for (int off = 16; off > 0; off >>= 1) {
    x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
    y += __shfl_xor_sync(0xFFFFFFFFu, y, off);
  }
  if (THREADS == 32) return {x, y};
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = {x, y};
  __syncthreads();
  float2 all = {0.0f, 0.0f};
  for (int w = 0; w < THREADS / 32; ++w) {
    all.x += sm[w].x;
    all.y += sm[w].y;
  }
  return all;
}

// A teacher's logit as it is stored, and its value.
__device__ __forceinline__ uint32_t teacher_bits(const RowArgs& a, int64_t i) {
  return a.teacher_bf16 ? static_cast<const uint16_t*>(a.teacher_logits)[i]
                        : static_cast<const uint32_t*>(a.teacher_logits)[i];
}
__device__ __forceinline__ float teacher_logit(const RowArgs& a, uint32_t bits) {
  return __uint_as_float(a.teacher_bf16 ? bits << 16 : bits);
}

// A row's labels: the target (-1: none), the teacher's record with the logits
// of its columns, the upstream gradients and normalisers. The loads of thread
// k's entry are issued, and waited for, in three steps between which the block
// does other work; a record longer than the block is read in the last one.
struct LabelsShared {
  int32_t id[ZS_MAX_TEACHER + 4];  // the teacher's ids, the target, -1 up to a multiple of 4
  float q[ZS_MAX_TEACHER + 4];     // u = t / T (-inf: unused), then x_k = exp(u - u_max); 0
  float z[ZS_MAX_TEACHER + 1];
};
template <typename T, int THREADS, bool LOSS, bool GRAD>
struct Labels {
  const RowArgs& a;
  const T* z;
  const int64_t r;
  const Part& part;
  const bool first, teacher;
  LabelsShared& sh;
  int32_t my_id = -1, target = -1;
  int64_t raw_target = -1;
  uint32_t my_t = 0;
  T my_z = T(0.0f), z_target = T(0.0f);  // (as stored: a conversion would wait for them)
  float w = 0.0f, al = 0.0f, b = 0.0f;  // d_loss, d_logprob, d_entropy
  float teacher_lse = 0.0f, lse = 0.0f, hard_lse = 0.0f, entropy = 0.0f;
  bool bad_target = false;

  // Whether this block needs the logit of a column: for the losses, or because
  // it writes that column's gradient. (Another block's columns may have been
  // overwritten in place when the gradient is computed alone.)
  __device__ __forceinline__ bool wanted(int32_t id) const {
    return id >= 0 && ((LOSS && first) || (id >= part.lo && id < part.hi));
  }
  __device__ __forceinline__ int32_t checked(int32_t id) const {
    if (id < a.vocab) return id;
    if (first) atomicOr(a.err, 4u);
    return -1;
  }
  __device__ __forceinline__ void put(int k, int32_t id, uint32_t t, float zk, float* u) {
    sh.id[k] = id;
    sh.q[k] = id >= 0 ? teacher_logit(a, t) * a.inv_t : -INFINITY;
    sh.z[k] = zk;
    *u = fmaxf(*u, sh.q[k]);
  }
  __device__ __forceinline__ void read() {
    const int k = threadIdx.x;
    if (teacher && k < a.teacher_k) {
      my_id = a.teacher_ids[r * a.teacher_k + k];
      my_t = teacher_bits(a, r * a.teacher_k + k);
    }
    if (a.targets) raw_target = a.targets[r];
    if (teacher && a.teacher_lse) teacher_lse = a.teacher_lse[r];
    if (GRAD) {
      if (a.d_loss) w = a.d_loss[r];
      if (a.d_logprob) al = a.d_logprob[r];
      if (!LOSS) {
        if (a.d_entropy) b = a.d_entropy[r];
        if (a.in_lse) lse = a.in_lse[r];
        if (a.in_hard_lse) hard_lse = a.in_hard_lse[r];
        if (a.in_entropy) entropy = a.in_entropy[r];
      }
    }
  }
  __device__ __forceinline__ void gather() {
    my_id = checked(my_id);
    if (wanted(my_id)) my_z = z[my_id];
    bad_target = raw_target >= a.vocab;
    if (bad_target && first && threadIdx.x == 0) atomicOr(a.err, 4u);
    if (raw_target >= 0 && !bad_target) target = (int32_t)raw_target;
    if (wanted(target)) z_target = z[target];
    if (target < 0) al = 0.0f;
  }
  __device__ __forceinline__ float finish() {
    const int K = a.teacher_k, tid = threadIdx.x;
    float u = -INFINITY;
    if (teacher) {
      if (tid < K) put(tid, my_id, my_t, value_of(my_z), &u);
      for (int k = tid + THREADS; k < K; k += THREADS) {
        const int32_t id = checked(a.teacher_ids[r * K + k]);
        put(k, id, teacher_bits(a, r * K + k), wanted(id) ? value_of(z[id]) : 0.0f, &u);
      }
    }
    if (GRAD && tid < 4) {
      sh.id[K + tid] = tid == 0 ? target : -1;
      sh.q[K + tid] = 0.0f;
      if (tid == 0) sh.z[K] = value_of(z_target);
    }
    return u;
  }
};

// A row per block, or per cluster of 2^shift blocks (LOSS) or as many independent
// ones (the gradient alone). LOSS: statistics and losses from the logits; GRAD:
// the gradient, from them or from the forward call's normalisers. The row is
// streamed by all threads; what else it takes is kept off that stream: labels
// are asked for behind its first loads, the blocks of an SM are at different
// points of their rows, the next kernel's are placed as the last rows retire.
// Of the 14.5 thousand cycles (7.6 us) of a 32000-logit bf16 row in a block of 256
// threads the stream was 10; a block of 128 spends the same on the rest of a row
// that it streams twice as long, with twice as many beside it (98 -> 86 us for
// 8192 rows).
template <typename T, int THREADS, bool LOSS, bool GRAD, bool ENTROPY, bool OWN, bool TOP>
__global__ void __launch_bounds__(THREADS, kResident / THREADS)
    rows_kernel(const __grid_constant__ RowArgs a) {
  overlap_wait();
  const int split = 1 << a.shift, rank = (int)(blockIdx.x & (unsigned)(split - 1));
  const int64_t r = blockIdx.x >> a.shift;
  const int V = a.vocab, K = a.teacher_k, tid = threadIdx.x;
  const T* z = static_cast<const T*>(a.logits) + r * a.row_stride;
  const Part part = part_of(z, V, rank, a.shift);
  // The first block of a row writes its statistics and losses.
  const bool first = rank == 0, teacher = K > 0 && (GRAD || first);
  __shared__ __align__(16) BlockSums sm_sums;
  __shared__ __align__(16) Sums sm_part;
  __shared__ float2 sm_add[THREADS / 32];
  __shared__ __align__(16) LabelsShared sl;
  Labels<T, THREADS, LOSS, GRAD> labels = {a, z, r, part, first, teacher, sl};
  float u_max = -INFINITY;
  // GRAD: the first chunks; for the gradient alone they are on their way while
  // the row's constants are made. (After the sums that early a load costs more in
  // registers than it hides: 4095 x 32000 94.5 against 95.1 us.)
  uint32_t ahead[kFlight][kWords];

  float M = 0.0f, S = 1.0f, S1 = 1.0f, lse = 0.0f, lse1 = 0.0f, ln_s = 0.0f;
  bool empty = false;
  if (LOSS) {
    extern __shared__ __align__(16) unsigned char dynamic[];
    TopShared* top = reinterpret_cast<TopShared*>(dynamic);
    T* maxima = nullptr;
    if (TOP) {
      const int capacity = list_capacity(a.top_k);
      uint64_t* list = reinterpret_cast<uint64_t*>(top + 1);
      maxima = reinterpret_cast<T*>(list + capacity);
      if (tid == 0) {
        top->capacity = capacity;
        top->list = list;
      }
    }
    uint64_t best = 0;
    Sums t = part_sums<T, THREADS, ENTROPY, OWN, TOP, GRAD ? kUntilRead : kUsual>(
        z, part, a.scale, sm_sums, maxima, &best, &u_max, a.err, labels);
    // (block_sums waited for the table)
    if (TOP) select_top<T, THREADS>(z, {part, maxima}, a.top_k, best, *top, a.err);
    if (split > 1) {
      if (tid == 0) sm_part = t;
      cluster_arrive();
      cluster_wait();
      if (GRAD || first) t = cluster_sums<ENTROPY, OWN>(&sm_part, split, a.scale);
      if (TOP && first) cluster_top<THREADS>(*top, a.top_k, split);
      cluster_arrive();  // this block has read the others' shared memory
    }
    const float m = t.m, U = t.u;
    M = m == -INFINITY ? 0.0f : m;  // a row masked throughout: every e is 2^-inf = 0
    S = t.s;
    S1 = OWN ? t.s1 : S;
    empty = m == -INFINITY && S == 0.0f;
    ln_s = logf(S);
    const float ln_s1 = OWN ? logf(S1) : ln_s;
    lse = empty ? -INFINITY : fmaf(M, a.inv_t, ln_s);
    lse1 = empty ? -INFINITY : M + ln_s1;
    if (first && tid == 0) {
      if (a.lse) a.lse[r] = lse;
      if (a.hard_lse) a.hard_lse[r] = lse1;
      if (a.entropy) a.entropy[r] = empty ? 0.0f : ln_s - kLn2 * (U / S);
      if (a.logprob) {
        const float t = a.distill ? 1.0f : a.inv_t;
        a.logprob[r] = labels.bad_target   ? NAN
                       : labels.target < 0 ? 0.0f
                       : empty             ? -INFINITY
                                           : (value_of(labels.z_target) - M) * t - (a.distill ? ln_s1 : ln_s);
      }
    }
    if (TOP && first) {
      for (int k = tid; k < a.top_k; k += THREADS) {
        const uint64_t key = top->best[k];
        a.top_ids[r * a.top_k + k] = (int32_t)~(uint32_t)key;
        a.top_logprobs[r * a.top_k + k] =
            empty ? -INFINITY : (key_value<T>(key) - M) * a.inv_t - ln_s;
      }
    }
  } else {
    labels.read();
    load_ahead<T, THREADS>(ahead, z, part, 0, a.err);
    labels.gather();
    u_max = labels.finish();
    block_sums<THREADS, false, false>({0.0f, 0.0f, 0.0f, 0.0f}, 0.0f, &u_max, sm_sums);
  }

  // The teacher's q_k = x_k / X with x_k = exp(u_k - u_max), X their sum (or
  // x_k = exp(u_k - teacher_lse), X = 1); Q = sum q. The loss in one more sum,
  //   sum_k q_k (ln q_k - ln p_k) = (1/X) sum_k x_k (ln x_k - ln p_k) - Q ln X.
  float Q = 0.0f, per_x = 1.0f;
  if (teacher) {
    const float u0 = a.teacher_lse ? labels.teacher_lse : u_max == -INFINITY ? 0.0f : u_max;
    float x_sum = 0.0f, l_sum = 0.0f;
    for (int k = tid; k < K; k += THREADS) {
      // (an entry without mass has none whatever u0: a teacher's row masked
      // throughout has lse -infinity)
      const float ln_x = sl.q[k] - u0, x = sl.q[k] == -INFINITY ? 0.0f : expf(ln_x);
      sl.q[k] = x;
      x_sum += x;
      if (LOSS && !(x == 0.0f))
        l_sum += x * (ln_x - (empty ? -INFINITY : (sl.z[k] - M) * a.inv_t - ln_s));
    }
    const float2 t = block_add<THREADS>(x_sum, l_sum, sm_add);
    Q = t.x;
    float loss = t.y;
    if (!a.teacher_lse && !(Q == 0.0f)) {
      per_x = 1.0f / Q;
      loss = loss * per_x - logf(Q);
      Q = Q * per_x;
    }
    if (LOSS && first && tid == 0 && a.loss) a.loss[r] = loss;
  }

  if (GRAD) {
    T* g = static_cast<T*>(a.d_logits) + r * a.grad_stride;
    const float al = labels.al, w = labels.w, b = labels.b;
    float A = 0.0f, B = 0.0f, A1 = 0.0f, M1 = M, at_target = 0.0f;
    bool zero;
    if (LOSS) {
      zero = empty;  // (lse may be -infinity without: the lowest value over T < 1)
      A = w * a.inv_t * Q / S;
      if (OWN)
        A1 = -al / S1;
      else
        A -= al / S;
      at_target = al;
    } else if (a.distill) {
      if (a.in_hard_lse) lse = lse1 = labels.hard_lse;
      if (a.in_lse) lse = labels.lse;
      zero = lse == -INFINITY;
      M = lse / a.inv_t;
      M1 = lse1;
      A = w * a.inv_t * Q;
      if (OWN)
        A1 = -al;
      else
        A -= al;
      at_target = al;
    } else {
      lse = labels.lse;
      zero = lse == -INFINITY;
      M = lse / a.inv_t;
      A = -(al + (b == 0.0f ? 0.0f : b * labels.entropy)) * a.inv_t;
      B = -b * kLn2 * a.inv_t;
      at_target = al * a.inv_t;
    }
    zero = zero || (al == 0.0f && w == 0.0f && b == 0.0f);
    // A softmax without weight must not meet its normaliser (it may belong to
    // another temperature): infinity turns its exponentials into 0.
    if (A == 0.0f && B == 0.0f) M = INFINITY;
    if (A1 == 0.0f) M1 = INFINITY;
    const GradRow row = {A, B, A1, M, M1, a.scale, zero};
    __syncthreads();  // the labels, before anything is overwritten in place
    if (LOSS) load_ahead<T, THREADS>(ahead, z, part, 0, a.err);
    write_part<T, THREADS, ENTROPY, OWN>(ahead, z, g, part, row, a.err);
    __syncthreads();
    // The columns of the target and the teacher's ids, from the logits kept
    // above (z may be overwritten by now). Equal ids all store the same value.
    for (int k = tid; k <= K; k += THREADS) {
      const int32_t id = sl.id[k];
      if (id < part.lo || id >= part.hi || zero) continue;
      float q = 0.0f;
#pragma unroll 4
      for (int i = 0; i < K; i += 4) {
        const int4 ids = *reinterpret_cast<const int4*>(sl.id + i);
        const float4 x = *reinterpret_cast<const float4*>(sl.q + i);
        q += ids.x == id ? x.x : 0.0f;
        q += ids.y == id ? x.y : 0.0f;
        q += ids.z == id ? x.z : 0.0f;
        q += ids.w == id ? x.w : 0.0f;
      }
      float x = smooth<ENTROPY, OWN>(row, {sl.z[k], 0.0f}).x - w * a.inv_t * (q * per_x);
      if (id == labels.target) x += at_target;
      store(g + id, x);
    }
  }
  if (LOSS && split > 1) cluster_wait();  // the others have read this block's shared memory
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

// The threads of a row's block. A block's fixed work (labels, joining its
// threads' sums, the hand-over to the next block: some 3 us) is hidden by the
// other blocks of its SM, so many rows want small blocks, as long as a thread's
// share of the row does not outgrow what the SM keeps in flight. By the row's
// bytes, from sweeps of 32..256 threads over 1000..64000 logits of both types
// (about 16000 rows, us with 32 / 64 / 128 / 256 threads, bf16):
//   sums alone      8 KB 25.5 / 29.5 / 41 / 71, 64 KB 84 / 82 / 80 / 87,
//                   300 KB (4096 rows) - / - / 189 / 180
//   alternatives    4 KB 128 / 90 / 95 / 175, 64 KB 264 / 172 / 139 / 171,
//                   128 KB - / - / 123 / 130
//   gradient alone  4 KB 21 / 25 / 39 / 75, 16 KB 81 / 78 / 82 / 100, 64 KB 158 / 154 / 150 / 148
//   both in one     8 KB 55 / 56 / 77 / 133, 16 KB 105 / 91 / 101 / 152,
//                   32 KB 230 / 186 / 170 / 199, 64 KB 235 / 224 / 184 / 174
// Few rows want larger ones, until the SMs are full. The search for the
// alternatives starts from the threads' best chunks: three for each alternative.
template <typename T, bool LOSS, bool GRAD, bool TOP>
int threads_of(const VocabLaunch& in) {
  const int64_t bytes = in.vocab * (int64_t)sizeof(T), chunks = in.vocab / kPer<T>;
  const int64_t kb = 1024;
  int threads;
  if (TOP)
    threads = bytes <= 8 * kb ? 64 : bytes <= 80 * kb ? 128 : 256;
  else if (!GRAD)
    threads = bytes <= 20 * kb ? 32 : bytes <= 48 * kb ? 64 : bytes <= 256 * kb ? 128 : 256;
  else
    threads = bytes <= 10 * kb ? 32 : bytes <= 20 * kb ? 64 : bytes <= 48 * kb ? 128 : 256;
  while (threads < kMaxThreads &&
         ((in.rows * threads < kSMs * kResident && chunks >= 2 * threads) ||
          (TOP && threads < 3 * in.top_k)))
    threads *= 2;
  return threads;
}

// How many blocks share a row (1, 2, 4 or 8; a cluster when they must meet).
//  - Few rows: until every SM has a block (the gradient alone, whose blocks need
//    not meet: 16), as long as every thread has a chunk.
//  - Loss and gradient in one call: the rows in flight are read twice, so they
//    are to stay in L2. With one, two and four blocks, us, the rule's in brackets:
//      bf16  4062 x 64000 [180.5] 182.5 -, 2031 x 128000 218 [184.8] 188.6,
//            1711 x 151936 225 [195.5] 188.6, 8192 x 151936 1065 [954] 983
//      fp32  4062 x 64000 431 [361.8] 361, 2031 x 128000 430 [363.4] 373,
//            1711 x 151936 440 [387] 379.5
//    (a few rounds of the largest rows want four, many want two: by bytes alone the
//    rule is up to 4 % from the better one there).
//  - Top alternatives: the table of a block's part stays under a quarter of an
//    SM's shared memory.
template <typename T, bool LOSS, bool GRAD, bool TOP>
int split_of(const VocabLaunch& in, int threads) {
  const int64_t chunks = in.vocab / kPer<T>, blocks = kSMs * (kResident / threads);
  const int64_t fill = LOSS ? kSMs : 16 * kSMs;
  int split = 1;
  while (split < kMaxSplit && in.rows * split < fill && chunks >= 2 * split * threads) split *= 2;
  if (LOSS && GRAD)
    while (split < kMaxSplit && blocks / split * in.vocab * (int64_t)sizeof(T) > kRowsInL2)
      split *= 2;
  if (TOP)
    while (split < kMaxSplit && chunks / split * (int64_t)sizeof(T) > kTableBytes) split *= 2;
  return split;
}

// launch_kernel's launch, in clusters of `cluster` blocks (1: no clusters).
cudaError_t launch_clusters(int cluster, void (*kernel)(RowArgs), dim3 grid, dim3 block,
                            size_t smem, cudaStream_t stream, const RowArgs& a) {
  if (cluster == 1) return launch_kernel(kernel, grid, block, smem, stream, a);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = launch_overlap() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T, int THREADS, bool LOSS, bool GRAD, bool ENTROPY, bool OWN, bool TOP>
cudaError_t launch_rows(const VocabLaunch& in, int split, cudaStream_t stream) {
  RowArgs a = row_args(in);
  if (!a.err) return cudaErrorInvalidSymbol;
  a.shift = split == 8 ? 3 : split / 2;
  const auto kernel = rows_kernel<T, THREADS, LOSS, GRAD, ENTROPY, OWN, TOP>;
  size_t smem = 0;
  if (TOP) {
    // The table: an entry for each 32 bytes of the part, and two ends.
    smem = sizeof(TopShared) + list_capacity(in.top_k) * 8 +
           (in.vocab / kPer<T> / split + 4) * sizeof(T);
    static std::atomic<bool> allowed[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!allowed[dev & 63].load(std::memory_order_acquire)) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
      if (e != cudaSuccess) return e;
      allowed[dev & 63].store(true, std::memory_order_release);
    }
  }
  return launch_clusters(LOSS ? split : 1, kernel, dim3((unsigned)(in.rows * split)),
                         dim3(THREADS), smem, stream, a);
}

template <typename T, bool LOSS, bool GRAD, bool ENTROPY, bool OWN, bool TOP>
cudaError_t launch_typed(const VocabLaunch& in, cudaStream_t stream) {
  const int threads = threads_of<T, LOSS, GRAD, TOP>(in);
  const int split = split_of<T, LOSS, GRAD, TOP>(in, threads);
  if (threads == 256)
    return launch_rows<T, 256, LOSS, GRAD, ENTROPY, OWN, TOP>(in, split, stream);
  if (threads == 128)
    return launch_rows<T, 128, LOSS, GRAD, ENTROPY, OWN, TOP>(in, split, stream);
  if (TOP || threads == 64)
    return launch_rows<T, 64, LOSS, GRAD, ENTROPY, OWN, TOP>(in, split, stream);
  return launch_rows<T, TOP ? 64 : 32, LOSS, GRAD, ENTROPY, OWN, TOP>(in, split, stream);
}

template <bool LOSS, bool GRAD, bool ENTROPY, bool OWN, bool TOP>
cudaError_t launch(const VocabLaunch& in, cudaStream_t stream) {
  return in.dtype == ZS_BF16
             ? launch_typed<__nv_bfloat16, LOSS, GRAD, ENTROPY, OWN, TOP>(in, stream)
             : launch_typed<float, LOSS, GRAD, ENTROPY, OWN, TOP>(in, stream);
}

// The hard labels need a softmax of their own: T is not 1, and one of their
// values is wanted.
bool own_softmax(const VocabLaunch& a) {
  return a.distill && a.temperature != 1.0 && (a.logprob || a.hard_lse || a.d_logprob);
}

}  // namespace

cudaError_t launch_vocab_loss(const VocabLaunch& a, cudaStream_t stream) {
  if (a.d_logits)
    return own_softmax(a) ? launch<true, true, false, true, false>(a, stream)
                          : launch<true, true, false, false, false>(a, stream);
  if (a.top_k) return launch<true, false, true, false, true>(a, stream);
  if (a.entropy) return launch<true, false, true, false, false>(a, stream);
  return own_softmax(a) ? launch<true, false, false, true, false>(a, stream)
                        : launch<true, false, false, false, false>(a, stream);
}

cudaError_t launch_vocab_grad(const VocabLaunch& a, cudaStream_t stream) {
  if (a.d_entropy) return launch<false, true, true, false, false>(a, stream);
  return own_softmax(a) ? launch<false, true, false, true, false>(a, stream)
                        : launch<false, true, false, false, false>(a, stream);
}

}  // namespace zs
