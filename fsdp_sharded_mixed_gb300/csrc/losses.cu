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

#include <atomic>

#include "bounds.cuh"
#include "overlap.cuh"
#include "zs_internal.h"

namespace zs {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 256;
constexpr int kMaxSmem = 200 * 1024;  // dynamic shared memory of a block

struct RowArgs {
  const void* logits;
  void* d_logits;
  int64_t row_stride, grad_stride;
  int32_t vocab, top_k, teacher_k;
  bool teacher_bf16;
  bool distill;   // targets are hard labels at T = 1
  float inv_t, scale, slack;  // 1/T, log2(e)/T, how far logits may exceed a reference
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

struct Span {
  int head, body, tail;  // elements, chunks, elements
};
template <typename T>
__device__ __forceinline__ Span span_of(const T* z, int V) {
  const int head = min(V, (int)((0 - (uintptr_t)z) % kChunkBytes / sizeof(T)));
  const int body = (V - head) / kPer<T>;
  return {head, body, V - head - body * kPer<T>};
}

__device__ __forceinline__ void load_chunk(uint32_t* w, const void* p) {
  asm volatile("ld.global.L1::no_allocate.v8.u32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                 "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
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

// 2^x to 2 units in the last place; results below the normal range become 0.
__device__ __forceinline__ float exp2_fast(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
  return e;
}
// A log2 weight that is 2^-10000 = 0 rather than 2^-inf: 0 * -inf is not 0.
__device__ __forceinline__ float clamped(float d) { return fmaxf(d, -1e4f); }

// ---- one pass over the row ------------------------------------------------------
// S and U (and S1, the sum at T = 1) relative to a reference logit m that
// follows the maximum: it moves only when a chunk exceeds it by more than 8
// powers of two, so that the sums are rescaled a few times a row and no e
// exceeds 2^8. m = -inf until a finite logit was seen (ref is 0 meanwhile).
template <bool ENTROPY, bool OWN>
struct Stats {
  float m = -INFINITY, ref = 0.0f, limit = -INFINITY;
  float2 s = {0.0f, 0.0f}, u = {0.0f, 0.0f}, s1 = {0.0f, 0.0f};

  __device__ __forceinline__ void move_to(float to, float scale, float slack) {
    const float delta = limit == -INFINITY ? -1e4f : clamped((ref - to) * scale);
    const float f = exp2_fast(delta);
    if (ENTROPY) {
      u.x = f * fmaf(s.x, delta, u.x);
      u.y = f * fmaf(s.y, delta, u.y);
    }
    s.x *= f;
    s.y *= f;
    if (OWN) {
      const float f1 = limit == -INFINITY ? 0.0f : exp2_fast((ref - to) * kLog2e);
      s1.x *= f1;
      s1.y *= f1;
    }
    m = ref = to;
    limit = to + slack;
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
  __device__ __forceinline__ float add_chunk(const uint32_t* w, float scale, float slack) {
    const float cm = max_of(w, T());
    if (cm > limit) move_to(cm, scale, slack);
#pragma unroll
    for (int i = 0; i < kPer<T> / 2; ++i) add(pair_of(w, i, T()), scale);
    return cm;
  }
  __device__ __forceinline__ void add_one(float z, float scale, float slack) {
    if (z > limit) move_to(z, scale, slack);
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
__device__ __forceinline__ Sums moved(const Sums& a, float M, float scale) {
  const float delta = toward(a.m, M, scale), f = exp2_fast(delta);
  const float f1 = exp2_fast(toward(a.m, M, kLog2e));
  return {M, f * a.s, f * fmaf(a.s, delta, a.u), f1 * a.s1};
}

// The block's sums, in a fixed order; every thread gets them.
template <int THREADS>
__device__ __forceinline__ Sums block_sums(Sums t, float scale, Sums* sm) {
  float M = t.m;
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
  t = moved(t, M, scale);
  for (int off = 16; off > 0; off >>= 1) {
    t.s += __shfl_xor_sync(0xFFFFFFFFu, t.s, off);
    t.u += __shfl_xor_sync(0xFFFFFFFFu, t.u, off);
    t.s1 += __shfl_xor_sync(0xFFFFFFFFu, t.s1, off);
  }
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = t;
  __syncthreads();
  M = sm[0].m;
  for (int w = 1; w < THREADS / 32; ++w) M = fmaxf(M, sm[w].m);
  Sums all = {M, 0.0f, 0.0f, 0.0f};
  for (int w = 0; w < THREADS / 32; ++w) {
    const Sums x = moved(sm[w], M, scale);
    all.s += x.s;
    all.u += x.u;
    all.s1 += x.s1;
  }
  return all;
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

// The pass over the row leaves every chunk's maximum in shared memory, and each
// thread knows the best of its own chunks. A chunk is ranked by its maximum,
// equal ones by position. If k chunks reach a bound, the row's top k elements
// do, each taken at its chunk's position: an element below the bound is beaten
// by the maxima of all k. So a bound that about k of the threads' best chunks
// reach leaves few chunks to read again and few elements to rank.
// Table entry p: body chunk p; then the tail and the head (whose position comes
// first). An end without elements has key 0. Entry p belongs to thread p modulo
// the block.
constexpr int kListed = 2048;  // elements that are ranked; 16 * ZS_MAX_TOP at least
struct TopShared {
  uint64_t list[kListed];
  uint64_t best[ZS_MAX_TOP];
  int count, total;
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
struct Chunks {  // the table of a row
  Span sp;
  int V;
  const T* maxima;
  __device__ __forceinline__ int count() const { return sp.body + 2; }
  __device__ __forceinline__ int position(int p) const { return p == sp.body + 1 ? 0 : p + 1; }
  __device__ __forceinline__ uint64_t key(int p) const {
    if ((p == sp.body && sp.tail == 0) || (p == sp.body + 1 && sp.head == 0)) return 0;
    return rank_key<T>(value_of(maxima[p]), position(p));
  }
  __device__ __forceinline__ void elements(int p, int* lo, int* hi) const {
    *lo = p == sp.body + 1 ? 0 : sp.head + p * kPer<T>;
    *hi = p == sp.body + 1 ? sp.head : min(V, *lo + kPer<T>);
  }
};

// Ranks the row's top k into sh.best (keys, best first; position = column).
// `mine`: the best key of the thread's body chunks.
template <typename T, int THREADS>
__device__ __forceinline__ void select_top(const T* z, const Chunks<T>& ch, int k, uint64_t mine,
                                           TopShared& sh, unsigned int* err) {
  const int tid = threadIdx.x;
  for (int p = ch.sp.body; p < ch.count(); ++p)
    if (p % THREADS == tid) mine = max(mine, ch.key(p));
  auto total_of = [&](int n) {
    __syncthreads();
    if (tid == 0) sh.total = 0;
    __syncthreads();
    if (n) atomicAdd(&sh.total, n);
    __syncthreads();
    return sh.total;
  };
  // Lists the elements at or above the bound, from the chunks that reach it.
  auto list_from = [&](uint64_t bound, bool look) {
    if (tid == 0) sh.count = 0;
    __syncthreads();
    for (int p = tid; look && p < ch.count(); p += THREADS) {
      if (ch.key(p) < bound || ch.key(p) == 0) continue;
      int lo, hi;
      ch.elements(p, &lo, &hi);
      for (int j = lo; j < hi; ++j) {
        if (!within(j, j + 1, 0, ch.V, err)) continue;
        const float x = value_of(z[j]);
        if (rank_key<T>(x, ch.position(p)) < bound) continue;
        const int at = atomicAdd(&sh.count, 1);
        if (at < kListed) sh.list[at] = rank_key<T>(x, j);
      }
    }
    __syncthreads();
    return sh.count;
  };
  uint64_t bound =
      bound_of<T>(k, 2 * k, [&](uint64_t b) { return __syncthreads_count(mine >= b); });
  int n = list_from(bound, mine >= bound);
  if (n > kListed) {
    // Very many in a few threads' chunks: the exact k-th best chunk leaves the
    // elements of k chunks at most.
    bound = bound_of<T>(k, k, [&](uint64_t b) {
      int reach = 0;
      for (int p = tid; p < ch.count(); p += THREADS) reach += ch.key(p) >= b;
      return total_of(reach);
    });
    n = list_from(bound, true);
  }
  bound = 0;
  if (n > kListed / 4)  // ranking is quadratic: first the exact k-th best
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
    for (int j = 0; j < n; ++j) rank += sh.list[j] > key;
    if (rank < k) sh.best[rank] = key;
  }
  __syncthreads();
}

// The sums of a row by one block: each thread keeps kFlight chunks in flight
// ahead of those that it works on. TOP: maxima and the thread's best chunk.
constexpr int kFlight = 2;
template <typename T, bool ENTROPY, bool OWN, bool TOP>
__device__ __forceinline__ Sums row_sums(const T* z, int V, float scale, float slack, Sums* sm,
                                         T* maxima, uint64_t* best, unsigned int* err) {
  const int tid = threadIdx.x;
  const Span sp = span_of(z, V);
  const T* body = z + sp.head;
  Stats<ENTROPY, OWN> st;
  uint32_t now[kFlight][kWords], next[kFlight][kWords];
  auto load = [&](uint32_t(*w)[kWords], int q0) {
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int q = q0 + f * kThreads + tid;
      if (q < sp.body && within(sp.head + (int64_t)q * kPer<T>,
                                sp.head + (int64_t)(q + 1) * kPer<T>, 0, V, err))
        load_chunk(w[f], body + (int64_t)q * kPer<T>);
    }
  };
  load(now, 0);
  if (tid < sp.head) st.add_one(value_of(z[tid]), scale, slack);
  if (tid < sp.tail) st.add_one(value_of(z[V - sp.tail + tid]), scale, slack);
  if (TOP && tid < 32) {
    float h = tid < sp.head ? value_of(z[tid]) : -INFINITY;
    float t = tid < sp.tail ? value_of(z[V - sp.tail + tid]) : -INFINITY;
    for (int off = 16; off > 0; off >>= 1) {
      h = max_nan(h, __shfl_xor_sync(0xFFFFFFFFu, h, off));
      t = max_nan(t, __shfl_xor_sync(0xFFFFFFFFu, t, off));
    }
    if (tid == 0) {
      store(maxima + sp.body, t);
      store(maxima + sp.body + 1, h);
    }
  }
  for (int q0 = 0; q0 < sp.body; q0 += kFlight * kThreads) {
    load(next, q0 + kFlight * kThreads);
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
      if (q0 + f * kThreads + tid < sp.body) {
        const float cm = st.template add_chunk<T>(now[f], scale, slack);
        if (TOP) {
          const int p = q0 + f * kThreads + tid;
          store(maxima + p, cm);
          *best = max(*best, rank_key<T>(cm, p + 1));
        }
      }
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
#pragma unroll
      for (int i = 0; i < kWords; ++i) now[f][i] = next[f][i];
  }
  return block_sums<kThreads>({st.m, st.s.x + st.s.y, st.u.x + st.u.y, st.s1.x + st.s1.y}, scale,
                              sm);
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
__device__ __forceinline__ void store_chunk(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.u32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Writes the smooth part of a row's gradient. Each element is read and written
// by one thread, so g may be z. Rows of z and g that sit differently in their
// 32-byte chunks (other strides or bases) go element by element.
template <typename T, bool ENTROPY, bool OWN>
__device__ __forceinline__ void write_row(const T* z, T* g, int V, const GradRow& r,
                                          unsigned int* err) {
  const int tid = threadIdx.x;
  if (((uintptr_t)z ^ (uintptr_t)g) % kChunkBytes != 0) {
#pragma unroll 4
    for (int j = tid; j < V; j += kThreads)
      store(g + j, r.zero ? 0.0f : smooth<ENTROPY, OWN>(r, {value_of(z[j]), 0.0f}).x);
    return;
  }
  const Span sp = span_of(z, V);
  auto one = [&](int j) {
    store(g + j, r.zero ? 0.0f : smooth<ENTROPY, OWN>(r, {value_of(z[j]), 0.0f}).x);
  };
  if (tid < sp.head) one(tid);
  if (tid < sp.tail) one(V - sp.tail + tid);
  const T* zb = z + sp.head;
  T* gb = g + sp.head;
  auto in_row = [&](int q) {
    return q < sp.body && within(sp.head + (int64_t)q * kPer<T>,
                                 sp.head + (int64_t)(q + 1) * kPer<T>, 0, V, err);
  };
  uint32_t now[kFlight][kWords], next[kFlight][kWords], out[kWords];
  if (r.zero) {  // not read at all: it may hold anything
#pragma unroll
    for (int i = 0; i < kWords; ++i) out[i] = 0;
    for (int q = tid; q < sp.body; q += kThreads)
      if (in_row(q)) store_chunk(gb + (int64_t)q * kPer<T>, out);
    return;
  }
  auto load = [&](uint32_t(*w)[kWords], int q0) {
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int q = q0 + f * kThreads + tid;
      if (in_row(q)) load_chunk(w[f], zb + (int64_t)q * kPer<T>);
    }
  };
  load(now, 0);
  for (int q0 = 0; q0 < sp.body; q0 += kFlight * kThreads) {
    load(next, q0 + kFlight * kThreads);
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int q = q0 + f * kThreads + tid;
      if (!in_row(q)) continue;
#pragma unroll
      for (int i = 0; i < kPer<T> / 2; ++i)
        put_pair(out, i, smooth<ENTROPY, OWN>(r, pair_of(now[f], i, T())), T());
      store_chunk(gb + (int64_t)q * kPer<T>, out);
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
#pragma unroll
      for (int i = 0; i < kWords; ++i) now[f][i] = next[f][i];
  }
}

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

__device__ __forceinline__ float teacher_logit(const RowArgs& a, int64_t i) {
  return a.teacher_bf16 ? value_of(static_cast<const __nv_bfloat16*>(a.teacher_logits)[i])
                        : static_cast<const float*>(a.teacher_logits)[i];
}

// One block per row. LOSS: statistics and losses from the logits; GRAD: the
// gradient, from them or from the forward call's normalisers.
template <typename T, bool LOSS, bool GRAD, bool ENTROPY, bool OWN, bool TOP>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ RowArgs a) {
  overlap_wait();
  const int64_t r = blockIdx.x;
  const int V = a.vocab, K = a.teacher_k, tid = threadIdx.x;
  const T* z = static_cast<const T*>(a.logits) + r * a.row_stride;
  __shared__ float sm[kThreads / 32];
  __shared__ Sums sm_sums[kThreads / 32];
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
    extern __shared__ __align__(16) unsigned char dynamic[];
    TopShared* top = reinterpret_cast<TopShared*>(dynamic);
    T* maxima = reinterpret_cast<T*>(top + 1);
    uint64_t best = 0;
    const Sums t = row_sums<T, ENTROPY, OWN, TOP>(z, V, a.scale, a.slack, sm_sums, maxima, &best,
                                                  a.err);
    const float m = t.m, U = t.u;
    M = m == -INFINITY ? 0.0f : m;  // a row masked throughout: every e is 2^-inf = 0
    S = t.s;
    S1 = OWN ? t.s1 : S;
    const bool empty = m == -INFINITY && S == 0.0f;
    const float ln_s = logf(S), ln_s1 = OWN ? logf(S1) : ln_s;
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
    if (TOP) {
      // block_sums waited for the table
      select_top<T, kThreads>(z, {span_of(z, V), V, maxima}, a.top_k, best, *top, a.err);
      for (int k = tid; k < a.top_k; k += kThreads) {
        const int32_t id = (int32_t)~(uint32_t)top->best[k];
        a.top_ids[r * a.top_k + k] = id;
        a.top_logprobs[r * a.top_k + k] =
            empty ? -INFINITY : (value_of(z[id]) - M) * a.inv_t - ln_s;
      }
    }
  }

  if (GRAD) {
    T* g = static_cast<T*>(a.d_logits) + r * a.grad_stride;
    const float al = a.d_logprob && target >= 0 ? a.d_logprob[r] : 0.0f;
    const float w = a.d_loss ? a.d_loss[r] : 0.0f, b = a.d_entropy ? a.d_entropy[r] : 0.0f;
    float A = 0.0f, B = 0.0f, A1 = 0.0f, M1 = M, at_target = 0.0f;
    bool zero;
    if (LOSS) {
      zero = lse == -INFINITY;
      A = w * a.inv_t * Q / S;
      if (OWN)
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
      if (OWN)
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
    // A softmax without weight must not meet its normaliser (it may belong to
    // another temperature): infinity turns its exponentials into 0.
    if (A == 0.0f && B == 0.0f) M = INFINITY;
    if (A1 == 0.0f) M1 = INFINITY;
    const GradRow row = {A, B, A1, M, M1, a.scale, zero};
    write_row<T, ENTROPY, OWN>(z, g, V, row, a.err);
    __syncthreads();
    // The columns of the target and the teacher's ids, from the logits kept
    // above (z may be overwritten by now). Equal ids all store the same value.
    for (int k = tid; k <= K; k += kThreads) {
      const int32_t id = s_id[k];
      if (id < 0 || zero) continue;
      float q = 0.0f;
      for (int i = 0; i < K; ++i)
        if (s_id[i] == id) q += s_q[i];
      float x = smooth<ENTROPY, OWN>(row, {s_z[k], 0.0f}).x - w * a.inv_t * q;
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
  a.inv_t = (float)(1.0 / in.temperature);
  a.scale = (float)(1.4426950408889634 / in.temperature);
  a.slack = (float)(8.0 / 1.4426950408889634 * (in.temperature < 1.0 ? in.temperature : 1.0));
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

template <typename T, bool LOSS, bool GRAD, bool ENTROPY, bool OWN, bool TOP>
cudaError_t launch_rows(const VocabLaunch& in, cudaStream_t stream) {
  const RowArgs a = row_args(in);
  if (!a.err) return cudaErrorInvalidSymbol;
  const auto kernel = rows_kernel<T, LOSS, GRAD, ENTROPY, OWN, TOP>;
  size_t smem = 0;
  if (TOP) {
    // A row's table has an entry for each 32 bytes of its logits and two ends.
    smem = sizeof(TopShared) + (in.vocab / kPer<T> + 3) * sizeof(T);
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
  return launch_kernel(kernel, dim3((unsigned)in.rows), dim3(kThreads), smem, stream, a);
}

template <bool LOSS, bool GRAD, bool ENTROPY, bool OWN, bool TOP>
cudaError_t launch(const VocabLaunch& in, cudaStream_t stream) {
  return in.dtype == ZS_BF16
             ? launch_rows<__nv_bfloat16, LOSS, GRAD, ENTROPY, OWN, TOP>(in, stream)
             : launch_rows<float, LOSS, GRAD, ENTROPY, OWN, TOP>(in, stream);
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
