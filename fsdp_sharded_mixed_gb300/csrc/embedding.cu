// embedding.cu — the table's rows of given tokens, scaled, and the gradient of
// the table: for each row the sum of the gradients of its tokens.
//
//   out_t = scale * E[tok_t]
//   dE_v  = add_v + scale * sum_{t: tok_t = v} d_out_t
//
// The gradient sorts the tokens (a stable counting sort, so that a row's sum
// runs over its tokens in their order) and then takes the sorted positions in
// blocks of 32, a warp to a block and a slab of 256 columns. A run of up to 64
// equal tokens is summed by the warp in whose block it starts; of a longer one
// each block's part goes to scratch memory, and the warp that finishes last adds
// the parts in their order. So the work of a warp is bounded however often a
// token occurs, each table row is written once, and no sum depends on timing.
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
constexpr int kWarps = kThreads / 32;

// ---- lookup ---------------------------------------------------------------------
struct LookupArgs {
  const void* table;
  const int64_t* tokens;
  void* out;
  int64_t rows, table_stride, out_stride;
  int32_t vocab, dim;
  float scale;
  unsigned int* err;
};

// A warp to a row and kAtOnce slabs of it.
constexpr int kAtOnce = 4;

template <typename TT, typename OT, Lay LAY>
__global__ void __launch_bounds__(kThreads) embedding_kernel(const __grid_constant__ LookupArgs a) {
  overlap_wait();
  const int64_t row = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  const int lane = threadIdx.x & 31, col0 = blockIdx.y * kAtOnce * kSlab;
  if (row >= a.rows) return;
  const int64_t token = a.tokens[row];
  OT* out = static_cast<OT*>(a.out) + row * a.out_stride;
  const bool in = token >= 0 && token < a.vocab;
  if (!in && token >= 0 && lane == 0 && blockIdx.y == 0) atomicOr(a.err, 4u);
  if (!in || !within(token, token + 1, 0, a.vocab, a.err)) {
    float v[kLane];
#pragma unroll
    for (int k = 0; k < kLane; ++k) v[k] = token < 0 ? 0.0f : NAN;
#pragma unroll
    for (int s = 0; s < kAtOnce; ++s) store8<OT, LAY>(out, col0 + s * kSlab, lane, a.dim, v);
    return;
  }
  const TT* from = static_cast<const TT*>(a.table) + token * a.table_stride;
  Raw8<TT> r[kAtOnce];
#pragma unroll
  for (int s = 0; s < kAtOnce; ++s) r[s] = load8<TT, LAY>(from, col0 + s * kSlab, lane, a.dim);
#pragma unroll
  for (int s = 0; s < kAtOnce; ++s) {
    float v[kLane];
#pragma unroll
    for (int k = 0; k < kLane; ++k) v[k] = raw_value(r[s], k) * a.scale;
    store8<OT, LAY>(out, col0 + s * kSlab, lane, a.dim, v);
  }
}

// ---- the tokens sorted ----------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigits = 1024;

struct SortArgs {
  const int64_t* tokens;
  uint32_t *keys, *order;    // sorted: the row of the table, and which token it was
  uint32_t *keys2, *order2;  // between passes
  uint32_t* tickets;         // cleared for the reduction
  int64_t rows, n_tickets;
  int32_t vocab, passes, bits;
  unsigned int* err;
};

// Tokens without a row (negative, or past the vocabulary, which sets the error
// word) get the key `vocab` and come last.
__device__ __forceinline__ uint32_t key_of(const SortArgs& a, int64_t i) {
  const int64_t token = a.tokens[i];
  if (token >= 0 && token < a.vocab) return (uint32_t)token;
  if (token >= 0) atomicOr(a.err, 4u);
  return (uint32_t)a.vocab;
}

// One block; each warp keeps its share of the tokens in order. A pass counts
// the digits warp by warp, turns the counts into places (digit first, then
// warp) and moves each warp's tokens to theirs, 32 at a time.
__global__ void __launch_bounds__(kSortThreads, 1) sort_tokens_kernel(const __grid_constant__ SortArgs a) {
  extern __shared__ uint32_t hist[];  // [kSortWarps][digits]
  __shared__ uint32_t warp_total[kSortWarps];
  overlap_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const int digits = 1 << a.bits;
  const int64_t share = ((a.rows + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int64_t lo = min(a.rows, share * warp), hi = min(a.rows, share * (warp + 1));
  for (int64_t i = tid; i < a.n_tickets; i += kSortThreads) a.tickets[i] = 0;
  uint32_t* mine = hist + warp * digits;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    // the last pass ends in keys, order
    const bool to_first = (a.passes - 1 - pass) % 2 == 0;
    const uint32_t* ks = to_first ? a.keys2 : a.keys;
    const uint32_t* os = to_first ? a.order2 : a.order;
    uint32_t* kd = to_first ? a.keys : a.keys2;
    uint32_t* od = to_first ? a.order : a.order2;
    for (int i = tid; i < kSortWarps * digits; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    for (int64_t i = lo + lane; i < hi; i += 32) {
      const uint32_t key = pass == 0 ? key_of(a, i) : ks[i];
      atomicAdd(&mine[(key >> shift) & (digits - 1)], 1u);
    }
    __syncthreads();
    uint32_t total = 0;
    if (tid < digits)
      for (int w = 0; w < kSortWarps; ++w) total += hist[w * digits + tid];
    uint32_t upto = total;  // inclusive, over the warp's digits
    for (int off = 1; off < 32; off *= 2) {
      const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, upto, off);
      if (lane >= off) upto += x;
    }
    if (lane == 31) warp_total[warp] = upto;
    __syncthreads();
    uint32_t at = upto - total;
    for (int w = 0; w < warp; ++w) at += warp_total[w];
    if (tid < digits)
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t n = hist[w * digits + tid];
        hist[w * digits + tid] = at;
        at += n;
      }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
      const int64_t i = i0 + lane;
      const bool some = i < hi;
      const uint32_t key = !some ? 0 : pass == 0 ? key_of(a, i) : ks[i];
      const uint32_t from = !some ? 0 : pass == 0 ? (uint32_t)i : os[i];
      const uint32_t digit = some ? (key >> shift) & (digits - 1) : 0xFFFFFFFFu;
      const uint32_t peers = __match_any_sync(0xFFFFFFFFu, digit);
      const uint32_t place = some ? mine[digit] + __popc(peers & ((1u << lane) - 1)) : 0;
      __syncwarp();
      if (some && lane == __ffs(peers) - 1) mine[digit] += __popc(peers);
      __syncwarp();
      if (some && within(place, (int64_t)place + 1, 0, a.rows, a.err)) {
        kd[place] = key;
        od[place] = from;
      }
    }
    __syncthreads();
  }
}

// ---- rows without tokens ---------------------------------------------------------
struct GradArgs {
  const void* d_out;
  const void* add;    // or NULL
  void* d_table;
  const uint32_t *keys, *order;
  float* parts;       // [2 * blocks][part_dim]
  uint32_t* tickets;  // [slabs][blocks]
  int64_t rows, blocks, row_stride, table_stride;
  int32_t vocab, dim, slabs, part_dim;
  float scale;
  unsigned int* err;
};

// Every row: zero, or what the gradient is added to.
template <typename GT, Lay LAY>
__global__ void __launch_bounds__(kThreads) fill_rows_kernel(const __grid_constant__ GradArgs a) {
  overlap_wait();
  const int lane = threadIdx.x & 31;
  const int64_t v = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  if (v >= a.vocab || !within(v, v + 1, 0, a.vocab, a.err)) return;
  GT* row = static_cast<GT*>(a.d_table) + v * a.table_stride;
  const GT* add = a.add ? static_cast<const GT*>(a.add) + v * a.table_stride : nullptr;
  for (int col0 = 0; col0 < a.dim; col0 += kSlab) {
    float x[kLane];
    Raw8<GT> r;
    if (add) r = load8<GT, LAY>(add, col0, lane, a.dim);
#pragma unroll
    for (int k = 0; k < kLane; ++k) x[k] = add ? raw_value(r, k) : 0.0f;
    store8<GT, LAY>(row, col0, lane, a.dim, x);
  }
}

// ---- sums over sorted tokens -----------------------------------------------------
constexpr int kBlock = 32;    // sorted positions of a warp
constexpr int kLongRun = 64;  // equal tokens that one warp sums by itself

template <typename T, typename GT, Lay LAY>
struct Reduce {
  const GradArgs& a;
  const int lane, col0;
  float acc[kLane];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < kLane; ++k) acc[k] = 0.0f;
  }
  __device__ __forceinline__ void add(const Raw8<T>& r) {
#pragma unroll
    for (int k = 0; k < kLane; ++k) acc[k] = __fadd_rn(acc[k], raw_value(r, k));
  }
  __device__ __forceinline__ Raw8<T> row(uint32_t t) {
    if (!within(t, (int64_t)t + 1, 0, a.rows, a.err)) t = 0;
    return load8<T, LAY>(static_cast<const T*>(a.d_out) + (int64_t)t * a.row_stride, col0, lane,
                         a.dim);
  }
  // The rows of lanes [l, l + n) of `order`.
  __device__ __forceinline__ void add_rows(uint32_t order, int l, int n) {
    int i = 0;
    for (; i + 4 <= n; i += 4) {
      Raw8<T> r[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) r[u] = row(__shfl_sync(0xFFFFFFFFu, order, l + i + u));
#pragma unroll
      for (int u = 0; u < 4; ++u) add(r[u]);
    }
    for (; i < n; ++i) add(row(__shfl_sync(0xFFFFFFFFu, order, l + i)));
  }
  __device__ __forceinline__ void write(uint32_t v) {
    if (!within(v, (int64_t)v + 1, 0, a.vocab, a.err)) return;
    const int64_t at = (int64_t)v * a.table_stride;
    float x[kLane];
    if (a.add) {
      const Raw8<GT> r = load8<GT, LAY>(static_cast<const GT*>(a.add) + at, col0, lane, a.dim);
#pragma unroll
      for (int k = 0; k < kLane; ++k) x[k] = __fmaf_rn(acc[k], a.scale, raw_value(r, k));
    } else {
#pragma unroll
      for (int k = 0; k < kLane; ++k) x[k] = acc[k] * a.scale;
    }
    store8<GT, LAY>(static_cast<GT*>(a.d_table) + at, col0, lane, a.dim, x);
  }
  // Parts are part_dim apart, a whole number of lanes: a lane finds its elements
  // where it left them, in either order of columns.
  __device__ __forceinline__ void write_part(int64_t slot) {
    if (!within(slot, slot + 1, 0, 2 * a.blocks, a.err)) return;
    store8<float, LAY>(a.parts + slot * a.part_dim, col0, lane, a.part_dim, acc);
  }
  __device__ __forceinline__ void add_part(int64_t slot) {
    if (!within(slot, slot + 1, 0, 2 * a.blocks, a.err)) return;
    const float* p = a.parts + slot * a.part_dim;
#pragma unroll
    for (int k = 0; k < kLane; ++k) {
      const int c = column<LAY>(col0, lane, k);
      if (c < a.part_dim) acc[k] = __fadd_rn(acc[k], __ldcg(p + c));
    }
  }
};

// The first sorted position whose key is at least v (32 probes a step).
__device__ __forceinline__ int64_t lower_bound(const GradArgs& a, uint32_t v, int lane) {
  int64_t lo = 0, hi = a.rows;  // keys before lo are below v, from hi on they are not
  while (lo < hi) {
    const int64_t step = (hi - lo + 31) / 32, at = lo + lane * step;
    const uint32_t below = __ballot_sync(0xFFFFFFFFu, at < hi && a.keys[at] < v);
    const int n = __popc(below);
    if (n < 32 && lo + n * step < hi) hi = lo + n * step;
    if (n > 0) lo += (n - 1) * step + 1;
  }
  return lo;
}

template <typename T, typename GT, Lay LAY>
__global__ void __launch_bounds__(kThreads) sum_tokens_kernel(const __grid_constant__ GradArgs a) {
  overlap_wait();
  const int lane = threadIdx.x & 31;
  const int64_t b = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  if (b >= a.blocks) return;
  // keys and tokens of this block, of the two before and the two after it
  const uint32_t none = 0xFFFFFFFFu;
  auto key_at = [&](int64_t i) { return i >= 0 && i < a.rows ? a.keys[i] : none; };
  auto order_at = [&](int64_t i) { return i < a.rows ? a.order[i] : 0u; };
  const int64_t p = b * kBlock + lane;
  const uint32_t before2 = key_at(p - 64), before = key_at(p - 32), here = key_at(p),
                 after = key_at(p + 32), after2 = key_at(p + 64);
  const uint32_t order = order_at(p), order1 = order_at(p + 32), order2 = order_at(p + 64);
  Reduce<T, GT, LAY> r{a, lane, (int)blockIdx.y * kSlab, {}};
  for (int l = 0; l < kBlock;) {
    const uint32_t v = __shfl_sync(none, here, l);
    if (v >= (uint32_t)a.vocab) return;  // the tokens without a row, and the end
    const int n = __popc(__ballot_sync(none, here == v));
    const bool starts = l > 0 || __shfl_sync(none, before, 31) != v;
    const int n_before =
        starts ? 0
               : __popc(__ballot_sync(none, before == v)) + __popc(__ballot_sync(none, before2 == v));
    const int n1 = l + n < kBlock ? 0 : __popc(__ballot_sync(none, after == v));
    const int n2 = n1 < 32 ? 0 : __popc(__ballot_sync(none, after2 == v));
    r.clear();
    if (n_before + n + n1 + n2 <= kLongRun) {
      if (starts) {
        r.add_rows(order, l, n);
        r.add_rows(order1, 0, n1);
        r.add_rows(order2, 0, n2);
        r.write(v);
      }
    } else {
      // This block's part: place 2b + 1 if the run starts here, else 2b.
      r.add_rows(order, l, n);
      r.write_part(2 * b + starts);
      const int64_t from = lower_bound(a, v, lane) / kBlock;
      const int64_t to = (lower_bound(a, v + 1, lane) - 1) / kBlock;
      __threadfence();
      __syncwarp();
      uint32_t done = 0;
      if (lane == 0) done = atomicAdd(&a.tickets[blockIdx.y * a.blocks + from], 1u);
      done = __shfl_sync(none, done, 0);
      if (done == (uint32_t)(to - from)) {
        __threadfence();
        r.clear();
        r.add_part(2 * from + 1);
        for (int64_t j = from + 1; j <= to; ++j) r.add_part(2 * j);
        r.write(v);
      }
    }
    l += n;
  }
}

template <typename TT, typename OT>
cudaError_t launch_lookup(const LookupArgs& a, bool vec, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.rows + kWarps - 1) / kWarps),
                  (unsigned)((a.dim + kAtOnce * kSlab - 1) / (kAtOnce * kSlab)));
  return vec ? launch_kernel(embedding_kernel<TT, OT, kEight>, grid, dim3(kThreads), 0, stream, a)
             : launch_kernel(embedding_kernel<TT, OT, kOne>, grid, dim3(kThreads), 0, stream, a);
}

template <typename T, typename GT, Lay LAY>
cudaError_t launch_sums(const GradArgs& a, bool fill, bool sums, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (fill)
    e = launch_kernel(fill_rows_kernel<GT, LAY>, dim3((unsigned)((a.vocab + kWarps - 1) / kWarps)),
                      dim3(kThreads), 0, stream, a);
  if (e != cudaSuccess || !sums) return e;
  const dim3 grid((unsigned)((a.blocks + kWarps - 1) / kWarps), (unsigned)a.slabs);
  return launch_kernel(sum_tokens_kernel<T, GT, LAY>, grid, dim3(kThreads), 0, stream, a);
}

int64_t align16(int64_t n) { return (n + 15) / 16 * 16; }

// Where the pieces of the gradient's scratch lie.
struct Scratch {
  int64_t blocks, n_tickets, part_dim, keys, order, keys2, order2, tickets, parts, bytes;
};
Scratch scratch_of(int64_t rows, int64_t dim) {
  Scratch s;
  const int64_t slabs = (dim + kSlab - 1) / kSlab, list = align16(rows * 4);
  s.blocks = (rows + kBlock - 1) / kBlock;
  s.n_tickets = s.blocks * slabs;
  s.keys = 0;
  s.order = list;
  s.keys2 = 2 * list;
  s.order2 = 3 * list;
  s.tickets = 4 * list;
  s.parts = s.tickets + align16(4 * s.n_tickets);
  s.part_dim = (dim + kLane - 1) / kLane * kLane;
  s.bytes = s.parts + 8 * s.blocks * s.part_dim;
  return s;
}

}  // namespace

int64_t embedding_grad_workspace_bytes(int64_t rows, int64_t dim) {
  return scratch_of(rows, dim).bytes;
}

cudaError_t launch_embedding(const EmbeddingLaunch& in, cudaStream_t stream) {
  LookupArgs a;
  a.table = in.table;
  a.tokens = in.tokens;
  a.out = in.rows_out;
  a.rows = in.rows;
  a.table_stride = in.table_stride;
  a.out_stride = in.row_stride;
  a.vocab = (int32_t)in.vocab;
  a.dim = (int32_t)in.dim;
  a.scale = (float)in.scale;
  a.err = device_error_word();
  if (!a.err) return cudaErrorInvalidSymbol;
  const bool bt = in.table_dtype == ZS_BF16, br = in.dtype == ZS_BF16;
  const bool vec = rows_aligned(a.table, a.table_stride, bt ? 2 : 4) &&
                   rows_aligned(a.out, a.out_stride, br ? 2 : 4);
  if (bt)
    return br ? launch_lookup<__nv_bfloat16, __nv_bfloat16>(a, vec, stream)
              : launch_lookup<__nv_bfloat16, float>(a, vec, stream);
  return br ? launch_lookup<float, __nv_bfloat16>(a, vec, stream)
            : launch_lookup<float, float>(a, vec, stream);
}

cudaError_t launch_embedding_grad(const EmbeddingLaunch& in, cudaStream_t stream) {
  const Scratch s = scratch_of(in.rows, in.dim);
  unsigned char* ws = static_cast<unsigned char*>(in.workspace);
  GradArgs a = {};
  a.d_out = in.rows_in;
  a.add = in.add;
  a.d_table = in.d_table;
  a.rows = in.rows;
  a.row_stride = in.row_stride;
  a.table_stride = in.table_stride;
  a.vocab = (int32_t)in.vocab;
  a.dim = (int32_t)in.dim;
  a.slabs = (int32_t)((in.dim + kSlab - 1) / kSlab);
  a.blocks = s.blocks;
  a.part_dim = (int32_t)s.part_dim;
  a.scale = (float)in.scale;
  a.err = device_error_word();
  if (!a.err) return cudaErrorInvalidSymbol;
  if (in.rows > 0) {
    a.keys = reinterpret_cast<uint32_t*>(ws + s.keys);
    a.order = reinterpret_cast<uint32_t*>(ws + s.order);
    a.tickets = reinterpret_cast<uint32_t*>(ws + s.tickets);
    a.parts = reinterpret_cast<float*>(ws + s.parts);
    SortArgs k;
    k.tokens = in.tokens;
    k.keys = reinterpret_cast<uint32_t*>(ws + s.keys);
    k.order = reinterpret_cast<uint32_t*>(ws + s.order);
    k.keys2 = reinterpret_cast<uint32_t*>(ws + s.keys2);
    k.order2 = reinterpret_cast<uint32_t*>(ws + s.order2);
    k.tickets = a.tickets;
    k.rows = in.rows;
    k.n_tickets = s.n_tickets;
    k.vocab = a.vocab;
    int bits = 1;
    while (in.vocab >> bits) ++bits;  // keys 0..vocab
    k.passes = (bits + 9) / 10;
    k.bits = (bits + k.passes - 1) / k.passes;
    k.err = a.err;
    const int smem = kSortWarps * (int)sizeof(uint32_t) << k.bits;
    cudaError_t e = cudaFuncSetAttribute(sort_tokens_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSortWarps * kMaxDigits * (int)sizeof(uint32_t));
    if (e == cudaSuccess)
      e = launch_kernel(sort_tokens_kernel, dim3(1), dim3(kSortThreads), smem, stream, k);
    if (e != cudaSuccess) return e;
  }
  const bool br = in.dtype == ZS_BF16, bt = in.table_dtype == ZS_BF16;
  const bool vec = rows_aligned(a.d_out, a.row_stride, br ? 2 : 4) &&
                   rows_aligned(a.d_table, a.table_stride, bt ? 2 : 4) &&
                   rows_aligned(a.add, a.table_stride, bt ? 2 : 4);
  const bool fill = a.add != a.d_table, sums = in.rows > 0;
  if (br) {
    if (bt)
      return vec ? launch_sums<__nv_bfloat16, __nv_bfloat16, kEight>(a, fill, sums, stream)
                 : launch_sums<__nv_bfloat16, __nv_bfloat16, kOne>(a, fill, sums, stream);
    return vec ? launch_sums<__nv_bfloat16, float, kEight>(a, fill, sums, stream)
               : launch_sums<__nv_bfloat16, float, kOne>(a, fill, sums, stream);
  }
  if (bt)
    return vec ? launch_sums<float, __nv_bfloat16, kEight>(a, fill, sums, stream)
               : launch_sums<float, __nv_bfloat16, kOne>(a, fill, sums, stream);
  return vec ? launch_sums<float, float, kEight>(a, fill, sums, stream)
             : launch_sums<float, float, kOne>(a, fill, sums, stream);
}

}  // namespace zs
