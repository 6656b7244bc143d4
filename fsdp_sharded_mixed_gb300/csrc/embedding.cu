// embedding.cu — the table's rows of given tokens, scaled, and the gradient of
// the table: for each row the sum of the gradients of its tokens.
//
//   out_t = scale * E[tok_t]
//   dE_v  = add_v + scale * sum_{t: tok_t = v} d_out_t
//
// The gradient sorts the tokens (a stable counting sort, so that a row's sum
// runs over its tokens in their order) and then takes the sorted positions in
// blocks of 128, 16 a warp, for a slab of 256 columns. A run of equal tokens
// within a warp's 16 is summed by it; the parts of longer ones and of those that
// cross warps are added in their order, through shared memory and, across blocks,
// scratch memory. So the work of a warp is bounded however often a token occurs,
// and no sum depends on timing. Sums are fp32; a result is rounded once.
//
// Bound: HBM for large tables, which are written whole (16384 tokens of 151936 x
// 2048 bf16: 106 us, 0.95 of the measured copy rate; 8 tokens: 87, 1.05); latency
// for middling ones: 8191 of 50257 x 768 added to another matrix 33.6 us (0.73), of
// which the sort takes 10. The lookup: 16384 rows of 2048 16.1 us (0.86).
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
  bool once;  // the output is written past L2
  unsigned int* err;
};

// A warp to a row and kAtOnce slabs of it (16384 rows of 2048 bf16: 17.5 us with two,
// 18.3 with four, 17.9 with eight; 8192 of 768: 4.8, 4.8, 7.7).
constexpr int kAtOnce = 4;
// Outputs that L2 (129 MB) would not hold beside the table are written past it, so
// that the table's frequent rows stay there (the same 16384 rows, with four slabs:
// 18.3 -> 16.0 us, with two 18.5); smaller ones are left to their reader.
constexpr int64_t kKeptOutput = 48 << 20;

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
    store8<OT, LAY>(out, col0 + s * kSlab, lane, a.dim, v, a.once);
  }
}

// ---- the tokens sorted, the other rows written ------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortBlocks = 8;  // one cluster (the portable size)
constexpr int kMaxDigits = 1024;
constexpr int kAtHand = 4;      // rounds of a warp's tokens on their way at once

struct SortArgs {
  const int64_t* tokens;
  uint32_t *keys, *order;    // sorted: the row of the table, and which token it was
  uint32_t *keys2, *order2;  // between passes
  uint32_t* tickets;         // cleared for the reduction
  int64_t rows, n_tickets, share;  // share: tokens of a warp
  int32_t vocab, passes, bits;
  unsigned int* err;
};

struct GradArgs {
  const void* d_out;
  const int64_t* tokens;
  const void* add;    // or NULL
  void* d_table;
  const uint32_t *keys, *order;
  float* parts;       // [2 * blocks][part_dim]
  uint32_t* tickets;  // [slabs][blocks]
  int64_t rows, blocks, row_stride, table_stride;
  int32_t vocab, dim, slabs, part_dim;
  int32_t fill_blocks;  // of the launch, which write the rows without tokens
  float scale;
  unsigned int* err;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
// A word of another block's shared memory, at the place of this block's p.
__device__ __forceinline__ uint32_t word_of(const uint32_t* p, int rank) {
  uint32_t at = (uint32_t)__cvta_generic_to_shared(p), x;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}

// Tokens without a row (negative, or past the vocabulary, which sets the error
// word) get the key `vocab` and come last.
__device__ __forceinline__ uint32_t key_of(const SortArgs& a, int64_t i, unsigned int* err) {
  const int64_t token = a.tokens[i];
  if (token >= 0 && token < a.vocab) return (uint32_t)token;
  if (token >= 0) atomicOr(err, 4u);
  return (uint32_t)a.vocab;
}

// A stable counting sort by digits, the lowest first, by the kSortBlocks blocks of
// one cluster; each warp keeps its share of the tokens in order. A pass counts the
// digits warp by warp, turns the counts into places (by digit, then block, then
// warp) and moves each warp's tokens to theirs, 32 at a time.
struct SortShared {
  uint32_t of_block[kMaxDigits];    // the block's counts, read by the others
  uint32_t of_warp[kSortWarps];
  uint32_t count[1];                // [kSortWarps][digits]
};
__device__ void sort_tokens(const SortArgs& a, SortShared& sh, int rank, unsigned int* err) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const int digits = 1 << a.bits;
  const int64_t lo = min(a.rows, a.share * (rank * kSortWarps + warp));
  const int64_t hi = min(a.rows, lo + a.share);
  for (int64_t i = rank * kSortThreads + tid; i < a.n_tickets; i += kSortBlocks * kSortThreads)
    a.tickets[i] = 0;
  uint32_t* mine = sh.count + warp * digits;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    // the last pass ends in keys, order
    const bool to_first = (a.passes - 1 - pass) % 2 == 0;
    const uint32_t* ks = to_first ? a.keys2 : a.keys;
    const uint32_t* os = to_first ? a.order2 : a.order;
    uint32_t* kd = to_first ? a.keys : a.keys2;
    uint32_t* od = to_first ? a.order : a.order2;
    for (int i = tid; i < kSortWarps * digits; i += kSortThreads) sh.count[i] = 0;
    __syncthreads();
    // A warp's tokens, 32 * kAtHand at a time; few stay in registers until they are moved.
    uint32_t keys[kAtHand], from[kAtHand];
    auto load = [&](int64_t i0) {
#pragma unroll
      for (int u = 0; u < kAtHand; ++u) {
        const int64_t i = i0 + u * 32 + lane;
        const bool some = i < hi;
        keys[u] = !some ? 0 : pass == 0 ? key_of(a, i, err) : __ldcg(ks + i);
        from[u] = !some ? 0 : pass == 0 ? (uint32_t)i : __ldcg(os + i);
      }
    };
    const bool held = hi - lo <= 32 * kAtHand;
    if (held) load(lo);
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kAtHand) {
      if (!held) load(i0);
#pragma unroll
      for (int u = 0; u < kAtHand; ++u)
        if (i0 + u * 32 + lane < hi)
          atomicAdd(&mine[(keys[u] >> shift) & (digits - 1)], 1u);
    }
    __syncthreads();
    uint32_t total = 0;
    if (tid < digits) {
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) total += sh.count[w * digits + tid];
      sh.of_block[tid] = total;
    }
    cluster_sync();
    uint32_t all = 0, before = 0;
    if (tid < digits)
#pragma unroll
      for (int r = 0; r < kSortBlocks; ++r) {
        const uint32_t n = word_of(sh.of_block + tid, r);
        before += r < rank ? n : 0;
        all += n;
      }
    // (What the last pass moves is not read in this launch; a block may only not leave
    // before the others have read its counts, which they say here. The release makes
    // sure that they have.)
    const bool ends = pass + 1 == a.passes;
    if (ends) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    uint32_t upto = all;  // inclusive, over the warp's digits
    for (int off = 1; off < 32; off *= 2) {
      const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, upto, off);
      if (lane >= off) upto += x;
    }
    if (lane == 31) sh.of_warp[warp] = upto;
    __syncthreads();
    const uint32_t ahead = lane < warp ? sh.of_warp[lane] : 0;
    uint32_t at = upto - all + before + __reduce_add_sync(0xFFFFFFFFu, ahead);
    if (tid < digits) {
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t n = sh.count[w * digits + tid];
        sh.count[w * digits + tid] = at;
        at += n;
      }
    }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kAtHand) {
      if (!held) load(i0);
#pragma unroll
      for (int u = 0; u < kAtHand; ++u) {
        if (i0 + u * 32 >= hi) break;
        const bool some = i0 + u * 32 + lane < hi;
        const uint32_t digit = some ? (keys[u] >> shift) & (digits - 1) : 0xFFFFFFFFu;
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, digit);
        const uint32_t place = some ? mine[digit] + __popc(peers & ((1u << lane) - 1)) : 0;
        __syncwarp();
        if (some && lane == __ffs(peers) - 1) mine[digit] += __popc(peers);
        __syncwarp();
        if (some && within(place, (int64_t)place + 1, 0, a.rows, err)) {
          kd[place] = keys[u];
          od[place] = from[u];
        }
      }
    }
    if (ends)
      asm volatile("barrier.cluster.wait;" ::: "memory");
    else
      cluster_sync();  // what was moved is there for all, and the counts have been read
  }
}

__global__ void __launch_bounds__(kSortThreads, 1) __cluster_dims__(kSortBlocks, 1, 1)
    sort_tokens_kernel(const __grid_constant__ SortArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  overlap_wait();
  sort_tokens(a, *reinterpret_cast<SortShared*>(smem), (int)blockIdx.x, a.err);
}

// ---- rows without tokens ----------------------------------------------------------
constexpr int kFillBlocks = 304;      // two to an SM of 152
constexpr int kMostFillBlocks = 1216;
constexpr int kMetWords = (ZS_MAX_VOCAB / kFillBlocks + 32) / 32;

// The lane's elements, past L1: a block that writes rows beside the sort does not wait
// for it, and it is that wait which would make sure of what L1 holds.
template <typename T, Lay LAY>
__device__ __forceinline__ Raw8<T> load8_from_l2(const T* row, int col0, int lane, int D) {
  constexpr int kWords = kLane * (int)sizeof(T) / 4;
  Raw8<T> r;
  if (LAY == kEight && col0 + lane * 8 + 8 <= D) {
    const T* p = row + col0 + lane * 8;
    if (kWords == 8 && (uintptr_t)p % 32 == 0) {
      asm volatile("ld.relaxed.gpu.global.v8.u32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]),
                     "=r"(r.w[kWords - 4]), "=r"(r.w[kWords - 3]), "=r"(r.w[kWords - 2]),
                     "=r"(r.w[kWords - 1])
                   : "l"(p)
                   : "memory");
      return r;
    }
#pragma unroll
    for (int i = 0; i < kWords; i += 4)
      asm volatile("ld.relaxed.gpu.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(r.w[i]), "=r"(r.w[i + 1]), "=r"(r.w[i + 2]), "=r"(r.w[i + 3])
                   : "l"(reinterpret_cast<const uint32_t*>(p) + i)
                   : "memory");
    return r;
  }
#pragma unroll
  for (int k = 0; k < kLane; ++k) {
    const int c = column<LAY>(col0, lane, k);
    set_raw(r, k, c < D ? __ldcg(row + c) : T(0.0f));
  }
  return r;
}

// A block's rows first, first + step, ...: `met` has a bit for each, set where the
// batch has tokens of it. The others become zero, or what the gradient is added to: a
// warp to a row.
template <typename GT, Lay LAY, bool ADD>
__device__ __forceinline__ void fill_rows(const GradArgs& a, const uint32_t* met, uint32_t first,
                                          uint32_t step, uint32_t rows) {
  // (two rows' loads on their way at once where they are few bytes: 8191 tokens of 50257
  // x 768 bf16 33.6 us against 35.0)
  constexpr int kSlabs = 4, kRowsAtOnce = ADD && sizeof(GT) == 2 ? 2 : 1;
  const int lane = threadIdx.x & 31;
  for (uint32_t i0 = threadIdx.x / 32; i0 < rows; i0 += kRowsAtOnce * kWarps) {
    bool write[kRowsAtOnce];
    int64_t at[kRowsAtOnce];
#pragma unroll
    for (int k = 0; k < kRowsAtOnce; ++k) {
      const uint32_t i = i0 + k * kWarps;
      const int64_t v = first + i * (int64_t)step;
      write[k] = i < rows && !(met[i / 32] >> (i & 31) & 1) && within(v, v + 1, 0, a.vocab, a.err);
      at[k] = v * a.table_stride;
    }
    for (int s0 = 0; s0 < a.slabs; s0 += kSlabs) {
      Raw8<GT> x[kRowsAtOnce][kSlabs];
#pragma unroll
      for (int k = 0; k < kRowsAtOnce; ++k)
#pragma unroll
        for (int s = 0; s < kSlabs; ++s) {
          x[k][s] = {};
          if (ADD && write[k] && s0 + s < a.slabs)
            x[k][s] = load8_from_l2<GT, LAY>(static_cast<const GT*>(a.add) + at[k],
                                             (s0 + s) * kSlab, lane, a.dim);
        }
#pragma unroll
      for (int k = 0; k < kRowsAtOnce; ++k)
#pragma unroll
        for (int s = 0; s < kSlabs; ++s)
          if (write[k] && s0 + s < a.slabs)
            store_raw8<GT, LAY>(static_cast<GT*>(a.d_table) + at[k], (s0 + s) * kSlab, lane, a.dim,
                                x[k][s]);
    }
  }
}

// ---- sums over sorted tokens -----------------------------------------------------
constexpr int kEach = 16;               // sorted positions of a warp
constexpr int kBlock = kEach * kWarps;  // and of a block

// What a warp of a block knows of its first and its last run.
struct Edges {
  uint32_t v_first, v_last;
  bool from_before, to_next;  // the first began before this warp, the last goes on behind it
  bool one;                   // they are one run (and its part is that of the first)
};
// The parts of runs that cross warps: of the first run, if it began before, and of
// the last, if it goes on.
struct Crossing {
  Edges edges[kWarps];
  int64_t from[2], to[2];  // of the block's first run and its last, where they cross blocks
  float2 parts[kWarps][2][kLane / 2][32];
};

// ADD: the sums are added to something.
template <typename T, typename GT, Lay LAY, bool ADD>
struct Reduce {
  static constexpr int kWords = kLane / 4 * ((int)sizeof(T) + (ADD ? (int)sizeof(GT) : 0));
  static constexpr int kRows = kWords <= 4 ? 8 : kWords <= 8 ? 4 : 2;  // on their way at once
  const GradArgs& a;
  const int lane;
  int col0;
  float2 acc[kLane / 2];
  Raw8<GT> base;

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kLane / 2; ++i) acc[i] = {0.0f, 0.0f};
  }
  __device__ __forceinline__ void add(const Raw8<T>& r) {
#pragma unroll
    for (int i = 0; i < kLane / 2; ++i) acc[i] = __fadd2_rn(acc[i], pair_of(r, i));
  }
  __device__ __forceinline__ Raw8<T> row(uint32_t t) const {
    if (!within(t, (int64_t)t + 1, 0, a.rows, a.err)) t = 0;
    return load8<T, LAY>(static_cast<const T*>(a.d_out) + (int64_t)t * a.row_stride, col0, lane,
                         a.dim);
  }
  __device__ __forceinline__ Raw8<GT> base_of(uint32_t v) const {
    if (!within(v, (int64_t)v + 1, 0, a.vocab, a.err)) v = 0;
    return load8<GT, LAY>(static_cast<const GT*>(a.add) + (int64_t)v * a.table_stride, col0, lane,
                          a.dim);
  }
  __device__ __forceinline__ void write(uint32_t v) const {
    if (!within(v, (int64_t)v + 1, 0, a.vocab, a.err)) return;
    Raw8<GT> r;
#pragma unroll
    for (int i = 0; i < kLane / 2; ++i) {
      const float2 scale = {a.scale, a.scale};
      set_pair(r, i, ADD ? __ffma2_rn(acc[i], scale, pair_of(base, i))
                         : __fmul2_rn(acc[i], scale));
    }
    store_raw8<GT, LAY>(static_cast<GT*>(a.d_table) + (int64_t)v * a.table_stride, col0, lane,
                        a.dim, r);
  }
  __device__ __forceinline__ void keep(float2 (*part)[32]) const {
#pragma unroll
    for (int i = 0; i < kLane / 2; ++i) part[i][lane] = acc[i];
  }
  __device__ __forceinline__ void add_kept(const float2 (*part)[32]) {
#pragma unroll
    for (int i = 0; i < kLane / 2; ++i) acc[i] = __fadd2_rn(acc[i], part[i][lane]);
  }
  // Parts in scratch memory are part_dim apart, a whole number of lanes: a lane
  // finds its elements where it left them, in either order of columns.
  __device__ __forceinline__ void write_part(int64_t slot) const {
    if (!within(slot, slot + 1, 0, 2 * a.blocks, a.err)) return;
    Raw8<float> r;
#pragma unroll
    for (int i = 0; i < kLane / 2; ++i) set_pair(r, i, acc[i]);
    store_raw8<float, LAY>(a.parts + slot * a.part_dim, col0, lane, a.part_dim, r);
  }
  // The parts of blocks from..to of one run, in their order.
  __device__ __forceinline__ void add_parts(int64_t from, int64_t to) {
    constexpr int kAtOnce = 4;
    for (int64_t j0 = from; j0 <= to; j0 += kAtOnce) {
      Raw8<float> r[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int64_t j = j0 + u, slot = j == from ? 2 * j + 1 : 2 * j;
        r[u] = {};
        if (j <= to && within(slot, slot + 1, 0, 2 * a.blocks, a.err)) {
          const float* p = a.parts + slot * a.part_dim;
#pragma unroll
          for (int k = 0; k < kLane; ++k) {
            const int c = column<LAY>(col0, lane, k);
            if (c < a.part_dim) r[u].w[k] = __float_as_uint(__ldcg(p + c));
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
        for (int i = 0; i < kLane / 2; ++i) acc[i] = __fadd2_rn(acc[i], pair_of(r[u], i));
    }
  }
};

// The first sorted positions whose keys are at least v and v + 1 (32 probes a step,
// both searches' on their way together).
__device__ __forceinline__ void run_of(const GradArgs& a, uint32_t v, int lane, int64_t* from,
                                       int64_t* to) {
  int64_t lo[2] = {0, 0}, hi[2] = {a.rows, a.rows};  // keys before lo are below, from hi on not
  while (lo[0] < hi[0] || lo[1] < hi[1]) {
    int64_t step[2];
    bool below[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      step[k] = (hi[k] - lo[k] + 31) / 32;
      const int64_t at = lo[k] + lane * step[k];
      below[k] = at < hi[k] && __ldcg(a.keys + at) < v + k;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int n = __popc(__ballot_sync(0xFFFFFFFFu, below[k]));
      if (lo[k] >= hi[k]) continue;
      if (n < 32 && lo[k] + n * step[k] < hi[k]) hi[k] = lo[k] + n * step[k];
      if (n > 0) lo[k] += (n - 1) * step[k] + 1;
    }
  }
  *from = lo[0];
  *to = lo[1];
}

// A block to kBlock sorted positions and a slab of columns. A warp's rows are asked
// for kRows at a time whatever runs they belong to; a run's sum is written when the
// next one starts. Runs that cross warps are put together in shared memory by the
// warp in which they start, those that cross blocks from scratch memory by the
// block that is through with its part last.
template <typename T, typename GT, Lay LAY, bool ADD>
__device__ __forceinline__ void sum_tokens(const GradArgs& a, Crossing& sh, int64_t item) {
  using R = Reduce<T, GT, LAY, ADD>;
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t b = item / a.slabs;
  const int slab = (int)(item - b * a.slabs);
  const int64_t p0 = b * kBlock + warp * kEach;
  // the warp's keys, and one to either side
  const int64_t p = p0 + lane, q = lane == 0 ? p0 - 1 : p0 + kEach;
  const bool mine = lane < kEach && p < a.rows;
  const uint32_t here = mine ? a.keys[p] : kAll;
  const uint32_t beside = q >= 0 && q < a.rows ? a.keys[q] : kAll;
  const uint32_t order = mine ? a.order[p] : 0;
  const uint32_t up = __shfl_up_sync(kAll, here, 1), left = lane == 0 ? beside : up;
  const uint32_t next = __shfl_sync(kAll, beside, 31);
  // tokens with a row, and the first ones of their runs
  const int n = __popc(__ballot_sync(kAll, lane < kEach && here < (uint32_t)a.vocab));
  const uint32_t starts = __ballot_sync(kAll, lane < n && here != left);
  R r{a, lane, slab * kSlab, {}, {}};
  Edges e = {};
  if (n > 0) {
    e.v_first = __shfl_sync(kAll, here, 0);
    e.v_last = __shfl_sync(kAll, here, n - 1);
    e.from_before = !(starts & 1);
    e.to_next = n == kEach && next == e.v_last;
    e.one = starts == 0;
  }
  if (lane == 0) sh.edges[warp] = e;
  uint32_t v = e.v_first;
  bool before_me = e.from_before;  // of the run at work
  r.clear();
#pragma unroll
  for (int i0 = 0; i0 < kEach; i0 += R::kRows) {
    Raw8<T> rows[R::kRows];
    Raw8<GT> bases[ADD ? R::kRows : 1];
#pragma unroll
    for (int u = 0; u < R::kRows; ++u) {
      const int i = i0 + u;
      if (i >= n) break;
      rows[u] = r.row(__shfl_sync(kAll, order, i));
      if (ADD && (starts >> i & 1)) bases[ADD ? u : 0] = r.base_of(__shfl_sync(kAll, here, i));
    }
    // while they are on their way: how far the runs that cross the block's ends go
    if (i0 == 0 && ((warp == 0 && e.from_before) || (warp == kWarps - 1 && e.to_next))) {
      const int end = warp == 0 && e.from_before ? 0 : 1;
      int64_t from, to;
      run_of(a, end ? e.v_last : e.v_first, lane, &from, &to);
      if (lane == 0) {
        sh.from[end] = from / kBlock;
        sh.to[end] = (to - 1) / kBlock;
      }
    }
#pragma unroll
    for (int u = 0; u < R::kRows; ++u) {
      const int i = i0 + u;
      if (i >= n) break;
      if (starts >> i & 1) {
        if (i > 0) {
          if (before_me)
            r.keep(sh.parts[warp][0]);
          else
            r.write(v);
        }
        v = __shfl_sync(kAll, here, i);
        before_me = false;
        r.clear();
        if (ADD) r.base = bases[ADD ? u : 0];
      }
      r.add(rows[u]);
    }
  }
  if (n > 0) {
    if (before_me)
      r.keep(sh.parts[warp][0]);
    else if (e.to_next)
      r.keep(sh.parts[warp][1]);
    else
      r.write(v);
  }
  __syncthreads();
  if (n == 0) return;

  // Adds the parts of a run from warp w on; whether it ends within the block.
  auto add_from = [&](int w) {
    for (; w < kWarps; ++w) {
      r.add_kept(sh.parts[w][0]);
      if (!sh.edges[w].one || !sh.edges[w].to_next) return true;
    }
    return false;
  };
  // Joins the run of v, whose part of this block was written.
  auto join = [&](uint32_t v, int end) {
    const int64_t from = sh.from[end], to = sh.to[end];
    __threadfence();
    __syncwarp();
    uint32_t done = 0;
    if (lane == 0 && within(from, from + 1, 0, a.blocks, a.err))
      done = atomicAdd(&a.tickets[slab * a.blocks + from], 1u);
    done = __shfl_sync(kAll, done, 0);
    if (done != (uint32_t)(to - from)) return;
    __threadfence();
    if (ADD) r.base = r.base_of(v);
    r.clear();
    r.add_parts(from, to);
    r.write(v);
  };
  if (warp == 0 && e.from_before) {  // began in a block before
    r.clear();
    add_from(0);
    r.write_part(2 * b);
    join(e.v_first, 0);
  }
  if (e.to_next && !(e.one && e.from_before)) {  // starts in this warp
    r.clear();
    r.add_kept(sh.parts[warp][1]);
    if (add_from(warp + 1)) {
      if (ADD) r.base = r.base_of(e.v_last);
      r.write(e.v_last);
    } else {
      r.write_part(2 * b + 1);
      join(e.v_last, 1);
    }
  }
}

// The first blocks write the rows without tokens, which they see from the tokens
// themselves; the others take a block of sorted positions and a slab each, and
// three blocks share an SM, so that the sums run beside the writing. The launch
// follows the sort's, but only the sums wait for that: the rows are written while it
// runs. (What came before the sort has ended by then: the sort waited for it before
// it let this launch start.)
template <typename T, typename GT, Lay LAY, bool ADD>
__global__ void __launch_bounds__(kThreads, 3)
    embedding_grad_kernel(const __grid_constant__ GradArgs a) {
  __shared__ union {
    Crossing sums;
    uint32_t met[kMetWords];
  } sh;
  if ((int)blockIdx.x >= a.fill_blocks) {
    overlap_wait();
    sum_tokens<T, GT, LAY, ADD>(a, sh.sums, (int64_t)blockIdx.x - a.fill_blocks);
    return;
  }
  if (a.rows == 0) overlap_wait();  // there is no sort
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = threadIdx.x; i < kMetWords; i += kThreads) sh.met[i] = 0;
  __syncthreads();
  const uint64_t lo = (uint64_t)a.vocab * blockIdx.x / a.fill_blocks,
                 hi = (uint64_t)a.vocab * (blockIdx.x + 1) / a.fill_blocks;
  constexpr int kTokens = 16;  // of a thread, on their way at once
  for (int64_t t0 = threadIdx.x; t0 < a.rows; t0 += kTokens * kThreads) {
    uint64_t v[kTokens];
#pragma unroll
    for (int u = 0; u < kTokens; ++u) {
      const int64_t t = t0 + u * kThreads;
      v[u] = t < a.rows ? __ldcg(reinterpret_cast<const unsigned long long*>(a.tokens) + t) : hi;
    }
#pragma unroll
    for (int u = 0; u < kTokens; ++u)
      if (v[u] - lo < hi - lo) atomicOr(&sh.met[(v[u] - lo) / 32], 1u << ((v[u] - lo) & 31));
  }
  __syncthreads();
  fill_rows<GT, LAY, ADD>(a, sh.met, (uint32_t)lo, 1, (uint32_t)(hi - lo));
}

// ---- few tokens -------------------------------------------------------------------
// One launch (512 tokens of 1000 x 256: 5.9 us against 13.9 by sorting; 50 of 50257 x
// 768 13.6 against 19; 1000 of 50257 x 512 14.6 against 16.5, about where they meet):
// block b owns rows b, b + B, ... of the table. It picks its tokens from the batch,
// ranks them by row (counting, in order), sums them, 16 a part, and writes its rows
// without tokens. For batches whose tokens a block reads at a glance, and whose rows
// it could sum alone if all went to one of the table's.
constexpr int kFewTokens = 1024;
constexpr int kFewItems = 2048;  // tokens times slabs
struct FewShared {
  uint32_t row[kFewTokens], token[kFewTokens];    // the block's, as they come
  uint32_t sorted_row[kFewTokens], sorted[kFewTokens];
  int begin[kFewTokens + 1];                      // of the runs of one row
  int count, runs;
  uint32_t met[kMetWords];
  float2 parts[kWarps][kLane / 2][32];
};

template <typename T, typename GT, Lay LAY, bool ADD>
__global__ void __launch_bounds__(kThreads, 3)
    few_tokens_kernel(const __grid_constant__ GradArgs a) {
  using R = Reduce<T, GT, LAY, ADD>;
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  __shared__ FewShared sh;
  overlap_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  const uint32_t B = gridDim.x, me = blockIdx.x;
  const bool fill = a.fill_blocks > 0;
  for (int i = tid; i < kMetWords; i += kThreads) sh.met[i] = 0;
  if (tid == 0) sh.count = 0;
  __syncthreads();
  // Its tokens, as they come (they are put in order below).
  for (int t = tid; t < (int)a.rows; t += kThreads) {
    const int64_t v = a.tokens[t];
    if (v >= a.vocab && me == 0) atomicOr(a.err, 4u);
    if (v < 0 || v >= a.vocab || (uint32_t)v % B != me) continue;
    const int at = atomicAdd(&sh.count, 1);
    if (!within(at, at + 1, 0, kFewTokens, a.err)) continue;
    sh.row[at] = (uint32_t)v;
    sh.token[at] = (uint32_t)t;
    const uint32_t i = (uint32_t)v / B;
    if (fill) atomicOr(&sh.met[i / 32], 1u << (i & 31));
  }
  __syncthreads();
  const int n = sh.count;
  // by row, then by token (unique, so that the order they were listed in is nothing)
  for (int j = tid; j < n; j += kThreads) {
    const uint64_t mine = (uint64_t)sh.row[j] << 32 | sh.token[j];
    int place = 0;
    for (int i = 0; i < n; ++i) place += ((uint64_t)sh.row[i] << 32 | sh.token[i]) < mine;
    sh.sorted_row[place] = (uint32_t)(mine >> 32);
    sh.sorted[place] = (uint32_t)mine;
  }
  __syncthreads();
  if (warp == 0) {
    int runs = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      const bool first = i < n && (i == 0 || sh.sorted_row[i] != sh.sorted_row[i - 1]);
      const uint32_t firsts = __ballot_sync(kAll, first);
      if (first) sh.begin[runs + __popc(firsts & ((1u << lane) - 1))] = i;
      runs += __popc(firsts);
    }
    if (lane == 0) {
      sh.begin[runs] = n;
      sh.runs = runs;
    }
  }
  __syncthreads();
  const int runs = sh.runs;
  R r{a, lane, 0, {}, {}};
  // The sum of sorted tokens [from, to).
  auto sum = [&](int from, int to) {
    r.clear();
    for (int i0 = from; i0 < to; i0 += R::kRows) {
      Raw8<T> rows[R::kRows];
#pragma unroll
      for (int u = 0; u < R::kRows; ++u)
        if (i0 + u < to) rows[u] = r.row(sh.sorted[i0 + u]);
#pragma unroll
      for (int u = 0; u < R::kRows; ++u)
        if (i0 + u < to) r.add(rows[u]);
    }
  };
  // Rows of a part, a warp to a slab each.
  for (int u = warp; u < runs * a.slabs; u += kWarps) {
    const int run = u / a.slabs, from = sh.begin[run], to = sh.begin[run + 1];
    if (to - from > kEach) continue;
    r.col0 = (u - run * a.slabs) * kSlab;
    const uint32_t v = sh.sorted_row[from];
    if (ADD) r.base = r.base_of(v);
    sum(from, to);
    r.write(v);
  }
  // Rows of more, the block together: a part a warp, added in order by the first.
  for (int run = 0; run < runs; ++run) {
    const int from = sh.begin[run], to = sh.begin[run + 1];
    if (to - from <= kEach) continue;
    const uint32_t v = sh.sorted_row[from];
    for (int slab = 0; slab < a.slabs; ++slab) {
      r.col0 = slab * kSlab;
      float2 total[kLane / 2] = {};
      for (int p0 = from; p0 < to; p0 += kWarps * kEach) {
        const int p = p0 + warp * kEach;
        if (p < to) {
          sum(p, min(to, p + kEach));
          r.keep(sh.parts[warp]);
        }
        __syncthreads();
        if (warp == 0) {
#pragma unroll
          for (int i = 0; i < kLane / 2; ++i) r.acc[i] = total[i];
          for (int w = 0; w < kWarps && p0 + w * kEach < to; ++w) r.add_kept(sh.parts[w]);
#pragma unroll
          for (int i = 0; i < kLane / 2; ++i) total[i] = r.acc[i];
        }
        __syncthreads();
      }
      if (warp == 0) {
        if (ADD) r.base = r.base_of(v);
        r.write(v);
      }
    }
  }
  if (fill) fill_rows<GT, LAY, ADD>(a, sh.met, me, B, (a.vocab - 1 - me) / B + 1);
}

template <typename TT, typename OT>
cudaError_t launch_lookup(const LookupArgs& a, bool vec, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.rows + kWarps - 1) / kWarps),
                  (unsigned)((a.dim + kAtOnce * kSlab - 1) / (kAtOnce * kSlab)));
  return vec ? launch_kernel(embedding_kernel<TT, OT, kEight>, grid, dim3(kThreads), 0, stream, a)
             : launch_kernel(embedding_kernel<TT, OT, kOne>, grid, dim3(kThreads), 0, stream, a);
}

template <typename T, typename GT, Lay LAY>
cudaError_t launch_sums(const SortArgs& k, GradArgs a, cudaStream_t stream) {
  // Blocks that write rows: 304, or up to 1216 where a block's rows are many bytes (of
  // writing and reading) for the 8 a token that it looks through. 304 / 1216: 16384 tokens
  // of 151936 x 2048 bf16 112 / 106 us, 2048 of 32000 x 4096 fp32 added to another 182 /
  // 162; but 8191 of 50257 x 768 bf16 added 34.5 / 38.4, 32768 of 32000 x 2048 fp32 73 / 80.
  const int64_t fill = a.add == a.d_table ? 0 : (a.vocab + kWarps - 1) / kWarps;
  int64_t most = kMostFillBlocks;
  if (k.rows > 0) {
    const int64_t bytes = (int64_t)a.vocab * a.dim * (int)sizeof(GT) * (a.add ? 2 : 1);
    const int64_t worth = bytes / (4 * 8 * k.rows);
    most = worth < kFillBlocks ? kFillBlocks : worth < most ? worth : most;
  }
  a.fill_blocks = (int32_t)(fill < most ? fill : most);
  if (k.rows == 0 && !fill) return cudaSuccess;
  if (k.rows > 0 && k.rows <= kFewTokens && k.rows * a.slabs <= kFewItems) {
    // as many blocks as there are rows for their warps, or tokens
    const int64_t work = fill ? a.fill_blocks : k.rows < kFillBlocks ? k.rows : kFillBlocks;
    return launch_kernel(a.add ? few_tokens_kernel<T, GT, LAY, true>
                               : few_tokens_kernel<T, GT, LAY, false>,
                         dim3((unsigned)work), dim3(kThreads), 0, stream, a);
  }
  if (k.rows > 0) {
    const int smem = (int)sizeof(SortShared) + (kSortWarps * (int)sizeof(uint32_t) << k.bits);
    cudaError_t e = cudaFuncSetAttribute(sort_tokens_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(SortShared) +
                                             kSortWarps * kMaxDigits * (int)sizeof(uint32_t));
    if (e == cudaSuccess)
      e = launch_kernel(sort_tokens_kernel, dim3(kSortBlocks), dim3(kSortThreads), smem, stream,
                        k);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(a.add ? embedding_grad_kernel<T, GT, LAY, true>
                             : embedding_grad_kernel<T, GT, LAY, false>,
                       dim3((unsigned)(a.fill_blocks + (k.rows > 0 ? a.blocks * a.slabs : 0))),
                       dim3(kThreads), 0, stream, a);
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
  a.once = in.rows * in.dim * (in.dtype == ZS_BF16 ? 2 : 4) > kKeptOutput;
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
  a.tokens = in.tokens;
  SortArgs k = {};
  k.rows = in.rows;
  k.err = a.err;
  k.bits = 1;
  if (in.rows > 0) {
    k.tokens = in.tokens;
    k.keys = reinterpret_cast<uint32_t*>(ws + s.keys);
    k.order = reinterpret_cast<uint32_t*>(ws + s.order);
    k.keys2 = reinterpret_cast<uint32_t*>(ws + s.keys2);
    k.order2 = reinterpret_cast<uint32_t*>(ws + s.order2);
    k.tickets = reinterpret_cast<uint32_t*>(ws + s.tickets);
    k.n_tickets = s.n_tickets;
    constexpr int64_t kAllWarps = kSortBlocks * kSortWarps;
    k.share = ((in.rows + kAllWarps - 1) / kAllWarps + 31) / 32 * 32;
    k.vocab = a.vocab;
    int bits = 1;
    while (in.vocab >> bits) ++bits;  // keys 0..vocab
    k.passes = (bits + 9) / 10;
    k.bits = (bits + k.passes - 1) / k.passes;
    a.keys = k.keys;
    a.order = k.order;
    a.tickets = k.tickets;
    a.parts = reinterpret_cast<float*>(ws + s.parts);
  }
  const bool br = in.dtype == ZS_BF16, bt = in.table_dtype == ZS_BF16;
  const bool vec = rows_aligned(a.d_out, a.row_stride, br ? 2 : 4) &&
                   rows_aligned(a.d_table, a.table_stride, bt ? 2 : 4) &&
                   rows_aligned(a.add, a.table_stride, bt ? 2 : 4);
  if (br) {
    if (bt)
      return vec ? launch_sums<__nv_bfloat16, __nv_bfloat16, kEight>(k, a, stream)
                 : launch_sums<__nv_bfloat16, __nv_bfloat16, kOne>(k, a, stream);
    return vec ? launch_sums<__nv_bfloat16, float, kEight>(k, a, stream)
               : launch_sums<__nv_bfloat16, float, kOne>(k, a, stream);
  }
  if (bt)
    return vec ? launch_sums<float, __nv_bfloat16, kEight>(k, a, stream)
               : launch_sums<float, __nv_bfloat16, kOne>(k, a, stream);
  return vec ? launch_sums<float, float, kEight>(k, a, stream)
             : launch_sums<float, float, kOne>(k, a, stream);
}

}  // namespace zs
