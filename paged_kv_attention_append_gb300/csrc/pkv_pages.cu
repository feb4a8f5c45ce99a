// Pages of the cache: copies of whole blocks, and the bookkeeping of block tables and
// reference counts (fork, free, reserve with copy-on-write, compaction).
//
// A block is free iff its count is 0, and free blocks are handed out from the lowest id
// up.  So every result is a function of the inputs alone: ranks come from prefix sums
// over the counts (segments of 4096 ids: one kernel counts, the next one adds up the
// segments before its own and ranks its ids), and the only atomics are sums, whose
// order does not matter.
//
// The bookkeeping is bound by latency: a few hundred KB of counts and tables, one or
// two launches a call, the second one launched while the first runs (programmatic
// dependent launch).  Copies are bound by HBM.
#include <cuda_runtime.h>

#include <algorithm>

#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kSegIds = 4096;               // block ids a CTA ranks
constexpr int kSegPer = kSegIds / kThreads;  // ids of a thread, consecutive
constexpr int kRowThreads = 1024;           // the CTA of reserve that goes over the rows

__device__ __forceinline__ int32_t used_blocks(int32_t ctx, int32_t width) {
  return ctx <= 0 ? 0 : min((ctx - 1) / kBlockSize + 1, width);
}

// Sum over the CTA's threads, returned to every thread.  s: one int per warp.
__device__ __forceinline__ int32_t cta_sum(int32_t v, int32_t *s) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  int32_t t = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) t += s[w];
  return t;
}

// Sum of v over the threads before this one; `total` over all of them.
__device__ __forceinline__ int32_t cta_scan(int32_t v, int32_t *s, int32_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s[warp] = x;
  __syncthreads();
  int32_t before = 0;
  total = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
    if (w < warp) before += s[w];
    total += s[w];
  }
  return before + x - v;
}

// ---------------------------------------------------------------- copies
//
// The arrays' rows are cut into units of 4 KB (8 vectors of 16 bytes a lane, all loads
// in flight before the first store; 1 KB where an array allows 4-byte accesses only),
// one warp a unit, units of a pair next to each other.

struct CopyParams {
  void *data[PKV_COPY_ARRAYS];
  int64_t row_bytes[PKV_COPY_ARRAYS];
  int32_t unit_end[PKV_COPY_ARRAYS];  // units of a pair in the arrays up to this one
  uint32_t narrow[PKV_COPY_ARRAYS / 32];
  int32_t num_arrays, num_blocks, num_pairs;
  const int32_t *src, *dst, *num_pairs_dev;
  int32_t *dev_status;
};
constexpr int kCopyVecs = 8;

template <typename V>
__device__ __forceinline__ void copy_unit(char *data, int64_t row_bytes, int32_t src, int32_t dst,
                                          int64_t at, int lane) {
  const char *s = data + src * row_bytes;
  char *d = data + dst * row_bytes;
  V v[kCopyVecs];
  const int64_t first = at + lane * (int)sizeof(V);
#pragma unroll
  for (int u = 0; u < kCopyVecs; ++u) {
    const int64_t o = first + u * 32 * (int)sizeof(V);
    if (o < row_bytes) v[u] = __ldg(reinterpret_cast<const V *>(s + o));
  }
#pragma unroll
  for (int u = 0; u < kCopyVecs; ++u) {
    const int64_t o = first + u * 32 * (int)sizeof(V);
    if (o < row_bytes) *reinterpret_cast<V *>(d + o) = v[u];
  }
}

__global__ void __launch_bounds__(kThreads) copy_blocks_kernel(const __grid_constant__ CopyParams p) {
  const int lane = threadIdx.x & 31;
  const int32_t per_pair = p.unit_end[p.num_arrays - 1];
  const int32_t pairs =
      p.num_pairs_dev ? min(max(__ldg(p.num_pairs_dev), 0), p.num_pairs) : p.num_pairs;
  // this warp's unit (pair, rem), then every `stride`-th one
  const int64_t stride = (int64_t)gridDim.x * (kThreads / 32);
  const int64_t first = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t step_pair = stride / per_pair;
  const int32_t step_rem = (int32_t)(stride - step_pair * per_pair);
  int64_t pair = first / per_pair;
  int32_t rem = (int32_t)(first - pair * per_pair);
  while (pair < pairs) {
    const int32_t s = __ldg(p.src + pair), d = __ldg(p.dst + pair);
    if (s >= p.num_blocks || d >= p.num_blocks) {
      if (s >= 0 && d >= 0 && rem == 0 && lane == 0) report(p.dev_status, PKV_DEV_BAD_BLOCK);
    } else if (s >= 0 && d >= 0) {
      int lo = 0, hi = p.num_arrays - 1;  // the array whose units hold rem
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (rem < p.unit_end[mid]) hi = mid; else lo = mid + 1;
      }
      const int64_t unit = rem - (lo ? p.unit_end[lo - 1] : 0);
      char *data = static_cast<char *>(p.data[lo]);
      if ((p.narrow[lo >> 5] >> (lo & 31)) & 1u)
        copy_unit<uint32_t>(data, p.row_bytes[lo], s, d, unit * (kCopyVecs * 32 * 4), lane);
      else
        copy_unit<uint4>(data, p.row_bytes[lo], s, d, unit * (kCopyVecs * 32 * 16), lane);
    }
    pair += step_pair;
    rem += step_rem;
    if (rem >= per_pair) {
      rem -= per_pair;
      ++pair;
    }
  }
}

// ---------------------------------------------------------------- fork, free

constexpr int kForkCols = 4 * kThreads;  // table columns of one CTA

// CTAs (row, column range): the new rows' copies first, then the old rows' counts.  An
// old row with c children changes its blocks' counts by c (less one when it ends), one
// atomic an entry and none when c = 1 and the row ends, beam search's usual case.
__global__ void __launch_bounds__(kThreads)
    fork_kernel(const int32_t *__restrict__ parents, int32_t num_new,
                const int32_t *__restrict__ tables, const int32_t *__restrict__ ctx_lens,
                int32_t num_rows, int32_t width, int32_t col_ctas, int32_t *__restrict__ refs,
                int32_t num_blocks, int32_t keep_parents, int32_t *__restrict__ new_tables,
                int32_t *__restrict__ new_ctx, int32_t *dev_status) {
  __shared__ int32_t s_sum[kThreads / 32];
  const int64_t row = blockIdx.x / col_ctas;
  const int32_t col0 = (int32_t)(blockIdx.x % col_ctas) * kForkCols;
  if (row < num_new) {
    const int32_t p = __ldg(parents + row);
    int32_t ctx = 0;
    if (p >= num_rows) {
      if (col0 == 0 && threadIdx.x == 0) report(dev_status, PKV_DEV_BAD_ROW);
    } else if (p >= 0) {
      ctx = max(__ldg(ctx_lens + p), 0);
    }
    if (col0 == 0 && threadIdx.x == 0) new_ctx[row] = ctx;
    const int32_t used = used_blocks(ctx, width);
    const int32_t end = min(used, col0 + kForkCols);
    for (int32_t j = col0 + threadIdx.x; j < end; j += kThreads)
      new_tables[row * width + j] = __ldg(tables + (int64_t)p * width + j);
    return;
  }
  const int64_t old = row - num_new;
  const int32_t used = used_blocks(__ldg(ctx_lens + old), width);
  if (col0 >= used) return;
  int32_t mine = 0;
  for (int32_t i = threadIdx.x; i < num_new; i += kThreads) mine += __ldg(parents + i) == old;
  const int32_t delta = cta_sum(mine, s_sum) - (keep_parents ? 0 : 1);
  const int32_t end = min(used, col0 + kForkCols);
  for (int32_t j = col0 + threadIdx.x; j < end; j += kThreads) {
    const int32_t b = __ldg(tables + old * width + j);
    if (b < 0 || b >= num_blocks)
      report(dev_status, PKV_DEV_BAD_BLOCK);
    else if (delta != 0 && atomicAdd(refs + b, delta) + delta < 0)
      report(dev_status, PKV_DEV_BAD_COUNT);
  }
}

// One CTA a listed row: the first to take its length (an exchange) frees it, another
// listing of the row finds it empty.
constexpr int kFreeThreads = 512;
__global__ void __launch_bounds__(kFreeThreads)
    free_kernel(const int32_t *__restrict__ rows, const int32_t *__restrict__ tables,
                int32_t *__restrict__ ctx_lens, int32_t num_rows, int32_t width,
                int32_t *__restrict__ refs, int32_t num_blocks, int32_t *dev_status) {
  __shared__ int32_t s_ctx;
  const int64_t row = __ldg(rows + blockIdx.x);
  if (row < 0) return;
  if (row >= num_rows) {
    if (threadIdx.x == 0) report(dev_status, PKV_DEV_BAD_ROW);
    return;
  }
  if (threadIdx.x == 0) s_ctx = atomicExch(ctx_lens + row, 0);
  __syncthreads();
  const int32_t used = used_blocks(s_ctx, width);
  const int32_t *entries = tables + row * width;
#pragma unroll 4
  for (int32_t j = threadIdx.x; j < used; j += kFreeThreads) {
    const int32_t b = __ldg(entries + j);
    if (b < 0 || b >= num_blocks) {
      report(dev_status, PKV_DEV_BAD_BLOCK);
    } else if (atomicSub(refs + b, 1) <= 0) {
      atomicAdd(refs + b, 1);
      report(dev_status, PKV_DEV_BAD_COUNT);
    }
  }
}

// ---------------------------------------------------------------- segments

// Blocks in use of this thread's kSegPer ids (bit u: id0 + u has a count), ids past the
// pool as used when `past` says so.
__device__ __forceinline__ uint32_t load_used(const int32_t *refs, int64_t id0, int32_t num_blocks,
                                              bool past) {
  uint32_t bits = 0;
  if (id0 + kSegPer <= num_blocks && (reinterpret_cast<uintptr_t>(refs) & 15u) == 0) {
    int4 v[kSegPer / 4];
#pragma unroll
    for (int u = 0; u < kSegPer / 4; ++u) v[u] = *reinterpret_cast<const int4 *>(refs + id0 + 4 * u);
#pragma unroll
    for (int u = 0; u < kSegPer / 4; ++u)
      bits |= ((uint32_t)(v[u].x != 0) | (uint32_t)(v[u].y != 0) << 1 | (uint32_t)(v[u].z != 0) << 2 |
               (uint32_t)(v[u].w != 0) << 3)
              << (4 * u);
  } else {
#pragma unroll
    for (int u = 0; u < kSegPer; ++u) {
      const bool in = id0 + u < num_blocks;
      bits |= (uint32_t)(in ? refs[id0 + u] != 0 : past) << u;
    }
  }
  return bits;
}

// Counts of the segments before `seg` and of all, to every thread.
__device__ __forceinline__ void sum_segments(const int32_t *counts, int32_t num_segs, int32_t seg,
                                             int32_t *s_sum, int32_t &before, int32_t &total) {
  int32_t b = 0, t = 0;
  for (int32_t i = threadIdx.x; i < num_segs; i += blockDim.x) {
    const int32_t c = counts[i];
    t += c;
    if (i < seg) b += c;
  }
  before = cta_sum(b, s_sum);
  total = cta_sum(t, s_sum);
}

// Blocks in use of each segment (compaction's first kernel).
__global__ void __launch_bounds__(kThreads)
    count_used_kernel(const int32_t *__restrict__ refs, int32_t num_blocks,
                      int32_t *__restrict__ counts) {
  __shared__ int32_t s_sum[kThreads / 32];
  pdl_trigger();
  const int64_t id0 = (int64_t)blockIdx.x * kSegIds + threadIdx.x * kSegPer;
  const int32_t n = cta_sum(__popc(load_used(refs, id0, num_blocks, false)), s_sum);
  if (threadIdx.x == 0) counts[blockIdx.x] = n;
}

// ---------------------------------------------------------------- reserve

// What the first kernel finds for a row (16 bytes) ahead of any change.
struct RowPlan {
  int32_t ctx, n;      // old length, new tokens
  int32_t first;       // first table column that takes a new block
  int32_t old_block;   // >= 0: that column's block is shared; its new one gets a copy
};
struct ReserveHead {
  int32_t demand;      // new blocks of the step; -1: tables or pool too small; -2: a block
                       // outside the pool; -3: counts that do not fit the tables
  int32_t pad[3];
};

struct ReserveParams {
  const int32_t *cu_new;
  int32_t *tables, *ctx_lens, *refs, *slots, *copy_src, *copy_dst;
  int32_t num_rows, width, num_blocks, num_tokens, num_segs, hash_size;
  ReserveHead *head;
  int32_t *seg_free;   // [num_segs]
  int32_t *row_base;   // [num_rows]: new blocks of the rows before
  RowPlan *row_plan;   // [num_rows]
  int32_t *dev_status;
};

// CTA 0 goes over the rows; the others count the free blocks of 4096 ids each.
// Who copies: of the rows that write into a partly filled shared block all do, unless
// they are all its holders: then the last one keeps it.  Their number and the last of
// them come from a hash table in shared memory (block, writers, last writer).
__global__ void __launch_bounds__(kRowThreads) reserve_rows_kernel(const ReserveParams p) {
  extern __shared__ int32_t s_hash[];  // [3][hash_size]
  __shared__ int32_t s_sum[kRowThreads / 32];
  __shared__ int32_t s_fail;
  pdl_trigger();
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    // four segments a CTA
    const int64_t seg = (int64_t)(blockIdx.x - 1) * (kRowThreads / kThreads) + tid / kThreads;
    const int64_t id0 = seg * kSegIds + (tid % kThreads) * kSegPer;
    const int32_t n = kSegPer - __popc(load_used(p.refs, id0, p.num_blocks, true));
    const int32_t w = __reduce_add_sync(0xffffffffu, n);
    if ((tid & 31) == 0) s_sum[tid >> 5] = w;
    __syncthreads();
    if (tid % kThreads == 0 && seg < p.num_segs) {
      int32_t t = 0;
      for (int u = 0; u < kThreads / 32; ++u) t += s_sum[tid / 32 + u];
      p.seg_free[seg] = t;
    }
    return;
  }
  int32_t *key = s_hash, *writers = s_hash + p.hash_size, *last = s_hash + 2 * p.hash_size;
  for (int i = tid; i < p.hash_size; i += kRowThreads) {
    key[i] = -1;
    writers[i] = 0;
    last[i] = -1;
  }
  if (tid == 0) s_fail = 0;
  __syncthreads();
  const uint32_t mask = (uint32_t)p.hash_size - 1;  // a power of two, twice the rows or more
  // the row's partly filled last block where other rows hold it too, else -1
  auto shared_part = [&](int32_t ctx, int32_t n, int64_t r, int32_t &refs) -> int32_t {
    if (n <= 0 || ctx % kBlockSize == 0 || ctx / kBlockSize >= p.width) return -1;
    const int32_t b = p.tables[r * p.width + ctx / kBlockSize];
    if (b < 0 || b >= p.num_blocks) {
      atomicMin(&s_fail, -2);
      return -1;
    }
    refs = p.refs[b];
    if (refs < 1) atomicMin(&s_fail, -3);
    return refs > 1 ? b : -1;
  };
  for (int32_t r = tid; r < p.num_rows; r += kRowThreads) {
    int32_t refs;
    const int32_t b = shared_part(max(p.ctx_lens[r], 0), __ldg(p.cu_new + r + 1) - __ldg(p.cu_new + r),
                                  r, refs);
    if (b < 0) continue;
    uint32_t h = (uint32_t)b * 2654435761u & mask;
    while (true) {  // ends: fewer keys than places
      const int32_t was = atomicCAS(key + h, -1, b);
      if (was == -1 || was == b) break;
      h = (h + 1) & mask;
    }
    atomicAdd(writers + h, 1);
    atomicMax(last + h, r);
  }
  __syncthreads();
  int32_t done = 0;  // new blocks of the rows so far
  for (int32_t r0 = 0; r0 < p.num_rows; r0 += kRowThreads) {
    const int32_t r = r0 + tid;
    int32_t need = 0;
    if (r < p.num_rows) {
      RowPlan pl;
      pl.ctx = max(p.ctx_lens[r], 0);
      pl.n = max(__ldg(p.cu_new + r + 1) - __ldg(p.cu_new + r), 0);
      pl.first = pl.ctx <= 0 ? 0 : (pl.ctx - 1) / kBlockSize + 1;
      pl.old_block = -1;
      int32_t refs;
      const int32_t b = shared_part(pl.ctx, pl.n, r, refs);
      if (b >= 0) {
        uint32_t h = (uint32_t)b * 2654435761u & mask;
        while (key[h] != b) h = (h + 1) & mask;
        if (writers[h] > refs) atomicMin(&s_fail, -3);
        if (writers[h] < refs || last[h] != r) {
          pl.old_block = b;
          --pl.first;
        }
      }
      if (pl.n > 0) {
        const int64_t end = ((int64_t)pl.ctx + pl.n - 1) / kBlockSize + 1;
        if (end > p.width || end - pl.first > p.num_blocks) atomicMin(&s_fail, -1);
        else need = (int32_t)end - pl.first;
      }
      p.row_plan[r] = pl;
    }
    // (in 128s first: the sum itself may pass 32 bits where the pool is far too small)
    if (cta_sum(need >> 7, s_sum) > p.num_blocks >> 7 || done > p.num_blocks) {
      if (tid == 0) atomicMin(&s_fail, -1);
      break;
    }
    int32_t total;
    const int32_t before = cta_scan(need, s_sum, total);
    if (r < p.num_rows) p.row_base[r] = done + before;
    done += total;
  }
  __syncthreads();
  if (tid == 0) p.head->demand = s_fail < 0 ? s_fail : done;
}

// The free id of rank k goes to the row whose range of new blocks holds k; its thread
// writes everything that follows from it.  What does not depend on new blocks is done
// row by row, by all CTAs together.
__global__ void __launch_bounds__(kThreads) reserve_assign_kernel(const ReserveParams p) {
  __shared__ int32_t s_sum[kThreads / 32];
  pdl_wait();
  const int tid = threadIdx.x;
  const int32_t demand = p.head->demand;
  int32_t before, total;
  sum_segments(p.seg_free, p.num_segs, blockIdx.x, s_sum, before, total);
  const int64_t gtid = (int64_t)blockIdx.x * kThreads + tid, threads = (int64_t)gridDim.x * kThreads;
  if (demand < 0 || demand > total) {
    for (int64_t i = gtid; i < p.num_tokens; i += threads) p.slots[i] = -1;
    for (int64_t r = gtid; r < p.num_rows; r += threads) p.copy_src[r] = p.copy_dst[r] = -1;
    if (gtid == 0)
      report(p.dev_status, demand == -2   ? PKV_DEV_BAD_BLOCK
                           : demand == -3 ? PKV_DEV_BAD_COUNT
                                          : PKV_DEV_NO_BLOCKS);
    return;
  }
  const int64_t id0 = (int64_t)blockIdx.x * kSegIds + tid * kSegPer;
  uint32_t free_ids = 0;
  if (before < demand) free_ids = ~load_used(p.refs, id0, p.num_blocks, true) & ((1u << kSegPer) - 1);
  int32_t dummy;
  int32_t rank = before + cta_scan(__popc(free_ids), s_sum, dummy);
  while (free_ids && rank < demand) {
    const int32_t id = (int32_t)id0 + __ffs(free_ids) - 1;
    free_ids &= free_ids - 1;
    int32_t lo = 0, hi = p.num_rows - 1;  // the last row whose base is <= rank
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) >> 1;
      if (p.row_base[mid] <= rank) lo = mid; else hi = mid - 1;
    }
    const RowPlan pl = p.row_plan[lo];
    const int32_t j = rank - p.row_base[lo], col = pl.first + j;
    p.tables[(int64_t)lo * p.width + col] = id;
    p.refs[id] = 1;
    if (j == 0 && pl.old_block >= 0) p.copy_dst[lo] = id;
    const int32_t c0 = __ldg(p.cu_new + lo);
    const int32_t a = max(pl.ctx, col * kBlockSize);
    const int32_t e = (int32_t)min((int64_t)pl.ctx + pl.n, (int64_t)(col + 1) * kBlockSize);
    for (int32_t pos = a; pos < e; ++pos) {
      const int64_t t = (int64_t)c0 + pos - pl.ctx;
      if (t >= 0 && t < p.num_tokens) p.slots[t] = id * kBlockSize + pos % kBlockSize;
    }
    ++rank;
  }
  for (int64_t r = gtid; r < p.num_rows; r += threads) {
    const RowPlan pl = p.row_plan[r];
    p.copy_src[r] = pl.old_block;
    if (pl.old_block < 0) p.copy_dst[r] = -1;
    else atomicSub(p.refs + pl.old_block, 1);
    if (pl.n <= 0) continue;
    p.ctx_lens[r] = pl.ctx + pl.n;
    if (pl.old_block < 0 && pl.ctx % kBlockSize != 0) {  // slots in the block it goes on filling
      const int32_t b = p.tables[r * p.width + pl.ctx / kBlockSize];
      const int32_t c0 = __ldg(p.cu_new + r);
      const int32_t room = min(pl.n, kBlockSize - pl.ctx % kBlockSize);
      for (int32_t i = 0; i < room; ++i) {
        const int64_t t = (int64_t)c0 + i;
        if (t >= 0 && t < p.num_tokens) p.slots[t] = b * kBlockSize + pl.ctx % kBlockSize + i;
      }
    }
  }
}

// ---------------------------------------------------------------- compact

struct CompactParams {
  const int32_t *tables, *ctx_lens, *refs;
  int32_t *new_tables, *new_refs, *copy_src, *copy_dst, *num_pairs;
  int32_t num_rows, width, num_blocks, num_pairs_max, num_segs;
  int32_t *seg_used;   // [num_segs]
  int32_t *move;       // [num_blocks]: of an id that moves or is moved to, its pair, else -1
  int32_t *pair_ref;   // [num_blocks / 2]: the count that moves
  int32_t *dev_status;
};

// Live ids below L (the number of live blocks): those that stay.
__device__ __forceinline__ int32_t live_below(const CompactParams &p, int32_t L, int32_t *s_sum) {
  const int32_t seg = L / kSegIds;
  int32_t before, total;
  sum_segments(p.seg_used, p.num_segs, seg, s_sum, before, total);
  int32_t n = 0;
  if (seg < p.num_segs) {
    const int64_t id0 = (int64_t)seg * kSegIds + threadIdx.x * kSegPer;
    const uint32_t bits = load_used(p.refs, id0, p.num_blocks, false);
    const int64_t left = L - id0;
    if (left > 0) n = __popc(left >= kSegPer ? bits : bits & ((1u << left) - 1));
  }
  return before + cta_sum(n, s_sum);
}

// The i-th live id past L pairs with the i-th free id below it; each is known to the
// thread that ranks it, so both sides of a pair are written independently.
__global__ void __launch_bounds__(kThreads) compact_pairs_kernel(const CompactParams p) {
  __shared__ int32_t s_sum[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  int32_t before, L;
  sum_segments(p.seg_used, p.num_segs, blockIdx.x, s_sum, before, L);
  const int32_t stay = live_below(p, L, s_sum), pairs = L - stay;
  const int64_t id0 = (int64_t)blockIdx.x * kSegIds + threadIdx.x * kSegPer;
  const uint32_t bits = load_used(p.refs, id0, p.num_blocks, false);
  int32_t dummy;
  int32_t live = before + cta_scan(__popc(bits), s_sum, dummy);  // live ids before this one
#pragma unroll
  for (int u = 0; u < kSegPer; ++u) {
    const int64_t id = id0 + u;
    if (id >= p.num_blocks) break;
    const bool on = (bits >> u) & 1u;
    int32_t m = -1;
    if (id < L && !on) {
      m = (int32_t)id - live;
      p.copy_dst[m] = (int32_t)id;
    } else if (id >= L && on) {
      m = live - stay;
      p.copy_src[m] = (int32_t)id;
      p.pair_ref[m] = p.refs[id];
    }
    p.move[id] = m;
    live += on;
  }
  const int64_t gtid = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (gtid == 0) *p.num_pairs = pairs;
  for (int64_t i = pairs + gtid; i < p.num_pairs_max; i += (int64_t)gridDim.x * kThreads)
    p.copy_src[i] = p.copy_dst[i] = -1;
}

// Tables and counts under the new names, each entry by one thread (so in place, too).
__global__ void __launch_bounds__(kThreads)
    compact_rename_kernel(const CompactParams p, int32_t ref_ctas, int32_t col_ctas) {
  __shared__ int32_t s_sum[kThreads / 32];
  pdl_wait();
  int32_t before, L;
  sum_segments(p.seg_used, p.num_segs, 0, s_sum, before, L);
  if ((int32_t)blockIdx.x < ref_ctas) {
    for (int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x; id < p.num_blocks;
         id += (int64_t)ref_ctas * kThreads) {
      const int32_t m = p.move[id];
      p.new_refs[id] = id >= L ? 0 : m >= 0 ? p.pair_ref[m] : p.refs[id];
    }
    return;
  }
  const int64_t row = (blockIdx.x - ref_ctas) / col_ctas;
  const int32_t col0 = (int32_t)((blockIdx.x - ref_ctas) % col_ctas) * kForkCols;
  const int32_t end = min(used_blocks(__ldg(p.ctx_lens + row), p.width), col0 + kForkCols);
  for (int32_t j = col0 + threadIdx.x; j < end; j += kThreads) {
    int32_t b = p.tables[row * p.width + j];
    if (b < 0 || b >= p.num_blocks) {
      report(p.dev_status, PKV_DEV_BAD_BLOCK);
    } else if (b >= L) {
      const int32_t m = p.move[b];
      if (m >= 0) b = p.copy_dst[m];
      else report(p.dev_status, PKV_DEV_BAD_COUNT);
    }
    p.new_tables[row * p.width + j] = b;
  }
}

int32_t segments(int32_t num_blocks) { return (num_blocks + kSegIds - 1) / kSegIds; }
bool misaligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

// Runs `launches` under the profiling hook of kernel id `which`.
template <typename F>
int profiled(int which, pkv_stream stream, F &&launches) {
  profile_begin(which, stream);
  const cudaError_t e = launches();
  profile_end(which, stream);
  return e != cudaSuccess ? (int)e : (int)cudaGetLastError();
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_copy_blocks(const pkv_block_array *arrays, int32_t num_arrays,
                                      int32_t num_blocks, const int32_t *src, const int32_t *dst,
                                      int32_t num_pairs, const int32_t *num_pairs_dev,
                                      int32_t *dev_status, pkv_stream stream) {
  if (num_arrays < 0 || num_blocks < 0 || num_pairs < 0) return PKV_ERR_SHAPE;
  if (num_arrays == 0 || num_pairs == 0) return PKV_OK;
  if (!arrays || !src || !dst) return PKV_ERR_NULL;
  if (misaligned4(src) || misaligned4(dst) || misaligned4(num_pairs_dev)) return PKV_ERR_ALIGN;
  for (int32_t i = 0; i < num_arrays; ++i) {
    if (!arrays[i].data) return PKV_ERR_NULL;
    if (arrays[i].row_bytes <= 0 || arrays[i].row_bytes % 4 != 0 ||
        arrays[i].row_bytes > (int64_t)1 << 36)
      return PKV_ERR_SHAPE;
    if (misaligned4(arrays[i].data)) return PKV_ERR_ALIGN;
  }
  const cudaError_t pe = prepare_kernel<copy_blocks_kernel>(0);
  if (pe != cudaSuccess) return PKV_ERR_CUDA;
  for (int32_t a0 = 0; a0 < num_arrays; a0 += PKV_COPY_ARRAYS) {
    CopyParams p = {};
    p.num_arrays = std::min(num_arrays - a0, PKV_COPY_ARRAYS);
    int64_t units = 0;
    for (int32_t i = 0; i < p.num_arrays; ++i) {
      const pkv_block_array &a = arrays[a0 + i];
      const bool narrow = a.row_bytes % 16 != 0 || (reinterpret_cast<uintptr_t>(a.data) & 15u);
      const int64_t unit = kCopyVecs * 32 * (narrow ? 4 : 16);
      units += (a.row_bytes + unit - 1) / unit;
      if (units > INT32_MAX / 2) return PKV_ERR_SHAPE;
      p.data[i] = a.data;
      p.row_bytes[i] = a.row_bytes;
      p.unit_end[i] = (int32_t)units;
      if (narrow) p.narrow[i >> 5] |= 1u << (i & 31);
    }
    p.num_blocks = num_blocks;
    p.num_pairs = num_pairs;
    p.src = src;
    p.dst = dst;
    p.num_pairs_dev = num_pairs_dev;
    p.dev_status = dev_status;
    const int64_t ctas = (units * num_pairs + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t cap = 4ll * std::max(device_sm_count(), 1);  // one resident wave
    const int e = profiled(PKV_KERNEL_COPY, stream, [&] {
      return launch_kernel(copy_blocks_kernel, dim3((unsigned)std::min(ctas, cap)), dim3(kThreads), 0,
                           stream, false, p);
    });
    if (e) return PKV_ERR_CUDA;
    count_launches(1);
  }
  return PKV_OK;
}

extern "C" pkv_status pkv_fork_sequences(const int32_t *parents, int32_t num_new,
                                         const int32_t *block_tables, const int32_t *context_lens,
                                         int32_t num_rows, int32_t max_blocks_per_seq,
                                         int32_t *ref_counts, int32_t num_blocks,
                                         int32_t keep_parents, int32_t *new_tables,
                                         int32_t *new_context_lens, int32_t *dev_status,
                                         pkv_stream stream) {
  if (num_new < 0 || num_rows < 0 || max_blocks_per_seq < 0 || num_blocks < 0) return PKV_ERR_SHAPE;
  if (keep_parents != 0 && keep_parents != 1) return PKV_ERR_RANGE;
  if (num_new == 0 && num_rows == 0) return PKV_OK;
  if ((num_new > 0 && (!parents || !new_tables || !new_context_lens)) ||
      (num_rows > 0 && (!block_tables || !context_lens || !ref_counts)))
    return PKV_ERR_NULL;
  if (misaligned4(parents) || misaligned4(block_tables) || misaligned4(context_lens) ||
      misaligned4(ref_counts) || misaligned4(new_tables) || misaligned4(new_context_lens))
    return PKV_ERR_ALIGN;
  if ((num_new > 0 && num_rows > 0) &&
      (new_tables == block_tables || new_context_lens == context_lens))
    return PKV_ERR_SHAPE;
  const int64_t cols = std::max((max_blocks_per_seq + kForkCols - 1) / kForkCols, 1);
  const int64_t ctas = ((int64_t)num_new + num_rows) * cols;
  if (ctas > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  const int e = profiled(PKV_KERNEL_PAGES, stream, [&] {
    return launch_kernel(fork_kernel, dim3((unsigned)ctas), dim3(kThreads), 0, stream, false, parents,
                         num_new, block_tables, context_lens, num_rows, max_blocks_per_seq,
                         (int32_t)cols, ref_counts, num_blocks, keep_parents, new_tables,
                         new_context_lens, dev_status);
  });
  if (e) return PKV_ERR_CUDA;
  count_launches(1);
  return PKV_OK;
}

extern "C" pkv_status pkv_free_sequences(const int32_t *rows, int32_t num_listed,
                                         const int32_t *block_tables, int32_t *context_lens,
                                         int32_t num_rows, int32_t max_blocks_per_seq,
                                         int32_t *ref_counts, int32_t num_blocks,
                                         int32_t *dev_status, pkv_stream stream) {
  if (num_listed < 0 || num_rows < 0 || max_blocks_per_seq < 0 || num_blocks < 0)
    return PKV_ERR_SHAPE;
  if (num_listed == 0) return PKV_OK;
  if (!rows || (num_rows > 0 && (!block_tables || !context_lens || !ref_counts))) return PKV_ERR_NULL;
  if (misaligned4(rows) || misaligned4(block_tables) || misaligned4(context_lens) ||
      misaligned4(ref_counts))
    return PKV_ERR_ALIGN;
  const int e = profiled(PKV_KERNEL_PAGES, stream, [&] {
    return launch_kernel(free_kernel, dim3((unsigned)num_listed), dim3(kFreeThreads), 0, stream, false,
                         rows, block_tables, context_lens, num_rows, max_blocks_per_seq, ref_counts,
                         num_blocks, dev_status);
  });
  if (e) return PKV_ERR_CUDA;
  count_launches(1);
  return PKV_OK;
}

namespace {

// Workspace: [head 16 B][segments][move | row_base][pair_ref | row_plan], each 16-byte
// aligned; one size serves both calls.
struct PagesOffsets {
  int64_t seg, a, b, total;
};
PagesOffsets pages_offsets(int64_t rows, int64_t blocks) {
  PagesOffsets o;
  o.seg = 16;
  o.a = align_up(o.seg + 4 * (blocks / kSegIds + 1), 16);
  o.b = align_up(o.a + 4 * std::max(rows, blocks), 16);
  o.total = align_up(o.b + std::max<int64_t>(16 * rows, 2 * blocks + 4), 16);
  return o;
}

}  // namespace

extern "C" size_t pkv_pages_workspace_size(int32_t num_rows, int32_t num_blocks) {
  return num_rows < 0 || num_blocks < 0 ? 0 : (size_t)pages_offsets(num_rows, num_blocks).total;
}

extern "C" pkv_status pkv_reserve_blocks(const int32_t *cu_new, int32_t *block_tables,
                                         int32_t *context_lens, int32_t num_rows,
                                         int32_t max_blocks_per_seq, int32_t *ref_counts,
                                         int32_t num_blocks, int32_t *slot_mapping,
                                         int32_t num_tokens, int32_t *copy_src, int32_t *copy_dst,
                                         void *workspace, int64_t workspace_bytes,
                                         int32_t *dev_status, pkv_stream stream) {
  if (num_rows < 0 || max_blocks_per_seq < 0 || num_blocks < 0 || num_tokens < 0)
    return PKV_ERR_SHAPE;
  if (num_rows > 8192 || (int64_t)num_blocks * kBlockSize > INT32_MAX ||
      (int64_t)max_blocks_per_seq * kBlockSize > INT32_MAX)
    return PKV_ERR_UNSUPPORTED;
  if (num_rows == 0) return PKV_OK;
  if (!cu_new || !context_lens || !copy_src || !copy_dst || !workspace ||
      (max_blocks_per_seq > 0 && !block_tables) || (num_blocks > 0 && !ref_counts) ||
      (num_tokens > 0 && !slot_mapping))
    return PKV_ERR_NULL;
  if (misaligned4(cu_new) || misaligned4(block_tables) || misaligned4(context_lens) ||
      misaligned4(ref_counts) || misaligned4(slot_mapping) || misaligned4(copy_src) ||
      misaligned4(copy_dst) || (reinterpret_cast<uintptr_t>(workspace) & 15u))
    return PKV_ERR_ALIGN;
  const PagesOffsets o = pages_offsets(num_rows, num_blocks);
  if (workspace_bytes < o.total) return PKV_ERR_WORKSPACE;
  char *w = static_cast<char *>(workspace);
  ReserveParams p;
  p.cu_new = cu_new;
  p.tables = block_tables;
  p.ctx_lens = context_lens;
  p.refs = ref_counts;
  p.slots = slot_mapping;
  p.copy_src = copy_src;
  p.copy_dst = copy_dst;
  p.num_rows = num_rows;
  p.width = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.num_tokens = num_tokens;
  p.num_segs = segments(num_blocks);
  p.hash_size = 64;
  while (p.hash_size < 2 * num_rows) p.hash_size *= 2;
  p.head = reinterpret_cast<ReserveHead *>(w);
  p.seg_free = reinterpret_cast<int32_t *>(w + o.seg);
  p.row_base = reinterpret_cast<int32_t *>(w + o.a);
  p.row_plan = reinterpret_cast<RowPlan *>(w + o.b);
  p.dev_status = dev_status;
  const int smem = 12 * p.hash_size;  // at most 192 KB
  if (prepare_kernel<reserve_rows_kernel>(12 * 16384) != cudaSuccess) return PKV_ERR_CUDA;
  constexpr int kSegsPerCta = kRowThreads / kThreads;
  const int e = profiled(PKV_KERNEL_PAGES, stream, [&] {
    cudaError_t le = launch_kernel(reserve_rows_kernel,
                                   dim3(1 + (p.num_segs + kSegsPerCta - 1) / kSegsPerCta),
                                   dim3(kRowThreads), (size_t)smem, stream, false, p);
    if (le != cudaSuccess) return le;
    return launch_kernel(reserve_assign_kernel, dim3(std::max(p.num_segs, 1)), dim3(kThreads), 0,
                         stream, !profiling_active(), p);
  });
  if (e) return PKV_ERR_CUDA;
  count_launches(2);
  return PKV_OK;
}

extern "C" pkv_status pkv_compact_blocks(const int32_t *block_tables, const int32_t *context_lens,
                                         int32_t num_rows, int32_t max_blocks_per_seq,
                                         const int32_t *ref_counts, int32_t num_blocks,
                                         int32_t *new_tables, int32_t *new_ref_counts,
                                         int32_t *copy_src, int32_t *copy_dst,
                                         int32_t num_pairs_max, int32_t *num_pairs,
                                         void *workspace, int64_t workspace_bytes,
                                         int32_t *dev_status, pkv_stream stream) {
  if (num_rows < 0 || max_blocks_per_seq < 0 || num_blocks < 0 || num_pairs_max < num_blocks / 2)
    return PKV_ERR_SHAPE;
  if (num_blocks > INT32_MAX - 2 * kSegIds) return PKV_ERR_UNSUPPORTED;
  if (num_blocks == 0 && num_pairs_max == 0 && num_rows == 0 && !num_pairs) return PKV_OK;
  if (!num_pairs || !workspace || (num_pairs_max > 0 && (!copy_src || !copy_dst)) ||
      (num_blocks > 0 && (!ref_counts || !new_ref_counts)) ||
      (num_rows > 0 && (!context_lens || (max_blocks_per_seq > 0 && (!block_tables || !new_tables)))))
    return PKV_ERR_NULL;
  if (misaligned4(block_tables) || misaligned4(context_lens) || misaligned4(ref_counts) ||
      misaligned4(new_tables) || misaligned4(new_ref_counts) || misaligned4(copy_src) ||
      misaligned4(copy_dst) || misaligned4(num_pairs) ||
      (reinterpret_cast<uintptr_t>(workspace) & 15u))
    return PKV_ERR_ALIGN;
  const PagesOffsets o = pages_offsets(num_rows, num_blocks);
  if (workspace_bytes < o.total) return PKV_ERR_WORKSPACE;
  char *w = static_cast<char *>(workspace);
  CompactParams p;
  p.tables = block_tables;
  p.ctx_lens = context_lens;
  p.refs = ref_counts;
  p.new_tables = new_tables;
  p.new_refs = new_ref_counts;
  p.copy_src = copy_src;
  p.copy_dst = copy_dst;
  p.num_pairs = num_pairs;
  p.num_rows = num_rows;
  p.width = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.num_pairs_max = num_pairs_max;
  p.num_segs = segments(num_blocks);
  p.seg_used = reinterpret_cast<int32_t *>(w + o.seg);
  p.move = reinterpret_cast<int32_t *>(w + o.a);
  p.pair_ref = reinterpret_cast<int32_t *>(w + o.b);
  p.dev_status = dev_status;
  const int32_t segs = std::max(p.num_segs, 1);
  const int32_t ref_ctas = std::max(std::min((num_blocks + kThreads - 1) / kThreads,
                                             2 * std::max(device_sm_count(), 1)), 1);
  const int64_t cols = std::max((max_blocks_per_seq + kForkCols - 1) / kForkCols, 1);
  const int64_t ctas = ref_ctas + num_rows * cols;
  if (ctas > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  const bool pdl = !profiling_active();
  const int e = profiled(PKV_KERNEL_PAGES, stream, [&] {
    cudaError_t le = launch_kernel(count_used_kernel, dim3(segs), dim3(kThreads), 0, stream, false,
                                   ref_counts, num_blocks, p.seg_used);
    if (le != cudaSuccess) return le;
    le = launch_kernel(compact_pairs_kernel, dim3(segs), dim3(kThreads), 0, stream, pdl, p);
    if (le != cudaSuccess) return le;
    return launch_kernel(compact_rename_kernel, dim3((unsigned)ctas), dim3(kThreads), 0, stream, pdl,
                         p, ref_ctas, (int32_t)cols);
  });
  if (e) return PKV_ERR_CUDA;
  count_launches(3);
  return PKV_OK;
}
