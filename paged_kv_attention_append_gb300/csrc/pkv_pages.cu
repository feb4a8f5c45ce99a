// Pages of the cache: copies of whole blocks, and the bookkeeping of block tables and
// reference counts (fork, free, reserve with copy-on-write, compaction).
//
// A block is free iff its count is 0, and free blocks are handed out from the lowest id
// up.  So every result is a function of the inputs alone: ranks come from prefix sums
// over the counts, and the only atomics are sums, whose order does not matter.
//
// The bookkeeping is bound by latency: a few hundred KB of counts and tables.  Reserve and
// the pairing of compact run as one cluster of up to eight CTAs (one for 4096 ids): each
// counts a range of ids, the counts meet in distributed shared memory, and each ranks its
// range, with a cluster barrier where a second kernel would be launched.  A pool of a
// million blocks takes 32 rounds of that.  Copies are bound by HBM.
//
// Every kernel here may be launched while the one before it ends, and waits for it before
// it touches anything; none but compact's first lets its own dependents launch early.  The
// selection and the attention read lengths ahead of their wait, so a thread that writes some
// makes them visible to the whole GPU (a fence) before its CTA ends.
#include <cuda_runtime.h>

#include <algorithm>

#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int32_t used_blocks(int32_t ctx, int32_t width) {
  return ctx <= 0 ? 0 : min((ctx - 1) / kBlockSize + 1, width);
}

// Sum over the CTA's threads, returned to every thread.  s: one int per warp.
__device__ __forceinline__ int32_t cta_sum(int32_t v, int32_t *s) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return __reduce_add_sync(0xffffffffu, lane < (int)(blockDim.x >> 5) ? s[lane] : 0);
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
  const int32_t w = lane < (int)(blockDim.x >> 5) ? s[lane] : 0;
  total = __reduce_add_sync(0xffffffffu, w);
  return __reduce_add_sync(0xffffffffu, lane < warp ? w : 0) + x - v;
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
  pdl_wait();
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
  pdl_wait();
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
    if (col0 == 0 && threadIdx.x == kThreads - 1) {  // (beside the others' copies)
      new_ctx[row] = ctx;
      __threadfence();
    }
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
  pdl_wait();
  const int64_t row = __ldg(rows + blockIdx.x);
  if (row < 0) return;
  if (row >= num_rows) {
    if (threadIdx.x == 0) report(dev_status, PKV_DEV_BAD_ROW);
    return;
  }
  if (threadIdx.x == 0) s_ctx = atomicExch(ctx_lens + row, 0);
  __syncthreads();
  if (threadIdx.x == kFreeThreads - 1) __threadfence();  // (what came before the barrier, too)
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

// ---------------------------------------------------------------- ranges of ids
//
// CTA `rank` of the cluster (the whole grid) looks after the ids [rank, rank + 1)
// range_ids(..), a multiple of kSegIds, kSegIds of them at a time: kSegPer consecutive ids
// a thread.

constexpr int kMaxRanks = 8;
constexpr int kRankThreads = 1024;
constexpr int kSegPer = 4;
constexpr int kSegIds = kRankThreads * kSegPer;

__device__ __forceinline__ int64_t range_ids(int32_t num_blocks, int32_t ranks) {
  const int64_t per = ((int64_t)num_blocks + ranks - 1) / ranks;
  return (per + kSegIds - 1) / kSegIds * kSegIds;
}

// Blocks in use of the ids [id0, id0 + kSegPer) (bit u: id0 + u has a count); ids past the
// pool as used when `past` says so.
__device__ __forceinline__ uint32_t load_used(const int32_t *refs, int64_t id0, int32_t num_blocks,
                                              bool past) {
  if (id0 + kSegPer <= num_blocks && (reinterpret_cast<uintptr_t>(refs) & 15u) == 0) {
    const int4 v = *reinterpret_cast<const int4 *>(refs + id0);
    return (uint32_t)(v.x != 0) | (uint32_t)(v.y != 0) << 1 | (uint32_t)(v.z != 0) << 2 |
           (uint32_t)(v.w != 0) << 3;
  }
  uint32_t bits = 0;
#pragma unroll
  for (int u = 0; u < kSegPer; ++u)
    bits |= (uint32_t)((id0 + u < num_blocks ? refs[id0 + u] : (int32_t)past) != 0) << u;
  return bits;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// An int of CTA `rank`'s shared memory, at the place `p` has in this one's.
__device__ __forceinline__ int32_t peer_int(const int32_t *p, uint32_t rank) {
  uint32_t a;
  int32_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

template <auto Kern, typename P>
cudaError_t launch_cluster(int smem, pkv_stream stream, bool pdl, const P &p) {
  const int64_t segs = ((int64_t)p.num_blocks + kSegIds - 1) / kSegIds;
  const unsigned ranks = (unsigned)std::min<int64_t>(std::max<int64_t>(segs, 1), kMaxRanks);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(kRankThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, Kern, p);
}

// ---------------------------------------------------------------- reserve

// What the first kernel finds for a row (16 bytes) ahead of any change.
struct RowPlan {
  int32_t ctx, n;      // old length, new tokens
  int32_t first;       // first table column that takes a new block
  int32_t old_block;   // >= 0: that column's block is shared; its new one gets a copy
};
struct ReserveParams {
  const int32_t *cu_new;
  int32_t *tables, *ctx_lens, *refs, *slots, *copy_src, *copy_dst;
  int32_t num_rows, width, num_blocks, num_tokens, hash_size;
  int32_t *row_base;   // [num_rows]: new blocks of the rows before
  RowPlan *row_plan;   // [num_rows]
  int32_t *dev_status;
};

// What the rows need, by all threads of one CTA: row_plan, row_base and the number of new
// blocks (-1: tables or pool too small; -2: a block outside the pool; -3: counts that do not
// fit the tables).  Who copies: of the rows that write into a partly filled shared block all
// do, unless they are all its holders: then the last one keeps it.  Their number and the
// last of them come from a hash table in shared memory (block, writers, last writer).
__device__ __forceinline__ int32_t plan_rows(const ReserveParams &p, int32_t *s_hash, int32_t *s_sum,
                                             int32_t *s_fail) {
  const int tid = threadIdx.x;
  int32_t *key = s_hash, *writers = s_hash + p.hash_size, *last = s_hash + 2 * p.hash_size;
  for (int i = tid; i < p.hash_size; i += kRankThreads) {
    key[i] = -1;
    writers[i] = 0;
    last[i] = -1;
  }
  if (tid == 0) *s_fail = 0;
  __syncthreads();
  const uint32_t mask = (uint32_t)p.hash_size - 1;  // a power of two, twice the rows or more
  struct Row {
    int32_t ctx, n, part, refs;  // part: its partly filled last block where others hold it, else -1
  };
  auto load = [&](int32_t r) {
    Row x;
    x.ctx = max(p.ctx_lens[r], 0);
    x.n = max(__ldg(p.cu_new + r + 1) - __ldg(p.cu_new + r), 0);
    x.part = -1;
    if (x.n > 0 && x.ctx % kBlockSize != 0 && x.ctx / kBlockSize < p.width) {
      const int32_t b = p.tables[(int64_t)r * p.width + x.ctx / kBlockSize];
      if (b < 0 || b >= p.num_blocks) {
        atomicMin(s_fail, -2);
      } else {
        x.refs = p.refs[b];
        if (x.refs < 1) atomicMin(s_fail, -3);
        if (x.refs > 1) x.part = b;
      }
    }
    return x;
  };
  auto insert = [&](int32_t r, const Row &x) {
    if (x.part < 0) return;
    uint32_t h = (uint32_t)x.part * 2654435761u & mask;
    while (true) {  // ends: fewer keys than places
      const int32_t was = atomicCAS(key + h, -1, x.part);
      if (was == -1 || was == x.part) break;
      h = (h + 1) & mask;
    }
    atomicAdd(writers + h, 1);
    atomicMax(last + h, r);
  };
  Row first;  // the first 1024 rows stay in registers
  if (tid < p.num_rows) {
    first = load(tid);
    insert(tid, first);
  }
  for (int32_t r = tid + kRankThreads; r < p.num_rows; r += kRankThreads) insert(r, load(r));
  __syncthreads();
  int32_t done = 0;  // new blocks of the rows so far
  for (int32_t r0 = 0; r0 < p.num_rows; r0 += kRankThreads) {
    const int32_t r = r0 + tid;
    int32_t need = 0;
    if (r < p.num_rows) {
      const Row x = r0 == 0 ? first : load(r);
      RowPlan pl;
      pl.ctx = x.ctx;
      pl.n = x.n;
      pl.first = x.ctx <= 0 ? 0 : (x.ctx - 1) / kBlockSize + 1;
      pl.old_block = -1;
      if (x.part >= 0) {
        uint32_t h = (uint32_t)x.part * 2654435761u & mask;
        while (key[h] != x.part) h = (h + 1) & mask;
        if (writers[h] > x.refs) atomicMin(s_fail, -3);
        if (writers[h] < x.refs || last[h] != r) {
          pl.old_block = x.part;
          --pl.first;
        }
      }
      if (pl.n > 0) {
        const int64_t end = ((int64_t)pl.ctx + pl.n - 1) / kBlockSize + 1;
        if (end > p.width || end - pl.first > p.num_blocks) atomicMin(s_fail, -1);
        else need = (int32_t)end - pl.first;
      }
      p.row_plan[r] = pl;
    }
    // (in 128s first: the sum itself may pass 32 bits where the pool is far too small)
    if (cta_sum(need >> 7, s_sum) > p.num_blocks >> 7 || done > p.num_blocks) {
      if (tid == 0) atomicMin(s_fail, -1);
      break;
    }
    int32_t total;
    const int32_t before = cta_scan(need, s_sum, total);
    if (r < p.num_rows) p.row_base[r] = done + before;
    done += total;
  }
  __syncthreads();
  return *s_fail < 0 ? *s_fail : done;
}

// Every CTA counts the free ids of its range, the first one plans the rows meanwhile; then
// each ranks its free ids: the one of rank k goes to the row whose range of new blocks holds
// k, and the thread that takes it writes everything that follows from it.  What does not
// depend on new blocks is done row by row, by all CTAs together.
__global__ void __launch_bounds__(kRankThreads) reserve_kernel(const ReserveParams p) {
  extern __shared__ int32_t s_mem[];  // plan_rows' hash table, then [kSegIds] free ids and
  int32_t *s_base = s_mem + kSegIds;  // [num_rows] row_base
  __shared__ int32_t s_sum[32], s_fail, s_free, s_demand;
  const int tid = threadIdx.x;
  const int32_t rank = (int32_t)blockIdx.x, ranks = (int32_t)gridDim.x;
  pdl_wait();
  const int64_t range = range_ids(p.num_blocks, ranks), id_lo = rank * range;
  const int64_t id_hi = min(id_lo + range, (int64_t)p.num_blocks);
  int32_t n = 0;
  for (int64_t i = id_lo; i < id_hi; i += kSegIds)
    n += kSegPer - __popc(load_used(p.refs, i + tid * kSegPer, p.num_blocks, true));
  n = cta_sum(n, s_sum);
  const int32_t gtid = rank * kRankThreads + tid, threads = ranks * kRankThreads;
  // slots that are no row's (the padding of a step behind its last row); before the barrier,
  // the rows' own come after it
  const int32_t cu_lo = __ldg(p.cu_new), cu_hi = __ldg(p.cu_new + p.num_rows);
  for (int64_t i = gtid; i < min(cu_lo, p.num_tokens); i += threads) p.slots[i] = -1;
  for (int64_t i = (int64_t)max(cu_hi, 0) + gtid; i < p.num_tokens; i += threads) p.slots[i] = -1;
  int32_t demand = 0;
  if (rank == 0) demand = plan_rows(p, s_mem, s_sum, &s_fail);
  if (tid == 0) {
    s_free = n;
    s_demand = demand;
  }
  cluster_sync();
  demand = peer_int(&s_demand, 0);
  int32_t before = 0, total = 0;
  for (int k = 0; k < ranks; ++k) {
    const int32_t f = peer_int(&s_free, k);
    if (k < rank) before += f;
    total += f;
  }
  cluster_arrive();  // what the others keep for this CTA is read; they wait for it at their end
  if (demand < 0 || demand > total) {
    for (int64_t i = gtid; i < p.num_tokens; i += threads) p.slots[i] = -1;
    for (int32_t r = gtid; r < p.num_rows; r += threads) p.copy_src[r] = p.copy_dst[r] = -1;
    if (gtid == 0)
      report(p.dev_status, demand == -2   ? PKV_DEV_BAD_BLOCK
                           : demand == -3 ? PKV_DEV_BAD_COUNT
                                          : PKV_DEV_NO_BLOCKS);
    cluster_wait();
    return;
  }
  // the lengths, by the threads that have least to do with the ids (the fence takes 0.5 us)
  if (threads - 1 - gtid < p.num_rows) {
    for (int32_t r = threads - 1 - gtid; r < p.num_rows; r += threads) {
      const RowPlan pl = p.row_plan[r];
      if (pl.n > 0) p.ctx_lens[r] = pl.ctx + pl.n;
    }
    __threadfence();
  }
  if (id_lo < id_hi && before < demand)
    for (int32_t r = tid; r < p.num_rows; r += kRankThreads) s_base[r] = p.row_base[r];
  for (int64_t i = id_lo; i < id_hi && before < demand; i += kSegIds) {
    // the free ids of the segment, in order, then an id a thread
    uint32_t bits = ~load_used(p.refs, i + tid * kSegPer, p.num_blocks, true) & ((1u << kSegPer) - 1);
    int32_t found;
    int32_t at = cta_scan(__popc(bits), s_sum, found);
    while (bits) {
      s_mem[at++] = (int32_t)i + tid * kSegPer + __ffs(bits) - 1;
      bits &= bits - 1;
    }
    __syncthreads();
    const int32_t take = min(found, demand - before);
    for (int32_t k = tid; k < take; k += kRankThreads) {
      const int32_t id = s_mem[k], place = before + k;
      int32_t lo = 0, hi = p.num_rows - 1;  // the last row whose base is <= place
      while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (s_base[mid] <= place) lo = mid; else hi = mid - 1;
      }
      const RowPlan pl = p.row_plan[lo];
      const int32_t j = place - s_base[lo], col = pl.first + j;
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
    }
    before += found;
    __syncthreads();
  }
  for (int32_t r = gtid; r < p.num_rows; r += threads) {
    const RowPlan pl = p.row_plan[r];
    p.copy_src[r] = pl.old_block;
    if (pl.old_block < 0) p.copy_dst[r] = -1;
    else atomicSub(p.refs + pl.old_block, 1);
    if (pl.n <= 0) continue;
    if (pl.old_block < 0 && pl.ctx % kBlockSize != 0) {  // slots in the block it goes on filling
      const int32_t b = p.tables[(int64_t)r * p.width + pl.ctx / kBlockSize];
      const int32_t c0 = __ldg(p.cu_new + r);
      const int32_t room = min(pl.n, kBlockSize - pl.ctx % kBlockSize);
      for (int32_t i = 0; i < room; ++i) {
        const int64_t t = (int64_t)c0 + i;
        if (t >= 0 && t < p.num_tokens) p.slots[t] = b * kBlockSize + pl.ctx % kBlockSize + i;
      }
    }
  }
  cluster_wait();
}

// ---------------------------------------------------------------- compact

struct CompactParams {
  const int32_t *tables, *ctx_lens, *refs;
  int32_t *new_tables, *new_refs, *copy_src, *copy_dst, *num_pairs;
  int32_t num_rows, width, num_blocks, num_pairs_max;
  int32_t *live;       // L, the number of blocks in use
  int32_t *move;       // [num_blocks]: of an id that moves or is moved to, its pair, else -1
  int32_t *pair_ref;   // [num_blocks / 2]: the count that moves
  int32_t *dev_status;
};

// The i-th live id past L pairs with the i-th free id below it; each is known to the
// thread that ranks it, so both sides of a pair are written independently.
__global__ void __launch_bounds__(kRankThreads) compact_pairs_kernel(const CompactParams p) {
  __shared__ int32_t s_sum[32], s_live, s_stay;
  const int tid = threadIdx.x;
  const int32_t rank = (int32_t)blockIdx.x, ranks = (int32_t)gridDim.x;
  pdl_wait();
  pdl_trigger();  // the renaming waits for all of this
  const int64_t range = range_ids(p.num_blocks, ranks), id_lo = rank * range;
  const int64_t id_hi = min(id_lo + range, (int64_t)p.num_blocks);
  int32_t n = 0;
  for (int64_t i = id_lo; i < id_hi; i += kSegIds)
    n += __popc(load_used(p.refs, i + tid * kSegPer, p.num_blocks, false));
  n = cta_sum(n, s_sum);
  if (tid == 0) s_live = n;
  cluster_sync();
  int32_t before = 0, L = 0;
  for (int k = 0; k < ranks; ++k) {
    const int32_t f = peer_int(&s_live, k);
    if (k < rank) before += f;
    L += f;
  }
  // live ids below L, which stay
  n = 0;
  for (int64_t i = id_lo; i < min(id_hi, (int64_t)L); i += kSegIds) {
    const int64_t id0 = i + tid * kSegPer, left = L - id0;
    const uint32_t bits = load_used(p.refs, id0, p.num_blocks, false);
    if (left > 0) n += __popc(left >= kSegPer ? bits : bits & ((1u << left) - 1));
  }
  n = cta_sum(n, s_sum);
  if (tid == 0) s_stay = n;
  cluster_sync();
  int32_t stay = 0;
  for (int k = 0; k < ranks; ++k) stay += peer_int(&s_stay, k);
  cluster_arrive();  // (waited for at the end: no CTA ends while others read its counts)
  const int32_t pairs = L - stay;
  int32_t live = before;  // live ids before the segment
  for (int64_t i = id_lo; i < id_hi; i += kSegIds) {
    const int64_t id0 = i + tid * kSegPer;
    const uint32_t bits = load_used(p.refs, id0, p.num_blocks, false);
    int32_t all;
    int32_t mine = live + cta_scan(__popc(bits), s_sum, all);
    live += all;
#pragma unroll
    for (int u = 0; u < kSegPer; ++u) {
      const int64_t id = id0 + u;
      if (id >= p.num_blocks) break;
      const bool on = (bits >> u) & 1u;
      int32_t m = -1;
      if (id < L && !on) {
        m = (int32_t)id - mine;
        p.copy_dst[m] = (int32_t)id;
      } else if (id >= L && on) {
        m = mine - stay;
        p.copy_src[m] = (int32_t)id;
        p.pair_ref[m] = p.refs[id];
      }
      p.move[id] = m;
      mine += on;
    }
  }
  const int32_t gtid = rank * kRankThreads + tid;
  if (gtid == 0) {
    *p.num_pairs = pairs;
    *p.live = L;
  }
  for (int64_t i = pairs + gtid; i < p.num_pairs_max; i += ranks * kRankThreads)
    p.copy_src[i] = p.copy_dst[i] = -1;
  cluster_wait();
}

// Tables and counts under the new names, each entry by one thread (so in place, too).
__global__ void __launch_bounds__(kThreads)
    compact_rename_kernel(const CompactParams p, int32_t ref_ctas, int32_t col_ctas) {
  pdl_wait();
  const int32_t L = *p.live;
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

// CTAs of a row of a table.
int64_t fork_ctas(int32_t width) {
  return std::max<int64_t>(((int64_t)width + kForkCols - 1) / kForkCols, 1);
}

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
                           stream, !profiling_active(), p);
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
  const int64_t cols = fork_ctas(max_blocks_per_seq);
  const int64_t ctas = ((int64_t)num_new + num_rows) * cols;
  if (ctas > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  const int e = profiled(PKV_KERNEL_PAGES, stream, [&] {
    return launch_kernel(fork_kernel, dim3((unsigned)ctas), dim3(kThreads), 0, stream, !profiling_active(), parents,
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
    return launch_kernel(free_kernel, dim3((unsigned)num_listed), dim3(kFreeThreads), 0, stream, !profiling_active(),
                         rows, block_tables, context_lens, num_rows, max_blocks_per_seq, ref_counts,
                         num_blocks, dev_status);
  });
  if (e) return PKV_ERR_CUDA;
  count_launches(1);
  return PKV_OK;
}

namespace {

// Workspace: [L 16 B][move | row_base][pair_ref | row_plan], each 16-byte aligned; one size
// serves both calls.
struct PagesOffsets {
  int64_t a, b, total;
};
PagesOffsets pages_offsets(int64_t rows, int64_t blocks) {
  PagesOffsets o;
  o.a = 16;
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
  p.hash_size = 64;
  while (p.hash_size < 2 * num_rows) p.hash_size *= 2;
  p.row_base = reinterpret_cast<int32_t *>(w + o.a);
  p.row_plan = reinterpret_cast<RowPlan *>(w + o.b);
  p.dev_status = dev_status;
  const int smem = std::max(12 * p.hash_size, 4 * (kSegIds + num_rows));  // 16 to 192 KB
  if (prepare_kernel<reserve_kernel>(12 * 16384) != cudaSuccess) return PKV_ERR_CUDA;
  const int e = profiled(PKV_KERNEL_PAGES, stream,
                         [&] { return launch_cluster<reserve_kernel>(smem, stream, !profiling_active(), p); });
  if (e) return PKV_ERR_CUDA;
  count_launches(1);
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
  if (num_blocks > INT32_MAX / 4) return PKV_ERR_UNSUPPORTED;
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
  p.live = reinterpret_cast<int32_t *>(w);
  p.move = reinterpret_cast<int32_t *>(w + o.a);
  p.pair_ref = reinterpret_cast<int32_t *>(w + o.b);
  p.dev_status = dev_status;
  const int32_t ref_ctas = std::max(std::min((num_blocks + kThreads - 1) / kThreads,
                                             2 * std::max(device_sm_count(), 1)), 1);
  const int64_t cols = fork_ctas(max_blocks_per_seq);
  const int64_t ctas = ref_ctas + num_rows * cols;
  if (ctas > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  const bool pdl = !profiling_active();
  const int e = profiled(PKV_KERNEL_PAGES, stream, [&] {
    const cudaError_t le = launch_cluster<compact_pairs_kernel>(0, stream, pdl, p);
    if (le != cudaSuccess) return le;
    return launch_kernel(compact_rename_kernel, dim3((unsigned)ctas), dim3(kThreads), 0, stream, pdl,
                         p, ref_ctas, (int32_t)cols);
  });
  if (e) return PKV_ERR_CUDA;
  count_launches(2);
  return PKV_OK;
}
