// Attention of each query token over the blocks selected for it and a KV head.
//
//   out[t][hq] = sum_p softmax_p(scale q . K[p]) V[p],  p over the visible keys of the
//   selected blocks.
//
// A CTA of four warps (or two), or a cluster of up to eight such CTAs, takes one (token, KV head):
// the G query heads are the rows of the m16 tiles, so a block is read once for all of
// them.  The selected blocks are dealt out over the warps; each streams its share through
// a ring of its own (TMA boxes of a block's K and V, as the split-KV kernel reads them)
// with an online softmax in registers.  The warps' (m, l, O) meet in shared memory, over
// the cluster through distributed shared memory, each CTA joining a part of the columns:
// one launch, no workspace, and a fixed order of every sum.  (A pair of one CTA is launched
// without clusters: 256 decodes of 64 blocks 84 us for the three calls, with them 89.)
//
// Weights go into the product with V as two bf16 parts, so that the output is as exact as with
// weights of 32 bits (2-norm error 0.0017, all of it the last rounding; with one part 0.0021;
// 24 decodes of 128 blocks 107.2 us for the three calls, 107.0 with one; 61 windows 20.1, 19.0).
//
// Bound: the selected blocks' K and V, 64 D bytes a block and KV head.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pkv_block.cuh"
#include "pkv_device.cuh"
#include "pkv_sparse.cuh"

namespace pkv {

namespace {

struct SparseParams {
  const __nv_bfloat16 *q;
  __nv_bfloat16 *out;
  const int32_t *cu_q_lens, *context_lens, *block_tables, *selected;
  int32_t max_blocks, num_seqs, num_blocks, num_q_heads, hkv, group, num_select;
  float scale_log2;
  int32_t *dev_status;
};

template <int D, int kWarps>
struct SparseCfg {
  static constexpr int kCtasPerSm = 12 / kWarps;
  // 8 KB a warp and stage at D = 128: with two stages three CTAs share an SM, so that the
  // (token, head) pairs of a call spread more evenly (192 pairs of 128 blocks: 38 us; three
  // stages and two CTAs 45)
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kSlabBytes = D / 64 * kBoxBytes;
  static constexpr int kStageBytes = 2 * kSlabBytes;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kRow = D + 8;  // floats of a partial row in shared memory
  static constexpr int kMlOffset = kWarps * kRingBytes;               // [warp][16] (m, l)
  static constexpr int kBarOffset = kMlOffset + kWarps * kRowsPerTile * 8;
  static constexpr int kSmemBytes = kBarOffset + kWarps * kStages * 8 + 1024;
  static_assert(kRowsPerTile * kRow * 4 <= kRingBytes, "a warp's partial fits its ring");
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// All threads of the cluster; shared memory written before it is visible after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// The address, in CTA `rank` of the cluster, of what `addr` is in this one.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

template <int D, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, SparseCfg<D, kWarps>::kCtasPerSm)
    sparse_kernel(const __grid_constant__ CUtensorMap pool_map, const SparseParams p) {
  using C = SparseCfg<D, kWarps>;
  constexpr int kThreads = 32 * kWarps;
  constexpr int kL = D / 32, kNt = D / 8, kStages = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ int32_t s_sum[kWarps];
  // (the same offset in every CTA of a cluster, which map_rank relies on)
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  const int64_t pair = blockIdx.x / ranks;
  const int64_t token = pair / p.hkv;
  const int h = (int)(pair % p.hkv);
  pdl_trigger();
  if (lane == 0) prefetch_tmap(&pool_map);
  uint8_t *ring = smem + warp * C::kRingBytes;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBarOffset) + warp * kStages;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(smem_u32(&bars[s]), 1);
    fence_mbar_init();
  }
  // (the kernels that write lengths make them visible before they let this one be launched)
  const TokenPlace at =
      find_token(p.cu_q_lens, p.context_lens, p.num_seqs, p.max_blocks, token, s_sum);
  pdl_wait();
  uint32_t qa[2 * kL][4];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int row = r + 8 * half;
    const __nv_bfloat16 *q =
        p.q + (token * p.num_q_heads + (int64_t)h * p.group + (row < p.group ? row : 0)) * D;
#pragma unroll
    for (int L = 0; L < kL; ++L) {
      const int e = 8 * (L >> 1) + 2 * c + (L & 1);
      const uint4 v = row < p.group ? ldg128_nc(q + 8 * e) : make_uint4(0, 0, 0, 0);
      qa[2 * L][half] = v.x;
      qa[2 * L][2 + half] = v.y;
      qa[2 * L + 1][half] = v.z;
      qa[2 * L + 1][2 + half] = v.w;
    }
  }
  // (the same for the whole cluster)
  const int32_t own = at.pos / kBlockSize;
  if (at.pos < 0) {
    if (at.seq < p.num_seqs && h == 0 && rank == 0 && threadIdx.x == 0)
      report(p.dev_status, PKV_DEV_PLAN_MISMATCH);
    return;
  }
  const int32_t *sel = p.selected + (token * p.hkv + h) * p.num_select;
  const int32_t *table = p.block_tables + (int64_t)at.seq * p.max_blocks;
  const int deal = kWarps * (int)ranks, first = (int)rank * kWarps + warp;
  const int lim_lo = r < p.group ? at.pos : -1, lim_hi = r + 8 < p.group ? at.pos : -1;
  float o[kNt][4];
#pragma unroll
  for (int nt = 0; nt < kNt; ++nt) o[nt][0] = o[nt][1] = o[nt][2] = o[nt][3] = 0.f;
  float m_lo = -INFINITY, m_hi = -INFINITY, l_lo = 0.f, l_hi = 0.f;
  int issued = 0, done = 0;
  bool good = true;
  // the warp's entries 32 at a time: lane i resolves entry first + (i0 + i) deal
  for (int i0 = 0; good && first + (int64_t)i0 * deal < p.num_select; i0 += 32) {
    const int64_t i = first + (int64_t)(i0 + lane) * deal;
    int32_t block = i < p.num_select ? __ldg(sel + i) : -1;
    if (block > own) block = -1;
    int32_t phys = block >= 0 ? __ldg(table + block) : -1;
    if (block >= 0 && (phys < 0 || phys >= p.num_blocks)) {
      report(p.dev_status, PKV_DEV_BAD_BLOCK);
      phys = -1;
    }
    uint32_t to_issue = __ballot_sync(0xffffffffu, phys >= 0), to_use = to_issue;
    auto issue = [&] {  // the next block of the window into the ring
      const int b = __ffs(to_issue) - 1;
      to_issue &= to_issue - 1;
      const int32_t ph = __shfl_sync(0xffffffffu, phys, b);
      if (lane == 0) {
        const int s = issued % kStages;
        const uint32_t bar = smem_u32(&bars[s]), dst = smem_u32(ring + s * C::kStageBytes);
        mbar_arrive_expect_tx(bar, C::kStageBytes);
        const int row = (int)(((int64_t)ph * 2 * p.hkv + h) * kBlockSize >> 3);
        tma_load_4d(dst, &pool_map, 0, 0, 0, row, bar);
        tma_load_4d(dst + C::kSlabBytes, &pool_map, 0, 0, 0, row + p.hkv * (kBlockSize >> 3), bar);
      }
      ++issued;
    };
    for (int k = 0; k < kStages && to_issue; ++k) issue();
    while (to_use) {
      const int b = __ffs(to_use) - 1;
      to_use &= to_use - 1;
      const int32_t logical = __shfl_sync(0xffffffffu, block, b);
      const int s = done % kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&bars[s]), (uint32_t)(done / kStages & 1)))) {
        if (lane == 0) report(p.dev_status, PKV_DEV_TIMEOUT);
        good = false;
        break;
      }
      ++done;
      const uint32_t sK = smem_u32(ring + s * C::kStageBytes), sV = sK + C::kSlabBytes;
      if (logical == own) {
        // the token's own block: V rows past it weigh 0, but 0 x NaN would not
        const int past = at.pos % kBlockSize + 1;
        for (int x = past * (D / 8) + lane; x < kBlockSize * (D / 8); x += 32)
          asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(
                           sV + blk_off<D / 64>(x / (D / 8), x % (D / 8))),
                       "r"(0)
                       : "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // ahead of the next copy here
        __syncwarp();
      }
      block_update<D, true>(sK, sV, qa, logical * kBlockSize, at.pos, lim_lo, lim_hi, p.scale_log2,
                            r, c, m_lo, m_hi, l_lo, l_hi, o);
      __syncwarp();
      if (to_issue) issue();
    }
  }
  if (lane == 0)  // after a timeout: what is still in flight lands before the CTA ends
    for (int j = done; j < issued; ++j)
      mbar_wait(smem_u32(&bars[j % kStages]), (uint32_t)(j / kStages & 1));
  __syncwarp();
  // the warp's partial, over its ring: lane (r, c) holds of rows r and r + 8 the 16 columns
  // from (8 hh + 2 c) 8 on, in each half hh
  l_lo += __shfl_xor_sync(0xffffffffu, l_lo, 1);
  l_lo += __shfl_xor_sync(0xffffffffu, l_lo, 2);
  l_hi += __shfl_xor_sync(0xffffffffu, l_hi, 1);
  l_hi += __shfl_xor_sync(0xffffffffu, l_hi, 2);
  float *part = reinterpret_cast<float *>(ring);
  float2 *ml = reinterpret_cast<float2 *>(smem + C::kMlOffset) + warp * kRowsPerTile;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int row = r + 8 * half;
    if (row >= p.group) continue;
#pragma unroll
    for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 8; j += 4) {
          float4 v;
          v.x = o[8 * hh + j][2 * half + u];
          v.y = o[8 * hh + j + 1][2 * half + u];
          v.z = o[8 * hh + j + 2][2 * half + u];
          v.w = o[8 * hh + j + 3][2 * half + u];
          *reinterpret_cast<float4 *>(part + row * C::kRow + (8 * hh + 2 * c + u) * 8 + j) = v;
        }
    if (c == 0) ml[row] = half ? make_float2(m_hi, l_hi) : make_float2(m_lo, l_lo);
  }
  if (ranks == 1) __syncthreads();
  else cluster_sync();
  // (row, 4 columns) by thread, over the warps of every CTA of the cluster
  constexpr int kChunks = D / 4;
  for (int x = (int)rank * kThreads + threadIdx.x; x < p.group * kChunks; x += (int)ranks * kThreads) {
    const int row = x / kChunks, ch = x % kChunks;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (uint32_t k = 0; k < ranks; ++k) {
      const uint32_t base = map_rank(smem_u32(smem), k);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = ld_cluster2(base + C::kMlOffset + (w * kRowsPerTile + row) * 8);
        const float4 y = ld_cluster4(base + w * C::kRingBytes + (row * C::kRow + 4 * ch) * 4);
        if (v.x == -INFINITY && v.y == 0.f) continue;  // no visible key in that warp's share
        const float mn = fmaxf(M, v.x);
        const float a = fast_exp2(M - mn), b = fast_exp2(v.x - mn);
        L = L * a + v.y * b;
        acc.x = acc.x * a + y.x * b;
        acc.y = acc.y * a + y.y * b;
        acc.z = acc.z * a + y.z * b;
        acc.w = acc.w * a + y.w * b;
        M = mn;
      }
    }
    const float inv = L > 0.f ? 1.f / L : L == L ? 0.f : L;
    uint2 pk;
    pk.x = pack_bf16x2(acc.x * inv, acc.y * inv);
    pk.y = pack_bf16x2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2 *>(p.out + (token * p.num_q_heads + (int64_t)h * p.group + row) * D +
                               4 * ch) = pk;
  }
  if (ranks > 1) cluster_sync();  // no CTA ends while another reads its shared memory
}

template <int D, int kWarps>
cudaError_t launch_sparse_t(const CUtensorMap &map, const SparseParams &p, int64_t total_q,
                            int ranks, pkv_stream stream) {
  using C = SparseCfg<D, kWarps>;
  const cudaError_t pe = prepare_kernel<sparse_kernel<D, kWarps>>(C::kSmemBytes);
  if (pe != cudaSuccess) return pe;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(total_q * p.hkv * ranks));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (ranks > 1) {  // (without: a cluster of one)
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = (unsigned)ranks;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (!profiling_active()) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, sparse_kernel<D, kWarps>, map, p);
}

template <int D>
cudaError_t launch_sparse(const CUtensorMap &map, const SparseParams &p, int64_t total_q,
                          pkv_stream stream) {
  // CTAs of a (token, KV head): more while there are fewer than two CTAs an SM and every
  // warp would still have two blocks (192 pairs of 128 blocks: two each 38 us, four 42.5; the
  // 8 pairs of one token, 32 blocks: the three calls 11.8 us with four each, 12.2 with
  // eight, 12.8 with two)
  int ranks = 1;
  while (ranks < 8 && total_q * p.hkv * ranks < 2ll * std::max(device_sm_count(), 1) &&
         16 * ranks <= p.num_select)
    ranks *= 2;
  // CTAs of two warps, twice as many of them an SM, where there are more (token, KV head)s than
  // CTAs of four fit at a time: their start and end overlap more.  Few blocks gain most (this call
  // alone at D = 128: 2400 pairs of 8 blocks 38.2 -> 34.6 us, 4000 of 4 48.4 -> 35.2; D = 64: 25.8
  // -> 18.7, 32.6 -> 23.5).  More blocks each gain where the waves come out even (1600 pairs of 28
  // 64.6 -> 61.4 us, 480 of 32 29.2 -> 24.3, 2400 of 48 143.3 -> 140.8); an odd number of waves of
  // four-warp CTAs ends with a wave of two-warp ones that is half empty (1200 of 28 50.0 -> 52.3,
  // 2048 of 32 88.3 -> 90.0), which nine waves no longer feel (4000 of 24: 125 either way, D = 64
  // 78.8 -> 71.9).  2048 of 64 take 81 -> 87 us with the selection.
  constexpr int32_t kFewBlocks = 16, kMostBlocks = 48;
  const int64_t slots = 3ll * std::max(device_sm_count(), 1), pairs = total_q * p.hkv;
  const int64_t waves = (pairs + slots - 1) / slots;
  if (waves > 1 && (p.num_select <= kFewBlocks ||
                    (p.num_select <= kMostBlocks && (waves % 2 == 0 || waves > 8))))
    return launch_sparse_t<D, 2>(map, p, total_q, ranks, stream);
  return launch_sparse_t<D, 4>(map, p, total_q, ranks, stream);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_paged_sparse_attention(
    const void *q, const int32_t *cu_q_lens, const int32_t *context_lens,
    const int32_t *block_tables, int32_t max_blocks_per_seq, int32_t num_seqs, int64_t total_q,
    int32_t num_q_heads, const int32_t *selected, int32_t num_select, const void *kv_pool,
    const pkv_pool_desc *desc, float scale, void *out, int32_t *dev_status, pkv_stream stream) {
  pkv_status st = check_pool(desc);
  if (st != PKV_OK) return st;
  st = check_sparse(desc, max_blocks_per_seq, num_seqs, total_q, num_q_heads, num_select);
  if (st != PKV_OK) return st;
  if (!std::isfinite(scale)) return PKV_ERR_RANGE;
  if (total_q == 0) return PKV_OK;
  if (!q || !cu_q_lens || !context_lens || !block_tables || !selected || !kv_pool || !out)
    return PKV_ERR_NULL;
  if (!aligned16(q) || !aligned16(out) || !aligned16(kv_pool) ||
      (reinterpret_cast<uintptr_t>(selected) & 3u))
    return PKV_ERR_ALIGN;
  CUtensorMap map;
  if (make_pool_map(&map, kv_pool, *desc)) return PKV_ERR_CUDA;
  SparseParams p;
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.cu_q_lens = cu_q_lens;
  p.context_lens = context_lens;
  p.block_tables = block_tables;
  p.selected = selected;
  p.max_blocks = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.num_blocks = desc->num_blocks;
  p.num_q_heads = num_q_heads;
  p.hkv = desc->num_kv_heads;
  p.group = num_q_heads / desc->num_kv_heads;
  p.num_select = num_select;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.dev_status = dev_status;
  profile_begin(PKV_KERNEL_SPARSE, stream);
  cudaError_t e = desc->head_dim == 128 ? launch_sparse<128>(map, p, total_q, stream)
                                        : launch_sparse<64>(map, p, total_q, stream);
  profile_end(PKV_KERNEL_SPARSE, stream);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return PKV_ERR_CUDA;
  count_launches(1);
  return PKV_OK;
}
