// What the split-KV kernels of the bf16 pool (pkv_decode.cu) and of the 8-bit pool
// (pkv_decode8.cu) share: their parameters, made from one attention call's
// arguments, and the partial-result conventions the merge kernel reads.
#pragma once

#include <cuda_bf16.h>

#include <mutex>

#include "pkv_device.cuh"

namespace pkv {

// Split-KV launch of an 8-bit pool (pkv_decode8.cu); a cudaError_t value.
int launch_decode8(const AttnArgs &a);

namespace {

constexpr int kWarps = kDecodeWarpsPerCta;
constexpr int kThreads = kWarps * 32;

struct DecodeParams {
  const __nv_bfloat16 *q;
  __nv_bfloat16 *out;
  const int32_t *cu_q_lens;
  const int32_t *context_lens;
  const int32_t *block_tables;
  const int32_t *warp_begin;
  const WarpHead *warp_head;
  const Piece *pieces;
  const SharedItem *shared;    // shared-prefix CTAs, after the num_indep_ctas CTAs of warp ranges
  int32_t num_indep_ctas;
  int32_t num_shared_items;    // entries of `shared` (the pairs' chains)
  const MergeGroup *merges;
  float *part_o;
  float2 *part_ml;
  const float *ppart_o;
  const float2 *ppart_ml;
  int32_t *dev_status;
  int32_t lookahead;           // plan sized for this many further steps (chained decode)
  int32_t after_prefill;       // launched right behind this call's tensor-core kernel: the
                               // pool is complete when this kernel starts (that kernel lets
                               // it launch only after its own wait for the append), so no
                               // wait precedes the pool reads; every warp waits at its end
                               // instead, so this kernel completes after that one
  int32_t num_merges;          // all merge groups: decode ones, then prefill ones
  int32_t num_decode_merges;
  int32_t merge_lanes_log2;    // lanes that share one decode row's splits (merge kernel)
  int32_t merge_rows;          // rows the merge launch covers per decode group
  int32_t num_partials;
  int32_t num_warps;
  int32_t num_seqs;
  int32_t max_blocks_per_seq;
  int32_t num_blocks;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group;
  float scale_log2;
  int64_t total_q;
  const uint8_t *pool;  // for address-translation warm-up only (data goes through pool_map)
  int64_t pool_bytes;
  const float2 *kv_scales;  // 8-bit pool: [num_blocks][Hkv] (K scale, V scale)
};

// A piece that cannot contribute a result (its plan disagrees with the device
// metadata) writes nothing to out; when it is one part of a merge group, every
// row of its partial slot is marked (m = NaN) so the merge writes none of the
// group's rows either.
__device__ __forceinline__ void poison_piece(const DecodeParams &p, int part, int lane) {
  if (part < 0 || part >= p.num_partials) return;
  if (lane < kRowsPerTile)
    p.part_ml[(int64_t)part * kRowsPerTile + lane] = make_float2(__int_as_float(0x7fc00000), 0.f);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

inline DecodeParams make_params(const AttnArgs &a) {
  DecodeParams p;
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.cu_q_lens = a.cu_q_lens;
  p.context_lens = a.context_lens;
  p.block_tables = a.block_tables;
  p.warp_begin = a.warp_begin;
  p.warp_head = a.warp_head;
  p.shared = a.shared_items;
  p.num_indep_ctas = (a.num_decode_warps + kWarps - 1) / kWarps;
  p.num_shared_items = a.num_shared_items;
  p.pieces = a.pieces;
  p.merges = a.merge_groups;
  p.part_o = a.part_o;
  p.part_ml = reinterpret_cast<float2 *>(a.part_ml);
  p.num_merges = a.num_merge_groups;
  p.lookahead = a.lookahead;
  p.after_prefill = a.num_prefill_tiles > 0 && a.num_prefill_ctas > 0 ? 1 : 0;
  p.num_decode_merges = a.num_decode_merges;
  p.merge_lanes_log2 = 0;
  p.merge_rows = a.merge_rows;
  p.num_partials = a.num_partials;
  p.ppart_o = a.ppart_o;
  p.ppart_ml = reinterpret_cast<const float2 *>(a.ppart_ml);
  p.dev_status = a.dev_status;
  p.num_warps = a.num_decode_warps;
  p.num_seqs = a.num_seqs;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.num_blocks = a.desc.num_blocks;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.desc.num_kv_heads;
  p.group = a.num_q_heads / a.desc.num_kv_heads;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.total_q = a.total_q;
  p.pool = static_cast<const uint8_t *>(a.kv_pool);
  p.pool_bytes = (int64_t)a.desc.num_blocks * 2 * a.desc.num_kv_heads * kBlockSize *
                 a.desc.head_dim * (a.kv_scales ? 1 : 2);
  p.kv_scales = reinterpret_cast<const float2 *>(a.kv_scales);
  return p;
}

}  // namespace
}  // namespace pkv
