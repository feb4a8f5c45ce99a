// What the selection of blocks (pkv_index.cu) and the attention over selected blocks
// (pkv_sparse.cu) share: a query token's place, and the checks of their arguments.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

namespace {

// A query token's sequence and position; pos < 0: none (seq = num_seqs: past the last
// sequence, else a context shorter than its window or longer than the table's row).
struct TokenPlace {
  int32_t seq, pos;
};

// By all threads of the CTA: the sequences that end at or before the token are counted,
// one round of loads for as many sequences as threads.  s: one int per warp.
__device__ __forceinline__ TokenPlace find_token(const int32_t *cu_q_lens,
                                                 const int32_t *context_lens, int32_t num_seqs,
                                                 int32_t max_blocks, int64_t token, int32_t *s) {
  int32_t n = 0;
  for (int32_t i = threadIdx.x; i < num_seqs; i += blockDim.x) n += __ldg(cu_q_lens + i + 1) <= token;
  n = __reduce_add_sync(0xffffffffu, n);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = n;
  __syncthreads();
  TokenPlace at;
  at.seq = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) at.seq += s[w];
  at.pos = -1;
  if (at.seq < num_seqs) {
    const int32_t end = __ldg(cu_q_lens + at.seq + 1), first = __ldg(cu_q_lens + at.seq);
    const int32_t ctx = __ldg(context_lens + at.seq);
    // (token < end always, unless cu_q_lens falls: then a position may be past the table)
    if (end - first <= ctx && (ctx - 1) / kBlockSize < max_blocks && token >= first && token < end)
      at.pos = ctx - (int32_t)(end - token);
  }
  return at;
}

inline pkv_status check_sparse(const pkv_pool_desc *desc, int32_t max_blocks_per_seq,
                               int32_t num_seqs, int64_t total_q, int32_t num_q_heads,
                               int32_t num_select) {
  if (max_blocks_per_seq < 0 || num_seqs < 0 || total_q < 0 || num_select < 1) return PKV_ERR_SHAPE;
  if (num_q_heads < 1 || num_q_heads % desc->num_kv_heads != 0) return PKV_ERR_SHAPE;
  if (num_q_heads / desc->num_kv_heads > kRowsPerTile) return PKV_ERR_UNSUPPORTED;
  if (total_q > INT32_MAX || total_q * desc->num_kv_heads > INT32_MAX / 8) return PKV_ERR_UNSUPPORTED;
  if (total_q > 0 && (num_seqs == 0 || max_blocks_per_seq == 0)) return PKV_ERR_SHAPE;
  return PKV_OK;
}

}  // namespace
}  // namespace pkv
