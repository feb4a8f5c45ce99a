// bf16 copies of the 8-bit blocks the tensor-core kernel needs, each KV head's blocks of a
// sequence one after another, so that a key tile is one box of a tensor map.
//
// A tensor-core sequence of q_len query tokens and context ctx does 4 D q_len ctx
// FLOPs a head and reads D ctx e4m3 values once more per 128-token tile; its keys
// and values are turned into bf16 here once (3 bytes moved a value, in L2 for
// all but the longest contexts), instead of once per query tile inside the
// attention kernel, whose shared-memory bandwidth the two MMAs already fill.
// Each value is c s rounded to bf16: exact for the power-of-two scales the
// append writes (e4m3 has 4 significant bits, bf16 8), one rounding of 2^-8 for
// any other scale.  Rows past the context are written as zeros, so that stale
// bytes (NaN codes among them) never meet a zero weight.
//
// Bound by latency on all but the longest contexts: launch, the three dependent
// reads from a block's number to its bytes, the stores.  One CTA a block, a warp per
// (K|V, head) slab, 64 bytes in and 128 out a lane at D = 128; a sequence's range and
// context are read together, before the wait for the preceding kernel.  288 blocks of 8
// heads: 6.4 us, 1024: 18.5 us (100 MB moved, 5.4 TB/s).  The tensor-core
// kernel is let launch early only when its CTAs, each a whole SM, leave half of the SMs
// to the CTAs here (64 CTAs of a gathered prefix: 44.8 us a step with the early
// launch, 48.7 without; 152 CTAs of a 2048-token chunk: 153 us with, 144 without).
#include <cuda_runtime.h>

#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 512;

struct StageParams {
  const uint8_t *pool;
  const float *scales;         // [num_blocks][Hkv][2]
  const int32_t *stage_begin;  // [num_seqs + 1]
  const int32_t *context_lens;
  const int32_t *block_tables;
  uint4 *staged;               // bf16 [2][Hkv][staged_blocks][16][D]
  int32_t num_seqs, max_blocks_per_seq, num_blocks, hkv, staged_blocks;
  int32_t early;
  int32_t *dev_status;
};

template <int D>
__global__ void __launch_bounds__(kThreads) stage_kernel(const StageParams p) {
  constexpr int kIn = kBlockSize * D / (32 * 16);  // 16-byte loads a lane
  if (p.early) pdl_trigger();  // the tensor-core kernel waits before it reads `staged`
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blk = blockIdx.x;
  // the sequence whose range holds this block: the last s with stage_begin[s] <= blk
  // (step metadata, not written by the kernels before this one)
  int seq = 0, kb = -1, ctx = 0;
  for (int s0 = 0; s0 < p.num_seqs; s0 += 32) {
    const int s = s0 + lane;
    const bool in = s < p.num_seqs;
    const int b0 = in ? __ldg(p.stage_begin + s) : 0, b1 = in ? __ldg(p.stage_begin + s + 1) : 0;
    const int c = in ? __ldg(p.context_lens + s) : 0;
    const uint32_t here = __ballot_sync(0xffffffffu, in && b0 <= blk && blk < b1);
    if (here) {
      const int src = __ffs((int)here) - 1;
      seq = s0 + src;
      kb = blk - __shfl_sync(0xffffffffu, b0, src);
      ctx = __shfl_sync(0xffffffffu, c, src);
      break;
    }
  }
  int phys = -1;
  const int64_t left = kb < 0 ? 0 : (int64_t)ctx - (int64_t)kb * kBlockSize;
  const int rows = left >= kBlockSize ? kBlockSize : left > 0 ? (int)left : 0;
  if (kb >= 0 && kb < p.max_blocks_per_seq && rows > 0) {
    phys = __ldg(p.block_tables + (int64_t)seq * p.max_blocks_per_seq + kb);
    if (phys < 0 || phys >= p.num_blocks) {
      if (threadIdx.x == 0) report(p.dev_status, PKV_DEV_BAD_BLOCK);
      phys = -1;
    }
  }
  pdl_wait();  // the pool is complete, and the workspace's last readers are done
  const int slabs = 2 * p.hkv;
  for (int sl = warp; sl < slabs; sl += kThreads / 32) {
    const int kv = sl >= p.hkv, h = sl - kv * p.hkv;
    const uint4 *src = reinterpret_cast<const uint4 *>(
        p.pool + ((int64_t)(phys < 0 ? 0 : phys) * slabs + sl) * kBlockSize * D);
    uint4 x[kIn];
    const float s =
        phys >= 0 ? __ldg(p.scales + ((int64_t)phys * p.hkv + h) * 2 + kv) : 0.f;
#pragma unroll
    for (int i = 0; i < kIn; ++i) {
      const int row = (i * 32 + lane) * 16 / D;
      x[i] = phys >= 0 && row < rows ? ldg128_nc(src + i * 32 + lane) : make_uint4(0, 0, 0, 0);
    }
    uint4 *dst = p.staged + ((int64_t)sl * p.staged_blocks + blk) * (kBlockSize * D / 8);
#pragma unroll
    for (int i = 0; i < kIn; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t a = e4m3x2_to_f16x2(w[k]), b = e4m3x2_to_f16x2(w[k] >> 16);
        const float2 fa = __half22float2(*reinterpret_cast<const __half2 *>(&a));
        const float2 fb = __half22float2(*reinterpret_cast<const __half2 *>(&b));
        o[2 * k] = pack_bf16x2(fa.x * s, fa.y * s);
        o[2 * k + 1] = pack_bf16x2(fb.x * s, fb.y * s);
      }
      dst[2 * (i * 32 + lane)] = make_uint4(o[0], o[1], o[2], o[3]);
      dst[2 * (i * 32 + lane) + 1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

}  // namespace

int launch_stage(const AttnArgs &a, int *launches) {
  if (!a.kv_scales || a.num_prefill_tiles <= 0 || a.staged_blocks <= 0) return 0;
  StageParams p;
  p.pool = static_cast<const uint8_t *>(a.kv_pool);
  p.scales = a.kv_scales;
  p.stage_begin = a.stage_begin;
  p.context_lens = a.context_lens;
  p.block_tables = a.block_tables;
  p.staged = static_cast<uint4 *>(a.staged);
  p.num_seqs = a.num_seqs;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.num_blocks = a.desc.num_blocks;
  p.hkv = a.desc.num_kv_heads;
  p.staged_blocks = a.staged_blocks;
  p.early = 2 * a.num_prefill_ctas <= device_sm_count() ? 1 : 0;
  p.dev_status = a.dev_status;
  const bool d128 = a.desc.head_dim == 128;
  cudaError_t e = d128 ? prepare_kernel<stage_kernel<128>>(0) : prepare_kernel<stage_kernel<64>>(0);
  if (e != cudaSuccess) return (int)e;
  profile_begin(PKV_KERNEL_STAGE, a.stream);
  e = launch_kernel(d128 ? stage_kernel<128> : stage_kernel<64>, dim3((unsigned)a.staged_blocks),
                    dim3(kThreads), 0, a.stream, !profiling_active(), p);
  profile_end(PKV_KERNEL_STAGE, a.stream);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) {
    ++*launches;
    count_launches(1);
  }
  return (int)e;
}

}  // namespace pkv
