// The block index of a bf16 pool and the selection of blocks by it.
//
// Index.  For each block and KV head, bounds of the keys in 8 bits: with s the smallest
// power of two >= 2^-64 with |K| <= 127 s, lo = floor(min K / s), hi = ceil(max K / s).
// For any q, sum_d max(q_d lo_d, q_d hi_d) s >= q . k for every key of the block (the published
// idea of bounding a page's q . k by its keys' least and largest values).
//
// Score of a block for a query token and KV head: that bound summed over the G query
// heads of the group, with q in 11 bits and a sign.  max(q lo, q hi) is q hi for q > 0 and
// q lo for q < 0, so the sum over the heads needs two vectors only, P and N (the positive
// and the negative parts, summed): 2 D products a block, whatever G.  All of it is
// integer arithmetic (P, N in 16 bits, lo, hi in 8, the sum below 2^30), rounded once
// to fp32 and scaled by a power of two: every order of summation gives the same score,
// so the selection is reproducible to the last tie.
//
// Bound: the index bytes, 2 D + 4 a block and KV head, 1/32 of the block's K and V.
#include <cuda_runtime.h>

#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_sparse.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kWarpsCta = kThreads / 32;
constexpr int kMaxTok = 64;  // tokens of an index update's CTA at most

// Two bf16 of a word; infinities and NaN as 0.
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  return ((w & 0x7f80u) == 0x7f80u ? 0u : w & 0xffffu) |
         ((w & 0x7f800000u) == 0x7f800000u ? 0u : w & 0xffff0000u);
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float pow2f(int e) {  // 2^e, -126 <= e <= 127
  return __int_as_float((e + 127) << 23);
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// ---------------------------------------------------------------- index update
//
// A CTA takes `tok` consecutive tokens.  Of a block's tokens in the step the one with the
// largest offset makes the bounds, from the block's rows up to it (read back from the pool:
// a slot written again after rejected tokens gives the bounds of what is there now); the
// CTA lists its tokens that do and its warps take them, a KV head at a time.  Few tokens:
// one a CTA, a warp a head (256 tokens 3.4 us); a prefill: 64, of which 4 do (35000 tokens
// of 8 heads of 128, 76 MB: 16.4 us, 4.6 TB/s; with 16 a CTA 4 us more, with a warp for
// every (token, head) 74; unpacking every value to fp32 took 7 us more).
template <int D>
__global__ void __launch_bounds__(kThreads)
    index_update_kernel(const uint4 *__restrict__ pool, const int32_t *__restrict__ slots,
                        int32_t num_tokens, int32_t num_blocks, int32_t hkv, int32_t tok,
                        int8_t *__restrict__ index, float *__restrict__ scales,
                        int32_t *dev_status) {
  constexpr int kLanes = D / 8;          // lanes of a key row, 8 elements each
  constexpr int kRows = 32 / kLanes;     // rows of one warp load
  constexpr int kLoads = kBlockSize / kRows;
  constexpr int kReach = kBlockSize - 1;  // how far apart a block's tokens lie at most
  __shared__ int32_t s_slot[kMaxTok + 2 * kReach];
  __shared__ int32_t s_list[kMaxTok], s_num;
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t0 = (int64_t)blockIdx.x * tok;
  for (int i = threadIdx.x; i < tok + 2 * kReach; i += kThreads) {
    const int64_t t = t0 - kReach + i;
    s_slot[i] = t >= 0 && t < num_tokens ? __ldg(slots + t) : -1;
  }
  if (threadIdx.x == 0) s_num = 0;
  __syncthreads();
  if ((int)threadIdx.x < tok) {
    const int at = threadIdx.x + kReach;
    const int32_t slot = s_slot[at], block = slot / kBlockSize;
    if (slot >= 0 && block >= num_blocks) {
      report(dev_status, PKV_DEV_BAD_SLOT);
    } else if (slot >= 0) {
      // another token that writes further into the block (or the same slot, later)
      bool other = false;
#pragma unroll
      for (int o = -kReach; o <= kReach; ++o) {
        const int32_t s = s_slot[at + o];
        other |= s >= 0 && s / kBlockSize == block && (s > slot || (s == slot && o > 0));
      }
      if (!other) s_list[atomicAdd(&s_num, 1)] = slot;
    }
  }
  __syncthreads();
  const int units = s_num * hkv;
  for (int unit = warp; unit < units; unit += kWarpsCta) {
    const int32_t slot = s_list[unit / hkv], h = unit % hkv;
    const int32_t block = slot / kBlockSize, off = slot % kBlockSize;
    const uint4 *rows = pool + ((int64_t)block * 2 * hkv + h) * kBlockSize * kLanes;
    uint4 v[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      if (u * kRows + lane / kLanes <= off) v[u] = ldg128(rows + u * 32 + lane);
    // bounds of pairs of elements; values that are not finite (found by their exponent, a
    // carry into the sign's place) count as 0
    uint32_t odd = 0;
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      if (u * kRows + lane / kLanes <= off)
        odd |= (((v[u].x & 0x7f807f80u) + 0x00800080u) | ((v[u].y & 0x7f807f80u) + 0x00800080u) |
                ((v[u].z & 0x7f807f80u) + 0x00800080u) | ((v[u].w & 0x7f807f80u) + 0x00800080u)) &
               0x80008000u;
    if (__any_sync(0xffffffffu, odd != 0)) {
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
        v[u] = make_uint4(finite_only(v[u].x), finite_only(v[u].y), finite_only(v[u].z),
                          finite_only(v[u].w));
    }
    uint32_t l2[4] = {0x7f807f80u, 0x7f807f80u, 0x7f807f80u, 0x7f807f80u};  // inf
    uint32_t h2[4] = {0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u};
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      if (u * kRows + lane / kLanes <= off) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          l2[i] = min_bf16x2(l2[i], w[i]);
          h2[i] = max_bf16x2(h2[i], w[i]);
        }
      }
    float lo[8], hi[8], top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int w = kLanes; w < 32; w <<= 1) {
        l2[i] = min_bf16x2(l2[i], __shfl_xor_sync(0xffffffffu, l2[i], w));
        h2[i] = max_bf16x2(h2[i], __shfl_xor_sync(0xffffffffu, h2[i], w));
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        lo[2 * i + j] = __uint_as_float(j ? l2[i] & 0xffff0000u : l2[i] << 16);
        hi[2 * i + j] = __uint_as_float(j ? h2[i] & 0xffff0000u : h2[i] << 16);
        top = fmaxf(top, fmaxf(fabsf(lo[2 * i + j]), fabsf(hi[2 * i + j])));
      }
    }
    top = warp_max(top);
    // top is 1.f 2^E with 7 bits of f; 127 = 1.984375 2^6 has f = 126
    const uint32_t bits = __float_as_uint(top);
    const int e = max((int)(bits >> 23) - 127 - 6 + ((bits >> 16 & 127u) == 127u), -64);
    const float inv = pow2f(-e);
    uint32_t w[2][2] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // a product that underflows to 0 is still below (above) 0
      const float a = lo[i] * inv, b = hi[i] * inv;
      const int f = a == 0.f && lo[i] < 0.f ? -1 : __float2int_rd(a);
      const int c = b == 0.f && hi[i] > 0.f ? 1 : __float2int_ru(b);
      w[0][i >> 2] |= (uint32_t)(f & 255) << (8 * (i & 3));
      w[1][i >> 2] |= (uint32_t)(c & 255) << (8 * (i & 3));
    }
    const int64_t row = (int64_t)block * hkv + h;
    if (lane < 2 * kLanes) {  // the second set of lanes (the same values) writes hi
      const bool up = lane >= kLanes;
      *reinterpret_cast<uint2 *>(index + row * 2 * D + (up ? D : 0) + (lane % kLanes) * 8) =
          make_uint2(up ? w[1][0] : w[0][0], up ? w[1][1] : w[0][1]);
    }
    if (lane == 0) scales[row] = pow2f(e);
  }
}

// ---------------------------------------------------------------- scores

constexpr int kScoreCtas = 4;  // an SM, by their registers

struct SelectParams {
  const __nv_bfloat16 *q;
  const int32_t *cu_q_lens, *context_lens, *block_tables;
  const int8_t *index;
  const float *scales;
  float *scores;          // [tokens of the pass][Hkv][stride]
  int32_t *selected;
  int64_t token0, tokens;  // tokens of the pass
  int64_t stride;
  int32_t max_blocks, num_seqs, num_blocks, num_q_heads, hkv, group;
  int32_t num_select, sink, recent;
  int32_t shares;         // into how many the blocks to score are cut
  int32_t *dev_status;
};

// A token's blocks to score are cut into equal ranges, one a CTA, of about a kScoreCtas * SMs'th
// of all that the pass has to score: every CTA finds that share, and which range is its
// own, from the lengths (a sequence's tokens count with the last one's blocks), so wide
// tables and ragged contexts cost nothing.  A warp takes one KV head (or a part of the range
// where there are fewer heads than warps), so the CTA reads the heads of a block together.
// kLpr lanes hold a block's 2 D bytes, 16 each, against weights that stay in registers;
// eight loads are in flight a lane, and their sums over the lanes are transposed on the
// way (8 shuffles for 16 or 32 blocks).  The loads are not predicated (a block that is not
// there reads block 0's row): with a branch each, 24 tokens of 1900 to 8200 blocks (254 MB)
// took 62 us, now 48.  Loads alone, in one even wave, take 40.
template <int D>
__global__ void __launch_bounds__(kThreads, kScoreCtas) score_kernel(const SelectParams p) {
  constexpr int kLpr = 2 * D / 16;     // lanes of an index row
  constexpr int kRpi = 32 / kLpr;      // blocks of one warp load
  constexpr int kUnroll = 8;
  constexpr int kBatch = kRpi * kUnroll;
  __shared__ int32_t s_sum[kWarpsCta], s_seq, s_range;
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int subs = p.hkv >= kWarpsCta ? 1 : kWarpsCta / p.hkv;
  // a sequence's tokens in this pass, and the blocks to score of the last of them
  struct Span {
    int32_t first, tokens, blocks, pos;  // first: counted from token0; pos: of the first
  };
  auto span = [&](int32_t s) {
    const int32_t c0 = __ldg(p.cu_q_lens + s), c1 = __ldg(p.cu_q_lens + s + 1);
    const int32_t ctx = __ldg(p.context_lens + s);
    const int64_t a = max((int64_t)c0, p.token0), e = min((int64_t)c1, p.token0 + p.tokens);
    Span x;
    x.first = (int32_t)(a - p.token0);
    x.tokens = e > a ? (int32_t)(e - a) : 0;
    x.pos = ctx - (int32_t)(c1 - a);
    const int32_t nb = (x.pos + x.tokens - 1) / kBlockSize + 1;
    x.blocks = x.tokens > 0 && c1 - c0 <= ctx && (ctx - 1) / kBlockSize < p.max_blocks &&
                       nb > p.num_select
                   ? nb - p.sink - p.recent
                   : 0;
    return x;
  };
  // sum over the CTA (one barrier round), or over the threads before this one
  auto cta_sum = [&](int32_t v, int32_t &before) {
    int32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    const int32_t w = lane < kWarpsCta ? s_sum[lane] : 0;
    before = x - v + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
    return __reduce_add_sync(0xffffffffu, w);
  };
  int32_t work = 0, before;
  for (int32_t s = threadIdx.x; s < p.num_seqs; s += kThreads) {
    const Span x = span(s);
    work += x.tokens * x.blocks;
  }
  const int32_t total = cta_sum(work, before), grain = kBatch * subs;
  const int32_t share = max((total + p.shares - 1) / p.shares + grain - 1, grain) / grain * grain;
  if (threadIdx.x == 0) s_seq = -1;
  int32_t base = 0;
  for (int32_t s0 = 0; s0 < p.num_seqs && base <= (int32_t)blockIdx.x; s0 += kThreads) {
    const int32_t s = s0 + threadIdx.x;
    int32_t own = 0;
    if (s < p.num_seqs) {
      const Span x = span(s);
      own = x.tokens * ((x.blocks + share - 1) / share);
    }
    const int32_t sum = cta_sum(own, before), at = (int32_t)blockIdx.x - base - before;
    if (at >= 0 && at < own) {  // one thread, in one of the rounds
      s_seq = s;
      s_range = at;
    }
    base += sum;
  }
  __syncthreads();
  const int32_t seq = s_seq;
  if (seq < 0) {
    pdl_wait();
    return;
  }
  const Span sp = span(seq);
  const int32_t ranges = (sp.blocks + share - 1) / share;
  const int32_t range = ((sp.blocks + ranges - 1) / ranges + grain - 1) / grain * grain;
  const int64_t local = sp.first + s_range / ranges;
  const int32_t c0 = p.sink + s_range % ranges * range;
  const int32_t nb = (sp.pos + s_range / ranges) / kBlockSize + 1;
  const int32_t b_lo = c0, b_hi = min(c0 + range, nb - p.recent);
  if (nb <= p.num_select || b_lo >= b_hi) {  // (an earlier token of a window: fewer blocks)
    pdl_wait();
    return;
  }
  const int32_t *table = p.block_tables + (int64_t)seq * p.max_blocks;
  const int32_t sub_len = range / subs;  // a multiple of kBatch
  // Queries, tables, index and the scores' space.  (With the queries read before this, one decode
  // took 10.9 us in a loop of the three calls, now 11.8; but they may be what the attention of
  // the call before is still writing.)
  pdl_wait();
  for (int item = warp; item < p.hkv * subs; item += kWarpsCta) {
    const int h = item % p.hkv;
    const int32_t lo = c0 + item / p.hkv * sub_len, hi = min(lo + sub_len, b_hi);
    auto entry = [&](int32_t b0) {  // lane i: the id of block b0 + i
      return lane < kBatch && b0 + lane < hi ? __ldg(table + b0 + lane) : -1;
    };
    // a batch's ids are read while the one before is scored, the first ones beside the queries
    int32_t next = entry(lo);
    // this lane's weights: of 16 elements from d0, N against lo or P against hi.  The
    // kRpi sets of lanes that hold the same ones take every kRpi-th head each.
    const int d0 = lane % (D / 16) * 16, part = lane / kLpr;
    const bool up = lane % kLpr >= D / 16;
    const __nv_bfloat16 *q =
        p.q + ((p.token0 + local) * p.num_q_heads + (int64_t)h * p.group) * D + d0;
    uint32_t top2 = 0;  // the largest |element| by pairs, as bits
    bool odd = false;
    for (int g = part; g < p.group; g += kRpi) {
      const uint4 a = ldg128_nc(q + g * D), b = ldg128_nc(q + g * D + 8);
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t m = w[i] & 0x7fff7fffu;
        odd |= (((m & 0x7f807f80u) + 0x00800080u) & 0x80008000u) != 0;
        top2 = __vmaxu2(top2, m);
      }
    }
    odd = __any_sync(0xffffffffu, odd);
    if (odd) {  // infinities and NaN count as 0
      top2 = 0;
      for (int g = part; g < p.group; g += kRpi)
        for (int i = 0; i < 8; ++i)
          top2 = __vmaxu2(top2, finite_only(__ldg(reinterpret_cast<const uint32_t *>(q + g * D) + i)) &
                                    0x7fff7fffu);
    }
    const uint32_t tops = __reduce_max_sync(0xffffffffu, max(top2 & 0xffffu, top2 >> 16));
    const float top = __uint_as_float(tops << 16);
    // u = 2^(E - 10) for top = 1.f 2^E (7 bits of f: below 2047 / 1024); q / u in two
    // exact steps
    int e = 0;
    if (top > 0.f) e = 10 - ((int)(__float_as_uint(top * 16777216.f) >> 23) - 127 - 24);
    if (top >= 16777216.f) e = 10 - ((int)(__float_as_uint(top) >> 23) - 127);
    const float f1 = pow2f(e >> 1), f2 = pow2f(e - (e >> 1));
    // rounded by adding and taking away 1.5 2^23; sums of integers below 2^15 are exact
    constexpr float kRound = 12582912.f;
    float sum[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) sum[i] = 0.f;
    for (int g = part; g < p.group; g += kRpi) {
      const uint4 a = ldg128_nc(q + g * D), b = ldg128_nc(q + g * D + 8);
      uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      if (odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = finite_only(w[i]);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float x = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        sum[i] += __fadd_rn(fmaf((up ? fmaxf(x, 0.f) : fminf(x, 0.f)) * f1, f2, kRound), -kRound);
      }
    }
    int32_t wt[8];  // 16-bit pairs
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a = sum[2 * i], b = sum[2 * i + 1];
#pragma unroll
      for (int o = kLpr; o < 32; o <<= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
      }
      wt[i] = (__float2int_rn(a) & 0xffff) | __float2int_rn(b) << 16;
    }
    float *out = p.scores + (local * p.hkv + h) * p.stride;
    // (index vectors and scales are numbered below 2^31)
    const uint4 *rows = reinterpret_cast<const uint4 *>(p.index + (int64_t)h * 2 * D) + lane % kLpr;
    const uint32_t block_vecs = (uint32_t)(p.hkv * 2 * D / 16);
    const float *scales = p.scales + h;
    bool bad = false;  // a block outside the pool: reported behind the loop
    for (int32_t b0 = lo; b0 < hi; b0 += kBatch) {
      int32_t phys = next;
      next = entry(b0 + kBatch);
      if ((uint32_t)phys >= (uint32_t)p.num_blocks) {
        phys = -1;
        bad |= lane < kBatch && b0 + lane < hi;
      }
      uint4 v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        // (block 0 in the place of none: a load without a branch)
        const uint32_t ph = (uint32_t)max(__shfl_sync(0xffffffffu, phys, u * kRpi + lane / kLpr), 0);
        v[u] = __ldg(rows + ph * block_vecs);
      }
      // the block whose score this lane ends up with
      const int mine = kLpr == 16 ? (lane >> 1 & 7) * 2 + (lane >> 4) : (lane & 7) * 4 + (lane >> 3);
      const int32_t ph = __shfl_sync(0xffffffffu, phys, mine);
      const float scale = __ldg(scales + (uint32_t)max(ph, 0) * (uint32_t)p.hkv);
      int32_t a[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        int32_t s = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s = __dp2a_lo(wt[2 * i], (int32_t)w[i], s);
          s = __dp2a_hi(wt[2 * i + 1], (int32_t)w[i], s);
        }
        a[u] = s;
      }
      // sums over the kLpr lanes of a row: halve the values and the lanes together
      int width = kLpr / 2;
#pragma unroll
      for (int n = kUnroll / 2; n >= 1; n >>= 1) {
        const bool upper = (lane & width) != 0;
#pragma unroll
        for (int u = 0; u < n; ++u) {
          const int32_t keep = upper ? a[u + n] : a[u], send = upper ? a[u] : a[u + n];
          a[u] = keep + __shfl_xor_sync(0xffffffffu, send, width);
        }
        width >>= 1;
      }
      if (kLpr == 16) a[0] += __shfl_xor_sync(0xffffffffu, a[0], 1);
      if (b0 + mine < hi && (kLpr == 8 || (lane & 1) == 0))
        out[b0 + mine] = ph >= 0 ? __int2float_rn(a[0]) * scale : -INFINITY;
    }
    if (bad) report(p.dev_status, PKV_DEV_BAD_BLOCK);
  }
}

// ---------------------------------------------------------------- selection
//
// One CTA a (token, KV head): the threshold, the score of the last block taken, by
// histograms over the scores' range (each over the bin before, at most four; mostly the
// second bin holds one score and ends it), then one ordered pass that writes the blocks
// above it and the first of those equal to it.  Two bins a thread, and eight scores a
// thread kept in shared memory (longer rows are read again).
template <int kT>
__global__ void __launch_bounds__(kT) select_kernel(const SelectParams p) {
  constexpr int kW = kT / 32, kPer = 2, kBins = kPer * kT, kCached = 8 * kT;
  constexpr int kBinBits = kT == 256 ? 9 : 11;
  static_assert(kBins == 1 << kBinBits, "a bin for every value of the digit");
  __shared__ uint32_t s_key[kCached];
  __shared__ int32_t s_bin[kBins];
  __shared__ int32_t s_sum[kW], s_gt[kW], s_eq[kW];
  __shared__ uint32_t s_min[kW], s_max[kW];
  __shared__ int32_t s_found, s_above, s_count;
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t local = blockIdx.x / p.hkv;
  const int h = (int)(blockIdx.x % p.hkv);
  const int64_t token = p.token0 + local;
  const TokenPlace at =
      find_token(p.cu_q_lens, p.context_lens, p.num_seqs, p.max_blocks, token, s_sum);
  int32_t *out = p.selected + (token * p.hkv + h) * p.num_select;
  const int32_t K = p.num_select;
  int32_t nb = at.pos / kBlockSize + 1;
  pdl_wait();
  if (at.pos < 0) {
    if (h == 0 && tid == 0 && at.seq < p.num_seqs) report(p.dev_status, PKV_DEV_PLAN_MISMATCH);
    nb = 0;
  }
  if (nb <= K) {
    for (int i = tid; i < K; i += kT) out[i] = i < nb ? i : -1;
    return;
  }
  for (int i = tid; i < p.sink; i += kT) out[i] = i;
  for (int i = tid; i < p.recent; i += kT) out[K - p.recent + i] = nb - p.recent + i;
  const int32_t need = K - p.sink - p.recent, n = nb - p.sink - p.recent;  // n > need
  if (need == 0) return;
  const float *scores = p.scores + (local * p.hkv + h) * p.stride + p.sink;
  auto key_of = [](float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
  };
  uint32_t lo = ~0u, hi = 0;
  constexpr int kAhead = 8;
  for (int32_t i0 = tid; i0 < n; i0 += kAhead * kT) {
    float x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i0 + u * kT < n) x[u] = scores[i0 + u * kT];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int32_t i = i0 + u * kT;
      if (i >= n) break;
      const uint32_t k = key_of(x[u]);
      if (i < kCached) s_key[i] = k;
      lo = min(lo, k);
      hi = max(hi, k);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    s_min[warp] = lo;
    s_max[warp] = hi;
  }
  for (int i = tid; i < kBins; i += kT) s_bin[i] = 0;
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, s_min[lane % kW]);
  hi = __reduce_max_sync(0xffffffffu, s_max[lane % kW]);
  auto key_at = [&](int32_t i) { return i < kCached ? s_key[i] : key_of(scores[i]); };
  // keys of [lo, lo + 2^bits): the need-th largest lies there, `above` keys beyond it
  int bits = 32 - __clz(hi - lo);
  int32_t above = 0;
  while (bits > 0) {
    const int shift = max(bits - kBinBits, 0);
#pragma unroll 4
    for (int32_t i = tid; i < n; i += kT) {
      const uint32_t k = key_at(i) - lo;
      if (bits == 32 || (k >> bits) == 0) atomicAdd(s_bin + (k >> shift), 1);
    }
    __syncthreads();
    // thread t: bins [kPer (kT - 1 - t), + kPer), from the top down
    const int base = kPer * (kT - 1 - tid);
    int32_t own = 0, bin[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      bin[u] = s_bin[base + u];
      s_bin[base + u] = 0;  // for the next round
      own += bin[u];
    }
    int32_t x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    const int32_t before = above + x - own + __reduce_add_sync(0xffffffffu, lane < warp ? s_sum[lane] : 0);
    if (before < need && before + own >= need) {  // one thread
      int32_t c = before;
#pragma unroll
      for (int u = kPer - 1; u >= 0; --u) {
        if (c < need && c + bin[u] >= need) {
          s_found = base + u;
          s_above = c;
          s_count = bin[u];
        }
        c += bin[u];
      }
    }
    __syncthreads();
    lo += (uint32_t)s_found << shift;
    above = s_above;
    bits = shift;
    if (above + s_count == need) {  // the whole bin is taken: all keys from lo on
      --lo;                         // (no key is 0)
      above = need;
      bits = 0;
    }
  }
  // `above` keys are larger than lo, the first need - above equal ones go along
  const int32_t ties = need - above;
  const int32_t per = ((n + kT - 1) / kT) | 1;  // odd: no bank conflicts
  const int32_t i0 = (int32_t)min((int64_t)tid * per, (int64_t)n), i1 = min(i0 + per, n);
  int32_t gt = 0, eq = 0;
#pragma unroll 4
  for (int32_t i = i0; i < i1; ++i) {
    const uint32_t k = key_at(i);
    gt += k > lo;
    eq += k == lo;
  }
  int32_t x = gt, y = eq;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += a;
      y += b;
    }
  }
  if (lane == 31) {
    s_gt[warp] = x;
    s_eq[warp] = y;
  }
  __syncthreads();
  int32_t gt0 = x - gt + __reduce_add_sync(0xffffffffu, lane < warp ? s_gt[lane] : 0);
  int32_t eq0 = y - eq + __reduce_add_sync(0xffffffffu, lane < warp ? s_eq[lane] : 0);
  if (gt == 0 && (eq == 0 || eq0 >= ties)) return;
  for (int32_t i = i0; i < i1; ++i) {
    const uint32_t k = key_at(i);
    const bool tie = k == lo;
    if (k > lo || (tie && eq0 < ties)) out[p.sink + gt0 + min(eq0, ties)] = p.sink + i;
    gt0 += k > lo;
    eq0 += tie;
  }
}

template <int D>
int launch_select_t(SelectParams p, int64_t total_q, int64_t pass_tokens, pkv_stream stream) {
  if (prepare_kernel<score_kernel<D>>(0) != cudaSuccess ||
      prepare_kernel<select_kernel<256>>(0) != cudaSuccess ||
      prepare_kernel<select_kernel<1024>>(0) != cudaSuccess)
    return (int)cudaErrorUnknown;
  const bool pdl = !profiling_active();
  for (int64_t t0 = 0; t0 < total_q; t0 += pass_tokens) {
    const int64_t n = std::min(pass_tokens, total_q - t0);
    p.token0 = t0;
    p.tokens = n;
    // one resident wave of shares, and a remainder for every token
    p.shares = kScoreCtas * std::max(device_sm_count(), 1);
    // (chunks: more of them, so that many CTAs read one part of a sequence's index at a time;
    // 512 tokens of 8192 blocks: 742 us with both kernels, in one wave 940)
    if (n > 4ll * p.num_seqs)
      p.shares = (int32_t)std::max<int64_t>(
          p.shares, std::min<int64_t>(n * p.max_blocks / 1024, 16ll * p.shares));
    cudaError_t e = launch_kernel(score_kernel<D>, dim3((unsigned)(p.shares + n)), dim3(kThreads), 0,
                                  stream, pdl, p);
    // (few rows of more than 1024 scores by four times the threads: 192 of 1900 to 8200 in 14
    // us, with 256 threads 22; 2048 rows of 60 under a table of 8192 take 24 us more with them)
    const bool wide = p.max_blocks > 1024 && n * p.hkv <= 2 * std::max(device_sm_count(), 1);
    if (e == cudaSuccess)
      e = launch_kernel(wide ? select_kernel<1024> : select_kernel<256>, dim3((unsigned)(n * p.hkv)),
                        dim3(wide ? 1024 : 256), 0, stream, pdl, p);
    if (e != cudaSuccess) return (int)e;
    count_launches(2);
  }
  return (int)cudaGetLastError();
}

// fp32 scores of a token: [Hkv][max_blocks, padded to 16 bytes]
int64_t score_bytes(int64_t hkv, int64_t max_blocks) { return hkv * align_up(max_blocks * 4, 16); }
constexpr int64_t kMaxWorkspace = 512ll << 20;

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_update_block_index(const void *kv_pool, const pkv_pool_desc *desc,
                                             const int32_t *slot_mapping, int32_t num_tokens,
                                             int8_t *index, float *index_scales,
                                             int32_t *dev_status, pkv_stream stream) {
  const pkv_status st = check_pool(desc);
  if (st != PKV_OK) return st;
  if (num_tokens < 0) return PKV_ERR_SHAPE;
  if (num_tokens == 0) return PKV_OK;
  if (!kv_pool || !slot_mapping || !index || !index_scales) return PKV_ERR_NULL;
  if (!aligned16(kv_pool) || !aligned16(index) || !aligned16(index_scales) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 3u))
    return PKV_ERR_ALIGN;
  // tokens a CTA: about two CTAs an SM
  const int64_t share = num_tokens / (2 * std::max(device_sm_count(), 1));
  int tok = 1;
  while (tok < kMaxTok && tok * 2 <= share) tok *= 2;
  const int64_t ctas = ((int64_t)num_tokens + tok - 1) / tok;
  const bool wide = desc->head_dim == 128;
  profile_begin(PKV_KERNEL_INDEX, stream);
  cudaError_t e = launch_kernel(wide ? index_update_kernel<128> : index_update_kernel<64>,
                                dim3((unsigned)ctas), dim3(kThreads), 0, stream, !profiling_active(),
                                static_cast<const uint4 *>(kv_pool), slot_mapping, num_tokens,
                                desc->num_blocks, desc->num_kv_heads, tok, index, index_scales,
                                dev_status);
  profile_end(PKV_KERNEL_INDEX, stream);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return PKV_ERR_CUDA;
  count_launches(1);
  return PKV_OK;
}

extern "C" size_t pkv_select_workspace_size(int64_t total_q, int32_t num_kv_heads,
                                            int32_t max_blocks_per_seq) {
  if (total_q <= 0 || num_kv_heads < 1 || max_blocks_per_seq < 1) return 0;
  const int64_t token = score_bytes(num_kv_heads, max_blocks_per_seq);
  return (size_t)(std::min(total_q, std::max<int64_t>(kMaxWorkspace / token, 1)) * token);
}

extern "C" pkv_status pkv_select_blocks(const void *q, const int32_t *cu_q_lens,
                                        const int32_t *context_lens, const int32_t *block_tables,
                                        int32_t max_blocks_per_seq, int32_t num_seqs,
                                        int64_t total_q, int32_t num_q_heads, const int8_t *index,
                                        const float *index_scales, const pkv_pool_desc *desc,
                                        int32_t num_select, int32_t sink_blocks,
                                        int32_t recent_blocks, int32_t *selected, void *workspace,
                                        int64_t workspace_bytes, int32_t *dev_status,
                                        pkv_stream stream) {
  pkv_status st = check_pool(desc);
  if (st != PKV_OK) return st;
  st = check_sparse(desc, max_blocks_per_seq, num_seqs, total_q, num_q_heads, num_select);
  if (st != PKV_OK) return st;
  if (sink_blocks < 0 || recent_blocks < 1 || (int64_t)sink_blocks + recent_blocks > num_select)
    return PKV_ERR_RANGE;
  if (total_q == 0) return PKV_OK;
  if (desc->num_blocks == 0) return PKV_ERR_SHAPE;
  if (!q || !cu_q_lens || !context_lens || !block_tables || !index || !index_scales || !selected ||
      !workspace)
    return PKV_ERR_NULL;
  if (!aligned16(q) || !aligned16(index) || (reinterpret_cast<uintptr_t>(index_scales) & 3u) ||
      !aligned16(workspace) || (reinterpret_cast<uintptr_t>(selected) & 3u))
    return PKV_ERR_ALIGN;
  const int64_t token = score_bytes(desc->num_kv_heads, max_blocks_per_seq);
  if (workspace_bytes < token) return PKV_ERR_WORKSPACE;
  SelectParams p;
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.cu_q_lens = cu_q_lens;
  p.context_lens = context_lens;
  p.block_tables = block_tables;
  p.index = index;
  p.scales = index_scales;
  p.scores = static_cast<float *>(workspace);
  p.selected = selected;
  p.stride = align_up((int64_t)max_blocks_per_seq * 4, 16) / 4;
  p.max_blocks = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.num_blocks = desc->num_blocks;
  p.num_q_heads = num_q_heads;
  p.hkv = desc->num_kv_heads;
  p.group = num_q_heads / desc->num_kv_heads;
  p.num_select = num_select;
  p.sink = sink_blocks;
  p.recent = recent_blocks;
  p.dev_status = dev_status;
  // a pass: what the workspace holds, its blocks and the grids counted in 32 bits
  int64_t pass = std::min(workspace_bytes / token, total_q);
  pass = std::min(pass, (int64_t)(1 << 30) / std::max(max_blocks_per_seq, p.hkv));
  if (pass < 1) return PKV_ERR_UNSUPPORTED;  // more columns than a pass may count
  profile_begin(PKV_KERNEL_SELECT, stream);
  const int e = desc->head_dim == 128 ? launch_select_t<128>(p, total_q, pass, stream)
                                      : launch_select_t<64>(p, total_q, pass, stream);
  profile_end(PKV_KERNEL_SELECT, stream);
  return e ? PKV_ERR_CUDA : PKV_OK;
}
