// One paged block of a bf16 pool in shared memory and its contribution to a row group
// of at most 16 query rows: what the split-KV kernels of the bf16 pool share.
#pragma once

#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kBoxBytes = kBlockSize * 128;  // 16 rows x 64 bf16, 128-byte swizzled

// Byte offset of 16-byte chunk `chunk` (0 .. D/8-1) of key row `row` (0..15) of
// a paged block as one 4-D TMA box lands it: [8-row group][64-column half]
// [8 rows][128 B], 128-byte swizzled (the 16-byte chunk index XOR the row within
// its 8-row atom).
template <int kHalves>
__device__ __forceinline__ uint32_t blk_off(int row, int chunk) {
  return (uint32_t)((((row >> 3) * kHalves + (chunk >> 3)) << 10) + ((row & 7) << 7) +
                    (((chunk & 7) ^ (row & 7)) << 4));
}

// One paged block (16 keys at positions p0 ..) of a row group: S = Q K^T, causal
// mask, online softmax in log2 units, O += P V.  sK / sV: the block's K and V in
// shared memory (blk_off layout).  The warp's running (m, l, O) are updated.
// P goes into the product as one bf16 (2^-8 of a weight at most is lost), or with kTwoParts as
// the sum of two, 2^-14: the first is the leading bits of P (1 - 2^-8), so that the second is
// never 0 (nor negative) beside a weight, and an infinite V keeps its sign.
template <int D, bool kTwoParts = false>
__device__ __forceinline__ void block_update(uint32_t sK, uint32_t sV, const uint32_t (&qa)[D / 16][4],
                                             int p0, int q_pos0, int lim_lo, int lim_hi, float sl2,
                                             int r, int c, float &m_lo, float &m_hi, float &l_lo,
                                             float &l_hi, float (&o)[D / 8][4]) {
  constexpr int kL = D / 32;
  constexpr int kNt = D / 8;
  constexpr int kHalves = D / 64;
  // S = Q K^T for the block's 16 keys (two n-tiles of 8 keys)
  float s[2][4];
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
    const int t = r + 8 * nt;
#pragma unroll
    for (int L = 0; L < kL; ++L) {
      const int e = 8 * (L >> 1) + 2 * c + (L & 1);
      const uint4 kv = lds128(sK + blk_off<kHalves>(t, e));
      mma_16816(s[nt], qa[2 * L][0], qa[2 * L][1], qa[2 * L][2], qa[2 * L][3], kv.x, kv.y);
      mma_16816(s[nt], qa[2 * L + 1][0], qa[2 * L + 1][1], qa[2 * L + 1][2],
                qa[2 * L + 1][3], kv.z, kv.w);
    }
  }
  // scale to log2 units; causal / context mask on the boundary blocks
  const bool need_mask = p0 + kBlockSize - 1 > q_pos0;
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x = s[nt][j] * sl2;
      if (need_mask) {
        const int pos = p0 + 8 * nt + 2 * c + (j & 1);
        if (pos > (j < 2 ? lim_lo : lim_hi)) x = -INFINITY;
      }
      s[nt][j] = x;
    }
  // online softmax (rows r and r + 8; the 4 lanes of a row hold 4 keys each)
  float mx_lo = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
  float mx_hi = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
  mx_lo = fmaxf(mx_lo, __shfl_xor_sync(0xffffffffu, mx_lo, 1));
  mx_lo = fmaxf(mx_lo, __shfl_xor_sync(0xffffffffu, mx_lo, 2));
  mx_hi = fmaxf(mx_hi, __shfl_xor_sync(0xffffffffu, mx_hi, 1));
  mx_hi = fmaxf(mx_hi, __shfl_xor_sync(0xffffffffu, mx_hi, 2));
  const float mn_lo = fmaxf(m_lo, mx_lo), mn_hi = fmaxf(m_hi, mx_hi);
  const float base_lo = mn_lo == -INFINITY ? 0.f : mn_lo;
  const float base_hi = mn_hi == -INFINITY ? 0.f : mn_hi;
  const float a_lo = fast_exp2(m_lo - base_lo), a_hi = fast_exp2(m_hi - base_hi);
  m_lo = mn_lo;
  m_hi = mn_hi;
#pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    s[nt][0] = fast_exp2(s[nt][0] - base_lo);
    s[nt][1] = fast_exp2(s[nt][1] - base_lo);
    s[nt][2] = fast_exp2(s[nt][2] - base_hi);
    s[nt][3] = fast_exp2(s[nt][3] - base_hi);
  }
  l_lo = l_lo * a_lo + (s[0][0] + s[0][1]) + (s[1][0] + s[1][1]);
  l_hi = l_hi * a_hi + (s[0][2] + s[0][3]) + (s[1][2] + s[1][3]);
  if (__any_sync(0xffffffffu, a_lo != 1.f || a_hi != 1.f)) {
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
      o[nt][0] *= a_lo;
      o[nt][1] *= a_lo;
      o[nt][2] *= a_hi;
      o[nt][3] *= a_hi;
    }
  }
  // P (bf16) as the A operand: keys are the k dimension
  uint32_t pb[2][2];  // the first parts, if there are two
  if constexpr (kTwoParts) {
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t b[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float &x = s[nt][2 * u + j];
          b[j] = __float_as_uint(x * 0.99609375f) & 0xffff0000u;
          x -= __uint_as_float(b[j]);  // exact
        }
        pb[nt][u] = __byte_perm(b[0], b[1], 0x7632);
      }
  }
  const uint32_t pa0 = pack_bf16x2(s[0][0], s[0][1]);
  const uint32_t pa1 = pack_bf16x2(s[0][2], s[0][3]);
  const uint32_t pa2 = pack_bf16x2(s[1][0], s[1][1]);
  const uint32_t pa3 = pack_bf16x2(s[1][2], s[1][3]);
  // O += P V: lane (r, c) reads keys 2c, 2c+1, 2c+8, 2c+9 at head_dim chunk r (+8 per half)
#pragma unroll
  for (int hh = 0; hh < kHalves; ++hh) {
    const int ch = hh * 8 + r;  // head_dim chunk
    const uint4 v0 = lds128(sV + blk_off<kHalves>(2 * c, ch));
    const uint4 v1 = lds128(sV + blk_off<kHalves>(2 * c + 1, ch));
    const uint4 v2 = lds128(sV + blk_off<kHalves>(2 * c + 8, ch));
    const uint4 v3 = lds128(sV + blk_off<kHalves>(2 * c + 9, ch));
    const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w};
    const uint32_t w1[4] = {v1.x, v1.y, v1.z, v1.w};
    const uint32_t w2[4] = {v2.x, v2.y, v2.z, v2.w};
    const uint32_t w3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t even0 = __byte_perm(w0[k], w1[k], 0x5410);
      const uint32_t even1 = __byte_perm(w2[k], w3[k], 0x5410);
      const uint32_t odd0 = __byte_perm(w0[k], w1[k], 0x7632);
      const uint32_t odd1 = __byte_perm(w2[k], w3[k], 0x7632);
      mma_16816(o[8 * hh + 2 * k], pa0, pa1, pa2, pa3, even0, even1);
      mma_16816(o[8 * hh + 2 * k + 1], pa0, pa1, pa2, pa3, odd0, odd1);
      if constexpr (kTwoParts) {
        mma_16816(o[8 * hh + 2 * k], pb[0][0], pb[0][1], pb[1][0], pb[1][1], even0, even1);
        mma_16816(o[8 * hh + 2 * k + 1], pb[0][0], pb[0][1], pb[1][0], pb[1][1], odd0, odd1);
      }
    }
  }
}

}  // namespace
}  // namespace pkv
