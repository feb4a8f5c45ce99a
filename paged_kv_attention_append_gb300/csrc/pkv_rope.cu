// KV append with the position rotation applied on the way, into a bf16 or an
// 8-bit pool.
//
// The append of pkv_append.cu scatters rows that another kernel has already
// rotated; here the rotation, the append and (8-bit pool) the quantisation are
// one pass over q, k and v.  With position p, pair i < R/2 of a head,
//   a' = a cos[p][i] - b sin[p][i],   b' = b cos[p][i] + a sin[p][i],
// (a, b) = elements (i, i + R/2), or (2i, 2i + 1) when interleaved; elements past
// R pass through.  q goes to q_out, k and v to the pool.  Every product and sum
// is rounded to fp32 on its own (no fused multiply-add), so the values match
// the formula evaluated in fp32 exactly, and each result is rounded once, to
// bf16 or to e4m3.
//
// 8-bit pool: for each (block, KV head, K or V) this step writes to, with N the
// new rows and `first` the smallest offset among them, rows below `first` are
// kept rows of the same sequence (a sequence fills its blocks in order), rows
// from `first` on that are not in N are stale.
//   s' = s when first > 0 and 448 s >= max |N|, else the smallest power of two
//        >= 2^-64 with 448 s' >= max |N|
//   new rows: rn_sat(x / s');   kept rows, when s' != s: rn(c s / s').
// Powers of two make x / s' and c s / s' exact before the rounding, so a kept
// row loses nothing but bits that fall below e4m3's smallest step.
//
// What bounds it: HBM.  Per token and head q is read and written, k and v are
// read and written (at half the bytes for the 8-bit pool).  16-byte loads, a row
// of 64 or 128 elements on 8 or 16 lanes, several rows in flight a lane; the
// token's cosines and sines are loaded once per warp and stay in registers
// across its heads.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>

#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kWarpsPerCta = kThreads / 32;
constexpr int kWindow = 16;   // tokens from a block's first new token that may write it
constexpr float kE4m3Max = 448.f;

struct RopeParams {
  const uint4 *q, *k, *v;
  uint4 *q_out;
  int64_t qs, ks, vs, qos;  // token strides in 16-byte vectors
  const float *cos_sin;
  const int32_t *positions;
  const int32_t *slots;
  int32_t max_pos, rot;     // rot = 0: no rotation
  int32_t n, hq, hkv;
  int32_t num_blocks;
  void *pool;
  float *scales;            // [num_blocks][Hkv][2]
  int32_t chunks, rows_per_chunk;  // rows of a token are cut into chunks, one per warp
  int32_t q_ctas;                  // 8-bit pool: CTAs that rotate q; the others append
  int32_t tile;                    // 8-bit pool: tokens whose blocks one warp looks after
  int32_t *dev_status;
};

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The cosines and sines of a lane's 8 elements 8 l .. 8 l + 7 at one position.
// Half split: 8 of each (the lane's partner elements are R/2 away and use the
// same ones).  Interleaved: 4 of each (c[4..7], s[4..7] are not used).
template <bool kInter>
struct Angles {
  float c[kInter ? 4 : 8], s[kInter ? 4 : 8];
  __device__ __forceinline__ void load(const RopeParams &p, int pos, int l) {
    const int half = p.rot >> 1;
    const float *row = p.cos_sin + (int64_t)pos * p.rot;
    if (8 * l >= p.rot) return;
    const int i0 = kInter ? 4 * l : 8 * l < half ? 8 * l : 8 * l - half;
#pragma unroll
    for (int j = 0; j < (kInter ? 1 : 2); ++j) {
      const float4 a = __ldg(reinterpret_cast<const float4 *>(row + i0) + j);
      const float4 b = __ldg(reinterpret_cast<const float4 *>(row + half + i0) + j);
      c[4 * j] = a.x, c[4 * j + 1] = a.y, c[4 * j + 2] = a.z, c[4 * j + 3] = a.w;
      s[4 * j] = b.x, s[4 * j + 1] = b.y, s[4 * j + 2] = b.z, s[4 * j + 3] = b.w;
    }
  }
  // The lane's 8 elements of one row, rotated.  Whole warp (the half-split form
  // shuffles); partner: the lane that holds the elements R/2 away; lanes past R
  // or with turn = false pass their elements through.
  __device__ __forceinline__ void turn(const RopeParams &p, const uint4 &raw, int l, int partner,
                                       bool on, float (&y)[8]) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = lo16(w[i]);
      y[2 * i + 1] = hi16(w[i]);
    }
    if constexpr (kInter) {
      if (on && 8 * l < p.rot) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = y[2 * i], b = y[2 * i + 1];
          y[2 * i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
          y[2 * i + 1] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
        }
      }
    } else {
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __shfl_sync(0xffffffffu, w[i], partner);
      if (on && 8 * l < p.rot) {
        const bool low = 8 * l < (p.rot >> 1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float other = (i & 1) ? hi16(o[i >> 1]) : lo16(o[i >> 1]);
          const float xc = __fmul_rn(y[i], c[i]), os = __fmul_rn(other, s[i]);
          y[i] = low ? __fsub_rn(xc, os) : __fadd_rn(xc, os);
        }
      }
    }
  }
};

template <int D>
__device__ __forceinline__ int partner_lane(const RopeParams &p, int lane) {
  constexpr int kLpr = D / 8;
  const int l = lane % kLpr, h = p.rot >> 4;  // lanes of half the rotated elements
  if (8 * l >= p.rot) return lane;
  return l < h ? lane + h : lane - h;
}

__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
  return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                    pack_bf16x2(y[6], y[7]));
}

// Rows of tokens, a chunk of one token's rows per warp: its q heads, then
// (kPool) its k and v heads.  U rows of each lane group are in flight.
template <int D, bool kInter, bool kPool>
__device__ __forceinline__ void token_rows(const RopeParams &p, int64_t unit, int lane) {
  constexpr int kLpr = D / 8, kRpw = 32 / kLpr, kU = 4;
  const int t = (int)(unit / p.chunks), ch = (int)(unit % p.chunks);
  if (t >= p.n) return;
  const int l = lane % kLpr, sub = lane / kLpr;
  const int rows = p.hq + (kPool ? 2 * p.hkv : 0);
  const int r0 = ch * p.rows_per_chunk, r1 = min(rows, r0 + p.rows_per_chunk);
  const int pos = p.positions ? __ldg(p.positions + t) : 0;
  const int64_t slot = kPool ? __ldg(p.slots + t) : -1;
  const bool bad_pos = pos >= p.max_pos && p.rot > 0;
  if (ch == 0 && lane == 0) {
    if (bad_pos) report(p.dev_status, PKV_DEV_BAD_POSITION);
    if (kPool && slot >= (int64_t)p.num_blocks * kBlockSize) report(p.dev_status, PKV_DEV_BAD_SLOT);
  }
  if (pos < 0 || bad_pos) return;
  const bool put = kPool && slot >= 0 && slot < (int64_t)p.num_blocks * kBlockSize;
  Angles<kInter> ang;
  const int turned = p.rot > 0 ? p.hq + p.hkv : 0;  // rows that are rotated
  if (r0 < turned) ang.load(p, pos, l);
  const int partner = partner_lane<D>(p, lane);
  const int64_t blk = put ? slot / kBlockSize : 0, off = put ? slot % kBlockSize : 0;
  for (int base = r0; base < r1; base += kU * kRpw) {
    uint4 x[kU];
    uint4 *dst[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int r = base + u * kRpw + sub;
      const uint4 *src = nullptr;
      dst[u] = nullptr;
      if (r < r1) {
        if (r < p.hq) {
          src = p.q + t * p.qs + r * kLpr + l;
          dst[u] = p.q_out + t * p.qos + r * kLpr + l;
        } else if (put) {
          const int kv = r >= p.hq + p.hkv, h = r - p.hq - (kv ? p.hkv : 0);
          src = (kv ? p.v + t * p.vs : p.k + t * p.ks) + h * kLpr + l;
          dst[u] = static_cast<uint4 *>(p.pool) +
                   (((blk * 2 + kv) * p.hkv + h) * kBlockSize + off) * kLpr + l;
        }
      }
      x[u] = src ? ldg128(src) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int r = base + u * kRpw + sub;
      float y[8];
      ang.turn(p, x[u], l, partner, r < turned, y);
      if (dst[u]) *dst[u] = r < turned ? pack8(y) : x[u];
    }
  }
}

// The smallest power of two s >= 2^-64 with amax <= 448 s (amax finite, >= 0):
// 448 = 1.75 * 2^8, so with amax = f 2^e the exponent is e - 8, or e - 7 when f > 1.75.
__device__ __forceinline__ float pow2_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, -64);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// One warp: the blocks whose first new token lies among tokens t0 .. t0 + tile - 1,
// for one KV head and K (kv = 0) or V (kv = 1).
template <int D, bool kInter>
__device__ __forceinline__ void append_blocks(const RopeParams &p, int64_t unit, int lane) {
  constexpr int kLpr = D / 8, kRpw = 32 / kLpr, kIt = kWindow / kRpw;
  const int kv = (int)(unit & 1);
  const int h = (int)((unit >> 1) % p.hkv);
  const int64_t t0 = (unit >> 1) / p.hkv * p.tile;
  if (t0 >= p.n) return;
  const int l = lane % kLpr, sub = lane / kLpr;
  const int64_t nslots = (int64_t)p.num_blocks * kBlockSize;
  // slots and positions of tokens t0 - 32 .. t0 + 31: lane i holds t0 - 32 + i and t0 + i;
  // a token that writes nothing has slot -1
  int32_t slot[2], pos[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t t = t0 + lane - 32 * (1 - i);
    const bool in = t >= 0 && t < p.n;
    slot[i] = in ? __ldg(p.slots + t) : -1;
    pos[i] = in && p.rot > 0 ? __ldg(p.positions + t) : 0;
    const bool bad_slot = slot[i] >= nslots, bad_pos = p.rot > 0 && pos[i] >= p.max_pos;
    if (i == 1 && lane < p.tile && h == 0 && kv == 0) {
      if (bad_slot) report(p.dev_status, PKV_DEV_BAD_SLOT);
      if (bad_pos) report(p.dev_status, PKV_DEV_BAD_POSITION);
    }
    if (bad_slot || bad_pos || pos[i] < 0 || slot[i] < 0) slot[i] = -1;
  }
  const int32_t blk0 = slot[0] < 0 ? -1 : slot[0] / kBlockSize;
  const int32_t blk1 = slot[1] < 0 ? -1 : slot[1] / kBlockSize;
  const int partner = partner_lane<D>(p, lane);
  const uint4 *src = (kv ? p.v : p.k) + h * kLpr + l;
  const int64_t stride = kv ? p.vs : p.ks;
  const bool rotate = kv == 0 && p.rot > 0;

  for (int j = 0; j < p.tile; ++j) {
    const int32_t blk = __shfl_sync(0xffffffffu, blk1, j);
    // bit 32 + i: token t0 + i writes this block
    const uint64_t same = ((uint64_t)__ballot_sync(0xffffffffu, blk1 == blk) << 32) |
                          __ballot_sync(0xffffffffu, blk0 == blk);
    if (blk < 0) continue;
    const uint64_t before = (same >> (32 + j - (kWindow - 1))) & ((1u << (kWindow - 1)) - 1);
    if (before) {
      // an earlier token's warp takes it, unless that token itself follows an
      // earlier one and this one lies outside the first one's window
      const int f = 32 + j - (kWindow - 1) + __ffsll((long long)before) - 1;
      const bool lost = ((same >> (f - (kWindow - 1))) & ((1u << (kWindow - 1)) - 1)) != 0;
      if (lost && lane == 0 && h == 0 && kv == 0) report(p.dev_status, PKV_DEV_BAD_SLOT);
      continue;
    }
    const uint32_t members = (uint32_t)(same >> (32 + j)) & 0xffffu;  // token t0 + j + i
    // offsets of the members; the smallest one
    int first = kBlockSize;
    const int my_off = slot[1] >= 0 ? slot[1] % kBlockSize : kBlockSize;
    {
      const bool mine = lane >= j && lane < j + kWindow && ((members >> (lane - j)) & 1);
      first = __reduce_min_sync(0xffffffffu, mine ? my_off : kBlockSize);
    }
    float *scale_at = p.scales + ((int64_t)blk * p.hkv + h) * 2 + kv;
    const float s_old = first > 0 ? __ldcg(scale_at) : 0.f;
    uint8_t *slab = static_cast<uint8_t *>(p.pool) +
                    (((int64_t)blk * 2 + kv) * p.hkv + h) * kBlockSize * D;
    // ---- the new rows, rotated, in registers; their largest value
    const int its = (32 - __clz((int)members) + kRpw - 1) / kRpw;
    uint4 x[kIt];
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      const int i = it * kRpw + sub;
      x[it] = it < its && ((members >> i) & 1) ? ldg128(src + (t0 + j + i) * stride)
                                               : make_uint4(0, 0, 0, 0);
    }
    float y[kIt][8];
    float amax = 0.f;
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      if (it >= its) break;
      const int i = it * kRpw + sub;
      const int ps = __shfl_sync(0xffffffffu, pos[1], (j + i) & 31);
      const bool on = rotate && ((members >> i) & 1);
      Angles<kInter> ang;
      if (on) ang.load(p, ps, l);
      ang.turn(p, x[it], l, partner, on, y[it]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = fabsf(y[it][e]);
        amax = fmaxf(amax, a <= FLT_MAX ? a : 0.f);  // infinities saturate, NaN stays NaN
      }
    }
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    // ---- the block's scale
    const bool keep = s_old > 0.f && s_old * kE4m3Max >= amax;
    const float s_new = keep ? s_old : pow2_scale(amax);
    const bool pow2 = (__float_as_uint(s_new) & 0x7fffffu) == 0 && s_new >= 0x1p-120f;
    const float inv = pow2 ? 1.f / s_new : 0.f;
    // ---- rows the block already holds, when its scale grew
    if (!keep && s_old > 0.f) {
      const float ratio = s_old / s_new;
      for (int r = sub; r < first; r += kRpw) {
        uint2 *at = reinterpret_cast<uint2 *>(slab + r * D) + l;
        const uint2 w = __ldcg(at);
        uint2 z;
        auto requant = [&](uint32_t v) {
          const uint32_t a = e4m3x2_to_f16x2(v), b = e4m3x2_to_f16x2(v >> 16);
          const float2 fa = __half22float2(*reinterpret_cast<const __half2 *>(&a));
          const float2 fb = __half22float2(*reinterpret_cast<const __half2 *>(&b));
          return f32x2_to_e4m3x2(fa.x * ratio, fa.y * ratio) |
                 (f32x2_to_e4m3x2(fb.x * ratio, fb.y * ratio) << 16);
        };
        z.x = requant(w.x);
        z.y = requant(w.y);
        *at = z;
      }
    }
    if (!keep && lane == 0) *scale_at = s_new;
    // ---- the new rows
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      if (it >= its) break;
      const int i = it * kRpw + sub;
      const int off = __shfl_sync(0xffffffffu, my_off, (j + i) & 31);
      if (!((members >> i) & 1)) continue;
      float z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = pow2 ? y[it][e] * inv : __fdiv_rn(y[it][e], s_new);
      uint2 w;
      w.x = f32x2_to_e4m3x2(z[0], z[1]) | (f32x2_to_e4m3x2(z[2], z[3]) << 16);
      w.y = f32x2_to_e4m3x2(z[4], z[5]) | (f32x2_to_e4m3x2(z[6], z[7]) << 16);
      reinterpret_cast<uint2 *>(slab + off * D)[l] = w;
    }
    __syncwarp();
  }
}

// No early release of the next kernel: the attention kernels read q before they
// wait for this one, so q_out has to be complete and visible when they start.
template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
  token_rows<D, kInter, true>(p, unit, lane);
  __threadfence();
}

template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads) rope_append_fp8_kernel(const RopeParams p) {
  const int lane = threadIdx.x & 31;
  if ((int)blockIdx.x < p.q_ctas)
    token_rows<D, kInter, false>(p, (int64_t)blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5), lane);
  else
    append_blocks<D, kInter>(
        p, (int64_t)(blockIdx.x - p.q_ctas) * kWarpsPerCta + (threadIdx.x >> 5), lane);
  __threadfence();
}

template <int D, bool kInter>
int launch_t(const RopeAppendArgs &a) {
  constexpr int kRpw = 32 / (D / 8);
  RopeParams p;
  p.q = static_cast<const uint4 *>(a.q);
  p.k = static_cast<const uint4 *>(a.k);
  p.v = static_cast<const uint4 *>(a.v);
  p.q_out = static_cast<uint4 *>(a.q_out);
  p.qs = a.q_stride / 8;
  p.ks = a.k_stride / 8;
  p.vs = a.v_stride / 8;
  p.qos = a.q_out_stride / 8;
  p.cos_sin = a.cos_sin;
  p.positions = a.cos_sin ? a.positions : nullptr;
  p.slots = a.slot_mapping;
  p.max_pos = a.max_positions;
  p.rot = a.cos_sin ? a.rotary_dim : 0;
  p.n = a.num_tokens;
  p.hq = a.num_q_heads;
  p.hkv = a.desc.num_kv_heads;
  p.num_blocks = a.desc.num_blocks;
  p.pool = a.kv_pool;
  p.scales = a.kv_scales;
  p.dev_status = a.dev_status;
  p.tile = 1;
  p.q_ctas = 0;
  const bool f8 = a.kv_scales != nullptr;
  const int sms = std::max(device_sm_count(), 1);
  // a token's rows on as many warps as it takes to give every SM 16 warps, up to
  // one step of rows a warp; a long chunk keeps a token's rows on one warp, which
  // loads its cosines and sines once
  const int rows = p.hq + (f8 ? 0 : 2 * p.hkv);
  const int steps = std::max(1, (rows + kRpw - 1) / kRpw);
  const int64_t want = (16ll * sms + p.n - 1) / p.n;
  const int chunks = (int)std::min<int64_t>(steps, std::max<int64_t>(1, want));
  p.rows_per_chunk = (steps + chunks - 1) / chunks * kRpw;
  p.chunks = std::max(1, (rows + p.rows_per_chunk - 1) / p.rows_per_chunk);
  const int64_t row_units = rows > 0 ? (int64_t)p.n * p.chunks : 0;
  int64_t ctas = (row_units + kWarpsPerCta - 1) / kWarpsPerCta;
  if (f8) {
    p.q_ctas = (int32_t)ctas;
    p.tile = p.n <= 1024 ? 1 : 4;
    const int64_t units = ((int64_t)p.n + p.tile - 1) / p.tile * p.hkv * 2;
    ctas += (units + kWarpsPerCta - 1) / kWarpsPerCta;
  }
  if (ctas > 0x7fffffffll) return (int)cudaErrorInvalidValue;
  const cudaError_t pe = f8 ? prepare_kernel<rope_append_fp8_kernel<D, kInter>>(0)
                            : prepare_kernel<rope_append_kernel<D, kInter>>(0);
  if (pe != cudaSuccess) return (int)pe;
  profile_begin(PKV_KERNEL_ROPE, a.stream);
  if (f8)
    rope_append_fp8_kernel<D, kInter><<<(unsigned)ctas, kThreads, 0, a.stream>>>(p);
  else
    rope_append_kernel<D, kInter><<<(unsigned)ctas, kThreads, 0, a.stream>>>(p);
  profile_end(PKV_KERNEL_ROPE, a.stream);
  const int e = (int)cudaGetLastError();
  if (!e) count_launches(1);
  return e;
}

}  // namespace

int launch_rope_append(const RopeAppendArgs &a) {
  if (a.desc.head_dim == 128)
    return a.interleaved ? launch_t<128, true>(a) : launch_t<128, false>(a);
  return a.interleaved ? launch_t<64, true>(a) : launch_t<64, false>(a);
}

}  // namespace pkv
