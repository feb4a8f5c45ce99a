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
//   s' = s when first > 0, s > 0 and 448 s >= max |N|, else the smallest power of two
//        >= 2^-64 with 448 s' >= max |N|
//   new rows: rn_sat(x / s');   kept rows, when s' != s: rn(c s / s'), an s that is not
//   positive and finite counting as 0.
// Powers of two make x / s' and c s / s' exact before the rounding, so a kept
// row loses nothing but bits that fall below e4m3's smallest step.
//
// What bounds it: HBM for long chunks.  Per token and head q is read and written, k
// and v are read and written (at half the bytes for the 8-bit pool).  A row of 64 or
// 128 elements lies on 8 or 16 lanes, four rows are in flight a lane, and a token's
// cosines and sines stay in registers across its heads.  35 000 tokens of 40 q and 8 KV
// heads, D = 128: 1.02 GB in 154 us (6.6 TB/s, 0.97 of the copy bandwidth); into the
// 8-bit pool 0.95 GB in 162 us (0.86: k and v are read twice, the second time from L1
// or L2).  Short steps are the launch: 16 decodes 3.0 us (2.7 in a graph), 256 decodes into
// the 8-bit pool 4.3 us (three dependent reads and two barriers).
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
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *q_out;
  int64_t qs, ks, vs, qos;  // token strides
  const float *cos_sin;
  const int32_t *positions;
  const int32_t *slots;
  int32_t max_pos, rot;     // rot = 0: no rotation
  uint64_t zero;            // two fp32 -0 (Lane)
  int32_t n, hq, hkv;
  int32_t num_blocks;
  void *pool;
  float *scales;            // [num_blocks][Hkv][2]
  int32_t chunks, rows_per_chunk;  // rows of a token are cut into chunks, one per warp
  int32_t append_ctas;             // 8-bit pool: CTAs that append; the others rotate q
  int32_t every;                   // 8-bit pool: CTAs 0, every, 2 every, .. append
  int32_t tile;                    // 8-bit pool: tokens whose blocks one CTA looks after
  int32_t *dev_status;
};

// A row of D elements lies on D / 8 lanes, 8 elements a lane, as four pairs to be
// rotated: (a[j], b[j]), j < 4, pair indices 4 l + j.
//   half split:  a = elements 4 l .. 4 l + 3, b = the four R / 2 further on (two
//                8-byte accesses, so no lane needs another's elements);
//   interleaved: a = the even, b = the odd ones of elements 8 l .. 8 l + 7.
// Lanes past the rotated part hold elements 8 l .. 8 l + 7 and pass them through.
// The arithmetic runs on packed fp32 pairs, each product and sum rounded.
template <bool kInter>
struct Lane {
  int a, b;     // element offsets of the lane's two runs of four
  bool turns;
  // two -0, from the launch: a product x y is computed as x y + zero, which changes no
  // bit of it and which the compiler, not knowing the value, cannot fuse with the sum
  // that follows (a packed mul.rn and add.rn came out as one multiply-add)
  uint64_t zero;
  float4 c, s;  // cosines and sines of the lane's pairs at one position

  __device__ __forceinline__ void place(const RopeParams &p, int l) {
    turns = 8 * l < p.rot;
    zero = p.zero;
    a = kInter || !turns ? 8 * l : 4 * l;
    b = kInter || !turns ? 8 * l + 4 : (p.rot >> 1) + 4 * l;
    c = s = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void angles(const RopeParams &p, int pos, int l) {
    if (!turns) return;
    const float *row = p.cos_sin + (int64_t)pos * p.rot + 4 * l;
    c = __ldg(reinterpret_cast<const float4 *>(row));
    s = __ldg(reinterpret_cast<const float4 *>(row + (p.rot >> 1)));
  }
  __device__ __forceinline__ uint4 load(const __nv_bfloat16 *row) const {
    if constexpr (kInter) return ldg128(row + a);
    const uint2 x = ldg64(row + a), y = ldg64(row + b);
    return make_uint4(x.x, x.y, y.x, y.y);
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *row, const uint4 &v) const {
    if constexpr (kInter) {
      *reinterpret_cast<uint4 *>(row + a) = v;
    } else {
      *reinterpret_cast<uint2 *>(row + a) = make_uint2(v.x, v.y);
      *reinterpret_cast<uint2 *>(row + b) = make_uint2(v.z, v.w);
    }
  }
  // the eight elements as fp32 in memory order (y), rotated when `on`
  __device__ __forceinline__ void turn(const uint4 &raw, bool on, float (&y)[8]) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = __uint_as_float(w[i] << 16);
      y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    if (!on || !turns) return;
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      constexpr int kA = kInter ? 2 : 1, kB = kInter ? 1 : 4;  // element of pair j: a kA j, b + kB
      float &a0 = y[kA * j], &a1 = y[kA * (j + 1)], &b0 = y[kA * j + kB], &b1 = y[kA * (j + 1) + kB];
      const uint64_t av = f2_pack(a0, a1), bv = f2_pack(b0, b1);
      const uint64_t cv = f2_pack(cc[j], cc[j + 1]), sv = f2_pack(ss[j], ss[j + 1]);
      const uint64_t nv = f2_pack(-ss[j], -ss[j + 1]);
      f2_unpack(f2_add(f2_fma(av, cv, zero), f2_fma(bv, nv, zero)), a0, a1);
      f2_unpack(f2_add(f2_fma(bv, cv, zero), f2_fma(av, sv, zero)), b0, b1);
    }
  }
};

__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
  return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                    pack_bf16x2(y[6], y[7]));
}

// Rows [r0, r1) of one segment of a token (its q, k or v heads): row r at src + r D,
// written to dst + r * dst_row, rotated or copied.  kU rows of each lane group are
// in flight.
template <int D, bool kInter, bool kTurn>
__device__ __forceinline__ void rows_segment(const Lane<kInter> &ln, const __nv_bfloat16 *src,
                                             __nv_bfloat16 *dst, int64_t dst_row, int r0, int r1,
                                             int sub) {
  constexpr int kRpw = 256 / D, kU = 4;
  for (int r = r0 + sub; r < r1; r += kU * kRpw) {
    uint4 x[kU];
    const __nv_bfloat16 *s = src + r * D;
    __nv_bfloat16 *d = dst + r * dst_row;
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (r + u * kRpw < r1) x[u] = ln.load(s + u * kRpw * D);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (r + u * kRpw >= r1) break;
      if constexpr (kTurn) {
        float y[8];
        ln.turn(x[u], true, y);
        x[u] = pack8(y);
      }
      ln.store(d + u * kRpw * dst_row, x[u]);
    }
  }
}

// Rows of tokens, a chunk of one token's rows per warp: its q heads, then
// (kPool) its k and v heads.
template <int D, bool kInter, bool kPool>
__device__ __forceinline__ void token_rows(const RopeParams &p, int64_t unit, int lane) {
  const int t = (int)(unit / p.chunks), ch = (int)(unit - (int64_t)t * p.chunks);
  if (t >= p.n) return;
  const int l = lane % (D / 8), sub = lane / (D / 8);
  const int rows = p.hq + (kPool ? 2 * p.hkv : 0);
  const int r0 = ch * p.rows_per_chunk, r1 = min(rows, r0 + p.rows_per_chunk);
  const int pos = __ldg(p.positions + t);
  const int64_t slot = kPool ? __ldg(p.slots + t) : -1;
  const bool bad_pos = pos >= p.max_pos;
  if (ch == 0 && lane == 0) {
    // a skipped token's slot is not looked at: padding (pos < 0) may hold any
    if (bad_pos)
      report(p.dev_status, PKV_DEV_BAD_POSITION);
    else if (kPool && pos >= 0 && slot >= (int64_t)p.num_blocks * kBlockSize)
      report(p.dev_status, PKV_DEV_BAD_SLOT);
  }
  if (pos < 0 || bad_pos) return;
  const bool put = kPool && slot >= 0 && slot < (int64_t)p.num_blocks * kBlockSize;
  Lane<kInter> ln;
  ln.place(p, l);
  if (r0 < p.hq + (put ? p.hkv : 0)) ln.angles(p, pos, l);
  if (r0 < p.hq)
    rows_segment<D, kInter, true>(ln, p.q + t * p.qs, p.q_out + t * p.qos, D, r0, min(r1, p.hq),
                                  sub);
  if (put) {
    // head h of K or V: 16 rows of D, this token's at its slot's offset
    constexpr int64_t kHead = kBlockSize * D;
    __nv_bfloat16 *slab = static_cast<__nv_bfloat16 *>(p.pool) +
                          (slot / kBlockSize) * 2 * p.hkv * kHead + slot % kBlockSize * D;
    rows_segment<D, kInter, true>(ln, p.k + t * p.ks, slab, kHead, max(r0 - p.hq, 0),
                                  min(r1 - p.hq, p.hkv), sub);
    rows_segment<D, kInter, false>(ln, p.v + t * p.vs, slab + p.hkv * kHead, kHead,
                                   max(r0 - p.hq - p.hkv, 0), r1 - p.hq - p.hkv, sub);
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

// One CTA: the blocks whose first new token lies among tokens t0 .. t0 + tile - 1 (a
// group each), for up to kSlabHeads KV heads, K and V (a slab each).
//   1. warp 0 finds the groups and lists their tokens (at most tile + 15);
//   2. each lane group takes rows of one token, rotates them, and their largest
//      value goes to its (group, slab)'s maximum in shared memory;
//   3. one thread per (group, slab) settles the scale; lane groups re-express the
//      rows a block holds where its scale grew;
//   4. the lane groups read their rows again (from L1 or L2), rotate, round and
//      store them.
// The lane groups of a CTA are laid out over (tokens x slabs) to fit the number
// of tokens: a whole block's 16 tokens side by side, each with its cosines and
// sines in registers across the slabs, or one decode token's slabs side by side.
constexpr int kMaxTile = 16;
constexpr int kSlabHeads = 8;
constexpr int kMaxSlabs = 2 * kSlabHeads;
struct AppendSmem {
  int n_rows, n_groups;
  int tok[kMaxTile + kWindow], grp[kMaxTile + kWindow], off[kMaxTile + kWindow];
  int pos[kMaxTile + kWindow];
  int blk[kMaxTile], first[kMaxTile];
  uint32_t amax[kMaxTile][kMaxSlabs];
  float scale[kMaxTile][kMaxSlabs], ratio[kMaxTile][kMaxSlabs];  // ratio 1: nothing to re-express
};

template <int D, bool kInter>
__device__ __forceinline__ void append_blocks(const RopeParams &p, int64_t unit, AppendSmem &sm) {
  constexpr int kLpr = D / 8, kLaneGroups = kThreads / kLpr;
  static_assert(kMaxTile * kMaxSlabs <= kThreads, "a thread per (group, slab)");
  const int lane = threadIdx.x & 31;
  const int hc = (p.hkv + kSlabHeads - 1) / kSlabHeads;
  const int64_t t0 = unit / hc * p.tile;
  const int h0 = (int)(unit % hc) * kSlabHeads, nh = min(kSlabHeads, p.hkv - h0), slabs = 2 * nh;
  sm.amax[threadIdx.x / kMaxSlabs][threadIdx.x % kMaxSlabs] = 0;
  if (threadIdx.x < 32) {
    const int64_t nslots = (int64_t)p.num_blocks * kBlockSize;
    // slots and positions of tokens t0 - 32 .. t0 + 31: lane i holds t0 - 32 + i and
    // t0 + i; a token that writes nothing has slot -1
    int32_t slot[2], pos[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t t = t0 + lane - 32 * (1 - i);
      const bool in = t >= 0 && t < p.n;
      slot[i] = in ? __ldg(p.slots + t) : -1;
      pos[i] = in && p.rot > 0 ? __ldg(p.positions + t) : 0;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool bad_pos = p.rot > 0 && pos[i] >= p.max_pos;
      // (a skipped token's slot is not looked at: padding may hold any)
      const bool bad_slot = !bad_pos && pos[i] >= 0 && slot[i] >= nslots;
      if (i == 1 && lane < p.tile && h0 == 0) {
        if (bad_slot) report(p.dev_status, PKV_DEV_BAD_SLOT);
        if (bad_pos) report(p.dev_status, PKV_DEV_BAD_POSITION);
      }
      if (bad_slot || bad_pos || pos[i] < 0 || slot[i] < 0) slot[i] = -1;
    }
    const int32_t blk0 = slot[0] < 0 ? -1 : slot[0] / kBlockSize;
    const int32_t blk1 = slot[1] < 0 ? -1 : slot[1] / kBlockSize;
    const int off = slot[1] < 0 ? kBlockSize : slot[1] % kBlockSize;
    int my_grp = -1, n_groups = 0;
    for (int j = 0; j < p.tile; ++j) {
      const int32_t blk = __shfl_sync(0xffffffffu, blk1, j);
      if (blk < 0) continue;
      // bit 32 + i: token t0 + i writes this block
      const uint64_t same = ((uint64_t)__ballot_sync(0xffffffffu, blk1 == blk) << 32) |
                            __ballot_sync(0xffffffffu, blk0 == blk);
      constexpr uint32_t kBack = (1u << (kWindow - 1)) - 1;
      const uint32_t before = (uint32_t)(same >> (32 + j - (kWindow - 1))) & kBack;
      if (before) {
        // an earlier token's group takes it, unless that token itself follows an
        // earlier one and this one lies outside the first one's window
        const int f = 32 + j - (kWindow - 1) + __ffs((int)before) - 1;
        if ((uint32_t)(same >> (f - (kWindow - 1))) & kBack) {
          if (lane == 0 && h0 == 0) report(p.dev_status, PKV_DEV_BAD_SLOT);
        }
        continue;
      }
      const uint32_t members = (uint32_t)(same >> (32 + j)) & 0xffffu;  // token t0 + j + i
      const bool mine = lane >= j && lane < j + kWindow && ((members >> (lane - j)) & 1);
      const int first = __reduce_min_sync(0xffffffffu, mine ? off : kBlockSize);
      if (mine) my_grp = n_groups;
      if (lane == 0) {
        sm.blk[n_groups] = blk;
        sm.first[n_groups] = first;
      }
      ++n_groups;
    }
    const uint32_t listed = __ballot_sync(0xffffffffu, my_grp >= 0);
    if (my_grp >= 0) {
      const int at = __popc(listed & ((1u << lane) - 1));
      sm.tok[at] = lane;
      sm.grp[at] = my_grp;
      sm.off[at] = off;
      sm.pos[at] = pos[1];
    }
    if (lane == 0) {
      sm.n_rows = __popc(listed);
      sm.n_groups = n_groups;
    }
  }
  __syncthreads();
  const int n_rows = sm.n_rows, n_groups = sm.n_groups;
  if (n_rows == 0) return;
  // slab sl: K of head h0 + sl for sl < nh, then V of head h0 + sl - nh
  const int tg = threadIdx.x / kMaxSlabs, ts = threadIdx.x % kMaxSlabs;
  const bool settles = tg < n_groups && ts < slabs;  // this thread's (group, slab)
  float *scale_at = nullptr;
  float s_old = 0.f;
  if (settles) {
    const int kv = ts >= nh;
    scale_at = p.scales + ((int64_t)sm.blk[tg] * p.hkv + h0 + ts - kv * nh) * 2 + kv;
    if (sm.first[tg] > 0) s_old = __ldcg(scale_at);
  }
  const int l = lane % kLpr, lg = threadIdx.x / kLpr;
  // lane groups side by side over the tokens (a power of two of them); the rest
  // of the layout is over the slabs
  int by_tok = 1;
  while (by_tok < n_rows && by_tok < kLaneGroups) by_tok *= 2;
  const int by_slab = kLaneGroups / by_tok;
  const int r0 = lg % by_tok, sl0 = lg / by_tok;
  Lane<kInter> ln;
  ln.place(p, l);

  // both passes: the rows of this lane group's tokens, slab by slab
  constexpr int kU = 4;
  auto each_row = [&](auto &&start, auto &&use, auto &&batch_end) {
    for (int r = r0; r < n_rows; r += by_tok) {
      const int64_t t = t0 + sm.tok[r];
      ln.angles(p, sm.pos[r], l);
      const __nv_bfloat16 *kt = p.k + t * p.ks + h0 * D, *vt = p.v + t * p.vs + h0 * D;
      start(r);
      for (int sl = sl0; sl < slabs; sl += kU * by_slab) {
        uint4 x[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int su = sl + u * by_slab;
          if (su < slabs) x[u] = ln.load(su < nh ? kt + su * D : vt + (su - nh) * D);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int su = sl + u * by_slab;
          if (su >= slabs) break;
          float y[8];
          ln.turn(x[u], su < nh, y);
          use(su, u, y);
        }
        batch_end(sl);
      }
    }
  };
  // a batch's kU largest values per lane are reduced together over the row's lanes:
  // each exchange halves the values a lane holds, until lane l holds one slab's
  uint32_t *amax_row = nullptr;
  float top[kU];
  const uint32_t group_mask = (kLpr == 32 ? 0xffffffffu : (1u << kLpr) - 1) << (lane - l);
  each_row(
      [&](int r) {
        amax_row = sm.amax[sm.grp[r]];
#pragma unroll
        for (int u = 0; u < kU; ++u) top[u] = 0.f;
      },
      [&](int, int u, const float (&y)[8]) {
        float a = max3(max3(fabsf(y[0]), fabsf(y[1]), fabsf(y[2])),
                       max3(fabsf(y[3]), fabsf(y[4]), fabsf(y[5])),
                       fmaxf(fabsf(y[6]), fabsf(y[7])));
        if (!(a <= FLT_MAX)) {  // infinities saturate: they do not count (nor does NaN)
          a = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(y[e]) <= FLT_MAX ? fabsf(y[e]) : 0.f);
        }
        top[u] = a;
      },
      [&](int sl) {
        static_assert(kU == 4, "two halving exchanges");
        const bool hi = (l & 1) != 0, hi2 = (l & 2) != 0;
        const float s0 = hi ? top[0] : top[2], s1 = hi ? top[1] : top[3];
        float k0 = hi ? top[2] : top[0], k1 = hi ? top[3] : top[1];
        k0 = fmaxf(k0, __shfl_xor_sync(group_mask, s0, 1));
        k1 = fmaxf(k1, __shfl_xor_sync(group_mask, s1, 1));
        float m = fmaxf(hi2 ? k1 : k0, __shfl_xor_sync(group_mask, hi2 ? k0 : k1, 2));
#pragma unroll
        for (int o = 4; o < kLpr; o <<= 1) m = fmaxf(m, __shfl_xor_sync(group_mask, m, o));
        const int su = sl + ((hi ? 2 : 0) + (hi2 ? 1 : 0)) * by_slab;
        if (l < 4 && su < slabs) atomicMax(&amax_row[su], __float_as_uint(m));
#pragma unroll
        for (int u = 0; u < kU; ++u) top[u] = 0.f;
      });
  __syncthreads();
  if (settles) {
    const float amax = __uint_as_float(sm.amax[tg][ts]);
    if (!(s_old > 0.f && s_old <= FLT_MAX)) s_old = 0.f;  // not a scale: its rows become zeros
    const bool keep = s_old > 0.f && s_old * kE4m3Max >= amax;
    const float s_new = keep ? s_old : pow2_scale(amax);
    sm.scale[tg][ts] = s_new;
    sm.ratio[tg][ts] = keep || sm.first[tg] == 0 ? 1.f : s_old / s_new;
    if (!keep) *scale_at = s_new;
  }
  __syncthreads();
  // the K slab of head h0 of group g's block; slab sl lies slab_off(sl) further on
  constexpr int kSlab = kBlockSize * D;
  auto block_of = [&](int g) {
    return static_cast<uint8_t *>(p.pool) + ((int64_t)sm.blk[g] * 2 * p.hkv + h0) * kSlab;
  };
  auto slab_off = [&](int sl) { return (sl < nh ? sl : p.hkv + sl - nh) * kSlab; };
  const float *scale_row = nullptr;
  uint8_t *row = nullptr;
  each_row(
      [&](int r) {
        scale_row = sm.scale[sm.grp[r]];
        row = block_of(sm.grp[r]) + sm.off[r] * D;
      },
      [&](int sl, int, const float (&y)[8]) {
        const float s = scale_row[sl];
        float z[8];
        if ((__float_as_uint(s) & 0x7fffffu) == 0 && s >= 0x1p-120f && s <= 0x1p120f) {
          // a power of two: the product with its reciprocal is exact
          const float inv = __uint_as_float((254u << 23) - __float_as_uint(s));
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = y[e] * inv;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = __fdiv_rn(y[e], s);
        }
        uint2 w;
        w.x = f32x2_to_e4m3x2(z[0], z[1]) | (f32x2_to_e4m3x2(z[2], z[3]) << 16);
        w.y = f32x2_to_e4m3x2(z[4], z[5]) | (f32x2_to_e4m3x2(z[6], z[7]) << 16);
        uint8_t *at = row + slab_off(sl);
        if constexpr (kInter) {
          *reinterpret_cast<uint2 *>(at + ln.a) = w;
        } else {
          *reinterpret_cast<uint32_t *>(at + ln.a) = w.x;
          *reinterpret_cast<uint32_t *>(at + ln.b) = w.y;
        }
      },
      [](int) {});
  // rows the blocks already hold, where a scale grew
  for (int i = lg; i < n_groups * slabs; i += kLaneGroups) {
    const int g = i / slabs, sl = i % slabs;
    const float ratio = sm.ratio[g][sl];
    if (ratio == 1.f) continue;
    uint2 *at = reinterpret_cast<uint2 *>(block_of(g) + slab_off(sl)) + l;
    for (int r = 0; r < sm.first[g]; ++r, at += D / 8) {
      const uint2 w = __ldcg(at);
      auto requant = [&](uint32_t v) {
        const uint32_t a = e4m3x2_to_f16x2(v), b = e4m3x2_to_f16x2(v >> 16);
        const float2 fa = __half22float2(*reinterpret_cast<const __half2 *>(&a));
        const float2 fb = __half22float2(*reinterpret_cast<const __half2 *>(&b));
        return f32x2_to_e4m3x2(fa.x * ratio, fa.y * ratio) |
               (f32x2_to_e4m3x2(fb.x * ratio, fb.y * ratio) << 16);
      };
      *at = make_uint2(requant(w.x), requant(w.y));
    }
  }
}

// Launched early behind the preceding kernel, whose completion is waited for before
// anything is read.  No early release of the next kernel: the attention kernels read
// q before they wait for this one, so q_out has to be complete and visible when they
// start (the pool is read after that wait).
template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads, 4) rope_append_kernel(const RopeParams p) {
  pdl_wait();
  const int64_t unit = (int64_t)blockIdx.x * kWarpsPerCta + (threadIdx.x >> 5);
  token_rows<D, kInter, true>(p, unit, threadIdx.x & 31);
  __threadfence();
}

// Appending CTAs wait on shared memory and barriers, those that rotate q on HBM.  A
// grid of more than one wave takes one appending CTA in every p.every, so that the
// two kinds share the SMs (35 000 tokens: 179 -> 164 us); in a single wave the
// appending ones come first, theirs is the longer chain of dependent steps (256
// decodes: 4.3 us, against 4.8 us spread).
template <int D, bool kInter>
__global__ void __launch_bounds__(kThreads, 4) rope_append_fp8_kernel(const RopeParams p) {
  __shared__ AppendSmem sm;
  pdl_wait();
  const int b = (int)blockIdx.x, at = b / p.every;
  if (b % p.every == 0 && at < p.append_ctas) {
    append_blocks<D, kInter>(p, at, sm);
  } else {
    const int before = min(at + (b % p.every > 0 ? 1 : 0), p.append_ctas);
    token_rows<D, kInter, false>(p, (int64_t)(b - before) * kWarpsPerCta + (threadIdx.x >> 5),
                                 threadIdx.x & 31);
    __threadfence();
  }
}

template <int D, bool kInter>
int launch_t(const RopeAppendArgs &a) {
  constexpr int kRpw = 32 / (D / 8);
  RopeParams p;
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.k = static_cast<const __nv_bfloat16 *>(a.k);
  p.v = static_cast<const __nv_bfloat16 *>(a.v);
  p.q_out = static_cast<__nv_bfloat16 *>(a.q_out);
  p.qs = a.q_stride;
  p.ks = a.k_stride;
  p.vs = a.v_stride;
  p.qos = a.q_out_stride;
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
  p.zero = 0x8000000080000000ull;
  p.tile = 1;
  p.append_ctas = 0;
  p.every = 1;
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
    // about four CTAs an SM, if the tokens are that many
    const int64_t hc = (p.hkv + kSlabHeads - 1) / kSlabHeads;
    p.tile = 1;
    while (p.tile < kMaxTile &&
           ((int64_t)p.n + 2 * p.tile - 1) / (2 * p.tile) * hc >= 4ll * sms)
      p.tile *= 2;
    const int64_t units = ((int64_t)p.n + p.tile - 1) / p.tile * hc;
    if (units + ctas > 0x7fffffffll) return (int)cudaErrorInvalidValue;
    p.append_ctas = (int32_t)units;
    ctas += units;
    if (ctas > 4ll * sms) p.every = (int32_t)(ctas / units);
  }
  if (ctas > 0x7fffffffll) return (int)cudaErrorInvalidValue;
  const cudaError_t pe = f8 ? prepare_kernel<rope_append_fp8_kernel<D, kInter>>(0)
                            : prepare_kernel<rope_append_kernel<D, kInter>>(0);
  if (pe != cudaSuccess) return (int)pe;
  profile_begin(PKV_KERNEL_ROPE, a.stream);
  cudaError_t e = launch_kernel(
      f8 ? rope_append_fp8_kernel<D, kInter> : rope_append_kernel<D, kInter>,
      dim3((unsigned)ctas), dim3(kThreads), 0, a.stream, !profiling_active(), p);
  profile_end(PKV_KERNEL_ROPE, a.stream);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e == cudaSuccess) count_launches(1);
  return (int)e;
}

}  // namespace

int launch_rope_append(const RopeAppendArgs &a) {
  if (a.desc.head_dim == 128)
    return a.interleaved ? launch_t<128, true>(a) : launch_t<128, false>(a);
  return a.interleaved ? launch_t<64, true>(a) : launch_t<64, false>(a);
}

}  // namespace pkv
