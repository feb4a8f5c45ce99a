// Split-KV paged attention over an 8-bit pool: e4m3 values with one fp32 scale for
// each block of 16 tokens, KV head and K or V.
//
// The work, its order and its results are those of the bf16 kernel (pkv_decode.cu):
// one plan, pieces of equal cost per warp, row groups of at most 16 query rows, the
// same partial slots and merge.  With K8, V8 the stored values and ks, vs a block's
// scales it computes
//   x = (q . K8) ks scale log2 e,   w = 2^(x - m),   out = sum w vs V8 / sum w
// with m the running maximum of x.
//
// What bounds it.  A block of a head is 4 KB at D = 128, half a bf16 one, so at
// HBM's rate an SM has ~180 cycles for a block that took a bf16 warp ~200
// instructions.  The first version (the bf16 kernel's products on converted K and V,
// a block at a time, ~500 instructions a block) streamed 1.13 GB in 235 us where HBM
// needs 166: bound by instruction issue at 2 warps a scheduler.  Hence:
//  * The products are transposed, S^T = K Q^T and O^T = V^T P^T: keys and head_dims are
//    the 16-row side of an m16n8k16 product and the query rows the 8-column side, so a
//    row group of at most 8 rows (one token of up to 8 query heads a KV head, a verify
//    pair of 4) takes half the products, exponentials and accumulators; larger ones
//    take two column tiles.  The 8 x 8 transposes of P^T between the two products are
//    one movmatrix each.
//  * Both products run on fp16 operands with fp32 sums.  e4m3 values are exact in fp16;
//    a row of q is scaled by a power of two so that its largest value lies in [2^14,
//    2^15): fp16 then holds every bf16 value down to 2^-28 of the row's largest exactly
//    and smaller ones to 2^-39 of it.  (q in two e4m3 parts on the 8-bit mma.sync, which
//    needs no conversion of K, was right and slower: 239 us for the 256 decodes, where
//    this form then took 196.)
//  * V8 is read as fragments by ldmatrix (16 x 16 bytes, transposed), whose register
//    holds four keys of one head_dim: two fp16 pairs, no byte shuffling.  The weights
//    carry vs, relative to the largest V scale seen so far: u = w vs / vref * 2^14,
//    rounded to fp16 (2^-11; smallest step 2^-38 of the largest weight, at the largest V
//    scale) where bf16 would round to 2^-8.
//  * Two consecutive blocks are a stage of the ring (one barrier) and are attended
//    together: one maximum, one rescale, and independent chains of products.
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "pkv_decode.cuh"

namespace pkv {

namespace {

constexpr int kPair = 2;          // blocks of a stage
constexpr int kFillArrivals = 4;  // two lanes fill a stage, two arrivals each
constexpr float kUScale = 16384.f;  // 2^14: the largest weight as fp16

template <int D>
struct Stage8 {
  static constexpr int kSlabBytes = kBlockSize * D;  // K or V of one block
  static constexpr int kBlockBytes = 2 * kSlabBytes;
  static constexpr int kStageBytes = kPair * kBlockBytes;
};
// NT: the column tiles of the largest row group (1: at most 8 rows).
template <int D, int NT>
struct Decode8Cfg : Stage8<D> {
  // CTAs an SM: with one column tile a lane's state fits 128 registers (126 at D = 64; at
  // D = 128 but for 72 bytes of spills), so 16 warps (8 warps and 3 stages, 256 decodes:
  // 193 us, 12 and 2: 184, 16 and 1: 180).  With two
  // it does not (12 warps spill: 107 -> 152 us on 64 windows of 2 to 4 tokens).  Stages a
  // warp: 16 KB at D = 128, 8 KB at D = 64, where they fit; more ran slower (256 decodes
  // of 16 heads a KV head: 3 stages 130 us, 2 120, 1 133).
  static constexpr int kCtas = NT == 1 ? 4 : 2;
  static constexpr int kStages = NT == 1 && D == 128 ? 1 : 2;

  static constexpr int kRingBytes = kStages * Stage8<D>::kStageBytes;
  static constexpr int kScaleOffset = kWarps * kRingBytes;  // float2 x 2 a stage
  // a shared-prefix CTA uses as many empty barriers as full ones
  static constexpr int kBarOffset = kScaleOffset + kWarps * kStages * kPair * 8;
  static constexpr int kFlagOffset = kBarOffset + 2 * kWarps * kStages * 8;  // int x 2 a stage
  static constexpr int kSmemBytes = kFlagOffset + kWarps * kStages * kPair * 4 + 1024;
};

// A row group's running state in one lane: query rows 8 t + 2 c + j, t < NT, j < 2
// (NT column tiles: 1 for a row group of at most 8 rows, else 2), and this lane's
// fragments of q and O.
template <int D, int NT>
struct Rows {
  float m[NT][2];        // running maximum of x
  float l[NT][2];        // this lane's part of sum w
  float qs[NT][2];       // from a product to x, but for the block's K scale
  int lim[NT][2];        // last visible key
  float vref, inv_vref;  // the largest V scale seen; O is in units of vref / 2^14
  uint32_t q[D / 16][NT][2];
  float o[D / 16][NT][4];  // head_dims 16 i + r (+ 8 in the last two), rows 8 t + 2 c, + 1
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[t][j] = -INFINITY;
        l[t][j] = 0.f;
      }
    vref = inv_vref = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) o[i][t][0] = o[i][t][1] = o[i][t][2] = o[i][t][3] = 0.f;
  }
};

// 8 x 8 transpose across the warp: lane (r, c) gives row r, columns 2 c and 2 c + 1, and
// gets row r, columns 2 c and 2 c + 1 of the transposed matrix.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
// Two 16 x 16 byte matrices, transposed: register 2 m + i holds keys 4 (lane % 4) ..
// + 3 of column 8 i + lane / 4 of matrix m; lane j < 16 gives row j of matrix 0, lane
// 16 + j of matrix 1.
__device__ __forceinline__ void ldmatrix_t8x2(uint32_t (&v)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}

// Byte offset of 16-byte chunk `chunk` of key row `row` of a slab as the box lands
// it: rows of D bytes, swizzled over D bytes (128: chunk ^ row % 8; 64: two rows
// to 128 bytes, chunk ^ (row / 2) % 4).
template <int D>
__device__ __forceinline__ uint32_t slab_off(int row, int chunk) {
  return D == 128 ? (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4))
                  : (uint32_t)(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}

// q as B fragments (k16 x n8) in fp16, and what belongs to its rows: row 8 t + r of the
// row group's R rows (token row / G, head h * G + row % G from packed query row q_row0;
// rows >= R read as zeros and see no key).  Lane (r, c) of step 4 L + i holds head_dims
// 16 e + 4 i .. + 3 of chunk e = c D / 64 + L, the ones its K chunk loads supply.  A row
// that holds an infinity becomes NaN.  The sign of the softmax scale goes into q (a
// scale of 0 makes q zero), so x grows with the products.
template <int D, int NT>
__device__ __forceinline__ void load_rows(const DecodeParams &p, int q_row0, int R, int h,
                                          int q_pos0, int r, int c, Rows<D, NT> &rows) {
  constexpr int kL = D / 64;  // 16-element chunks per lane per row
  const int G = p.group;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row = r + 8 * t;
    const bool rv = row < R;
    const __nv_bfloat16 *qrow =
        p.q + ((int64_t)(q_row0 + (rv ? row / G : 0)) * p.num_q_heads + h * G +
               (rv ? row % G : 0)) * D + 16 * kL * c;
    uint4 raw[2 * kL];
#pragma unroll
    for (int i = 0; i < 2 * kL; ++i) raw[i] = rv ? ldg128_nc(qrow + 8 * i) : make_uint4(0, 0, 0, 0);
    const uint32_t *w = reinterpret_cast<const uint32_t *>(raw);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8 * kL; ++i)
      top = max3(top, fabsf(__uint_as_float(w[i] << 16)),
                 fabsf(__uint_as_float(w[i] & 0xffff0000u)));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = (int)(__float_as_uint(top) >> 23);  // biased exponent of the largest
    const int f = min(268 - e, 253);                  // of 2^(14 - exponent)
    const float sl2 = p.scale_log2;
    float up = e == 255 ? __int_as_float(0x7fc00000) : __uint_as_float((uint32_t)f << 23);
    float down = e == 255 ? 1.f : __uint_as_float((uint32_t)(254 - f) << 23);
    if (sl2 < 0.f) up = -up;
    if (sl2 == 0.f) up = 0.f;
    down = sl2 == 0.f ? 1.f : down * fabsf(sl2);
#pragma unroll
    for (int i = 0; i < 8 * kL; ++i)
      rows.q[i >> 1][t][i & 1] = pack_f16x2(__uint_as_float(w[i] << 16) * up,
                                            __uint_as_float(w[i] & 0xffff0000u) * up);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      rows.qs[t][j] = __shfl_sync(0xffffffffu, down, 4 * (2 * c + j));
      const int mine = 8 * t + 2 * c + j;
      rows.lim[t][j] = mine < R ? q_pos0 + mine / G : -1;
    }
  }
}

// Two blocks of a stage in shared memory: sc holds their scales (K0, V0, K1, V1), p0 the
// position of each one's first key (kNoBlock: no block, every key is masked).
constexpr int kNoBlock = 1 << 30;

template <int D, int NT>
__device__ __forceinline__ void attend_pair(uint32_t stage, const float4 sc, const int (&p0)[kPair],
                                            int q_pos0, int ctx, int lane, Rows<D, NT> &rows) {
  constexpr int kSlab = Stage8<D>::kSlabBytes;
  const int r = lane >> 2, c = lane & 3;
  // ---- S^T.  Row i of a tile is key 4 (i % 8 / 2) + 2 (i / 8) + i % 2 of the block: once
  // transposed, lane c holds keys 4 c .. 4 c + 3, as ldmatrix gives V
  const int key0 = 4 * (r >> 1) + (r & 1);
  float s[kPair][NT][4];  // keys key0 (first two) and key0 + 2; rows 2 c, 2 c + 1 of tile t
#pragma unroll
  for (int b = 0; b < kPair; ++b)
#pragma unroll
    for (int t = 0; t < NT; ++t) s[b][t][0] = s[b][t][1] = s[b][t][2] = s[b][t][3] = 0.f;
#pragma unroll
  for (int L = 0; L < D / 64; ++L) {
    const int chunk = D == 128 ? 2 * c + L : c;
    uint4 kv[kPair][2];
#pragma unroll
    for (int b = 0; b < kPair; ++b) {
      kv[b][0] = lds128(stage + b * 2 * kSlab + slab_off<D>(key0, chunk));
      kv[b][1] = lds128(stage + b * 2 * kSlab + slab_off<D>(key0 + 2, chunk));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int b = 0; b < kPair; ++b) {
        const uint4 &x = kv[b][0], &y = kv[b][1];
        const uint32_t w0 = i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
        const uint32_t w1 = i == 0 ? y.x : i == 1 ? y.y : i == 2 ? y.z : y.w;
        const uint32_t a0 = e4m3x2_to_f16x2(w0), a2 = e4m3x2_to_f16x2(w0 >> 16);
        const uint32_t a1 = e4m3x2_to_f16x2(w1), a3 = e4m3x2_to_f16x2(w1 >> 16);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma_16816_f16(s[b][t], a0, a1, a2, a3, rows.q[4 * L + i][t][0], rows.q[4 * L + i][t][1]);
      }
  }
  if (max(p0[0], p0[1]) + kBlockSize - 1 > q_pos0) {
#pragma unroll
    for (int b = 0; b < kPair; ++b)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (p0[b] + key0 + (j & 2) > rows.lim[t][j & 1]) s[b][t][j] = -INFINITY;
  }
  // A block past the context (not there, or one that a later step of a chain will fill)
  // weighs nothing, and its V scale, which may hold anything, is not looked at.  Its K
  // scale needs no care: a masked -inf times any f > 0 below stays -inf.
  const float vs[kPair] = {p0[0] < ctx ? sc.y : 0.f, p0[1] < ctx ? sc.w : 0.f};
  const float vmax = fmaxf(vs[0], vs[1]);
  float down = 1.f;
  if (vmax > rows.vref) {  // the same in every lane
    down = rows.vref / vmax;
    rows.vref = vmax;
    rows.inv_vref = 1.f / vmax;
  }
  // ---- weights: the running maximum, their sum, and as fp16 with their V scale
  uint32_t pb[kPair][NT][2];
  float alpha[NT][2];
  bool moved = down != 1.f;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    // f > 0, so the largest product is the largest x; kept off zero, where a masked
    // -inf would become NaN
    constexpr float kTiny = 1.17549435e-38f;
    float f[kPair][2], nbase[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      f[0][j] = fmaxf(rows.qs[t][j] * sc.x, kTiny);
      f[1][j] = fmaxf(rows.qs[t][j] * sc.z, kTiny);
      float mx = fmaxf(fmaxf(s[0][t][j], s[0][t][2 + j]) * f[0][j],
                       fmaxf(s[1][t][j], s[1][t][2 + j]) * f[1][j]);
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      mx = fmaxf(rows.m[t][j], mx);
      const float base = mx == -INFINITY ? 0.f : mx;  // a row that has seen no key
      const float a = fast_exp2(rows.m[t][j] - base);
      rows.m[t][j] = mx;
      rows.l[t][j] *= a;
      alpha[t][j] = a * down;
      moved |= a != 1.f;
      nbase[j] = -base;
    }
    uint64_t sum = 0;
    const uint64_t nb = f2_pack(nbase[0], nbase[1]);
#pragma unroll
    for (int b = 0; b < kPair; ++b) {
      const float g = vs[b] * rows.inv_vref * kUScale;
      const uint64_t fb = f2_pack(f[b][0], f[b][1]);
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        float e0, e1;
        f2_unpack(f2_fma(f2_pack(s[b][t][2 * hh], s[b][t][2 * hh + 1]), fb, nb), e0, e1);
        e0 = fast_exp2(e0);
        e1 = fast_exp2(e1);
        sum = f2_add(sum, f2_pack(e0, e1));
        pb[b][t][hh] = transpose8(pack_f16x2(e0 * g, e1 * g));
      }
    }
    float x, y;
    f2_unpack(sum, x, y);
    rows.l[t][0] += x;
    rows.l[t][1] += y;
  }
  if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        rows.o[i][t][0] *= alpha[t][0];
        rows.o[i][t][1] *= alpha[t][1];
        rows.o[i][t][2] *= alpha[t][0];
        rows.o[i][t][3] *= alpha[t][1];
      }
  }
  // ---- O^T += V8^T u; rows of V at or past the context end (stale bytes, NaN codes
  // among them) are read as zeros: 0 x NaN would reach O
#pragma unroll
  for (int b = 0; b < kPair; ++b) {
    const uint32_t sv = stage + b * 2 * kSlab + kSlab;
    const int left = ctx - p0[b] - 4 * c;  // keys of this lane's four that are the sequence's
    const bool edge = p0[b] + kBlockSize > ctx;
    const uint32_t keep = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
#pragma unroll
    for (int m = 0; m < D / 32; ++m) {
      uint32_t v[4];
      ldmatrix_t8x2(v, sv + slab_off<D>(lane & 15, 2 * m + (lane >> 4)));
      if (edge) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] &= keep;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t a0 = e4m3x2_to_f16x2(v[2 * k]), a2 = e4m3x2_to_f16x2(v[2 * k] >> 16);
        const uint32_t a1 = e4m3x2_to_f16x2(v[2 * k + 1]), a3 = e4m3x2_to_f16x2(v[2 * k + 1] >> 16);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          mma_16816_f16(rows.o[2 * m + k][t], a0, a1, a2, a3, pb[b][t][0], pb[b][t][1]);
      }
    }
  }
}

// A whole segment writes the normalised bf16 output (8 x 8 tiles of O^T transposed, so
// that a lane stores two head_dims of a row); a split piece its fp32 partial (O, m, l).
template <int D, int NT>
__device__ __forceinline__ void write_rows(const DecodeParams &p, int part, int64_t row0, int h,
                                           const Rows<D, NT> &rows, int R, int r, int c) {
  const int G = p.group;
  const float unit = rows.vref * (1.f / kUScale);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float l[2], f[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      l[j] = rows.l[t][j];
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) l[j] += __shfl_xor_sync(0xffffffffu, l[j], d);
      f[j] = part >= 0 ? unit : l[j] > 0.f ? unit / l[j] : 0.f;
    }
    if (part < 0) {
      const int row = 8 * t + r;
      __nv_bfloat16 *dst =
          p.out + ((row0 + row / G) * p.num_q_heads + h * G + row % G) * D + 2 * c;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const float *o = rows.o[i][t];
        const uint32_t x = transpose8(pack_bf16x2(o[0] * f[0], o[1] * f[1]));
        const uint32_t y = transpose8(pack_bf16x2(o[2] * f[0], o[3] * f[1]));
        if (row < R) {
          *reinterpret_cast<uint32_t *>(dst + 16 * i) = x;
          *reinterpret_cast<uint32_t *>(dst + 16 * i + 8) = y;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = 8 * t + 2 * c + j;
        if (row >= R) continue;
        float *dst = p.part_o + ((int64_t)part * kRowsPerTile + row) * D + r;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          dst[16 * i] = rows.o[i][t][j] * f[j];
          dst[16 * i + 8] = rows.o[i][t][2 + j] * f[j];
        }
        if (r == 0)
          p.part_ml[(int64_t)part * kRowsPerTile + row] = make_float2(rows.m[t][j], l[j]);
      }
    }
  }
}

// A ring of stages and its producer: lanes 0 and 1 of the issuing warp each fill
// one block of a stage (a box of its K and V slabs, and its two scales), or mark
// it bad; a stage's barrier completes after both.
template <int D>
struct Ring {
  uint32_t base, bars, scales;  // shared memory addresses
  int *flags;
  // block `lane` (of n) of the stage: physical block `phys` of KV head h; code: what to
  // report when it is not one of the pool's (0: nothing, there is no such block)
  __device__ __forceinline__ void fill(const CUtensorMap &map, const DecodeParams &p, int stage,
                                       int lane, int n, int phys, int h, int code) const {
    using C = Stage8<D>;
    if (lane >= kPair) return;
    const uint32_t bar = bars + stage * 8;
    const bool has = lane < n;
    const bool ok = has && code != PKV_DEV_PLAN_MISMATCH && phys >= 0 && phys < p.num_blocks;
    flags[stage * kPair + lane] = ok ? 1 : 0;
    if (ok) {
      mbar_arrive_expect_tx(bar, C::kBlockBytes);
      tma_load_4d(base + stage * C::kStageBytes + lane * C::kBlockBytes, &map, 0, 0, h, phys * 2,
                  bar);
      cp_async_8(scales + (stage * kPair + lane) * 8,
                 p.kv_scales + (int64_t)phys * p.num_kv_heads + h);
      cp_async_arrive(bar);
    } else {
      if (has) report(p.dev_status, code);
      mbar_arrive(bar);
      mbar_arrive(bar);
    }
  }
  // what the consumers read of a stage once its barrier completed; the scales of a block
  // that is not there (kNoBlock) may be anything
  __device__ __forceinline__ float4 scale_of(int stage, int n, int kb, int (&p0)[kPair]) const {
    const uint4 v = lds128(scales + stage * kPair * 8);
    const float4 sc = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                            __uint_as_float(v.w));
    const int2 ok = *reinterpret_cast<const int2 *>(flags + stage * kPair);
    p0[0] = ok.x ? kb * kBlockSize : kNoBlock;
    p0[1] = n > 1 && ok.y ? (kb + 1) * kBlockSize : kNoBlock;
    return sc;
  }
};

// Shared-block CTA: as in pkv_decode.cu, two pairs of warps, each pair streaming a chain
// of items once for two row groups through a ring pooled from its two warps' rings.
template <int D, int MAXT>
__device__ __forceinline__ void shared_cta8(const CUtensorMap &pool_map, const DecodeParams &p,
                                            uint8_t *smem, int warp, int lane) {
  using C = Decode8Cfg<D, MAXT>;
  constexpr int kS = kSharedRowGroups * C::kStages;  // stages of a pair's pooled ring
  const int r = lane >> 2, c = lane & 3;
  const int G = p.group, hkv = p.num_kv_heads;
  const int pair = warp / kSharedRowGroups, lw = warp % kSharedRowGroups;
  const int head = (blockIdx.x - p.num_indep_ctas) * kSharedItemsPerCta + pair;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kBarOffset) + pair * 2 * kS;
  uint64_t *empty = full + kS;
  Ring<D> ring;
  ring.base = smem_u32(smem + pair * kSharedRowGroups * C::kRingBytes);
  ring.bars = smem_u32(full);
  ring.scales = smem_u32(smem + C::kScaleOffset) + pair * kS * kPair * 8;
  ring.flags = reinterpret_cast<int *>(smem + C::kFlagOffset) + pair * kS * kPair;
  if (lw == 0 && lane == 0) {
    for (int s = 0; s < kS; ++s) {
      mbar_init(smem_u32(&full[s]), kFillArrivals);
      mbar_init(smem_u32(&empty[s]), kSharedRowGroups);
    }
    fence_mbar_init();
  }
  auto item_ok = [&](const SharedItem &it) {
    return it.seq0 >= 0 && it.seq0 < p.num_seqs && it.h >= 0 && it.h < hkv && it.kb_begin >= 0 &&
           it.kb_begin <= it.kb_end && it.kb_end <= p.max_blocks_per_seq && it.n_rg >= 1 &&
           it.n_rg <= kSharedRowGroups;
  };
  auto next_of = [&](int idx, const SharedItem &it) {
    return it.next > idx && it.next < p.num_shared_items ? it.next : -1;
  };
  const int first = head < p.num_shared_items ? head : -1;

  // ---- producer state (the pair's first warp, uniform): item p_idx, its next block
  // p_j of p_n, and a table window (lane i holds entry win_base + i)
  int p_idx = first, p_j = 0, p_n = 0, p_seq = 0, p_h = 0, p_kb0 = 0, p_next = -1;
  int win_base = 0, win_val = -1;
  auto p_window = [&](int kb) {
    win_base = kb;
    win_val = kb + lane < p_kb0 + p_n
                  ? __ldg(p.block_tables + (int64_t)p_seq * p.max_blocks_per_seq + kb + lane)
                  : -1;
  };
  auto p_load = [&](int idx) {
    const SharedItem &it = p.shared[idx];
    const bool ok = item_ok(it);
    p_seq = ok ? it.seq0 : 0;
    p_h = ok ? it.h : 0;
    p_kb0 = ok ? it.kb_begin : 0;
    p_n = ok ? it.kb_end - it.kb_begin : 0;
    p_next = next_of(idx, it);
    p_j = 0;
    p_window(p_kb0);
  };
  // true when the chain still has a block to issue (moving to later items)
  auto p_more = [&]() {
    while (p_idx >= 0 && p_j >= p_n) {
      p_idx = p_next;
      if (p_idx >= 0) p_load(p_idx);
    }
    return p_idx >= 0;
  };
  if (lw == 0 && first >= 0) p_load(first);

  // ---- the consumers' current item
  int c_idx = first, c_h = 0, c_kb0 = 0, c_kb1 = 0, c_next = -1;
  SharedRowGroup rg;
  int cu0 = 0, qs = 0, ctx = 0;
  bool has_rg = false, mine = false;
  auto c_setup = [&]() {  // both warps: item c_idx's row group and lengths
    const SharedItem &it = p.shared[c_idx];
    const bool ok = item_ok(it);
    const int n_rg = it.n_rg;
    if (!ok && n_rg != 0 && lw == 0 && lane == 0) report(p.dev_status, PKV_DEV_PLAN_MISMATCH);
    c_h = ok ? it.h : 0;
    c_kb0 = ok ? it.kb_begin : 0;
    c_kb1 = ok ? it.kb_end : 0;
    c_next = next_of(c_idx, it);
    rg.seq = -1;
    rg.qi0 = rg.n_q = rg.q_row0 = 0;
    rg.part = -1;
    has_rg = ok && lw < n_rg;
    if (has_rg) rg = it.rg[lw];
    mine = has_rg && rg.seq >= 0 && rg.seq < p.num_seqs && rg.qi0 >= 0 && rg.n_q >= 1 &&
           rg.n_q * G <= 8 * MAXT && rg.q_row0 >= 0 && rg.q_row0 + rg.n_q <= p.total_q;
    cu0 = qs = ctx = 0;
    if (mine) {
      cu0 = __ldg(p.cu_q_lens + rg.seq);
      qs = __ldg(p.cu_q_lens + rg.seq + 1) - cu0;
      ctx = __ldg(p.context_lens + rg.seq);
      mine = rg.qi0 + rg.n_q <= qs && qs <= ctx && rg.q_row0 == cu0 + rg.qi0 &&
             c_kb1 <= (ctx + p.lookahead * qs - qs + rg.qi0 + rg.n_q - 1) / kBlockSize + 1;
      if (!mine && lane == 0) report(p.dev_status, PKV_DEV_PLAN_MISMATCH);
    }
  };
  if (c_idx >= 0) c_setup();
  __syncthreads();  // barrier initialisation visible to every warp
  if (!p.after_prefill) pdl_wait();

  int issued = 0;  // stages issued into the pooled ring (the producer's count)
  auto issue = [&]() {  // the pair's first warp, whole warp: the chain's next stage
    const int kb = p_kb0 + p_j, n = min(kPair, p_n - p_j);
    if (kb + n > win_base + 32) p_window(kb);
    const int phys = __shfl_sync(0xffffffffu, win_val, (kb - win_base + lane) & 31);
    ring.fill(pool_map, p, issued % kS, lane, n, phys, p_h, PKV_DEV_BAD_BLOCK);
    p_j += n;
    ++issued;
  };
  if (lw == 0)
    for (int k = 0; k < kS && p_more(); ++k) issue();

  bool good = true;
  int done = 0;  // stages consumed (both warps walk the same chain)
  // one item: this warp's row group (of at most 8 NT rows) over the item's stages
  auto run_item = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    const int R = mine ? rg.n_q * G : 0;
    const int q_pos0 = ctx - qs + rg.qi0;
    Rows<D, NT> rows;
    load_rows<D, NT>(p, mine ? rg.q_row0 : 0, R, c_h, q_pos0, r, c, rows);
    rows.reset();
    for (int kb = c_kb0; kb < c_kb1; kb += kPair) {
      const int s = done % kS;
      const uint32_t par = (uint32_t)((done / kS) & 1);
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&full[s]), par))) {
        if (lane == 0) report(p.dev_status, PKV_DEV_TIMEOUT);
        good = false;
        return;
      }
      ++done;
      if (mine) {
        int p0[kPair];
        const float4 sc = ring.scale_of(s, min(kPair, c_kb1 - kb), kb, p0);
        attend_pair<D, NT>(ring.base + s * C::kStageBytes, sc, p0, q_pos0, ctx, lane, rows);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty[s]));
      if (lw == 0 && p_more()) {  // refill once both warps released the stage
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&empty[s]), par))) {
          if (lane == 0) report(p.dev_status, PKV_DEV_TIMEOUT);
          good = false;
          return;
        }
        issue();
      }
    }
    if (mine)
      write_rows<D, NT>(p, rg.part, cu0 + rg.qi0, c_h, rows, R, r, c);
    else if (has_rg)  // this warp's row group, which could not be attended
      poison_piece(p, rg.part, lane);
  };
  while (c_idx >= 0 && good) {
    if constexpr (MAXT == 2) {
      if (mine && rg.n_q * G > kDecode8SmallRows)
        run_item(std::integral_constant<int, 2>());
      else
        run_item(std::integral_constant<int, 1>());
    } else {
      run_item(std::integral_constant<int, 1>());
    }
    if (!good) break;
    c_idx = c_next;
    if (c_idx >= 0) c_setup();
  }
  // the issuing warp's copies still in flight land before the CTA exits
  if (lw == 0 && lane == 0)
    for (int j = done; j < issued; ++j)
      mbar_wait(smem_u32(&full[j % kS]), (uint32_t)((j / kS) & 1));
}

template <int D, int MAXT>
__global__ void __launch_bounds__(kThreads, (Decode8Cfg<D, MAXT>::kCtas))
    decode8_kernel(const __grid_constant__ CUtensorMap pool_map, const DecodeParams p) {
  using C = Decode8Cfg<D, MAXT>;
  constexpr int NSTAGE = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  // What may be read before the preceding kernel has completed, and why the pages of
  // the pool and the tables are touched first: see decode_kernel in pkv_decode.cu.
  pdl_trigger();
  if (lane == 0) prefetch_tmap(&pool_map);
  if (blockIdx.x >= p.num_indep_ctas) {  // CTA-uniform: a shared-prefix CTA
    shared_cta8<D, MAXT>(pool_map, p, smem, warp, lane);
    if (p.after_prefill) pdl_wait();
    return;
  }
  const int gw = blockIdx.x * kWarps + warp;
  const bool has_warp = gw < p.num_warps;
  {
    constexpr int64_t kPage = 2 << 20;
    const int64_t tab_bytes = (int64_t)p.num_seqs * p.max_blocks_per_seq * 4;
    const int64_t npool = (p.pool_bytes + kPage - 1) / kPage;
    const int nw_all = gridDim.x * kWarps;
    if (lane == 0 && (int64_t)gw * kPage < tab_bytes)
      prefetch_l2(reinterpret_cast<const uint8_t *>(p.block_tables) + (int64_t)gw * kPage);
    if (lane < 4) {  // a few pool pages per warp, spread over the whole pool
      const int64_t pg = (int64_t)gw + (int64_t)lane * nw_all;
      if (pg < npool) prefetch_l2(p.pool + pg * kPage);
    }
    if (gw == 0 && lane == 4) prefetch_l2(p.cu_q_lens);
    if (gw == 0 && lane == 5) prefetch_l2(p.context_lens);
    if (gw == 0 && lane == 6) prefetch_l2(p.q);
    if (gw == 0 && lane == 7) prefetch_l2(p.kv_scales);
  }
  const int pb = has_warp ? __ldg(p.warp_begin + gw) : 0;
  const int pe = has_warp ? __ldg(p.warp_begin + gw + 1) : 0;
  Piece pp;
  int fb = -1;  // lanes 0, 1: physical ids of the first piece's first stage, if known
  if (has_warp) {
    const WarpHead &wh = p.warp_head[gw];  // pp == pieces[pb], loaded beside the range
    pp = wh.first;
    const int b0 = wh.blk[0], b1 = wh.blk[1];
    fb = lane == 0 ? b0 : lane == 1 ? b1 : -1;
  }
  const int hkv = p.num_kv_heads;
  const int G = p.group;
  // The first copies use the block ids the plan carries, so no table read sits
  // between the plan read and the first copy; lanes 0 and 1 read the same entries
  // from the device table here, checked once the first stage has landed.
  const bool first_in = has_warp && pb < pe && pp.seq >= 0 && pp.seq < p.num_seqs;
  int head_chk = -1;
  if (first_in && pp.kb_begin >= 0 && lane < kPair &&
      pp.kb_begin + lane < min(pp.kb_end, p.max_blocks_per_seq))
    head_chk = __ldg(p.block_tables + (int64_t)pp.seq * p.max_blocks_per_seq + pp.kb_begin + lane);
  int f_cu0 = 0, f_cu1 = 0, f_ctx = 0;
  if (first_in) {
    f_cu0 = __ldg(p.cu_q_lens + pp.seq);
    f_cu1 = __ldg(p.cu_q_lens + pp.seq + 1);
    f_ctx = __ldg(p.context_lens + pp.seq);
  }
  Ring<D> ring;
  ring.base = smem_u32(smem + warp * C::kRingBytes);
  ring.bars = smem_u32(smem + C::kBarOffset) + warp * NSTAGE * 8;
  ring.scales = smem_u32(smem + C::kScaleOffset) + warp * NSTAGE * kPair * 8;
  ring.flags = reinterpret_cast<int *>(smem + C::kFlagOffset) + warp * NSTAGE * kPair;
  if (lane == 0 && has_warp) {
    for (int s = 0; s < NSTAGE; ++s) mbar_init(ring.bars + s * 8, kFillArrivals);
    fence_mbar_init();
  }
  if (!p.after_prefill) pdl_wait();
  if (!has_warp || pb >= pe) {
    if (p.after_prefill) pdl_wait();
    return;
  }
  __syncwarp();

  // ---- producer: walks the warp's pieces, a stage (two blocks of a piece) at a
  // time.  Whole warp, uniform; the table is read 32 entries at a time.
  const Piece first = pp;  // the producer below moves pp ahead of the consumer
  int ppi = pb, pkb = pp.kb_begin, issued = 0;
  int win_base = 0, win_val = -1;
  bool win_ok = false, pp_ok = false;
  auto check_piece = [&]() {
    pp_ok = pp.seq >= 0 && pp.seq < p.num_seqs && pp.h >= 0 && pp.h < hkv && pkb >= 0 &&
            pp.kb_end <= p.max_blocks_per_seq;
    win_ok = false;
  };
  check_piece();
  auto load_window = [&]() {  // entries pkb .. pkb + 31 of pp's table
    win_base = pkb;
    const int idx = pkb + lane;
    win_val = pp_ok && idx < pp.kb_end
                  ? __ldg(p.block_tables + (int64_t)pp.seq * p.max_blocks_per_seq + idx)
                  : -1;
    win_ok = true;
  };
  auto issue_next = [&](int stage) {
    while (pkb >= pp.kb_end) {
      if (ppi + 1 >= pe) return;
      pp = p.pieces[++ppi];
      pkb = pp.kb_begin;
      check_piece();
      // the consumer reaches this piece NSTAGE stages later: bring its q rows
      // (n_q tokens x the group's G heads, G * 2D contiguous bytes per token) into L2
      const int lpt = (G * D * 2 + 127) / 128;  // 128-byte lines per token
      const int t = lane / lpt;
      if (t < pp.n_q && pp.q_row0 >= 0 && pp.q_row0 + pp.n_q <= p.total_q && pp_ok)
        prefetch_l2(p.q + ((int64_t)(pp.q_row0 + t) * p.num_q_heads + pp.h * G) * D +
                    (lane % lpt) * 64);
    }
    const int n = min(kPair, pp.kb_end - pkb);
    int phys = fb;
    if (issued > 0 || __any_sync(0xffffffffu, lane < n && fb < 0)) {
      if (!win_ok || pkb + n > win_base + 32) load_window();
      phys = __shfl_sync(0xffffffffu, win_val, (pkb - win_base + lane) & 31);
    }
    ring.fill(pool_map, p, stage, lane, n, phys, pp.h,
              pp_ok ? PKV_DEV_BAD_BLOCK : PKV_DEV_PLAN_MISMATCH);
    pkb += n;
    ++issued;
  };
  for (int s = 0; s < NSTAGE; ++s) issue_next(s);

  int stage = 0;
  uint32_t phase = 0;
  int consumed = 0;
  bool abandoned = false;

  for (int pi = pb; pi < pe && !abandoned; ++pi) {
    // the producer runs ahead and usually already holds this piece
    const Piece pc = pi == pb ? first : (pi == ppi ? pp : p.pieces[pi]);
    // ---- piece metadata, checked against the device copies of the step arrays
    bool valid = pc.seq >= 0 && pc.seq < p.num_seqs && pc.h >= 0 && pc.h < hkv &&
                 pc.kb_begin >= 0 && pc.kb_begin <= pc.kb_end &&
                 pc.kb_end <= p.max_blocks_per_seq && pc.n_q >= 1 &&
                 pc.n_q * G <= 8 * MAXT && pc.q_row0 >= 0 &&
                 pc.q_row0 + pc.n_q <= p.total_q;
    int cu0 = 0, qs = 0, ctx = 0;
    if (valid) {
      cu0 = pi == pb ? f_cu0 : __ldg(p.cu_q_lens + pc.seq);
      qs = (pi == pb ? f_cu1 : __ldg(p.cu_q_lens + pc.seq + 1)) - cu0;
      ctx = pi == pb ? f_ctx : __ldg(p.context_lens + pc.seq);
      valid = pc.qi0 >= 0 && pc.qi0 + pc.n_q <= qs && qs <= ctx && pc.q_row0 == cu0 + pc.qi0 &&
              pc.kb_end <= (ctx + p.lookahead * qs - qs + pc.qi0 + pc.n_q - 1) / kBlockSize + 1;
    }
    if (!valid && lane == 0) report(p.dev_status, PKV_DEV_PLAN_MISMATCH);
    // the piece's row group (of at most 8 NT rows) over its stages
    auto run_piece = [&](auto nt) {
      constexpr int NT = decltype(nt)::value;
      const int R = valid ? pc.n_q * G : 0;
      const int q_pos0 = ctx - qs + pc.qi0;  // causal position of the group's first token
      Rows<D, NT> rows;
      load_rows<D, NT>(p, valid ? pc.q_row0 : 0, R, valid ? pc.h : 0, q_pos0, r, c, rows);
      rows.reset();
      bool head_bad = false;  // the plan's block ids for this piece disagree with the table
      for (int kb = pc.kb_begin; kb < pc.kb_end; kb += kPair) {
        if (!__all_sync(0xffffffffu, mbar_wait(ring.bars + stage * 8, phase))) {
          if (lane == 0) report(p.dev_status, PKV_DEV_TIMEOUT);
          abandoned = true;
          return;
        }
        if (consumed++ == 0) {  // the check entries have landed by now: compare the inline ids
          const bool bad = fb >= 0 && fb != head_chk;
          if (bad) report(p.dev_status, PKV_DEV_PLAN_MISMATCH);
          // blocks loaded from ids the table does not hold: nothing of this
          // piece is used or written
          head_bad = __any_sync(0xffffffffu, bad);
        }
        if (valid && !head_bad) {
          int p0[kPair];
          const float4 sc = ring.scale_of(stage, min(kPair, pc.kb_end - kb), kb, p0);
          attend_pair<D, NT>(ring.base + stage * C::kStageBytes, sc, p0, q_pos0, ctx, lane, rows);
        }
        __syncwarp();
        issue_next(stage);  // refill this stage with the stream's next blocks
        if (++stage == NSTAGE) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (valid && !head_bad)
        write_rows<D, NT>(p, pc.part, cu0 + pc.qi0, pc.h, rows, R, r, c);
      else
        poison_piece(p, pc.part, lane);
    };
    if constexpr (MAXT == 2) {
      if (valid && pc.n_q * G > kDecode8SmallRows)
        run_piece(std::integral_constant<int, 2>());
      else
        run_piece(std::integral_constant<int, 1>());
    } else {
      run_piece(std::integral_constant<int, 1>());
    }
  }
  if (abandoned) {
    // drain this warp's copies still in flight (bounded) before exiting
    for (int j = consumed; j < issued; ++j)
      mbar_wait(ring.bars + (j % NSTAGE) * 8, (uint32_t)((j / NSTAGE) & 1));
  }
  if (p.after_prefill) pdl_wait();
}

// 4-D view of an 8-bit pool: (D bytes, 16 rows, KV heads, K and V of every
// block); a box (D, 16, 1, 2) is the K and the V slab of one block and head.
int make_pool_map8(CUtensorMap *map, const void *pool, const pkv_pool_desc &desc) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return (int)cudaErrorNotSupported;
  const cuuint64_t d = (cuuint64_t)desc.head_dim, hkv = (cuuint64_t)desc.num_kv_heads;
  cuuint64_t dims[4] = {d, kBlockSize, hkv,
                        (cuuint64_t)(desc.num_blocks > 0 ? desc.num_blocks : 1) * 2};
  cuuint64_t strides[3] = {d, d * kBlockSize, d * kBlockSize * hkv};
  cuuint32_t box[4] = {(cuuint32_t)d, kBlockSize, 1, 2};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(pool), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? 0 : (int)cudaErrorInvalidValue;
}

template <int D, int MAXT>
int launch_t(const AttnArgs &a, const CUtensorMap &map) {
  using C = Decode8Cfg<D, MAXT>;
  static_assert((C::kSmemBytes + 1024) * C::kCtas <= 228 * 1024, "the CTAs share an SM");
  cudaError_t e = prepare_kernel<decode8_kernel<D, MAXT>>(C::kSmemBytes);
  if (e != cudaSuccess) return (int)e;
  const unsigned grid = (unsigned)((a.num_decode_warps + kWarps - 1) / kWarps + a.num_shared_ctas);
  profile_begin(PKV_KERNEL_DECODE, a.stream);
  e = launch_kernel(decode8_kernel<D, MAXT>, dim3(grid), dim3(kThreads), C::kSmemBytes, a.stream,
                    !profiling_active(), map, make_params(a));
  profile_end(PKV_KERNEL_DECODE, a.stream);
  return e != cudaSuccess ? (int)e : (int)cudaGetLastError();
}

}  // namespace

int launch_decode8(const AttnArgs &a) {
  CUtensorMap map;
  const int e = make_pool_map8(&map, a.kv_pool, a.desc);
  if (e) return e;
  // no row group of more than 8 rows: the kernel with one column tile and 16 warps an
  // SM (256 decodes of 4 heads: 193 us with 8 warps of either, 180 us with 16)
  if (a.max_rows <= kDecode8SmallRows)
    return a.desc.head_dim == 128 ? launch_t<128, 1>(a, map) : launch_t<64, 1>(a, map);
  return a.desc.head_dim == 128 ? launch_t<128, 2>(a, map) : launch_t<64, 2>(a, map);
}

}  // namespace pkv
