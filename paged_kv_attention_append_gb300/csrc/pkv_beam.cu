// Beam search's selection: log-softmax of each beam's logits, added to its score, and
// the best continuations over all beams of a request.
//
//   score(k, t) = cum_k + x_kt - log sum_u exp(x_ku);  the num_select largest of (k, t),
//   ties to the lower beam, then the lower token.
//
// Within a beam the score grows with the logit, so the best of a beam are its largest
// logits and need no logarithm.  The logits are read once: a CTA goes over a range of
// one row in tiles and takes from them, at the same time,
//  - the running sum of exponentials: a thread keeps s = sum 2^(x L - r), with L fp32's
//    log2 e and r its maximum of x L so far (one fma and one ex2 an element; s is rescaled
//    when r moves).  The row's lse is (r + log2 s) / L: as the same L divides it, its
//    rounding (2^-26 of L) moves the lse by 2^-26 times the softmax's entropy only.  r starts at
//    -kFar: far masked values (-1e30, whatever r would be rounded to there) weigh 0 from the first
//    on.  Where a range's largest x L is not within kFar, fp32's step is 64 or more, so that only
//    the logits equal to the largest one count, and they are counted;
//  - the candidates: 64-bit keys (logit, lowest token first), so that no two are equal.
//    A threshold T below the num_select-th largest key comes from the threads' maxima of
//    the first tile; keys above T go to their warp's buffer in shared memory, straight
//    from the registers and without atomics or barriers.  After the tiles 0, 1, 3, 7, ..
//    the CTA keeps its num_select largest keys and raises T to the last of them, so
//    about num_select keys pass between two such cuts.  (With the first tile's T kept,
//    that many passed in every tile: 512 rows of 128000 fp32 took 60 us; with keys put into
//    one buffer by atomics after each tile, 46.)
// A second kernel, one CTA a request, joins the rows' sums and merges the sorted lists
// by score in 64 bits, within a beam by key.
//
// Which elements a thread sums depends on their place in the row alone, not on the row's
// address: equal rows get equal sums, and their ties go by the beam.
//
// Bound by HBM for large calls, by latency (two launches) for small ones.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>

#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kBeamWarps = kThreads / 32;
constexpr int kMaxSelect = 128;
constexpr int kWarpKeys = 128;      // new candidate keys a warp keeps (>= kMaxSelect)
constexpr int kAllKeys = kBeamWarps * kWarpKeys + kMaxSelect + 64;
constexpr int kMaxLists = 1024;     // sorted lists (beam, split) of a request
constexpr int32_t kMaxVocab = INT32_MAX - 65536;  // tiles count past its end in 32 bits
constexpr int kMergeScores = 2048;  // scores a merge keeps in shared memory (>= kMaxLists)
constexpr float kLog2e = 1.4426950408889634f;  // L above
constexpr float kFar = 1073741824.f;  // 2^30: r is off by 32 below it, so s by 2^32

struct BeamParams {
  const void *logits;
  const float *cum;
  const uint8_t *finished;
  float *scores;
  int32_t *tokens, *parents;
  float2 *part;          // [rows][splits]: r, sum of 2^(x L - r); beyond kFar +-inf, a count
  uint64_t *keys;        // [rows][splits][num_select], descending, 0: none
  int64_t row_stride, num_rows;
  int32_t num_beams, vocab, num_select, pad_token, splits, tiles;
};

// Larger key: larger logit, then lower token.  (-0 counts as 0.)
__device__ __forceinline__ uint64_t make_key(float x, int32_t token) {
  const uint32_t b = __float_as_uint(x + 0.f);
  const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (uint64_t)o << 32 | (uint32_t)~token;
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// How a type's elements lie in 32-bit words, and its -inf.
template <typename T>
struct Words;
template <>
struct Words<float> {
  static constexpr int kPer = 1;
  static constexpr uint32_t kNegInf = 0xff800000u;
  static __device__ __forceinline__ float get(uint32_t w, int) { return __uint_as_float(w); }
};
template <>
struct Words<__nv_bfloat16> {
  static constexpr int kPer = 2;
  static constexpr uint32_t kNegInf = 0xff80u;
  static __device__ __forceinline__ float get(uint32_t w, int i) {
    return __uint_as_float(i ? w & 0xffff0000u : w << 16);
  }
};
template <>
struct Words<__half> {
  static constexpr int kPer = 2;
  static constexpr uint32_t kNegInf = 0xfc00u;
  static __device__ __forceinline__ float get(uint32_t w, int i) {
    return __half2float(__ushort_as_half((uint16_t)(i ? w >> 16 : w)));
  }
};
template <typename T>
__device__ __forceinline__ uint32_t raw_bits(const T *p) {
  if (sizeof(T) == 4) return __ldg(reinterpret_cast<const uint32_t *>(p));
  return __ldg(reinterpret_cast<const uint16_t *>(p));
}

// A row of logits, and the part of the tensor's memory that 16-byte loads may touch.
template <typename T>
struct Row {
  const T *data;
  const char *lo, *hi;  // the tensor's first byte and the one past its last
  int32_t vocab;
  uint32_t shift;       // data's offset from 16-byte alignment, in bytes
};

// Elements [at, at + kVec) of a row, as they lie in memory; those past its end as -inf.
// Rows of 16 bits that start off alignment (an odd vocabulary) are put together from the
// aligned 16-byte pieces around them; an element at a time only at the tensor's ends.
template <typename T, int kVec>
__device__ __forceinline__ void load_vec(const Row<T> &row, int32_t at, uint32_t *w) {
  using W = Words<T>;
  constexpr int kWords = kVec / W::kPer;
  const T *src = row.data + at;
  const bool whole = at + kVec <= row.vocab;
  if (kVec == 1) {  // (4-byte types)
    w[0] = whole ? raw_bits(src) : W::kNegInf;
    return;
  }
  if (row.shift == 0 && whole) {
    if (kWords == 2) {
      const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(src));
      w[0] = v.x;
      w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(src) + i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
    }
    return;
  }
  if (kWords >= 4 && sizeof(T) == 2) {
    const char *first = reinterpret_cast<const char *>(src) - row.shift;
    if (whole && first >= row.lo && first + kWords * 4 + 16 <= row.hi) {
      uint32_t v[kWords + 4];
#pragma unroll
      for (int i = 0; i < kWords / 4 + 1; ++i) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(first) + i);
        v[4 * i] = x.x;
        v[4 * i + 1] = x.y;
        v[4 * i + 2] = x.z;
        v[4 * i + 3] = x.w;
      }
      // by 8, by 4, then by 2 bytes
#pragma unroll
      for (int i = 0; i < kWords + 2; ++i) v[i] = row.shift & 8 ? v[i + 2] : v[i];
#pragma unroll
      for (int i = 0; i < kWords + 1; ++i) v[i] = row.shift & 4 ? v[i + 1] : v[i];
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        w[i] = __funnelshift_r(v[i], v[i + 1], (row.shift & 2) * 8);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    w[i] = 0;
#pragma unroll
    for (int j = 0; j < W::kPer; ++j) {
      const int e = i * W::kPer + j;
      w[i] |= (at + e < row.vocab ? raw_bits(src + e) : W::kNegInf) << (16 * j);
    }
  }
}

// How many of s[begin, end) are above k.  Eight at a time, all loads ahead of the compares
// (one by one, 150 keys took 7 us); begin and end multiples of 8, s 16-byte aligned.
__device__ __forceinline__ int count_above(const uint64_t *s, int begin, int end, uint64_t k) {
  int n = 0;
  for (int j = begin; j < end; j += 8) {
    ulonglong2 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = reinterpret_cast<const ulonglong2 *>(s + j)[u];
#pragma unroll
    for (int u = 0; u < 4; ++u) n += (v[u].x > k) + (v[u].y > k);
  }
  return n;
}

// The `cnt` keys of s_all in descending order, the first `keep` of them to s_top: each
// key's place is the number of larger ones.  Up to kT keys, the threads that are left over
// share the counting (s_rank: kT ints).  The 64 keys from cnt on are 0.  By all kT threads.
template <int kT>
__device__ __forceinline__ void sort_keys(const uint64_t *s_all, int cnt, uint64_t *s_top, int keep,
                                          int32_t *s_rank) {
  const int tid = threadIdx.x;
  if (cnt <= kT) {
    const int lanes = cnt <= 32 ? 32 : 1 << (32 - __clz(cnt - 1));
    const int parts = kT / lanes, i = tid & (lanes - 1), part = tid / lanes;
    const int len = ((cnt + parts - 1) / parts + 7) & ~7, all = (cnt + 7) & ~7;
    const uint64_t k = i < cnt ? s_all[i] : 0;
    s_rank[tid] = 0;
    __syncthreads();
    if ((i & ~31) < cnt) {
      const int rank = count_above(s_all, part * len, min(part * len + len, all), k);
      if (rank) atomicAdd(s_rank + i, rank);
    }
    __syncthreads();
    if (tid < cnt && s_rank[tid] < keep) s_top[s_rank[tid]] = k;
  } else {
    for (int i = tid; i < cnt; i += kT) {
      const uint64_t k = s_all[i];
      const int rank = count_above(s_all, 0, (cnt + 7) & ~7, k);
      if (rank < keep) s_top[rank] = k;
    }
  }
  __syncthreads();
}

// A value that at least M of the CTA's threads reach: the smallest over the first `warps` of its
// kWarps warps of their ceil(M / warps)-th largest (0: there are too few).  s: an int a warp.
template <int kWarps>
__device__ __forceinline__ uint32_t threads_threshold(uint32_t o, int M, int warps, uint32_t *s) {
  uint32_t kth = 0;
  for (int i = 0; i < M; i += warps) {
    kth = __reduce_max_sync(0xffffffffu, o);
    const uint32_t who = __ballot_sync(0xffffffffu, o == kth);
    if ((threadIdx.x & 31) == __ffs(who) - 1) o = 0;
  }
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = (int)threadIdx.x >> 5 < warps ? kth : ~0u;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) kth = min(kth, s[w]);
  return kth;
}

// A tile is 2 kHalf elements a thread, in two sets of registers: each is filled again as
// soon as it has been used, so loads are always in flight.
// kVec: consecutive elements a thread loads together.
template <typename T, int kHalf, int kVec>
__global__ void __launch_bounds__(kThreads, 4) beam_rows_kernel(const BeamParams p) {
  using W = Words<T>;
  constexpr int kWords = kHalf / W::kPer;
  constexpr int kHalfTile = kThreads * kHalf, kTile = 2 * kHalfTile;
  __shared__ uint64_t s_new[kBeamWarps][kWarpKeys];
  __shared__ alignas(16) uint64_t s_all[kAllKeys];
  __shared__ uint64_t s_top[kMaxSelect];
  __shared__ float s_m[kBeamWarps], s_s[kBeamWarps];
  __shared__ uint32_t s_kth[kBeamWarps];
  __shared__ int32_t s_rank[kThreads], s_cnt[kBeamWarps];
  pdl_wait();
  pdl_trigger();  // only now: the merge reads the call's inputs before its own wait
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row_id = blockIdx.x / p.splits;
  const int split = blockIdx.x % p.splits;
  if (p.finished && __ldg(p.finished + row_id)) return;  // the merge does not look at its parts
  Row<T> row;
  row.data = static_cast<const T *>(p.logits) + row_id * p.row_stride;
  row.lo = static_cast<const char *>(p.logits);
  row.hi = row.lo + ((p.num_rows - 1) * p.row_stride + p.vocab) * (int64_t)sizeof(T);
  row.vocab = p.vocab;
  row.shift = (uint32_t)(reinterpret_cast<uintptr_t>(row.data) & 15u);
  const int tile0 = (int)((int64_t)p.tiles * split / p.splits);
  const int tile1 = (int)((int64_t)p.tiles * (split + 1) / p.splits);
  const int M = p.num_select;
  float r = -kFar, s = 0.f;
  // candidates are the keys above T_key, their logits at least T_val (a cheaper test, false
  // for NaN too); logits of -inf never are
  uint64_t T_key = make_key(-INFINITY, 0);
  float T_val = -FLT_MAX;
  int num_top = 0;          // keys in s_top, the CTA's largest so far, sorted
  int cnt = 0;              // keys this warp found since
  // element i < 2 kHalf of this thread's in a tile
  auto token = [&](int tile, int i) {
    return tile * kTile + i / kVec * kThreads * kVec + tid * kVec + i % kVec;
  };
  auto key_at = [&](int at) -> uint64_t {
    if (at >= p.vocab) return 0;
    const float x = W::get(raw_bits(row.data + at), 0);
    return x >= -FLT_MAX ? make_key(x, at) : 0;
  };
  uint32_t w[2][kWords];
  auto load = [&](int tile, int half) {
#pragma unroll
    for (int j = 0; j < kHalf / kVec; ++j)
      load_vec<T, kVec>(row, token(tile, half * kHalf + j * kVec), w[half] + j * (kVec / W::kPer));
  };
  auto elements = [&](int half, float (&x)[kHalf]) {  // returns the largest
#pragma unroll
    for (int i = 0; i < kHalf; ++i) x[i] = W::get(w[half][i / W::kPer], i % W::kPer);
    float top = x[0];
#pragma unroll
    for (int i = 1; i < kHalf; i += 2)
      top = i + 1 < kHalf ? max3(top, x[i], x[i + 1]) : fmaxf(top, x[i]);
    return top;
  };
  auto push = [&](uint64_t k) {  // by the whole warp
    const bool pass = k > T_key;
    const uint32_t b = __ballot_sync(0xffffffffu, pass);
    const int place = cnt + __popc(b & ((1u << lane) - 1));
    if (pass && place < kWarpKeys) s_new[warp][place] = k;
    cnt += __popc(b);
  };
  // half a tile into the sum and the candidates
  auto use = [&](int tile, int half) {
    float x[kHalf];
    const float top = elements(half, x);
    const float r_new = fmaxf(r, top * kLog2e);
    s *= fast_exp2(r - r_new);
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < kHalf; i += 2) {
      a += fast_exp2(fmaf(x[i], kLog2e, -r_new));  // (a NaN makes the row's sum NaN)
      b += fast_exp2(fmaf(x[i + 1], kLog2e, -r_new));
    }
    s += a + b;
    r = r_new;
    if (__any_sync(0xffffffffu, top >= T_val)) {
#pragma unroll
      for (int i = 0; i < kHalf; ++i)
        if (__any_sync(0xffffffffu, x[i] >= T_val))
          push(x[i] >= T_val ? make_key(x[i], token(tile, half * kHalf + i)) : 0);
    }
  };
  // the CTA's largest keys of all found so far to s_top; by all threads
  auto cut = [&] {
    if (lane == 0) s_cnt[warp] = min(cnt, kWarpKeys);
    for (int i = tid; i < num_top; i += kThreads) s_all[i] = s_top[i];
    __syncthreads();
    int before = num_top, all = num_top;
#pragma unroll
    for (int v = 0; v < kBeamWarps; ++v) {
      if (v < warp) before += s_cnt[v];
      all += s_cnt[v];
    }
    for (int i = lane; i < s_cnt[warp]; i += 32) s_all[before + i] = s_new[warp][i];
    if (tid < 64) s_all[all + tid] = 0;
    __syncthreads();
    sort_keys<kThreads>(s_all, all, s_top, M, s_rank);
    num_top = min(all, M);
    cnt = 0;
    if (num_top == M && s_top[M - 1] > T_key) {
      // (the elements still to come are of higher tokens: equal logits do not pass any more)
      T_key = s_top[M - 1];
      T_val = key_value(T_key + (1ull << 32));
    }
  };
  load(tile0, 0);
  load(tile0, 1);
  {
    float x[kHalf];
    float top = elements(0, x);
    top = fmaxf(top, elements(1, x));
    // (warps whose threads all have elements: rows of 300 to 600, or as short a last range, took
    // 15 to 160 us with the others counted in, as then every element was a candidate)
    const int left = p.vocab - tile0 * kTile;
    const int full = max(min(left / (32 * kVec), kBeamWarps), 1);
    const uint32_t o = threads_threshold<kBeamWarps>((uint32_t)(make_key(top, 0) >> 32), M, full, s_kth);
    top = key_value((uint64_t)o << 32);  // (0 is a NaN)
    if (top >= T_val) {
      T_val = top;
      T_key = make_key(top, 0x7fffffff) - 1;  // below every key of that logit
    }
  }
  for (int tile = tile0; tile < tile1; ++tile) {
    int had = cnt;
    use(tile, 0);
    if (tile + 1 < tile1) load(tile + 1, 0);
    use(tile, 1);
    if (tile + 1 < tile1) load(tile + 1, 1);
    const int n = tile - tile0 + 1;
    // (the last few tiles bring fewer keys than a cut costs)
    const bool due = (n & (n - 1)) == 0 && tile + 3 < tile1;
    const bool full = __syncthreads_or(cnt > kWarpKeys);
    // Too many for a warp's buffer (ties, rows that rise from tile to tile): the tile once more,
    // an element a thread at a time, with a cut as soon as a warp has a few
    if (full) {
      cnt = had;
#pragma unroll 1
      for (int i = -1; i < 2 * kHalf; ++i) {
        if (i >= 0) push(key_at(token(tile, i)));
        if (__syncthreads_or(cnt > kWarpKeys / 8)) cut();
      }
    }
    if (due) cut();
  }
  cut();
  uint64_t *out = p.keys + ((int64_t)row_id * p.splits + split) * M;
  for (int i = tid; i < M; i += kThreads) out[i] = i < num_top ? s_top[i] : 0;
  // the threads' sums, at the CTA's r
  float top = r;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) s_m[warp] = top;
  __syncthreads();
  top = s_m[0];
#pragma unroll
  for (int i = 1; i < kBeamWarps; ++i) top = fmaxf(top, s_m[i]);
  s *= r == top ? 1.f : fast_exp2(r - top);
  if (fabsf(top) >= kFar) {
    if (num_top > 0) {  // how often its largest logit is there; NaN and +inf are still no numbers
      const float x0 = key_value(s_top[0]);
      const int end = min(tile1 * kTile, p.vocab);
      s = 0.f;
      for (int at = tile0 * kTile + tid; at < end; at += kThreads) {
        const float x = W::get(raw_bits(row.data + at), 0);
        s += !(x <= FLT_MAX) ? NAN : x == x0 ? 1.f : 0.f;
      }
    }  // (else all of it is -inf, or NaN: s is 0 or NaN)
    top = copysignf(INFINITY, top);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) s_s[warp] = s;
  __syncthreads();
  if (tid == 0) {
    float sum = s_s[0];
#pragma unroll
    for (int i = 1; i < kBeamWarps; ++i) sum += s_s[i];
    p.part[(int64_t)row_id * p.splits + split] = make_float2(top, sum);
  }
}

// A double as an integer of the same order, 0 for what is not finite in fp32.
__device__ __forceinline__ uint64_t order_double(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
  if ((b & ~(1ull << 63)) >= 0x47effffff0000000ull) return 0;  // 2^128 - 2^103 on, inf, NaN
  return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double unorder_double(uint64_t o) {
  return __longlong_as_double((long long)(o >> 63 ? o ^ 1ull << 63 : ~o));
}

// What the two functions below work on, which a merge needs where scores are coarse.
struct ByKey {
  const uint64_t *keys;     // [lists][num_select]
  const double *base;       // of each beam, as is what follows
  const float *shift;
  const bool *done;
  uint64_t *head, *low;     // [lists]: score and key of each list's first one left
  int32_t *next;            // [lists]: its place in the list
  uint64_t *won;            // [num_select]: of each round the score (0: none left),
  int32_t *list, *at;       // its list and place in it
  int lists, splits, num_select;
};
__device__ __forceinline__ uint64_t candidate_score(double base, float shift, uint64_t key) {
  return key ? order_double(base + (double)(key_value(key) - shift)) : 0;
}
// Whether that difference is rounded (then merge_by_key takes it in 64 bits).
__device__ __forceinline__ bool difference_is_rounded(float shift, uint64_t key) {
  const float x = key_value(key);
  return shift != 0.f && (x - shift) + shift != x;
}
// Whether another logit than this key's may have the same score, told apart as `reach` says.
__device__ __forceinline__ bool score_is_coarse(double base, float shift, uint64_t key, int reach) {
  const int e_base = (__double2hiint(base) >> 20 & 0x7ff) - 1023;
  const int e = (int)(__float_as_uint(key_value(key)) >> 23 & 0xff) - 127;
  return e_base - e > reach || shift != 0.f;
}

// Whether two of the `cnt` scores are one beam's, equal and of different logits, or one is of a
// rounded difference, as seen by this warp; by all threads.  Bits of `low` do not count; they
// hold a score's ~place in the lists, or (low 0) score i is that of list i / depth, place i % depth.
__device__ __noinline__ bool scores_hide_keys(const ByKey &m, const uint64_t *score, uint64_t low,
                                              int cnt, int depth, int reach) {
  const int lane = threadIdx.x & 31, M = m.num_select;
  auto place_of = [&](int i) { return low ? (int)(~score[i] & low) : i / depth * M + i % depth; };
  bool hidden = false;
  for (int i0 = threadIdx.x - lane; i0 < cnt; i0 += blockDim.x) {
    const int i = i0 + lane;
    uint64_t mine = 0;
    uint32_t logit = 0;
    int beam = 0;
    bool coarse = false;
    if (i < cnt && score[i] != 0) {
      const int at = place_of(i);
      const uint64_t key = m.keys[at];
      beam = at / M / m.splits;
      mine = score[i] | low;
      logit = (uint32_t)(key >> 32);
      coarse = !m.done[beam] && score_is_coarse(m.base[beam], m.shift[beam], key, reach);
      hidden |= coarse && difference_is_rounded(m.shift[beam], key);
    }
    // the warp goes over all scores for each of its coarse ones
    for (uint32_t left = __ballot_sync(0xffffffffu, coarse); left; left &= left - 1) {
      const int from = __ffs(left) - 1;
      const uint64_t o = __shfl_sync(0xffffffffu, mine, from);
      const uint32_t x = __shfl_sync(0xffffffffu, logit, from);
      const int k = __shfl_sync(0xffffffffu, beam, from);
      for (int j = lane; j < cnt; j += 32) {
        if (score[j] == 0 || (score[j] | low) != o) continue;
        const int at = place_of(j);
        if (at / M / m.splits == k && (uint32_t)(m.keys[at] >> 32) != x) hidden = true;
      }
      if (__any_sync(0xffffffffu, hidden)) return true;
    }
  }
  return hidden;
}

// A merge that compares candidates by score (all 64 bits), then beam, then key: by one warp, in
// num_select rounds over the lists' heads, with their keys beside their scores.
__device__ __noinline__ void merge_by_key(const ByKey &m) {
  const int lane = threadIdx.x & 31;
  auto enter = [&](int l, int n) {  // the n-th of list l as its head
    const int k = l / m.splits;
    const uint64_t key = n < m.num_select ? m.keys[(int64_t)l * m.num_select + n] : 0;
    m.next[l] = n;
    m.low[l] = key;
    if (!m.done[k])
      m.head[l] =
          key ? order_double(m.base[k] + ((double)key_value(key) - (double)m.shift[k])) : 0;
    else m.head[l] = n == 0 && l == k * m.splits ? order_double(m.base[k]) : 0;
  };
  for (int l = lane; l < m.lists; l += 32) enter(l, 0);
  uint64_t best, best_key;  // of this lane's lists
  int best_list, best_beam;
  auto look = [&] {
    best = best_key = 0;
    best_list = best_beam = 0;
    for (int l = lane; l < m.lists; l += 32) {
      const uint64_t o = m.head[l];
      if (o == 0 || o < best) continue;
      const int k = l / m.splits;
      if (o > best || (k == best_beam && m.low[l] > best_key)) {
        best = o;
        best_key = m.low[l];
        best_list = l;
        best_beam = k;
      }
    }
  };
  look();
  for (int i = 0; i < m.num_select; ++i) {
    bool mine = best != 0;  // of the lanes' best, by what is compared first
    auto keep_max = [&](uint32_t x) {  // (by all lanes)
      const uint32_t top = __reduce_max_sync(0xffffffffu, mine ? x : 0u);
      mine = mine && x == top;
    };
    keep_max((uint32_t)(best >> 32));
    keep_max((uint32_t)best);
    keep_max(~(uint32_t)best_beam);
    keep_max((uint32_t)(best_key >> 32));
    keep_max((uint32_t)best_key);
    if (!__any_sync(0xffffffffu, mine)) {
      if (lane == 0) m.won[i] = 0;
    } else if (mine) {  // one lane: a beam's keys are all different
      const int l = best_list, n = m.next[l];
      m.won[i] = best;
      m.list[i] = l;
      m.at[i] = n;
      enter(l, n + 1);
      look();
    }
    __syncwarp();
  }
}

// One CTA a request.  List k splits + j holds beam k's best of its j-th range: equal scores go
// to the lower list.  Where they are few (by_counting below) two sorts by counting do: of the
// lists' heads, so that the num_select best lists stay, and of the one of rank r num_select - r
// keys only; then of those (15 lists by 10: the call 19.7 us, merged by rounds or one sort of
// all 22.5; 11 lists by 31: this kernel 8.8, by rounds 14.7).  Of more than kFewLists heads a
// threshold leaves a few to sort (600 lists by 3: the call 13.7 us, by rounds 18).  Beyond
// kMostKeys (32 kept of 32 lists; the call with 63 lists, by counting / by rounds: 32 kept 17.8 /
// 19.1 us, 36 20.8 / 20.3, 44 31.3 / 22.9; by rounds 64 28.5, 128 49) and beyond kPlaces one warp
// merges them in num_select rounds over the heads, with as many scores as fit in shared memory (a
// list's further ones are read when it gets there).
//
// Scores are fp64; to be sorted they take their key's place in the lists into their last 13 bits:
// equal to 2^-39 they count as equal.  Within a beam that is the order of the keys as long as
// different logits have different scores: those of exponent e are 2^(e - 24) apart at least, scores
// of exponent E are told apart by 2^(E - 39), by 2^(E - 52) in the rounds.  Where a candidate
// fails that test (a beam at -1e9, a logit of 1e-5) and a beam has several lists, equal scores are
// looked for, and where they hide different logits all is done again by merge_by_key (4 beams
// of 32000 of which three are at -1e9: the call 20.7 us, else 7.5; 128 kept of a row at -1e12:
// 119, else 50; 8 beams of 128000 log-probabilities, whose best are next to 0: 17, without the
// look 47.  Keys compared everywhere instead: 8.8 us for any 4 beams, 79 for 128 of 63 lists).
constexpr int kMergeThreads = 512, kMergeWarps = kMergeThreads / 32;
constexpr int kFewLists = 64, kPlaces = 8192, kMostKeys = 512;
constexpr int kSortReach = 39 - 24 - 2, kRoundReach = 52 - 24 - 2;  // (E is the base's here)
// (two CTAs an SM, so 64 registers: left to itself the compiler takes 40 and spills about the call)
__global__ void __launch_bounds__(kMergeThreads, 2) beam_merge_kernel(const BeamParams p) {
  __shared__ double s_base[kMaxLists];       // cum - (lse - shift) of the request's beams,
  __shared__ float s_shift[kMaxLists];       // shift 0 unless a row's largest logit is beyond kFar
  __shared__ bool s_done[kMaxLists];
  // keys as they are (counting, if they fit), or [list][depth] ordered scores (rounds)
  __shared__ uint64_t s_score[kMergeScores];
  __shared__ alignas(16) uint64_t s_head[kMaxLists + 64];  // of each list the first score left
  __shared__ int32_t s_next[kMaxLists];
  __shared__ uint64_t s_won[kMaxSelect];     // of each round the score (0: none left),
  __shared__ int32_t s_list[kMaxSelect], s_at[kMaxSelect];  // its list and place in it
  __shared__ uint32_t s_kth[kMergeWarps];
  __shared__ int32_t s_count;
  const int tid = threadIdx.x;
  const int64_t row0 = (int64_t)blockIdx.x * p.num_beams;
  const int lists = p.num_beams * p.splits, M = p.num_select;
  const uint64_t *keys = p.keys + row0 * p.splits * M;
  // a beam's parts are joined by a group of up to 32 lanes (50 parts by one thread: 8 us)
  int group = 32;
  while (group > 1 && group / 2 >= p.splits) group /= 2;
  const int lead = tid / group, lane = tid % group;
  // (inputs of the call: the kernel before this one does not write them)
  float cum = 0.f;
  bool ended = false;
  auto inputs = [&](int k) {
    cum = __ldg(p.cum + row0 + k);
    ended = p.finished && __ldg(p.finished + row0 + k);
  };
  if (lead < p.num_beams) inputs(lead);
  // lists that can have keys among the best, and how many those can be together
  const int R = min(lists, M), most = R * M - R * (R - 1) / 2;
  const bool by_counting = most <= kMostKeys && lists * M <= kPlaces;
  const bool copied = by_counting && lists * M <= kMergeScores;
  if (tid == 0) s_count = 0;
  pdl_wait();
  // the first keys on their way beside the sums
  const uint64_t first = copied && tid < lists * M ? keys[tid] : 0;
  for (int k0 = 0; k0 < p.num_beams; k0 += kMergeThreads / group) {
    const int k = k0 + lead;
    if (k0 > 0 && k < p.num_beams) inputs(k);
    const int parts = k < p.num_beams && !ended ? p.splits : 0;
    const float2 *part = p.part + (row0 + k) * p.splits;
    const uint64_t *heads = keys + (int64_t)k * p.splits * M;  // every M-th
    float m = -INFINITY, s = 0.f, shift = 0.f;
#pragma unroll 4
    for (int j = lane; j < parts; j += group) m = fmaxf(m, part[j].x);
    for (int o = group / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll 4
    for (int j = lane; j < parts; j += group)
      s += part[j].y * (part[j].x == m ? 1.f : exp2f(part[j].x - m));
    for (int o = group / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const bool far = fabsf(m) == INFINITY && s > 0.f;
    if (__any_sync(0xffffffffu, far)) {
      // the parts are counts of their largest logits: those of the row's largest
      uint32_t best = 0;
      for (int j = lane; j < parts; j += group) best = max(best, (uint32_t)(heads[(int64_t)j * M] >> 32));
      for (int o = group / 2; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
      float n = 0.f;
      for (int j = lane; j < parts; j += group)
        if ((uint32_t)(heads[(int64_t)j * M] >> 32) == best) n += part[j].y;
      for (int o = group / 2; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      if (far) {
        s = n;
        shift = key_value((uint64_t)best << 32);
        m = 0.f;
      }
    }
    if (lane != 0 || k >= p.num_beams) continue;
    double base = cum;
    if (!ended) {
      // log2 s by its exponent and mantissa: off by half a step of a number below 1
      int e;
      const float f = frexpf(s, &e);
      base -= ((double)m + (e - 1) + (double)log2f(2.f * f)) * (1.0 / (double)kLog2e);
    }
    s_base[k] = base;
    s_shift[k] = shift;
    s_done[k] = ended;
  }
  if (copied) {
    s_score[tid] = first;
#pragma unroll 4
    for (int i = tid + kMergeThreads; i < lists * M; i += kMergeThreads) s_score[i] = keys[i];
  }
  __syncthreads();
  // the ordered score of a key of list l, its first or not (0: there is none)
  // (the order within a list is the keys' anyway, so with one list a beam only shifts matter)
  const int sort_reach = p.splits > 1 ? kSortReach : INT32_MAX;
  const int round_reach = p.splits > 1 ? kRoundReach : INT32_MAX;
  bool coarse = false;  // whether one of this thread's scores may be another logit's, too
  auto score_of = [&](int l, bool lead, uint64_t key, int reach) -> uint64_t {
    const int k = l / p.splits;
    const double base = s_base[k];
    if (s_done[k]) return lead && l == k * p.splits ? order_double(base) : 0;
    const float shift = s_shift[k];
    const uint64_t o = candidate_score(base, shift, key);
    if (o != 0 && score_is_coarse(base, shift, key, reach)) coarse = true;
    return o;
  };
  auto put = [&](int i, uint64_t score, int l, uint64_t key) {
    const int64_t o = (int64_t)blockIdx.x * M + i;
    const int k = l / p.splits;
    p.scores[o] = score ? (float)unorder_double(score) : -INFINITY;
    p.parents[o] = score ? (int32_t)(row0 + k) : -1;
    p.tokens[o] = score == 0 ? -1 : s_done[k] ? p.pad_token : (int32_t)~(uint32_t)key;
  };
  auto put_won = [&] {  // by one warp
    for (int i = tid; i < M; i += 32) {
      const uint64_t won = s_won[i];
      const int l = won ? s_list[i] : 0;
      put(i, won, l, won ? keys[(int64_t)l * M + s_at[i]] : 0);
    }
  };
  auto by_key = [&] {
    return ByKey{keys,  s_base, s_shift, s_done, s_head,   s_score, s_next,
                 s_won, s_list, s_at,    lists,  p.splits, M};
  };
  auto put_by_key = [&] {
    merge_by_key(by_key());
    put_won();
  };
  if (by_counting) {
    constexpr uint64_t kPlace = kPlaces - 1;
    auto place_of = [](uint64_t o) { return (int)(~o & kPlace); };
    auto key_at = [&](int at) { return copied ? s_score[at] : keys[at]; };
    // key `at` of all, the d-th of list l: lower lists, and earlier keys, go first
    auto sort_score = [&](int at, int l, int d) -> uint64_t {
      const uint64_t o = score_of(l, d == 0, key_at(at), sort_reach);
      return o ? (o & ~kPlace) | (kPlace - at) : 0;
    };
    uint64_t *s_some = s_head, *s_best = s_won;  // to be sorted, and the best of them
    if (tid < M) s_best[tid] = 0;
    int some = lists;
    if (lists <= kFewLists) {
      if (tid < lists) s_some[tid] = sort_score(tid * M, tid, 0);
    } else {
      static_assert(kMaxLists <= 2 * kMergeThreads, "two heads a thread");
      // every 16th list a warp's, so that each has some of every beam
      const int one = tid % 32 * kMergeWarps + tid / 32, other = one + kMergeThreads;
      const uint64_t a = one < lists ? sort_score(one * M, one, 0) : 0;
      const uint64_t b = other < lists ? sort_score(other * M, other, 0) : 0;
      const uint32_t T =
          threads_threshold<kMergeWarps>((uint32_t)(max(a, b) >> 32), M, kMergeWarps, s_kth);
      if (a && (uint32_t)(a >> 32) >= T) s_some[atomicAdd(&s_count, 1)] = a;
      if (b && (uint32_t)(b >> 32) >= T) s_some[atomicAdd(&s_count, 1)] = b;
      __syncthreads();
      some = s_count;
    }
    if (tid < 64) s_some[some + tid] = 0;
    bool look_closer = __syncthreads_or(coarse), hidden = false;
    if (look_closer) hidden = scores_hide_keys(by_key(), s_some, kPlace, some, 0, sort_reach);
    sort_keys<kMergeThreads>(s_some, some, s_best, M, s_next);
    // key d of the list of rank r, to place r M - r (r - 1) / 2 + d
    for (int i = tid; i < R * M; i += kMergeThreads) {
      const int r = i / M, d = i % M, at = place_of(s_best[r]) + d;
      if (r + d >= M) continue;
      s_some[i - r * (r - 1) / 2] = s_best[r] ? sort_score(at, at / M, d) : 0;
    }
    if (tid < 64) s_some[most + tid] = 0;
    look_closer = __syncthreads_or(coarse);
    if (look_closer)  // (by all threads, whatever they have seen)
      hidden |= scores_hide_keys(by_key(), s_some, kPlace, most, 0, sort_reach);
    if (tid < M) s_best[tid] = 0;
    __syncthreads();
    sort_keys<kMergeThreads>(s_some, most, s_best, M, s_next);
    if (!look_closer || !__syncthreads_or(hidden)) {
      if (tid < M) {
        const uint64_t best = s_best[tid];
        const int at = best ? place_of(best) : 0;
        put(tid, best & ~kPlace, at / M, key_at(at));
      }
      return;
    }
    if (tid >= 32) return;
    put_by_key();
    return;
  }
  const int depth = min(M, kMergeScores / lists);
  for (int i = tid; i < lists * depth; i += kMergeThreads) {
    const int l = i / depth, n = i % depth;
    const uint64_t o = score_of(l, n == 0, keys[(int64_t)l * M + n], round_reach);
    s_score[i] = o;
    if (n == 0) {
      s_head[l] = o;
      s_next[l] = 0;
    }
  }
  // (of many coarse ones each would be compared with up to 2048)
  const int num_coarse = __syncthreads_count(coarse);
  if (num_coarse > 0) {
    bool hidden = num_coarse > 32;
    if (!hidden)
      hidden = scores_hide_keys(by_key(), s_score, 0, lists * depth, depth, round_reach);
    coarse = false;
    if (__syncthreads_or(hidden)) {
      if (tid < 32) put_by_key();
      return;
    }
  }
  if (tid >= 32) return;
  uint64_t best = 0;  // the best head of this lane's lists
  int best_list = tid;
  auto look = [&] {
    best = 0;
    for (int l = tid; l < lists; l += 32)
      if (s_head[l] > best) {
        best = s_head[l];
        best_list = l;
      }
  };
  look();
  for (int i = 0; i < M; ++i) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32));
    const bool high = (uint32_t)(best >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(0xffffffffu, high ? (uint32_t)best : 0u);
    const uint64_t top = (uint64_t)hi << 32 | lo;
    const uint32_t l = __reduce_min_sync(0xffffffffu, best == top ? (uint32_t)best_list : ~0u);
    if (best == top && (uint32_t)best_list == l) {  // one lane: lists are dealt out by lane
      s_won[i] = top;
      if (top != 0) {
        const int n = s_next[l];
        s_list[i] = (int)l;
        s_at[i] = n;
        s_next[l] = n + 1;
        s_head[l] = n + 1 >= M       ? 0
                    : n + 1 < depth ? s_score[(int)l * depth + n + 1]
                                    : score_of((int)l, false, keys[(int64_t)l * M + n + 1],
                                               round_reach);
        look();
      }
    }
    __syncwarp();
  }
  if (__any_sync(0xffffffffu, coarse)) put_by_key();
  else put_won();
}

// How a call's rows are cut.  Tiles of 32 elements a thread where they give every SM a few
// CTAs and a row fills half of one, else of 8 (836 rows of 8009 fp16 19 us, by 8 23; 516 of 586
// bf16 14 us, by 32 16); splits of a row so that about kCtasPerSm CTAs an SM share the work (of
// 152 SMs: the cut must not depend on the device, the workspace goes by it).
struct BeamCut {
  int elems, tiles, splits;
};
BeamCut beam_cut(int64_t rows, int32_t num_beams, int32_t vocab) {
  constexpr int64_t kSms = 152, kCtasPerSm = 4, kLargeTiles = 4096;
  BeamCut c;
  c.elems = rows * (vocab / (kThreads * 32) + 1) >= 2 * kSms && vocab >= kLargeTiles ? 32 : 8;
  c.tiles = (vocab + kThreads * c.elems - 1) / (kThreads * c.elems);
  int64_t s = kCtasPerSm * kSms / std::max<int64_t>(rows, 1);
  s = std::min<int64_t>(s, std::min(c.tiles, std::max(kMaxLists / num_beams, 1)));
  c.splits = (int)std::max<int64_t>(s, 1);
  return c;
}
int64_t part_bytes(int64_t rows, int splits) { return align_up(rows * splits * 8, 16); }

template <typename T, int kHalf, int kVec>
cudaError_t launch_rows_t(const BeamParams &p, int64_t ctas, pkv_stream stream) {
  constexpr auto kern = beam_rows_kernel<T, kHalf, kVec>;
  const cudaError_t pe = prepare_kernel<kern>(0);
  if (pe != cudaSuccess) return pe;
  return launch_kernel(kern, dim3((unsigned)ctas), dim3(kThreads), 0, stream, !profiling_active(), p);
}

// fp32 rows of which some start off 16-byte alignment: an element a load, a warp's next to each
// other (512 rows of 128000 in 58 us; put together from 16-byte pieces 78, aligned ones 51).  It
// is the same for all rows of a call, so that equal rows get equal sums.
template <typename T>
cudaError_t launch_rows(const BeamParams &p, int elems, int64_t ctas, pkv_stream stream) {
  if constexpr (sizeof(T) == 4) {
    if ((reinterpret_cast<uintptr_t>(p.logits) & 15u) || (p.num_rows > 1 && p.row_stride % 4 != 0))
      return elems == 32 ? launch_rows_t<T, 16, 1>(p, ctas, stream)
                         : launch_rows_t<T, 4, 1>(p, ctas, stream);
  }
  return elems == 32 ? launch_rows_t<T, 16, 8>(p, ctas, stream)
                     : launch_rows_t<T, 4, 4>(p, ctas, stream);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_beam_workspace_size(int32_t num_requests, int32_t num_beams, int32_t vocab,
                                          int32_t num_select) {
  if (num_requests <= 0 || num_beams < 1 || num_beams > kMaxLists || vocab < 1 ||
      vocab > kMaxVocab || num_select < 1)
    return 0;
  const int64_t rows = (int64_t)num_requests * num_beams;
  const BeamCut c = beam_cut(rows, num_beams, vocab);
  return (size_t)(part_bytes(rows, c.splits) + rows * c.splits * num_select * 8);
}

extern "C" pkv_status pkv_beam_select(const void *logits, int32_t logit_type, int64_t row_stride,
                                      const float *cum_scores, const uint8_t *finished,
                                      int32_t num_requests, int32_t num_beams, int32_t vocab,
                                      int32_t num_select, int32_t pad_token, float *scores,
                                      int32_t *tokens, int32_t *parents, void *workspace,
                                      int64_t workspace_bytes, pkv_stream stream) {
  if (num_requests < 0 || num_beams < 1 || vocab < 1 || num_select < 1) return PKV_ERR_SHAPE;
  if (num_select > kMaxSelect || num_beams > kMaxLists) return PKV_ERR_UNSUPPORTED;
  if (logit_type != PKV_BF16 && logit_type != PKV_FP16 && logit_type != PKV_FP32)
    return PKV_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)num_requests * num_beams;
  if (rows > 1 && row_stride < vocab) return PKV_ERR_SHAPE;
  if (vocab > kMaxVocab) return PKV_ERR_UNSUPPORTED;
  if (num_requests == 0) return PKV_OK;
  if (!logits || !cum_scores || !scores || !tokens || !parents || !workspace) return PKV_ERR_NULL;
  const uintptr_t size = logit_type == PKV_FP32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(logits) & (size - 1)) ||
      (reinterpret_cast<uintptr_t>(cum_scores) & 3u) || (reinterpret_cast<uintptr_t>(scores) & 3u) ||
      (reinterpret_cast<uintptr_t>(tokens) & 3u) || (reinterpret_cast<uintptr_t>(parents) & 3u) ||
      (reinterpret_cast<uintptr_t>(workspace) & 15u))
    return PKV_ERR_ALIGN;
  const BeamCut c = beam_cut(rows, num_beams, vocab);
  if (rows * c.splits > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (workspace_bytes < part_bytes(rows, c.splits) + rows * c.splits * num_select * 8)
    return PKV_ERR_WORKSPACE;
  BeamParams p;
  p.logits = logits;
  p.cum = cum_scores;
  p.finished = finished;
  p.scores = scores;
  p.tokens = tokens;
  p.parents = parents;
  p.part = static_cast<float2 *>(workspace);
  p.keys = reinterpret_cast<uint64_t *>(static_cast<char *>(workspace) + part_bytes(rows, c.splits));
  p.row_stride = row_stride;
  p.num_rows = rows;
  p.num_beams = num_beams;
  p.vocab = vocab;
  p.num_select = num_select;
  p.pad_token = pad_token;
  p.splits = c.splits;
  p.tiles = c.tiles;
  if (prepare_kernel<beam_merge_kernel>(0) != cudaSuccess) return PKV_ERR_CUDA;
  profile_begin(PKV_KERNEL_BEAM, stream);
  const int64_t ctas = rows * c.splits;
  cudaError_t e = logit_type == PKV_BF16   ? launch_rows<__nv_bfloat16>(p, c.elems, ctas, stream)
                  : logit_type == PKV_FP16 ? launch_rows<__half>(p, c.elems, ctas, stream)
                                           : launch_rows<float>(p, c.elems, ctas, stream);
  if (e == cudaSuccess)
    e = launch_kernel(beam_merge_kernel, dim3((unsigned)num_requests), dim3(kMergeThreads), 0,
                      stream, !profiling_active(), p);
  profile_end(PKV_KERNEL_BEAM, stream);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return PKV_ERR_CUDA;
  count_launches(2);
  return PKV_OK;
}
