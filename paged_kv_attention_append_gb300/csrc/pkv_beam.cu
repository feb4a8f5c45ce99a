// Beam search's selection: log-softmax of each beam's logits, added to its score, and
// the best continuations over all beams of a request.
//
//   score(k, t) = cum_k + x_kt - log sum_u exp(x_ku);  the num_select largest of (k, t),
//   ties to the lower beam, then the lower token.
//
// Within a beam the score grows with the logit, so the best of a beam are its largest
// logits and need no logarithm.  The logits are read once: a CTA goes over a range of
// one row in tiles that stay in registers and takes from them, at the same time,
//  - the running maximum and sum of exponentials (per thread, rescaled when its maximum
//    moves; joined over the CTA at the end);
//  - the candidates: 64-bit keys (logit, lowest token first), so that no two are equal.
//    A threshold T below the num_select-th largest key comes from the threads' maxima of
//    the first tile; keys above T go to a buffer in shared memory, which is cut to its
//    num_select largest (and T raised) when it fills.  After the first tile hardly any
//    key passes: the expected number is num_select ln(tiles).
// A second kernel, one warp a request, joins the rows' sums and merges the sorted lists
// by score in 64 bits.
//
// Which elements a thread sums depends on their place in the row alone, not on the row's
// address: equal rows get equal sums, and their ties go by the beam.
//
// Bound by HBM for large calls, by latency (two launches) for small ones.
#include <cuda_runtime.h>

#include <algorithm>

#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kBeamWarps = kThreads / 32;
constexpr int kMaxSelect = 128;
constexpr int kBuffer = 512;        // candidate keys a CTA keeps (>= 2 kMaxSelect)
constexpr int kMaxLists = 1024;     // sorted lists (beam, split) of a request
constexpr int kVec = 8;             // consecutive elements a thread loads together
constexpr float kLog2e = 1.4426950408889634f;

struct BeamParams {
  const void *logits;
  const float *cum;
  const uint8_t *finished;
  float *scores;
  int32_t *tokens, *parents;
  float2 *part;          // [rows][splits]: maximum, sum of exp(x - maximum)
  uint64_t *keys;        // [rows][splits][num_select], descending, 0: none
  int64_t row_stride;
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

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// Elements [at, at + 8) of a row; those past its end as -inf.
template <typename T>
__device__ __forceinline__ void load8(const T *row, int32_t at, int32_t vocab, bool aligned,
                                      float *x) {
  if (aligned && at + kVec <= vocab) {
    union {
      uint4 v[sizeof(T) * kVec / 16];
      T e[kVec];
    } u;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) * kVec / 16); ++i)
      u.v[i] = __ldcs(reinterpret_cast<const uint4 *>(row + at) + i);
#pragma unroll
    for (int i = 0; i < kVec; ++i) x[i] = to_float(u.e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) x[i] = at + i < vocab ? to_float(row[at + i]) : -INFINITY;
  }
}

__device__ __forceinline__ int32_t block_sum(int32_t v, int32_t *s) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  int32_t t = 0;
#pragma unroll
  for (int w = 0; w < kBeamWarps; ++w) t += s[w];
  return t;
}

// The lane keys of a warp in descending order (bitonic).
__device__ __forceinline__ uint64_t warp_sort(uint64_t k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, k, o);
      const bool up = ((lane & size) == 0) == ((lane & o) == 0);  // keeps the larger
      k = up ? (k > other ? k : other) : (k < other ? k : other);
    }
  return k;
}

// The `cnt` keys of s_buf in descending order, its first min(cnt, keep) of them: each
// key's place is the number of larger ones.
__device__ __forceinline__ void sort_buffer(uint64_t *s_buf, int cnt, int keep) {
  uint64_t k[kBuffer / kThreads];
  int rank[kBuffer / kThreads];
#pragma unroll
  for (int u = 0; u < kBuffer / kThreads; ++u) {
    const int i = threadIdx.x + u * kThreads;
    k[u] = i < cnt ? s_buf[i] : 0;
    rank[u] = 0;
  }
  if (cnt <= kThreads) {
    for (int j = 0; j < cnt; ++j) rank[0] += s_buf[j] > k[0];
  } else {
    for (int j = 0; j < cnt; ++j) {
      const uint64_t o = s_buf[j];
#pragma unroll
      for (int u = 0; u < kBuffer / kThreads; ++u) rank[u] += o > k[u];
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kBuffer / kThreads; ++u)
    if (threadIdx.x + u * kThreads < cnt && rank[u] < keep) s_buf[rank[u]] = k[u];
  __syncthreads();
}

template <typename T, int kElems>
__global__ void __launch_bounds__(kThreads) beam_rows_kernel(const BeamParams p) {
  __shared__ uint64_t s_buf[kBuffer];
  __shared__ uint64_t s_warp[2 * kBeamWarps];
  __shared__ float s_m[kBeamWarps], s_s[kBeamWarps];
  __shared__ int32_t s_sum[kBeamWarps];
  __shared__ int32_t s_cnt;
  constexpr int kTile = kThreads * kElems;
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row_id = blockIdx.x / p.splits;
  const int split = blockIdx.x % p.splits;
  if (p.finished && __ldg(p.finished + row_id)) return;  // the merge does not look at its parts
  const T *row = static_cast<const T *>(p.logits) + row_id * p.row_stride;
  const bool aligned = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
  const int tile0 = (int)((int64_t)p.tiles * split / p.splits);
  const int tile1 = (int)((int64_t)p.tiles * (split + 1) / p.splits);
  const int M = p.num_select;
  float m = -INFINITY, s = 0.f;
  uint64_t T_key = 0;       // candidates are the keys above this
  float T_val = -INFINITY;  // its logit: a cheaper test that lets through no fewer
  if (tid == 0) s_cnt = 0;
  for (int tile = tile0; tile < tile1; ++tile) {
    const int32_t at0 = tile * kTile + tid * kVec;
    float x[kElems];
#pragma unroll
    for (int j = 0; j < kElems / kVec; ++j)
      load8(row, at0 + j * kThreads * kVec, p.vocab, aligned, x + j * kVec);
    float top = x[0];
#pragma unroll
    for (int i = 1; i < kElems; ++i) top = fmaxf(top, x[i]);
    const float m_new = fmaxf(m, top);
    if (m_new > -INFINITY) {
      s *= fast_exp2((m - m_new) * kLog2e);
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int i = 0; i < kElems; i += 2) {
        a += fast_exp2((x[i] - m_new) * kLog2e);
        b += fast_exp2((x[i + 1] - m_new) * kLog2e);
      }
      s += a + b;
      m = m_new;
    } else {
#pragma unroll
      for (int i = 0; i < kElems; ++i)  // all masked; a NaN makes the row's sum NaN
        if (x[i] != x[i]) s = x[i];
    }
    auto token = [&](int i) { return at0 + (i / kVec) * kThreads * kVec + i % kVec; };
    auto count_above = [&](uint64_t t) {
      int32_t n = 0;
#pragma unroll
      for (int i = 0; i < kElems; ++i) n += token(i) < p.vocab && make_key(x[i], token(i)) > t;
      return n;
    };
    if (tile == tile0) {
      // every warp's M-th largest thread maximum is a lower bound of the M-th largest
      // key, and so is the smallest over the warps of their ceil(M / 8)-th
      int32_t at = at0;
      float best = x[0];
#pragma unroll
      for (int i = 1; i < kElems; ++i)
        if (x[i] > best) {
          best = x[i];
          at = token(i);
        }
      const uint64_t k = warp_sort(at < p.vocab ? make_key(best, at) : 0);
      const uint64_t k1 = M <= 32 ? __shfl_sync(0xffffffffu, k, (M - 1) & 31) : 0;
      const uint64_t k2 = __shfl_sync(0xffffffffu, k, (M + kBeamWarps - 1) / kBeamWarps - 1);
      if (lane == 0) {
        s_warp[warp] = k1;
        s_warp[kBeamWarps + warp] = k2;
      }
      __syncthreads();
      uint64_t t1 = 0, t2 = ~0ull;
#pragma unroll
      for (int w = 0; w < kBeamWarps; ++w) {
        t1 = max(t1, s_warp[w]);
        t2 = min(t2, s_warp[kBeamWarps + w]);
      }
      T_key = max(t1, t2);
      if (T_key) --T_key;  // that key itself is a candidate
      T_val = T_key ? key_value(T_key + 1) : -INFINITY;
    }
    // (a tile without a candidate: one barrier)
    if (!__syncthreads_or(!(top < T_val))) continue;
    while (true) {
      const int32_t n = top < T_val ? 0 : count_above(T_key);
      const int32_t total = block_sum(n, s_sum);
      const int32_t cnt = s_cnt;
      if (total == 0) break;
      if (cnt + total <= kBuffer) {
        __syncthreads();  // every thread has read s_cnt
        if (n) {
          int32_t at = atomicAdd(&s_cnt, n);
#pragma unroll
          for (int i = 0; i < kElems; ++i) {
            const uint64_t k = make_key(x[i], token(i));
            if (token(i) < p.vocab && k > T_key) s_buf[at++] = k;
          }
        }
        __syncthreads();
        if (tile == tile0 && tile + 1 < tile1 && s_cnt > M) {
          sort_buffer(s_buf, s_cnt, M);
          if (tid == 0) s_cnt = M;
          T_key = s_buf[M - 1];
          T_val = key_value(T_key);
          __syncthreads();
        }
        break;
      }
      if (cnt > M) {  // the buffer's M largest stay, and T is the last of them
        sort_buffer(s_buf, cnt, M);
        if (tid == 0) s_cnt = M;
        T_key = s_buf[M - 1];
      } else {
        // rows that rise from tile to tile: the T that leaves M keys of this tile
        // above it, bit by bit (keys are unique, so there is one)
        uint64_t t = 0;
        for (int bit = 63; bit >= 0; --bit) {
          const uint64_t c = t | 1ull << bit;
          if (block_sum(count_above(c), s_sum) >= M) t = c;
        }
        T_key = max(T_key, t);
      }
      T_val = key_value(T_key);
      __syncthreads();
    }
  }
  __syncthreads();
  const int cnt = s_cnt;
  sort_buffer(s_buf, cnt, M);
  uint64_t *out = p.keys + ((int64_t)row_id * p.splits + split) * M;
  for (int i = tid; i < M; i += kThreads) out[i] = i < cnt ? s_buf[i] : 0;
  // the threads' sums, at the CTA's maximum
  float wm = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
  if (lane == 0) s_m[warp] = wm;
  __syncthreads();
  float bm = s_m[0];
#pragma unroll
  for (int w = 1; w < kBeamWarps; ++w) bm = fmaxf(bm, s_m[w]);
  s *= m == bm ? 1.f : fast_exp2((m - bm) * kLog2e);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) s_s[warp] = s;
  __syncthreads();
  if (tid == 0) {
    float t = s_s[0];
#pragma unroll
    for (int w = 1; w < kBeamWarps; ++w) t += s_s[w];
    p.part[(int64_t)row_id * p.splits + split] = make_float2(bm, t);
  }
}

// A double as an integer of the same order, 0 for what is not finite.
__device__ __forceinline__ uint64_t order_double(double x) {
  if (!isfinite(x)) return 0;
  const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
  return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double unorder_double(uint64_t o) {
  return __longlong_as_double((long long)(o >> 63 ? o ^ 1ull << 63 : ~o));
}

// One warp a request: M rounds over the heads of its sorted lists.  List k splits + j
// holds beam k's best of its j-th range: equal scores go to the lower list.
__global__ void __launch_bounds__(32) beam_merge_kernel(const BeamParams p) {
  __shared__ double s_base[kMaxLists];      // cum - lse of the request's beams
  __shared__ uint64_t s_head[kMaxLists];    // ordered score of each list's first key left
  __shared__ int32_t s_next[kMaxLists];
  const int lane = threadIdx.x;
  const int64_t row0 = (int64_t)blockIdx.x * p.num_beams;
  const int lists = p.num_beams * p.splits, M = p.num_select;
  pdl_wait();
  for (int k = lane; k < p.num_beams; k += 32) {
    double base = __ldg(p.cum + row0 + k);
    if (!(p.finished && __ldg(p.finished + row0 + k))) {
      const float2 *part = p.part + (row0 + k) * p.splits;
      float m = part[0].x;
      for (int j = 1; j < p.splits; ++j) m = fmaxf(m, part[j].x);
      float s = 0.f;
      for (int j = 0; j < p.splits; ++j)
        s += part[j].y * (part[j].x == m ? 1.f : exp2f((part[j].x - m) * kLog2e));
      base -= (double)m + log((double)s);
    }
    s_base[k] = base;
  }
  __syncwarp();
  // the ordered score of list l's key n (0: none left)
  auto score_of = [&](int l, int n) -> uint64_t {
    const int k = l / p.splits;
    if (p.finished && __ldg(p.finished + row0 + k))
      return n == 0 && l == k * p.splits ? order_double(s_base[k]) : 0;
    if (n >= M) return 0;
    const uint64_t key = p.keys[(row0 * p.splits + l) * M + n];
    return key ? order_double(s_base[k] + (double)key_value(key)) : 0;
  };
  uint64_t best = 0;
  int best_list = lane;
  auto look = [&] {
    best = 0;
    for (int l = lane; l < lists; l += 32)
      if (s_head[l] > best) {
        best = s_head[l];
        best_list = l;
      }
  };
  for (int l = lane; l < lists; l += 32) {
    s_head[l] = score_of(l, 0);
    s_next[l] = 0;
  }
  look();
  for (int i = 0; i < M; ++i) {
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32));
    const bool mine = (uint32_t)(best >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(0xffffffffu, mine ? (uint32_t)best : 0u);
    const uint64_t top = (uint64_t)hi << 32 | lo;
    const uint32_t l = __reduce_min_sync(0xffffffffu, best == top ? (uint32_t)best_list : ~0u);
    if (best == top && (uint32_t)best_list == l) {  // one lane: lists are dealt out by lane
      const int64_t o = (int64_t)blockIdx.x * M + i;
      const int k = (int)l / p.splits;
      if (top == 0) {
        p.scores[o] = -INFINITY;
        p.tokens[o] = p.parents[o] = -1;
      } else {
        p.scores[o] = (float)unorder_double(top);
        p.parents[o] = (int32_t)(row0 + k);
        p.tokens[o] = p.finished && __ldg(p.finished + row0 + k)
                          ? p.pad_token
                          : (int32_t)~(uint32_t)p.keys[(row0 * p.splits + l) * M + s_next[l]];
        s_head[l] = score_of((int)l, ++s_next[l]);
        look();
      }
    }
    __syncwarp();
  }
}

// How a call's rows are cut.  Tiles of 8192 elements (32 a thread) where they give every
// SM a few CTAs, else of 2048; splits of a row so that about 16 CTAs an SM share the
// work (of 152 SMs: the cut must not depend on the device, the workspace goes by it).
struct BeamCut {
  int elems, tiles, splits;
};
BeamCut beam_cut(int64_t rows, int32_t num_beams, int32_t vocab) {
  constexpr int64_t kSms = 152;
  BeamCut c;
  c.elems = rows * ((vocab + 8191) / 8192) >= 2 * kSms ? 32 : 8;
  c.tiles = (vocab + kThreads * c.elems - 1) / (kThreads * c.elems);
  int64_t s = (16 * kSms + rows - 1) / std::max<int64_t>(rows, 1);
  s = std::min<int64_t>(s, std::min(c.tiles, std::max(kMaxLists / num_beams, 1)));
  c.splits = (int)std::max<int64_t>(s, 1);
  return c;
}
int64_t part_bytes(int64_t rows, int splits) { return align_up(rows * splits * 8, 16); }

template <typename T>
cudaError_t launch_rows(const BeamParams &p, int elems, int64_t ctas, pkv_stream stream) {
  auto kern = elems == 32 ? beam_rows_kernel<T, 32> : beam_rows_kernel<T, 8>;
  const cudaError_t pe = elems == 32 ? prepare_kernel<beam_rows_kernel<T, 32>>(0)
                                     : prepare_kernel<beam_rows_kernel<T, 8>>(0);
  if (pe != cudaSuccess) return pe;
  return launch_kernel(kern, dim3((unsigned)ctas), dim3(kThreads), 0, stream, false, p);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_beam_workspace_size(int32_t num_requests, int32_t num_beams, int32_t vocab,
                                          int32_t num_select) {
  if (num_requests <= 0 || num_beams < 1 || num_beams > kMaxLists || vocab < 1 || num_select < 1)
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
  // tokens of a tile are numbered in 32 bits past the vocabulary's end
  if (vocab > INT32_MAX - 65536) return PKV_ERR_UNSUPPORTED;
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
  p.num_beams = num_beams;
  p.vocab = vocab;
  p.num_select = num_select;
  p.pad_token = pad_token;
  p.splits = c.splits;
  p.tiles = c.tiles;
  if (prepare_kernel<beam_merge_kernel>(0) != cudaSuccess) return PKV_ERR_CUDA;
  profile_begin(PKV_KERNEL_BEAM, stream);
  cudaError_t e = logit_type == PKV_BF16
                      ? launch_rows<__nv_bfloat16>(p, c.elems, rows * c.splits, stream)
                  : logit_type == PKV_FP16 ? launch_rows<__half>(p, c.elems, rows * c.splits, stream)
                                           : launch_rows<float>(p, c.elems, rows * c.splits, stream);
  if (e == cudaSuccess)
    e = launch_kernel(beam_merge_kernel, dim3((unsigned)num_requests), dim3(32), 0, stream,
                      !profiling_active(), p);
  profile_end(PKV_KERNEL_BEAM, stream);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return PKV_ERR_CUDA;
  count_launches(2);
  return PKV_OK;
}
