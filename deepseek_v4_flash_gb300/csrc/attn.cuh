// attn.cuh -- device helpers shared by the attention kernels: which positions
// a query sees, where a position lies in the paged cache, and the attention
// of one row by one warp.
//
// The query at position i sees position j when
//   j <= i  and  (window == 0  or  j > i - window  or  j < n_sink).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn.h"
#include "common.cuh"

namespace ds4 {

template <int DT>
struct Half16;  // the two 16-bit types
template <>
struct Half16<DS4MOE_DT_BF16> {
  static constexpr uint32_t INF = 0x7F80;  // bits of infinity; a larger magnitude is a NaN
  static __device__ __forceinline__ float2 up(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t down(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
};
template <>
struct Half16<DS4MOE_DT_F16> {
  static constexpr uint32_t INF = 0x7C00;
  static __device__ __forceinline__ float2 up(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
  }
  static __device__ __forceinline__ uint32_t down(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Row bounds of a ragged call (cu_q): each is brought into [0, n_tok] and
// raised to the largest before it. Sequences then never share a row, and their
// rows are at most n_tok in all: the workspace is sized by that.
__device__ __forceinline__ int clamp_row(int c, int n_tok) { return min(max(c, 0), n_tok); }

// Bounds (first row, end) of sequence b = b0 + threadIdx.x, by a block of
// 1024 threads for b0 = 0, 1024, ...; `base` (shared, 0 at first) is the
// largest bound of the sequences before. `bad` is set where a bound changed.
__device__ __forceinline__ int2 clean_rows(const int32_t *cu, int n_seq, int n_tok, int b, int *base, int *warp_top,
                                           bool &bad) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int raw0 = b < n_seq ? cu[b] : 0, raw1 = b < n_seq ? cu[b + 1] : 0, from = *base;
  int c0 = clamp_row(raw0, n_tok), c1 = clamp_row(raw1, n_tok);
  const bool wrong = b < n_seq && (c0 != raw0 || c1 != raw1 || c0 > c1 || c0 < from);
  if (__syncthreads_or(wrong)) {
    // running maximum of the first rows
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, c0, o);
      if (lane >= o) c0 = max(c0, x);
    }
    if (lane == 31) warp_top[w] = c0;
    __syncthreads();
    c0 = max(c0, from);
    for (int i = 0; i < w; i++) c0 = max(c0, warp_top[i]);
    c1 = max(c0, c1);
    bad |= b < n_seq && (c0 != raw0 || c1 != raw1);
  }
  if (threadIdx.x == 1023) *base = c1;  // (only used when another 1024 follow)
  __syncthreads();
  return make_int2(c0, c1);
}

// Rows and length of sequence b (a ragged call's bounds are clean); the length
// is clamped to what the table holds, and `bad` set where it had to be (the
// caller raises DS4MOE_DEVERR_LENGTH).
struct SeqInfo {
  int tok0, n, len;  // first row of q, rows, cached positions
};
__device__ __forceinline__ int seq_len(const AttnArgs &a, int b, bool &bad) {
  const int l = a.kv_len[b], len = min(max(l, 0), a.kv.width * a.kv.page_size);
  bad |= len != l;
  return len;
}
__device__ __forceinline__ SeqInfo seq_info(const AttnArgs &a, int b, bool &bad) {
  SeqInfo s;
  if (a.cu_q) {
    s.tok0 = a.cu_q[b];
    s.n = a.cu_q[b + 1] - s.tok0;
  } else {
    s.tok0 = b * a.n_new;
    s.n = a.n_new;
  }
  s.len = seq_len(a, b, bad);
  return s;
}

// ---- a batch with shared positions

// Shared positions of group g, within what the table holds.
__device__ __forceinline__ int shared_of(const SharedArgs &a, int g, bool &bad) {
  const int l = a.shared_len[g], s = min(max(l, 0), a.kv.width * a.kv.page_size);
  bad |= s != l;
  return s;
}

// The group of a call without a planning launch: its sequences (the bounds
// brought into the batch and in order, as clean_rows does), and the shared
// positions that are read once.
__device__ __forceinline__ int2 one_group(const SharedArgs &a, int &s, bool &bad) {
  const int r0 = a.group_start ? a.group_start[0] : 0, r1 = a.group_start ? a.group_start[1] : a.batch;
  s = shared_of(a, 0, bad);
  const int c0 = clamp_row(r0, a.batch), c1 = max(clamp_row(r1, a.batch), c0);
  bad |= c0 != r0 || c1 != r1;
  if (a.cost.gain(s, c1 - c0) <= a.cost.least) s = 0;
  return make_int2(c0, c1);
}

// Where sequence b's own positions begin. It shares its group's positions when
// its first new token sees all of them.
__device__ __forceinline__ int own_start(const SharedArgs &a, int b, int len) {
  if (a.start) return a.start[b];
  bool bad = false;
  int s;
  const int2 c = one_group(a, s, bad);
  return b >= c.x && b < c.y && len - a.n_new + 1 >= s ? s : 0;
}

// The rows of group g, no rows where nothing is read once; its positions; the
// table's row through which they are read.
__device__ __forceinline__ SeqInfo prefix_info(const SharedArgs &a, int g, int *tab) {
  SeqInfo i = {0, 0, 0};
  if (a.start) {
    i.tok0 = a.cu_q[g], i.len = a.plen[g];
    if (i.len > 0) i.n = a.cu_q[g + 1] - i.tok0;
    if (tab) *tab = a.ptab[g];
    return i;
  }
  bool bad = false, ignored = false;
  int s;
  const int2 c = one_group(a, s, bad);
  if (bad && blockIdx.x == 0) raise_flag(a.err, DS4MOE_DEVERR_LENGTH);
  i.tok0 = c.x * a.n_new;
  if (s == 0) return i;
  for (int b = c.x; b < c.y; b++) {  // (the first, unless a place in the batch is empty)
    if (seq_len(a, b, ignored) - a.n_new + 1 < s) continue;
    if (tab) *tab = b;
    i.n = (c.y - c.x) * a.n_new, i.len = s;
    break;
  }
  return i;
}

// (calls without shared positions)
__device__ __forceinline__ int own_start(const AttnArgs &, int, int) { return 0; }
__device__ __forceinline__ SeqInfo prefix_info(const AttnArgs &, int, int *) { return {0, 0, 0}; }
// The results over the shared positions and log2 of their sums.
__device__ __forceinline__ float *pre_results(const SharedArgs &a) { return a.pre; }
__device__ __forceinline__ float *pre_results(const AttnArgs &) { return nullptr; }
__device__ __forceinline__ float *pre_logs(const SharedArgs &a) { return a.pre_log; }
__device__ __forceinline__ float *pre_logs(const AttnArgs &) { return nullptr; }

// log2 of a sum of weights l relative to 2^m.
__device__ __forceinline__ float log_sum(float m, float l) { return l == 0.0f ? -INFINITY : m + __log2f(l); }

// Joins a result with log2 sum `lp` and an accumulator relative to 2^m with sum
// l: the factors of the two, 0 for one without a score above -infinity. Both
// results are multiplied and added whatever the factors, for 0 times a NaN or an
// infinity that a row sees is NaN, as it is among the positions of one call;
// `zero`: the row has no score above -infinity at all, and is 0 whatever the values.
__device__ __forceinline__ void join_two(float lp, float m, float l, float &from, float &inv, bool &zero) {
  zero = l == 0.0f && lp == -INFINITY;
  if (l == 0.0f) {
    from = lp == -INFINITY ? 0.0f : lp == lp ? 1.0f : lp, inv = 0.0f;
    return;
  }
  const float top = fmaxf(lp, log_sum(m, l));
  const float p = lp == -INFINITY ? 0.0f : ex2(lp - top), o = ex2(m - top), z = 1.0f / fmaf(o, l, p);
  from = p * z, inv = o * z;
}

// First position of the window of the query at position i >= 0, and the
// number of first positions visible before it.
__device__ __forceinline__ int window_lo(const AttnArgs &a, int i) {
  return a.window > 0 && i >= a.window ? i - a.window + 1 : 0;
}

// pos / page_size, 0 <= pos < 2^31: with l = ceil(log2 page_size) and mul =
// ceil(2^(31 + l) / page_size) < 2^32 the product's error pos * (mul - exact) is
// below 2^31, less than a page_size-th of 2^(31 + l).
__device__ __forceinline__ int page_index(const KvView &kv, int pos) {
  return (int)(((unsigned long long)(uint32_t)pos * kv.div_mul) >> kv.div_sh);
}
// Page of a sequence's position, or -1 for a table entry outside the cache.
__device__ __forceinline__ int page_of(const KvView &kv, int b, int pos) {
  const int p = kv.table[(long long)b * kv.table_stride + page_index(kv, pos)];
  return p >= 0 && p < kv.n_pages ? p : -1;
}

// The groups of 2^sh positions (16 in the streaming kernel, up to 128 in the
// tile kernel) that hold every position visible to a query at positions
// first .. last (0 <= first <= last): the groups of the first positions, then
// those of the windows.
struct Groups {
  int n_sink;  // leading groups
  int win0;    // position group of list entry n_sink
  int n;       // list entries
};
__device__ __forceinline__ Groups groups_of(const AttnArgs &a, int first, int last, int sh = 4) {
  Groups g;
  const int lo = window_lo(a, first), w0 = lo >> sh, w1 = (last >> sh) + 1;
  const int ns = (min(a.n_sink, lo) + (1 << sh) - 1) >> sh;
  if (ns >= w0) {  // no gap
    g.n_sink = 0, g.win0 = 0, g.n = w1;
  } else {
    g.n_sink = ns, g.win0 = w0, g.n = ns + w1 - w0;
  }
  return g;
}
__device__ __forceinline__ int group_pos(const Groups &g, int i, int sh = 4) {
  return (i < g.n_sink ? i : g.win0 + i - g.n_sink) << sh;
}

// Rows whose products gave a NaN. Positions that a row does not see have a
// weight of 0 there, and 0 x NaN and 0 x infinity are NaN; so the row may have
// to be computed once more from what it sees alone. That takes a warp some 1000
// cycles per position, so first (every row behind one NaN in a prompt comes
// here: computing them all again took 44 ms instead of 0.08 for 2048 tokens of
// 32 heads):
//   - a row whose sum of weights l is NaN saw a NaN or infinite score, for
//     hidden scores weigh 0 in l: it stays NaN;
//   - a row with l = 0 has no score above -infinity: zeros;
//   - else a look (unseen_nonfinite) at the values that the products read and
//     the row does not see, for a warp's rows together, then for each. They lie
//     at the edges of a row tile's positions, a few hundred at most. All
//     finite: the NaN is the row's own;
//   - nor is there doubt when the row's own position has a NaN wherever the
//     result has one (own_nan): a prompt whose values are NaN from a token on.

// Whether a position that a query at pos0 .. pos1 does not see, among those of
// the products, has an infinity or NaN in columns [c0, c1) of its value (whole
// warp). The products read the positions from `win0` to `end` and the first
// `sinks` ones.
template <int DT>
__device__ __noinline__ bool unseen_nonfinite(const AttnArgs &a, int b, int kvh, int pos0, int pos1, int win0, int sinks,
                                            int end, int c0, int c1) {
  constexpr uint32_t LO = Half16<DT>::INF, HI = LO << 16;  // exponent bits
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (int part = 0; part < 3; part++) {
    // after the first query, between the last one's window and the first positions, in the first positions' groups
    int j = part == 0 ? pos0 + 1 : part == 1 ? max(win0, a.n_sink) : a.n_sink;
    const int to = part == 0 ? end : part == 1 ? window_lo(a, pos1) : sinks;
    while (j < to) {
      const int e = min(to, (j | 15) + 1), page = page_of(a.kv, b, j);  // 16 of them share a page
      if (page >= 0) {
        const uint16_t *vp = a.kv.v + (long long)page * a.kv.v_page + (long long)kvh * a.kv.v_head +
                             (long long)(j - page_index(a.kv, j) * a.kv.page_size) * a.kv.v_row;
        for (int c = c0 / 2 + lane; c < c1 / 2; c += 32) {
#pragma unroll 8
          for (int i = 0; i < e - j; i++) {
            const uint32_t u = reinterpret_cast<const uint32_t *>(vp + (long long)i * a.kv.v_row)[c];
            bad |= (u & LO) == LO || (u & HI) == HI;
          }
        }
      }
      j = e;
    }
  }
  return __any_sync(0xffffffffu, bad);
}

// Whether the value of the row's own position, `pos`, is NaN in each of the
// columns [c0, c1) where the row's result (`o`, column 0) is (whole warp).
template <int DT>
__device__ __noinline__ bool own_nan(const AttnArgs &a, const uint16_t *o, int b, int kvh, int pos, int c0, int c1) {
  constexpr uint32_t INF = Half16<DT>::INF;
  const int lane = threadIdx.x & 31, page = page_of(a.kv, b, pos);
  if (page < 0) return false;
  const uint16_t *vp = a.kv.v + (long long)page * a.kv.v_page + (long long)kvh * a.kv.v_head +
                       (long long)(pos - page_index(a.kv, pos) * a.kv.page_size) * a.kv.v_row;
  bool other = false;
  for (int c = c0 + lane; c < c1; c += 32)
    other |= (*(volatile const uint16_t *)(o + c) & 0x7FFFu) > INF && (vp[c] & 0x7FFFu) <= INF;
  return !__any_sync(0xffffffffu, other);
}

// One row (a token's head) over list entries [g0, g1) by one warp, 32 positions
// at a time, in 32 bits: nothing of a position that the row does not see enters.
// A lane takes one position's score, then the values' elements 2l + 64c and
// 2l + 64c + 1, which it accumulates. `m` is the running maximum of scale_log2 *
// score and `l` the sum of the weights relative to it (l = 0: no score above
// -infinity).
template <int DT, int D>
__device__ __forceinline__ void attn_row_warp(const AttnArgs &a, const uint16_t *q, int b, int kvh, int pos,
                                           const Groups &gr, int g0, int g1, float2 (&acc)[D / 64], float &m,
                                           float &l, bool &bad_page) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < D / 64; c++) acc[c] = make_float2(0.0f, 0.0f);
  m = -INFINITY, l = 0.0f;
  if (pos < 0) return;
  const int lo = window_lo(a, pos), sink = min(a.n_sink, lo);
  for (int g = g0; g < g1; g += 2) {
    const int mine = g + (lane >> 4), j = group_pos(gr, mine) + (lane & 15);
    const bool see = mine < g1 && j <= pos && (j >= lo || j < sink);
    const int page = see ? page_of(a.kv, b, j) : 0;
    if (page < 0) bad_page = true;
    const bool read = see && page >= 0;
    const int row = j - page_index(a.kv, j) * a.kv.page_size;
    float s = 0.0f, s2 = 0.0f;
    if (read) {
      const uint4 *k = reinterpret_cast<const uint4 *>(a.kv.k + (long long)page * a.kv.k_page + (long long)kvh * a.kv.k_head +
                                                       (long long)row * a.kv.k_row);
#pragma unroll 4
      for (int c = 0; c < D / 8; c++) {
        const uint4 x = k[c], y = reinterpret_cast<const uint4 *>(q)[c];
        float2 u = Half16<DT>::up(x.x), v = Half16<DT>::up(y.x);
        s = fmaf(u.x, v.x, s), s2 = fmaf(u.y, v.y, s2);
        u = Half16<DT>::up(x.y), v = Half16<DT>::up(y.y);
        s = fmaf(u.x, v.x, s), s2 = fmaf(u.y, v.y, s2);
        u = Half16<DT>::up(x.z), v = Half16<DT>::up(y.z);
        s = fmaf(u.x, v.x, s), s2 = fmaf(u.y, v.y, s2);
        u = Half16<DT>::up(x.w), v = Half16<DT>::up(y.w);
        s = fmaf(u.x, v.x, s), s2 = fmaf(u.y, v.y, s2);
      }
    }
    s = see ? (s + s2) * a.scale_log2 : -INFINITY;
    const float mn = fmaxf(m, warp_max(s)), f = mn == -INFINITY ? 1.0f : ex2(m - mn);
    const float w = s == -INFINITY ? 0.0f : ex2(s - mn);
    float sum = w;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    m = mn, l = fmaf(l, f, sum);
#pragma unroll
    for (int c = 0; c < D / 64; c++) acc[c].x *= f, acc[c].y *= f;
    const long long at = (long long)page * a.kv.v_page + (long long)kvh * a.kv.v_head + (long long)row * a.kv.v_row;
    auto add = [&](int u) {
      const float wu = __shfl_sync(0xffffffffu, w, u);
      const uint32_t *v = reinterpret_cast<const uint32_t *>(a.kv.v + __shfl_sync(0xffffffffu, at, u));
#pragma unroll
      for (int c = 0; c < D / 64; c++) {
        const float2 x = Half16<DT>::up(v[lane + 32 * c]);
        acc[c].x = fmaf(wu, x.x, acc[c].x), acc[c].y = fmaf(wu, x.y, acc[c].y);
      }
    };
    unsigned live = __ballot_sync(0xffffffffu, read);
    if (live == 0xffffffffu) {
#pragma unroll 4
      for (int u = 0; u < 32; u++) add(u);
    } else {
      for (; live; live &= live - 1) add(__ffs(live) - 1);
    }
  }
}

}  // namespace ds4
