// attn.cu -- the attention handle (ds4moe_attn_*): argument checks, the
// append of new keys and values to the paged cache, and the choice of kernel.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>

#include "attn.cuh"
#include "internal.h"

namespace ds4 {

// Copies rows of new keys and values to their places in the pages, rounding
// to the cache's type. One thread per 8 elements (16 bytes of the cache);
// neighbouring threads take neighbouring elements of a row. Bound by the bytes:
// 12291 tokens of 8 x 128 from fp32 26.5 us, 5.7 TB/s.
//
// Ragged calls: every block needs the row bounds ascending (see clean_rows). Up
// to AP_SEQS sequences it reads and checks them itself, for a search in shared
// memory (the reads go with those of the rows); for more, k_clean_rows puts
// them in the workspace first.
constexpr int AP_SEQS = 1024;
struct AppendArgs {
  KvView kv;
  const void *k, *v;           // v null: the keys only
  long long k_stride, v_stride;
  const int32_t *kv_len, *cu_q;
  int32_t n_seq, n_tok, n_new, n_kv, D, per_tok;  // per_tok: 8-element pieces of a token's keys
  uint32_t *err;
};

__global__ void __launch_bounds__(1024) k_clean_rows(const int32_t *cu, int n_seq, int n_tok, int32_t *clean, uint32_t *err) {
  __shared__ int top[32], base;
  pdl_launch_dependents();
  pdl_wait();
  if (threadIdx.x == 0) base = 0;
  __syncthreads();
  bool bad = false;
  for (int b0 = 0; b0 < n_seq; b0 += 1024) {
    const int b = b0 + threadIdx.x;
    const int2 c = clean_rows(cu, n_seq, n_tok, b, &base, top, bad);
    if (b < n_seq) clean[b] = c.x;
    if (b + 1 == n_seq) clean[n_seq] = c.y;
  }
  if (bad) raise_flag(err, DS4MOE_DEVERR_LENGTH);
}

template <int DT, bool F32, int P>
__global__ void __launch_bounds__(128) k_kv_append(const AppendArgs a) {
  __shared__ int s_cu[AP_SEQS + 1];
  pdl_launch_dependents();
  pdl_wait();
  const long long total = (long long)a.n_tok * a.per_tok;
  const int kv = blockIdx.y;
  const char *src = (const char *)(kv ? a.v : a.k);
  const long long stride = kv ? a.v_stride : a.k_stride;
  uint4 x[P], y[P];
  uint16_t *dst[P];
  int row_t[P], row_e[P];  // this thread's pieces: token (-1: none) and element
#pragma unroll
  for (int j = 0; j < P; j++) {
    dst[j] = nullptr, row_t[j] = -1;
    const long long i = (long long)blockIdx.x * (128 * P) + j * 128 + threadIdx.x;
    if (i >= total) continue;
    const int t = (int)(i / a.per_tok), e = (int)(i - (long long)t * a.per_tok) * 8;
    const char *p = src + ((long long)t * stride + e) * (F32 ? 4 : 2);
    x[j] = reinterpret_cast<const uint4 *>(p)[0];
    if (F32) y[j] = reinterpret_cast<const uint4 *>(p)[1];
    row_t[j] = t, row_e[j] = e;
  }
  const int *cu = a.cu_q;
  if (a.cu_q && a.n_seq <= AP_SEQS) {
    bool bad = false;
    int last = 0;
    for (int i = threadIdx.x; i <= a.n_seq; i += 128) {
      const int raw = a.cu_q[i], c = clamp_row(raw, a.n_tok);
      bad |= raw != c || (i > 0 && clamp_row(a.cu_q[i - 1], a.n_tok) > c);
      s_cu[i] = c;
    }
    if (__syncthreads_or(bad)) {
      if (threadIdx.x == 0) {
        if (blockIdx.x == 0) raise_flag(a.err, DS4MOE_DEVERR_LENGTH);
        for (int i = 0; i <= a.n_seq; i++) s_cu[i] = last = max(last, s_cu[i]);
      }
      __syncthreads();
    }
    cu = s_cu;
  }
#pragma unroll
  for (int j = 0; j < P; j++) {
    if (row_t[j] < 0) continue;
    const int t = row_t[j], e = row_e[j];
    int b, at, n;
    if (!a.cu_q) {
      b = t / a.n_new, at = t - b * a.n_new, n = a.n_new;
    } else {
      // the last sequence that starts at or before row t
      int lo = 0, hi = a.n_seq;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
      }
      b = lo;
      const int c0 = cu[b], c1 = cu[b + 1];
      if (t < c0 || t >= c1) continue;  // a row of no sequence
      at = t - c0, n = c1 - c0;
    }
    const long long pos = (long long)a.kv_len[b] - n + at;
    if (pos < 0 || pos >= (long long)a.kv.width * a.kv.page_size) {
      raise_flag(a.err, DS4MOE_DEVERR_LENGTH);
      continue;
    }
    const int page = page_of(a.kv, b, (int)pos);
    if (page < 0) {
      raise_flag(a.err, DS4MOE_DEVERR_PAGE);
      continue;
    }
    const int row = (int)pos - page_index(a.kv, (int)pos) * a.kv.page_size, h = e / a.D, d = e - h * a.D;
    dst[j] = const_cast<uint16_t *>(kv ? a.kv.v : a.kv.k);
    dst[j] += kv ? (long long)page * a.kv.v_page + (long long)row * a.kv.v_row + (long long)h * a.kv.v_head + d
                 : (long long)page * a.kv.k_page + (long long)row * a.kv.k_row + (long long)h * a.kv.k_head + d;
  }
#pragma unroll
  for (int j = 0; j < P; j++) {
    if (!dst[j]) continue;
    uint4 o = x[j];
    if (F32) {
      auto f = [](uint32_t u) { return __uint_as_float(u); };
      o = make_uint4(Half16<DT>::down(f(x[j].x), f(x[j].y)), Half16<DT>::down(f(x[j].z), f(x[j].w)),
                     Half16<DT>::down(f(y[j].x), f(y[j].y)), Half16<DT>::down(f(y[j].z), f(y[j].w)));
    }
    *reinterpret_cast<uint4 *>(dst[j]) = o;
  }
}

// The steps of k_kv_append for k_append_rope, below. (k_kv_append on these took
// 28.0 us instead of 26.4 for the 12291 tokens: it keeps them in its loop.)

// The row bounds of a ragged append, ascending: in shared memory (s_cu) by a
// whole block of 128 threads, or (more than AP_SEQS sequences) as they are, for
// k_clean_rows has been there. Null: no bounds.
__device__ __forceinline__ const int *append_bounds(const int32_t *cu_q, int n_seq, int n_tok, int *s_cu, uint32_t *err) {
  if (!cu_q || n_seq > AP_SEQS) return cu_q;
  bool bad = false;
  int last = 0;
  for (int i = threadIdx.x; i <= n_seq; i += 128) {
    const int raw = cu_q[i], c = clamp_row(raw, n_tok);
    bad |= raw != c || (i > 0 && clamp_row(cu_q[i - 1], n_tok) > c);
    s_cu[i] = c;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      if (blockIdx.x == 0) raise_flag(err, DS4MOE_DEVERR_LENGTH);
      for (int i = 0; i <= n_seq; i++) s_cu[i] = last = max(last, s_cu[i]);
    }
    __syncthreads();
  }
  return s_cu;
}

// Sequence and position of new row t; false for a row of no sequence.
__device__ __forceinline__ bool append_seq(const int32_t *kv_len, const int *cu, int n_seq, int n_new, int t, int &b,
                                          long long &pos) {
  int at, n;
  if (!cu) {
    b = t / n_new, at = t - b * n_new, n = n_new;
  } else {
    // the last sequence that starts at or before row t
    int lo = 0, hi = n_seq;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
    const int c0 = cu[b], c1 = cu[b + 1];
    if (t < c0 || t >= c1) return false;
    at = t - c0, n = c1 - c0;
  }
  pos = (long long)kv_len[b] - n + at;
  return true;
}

// Page of a position to be written; false, with the flag, where there is none.
__device__ __forceinline__ bool append_page(const KvView &kv, int b, long long pos, uint32_t *err, int &page) {
  if (pos < 0 || pos >= (long long)kv.width * kv.page_size) {
    raise_flag(err, DS4MOE_DEVERR_LENGTH);
    return false;
  }
  page = page_of(kv, b, (int)pos);
  if (page < 0) raise_flag(err, DS4MOE_DEVERR_PAGE);
  return page >= 0;
}

// The append with the positions' rotation on the way, for the keys and, in the
// same launch, the queries. Pair (x, y) of a head at position p becomes
//   (x cos - y sin, y cos + x sin),  angle p * inv_freq[i],
// in 32 bits, rounded once. A thread takes 16 elements (two pieces of 8, so
// that it holds both halves of its pairs) of `per` rows of one token; a block
// computes the sines of its tokens' angles once, for all their heads (every
// thread its own eight: 1.1 times as long for 12291 tokens of 32 + 2 x 8 heads of 128
// from fp32, 1064 rows of 48 heads of 64 13.0 us instead of 9.0). Bound by the
// bytes: 12291 tokens 76 us, 5.9 TB/s, of 6.8 for a copy. Rows one at a time: four of
// them in registers took 151 of these and 1.4 times as long, for fewer blocks fit.
//
// Angles: p * inv_freq / 2 pi in turns, modulo one turn, in 64-bit fixed point
// (a phase accumulator): the product with the integer p wraps by itself. An
// fp32 frequency is m 2^e, and 2^64 / 2 pi a constant of 64 bits, so the phase of
// position 2^31 is off by inv_freq 2^-33 turns at most, where fp32 would leave
// nothing of the angle. FP64, of which this GPU has little, is not needed.
struct RopeArgs {
  KvView kv;
  const void *q, *k, *v;  // q, v may be null
  uint16_t *q_out;
  long long q_stride, k_stride, v_stride, qo_stride;
  const int32_t *kv_len, *cu_q;
  int32_t n_seq, n_tok, n_new, nq, n_kv, rows;  // rows of a token: nq queries, n_kv keys, n_kv (or no) values
  int32_t D, ish;                               // log2 of the 16-element items of a row
  int32_t rot, off, interleaved;
  int32_t per, slices;                          // rows of a thread, threads of a token's item
  const float *inv_freq;
  float scale;
  uint32_t *err;
};

// inv_freq / 2 pi in turns, modulo 1, times 2^64 (f finite).
__device__ __forceinline__ unsigned long long turns_of(float f) {
  const uint32_t u = __float_as_uint(f), ex = u >> 23 & 255;
  const unsigned long long m = ex ? (u & 0x7FFFFF) | 0x800000 : u & 0x7FFFFF;
  // 2^66 / 2 pi = 2^64 * 2 / pi, so inv_freq / 2 pi = m * C * 2^(e - 2), e = ex - 150
  constexpr unsigned long long C = 0xA2F9836E4E441529ull;
  const unsigned long long lo = m * C, hi = __umul64hi(m, C);
  const int s = 152 - (int)max(ex, 1u);
  const unsigned long long t = s >= 128 ? 0 : s >= 64 ? hi >> (s - 64) : s > 0 ? hi << (64 - s) | lo >> s : s > -64 ? lo << -s : 0;
  return u >> 31 ? 0ull - t : t;
}

// Cosine and sine of position p at frequency f.
__device__ __forceinline__ void rope_angle(float f, int p, float scale, float &c, float &s) {
  const unsigned long long phase = turns_of(f) * (unsigned long long)(long long)p;
  // the nearest quarter turn, and what is left of at most an eighth
  const int q = (int)((phase + (1ull << 61)) >> 62);
  const int r = (int)((long long)(phase - ((unsigned long long)q << 62)) >> 32);
  float c0, s0;
  sincospif((float)r * 0x1p-31f, &s0, &c0);
  if (!isfinite(f)) c0 = s0 = __int_as_float(0x7FC00000);
  c0 *= scale, s0 *= scale;
  c = q & 1 ? s0 : c0, s = q & 1 ? c0 : s0;
  if (q == 1 || q == 2) c = -c;
  if (q & 2) s = -s;
}

// Angles that a block's 128 threads need at most: its tokens (128 / (D / 16) and
// two begun ones) times rot / 2.
constexpr int AR_ANGLES = 1024 + 512;

template <int DT, bool F32>
__global__ void __launch_bounds__(128) k_append_rope(const RopeArgs a) {
  __shared__ int s_cu[AP_SEQS + 1];
  __shared__ __align__(16) float s_cos[AR_ANGLES], s_sin[AR_ANGLES];
  pdl_launch_dependents();
  pdl_wait();
  const long long idx = (long long)blockIdx.x * 128 + threadIdx.x, rest = idx >> a.ish;
  const int i = (int)(idx & ((1 << a.ish) - 1));
  const long long tt = rest / a.slices;
  const int sl = (int)(rest - tt * a.slices), t = (int)min(tt, (long long)a.n_tok);
  const int r1 = t < a.n_tok ? min(a.rows, (sl + 1) * a.per) : 0;
  // the two pieces: of the turned part first (item i < rot / 16), then what passes
  const bool turns = i < a.rot >> 4;
  int ea, eb;
  if (turns) {
    ea = a.off + (a.interleaved ? 16 * i : 8 * i), eb = ea + (a.interleaved ? 8 : a.rot >> 1);
  } else {
    ea = 16 * i - a.rot, eb = ea + 8;
    if (ea >= a.off) ea += a.rot;
    if (eb >= a.off) eb += a.rot;
  }
  int angle0 = 0;
  constexpr int W = F32 ? 2 : 1;  // 16-byte words of a piece
  uint4 x[2 * W];
  auto load = [&](int r) {
    if (r >= r1) return;
    const char *p;
    if (r < a.nq) p = (const char *)a.q + ((long long)t * a.q_stride + (long long)r * a.D) * (F32 ? 4 : 2);
    else if (r < a.nq + a.n_kv) p = (const char *)a.k + ((long long)t * a.k_stride + (long long)(r - a.nq) * a.D) * (F32 ? 4 : 2);
    else p = (const char *)a.v + ((long long)t * a.v_stride + (long long)(r - a.nq - a.n_kv) * a.D) * (F32 ? 4 : 2);
#pragma unroll
    for (int w = 0; w < W; w++) {
      x[w] = reinterpret_cast<const uint4 *>(p + ea * (F32 ? 4 : 2))[w];
      x[W + w] = reinterpret_cast<const uint4 *>(p + eb * (F32 ? 4 : 2))[w];
    }
  };
  load(sl * a.per);
  const int *cu = append_bounds(a.cu_q, a.n_seq, a.n_tok, s_cu, a.err);
  int b, page = 0, row = 0;
  long long pos;
  {
    // angles by token and frequency
    const int half = a.rot >> 1, t0 = (int)min(((long long)blockIdx.x * 128 >> a.ish) / a.slices, (long long)a.n_tok);
    const int t1 = (int)min((((long long)blockIdx.x * 128 + 127) >> a.ish) / a.slices + 1, (long long)a.n_tok);
    for (int e = threadIdx.x; e < (t1 - t0) * half; e += 128) {
      const int k = e / half;
      if (append_seq(a.kv_len, cu, a.n_seq, a.n_new, t0 + k, b, pos)) rope_angle(a.inv_freq[e - k * half], (int)pos, a.scale, s_cos[e], s_sin[e]);
    }
    __syncthreads();
    if (sl * a.per >= r1 || !append_seq(a.kv_len, cu, a.n_seq, a.n_new, t, b, pos)) return;
    if (turns) angle0 = (t - t0) * half + 8 * i;
  }
  bool store = true;  // the cache has a place for the token
  if (r1 > a.nq) {
    store = append_page(a.kv, b, pos, a.err, page);
    if (store) row = (int)pos - page_index(a.kv, (int)pos) * a.kv.page_size;
  }
  float cs[8], sn[8];
  if (turns) {
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      *reinterpret_cast<float4 *>(cs + e) = *reinterpret_cast<const float4 *>(s_cos + angle0 + e);
      *reinterpret_cast<float4 *>(sn + e) = *reinterpret_cast<const float4 *>(s_sin + angle0 + e);
    }
  }
  for (int r = sl * a.per; r < r1; r++) {
    if (r != sl * a.per) load(r);
    const bool is_q = r < a.nq, is_v = r >= a.nq + a.n_kv;
    uint16_t *dst;
    if (is_q) {
      dst = a.q_out + (long long)t * a.qo_stride + (long long)r * a.D;
    } else {
      if (!store) continue;
      dst = is_v ? const_cast<uint16_t *>(a.kv.v) + (long long)page * a.kv.v_page + (long long)row * a.kv.v_row + (long long)(r - a.nq - a.n_kv) * a.kv.v_head
                 : const_cast<uint16_t *>(a.kv.k) + (long long)page * a.kv.k_page + (long long)row * a.kv.k_row + (long long)(r - a.nq) * a.kv.k_head;
    }
    if (!F32 && (is_v || !turns)) {  // bits are copied
      *reinterpret_cast<uint4 *>(dst + ea) = x[0];
      *reinterpret_cast<uint4 *>(dst + eb) = x[W];
      continue;
    }
    float v[16];
    const uint32_t *u = reinterpret_cast<const uint32_t *>(x);
    if (F32) {
#pragma unroll
      for (int e = 0; e < 16; e++) v[e] = __uint_as_float(u[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const float2 y = Half16<DT>::up(u[e]);
        v[2 * e] = y.x, v[2 * e + 1] = y.y;
      }
    }
    if (turns && !is_v) {
#pragma unroll
      for (int e = 0; e < 8; e++) {
        if (a.interleaved) {
          const float p = v[2 * e], q = v[2 * e + 1];
          v[2 * e] = fmaf(p, cs[e], -(q * sn[e])), v[2 * e + 1] = fmaf(q, cs[e], p * sn[e]);
        } else {
          const float p = v[e], q = v[8 + e];
          v[e] = fmaf(p, cs[e], -(q * sn[e])), v[8 + e] = fmaf(q, cs[e], p * sn[e]);
        }
      }
    }
    *reinterpret_cast<uint4 *>(dst + ea) = make_uint4(Half16<DT>::down(v[0], v[1]), Half16<DT>::down(v[2], v[3]),
                                                      Half16<DT>::down(v[4], v[5]), Half16<DT>::down(v[6], v[7]));
    *reinterpret_cast<uint4 *>(dst + eb) = make_uint4(Half16<DT>::down(v[8], v[9]), Half16<DT>::down(v[10], v[11]),
                                                      Half16<DT>::down(v[12], v[13]), Half16<DT>::down(v[14], v[15]));
  }
}

}  // namespace ds4

namespace {

using namespace ds4;

bool at_dev_ptr(const void *p) {
  if (!p) return false;
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged;
}

ds4moe_status at_status(cudaError_t e) {
  if (e == cudaSuccess) return DS4MOE_OK;
  cudaGetLastError();
  return e == cudaErrorMemoryAllocation ? DS4MOE_ERR_OOM : DS4MOE_ERR_CUDA;
}

bool al16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// Strides the kernels take: multiples of 16 bytes, below 2^39 elements.
bool stride_ok(long long s, long long least) { return s >= least && s % 8 == 0 && s < (1ll << 39); }

// The cache as the kernels see it; false when the description is not one
// they can read.
bool view_of(const ds4moe_attn *h, const ds4moe_kv_cache *c, KvView &v) {
  const int D = h->d.head_dim, H = h->d.n_kv_heads;
  if (!c || c->n_pages < 1 || c->n_pages > INT32_MAX - 1 || c->page_size < 16 || c->page_size > 65536 ||
      c->page_size % 16)
    return false;
  if (c->max_pages < 1 || c->table_stride < c->max_pages || c->table_stride >= (1ll << 39) ||
      (long long)c->max_pages * c->page_size > INT32_MAX - 1024)
    return false;
  v.k = (const uint16_t *)c->k, v.v = (const uint16_t *)c->v;
  // the stride over a single head is never used
  v.k_page = c->k_page_stride, v.k_row = c->k_row_stride, v.k_head = H == 1 ? D : c->k_head_stride;
  v.v_page = c->v_page_stride, v.v_row = c->v_row_stride, v.v_head = H == 1 ? D : c->v_head_stride;
  if (c->n_pages == 1) v.k_page = v.v_page = (long long)c->page_size * H * D;
  for (long long s : {v.k_page, v.k_row, v.k_head, v.v_page, v.v_row, v.v_head})
    if (!stride_ok(s, D)) return false;
  v.table = c->block_table, v.table_stride = c->table_stride;
  int l = 0;
  while ((1 << l) < c->page_size) l++;
  v.div_sh = 31 + l, v.div_mul = (uint32_t)(((1ull << (31 + l)) + c->page_size - 1) / c->page_size);
  v.page_size = c->page_size, v.width = c->max_pages, v.n_pages = (int32_t)c->n_pages;
  return at_dev_ptr(c->k) && at_dev_ptr(c->v) && al16(c->k) && al16(c->v) && at_dev_ptr(c->block_table);
}

const void *append_fn(bool bf, bool f32, bool two) {
  constexpr int B = DS4MOE_DT_BF16, F = DS4MOE_DT_F16;
  if (two)
    return !f32 ? (const void *)k_kv_append<B, false, 2> : bf ? (const void *)k_kv_append<B, true, 2> : (const void *)k_kv_append<F, true, 2>;
  return !f32 ? (const void *)k_kv_append<B, false, 1> : bf ? (const void *)k_kv_append<B, true, 1> : (const void *)k_kv_append<F, true, 1>;
}

const void *rope_fn(bool bf, bool f32) {
  constexpr int B = DS4MOE_DT_BF16, F = DS4MOE_DT_F16;
  return bf ? f32 ? (const void *)k_append_rope<B, true> : (const void *)k_append_rope<B, false>
            : f32 ? (const void *)k_append_rope<F, true> : (const void *)k_append_rope<F, false>;
}

ds4moe_status attn_call(ds4moe_attn *h, const ds4moe_kv_cache *cache, const void *q, int64_t q_stride,
                        const int32_t *cu_q, bool ragged, const int32_t *kv_len, int32_t n_seq, int32_t n_tok,
                        int32_t n_new, void *out, int64_t out_stride, void *stream, const int32_t *shared_len = nullptr,
                        const int32_t *group_start = nullptr, int32_t n_groups = 0) {
  const ds4moe_attn_desc &d = h->d;
  AttnArgs a = {};
  if (!view_of(h, cache, a.kv)) return DS4MOE_ERR_INVALID_ARG;
  const long long row = (long long)d.n_heads * d.head_dim;
  if (n_tok == 1) q_stride = out_stride = row;
  if (!stride_ok(q_stride, row) || !stride_ok(out_stride, row) || !al16(q) || !al16(out)) return DS4MOE_ERR_INVALID_ARG;
  if (!at_dev_ptr(q) || !at_dev_ptr(out) || !at_dev_ptr(kv_len) || (ragged && !at_dev_ptr(cu_q)))
    return DS4MOE_ERR_INVALID_ARG;
  a.q = (const uint16_t *)q, a.out = (uint16_t *)out, a.q_stride = q_stride, a.out_stride = out_stride;
  a.kv_len = kv_len, a.cu_q = ragged ? cu_q : nullptr;
  a.n_seq = n_seq, a.n_tok = n_tok, a.n_new = n_new;
  a.n_heads = d.n_heads, a.n_kv = d.n_kv_heads, a.group = d.n_heads / d.n_kv_heads;
  a.window = d.window, a.n_sink = d.window ? d.n_sink : 0;
  a.scale_log2 = d.scale * 1.44269504088896340736f;  // log2(e)
  a.err = h->err;
  const bool rows16 = !ragged && n_new * a.group <= AD_MAX_ROWS && d.head_dim <= 128;
  if (shared_len) {
    if (!at_dev_ptr(shared_len) || (group_start && !at_dev_ptr(group_start))) return DS4MOE_ERR_INVALID_ARG;
    // With a window a row sees few of the shared positions, or none; and where
    // even a table full of them would gain nothing: the plain call. (In a wider
    // table the device decides, and launches that find nothing to do, and the
    // own parts' kernels over whole histories, cost 8 to 15 us: 8 sequences of 1700
    // 16 and 28, 64 of 5000 196 and 211.)
    const ShareCost cost = h->share_always ? ShareCost{1.0f, 0.0f, 0.0f, 0.0f} : share_cost(d, n_seq, n_new);
    if (d.window == 0 && cost.gain(a.kv.width * a.kv.page_size, n_seq) > cost.least) {
      SharedArgs sa = {};
      static_cast<AttnArgs &>(sa) = a;
      sa.cost = cost, sa.shared_len = shared_len, sa.group_start = group_start, sa.n_groups = n_groups, sa.batch = n_seq;
      sa.pre = h->shared.pre, sa.pre_log = h->shared.pre_log;
      int launches = 0;
      cudaError_t e = launch_attn_prefix(sa, d.head_dim, d.dtype, h->tile, h->shared, h->n_sm, &launches, (cudaStream_t)stream);
      if (e == cudaSuccess && rows16) {
        e = launch_attn_decode(sa, d.head_dim, d.dtype, h->part, h->ticket, h->n_sm, (cudaStream_t)stream);
        launches++;
      } else if (e == cudaSuccess) {
        e = launch_attn_own(sa, d.head_dim, d.dtype, h->tile, h->n_sm, &launches, (cudaStream_t)stream);
      }
      h->launches += launches;
      return at_status(e);
    }
  }
  // Few rows of a short head: the streaming kernel (a unit's 16-row product
  // there costs what a quarter of a 128-row tile does here, and needs no
  // tensor memory, descriptors or second launch). All else: tiles of 128 rows.
  // Both at dimension 128, one key-value head, streaming against tiles, us: 4
  // rows, 1 sequence of 8192 14 and 25, 24 of them 35 and 39; 16 rows 18 and 25,
  // 39 and 39. 20 rows (two products of 16 in the streaming kernel): tiles, 25 and 39.
  if (rows16) {
    const cudaError_t e = launch_attn_decode(a, d.head_dim, d.dtype, h->part, h->ticket, h->n_sm, (cudaStream_t)stream);
    h->launches++;
    return at_status(e);
  }
  int launches = 0;
  const cudaError_t e = launch_attn_tile(a, d.head_dim, d.dtype, h->tile, h->n_sm, &launches, (cudaStream_t)stream);
  h->launches += launches;
  return at_status(e);
}

}  // namespace

extern "C" {

ds4moe_status ds4moe_attn_create(const ds4moe_attn_desc *desc, ds4moe_attn **out) {
  if (!out) return DS4MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (!desc || desc->abi_version != DS4MOE_ABI_VERSION) return DS4MOE_ERR_INVALID_ARG;
  const ds4moe_attn_desc &d = *desc;
  if (d.n_kv_heads < 1 || d.n_kv_heads > 1024 || d.n_heads < d.n_kv_heads || d.n_heads % d.n_kv_heads)
    return DS4MOE_ERR_INVALID_ARG;
  if (d.dtype != DS4MOE_DT_BF16 && d.dtype != DS4MOE_DT_F16) return DS4MOE_ERR_INVALID_ARG;
  if (d.window < 0 || d.n_sink < 0) return DS4MOE_ERR_INVALID_ARG;
  if (!isfinite(d.scale) || d.scale <= 0.0f) return DS4MOE_ERR_INVALID_ARG;
  if (d.max_seqs < 1 || d.max_seqs > 65536 || d.max_tokens < 1 || d.max_tokens > (1 << 20))
    return DS4MOE_ERR_INVALID_ARG;
  if (d.head_dim < 1) return DS4MOE_ERR_INVALID_ARG;
  if ((d.head_dim != 64 && d.head_dim != 128 && d.head_dim != 256 && d.head_dim != 512) ||
      d.n_heads / d.n_kv_heads > 128)
    return DS4MOE_ERR_UNSUPPORTED;
  ds4moe_attn *h = new (std::nothrow) ds4moe_attn;
  if (!h) return DS4MOE_ERR_OOM;
  memset(h, 0, sizeof(*h));
  h->d = d;
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->n_sm, cudaDevAttrMultiProcessorCount, h->device);
  // one allocation: flags, tickets, the ragged plan, the partials
  const size_t groups = attn_tile_groups(d.n_heads / d.n_kv_heads, d.head_dim, d.max_tokens, d.max_seqs);
  const size_t parts = std::max(attn_decode_part_floats(h->n_sm), attn_tile_part_floats(d.head_dim, h->n_sm));
  size_t at = 0;
  auto place = [&](size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) & ~(size_t)255;
    return p;
  };
  const size_t o_err = place(64), o_ticket = place((size_t)2 * h->n_sm * 4), o_marked = place((size_t)h->n_sm * 4);
  const size_t o_split = place((size_t)h->n_sm * 32);
  const size_t o_count = place(4), o_seq = place((size_t)d.max_seqs * 4), o_cu = place(((size_t)d.max_seqs + 1) * 4);
  const size_t o_first = place((groups + 1) * 8);
  const size_t o_info = place(groups * 8), o_part = place(parts * 4);
  if (e == cudaSuccess) e = attn_decode_set_attributes();
  if (e == cudaSuccess) e = attn_tile_set_attributes(d.dtype, d.head_dim);
  if (e == cudaSuccess) e = cudaMalloc((void **)&h->mem, at);
  if (e == cudaSuccess) e = cudaMemsetAsync(h->mem, 0, o_split, 0);
  if (e == cudaSuccess) e = cudaStreamSynchronize(0);
  if (e != cudaSuccess) {
    const ds4moe_status st = at_status(e);
    if (h->mem) cudaFree(h->mem);
    cudaGetLastError();
    delete h;
    return st;
  }
  h->err = (uint32_t *)(h->mem + o_err), h->ticket = (int *)(h->mem + o_ticket), h->part = (float *)(h->mem + o_part);
  h->tile.split = h->mem + o_split, h->tile.marked = (int *)(h->mem + o_marked), h->tile.count = (int *)(h->mem + o_count);
  h->tile.seq_first = (int *)(h->mem + o_seq), h->tile.cu = (int32_t *)(h->mem + o_cu), h->tile.first = (long long *)(h->mem + o_first);
  h->tile.info = h->mem + o_info, h->tile.part = h->part;
  h->tile.pairs = attn_tile_pairs(d.dtype, d.head_dim);
  h->bytes = at;
  *out = h;
  return DS4MOE_OK;
}

void ds4moe_attn_destroy(ds4moe_attn *h) {
  if (!h) return;
  cudaDeviceSynchronize();
  cudaFree(h->mem);
  if (h->shared_mem) cudaFree(h->shared_mem);
  delete h;
}

ds4moe_status ds4moe_attn_reserve_shared(ds4moe_attn *h, int32_t max_tokens) {
  if (!h || max_tokens < 0 || max_tokens > h->d.max_tokens) return DS4MOE_ERR_INVALID_ARG;
  if (max_tokens <= h->shared_tokens) return DS4MOE_OK;
  const size_t rows = (size_t)max_tokens * h->d.n_heads;
  size_t at = 0;
  auto place = [&](size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) & ~(size_t)255;
    return p;
  };
  const size_t o_start = place((size_t)h->d.max_seqs * 4), o_plen = place((size_t)h->d.max_seqs * 4);
  const size_t o_ptab = place((size_t)h->d.max_seqs * 4), o_log = place(rows * 4), o_pre = place(rows * h->d.head_dim * 4);
  uint8_t *mem = nullptr;
  cudaError_t e = attn_shared_set_attributes(h->d.dtype, h->d.head_dim);
  if (e == cudaSuccess) e = cudaMalloc((void **)&mem, at);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();  // calls that use the old one
  if (e != cudaSuccess) {
    if (mem) cudaFree(mem);
    return at_status(e);
  }
  if (h->shared_mem) cudaFree(h->shared_mem);
  h->shared_mem = mem, h->shared_tokens = max_tokens, h->shared_bytes = at;
  h->shared.start = (int32_t *)(mem + o_start), h->shared.plen = (int32_t *)(mem + o_plen), h->shared.ptab = (int32_t *)(mem + o_ptab);
  h->shared.pre = (float *)(mem + o_pre), h->shared.pre_log = (float *)(mem + o_log);
  return DS4MOE_OK;
}

ds4moe_status ds4moe_kv_append(ds4moe_attn *h, const ds4moe_kv_cache *cache, const void *k_new, int64_t k_stride,
                               const void *v_new, int64_t v_stride, int32_t src_dtype, const int32_t *cu_q,
                               const int32_t *kv_len, int32_t n_seq, int32_t n_tok, void *stream) {
  if (!h || n_seq < 0 || n_seq > h->d.max_seqs || n_tok < 0 || n_tok > h->d.max_tokens) return DS4MOE_ERR_INVALID_ARG;
  if (src_dtype != DS4MOE_DT_F32 && src_dtype != h->d.dtype) return DS4MOE_ERR_INVALID_ARG;
  if (n_seq == 0 || n_tok == 0) return DS4MOE_OK;
  if (!cu_q && n_tok % n_seq) return DS4MOE_ERR_INVALID_ARG;
  const int row = h->d.n_kv_heads * h->d.head_dim;
  AppendArgs a = {};
  if (!view_of(h, cache, a.kv)) return DS4MOE_ERR_INVALID_ARG;
  if (n_tok == 1) k_stride = v_stride = row;
  if (!stride_ok(k_stride, row) || !al16(k_new) || !at_dev_ptr(k_new)) return DS4MOE_ERR_INVALID_ARG;
  if (v_new && (!stride_ok(v_stride, row) || !al16(v_new) || !at_dev_ptr(v_new))) return DS4MOE_ERR_INVALID_ARG;
  if (!at_dev_ptr(kv_len) || (cu_q && !at_dev_ptr(cu_q))) return DS4MOE_ERR_INVALID_ARG;
  a.k = k_new, a.v = v_new, a.k_stride = k_stride, a.v_stride = v_stride;
  a.kv_len = kv_len, a.cu_q = cu_q, a.n_seq = n_seq, a.n_tok = n_tok, a.n_new = cu_q ? 0 : n_tok / n_seq;
  a.n_kv = h->d.n_kv_heads, a.D = h->d.head_dim, a.per_tok = row / 8, a.err = h->err;
  // More than one wave of threads: two pieces per thread (12291 tokens of
  // 8 x 128: 27.4 -> 26.6 us), their loads in flight together; else one (64
  // rows of 512: 2.8 us, with two 3.9).
  const long long total = (long long)n_tok * a.per_tok * (v_new ? 2 : 1);
  const bool two = total > (long long)h->n_sm * 2048;
  const bool f32 = src_dtype == DS4MOE_DT_F32;
  // (the cache's own type: bits are copied)
  const void *fn = append_fn(!f32 || h->d.dtype == DS4MOE_DT_BF16, f32, two);
  void *args[] = {&a};
  const int per = two ? 256 : 128;
  cudaError_t e = cudaSuccess;
  if (cu_q && n_seq > AP_SEQS) {
    a.cu_q = h->tile.cu;
    void *clean[] = {(void *)&cu_q, &n_seq, &n_tok, &h->tile.cu, &h->err};
    e = launch_pdl((const void *)k_clean_rows, dim3(1), dim3(1024), 0, (cudaStream_t)stream, clean, true);
    h->launches++;
    if (e != cudaSuccess) return at_status(e);
  }
  e = launch_pdl(fn, dim3((unsigned)(((long long)n_tok * a.per_tok + per - 1) / per), v_new ? 2 : 1),
                                   dim3(128), 0, (cudaStream_t)stream, args, true);
  h->launches++;
  return at_status(e);
}

ds4moe_status ds4moe_kv_append_rope(ds4moe_attn *h, const ds4moe_kv_cache *cache, const ds4moe_rope *rope,
                                    const void *q_new, int64_t q_stride, void *q_out, int64_t q_out_stride,
                                    const void *k_new, int64_t k_stride, const void *v_new, int64_t v_stride,
                                    int32_t src_dtype, const int32_t *cu_q, const int32_t *kv_len, int32_t n_seq,
                                    int32_t n_tok, void *stream) {
  if (!h || n_seq < 0 || n_seq > h->d.max_seqs || n_tok < 0 || n_tok > h->d.max_tokens) return DS4MOE_ERR_INVALID_ARG;
  if (src_dtype != DS4MOE_DT_F32 && src_dtype != h->d.dtype) return DS4MOE_ERR_INVALID_ARG;
  const int D = h->d.head_dim;
  if (!rope || rope->rot_dim < 16 || rope->rot_dim % 16 || rope->offset < 0 || rope->offset % 8 || rope->rot_dim > D ||
      rope->offset > D - rope->rot_dim || (rope->interleaved != 0 && rope->interleaved != 1) || !isfinite(rope->scale))
    return DS4MOE_ERR_INVALID_ARG;
  if (!q_new != !q_out) return DS4MOE_ERR_INVALID_ARG;
  if (n_seq == 0 || n_tok == 0) return DS4MOE_OK;
  if (!cu_q && n_tok % n_seq) return DS4MOE_ERR_INVALID_ARG;
  const long long row = (long long)h->d.n_kv_heads * D, q_row = (long long)h->d.n_heads * D;
  const bool f32 = src_dtype == DS4MOE_DT_F32;
  RopeArgs a = {};
  if (!view_of(h, cache, a.kv)) return DS4MOE_ERR_INVALID_ARG;
  if (n_tok == 1) k_stride = v_stride = row, q_stride = q_out_stride = q_row;
  if (!stride_ok(k_stride, row) || !al16(k_new) || !at_dev_ptr(k_new)) return DS4MOE_ERR_INVALID_ARG;
  if (v_new && (!stride_ok(v_stride, row) || !al16(v_new) || !at_dev_ptr(v_new))) return DS4MOE_ERR_INVALID_ARG;
  if (q_new) {
    if (!stride_ok(q_stride, q_row) || !al16(q_new) || !at_dev_ptr(q_new)) return DS4MOE_ERR_INVALID_ARG;
    if (!stride_ok(q_out_stride, q_row) || !al16(q_out) || !at_dev_ptr(q_out)) return DS4MOE_ERR_INVALID_ARG;
    // in place: every element is read and written by the same thread
    const bool same = q_new == q_out && !f32 && q_stride == q_out_stride;
    const int src = f32 ? 4 : 2;
    auto over = [&](const void *p, long long stride, long long len) {
      return rows_overlap(q_out, q_row * 2, q_out_stride * 2, p, len * src, stride * src, n_tok);
    };
    if ((!same && over(q_new, q_stride, q_row)) || over(k_new, k_stride, row) || (v_new && over(v_new, v_stride, row)))
      return DS4MOE_ERR_INVALID_ARG;
  }
  if (!at_dev_ptr(kv_len) || (cu_q && !at_dev_ptr(cu_q)) || !at_dev_ptr(rope->inv_freq) || !al16(rope->inv_freq))
    return DS4MOE_ERR_INVALID_ARG;
  a.q = q_new, a.k = k_new, a.v = v_new, a.q_out = (uint16_t *)q_out;
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride, a.qo_stride = q_out_stride;
  a.kv_len = kv_len, a.cu_q = cu_q, a.n_seq = n_seq, a.n_tok = n_tok, a.n_new = cu_q ? 0 : n_tok / n_seq;
  a.nq = q_new ? h->d.n_heads : 0, a.n_kv = h->d.n_kv_heads, a.rows = a.nq + a.n_kv * (v_new ? 2 : 1);
  a.D = D;
  while (16 << a.ish < D) a.ish++;
  a.rot = rope->rot_dim, a.off = rope->offset, a.interleaved = rope->interleaved;
  a.inv_freq = rope->inv_freq, a.scale = rope->scale, a.err = h->err;
  // More than one wave of threads: six rows of a token per thread (12291 tokens of
  // 48 rows, in one run of all: 74 us; one 81, two 81, four 75, sixteen 76); else one.
  const long long items = (long long)n_tok * a.rows << a.ish;
  a.per = items > (long long)h->n_sm * 2048 ? 6 : 1;
  a.slices = (a.rows + a.per - 1) / a.per;
  cudaError_t e = cudaSuccess;
  if (cu_q && n_seq > AP_SEQS) {
    a.cu_q = h->tile.cu;
    void *clean[] = {(void *)&cu_q, &n_seq, &n_tok, &h->tile.cu, &h->err};
    e = launch_pdl((const void *)k_clean_rows, dim3(1), dim3(1024), 0, (cudaStream_t)stream, clean, true);
    h->launches++;
    if (e != cudaSuccess) return at_status(e);
  }
  void *args[] = {&a};
  const long long threads = (long long)n_tok * a.slices << a.ish;
  e = launch_pdl(rope_fn(h->d.dtype == DS4MOE_DT_BF16, f32), dim3((unsigned)((threads + 127) / 128)), dim3(128), 0,
                 (cudaStream_t)stream, args, true);
  h->launches++;
  return at_status(e);
}

ds4moe_status ds4moe_attn_decode(ds4moe_attn *h, const ds4moe_kv_cache *cache, const void *q, int64_t q_stride,
                                 const int32_t *kv_len, int32_t n_seq, int32_t n_new, void *out, int64_t out_stride,
                                 void *stream) {
  if (!h || n_seq < 0 || n_seq > h->d.max_seqs || n_new < 1 || n_new > DS4MOE_ATTN_MAX_NEW ||
      (long long)n_seq * n_new > h->d.max_tokens)
    return DS4MOE_ERR_INVALID_ARG;
  if (n_seq == 0) return DS4MOE_OK;
  return attn_call(h, cache, q, q_stride, nullptr, false, kv_len, n_seq, n_seq * n_new, n_new, out, out_stride, stream);
}

ds4moe_status ds4moe_attn_debug_share(ds4moe_attn *h, int32_t always) {
  if (!h || (always != 0 && always != 1)) return DS4MOE_ERR_INVALID_ARG;
  h->share_always = always;
  return DS4MOE_OK;
}

ds4moe_status ds4moe_attn_decode_shared(ds4moe_attn *h, const ds4moe_kv_cache *cache, const void *q, int64_t q_stride,
                                        const int32_t *kv_len, const int32_t *shared_len, const int32_t *group_start,
                                        int32_t n_groups, int32_t n_seq, int32_t n_new, void *out, int64_t out_stride,
                                        void *stream) {
  if (!h || n_seq < 0 || n_seq > h->d.max_seqs || n_new < 1 || n_new > DS4MOE_ATTN_MAX_NEW ||
      (long long)n_seq * n_new > h->d.max_tokens)
    return DS4MOE_ERR_INVALID_ARG;
  if (n_groups < 1 || (n_seq > 0 && n_groups > n_seq) || (!group_start && n_groups != 1)) return DS4MOE_ERR_INVALID_ARG;
  if (n_seq * n_new > h->shared_tokens) return DS4MOE_ERR_INVALID_ARG;
  if (n_seq == 0) return DS4MOE_OK;
  if (!shared_len) return DS4MOE_ERR_INVALID_ARG;
  return attn_call(h, cache, q, q_stride, nullptr, false, kv_len, n_seq, n_seq * n_new, n_new, out, out_stride, stream,
                   shared_len, group_start, n_groups);
}

ds4moe_status ds4moe_attn_prefill(ds4moe_attn *h, const ds4moe_kv_cache *cache, const void *q, int64_t q_stride,
                                  const int32_t *cu_q, const int32_t *kv_len, int32_t n_seq, int32_t n_tok, void *out,
                                  int64_t out_stride, void *stream) {
  if (!h || n_seq < 0 || n_seq > h->d.max_seqs || n_tok < 0 || n_tok > h->d.max_tokens) return DS4MOE_ERR_INVALID_ARG;
  if (n_seq == 0 || n_tok == 0) return DS4MOE_OK;
  return attn_call(h, cache, q, q_stride, cu_q, true, kv_len, n_seq, n_tok, 0, out, out_stride, stream);
}

ds4moe_status ds4moe_attn_get_device_error(ds4moe_attn *h, void *stream, uint32_t *flags_out) {
  if (!h) return DS4MOE_ERR_INVALID_ARG;
  uint32_t f = 0;
  cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaMemcpy(&f, h->err, 4, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(h->err, 0, 4);
  if (e != cudaSuccess) return at_status(e);
  if (flags_out) *flags_out = f;
  return f ? DS4MOE_ERR_DEVICE : DS4MOE_OK;
}

uint64_t ds4moe_attn_device_bytes(const ds4moe_attn *h) { return h ? h->bytes + h->shared_bytes : 0; }
uint64_t ds4moe_attn_launch_count(const ds4moe_attn *h) { return h ? h->launches : 0; }

}  // extern "C"
