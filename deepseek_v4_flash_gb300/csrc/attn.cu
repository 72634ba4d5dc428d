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

ds4moe_status attn_call(ds4moe_attn *h, const ds4moe_kv_cache *cache, const void *q, int64_t q_stride,
                        const int32_t *cu_q, bool ragged, const int32_t *kv_len, int32_t n_seq, int32_t n_tok,
                        int32_t n_new, void *out, int64_t out_stride, void *stream) {
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
  // Few rows of a short head: the streaming kernel (a unit's 16-row product
  // there costs what a quarter of a 128-row tile does here, and needs no
  // tensor memory, descriptors or second launch). All else: tiles of 128 rows.
  // Both at dimension 128, one key-value head, streaming against tiles, us: 4
  // rows, 1 sequence of 8192 14 and 25, 24 of them 35 and 39; 16 rows 18 and 25,
  // 39 and 39. 20 rows (two products of 16 in the streaming kernel): tiles, 25 and 39.
  if (!ragged && n_new * a.group <= AD_MAX_ROWS && d.head_dim <= 128) {
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
  const size_t o_err = place(64), o_ticket = place((size_t)h->n_sm * 4), o_marked = place((size_t)h->n_sm * 4);
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
  delete h;
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

ds4moe_status ds4moe_attn_decode(ds4moe_attn *h, const ds4moe_kv_cache *cache, const void *q, int64_t q_stride,
                                 const int32_t *kv_len, int32_t n_seq, int32_t n_new, void *out, int64_t out_stride,
                                 void *stream) {
  if (!h || n_seq < 0 || n_seq > h->d.max_seqs || n_new < 1 || n_new > DS4MOE_ATTN_MAX_NEW ||
      (long long)n_seq * n_new > h->d.max_tokens)
    return DS4MOE_ERR_INVALID_ARG;
  if (n_seq == 0) return DS4MOE_OK;
  return attn_call(h, cache, q, q_stride, nullptr, false, kv_len, n_seq, n_seq * n_new, n_new, out, out_stride, stream);
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

uint64_t ds4moe_attn_device_bytes(const ds4moe_attn *h) { return h ? h->bytes : 0; }
uint64_t ds4moe_attn_launch_count(const ds4moe_attn *h) { return h ? h->launches : 0; }

}  // extern "C"
