// sample.cu -- what follows the output head: probabilities of a row of logits
// (ds4moe_token_probs) and the verification of drafted tokens against them
// (ds4moe_verify_drafts).
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace ds4 {

constexpr int SP_THREADS = 512;
constexpr int SP_WARPS = SP_THREADS / 32;

// (value, index) of the larger value, the lower index among equals.
__device__ __forceinline__ void arg_max(float &v, int &i, float w, int j) {
  if (w > v || (w == v && j < i)) v = w, i = j;
}

// d / T from 1 / T with one correction step: (x - max) / T reaches -40 and
// more, where the rounding of 1 / T alone would show in the exponential.
__device__ __forceinline__ float over_t(float d, float t, float inv_t) {
  const float z = d * inv_t;
  return isfinite(z) ? fmaf(fmaf(-z, t, d), inv_t, z) : z;
}

// Softmax of one row per block: the maximum, the sum of exp((x - max) / T),
// then the quotients. T = 0: 1 at the lowest index of the maximum, 0
// elsewhere. A row whose maximum is not finite, or that holds a NaN, gives
// what the formula gives (NaN).
__global__ void __launch_bounds__(SP_THREADS) k_token_probs(const float *x, long long xs, int V, float t, float inv_t, float *out,
                                                        long long os) {
  __shared__ float sv[SP_WARPS], ss[SP_WARPS];
  __shared__ int si[SP_WARPS];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  pdl_wait();
  const float *r = x + (long long)blockIdx.x * xs;
  float *o = out + (long long)blockIdx.x * os;
  float m = -INFINITY;
  int at = V;
  bool nan = false;
  for (int i = tid; i < V; i += SP_THREADS) {
    const float v = r[i];
    nan |= v != v;
    arg_max(m, at, v, i);
  }
#pragma unroll
  for (int s = 16; s; s >>= 1)
    arg_max(m, at, __shfl_xor_sync(0xffffffffu, m, s), __shfl_xor_sync(0xffffffffu, at, s));
  if (lane == 0) sv[w] = m, si[w] = at;
  nan = __syncthreads_or(nan);
  for (int i = 0; i < SP_WARPS; i++) arg_max(m, at, sv[i], si[i]);
  if (nan) m = NAN;
  if (inv_t == 0.0f) {
    for (int i = tid; i < V; i += SP_THREADS) o[i] = nan ? NAN : i == at ? 1.0f : 0.0f;
    return;
  }
  float sum = 0.0f;
  for (int i = tid; i < V; i += SP_THREADS) sum += expf(over_t(r[i] - m, t, inv_t));
#pragma unroll
  for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
  if (lane == 0) ss[w] = sum;
  __syncthreads();
  sum = 0.0f;
  for (int i = 0; i < SP_WARPS; i++) sum += ss[i];
  const float inv = 1.0f / sum;
  for (int i = tid; i < V; i += SP_THREADS) o[i] = expf(over_t(r[i] - m, t, inv_t)) * inv;
}

// ---------------------------------------------------------------------------
// Verification. Sums of probabilities decide a whole number, so they are
// exact: a probability is rounded to a multiple of 2^-shift (shift = 62 -
// ceil(log2 V), 45 for a vocabulary of 129280) and summed in 64-bit integers,
// whose sum does not depend on the order and cannot overflow.

struct VerifyArgs {
  const float *target, *draft;       // [n_seq][G + 1][V], [n_seq][G][V] or null
  long long t_pitch, d_pitch;        // elements from row to row
  const int32_t *tok, *n_draft;      // [n_seq][G], [n_seq] or null
  const float *u_accept, *u_sample;  // [n_seq][G], [n_seq]
  int32_t G, V, shift;
  int32_t *n_accepted, *tokens;      // [n_seq], [n_seq][G + 1]
  uint32_t *err;
};

// A probability in units of 2^-shift, clamped to [0, 1]; NaN counts as 0.
__device__ __forceinline__ long long fixed_prob(float p, int shift) {
  if (!(p > 0.0f)) return 0;
  p = fminf(p, 1.0f);
  const int b = __float_as_int(p), e = b >> 23;
  if (e == 0) return 0;  // below 2^-126
  const unsigned long long mant = (b & 0x7FFFFF) | 0x800000;
  const int s = e - 150 + shift;  // value = mant * 2^s units
  if (s >= 0) return (long long)(mant << s);
  if (s < -24) return 0;
  return (long long)((mant + (1ull << (-s - 1))) >> -s);
}

// u in [0, 1) in units of 2^-64 (bits below are dropped: they lie under one
// unit of any sum).
__device__ __forceinline__ unsigned long long fixed_u(float u) {
  if (!(u > 0.0f)) return 0;
  u = fminf(u, 0x1.fffffep-1f);
  const int b = __float_as_int(u), s = (b >> 23) - 150 + 64;
  const unsigned long long mant = (b & 0x7FFFFF) | 0x800000;
  return s >= 0 ? mant << s : s > -24 ? mant >> -s : 0;
}

// What the last token is drawn from: row p less row q (dropped below 0).
// dtok >= 0: q is 1 at dtok and 0 elsewhere.
__device__ __forceinline__ long long mass_at(const float *p, const float *q, int dtok, int i, int shift) {
  long long r = fixed_prob(p[i], shift);
  if (q) r = max(0ll, r - fixed_prob(q[i], shift));
  if (i == dtok) r = 0;
  return r;
}

__device__ __forceinline__ long long warp_sum64(long long v) {
#pragma unroll
  for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

__global__ void __launch_bounds__(SP_THREADS) k_verify_drafts(const VerifyArgs a) {
  __shared__ long long part[SP_WARPS];
  __shared__ int s_n;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, b = blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  int cnt = a.G;
  if (a.n_draft) {
    cnt = min(max(a.n_draft[b], 0), a.G);
    if (cnt != a.n_draft[b] && tid == 0) raise_flag(a.err, DS4MOE_DEVERR_LENGTH);
  }
  if (w == 0) {
    // draft i is accepted when u * q < p: the product of two 24-bit
    // significands is exact in 64 bits
    int n = cnt;
    for (int i = lane; i < cnt; i += 32) {
      const int t = a.tok[(long long)b * a.G + i];
      bool ok = false;
      if (t >= 0 && t < a.V) {
        const double p = a.target[((long long)b * (a.G + 1) + i) * a.t_pitch + t];
        const double q = a.draft ? a.draft[((long long)b * a.G + i) * a.d_pitch + t] : 1.0;
        ok = (double)a.u_accept[(long long)b * a.G + i] * q < p;
      } else {
        raise_flag(a.err, DS4MOE_DEVERR_TOKEN_ID);
      }
      if (!ok) n = min(n, i);
    }
    n = __reduce_min_sync(0xffffffffu, n);
    if (lane == 0) s_n = n;
  }
  __syncthreads();
  const int n = s_n;
  const float *p = a.target + ((long long)b * (a.G + 1) + n) * a.t_pitch;
  const float *q = n < cnt && a.draft ? a.draft + ((long long)b * a.G + n) * a.d_pitch : nullptr;
  int dtok = n < cnt && !a.draft ? a.tok[(long long)b * a.G + n] : -1;
  const int per = (a.V + SP_WARPS - 1) / SP_WARPS, i0 = w * per, i1 = min(a.V, i0 + per);
  long long total = 0;
  for (int round = 0; round < 2; round++) {
    long long s = 0;
    for (int i = i0 + lane; i < i1; i += 32) s += mass_at(p, q, dtok, i, a.shift);
    s = warp_sum64(s);
    __syncthreads();
    if (lane == 0) part[w] = s;
    __syncthreads();
    total = 0;
    for (int i = 0; i < SP_WARPS; i++) total += part[i];
    if (total > 0 || (!q && dtok < 0)) break;
    q = nullptr, dtok = -1;  // nothing is left: draw from p itself
  }
  const long long thr = (long long)__umul64hi((unsigned long long)total, fixed_u(a.u_sample[b]));
  if (total == 0) {
    if (tid == 0) a.tokens[(long long)b * (a.G + 1) + n] = -1;
  } else {
    // the warp whose run holds the first cumulative sum above thr
    long long before = 0;
    for (int i = 0; i < w; i++) before += part[i];
    if (before <= thr && thr < before + part[w]) {
      for (int c = i0; c < i1; c += 32) {
        const int i = c + lane;
        long long s = i < i1 ? mass_at(p, q, dtok, i, a.shift) : 0;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
          const long long o = __shfl_up_sync(0xffffffffu, s, k);
          if (lane >= k) s += o;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + s > thr);
        if (hit) {
          if (lane == 0) a.tokens[(long long)b * (a.G + 1) + n] = c + __ffs(hit) - 1;
          break;
        }
        before += __shfl_sync(0xffffffffu, s, 31);
      }
    }
  }
  if (tid <= a.G && tid != n)
    a.tokens[(long long)b * (a.G + 1) + tid] = tid < n ? a.tok[(long long)b * a.G + tid] : -1;
  if (tid == 0) a.n_accepted[b] = n;
}

}  // namespace ds4

namespace {

bool sp_dev_ptr(const void *p) {
  if (!p) return false;
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged;
}

ds4moe_status sp_status(cudaError_t e) {
  if (e == cudaSuccess) return DS4MOE_OK;
  cudaGetLastError();
  return DS4MOE_ERR_CUDA;
}

}  // namespace

extern "C" {

using namespace ds4;

ds4moe_status ds4moe_token_probs(const float *logits, int64_t logits_stride, int32_t n_rows, int32_t vocab,
                                 float temperature, float *probs, int64_t probs_stride, void *stream) {
  if (n_rows < 0 || n_rows > (1 << 24) || vocab < 1 || vocab > (1 << 24)) return DS4MOE_ERR_INVALID_ARG;
  if (!isfinite(temperature) || temperature < 0.0f || (temperature > 0.0f && !isfinite(1.0f / temperature)))
    return DS4MOE_ERR_INVALID_ARG;
  if (n_rows == 0) return DS4MOE_OK;
  if (n_rows > 1 && (logits_stride < vocab || probs_stride < vocab)) return DS4MOE_ERR_INVALID_ARG;
  if (!sp_dev_ptr(logits) || !sp_dev_ptr(probs)) return DS4MOE_ERR_INVALID_ARG;
  float inv_t = temperature > 0.0f ? 1.0f / temperature : 0.0f;
  long long xs = logits_stride, os = probs_stride;
  void *args[] = {(void *)&logits, &xs, &vocab, &temperature, &inv_t, (void *)&probs, &os};
  return sp_status(launch_pdl((const void *)k_token_probs, dim3(n_rows), dim3(SP_THREADS), 0, (cudaStream_t)stream, args,
                              true));
}

ds4moe_status ds4moe_verify_drafts(const float *target, int64_t target_stride, const float *draft, int64_t draft_stride,
                                   const int32_t *draft_tokens, const int32_t *n_draft, const float *u_accept,
                                   const float *u_sample, int32_t n_seq, int32_t max_draft, int32_t vocab,
                                   int32_t *n_accepted, int32_t *tokens_out, uint32_t *err_flags, void *stream) {
  if (n_seq < 0 || n_seq > (1 << 20) || max_draft < 0 || max_draft > DS4MOE_MAX_DRAFT || vocab < 1 || vocab > (1 << 24))
    return DS4MOE_ERR_INVALID_ARG;
  if (n_seq == 0) return DS4MOE_OK;
  if (target_stride < vocab || (draft && draft_stride < vocab)) return DS4MOE_ERR_INVALID_ARG;
  if (!sp_dev_ptr(target) || !sp_dev_ptr(u_sample) || !sp_dev_ptr(n_accepted) || !sp_dev_ptr(tokens_out))
    return DS4MOE_ERR_INVALID_ARG;
  if (max_draft > 0 && (!sp_dev_ptr(draft_tokens) || !sp_dev_ptr(u_accept) || (draft && !sp_dev_ptr(draft))))
    return DS4MOE_ERR_INVALID_ARG;
  if ((n_draft && !sp_dev_ptr(n_draft)) || (err_flags && !sp_dev_ptr(err_flags))) return DS4MOE_ERR_INVALID_ARG;
  VerifyArgs a = {};
  a.target = target, a.draft = max_draft > 0 ? draft : nullptr, a.t_pitch = target_stride, a.d_pitch = draft_stride;
  a.tok = draft_tokens, a.n_draft = n_draft, a.u_accept = u_accept, a.u_sample = u_sample;
  a.G = max_draft, a.V = vocab, a.n_accepted = n_accepted, a.tokens = tokens_out, a.err = err_flags;
  int lg = 0;
  while ((1 << lg) < vocab) lg++;
  a.shift = 62 - lg;
  void *args[] = {&a};
  return sp_status(launch_pdl((const void *)k_verify_drafts, dim3(n_seq), dim3(SP_THREADS), 0, (cudaStream_t)stream, args,
                              true));
}

}  // extern "C"
