// sample.cu -- what follows the output head: probabilities of a row of logits
// (ds4moe_token_probs) and the verification of drafted tokens against them
// (ds4moe_verify_drafts).
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace ds4 {

constexpr int SP_THREADS = 512;
constexpr int SP_WARPS = SP_THREADS / 32;

// Both kernels give a row to a cluster of 1, 2, 4 or 8 blocks: enough blocks
// that a block's part is about 4096 entries, so that a single row is read by
// eight SMs (a call for one sequence is all latency) and a whole batch keeps
// every SM's loads in flight. Parts are multiples of 4 entries.
constexpr int SP_PART = 4096;
int cluster_of(int V) {
  int c = 1;
  while (c < 8 && (long long)c * SP_PART < V) c *= 2;
  return c;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word of another block's shared memory.
__device__ __forceinline__ uint32_t ld_peer(const void *p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// (value, index) of the larger value, the lower index among equals.
__device__ __forceinline__ void arg_max(float &v, int &i, float w, int j) {
  if (w > v || (w == v && j < i)) v = w, i = j;
}

// exp(d / T) for d <= 0 as 2^(d c), c = log2(e) / T given as hi + lo: the
// product's rounding and lo come back as a first-order factor, for d c reaches
// -60 and more, where they would show in a 32-bit exponential. Eight
// instructions (a division and expf took 25, and the kernel was bound by
// them). d is kept above dmin = -200 / c, where the result is 0, so that
// -infinity gives 0 and not infinity less infinity; a NaN stays one.
struct ExpScale {
  float hi, lo, dmin, t;
};
__device__ __forceinline__ float exp_over_t(float d, const ExpScale &c) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(d) : "f"(c.dmin));
  const float x = __fmul_rn(d, c.hi), err = __fmaf_rn(d, c.lo, __fmaf_rn(d, c.hi, -x));
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
  return __fmaf_rn(e, err * 0.693147180559945f, e);
}

// Four entries of a row (those below end; `fill` elsewhere): i .. i + 3 in one
// access where rows are 16-byte aligned, else i, i + S, i + 2 S, i + 3 S, so
// that neighbouring threads take neighbouring entries. `inner`: the whole
// block's, or warp's, entries are known to lie below end.
template <bool VEC, int S>
__device__ __forceinline__ float4 row4(const float *r, int i, int end, float fill, bool inner = false) {
  if (VEC && (inner || i + 3 < end)) return *reinterpret_cast<const float4 *>(r + i);
  if (inner) return make_float4(r[i], r[i + S], r[i + 2 * S], r[i + 3 * S]);
  return make_float4(i < end ? r[i] : fill, i + S < end ? r[i + S] : fill, i + 2 * S < end ? r[i + 2 * S] : fill,
                     i + 3 * S < end ? r[i + 3 * S] : fill);
}
template <bool VEC, int S>
__device__ __forceinline__ void put4(float *o, int i, int end, float4 v, bool inner = false) {
  if (VEC && (inner || i + 3 < end)) {
    *reinterpret_cast<float4 *>(o + i) = v;
    return;
  }
  if (inner || i < end) o[i] = v.x;
  if (inner || i + S < end) o[i + S] = v.y;
  if (inner || i + 2 * S < end) o[i + 2 * S] = v.z;
  if (inner || i + 3 * S < end) o[i + 3 * S] = v.w;
}

// Softmax of one row per cluster, bound by the row's bytes (read once, written
// once): a block keeps up to SP_KEEP x 2048 entries of its part in registers
// (the rest of a longer part is read again, from L2), takes the exponentials
// relative to its own maximum, and one exchange of (maximum, sum) between the
// blocks gives the factor that turns them into probabilities.
// T = 0: 1 at the lowest index of the maximum, 0 elsewhere.
// 320 rows of 129280: 68 us, 4.9 TB/s read and written (0.73 of the copy rate):
// the registers that hold a part allow two blocks per SM, whose load, compute
// and store phases overlap only with each other's. Rows that are not 16-byte
// aligned take four accesses for one: 320 of 129281 75 us. One row's latency: 5 us.
constexpr int SP_KEEP = 8, PR_THREADS = 512, PR_WARPS = PR_THREADS / 32;
template <bool VEC>
__global__ void __launch_bounds__(PR_THREADS, 2) k_token_probs(const float *x, long long xs, int V, ExpScale c,
                                                           float *out, long long os) {
  __shared__ float sv[PR_WARPS], ss[PR_WARPS];
  __shared__ int si[PR_WARPS];
  __shared__ float pub[3];  // this block's maximum, sum, index of the maximum
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int rank = cluster_rank(), n_blk = cluster_size();
  pdl_launch_dependents();
  pdl_wait();
  const long long row = blockIdx.x / n_blk;
  const float *r = x + row * xs;
  float *o = out + row * os;
  constexpr int S = VEC ? 1 : PR_THREADS;  // between a thread's entries
  const int lead = VEC ? 4 * tid : tid;
  const int part = ((V + n_blk - 1) / n_blk + 3) & ~3;
  const int begin = min(V, rank * part), end = min(V, begin + part);
  float4 v[SP_KEEP];
#pragma unroll
  for (int k = 0; k < SP_KEEP; k++)
    v[k] = row4<VEC, S>(r, begin + lead + 4 * k * PR_THREADS, end, -INFINITY, begin + 4 * (k + 1) * PR_THREADS <= end);
  const int rest = begin + lead + 4 * SP_KEEP * PR_THREADS;
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < SP_KEEP; k++) m = fmaxf(fmaxf(fmaxf(m, v[k].x), fmaxf(v[k].y, v[k].z)), v[k].w);
  for (int i = rest; i < end; i += 4 * PR_THREADS) {
    const float4 y = row4<VEC, S>(r, i, end, -INFINITY);
    m = fmaxf(fmaxf(fmaxf(m, y.x), fmaxf(y.y, y.z)), y.w);
  }
  m = warp_max(m);
  if (lane == 0) sv[w] = m;
  __syncthreads();
  m = warp_max(sv[lane & (PR_WARPS - 1)]);
  if (c.t == 0.0f) {
    // the lowest index that holds the maximum, and whether there is a NaN
    int at = V;
    bool nan = false;
    auto look = [&](float a, int i) {
      nan |= a != a;
      if (a == m && i < end) at = min(at, i);
    };
#pragma unroll
    for (int k = 0; k < SP_KEEP; k++) {
      const int i = begin + lead + 4 * k * PR_THREADS;
      look(v[k].x, i), look(v[k].y, i + S), look(v[k].z, i + 2 * S), look(v[k].w, i + 3 * S);
    }
    for (int i = rest; i < end; i += 4 * PR_THREADS) {
      const float4 y = row4<VEC, S>(r, i, end, -INFINITY);
      look(y.x, i), look(y.y, i + S), look(y.z, i + 2 * S), look(y.w, i + 3 * S);
    }
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) si[w] = at;
    nan = __syncthreads_or(nan);
    if (tid == 0) {
      for (int i = 0; i < PR_WARPS; i++) at = min(at, si[i]);
      pub[0] = nan ? NAN : m, pub[2] = __int_as_float(at);
    }
    cluster_sync();
    float best = -INFINITY;
    int where = V;
    for (int b = 0; b < n_blk; b++) {
      const float pm = __uint_as_float(ld_peer(&pub[0], b));
      if (pm != pm) best = NAN;
      else arg_max(best, where, pm, (int)ld_peer(&pub[2], b));
    }
    cluster_sync();  // a block's shared memory outlives its readers
    const bool bad = best != best;
    for (int i = begin + lead; i < end; i += 4 * PR_THREADS) {
      const float one[2] = {bad ? NAN : 0.0f, bad ? NAN : 1.0f};
      put4<VEC, S>(o, i, end, make_float4(one[i == where], one[i + S == where], one[i + 2 * S == where], one[i + 3 * S == where]));
    }
    return;
  }
  // (a part of nothing but -infinity weighs nothing)
  const float mz = m == -INFINITY ? 0.0f : m;
  auto e = [&](float a) { return exp_over_t(a - mz, c); };
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < SP_KEEP; k++) {
    v[k] = make_float4(e(v[k].x), e(v[k].y), e(v[k].z), e(v[k].w));
    sum += (v[k].x + v[k].y) + (v[k].z + v[k].w);
  }
  for (int i = rest; i < end; i += 4 * PR_THREADS) {
    const float4 y = row4<VEC, S>(r, i, end, -INFINITY);
    sum += (e(y.x) + e(y.y)) + (e(y.z) + e(y.w));
  }
#pragma unroll
  for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
  if (lane == 0) ss[w] = sum;
  __syncthreads();
  if (w == 0) {
    sum = lane < PR_WARPS ? ss[lane] : 0.0f;
#pragma unroll
    for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    if (lane == 0) pub[0] = m, pub[1] = sum;
  }
  cluster_sync();
  if (w == 0) {
    // one warp, a lane per block: the row's maximum and sum, this block's factor
    const float pm = lane < n_blk ? __uint_as_float(ld_peer(&pub[0], lane)) : -INFINITY;
    const float ps = lane < n_blk ? __uint_as_float(ld_peer(&pub[1], lane)) : 0.0f;
    const float top = warp_max(pm);
    float total = pm == -INFINITY ? ps : ps * exp_over_t(pm - top, c);
#pragma unroll
    for (int k = 4; k; k >>= 1) total += __shfl_xor_sync(0xffffffffu, total, k);
    if (lane == 0) ss[0] = (m == -INFINITY ? 0.0f : exp_over_t(m - top, c)) / total;
  }
  // a block's shared memory outlives its readers (nothing is handed over: relaxed)
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  __syncthreads();
  const float f = ss[0];
#pragma unroll
  for (int k = 0; k < SP_KEEP; k++) {
    const int i = begin + lead + 4 * k * PR_THREADS;
    put4<VEC, S>(o, i, end, make_float4(v[k].x * f, v[k].y * f, v[k].z * f, v[k].w * f),
              begin + 4 * (k + 1) * PR_THREADS <= end);
  }
  for (int i = rest; i < end; i += 4 * PR_THREADS) {
    const float4 y = row4<VEC, S>(r, i, end, -INFINITY);
    put4<VEC, S>(o, i, end, make_float4(e(y.x) * f, e(y.y) * f, e(y.z) * f, e(y.w) * f));
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Verification. Sums of probabilities decide a whole number, so they are
// exact: a probability is rounded to a multiple of 2^-shift, shift = 45 (less
// for a vocabulary above 2^17, so that sums stay below 2^62), and summed in
// integers, whose sum does not depend on the order. A fixed-point value is
// hi 2^(shift - 22) + lo with hi = rint(p 2^22) and lo the rounded remainder;
// both come from adding 1.5 2^23 to a float, so that an entry costs 5 float
// operations and two 32-bit additions where a 64-bit shift would take three
// times as many.

struct VerifyArgs {
  const float *target, *draft;       // [n_seq][G + 1][V], [n_seq][G][V] or null
  long long t_pitch, d_pitch;        // elements from row to row
  const int32_t *tok, *n_draft;      // [n_seq][G], [n_seq] or null
  const float *u_accept, *u_sample;  // [n_seq][G], [n_seq]
  int32_t G, V, shift;
  int32_t *n_accepted, *tokens;      // [n_seq], [n_seq][G + 1]
  uint32_t *err;
};

constexpr float SP_MAGIC = 12582912.0f;  // 1.5 2^23: x + SP_MAGIC holds rint(x) in its low bits

// hi and lo of p, each plus the bits of SP_MAGIC. NaN and negative p: 0;
// above 1: 1. lo_scale = 2^(shift - 22).
__device__ __forceinline__ void split_prob(float p, float lo_scale, int &hi, int &lo) {
  const float t = __saturatef(p) * 4194304.0f;
  const float h = __fadd_rn(t, SP_MAGIC);
  const float l = __fadd_rn(t, -__fadd_rn(h, -SP_MAGIC));  // exact
  hi = __float_as_int(h), lo = __float_as_int(__fmaf_rn(l, lo_scale, SP_MAGIC));
}

// What the last token is drawn from at one entry: p less q (dropped below 0:
// the rounding is monotonic, so p > q decides) as (hi, lo).
__device__ __forceinline__ void mass_of(float p, float q, float lo_scale, int &hi, int &lo) {
  int ph, pl, qh, ql;
  split_prob(p, lo_scale, ph, pl);
  split_prob(q, lo_scale, qh, ql);
  const bool more = __saturatef(p) > __saturatef(q);
  hi = more ? ph - qh : 0, lo = more ? pl - ql : 0;
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

__device__ __forceinline__ long long warp_sum64(long long v) {
#pragma unroll
  for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// One sequence per cluster. Every block finds the first draft that is not
// accepted, then sums its part of the one row (of p, and of q) that the token
// is drawn from; the sums meet in shared memory of the cluster, and the warp
// whose run of entries holds the border scans that run again. Bound by three
// dependent reads (count and token, the probabilities at the token, the rows)
// and then by the rows' bytes: 7.3 us for one sequence of 129280, 20 us for 64
// (66 MB; the four blocks of a sequence fill the SMs unevenly, 1 or 2 each).
template <bool VEC>
__global__ void __launch_bounds__(SP_THREADS) k_verify_drafts(const VerifyArgs a) {
  __shared__ long long part[SP_WARPS];
  __shared__ __align__(8) int pub[2];  // this block's sum, low and high word
  __shared__ long long s_sum[2];  // of all blocks, of those before this one
  __shared__ int s_n;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int rank = cluster_rank(), n_blk = cluster_size(), b = blockIdx.x / n_blk;
  pdl_launch_dependents();
  pdl_wait();
  int cnt = a.G;
  if (a.n_draft) {
    const int given = a.n_draft[b];
    cnt = min(max(given, 0), a.G);
    if (cnt != given && tid == 0) raise_flag(a.err, DS4MOE_DEVERR_LENGTH);
  }
  if (w == 0) {
    // draft i is accepted when u * q < p, both clamped as where the token is
    // drawn (__saturatef: to [0, 1], NaN to 0): the product of two 24-bit
    // significands is exact in 64 bits
    int n = cnt;
    for (int i = lane; i < cnt; i += 32) {
      const int t = a.tok[(long long)b * a.G + i];
      bool ok = false;
      if (t >= 0 && t < a.V) {
        const double p = __saturatef(a.target[((long long)b * (a.G + 1) + i) * a.t_pitch + t]);
        const double q = a.draft ? __saturatef(a.draft[((long long)b * a.G + i) * a.d_pitch + t]) : 1.0f;
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
  // a warp's run: a multiple of 128 entries, four per lane and step
  const int per = ((a.V + n_blk * SP_WARPS - 1) / (n_blk * SP_WARPS) + 127) & ~127;
  const int i0 = min(a.V, (rank * SP_WARPS + w) * per), i1 = min(a.V, i0 + per);
  const int lo_bits = a.shift - 22;
  const float lo_scale = (float)(1 << lo_bits);
  // hi and lo of four entries, `step` apart
  constexpr int S = VEC ? 1 : 32;
  auto four = [&](auto step, int i, int (&hi)[4], int (&lo)[4], bool inner) {
    constexpr int N = decltype(step)::value;
    const float4 x = row4<VEC, N>(p, i, i1, 0.0f, inner);
    const float4 y = q ? row4<VEC, N>(q, i, i1, 0.0f, inner) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float px[4] = {x.x, x.y, x.z, x.w}, qx[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int k = 0; k < 4; k++) {
      mass_of(px[k], qx[k], lo_scale, hi[k], lo[k]);
      if (dtok >= 0 && i + k * N == dtok) hi[k] = lo[k] = 0;
    }
  };
  long long total = 0, before = 0, mine = 0;
  for (int round = 0; round < 2; round++) {
    long long s = 0;
    for (int c = i0 + (VEC ? 4 * lane : lane); c < i1; c += 8 * 128) {
      int sh = 0, sl = 0;  // 32 entries: |hi|, |lo| < 2^28
#pragma unroll
      for (int k = 0; k < 8; k++) {
        int hi[4], lo[4];
        four(std::integral_constant<int, S>(), c + 128 * k, hi, lo, c - (VEC ? 4 * lane : lane) + 128 * (k + 1) <= i1);
        sh += (hi[0] + hi[1]) + (hi[2] + hi[3]), sl += (lo[0] + lo[1]) + (lo[2] + lo[3]);
      }
      s += ((long long)sh << lo_bits) + sl;
    }
    mine = warp_sum64(s);
    if (lane == 0) part[w] = mine;
    __syncthreads();
    if (w == 0) {
      const long long t = warp_sum64(lane < SP_WARPS ? part[lane] : 0);
      if (lane == 0) pub[0] = (int)(uint32_t)t, pub[1] = (int)(t >> 32);
    }
    cluster_sync();
    if (w == 0) {
      const long long t =
          lane < n_blk ? (long long)ld_peer(&pub[0], lane) | (long long)ld_peer(&pub[1], lane) << 32 : 0;
      const long long all = warp_sum64(t), mine_from = warp_sum64(lane < rank ? t : 0);
      if (lane == 0) s_sum[0] = all, s_sum[1] = mine_from;
    }
    __syncthreads();
    total = s_sum[0], before = s_sum[1];
    for (int i = 0; i < w; i++) before += part[i];
    // read by all before it is written again or the block leaves
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (total > 0 || (!q && dtok < 0)) break;
    q = nullptr, dtok = -1;  // nothing is left: draw from p itself
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  int32_t *out = a.tokens + (long long)b * (a.G + 1);
  if (total > 0) {
    const long long thr = (long long)__umul64hi((unsigned long long)total, fixed_u(a.u_sample[b]));
    if (before <= thr && thr < before + mine) {
      for (int c = i0; c < i1; c += 128) {
        int hi[4], lo[4];
        four(std::integral_constant<int, 1>(), c + 4 * lane, hi, lo, c + 128 <= i1);
        long long e[4];
#pragma unroll
        for (int k = 0; k < 4; k++) e[k] = ((long long)hi[k] << lo_bits) + lo[k] + (k ? e[k - 1] : 0);
        long long s = e[3];
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
          const long long o = __shfl_up_sync(0xffffffffu, s, k);
          if (lane >= k) s += o;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + s > thr);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            const long long at = before + s - e[3];
            int k = 0;
            while (k < 3 && at + e[k] <= thr) k++;
            out[n] = c + 4 * lane + k;
          }
          break;
        }
        before += __shfl_sync(0xffffffffu, s, 31);
      }
    }
  } else if (rank == 0 && tid == 0) {
    out[n] = -1;
  }
  if (rank == 0) {
    if (tid <= a.G && tid != n) out[tid] = tid < n ? a.tok[(long long)b * a.G + tid] : -1;
    if (tid == 0) a.n_accepted[b] = n;
  }
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

static cudaError_t launch_rows(const void *fn, int rows, int cluster, int threads, cudaStream_t s, void **args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * cluster);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelExC(&cfg, fn, args);
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

// SMs of the current device, 0 on an error.
int sp_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
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
  if (!(temperature == 0.0f || (temperature >= 1e-6f && temperature <= 1e6f))) return DS4MOE_ERR_INVALID_ARG;
  if (n_rows == 0) return DS4MOE_OK;
  if (n_rows > 1 && (logits_stride < vocab || probs_stride < vocab)) return DS4MOE_ERR_INVALID_ARG;
  if (!sp_dev_ptr(logits) || !sp_dev_ptr(probs)) return DS4MOE_ERR_INVALID_ARG;
  const double scale = temperature > 0.0f ? 1.4426950408889634 / temperature : 0.0;  // log2(e) / T
  ExpScale c = {(float)scale, (float)(scale - (float)scale), temperature > 0.0f ? (float)(-200.0 / scale) : 0.0f,
                temperature};
  long long xs = logits_stride, os = probs_stride;
  void *args[] = {(void *)&logits, &xs, &vocab, &c, (void *)&probs, &os};
  const bool vec = (n_rows == 1 || (xs % 4 == 0 && os % 4 == 0)) && ((uintptr_t)logits & 15) == 0 && ((uintptr_t)probs & 15) == 0;
  // Many rows: as few blocks per row as keep a part in registers (320 rows of
  // 50001: 63 -> 39 us); few: as many as share the latency.
  const int n_sm = sp_sms();
  if (!n_sm) return sp_status(cudaErrorUnknown);
  int cluster = cluster_of(vocab);
  while (cluster > 1 && (long long)n_rows * cluster > 2 * n_sm && vocab <= cluster / 2 * SP_KEEP * 4 * PR_THREADS) cluster /= 2;
  return sp_status(launch_rows(vec ? (const void *)k_token_probs<true> : (const void *)k_token_probs<false>, n_rows,
                               cluster, PR_THREADS, (cudaStream_t)stream, args));
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
  a.shift = lg > 17 ? 62 - lg : 45;
  const bool vec = target_stride % 4 == 0 && ((uintptr_t)target & 15) == 0 &&
                   (!a.draft || (draft_stride % 4 == 0 && ((uintptr_t)draft & 15) == 0));
  void *args[] = {&a};
  // Smaller clusters where a batch would not be resident at once (two blocks
  // per SM): a second wave of short blocks costs as much as the first.
  const int n_sm = sp_sms();
  if (!n_sm) return sp_status(cudaErrorUnknown);
  int cluster = cluster_of(vocab);
  while (cluster > 1 && (long long)n_seq * cluster > 2 * n_sm) cluster /= 2;
  return sp_status(launch_rows(vec ? (const void *)k_verify_drafts<true> : (const void *)k_verify_drafts<false>, n_seq,
                               cluster, SP_THREADS, (cudaStream_t)stream, args));
}

}  // extern "C"
