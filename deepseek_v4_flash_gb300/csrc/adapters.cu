// adapters.cu -- low-rank adapters of many requests beside a shared projection:
//   y[t] = base[t] + scale_s B_s (A_s x[t]),  s = slots[t]  (no adapter: base[t]).
//
// A_s is [rank][n_in], B_s [n_out][rank] in 16 bits, x, base and y rows of tokens.
// Sums are in 32 bits, A x stays in 32 bits between the two products.
//
// Few tokens (LR_TOKENS): k_adapt_token, a cluster of eight blocks per token,
// one launch. A block takes an eighth of the columns of A, the eight exchange
// their partial sums through distributed shared memory, then each computes an
// eighth of y. Bound by the latency of that chain and, with many adapters, by
// the adapters' bytes.
//
// Many tokens: bound by the bytes of x, base and y, provided that the products
// run on the tensor cores. k_adapt_plan sorts the tokens by adapter and cuts
// them into tiles of up to 128; k_adapt_shrink computes V = scale A x per tile
// (a cluster per tile, the columns of A split over its blocks); k_adapt_expand
// y = base + B V per tile and 128 columns. Products are tcgen05.mma kind::tf32:
// a 16-bit weight is exact in tf32, and an fp32 operand is the sum of two tf32
// numbers to 2^-20, so two products give what fp32 would.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>

#include "attn.cuh"
#include "internal.h"
#include "umma.cuh"

struct ds4moe_adapters {
  int N, K, slots, max_rank, dtype, max_tokens, device, n_sm;
  int R32;           // rows of a slot's A: max_rank rounded up to 32
  long long b_slot;  // elements of a slot's B: n_out times max_rank rounded up to 8
  uint8_t *mem;      // one allocation; the rest points into it
  uint32_t *err;
  int2 *info;        // [slots] {rank, bits of the scale}
  uint16_t *A;       // [slots][R32][K]
  uint16_t *B;       // [slots] of [N][rank rounded up to 8]
  int *perm;         // [max_tokens] tokens in the order of their adapters
  int4 *tiles;       // {slot, first place in perm, tokens | rank << 16, bits of the scale}
  int *n_tiles;
  float *v;          // [max_tokens][R32] scale A x by place in perm
  int clusters[9];   // clusters of so many blocks of k_adapt_shrink that run at once
  uint64_t bytes, launches;
};

namespace ds4 {

constexpr int LR_CLUSTER = 8;
constexpr int LR_MAX_RANK = 256, LR_MAX_SLOTS = 4096;
// Largest call of k_adapt_token.
constexpr int LR_TOKENS = 64;

struct AdaptArgs {
  int N, K, slots, T, R32;
  long long b_slot, x_stride, y_stride, base_stride;
  const void *x;
  const float *base;  // null: y itself
  float *y;
  const int32_t *slot_of;
  const int2 *info;
  const uint16_t *A, *B;
  int *perm;
  int4 *tiles;
  int *n_tiles;
  float *v;
  int wide;  // y and base take 16-byte accesses
  uint32_t *err;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ float remote_f32(uint32_t addr, int rank) {
  uint32_t r;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
  return v;
}
__device__ __forceinline__ float4 remote_f32x4(uint32_t addr, int rank) {
  uint32_t r;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(r) : "memory");
  return v;
}

// Slot of a token, -1 for none (and, with the flag, for one that there is not).
__device__ __forceinline__ int slot_at(const AdaptArgs &a, int t, bool &bad) {
  const int s = a.slot_of[t];
  if (s >= -1 && s < a.slots) return s;
  bad = true;
  return -1;
}

// ---------------------------------------------------------------------------
// Few tokens.

// Eight 16-bit weights times eight floats.
template <int DT>
__device__ __forceinline__ float dot8(const uint4 &w, const float *x, float s) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float2 f = Half16<DT>::up(u[i]);
    s = fmaf(f.x, x[2 * i], s), s = fmaf(f.y, x[2 * i + 1], s);
  }
  return s;
}

template <int DT, bool F32>
__global__ void __launch_bounds__(256) k_adapt_token(const AdaptArgs a) {
  extern __shared__ __align__(16) float s_x[];  // this block's columns of x
  __shared__ float s_part[LR_MAX_RANK];
  __shared__ __align__(16) float s_v[LR_MAX_RANK];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, c = (int)cluster_rank(), t = blockIdx.x / LR_CLUSTER;
  pdl_launch_dependents();
  pdl_wait();
  bool bad = false;
  const int s = slot_at(a, t, bad);
  if (bad && c == 0 && tid == 0) raise_flag(a.err, DS4MOE_DEVERR_ADAPTER);
  const int2 in = s >= 0 ? a.info[s] : make_int2(0, 0);
  const int rank = in.x;
  const int n0 = (int)((long long)a.N * c / LR_CLUSTER), n1 = (int)((long long)a.N * (c + 1) / LR_CLUSTER);
  const float *base = a.base ? a.base + (long long)t * a.base_stride : a.y + (long long)t * a.y_stride;
  float *y = a.y + (long long)t * a.y_stride;
  if (rank == 0) {  // (the same for all blocks of the cluster)
    if (a.base)
      for (int n = n0 + tid; n < n1; n += 256) y[n] = base[n];
    return;
  }
  const int r8 = (rank + 7) & ~7;
  const uint16_t *A = a.A + (long long)s * a.R32 * a.K, *B = a.B + (long long)s * a.b_slot;
  if (tid == 0) {  // this block's part of B on its way
    const uint32_t bytes = (uint32_t)min((long long)(n1 - n0) * r8 * 2, 1ll << 20);
    if (bytes) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(B + (long long)n0 * r8), "r"(bytes) : "memory");
  }
  // pieces of eight columns
  const int u0 = (int)((long long)(a.K / 8) * c / LR_CLUSTER), nu = (int)((long long)(a.K / 8) * (c + 1) / LR_CLUSTER) - u0;
  for (int u = tid; u < nu; u += 256) {
    float4 lo, hi;
    if (F32) {
      const float4 *p = reinterpret_cast<const float4 *>((const float *)a.x + (long long)t * a.x_stride) + 2 * (u0 + u);
      lo = p[0], hi = p[1];
    } else {
      const uint4 q = reinterpret_cast<const uint4 *>((const uint16_t *)a.x + (long long)t * a.x_stride)[u0 + u];
      const float2 f0 = Half16<DT>::up(q.x), f1 = Half16<DT>::up(q.y), f2 = Half16<DT>::up(q.z), f3 = Half16<DT>::up(q.w);
      lo = make_float4(f0.x, f0.y, f1.x, f1.y), hi = make_float4(f2.x, f2.y, f3.x, f3.y);
    }
    reinterpret_cast<float4 *>(s_x)[2 * u] = lo, reinterpret_cast<float4 *>(s_x)[2 * u + 1] = hi;
  }
  __syncthreads();
  // four rows of A per warp at a time
  for (int r0 = 4 * w; r0 < rank; r0 += 32) {
    float sum[4] = {};
    const uint4 *p = reinterpret_cast<const uint4 *>(A + (long long)r0 * a.K) + u0;
    for (int u = lane; u < nu; u += 32) {
      float x[8];
      *reinterpret_cast<float4 *>(x) = reinterpret_cast<const float4 *>(s_x)[2 * u];
      *reinterpret_cast<float4 *>(x + 4) = reinterpret_cast<const float4 *>(s_x)[2 * u + 1];
#pragma unroll
      for (int j = 0; j < 4; j++) sum[j] = dot8<DT>(p[(long long)j * (a.K / 8) + u], x, sum[j]);  // (rows past the rank are zeros)
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int j = 0; j < 4; j++) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < 4; j++) s_part[r0 + j] = sum[j];
    }
  }
  cluster_arrive();
  cluster_wait();
  const float scale = __int_as_float(in.y);
  for (int r = tid; r < r8; r += 256) {
    float v = 0.0f;
    if (r < rank)
#pragma unroll
      for (int i = 0; i < LR_CLUSTER; i++) v += remote_f32(smem_u32(s_part + r), i);
    s_v[r] = v * scale;
  }
  __syncthreads();
  cluster_arrive();  // the others' sums are read: they may leave
  for (int n = n0 + tid; n < n1; n += 256) {
    const uint4 *p = reinterpret_cast<const uint4 *>(B + (long long)n * r8);
    float sum = 0.0f;
    for (int u = 0; u < r8 / 8; u++) sum = dot8<DT>(p[u], s_v + 8 * u, sum);
    y[n] = base[n] + sum;
  }
  cluster_wait();
}

// ---------------------------------------------------------------------------
// Many tokens.

// Tokens by adapter (no adapter last, only where base has to be copied), and
// the tiles. One block; a thread keeps the slots of its first LR_KEEP tokens.
constexpr int LR_KEEP = 8;
__global__ void __launch_bounds__(1024) k_adapt_plan(const AdaptArgs a) {
  __shared__ int s_n[LR_MAX_SLOTS + 1], s_at[LR_MAX_SLOTS + 1];
  __shared__ int w_rows[32], w_tiles[32];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  pdl_wait();
  int raw[LR_KEEP];
#pragma unroll
  for (int i = 0; i < LR_KEEP; i++) raw[i] = tid + 1024 * i < a.T ? a.slot_of[tid + 1024 * i] : -1;
  for (int s = tid; s <= a.slots; s += 1024) s_n[s] = 0, s_at[s] = s < a.slots ? a.info[s].x : 0;  // (ranks, for now)
  __syncthreads();
  bool bad = false;
  // a token's bucket, -1 for none; a.slots: base is copied
  auto bucket = [&](int t, int s) {
    if (t >= a.T) return -1;
    if (s < -1 || s >= a.slots) bad = true, s = -1;
    if (s >= 0 && s_at[s] == 0) s = -1;
    return s >= 0 ? s : a.base ? a.slots : -1;
  };
  auto count = [&](int *at, int s) {  // the warp's tokens of one bucket together; a token's place
    const unsigned m = __match_any_sync(0xffffffffu, s);
    const int first = __ffs(m) - 1;
    int p = 0;
    if (lane == first && s >= 0) p = atomicAdd(at + s, __popc(m));
    return __shfl_sync(0xffffffffu, p, first) + __popc(m & ((1u << lane) - 1));
  };
#pragma unroll
  for (int i = 0; i < LR_KEEP; i++) {
    if (1024 * i >= a.T) break;
    raw[i] = bucket(tid + 1024 * i, raw[i]);
    count(s_n, raw[i]);
  }
  for (int t = 1024 * LR_KEEP + tid; t - tid < a.T; t += 1024) count(s_n, bucket(t, t < a.T ? a.slot_of[t] : -1));
  __syncthreads();
  // exclusive sums of rows and tiles over the buckets, five per thread
  constexpr int PER = (LR_MAX_SLOTS + 1 + 1023) / 1024;
  int rows = 0, tiles = 0, rank[PER];
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int s = tid * PER + i;
    rank[i] = 0;
    if (s <= a.slots) rows += s_n[s], tiles += (s_n[s] + 127) / 128, rank[i] = s_at[s];
  }
  int ri = rows, ti = tiles;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, ri, o), z = __shfl_up_sync(0xffffffffu, ti, o);
    if (lane >= o) ri += x, ti += z;
  }
  if (lane == 31) w_rows[w] = ri, w_tiles[w] = ti;
  __syncthreads();
  int r0 = ri - rows, t0 = ti - tiles;
  for (int i = 0; i < w; i++) r0 += w_rows[i], t0 += w_tiles[i];
  // tokens beyond the kept ones need the ranks once more
  int places[PER];
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int s = tid * PER + i;
    places[i] = r0;
    if (s > a.slots) continue;
    const int scale = s < a.slots && s_n[s] ? a.info[s].y : 0;
    for (int k = 0; k < s_n[s]; k += 128) a.tiles[t0++] = make_int4(s, r0 + k, min(128, s_n[s] - k) | rank[i] << 16, scale);
    r0 += s_n[s];
  }
  if (tid == 1023) *a.n_tiles = t0;
#pragma unroll
  for (int i = 0; i < PER; i++)
    if (tid * PER + i <= a.slots) s_n[tid * PER + i] = places[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < LR_KEEP; i++) {
    if (1024 * i >= a.T) break;
    const int p = count(s_n, raw[i]);
    if (raw[i] >= 0) a.perm[p] = tid + 1024 * i;
  }
  for (int t = 1024 * LR_KEEP + tid; t - tid < a.T; t += 1024) {
    const int s = bucket(t, t < a.T ? a.slot_of[t] : -1), p = count(s_n, s);
    if (s >= 0) a.perm[p] = t;
  }
  if (bad) raise_flag(a.err, DS4MOE_DEVERR_ADAPTER);
}

// kind::tf32, both operands K-major, fp32 accumulator.
__device__ __forceinline__ uint32_t idesc_tf32(int n) {
  return (1u << 4) | (2u << 7) | (2u << 10) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void umma_tf32(uint32_t d, uint64_t x, uint64_t y, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::tf32 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(x), "l"(y), "r"(id), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void sts4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
template <int N>
__device__ __forceinline__ void named_sync(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(N) : "memory");
}
// Byte of 16-byte piece p (0..7) of row r in a 128-byte swizzled operand.
__device__ __forceinline__ uint32_t sw128(int r, int p) { return (uint32_t)(r * 128 + ((p ^ (r & 7)) << 4)); }

// Four floats as a 16-byte piece of the two operands: x = hi + lo, each cut to
// the 11 bits of a tf32 number (an error of 2^-20 of x at most). For an infinity
// lo is NaN: either sums whose high part is not finite leave the low part out
// (add_low), or it is made 0 (INF).
constexpr uint32_t TF32 = 0xFFFFE000u;
template <bool INF>
__device__ __forceinline__ void put_split(uint32_t hi_at, uint32_t lo_at, const uint4 &x) {
  const uint32_t h0 = x.x & TF32, h1 = x.y & TF32, h2 = x.z & TF32, h3 = x.w & TF32;
  auto rest = [](uint32_t v, uint32_t h) {
    const float d = __uint_as_float(v) - __uint_as_float(h);
    return INF && isinf(__uint_as_float(v)) ? 0u : __float_as_uint(d) & TF32;
  };
  sts4(hi_at, h0, h1, h2, h3);
  sts4(lo_at, rest(x.x, h0), rest(x.y, h1), rest(x.z, h2), rest(x.w, h3));
}
__device__ __forceinline__ float add_low(float hi, float lo) { return isfinite(hi) ? hi + lo : hi; }
// Eight 16-bit numbers as two pieces of one operand: pieces 2 p and 2 p + 1 of row r.
template <int DT>
__device__ __forceinline__ void put_wide(uint32_t at, int r, int p, const uint4 &w) {
  auto f = [](float v) { return __float_as_uint(v); };
  const float2 f0 = Half16<DT>::up(w.x), f1 = Half16<DT>::up(w.y), f2 = Half16<DT>::up(w.z), f3 = Half16<DT>::up(w.w);
  sts4(at + sw128(r, 2 * p), f(f0.x), f(f0.y), f(f1.x), f(f1.y));
  sts4(at + sw128(r, 2 * p + 1), f(f2.x), f(f2.y), f(f3.x), f(f3.y));
}

// After a wait has run out the others that follow from it are short.
struct Waits {
  bool ok = true;
  __device__ __forceinline__ void wait(uint32_t bar, uint32_t parity) {
    if (!mbar_wait_bounded(bar, parity, ok ? WAIT_LIMIT : 1000)) ok = false;
  }
};

constexpr int LR_HALF = 128 * 128;  // 128 rows of 32 tf32 numbers
constexpr int LR_SMEM = 224 * 1024;  // a block has an SM (and all of its tensor memory) to itself

// ---- V = scale A x. One tile per cluster at a time; block k of the cluster
// takes a part of the columns, 32 at a time. Sixteen warps split x (and widen
// A) on the way from registers, where the next AHEAD chunks are under way, to
// a ring in shared memory; one warp issues the products.
//
// The tensor cores add a product to an accumulator with the sum cut, not rounded,
// to 24 bits, so a long chain of additions drifts: 256 of them (1024 columns)
// were off by 4e-6 of the result, five times what 32-bit sums are. So chunks go
// round several accumulators, the low parts of x to one of their own, added up
// in 32 bits at the end.
constexpr int LR_WARPS = 16;
__host__ __device__ constexpr int shrink_stage(bool f32, int r32) { return LR_HALF * (f32 ? 2 : 1) + r32 * 128; }
__host__ __device__ constexpr int shrink_stages(bool f32, int r32) {
  const int n = (LR_SMEM - 1024) / shrink_stage(f32, r32);
  return n < 6 ? n : 6;
}
__host__ __device__ constexpr int shrink_accs(int r32) { return 512 / r32 < 8 ? 512 / r32 : 8; }

// WP: pieces of A per thread and chunk: one for ranks up to 128, else two.
template <int DT, bool F32, int WP>
__global__ void __launch_bounds__(LR_WARPS * 32 + 32, 1) k_adapt_shrink(const AdaptArgs a, int ks) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[2 * 6 + 1];
  __shared__ uint32_t s_tmem;
  const int tid = threadIdx.x, w = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const int stage_bytes = shrink_stage(F32, a.R32), nst = shrink_stages(F32, a.R32);
  const uint32_t bar0 = smem_u32(s_bar);
  auto full = [&](int i) { return bar0 + 8 * i; };
  auto empty = [&](int i) { return bar0 + 8 * (6 + i); };
  const uint32_t b_done = bar0 + 8 * 12;
  if (w == LR_WARPS) {
    if (lane == 0) {
      for (int i = 0; i < 6; i++) mbar_init(full(i), LR_WARPS), mbar_init(empty(i), 1);
      mbar_init(b_done, 1);
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(smem_u32(&s_tmem), 512);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  pdl_launch_dependents();
  pdl_wait();
  const int k = (int)cluster_rank(), n_tiles = *a.n_tiles, n_cl = gridDim.x / ks;
  const int ch0 = (a.K / 32) * k / ks, nc = (a.K / 32) * (k + 1) / ks - ch0;  // chunks of 32 columns
  // accumulators of the high parts; the low parts' one comes after them
  const int n_acc = shrink_accs(a.R32) - (F32 ? 1 : 0);
  Waits ws;
  constexpr int XP = F32 ? 2 : 1, PR = F32 ? 8 : 4;  // 16-byte pieces of x per thread and chunk; pieces of a row
  constexpr int AHEAD = WP == 1 ? 4 : 2;
  uint4 x[AHEAD][XP], wt[AHEAD][WP];
  const char *xp[XP];
  const uint16_t *ap;
  int r32 = 0;
  // the next tile with a rank, from i on, and this thread's part of it
  auto begin = [&](int i) {
    int4 tile = make_int4(0, 0, 0, 0);
    for (; i < n_tiles; i += n_cl) {
      tile = a.tiles[i];
      if (tile.z >> 16) break;
    }
    if (i >= n_tiles || w == LR_WARPS) return i;
    r32 = ((tile.z >> 16) + 31) & ~31;
#pragma unroll
    for (int j = 0; j < XP; j++) {
      const int r = tid / PR + j * (LR_WARPS * 32 / PR);
      xp[j] = nullptr;
      if (r < (tile.z & 0xFFFF))
        xp[j] = (const char *)a.x + ((long long)a.perm[tile.y + r] * a.x_stride + ch0 * 32) * (F32 ? 4 : 2) + tid % PR * 16;
    }
    ap = a.A + ((long long)tile.x * a.R32 + tid / 4) * a.K + ch0 * 32 + tid % 4 * 8;
    return i;
  };
  auto fetch = [&](int c, uint4 (&x)[XP], uint4 (&wt)[WP]) {
#pragma unroll
    for (int j = 0; j < XP; j++)
      x[j] = xp[j] && c < nc ? __ldcs(reinterpret_cast<const uint4 *>(xp[j] + (long long)c * (F32 ? 128 : 64))) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < WP; j++)
      if (128 * j + tid / 4 < r32 && c < nc) wt[j] = *reinterpret_cast<const uint4 *>(ap + (long long)128 * j * a.K + c * 32);
  };
  int used = 0, tiles = 0;  // chunks, tiles so far
  int i = begin(blockIdx.x / ks);
  if (i < n_tiles && w < LR_WARPS) {
#pragma unroll
    for (int c = 0; c < AHEAD; c++) fetch(c, x[c], wt[c]);
  }
  while (i < n_tiles) {
    const int4 tile = a.tiles[i];
    const int rank = tile.z >> 16, rows = tile.z & 0xFFFF, r32_now = (rank + 31) & ~31;
    int next;
    if (w < LR_WARPS) {
      for (int c0 = 0; c0 < nc; c0 += AHEAD) {
#pragma unroll
        for (int j = 0; j < AHEAD; j++) {
          const int c = c0 + j;
          if (c >= nc) break;
          const int u = used + c, st = u % nst;
          if (u >= nst) ws.wait(empty(st), (u / nst - 1) & 1);
          const uint32_t at = base + st * stage_bytes, wa = at + LR_HALF * (F32 ? 2 : 1);
#pragma unroll
          for (int p = 0; p < XP; p++) {
            const int r = tid / PR + p * (LR_WARPS * 32 / PR);
            if (F32) {
              const uint32_t o = sw128(r, tid % PR);
              put_split<false>(at + o, at + LR_HALF + o, x[j][p]);
            } else {
              put_wide<DT>(at, r, tid % PR, x[j][p]);
            }
          }
#pragma unroll
          for (int p = 0; p < WP; p++)
            if (128 * p + tid / 4 < r32_now) put_wide<DT>(wa, 128 * p + tid / 4, tid % 4, wt[j][p]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full(st));
          fetch(c + AHEAD, x[j], wt[j]);
        }
      }
      // the next tile's first chunks come in while this one is added up
      next = begin(i + n_cl);
      if (next < n_tiles) {
#pragma unroll
        for (int c = 0; c < AHEAD; c++) fetch(c, x[c], wt[c]);
      }
    } else {
      const uint32_t id = idesc_tf32(__shfl_sync(0xffffffffu, r32_now, 0));
      for (int c = 0; c < nc; c++) {
        const int u = __shfl_sync(0xffffffffu, used + c, 0), uc = __shfl_sync(0xffffffffu, c, 0), st = u % nst;
        ws.wait(full(st), (u / nst) & 1);
        __syncwarp();
        tc_fence_after();
        const uint32_t sa = base + st * stage_bytes;
        const uint64_t dh = desc_sw128(sa, 0), dl = desc_sw128(sa + LR_HALF, 0), dw = desc_sw128(sa + LR_HALF * (F32 ? 2 : 1), 0);
        const uint32_t acc = tmem + uc % n_acc * a.R32, low = tmem + n_acc * a.R32;
        if (elect_one()) {
#pragma unroll
          for (int q = 0; q < 4; q++) umma_tf32(acc, dh + 2 * q, dw + 2 * q, id, uc >= n_acc || q != 0);
          if (F32) {
#pragma unroll
            for (int q = 0; q < 4; q++) umma_tf32(low, dl + 2 * q, dw + 2 * q, id, uc != 0 || q != 0);
          }
          umma_commit(empty(st));
          if (uc + 1 == nc) umma_commit(b_done);
        }
        __syncwarp();
      }
      next = begin(i + n_cl);
    }
    if (nc) ws.wait(b_done, tiles & 1);
    __syncwarp();
    tc_fence_after();
    // the block's sums, over the ring
    float *sums = reinterpret_cast<float *>(smem_raw + (base - smem_u32(smem_raw)));
    const int pitch = r32_now + 4;
    if (w < LR_WARPS)
      for (int c = (w >> 2) * 16; c < r32_now; c += 64) {
        float v[16];
        const int row = (w & 3) * 32 + lane, n_high = min(nc, n_acc);  // (the others are not written)
        const uint32_t t0 = tmem + ((uint32_t)((w & 3) * 32) << 16) + c;
#pragma unroll
        for (int e = 0; e < 16; e++) v[e] = 0.0f;
        for (int q = 0; q < n_high; q += 2) {
          float y[16], z[16];
          tmem_ld16x2(t0 + q * a.R32, t0 + min(q + 1, n_high - 1) * a.R32, y, z);
#pragma unroll
          for (int e = 0; e < 16; e++) v[e] += q + 1 < n_high ? y[e] + z[e] : y[e];
        }
        if (F32 && nc) {
          float y[16], z[16];
          tmem_ld16x2(t0 + n_acc * a.R32, t0 + n_acc * a.R32, y, z);
#pragma unroll
          for (int e = 0; e < 16; e++) v[e] = add_low(v[e], y[e]);
        }
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          *reinterpret_cast<float4 *>(sums + row * pitch + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
      }
    tc_fence_before();
    cluster_arrive();
    cluster_wait();
    // this block's rows of the cluster's sum
    const float scale = __int_as_float(tile.w);
    const int q4 = r32_now / 4, m0 = 128 * k / ks, m1 = 128 * (k + 1) / ks;
    for (int e = tid; e < (m1 - m0) * q4; e += LR_WARPS * 32 + 32) {
      const int row = m0 + e / q4, c = e % q4 * 4;
      if (row >= rows) continue;
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int b = 0; b < ks; b++) {
        const float4 o = remote_f32x4(smem_u32(sums + row * pitch + c), b);
        s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
      }
      // what lies past the rank may be 0 x infinity
      s.x = c < rank ? s.x * scale : 0.0f, s.y = c + 1 < rank ? s.y * scale : 0.0f;
      s.z = c + 2 < rank ? s.z * scale : 0.0f, s.w = c + 3 < rank ? s.w * scale : 0.0f;
      *reinterpret_cast<float4 *>(a.v + (long long)(tile.y + row) * a.R32 + c) = s;
    }
    cluster_arrive();
    cluster_wait();
    tc_fence_after();
    used += nc, tiles += nc != 0;
    i = next;
  }
  if (!ws.ok && lane == 0) raise_flag(a.err, DS4MOE_DEVERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (w == LR_WARPS) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---- y = base + B V, 128 tokens of a tile and 128 columns at a time; a block
// takes a run of them. Four warps bring V (split) and B (widened) chunk by chunk
// of 32 ranks into a ring and issue the products, into two accumulators in turn;
// sixteen add base, which they request an item ahead, and store y. Bound by the
// bytes of base and y.
constexpr int LE_STAGE = 3 * LR_HALF, LE_NST = 4, LE_FEED = 128, LE_THREADS = LE_FEED + 512;

template <int DT>
__global__ void __launch_bounds__(LE_THREADS, 1) k_adapt_expand(const AdaptArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[LE_NST + 4];
  __shared__ uint32_t s_tmem;
  const int tid = threadIdx.x, w = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t bar0 = smem_u32(s_bar);
  auto empty = [&](int i) { return bar0 + 8 * i; };
  auto acc_full = [&](int i) { return bar0 + 8 * (LE_NST + i); };
  auto acc_empty = [&](int i) { return bar0 + 8 * (LE_NST + 2 + i); };
  if (w == 0) {
    if (lane == 0) {
      for (int i = 0; i < LE_NST; i++) mbar_init(empty(i), 1);
      for (int i = 0; i < 2; i++) mbar_init(acc_full(i), 1), mbar_init(acc_empty(i), 16);
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(smem_u32(&s_tmem), 256);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  pdl_launch_dependents();
  pdl_wait();
  const int n_col = (a.N + 127) / 128;
  const long long total = (long long)*a.n_tiles * n_col;
  const long long i0 = total * blockIdx.x / gridDim.x, i1 = total * (blockIdx.x + 1) / gridDim.x;
  Waits ws;
  if (w < LE_FEED / 32) {
    const uint32_t id = idesc_tf32(128);
    int used = 0, accs = 0;
    uint4 v[8], wt[4];
    // the chunk of 32 ranks from c on of item i
    auto fetch = [&](const int4 &tile, int n0, int c) {
      const int rows = tile.z & 0xFFFF, r8 = ((tile.z >> 16) + 7) & ~7;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int r = tid / 8 + 16 * j;
        v[j] = make_uint4(0, 0, 0, 0);
        if (r < rows) v[j] = *reinterpret_cast<const uint4 *>(a.v + (long long)(tile.y + r) * a.R32 + c + tid % 8 * 4);
      }
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int r = tid / 4 + 32 * j, e = c + tid % 4 * 8;
        wt[j] = make_uint4(0, 0, 0, 0);
        if (n0 + r < a.N && e < r8) wt[j] = *reinterpret_cast<const uint4 *>(a.B + (long long)tile.x * a.b_slot + (long long)(n0 + r) * r8 + e);
      }
    };
    int at_tile = -1;
    int4 tile = make_int4(0, 0, 0, 0);
    auto load_tile = [&](long long i) {
      const int t = (int)(i / n_col);
      if (t != at_tile) at_tile = t, tile = a.tiles[t];
    };
    long long i = i0;
    int c = 0;
    auto skip = [&]() {  // to an item with products
      for (; i < i1; i++) {
        load_tile(i);
        if (tile.z >> 16) break;
        i = (long long)(at_tile + 1) * n_col - 1;  // (a tile without: all of its columns)
      }
    };
    skip();
    if (i < i1) fetch(tile, (int)(i % n_col) * 128, 0);
    while (i < i1) {
      const int r32 = ((tile.z >> 16) + 31) & ~31, buf = accs & 1, st = used % LE_NST;
      const bool first = c == 0, last = c + 32 >= r32;
      if (used >= LE_NST) ws.wait(empty(st), (used / LE_NST - 1) & 1);
      const uint32_t at = base + st * LE_STAGE;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const uint32_t o = sw128(tid / 8 + 16 * j, tid % 8);
        put_split<true>(at + o, at + LR_HALF + o, v[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; j++) put_wide<DT>(at + 2 * LR_HALF, tid / 4 + 32 * j, tid % 4, wt[j]);
      // the next chunk under way
      if (last) {
        i++, c = 0;
        skip();
      } else {
        c += 32;
      }
      if (i < i1) fetch(tile, (int)(i % n_col) * 128, c);
      if (first && accs >= 2) ws.wait(acc_empty(buf), (accs / 2 - 1) & 1);
      fence_proxy_async_smem();
      named_sync<LE_FEED>(1);
      if (w == 0) {
        const uint32_t sa = base + __shfl_sync(0xffffffffu, st, 0) * LE_STAGE, d = tmem + __shfl_sync(0xffffffffu, buf, 0) * 128;
        const uint64_t dh = desc_sw128(sa, 0), dl = desc_sw128(sa + LR_HALF, 0), dw = desc_sw128(sa + 2 * LR_HALF, 0);
        const uint32_t more = __shfl_sync(0xffffffffu, (int)!first, 0), ends = __shfl_sync(0xffffffffu, (int)last, 0);
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int q = 0; q < 4; q++) umma_tf32(d, dh + 2 * q, dw + 2 * q, id, more || q != 0);
#pragma unroll
          for (int q = 0; q < 4; q++) umma_tf32(d, dl + 2 * q, dw + 2 * q, id, 1);
          umma_commit(empty(st));
          if (ends) umma_commit(acc_full(buf));
        }
        __syncwarp();
      }
      used++, accs += last;
    }
    // nothing is in flight when the block leaves
    if (used) ws.wait(empty((used - 1) % LE_NST), ((used - 1) / LE_NST) & 1);
  } else {
    const int q = w & 3, g = (w - LE_FEED / 32) >> 2;  // the warp's quarter of the rows, of the columns
    const float *from = a.base ? a.base : a.y;
    const long long from_stride = a.base ? a.base_stride : a.y_stride;
    int at_tile = -1, tok = -1, accs = 0;
    int4 tile = make_int4(0, 0, 0, 0);
    // this lane's pieces of y: row (lane & 24) + j of the warp's 32, 16 bytes at
    // piece lane % 8 of its 32 columns
    float4 b[8];
    auto load = [&](long long i) {
      const int t = (int)(i / n_col), n = (int)(i % n_col) * 128 + 32 * g + 4 * (lane & 7);
      if (t != at_tile) {
        at_tile = t, tile = a.tiles[t];
        const int row = 32 * q + lane;
        tok = row < (tile.z & 0xFFFF) ? a.perm[tile.y + row] : -1;
      }
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int t_j = __shfl_sync(0xffffffffu, tok, (lane & 24) + j);
        b[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (t_j < 0) continue;
        const float *p = from + (long long)t_j * from_stride + n;
        if (a.wide) {
          if (n < a.N) b[j] = __ldcs(reinterpret_cast<const float4 *>(p));
        } else {
          if (n < a.N) b[j].x = p[0];
          if (n + 1 < a.N) b[j].y = p[1];
          if (n + 2 < a.N) b[j].z = p[2];
          if (n + 3 < a.N) b[j].w = p[3];
        }
      }
    };
    if (i0 < i1) load(i0);
    for (long long i = i0; i < i1; i++) {
      const int n = (int)(i % n_col) * 128 + 32 * g + 4 * (lane & 7), mine = tok;
      uint32_t u[32];
      if (tile.z >> 16) {
        const int buf = accs & 1;
        ws.wait(acc_full(buf), (accs / 2) & 1);
        __syncwarp();
        tc_fence_after();
        float v[32];
        tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + buf * 128 + 32 * g, v);
        tmem_wait_ld(v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty(buf));
        accs++;
#pragma unroll
        for (int e = 0; e < 32; e++) u[e] = __float_as_uint(v[e]);
        transpose8(u);
#pragma unroll
        for (int j = 0; j < 8; j++) {
          b[j].x += __uint_as_float(u[4 * j]), b[j].y += __uint_as_float(u[4 * j + 1]);
          b[j].z += __uint_as_float(u[4 * j + 2]), b[j].w += __uint_as_float(u[4 * j + 3]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int t_j = __shfl_sync(0xffffffffu, mine, (lane & 24) + j);
        if (t_j < 0) continue;
        float *p = a.y + (long long)t_j * a.y_stride + n;
        if (a.wide) {
          if (n < a.N) __stcs(reinterpret_cast<float4 *>(p), b[j]);
        } else {
          if (n < a.N) p[0] = b[j].x;
          if (n + 1 < a.N) p[1] = b[j].y;
          if (n + 2 < a.N) p[2] = b[j].z;
          if (n + 3 < a.N) p[3] = b[j].w;
        }
      }
      if (i + 1 < i1) load(i + 1);
    }
  }
  if (!ws.ok && lane == 0) raise_flag(a.err, DS4MOE_DEVERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (w == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// A slot's weights into its place: rows of A padded with zeros to r32, rows of B
// to r8.
__global__ void __launch_bounds__(256) k_adapt_set(const uint16_t *A, const uint16_t *B, int rank, float scale, int K, int N,
                                               uint16_t *dA, uint16_t *dB, int2 *info) {
  pdl_launch_dependents();
  pdl_wait();
  const long long r8 = (rank + 7) & ~7, r32 = (rank + 31) & ~31, na = r32 * K, n = na + (long long)N * r8;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    if (i < na) {
      dA[i] = i < (long long)rank * K ? A[i] : 0;
    } else {
      const long long row = (i - na) / r8, c = (i - na) % r8;
      dB[i - na] = c < rank ? B[row * rank + c] : 0;
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *info = make_int2(rank, __float_as_int(scale));
}

}  // namespace ds4

namespace {

using namespace ds4;

bool ap_dev_ptr(const void *p) {
  if (!p) return false;
  cudaPointerAttributes at;
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged;
}

ds4moe_status ap_status(cudaError_t e) {
  if (e == cudaSuccess) return DS4MOE_OK;
  cudaGetLastError();
  return e == cudaErrorMemoryAllocation ? DS4MOE_ERR_OOM : DS4MOE_ERR_CUDA;
}

struct AdaptFns {
  const void *token, *shrink, *expand;
};
template <int DT, bool F32>
AdaptFns fns_of(bool two) {
  return {(const void *)k_adapt_token<DT, F32>, two ? (const void *)k_adapt_shrink<DT, F32, 2> : (const void *)k_adapt_shrink<DT, F32, 1>,
          (const void *)k_adapt_expand<DT>};
}
AdaptFns adapt_fns(int dtype, bool f32, int r32) {
  constexpr int B = DS4MOE_DT_BF16, F = DS4MOE_DT_F16;
  const bool two = r32 > 128;
  return dtype == B ? f32 ? fns_of<B, true>(two) : fns_of<B, false>(two) : f32 ? fns_of<F, true>(two) : fns_of<F, false>(two);
}

cudaError_t launch_cluster(const void *fn, int grid, int cluster, int threads, size_t smem, cudaStream_t s, void **args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid), cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr, cfg.numAttrs = 2;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

bool rows_overlap(const void *p, long long n, const void *q, long long m) {
  const uintptr_t x = (uintptr_t)p, y = (uintptr_t)q;
  return x < y + (uintptr_t)m && y < x + (uintptr_t)n;
}

}  // namespace

extern "C" {

ds4moe_status ds4moe_adapters_create(int32_t n_out, int32_t n_in, int32_t n_slots, int32_t max_rank, int32_t dtype,
                                     int32_t max_tokens, ds4moe_adapters **out) {
  if (!out) return DS4MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (n_out < 1 || n_out > (1 << 24) || n_in < 32 || n_in > (1 << 16) || n_in % 32) return DS4MOE_ERR_INVALID_ARG;
  if (n_slots < 1 || max_rank < 1 || max_tokens < 1 || max_tokens > (1 << 16)) return DS4MOE_ERR_INVALID_ARG;
  if (dtype != DS4MOE_DT_BF16 && dtype != DS4MOE_DT_F16) return DS4MOE_ERR_INVALID_ARG;
  if (n_slots > LR_MAX_SLOTS || max_rank > LR_MAX_RANK) return DS4MOE_ERR_UNSUPPORTED;
  ds4moe_adapters *h = new (std::nothrow) ds4moe_adapters;
  if (!h) return DS4MOE_ERR_OOM;
  memset(h, 0, sizeof(*h));
  h->N = n_out, h->K = n_in, h->slots = n_slots, h->max_rank = max_rank, h->dtype = dtype, h->max_tokens = max_tokens;
  h->R32 = (max_rank + 31) & ~31, h->b_slot = (long long)n_out * ((max_rank + 7) & ~7);
  size_t at = 0;
  auto place = [&](size_t bytes) {
    const size_t p = at;
    at += (bytes + 255) & ~(size_t)255;
    return p;
  };
  const size_t o_err = place(64), o_info = place((size_t)n_slots * 8), zeroed = at;
  const size_t o_perm = place((size_t)max_tokens * 4), o_n = place(4);
  const size_t o_tiles = place(((size_t)max_tokens / 128 + std::min(n_slots + 1, max_tokens) + 1) * 16);
  const size_t o_v = place((size_t)max_tokens * h->R32 * 4);
  const size_t o_a = place((size_t)n_slots * h->R32 * n_in * 2), o_b = place((size_t)n_slots * h->b_slot * 2);
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->n_sm, cudaDevAttrMultiProcessorCount, h->device);
  for (bool f32 : {false, true}) {
    const AdaptFns f = adapt_fns(dtype, f32, h->R32);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f.token, cudaFuncAttributeMaxDynamicSharedMemorySize, ((1 << 16) / LR_CLUSTER + 8) * 4);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(f.shrink, cudaFuncAttributeMaxDynamicSharedMemorySize, LR_SMEM);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f.expand, cudaFuncAttributeMaxDynamicSharedMemorySize, LR_SMEM);
    for (int ks = 1; ks <= LR_CLUSTER && e == cudaSuccess; ks++) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      cfg.gridDim = dim3(ks), cfg.blockDim = dim3(LR_WARPS * 32 + 32), cfg.dynamicSmemBytes = LR_SMEM;
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = ks, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr, cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&h->clusters[ks], f.shrink, &cfg);
      if (e == cudaSuccess && h->clusters[ks] < 1) h->clusters[ks] = 1;
    }
  }
  if (e == cudaSuccess) e = cudaMalloc((void **)&h->mem, at);
  if (e == cudaSuccess) e = cudaMemsetAsync(h->mem, 0, zeroed, 0);
  if (e == cudaSuccess) e = cudaStreamSynchronize(0);
  if (e != cudaSuccess) {
    const ds4moe_status st = ap_status(e);
    if (h->mem) cudaFree(h->mem);
    cudaGetLastError();
    delete h;
    return st;
  }
  h->err = (uint32_t *)(h->mem + o_err), h->info = (int2 *)(h->mem + o_info), h->perm = (int *)(h->mem + o_perm);
  h->n_tiles = (int *)(h->mem + o_n), h->tiles = (int4 *)(h->mem + o_tiles), h->v = (float *)(h->mem + o_v);
  h->A = (uint16_t *)(h->mem + o_a), h->B = (uint16_t *)(h->mem + o_b);
  h->bytes = at;
  *out = h;
  return DS4MOE_OK;
}

void ds4moe_adapters_destroy(ds4moe_adapters *h) {
  if (!h) return;
  cudaDeviceSynchronize();
  cudaFree(h->mem);
  delete h;
}

ds4moe_status ds4moe_adapters_set(ds4moe_adapters *h, int32_t slot, int32_t rank, const void *A, const void *B,
                                  float scale, void *stream) {
  if (!h || slot < 0 || slot >= h->slots || rank < 0 || rank > h->max_rank) return DS4MOE_ERR_INVALID_ARG;
  if (rank && (!isfinite(scale) || !ap_dev_ptr(A) || !ap_dev_ptr(B) || ((uintptr_t)A & 1) || ((uintptr_t)B & 1)))
    return DS4MOE_ERR_INVALID_ARG;
  const uint16_t *pa = (const uint16_t *)A, *pb = (const uint16_t *)B;
  uint16_t *dA = h->A + (long long)slot * h->R32 * h->K, *dB = h->B + (long long)slot * h->b_slot;
  int2 *info = h->info + slot;
  void *args[] = {&pa, &pb, &rank, &scale, &h->K, &h->N, &dA, &dB, &info};
  const long long n = (long long)((rank + 31) & ~31) * h->K + (long long)h->N * ((rank + 7) & ~7);
  const int grid = (int)std::min<long long>((n + 255) / 256 + 1, 8 * h->n_sm);
  const cudaError_t e = launch_pdl((const void *)k_adapt_set, dim3(grid), dim3(256), 0, (cudaStream_t)stream, args, true);
  h->launches++;
  return ap_status(e);
}

ds4moe_status ds4moe_adapters_forward(ds4moe_adapters *h, const void *x, int64_t x_stride, int32_t x_dtype,
                                      const int32_t *slots, int32_t n_tok, const float *base, int64_t base_stride,
                                      float *y, int64_t y_stride, void *stream) {
  if (!h || n_tok < 0 || n_tok > h->max_tokens) return DS4MOE_ERR_INVALID_ARG;
  if (x_dtype != DS4MOE_DT_F32 && x_dtype != h->dtype) return DS4MOE_ERR_INVALID_ARG;
  if (n_tok == 0) return DS4MOE_OK;
  const bool f32 = x_dtype == DS4MOE_DT_F32;
  const long long K = h->K, N = h->N, lim = 1ll << 39;
  if (n_tok == 1) x_stride = K, base_stride = y_stride = N;
  if (x_stride < K || x_stride >= lim || x_stride % (f32 ? 4 : 8) || ((uintptr_t)x & 15)) return DS4MOE_ERR_INVALID_ARG;
  if (y_stride < N || y_stride >= lim || ((uintptr_t)y & 3)) return DS4MOE_ERR_INVALID_ARG;
  if (base && (base_stride < N || base_stride >= lim || ((uintptr_t)base & 3))) return DS4MOE_ERR_INVALID_ARG;
  if (!ap_dev_ptr(x) || !ap_dev_ptr(slots) || !ap_dev_ptr(y) || (base && !ap_dev_ptr(base))) return DS4MOE_ERR_INVALID_ARG;
  const long long n = n_tok - 1, y_bytes = (n * y_stride + N) * 4;
  if (rows_overlap(y, y_bytes, x, (n * x_stride + K) * (f32 ? 4 : 2))) return DS4MOE_ERR_INVALID_ARG;
  if (base == y && base_stride == y_stride) base = nullptr;
  if (base && rows_overlap(y, y_bytes, base, (n * base_stride + N) * 4)) return DS4MOE_ERR_INVALID_ARG;
  AdaptArgs a = {};
  a.N = h->N, a.K = h->K, a.slots = h->slots, a.T = n_tok, a.R32 = h->R32, a.b_slot = h->b_slot;
  a.x = x, a.x_stride = x_stride, a.base = base, a.base_stride = base_stride, a.y = y, a.y_stride = y_stride;
  a.slot_of = slots, a.info = h->info, a.A = h->A, a.B = h->B;
  a.perm = h->perm, a.tiles = h->tiles, a.n_tiles = h->n_tiles, a.v = h->v, a.err = h->err;
  a.wide = N % 4 == 0 && y_stride % 4 == 0 && !((uintptr_t)y & 15) && (!base || (base_stride % 4 == 0 && !((uintptr_t)base & 15)));
  const AdaptFns f = adapt_fns(h->dtype, f32, h->R32);
  const cudaStream_t s = (cudaStream_t)stream;
  if (n_tok <= LR_TOKENS) {
    void *args[] = {&a};
    const cudaError_t e = launch_cluster(f.token, LR_CLUSTER * n_tok, LR_CLUSTER, 256, (size_t)(K / 8 / LR_CLUSTER + 1) * 32, s, args);
    h->launches++;
    return ap_status(e);
  }
  void *plan[] = {&a};
  cudaError_t e = launch_pdl((const void *)k_adapt_plan, dim3(1), dim3(1024), 0, s, plan, true);
  if (e == cudaSuccess) {
    // Blocks of a tile: the fewest chunks of 32 columns one after another, six
    // more for a tile's start and sum, with some tiles that are not full; and
    // chains of additions that stay exact (11 chunks per accumulator, see k_adapt_shrink).
    const int most = n_tok / 128 + std::min(h->slots + 1, n_tok) + 1, full = n_tok / 128 + 1, guess = full + std::min(h->slots, full) / 2;
    const int n_acc = shrink_accs(h->R32) - (f32 ? 1 : 0);
    int ks = LR_CLUSTER;
    long long best = -1;
    for (int c = LR_CLUSTER; c >= 1; c--) {
      const long long chunks = (K / 32 + c - 1) / c, cost = (guess + h->clusters[c] - 1) / h->clusters[c] * (chunks + 6);
      if (best < 0 || (cost < best && chunks <= 11 * n_acc)) best = cost, ks = c;
    }
    const int grid = std::min(h->clusters[ks], most) * ks;
    void *args[] = {&a, &ks};
    e = launch_cluster(f.shrink, grid, ks, LR_WARPS * 32 + 32, LR_SMEM, s, args);
    if (e == cudaSuccess) {
      const long long items = (long long)most * ((N + 127) / 128);
      e = launch_pdl(f.expand, dim3((unsigned)std::min<long long>(items, h->n_sm)), dim3(LE_THREADS), LR_SMEM, s, plan, true);
    }
  }
  h->launches += 3;
  return ap_status(e);
}

ds4moe_status ds4moe_adapters_get_device_error(ds4moe_adapters *h, void *stream, uint32_t *flags_out) {
  if (!h) return DS4MOE_ERR_INVALID_ARG;
  uint32_t f = 0;
  cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaMemcpy(&f, h->err, 4, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(h->err, 0, 4);
  if (e != cudaSuccess) return ap_status(e);
  if (flags_out) *flags_out = f;
  return f ? DS4MOE_ERR_DEVICE : DS4MOE_OK;
}

uint64_t ds4moe_adapters_device_bytes(const ds4moe_adapters *h) { return h ? h->bytes : 0; }
uint64_t ds4moe_adapters_launch_count(const ds4moe_adapters *h) { return h ? h->launches : 0; }

}  // extern "C"
