// adapters.cu -- low-rank adapters of many requests beside a shared projection:
//   y[t] = base[t] + scale_s B_s (A_s x[t]),  s = slots[t]  (no adapter: base[t]).
//
// A_s is [rank][n_in], B_s [n_out][rank] in 16 bits, x, base and y rows of tokens.
// Sums are in 32 bits, A x stays in 32 bits between the two products.
//
// Few tokens (choose_way): k_adapt_token, a cluster of eight blocks per token,
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
#include <type_traits>

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
  int *n_tiles;      // then, for calls that decide on the device: whether they go token by token, tokens given out
  float *v;          // [max_tokens][R32] scale A x by place in perm
  int path;          // ds4moe_adapters_debug_path
  int clusters[17];  // clusters of so many blocks of k_adapt_shrink that run at once
  int token_clusters[2];  // clusters of k_adapt_token that run at once, by the type of x
  uint64_t bytes, launches;
};

namespace ds4 {

constexpr int LR_CLUSTER = 8;
constexpr int LR_MAX_RANK = 256, LR_MAX_SLOTS = 4096;

struct AdaptArgs {
  int N, K, slots, T, R32;
  int x_stride, y_stride, base_stride;
  long long b_slot;
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
  int most;  // tiles above which the call goes token by token (k_adapt_plan decides), or 0: by tiles
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
__device__ __forceinline__ void remote_store(uint32_t addr, int rank, int v) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(r), "r"(v) : "memory");
}
__device__ __forceinline__ float4 remote_f32x4(uint32_t addr, int rank) {
  uint32_t r;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(r) : "memory");
  return v;
}

// Asks L2 for `bytes` from p on (multiples of 16).
__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
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

// (four blocks per SM: all of 64 tokens' blocks run at once) LOOP: if k_adapt_plan
// has decided so, by as many clusters as run at once.
template <int DT, bool F32, bool LOOP>
__global__ void __launch_bounds__(256, 4) k_adapt_token(const AdaptArgs a) {
  extern __shared__ __align__(16) float s_x[];  // this block's columns of x
  __shared__ float s_part[LR_MAX_RANK];
  __shared__ __align__(16) float s_v[LR_MAX_RANK];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, c = (int)cluster_rank();
  int t = blockIdx.x / LR_CLUSTER, turn = 0;
  __shared__ int s_then[2];  // LOOP: the cluster's next token, from its first block, in turns
  pdl_launch_dependents();
  pdl_wait();
  if (LOOP && !a.n_tiles[1]) return;
  // Tokens go to clusters as they come free (dealt out ahead: 1000 adapters of rank
  // 64, 1000 tokens 339 us instead of 286). A block writes a buffer that another
  // token's values were in when all who read them have passed a barrier since.
  do {
    // Loads that do not wait for one another go first: the slot's own chain (slot,
    // rank, weights) runs beside x's.
    bool bad = false;
    const int s = slot_at(a, t, bad);
    if (LOOP && c == 0 && tid < LR_CLUSTER) {
      int then = 0;
      if (tid == 0) then = gridDim.x / LR_CLUSTER + atomicAdd(a.n_tiles + 2, 1);
      remote_store(smem_u32(s_then + turn), tid, __shfl_sync((1 << LR_CLUSTER) - 1, then, 0));
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
    if (bad && c == 0 && tid == 0) raise_flag(a.err, DS4MOE_DEVERR_ADAPTER);
    const int2 in = s >= 0 ? a.info[s] : make_int2(0, 0);
    const int rank = in.x;
    const int n0 = (int)((long long)a.N * c / LR_CLUSTER), n1 = (int)((long long)a.N * (c + 1) / LR_CLUSTER);
    const float *base = a.base ? a.base + (long long)t * a.base_stride : a.y + (long long)t * a.y_stride;
    float *y = a.y + (long long)t * a.y_stride;
    if (rank == 0) {  // (the same for all blocks of the cluster)
      if (a.base)
        for (int n = n0 + tid; n < n1; n += 256) y[n] = base[n];
      if (LOOP) {
        cluster_arrive();
        cluster_wait();
      }
      continue;
    }
    const int r8 = (rank + 7) & ~7;
    const uint16_t *A = a.A + (long long)s * a.R32 * a.K, *B = a.B + (long long)s * a.b_slot;
    if (tid == 0) {  // this block's part of B on its way
      const uint32_t bytes = (uint32_t)min((long long)(n1 - n0) * r8 * 2, 1ll << 20);
      if (bytes) prefetch_l2(B + (long long)n0 * r8, bytes);
    }
    // J rows of A per warp at a time (rows past the rank are zeros up to a multiple
    // of 32); the first pieces are requested before x is waited for
    auto rows_of_a = [&](auto per_warp) {
      constexpr int J = decltype(per_warp)::value;
      const uint4 *p = reinterpret_cast<const uint4 *>(A + (long long)(J * w) * a.K) + u0;
      const long long row = a.K / 8;
      uint4 first[J];
#pragma unroll
      for (int j = 0; j < J; j++) {
        first[j] = make_uint4(0, 0, 0, 0);
        if (J * w < rank && lane < nu) first[j] = p[j * row + lane];
      }
      __syncthreads();
      auto add = [&](const uint4 (&wt)[J], int u, float (&sum)[J]) {
        float x[8];
        *reinterpret_cast<float4 *>(x) = reinterpret_cast<const float4 *>(s_x)[2 * u];
        *reinterpret_cast<float4 *>(x + 4) = reinterpret_cast<const float4 *>(s_x)[2 * u + 1];
#pragma unroll
        for (int j = 0; j < J; j++) sum[j] = dot8<DT>(wt[j], x, sum[j]);
      };
      for (int r0 = J * w; r0 < rank; r0 += 8 * J, p += 8 * J * row) {
        float sum[J] = {};
        int u = lane;
        if (r0 == J * w) {
          if (u < nu) add(first, u, sum);
          u += 32;
        }
#pragma unroll 2
        for (; u < nu; u += 32) {
          uint4 wt[J];
#pragma unroll
          for (int j = 0; j < J; j++) wt[j] = p[j * row + u];
          add(wt, u, sum);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
#pragma unroll
          for (int j = 0; j < J; j++) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
        if (lane == 0) {
#pragma unroll
          for (int j = 0; j < J; j++) s_part[r0 + j] = sum[j];
        }
      }
    };
    if (rank <= 16) rows_of_a(std::integral_constant<int, 2>());
    else rows_of_a(std::integral_constant<int, 4>());
    cluster_arrive();
    const float scale = __int_as_float(in.y);
    // U lanes per row of B, so that a load takes whole lines: the lane's piece of
    // eight ranks is the same for all rows. A warp takes 32 rows, 32 / U at a time,
    // of which lane l ends up with row (l % U) * (32 / U) + l / U. The first pieces
    // are requested before the other blocks' sums are waited for.
    const int units = r8 / 8;
    auto rows_of_b = [&](auto lanes) {
      constexpr int U = decltype(lanes)::value, G = 32 / U, H = U < 4 ? U : 4;
      const int u = lane % U, g = lane / U;
      uint4 wt[H];
      auto request = [&](int r0, int b) {
#pragma unroll
        for (int k = 0; k < H; k++) {
          const int n = r0 + (b + k) * G + g;
          wt[k] = make_uint4(0, 0, 0, 0);
          if (n < n1 && u < units) wt[k] = *reinterpret_cast<const uint4 *>(B + (long long)n * r8 + 8 * u);
        }
      };
      int r0 = n0 + 32 * w;
      float from = r0 + u * G + g < n1 ? base[r0 + u * G + g] : 0.0f;
      request(r0, 0);
      cluster_wait();
      if (tid < r8) {
        float v = 0.0f;
        if (tid < rank)
#pragma unroll
          for (int i = 0; i < LR_CLUSTER; i++) v += remote_f32(smem_u32(s_part + tid), i);
        s_v[tid] = v * scale;
      }
      __syncthreads();
      cluster_arrive();  // the others' sums are read: they may leave
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; e++) v[e] = u < units ? s_v[8 * u + e] : 0.0f;
      for (; r0 < n1; r0 += 256) {
        const int mine = r0 + u * G + g;
        float keep = 0.0f;
#pragma unroll
        for (int b = 0; b < U; b += H) {
#pragma unroll
          for (int k = 0; k < H; k++) {
            float sum = dot8<DT>(wt[k], v, 0.0f);
#pragma unroll
            for (int o = U / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (b + k == u) keep = sum;
          }
          if (b + H < U) request(r0, b + H);
          else if (r0 + 256 < n1) request(r0 + 256, 0);
        }
        if (mine < n1) y[mine] = from + keep;
        from = mine + 256 < n1 ? base[mine + 256] : 0.0f;
      }
    };
    if (units == 1) rows_of_b(std::integral_constant<int, 1>());
    else if (units == 2) rows_of_b(std::integral_constant<int, 2>());
    else if (units <= 4) rows_of_b(std::integral_constant<int, 4>());
    else if (units <= 8) rows_of_b(std::integral_constant<int, 8>());
    else if (units <= 16) rows_of_b(std::integral_constant<int, 16>());
    else rows_of_b(std::integral_constant<int, 32>());
    cluster_wait();
  } while (LOOP && (t = s_then[turn], turn ^= 1, t < a.T));
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
  if (tid == 1023) {
    const bool tokens = a.most && t0 > a.most;
    a.n_tiles[0] = tokens ? 0 : t0, a.n_tiles[1] = tokens, a.n_tiles[2] = 0;
  }
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
// the 11 bits of a tf32 number (an error of 2^-20 of x at most). The products
// leave the low 13 bits of a word out themselves. For an
// infinity lo is NaN, and a lo of 0 is NaN times an infinite weight. So either sums
// whose high part is not finite leave the low part out (add_low), or (INF) lo is
// never one of these: infinite as x is, and 2^-30 of x for 0, which gives the low
// sum the infinities of the high one (add_low there: 6 of the prompts' 103 us).
template <bool INF>
__device__ __forceinline__ void put_split(uint32_t hi_at, uint32_t lo_at, const uint4 &x) {
  auto rest = [](uint32_t v) {
    const float f = __uint_as_float(v), d = f - __uint_as_float(v & 0xFFFFE000u);
    if (!INF) return __float_as_uint(d);
    return isinf(f) ? v : __float_as_uint(d == 0.0f ? f * 0x1p-30f : d);
  };
  sts4(hi_at, x.x, x.y, x.z, x.w);
  sts4(lo_at, rest(x.x), rest(x.y), rest(x.z), rest(x.w));
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
// takes a part of the columns, in chunks of CH * 32. Two groups of four warps take
// the chunks in turn: they split x (and widen A) on the way from registers, where
// the group's next chunk is under way, to a ring in shared memory; one warp
// issues the products. What bounds it is issuing that work: sixteen warps that
// all took a part of every chunk of 32 columns passed too many barriers and proxy
// fences (73 us for the prompts of 6.6 thousand tokens; groups of them 57).
//
// The tensor cores add a product to an accumulator with the sum cut, not rounded,
// to 24 bits, so a long chain of additions drifts: 256 of them (1024 columns)
// were off by 4e-6 of the result, five times what 32-bit sums are. So chunks go
// round several accumulators, the low parts of x to one of their own, added up
// in 32 bits at the end. Where the accumulators that there is room for would take
// more than 37 additions each (fp32 inputs: ranks of 161 to 256 from 4128 columns on,
// of 128 from 12320, up to 64 from 28704; 16-bit ones, which need no accumulator for
// low parts: 8224, 16416, 32800), a block takes its columns in `passes`, whose sums
// meet in 32 bits in V. Measured, error of the result and time of 4096 tokens, in one
// pass and so: rank 256, 8192 columns and 8192 outputs 1.8e-6 322 us, 1.2e-6 367 us;
// 65536 columns and 512 outputs 1.0e-5 729 us, 1.2e-6 1512 us.
constexpr int LR_WARPS = 8, LR_GROUPS = 2, LR_FEED = LR_WARPS * 32 / LR_GROUPS;
// 32-column parts of a chunk: two, while two stages of them fit.
__host__ __device__ constexpr int shrink_ch(int r32) { return r32 <= 128 ? 2 : 1; }
// A part: the high numbers of x, the low ones (fp32), the rows of A.
__host__ __device__ constexpr int shrink_part(bool f32, int r32) { return LR_HALF * (f32 ? 2 : 1) + r32 * 128; }
__host__ __device__ constexpr int shrink_stage(bool f32, int r32) { return shrink_ch(r32) * shrink_part(f32, r32); }
__host__ __device__ constexpr int shrink_stages(bool f32, int r32) {
  const int n = (LR_SMEM - 1024) / shrink_stage(f32, r32);
  return n < 6 ? n : 6;  // (two at least)
}
__host__ __device__ constexpr int shrink_accs(int r32) { return 512 / r32 < 8 ? 512 / r32 : 8; }

// WP: 16-byte pieces of A per thread and part, a 32nd of the largest rank. MANY:
// more than one pass (of its own: the others' registers are all in use).
template <int DT, bool F32, int WP, bool MANY>
__global__ void __launch_bounds__(LR_WARPS * 32 + 32, 1) k_adapt_shrink(const AdaptArgs a, int ks, int n_passes) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[2 * 6 + 1];
  __shared__ uint32_t s_tmem;
  constexpr int CH = shrink_ch(WP * 32);
  const int tid = threadIdx.x, w = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const int part_bytes = shrink_part(F32, a.R32), nst = shrink_stages(F32, a.R32);
  const uint32_t bar0 = smem_u32(s_bar);
  auto full = [&](int i) { return bar0 + 8 * i; };
  auto empty = [&](int i) { return bar0 + 8 * (6 + i); };
  const uint32_t b_done = bar0 + 8 * 12;
  if (w == LR_WARPS) {
    if (lane == 0) {
      for (int i = 0; i < 6; i++) mbar_init(full(i), LR_FEED / 32), mbar_init(empty(i), 1);
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
  // this block's parts of 32 columns; those of a pass, and its chunks
  const int all0 = (a.K / 32) * k / ks, all = (a.K / 32) * (k + 1) / ks - all0;
  const int passes = MANY ? n_passes : 1;
  int p0, np, nc;
  auto set_pass = [&](int r) {
    const int from = all * r / passes;
    p0 = all0 + from, np = all * (r + 1) / passes - from, nc = (np + CH - 1) / CH;
  };
  set_pass(0);
  // accumulators of the high parts; the low parts' one comes after them
  const int n_acc = shrink_accs(a.R32) - (F32 ? 1 : 0);
  Waits ws;
  constexpr int PR = F32 ? 8 : 4, XP = 128 * PR / LR_FEED;  // 16-byte pieces of a row's part of x; of a thread
  const int ft = tid & (LR_FEED - 1), group = tid / LR_FEED;
  uint4 x[CH][XP], wt[CH][WP];
  int tok[XP];
  const uint16_t *ap;
  int r32 = 0;
  // the next tile with a rank, from i on, pass r of it, and this thread's part of that
  auto begin = [&](int i, int r) {
    int4 tile = make_int4(0, 0, 0, 0);
    if (MANY) set_pass(r);
    for (; i < n_tiles; i += n_cl) {
      tile = a.tiles[i];
      if (tile.z >> 16) break;
    }
    if (i >= n_tiles || w == LR_WARPS) return i;
    r32 = ((tile.z >> 16) + 31) & ~31;
#pragma unroll
    for (int j = 0; j < XP; j++) {
      const int r = ft / PR + j * (LR_FEED / PR);
      tok[j] = a.perm[tile.y + min(r, (tile.z & 0xFFFF) - 1)];  // (rows past the last are not stored)
    }
    ap = a.A + ((long long)tile.x * a.R32 + ft / 4) * a.K + p0 * 32 + ft % 4 * 8;
    return i;
  };
  auto fetch = [&](int c) {
    const char *p = (const char *)a.x + (p0 + c * CH) * (F32 ? 128 : 64) + ft % PR * 16;
    const bool two = c * CH + 1 < np;
    if (c * CH >= np) return;
#pragma unroll
    for (int j = 0; j < XP; j++) {
      const char *row = p + (long long)tok[j] * (a.x_stride * (F32 ? 4ll : 2ll));
      x[0][j] = __ldcs(reinterpret_cast<const uint4 *>(row));
      if (CH == 2 && two) x[CH - 1][j] = __ldcs(reinterpret_cast<const uint4 *>(row + (F32 ? 128 : 64)));
    }
#pragma unroll
    for (int j = 0; j < WP; j++)
      if (32 * j + ft / 4 < r32) {
        const uint16_t *row = ap + (long long)32 * j * a.K + c * CH * 32;
        wt[0][j] = *reinterpret_cast<const uint4 *>(row);
        if (CH == 2 && two) wt[CH - 1][j] = *reinterpret_cast<const uint4 *>(row + 32);
      }
  };
  // Rows of x lie far apart and a chunk takes 128 bytes or two of each: the rows'
  // next SPAN chunks are asked for at once, SPAN to 2 SPAN chunks ahead (thread: row).
  constexpr int SPAN = 8 / CH, CHUNK = CH * (F32 ? 128 : 64);
  const char *row_x = nullptr;
  auto ask = [&](int c) {
    if (row_x && c < nc) prefetch_l2(row_x + (long long)c * CHUNK, (uint32_t)min(SPAN * CHUNK, (np - c * CH) * (CHUNK / CH)));
  };
  auto ask_first = [&](int i) {
    const int4 tile = a.tiles[i];
    row_x = nullptr;
    if (tid < (tile.z & 0xFFFF)) row_x = (const char *)a.x + ((long long)a.perm[tile.y + tid] * a.x_stride + p0 * 32) * (F32 ? 4 : 2);
    ask(0), ask(SPAN);
  };
  // the ring: stage and lap of the warp's next chunk (of the group's, or of the products')
  int st = 0, lap = 0;
  auto advance = [&](int n) {
    for (st += n; st >= nst; st -= nst) lap++;
    for (; st < 0; st += nst) lap--;
  };
  int tiles = 0;
  int i = begin(blockIdx.x / ks, 0), pass = 0;
  if (w < LR_WARPS) {
    if (i < n_tiles) {
      if (group == 0) ask_first(i);
      fetch(group);
    }
    advance(group);
  }
  while (i < n_tiles) {
    const int4 tile = a.tiles[i];
    const int rank = tile.z >> 16, rows = tile.z & 0xFFFF, r32_now = (rank + 31) & ~31;
    const int np_now = np, nc_now = nc;
    const bool again = MANY && pass + 1 < passes;  // the tile's next pass follows
    int next;
    if (w < LR_WARPS) {
      int c = group;
      for (; c < nc; c += LR_GROUPS, advance(LR_GROUPS)) {
        if (group == 0 && c % SPAN == 0) ask(c + 2 * SPAN);
        if (lap > 0) ws.wait(empty(st), (lap - 1) & 1);
#pragma unroll
        for (int h = 0; h < CH; h++) {
          if (c * CH + h >= np) break;
          const uint32_t at = base + (st * CH + h) * part_bytes, wa = at + LR_HALF * (F32 ? 2 : 1);
#pragma unroll
          for (int p = 0; p < XP; p++) {
            const int r = ft / PR + p * (LR_FEED / PR);
            if (F32) {
              const uint32_t o = sw128(r, ft % PR);
              put_split<false>(at + o, at + LR_HALF + o, x[h][p]);
            } else {
              put_wide<DT>(at, r, ft % PR, x[h][p]);
            }
          }
#pragma unroll
          for (int p = 0; p < WP; p++)
            if (32 * p + ft / 4 < r32_now) put_wide<DT>(wa, 32 * p + ft / 4, ft % 4, wt[h][p]);
        }
        fetch(c + LR_GROUPS);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full(st));
      }
      advance(nc + group - c);  // all warps' chunks follow on the tile's nc chunks
      // the next tile's (or pass's) first chunks come in while this one is added up
      next = begin(again ? i : i + n_cl, again ? pass + 1 : 0);
      if (next < n_tiles) {
        if (group == 0) ask_first(next);
        fetch(group);
      }
    } else {
      const uint32_t id = idesc_tf32(__shfl_sync(0xffffffffu, r32_now, 0));
      for (int c = 0; c < nc; c++, advance(1)) {
        const int uc = __shfl_sync(0xffffffffu, c, 0), us = __shfl_sync(0xffffffffu, st, 0);
        ws.wait(full(us), lap & 1);
        __syncwarp();
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < CH; h++) {
            const int part = uc * CH + h;
            if (part >= np) break;
            const uint32_t sa = base + (us * CH + h) * part_bytes;
            const uint64_t dh = desc_sw128(sa, 0), dl = desc_sw128(sa + LR_HALF, 0), dw = desc_sw128(sa + LR_HALF * (F32 ? 2 : 1), 0);
            const uint32_t acc = tmem + part % n_acc * a.R32, low = tmem + n_acc * a.R32;
#pragma unroll
            for (int q = 0; q < 4; q++) umma_tf32(acc, dh + 2 * q, dw + 2 * q, id, part >= n_acc || q != 0);
            if (F32) {
#pragma unroll
              for (int q = 0; q < 4; q++) umma_tf32(low, dl + 2 * q, dw + 2 * q, id, part != 0 || q != 0);
            }
          }
          umma_commit(empty(us));
          if (uc + 1 == nc) umma_commit(b_done);
        }
        __syncwarp();
      }
      next = begin(again ? i : i + n_cl, again ? pass + 1 : 0);
    }
    if (nc_now) ws.wait(b_done, tiles & 1);
    __syncwarp();
    tc_fence_after();
    // the block's sums, over the ring
    float *sums = reinterpret_cast<float *>(smem_raw + (base - smem_u32(smem_raw)));
    const int pitch = r32_now + 4;
    if (w < LR_WARPS)
      for (int c = (w >> 2) * 16; c < r32_now; c += 32) {
        float v[16];
        const int row = (w & 3) * 32 + lane, n_high = min(np_now, n_acc);  // (the others are not written)
        const uint32_t t0 = tmem + ((uint32_t)((w & 3) * 32) << 16) + c;
#pragma unroll
        for (int e = 0; e < 16; e++) v[e] = 0.0f;
        for (int q = 0; q < n_high; q += 2) {
          float y[16], z[16];
          tmem_ld16x2(t0 + q * a.R32, t0 + min(q + 1, n_high - 1) * a.R32, y, z);
#pragma unroll
          for (int e = 0; e < 16; e++) v[e] += q + 1 < n_high ? y[e] + z[e] : y[e];
        }
        if (F32 && nc_now) {
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
      const int row = m0 + e / q4, c = (e - (row - m0) * q4) * 4;
      if (row >= rows) continue;
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int b = 0; b < ks; b++) {
        const float4 o = remote_f32x4(smem_u32(sums + row * pitch + c), b);
        s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
      }
      // what lies past the rank may be 0 x infinity
      s.x = c < rank ? s.x * scale : 0.0f, s.y = c + 1 < rank ? s.y * scale : 0.0f;
      s.z = c + 2 < rank ? s.z * scale : 0.0f, s.w = c + 3 < rank ? s.w * scale : 0.0f;
      float4 *v = reinterpret_cast<float4 *>(a.v + (long long)(tile.y + row) * a.R32 + c);
      if (MANY && pass) {  // (this thread stored the passes before)
        const float4 o = *v;
        s.x += o.x, s.y += o.y, s.z += o.z, s.w += o.w;
      }
      *v = s;
    }
    cluster_arrive();
    cluster_wait();
    tc_fence_after();
    tiles += nc_now != 0;
    i = next, pass = again ? pass + 1 : 0;
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
// takes a run of them. Four warps bring B (widened) into a ring, by 64 ranks, and
// V (split), which stays for all columns of a tile, and issue the products, into
// two pairs of accumulators (high and low parts) in turn; sixteen add base, which they request an item ahead,
// and store y. Base comes through shared memory where that has room (ranks up to
// 64), so that an item's is under way all the time that the one before it takes,
// not only after its stores (57 -> 52 us). Bound by the bytes of base and y. Ranks
// above 128 leave no room for
// V: there (not KEEP) the ring has it too, by 32 ranks. (So for all ranks, the
// four warps were what bound it: 64 us for the prompts of 6.6 thousand tokens.)
constexpr int LE_STAGE = 3 * LR_HALF, LE_NST = 4, LE_FEED = 128, LE_THREADS = LE_FEED + 512;

template <int DT, bool KEEP>
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
    tmem_alloc(smem_u32(&s_tmem), 512);
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
  const int t0 = (int)(i0 / n_col), c0 = (int)(i0 - (long long)t0 * n_col);
  Waits ws;
  if (w < LE_FEED / 32) {
    const uint32_t id = idesc_tf32(128);
    // KEEP: V, 32 ranks of it after another (high, low), then stages of two parts of B
    const uint32_t ring = KEEP ? base + a.R32 / 32 * (2 * LR_HALF) : base;
    const int nst = KEEP ? 2 : LE_NST;
    constexpr int STEP = KEEP ? 64 : 32, PARTS = STEP / 32, STAGE = KEEP ? 2 * LR_HALF : LE_STAGE;
    int used = 0, accs = 0, st = 0, lap = 0;
    uint4 v[8], wt[PARTS][4];
    auto fetch_v = [&](const int4 &tile, int c) {
      const int rows = tile.z & 0xFFFF;
      const float *p = a.v + (long long)tile.y * a.R32 + c + tid % 8 * 4;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        v[j] = make_uint4(0, 0, 0, 0);
        if (tid / 8 + 16 * j < rows) v[j] = *reinterpret_cast<const uint4 *>(p + (tid / 8 + 16 * j) * a.R32);
      }
    };
    auto put_v = [&](uint32_t at) {
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const uint32_t o = sw128(tid / 8 + 16 * j, tid % 8);
        put_split<true>(at + o, at + LR_HALF + o, v[j]);
      }
    };
    // STEP ranks from c on of B's rows
    auto fetch = [&](const int4 &tile, int n0, int c) {
      const int r8 = ((tile.z >> 16) + 7) & ~7;
      const uint16_t *p = a.B + (long long)tile.x * a.b_slot + (long long)(n0 + tid / 4) * r8 + c + tid % 4 * 8;
#pragma unroll
      for (int h = 0; h < PARTS; h++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          wt[h][j] = make_uint4(0, 0, 0, 0);
          if (n0 + tid / 4 + 32 * j < a.N && c + 32 * h + tid % 4 * 8 < r8)
            wt[h][j] = *reinterpret_cast<const uint4 *>(p + (long long)32 * j * r8 + 32 * h);
        }
      if (!KEEP) fetch_v(tile, c);
    };
    int t = t0, col = c0, c = 0, kept = -1;  // tile, its part of the columns, of its ranks; the tile whose V is kept
    long long i = i0;
    int4 tile = make_int4(0, 0, 0, 0);
    if (i < i1) tile = a.tiles[t];
    auto skip = [&]() {  // to an item with products
      while (i < i1 && (col == n_col || !(tile.z >> 16))) {
        i += n_col - col, col = 0;  // (a tile without: all of its columns)
        if (i < i1) tile = a.tiles[++t];
      }
    };
    skip();
    if (i < i1) fetch(tile, col * 128, 0);
    while (i < i1) {
      const int r32 = ((tile.z >> 16) + 31) & ~31, buf = accs & 1, c_now = c;
      const bool first = c == 0, last = c + STEP >= r32;
      if (KEEP && t != kept) {
        // the products with the last tile's V are done
        if (used) ws.wait(empty(st == 0 ? nst - 1 : st - 1), (st == 0 ? lap - 1 : lap) & 1);
        for (int e = 0; e < r32; e += 32) {
          fetch_v(tile, e);
          put_v(base + e / 32 * (2 * LR_HALF));
        }
        kept = t;
      }
      if (lap > 0) ws.wait(empty(st), (lap - 1) & 1);
      const uint32_t at = ring + st * STAGE;
      if (!KEEP) put_v(at);
#pragma unroll
      for (int h = 0; h < PARTS; h++)
#pragma unroll
        for (int j = 0; j < 4; j++) put_wide<DT>(at + (KEEP ? h : 2) * LR_HALF, tid / 4 + 32 * j, tid % 4, wt[h][j]);
      // the next chunk under way
      if (last) {
        i++, col++, c = 0;
        skip();
      } else {
        c += STEP;
      }
      if (i < i1) fetch(tile, col * 128, c);
      if (first && accs >= 2) ws.wait(acc_empty(buf), (accs / 2 - 1) & 1);
      fence_proxy_async_smem();
      named_sync<LE_FEED>(1);
      if (w == 0) {
        const int us = __shfl_sync(0xffffffffu, st, 0), uc = __shfl_sync(0xffffffffu, c_now, 0), ur = __shfl_sync(0xffffffffu, r32, 0);
        const uint32_t sa = ring + us * STAGE, d = tmem + __shfl_sync(0xffffffffu, buf, 0) * 128;
        const uint32_t ends = __shfl_sync(0xffffffffu, (int)last, 0);
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < PARTS; h++) {
            if (uc + 32 * h >= ur) break;
            const uint32_t va = KEEP ? base + (uc / 32 + h) * (2 * LR_HALF) : sa;
            const uint64_t dh = desc_sw128(va, 0), dl = desc_sw128(va + LR_HALF, 0), dw = desc_sw128(sa + (KEEP ? h : 2) * LR_HALF, 0);
#pragma unroll
            for (int q = 0; q < 4; q++) umma_tf32(d, dh + 2 * q, dw + 2 * q, id, uc != 0 || h != 0 || q != 0);
#pragma unroll
            for (int q = 0; q < 4; q++) umma_tf32(d + 256, dl + 2 * q, dw + 2 * q, id, uc != 0 || h != 0 || q != 0);
          }
          umma_commit(empty(us));
          if (ends) umma_commit(acc_full(buf));
        }
        __syncwarp();
      }
      used++, accs += last;
      if (++st == nst) st = 0, lap++;
    }
    // nothing is in flight when the block leaves
    if (used) ws.wait(empty(st == 0 ? nst - 1 : st - 1), (st == 0 ? lap - 1 : lap) & 1);
  } else {
    const int q = w & 3, g = (w - LE_FEED / 32) >> 2;  // the warp's quarter of the rows, of the columns
    // this lane's pieces of y: row (lane & 24) + j of the warp's 32, 16 bytes at
    // piece lane % 8 of its 32 columns
    const float *from = (a.base ? a.base : a.y) + 32 * g + 4 * (lane & 7);
    float *to = a.y + 32 * g + 4 * (lane & 7);
    const int from_stride = a.base ? a.base_stride : a.y_stride;
    int accs = 0, t = t0, col = c0, tok[8], rank = 0;  // tile, its part of the columns; tokens of the lane's rows, rank
    auto load_tile = [&]() {
      const int4 tile = a.tiles[t];
      rank = tile.z >> 16;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int row = 32 * q + (lane & 24) + j;
        tok[j] = row < (tile.z & 0xFFFF) ? a.perm[tile.y + row] : -1;
      }
    };
    auto left_of = [&]() { return a.N - col * 128 - 32 * g - 4 * (lane & 7); };
    float4 b[8];
    // y of an item whose base is in b
    auto finish = [&](const int (&rows)[8], int n, int left, int rk) {
      if (rk) {
        const int buf = accs & 1;
        ws.wait(acc_full(buf), (accs / 2) & 1);
        __syncwarp();
        tc_fence_after();
        uint32_t u[32];
        const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + buf * 128 + 32 * g;
#pragma unroll
        for (int e = 0; e < 32; e += 16) {
          float hi[16], lo[16];
          tmem_ld16x2(at + e, at + 256 + e, hi, lo);
#pragma unroll
          for (int k = 0; k < 16; k++) u[e + k] = __float_as_uint(hi[k] + lo[k]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty(buf));
        accs++;
        transpose8(u);
#pragma unroll
        for (int j = 0; j < 8; j++) {
          b[j].x += __uint_as_float(u[4 * j]), b[j].y += __uint_as_float(u[4 * j + 1]);
          b[j].z += __uint_as_float(u[4 * j + 2]), b[j].w += __uint_as_float(u[4 * j + 3]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; j++) {
        if (rows[j] < 0) continue;
        float *p = to + (long long)rows[j] * a.y_stride + n;
        if (a.wide) {
          if (left > 0) __stcs(reinterpret_cast<float4 *>(p), b[j]);
        } else {
          if (left > 0) p[0] = b[j].x;
          if (left > 1) p[1] = b[j].y;
          if (left > 2) p[2] = b[j].z;
          if (left > 3) p[3] = b[j].w;
        }
      }
    };
    if (KEEP && a.R32 <= 64 && a.wide) {
      // through this thread's eight places of 16 bytes, behind V and the ring
      const uint32_t slot = base + 4 * (2 * LR_HALF) + (uint32_t)(tid - LE_FEED) * 16;
      auto request = [&]() {
        const bool in = left_of() > 0;
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const bool live = in && tok[j] >= 0;
          const float *p = live ? from + (long long)tok[j] * from_stride + col * 128 : a.y;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot + j * (512 * 16)), "l"(p), "r"(live ? 16 : 0) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      if (i0 < i1) load_tile(), request();
      for (long long i = i0; i < i1; i++) {
        const int n = col * 128, left = left_of(), rk = rank;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const uint4 x = ld_shared_v4(slot + j * (512 * 16));
          b[j] = make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w));
        }
        if (i + 1 < i1 && col + 1 < n_col) {  // (the next tile's first item is requested when this one is stored)
          col++;
          request();
          finish(tok, n, left, rk);
        } else {
          finish(tok, n, left, rk);
          if (i + 1 < i1) {
            col = 0, t++;
            load_tile();
            request();
          }
        }
      }
    } else {
      auto request = [&]() {
        const int n = col * 128, left = left_of();
#pragma unroll
        for (int j = 0; j < 8; j++) {
          b[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (tok[j] < 0) continue;
          const float *p = from + (long long)tok[j] * from_stride + n;
          if (a.wide) {
            if (left > 0) b[j] = __ldcs(reinterpret_cast<const float4 *>(p));
          } else {
            if (left > 0) b[j].x = p[0];
            if (left > 1) b[j].y = p[1];
            if (left > 2) b[j].z = p[2];
            if (left > 3) b[j].w = p[3];
          }
        }
      };
      if (i0 < i1) load_tile(), request();
      for (long long i = i0; i < i1; i++) {
        finish(tok, col * 128, left_of(), rank);
        if (i + 1 == i1) break;
        if (++col == n_col) {
          col = 0, t++;
          load_tile();
        }
        request();
      }
    }
  }
  if (!ws.ok && lane == 0) raise_flag(a.err, DS4MOE_DEVERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (w == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// A slot's weights into its place: rows of A padded with zeros to r32, rows of B
// to r8. Two bytes a thread: up to 4 MB of weights (rank 128, 8192 x 8192) a call takes
// the 5.7 to 6 us of its host side, 8 MB 8.6, 9.4 MB 11.2 (read and written, 1.7 to 2.0
// TB/s): what one adapter of a step's next request costs, not every step.
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
  const void *token, *token_loop, *shrink, *shrink_many, *expand;
};
template <int DT, bool F32, bool MANY>
const void *shrink_of(int r32) {
  return r32 <= 64 ? (const void *)k_adapt_shrink<DT, F32, 2, MANY> : r32 <= 128 ? (const void *)k_adapt_shrink<DT, F32, 4, MANY>
                                                                                  : (const void *)k_adapt_shrink<DT, F32, 8, MANY>;
}
template <int DT, bool F32>
AdaptFns fns_of(int r32) {
  return {(const void *)k_adapt_token<DT, F32, false>, (const void *)k_adapt_token<DT, F32, true>, shrink_of<DT, F32, false>(r32), shrink_of<DT, F32, true>(r32),
          r32 <= 128 ? (const void *)k_adapt_expand<DT, true> : (const void *)k_adapt_expand<DT, false>};
}
AdaptFns adapt_fns(int dtype, bool f32, int r32) {
  constexpr int B = DS4MOE_DT_BF16, F = DS4MOE_DT_F16;
  return dtype == B ? f32 ? fns_of<B, true>(r32) : fns_of<B, false>(r32) : f32 ? fns_of<F, true>(r32) : fns_of<F, false>(r32);
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

size_t token_smem(int n_in) { return (size_t)(n_in / 8 / LR_CLUSTER + 1) * 32; }

// Whether a call goes token by token (-1), by tiles (0), or whichever is shorter
// once the number of tiles is known on the device: the most for which tiles are.
//
// Tiles are a 128th of the tokens if all have one adapter, and with as many adapters
// as there are slots or tokens one more for each. Times in us, measured with 64 to
// 4096 tokens (tokens, tiles): token by token a wave of four blocks per SM reads the
// adapter again, out of L2; by tiles every tile costs its turn in three kernels.
//   4096 x 4096, rank 16    512 tokens of 1 adapter 37, 25; of 64 37, 88; of 512 52, 529; 4096 of 1 289, 71
//                rank 64    64 of 1 20, 25; 512 of 1 74, 27; of 64 82, 96; of 512 128, 567; 4096 of 512 603, 719
//                rank 256   64 of 1 39, 36; 512 of 1 231, 40; of 64 270, 330; 4096 of 512 2015, 2405
//   512 x 512, rank 16      512 of 1 28, 23; of 512 29, 160; 4096 of 1 191, 24; of 512 193, 89
//   8192 x 8192, rank 128   64 of 1 35, 31; 512 of 64 235, 240; of 512 497, 1586
// A decision on the device takes launches that find nothing to do (2 to 3 us for tiles;
// some 10 token by token, and blocks that take several tokens, 1.3 times the time at
// most: 256 to 1000 of rank 64 and as many adapters 69, 90 and 243, 286). It is left to the
// device where tiles may take 0.6 of the time or less.
int choose_way(const ds4moe_adapters *h, int n_tok) {
  if (h->path) return h->path == 1 ? -1 : 0;
  const double r = h->max_rank, size = (double)h->K + h->N;
  const int waves = (n_tok * LR_CLUSTER + 4 * h->n_sm - 1) / (4 * h->n_sm);
  const double tokens = waves * (2.9 + 0.05 * r + 1e-6 * r * (14.0 * h->N + 5.8 * h->K));
  const double start = 20.0 + size * (6e-4 + 4.5e-7 * n_tok), tile = 0.2 + size * (h->R32 <= 64 ? 1e-4 : h->R32 <= 128 ? 1.6e-4 : 4.6e-4);
  const int full = n_tok / 128, least = (n_tok + 127) / 128, most = full + std::min(h->slots + 1, n_tok);
  const double surely = start + tile * (most - 1), at_best = start + tile * (least - 1);
  if (tokens >= surely) return 0;
  if (tokens <= 1.7 * at_best) return -1;
  if (tokens + 10.0 >= surely) return 0;
  return 1 + (int)((tokens - start) / tile);
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
  const size_t o_perm = place((size_t)max_tokens * 4), o_n = place(12);
  const size_t o_tiles = place(((size_t)max_tokens / 128 + std::min(n_slots + 1, max_tokens) + 1) * 16);
  const size_t o_v = place((size_t)max_tokens * h->R32 * 4);
  const size_t o_a = place((size_t)n_slots * h->R32 * n_in * 2), o_b = place((size_t)n_slots * h->b_slot * 2);
  cudaError_t e = cudaGetDevice(&h->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->n_sm, cudaDevAttrMultiProcessorCount, h->device);
  for (bool f32 : {false, true}) {
    const AdaptFns f = adapt_fns(dtype, f32, h->R32);
    for (const void *fn : {f.token, f.token_loop})
      if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, ((1 << 16) / LR_CLUSTER + 8) * 4);
    for (const void *fn : {f.shrink, f.shrink_many, f.expand})
      if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, LR_SMEM);
    for (const void *fn : {f.shrink, f.shrink_many})
      if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      cfg.gridDim = dim3(LR_CLUSTER), cfg.blockDim = dim3(256), cfg.dynamicSmemBytes = token_smem(n_in);
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = LR_CLUSTER, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr, cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&h->token_clusters[f32], f.token_loop, &cfg);
      if (e == cudaSuccess && h->token_clusters[f32] < 1) h->token_clusters[f32] = 1;
    }
    for (int ks = 1; ks <= 2 * LR_CLUSTER && e == cudaSuccess; ks += ks < LR_CLUSTER ? 1 : LR_CLUSTER) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      cfg.gridDim = dim3(ks), cfg.blockDim = dim3(LR_WARPS * 32 + 32), cfg.dynamicSmemBytes = LR_SMEM;
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = ks, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr, cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&h->clusters[ks], f.shrink, &cfg);
      if (e == cudaSuccess && h->clusters[ks] < 1 && ks <= LR_CLUSTER) h->clusters[ks] = 1;
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
  const long long K = h->K, N = h->N, lim = 1ll << 31;  // strides are 32-bit numbers on the device
  if (n_tok == 1) x_stride = K, base_stride = y_stride = N;
  if (x_stride < K || x_stride >= lim || x_stride % (f32 ? 4 : 8) || ((uintptr_t)x & 15)) return DS4MOE_ERR_INVALID_ARG;
  if (y_stride < N || y_stride >= lim || ((uintptr_t)y & 3)) return DS4MOE_ERR_INVALID_ARG;
  if (base && (base_stride < N || base_stride >= lim || ((uintptr_t)base & 3))) return DS4MOE_ERR_INVALID_ARG;
  if (!ap_dev_ptr(x) || !ap_dev_ptr(slots) || !ap_dev_ptr(y) || (base && !ap_dev_ptr(base))) return DS4MOE_ERR_INVALID_ARG;
  if (rows_overlap(y, N * 4, y_stride * 4, x, K * (f32 ? 4 : 2), x_stride * (f32 ? 4 : 2), n_tok)) return DS4MOE_ERR_INVALID_ARG;
  if (base == y && base_stride == y_stride) base = nullptr;
  if (base && rows_overlap(y, N * 4, y_stride * 4, base, N * 4, base_stride * 4, n_tok)) return DS4MOE_ERR_INVALID_ARG;
  AdaptArgs a = {};
  a.N = h->N, a.K = h->K, a.slots = h->slots, a.T = n_tok, a.R32 = h->R32, a.b_slot = h->b_slot;
  a.x = x, a.x_stride = (int)x_stride, a.base = base, a.base_stride = (int)base_stride, a.y = y, a.y_stride = (int)y_stride;
  a.slot_of = slots, a.info = h->info, a.A = h->A, a.B = h->B;
  a.perm = h->perm, a.tiles = h->tiles, a.n_tiles = h->n_tiles, a.v = h->v, a.err = h->err;
  a.wide = N % 4 == 0 && y_stride % 4 == 0 && !((uintptr_t)y & 15) && (!base || (base_stride % 4 == 0 && !((uintptr_t)base & 15)));
  const AdaptFns f = adapt_fns(h->dtype, f32, h->R32);
  const cudaStream_t s = (cudaStream_t)stream;
  const int way = choose_way(h, n_tok);
  if (way < 0) {
    void *args[] = {&a};
    const cudaError_t e = launch_cluster(f.token, LR_CLUSTER * n_tok, LR_CLUSTER, 256, token_smem(h->K), s, args);
    h->launches++;
    return ap_status(e);
  }
  a.most = way;
  void *plan[] = {&a};
  cudaError_t e = launch_pdl((const void *)k_adapt_plan, dim3(1), dim3(1024), 0, s, plan, true);
  if (e == cudaSuccess && way) {
    e = launch_cluster(f.token_loop, h->token_clusters[f32] * LR_CLUSTER, LR_CLUSTER, 256, token_smem(h->K), s, plan);
    h->launches++;
  }
  if (e == cudaSuccess) {
    // Blocks of a tile: the fewest chunks of 32 columns one after another, six
    // more for a tile's start and sum, with some tiles that are not full; but chains
    // of additions that stay exact (four of each chunk, up to 37 to an accumulator,
    // see k_adapt_shrink: 41 were off by 1.06e-6, twice what 32-bit sums are), where
    // need be with twice the largest portable cluster and in passes of eight chunks to
    // an accumulator.
    const int most = n_tok / 128 + std::min(h->slots + 1, n_tok) + 1, full = n_tok / 128 + 1, guess = full + std::min(h->slots, full) / 2;
    const int n_acc = shrink_accs(h->R32) - (f32 ? 1 : 0);
    int ks = 0;
    long long best = 0;
    for (int c = LR_CLUSTER; c >= 1; c--) {
      const long long chunks = (K / 32 + c - 1) / c, cost = (guess + h->clusters[c] - 1) / h->clusters[c] * (chunks + 6);
      if (4 * chunks <= 37 * n_acc && (!ks || cost < best)) best = cost, ks = c;
    }
    int passes = 1;
    if (!ks) {
      ks = h->clusters[2 * LR_CLUSTER] ? 2 * LR_CLUSTER : LR_CLUSTER;
      passes = ((h->K / 32 + ks - 1) / ks + 8 * n_acc - 1) / (8 * n_acc);
    }
    const int grid = std::min(h->clusters[ks], most) * ks;
    void *args[] = {&a, &ks, &passes};
    e = launch_cluster(passes > 1 ? f.shrink_many : f.shrink, grid, ks, LR_WARPS * 32 + 32, LR_SMEM, s, args);
    if (e == cudaSuccess) {
      const long long items = (long long)most * ((N + 127) / 128);
      e = launch_pdl(f.expand, dim3((unsigned)std::min<long long>(items, h->n_sm)), dim3(LE_THREADS), LR_SMEM, s, plan, true);
    }
  }
  h->launches += 3;
  return ap_status(e);
}

ds4moe_status ds4moe_adapters_debug_path(ds4moe_adapters *h, int32_t path) {
  if (!h || path < 0 || path > 2) return DS4MOE_ERR_INVALID_ARG;
  h->path = path;
  return DS4MOE_OK;
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
