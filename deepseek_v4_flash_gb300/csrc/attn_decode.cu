// attn_decode.cu -- attention of few new tokens over the paged cache: at most
// 16 rows (new tokens x heads of a key-value head), head dimension 64 or 128.
//
// out = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m), s_j = <q, k_j> scale log2(e),
// in one pass: a running maximum m per row, the sum l and the accumulator O
// relative to it. Bound by the cache's bytes (each key and value is read
// once; 4 G n_new operations per 4 bytes), so all that matters is enough bytes
// in flight on every SM and no SM without work:
//   - The cache is cut into units of 128 positions of one (sequence, key-value
//     head); the call's units, in order, are dealt to the blocks in equal
//     contiguous runs, whatever the sequences' lengths. A (sequence, head) that
//     lies in several runs leaves one partial (O, m, l) per block, and the
//     block that arrives last adds them up in block order: the same bits every
//     time, one launch.
//   - A warp owns 16 positions of each unit and streams them through its own
//     ring of cp.async stages, without a block barrier until the run leaves
//     the (sequence, head): 192 KB per SM are in flight.
//   - Rows are the M = 16 of mma.sync m16n8k16 (f32 accumulation): with at
//     most 16 rows the instruction's legacy rate is far above what the memory
//     feeds, and scores, weights and O stay in registers.
// Measured: 24 sequences of 300 to 65537 positions, 8 heads of 128 (1.39 GB):
// 228 to 235 us, 5.9 to 6.1 TB/s, 0.88 to 0.91 of the copy rate; one sequence of
// 701: 8.8 us, a chain of dependent reads and the join's round trips.
// Rows of the cache that no query row sees are zero-filled on their way in, so
// that a weight of 0 never meets what they hold.
#include <type_traits>

#include "attn.cuh"
#include "internal.h"

namespace ds4 {

// Warps of a block; a unit has a group of 16 positions for each. Eight, and one
// block per SM; with shared positions two blocks of four: there the items, of
// the sequences' own positions, are short, and while one block joins its warps'
// results the other one streams.
template <bool SHARED>
constexpr int AD_WARPS = SHARED ? 4 : 8;
// A block's least run: below two units the join costs more than the split
// gains (1 sequence of 8192, 8 heads on 1: 16.9 us with one, 13.0 with two, 14.6 with four).
constexpr int AD_LEAST = 2;
constexpr int AD_MAX_BLOCKS = 160;  // blocks of eight warps (one per SM): the joining block's table of factors
template <bool SHARED>
constexpr int AD_RING = AD_WARPS<SHARED> * 24 * 1024;
// fp16 weights are scaled by 2^14 (the largest is 16384): a weight then
// vanishes below 2^-39 of the largest instead of 2^-25, and a long cache's
// many small weights are not lost.
template <int DT>
constexpr float AD_BIAS = DT == DS4MOE_DT_F16 ? 14.0f : 0.0f;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
template <int DT>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (DT == DS4MOE_DT_BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool SHARED>
using DecArgs = typename std::conditional<SHARED, SharedArgs, AttnArgs>::type;

// A sequence's part in a decode call.
struct DecSeq {
  int first, last, len;  // positions of its first and last new token
  int own;               // SHARED: where its own positions begin
  Groups gr;
  int units;             // at least one, so that every row is written
};
template <bool SHARED>
__device__ __forceinline__ DecSeq dec_seq(const DecArgs<SHARED> &a, int b, bool &bad) {
  DecSeq s;
  const SeqInfo si = seq_info(a, b, bad);
  s.len = si.len, s.first = si.len - si.n, s.last = si.len - 1;
  s.gr = Groups{0, 0, 0};
  if (s.last >= 0) s.gr = groups_of(a, max(s.first, 0), s.last);
  s.own = 0;
  if (SHARED) {
    s.own = own_start(a, b, si.len);
    s.gr.win0 = s.own >> 4, s.gr.n = s.last < s.own ? 0 : s.gr.n - s.gr.win0;  // (no window)
  }
  s.units = max(1, (s.gr.n + AD_WARPS<SHARED> - 1) / AD_WARPS<SHARED>);
  return s;
}

// Where a block stands in its run of units.
struct DecCursor {
  DecSeq s;
  int b, kvh, lu;  // sequence, key-value head, unit of that pair
};
template <bool SHARED>
__device__ __forceinline__ void dec_next(const DecArgs<SHARED> &a, DecCursor &c) {
  if (++c.lu < c.s.units) return;
  c.lu = 0;
  if (++c.kvh < a.n_kv) return;
  c.kvh = 0;
  bool bad = false;
  if (++c.b < a.n_seq) c.s = dec_seq<SHARED>(a, c.b, bad);
}

// A sequence's units by lane (sequences b0 .. b0 + 31), inclusive prefix and
// the warp's sum.
template <bool SHARED>
__device__ __forceinline__ long long dec_prefix(const DecArgs<SHARED> &a, int b0, bool &bad, long long &incl, long long &sum) {
  const int lane = threadIdx.x & 31;
  const long long n = b0 + lane < a.n_seq ? (long long)dec_seq<SHARED>(a, b0 + lane, bad).units * a.n_kv : 0;
  incl = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  sum = __shfl_sync(0xffffffffu, incl, 31);
  return n;
}
// The block's run of units [u0, u1) out of U, dealt to N blocks, and the
// cursor at u0 (whole warp). False when there is nothing for this block.
template <bool SHARED>
__device__ __forceinline__ bool dec_start(const DecArgs<SHARED> &a, int n_cta, long long &U, long long &N, long long &u0,
                                        long long &u1, DecCursor &c) {
  long long incl, sum, n;
  bool bad = false;
  n = dec_prefix<SHARED>(a, 0, bad, incl, sum);  // up to 32 sequences: the only pass
  U = sum;
  for (int b0 = 32; b0 < a.n_seq; b0 += 32) {
    long long i, s;
    dec_prefix<SHARED>(a, b0, bad, i, s);
    U += s;
  }
  if (bad && blockIdx.x == 0 && threadIdx.x < 32) raise_flag(a.err, DS4MOE_DEVERR_LENGTH);
  N = (U + AD_LEAST - 1) / AD_LEAST;
  if (N > n_cta) N = n_cta;  // (at most AD_MAX_BLOCKS)
  if (blockIdx.x >= N) return false;
  u0 = U * blockIdx.x / N, u1 = U * (blockIdx.x + 1) / N;
  long long u = u0;
  for (int b0 = 0; b0 < a.n_seq; b0 += 32) {
    if (b0) n = dec_prefix<SHARED>(a, b0, bad, incl, sum);
    const unsigned hit = __ballot_sync(0xffffffffu, u < incl);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const long long rem = u - __shfl_sync(0xffffffffu, incl - n, l);
      c.b = b0 + l;
      c.s = dec_seq<SHARED>(a, c.b, bad);
      c.kvh = (int)(rem / c.s.units), c.lu = (int)(rem - (long long)c.kvh * c.s.units);
      break;
    }
    u -= sum;
  }
  return true;
}

// A row whose result holds a NaN that may come from a position it does not see
// (another of several new tokens does), once more from what it sees alone.
template <int DT, int D>
__device__ __noinline__ void redo_row(const AttnArgs &a, int t, int h, int b, int pos, const Groups &gr) {
  float2 acc[D / 64];
  float m, l;
  bool bad = false;
  attn_row_warp<DT, D>(a, a.q + (long long)t * a.q_stride + (long long)h * D, b, h / a.group, pos, gr, 0, gr.n, acc, m,
                       l, bad);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint32_t *o = reinterpret_cast<uint32_t *>(a.out + (long long)t * a.out_stride + (long long)h * D);
#pragma unroll
  for (int c = 0; c < D / 64; c++)
    o[(threadIdx.x & 31) + 32 * c] = l == 0.0f ? 0u : Half16<DT>::down(acc[c].x * inv, acc[c].y * inv);
}

// SHARED: the positions before each sequence's own ones are in a.pre, whose
// result joins the row's as it is stored (attn_shared.cu).
template <int DT, int D, bool SHARED>
__global__ void __launch_bounds__(AD_WARPS<SHARED> * 32, SHARED ? 2 : 1) k_attn_decode(const DecArgs<SHARED> a, float *part, int *ticket, int n_cta) {
  constexpr int STAGE = 64 * D;  // a warp's 16 keys and 16 values; also 16 rows of O in 32 bits
  constexpr int NST = AD_RING<SHARED> / (AD_WARPS<SHARED> * STAGE);
  constexpr int CH = D / 8;      // 16-byte pieces of a row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[AD_WARPS<SHARED>][16], s_l[AD_WARPS<SHARED>][16], s_mt[16], s_lt[16];
  __shared__ float s_f[SHARED ? 1 : AD_MAX_BLOCKS][16];  // (SHARED: two blocks' tables would not fit beside their rings)
  __shared__ int s_last, s_nan;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int rows = a.n_new * a.group;
  uint8_t *ring = smem + w * NST * STAGE;
  const uint32_t ring_u = smem_u32(ring);
  pdl_launch_dependents();
  // (SHARED: when this kernel starts, all that came before the call is done, see
  // k_attn_tile; only results of the call's own kernels are waited for, below)
  if (!SHARED) pdl_wait();

  long long U, N, u0, u1;
  DecCursor lc, cc;  // where loading and computing stand
  if (!dec_start<SHARED>(a, n_cta, U, N, u0, u1, lc)) {
    if (SHARED) pdl_wait();  // (a kernel that is done stands for all before it)
    return;
  }
  cc = lc;

  // one unit's 16 positions of this warp into ring slot `slot`
  bool bad_page = false;
  // the table's entry for the next unit is read one unit ahead
  int entry = 0, row0 = 0;
  auto look = [&]() {
    const int g = lc.lu * AD_WARPS<SHARED> + w;
    if (lc.b < a.n_seq && g < lc.s.gr.n) {
      const int p0 = group_pos(lc.s.gr, g), pi = page_index(a.kv, p0);
      entry = a.kv.table[(long long)lc.b * a.kv.table_stride + pi], row0 = p0 - pi * a.kv.page_size;
    }
  };
  auto load = [&](int slot) {
    const int g = lc.lu * AD_WARPS<SHARED> + w;
    if (g < lc.s.gr.n) {
      const int p0 = group_pos(lc.s.gr, g);
      const int page = entry >= 0 && entry < a.kv.n_pages ? entry : -1;
      if (page < 0) bad_page = true;
      // rows some query row sees: within the length, in the first query's
      // window or after it, or among the first positions
      const int lo = SHARED ? lc.s.own : window_lo(a, max(lc.s.first, 0)), sink = min(a.n_sink, window_lo(a, lc.s.last));
      // this lane's piece of the row (lane / CH), and of every (32 / CH)-th after it
      constexpr int STEP = 32 / CH;
      const int r0 = lane / CH, c = lane % CH;
      const long long row = row0 + r0;
      const uint16_t *kp = a.kv.k + (long long)max(page, 0) * a.kv.k_page + (long long)lc.kvh * a.kv.k_head + row * a.kv.k_row + c * 8;
      const uint16_t *vp = a.kv.v + (long long)max(page, 0) * a.kv.v_page + (long long)lc.kvh * a.kv.v_head + row * a.kv.v_row + c * 8;
      const uint32_t dst = ring_u + slot * STAGE + r0 * (2 * D);
      if (page >= 0 && p0 + 15 <= lc.s.last && (p0 >= lo || p0 + 15 < sink)) {  // all of them
#pragma unroll
        for (int i = 0; i < 16 / STEP; i++) {
          const uint32_t d = dst + i * STEP * (2 * D) + ((c ^ ((r0 + i * STEP) & 7)) << 4);
          cp_async16(d, kp, true);
          cp_async16(d + 32 * D, vp, true);
          kp += STEP * a.kv.k_row, vp += STEP * a.kv.v_row;
        }
      } else {
        for (int i = 0; i < 16 / STEP; i++) {
          const int j = p0 + r0 + i * STEP;
          const bool live = page >= 0 && j <= lc.s.last && (j >= lo || j < sink);
          const uint32_t d = dst + i * STEP * (2 * D) + ((c ^ ((r0 + i * STEP) & 7)) << 4);
          cp_async16(d, live ? kp : a.kv.k, live);
          cp_async16(d + 32 * D, live ? vp : a.kv.v, live);
          kp += STEP * a.kv.k_row, vp += STEP * a.kv.v_row;
        }
      }
    }
    cp_commit();
  };

  const int n_it = (int)(u1 - u0);
  look();
#pragma unroll
  for (int i = 0; i < NST - 1; i++) {
    if (i < n_it) {
      load(i);
      dec_next<SHARED>(a, lc);
      look();
    } else {
      cp_commit();
    }
  }

  if (SHARED) pdl_wait();

  // SHARED: this thread's pieces of the item's results over the shared positions,
  // requested when the item begins
  constexpr int PIECES = SHARED ? 16 * (D / 4) / (AD_WARPS<SHARED> * 32) : 1;
  float4 pre[PIECES];
  float pre_log[PIECES];
  uint32_t qf[D / 16][4];
  float o[D / 8][4], m[2], l[2];
  const int r0 = lane >> 2, r1 = r0 + 8, c2 = (lane & 3) * 2;
  long long item0 = u0 - cc.lu;  // first unit of the current (sequence, head)
  bool fresh = true;
  for (int it = 0; it < n_it; it++) {
    // the next unit into the slot that the last iteration emptied
    if (it + NST - 1 < n_it) {
      load((it + NST - 1) % NST);
      dec_next<SHARED>(a, lc);
      look();
    } else {
      cp_commit();
    }
    if (fresh) {
      fresh = false;
      // row r = token * group + head; rows past the last read row 0 and are not stored
      const int t0 = cc.b * a.n_new, h0 = cc.kvh * a.group;
      const int ra = r0 < rows ? r0 : 0, rb = r1 < rows ? r1 : 0;
      const uint16_t *qa = a.q + (long long)(t0 + ra / a.group) * a.q_stride + (long long)(h0 + ra % a.group) * D;
      const uint16_t *qb = a.q + (long long)(t0 + rb / a.group) * a.q_stride + (long long)(h0 + rb % a.group) * D;
#pragma unroll
      for (int k = 0; k < D / 16; k++) {
        qf[k][0] = *reinterpret_cast<const uint32_t *>(qa + k * 16 + c2);
        qf[k][1] = *reinterpret_cast<const uint32_t *>(qb + k * 16 + c2);
        qf[k][2] = *reinterpret_cast<const uint32_t *>(qa + k * 16 + 8 + c2);
        qf[k][3] = *reinterpret_cast<const uint32_t *>(qb + k * 16 + 8 + c2);
      }
      if (SHARED) {
#pragma unroll
        for (int j = 0; j < PIECES; j++) {
          const int i = tid + j * AD_WARPS<SHARED> * 32, r = i / (D / 4), c = (i % (D / 4)) * 4;
          pre_log[j] = -INFINITY, pre[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (r >= rows || cc.s.own == 0) continue;
          const long long at = (long long)(t0 + r / a.group) * a.n_heads + h0 + r % a.group;
          pre_log[j] = pre_logs(a)[at], pre[j] = *reinterpret_cast<const float4 *>(pre_results(a) + at * D + c);
        }
      }
#pragma unroll
      for (int i = 0; i < D / 8; i++) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
      m[0] = m[1] = -INFINITY, l[0] = l[1] = 0.0f;
    }
    cp_wait<NST - 1>();
    __syncwarp();
    const uint32_t kb = ring_u + (it % NST) * STAGE, vb = kb + 32 * D;
    const int g = cc.lu * AD_WARPS<SHARED> + w;
    if (g < cc.s.gr.n) {
      // two chains of products each (even and odd steps): half the latency
      float s[2][4] = {}, s2[2][4] = {};
      {
        // matrices: keys 0-7 and 8-15 x halves of the 16 elements. A step
        // along the row flips address bits 5 to 7 (the swizzle is a xor).
        const int r = (lane & 7) + ((lane >> 4) << 3);
        const uint32_t ka = kb + r * (2 * D) + ((((lane >> 3) & 1) ^ (r & 7)) << 4);
#pragma unroll
        for (int k = 0; k < D / 16; k += 2) {
          uint32_t bf[4], bg[4];
          ldsm4(bf, ka ^ (k << 5));
          ldsm4(bg, ka ^ ((k + 1) << 5));
          mma16816<DT>(s[0], qf[k], bf[0], bf[1]);
          mma16816<DT>(s[1], qf[k], bf[2], bf[3]);
          mma16816<DT>(s2[0], qf[k + 1], bg[0], bg[1]);
          mma16816<DT>(s2[1], qf[k + 1], bg[2], bg[3]);
        }
      }
      const int p0 = group_pos(cc.s.gr, g);
      const int pa = cc.s.first + (a.n_new == 1 ? 0 : r0 / a.group), pb = cc.s.first + (a.n_new == 1 ? 0 : r1 / a.group);
#pragma unroll
      for (int n = 0; n < 2; n++)
#pragma unroll
        for (int i = 0; i < 4; i++) s[n][i] = (s[n][i] + s2[n][i]) * a.scale_log2;
      // some position not seen by some row (rows past the last take any mask)
      if (p0 + 15 > cc.s.first || (SHARED && p0 < cc.s.own) || (a.window > 0 && p0 < window_lo(a, max(cc.s.last, 0)) && p0 + 15 >= min(a.n_sink, window_lo(a, max(cc.s.first, 0))))) {
        const int la = SHARED ? cc.s.own : window_lo(a, max(pa, 0)), lb = SHARED ? cc.s.own : window_lo(a, max(pb, 0));
#pragma unroll
        for (int n = 0; n < 2; n++)
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int j = p0 + n * 8 + c2 + (i & 1), p = i < 2 ? pa : pb, lo = i < 2 ? la : lb;
            if (j > p || (j < lo && j >= a.n_sink)) s[n][i] = -INFINITY;
          }
      }
      float mx[2];
#pragma unroll
      for (int h = 0; h < 2; h++) {
        mx[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2)) - AD_BIAS<DT>;
      }
      if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const float mn = fmaxf(m[h], mx[h]);
          f[h] = mn == -INFINITY ? 1.0f : ex2(m[h] - mn);
          m[h] = mn, l[h] *= f[h];
        }
#pragma unroll
        for (int i = 0; i < D / 8; i++) o[i][0] *= f[0], o[i][1] *= f[0], o[i][2] *= f[1], o[i][3] *= f[1];
      }
      // a row that has seen nothing yet keeps weights of 0
      const float ma = m[0] == -INFINITY ? 0.0f : m[0], mb = m[1] == -INFINITY ? 0.0f : m[1];
#pragma unroll
      for (int n = 0; n < 2; n++) {
        s[n][0] = ex2(s[n][0] - ma), s[n][1] = ex2(s[n][1] - ma);
        s[n][2] = ex2(s[n][2] - mb), s[n][3] = ex2(s[n][3] - mb);
        l[0] += s[n][0] + s[n][1], l[1] += s[n][2] + s[n][3];
      }
      const uint32_t pf[4] = {Half16<DT>::down(s[0][0], s[0][1]), Half16<DT>::down(s[0][2], s[0][3]),
                              Half16<DT>::down(s[1][0], s[1][1]), Half16<DT>::down(s[1][2], s[1][3])};
      {
        // matrices: positions 0-7 and 8-15 x two 8-element columns
        const int r = (lane & 7) + (((lane >> 3) & 1) << 3);
        const uint32_t va = vb + r * (2 * D) + (((lane >> 4) ^ (r & 7)) << 4);
#pragma unroll
        for (int d = 0; d < D / 16; d++) {
          uint32_t bf[4];
          ldsm4t(bf, va ^ (d << 5));
          mma16816<DT>(o[2 * d], pf, bf[0], bf[1]);
          mma16816<DT>(o[2 * d + 1], pf, bf[2], bf[3]);
        }
      }
    }

    const bool item_ends = cc.lu + 1 == cc.s.units;
    if (item_ends || it + 1 == n_it) {
      // the block's eight warps: O into the slot just read, m and l beside it
#pragma unroll
      for (int h = 0; h < 2; h++) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if ((lane & 3) == 0) s_m[w][r0 + 8 * h] = m[h], s_l[w][r0 + 8 * h] = l[h];
      }
      __syncwarp();
      float *so = reinterpret_cast<float *>(ring + (it % NST) * STAGE);
#pragma unroll
      for (int i = 0; i < D / 8; i++) {
        const int c = (i * 8 + c2) ^ ((r0 & 7) << 3);
        if (r0 < rows) *reinterpret_cast<float2 *>(so + r0 * D + c) = make_float2(o[i][0], o[i][1]);
        if (r1 < rows) *reinterpret_cast<float2 *>(so + r1 * D + c) = make_float2(o[i][2], o[i][3]);
      }
      if (tid == 0) s_nan = 0;
      __syncthreads();
      if (tid < 16) {
        float mt = -INFINITY, lt = 0.0f;
        for (int i = 0; i < AD_WARPS<SHARED>; i++) mt = fmaxf(mt, s_m[i][tid]);
        for (int i = 0; i < AD_WARPS<SHARED>; i++) {
          const float f = s_m[i][tid] == -INFINITY ? 0.0f : ex2(s_m[i][tid] - mt);
          lt += s_l[i][tid] * f;
          s_m[i][tid] = f;
        }
        s_mt[tid] = mt, s_lt[tid] = lt;
      }
      __syncthreads();
      const long long end = item0 + cc.s.units;
      const bool whole = item0 >= u0 && end <= u1;
      const int slot = 2 * blockIdx.x + (item0 < u0 ? 0 : 1);
      float *pp = part + (size_t)slot * (16 * (D + 2));
      const int nan_rows_possible = a.n_new > 1;
      auto store = [&](int r, int c, float4 x, float m, float l, int piece) {
        const int t = cc.b * a.n_new + r / a.group, h = cc.kvh * a.group + r % a.group;
        float inv = 1.0f / l, from = 0.0f;
        bool zero = l == 0.0f;  // no score above -infinity (whatever the values: 0 x NaN is NaN)
        if (SHARED) join_two(pre_log[piece], m, l, from, inv, zero);
        x.x *= inv, x.y *= inv, x.z *= inv, x.w *= inv;
        if (SHARED) {
          const float4 p = pre[piece];
          x.x = fmaf(from, p.x, x.x), x.y = fmaf(from, p.y, x.y), x.z = fmaf(from, p.z, x.z), x.w = fmaf(from, p.w, x.w);
        }
        if (zero) x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const uint2 u = make_uint2(Half16<DT>::down(x.x, x.y), Half16<DT>::down(x.z, x.w));
        *reinterpret_cast<uint2 *>(a.out + (long long)t * a.out_stride + (long long)h * D + c) = u;
        if (nan_rows_possible && l == l) {
          const float z = x.x + x.y + x.z + x.w;  // NaN, or two infinities that cancel: both are looked at again
          if (z != z) atomicOr(&s_nan, 1 << r);
        }
      };
      auto sum_warps = [&](int i, int piece) {
        const int r = i / (D / 4), c = (i % (D / 4)) * 4;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < AD_WARPS<SHARED>; v++) {
          const float f = s_m[v][r];
          const float4 y = *reinterpret_cast<const float4 *>(smem + (size_t)(v * NST + it % NST) * STAGE +
                                                             4 * (r * D + (c ^ ((r & 7) << 3))));
          x.x = fmaf(f, y.x, x.x), x.y = fmaf(f, y.y, x.y), x.z = fmaf(f, y.z, x.z), x.w = fmaf(f, y.w, x.w);
        }
        if (whole) store(r, c, x, s_mt[r], s_lt[r], piece);
        else *reinterpret_cast<float4 *>(pp + r * D + c) = x;
      };
      // (SHARED: pieces are numbered at compile time, or they would not stay in registers)
      auto each_piece = [&](auto f) {
        if (SHARED) {
#pragma unroll
          for (int j = 0; j < PIECES; j++)
            if (tid + j * AD_WARPS<SHARED> * 32 < rows * (D / 4)) f(tid + j * AD_WARPS<SHARED> * 32, j);
        } else {
          for (int i = tid; i < rows * (D / 4); i += AD_WARPS<SHARED> * 32) f(i, 0);
        }
      };
      each_piece(sum_warps);
      bool done = whole;
      if (!whole) {
        if (tid < 16) pp[16 * D + tid] = s_mt[tid], pp[16 * D + 16 + tid] = s_lt[tid];
        // the last of the blocks that share this (sequence, head) joins
        const long long b0 = ((item0 + 1) * N - 1) / U, b1 = (end * N - 1) / U;
        __threadfence();
        __syncthreads();
        if (tid == 0) {
          const int n = atomicAdd(&ticket[b0], 1);
          s_last = n == (int)(b1 - b0);
          if (s_last) ticket[b0] = 0;
        }
        __syncthreads();
        done = s_last;
        if (s_last) {
          __threadfence();
          const int np = (int)(b1 - b0) + 1;
          // the block where the item starts holds it in its second slot, the others in their first
          auto at = [&](int p) { return part + (size_t)(2 * (b0 + p) + (p == 0 ? 1 : 0)) * (16 * (D + 2)); };
          // a row's factors 2^(m_p - m) / l: lanes over the partials
          for (int r = w; r < rows; r += AD_WARPS<SHARED>) {
            float mt = -INFINITY, lt = 0.0f;
            for (int p = lane; p < np; p += 32) {
              const float mp = __ldcg(at(p) + 16 * D + r);
              if (!SHARED) s_f[p][r] = mp;
              mt = fmaxf(mt, mp);
            }
            mt = warp_max(mt);
            for (int p = lane; p < np; p += 32) {
              const float mp = SHARED ? __ldcg(at(p) + 16 * D + r) : s_f[p][r];
              const float f = mp == -INFINITY ? 0.0f : ex2(mp - mt);
              if (!SHARED) s_f[p][r] = f;
              lt = fmaf(f, __ldcg(at(p) + 16 * D + 16 + r), lt);
            }
#pragma unroll
            for (int k = 16; k; k >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, k);
            if (lane == 0) s_lt[r] = lt, s_mt[r] = mt;
          }
          __syncthreads();
          each_piece([&](int i, int piece) {
            const int r = i / (D / 4), c = (i % (D / 4)) * 4;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 16
            for (int p = 0; p < np; p++) {
              const float4 y = __ldcg(reinterpret_cast<const float4 *>(at(p) + r * D + c));
              const float mp = SHARED ? __ldcg(at(p) + 16 * D + r) : 0.0f;
              const float f = SHARED ? mp == -INFINITY ? 0.0f : ex2(mp - s_mt[r]) : s_f[p][r];
              x.x = fmaf(f, y.x, x.x), x.y = fmaf(f, y.y, x.y), x.z = fmaf(f, y.z, x.z), x.w = fmaf(f, y.w, x.w);
            }
            store(r, c, x, s_mt[r], s_lt[r], piece);
          });
        }
      }
      __syncthreads();
      if (nan_rows_possible && done && s_nan) {
        for (int r = w; r < rows; r += AD_WARPS<SHARED>) {
          const int pos = cc.s.first + r / a.group, t = cc.b * a.n_new + r / a.group, h = cc.kvh * a.group + r % a.group;
          if ((s_nan >> r & 1) &&
              unseen_nonfinite<DT>(a, cc.b, cc.kvh, pos, pos, window_lo(a, max(cc.s.first, 0)), 0, cc.s.last + 1, 0, D) &&
              !own_nan<DT>(a, a.out + (long long)t * a.out_stride + (long long)h * D, cc.b, cc.kvh, pos, 0, D))
            redo_row<DT, D>(a, t, h, cc.b, pos, SHARED ? groups_of(a, max(pos, 0), max(pos, 0)) : cc.s.gr);
        }
        __syncthreads();
      }
      item0 = end;
      fresh = true;
    }
    dec_next<SHARED>(a, cc);
  }
  if (bad_page) raise_flag(a.err, DS4MOE_DEVERR_PAGE);
}

template <int DT>
static const void *dec_fn(int D, bool shared) {
  if (shared) return D == 64 ? (const void *)k_attn_decode<DT, 64, true> : (const void *)k_attn_decode<DT, 128, true>;
  return D == 64 ? (const void *)k_attn_decode<DT, 64, false> : (const void *)k_attn_decode<DT, 128, false>;
}

size_t attn_decode_part_floats(int n_sm) { return (size_t)2 * 2 * n_sm * 16 * (128 + 2); }

cudaError_t attn_decode_set_attributes() {
  for (bool shared : {false, true})
    for (int D : {64, 128})
      for (const void *fn : {dec_fn<DS4MOE_DT_BF16>(D, shared), dec_fn<DS4MOE_DT_F16>(D, shared)}) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   shared ? AD_RING<true> : AD_RING<false>);
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

template <bool SHARED>
static cudaError_t launch(const DecArgs<SHARED> &a, int head_dim, int dtype, float *part, int *ticket, int n_cta, cudaStream_t s) {
  void *args[] = {(void *)&a, &part, &ticket, &n_cta};
  const void *fn = dtype == DS4MOE_DT_BF16 ? dec_fn<DS4MOE_DT_BF16>(head_dim, SHARED) : dec_fn<DS4MOE_DT_F16>(head_dim, SHARED);
  return launch_pdl(fn, dim3(n_cta), dim3(AD_WARPS<SHARED> * 32), AD_RING<SHARED>, s, args, true);
}

cudaError_t launch_attn_decode(const AttnArgs &a, int head_dim, int dtype, float *part, int *ticket, int n_sm,
                               cudaStream_t s) {
  return launch<false>(a, head_dim, dtype, part, ticket, n_sm > AD_MAX_BLOCKS ? AD_MAX_BLOCKS : n_sm, s);
}

cudaError_t launch_attn_decode(const SharedArgs &a, int head_dim, int dtype, float *part, int *ticket, int n_sm,
                               cudaStream_t s) {
  return launch<true>(a, head_dim, dtype, part, ticket, 2 * n_sm, s);
}

}  // namespace ds4
