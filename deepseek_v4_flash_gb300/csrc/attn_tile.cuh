// attn_tile.cuh -- attention of tiles of 128 rows (new tokens x heads of a
// key-value head) on the tensor cores (tcgen05): prefill, drafted tokens of
// many heads per key-value head, and the long head dimensions 256 and 512.
//
// One pass over the visible positions in tiles of up to 128:
//   S = Q K^T           tcgen05.mma, Q and K in shared memory, S in tensor memory
//   P = 2^(S c - m)     two warpgroups, two threads per row
//   O += P V            tcgen05.mma, P in tensor memory (over S), V in shared memory
// with m the running maximum of a row. m only follows a new maximum that is
// more than 2^AT_LAZY above it, so that O is rarely rescaled (weights up to
// 2^AT_LAZY lose nothing: sums are kept in 32 bits and the quotient O / l does
// not depend on m).
//
// Warps: 0 loads (TMA out of the pages, a ring of stages), 1 issues the
// products, 2 works out which tiles come next, two warpgroups per row tile do
// the softmax and the output. Two tiles of S are in flight: while one is
// turned into P, the next one's product runs.
//   Head dimension 64 and 128, ragged calls: two row tiles per block share
//     every key and value tile, which halves the traffic from L2. Bound by a
//     row tile's chain S -> P -> O -> next S, two of which alternate (4096
//     tokens of 32/8 heads of 128: 122 us, 1126 TFLOP/s; one thread per row
//     192 us, as the chain was twice as long in the softmax).
//   Dimension 512: O has 512 columns and S needs room too, so a block computes
//     one half of O's columns (S is then computed twice), and Q takes 128 of
//     224 KB. Two row tiles therefore work as a pair of blocks (cta_group::2):
//     one product has 256 rows, each block holds half of the keys' rows and of
//     the values' columns, and what comes through L2 and the ring per row
//     halves (4096 tokens of 16 heads: 297 us alone, 238 us in pairs, 1154
//     TFLOP/s and half as much again for the second S; the products' own
//     24 cycles per position are reached). A single row tile (a decode
//     call of up to 128 rows) runs alone.
//
// Visible positions are listed in groups (the first positions' groups, then
// the windows' groups), one TMA box each, and a tile is 128 positions of that
// list. Small windows take groups of 16 to 32: a window of 128 positions costs
// 160 to 192 of them, not 3 tiles of 128. Else groups are as large as the pages
// allow (see box_shift).
//
// The call's tiles, in order, are dealt to the blocks in equal contiguous
// runs. A row tile whose positions lie in several runs leaves one partial
// (O, m, l) per block; k_attn_join adds them in block order. Where a window
// leaves an item few tiles it stays whole (AT_WHOLE).
//
// What the compiler makes of the softmax's loop depends on code far from it: at
// dimension 128, two row tiles and 96 registers, the same loop ran between 395
// and 513 us (prompts of 8192 and 4099, window 4096) with other forms of the
// rare second look at a row. A change here is timed there too.
#pragma once
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "attn.cuh"
#include "internal.h"
#include "umma.cuh"

namespace ds4 {

// What a call computes:
//   AT_ALL     every position that a row sees (attn_tile.cu);
//   AT_PREFIX  for a batch with shared positions (attn_shared.cu): every row of a
//              group of sequences over the group's shared positions, all of
//              which it sees. The call's "sequences" are the groups; results
//              stay in 32 bits, with the sum of weights as its logarithm;
//   AT_OWN     there, every sequence over its positions behind the shared
//              ones, joined with its rows' AT_PREFIX results.
enum { AT_ALL = 0, AT_PREFIX = 1, AT_OWN = 2 };

template <int MODE>
using Args = typename std::conditional<MODE == AT_ALL, AttnArgs, SharedArgs>::type;

// Whether row groups come from row bounds (ragged) or are the new tokens of
// every sequence.
template <int MODE>
__device__ __forceinline__ bool ragged(const AttnArgs &a) {
  return MODE == AT_ALL ? a.cu_q != nullptr : MODE == AT_PREFIX;
}

constexpr float AT_LAZY = 8.0f;
// fp16 weights are scaled by 2^7 (at most 2^15 with the lazy maximum): small
// weights keep 2^-31 of the largest instead of 2^-24.
template <int DT>
constexpr float AT_BIAS = DT == DS4MOE_DT_F16 ? 7.0f : 0.0f;

constexpr int AT_CHUNK = 128 * 128;     // 128 rows of 64 elements, 128-byte swizzled
constexpr int AT_SMEM = 224 * 1024;     // Q and the ring
constexpr int AT_MISC = 3 * 1024;       // what precedes them: barriers, segments, exchanged values
// What an item costs beside its tiles (loading Q, filling the pipeline,
// writing O), in tiles: counted into the runs, or a block with a prompt's first
// row groups, of one or two tiles each, would have three times the items of
// the others.
constexpr int AT_ITEM = 2;
// Most tiles of an item that is never split, 4 drafted tokens with 64 heads
// over one of 512: window 64, 1 and 64 sequences, 10.2 and 16.7 us whole, 17.2
// and 23.4 us as equal runs and their join; window 600 (7 tiles), 17.9 and 37.3
// us against 19.1 and 53.8 us; dimension 128 and one sequence is even there.
constexpr int AT_WHOLE = 8;
constexpr int AT_WALK = 512;            // most row groups that every block walks through itself
constexpr int AT_SEGS = 4;              // segments the scheduling warp is ahead

template <int D, int NT, bool PAIR>
struct TileCfg {
  static constexpr int DV = D < 256 ? D : 256;         // columns of O a block computes
  static constexpr int HALVES = D / DV;
  // Ring stages: KC chunks of 64 elements of a key tile's rows, VC of a value
  // tile's. Of a pair, each block holds half of the keys' rows and half of
  // the values' columns.
  static constexpr int KC = D == 64 ? 1 : 2, VC = D == 64 || PAIR ? 1 : 2;
  static constexpr int KPITCH = PAIR ? AT_CHUNK / 2 : AT_CHUNK;  // bytes of a chunk of keys
  static constexpr int STAGE = KC * KPITCH;
  static constexpr int KST = D / 64 / KC, VST = DV / 64 / VC / (PAIR ? 2 : 1);  // stages of a key and a value tile
  static constexpr int PV_N = VC * 64 * (PAIR ? 2 : 1);          // columns of one product into O
  static constexpr int Q = NT * (D / 64) * AT_CHUNK;
  static constexpr int NST_ = (AT_SMEM - Q) / STAGE;
  static constexpr int NST = NST_ > 10 ? 10 : NST_;
  static constexpr int THREADS = 128 + 256 * NT;
  static constexpr int SPAN = PAIR ? 2 : NT;           // row tiles of a ragged call's row group
  static constexpr int PITCH = DV + 4;                 // floats of a partial's row: O, m, l
  static constexpr int JROWS = 1024 / DV;              // rows that a joining block's threads cover at once
  static constexpr int O_COL = 256;                    // O's first tensor-memory column (S: 0 and 128)
  static_assert(VC * AT_CHUNK <= STAGE, "a stage holds either");
};

struct TileMaps {
  CUtensorMap q, k, v;
};

// What the blocks of a call share.
struct TileArgs {
  int gsh;           // log2 of a group's positions
  int tpt;           // tokens of a row tile: 128 / group
  int members;       // blocks that work on the same (item, key tiles): row tiles (decode calls, pairs) x halves
  int gangs;
  int whole;         // items are not split: each goes to the block whose run holds its first unit
  int join;          // AT_PREFIX: blocks of k_attn_join share the gangs among so many
  long long *first;  // ragged: first unit of each row group, then the total (k_attn_plan); null: no plan
  int2 *info;        // ragged: {sequence, first token of the row group in it}
  int *count;        // ragged: number of row groups
  float *part;       // [2 * grid][NT][128][DV + 4]: partials
  int4 *split;       // [2 * gangs]: what k_attn_join adds up
};

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap *m, int c0, int c1, int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *m, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
// ---- pairs of blocks (cta_group::2): one product of 256 rows, 128 in each
// block's tensor memory, the other operand's halves in the two blocks' shared
// memories. The even block issues the products and owns the barriers that say
// what is ready; all other barriers are told in both.
__device__ __forceinline__ uint32_t of_block(uint32_t addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void tma_4d_pair(uint32_t dst, const CUtensorMap *m, int c0, int c1, int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_3d_pair(uint32_t dst, const CUtensorMap *m, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void arrive_leader(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(of_block(bar, 0)) : "memory");
}
// (relaxed: the copies count their bytes themselves, and a release at cluster
// scope took 1000 cycles per stage)
__device__ __forceinline__ void expect_leader(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(of_block(bar, 0)),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void umma_f16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_f16_ts_pair(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The barrier at this place of both blocks.
__device__ __forceinline__ void umma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int DT>
__device__ __forceinline__ uint32_t idesc(int n, bool b_mn_major, int m = 128) {
  constexpr uint32_t t = DT == DS4MOE_DT_BF16 ? 1u : 0u;
  return (1u << 4) | (t << 7) | (t << 10) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// D[tmem] (+)= A[tmem] B
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Cycles that a warp waits for another, which may compute rows once more
// (AT_REDO).
constexpr long long AT_WAIT = 1ll << 33;

// A bounded wait of the whole warp: false for every lane when one gave up.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, AT_WAIT));
}

// ---------------------------------------------------------------------------
// The order of work.

// A run of key tiles [kt0, kt1) of one item: a row group (NT row tiles of tpt
// tokens) of one sequence and key-value head.
struct Seg {
  int b, kvh;
  int row0, n;       // first row of q, tokens
  int pos0;          // position of the first token
  int len;           // cached positions of the sequence
  int last;          // last position that any row of the list's range sees
  Groups gr;
  int kt0, kt1;      // empty: nothing is visible, the rows are 0; kt1 < 0: no more work
  int starts, ends;  // the run holds the item's first, last tile
};

// With AT_OWN's first position that counts.
template <int MODE>
struct SegOf : Seg {
  static constexpr int lo = 0;
};
template <>
struct SegOf<AT_OWN> : Seg {
  int lo;
};

__device__ __forceinline__ int tiles_of(const Groups &g, int sh) { return ((g.n << sh) + 127) >> 7; }

__device__ __forceinline__ Groups range_groups(const AttnArgs &a, int first, int last, int sh) {
  return last >= 0 ? groups_of(a, max(first, 0), last, sh) : Groups{0, 0, 0};
}

// The groups of 2^sh positions that hold positions first .. last.
__device__ __forceinline__ Groups own_groups(int first, int last, int sh) {
  if (last < first) return Groups{0, 0, 0};
  return Groups{0, first >> sh, (last >> sh) - (first >> sh) + 1};
}

// Columns of key tile kt that the products need, in 16s: up to the last
// visible position.
__device__ __forceinline__ int cols16(const Seg &s, int kt, int sh) {
  const int ng = s.gr.n - (kt << (7 - sh));  // groups from this tile on
  if (ng > 1 << (7 - sh)) return 8;
  return ((ng - 1) << (sh - 4)) + ((s.last - group_pos(s.gr, s.gr.n - 1, sh)) >> 4) + 1;
}

template <int MODE>
struct Sched {
  // In units of a tile, AT_ITEM of them before each item's first tile: where
  // the run stands, its end, the current item.
  long long u, u1, item0, item1;
  int b, kvh;
  int t0, span;                   // ragged calls: the row group's first token in its sequence, tokens of one
  int row0, row1, slen;           // ragged calls without a plan: first row, end and length of sequence `lane`
  int stab;                       // AT_PREFIX: the block table's row of it
  long long U, N;                 // the call's units, the gangs that have some

  // Rows and length of a sequence (whole warp, the same one).
  __device__ __forceinline__ SeqInfo seq(const Args<MODE> &a, const TileArgs &t, int bb) const {
    if (ragged<MODE>(a) && !t.first) {
      SeqInfo s;
      s.tok0 = __shfl_sync(0xffffffffu, row0, bb), s.n = __shfl_sync(0xffffffffu, row1, bb) - s.tok0;
      s.len = __shfl_sync(0xffffffffu, slen, bb);
      return s;
    }
    bool bad = false;
    if (MODE == AT_PREFIX) return prefix_info(a, bb, nullptr);
    return seq_info(a, bb, bad);
  }
  // A ragged call without a plan (up to 32 sequences): its row bounds, made
  // ascending as k_attn_plan does.
  __device__ __forceinline__ void read_rows(const Args<MODE> &a, bool &bad) {
    const int lane = threadIdx.x & 31;
    const bool in = lane < a.n_seq;
    if (MODE == AT_PREFIX) {
      SeqInfo s = {0, 0, 0};
      if (in) s = prefix_info(a, lane, &stab);
      row0 = s.tok0, row1 = s.tok0 + s.n, slen = s.len;
      return;
    }
    const int raw0 = in ? a.cu_q[lane] : 0, raw1 = in ? a.cu_q[lane + 1] : 0;
    slen = in ? seq_len(a, lane, bad) : 0;
    row0 = clamp_row(raw0, a.n_tok), row1 = clamp_row(raw1, a.n_tok);
    if (__any_sync(0xffffffffu, in && (row0 != raw0 || row1 != raw1 || row0 > row1))) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, row0, o);
        if (lane >= o) row0 = max(row0, x);
      }
      row1 = max(row0, row1);
      bad |= in && (row0 != raw0 || row1 != raw1);
    }
  }

  // the current item's sequence and rows; its tiles
  __device__ __forceinline__ int load(const Args<MODE> &a, const TileArgs &t, int member_rt, SegOf<MODE> &s) const {
    const SeqInfo si = seq(a, t, b);
    s.b = b, s.kvh = kvh, s.len = si.len;
    if (MODE == AT_PREFIX) {
      if (t.first) prefix_info(a, b, &s.b);
      else s.b = __shfl_sync(0xffffffffu, stab, b);
      s.row0 = si.tok0 + t0;
      s.n = min(span, si.n - t0);
      s.pos0 = s.last = si.len - 1;  // of every row
      s.gr = range_groups(a, s.last, s.last, t.gsh);
    } else if (ragged<MODE>(a)) {
      s.row0 = si.tok0 + t0;
      s.n = min(span, si.n - t0);
      s.pos0 = si.len - si.n + t0;
      s.last = s.pos0 + s.n - 1;
      s.gr = range_groups(a, s.pos0, s.last, t.gsh);
    } else {
      // every row tile of the sequence reads the same positions
      s.last = si.len - 1;
      s.gr = range_groups(a, si.len - si.n, s.last, t.gsh);
      if constexpr (MODE == AT_OWN) s.lo = own_start(a, b, si.len), s.gr = own_groups(s.lo, s.last, t.gsh);
      s.row0 = si.tok0 + member_rt * t.tpt;
      s.n = min(t.tpt, si.n - member_rt * t.tpt);
      s.pos0 = si.len - si.n + member_rt * t.tpt;
    }
    return tiles_of(s.gr, t.gsh);
  }

  // units of the tokens t0 .. t0 + n - 1 of a sequence
  static __device__ __forceinline__ int units(const Args<MODE> &a, int gsh, const SeqInfo &si, int t0, int n) {
    if (MODE == AT_PREFIX) return AT_ITEM + max(1, tiles_of(range_groups(a, si.len - 1, si.len - 1, gsh), gsh));
    const int p0 = si.len - si.n + t0;
    return AT_ITEM + max(1, tiles_of(range_groups(a, p0, p0 + n - 1, gsh), gsh));
  }
  __device__ __forceinline__ int seq_units(const Args<MODE> &a, int gsh, int bb, bool &bad) const {
    const SeqInfo si = seq_info(a, bb, bad);
    if (MODE == AT_OWN) return AT_ITEM + max(1, tiles_of(own_groups(own_start(a, bb, si.len), si.len - 1, gsh), gsh));
    return units(a, gsh, si, 0, si.n);
  }

  // Row groups of all sequences in order: their units' sum, or (r >= 0) the
  // one that holds unit r, into b, t0 and item0 (relative to the sum's start).
  __device__ long long walk(const Args<MODE> &a, const TileArgs &t, long long r) {
    const int lane = threadIdx.x & 31;
    long long base = 0, mine = 0;
    for (int l = 0; l < a.n_seq; l++) {
      const SeqInfo x = seq(a, t, l);
      for (int j0 = 0; j0 < x.n; j0 += 32 * span) {
        const int j = j0 + lane * span;
        const int un = j < x.n ? units(a, t.gsh, x, j, min(span, x.n - j)) : 0;
        if (r < 0) {
          mine += un;
          continue;
        }
        int incl = un;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, r < base + incl);
        if (hit) {
          const int k = __ffs(hit) - 1;
          b = l, t0 = j0 + k * span;
          item0 = base + __shfl_sync(0xffffffffu, incl - un, k), item1 = item0 + __shfl_sync(0xffffffffu, un, k);
          return 0;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    return mine;
  }

  // Whole warp. False when gang g has no tiles.
  __device__ bool init(const Args<MODE> &a, const TileArgs &t, int g, int nt, bool &bad) {
    const int lane = threadIdx.x & 31;
    long long head = 0;  // ragged: units of one key-value head
    int n_idx = 0;
    t0 = 0, span = nt * t.tpt;
    if (ragged<MODE>(a) && t.first) {
      n_idx = *t.count, head = t.first[n_idx];
      U = head * a.n_kv;
    } else if (ragged<MODE>(a)) {
      read_rows(a, bad);
      head = walk(a, t, -1);
      U = head * a.n_kv;
    } else {
      long long n = 0;
      for (int i = lane; i < a.n_seq; i += 32) n += seq_units(a, t.gsh, i, bad);
#pragma unroll
      for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      U = n * a.n_kv;
    }
    N = U < t.gangs ? U : t.gangs;
    if (g >= N) return false;
    u = U * g / N, u1 = U * (g + 1) / N;
    if (ragged<MODE>(a)) {
      kvh = (int)(u / head);
      const long long r = u - kvh * head;
      if (t.first) {
        // the last row group whose first unit is at or before r
        int lo = 0, hi = n_idx;  // first[lo] <= r < first[hi]
        while (hi - lo > 1) {
          const int step = (hi - lo + 31) / 32, i = min(hi, lo + (lane + 1) * step);
          const unsigned le = __ballot_sync(0xffffffffu, i < hi && t.first[i] <= r);
          const int k = __popc(le);  // ascending: a prefix of the lanes
          const int nlo = k ? lo + k * step : lo;
          hi = min(hi, lo + (k + 1) * step), lo = nlo;
        }
        const int2 in = t.info[lo];
        b = in.x, t0 = in.y;
        item0 = t.first[lo], item1 = t.first[lo + 1];
      } else {
        walk(a, t, r);
      }
      item0 += kvh * head, item1 += kvh * head;
    } else {
      long long r = u;
      for (int b0 = 0; b0 < a.n_seq; b0 += 32) {
        const long long n = b0 + lane < a.n_seq ? (long long)seq_units(a, t.gsh, b0 + lane, bad) * a.n_kv : 0;
        long long incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long x = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, r < incl);
        if (hit) {
          const int l = __ffs(hit) - 1;
          r -= __shfl_sync(0xffffffffu, incl - n, l);
          b = b0 + l;
          const int un = seq_units(a, t.gsh, b, bad);
          kvh = (int)(r / un);
          item0 = u - (r - (long long)kvh * un), item1 = item0 + un;
          break;
        }
        r -= __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    if (t.whole) {
      if (u != item0) advance(a, t);
      u = item0;
    } else if (u - item0 <= AT_ITEM) {
      u = item0;  // before the item's first tile: all of it
    }
    return true;
  }

  // The next item; item0 = U after the last one.
  __device__ __forceinline__ void advance(const Args<MODE> &a, const TileArgs &t) {
    bool bad = false;
    item0 = item1;
    if (item0 >= U) return;
    if (ragged<MODE>(a)) {
      SeqInfo si = seq(a, t, b);
      for (t0 += span; t0 >= si.n; t0 = 0) {
        if (++b == a.n_seq) b = 0, kvh++;
        si = seq(a, t, b);
        if (si.n > 0) {
          t0 = 0;
          break;
        }
      }
      item1 = item0 + units(a, t.gsh, si, t0, min(span, si.n - t0));
    } else {
      if (++kvh == a.n_kv) kvh = 0, b++;
      item1 = item0 + seq_units(a, t.gsh, b, bad);
    }
  }

  __device__ __forceinline__ bool next(const Args<MODE> &a, const TileArgs &t, int member_rt, SegOf<MODE> &s) {
    if (u >= u1 || (!t.whole && u1 < item1 && u1 - item0 <= AT_ITEM)) return false;  // (the next gang's from its start)
    const int n_kt = load(a, t, member_rt, s);
    const long long e = t.whole || item1 < u1 ? item1 : u1;
    s.starts = u == item0, s.ends = e == item1;
    s.kt0 = max(0, (int)(u - item0) - AT_ITEM), s.kt1 = min(n_kt, (int)(e - item0) - AT_ITEM);
    u = e;
    if (u == item1 && u < u1) advance(a, t);
    return true;
  }
};

// Ragged calls of many sequences or row groups: the row bounds (`cu`, as the
// caller gave them) made ascending into a.cu_q, the groups of `span` tokens in
// sequence order, and the running count of their units, by one block. Small
// calls do without (Sched::walk, in every block): up to AT_WALK groups of up to
// 32 sequences a block's walk is shorter than this kernel's 4 to 6 us.
template <int MODE>
__global__ void __launch_bounds__(1024) k_attn_plan(const Args<MODE> a, const int32_t *cu, int32_t *clean, int span, int gsh,
                                                long long *first, int2 *info, int *count, int *seq_first) {
  __shared__ long long warp_sum[32];
  __shared__ long long s_base;
  __shared__ int s_top[32], s_row;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  pdl_wait();
  // exclusive prefix of v over the block, plus the running base
  auto scan = [&](long long v) {
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[w] = x;
    __syncthreads();
    if (w == 0) {
      long long y = warp_sum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
      }
      warp_sum[lane] = y;
    }
    __syncthreads();
    const long long r = s_base + (w ? warp_sum[w - 1] : 0) + x - v;
    __syncthreads();
    if (tid == 0) s_base += warp_sum[31];
    __syncthreads();
    return r;
  };
  if (tid == 0) s_base = 0, s_row = 0;
  __syncthreads();
  bool bad = false;
  for (int b0 = 0; b0 < a.n_seq; b0 += 1024) {
    const int b = b0 + tid;
    const int2 c = clean_rows(cu, a.n_seq, a.n_tok, b, &s_row, s_top, bad);
    const int rows = b >= a.n_seq ? 0 : MODE == AT_PREFIX ? prefix_info(a, b, nullptr).n : c.y - c.x;
    const long long x = scan((rows + span - 1) / span);
    if (b < a.n_seq) {
      seq_first[b] = (int)x;
      clean[b] = c.x;
      if (b + 1 == a.n_seq) clean[b + 1] = c.y;
      if (MODE == AT_ALL) seq_len(a, b, bad);
    }
  }
  if (bad) raise_flag(a.err, DS4MOE_DEVERR_LENGTH);
  const int total = (int)s_base;  // at most n_tok / span + n_seq
  __syncthreads();
  if (tid == 0) s_base = 0, *count = total;
  __syncthreads();
  for (int i0 = 0; i0 < total; i0 += 1024) {
    const int i = i0 + tid;
    long long units = 0;
    int b = 0, t0 = 0;
    if (i < total) {
      int lo = 0, hi = a.n_seq;  // the last sequence that starts at or before i (empty ones start with the next)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seq_first[mid] <= i) lo = mid;
        else hi = mid;
      }
      b = lo, t0 = (i - seq_first[b]) * span;
      bool unused = false;
      const SeqInfo si = MODE == AT_PREFIX ? prefix_info(a, b, nullptr) : seq_info(a, b, unused);
      units = Sched<MODE>::units(a, gsh, si, t0, min(span, si.n - t0));
    }
    const long long x = scan(units);
    if (i < total) first[i] = x, info[i] = make_int2(b, t0);
  }
  if (tid == 0) first[total] = s_base;
}

// ---------------------------------------------------------------------------

// Bits [a, b) of a 128-bit row of flags, word w.
__device__ __forceinline__ uint32_t range_bits(int a, int b, int w) {
  const int lo = min(max(a - 32 * w, 0), 32), hi = min(max(b - 32 * w, 0), 32);
  const uint32_t h = hi == 32 ? 0xFFFFFFFFu : (1u << hi) - 1u, l = lo == 32 ? 0xFFFFFFFFu : (1u << lo) - 1u;
  return h & ~l;
}

// A row whose result holds a NaN that may come from a position it does not see
// (other rows of the tile do), once more from what it sees alone. Writes
// columns [c0, c1).
template <int DT, int D>
__device__ __noinline__ void redo_row_cols(const AttnArgs &a, int t, int h, int b, int pos, int c0, int c1) {
  float2 acc[D / 64];
  float m, l;
  bool bad = false;
  Groups gr = {0, 0, 0};
  if (pos >= 0) gr = groups_of(a, pos, pos);
  attn_row_warp<DT, D>(a, a.q + (long long)t * a.q_stride + (long long)h * D, b, h / a.group, pos, gr, 0, gr.n, acc, m,
                       l, bad);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint32_t *o = reinterpret_cast<uint32_t *>(a.out + (long long)t * a.out_stride + (long long)h * D);
#pragma unroll
  for (int c = 0; c < D / 64; c++)
    if (c * 64 >= c0 && c * 64 < c1)
      o[(threadIdx.x & 31) + 32 * c] = l == 0.0f ? 0u : Half16<DT>::down(acc[c].x * inv, acc[c].y * inv);
}

// Rows that see this many positions are not computed once more in the block,
// whose other warps wait for the next weights meanwhile (a warp's 32 rows take
// up to 50000 cycles a position), but by k_attn_mend. Until then the first
// column that the warp stores of such a row holds AT_MARK, bits that no result
// has: conversions give a NaN a positive sign.
constexpr int AT_REDO = 65536;
constexpr uint16_t AT_MARK = 0xFFFF;

// Rows of this warp whose result holds a NaN, although their sum of weights
// does not: token tq, head hq, position pos of sequence b (one row per lane;
// pos -1: the sum is 0, the row becomes zeros; -2: no such row). Those that may
// owe the NaN to a position they do not see are computed once more.
template <int DT, int D>
__device__ __noinline__ void look_again(const AttnArgs &a, int tq, int hq, int b, int pos, int c0, int c1) {
  const int lane = threadIdx.x & 31;
  unsigned m = __ballot_sync(0xffffffffu, pos >= 0);
  int kvh = 0, win0 = 0, sinks = 0, end = 0;
  if (m) {
    // the item's queries lie less than `span` positions apart
    bool bad = false;
    const int first = __reduce_min_sync(0xffffffffu, pos >= 0 ? pos : INT32_MAX), last = __reduce_max_sync(0xffffffffu, pos);
    const int len = seq_len(a, b, bad), p1 = min(first + a.span, len) - 1;
    const Groups gr = groups_of(a, max(last - a.span + 1, 0), p1, a.gsh);
    kvh = __shfl_sync(0xffffffffu, hq, __ffs(m) - 1) / a.group;
    win0 = gr.win0 << a.gsh, sinks = gr.n_sink << a.gsh, end = min(len, (p1 | 15) + 1);
    if (!unseen_nonfinite<DT>(a, b, kvh, first, last, win0, sinks, end, c0, c1)) m = 0;
  }
  for (m |= __ballot_sync(0xffffffffu, pos == -1); m; m &= m - 1) {
    const int x = __ffs(m) - 1, tx = __shfl_sync(0xffffffffu, tq, x), hx = __shfl_sync(0xffffffffu, hq, x);
    const int px = __shfl_sync(0xffffffffu, pos, x);
    uint16_t *o = a.out + (long long)tx * a.out_stride + (long long)hx * D;
    if (px >= 0 && (own_nan<DT>(a, o, b, kvh, px, c0, c1) ||
                    !unseen_nonfinite<DT>(a, b, kvh, px, px, win0, sinks, end, c0, c1)))
      continue;
    const int lo = window_lo(a, max(px, 0));
    if (px - lo + min(a.n_sink, lo) < AT_REDO) redo_row_cols<DT, D>(a, tx, hx, b, px, c0, c1);
    else if (lane == 0) o[c0] = AT_MARK, a.marked[blockIdx.x] = 1;
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <int DT, int D, int NT, bool PAIR, int MODE>
__global__ void __launch_bounds__(128 + 256 * NT, 1)
    k_attn_tile(const __grid_constant__ TileMaps maps, const Args<MODE> a, const TileArgs t) {
  using C = TileCfg<D, NT, PAIR>;
  // One window of dynamic shared memory, exactly what an SM has: a TMA tile
  // in the 128-byte swizzle starts on a multiple of 1024 bytes.
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  struct Misc {
    uint64_t bars[2 * 12 + 2 * AT_SEGS + 13 + 8];
    SegOf<MODE> segs[AT_SEGS];
    uint32_t tmem;
    // what the two threads of a row tell each other. Two row tiles: a row's S
    // follows both threads' P, so the next value cannot overtake the last.
    // One row tile: S runs ahead, two slots.
    float x[2][2][128];
  };
  static_assert(sizeof(Misc) <= AT_MISC && C::Q + C::NST * C::STAGE <= AT_SMEM, "shared memory");
  Misc &ms = *reinterpret_cast<Misc *>(smem_raw);
  const int tid = threadIdx.x, w = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t base = smem_u32(smem_raw) + AT_MISC;
  const uint32_t q_sm = base, ring = base + C::Q;
  const uint32_t bar0 = smem_u32(ms.bars);
  auto full = [&](int i) { return bar0 + 8 * i; };
  auto empty = [&](int i) { return bar0 + 8 * (12 + i); };
  auto seg_full = [&](int i) { return bar0 + 8 * (24 + i); };
  auto seg_empty = [&](int i) { return bar0 + 8 * (24 + AT_SEGS + i); };
  const uint32_t b_qf = bar0 + 8 * (24 + 2 * AT_SEGS), b_qe = b_qf + 16, b_sf = b_qe + 16, b_pa = b_sf + 16,
                 b_pb = b_pa + 16, b_of = b_pb + 16, b_done = b_of + 16, b_x = b_done + 8;
  if (base & 1023) {  // not where the swizzle needs it
    if (tid == 0) raise_flag(a.err, DS4MOE_DEVERR_INTERNAL);
    return;
  }
  const int gang = blockIdx.x / t.members, member = blockIdx.x % t.members;
  // which half of O's columns, which row tile of the row group (ragged pairs) or sequence (decode calls)
  const int rank = PAIR ? member & 1 : 0;
  const int half = PAIR ? member >> 1 & 1 : member % C::HALVES, rt = PAIR ? (member >> 2) * 2 + rank : member / C::HALVES;
  if (w == 0) {
    if (lane == 0) {
      for (int i = 0; i < C::NST; i++) mbar_init(full(i), PAIR ? 2 : 1), mbar_init(empty(i), 1);
      for (int i = 0; i < AT_SEGS; i++) mbar_init(seg_full(i), 1), mbar_init(seg_empty(i), 2 + 8 * NT);
      for (int i = 0; i < 2; i++) {
        mbar_init(b_qf + 8 * i, PAIR ? 2 : 1), mbar_init(b_qe + 8 * i, 1), mbar_init(b_sf + 8 * i, 1);
        // every thread of a warpgroup, or every warp of the two blocks'
        mbar_init(b_pa + 8 * i, PAIR ? 8 : 128), mbar_init(b_pb + 8 * i, PAIR ? 8 : 128), mbar_init(b_of + 8 * i, 1);
      }
      mbar_init(b_done, 1);
      for (int i = 0; i < 8; i++) mbar_init(b_x + 8 * i, 2);
      fence_mbar_init();
      fence_proxy_async_smem();
    }
    __syncwarp();
  } else if (w == 1) {
    if (PAIR) tmem_alloc_pair(smem_u32(&ms.tmem), 512);
    else tmem_alloc(smem_u32(&ms.tmem), 512);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (PAIR) cluster_sync_all();  // barriers are set up before the other block reaches for them
  const uint32_t tmem = ms.tmem;
  // AT_PREFIX: what follows the call's other kernels may then rely on all that
  // came before the call (the streaming kernel reads the cache before it waits)
  if (MODE == AT_PREFIX) pdl_wait();
  pdl_launch_dependents();
  pdl_wait();

  bool ok = true;  // no wait has run out

  // Operands of copies and products go through uniform(): the compiler then
  // keeps them in uniform registers, where these instructions want them.
  auto uniform = [&](int x) { return __shfl_sync(0xffffffffu, x, 0); };
  // The block's segments in order, from the scheduling warp; false after the
  // last one.
  int seg_n = 0;
  auto next_seg = [&](SegOf<MODE> &s) {
    const int i = seg_n % AT_SEGS;
    if (!wait_warp(seg_full(i), (seg_n / AT_SEGS) & 1)) return ok = false;
    s = ms.segs[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(seg_empty(i));
    seg_n++;
    return s.kt1 >= 0;
  };

  if (w == 2) {
    // ---- order of work: a few segments ahead of the others, so that nobody
    // else waits for lengths, row groups and tables of them
    Sched<MODE> sc;
    bool bad = false, split_out = false;
    bool more = sc.init(a, t, gang, C::SPAN, bad);
    if (bad && blockIdx.x == 0) raise_flag(a.err, DS4MOE_DEVERR_LENGTH);
    while (ok) {
      SegOf<MODE> s;
      s.kt1 = -1;
      if (more) more = sc.next(a, t, rt, s);
      if (!more) s.kt1 = -1;
      const int i = seg_n % AT_SEGS;
      if (seg_n >= AT_SEGS && !wait_warp(seg_empty(i), (seg_n / AT_SEGS - 1) & 1)) ok = false;
      if (lane == 0) {
        ms.segs[i] = s;
        mbar_arrive(seg_full(i));
        if (more && s.starts && !s.ends && member == 0) {
          // the first of an item's blocks says what k_attn_join adds up
          const int parts = (int)((sc.item1 * sc.N - 1) / sc.U) - gang + 1;
          t.split[2 * gang] = make_int4(parts, s.b, s.kvh, s.pos0);
          t.split[2 * gang + 1] = make_int4(s.row0, ragged<MODE>(a) ? s.n : a.n_new, s.lo, 0);
        }
      }
      split_out |= more && s.starts && !s.ends;
      __syncwarp();
      seg_n++;
      if (!more) break;
    }
    if (!split_out && member == 0 && lane == 0) t.split[2 * gang].x = 0;
  } else if (w == 0) {
    // ---- loads
    int st = 0;  // ring stages issued so far
    int qn = 0;  // items whose Q was issued
    bool bad_page = false;
    const int gpt = 1 << (7 - t.gsh);  // groups of a tile, one per lane
    // where this lane's group of a key tile lies; the table's entry is checked
    // when it is used, so that its latency is not waited for here
    struct Place {
      int page, row;
    };
    auto lookup = [&](const Seg &s, int kt) {
      const int ng = min(gpt, s.gr.n - kt * gpt);
      const int p0 = group_pos(s.gr, kt * gpt + min(lane, ng - 1), t.gsh), pi = page_index(a.kv, p0);
      return Place{a.kv.table[(long long)s.b * a.kv.table_stride + pi], p0 - pi * a.kv.page_size};
    };
    // one operand tile, nst stages of `chunks` chunks each: its boxes [g0, g1)
    auto load_tile = [&](const Seg &s, const Place &pl, const CUtensorMap *m, int nst, int chunks, int pitch, int chunk0,
                         int chunk_step, int g0, int g1) {
      int page = pl.page;
      if (page < 0 || page >= a.kv.n_pages) bad_page = true, page = a.kv.n_pages;  // past the pool: zeros
      const int kvh = uniform(s.kvh), n_box = uniform(g1 - g0), first = uniform(g0);
      for (int i = 0; i < nst && ok; i++) {
        const int slot = uniform(st % C::NST);
        if (st >= C::NST && !wait_warp(empty(slot), (st / C::NST - 1) & 1)) {
          ok = false;
          break;
        }
        const uint32_t dst = ring + slot * C::STAGE, bar = PAIR ? uniform(of_block(full(slot), 0)) : full(slot);
        const int x = uniform((chunk0 + i * chunk_step) * 64);
        if (elect_one()) {
          const uint32_t bytes = (chunks * 128u << t.gsh) * n_box;
          if (PAIR) expect_leader(full(slot), bytes);
          else mbar_arrive_expect_tx(bar, bytes);
        }
        for (int g = 0; g < n_box; g++) {
          const int pg = __shfl_sync(0xffffffffu, page, first + g), row = __shfl_sync(0xffffffffu, pl.row, first + g);
          const uint32_t to = dst + (g << (t.gsh + 7));
          if (elect_one()) {
            if (PAIR) {
              tma_4d_pair(to, m, x, row, kvh, pg, bar);
              if (chunks == 2) tma_4d_pair(to + pitch, m, x + 64, row, kvh, pg, bar);
            } else {
              tma_4d(to, m, x, row, kvh, pg, bar);
              if (chunks == 2) tma_4d(to + pitch, m, x + 64, row, kvh, pg, bar);
            }
          }
        }
        st++;
      }
    };
    auto load_k = [&](const Seg &s, int kt, const Place &pl) {
      const int ng = min(gpt, s.gr.n - kt * gpt), h = (ng + 1) >> 1;  // a pair: the first h boxes, the others
      load_tile(s, pl, &maps.k, C::KST, C::KC, C::KPITCH, 0, C::KC, PAIR && rank ? h : 0, PAIR && !rank ? h : ng);
    };
    auto load_v = [&](const Seg &s, int kt, const Place &pl) {
      const int ng = min(gpt, s.gr.n - kt * gpt);
      load_tile(s, pl, &maps.v, C::VST, C::VC, AT_CHUNK, half * (C::DV / 64) + rank, PAIR ? 2 : C::VC, 0, ng);
    };
    SegOf<MODE> s;
    while (ok && next_seg(s)) {
      if (s.kt0 >= s.kt1) continue;
      Place kp = lookup(s, s.kt0);
      for (int r = 0; r < NT && ok; r++) {
        if (qn > 0 && !wait_warp(b_qe + 8 * r, (qn - 1) & 1)) ok = false;
        const int qh = uniform(s.kvh * a.group), qt = uniform(s.row0 + (PAIR && ragged<MODE>(a) ? rank : r) * t.tpt);
        const uint32_t q_bar = PAIR ? uniform(of_block(b_qf, 0)) : 0;
        if (ok && elect_one()) {
          const uint32_t bytes = (D / 64) * t.tpt * a.group * 128;
          if (PAIR) expect_leader(b_qf, bytes);
          else mbar_arrive_expect_tx(b_qf + 8 * r, bytes);
          // rows past the call's last come in as zeros
#pragma unroll
          for (int c = 0; c < D / 64; c++) {
            if (PAIR) tma_3d_pair(q_sm + c * AT_CHUNK, &maps.q, c * 64, qh, qt, q_bar);
            else tma_3d(q_sm + (r * (D / 64) + c) * AT_CHUNK, &maps.q, c * 64, qh, qt, b_qf + 8 * r);
          }
        }
        __syncwarp();
      }
      qn++;
      // in the order in which the products use them: one row tile computes the
      // next tile's S before the current O
      if (NT == 1 && ok) load_k(s, s.kt0, kp);
      for (int kt = s.kt0; kt < s.kt1 && ok; kt++) {
        const Place vp = kp;
        if (kt + 1 < s.kt1) kp = lookup(s, kt + 1);
        if (NT == 2) load_k(s, kt, vp);
        else if (kt + 1 < s.kt1) load_k(s, kt + 1, kp);
        if (ok) load_v(s, kt, vp);
      }
    }
    if (bad_page) raise_flag(a.err, DS4MOE_DEVERR_PAGE);
    if (PAIR && ok) {
      // the leader's last arrivals have come in before the block leaves
      for (int i = max(0, st - C::NST); i < st; i++)
        if (!wait_warp(empty(i % C::NST), (i / C::NST) & 1)) ok = false;
      if (qn > 0 && !wait_warp(b_qe, (qn - 1) & 1)) ok = false;
    }
    if (PAIR && !ok) {
      // their landing is told to the leader alone: 10 ms, some thousand times what they need
      for (int i = 0; i < 100; i++) __nanosleep(100000);
    } else if (!ok) {
      // the copies in flight land before the block leaves (they need microseconds; a second full wait is not due)
      constexpr long long LAND = WAIT_LIMIT / 128;
      for (int i = max(0, st - C::NST); i < st; i++) mbar_wait_bounded(full(i % C::NST), (i / C::NST) & 1, LAND);
      for (int r = 0; r < NT; r++)
        if (qn > 0) mbar_wait_bounded(b_qf + 8 * r, (qn - 1) & 1, LAND);
    }
  } else if (w == 1) {
    // ---- products
    int st = 0, qn = 0;
    int steps = 0;  // (key tile, row tile) pairs before the current segment
    const uint32_t id_o = idesc<DT>(C::PV_N, true, PAIR ? 256 : 128);
    const uint32_t tmem_u = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dq = desc_sw128(q_sm, 0), dk = desc_sw128(ring, 0), dv = desc_sw128(ring, AT_CHUNK);
    int kst0 = 0, vst0 = 0;  // ring stages of the current key and value tile
    SegOf<MODE> s = {};
    auto wait_stage = [&](int i) {
      if (!wait_warp(full(i % C::NST), (i / C::NST) & 1)) ok = false;
    };
    auto commit = [&](uint32_t bar) {
      if (PAIR) umma_commit_pair(bar);
      else umma_commit(bar);
    };
    // S of key tile kt and row tile r, the segment's i-th such step
    auto qk = [&](int kt, int r, int i) {
      const int buf = NT == 2 ? r : uniform((steps + i) & 1);
      if (i < NT && !wait_warp(b_qf + 8 * r, (qn - 1) & 1)) ok = false;
      if (r == 0) kst0 = st, st += C::KST;
      // a pair's columns: as many of either block, in boxes
      const int boxes = min(1 << (7 - t.gsh), s.gr.n - (kt << (7 - t.gsh)));
      const int cols = PAIR ? ((boxes + 1) >> 1) << (t.gsh + 1) : 16 * cols16(s, kt, t.gsh);
      const uint32_t id = idesc<DT>(uniform(cols), false, PAIR ? 256 : 128);
      const uint32_t sd = tmem_u + buf * 128;
#pragma unroll
      for (int j = 0; j < C::KST; j++) {
        const int slot = uniform((kst0 + j) % C::NST);
        if (r == 0) wait_stage(kst0 + j);
        tc_fence_after();
        if (ok && elect_one()) {
          // descriptor addresses count 16 bytes
          const uint64_t qa = dq + ((r * (D / 64) + j * C::KC) * AT_CHUNK >> 4), kb = dk + (slot * C::STAGE >> 4);
#pragma unroll
          for (int c = 0; c < C::KC; c++)
#pragma unroll
            for (int k = 0; k < 4; k++) {
              const uint64_t qd = qa + (c * AT_CHUNK >> 4) + 2 * k, kd = kb + (c * C::KPITCH >> 4) + 2 * k;
              if (PAIR) umma_f16_pair(sd, qd, kd, id, (j | c | k) != 0);
              else umma_f16(sd, qd, kd, id, (j | c | k) != 0);
            }
          if (r == NT - 1) commit(empty(slot));
          if (j == C::KST - 1) {
            commit(b_sf + 8 * buf);
            if (kt + 1 == s.kt1) commit(b_qe + 8 * r);
          }
        }
        __syncwarp();
      }
    };
    // O of row tile r from its P of key tile kt
    auto pv = [&](int kt, int r, int i) {
      const int buf = NT == 2 ? r : uniform((steps + i) & 1), use = (steps + i) >> 1;
      const int n16 = uniform(cols16(s, kt, t.gsh)), later = uniform(kt != s.kt0);
      if (r == 0) {
        vst0 = st, st += C::VST;
        for (int j = 0; j < C::VST; j++) wait_stage(vst0 + j);
        // rows past the sequence's length: whatever the page holds there would
        // meet a weight of 0; zeros instead
        const int gpt = 1 << (7 - t.gsh), ng = min(gpt, s.gr.n - kt * gpt);
        const int live = ((ng - 1) << t.gsh) + s.len - group_pos(s.gr, kt * gpt + ng - 1, t.gsh);
        if (ok && live < 16 * n16) {
          const int n8 = (16 * n16 - live) * 8;
          for (int j = 0; j < C::VST * C::VC; j++)
            for (int e = lane; e < n8; e += 32) {
              const uint32_t p = ring + ((vst0 + j / C::VC) % C::NST) * C::STAGE + j % C::VC * AT_CHUNK + live * 128 + e * 16;
              asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(p), "r"(0) : "memory");
              if (PAIR)
                asm volatile("st.shared::cluster.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(of_block(p, 1)), "r"(0) : "memory");
            }
          if (PAIR) asm volatile("fence.proxy.async;" ::: "memory");
          else fence_proxy_async_smem();
          __syncwarp();
        }
        // nor do the positions of the first group count that lie before the
        // sequence's own
        const int head = s.lo - (s.gr.win0 << t.gsh);
        if (MODE == AT_OWN && ok && kt == 0 && head > 0) {
          for (int j = 0; j < C::VST * C::VC; j++)
            for (int e = lane; e < head * 8; e += 32) {
              const uint32_t p = ring + ((vst0 + j / C::VC) % C::NST) * C::STAGE + j % C::VC * AT_CHUNK + e * 16;
              asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(p), "r"(0) : "memory");
              if (PAIR)
                asm volatile("st.shared::cluster.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(of_block(p, 1)), "r"(0) : "memory");
            }
          if (PAIR) asm volatile("fence.proxy.async;" ::: "memory");
          else fence_proxy_async_smem();
          __syncwarp();
        }
      }
      uint64_t vb[C::VST];
      uint32_t eb[C::VST];
#pragma unroll
      for (int j = 0; j < C::VST; j++) {
        const int slot = uniform((vst0 + j) % C::NST);
        vb[j] = dv + (slot * C::STAGE >> 4), eb[j] = empty(slot);
      }
      const uint32_t o = tmem_u + C::O_COL + r * C::DV, pd = tmem_u + buf * 128;
      // P comes in two halves of 64 columns, from two warpgroups. An item's
      // first product overwrites the O that both have been reading.
#pragma unroll
      for (int h = 0; h < 2; h++) {
        if (ok && !later && h == 0 && !wait_warp(b_pb + 8 * buf, use & 1)) ok = false;
        if (ok && !wait_warp((h ? b_pb : b_pa) + 8 * buf, use & 1)) ok = false;
        tc_fence_after();
        if (ok && elect_one()) {
#pragma unroll
          for (int j = 0; j < C::VST; j++) {
#pragma unroll
            for (int k = 4 * h; k < 4 * h + 4; k++)
              if (k < n16) {
                const uint32_t od = o + j * C::PV_N;
                if (PAIR) umma_f16_ts_pair(od, pd + 8 * k, vb[j] + (2048 * k >> 4), id_o, later || k != 0);
                else umma_f16_ts(od, pd + 8 * k, vb[j] + (2048 * k >> 4), id_o, later || k != 0);
              }
            if (h == 1 && r == NT - 1) commit(eb[j]);
          }
          if (h == 1 && (NT == 1 || kt + 1 == s.kt1)) commit(b_of + 8 * r);
        }
        __syncwarp();
      }
    };
    while (ok && next_seg(s)) {
      if (s.kt0 >= s.kt1 || rank) continue;  // (the even block's products are the pair's)
      qn++;
      const int n = (s.kt1 - s.kt0) * NT;
      qk(s.kt0, 0, 0);
      for (int kt = s.kt0, i = 0; kt < s.kt1 && ok; kt++, i += NT) {
        // the next S before the current O
        if (NT == 2) {
          qk(kt, NT - 1, i + 1);
          pv(kt, 0, i);
          if (kt + 1 < s.kt1) qk(kt + 1, 0, i + 2);
          pv(kt, NT - 1, i + 1);
        } else {
          if (kt + 1 < s.kt1) qk(kt + 1, 0, i + 1);
          pv(kt, 0, i);
        }
      }
      steps += n;
    }
    if (!rank) {
      if (elect_one()) {
        if (PAIR) asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(b_done) : "memory");
        else umma_commit(b_done);
      }
      __syncwarp();
      mbar_wait_bounded(b_done, 0);  // nothing is in flight when the block leaves
    }
  } else if (w >= 4) {
    // ---- softmax and output: two warpgroups per row tile. A row belongs to
    // two threads, which take 64 columns of a tile each and agree on its
    // maximum through shared memory: half the latency between S and P, which
    // is what a row tile's products wait for.
    const int sw = w - 4, ch = sw >> 2 & 1, r = sw >> 3;
    const int row = (w & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((w & 3) * 32) << 16;
    const int tok = row / a.group, head = row - tok * a.group;  // within the tile and the key-value head
    // this block's first token of the row group
    const int tile0 = (PAIR && ragged<MODE>(a) ? rank : r) * t.tpt;
    const int my_tok = tok < t.tpt ? tile0 + tok : INT32_MAX;
    const uint32_t oa = tmem + lanes + C::O_COL + r * C::DV;
    const uint32_t b_pair = b_x + 8 * (r * 4 + (w & 3));
    int steps = 0;  // key tiles of this row tile so far
    int swaps = 0;  // values exchanged with the row's other thread
    // a value for the row's other thread, and the other's
    float *x_pair = &ms.x[0][0][0];
    auto tell = [&](float mine) {
      x_pair = &ms.x[NT == 2 ? r : swaps & 1][0][0];
      x_pair[ch * 128 + row] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(b_pair);
    };
    auto hear = [&](float &other) {
      if (!wait_warp(b_pair, swaps & 1)) return ok = false;
      swaps++;
      other = x_pair[(ch ^ 1) * 128 + row];
      return true;
    };
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(b_pair);
      if (!wait_warp(b_pair, swaps & 1)) return ok = false;
      swaps++;
      return true;
    };
    int items = 0;  // segments with tiles so far
    SegOf<MODE> s;
    while (ok && next_seg(s)) {
      const bool valid = my_tok < s.n;
      const int pos = valid ? s.pos0 + (MODE == AT_PREFIX ? 0 : my_tok) : -1;
      const int lo = MODE == AT_OWN ? s.lo : window_lo(a, max(pos, 0));
      // what every row of this tile sees: positions up to p_first, from lo_last
      const int p_first = s.pos0 + (MODE == AT_PREFIX ? 0 : tile0);
      const int lo_last = MODE == AT_OWN ? s.lo : window_lo(a, max(s.pos0 + s.n - 1, 0));
      const int shift = (s.gr.win0 - s.gr.n_sink) << t.gsh;
      float m = -INFINITY, l = 0.0f;
      for (int kt = s.kt0; kt < s.kt1; kt++, steps++) {
        const int buf = NT == 2 ? r : steps & 1, use = NT == 2 ? steps : steps >> 1;
        if (!wait_warp(b_sf + 8 * buf, use & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sa = tmem + lanes + buf * 128;
        float v[64];
        tmem_ld32(sa + 64 * ch, v);
        tmem_ld32(sa + 64 * ch + 32, v + 32);
        // columns c < cs: the first positions' groups, position 128 kt + c; others shifted
        const int cs = (s.gr.n_sink << t.gsh) - 128 * kt, off = 128 * kt + shift;
        const bool partly = cs > 0 || off + 127 > p_first || ((MODE == AT_OWN || a.window > 0) && off < lo_last);
        auto hide = [&](float *x, int c) {  // what the row does not see of its 32 columns c
          const int e0 = min(min(a.n_sink, pos + 1) - 128 * kt, cs), wd = 2 * ch + c;
          const uint32_t bits =
              range_bits(0, e0, wd) |
              ((range_bits(lo - off, pos + 1 - off, wd) | range_bits(0, min(a.n_sink, pos + 1) - off, wd)) &
               range_bits(cs, 128, wd));
#pragma unroll
          for (int i = 0; i < 32; i++)
            if (!(bits >> i & 1)) x[i] = -INFINITY;
        };
        tmem_wait_ld(v);
        tmem_wait_ld(v + 32);
        if (partly) hide(v, 0), hide(v + 32, 1);
        float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int i = 4; i < 60; i += 8) {
          mx[0] = max3(mx[0], v[i], v[i + 1]), mx[1] = max3(mx[1], v[i + 2], v[i + 3]);
          mx[2] = max3(mx[2], v[i + 4], v[i + 5]), mx[3] = max3(mx[3], v[i + 6], v[i + 7]);
        }
        mx[0] = max3(mx[0], v[60], v[61]), mx[1] = max3(mx[1], v[62], v[63]);
        float mt = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]), other;
        tell(mt);
        const unsigned long long sc2 = f2_pack(a.scale_log2, a.scale_log2);
        unsigned long long sum[2] = {0, 0};
        uint32_t p[16];
        auto weights = [&](const float *x) {  // of 32 columns, relative to m
          const float mz = m == -INFINITY ? 0.0f : m;
          const unsigned long long nm2 = f2_pack(-mz, -mz);
#pragma unroll
          for (int i = 0; i < 16; i++) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(x[2 * i], x[2 * i + 1]), sc2, nm2), x0, x1);
            x0 = ex2(x0), x1 = ex2(x1);
            sum[i & 1] = f2_add(sum[i & 1], f2_pack(x0, x1));
            p[i] = Half16<DT>::down(x0, x1);
          }
        };
        // the first 32 columns' weights with the maximum so far, while the
        // other thread's is on its way: it rarely changes
        weights(v);
        if (!hear(other)) break;
        mt = fmaxf(mt, other) * a.scale_log2 - AT_BIAS<DT>;
        const bool grow = mt > m + AT_LAZY || (m == -INFINITY && mt > m);
        if (__any_sync(0xffffffffu, grow)) {
          const float mn = grow ? mt : m;
          const float f = mn == -INFINITY ? 1.0f : ex2(m - mn);
          m = mn, l *= f;
          // O is the first warpgroup's to rescale: products start when its
          // half of P is there
          if (kt > s.kt0 && ch == 0) {
            // the last product into O has to be done; with two row tiles it
            // came before this S
            if (NT == 1 && !wait_warp(b_of, (steps - 1) & 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < C::DV; c += 16) {
              uint32_t x[16];
              asm volatile(
                  "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
                  "tcgen05.wait::ld.sync.aligned;"
                  : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]),
                    "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15])
                  : "r"(oa + c)
                  : "memory");
#pragma unroll
              for (int i = 0; i < 16; i++) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
              tmem_st16(oa + c, x);
            }
            tmem_wait_st();
          }
          // the first columns again (S is still there: P of these columns goes
          // over it, the other thread's P over the second 32 at most)
          float x[32];
          tmem_ld32(sa + 64 * ch, x);
          tmem_wait_ld(x);
          if (partly) hide(x, 0);
          sum[0] = sum[1] = 0;
          weights(x);
        }
        tmem_st16(sa + 32 * ch, p);
        weights(v + 32);
        tmem_st16(sa + 32 * ch + 16, p);
        // One row tile: every product into O is waited for before the next one
        // can end (a parity tells only neighbouring phases apart). It has
        // ended long since, in general.
        if (NT == 1 && kt > s.kt0 && !wait_warp(b_of, (steps - 1) & 1)) {
          ok = false;
          break;
        }
        tmem_wait_st();
        tc_fence_before();
        if (PAIR) {
          __syncwarp();
          if (lane == 0) arrive_leader((ch ? b_pb : b_pa) + 8 * buf);
        } else {
          mbar_arrive((ch ? b_pb : b_pa) + 8 * buf);
        }
        float s0, s1, s2, s3;
        f2_unpack(sum[0], s0, s1);
        f2_unpack(sum[1], s2, s3);
        l += (s0 + s1) + (s2 + s3);
      }
      if (!ok) break;
      const bool whole = s.starts && s.ends, none = s.kt0 >= s.kt1;
      const int tq = s.row0 + my_tok, hq = s.kvh * a.group + head;
      // each warpgroup stores half of O's columns (64: the first all of them)
      const int c0 = C::DV == 64 ? 0 : ch * (C::DV / 2), c1 = C::DV == 64 ? (ch ? 0 : 64) : c0 + C::DV / 2;
      const long long pre = valid ? (long long)tq * a.n_heads + hq : 0;  // the row among the AT_PREFIX results
      // AT_OWN: the rows' AT_PREFIX results, 32 columns at a time, the first
      // while the last product runs, the others one step ahead
      const long long pre_at = MODE == AT_OWN && whole && valid && s.lo > 0 ? pre * D + half * C::DV : -1;
      uint32_t z[32];
      float pre_log = -INFINITY;
      auto fetch = [&](int c) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const long long at = __shfl_sync(0xffffffffu, pre_at, (lane & 24) + i);
          uint4 u = make_uint4(0, 0, 0, 0);
          if (at >= 0 && c < c1) u = *reinterpret_cast<const uint4 *>(pre_results(a) + at + c + 4 * (lane & 7));
          z[4 * i] = u.x, z[4 * i + 1] = u.y, z[4 * i + 2] = u.z, z[4 * i + 3] = u.w;
        }
      };
      if (MODE == AT_OWN) {
        if (pre_at >= 0) pre_log = pre_logs(a)[pre];
        fetch(c0);
      }
      if (!none) {
        // the item's last product (two row tiles: the only one this barrier counts)
        if (!wait_warp(b_of + 8 * r, (NT == 1 ? steps - 1 : items) & 1)) {
          ok = false;
          break;
        }
        items++;
        tc_fence_after();
        float other;
        tell(l);
        if (!hear(other) || !meet()) break;  // both have read l when the next item writes
        l += other;
      }
      float inv = none || l == 0.0f ? 0.0f : 1.0f / l;
      float from = 0.0f;  // AT_OWN: the factor of the AT_PREFIX result
      bool zero = false;       // AT_OWN: no score above -infinity, neither here nor there
      if (MODE == AT_OWN && whole) join_two(pre_log, m, none ? 0.0f : l, from, inv, zero);
      const int slot = 2 * blockIdx.x + (s.starts ? 1 : 0);
      // rows 8 (lane / 8) + i are this lane's to store, 16 bytes at piece lane % 8
      float *pp = t.part + ((size_t)(slot * NT + r) * 128 + (w & 3) * 32 + (lane & 24)) * C::PITCH + 4 * (lane & 7);
      const long long own = valid ? (long long)tq * a.out_stride + (long long)hq * D + half * C::DV : -1;
      bool nan = false;
#pragma unroll 1
      for (int c = c0; c < c1; c += whole ? 64 : 32) {
        float x[32];
        uint32_t y[32];
        if (MODE == AT_PREFIX && whole) {
#pragma unroll
          for (int h = 0; h < 2; h++) {
            tmem_ld32(oa + c + 32 * h, x);
            tmem_wait_ld(x);
#pragma unroll
            for (int i = 0; i < 32; i++) y[i] = __float_as_uint(x[i] * inv);
            transpose8(y);
#pragma unroll
            for (int i = 0; i < 8; i++) {
              const long long at = __shfl_sync(0xffffffffu, valid ? pre : -1, (lane & 24) + i);
              if (at >= 0)
                *reinterpret_cast<uint4 *>(pre_results(a) + at * D + half * C::DV + c + 32 * h + 4 * (lane & 7)) =
                    make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
            }
          }
        } else if (whole) {
#pragma unroll
          for (int h = 0; h < 2; h++) {
            uint32_t zc[32];
            if (MODE == AT_OWN) {
#pragma unroll
              for (int i = 0; i < 32; i++) zc[i] = z[i];
              fetch(c + 32 * h + 32);
              transpose8(zc);
            }
            if (none) {
#pragma unroll
              for (int i = 0; i < 32; i++) x[i] = 0.0f;
            } else {
              tmem_ld32(oa + c + 32 * h, x);
              tmem_wait_ld(x);
            }
#pragma unroll
            for (int i = 0; i < 16; i++) {
              float x0 = x[2 * i] * inv, x1 = x[2 * i + 1] * inv;
              if (MODE == AT_OWN) {
                x0 = fmaf(from, __uint_as_float(zc[2 * i]), x0), x1 = fmaf(from, __uint_as_float(zc[2 * i + 1]), x1);
                if (zero) x0 = x1 = 0.0f;
              }
              nan |= x0 != x0 || x1 != x1;
              y[16 * h + i] = Half16<DT>::down(x0, x1);
            }
          }
          transpose8(y);
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const long long at = __shfl_sync(0xffffffffu, own, (lane & 24) + i);
            if (at >= 0)
              *reinterpret_cast<uint4 *>(a.out + at + c + 8 * (lane & 7)) =
                  make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          }
        } else {
          tmem_ld32(oa + c, x);
          tmem_wait_ld(x);
#pragma unroll
          for (int i = 0; i < 32; i++) y[i] = __float_as_uint(x[i]);
          transpose8(y);
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const int live = __shfl_sync(0xffffffffu, (int)valid, (lane & 24) + i);
            if (live)
              *reinterpret_cast<uint4 *>(pp + (size_t)i * C::PITCH + c) =
                  make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          }
        }
      }
      if (valid && !whole && ch == 0) {
        float *ml = t.part + ((size_t)(slot * NT + r) * 128 + row) * C::PITCH + C::DV;
        ml[0] = m, ml[1] = l;
      }
      if (MODE == AT_PREFIX && valid && whole && ch == 0 && half == 0) pre_logs(a)[pre] = log_sum(m, l);
      tc_fence_before();
      __syncwarp();  // other lanes have stored parts of these rows
      if (MODE == AT_PREFIX) continue;  // (a row sees all that the products read)
      const bool look = nan && valid && l == l;
      if (__any_sync(0xffffffffu, look))
        look_again<DT, D>(a, tq, hq, s.b, look ? (MODE == AT_ALL && l == 0.0f ? -1 : pos) : -2, half * C::DV + c0, half * C::DV + c1);
    }
  }
  if (!ok && lane == 0) raise_flag(a.err, DS4MOE_DEVERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (w == 1) {
    tc_fence_after();
    if (!PAIR) tmem_dealloc(tmem, 512);
  }
  if (PAIR) {
    // tensor memory is given back by both blocks, after both are done with it;
    // shared memory outlives the other block's arrivals
    __syncwarp();
    cluster_sync_all();
    if (w == 1) tmem_dealloc_pair(tmem, 512);
  }
}

// Adds up the partials of the row groups whose key tiles lie in several
// blocks' runs, in block order. Block (gang, member, row tile, rows); a thread
// takes four columns of R rows, with 8 / R partials of each in flight. The
// kernel is all latency: ragged calls (many split row groups of two or three
// partials) take R = 4, one wave of blocks instead of four; decode calls (few
// rows, up to a partial per gang) R = 1, four times the threads. Registers are
// limited to what the sums need (12291 tokens of 32/8 heads of 128: 13.8 -> 11.8
// us), not the rows computed once more.
constexpr int AJ_THREADS = 256;

// Rows r0 + i with bit i of `again` (a NaN, but not in their sum of weights), by
// the block's warps in turn; d0, d1: the item, as in k_attn_join.
template <int DT, int D, int NT, bool PAIR, int MODE, int ROWS>
__device__ __noinline__ void join_again(const AttnArgs &a, const TileArgs &t, unsigned long long again) {
  using C = TileCfg<D, NT, PAIR>;
  const int r0 = blockIdx.x % (128 / ROWS) * ROWS, r = blockIdx.x / (128 / ROWS) % NT;
  const int bid = blockIdx.x / (128 / ROWS * NT);
  const int gang = bid / t.members, member = bid % t.members;
  const int half = PAIR ? member >> 1 & 1 : member % C::HALVES;
  const int rt = PAIR ? (member >> 2) * 2 + (member & 1) : member / C::HALVES;
  const int4 d0 = t.split[2 * gang], d1 = t.split[2 * gang + 1];
  const int tok0 = (rt + r) * t.tpt, c0 = half * C::DV, c1 = c0 + C::DV;
  bool bad = false;
  const int last = d0.w + d1.y - 1;
  const Groups gr = range_groups(a, d0.w, last, t.gsh);  // as the item's blocks listed them
  const int win0 = gr.win0 << t.gsh, sinks = gr.n_sink << t.gsh, end = min(seq_len(a, d0.y, bad), (last | 15) + 1);
  const int p0 = d0.w + tok0 + (r0 + __ffsll(again) - 1) / a.group, p1 = d0.w + tok0 + (r0 + 63 - __clzll(again)) / a.group;
  if (!unseen_nonfinite<DT>(a, d0.y, d0.z, p0, p1, win0, sinks, end, c0, c1)) return;
  for (int i = threadIdx.x >> 5; i < 64; i += AJ_THREADS / 32)
    if (again >> i & 1) {
      const int row = r0 + i, tok = tok0 + row / a.group, pos = d0.w + tok, h = d0.z * a.group + row % a.group;
      if (!own_nan<DT>(a, a.out + (long long)(d1.x + tok) * a.out_stride + (long long)h * D, d0.y, d0.z, pos, c0, c1) &&
          unseen_nonfinite<DT>(a, d0.y, d0.z, pos, pos, win0, sinks, end, c0, c1))
        redo_row_cols<DT, D>(a, d1.x + tok, h, d0.y, pos, c0, c1);
    }
}

template <int DT, int D, int NT, bool PAIR, int MODE, int R>
__global__ void __launch_bounds__(AJ_THREADS, MODE == AT_PREFIX ? 2 : D * R < 512 || D == 128 ? 4 : D * R <= 1024 ? 3 : 2)
    k_attn_join(const __grid_constant__ Args<MODE> a, const __grid_constant__ TileArgs t) {
  using C = TileCfg<D, NT, PAIR>;
  constexpr int ROWS = C::JROWS * R, STEP = C::JROWS, P = MODE == AT_PREFIX ? 16 : 8 / R;  // rows of the block; distance of a thread's rows
  __shared__ unsigned long long s_nan;
  const int tid = threadIdx.x;
  const int r0 = blockIdx.x % (128 / ROWS) * ROWS, r = blockIdx.x / (128 / ROWS) % NT;
  const int jid = blockIdx.x / (128 / ROWS * NT), member = jid % t.members;
  const int half = PAIR ? member >> 1 & 1 : member % C::HALVES;
  const int rt = PAIR ? (member >> 2) * 2 + (member & 1) : member / C::HALVES;
  pdl_launch_dependents();
  pdl_wait();
  // The gang in whose run a split item starts: this block's, or (AT_PREFIX, whose
  // items are few, so that most gangs have none) those of a part of the gangs.
  int gang = jid / t.members, gang1 = gang + 1;
  if (MODE == AT_PREFIX) {
    const int j = gang;
    gang = t.gangs * j / t.join, gang1 = t.gangs * (j + 1) / t.join;  // (one at least)
  }
  do {
    const int bid = gang * t.members + member;
    const int4 d0 = t.split[2 * gang], d1 = t.split[2 * gang + 1];
    const int parts = d0.x;
    if (MODE == AT_PREFIX && parts == 0) continue;
    if (parts == 0) return;
    const int tok0 = (rt + r) * t.tpt;  // one of the two is 0
    const int rows = min(t.tpt, d1.y - tok0) * a.group;
    if (MODE == AT_PREFIX && r0 >= rows) continue;
    if (r0 >= rows) return;
    if (tid == 0) s_nan = 0;
    __syncthreads();
    const int row0 = r0 + tid / (C::DV / 4), c = tid % (C::DV / 4) * 4;
    float m[R], l[R];
    float4 x[R];
    // AT_OWN: the rows' AT_PREFIX results (R = 1)
    float pre_log[R];
    float4 pre_x[R];
    auto pre_of = [&](int k) {
      const int row = row0 + k * STEP;
      return (long long)(d1.x + tok0 + row / a.group) * a.n_heads + d0.z * a.group + row % a.group;
    };
#pragma unroll
    for (int k = 0; k < R; k++) {
      pre_log[k] = -INFINITY, pre_x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (MODE == AT_OWN && d1.z > 0 && row0 + k * STEP < rows)
        pre_log[k] = pre_logs(a)[pre_of(k)], pre_x[k] = *reinterpret_cast<const float4 *>(pre_results(a) + pre_of(k) * D + half * C::DV + c);
    }
#pragma unroll
    for (int k = 0; k < R; k++) m[k] = -INFINITY, l[k] = 0.0f, x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int p0 = 0; p0 < parts; p0 += P) {
      float2 ml[R][P];
      float4 y[R][P];
#pragma unroll
      for (int i = 0; i < P; i++) {
        // the block where the item starts holds it in its second slot, the others in their first
        const int slot = 2 * (bid + (p0 + i) * t.members) + (p0 + i == 0 ? 1 : 0);
        const float *q0 = t.part + ((size_t)(slot * NT + r) * 128 + row0) * C::PITCH;
#pragma unroll
        for (int k = 0; k < R; k++) {
          ml[k][i] = make_float2(-INFINITY, 0.0f), y[k][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (p0 + i < parts && row0 + k * STEP < rows) {
            const float *q = q0 + (size_t)k * STEP * C::PITCH;
            ml[k][i] = *reinterpret_cast<const float2 *>(q + C::DV), y[k][i] = *reinterpret_cast<const float4 *>(q + c);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < R; k++) {
        float mn = m[k];
#pragma unroll
        for (int i = 0; i < P; i++) mn = fmaxf(mn, ml[k][i].x);
        const float f = mn == -INFINITY ? 1.0f : ex2(m[k] - mn);
        m[k] = mn, l[k] *= f, x[k].x *= f, x[k].y *= f, x[k].z *= f, x[k].w *= f;
#pragma unroll
        for (int i = 0; i < P; i++) {
          const float g = ml[k][i].x == -INFINITY ? 0.0f : ex2(ml[k][i].x - mn);
          const float4 z = y[k][i];
          l[k] = fmaf(g, ml[k][i].y, l[k]);
          x[k].x = fmaf(g, z.x, x[k].x), x[k].y = fmaf(g, z.y, x[k].y), x[k].z = fmaf(g, z.z, x[k].z), x[k].w = fmaf(g, z.w, x[k].w);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < R; k++) {
      const int row = row0 + k * STEP;
      if (row >= rows) continue;
      // (AT_PREFIX without a score above -infinity: a value's NaN stays for the join)
      float inv = MODE == AT_PREFIX && l[k] == 0.0f ? 0.0f : 1.0f / l[k], from = 0.0f;
      bool zero = MODE != AT_PREFIX && l[k] == 0.0f;
      if (MODE == AT_OWN) join_two(pre_log[k], m[k], l[k], from, inv, zero);
      float4 z = make_float4(x[k].x * inv, x[k].y * inv, x[k].z * inv, x[k].w * inv);
      if (MODE != AT_OWN && zero) z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (MODE == AT_PREFIX) {
        *reinterpret_cast<float4 *>(pre_results(a) + pre_of(k) * D + half * C::DV + c) = z;
        if (c == 0 && half == 0) pre_logs(a)[pre_of(k)] = log_sum(m[k], l[k]);
        continue;
      }
      if (MODE == AT_OWN) {
        const float4 p = pre_x[k];
        z.x = fmaf(from, p.x, z.x), z.y = fmaf(from, p.y, z.y), z.z = fmaf(from, p.z, z.z), z.w = fmaf(from, p.w, z.w);
        if (zero) z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      if (l[k] == l[k] && (z.x != z.x || z.y != z.y || z.z != z.z || z.w != z.w)) atomicOr(&s_nan, 1ull << (row - r0));
      const int tok = row / a.group, h = d0.z * a.group + row % a.group;
      *reinterpret_cast<uint2 *>(a.out + (long long)(d1.x + tok0 + tok) * a.out_stride + (long long)h * D + half * C::DV + c) =
          make_uint2(Half16<DT>::down(z.x, z.y), Half16<DT>::down(z.z, z.w));
    }
    __syncthreads();
    const unsigned long long again = s_nan;
    if (MODE != AT_PREFIX && again) join_again<DT, D, NT, PAIR, MODE, ROWS>(a, t, again);
  } while (MODE == AT_PREFIX && ++gang < gang1);
}

// The marked rows (AT_MARK), all in items that a block of the tile kernel did
// alone: a block for each of its blocks.
template <int DT, int D, int NT, bool PAIR, int MODE>
__global__ void __launch_bounds__(AJ_THREADS)
    k_attn_mend(const __grid_constant__ Args<MODE> a, const __grid_constant__ TileArgs t) {
  using C = TileCfg<D, NT, PAIR>;
  pdl_launch_dependents();
  pdl_wait();
  if (!a.marked[blockIdx.x]) return;
  constexpr int COLS = C::DV == 64 ? 64 : C::DV / 2;  // of a warp of the tile kernel
  const int gang = blockIdx.x / t.members, member = blockIdx.x % t.members, rank = PAIR ? member & 1 : 0;
  const int half = PAIR ? member >> 1 & 1 : member % C::HALVES, rt = PAIR ? (member >> 2) * 2 + rank : member / C::HALVES;
  const int tile0 = PAIR && ragged<MODE>(a) ? rank * t.tpt : 0;
  Sched<MODE> sc;
  SegOf<MODE> s;
  bool bad = false;
  bool more = sc.init(a, t, gang, C::SPAN, bad);
  while (more && sc.next(a, t, rt, s)) {
    if (!s.starts || !s.ends || s.kt0 >= s.kt1) continue;
    for (int i = threadIdx.x >> 5; i < min(NT * t.tpt, s.n - tile0) * a.group; i += AJ_THREADS / 32) {
      const int tok = tile0 + i / a.group, tq = s.row0 + tok, hq = s.kvh * a.group + i % a.group;
      for (int c = half * C::DV; c < (half + 1) * C::DV; c += COLS)
        if (a.out[(long long)tq * a.out_stride + (long long)hq * D + c] == AT_MARK)
          redo_row_cols<DT, D>(a, tq, hq, s.b, s.pos0 + tok, c, c + COLS);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) a.marked[blockIdx.x] = 0;
}

// ---------------------------------------------------------------------------

namespace {

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
  static const EncodeTiled fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return (EncodeTiled)p;
  }();
  return fn;
}

// `n` dimensions, innermost first; strides in elements from the second on.
bool make_map(CUtensorMap *m, int dtype, const void *ptr, int n, const cuuint64_t *dims, const long long *strides,
              const cuuint32_t *box) {
  cuuint64_t sb[4];
  for (int i = 0; i + 1 < n; i++) sb[i] = (cuuint64_t)strides[i] * 2;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return encode_fn()(m, dtype == DS4MOE_DT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, n,
                     const_cast<void *>(ptr), dims, sb, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// log2 of a group's positions: groups lie within pages, and a window of W
// positions reads up to two groups too many, so at most W / 4. (Issuing a box
// costs the loading warp about as long as 2 KB take to arrive.)
int box_shift(int page_size, int window, int most) {
  int sh = 4;
  while (sh < most && page_size % (32 << (sh - 4)) == 0 && (window == 0 || window / 4 >= 32 << (sh - 4))) sh++;
  return sh;
}

struct TileFns {
  const void *tile, *join, *mend;
  int nt, halves, jrows, threads, span;
};

template <int DT, int D, int NT, bool PAIR, int MODE, bool RAGGED>
TileFns fns() {
  using C = TileCfg<D, NT, PAIR>;
  // a key tile's stages are freed one by one, a value tile's are all held at once
  static_assert(C::NST > C::VST && (NT == 1 || C::NST > 2 * C::KST) && C::NST <= 12, "ring");
  // (AT_PREFIX: few items of many partials, as a decode call)
  constexpr int R = RAGGED && MODE != AT_PREFIX ? 4 : 1;
  // (rows of AT_PREFIX see all that the products read: none is computed once more)
  const void *mend = nullptr;
  if constexpr (MODE != AT_PREFIX) mend = (const void *)k_attn_mend<DT, D, NT, PAIR, MODE>;
  return {(const void *)k_attn_tile<DT, D, NT, PAIR, MODE>, (const void *)k_attn_join<DT, D, NT, PAIR, MODE, R>, mend, NT,
          C::HALVES, C::JROWS * R, C::THREADS, C::SPAN};
}

template <int DT, int MODE, bool RAGGED>
TileFns fns_of(int D, bool pair) {
  constexpr int NT = RAGGED ? 2 : 1;
  if (D == 64) return fns<DT, 64, NT, false, MODE, RAGGED>();
  if (D == 128) return fns<DT, 128, NT, false, MODE, RAGGED>();
  if (D == 256) return fns<DT, 256, 1, false, MODE, RAGGED>();
  return pair ? fns<DT, 512, 1, true, MODE, RAGGED>() : fns<DT, 512, 1, false, MODE, RAGGED>();
}

template <int MODE>
TileFns tile_fns(int dtype, int D, bool ragged, bool pair) {
  constexpr int B = DS4MOE_DT_BF16, F = DS4MOE_DT_F16;
  if constexpr (MODE != AT_OWN)
    if (ragged) return dtype == B ? fns_of<B, MODE, true>(D, pair) : fns_of<F, MODE, true>(D, pair);
  if constexpr (MODE != AT_PREFIX)
    if (!ragged) return dtype == B ? fns_of<B, MODE, false>(D, pair) : fns_of<F, MODE, false>(D, pair);
  return {};
}

constexpr int AT_DYN = AT_MISC + AT_SMEM;

template <int MODE>
cudaError_t set_tile_attributes(int dtype, int D) {
  if (!encode_fn()) return cudaErrorNotSupported;
  for (bool ragged : {false, true})
    for (bool pair : {false, true}) {
      if ((ragged && MODE == AT_OWN) || (!ragged && MODE == AT_PREFIX)) continue;
      const cudaError_t e =
          cudaFuncSetAttribute(tile_fns<MODE>(dtype, D, ragged, pair).tile, cudaFuncAttributeMaxDynamicSharedMemorySize, AT_DYN);
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

template <int MODE>
cudaError_t launch_tile(const Args<MODE> &a, int D, int dtype, const TileWork &w, int n_sm, int *launches, cudaStream_t s) {
  const bool ragged = MODE == AT_ALL ? a.cu_q != nullptr : MODE == AT_PREFIX;
  TileArgs t = {};
  t.tpt = 128 / a.group;
  int row_tiles = ragged ? 1 : (a.n_new + t.tpt - 1) / t.tpt;
  // Dimension 512: pairs, where they fit nearly all SMs, for two row tiles and
  // more (a ragged call's row groups have two; an odd one of a decode call goes
  // with an empty one: three, 8 sequences of 16384, 145 us alone, 127 us so; a
  // single one 70 us alone, 75 us so).
  const bool pair = (ragged || row_tiles > 1) && w.pairs * 16 >= n_sm * 7;
  if (pair && !ragged) row_tiles = (row_tiles + 1) & ~1;
  const TileFns f = tile_fns<MODE>(dtype, D, ragged, pair);
  t.members = row_tiles * f.halves * (pair && ragged ? 2 : 1);
  t.gangs = (pair ? std::min(n_sm, 2 * w.pairs) : n_sm) / t.members;
  t.gsh = box_shift(a.kv.page_size, a.window, pair ? 6 : 7);
  // A window bounds an item's tiles: up to AT_WHOLE of them an item stays in one
  // block, and there is nothing to join.
  const long long reach = (long long)a.window + (ragged ? f.span * t.tpt : a.n_new) + a.n_sink + (2 << t.gsh);
  t.whole = a.window > 0 && reach <= AT_WHOLE * 128;
  // (a split item is a row group's, of at most so many)
  t.join = (int)std::min<long long>(t.gangs, 2ll * a.n_kv * (a.n_tok / (f.span * t.tpt) + a.n_seq));
  t.first = w.first, t.info = (int2 *)w.info, t.count = w.count, t.part = w.part, t.split = (int4 *)w.split;
  TileMaps maps;
  const cuuint64_t qd[3] = {(cuuint64_t)D, (cuuint64_t)a.n_heads, (cuuint64_t)a.n_tok};
  const long long qs[2] = {D, a.q_stride};
  const cuuint32_t qb[3] = {64, (cuuint32_t)a.group, (cuuint32_t)t.tpt};
  const cuuint64_t kd[4] = {(cuuint64_t)D, (cuuint64_t)a.kv.page_size, (cuuint64_t)a.n_kv, (cuuint64_t)a.kv.n_pages};
  const long long ks[3] = {a.kv.k_row, a.kv.k_head, a.kv.k_page}, vs[3] = {a.kv.v_row, a.kv.v_head, a.kv.v_page};
  const cuuint32_t kb[4] = {64, 1u << t.gsh, 1, 1};
  if (!make_map(&maps.q, dtype, a.q, 3, qd, qs, qb) || !make_map(&maps.k, dtype, a.kv.k, 4, kd, ks, kb) ||
      !make_map(&maps.v, dtype, a.kv.v, 4, kd, vs, kb))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  int span = f.span * t.tpt;
  Args<MODE> p = a;
  p.span = ragged ? span : a.n_new, p.gsh = t.gsh, p.marked = w.marked;
  if (ragged && a.n_seq <= 32 && a.n_tok / span + a.n_seq <= AT_WALK) t.first = nullptr;
  if (ragged && t.first) {
    p.cu_q = w.cu;
    void *args[] = {&p, (void *)&a.cu_q, (void *)&w.cu, &span, &t.gsh, &t.first, &t.info, &t.count, (void *)&w.seq_first};
    e = launch_pdl((const void *)k_attn_plan<MODE == AT_OWN ? AT_ALL : MODE>, dim3(1), dim3(1024), 0, s, args, true);
    ++*launches;
  }
  if (e == cudaSuccess) {
    void *args[] = {&maps, &p, &t};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(t.gangs * t.members), cfg.blockDim = dim3(f.threads), cfg.dynamicSmemBytes = AT_DYN, cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr, cfg.numAttrs = pair ? 2 : 1;
    e = cudaLaunchKernelExC(&cfg, f.tile, args);
    ++*launches;
  }
  if (e == cudaSuccess && !t.whole) {
    void *args[] = {&p, &t};
    e = launch_pdl(f.join, dim3((MODE == AT_PREFIX ? t.join : t.gangs) * t.members * f.nt * (128 / f.jrows)), dim3(AJ_THREADS), 0,
                   s, args, true);
    ++*launches;
  }
  if (e == cudaSuccess && f.mend && !t.whole && (long long)a.kv.width * a.kv.page_size >= AT_REDO &&
      (a.window == 0 || (long long)a.window + a.n_sink >= AT_REDO)) {
    void *args[] = {&p, &t};
    e = launch_pdl(f.mend, dim3(t.gangs * t.members), dim3(AJ_THREADS), 0, s, args, true);
    ++*launches;
  }
  return e;
}

}  // namespace

}  // namespace ds4
