// attn_shared.cu -- decode attention of a batch whose sequences begin with the
// same positions (a system prompt, a document): those are read once for all.
//
// A row's result over shared and own positions is joined from two:
//   out = (2^(Lp - M) Op + 2^(Ls - M) Os) / (2^(Lp - M) + 2^(Ls - M)),
//   L = log2 of the sum of weights, M the larger one.
//   1. Op, Lp: the rows of all the group's sequences are the rows of one matrix
//      product per key-value head (the tile kernel, AT_PREFIX): every shared key
//      and value comes out of HBM once and meets up to 256 rows in each block.
//   2. Os, and the join: every sequence over its own positions, by the streaming
//      kernel (few rows of a short head) or the tile kernel (AT_OWN), which read
//      Op and Lp as they write the output. Op stays in 32 bits.
// Sequences that do not reach past the shared positions, and groups for which
// the first part costs more than it saves (share_cost), read everything in
// the second part.
#include "attn_tile.cuh"

namespace ds4 {

constexpr float SHARE_LEAST = 20000.0f;

// Groups' bounds, ascending in [0, n_seq] (see clean_rows), as rows; the shared
// positions that are read once, and the first sequence that reaches past them,
// through whose table that happens; where each sequence's own positions begin.
__global__ void __launch_bounds__(1024) k_shared_plan(const SharedArgs a, int32_t *cu, int32_t *plen, int32_t *ptab, int32_t *start) {
  __shared__ int s_top[32], s_base;
  __shared__ float s_gain[32];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, n_groups = a.n_groups;
  pdl_launch_dependents();
  pdl_wait();
  if (tid == 0) s_base = 0;
  for (int b = tid; b < a.batch; b += 1024) start[b] = 0;
  __syncthreads();
  bool bad = false;
  if (!a.group_start) {
    if (tid == 0) cu[0] = 0, cu[1] = a.batch * a.n_new;
  } else {
    for (int g0 = 0; g0 < n_groups; g0 += 1024) {
      const int g = g0 + tid;
      const int2 c = clean_rows(a.group_start, n_groups, a.batch, g, &s_base, s_top, bad);
      if (g < n_groups) cu[g] = c.x * a.n_new;
      if (g + 1 == n_groups) cu[n_groups] = c.y * a.n_new;
    }
  }
  __syncthreads();
  // Launches, partials and joins cost the call once; a group shares when it gains
  // a little and all of them pay for that.
  float gain = 0.0f;
  for (int g = tid; g < n_groups; g += 1024) {
    const float x = a.cost.gain(shared_of(a, g, bad), (cu[g + 1] - cu[g]) / a.n_new);
    if (x > a.cost.least / 16) gain += x;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) gain += __shfl_xor_sync(0xffffffffu, gain, o);
  if (lane == 0) s_gain[w] = gain;
  __syncthreads();
  gain = 0.0f;
  for (int i = 0; i < 32; i++) gain += s_gain[i];
  const bool pays = gain > a.cost.least;
  for (int g = w; g < n_groups; g += 32) {
    const int b0 = cu[g] / a.n_new, b1 = cu[g + 1] / a.n_new;
    const int s = shared_of(a, g, bad);
    int first = INT32_MAX;
    if (pays && s > 0 && a.cost.gain(s, b1 - b0) > a.cost.least / 16)
      for (int b = b0 + lane; b < b1; b += 32) {
        bool wrong = false;
        if (seq_len(a, b, wrong) - a.n_new + 1 < s) continue;
        start[b] = s, first = min(first, b);
      }
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) plen[g] = first == INT32_MAX ? 0 : s, ptab[g] = first == INT32_MAX ? 0 : first;
  }
  if (bad) raise_flag(a.err, DS4MOE_DEVERR_LENGTH);
}

// Measured with bf16, own parts of 200 positions, 2 to 64 sequences (us, plain and
// shared; without this rule):
//   32/8 heads of 128         64 x 1024: 46, 42; 64 x 32768: 783, 81; 8 x 32768: 107, 57; 2 x 32768: 39, 56
//   16/4 heads of 64          64 x 2048: 35, 33; 64 x 32768: 350, 50
//   64 heads over 1 of 512    64 x 4096: 87, 87; 64 x 32768: 592, 262; four new tokens 64 x 32768: 871, 924
// Plain, the sequences' copies of a position come out of L2 at some 11 TB/s (heads
// of 64: 6.4), or its products bound it, in tiles of 128 rows; shared, its bytes
// come once out of HBM, with joins beside them, and the products of all rows run
// at some 1.25 PFLOP/s. Where a sequence fills its tiles already, sharing gains
// nothing.
ShareCost share_cost(const ds4moe_attn_desc &d, int n_seq, int n_new) {
  const float bytes = 4.0f * d.n_kv_heads * d.head_dim;
  const int rows = n_new * (d.n_heads / d.n_kv_heads);
  const bool streams = rows <= AD_MAX_ROWS && d.head_dim <= 128;
  ShareCost c;
  c.seq = bytes / (d.head_dim == 64 ? 6400.0f : 11000.0f);
  if (!streams) c.seq = std::max(c.seq, 4.0f * ((rows + 127) / 128 * 128) * d.n_kv_heads * d.head_dim / 1.6e6f);
  c.read = bytes / 5000.0f;
  c.rows = 4.0f * rows * d.n_kv_heads * d.head_dim / 1.25e6f;
  // the tile kernel's own parts: a block's items one after another, some 14 us each with their joins
  c.least = SHARE_LEAST + (streams ? 0.0f : 95.0f * n_seq * d.n_kv_heads * ((rows + 127) / 128) * (d.head_dim == 512 ? 2 : 1));
  return c;
}

cudaError_t attn_shared_set_attributes(int dtype, int D) {
  const cudaError_t e = set_tile_attributes<AT_PREFIX>(dtype, D);
  return e == cudaSuccess ? set_tile_attributes<AT_OWN>(dtype, D) : e;
}

cudaError_t launch_attn_prefix(SharedArgs &a, int D, int dtype, const TileWork &w, const SharedWork &sw, int n_sm, int *launches,
                               cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  // one group, of no more than AT_WALK row groups of a row at least: no planning launch (3 us)
  if (a.n_groups > 1 || a.n_tok >= AT_WALK) {
    int32_t *cu = w.cu;
    void *args[] = {&a, &cu, (void *)&sw.plen, (void *)&sw.ptab, (void *)&sw.start};
    e = launch_pdl((const void *)k_shared_plan, dim3(1), dim3(1024), 0, s, args, true);
    ++*launches;
    a.plen = sw.plen, a.ptab = sw.ptab, a.start = sw.start;
  }
  SharedArgs p = a;
  p.n_seq = a.n_groups, p.cu_q = a.start ? w.cu : nullptr;
  if (e == cudaSuccess) e = launch_tile<AT_PREFIX>(p, D, dtype, w, n_sm, launches, s);
  return e;
}

cudaError_t launch_attn_own(const SharedArgs &a, int D, int dtype, const TileWork &w, int n_sm, int *launches, cudaStream_t s) {
  return launch_tile<AT_OWN>(a, D, dtype, w, n_sm, launches, s);
}

}  // namespace ds4
