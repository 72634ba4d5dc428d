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
// the first part costs more than it saves (shared_worth), read everything in
// the second part. One group of all sequences needs no planning launch.
#include "attn_tile.cuh"

namespace ds4 {

// Groups' bounds, ascending in [0, n_seq] (see clean_rows), as rows; the shared
// positions that are read once, and the first sequence that reaches past them,
// through whose table that happens; where each sequence's own positions begin.
__global__ void __launch_bounds__(1024) k_shared_plan(const AttnArgs a, const int32_t *group_start, int n_groups, int32_t *cu,
                                                  int32_t *plen, int32_t *ptab, int32_t *start) {
  __shared__ int s_top[32], s_base;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  pdl_wait();
  if (tid == 0) s_base = 0;
  for (int b = tid; b < a.batch; b += 1024) start[b] = 0;
  __syncthreads();
  bool bad = false;
  if (!group_start) {
    if (tid == 0) cu[0] = 0, cu[1] = a.batch * a.n_new;
  } else {
    for (int g0 = 0; g0 < n_groups; g0 += 1024) {
      const int g = g0 + tid;
      const int2 c = clean_rows(group_start, n_groups, a.batch, g, &s_base, s_top, bad);
      if (g < n_groups) cu[g] = c.x * a.n_new;
      if (g + 1 == n_groups) cu[n_groups] = c.y * a.n_new;
    }
  }
  __syncthreads();
  for (int g = w; g < n_groups; g += 32) {
    const int b0 = cu[g] / a.n_new, b1 = cu[g + 1] / a.n_new;
    const int s = shared_of(a, g, bad);
    int first = INT32_MAX;
    if (shared_worth(s, b1 - b0))
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

cudaError_t attn_shared_set_attributes(int dtype, int D) {
  const cudaError_t e = set_tile_attributes<AT_PREFIX>(dtype, D);
  return e == cudaSuccess ? set_tile_attributes<AT_OWN>(dtype, D) : e;
}

cudaError_t launch_attn_prefix(AttnArgs &a, const int32_t *group_start, int n_groups, int D, int dtype, const TileWork &w,
                               const SharedWork &sw, int n_sm, int *launches, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  // one group of all sequences is walked by every block itself (AT_WALK row
  // groups, of a row at least)
  if (group_start || a.n_tok >= AT_WALK) {
    int32_t *cu = w.cu;
    void *args[] = {&a, &group_start, &n_groups, &cu, (void *)&sw.plen, (void *)&sw.ptab, (void *)&sw.start};
    e = launch_pdl((const void *)k_shared_plan, dim3(1), dim3(1024), 0, s, args, true);
    ++*launches;
    a.plen = sw.plen, a.ptab = sw.ptab, a.start = sw.start;
  }
  AttnArgs p = a;
  p.n_seq = n_groups, p.cu_q = a.start ? w.cu : nullptr;
  if (e == cudaSuccess) e = launch_tile<AT_PREFIX>(p, D, dtype, w, n_sm, launches, s);
  return e;
}

cudaError_t launch_attn_own(const AttnArgs &a, int D, int dtype, const TileWork &w, int n_sm, int *launches, cudaStream_t s) {
  return launch_tile<AT_OWN>(a, D, dtype, w, n_sm, launches, s);
}

}  // namespace ds4
