// attn_tile.cu -- the tile kernel (attn_tile.cuh) over every position that a row
// sees: prefill, and decode calls that the streaming kernel does not take.
#include "attn_tile.cuh"

namespace ds4 {

size_t attn_tile_part_floats(int D, int n_sm) {
  const int dv = D < 256 ? D : 256, nt = D <= 128 ? 2 : 1;
  return (size_t)2 * n_sm * nt * 128 * (dv + 4);
}

size_t attn_tile_groups(int group, int D, int max_tokens, int max_seqs) {
  const int nt = D <= 128 ? 2 : 1, span = nt * (128 / group);
  return (size_t)max_tokens / span + max_seqs + 1;
}

cudaError_t attn_tile_set_attributes(int dtype, int D) { return set_tile_attributes<AT_ALL>(dtype, D); }

// Pairs of blocks of dimension 512 that run at once, 0 where there are none.
int attn_tile_pairs(int dtype, int D) {
  if (D != 512) return 0;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  const TileFns f = tile_fns<AT_ALL>(dtype, D, true, true);
  cfg.gridDim = dim3(2), cfg.blockDim = dim3(f.threads), cfg.dynamicSmemBytes = AT_DYN;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2, at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at, cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, f.tile, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

cudaError_t launch_attn_tile(const AttnArgs &a, int D, int dtype, const TileWork &w, int n_sm, int *launches,
                             cudaStream_t s) {
  return launch_tile<AT_ALL>(a, D, dtype, w, n_sm, launches, s);
}

}  // namespace ds4
