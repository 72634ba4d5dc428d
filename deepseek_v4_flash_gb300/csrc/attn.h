// attn.h -- the attention handle, the arguments of its kernels and the
// launchers shared by attn.cu and the kernel translation units.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "ds4moe.h"

namespace ds4 {

// A paged cache as the kernels see it: strides in elements.
struct KvView {
  const uint16_t *k, *v;
  long long k_page, k_row, k_head, v_page, v_row, v_head;
  const int32_t *table;      // [n_seq][table_stride]
  long long table_stride;
  int32_t page_size, width;  // width: entries of a sequence's table row
  int32_t n_pages;
  uint32_t div_mul, div_sh;  // page number of a position (page_index)
};

// One attention call. Tokens of sequence b are rows tok0(b) .. tok0(b) +
// n_b - 1 of q; the j-th has position len(b) - n_b + j.
struct AttnArgs {
  KvView kv;
  const uint16_t *q;
  uint16_t *out;
  long long q_stride, out_stride;  // elements from one token's row to the next
  const int32_t *kv_len;           // [n_seq] cached positions, the new tokens among them
  const int32_t *cu_q;             // [n_seq + 1] first row of each sequence, or null: n_new rows each
                                   // (a planned call's kernels: the workspace's copy, ascending in [0, n_tok])
  int32_t n_seq, n_tok, n_new;
  int32_t n_heads, n_kv, group;    // group = n_heads / n_kv
  int32_t window, n_sink;
  float scale_log2;                // score scale * log2(e)
  // tile kernel: the positions of an item's queries span less than this; log2
  // of a group's positions; which of its blocks have marked rows
  int32_t span, gsh;
  int *marked;
  uint32_t *err;
};

// Workspace of the tile kernel.
struct TileWork {
  long long *first;  // [row groups + 1]
  void *info;        // int2 [row groups]
  int *count, *seq_first;
  int32_t *cu;       // [max_seqs + 1] row bounds, ascending in [0, n_tok]
  float *part;
  void *split;       // int4 [2 * n_sm]
  int *marked;       // [n_sm], 0 but between the tile kernel and k_attn_mend
  int pairs;         // pairs of blocks that run at once
};

}  // namespace ds4

struct ds4moe_attn {
  ds4moe_attn_desc d;
  int device, n_sm;
  uint8_t *mem;      // one allocation; the rest points into it
  uint32_t *err;     // device error flags
  float *part;       // partial results of the blocks that share a (sequence, head)
  int *ticket;       // arrivals of those blocks, by the first of them (self-resetting)
  ds4::TileWork tile;  // the tile kernel's share (its partials are `part`)
  uint64_t bytes, launches;
};

namespace ds4 {
// attn_decode.cu: few rows (new tokens x heads per key-value head), head
// dimension 64 or 128.
constexpr int AD_MAX_ROWS = 16;
size_t attn_decode_part_floats(int n_sm);
cudaError_t attn_decode_set_attributes();
cudaError_t launch_attn_decode(const AttnArgs &a, int head_dim, int dtype, float *part, int *ticket, int n_sm,
                               cudaStream_t s);
// attn_tile.cu: tiles of 128 rows on the tensor cores, every shape.
size_t attn_tile_part_floats(int head_dim, int n_sm);
size_t attn_tile_groups(int group, int head_dim, int max_tokens, int max_seqs);
cudaError_t attn_tile_set_attributes(int dtype, int head_dim);
int attn_tile_pairs(int dtype, int head_dim);
cudaError_t launch_attn_tile(const AttnArgs &a, int head_dim, int dtype, const TileWork &w, int n_sm, int *launches,
                             cudaStream_t s);
}  // namespace ds4
