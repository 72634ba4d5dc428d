// attn_rows.cu -- attention over the paged cache, one warp per (token, head):
// the plain kernel, right for every shape.
#include "attn.cuh"
#include "internal.h"

namespace ds4 {

template <int DT, int D>
__global__ void __launch_bounds__(128) k_attn_rows(const AttnArgs a) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.y, t = blockIdx.x * 4 + w;
  if (t >= a.n_tok) return;
  // the sequence that holds row t
  int b = -1;
  SeqInfo si = {};
  bool bad = false;
  if (!a.cu_q) {
    b = t / a.n_new;
    si = seq_info(a, b, bad);
  } else {
    for (int i = lane; i < a.n_seq; i += 32) {
      bool bd = false;
      const SeqInfo x = seq_info(a, i, bd);
      bad |= bd;
      if (t >= x.tok0 && t < x.tok0 + x.n) b = i;
    }
    b = __reduce_max_sync(0xffffffffu, b);
    bad = __any_sync(0xffffffffu, bad);
    bool unused = false;
    if (b >= 0) si = seq_info(a, b, unused);
  }
  if (bad && lane == 0) raise_flag(a.err, DS4MOE_DEVERR_LENGTH);
  if (b < 0) return;
  const int pos = si.len - si.n + (t - si.tok0);
  Groups gr = {};
  if (pos >= 0) gr = groups_of(a, pos, pos);
  float2 acc[D / 64];
  float m, l;
  bool bad_page = false;
  attn_row_warp<DT, D>(a, a.q + (long long)t * a.q_stride + (long long)h * D, b, h / a.group, pos, gr, 0, gr.n, acc, m,
                       l, bad_page);
  if (bad_page && lane == 0) raise_flag(a.err, DS4MOE_DEVERR_PAGE);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint32_t *o = reinterpret_cast<uint32_t *>(a.out + (long long)t * a.out_stride + (long long)h * D);
#pragma unroll
  for (int c = 0; c < D / 64; c++) o[lane + 32 * c] = Half16<DT>::down(acc[c].x * inv, acc[c].y * inv);
}

template <int DT>
static const void *rows_fn(int D) {
  return D == 64    ? (const void *)k_attn_rows<DT, 64>
         : D == 128 ? (const void *)k_attn_rows<DT, 128>
         : D == 256 ? (const void *)k_attn_rows<DT, 256>
                    : (const void *)k_attn_rows<DT, 512>;
}

cudaError_t launch_attn_rows(const AttnArgs &a, int head_dim, int dtype, cudaStream_t s) {
  void *args[] = {(void *)&a};
  const void *fn = dtype == DS4MOE_DT_BF16 ? rows_fn<DS4MOE_DT_BF16>(head_dim) : rows_fn<DS4MOE_DT_F16>(head_dim);
  return launch_pdl(fn, dim3((a.n_tok + 3) / 4, a.n_heads), dim3(128), 0, s, args, true);
}

}  // namespace ds4
