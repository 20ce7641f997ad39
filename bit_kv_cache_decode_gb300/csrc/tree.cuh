// Attention of a tree of drafted tokens over the mixed cache: the arguments its kernels share.
#pragma once

#include "kernels.cuh"

namespace oscar {

constexpr int kMaxTreeBf16Pages = 2040;   // sink and recent pages of a request

constexpr int kTreeRows = 128;            // query rows (node, head) of a tile, the tensor cores' M

struct TreeArgs {
  const __nv_bfloat16 *q, *kd, *vd;       // [B][T][hq][128], [B][T][hkv][128]
  const unsigned long long* mask;         // [B][T][W]: the drafted nodes a node attends to
  const int *n_draft, *seq_lens;          // n_draft may be null: T nodes
  const int* hist_pt;
  int max_hist_pages;
  const int* bf16_pt;
  int T, W;
  int gq_log2;                            // query heads of a kv head: 1, 2, 4 or 8
  int nsplit, pps;                        // history slots at most, pages a slot takes at most
  int nb;                                 // slots of BF16 and draft pages, after the nsplit history slots
  int rows;                               // rows of a tile that have partials: min(128, T gq rounded up to 8)
  float scale_log2;                       // sm_scale * log2(e)
  float* partials;                        // per (request, row tile, kv head) and slot: see tree_part
  void* out;
  int out_dtype;
  float* lse;
};

// query rows of a kv head that have partials in a tile, and tiles
inline int tree_tiles(int T, int gq) { return (T * gq + kTreeRows - 1) / kTreeRows; }
inline int tree_tile_rows(int T, int gq) { return T * gq >= kTreeRows ? kTreeRows : (T * gq + 7) / 8 * 8; }

// More than one tile: a CTA takes two, so that a page is unpacked once for 256 rows.
inline bool tree_wide(int T, int gq) { return T * gq > kTreeRows; }

// nodes of request b that take part
__device__ __forceinline__ int live_nodes(const TreeArgs& a, int b) {
  return a.n_draft != nullptr ? min(max(a.n_draft[b], 0), a.T) : a.T;
}
// history pages of a request (length L), and the slots they are spread over
__device__ __forceinline__ int tree_pages(const LayerView& lv, const TreeArgs& a, int L) {
  return min((max(0, max(L, 0) - lv.sink - lv.recent) + kP - 1) / kP, a.max_hist_pages);   // L below 0 counts as 0
}
// x / y for 0 <= x < 2^26, y > 0 and a quotient of at most 2^16: a quarter of the integer division's latency, which
// every CTA's start would wait for twice. The float quotient is off by less than one.
__device__ __forceinline__ int tree_div(int x, int y) {
  int q = (int)__fdividef((float)x, (float)y);
  const int rest = x - q * y;
  return q + (rest >= y) - (rest < 0);
}
__device__ __forceinline__ int tree_hist_slots(const TreeArgs& a, int pages) { return tree_div(pages + a.pps - 1, a.pps); }
// Partials of slot `slot` of tile qt: acc as [32 channel quads][rows] float4, then (m, l) as [rows] float2, so that
// the threads of a warp, one row each, write whole lines.
__device__ __forceinline__ float* tree_part(const LayerView& lv, const TreeArgs& a, int b, int qt, int h, int slot) {
  const int tiles = ((a.T << a.gq_log2) + kTreeRows - 1) / kTreeRows;
  return a.partials + ((((size_t)b * tiles + qt) * lv.hkv + h) * (a.nsplit + a.nb) + slot) * a.rows * kPartFloats;
}

int launch_tree_merge(const LayerView& lv, const TreeArgs& a, int B, int sms, cudaStream_t st);
int configure_tree_merge();

}  // namespace oscar
