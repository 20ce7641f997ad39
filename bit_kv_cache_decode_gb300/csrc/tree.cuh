// Attention of a tree of drafted tokens over the mixed cache: the arguments its kernels share.
#pragma once

#include "kernels.cuh"

namespace oscar {

constexpr int kMaxTreeBf16Pages = 2040;   // sink and recent pages of a request

struct TreeArgs {
  const __nv_bfloat16 *q, *kd, *vd;       // [B][T][hq][128], [B][T][hkv][128]
  const unsigned long long* mask;         // [B][T][W]: the drafted nodes a node attends to
  const int *n_draft, *seq_lens;          // n_draft may be null: T nodes
  const int* hist_pt;
  int max_hist_pages;
  const int* bf16_pt;
  int T, W;
  int nsplit;                             // history slots of a row, then nb slots of BF16 and draft pages
  int nb;
  float scale_log2;                       // sm_scale * log2(e)
  float* partials;                        // [B * T * hq][nsplit + nb][kPartFloats]
  void* out;
  int out_dtype;
  float* lse;
};

// nodes of request b that take part
__device__ __forceinline__ int live_nodes(const TreeArgs& a, int b) {
  return a.n_draft != nullptr ? min(max(a.n_draft[b], 0), a.T) : a.T;
}
// the slot row of query row (b, node, head)
__device__ __forceinline__ float* tree_part(const TreeArgs& a, int hq_total, int b, int node, int hq, int slot) {
  return a.partials + ((((size_t)b * a.T + node) * hq_total + hq) * (a.nsplit + a.nb) + slot) * kPartFloats;
}

int launch_tree_merge(const LayerView& lv, const TreeArgs& a, int B, cudaStream_t st);

}  // namespace oscar
