// Commit of accepted draft tokens (sm_103a): a ragged number of tokens per request goes into the cache in one
// call, as that many single appends would put them there.
//
// Token j of request r (0 <= j < n_accept[r]) takes position p = L + j. If p >= sink + recent, the oldest
// recent token, at position p - recent, is demoted first: rotated, clipped, quantised and packed into the
// history. Its ring slot is the slot of p itself, and with n_accept <= recent no two tokens share a slot, so
// the tokens are independent of one another: a CTA takes 16 of them (one tensor-core tile of demoted rows) of
// one (request, kv head, K / V), stages the old rows, then rotates, quantises and overwrites.
//
// Rotation and quantiser are the append's own (rotate_tile16, quantize_pack_row), so the bytes are those of a
// chain of oscar_append_kv calls. The call moves a few KB per request: its time is the latency of the launch,
// the 64 KB of rotation fragments (from L2) and one tile.
#include "kernels.cuh"
#include "qprep.cuh"
#include "rotate.cuh"
#include "tma.cuh"

namespace oscar {
namespace {

constexpr int kTileRows = 16;
constexpr int kTileFloats = kTileRows * kTileStride;
constexpr int kCommitSmem = (kRFragWords + kTileFloats + kD) * 4 + 64;

struct CommitArgs {
  const __nv_bfloat16 *k, *v;                      // [B][T][hkv][128]
  const int *seq_lens, *n_accept, *path;           // path [B][max_accept], or null: node j is token j
  const int *hist_pt, *bf16_pt;
  int T, max_accept, max_hist_pages;
};

__global__ void __launch_bounds__(kPrologueWarps * 32, 1) k_commit_draft(LayerView lv, CommitArgs a) {
  extern __shared__ __align__(128) float smem[];
  uint32_t* frag_s = reinterpret_cast<uint32_t*>(smem);
  float* rows = smem + kRFragWords;                // [16][kTileStride]
  float* tau_s = rows + kTileFloats;               // [128]
  const uint32_t bars = smem_addr(tau_s + kD);
  __shared__ int s_hpage[kTileRows], s_spage[kTileRows];   // demoted row's pages, -1: no demotion
  __shared__ int s_page[kTileRows], s_row[kTileRows], s_node[kTileRows];   // new token's place, -1: none
  const int b = blockIdx.x, h = blockIdx.y, kind = blockIdx.z & 1, j0 = (blockIdx.z >> 1) * kTileRows;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int L = a.seq_lens[b];
  int n = a.n_accept[b];
  if (L < 0 || n < 0 || n > a.max_accept || L > 0x7fffffff - n) {   // the whole request is left as it is
    if (tid == 0 && blockIdx.z == 0 && h == 0) flag(lv.status, OSCAR_STATUS_BAD_SEQLEN);
    return;
  }
  if (j0 >= n) return;
  const int nj = min(kTileRows, n - j0);
  const int per_req = (lv.sink + lv.recent) / kP;
  auto in = [](int p, int count) { return p >= 0 && p < count; };
  if (tid < kTileRows) {
    int hpage = -1, spage = -1, page = -1, row = 0, node = -1;
    if (tid < nj) {
      const int p = L + j0 + tid;
      node = a.path != nullptr ? a.path[(size_t)b * a.max_accept + j0 + tid] : j0 + tid;
      if (!in(node, a.T)) {
        flag(lv.status, OSCAR_STATUS_BAD_TREE);
        node = -1;
      }
      const int slot = p < lv.sink ? p : lv.sink + (p - lv.sink) % lv.recent;
      row = slot % kP;
      page = a.bf16_pt[(size_t)b * per_req + slot / kP];
      if (!in(page, lv.n_bf16)) {
        flag(lv.status, OSCAR_STATUS_BAD_PAGE);
        page = -1;
      }
      if (p >= lv.sink + lv.recent && page >= 0 && node >= 0) {
        const int hh = p - lv.recent - lv.sink;
        const bool fits = hh / kP < a.max_hist_pages;
        hpage = fits ? a.hist_pt[(size_t)b * a.max_hist_pages + hh / kP] : -1;
        if (!fits || !in(hpage, lv.n_int2)) {
          flag(lv.status, fits ? OSCAR_STATUS_BAD_PAGE : OSCAR_STATUS_BAD_SEQLEN);
          hpage = -1;
          node = -1;                               // the old token has nowhere to go: the new one stays out
        } else {
          spage = page;
        }
      }
      if (node < 0) page = -1;
    }
    s_hpage[tid] = hpage;
    s_spage[tid] = spage;
    s_page[tid] = page;
    s_row[tid] = row;
    s_node[tid] = node;
  }
  const bool demotes = (long long)L + j0 + nj > lv.sink + lv.recent;   // some row of the tile is demoted
  const bool rotate = demotes && (kind == OSCAR_KIND_K || lv.v_explicit);
  const float* prm = lv.params + (size_t)h * kParamFloats;
  if (rotate && tid == 0) {
    const float* f = prm + (kind == OSCAR_KIND_K ? kRKFragOff : kRVFragOff);
    constexpr int chunk = kRFragWords / 8;
    for (int c = 0; c < 8; ++c) {
      mbar_init(bars + 8 * c);
      bulk_load_hint(smem_addr(frag_s + c * chunk), f + c * chunk, chunk * 4, bars + 8 * c, l2_evict_last());
    }
  }
  if (tid < kD) tau_s[tid] = prm[(kind == OSCAR_KIND_K ? kTauKOff : kTauVOff) + tid];
  __syncthreads();
  {
    // the demoted rows, one 16-byte chunk per thread
    const int r = tid >> 4, c8 = tid & 15;
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (s_spage[r] >= 0) u = *reinterpret_cast<const uint4*>(bf16_row(lv, s_spage[r], h, kind, s_row[r]) + 8 * c8);
    const uint32_t wds[4] = {u.x, u.y, u.z, u.w};
    float4* dst = reinterpret_cast<float4*>(rows + r * kTileStride + 8 * c8);
    dst[0] = make_float4(__uint_as_float(wds[0] << 16), __uint_as_float(wds[0] & 0xffff0000u),
                         __uint_as_float(wds[1] << 16), __uint_as_float(wds[1] & 0xffff0000u));
    dst[1] = make_float4(__uint_as_float(wds[2] << 16), __uint_as_float(wds[2] & 0xffff0000u),
                         __uint_as_float(wds[3] << 16), __uint_as_float(wds[3] & 0xffff0000u));
  }
  __syncthreads();                                 // the old rows are staged: their slots may be overwritten
  if (rotate && !rotate_tile16(frag_s, rows, bars)) {
    if (tid == 0) flag(lv.status, OSCAR_STATUS_TIMEOUT);
    mbar_wait(bars + 8 * w, 0);                    // one more bounded wait for the copies in flight
    return;                                        // these tokens are left out
  }
  for (int r = w; r < nj; r += kPrologueWarps) {
    if (s_hpage[r] >= 0) {
      const int hh = L + j0 + r - lv.recent - lv.sink;
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = rows[r * kTileStride + rot_channel(lane, e)];
      quantize_pack_row(y, tau_s, int2_block_w(lv, s_hpage[r], h), hh % kP, kind,
                        lv.meta_u8 ? meta_consts(lv, h, kind) : nullptr, lv.meta_cb ? cb_consts(lv, h, kind) : nullptr,
                        lv.status);
    }
    if (s_page[r] >= 0) {
      const __nv_bfloat16* src =
          (kind == OSCAR_KIND_K ? a.k : a.v) + (((size_t)b * a.T + s_node[r]) * lv.hkv + h) * kD;
      const uint2 x = reinterpret_cast<const uint2*>(src)[lane];
      if (__any_sync(0xffffffffu, bf16x2_nonfinite(x.x) || bf16x2_nonfinite(x.y)) && lane == 0)
        flag(lv.status, OSCAR_STATUS_NONFINITE);
      reinterpret_cast<uint2*>(bf16_row(lv, s_page[r], h, kind, s_row[r]))[lane] = x;
    }
  }
}

}  // namespace

int launch_commit_draft(const LayerView& lv, int B, int T, const void* k, const void* v, const int* seq_lens,
                        const int* n_accept, int max_accept, const int* path, const int* hist_pt, int max_hist_pages,
                        const int* bf16_pt, cudaStream_t st) {
  CommitArgs a;
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.seq_lens = seq_lens;
  a.n_accept = n_accept;
  a.path = path;
  a.hist_pt = hist_pt;
  a.bf16_pt = bf16_pt;
  a.T = T;
  a.max_accept = max_accept;
  a.max_hist_pages = max_hist_pages;
  const dim3 grid(B, lv.hkv, 2 * ((max_accept + kTileRows - 1) / kTileRows));
  k_commit_draft<<<grid, kPrologueWarps * 32, kCommitSmem, st>>>(lv, a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

int configure_commit_kernel() {
  return cudaFuncSetAttribute(k_commit_draft, cudaFuncAttributeMaxDynamicSharedMemorySize, kCommitSmem) == cudaSuccess
             ? OSCAR_OK
             : OSCAR_ERR_CUDA;
}

}  // namespace oscar
