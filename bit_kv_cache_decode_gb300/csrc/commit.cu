// Commit of accepted draft tokens (sm_103a): a ragged number of tokens per request goes into the cache in one
// call, as that many single appends would put them there.
//
// Token j of request r (0 <= j < n_accept[r]) takes position p = L + j. If p >= sink + recent, the oldest
// recent token, at position p - recent, is demoted first: rotated, clipped, quantised and packed into the
// history. Its ring slot is the slot of p itself, and with n_accept <= recent no two tokens share a slot, so
// the tokens are independent of one another.
//
// A CTA serves one (kv head, K / V) and walks the requests in units of 16 tokens. The places of 8 units are looked up
// together and listed, tokens that demote a row first; the list is worked off 16 tokens at a time, so that a tile of
// the tensor cores is full though a request brings few. The 64 KB of rotation fragments are fetched once, and a
// tile's old and new rows are loaded while the tile before it is rotated. Half of the threads carry the old rows to
// the tile, the others the new rows to the slots, after a barrier that follows the old rows' arrival.
//
// Rotation and quantiser are the append's own (rotate_tile16, quantize_pack_row), so the bytes are those of a
// chain of oscar_append_kv calls. The call moves a few KB per request; its time is latency: the launch, the
// places, the fragments from L2, then a tile for every 16 tokens (its rows and the fragments from shared memory, its 16
// rows' quantisers). 64 requests x 1 to 15 tokens x 8 heads, explicit V: 19.7 us (a CTA per 16 tokens of one request:
// 28.8 us; V fields set row by row: 4 us more); one request, 3 tokens: 5.2 us.
#include <algorithm>

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

constexpr int kWarps = 16;                         // a warp rotates 8 channels of the tile and quantises a row of it
static_assert(kWarps * 32 == 4 * kD, "a thread for every word of the V fields");
constexpr int kUnits = 8;                          // units whose places are looked up together

// The 2-bit V fields of a tile's demoted rows, channel-major in their pages: a channel's 64 rows are four words. Thread
// (channel, word) gathers the fields of the rows in its word and sets them with one atomic pair per page (rows of a page
// follow one another). Atomics, as other rows of the same word may be another CTA's. hpage: -1 behind the last demoted row.
__device__ __forceinline__ void set_v_codes(const LayerView& lv, int h, const int* hpage, const int* hrow,
                                            const uint8_t (*codes)[kD / 4]) {
  const int c = threadIdx.x & (kD - 1), word = threadIdx.x >> 7;
  const uint32_t at_page = v_chan_off(c) + 4 * word;
  unsigned mask = 0, value = 0;
#pragma unroll 4
  for (int i = 0; i < kTileRows; ++i) {
    const int page = hpage[i], t = hrow[i];
    if (page < 0) break;                           // alike in all threads
    if (v_word(t) == word) {                       // alike in a warp
      mask |= 3u << v_bit(t);
      value |= ((codes[i][c >> 2] >> (2 * (c & 3))) & 3u) << v_bit(t);
    }
    if ((i + 1 == kTileRows || hpage[i + 1] != page) && mask != 0) {
      unsigned* at = reinterpret_cast<unsigned*>(int2_block_w(lv, page, h) + at_page);
      atomicAnd(at, ~mask);
      if (value != 0) atomicOr(at, value);
      mask = value = 0;
    }
  }
}

__global__ void __launch_bounds__(kWarps * 32, 2) k_commit_draft(LayerView lv, CommitArgs a, int B) {
  extern __shared__ __align__(128) float smem[];
  uint32_t* frag_s = reinterpret_cast<uint32_t*>(smem);
  float* rows = smem + kRFragWords;                // [16][kTileStride]
  float* tau_s = rows + kTileFloats;               // [128]
  const uint32_t bars = smem_addr(tau_s + kD);
  __shared__ int s_hpage[kUnits * kTileRows], s_hrow[kUnits * kTileRows];   // demoted row's place, -1: no demotion
  __shared__ int s_page[kUnits * kTileRows], s_row[kUnits * kTileRows];     // new token's place, -1: none
  __shared__ int s_node[kUnits * kTileRows], s_req[kUnits * kTileRows], s_count[2][kUnits / 2];
  __shared__ uint8_t codes[kTileRows][kD / 4];     // V rows' packed bytes
  const int h = blockIdx.y, kind = blockIdx.z;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int per_req = (lv.sink + lv.recent) / kP;
  const int tiles = (a.max_accept + kTileRows - 1) / kTileRows;
  const long long units = (long long)B * tiles, step = gridDim.x;
  const bool turns = kind == OSCAR_KIND_K || lv.v_explicit;   // this kind's rows are rotated
  const float* prm = lv.params + (size_t)h * kParamFloats;
  auto in = [](int p, int count) { return p >= 0 && p < count; };
  // every first load of a memory region takes thousands of cycles: what comes back is stored when the others are under way
  const float tau = tid < kD ? prm[(kind == OSCAR_KIND_K ? kTauKOff : kTauVOff) + tid] : 0.f;
  bool fetched = false, rotated = false;

  for (long long u0 = blockIdx.x; u0 < units; u0 += kUnits * step) {
    // ---- the places of 8 units' tokens, one per thread ----
    const long long u = u0 + (tid >> 4) * step;
    int b = 0, j = 0, L = 0, n = 0;
    bool live = false;
    if (tid < kUnits * kTileRows && u < units) {
      b = tiles == 1 ? (int)u : (int)(u / tiles);
      j = (int)(u - (long long)b * tiles) * kTileRows + (tid & 15);
      L = a.seq_lens[b];
      n = a.n_accept[b];
      live = L >= 0 && n >= 0 && n <= a.max_accept && L <= 0x7fffffff - n;   // else the whole request is left as it is
      if (!live && j == 0) flag(lv.status, OSCAR_STATUS_BAD_SEQLEN);
      live = live && j < n;
    }
    const int p = L + j;
    const bool full = live && p >= lv.sink + lv.recent;
    const bool may = __syncthreads_or(full);       // some row may be demoted: the fragments start now
    if (turns && may && !fetched) {
      fetched = true;
      if (lane == 0 && w < 8) {
        const float* f = prm + (kind == OSCAR_KIND_K ? kRKFragOff : kRVFragOff);
        constexpr int chunk = kRFragWords / 8;
        mbar_init(bars + 8 * w);
        bulk_load_hint(smem_addr(frag_s + w * chunk), f + w * chunk, chunk * 4, bars + 8 * w, l2_evict_last());
      }
    }
    if (tid < kUnits * kTileRows) {
      const int slot = !live ? 0 : p < lv.sink ? p : lv.sink + (p - lv.sink) % lv.recent;
      const int hh = p - lv.recent - lv.sink;
      const bool fits = full && hh / kP < a.max_hist_pages;
      // three independent loads, checked afterwards
      int node = !live ? -1 : a.path != nullptr ? a.path[(size_t)b * a.max_accept + j] : j;
      int page = live ? a.bf16_pt[(size_t)b * per_req + slot / kP] : -1;
      int hpage = fits ? a.hist_pt[(size_t)b * a.max_hist_pages + hh / kP] : -1;
      if (live) {
        const bool ok_node = in(node, a.T), ok_page = in(page, lv.n_bf16), ok_hist = !full || in(hpage, lv.n_int2);
        if (!ok_node) flag(lv.status, OSCAR_STATUS_BAD_TREE);
        if (!ok_page) flag(lv.status, OSCAR_STATUS_BAD_PAGE);
        // the old token has nowhere to go: the new one stays out
        if (ok_node && ok_page && !ok_hist) flag(lv.status, fits ? OSCAR_STATUS_BAD_PAGE : OSCAR_STATUS_BAD_SEQLEN);
        if (!ok_node || !ok_page || !ok_hist) page = hpage = -1;
      }
      // the list's order: demoting tokens by their place in the units, then the others
      const unsigned demoting = __ballot_sync(0xffffffffu, hpage >= 0);
      const unsigned other = __ballot_sync(0xffffffffu, hpage < 0 && page >= 0);
      if (lane == 0) {
        s_count[0][w] = __popc(demoting);
        s_count[1][w] = __popc(other);
      }
      s_hpage[tid] = -1;
      asm volatile("bar.sync 1, %0;" ::"n"(kUnits * kTileRows) : "memory");
      int at = 0;
      for (int i = 0; i < kUnits / 2; ++i) at += (i < w || hpage < 0 ? s_count[0][i] : 0) + (i < w && hpage < 0 ? s_count[1][i] : 0);
      at += __popc((hpage >= 0 ? demoting : other) & ((1u << lane) - 1u));
      if (page >= 0) {
        s_hpage[at] = hpage;
        s_hrow[at] = hh & (kP - 1);
        s_page[at] = page;
        s_row[at] = slot % kP;
        s_node[at] = node;
        s_req[at] = b;
      }
    }
    if (tid < kD) tau_s[tid] = tau;
    __syncthreads();
    int listed = 0;
    for (int i = 0; i < kUnits / 2; ++i) listed += s_count[0][i] + s_count[1][i];
    // ---- 16 tokens of the list at a time: 16 bytes of row r for each thread, an old row's or a new one's ----
    const bool is_new = tid >= 256;
    const int r = (tid >> 4) & 15, c8 = tid & 15;
    auto load = [&](int m) {
      const uint4* src = nullptr;
      if (m < listed) {
        if (is_new)
          src = reinterpret_cast<const uint4*>((kind == OSCAR_KIND_K ? a.k : a.v) +
                                               (((size_t)s_req[m] * a.T + s_node[m]) * lv.hkv + h) * kD + 8 * c8);
        else if (s_hpage[m] >= 0)
          src = reinterpret_cast<const uint4*>(bf16_row(lv, s_page[m], h, kind, s_row[m]) + 8 * c8);
      }
      return src != nullptr ? *src : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 next = load(r);
    for (int t0 = 0; t0 < listed; t0 += kTileRows) {
      const int m = t0 + r;
      const uint4 x = next;
      if (!is_new) {
        const uint32_t wds[4] = {x.x, x.y, x.z, x.w};
        float4* dst = reinterpret_cast<float4*>(rows + r * kTileStride + 8 * c8);
        dst[0] = make_float4(__uint_as_float(wds[0] << 16), __uint_as_float(wds[0] & 0xffff0000u),
                             __uint_as_float(wds[1] << 16), __uint_as_float(wds[1] & 0xffff0000u));
        dst[1] = make_float4(__uint_as_float(wds[2] << 16), __uint_as_float(wds[2] & 0xffff0000u),
                             __uint_as_float(wds[3] << 16), __uint_as_float(wds[3] & 0xffff0000u));
      }
      __syncthreads();                             // the tile is staged, the old rows are read
      next = load(m + kTileRows);
      const bool demotes = s_hpage[t0] >= 0;
      if (demotes) {
        if (turns) {
          rotated = true;
          if (!rotate_tile16<kD / 8 / kWarps>(frag_s, rows, bars)) {
            if (tid == 0) flag(lv.status, OSCAR_STATUS_TIMEOUT);
            if (w < 8) mbar_wait(bars + 8 * w, 0); // one more bounded wait for the copies in flight
            return;                                // these tokens are left out
          }
        }
        const int at = t0 + w;                     // a warp's row
        if (s_hpage[at] >= 0) {
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = rows[w * kTileStride + rot_channel(lane, e)];
          uint8_t* blk = int2_block_w(lv, s_hpage[at], h);
          const unsigned byte = quantize_row(y, tau_s, blk, s_hrow[at], kind,
                                             lv.meta_u8 ? meta_consts(lv, h, kind) : nullptr,
                                             lv.meta_cb ? cb_consts(lv, h, kind) : nullptr, lv.status);
          if (kind == OSCAR_KIND_K) blk[kKCodesOff + s_hrow[at] * (kD / 4) + rev5(lane)] = (uint8_t)byte;
          else codes[w][rev5(lane)] = (uint8_t)byte;
        }
      }
      if (is_new && m < listed) {
        if (bf16x2_nonfinite(x.x) || bf16x2_nonfinite(x.y) || bf16x2_nonfinite(x.z) || bf16x2_nonfinite(x.w))
          flag(lv.status, OSCAR_STATUS_NONFINITE);
        *reinterpret_cast<uint4*>(bf16_row(lv, s_page[m], h, kind, s_row[m]) + 8 * c8) = x;
      }
      __syncthreads();                             // the tile is free, the codes are complete
      if (demotes && kind == OSCAR_KIND_V) set_v_codes(lv, h, s_hpage + t0, s_hrow + t0, codes);
      // the next tile's codes are written after a barrier of its own
    }
    __syncthreads();                               // the places are free
  }
  if (fetched && !rotated && w < 8) mbar_wait(bars + 8 * w, 0);   // copies requested but unused: let them land
}

}  // namespace

int launch_commit_draft(const LayerView& lv, int B, int T, const void* k, const void* v, const int* seq_lens,
                        const int* n_accept, int max_accept, const int* path, const int* hist_pt, int max_hist_pages,
                        const int* bf16_pt, int sms, cudaStream_t st) {
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
  // two CTAs fit an SM; a (kv head, kind) gets its share of them, as many as it has units
  const long long units = (long long)B * ((max_accept + kTileRows - 1) / kTileRows);
  const int share = std::max(1, sms / lv.hkv);
  const dim3 grid((unsigned)std::min<long long>(units, share), lv.hkv, 2);
  k_commit_draft<<<grid, kWarps * 32, kCommitSmem, st>>>(lv, a, B);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

int configure_commit_kernel() {
  if (cudaFuncSetAttribute(k_commit_draft, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess)
    return OSCAR_ERR_CUDA;
  return cudaFuncSetAttribute(k_commit_draft, cudaFuncAttributeMaxDynamicSharedMemorySize, kCommitSmem) == cudaSuccess
             ? OSCAR_OK
             : OSCAR_ERR_CUDA;
}

}  // namespace oscar
