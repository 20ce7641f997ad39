// Page tables, token slots and tree masks built on the GPU (sm_103a), so that a serving loop that keeps its
// lengths on the device needs no host round trip between steps.
//
// k_build_tables. Request r goes from old_lens[r] to new_lens[r] tokens. With H(L) = ceil(max(0, L - sink -
// recent) / 64) history pages and F(L) = ceil(min(L, sink) / 64) + ceil(clamp(L - sink, 0, recent) / 64) BF16
// pages, the call pops H(new) - H(old) and F(new) - F(old) page ids from the free rings in (request, page)
// order, or, for new = 0, pushes the request's pages back. Ids are popped at `head` and pushed at head + count,
// so entries that are read and entries that are written never overlap and no thread waits for another.
//
// Every CTA scans the lengths itself (a few KB, in L2 after the first), then takes its share of the tables and
// of the new tokens' slots; a slot's page is looked up from the request's table or, for a page popped by this
// call, from the ring, never from an entry another CTA writes. The last CTA to finish reading writes the new
// ring positions, which may alias the old ones. The kernel is bound by latency: its launch, the lengths, the scan, a
// page id. 64 prompts of up to 16K tokens (slots 9 MB): 8.0 us; one prompt of 777: 4.2 us. Up to four CTAs per SM
// hide the slots' lookups (one: 18 us; two: 9.4 us; eight, each with a scan of its own: 11.0 us).
//
// k_tree_layout. Ancestor sets by pointer doubling: after step k a node's bit set holds its ancestors within
// 2^k steps, so T nodes take log2 T steps of one OR per word. Bound by latency: 26 nodes 2.6 us in a graph, 256 trees of
// 256 nodes (2.6 MB) 8.6 us.
#include <algorithm>

#include "kernels.cuh"

namespace oscar {
namespace {

constexpr int kTabThreads = 256;

struct TablesArgs {
  int B, sink, recent;
  const int *old_lens, *new_lens;
  int* hist_pt;
  int max_hist_pages;
  int* bf16_pt;
  int nbf;
  int *free_int2, *free_bf16;
  int cap_int2, cap_bf16;
  const int* rings_in;
  int* rings_out;
  int* cu_tokens;
  int4* slots;
  int max_tokens;
  int* status;
  unsigned* ticket;
};

__device__ __forceinline__ int hist_pages(int L, int sink, int recent) {
  return (int)(((long long)max(0, L - sink - recent) + kP - 1) / kP);
}
__device__ __forceinline__ int bf16_pages(int L, int sink, int recent) {
  return (min(L, sink) + kP - 1) / kP + (min(max(L - sink, 0), recent) + kP - 1) / kP;
}

// tokens; page ids popped and pushed, of history and BF16 pages. 64 bits: the lengths are checked after they are summed
struct Counts {
  long long v[5];
  __device__ void operator+=(const Counts& x) {
#pragma unroll
    for (int e = 0; e < 5; ++e) v[e] += x.v[e];
  }
};
enum { kTokens, kPopH, kPushH, kPopB, kPushB };

__global__ void __launch_bounds__(kTabThreads) k_build_tables(TablesArgs a) {
  extern __shared__ int smem[];
  int* tok0 = smem;                                // [B + 1] first new token of a request
  int* pop_h = tok0 + a.B + 1;                     // [B + 1] history pages popped before it (pushed, if it is released)
  int* pop_b = pop_h + a.B + 1;
  __shared__ Counts red[kTabThreads / 32];
  __shared__ int s_ring[4], s_bad;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int position = tid < 4 ? a.rings_in[tid] : 0;   // stored below, when the lengths are under way too

  // ---- the scan: each thread counts a run of requests, the CTA scans the threads' sums ----
  int bad = 0;
  auto counts = [&](int r) {
    Counts c = {};
    const int o = a.old_lens[r], n = a.new_lens[r];
    const int ho = hist_pages(o, a.sink, a.recent), hn = hist_pages(n, a.sink, a.recent);
    if (o < 0 || n < 0 || (n < o && n != 0) || hn > a.max_hist_pages || ho > a.max_hist_pages) {
      bad |= OSCAR_STATUS_BAD_SEQLEN;
    } else {
      const int bo = bf16_pages(o, a.sink, a.recent), bn = bf16_pages(n, a.sink, a.recent);
      c.v[kTokens] = max(0, n - o);
      c.v[kPopH] = n >= o ? hn - ho : 0;
      c.v[kPushH] = n >= o ? 0 : ho;
      c.v[kPopB] = n >= o ? bn - bo : 0;
      c.v[kPushB] = n >= o ? 0 : bo;
    }
    return c;
  };
  const int run = (a.B + kTabThreads - 1) / kTabThreads, r_lo = min(tid * run, a.B), r_hi = min(r_lo + run, a.B);
  Counts mine = {};
#pragma unroll 4
  for (int r = r_lo; r < r_hi; ++r) mine += counts(r);
  Counts upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    Counts x;
#pragma unroll
    for (int e = 0; e < 5; ++e) x.v[e] = __shfl_up_sync(0xffffffffu, upto.v[e], o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) red[w] = upto;
  if (tid < 4) s_ring[tid] = position;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  Counts all = {}, at = {};
#pragma unroll
  for (int i = 0; i < kTabThreads / 32; ++i) {
    if (i == w) at = all;
    all += red[i];
  }
#pragma unroll
  for (int e = 0; e < 5; ++e) at.v[e] += upto.v[e] - mine.v[e];
  for (int r = r_lo; r < r_hi; ++r) {              // a request pops or pushes
    const Counts c = counts(r);
    tok0[r] = (int)min(at.v[kTokens], (long long)0x7fffffff);
    pop_h[r] = (int)(c.v[kPushH] ? at.v[kPushH] : at.v[kPopH]);
    pop_b[r] = (int)(c.v[kPushB] ? at.v[kPushB] : at.v[kPopB]);
    at += c;
  }
  if (tid == 0) tok0[a.B] = (int)min(all.v[kTokens], (long long)0x7fffffff);
  if (all.v[kTokens] > (a.slots != nullptr ? a.max_tokens : 0x7fffffff)) bad |= OSCAR_STATUS_BAD_SEQLEN;
  for (int e = 0; e < 2; ++e) {
    const int head = s_ring[2 * e], count = s_ring[2 * e + 1], cap = e ? a.cap_bf16 : a.cap_int2;
    if (head < 0 || count < 0 || count > cap || (cap > 0 && head >= cap) || all.v[e ? kPushB : kPushH] > cap - count)
      bad |= OSCAR_STATUS_BAD_PAGE;
    else if (all.v[e ? kPopB : kPopH] > count)
      bad |= OSCAR_STATUS_NO_PAGES;
  }
  if (bad) atomicOr(&s_bad, bad);
  __syncthreads();
  bad = s_bad;
  const int total = tok0[a.B];
  // ---- the new ring positions, by the last CTA that has read the old ones (each has them in shared memory) ----
  if (tid == 0 && (gridDim.x == 1 || atomicInc(a.ticket, gridDim.x - 1) == gridDim.x - 1)) {   // wraps to 0: ready again
    const bool ok = bad == 0;
    a.rings_out[0] = ok && a.cap_int2 > 0 ? (int)((s_ring[0] + all.v[kPopH]) % a.cap_int2) : s_ring[0];
    a.rings_out[1] = s_ring[1] + (ok ? (int)(all.v[kPushH] - all.v[kPopH]) : 0);
    a.rings_out[2] = ok && a.cap_bf16 > 0 ? (int)((s_ring[2] + all.v[kPopB]) % a.cap_bf16) : s_ring[2];
    a.rings_out[3] = s_ring[3] + (ok ? (int)(all.v[kPushB] - all.v[kPopB]) : 0);
  }

  if (bad == 0) {
    auto ring = [](int head, int i, int cap) {        // head, i < cap (i: of the entries the call takes or adds)
      const unsigned x = (unsigned)head + (unsigned)i;
      return x - (x >= (unsigned)cap ? (unsigned)cap : 0u);
    };
    // page j of request r, whether it is in the table already or popped by this call
    auto hist_id = [&](int r, int j, int held) {
      return j < held ? a.hist_pt[(size_t)r * a.max_hist_pages + j]
                      : a.free_int2[ring(s_ring[0], pop_h[r] + j - held, a.cap_int2)];
    };
    auto bf16_id = [&](int r, int j, int held) {
      return j < held ? a.bf16_pt[(size_t)r * a.nbf + j] : a.free_bf16[ring(s_ring[2], pop_b[r] + j - held, a.cap_bf16)];
    };
    // ---- table entries: one warp per request ----
    const int warps = gridDim.x * (kTabThreads / 32);
    for (int r = blockIdx.x * (kTabThreads / 32) + w; r < a.B; r += warps) {
      const int o = a.old_lens[r], n = a.new_lens[r];
      const int ho = hist_pages(o, a.sink, a.recent), hn = hist_pages(n, a.sink, a.recent);
      const int bo = bf16_pages(o, a.sink, a.recent), bn = bf16_pages(n, a.sink, a.recent);
      if (n >= o) {
        for (int j = ho + lane; j < hn; j += 32) a.hist_pt[(size_t)r * a.max_hist_pages + j] = hist_id(r, j, ho);
        for (int j = bo + lane; j < bn; j += 32) a.bf16_pt[(size_t)r * a.nbf + j] = bf16_id(r, j, bo);
      } else {                                     // released: its pages to the rings' ends
        for (int j = lane; j < ho; j += 32) {
          int* e = a.hist_pt + (size_t)r * a.max_hist_pages + j;
          a.free_int2[ring(s_ring[0], s_ring[1] + pop_h[r] + j, a.cap_int2)] = *e;
          *e = -1;
        }
        for (int j = lane; j < bo; j += 32) {
          int* e = a.bf16_pt + (size_t)r * a.nbf + j;
          a.free_bf16[ring(s_ring[2], s_ring[3] + pop_b[r] + j, a.cap_bf16)] = *e;
          *e = -1;
        }
      }
    }
    // ---- slots: one new token per thread ----
    const int stride = gridDim.x * kTabThreads;
    for (long long t = (long long)blockIdx.x * kTabThreads + tid; t < total && a.slots != nullptr; t += stride) {
      int lo = 0, hi = a.B - 1;                    // the last request that starts at or before t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tok0[mid] <= t) lo = mid;
        else hi = mid - 1;
      }
      const int r = lo, o = a.old_lens[r], L = a.new_lens[r], pos = o + (int)(t - tok0[r]);
      const int bo = bf16_pages(o, a.sink, a.recent);
      int4 s;
      s.x = pos;
      if (pos < a.sink) {
        s.y = 0;
        s.z = bf16_id(r, pos / kP, bo);
        s.w = pos % kP;
      } else if (pos >= L - a.recent) {
        const int at = (pos - a.sink) % a.recent;
        s.y = 2;
        s.z = bf16_id(r, a.sink / kP + at / kP, bo);
        s.w = at % kP;
      } else {
        s.y = 1;
        s.z = hist_id(r, (pos - a.sink) / kP, hist_pages(o, a.sink, a.recent));
        s.w = (pos - a.sink) % kP;
      }
      a.slots[t] = s;
    }
    if (blockIdx.x == 0 && a.cu_tokens != nullptr)
      for (int r = tid; r <= a.B; r += kTabThreads) a.cu_tokens[r] = tok0[r];
  } else if (blockIdx.x == 0 && tid == 0) {
    flag(a.status, bad);
  }
}

// One CTA per request, one thread per node.
__global__ void __launch_bounds__(kMaxDraft) k_tree_layout(const int* __restrict__ parents, const int* __restrict__ n_draft,
                                                           const int* __restrict__ seq_lens, int T, int W,
                                                           unsigned long long* __restrict__ mask,
                                                           int* __restrict__ positions, int* status) {
  __shared__ unsigned long long anc[2][kMaxDraft][kMaxDraft / 64];
  __shared__ short up[2][kMaxDraft];               // the node 2^k steps above, -1 past the root, -2 past a bad parent
  const int b = blockIdx.x, i = threadIdx.x;
  const int asked = n_draft != nullptr ? n_draft[b] : T, L = seq_lens[b];   // independent loads
  const int parent = i < T ? parents[(size_t)b * T + i] : -1;
  if ((asked < 0 || asked > T) && i == 0) flag(status, OSCAR_STATUS_BAD_TREE);
  const bool fits = asked <= 0 || (L >= 0 && L <= 0x7fffffff - T);   // every node's position is a position
  if (!fits && i == 0) flag(status, OSCAR_STATUS_BAD_SEQLEN);
  const int n = fits ? min(max(asked, 0), T) : 0;
  if (i < T) {
    int p = i < n ? parent : -1;
    if (p < -1 || p >= i) {
      flag(status, OSCAR_STATUS_BAD_TREE);
      p = -2;
    }
    up[0][i] = (short)p;
    for (int wd = 0; wd < W; ++wd) anc[0][i][wd] = wd == (i >> 6) ? 1ull << (i & 63) : 0ull;
  }
  __syncthreads();
  int cur = 0;
  for (int step = 1; step < T; step <<= 1) {
    if (i < T) {
      const int p = up[cur][i];
      for (int wd = 0; wd < W; ++wd) anc[cur ^ 1][i][wd] = anc[cur][i][wd] | (p >= 0 ? anc[cur][p][wd] : 0ull);
      up[cur ^ 1][i] = p >= 0 ? up[cur][p] : (short)p;
    }
    cur ^= 1;
    __syncthreads();
  }
  if (i >= T) return;
  const bool live = i < n && up[cur][i] != -2;     // T steps up lead past the root, or to a bad parent
  int depth = 0;
  for (int wd = 0; wd < W; ++wd) {
    const unsigned long long m = live ? anc[cur][i][wd] : 0ull;
    depth += __popcll(m);
    mask[((size_t)b * T + i) * W + wd] = m;
  }
  positions[(size_t)b * T + i] = live ? L + depth - 1 : -1;
}

}  // namespace

int launch_build_tables(const oscar_layout& lay, int B, const int* old_lens, const int* new_lens, int* hist_pt,
                        int max_hist_pages, int* bf16_pt, int* free_int2, int* free_bf16, const int* rings_in,
                        int* rings_out, int* cu_tokens, int* slots, int max_tokens, int* status, unsigned* ticket,
                        int sms, cudaStream_t st) {
  TablesArgs a;
  a.B = B;
  a.sink = lay.sink;
  a.recent = lay.recent;
  a.old_lens = old_lens;
  a.new_lens = new_lens;
  a.hist_pt = hist_pt;
  a.max_hist_pages = max_hist_pages;
  a.bf16_pt = bf16_pt;
  a.nbf = (lay.sink + lay.recent) / kP;
  a.free_int2 = free_int2;
  a.free_bf16 = free_bf16;
  a.cap_int2 = lay.num_int2_pages;
  a.cap_bf16 = lay.num_bf16_pages;
  a.rings_in = rings_in;
  a.rings_out = rings_out;
  a.cu_tokens = cu_tokens;
  a.slots = reinterpret_cast<int4*>(slots);
  a.max_tokens = max_tokens;
  a.status = status;
  a.ticket = ticket;
  // a CTA per 512 tokens there may be (or per 8 requests), at most four per SM: each scans all lengths
  const int want = std::max(slots != nullptr ? max_tokens / 512 + 1 : 1, (B + 7) / 8);
  const int grid = std::max(1, std::min(4 * sms, want));
  k_build_tables<<<grid, kTabThreads, 3 * (B + 1) * sizeof(int), st>>>(a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

int configure_tables_kernel() {
  return cudaFuncSetAttribute(k_build_tables, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              3 * (kMaxTableBatch + 1) * (int)sizeof(int)) == cudaSuccess
             ? OSCAR_OK
             : OSCAR_ERR_CUDA;
}

int launch_tree_layout(int B, int T, const int* parents, const int* n_draft, const int* seq_lens, uint64_t* mask,
                       int* positions, int* status, cudaStream_t st) {
  k_tree_layout<<<B, (T + 31) / 32 * 32, 0, st>>>(parents, n_draft, seq_lens, T, (T + 63) / 64,
                                                  reinterpret_cast<unsigned long long*>(mask), positions, status);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

}  // namespace oscar
