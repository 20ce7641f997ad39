// Step prologue (sm_103a): the append with demotion and the decode's query
// prologue in one launch; optionally with the norm and the rotation of raw q and k on the way.
//
// * Append (news article "超越 TurboQuant…OSCAR…", section "OSCAR 的设计思路":
//   the new token enters the recent window, and the oldest recent token is
//   rotated, clipped, quantised and packed into the history).
// * Query prologue (MarkTechPost article "Together AI 开源 OSCAR…", section
//   "OSCAR 有何不同做法": R_K = U_Q H_Had P_br; the read path's inverse rotation
//   of the keys is applied once to the query instead, R_K being orthogonal).
//
// grid = (B, hkv, 2 kinds or 1), block = 256 (8 warps). CTA (b, h, kind):
// * The demoted row of this kind (if the recent window is full) is row 0 of a
//   16-row tile. For kind K with queries, the gq query rows of kv head h are
//   rows 1 .. gq.
// * One tensor-core pass multiplies the tile by the composite rotation (R_K, or
//   R_V in explicit-V mode; V in V-absorbed mode is not rotated). Its fragments
//   come from the rotation parameters in 8 bulk copies.
// * The last warp quantises and packs the demoted row (the same single-row quantiser
//   as everywhere) into its history row.
// * The query rows become q~, its group sums, scale factors and the MMA
//   fragments of the tensor-core decode (qprep.cuh).
// * The new token is written to its ring slot, after the slot's old row was
//   staged.
// The grid waits for the kernel before it on the stream (programmatic
// dependent launch) before it reads q, k and v, then lets the decode be
// scheduled. Sequence lengths, page tables and the pool's rows (inputs the
// kernel before does not produce) are read before that wait.
//
// From raw rows (RAW: oscar_append_kv_rope, oscar_decode_step_rope) the grid waits first: the raw rows, the length and the
// new token's page are then read side by side, one latency instead of three. Eight lanes a row normalise and
// rotate the gq query rows of the head and its new key row (norm_rope.cu's formulas: float32, one rounding to BF16), 16
// channels a lane; the sum of squares is three shuffles, a pair's partner comes through shared memory. The results are
// what the rest of the kernel takes for q and k, and the queries are written out for the kernels behind. The angles
// (64 of them) are the same for all heads of a request. Bound by latency (loads, two barriers, sums, stores): one request
// 2.7 us in a graph, 256 requests x 8 heads 11.9 us.
#include "kernels.cuh"
#include "rope.cuh"
#include "rotate.cuh"
#include "tma.cuh"
#include "timeline.cuh"
#include "qprep.cuh"

namespace oscar {
namespace {

__device__ __forceinline__ bool valid_page(int p, int n) { return p >= 0 && p < n; }

// smem: rotation fragments | 16-row tile | tau | 8 mbarriers
constexpr int kTileFloats = 16 * kTileStride;

// What a launch does: rows as they come; raw rows; raw rows, with the rotation's fragments read from L2 (and L1, which CTAs
// of one head share) when they are needed; the same without a decode behind it. The last two take 64 KB less of shared
// memory, so that more CTAs fit an SM.
enum { kPlain, kRaw, kRawLate, kRawAppend };

// Norm and rotation of a row by eight lanes: lane l has channels 8 l .. and 64 + 8 l .. in x, their weights in w. buf: a float
// row of the group's own.
__device__ __forceinline__ void norm_rope_row(float (&x)[16], const float (&w)[16], const RawStep& raw, const float2* cs,
                                              float* buf, int l) {
  if (raw.normed) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    const float r = rsqrtf(ss * (1.f / kD) + raw.eps);
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] *= r * w[e];
  }
  const int rot = raw.r.rot, half = rot / 2;
  if (raw.pairs) {
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      const int c = (e < 8 ? 8 * l : 56 + 8 * l) + e;
      if (c >= rot) continue;
      const float2 t = cs[c >> 1];
      const float u = x[e], v = x[e + 1];
      x[e] = u * t.x - v * t.y;
      x[e + 1] = v * t.x + u * t.y;
    }
  } else if (rot == kD) {                            // a pair is in one lane
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 t = cs[8 * l + e];
      const float u = x[e], v = x[e + 8];
      x[e] = u * t.x - v * t.y;
      x[e + 8] = v * t.x + u * t.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) buf[(e < 8 ? 8 * l : 56 + 8 * l) + e] = x[e];
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int c = (e < 8 ? 8 * l : 56 + 8 * l) + e;
      if (c >= rot) continue;
      const bool second = c >= half;
      const float2 t = cs[second ? c - half : c];
      x[e] = second ? x[e] * t.x + buf[c - half] * t.y : x[e] * t.x - buf[c + half] * t.y;
    }
  }
}
constexpr float kBf16End = 0x1.FFp127f;              // from here on a float32 rounds to an infinite BF16
__device__ __forceinline__ void widen8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

// CTAs an SM, and k-blocks of fragments in flight, of appends without a decode: 256 requests x 8 heads 11.9 us, 36.2 where all
// demote (4 and 8: 14.0, 39.5; 6 and 2: 12.8, 36.5); one request 2.7 and 3.1 (2.7, 2.9; 3.1, 3.3).
constexpr int kAppendCtas = 5, kAppendAhead = 2;
template <int MODE>
__global__ void __launch_bounds__(kPrologueWarps * 32, MODE == kRawAppend ? kAppendCtas : MODE == kRawLate ? 4 : 1)
    k_step_prologue(LayerView lv, DecodeWorkspace ws, const __nv_bfloat16* __restrict__ q,
                    const __nv_bfloat16* __restrict__ k, const __nv_bfloat16* __restrict__ v,
                    const int* __restrict__ seq_lens_before, const int* __restrict__ hist_pt, int max_hist_pages,
                    const int* __restrict__ bf16_pt, float scale_log2, RawStep raw) {
  TimelineSpan timeline_span(lv, k != nullptr ? kTlAppend : kTlQprep);
  constexpr int kTokenWarp = kPrologueWarps - 2, kRowWarps = 3;   // the raw rows' warps: 4 rows each, 9 at most
  constexpr bool RAW = MODE != kPlain, kLate = MODE == kRawLate || MODE == kRawAppend;
  extern __shared__ __align__(128) float smem[];
  uint32_t* frag_s = reinterpret_cast<uint32_t*>(smem);
  float* rows = smem + (kLate ? 0 : kRFragWords);    // [16][kTileStride]
  float* tau_s = rows + kTileFloats;                 // [128]
  const uint32_t bars = smem_addr(tau_s + kD);
  __shared__ int sig[8];
  const int b = blockIdx.x, h = blockIdx.y, kind = blockIdx.z;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int gq = lv.hq / lv.hkv;
  const float* prm = lv.params + (size_t)h * kParamFloats;
  const bool do_q = MODE != kRawAppend && q != nullptr && kind == OSCAR_KIND_K && (!RAW || raw.prepare);
  const bool rotate = (kind == OSCAR_KIND_K) || lv.v_explicit;
  // The rotation fragments do not depend on the kernel before: they are requested before the wait below,
  // while that kernel still runs (this grid is scheduled early). Every CTA that may rotate requests them.
  const bool fetch_frags = rotate && (do_q || k != nullptr) && !kLate;
  if (fetch_frags && tid == 0) {
    const float* f = prm + (kind == OSCAR_KIND_K ? kRKFragOff : kRVFragOff);
    const uint64_t keep = l2_evict_last();
    constexpr int chunk = kRFragWords / 8;             // one k-block: 2,048 words
    for (int c = 0; c < 8; ++c) {
      mbar_init(bars + 8 * c);
      bulk_load_hint(smem_addr(frag_s + c * chunk), f + c * chunk, chunk * 4, bars + 8 * c, keep);
    }
  }
  // --- demotion of the oldest recent token: where it comes from and goes to ---
  // Sequence lengths, page tables and the pool are not produced by the kernel before this one (the
  // caller's q, k, v are): they are read before the programmatic wait, so only q, k and v wait for it.
  const int bf16_per_req = (lv.sink + lv.recent) / kP;
  int L_old = 0;
  bool demote = false;
  int slot = 0, spage = -1, hh = 0, hpage = -1;
  if (!RAW && k != nullptr) L_old = __ldcg(seq_lens_before + b);   // L2 reads: nothing older may sit in this SM's L1
  // With raw rows everything waits, and all loads but those that follow from the length are in flight together: the kernel
  // before may be the one that counts the requests' lengths up.
  // Rows 0 .. gq - 1: queries, row gq: the new key; four rows a warp.
  const bool raw_k = RAW && kind == OSCAR_KIND_K;
  const int rrow = tid >> 3, rl = tid & 7;
  const bool rq = rrow < gq, rlive = raw_k && (rrow == gq || (rq && q != nullptr));
  uint4 rx[2] = {}, rw[2] = {};
  int rpos[kRopeAxes] = {}, new_page = -1;
  if constexpr (RAW) {
    pdl_wait();
    pdl_launch_dependents();
    L_old = __ldcg(seq_lens_before + b);
    if (rlive) {
      const __nv_bfloat16* src = rq ? q + b * raw.q_row + (h * gq + rrow) * kD : k + b * raw.k_row + h * kD;
      const __nv_bfloat16* wt = rq ? raw.qw : raw.kw;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        rx[part] = *reinterpret_cast<const uint4*>(src + 64 * part + 8 * rl);
        if (wt == nullptr) {
          rw[part] = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);   // BF16 ones
        } else if (raw.wide_weights) {
          rw[part] = *reinterpret_cast<const uint4*>(wt + 64 * part + 8 * rl);
        } else {
          __nv_bfloat162 p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) p[e] = __halves2bfloat162(wt[64 * part + 8 * rl + 2 * e], wt[64 * part + 8 * rl + 2 * e + 1]);
          rw[part] = *reinterpret_cast<const uint4*>(p);
        }
      }
    }
    if (RAW && !raw_k && w == kTokenWarp) {
      const uint2 x = reinterpret_cast<const uint2*>(v + b * raw.v_row + h * kD)[lane];
      rx[0].x = x.x;
      rx[0].y = x.y;
    }
    if (raw_k && raw.r.positions != nullptr && tid < raw.r.rot / 2)
      for (int a = 0; a < raw.r.n_axes; ++a) rpos[a] = raw.r.positions[(size_t)a * raw.r.n + b];
    if (L_old >= 0) {                                // the new token's page
      const int pos = L_old, s2 = pos < lv.sink ? pos : lv.sink + (pos - lv.sink) % lv.recent;
      new_page = __ldcg(bf16_pt + b * bf16_per_req + s2 / kP);
    }
  }
  if (k != nullptr) {
    if (L_old < 0 && tid == 0) flag(lv.status, OSCAR_STATUS_BAD_SEQLEN);
    demote = L_old >= lv.sink + lv.recent;
    if (demote) {
      const int old = L_old - lv.recent;
      slot = (old - lv.sink) % lv.recent;
      spage = __ldcg(bf16_pt + b * bf16_per_req + lv.sink / kP + slot / kP);
      hh = old - lv.sink;
      const bool ok_h = hh / kP < max_hist_pages;
      hpage = ok_h ? __ldcg(hist_pt + (size_t)b * max_hist_pages + hh / kP) : -1;
      if (!ok_h || !valid_page(spage, lv.n_bf16) || !valid_page(hpage, lv.n_int2)) {
        if (tid == 0) flag(lv.status, ok_h ? OSCAR_STATUS_BAD_PAGE : OSCAR_STATUS_BAD_SEQLEN);
        demote = false;
      }
    }
  }
  // An append that demotes nothing: the warps with raw rows, and the one that writes the new token.
  const bool light = MODE == kRawAppend && !demote;
  if (light && w != kTokenWarp && (kind != OSCAR_KIND_K || w >= kRowWarps)) return;
  auto sync = [&] {
    if (!light) __syncthreads();
    else if (kind == OSCAR_KIND_K) asm volatile("bar.sync 2, %0;" ::"n"(32 * (kRowWarps + 1)) : "memory");
  };
  // The next layer's prologue needs its rotation fragments from L2 about one layer's decode from now:
  // ask for them now, with the same evict-last priority, so the page stream of this layer does not
  // leave them to be fetched from HBM on the next critical path.
  if (lv.next_params != nullptr && b == 0 && tid == 0 && rotate && !kLate) {
    const float* nf = lv.next_params + (size_t)h * kParamFloats + (kind == OSCAR_KIND_K ? kRKFragOff : kRVFragOff);
    l2_prefetch(nf, kRFragWords * 4, l2_evict_last());
  }
  const bool need_frags = (demote && rotate) || do_q;      // fetch_frags holds whenever this does
  // --- the tile: row 0 the demoted row, rows 1 .. gq the queries, zeros elsewhere ---
  // one 16-byte chunk (8 values) per thread: 16 rows x 16 chunks; the demoted row's chunks are loaded
  // before the wait, the queries' after it
  static_assert(kPrologueWarps * 32 == 16 * 16, "one chunk per thread");
  const int r = tid >> 4, c8 = tid & 15;
  uint4 u = make_uint4(0u, 0u, 0u, 0u);
  if (r == 0 && demote) u = __ldcg(reinterpret_cast<const uint4*>(bf16_row(lv, spage, h, kind, slot % kP) + 8 * c8));
  __shared__ float2 cs[RAW ? kD / 2 : 1];                  // the request's angles
  __shared__ float raw_rows[RAW ? 12 * kTileStride : 1];    // raw rows (of three warps, four each) between norm and rotation
  __shared__ uint4 new_key[RAW ? kD / 8 : 1];              // the new key row, BF16
  // Wait for the grid before (in a model, the kernel that made q, k and v), then let the decode be
  // scheduled; it waits for this grid before it reads anything this kernel writes.
  if constexpr (!RAW) {
    pdl_wait();
    pdl_launch_dependents();
  }
  if constexpr (RAW) {
    if (raw_k) {
      if (tid < raw.r.rot / 2) {
        bool low = false;
        for (int a = 0; a < raw.r.n_axes; ++a) {
          if (raw.r.positions == nullptr) rpos[a] = L_old;
          low |= rpos[a] < 0;
          rpos[a] = max(rpos[a], 0);
        }
        if (low && tid == 0) flag(lv.status, OSCAR_STATUS_BAD_SEQLEN);
        cs[tid] = rope_turn(raw.r, rpos, tid, 1.f);
      }
      sync();
      if (4 * w < gq + 1) {                          // all lanes of a warp take part
        float x[16], wt[16];
        widen8(rx[0], x);
        widen8(rx[1], x + 8);
        widen8(rw[0], wt);
        widen8(rw[1], wt + 8);
        norm_rope_row(x, wt, raw, cs, raw_rows + rrow * kTileStride, rl);
        bool bad = false;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          __nv_bfloat162 p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            bad |= !(fabsf(x[8 * part + 2 * e]) < kBf16End) || !(fabsf(x[8 * part + 2 * e + 1]) < kBf16End);
            p[e] = __floats2bfloat162_rn(x[8 * part + 2 * e], x[8 * part + 2 * e + 1]);
          }
          const uint4 z = *reinterpret_cast<const uint4*>(p);
          if (rlive && rq) {
            reinterpret_cast<uint4*>(raw.q_out + ((size_t)b * lv.hq + h * gq + rrow) * kD)[8 * part + rl] = z;
            if (do_q) {
              widen8(z, x + 8 * part);
              float4* t = reinterpret_cast<float4*>(rows + (rrow + 1) * kTileStride + 64 * part + 8 * rl);
              t[0] = make_float4(x[8 * part], x[8 * part + 1], x[8 * part + 2], x[8 * part + 3]);
              t[1] = make_float4(x[8 * part + 4], x[8 * part + 5], x[8 * part + 6], x[8 * part + 7]);
            }
          } else if (rlive) {
            new_key[8 * part + rl] = z;
          }
        }
        if (rlive && bad) flag(lv.status, OSCAR_STATUS_NONFINITE);
      }
    }
  } else if (r >= 1 && r <= gq && do_q) {
    u = *reinterpret_cast<const uint4*>(q + ((size_t)b * lv.hq + h * gq + r - 1) * kD + 8 * c8);
    if (bf16x2_nonfinite(u.x) || bf16x2_nonfinite(u.y) || bf16x2_nonfinite(u.z) || bf16x2_nonfinite(u.w))
      flag(lv.status, OSCAR_STATUS_NONFINITE);
  }
  if (!light && (!RAW || !do_q || r == 0 || r > gq)) {   // rows 1 .. gq of raw queries are there
    const uint32_t wds[4] = {u.x, u.y, u.z, u.w};
    float4* dst = reinterpret_cast<float4*>(rows + r * kTileStride + 8 * c8);
    dst[0] = make_float4(__uint_as_float(wds[0] << 16), __uint_as_float(wds[0] & 0xffff0000u),
                         __uint_as_float(wds[1] << 16), __uint_as_float(wds[1] & 0xffff0000u));
    dst[1] = make_float4(__uint_as_float(wds[2] << 16), __uint_as_float(wds[2] & 0xffff0000u),
                         __uint_as_float(wds[3] << 16), __uint_as_float(wds[3] & 0xffff0000u));
  }
  if (!light && tid < kD) tau_s[tid] = prm[(kind == OSCAR_KIND_K ? kTauKOff : kTauVOff) + tid];
  sync();                                            // barriers initialised, tile staged, old slot read
  if (kLate) {
    if (need_frags) rotate_tile16_l2<MODE == kRawAppend ? kAppendAhead : 8>(reinterpret_cast<const uint32_t*>(prm + (kind == OSCAR_KIND_K ? kRKFragOff : kRVFragOff)), rows);
  } else if (need_frags && !rotate_tile16(frag_s, rows, bars)) {
    if (tid == 0) flag(lv.status, OSCAR_STATUS_TIMEOUT);
    mbar_wait(bars + 8 * w, 0);                      // one more bounded wait for the copies in flight
    return;                                          // the pool is left untouched
  }
  if (fetch_frags && !need_frags) mbar_wait(bars + 8 * w, 0);   // copies requested but unused: let them land
  timeline_span.mark();                              // rotation done (fragments and rows loaded)
  // rows now hold rotated values in rotated channel order (row 0 raw if V is not rotated). The last
  // warp quantises the demoted row while warps 0 .. 6 finish the queries (named barrier 1).
  if (w == kPrologueWarps - 1) {
    if (demote) {
      float y[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = rows[rot_channel(lane, r)];
      quantize_pack_row(y, tau_s, int2_block_w(lv, hpage, h), hh % kP, kind,
                        lv.meta_u8 ? meta_consts(lv, h, kind) : nullptr, lv.meta_cb ? cb_consts(lv, h, kind) : nullptr,
                        lv.status);
    }
  } else if (do_q) {
    constexpr int kQWarps = kPrologueWarps - 1;
    qprep_stats(lv, ws, rows + kTileStride, kTileStride, sig, b, h, kQWarps);
    asm volatile("bar.sync 1, %0;" ::"n"(kQWarps * 32) : "memory");
    qprep_finish(lv, ws, rows + kTileStride, kTileStride, sig, b, h, scale_log2, kQWarps);
  }
  // --- the new token into its slot (the old row was staged before the first barrier) ---
  if (k == nullptr || L_old < 0 || w != kTokenWarp) return;
  const int pos = L_old, at = pos < lv.sink ? pos : lv.sink + (pos - lv.sink) % lv.recent, row = at % kP;
  const int page = RAW ? new_page : bf16_pt[b * bf16_per_req + at / kP];
  if (!valid_page(page, lv.n_bf16)) {
    if (lane == 0) flag(lv.status, OSCAR_STATUS_BAD_PAGE);
    return;
  }
  uint2 x;
  if (raw_k) {
    x = reinterpret_cast<const uint2*>(new_key)[lane];
  } else if (RAW) {
    x = make_uint2(rx[0].x, rx[0].y);
  } else {
    x = reinterpret_cast<const uint2*>((kind == OSCAR_KIND_K ? k : v) + ((size_t)b * lv.hkv + h) * kD)[lane];
  }
  if (__any_sync(0xffffffffu, bf16x2_nonfinite(x.x) || bf16x2_nonfinite(x.y)) && lane == 0)
    flag(lv.status, OSCAR_STATUS_NONFINITE);
  reinterpret_cast<uint2*>(bf16_row(lv, page, h, kind, row))[lane] = x;
}

constexpr int kLateSmem = (kTileFloats + kD) * 4 + 64, kPrologueSmem = kRFragWords * 4 + kLateSmem;

}  // namespace

int launch_prologue(const LayerView& lv, const DecodeWorkspace& ws, int B, const void* q, const void* k,
                    const void* v, const int* seq_lens_before, const int* hist_pt, int max_hist_pages,
                    const int* bf16_pt, float sm_scale, cudaStream_t st, bool after_all, const RawStep* raw) {
  if (B == 0) return OSCAR_OK;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(B, lv.hkv, k != nullptr ? 2 : 1);   // query-only: the K CTAs
  cfg.blockDim = dim3(kPrologueWarps * 32);
  // An append of raw rows rotates demoted rows only (256 requests x 8 heads, none demoted: 12 us; with every CTA asking for
  // the fragments 40). A step's queries take them from L2 where there are more than four CTAs for each of 152 SMs: decode
  // steps of 256 requests x 8 heads 140 us (bulk copies: 158), of 64 38.1 (41.5), of 32 24.1 (23.8), of 8 13.5 (13.0).
  const bool late = raw != nullptr && (!raw->prepare || 2ll * B * lv.hkv > 4 * 152);
  cfg.dynamicSmemBytes = late ? kLateSmem : kPrologueSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = after_all ? 0 : 1;
  const auto kernel = raw == nullptr ? k_step_prologue<kPlain> : !raw->prepare ? k_step_prologue<kRawAppend>
                      : late ? k_step_prologue<kRawLate> : k_step_prologue<kRaw>;
  return cudaLaunchKernelEx(&cfg, kernel, lv, ws,
                            static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k),
                            static_cast<const __nv_bfloat16*>(v), seq_lens_before, hist_pt, max_hist_pages, bf16_pt,
                            sm_scale * kLog2e, raw ? *raw : RawStep{}) == cudaSuccess
             ? OSCAR_OK
             : OSCAR_ERR_CUDA;
}

int configure_prologue_kernel() {
  for (auto fn : {k_step_prologue<kPlain>, k_step_prologue<kRaw>, k_step_prologue<kRawLate>, k_step_prologue<kRawAppend>}) {
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kPrologueSmem) != cudaSuccess)
      return OSCAR_ERR_CUDA;
    if (int rc = set_max_shared_carveout(reinterpret_cast<const void*>(fn)); rc != OSCAR_OK) return rc;
  }
  return OSCAR_OK;
}

}  // namespace oscar
