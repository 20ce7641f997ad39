// Attention of a tree of drafted tokens over the mixed cache (sm_103a).
//
// Query row (node i, head) of a request attends to all committed tokens, read where they are (INT2 history in
// the rotated basis, BF16 sink and recent rows), and to the drafted nodes of its mask word i:
//   logits  history: s (q R_K) . khat   BF16, drafted: s q . k,   one softmax, o = sum p v.
//
// One warp per (query row, slot): a slot is a range of the request's history pages, or of its BF16 and draft
// pages. The running maximum and sum of the softmax pass over the tokens once.
#include <algorithm>

#include "rotate.cuh"
#include "tma.cuh"
#include "tree.cuh"

namespace oscar {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__global__ void __launch_bounds__(kWarps * 32) k_tree_rows(LayerView lv, TreeArgs a, int B) {
  __shared__ float xs[kWarps][kD];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y;
  const int b = blockIdx.z / (a.nsplit + a.nb), slot = blockIdx.z % (a.nsplit + a.nb);
  const int gq = lv.hq / lv.hkv, Q = blockIdx.x * kWarps + w, node = Q / gq, hq = h * gq + Q % gq;
  const int n = live_nodes(a, b);
  if (a.n_draft != nullptr && a.n_draft[b] != n && threadIdx.x == 0) flag(lv.status, OSCAR_STATUS_BAD_TREE);
  if (node >= n) return;
  const __nv_bfloat16* qr = a.q + (((size_t)b * a.T + node) * lv.hq + hq) * kD;
  float q[4];                                      // channels 4 lane .. 4 lane + 3
  for (int e = 0; e < 4; ++e) q[e] = __bfloat162float(qr[4 * lane + e]);
  if (__any_sync(0xffffffffu, nonfinite(q[0]) || nonfinite(q[1]) || nonfinite(q[2]) || nonfinite(q[3])) && lane == 0)
    flag(lv.status, OSCAR_STATUS_NONFINITE);
  int L = a.seq_lens[b];
  if (L < 0) {
    if (lane == 0) flag(lv.status, OSCAR_STATUS_BAD_SEQLEN);
    L = 0;
  }
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  auto token = [&](float dot, const float (&v)[4]) {
    const float x = dot * a.scale_log2;
    const float mn = fmaxf(m, x);
    const float c = m == -INFINITY ? 0.f : exp2f(m - mn), p = x == -INFINITY ? 0.f : exp2f(x - mn);
    m = mn;
    l = fmaf(l, c, p);
    for (int e = 0; e < 4; ++e) acc[e] = fmaf(acc[e], c, p * v[e]);
  };
  if (slot < a.nsplit) {
    for (int e = 0; e < 4; ++e) xs[w][4 * lane + e] = q[e];
    __syncwarp();
    float y[1][4];
    warp_rotate<1>(lv.params + (size_t)h * kParamFloats + kUKOff, xs[w], y);
    __syncwarp();
    for (int e = 0; e < 4; ++e) xs[w][rot_channel(lane, e)] = y[0][e];
    __syncwarp();
    for (int e = 0; e < 4; ++e) q[e] = xs[w][4 * lane + e];
    int Lh = max(0, L - lv.sink - lv.recent), np = (Lh + kP - 1) / kP;
    if (np > a.max_hist_pages) {
      if (lane == 0) flag(lv.status, OSCAR_STATUS_BAD_SEQLEN);
      np = a.max_hist_pages;
      Lh = np * kP;
    }
    const int p0 = (int)((long long)slot * np / a.nsplit), p1 = (int)((long long)(slot + 1) * np / a.nsplit);
    const int g = lane >> 4;
    for (int p = p0; p < p1; ++p) {
      const int id = a.hist_pt[(size_t)b * a.max_hist_pages + p];
      if (id < 0 || id >= lv.n_int2) {
        if (lane == 0) flag(lv.status, OSCAR_STATUS_BAD_PAGE);
        continue;
      }
      const uint8_t* blk = int2_block(lv, id, h);
      for (int t = 0; t < min(kP, Lh - p * kP); ++t) {
        float2 ks, vs;
        if (lv.meta_u8) {
          const float *ck = meta_consts(lv, h, 0) + 4 * g, *cv = meta_consts(lv, h, 1) + 4 * g;
          const uint8_t *mk = blk + kKMetaOff + 4 * t + 2 * g, *mv = blk + kVMetaOffU8 + 4 * t + 2 * g;
          ks = u8_scale_zero(mk[0], mk[1], ck[0], ck[1], ck[2]);
          vs = u8_scale_zero(mv[0], mv[1], cv[0], cv[1], cv[2]);
        } else {
          ks = __half22float2(*reinterpret_cast<const __half2*>(blk + kKMetaOff + 8 * t + 4 * g));
          vs = __half22float2(*reinterpret_cast<const __half2*>(blk + kVMetaOff + 8 * t + 4 * g));
        }
        const unsigned kb = blk[kKCodesOff + 32 * t + lane];
        float dot = 0.f, v[4];
        for (int e = 0; e < 4; ++e) {
          const int kc = (kb >> (2 * e)) & 3, c = 4 * lane + e;
          const int vc = (*reinterpret_cast<const uint32_t*>(blk + v_chan_off(c) + 4 * v_word(t)) >> v_bit(t)) & 3;
          const float kl = lv.meta_cb ? cb_consts(lv, h, 0)[kc] / 255.f : (float)kc;
          const float vl = lv.meta_cb ? cb_consts(lv, h, 1)[vc] / 255.f : (float)vc;
          dot = fmaf(q[e], fmaf(ks.x, kl, ks.y), dot);
          v[e] = fmaf(vs.x, vl, vs.y);
        }
        token(warp_sum(dot), v);
      }
    }
  } else {
    const int nbf = (lv.sink + lv.recent) / kP, units = nbf + (a.T + kP - 1) / kP, s = slot - a.nsplit;
    for (int u = s * units / a.nb; u < (s + 1) * units / a.nb; ++u) {
      const bool draft = u >= nbf;
      int rows, id = 0;
      if (draft) rows = min(kP, n - (u - nbf) * kP);
      else if (u < lv.sink / kP) rows = min(kP, min(L, lv.sink) - u * kP);
      else rows = min(kP, min(max(L - lv.sink, 0), lv.recent) - (u - lv.sink / kP) * kP);
      if (!draft && rows > 0) {
        id = a.bf16_pt[(size_t)b * nbf + u];
        if (id < 0 || id >= lv.n_bf16) {
          if (lane == 0) flag(lv.status, OSCAR_STATUS_BAD_PAGE);
          continue;
        }
      }
      for (int t = 0; t < rows; ++t) {
        const int j = (u - nbf) * kP + t;          // drafted node
        if (draft && !(a.mask[((size_t)b * a.T + node) * a.W + (j >> 6)] >> (j & 63) & 1)) continue;
        const __nv_bfloat16* kr = draft ? a.kd + (((size_t)b * a.T + j) * lv.hkv + h) * kD : bf16_row(lv, id, h, 0, t);
        const __nv_bfloat16* vr = draft ? a.vd + (((size_t)b * a.T + j) * lv.hkv + h) * kD : bf16_row(lv, id, h, 1, t);
        float dot = 0.f, v[4];
        for (int e = 0; e < 4; ++e) {
          dot = fmaf(q[e], __bfloat162float(kr[4 * lane + e]), dot);
          v[e] = __bfloat162float(vr[4 * lane + e]);
          if (draft && (nonfinite(v[e]) || nonfinite(__bfloat162float(kr[4 * lane + e]))))
            flag(lv.status, OSCAR_STATUS_NONFINITE);
        }
        token(warp_sum(dot), v);
      }
    }
  }
  float* part = tree_part(a, lv.hq, b, node, hq, slot);
  if (lane == 0) {
    part[0] = m;
    part[1] = l;
  }
  *reinterpret_cast<float4*>(part + 4 + 4 * lane) = make_float4(acc[0], acc[1], acc[2], acc[3]);
}

}  // namespace

// Slots of a query row: the history over nsplit of them, the BF16 and draft pages over nb.
void tree_splits(int B, int T, int hkv, int gq, int nbf, int max_hist_pages, int sms, int max_slots, int* nsplit,
                 int* nb) {
  *nsplit = std::max(1, std::min(std::min(max_hist_pages, max_slots - 1), 32));
  *nb = 1;
}

int launch_tree_attention(const LayerView& lv, const TreeArgs& a, int B, cudaStream_t st) {
  const dim3 grid((a.T * (lv.hq / lv.hkv) + kWarps - 1) / kWarps, lv.hkv, B * (a.nsplit + a.nb));
  k_tree_rows<<<grid, kWarps * 32, 0, st>>>(lv, a, B);
  if (cudaGetLastError() != cudaSuccess) return OSCAR_ERR_CUDA;
  return launch_tree_merge(lv, a, B, st);
}

}  // namespace oscar
