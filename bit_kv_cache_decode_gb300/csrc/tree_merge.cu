// Log-sum-exp merge of the tree attention's partials (sm_103a): per query row (request, drafted node, head) the
// slots (m, l, acc[128]), m in log2 units and l, acc relative to 2^m, become
//   M = max m_s,  o = sum 2^(m_s - M) acc_s / sum 2^(m_s - M) l_s,  lse = ln 2 (M + log2 L).
// In explicit-V mode the history slots' sum is in the rotated value basis and is multiplied by
// R_V^T = P_br H U_V^T before it meets the BF16 slots' sum. A row that attends to nothing is 0 with lse -inf.
//
// A CTA takes 8 rows of one kv head, a thread one row and four channels, so a warp reads four whole lines of a slot;
// every slot's loads are independent. The kernel reads each partial once, mostly from L2, where the attention kernel has
// just written it.
// In explicit-V mode U_V^T (64 KB) is brought to shared memory by bulk copies. With few rows they are issued before the
// wait for the attention kernel; with many a CTA takes 32 rows, four to a thread, which reads U_V^T a quarter as often
// and is bound by the products (16,384 a row), and fetches it only for a request that has history. With the attention, 16
// x 100 nodes x 4 heads over 2,000 tokens take 174 us so, 178 us with 8 rows to a CTA; 12 x 130 nodes x 8 heads over 125
// to 252 tokens, which have no history, 107 and 195 us.
#include "rotate.cuh"
#include "tma.cuh"
#include "tree.cuh"

namespace oscar {
namespace {

constexpr int kTmRows = 8, kTmThreads = kTmRows * (kD / 4);
constexpr int kTmSmem = kD * kD * 4 + 16;          // explicit-V mode: U_V^T, a barrier

// G rows to a thread, 8 apart
template <bool EXPLICIT, int G>
__global__ void __launch_bounds__(kTmThreads) k_tree_merge(LayerView lv, TreeArgs a) {
  __shared__ __align__(16) float zs[EXPLICIT ? G * kTmRows : 1][kD + 4];
  const int r = threadIdx.x & (kTmRows - 1), quad = threadIdx.x / kTmRows, h = blockIdx.y, b = blockIdx.z;
  const int gq = 1 << a.gq_log2, Q0 = blockIdx.x * G * kTmRows;
  extern __shared__ __align__(128) float uvt[];
  const uint32_t bar = smem_addr(uvt + kD * kD);
  auto fetch = [&]() {                             // the parameters come from no kernel
    mbar_init(bar);
    mbar_expect_tx(bar, kD * kD * 4);
    const float* src = lv.params + (size_t)h * kParamFloats + kUVtOff;
    for (int i = 0; i < 4; ++i)
      bulk_copy_hint(smem_addr(uvt) + i * kD * kD, src + i * kD * kD / 4, kD * kD, bar, l2_evict_last());
  };
  if (EXPLICIT && G == 1 && threadIdx.x == 0) fetch();
  pdl_wait();                                      // the partials are written by the preceding grid
  pdl_launch_dependents();
  const int nodes = live_nodes(a, b), len = a.seq_lens[b];   // independent loads
  if (Q0 >= nodes * gq) {                          // nothing here: let the copies land, then leave
    if (EXPLICIT && G == 1 && threadIdx.x == 0) mbar_wait(bar, 0);
    return;
  }
  const int hist_slots = tree_hist_slots(a, tree_pages(lv, a, len));
  if (EXPLICIT && G > 1 && hist_slots > 0 && threadIdx.x == 0) fetch();
  const size_t step = (size_t)a.rows * kPartFloats;
  float4 hist[G], o[G];
  float M[G], L[G];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int Q = Q0 + kTmRows * g + r, row = Q % kTreeRows;
    hist[g] = o[g] = make_float4(0.f, 0.f, 0.f, 0.f);
    M[g] = -INFINITY;
    L[g] = 0.f;
    if (Q >= nodes * gq) continue;                 // behind the last node: its partials were not written
    const float* p0 = tree_part(lv, a, b, Q / kTreeRows, h, 0);
    const float *acc0 = p0 + 4 * (quad * a.rows + row), *ml0 = p0 + a.rows * kD + 2 * row;
    const float *near = acc0 + a.nsplit * step, *near_ml = ml0 + a.nsplit * step;
#pragma unroll 8
    for (int s = 0; s < hist_slots; ++s) M[g] = fmaxf(M[g], ml0[s * step]);
#pragma unroll 4
    for (int s = 0; s < a.nb; ++s) M[g] = fmaxf(M[g], near_ml[s * step]);
    const float Mb = M[g] == -INFINITY ? 0.f : M[g];
    auto add = [&](float4& acc, const float* ml, const float* v4) {
      const float2 x = *reinterpret_cast<const float2*>(ml);
      const float4 v = *reinterpret_cast<const float4*>(v4);
      const float wt = exp2f(x.x - Mb);
      L[g] = fmaf(wt, x.y, L[g]);
      acc.x = fmaf(wt, v.x, acc.x);
      acc.y = fmaf(wt, v.y, acc.y);
      acc.z = fmaf(wt, v.z, acc.z);
      acc.w = fmaf(wt, v.w, acc.w);
    };
#pragma unroll 8
    for (int s = 0; s < hist_slots; ++s) add(hist[g], ml0 + s * step, acc0 + s * step);
#pragma unroll 4
    for (int s = 0; s < a.nb; ++s) add(o[g], near_ml + s * step, near + s * step);
  }
  if (EXPLICIT && hist_slots > 0) {                // hist R_V^T: the permutation and H by a warp per row, then U_V^T
#pragma unroll
    for (int g = 0; g < G; ++g) *reinterpret_cast<float4*>(&zs[kTmRows * g + r][4 * quad]) = hist[g];
    __syncthreads();                               // also: the barrier is set up
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int w = threadIdx.x >> 5; w < G * kTmRows; w += kTmThreads / 32) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = zs[w][rot_channel(lane, e)];   // (hist P_br)[lane + 32 e]
      fwht128(v);
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 4; ++e) zs[w][lane + 32 * e] = v[e];
    }
    if (!__syncthreads_and(mbar_wait(bar, 0))) {   // bounded; no output rather than a wrong one
      if (threadIdx.x == 0) flag(lv.status, OSCAR_STATUS_TIMEOUT);
      return;
    }
#pragma unroll
    for (int g = 0; g < G; ++g) hist[g] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int i = 0; i < kD; i += 4) {
      float4 z[G];
#pragma unroll
      for (int g = 0; g < G; ++g) z[g] = *reinterpret_cast<const float4*>(&zs[kTmRows * g + r][i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 u = *reinterpret_cast<const float4*>(uvt + (i + e) * kD + 4 * quad);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float x = e == 0 ? z[g].x : e == 1 ? z[g].y : e == 2 ? z[g].z : z[g].w;
          hist[g].x = fmaf(x, u.x, hist[g].x);
          hist[g].y = fmaf(x, u.y, hist[g].y);
          hist[g].z = fmaf(x, u.z, hist[g].z);
          hist[g].w = fmaf(x, u.w, hist[g].w);
        }
      }
    }
  } else if (EXPLICIT && G == 1 && threadIdx.x == 0) {
    mbar_wait(bar, 0);                             // copies requested but unused: let them land
  }
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int Q = Q0 + kTmRows * g + r, node = Q >> a.gq_log2, hq = h * gq + (Q & (gq - 1));
    if (node >= nodes) continue;                   // rows behind the last node stay as they are
    const bool empty = M[g] == -INFINITY && L[g] == 0.f;   // not: NaN weights, which leave no maximum either
    const float inv = empty ? 0.f : 1.f / L[g];
    const float4 x = make_float4((hist[g].x + o[g].x) * inv, (hist[g].y + o[g].y) * inv, (hist[g].z + o[g].z) * inv,
                                 (hist[g].w + o[g].w) * inv);
    const size_t orow = ((size_t)b * a.T + node) * lv.hq + hq;
    if (a.out_dtype == OSCAR_OUT_FP32) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * kD + 4 * quad) = x;
    } else {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
      uint2 u;
      u.x = *reinterpret_cast<const uint32_t*>(&lo);
      u.y = *reinterpret_cast<const uint32_t*>(&hi);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * kD + 4 * quad) = u;
    }
    if (a.lse != nullptr && quad == 0)
      a.lse[orow] = empty ? -INFINITY : (M[g] + log2f(L[g])) * 0.6931471805599453f;
  }
}

template <bool EXPLICIT, int G>
int launch_as(const LayerView& lv, const TreeArgs& a, int B, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(((a.T << a.gq_log2) + G * kTmRows - 1) / (G * kTmRows), lv.hkv, B);
  cfg.blockDim = dim3(kTmThreads);
  cfg.dynamicSmemBytes = EXPLICIT ? kTmSmem : 0;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_tree_merge<EXPLICIT, G>, lv, a) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

template <bool EXPLICIT, int G>
int configure_as() {
  if (EXPLICIT && cudaFuncSetAttribute(k_tree_merge<EXPLICIT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTmSmem) != cudaSuccess)
    return OSCAR_ERR_CUDA;
  return set_max_shared_carveout(reinterpret_cast<const void*>(k_tree_merge<EXPLICIT, G>));
}

}  // namespace

int launch_tree_merge(const LayerView& lv, const TreeArgs& a, int B, int sms, cudaStream_t st) {
  if (!lv.v_explicit) return launch_as<false, 1>(lv, a, B, st);
  // 32 rows to a CTA once that gives every SM eight (5 x 60 nodes, 2 CTAs an SM: 72 us so, 69 us with 8 rows)
  const long long ctas = (long long)B * lv.hkv * (((a.T << a.gq_log2) + 31) / 32);
  return ctas >= 8 * sms ? launch_as<true, 4>(lv, a, B, st) : launch_as<true, 1>(lv, a, B, st);
}

int configure_tree_merge() {
  if (configure_as<false, 1>() != OSCAR_OK || configure_as<true, 1>() != OSCAR_OK) return OSCAR_ERR_CUDA;
  return configure_as<true, 4>();
}

}  // namespace oscar
