// Log-sum-exp merge of the tree attention's partials (sm_103a): per query row (request, drafted node, head) the
// slots (m, l, acc[128]), m in log2 units and l, acc relative to 2^m, become
//   M = max m_s,  o = sum 2^(m_s - M) acc_s / sum 2^(m_s - M) l_s,  lse = ln 2 (M + log2 L).
// In explicit-V mode the history slots' sum is in the rotated value basis and is multiplied by
// R_V^T = P_br H U_V^T before it meets the BF16 slots' sum. A row that attends to nothing is 0 with lse -inf.
//
// A CTA takes 8 rows of one kv head, a thread one row and four channels, so a warp reads four whole lines of a slot;
// every slot's loads are independent. In explicit-V mode U_V^T (64 KB) is brought to shared memory by bulk copies that
// are issued before the wait for the attention kernel. The kernel reads each partial once, mostly from L2, where the
// attention kernel has just written it.
#include "rotate.cuh"
#include "tma.cuh"
#include "tree.cuh"

namespace oscar {
namespace {

constexpr int kTmRows = 8, kTmThreads = kTmRows * (kD / 4);
constexpr int kTmSmem = kD * kD * 4 + 16;          // explicit-V mode: U_V^T, a barrier

__global__ void __launch_bounds__(kTmThreads) k_tree_merge(LayerView lv, TreeArgs a) {
  __shared__ __align__(16) float zs[kTmRows][kD + 4];
  const int r = threadIdx.x & (kTmRows - 1), quad = threadIdx.x / kTmRows, h = blockIdx.y, b = blockIdx.z;
  const int gq = 1 << a.gq_log2, Q = blockIdx.x * kTmRows + r, node = Q >> a.gq_log2, hq = h * gq + (Q & (gq - 1));
  extern __shared__ __align__(128) float uvt[];
  const uint32_t bar = smem_addr(uvt + kD * kD);
  if (lv.v_explicit && threadIdx.x == 0) {         // the parameters come from no kernel
    mbar_init(bar);
    mbar_expect_tx(bar, kD * kD * 4);
    const float* src = lv.params + (size_t)h * kParamFloats + kUVtOff;
    for (int i = 0; i < 4; ++i)
      bulk_copy_hint(smem_addr(uvt) + i * kD * kD, src + i * kD * kD / 4, kD * kD, bar, l2_evict_last());
  }
  pdl_wait();                                      // the partials are written by the preceding grid
  pdl_launch_dependents();
  const int nodes = live_nodes(a, b), len = a.seq_lens[b];   // independent loads
  if (blockIdx.x * kTmRows >= nodes * gq) {        // nothing here: let the copies land, then leave
    if (lv.v_explicit && threadIdx.x == 0) mbar_wait(bar, 0);
    return;
  }
  const int hist_slots = tree_hist_slots(a, tree_pages(lv, a, len));
  const int qt = Q / kTreeRows, row = Q % kTreeRows;
  const size_t step = (size_t)a.rows * kPartFloats;
  const float* p0 = tree_part(lv, a, b, qt, h, 0);
  const float *acc0 = p0 + 4 * (quad * a.rows + row), *ml0 = p0 + a.rows * kD + 2 * row;
  const float *near = acc0 + a.nsplit * step, *near_ml = ml0 + a.nsplit * step;
  float M = -INFINITY;
#pragma unroll 8
  for (int s = 0; s < hist_slots; ++s) M = fmaxf(M, ml0[s * step]);
#pragma unroll 4
  for (int s = 0; s < a.nb; ++s) M = fmaxf(M, near_ml[s * step]);
  const float Mb = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  auto add = [&](float4& acc, const float* ml, const float* v4) {
    const float2 x = *reinterpret_cast<const float2*>(ml);
    const float4 v = *reinterpret_cast<const float4*>(v4);
    const float wt = exp2f(x.x - Mb);
    L = fmaf(wt, x.y, L);
    acc.x = fmaf(wt, v.x, acc.x);
    acc.y = fmaf(wt, v.y, acc.y);
    acc.z = fmaf(wt, v.z, acc.z);
    acc.w = fmaf(wt, v.w, acc.w);
  };
  float4 hist = make_float4(0.f, 0.f, 0.f, 0.f), o = hist;
#pragma unroll 8
  for (int s = 0; s < hist_slots; ++s) add(hist, ml0 + s * step, acc0 + s * step);
#pragma unroll 4
  for (int s = 0; s < a.nb; ++s) add(o, near_ml + s * step, near + s * step);
  if (lv.v_explicit) {                             // hist R_V^T: the permutation and H by a warp per row, then U_V^T
    *reinterpret_cast<float4*>(&zs[r][4 * quad]) = hist;
    __syncthreads();                               // also: the barrier is set up
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = zs[w][rot_channel(lane, e)];   // (hist P_br)[lane + 32 e]
    fwht128(v);
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 4; ++e) zs[w][lane + 32 * e] = v[e];
    if (!__syncthreads_and(mbar_wait(bar, 0))) {   // bounded; no output rather than a wrong one
      if (threadIdx.x == 0) flag(lv.status, OSCAR_STATUS_TIMEOUT);
      return;
    }
    hist = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = 0; i < kD; ++i) {
      const float4 u = *reinterpret_cast<const float4*>(uvt + i * kD + 4 * quad);
      const float z = zs[r][i];
      hist.x = fmaf(z, u.x, hist.x);
      hist.y = fmaf(z, u.y, hist.y);
      hist.z = fmaf(z, u.z, hist.z);
      hist.w = fmaf(z, u.w, hist.w);
    }
  }
  if (node >= nodes) return;                       // rows behind the last node stay as they are
  const float inv = M == -INFINITY ? 0.f : 1.f / L;
  o = make_float4((hist.x + o.x) * inv, (hist.y + o.y) * inv, (hist.z + o.z) * inv, (hist.w + o.w) * inv);
  const size_t orow = ((size_t)b * a.T + node) * lv.hq + hq;
  if (a.out_dtype == OSCAR_OUT_FP32) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * kD + 4 * quad) = o;
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
    uint2 u;
    u.x = *reinterpret_cast<const uint32_t*>(&lo);
    u.y = *reinterpret_cast<const uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * kD + 4 * quad) = u;
  }
  if (a.lse != nullptr && quad == 0)
    a.lse[orow] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

}  // namespace

int launch_tree_merge(const LayerView& lv, const TreeArgs& a, int B, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((a.T * (lv.hq / lv.hkv) + kTmRows - 1) / kTmRows, lv.hkv, B);
  cfg.blockDim = dim3(kTmThreads);
  cfg.dynamicSmemBytes = lv.v_explicit ? kTmSmem : 0;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_tree_merge, lv, a) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

int configure_tree_merge() {
  if (cudaFuncSetAttribute(k_tree_merge, cudaFuncAttributeMaxDynamicSharedMemorySize, kTmSmem) != cudaSuccess)
    return OSCAR_ERR_CUDA;
  return set_max_shared_carveout(reinterpret_cast<const void*>(k_tree_merge));
}

}  // namespace oscar
