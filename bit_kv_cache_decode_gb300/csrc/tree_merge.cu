// Log-sum-exp merge of the tree attention's partials (sm_103a): per query row (request, drafted node, head) the
// slots (m, l, acc[128]), m in log2 units and l, acc relative to 2^m, become
//   M = max m_s,  o = sum 2^(m_s - M) acc_s / sum 2^(m_s - M) l_s,  lse = ln 2 (M + log2 L).
// In explicit-V mode the history slots' sum is in the rotated value basis and is multiplied by
// R_V^T = P_br H U_V^T before it meets the BF16 slots' sum. A row that attends to nothing is 0 with lse -inf.
//
// One warp per row; lane l owns channels 4l .. 4l + 3, so a slot is one coalesced 512-byte read, and four slots
// are in flight. A CTA's rows belong to one kv head, so that U_V stays in L1. The kernel reads each partial once,
// mostly from L2, where the attention kernel has just written it.
#include "rotate.cuh"
#include "tma.cuh"
#include "tree.cuh"

namespace oscar {
namespace {

constexpr int kTmWarps = 8;

__global__ void __launch_bounds__(kTmWarps * 32) k_tree_merge(LayerView lv, TreeArgs a) {
  __shared__ float zs[kTmWarps][kD];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y, b = blockIdx.z;
  const int gq = lv.hq / lv.hkv;
  pdl_wait();                                      // the partials are written by the preceding grid
  pdl_launch_dependents();
  const int Q = blockIdx.x * kTmWarps + w, node = Q / gq, hq = h * gq + Q % gq;
  if (node >= live_nodes(a, b)) return;            // rows behind the last node stay as they are
  const float* row = tree_part(a, lv.hq, b, node, hq, 0);
  const int ns = a.nsplit + a.nb;
  float M = -INFINITY;
  for (int s = lane; s < ns; s += 32) M = fmaxf(M, row[(size_t)s * kPartFloats]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float Mb = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  float4 hist = make_float4(0.f, 0.f, 0.f, 0.f), near = hist;
  auto add = [&](float4& acc, int s) {
    const float* p = row + (size_t)s * kPartFloats;
    const float2 ml = *reinterpret_cast<const float2*>(p);
    const float4 v = *reinterpret_cast<const float4*>(p + 4 + 4 * lane);
    const float wt = exp2f(ml.x - Mb);
    L = fmaf(wt, ml.y, L);
    acc.x = fmaf(wt, v.x, acc.x);
    acc.y = fmaf(wt, v.y, acc.y);
    acc.z = fmaf(wt, v.z, acc.z);
    acc.w = fmaf(wt, v.w, acc.w);
  };
#pragma unroll 4
  for (int s = 0; s < a.nsplit; ++s) add(hist, s);
#pragma unroll 4
  for (int s = a.nsplit; s < ns; ++s) add(near, s);
  if (lv.v_explicit) {
    float* z = zs[w];
    *reinterpret_cast<float4*>(z + 4 * lane) = hist;
    __syncwarp();
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = z[rot_channel(lane, e)];       // (hist P_br)[lane + 32 e]
    fwht128(v);
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 4; ++e) z[lane + 32 * e] = v[e];
    __syncwarp();
    const float* uvt = lv.params + (size_t)h * kParamFloats + kUVtOff;
    hist = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = 0; i < kD; ++i) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(uvt + i * kD + 4 * lane));
      hist.x = fmaf(z[i], u.x, hist.x);
      hist.y = fmaf(z[i], u.y, hist.y);
      hist.z = fmaf(z[i], u.z, hist.z);
      hist.w = fmaf(z[i], u.w, hist.w);
    }
  }
  const float inv = M == -INFINITY ? 0.f : 1.f / L;
  const float4 o = make_float4((hist.x + near.x) * inv, (hist.y + near.y) * inv, (hist.z + near.z) * inv,
                               (hist.w + near.w) * inv);
  const size_t orow = ((size_t)b * a.T + node) * lv.hq + hq;
  if (a.out_dtype == OSCAR_OUT_FP32) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * kD + 4 * lane) = o;
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
    uint2 u;
    u.x = *reinterpret_cast<const uint32_t*>(&lo);
    u.y = *reinterpret_cast<const uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * kD + 4 * lane) = u;
  }
  if (a.lse != nullptr && lane == 0)
    a.lse[orow] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

}  // namespace

int launch_tree_merge(const LayerView& lv, const TreeArgs& a, int B, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((a.T * (lv.hq / lv.hkv) + kTmWarps - 1) / kTmWarps, lv.hkv, B);
  cfg.blockDim = dim3(kTmWarps * 32);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_tree_merge, lv, a) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

}  // namespace oscar
