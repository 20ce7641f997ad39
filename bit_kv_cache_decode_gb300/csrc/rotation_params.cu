// Operands of a layer's rotations, made when they are loaded (sm_103a).
//
// R = U H P_br (MarkTechPost article "Together AI 开源 OSCAR…", section "OSCAR 有何不同做法"), composed in
// double from the float32 U as loaded: (U H)[i][c] = sum_m U[i][m] (-1)^popcount(m & c) / sqrt(128), and
// column j of R is column bitrev7(j) of U H. R[i][j]: i = input channel, j = rotated channel.
//
// Thread = rotated channel, a CTA 8 input channels: each R element is 128 products in the order of m. 8 heads, K and V:
// 33.6 million double-precision multiply-adds. Loading a layer of 8 heads takes 0.5 ms with V absorbed and 0.6 ms with
// V rotated, most of it the orthogonality check and the copies (the same sums and conversions in loops on the host: 25
// and 40 ms).
#include <cmath>

#include "kernels.cuh"

namespace oscar {
namespace {

constexpr int kRpRows = 8;

__global__ void __launch_bounds__(kD) k_rotation_params(float* params, double inv, int v_rotated) {
  __shared__ float u[kRpRows][kD];
  const int i0 = kRpRows * blockIdx.x, kind = blockIdx.z, j = threadIdx.x;
  float* p = params + (size_t)blockIdx.y * kParamFloats;
  const float* U = p + (kind == OSCAR_KIND_K ? kUKOff : kUVOff);
#pragma unroll
  for (int e = 0; e < kRpRows; ++e) {
    u[e][j] = U[(i0 + e) * kD + j];
    if (kind == OSCAR_KIND_V) p[kUVtOff + j * kD + i0 + e] = u[e][j];
  }
  if (kind == OSCAR_KIND_V && !v_rotated) return;
  __syncthreads();
  const int rj = __brev(j) >> 25;
  double r[kRpRows] = {};
#pragma unroll 4
  for (int m = 0; m < kD; ++m) {
    const double h = __popc(m & rj) & 1 ? -inv : inv;
#pragma unroll
    for (int e = 0; e < kRpRows; ++e) r[e] = fma((double)u[e][m], h, r[e]);
  }
  // R as fp16 hi = fp16(R), lo = fp16(R - hi) (about 22 significant bits) in the B-fragment order of
  // mma.m16n8k16 (k = input channel, n = rotated channel): for k-block kb, n-tile nt and lane (g = lane / 4,
  // t = lane % 4), b0 holds rows 16 kb + 2t, +1 and b1 rows 16 kb + 2t + 8, +9, all of column 8 nt + g; the words of a
  // lane are hi b0, hi b1, lo b0, lo b1.
  __half* frag = reinterpret_cast<__half*>(p + (kind == OSCAR_KIND_K ? kRKFragOff : kRVFragOff));
  // R as three bf16 parts b1 = bf16(R), b2 = bf16(R - b1), b3 = bf16(R - b1 - b2), each laid out as the
  // bulk prefill's tensor-core B operand (n = rotated channel, k = input channel, K-major, 128-byte swizzle):
  // element (n, k) of part p at byte p * 32768 + (k / 64) * 16384 + n * 128 + (((k % 64) / 8) ^ (n % 8)) * 16
  // + (k % 8) * 2.
  uint8_t* img = reinterpret_cast<uint8_t*>(p + (kind == OSCAR_KIND_K ? kRKImgOff : kRVImgOff));
#pragma unroll
  for (int e = 0; e < kRpRows; ++e) {
    const int i = i0 + e, lane = (j & 7) * 4 + ((i & 7) >> 1);
    __half* at = frag + ((((i >> 4) * 16 + (j >> 3)) * 32 + lane) * 4 + ((i >> 3) & 1)) * 2 + (i & 1);
    const __half hi = __double2half(r[e]);
    at[0] = hi;
    at[4] = __double2half(r[e] - (double)__half2float(hi));
    uint8_t* to = img + (i >> 6) * 16384 + j * 128 + ((((i & 63) >> 3) ^ (j & 7)) << 4) + (i & 7) * 2;
    double rest = r[e];
#pragma unroll
    for (int part = 0; part < 3; ++part) {
      const __nv_bfloat16 b = __float2bfloat16_rn((float)rest);
      *reinterpret_cast<__nv_bfloat16*>(to + part * 32768) = b;
      rest -= (double)__bfloat162float(b);
    }
  }
}

}  // namespace

int launch_rotation_params(float* params, int hkv, bool v, bool v_rotated, cudaStream_t st) {
  k_rotation_params<<<dim3(kD / kRpRows, hkv, v ? 2 : 1), kD, 0, st>>>(params, 1.0 / std::sqrt((double)kD), v_rotated);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

}  // namespace oscar
