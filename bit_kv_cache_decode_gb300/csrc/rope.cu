// Rotary positions (sm_103a): pairs of a head's channels turned by position * frequency, forward and
// inverse (the inverse is the gradient: the rotation is orthogonal up to its scale).
//
//   (a, b) -> s (a cos t - b sin t, b cos t + a sin t),   t = pos * f,
//
// pairs are (i, i + rot/2) (half layout) or (2i, 2i + 1) (pairs layout), i < rot/2; the channels from rot on
// are passed through.
//
// Angles. A float32 product pos * f loses the angle of far positions (at pos 1e5 its half unit is 4e-3
// radians). The plan therefore holds each frequency as a 64-bit fraction of a turn, F = round(f / (2 pi) 2^64),
// and the angle is the integer product pos * F modulo 2^64: the full turns fall off by themselves, and the
// error stays below pos 2^-65 turns. Its upper 32 bits (2^-32 turns), as a signed number of half turns in float32
// (2^-26 turns, or 1e-7 radians, at most), go to sincospif: what is left of the angle's error is float32's, the same
// at any position.
//
// Positions with several axes (time, height and width of images and video): each pair has its axis, and turns by the
// token's position on it. The axes' positions and the pairs' axes are read by the CTA's angles alone, so the time is the
// rows': 40,961 tokens x 40 heads x 128 bf16, 3 axes, all turned in halves (0.84 GB), 129 us (6.5 TB/s, 98 % of the copy rate).
//
// Each (token, pair) angle is computed once per CTA into shared memory and serves all heads. A thread keeps
// one unit of the head (16 bytes, or the 8 or 4 that the strides and the halves allow) and walks tokens and heads,
// two units in flight; every element is read and written once, so the kernel is bound by memory. For 49,153 tokens
// x 40 heads x 128 bf16 (1.007 GB): pairs layout 157 us (half of the head rotated; 6.40 TB/s, 96 % of the copy rate),
// half layout 152 us (whole head; 6.61 TB/s). What carried it: streaming loads and stores (206 us with the default policy);
// short CTAs of 8 tokens (32 tokens: 239 us); two units per thread (one: 166 us; four: 230 us, fewer threads fit);
// 8 CTAs per SM for the pairs layout (6: 167 us) and 5 for the half layout, whose unit has two parts (6: 154.6 us; where only
// a part of a head is turned see launch_as);
// narrower units rather than single elements, and 16 bytes for the channels behind them where those allow it (head 64, 24
// channels rotated in halves: 99 us, all of it in 8-byte units 138 us, in elements 364 us).
#include <algorithm>

#include "rope.cuh"

namespace oscar {
namespace {

struct RopeArgs {
  RopeSide q, k;
  Rotary r;
  int dim;
  int tokens;                                      // tokens per CTA
  unsigned per_head;                               // i / heads as the upper half of i times this; 0 for one head: i itself
  int inverse;
};

// Where a token's pair j lies among its (cos, sin), for units of PER pairs: two pairs (16 bytes) of all units side by side, then
// the next two, so that threads of neighbouring units read without bank conflicts (pair by pair, 16,384 tokens x 40 heads x 256
// in halves took 186 us instead of 109).
template <int PER>
__device__ __forceinline__ int slot(int j, int units) {
  const int u = j / PER, e = j % PER;
  return PER == 1 ? j : ((e >> 1) * units + u) * 2 + (e & 1);
}

// BATCH: units a thread has in flight; CTAS: CTAs an SM
template <typename T, int V, int VP, bool HALF, bool WIDE, int BATCH, int CTAS>
__global__ void __launch_bounds__(kRopeThreads, CTAS) k_rope(RopeArgs a) {
  __shared__ __align__(16) float2 table[kRopeTable];   // [token][slot of a pair]: (cos, sin) times the scale
  __shared__ int pos_s[kRopeTokens * kRopeAxes];
  const int rot = a.r.rot, half = rot / 2, t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.r.n - t0);
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, nthr = blockDim.x * blockDim.y;
  constexpr int kPer = HALF ? V : V / 2;           // pairs of a unit
  const int rot_units = HALF ? half / V : rot / V;
  load_positions<!HALF && sizeof(T) == 4>(a.r, t0, nt, pos_s, tid, nthr);
  __syncthreads();
  for (int i = tid; i < nt * half; i += nthr) {
    const int t = i / half, j = i - t * half;
    table[t * half + slot<kPer>(j, rot_units)] = rope_turn(a.r, pos_s + t * kRopeAxes, j, a.inverse ? -1.f : 1.f);
  }
  __syncthreads();
  const int units = rot_units + (a.dim - rot) / VP;
  const int heads = a.q.heads + a.k.heads, items = nt * heads;
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    const bool rotary = u < rot_units;
    const int at = rotary ? u * V : rot + (u - rot_units) * VP;
    for (int i0 = threadIdx.y; i0 < items; i0 += BATCH * blockDim.y) {
      Unit<T, V, VP, HALF, WIDE> x[BATCH];
      T* out[BATCH];
      int tok[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const unsigned i = i0 + k * blockDim.y;    // (token, head): i = t heads + h
        const int t = a.per_head != 0u ? __umulhi(i, a.per_head) : i, h = (int)i - t * heads;
        const bool isq = h < a.q.heads;
        const RopeSide& s = isq ? a.q : a.k;
        const int hh = isq ? h : h - a.q.heads;
        const T* in = static_cast<const T*>(s.in) + (t0 + t) * s.in_tok + hh * s.in_head;
        out[k] = static_cast<T*>(s.out) + (t0 + t) * s.out_tok + hh * s.out_head;
        tok[k] = t;
        // a padded row is left as it is, and so is what is passed through in place
        if ((int)i >= items || pos_s[t * kRopeAxes] < 0 || (!rotary && in == out[k])) out[k] = nullptr;
        if (out[k] != nullptr) x[k].load(in, at, half, rotary);
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        if (out[k] == nullptr) continue;
        if (rotary) {
          float2 cs[kPer];
#pragma unroll
          for (int e = 0; e < kPer; e += 2) {
            const float2* at = table + tok[k] * half + slot<kPer>(u * kPer + e, rot_units);
            if constexpr (kPer == 1) {
              cs[e] = *at;
            } else {
              const float4 two = *reinterpret_cast<const float4*>(at);
              cs[e] = make_float2(two.x, two.y);
              cs[e + 1] = make_float2(two.z, two.w);
            }
          }
          x[k].turn(cs);
        }
        x[k].store(out[k], at, half, rotary);
      }
    }
  }
}

template <typename T, int V, int VP, bool HALF, bool WIDE, int BATCH, int CTAS>
int launch_with(RopeArgs a, cudaStream_t st) {
  const int rot = a.r.rot, half = rot / 2;
  const int units = (HALF ? half / V : rot / V) + (a.dim - rot) / VP;
  // four CTAs per SM and more while there are tokens for them (3,000 tokens x 40 heads: 12.2 us; two: 14.9, eight: 14.3)
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return OSCAR_ERR_CUDA;
  a.tokens = std::max(1, std::min(std::min(kRopeTable / half, kRopeTokens), a.r.n / (4 * sms)));
  // i / heads is the upper half of i ceil(2^32 / heads) while i heads <= 2^32: for all rows of a CTA's tokens, so many heads
  // leave it fewer of them. A single token's rows are all its own: 1 gives 0 for each.
  const unsigned long long heads = a.q.heads + a.k.heads;
  a.tokens = (int)std::max(1ull, std::min((unsigned long long)a.tokens, 0x100000000ull / (heads * heads)));
  a.per_head = heads == 1 ? 0u : a.tokens == 1 ? 1u : (unsigned)((0x100000000ull + heads - 1) / heads);
  const int bx = std::min(units, kRopeThreads), by = std::max(1, std::min(kRopeThreads / bx, a.q.heads + a.k.heads));
  k_rope<T, V, VP, HALF, WIDE, BATCH, CTAS><<<(a.r.n - 1) / a.tokens + 1, dim3(bx, by), 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

// Units in flight and CTAs an SM of the half layout where a part of a head is turned, whose threads do unequal work. One and 8
// while L2 holds the call (2,400 tokens x 24 heads x 160 float32, 80 turned: 12.2 us; two and 6: 13.9; 1,024 x 9 x 512 bf16, 128
// turned: 5.8; two and 5: 7.4), for rows of a power of two of bytes up to 512 (8,192 x 40 x 128 float32, 64 turned: 60 us; two
// and 5: 74), and of 16 bits unless a quarter or less is turned (6,553 x 40 x 160, 80 turned: 35 us, 40; 10,922 x 40 x 96, 24
// turned: 41, 37). Other float32 rows two and 6 (6,553 x 40 x 160, 80 turned: 60 us; one and 8: 65; two and 5: 74), all else
// two and 5 (single elements, 4,096 x 40 x 128 float32, 64 turned: 72 us; one and 8: 85).
template <typename T, int V, int VP, bool HALF, bool WIDE>
int launch_as(const RopeArgs& a, cudaStream_t st) {
  if constexpr (!HALF) {
    return launch_with<T, V, VP, HALF, WIDE, 2, 8>(a, st);
  } else {
    if constexpr (WIDE) {
      const int row = a.dim * (int)sizeof(T);
      const bool even = row <= 512 && (row & (row - 1)) == 0;
      const bool in_l2 = 2.0 * a.r.n * (a.q.heads + a.k.heads) * row <= 1 << 27;   // input and output
      if (a.r.rot < a.dim && (even || in_l2 || (sizeof(T) == 2 && 4 * a.r.rot > a.dim)))
        return launch_with<T, V, VP, HALF, WIDE, 1, 8>(a, st);
      if constexpr (sizeof(T) == 4)
        if (a.r.rot < a.dim) return launch_with<T, V, VP, HALF, WIDE, 2, 6>(a, st);
    }
    return launch_with<T, V, VP, HALF, WIDE, 2, 5>(a, st);
  }
}

// bytes: the widest access, of 16 at most, that every row, half and remainder starts on a multiple of; else elements.
// Where only the halves are narrower, which are then 8 bytes' multiples, the channels behind them are copied 16 bytes at
// a time (copy16).
template <typename T, bool HALF>
int launch_layout(const RopeArgs& a, int bytes, bool copy16, cudaStream_t st) {
  constexpr int V16 = 16 / sizeof(T), V8 = 8 / sizeof(T), V4 = 4 / sizeof(T), kLeast = HALF ? 1 : 2;
  if (bytes == 16) return launch_as<T, V16, V16, HALF, true>(a, st);
  if constexpr (HALF) {
    if (bytes == 8 && copy16) return launch_as<T, V8, V16, HALF, true>(a, st);
  }
  if (bytes == 8) return launch_as<T, V8, V8, HALF, true>(a, st);
  if constexpr (V4 > 1) {
    if (bytes == 4) return launch_as<T, V4, V4, HALF, true>(a, st);
  }
  return launch_as<T, kLeast, kLeast, HALF, false>(a, st);
}
template <typename T>
int launch_typed(const RopeArgs& a, bool half_layout, int bytes, bool copy16, cudaStream_t st) {
  return half_layout ? launch_layout<T, true>(a, bytes, copy16, st) : launch_layout<T, false>(a, bytes, copy16, st);
}

}  // namespace

int launch_rope(const oscar_rope_tensor& q, const oscar_rope_tensor& k, int n, int dim, int dtype, const int* positions,
                const oscar_rotary& r, int inverse, cudaStream_t st) {
  RopeArgs a;
  a.q = side(q);
  a.k = side(k);
  a.r = rotary_of(r, positions, n);
  a.dim = dim;
  a.inverse = inverse;
  const bool half_layout = r.layout == OSCAR_ROPE_HALF;
  const int rot = r.rotary_dim;
  const int size = dtype == OSCAR_DTYPE_FP32 ? 4 : 2;
  const int v16 = 16 / size;
  const bool copy16 = half_layout && fits(q, size, v16) && fits(k, size, v16) && rot % v16 == 0 && (dim - rot) % v16 == 0;
  int bytes = 16;
  for (; bytes > size; bytes /= 2) {
    const int v = bytes / size;
    if (fits(q, size, v) && fits(k, size, v) && (half_layout ? rot / 2 : rot) % v == 0 && (copy16 || (dim - rot) % v == 0)) break;
  }
  if (dtype == OSCAR_DTYPE_FP32) return launch_typed<float>(a, half_layout, bytes, copy16, st);
  if (dtype == OSCAR_DTYPE_FP16) return launch_typed<__half>(a, half_layout, bytes, copy16, st);
  return launch_typed<__nv_bfloat16>(a, half_layout, bytes, copy16, st);
}

}  // namespace oscar
