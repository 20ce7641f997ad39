// What the kernels that rotate heads share (sm_103a): tensors by strides, units of a head's channels, angles.
#pragma once

#include "kernels.cuh"

namespace oscar {

constexpr int kRopeThreads = 256;
constexpr int kRopeTable = 1024;                   // (cos, sin) entries of a CTA's tokens
constexpr int kRopeTokens = 8;                     // tokens of a CTA, at most

struct RopeSide {                                  // q or k
  const void* in;
  void* out;
  long long in_tok, in_head, out_tok, out_head;    // strides in elements
  int heads;
};
// Positions of tokens t0 .. t0 + nt - 1 into shared memory [token][axis]; axis 0 is negative where any is (a padded row).
// TIGHT: fewer loads at a time, for kernels that spill otherwise (float32 pairs, 64 tokens x 40 heads x 128: 4.4 us instead of
// 4.6); bf16 pairs do not, and take longer so (4,096 tokens x 40 heads x 256: 34.8 us instead of 34.2).
template <bool TIGHT = false>
__device__ __forceinline__ void load_positions(const Rotary& r, int t0, int nt, int* pos_s, int tid, int nthr) {
  int first;
  auto axis = [&](int i, int a) {
    const int p = r.positions[(size_t)a * r.n + t0 + i];
    pos_s[i * kRopeAxes + a] = p;
    if (p < 0) first = -1;
  };
  if constexpr (TIGHT) {
#pragma unroll 1
    for (int i = tid; i < nt; i += nthr) {
      first = r.positions[t0 + i];
#pragma unroll 2
      for (int a = 1; a < r.n_axes; ++a) axis(i, a);
      pos_s[i * kRopeAxes] = first;
    }
  } else {
    for (int i = tid; i < nt; i += nthr) {
      first = r.positions[t0 + i];
      for (int a = 1; a < r.n_axes; ++a) axis(i, a);
      pos_s[i * kRopeAxes] = first;
    }
  }
}
// (cos, sin) times the scale of pair j at the positions of one token; sign -1 turns backwards. See rope.cu on the angle.
__device__ __forceinline__ float2 rope_turn(const Rotary& r, const int* pos, int j, float sign) {
  const int axis = r.axes != nullptr ? min((int)r.axes[j], r.n_axes - 1) : 0;
  const unsigned long long turn = (unsigned long long)(unsigned)pos[axis] * r.turns[j];
  float s, c;
  sincospif((float)(int)(turn >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
  return make_float2(c * r.scale, s * sign * r.scale);
}
template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f(float x) { return x; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }

// V elements, loaded and stored as one access (WIDE: 16, 8 or 4 bytes) or one by one (rows on any element boundary)
template <int BYTES> struct AccessOf;
template <> struct AccessOf<16> { using type = uint4; };
template <> struct AccessOf<8> { using type = uint2; };
template <> struct AccessOf<4> { using type = unsigned; };
template <typename T, int V, bool WIDE> struct alignas(WIDE ? sizeof(T) * V : sizeof(T)) Vec { T v[V]; };

// One head's unit u: half layout: V channels from V u of the first half and their partners; pairs layout: V
// channels (V / 2 pairs) from V u; units past the rotary part copy VP channels. Loading and turning are apart, so that
// a thread has several units' loads in flight before it stores any (in place, the compiler may not reorder them).
template <typename T, int V, int VP, bool HALF, bool WIDE>
struct Unit {
  Vec<T, VP, WIDE> a;                              // V <= VP: a rotary unit is its first V elements
  Vec<T, V, WIDE> b;
  // each element is touched once: streaming accesses where they are wide
  template <int N>
  static __device__ __forceinline__ void get(T* x, const T* at) {
    if constexpr (WIDE) {
      using Bits = typename AccessOf<sizeof(T) * N>::type;
      *reinterpret_cast<Bits*>(x) = __ldcs(reinterpret_cast<const Bits*>(at));
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = at[e];
    }
  }
  template <int N>
  static __device__ __forceinline__ void put(T* at, const T* x) {
    if constexpr (WIDE) {
      using Bits = typename AccessOf<sizeof(T) * N>::type;
      __stcs(reinterpret_cast<Bits*>(at), *reinterpret_cast<const Bits*>(x));
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) at[e] = x[e];
    }
  }
  __device__ __forceinline__ void load(const T* in, int at, int half, bool rotary) {
    if (V == VP || !rotary) get<VP>(a.v, in + at);
    else get<V>(a.v, in + at);
    if (HALF && rotary) get<V>(b.v, in + at + half);
  }
  __device__ __forceinline__ void turn(const float2* cs) {
    if (HALF) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float x = to_f(a.v[e]), y = to_f(b.v[e]);
        a.v[e] = from_f<T>(x * cs[e].x - y * cs[e].y);
        b.v[e] = from_f<T>(y * cs[e].x + x * cs[e].y);
      }
    } else {
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        const float x = to_f(a.v[2 * e]), y = to_f(a.v[2 * e + 1]);
        a.v[2 * e] = from_f<T>(x * cs[e].x - y * cs[e].y);
        a.v[2 * e + 1] = from_f<T>(y * cs[e].x + x * cs[e].y);
      }
    }
  }
  __device__ __forceinline__ void store(T* out, int at, int half, bool rotary) const {
    if (V == VP || !rotary) put<VP>(out + at, a.v);
    else put<V>(out + at, a.v);
    if (HALF && rotary) put<V>(out + at + half, b.v);
  }
};

// whether accesses of v elements of `size` bytes fit a tensor's rows
inline bool fits(const oscar_rope_tensor& t, int size, int v) {
  if (t.heads == 0) return true;
  const uintptr_t p = reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out);
  return p % (size * v) == 0 && t.in_token % v == 0 && t.in_head % v == 0 && t.out_token % v == 0 && t.out_head % v == 0;
}

inline RopeSide side(const oscar_rope_tensor& t) {
  return {t.in, t.out, t.in_token, t.in_head, t.out_token, t.out_head, t.heads};
}

}  // namespace oscar
