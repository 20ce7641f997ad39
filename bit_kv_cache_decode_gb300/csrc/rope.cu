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
// Each (token, pair) angle is computed once per CTA into shared memory and serves all heads. A thread keeps
// one unit of the head (16 bytes, or the 8 or 4 that the strides and the halves allow) and walks tokens and heads,
// two units in flight; every element is read and written once, so the kernel is bound by memory. For 49,153 tokens
// x 40 heads x 128 bf16 (1.007 GB): pairs layout 157 us (half of the head rotated; 6.42 TB/s, 95 % of the copy rate),
// half layout 161 us (whole head). What carried it: streaming loads and stores (206 us with the default policy);
// short CTAs of 8 tokens (32 tokens: 239 us); two units per thread (one: 166 us; four: 230 us, fewer threads fit);
// 8 CTAs per SM for the pairs layout (6: 167 us) and 6 for the half layout, whose unit has two parts (8: 171 us);
// narrower units rather than single elements, and 16 bytes for the channels behind them where those allow it (head 64, 24
// channels rotated in halves: 99 us, all of it in 8-byte units 138 us, in elements 364 us).
#include <algorithm>

#include "kernels.cuh"

namespace oscar {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTable = 1024;                   // (cos, sin) entries of a CTA's tokens
constexpr int kRopeTokens = 8;                     // tokens of a CTA, at most

struct RopeSide {                                  // q or k
  const void* in;
  void* out;
  long long in_tok, in_head, out_tok, out_head;    // strides in elements
  int heads;
};
struct RopeArgs {
  RopeSide q, k;
  const int* positions;
  const unsigned long long* turns;                 // [rot / 2]
  int n, dim, rot;
  int tokens;                                      // tokens per CTA
  unsigned per_head;                               // ceil(2^32 / heads), i / heads for i heads < 2^32; 0 for one head
  float scale;
  int inverse;
};

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

template <typename T, int V, int VP, bool HALF, bool WIDE>
__global__ void __launch_bounds__(kRopeThreads, HALF ? 6 : 8) k_rope(RopeArgs a) {
  __shared__ float2 table[kRopeTable];             // [token][pair]: (cos, sin) times the scale
  __shared__ int pos_s[kRopeTokens];
  const int half = a.rot / 2, t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.n - t0);
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, nthr = blockDim.x * blockDim.y;
  for (int i = tid; i < nt; i += nthr) pos_s[i] = a.positions[t0 + i];
  __syncthreads();
  for (int i = tid; i < nt * half; i += nthr) {
    const int t = i / half, j = i - t * half;
    const unsigned long long turn = (unsigned long long)(unsigned)pos_s[t] * a.turns[j];
    float s, c;
    sincospif((float)(int)(turn >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
    table[i] = make_float2(c * a.scale, (a.inverse ? -s : s) * a.scale);
  }
  __syncthreads();
  constexpr int kPer = HALF ? V : V / 2;           // pairs of a unit
  constexpr int kBatch = 2;                        // units a thread has in flight
  const int rot_units = HALF ? half / V : a.rot / V;
  const int units = rot_units + (a.dim - a.rot) / VP;
  const int heads = a.q.heads + a.k.heads, items = nt * heads;
  for (int u = threadIdx.x; u < units; u += blockDim.x) {
    const bool rotary = u < rot_units;
    const int at = rotary ? u * V : a.rot + (u - rot_units) * VP;
    for (int i0 = threadIdx.y; i0 < items; i0 += kBatch * blockDim.y) {
      Unit<T, V, VP, HALF, WIDE> x[kBatch];
      T* out[kBatch];
      int tok[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const unsigned i = i0 + k * blockDim.y;    // (token, head): i = t heads + h
        const int t = a.per_head != 0u ? __umulhi(i, a.per_head) : i, h = (int)i - t * heads;
        const bool isq = h < a.q.heads;
        const RopeSide& s = isq ? a.q : a.k;
        const int hh = isq ? h : h - a.q.heads;
        const T* in = static_cast<const T*>(s.in) + (t0 + t) * s.in_tok + hh * s.in_head;
        out[k] = static_cast<T*>(s.out) + (t0 + t) * s.out_tok + hh * s.out_head;
        tok[k] = t;
        // a padded row is left as it is, and so is what is passed through in place
        if ((int)i >= items || pos_s[t] < 0 || (!rotary && in == out[k])) out[k] = nullptr;
        if (out[k] != nullptr) x[k].load(in, at, half, rotary);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (out[k] == nullptr) continue;
        if (rotary) {
          float2 cs[kPer];
#pragma unroll
          for (int e = 0; e < kPer; ++e) cs[e] = table[tok[k] * half + u * kPer + e];
          x[k].turn(cs);
        }
        x[k].store(out[k], at, half, rotary);
      }
    }
  }
}

template <typename T, int V, int VP, bool HALF, bool WIDE>
int launch_as(RopeArgs a, cudaStream_t st) {
  const int half = a.rot / 2;
  const int units = (HALF ? half / V : a.rot / V) + (a.dim - a.rot) / VP;
  // four CTAs per SM and more while there are tokens for them (3,000 tokens x 40 heads: 12.2 us; two: 14.9, eight: 14.3)
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return OSCAR_ERR_CUDA;
  a.tokens = std::max(1, std::min(std::min(kRopeTable / half, kRopeTokens), a.n / (4 * sms)));
  const unsigned heads = a.q.heads + a.k.heads;
  a.per_head = heads == 1 ? 0u : (unsigned)((0x100000000ull + heads - 1) / heads);
  const int bx = std::min(units, kRopeThreads), by = std::max(1, std::min(kRopeThreads / bx, a.q.heads + a.k.heads));
  k_rope<T, V, VP, HALF, WIDE><<<(a.n - 1) / a.tokens + 1, dim3(bx, by), 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
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

// whether accesses of v elements of `size` bytes fit a tensor's rows
bool fits(const oscar_rope_tensor& t, int size, int v) {
  if (t.heads == 0) return true;
  const uintptr_t p = reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out);
  return p % (size * v) == 0 && t.in_token % v == 0 && t.in_head % v == 0 && t.out_token % v == 0 && t.out_head % v == 0;
}

RopeSide side(const oscar_rope_tensor& t) {
  return {t.in, t.out, t.in_token, t.in_head, t.out_token, t.out_head, t.heads};
}

}  // namespace

int launch_rope(const oscar_rope_tensor& q, const oscar_rope_tensor& k, int n, int dim, int rot, int dtype,
                const int* positions, const uint64_t* turns, int layout, float scale, int inverse, cudaStream_t st) {
  RopeArgs a;
  a.q = side(q);
  a.k = side(k);
  a.positions = positions;
  a.turns = reinterpret_cast<const unsigned long long*>(turns);
  a.n = n;
  a.dim = dim;
  a.rot = rot;
  a.scale = scale;
  a.inverse = inverse;
  const bool half_layout = layout == OSCAR_ROPE_HALF;
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
