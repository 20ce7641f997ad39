// Norm and rotary position of a head's row in one pass, and the gradient (sm_103a).
//
//   r = (mean x^2 + eps)^-1/2,   y = Rot(x r w):   the root-mean-square norm with a weight per channel, then rope.cu's
//   rotation. Gradient of a loss with g = dL/dy:  h = Rot^T g (turned backwards, times the scale),
//   dL/dw = sum over rows of h x r,   u = h w,   dL/dx = r (u - x r^2 mean(u x)).
//
// A row of a head is held by a group of 1 to 32 lanes, each with whole units of it (rope.cuh: 16 bytes, and for the half
// layout their partners, so a rotation stays within a thread); the sums of a row are shuffles within its group. Angles
// are computed once per CTA and token into shared memory and serve all heads. Everything between the load and the one
// rounding at the store is float32. A row is read once and written once: bound by memory.
//
// Gradient: the weights' sums are held in registers over all rows of a CTA, which walks tokens of q or of k; CTAs'
// partial sums go to the workspace and are added in a fixed order by a second kernel, so results do not depend on timing.
#include <algorithm>
#include <type_traits>

#include "rope.cuh"
#include "smem.cuh"
#include "tma.cuh"

namespace oscar {
namespace {

constexpr int kGradCtas = 304;                     // partial sums of the weights' gradients, at most: two CTAs per SM of 152
constexpr int kGradTable = 2048, kGradTokens = 32; // as kRopeTable and kRopeTokens, for the gradient's CTAs
constexpr int kSumRows = 8;                        // threads that share a channel's partial sums

struct NormArgs {
  RopeSide q, k;
  RopeSide gq, gk;                                 // gradient: dL/dy (in); q, k: x (in) and dL/dx (out)
  const void *qw, *kw;                             // weights of the rows' type, or null: ones
  Rotary r;
  int dim, tokens, lanes;                          // tokens per CTA (gradient: at a time), lanes per row
  int q_ctas;                                      // gradient: the first CTAs walk q, the others k
  float eps;
  float* partials;                                 // gradient: [CTA][dim], or null
};

// whether a lane holds no more than 32 bytes of a row
template <typename T, int V, bool HALF, int K>
constexpr bool few() {
  return sizeof(T) * V * K * (HALF ? 2 : 1) <= 32;
}

// What a lane holds of a row: K units.
template <typename T, int V, bool HALF, int K>
struct Place {
  int at[K], unit[K], rot_units;                   // first channel of unit k
  bool there[K], rotary[K];
  __device__ __forceinline__ Place(int lane, int lanes, int dim, int rot) {
    rot_units = HALF ? rot / 2 / V : rot / V;
    const int units = rot_units + (dim - rot) / V;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = lane + k * lanes;
      unit[k] = u;
      there[k] = u < units;
      rotary[k] = u < rot_units;
      at[k] = rotary[k] ? u * V : rot + (u - rot_units) * V;
    }
  }
};

// Two values an instruction where there are two.
template <int N>
__device__ __forceinline__ void mul(float (&d)[N], const float (&a)[N], const float (&b)[N]) {
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) {
    const float2 r = __fmul2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
    d[i] = r.x;
    d[i + 1] = r.y;
  }
  if constexpr (N % 2) d[N - 1] = a[N - 1] * b[N - 1];
}
template <int N>
__device__ __forceinline__ void mul(float (&d)[N], const float (&a)[N], float b) {
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) {
    const float2 r = __fmul2_rn(make_float2(a[i], a[i + 1]), make_float2(b, b));
    d[i] = r.x;
    d[i + 1] = r.y;
  }
  if constexpr (N % 2) d[N - 1] = a[N - 1] * b;
}
template <int N>
__device__ __forceinline__ void fma(float (&d)[N], const float (&a)[N], const float (&b)[N], const float (&c)[N]) {
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) {
    const float2 r = __ffma2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), make_float2(c[i], c[i + 1]));
    d[i] = r.x;
    d[i + 1] = r.y;
  }
  if constexpr (N % 2) d[N - 1] = fmaf(a[N - 1], b[N - 1], c[N - 1]);
}
template <int N>
__device__ __forceinline__ void fma(float (&d)[N], const float (&a)[N], float b, const float (&c)[N]) {
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) {
    const float2 r = __ffma2_rn(make_float2(a[i], a[i + 1]), make_float2(b, b), make_float2(c[i], c[i + 1]));
    d[i] = r.x;
    d[i + 1] = r.y;
  }
  if constexpr (N % 2) d[N - 1] = fmaf(a[N - 1], b, c[N - 1]);
}
// sum of a b, added to two partial sums
template <int N>
__device__ __forceinline__ void dot(float2& s, const float (&a)[N], const float (&b)[N]) {
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) s = __ffma2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), s);
  if constexpr (N % 2) s.x = fmaf(a[N - 1], b[N - 1], s.x);
}

// A unit's values in float32: V channels and, for a rotary unit of the half layout, their V partners (else zeros).
template <int V, bool HALF> struct Values {
  float a[V], b[HALF ? V : 1];
};
// N values to and from float32, two of a 16-bit type at a time where they come as words
template <typename T, int N, bool WIDE>
__device__ __forceinline__ void widen(float (&f)[N], const T* x) {
  if constexpr (WIDE && sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(x)[i];
      if constexpr (std::is_same<T, __half>::value) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      } else {
        f[2 * i] = __uint_as_float(w << 16);
        f[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = to_f(x[i]);
  }
}
template <typename T, int N, bool WIDE>
__device__ __forceinline__ void narrow(T* x, const float (&f)[N]) {
  if constexpr (WIDE && sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        reinterpret_cast<uint32_t*>(x)[i] = *reinterpret_cast<const uint32_t*>(&v);
      } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        reinterpret_cast<uint32_t*>(x)[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = from_f<T>(f[i]);
  }
}
template <typename T, int V, bool HALF, bool WIDE>
__device__ __forceinline__ Values<V, HALF> values_of(const Unit<T, V, V, HALF, WIDE>& x) {
  Values<V, HALF> f;
  widen<T, V, WIDE>(f.a, x.a.v);
  if constexpr (HALF) widen<T, V, WIDE>(f.b, x.b.v);
  else f.b[0] = 0.f;
  return f;
}

// The rotations of a token, as its rotary units read them: 4 floats a pair, weights included (wa, wb: of the pair's
// channels). Half layout: V floats each of wa cos, -wb sin, wb cos, wa sin; pairs layout: V floats of (wa cos, wb cos) and V
// of (-wb sin, wa sin). The 16-byte chunks of a unit are rot_units apart, so that the lanes of a row read without bank
// conflicts.
template <int V, bool HALF>
__device__ __forceinline__ void put_turn(float* token, int rot_units, int j, float2 cs, float wa, float wb) {
  constexpr int kPer = HALF ? V : V / 2;           // pairs of a unit
  const int u = j / kPer, e = j - u * kPer;
  const float f[4] = {wa * cs.x, HALF ? -wb * cs.y : wb * cs.x, HALF ? wb * cs.x : -wb * cs.y, wa * cs.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = HALF ? i * V + e : (i >> 1) * V + 2 * e + (i & 1);
    token[((at >> 2) * rot_units + u) * 4 + (at & 3)] = f[i];
  }
}
// a unit's values turned: Rot(w x) for the table's weights w
template <int V, bool HALF>
__device__ __forceinline__ void turn(Values<V, HALF>& f, const float* token, int rot_units, int u) {
  constexpr int kFloats = HALF ? 4 * V : 2 * V;
  float t[kFloats];
#pragma unroll
  for (int i = 0; i < kFloats / 4; ++i) {
    const float4 c = *reinterpret_cast<const float4*>(token + (i * rot_units + u) * 4);
    t[4 * i] = c.x;
    t[4 * i + 1] = c.y;
    t[4 * i + 2] = c.z;
    t[4 * i + 3] = c.w;
  }
  float swapped[V];
  if constexpr (HALF) {
    float ac[V], bs[V], bc[V], as[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      ac[e] = t[e];
      bs[e] = t[V + e];
      bc[e] = t[2 * V + e];
      as[e] = t[3 * V + e];
      swapped[e] = f.a[e];
    }
    mul<V>(f.a, f.a, ac);
    fma<V>(f.a, f.b, bs, f.a);
    mul<V>(f.b, f.b, bc);
    fma<V>(f.b, swapped, as, f.b);
  } else {
    float c2[V], s2[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      c2[e] = t[e];
      s2[e] = t[V + e];
      swapped[e] = f.a[e ^ 1];
    }
    mul<V>(f.a, f.a, c2);
    fma<V>(f.a, swapped, s2, f.a);
  }
}
template <typename T, int V, bool HALF, bool WIDE>
__device__ __forceinline__ void store(T* out, const Values<V, HALF>& f, int at, int half, bool rotary) {
  Unit<T, V, V, HALF, WIDE> x;
  narrow<T, V, WIDE>(x.a.v, f.a);
  if constexpr (HALF) narrow<T, V, WIDE>(x.b.v, f.b);
  x.store(out, at, half, rotary);
}
// What a lane has nothing of is zeros, so that the arithmetic needs no conditions: only loads and stores do.
template <typename T, int V, bool HALF, bool WIDE>
__device__ __forceinline__ Unit<T, V, V, HALF, WIDE> zeros() {
  Unit<T, V, V, HALF, WIDE> x;
#pragma unroll
  for (int e = 0; e < V; ++e) x.a.v[e] = x.b.v[e] = from_f<T>(0.f);
  return x;
}
template <typename T, int V, bool HALF, bool WIDE>
__device__ __forceinline__ Unit<T, V, V, HALF, WIDE> weights(const void* w, int at, int half, bool rotary) {
  Unit<T, V, V, HALF, WIDE> x = zeros<T, V, HALF, WIDE>();
  if (w != nullptr) {
    x.load(static_cast<const T*>(w), at, half, rotary);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) x.a.v[e] = x.b.v[e] = from_f<T>(1.f);
  }
  return x;
}
__device__ __forceinline__ float group_sum(float s, int lanes) {
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    if (m >= lanes) break;
    s += __shfl_xor_sync(0xffffffffu, s, m);
  }
  return s;
}
__device__ __forceinline__ float2 group_sum(float2 s, int lanes) {
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    if (m >= lanes) break;
    const float x = __shfl_xor_sync(0xffffffffu, s.x, m), y = __shfl_xor_sync(0xffffffffu, s.y, m);
    s = make_float2(s.x + x, s.y + y);
  }
  return s;
}

// A group's rows (token, head) of a CTA's tokens, head after head: rows group, group + groups, ... Steps are additions.
template <typename T>
struct Walk {
  const T* in;
  T* out;
  int t, h, dt, dh, heads;
  long long in_step, in_wrap, out_step, out_wrap;  // a step, and what a step past the last head adds
  __device__ __forceinline__ Walk(const RopeSide& s, long long t0, int group, int groups) {
    heads = s.heads;
    t = group / heads;
    h = group - t * heads;
    dt = groups / heads;
    dh = groups - dt * heads;
    in = static_cast<const T*>(s.in) + (t0 + t) * s.in_tok + h * s.in_head;
    out = static_cast<T*>(s.out) + (t0 + t) * s.out_tok + h * s.out_head;
    in_step = dt * s.in_tok + dh * s.in_head;
    in_wrap = s.in_tok - heads * s.in_head;
    out_step = dt * s.out_tok + dh * s.out_head;
    out_wrap = s.out_tok - heads * s.out_head;
  }
  __device__ __forceinline__ void next() {
    t += dt;
    h += dh;
    in += in_step;
    out += out_step;
    if (h >= heads) {
      h -= heads;
      ++t;
      in += in_wrap;
      out += out_wrap;
    }
  }
};

template <typename T>
__device__ __forceinline__ float weight_at(const void* w, int c) {
  return w != nullptr ? to_f(static_cast<const T*>(w)[c]) : 1.f;
}

template <typename T, int V, bool HALF, bool WIDE, int K>
__global__ void __launch_bounds__(kRopeThreads, few<T, V, HALF, K>() ? 4 : 2) k_norm_rope(NormArgs a) {
  __shared__ __align__(16) float table[2][4 * kRopeTable];   // of q, of k: [token][4 rot / 2]
  __shared__ __align__(16) float rest[2][512];     // the weights of the channels behind the rotated ones
  __shared__ int pos_s[kRopeTokens * kRopeAxes];
  constexpr bool kFew = few<T, V, HALF, K>();      // of wide rows, units that a lane does not have are skipped
  constexpr int kBatch = kFew ? 2 : 1;           // rows a group has in flight
  const int rot = a.r.rot, half = rot / 2, t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.r.n - t0), tid = threadIdx.x;
  const int lane = tid & (a.lanes - 1), group = tid / a.lanes, groups = kRopeThreads / a.lanes;
  const Place<T, V, HALF, K> p(lane, a.lanes, a.dim, rot);
  load_positions(a.r, t0, nt, pos_s, tid, kRopeThreads);
  __syncthreads();
  for (int i = tid; i < nt * half; i += kRopeThreads) {
    const int t = i / half, j = i - t * half, ca = HALF ? j : 2 * j, cb = HALF ? j + half : 2 * j + 1;
    const float2 cs = rope_turn(a.r, pos_s + t * kRopeAxes, j, 1.f);
    put_turn<V, HALF>(table[0] + t * 2 * rot, p.rot_units, j, cs, weight_at<T>(a.qw, ca), weight_at<T>(a.qw, cb));
    put_turn<V, HALF>(table[1] + t * 2 * rot, p.rot_units, j, cs, weight_at<T>(a.kw, ca), weight_at<T>(a.kw, cb));
  }
  for (int c = rot + tid; c < a.dim; c += kRopeThreads) {
    rest[0][c - rot] = weight_at<T>(a.qw, c);
    rest[1][c - rot] = weight_at<T>(a.kw, c);
  }
  __syncthreads();
  const float inv_dim = 1.f / (float)a.dim;
#pragma unroll 1
  for (int isk = 0; isk < 2; ++isk) {              // the heads of q, then of k
    const RopeSide s = isk ? a.k : a.q;
    if (s.heads == 0) continue;
    Walk<T> row(s, t0, group, groups);
    // the same trips for every lane of a warp: the row's sum is a shuffle
#pragma unroll 1
    for (int i0 = 0; i0 < nt * s.heads; i0 += kBatch * groups) {
      Unit<T, V, V, HALF, WIDE> x[kBatch][K];
      T* out[kBatch];
      const float* turns[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const bool live = row.t < nt && pos_s[row.t * kRopeAxes] >= 0;   // a padded row is left as it is
        out[b] = live ? row.out : nullptr;
        turns[b] = table[isk] + (live ? row.t : 0) * 2 * rot;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          x[b][k] = zeros<T, V, HALF, WIDE>();
          if (live && p.there[k]) x[b][k].load(row.in, p.at[k], half, p.rotary[k]);
        }
        row.next();
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        float2 ss = make_float2(0.f, 0.f);
        Values<V, HALF> f[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (!kFew && !p.there[k]) continue;
          f[k] = values_of<T, V, HALF, WIDE>(x[b][k]);
          dot(ss, f[k].a, f[k].a);
          if (HALF && (kFew || p.rotary[k])) dot(ss, f[k].b, f[k].b);
        }
        const float r = rsqrtf(group_sum(ss.x + ss.y, a.lanes) * inv_dim + a.eps);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (!kFew && !p.there[k]) continue;
          mul(f[k].a, f[k].a, r);
          if (HALF && (kFew || p.rotary[k])) mul(f[k].b, f[k].b, r);
          if (p.rotary[k]) {
            turn<V, HALF>(f[k], turns[b], p.rot_units, p.unit[k]);
          } else if (p.there[k]) {
#pragma unroll
            for (int e = 0; e < V; ++e) f[k].a[e] *= rest[isk][p.at[k] - rot + e];
          }
          if (out[b] != nullptr && p.there[k]) store<T, V, HALF, WIDE>(out[b], f[k], p.at[k], half, p.rotary[k]);
        }
      }
    }
  }
}

// What a lane has loaded of a row for the gradient.
template <typename T, int V, bool HALF, bool WIDE, int K>
struct GradRow {
  Unit<T, V, V, HALF, WIDE> x[K], g[K];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = g[k] = zeros<T, V, HALF, WIDE>();
  }
  template <typename P>
  __device__ __forceinline__ void load(const P& p, const T* in, const T* gin, int half) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (p.there[k]) {
        x[k].load(in, p.at[k], half, p.rotary[k]);
        g[k].load(gin, p.at[k], half, p.rotary[k]);
      }
  }
  // The same through shared memory: asynchronous 16-byte copies into slots of the thread's own, chunk j of all threads side by
  // side at slot + j * 16 * kRopeThreads.
  static constexpr int kParts = HALF ? 2 : 1, kChunks = 2 * K * kParts;
  template <typename P>
  static __device__ __forceinline__ void copy(uint32_t slot, const P& p, const T* in, const T* gin, int half) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int part = 0; part < kParts; ++part)
        if (p.there[k] && (part == 0 || p.rotary[k])) {
          const int at = p.at[k] + part * half, j = 2 * (k * kParts + part);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + j * 16 * kRopeThreads), "l"(in + at) : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(slot + (j + 1) * 16 * kRopeThreads), "l"(gin + at)
                       : "memory");
        }
  }
  template <typename P>
  __device__ __forceinline__ void take(uint32_t slot, const P& p) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int part = 0; part < kParts; ++part)
        if (p.there[k] && (part == 0 || p.rotary[k])) {
          const int j = 2 * (k * kParts + part);
          const uint4 cx = lds128(slot + j * 16 * kRopeThreads), cg = lds128(slot + (j + 1) * 16 * kRopeThreads);
          *reinterpret_cast<uint4*>(part ? x[k].b.v : x[k].a.v) = cx;
          *reinterpret_cast<uint4*>(part ? g[k].b.v : g[k].a.v) = cg;
        }
  }
};

// The rows of a group, some trips ahead of those it works on: trip by trip, tokens by tokens as the CTA walks them.
template <typename T>
struct Ahead {
  RopeSide s;
  Walk<T> row;                                     // out: the gradient's row
  long long t0, step, n;
  int tokens, group, groups, i0, nt;
  __device__ __forceinline__ Ahead(const RopeSide& s_, long long t0_, long long step_, long long n_, int tokens_, int group_, int groups_)
      : s(s_), row(s_, t0_, group_, groups_), t0(t0_), step(step_), n(n_), tokens(tokens_), group(group_), groups(groups_), i0(0),
        nt((int)min((long long)tokens_, n_ - t0_)) {}
  __device__ __forceinline__ bool there() const { return row.t < nt; }     // nt < 1 behind the last tokens
  __device__ __forceinline__ void next() {
    i0 += groups;
    if (i0 < nt * s.heads) {
      row.next();
    } else {
      t0 += step;
      i0 = 0;
      nt = (int)max(min((long long)tokens, n - t0), 0ll);
      row = Walk<T>(s, t0, group, groups);
    }
  }
};

template <typename T, int V, bool HALF, bool WIDE, int K>
constexpr bool grad_async() {
  return WIDE && sizeof(T) * V == 16 && few<T, V, HALF, K>();
}
constexpr int kSlots = 3;                          // rows of a thread in shared memory: one worked on, two on their way
template <typename T, int V, bool HALF, bool WIDE, int K>
constexpr int grad_smem() {
  return 16 * kGradTable + (grad_async<T, V, HALF, WIDE, K>() ? kSlots * GradRow<T, V, HALF, WIDE, K>::kChunks * 16 * kRopeThreads : 0);
}

template <typename T, int V, bool HALF, bool WIDE, int K>
__global__ void __launch_bounds__(kRopeThreads, few<T, V, HALF, K>() ? 2 : 1) k_norm_rope_grad(NormArgs a) {
  extern __shared__ __align__(16) float smem[];
  float* const table = smem;                       // [token][4 rot / 2]; at the end a warp's share of dw: [8][512]
  __shared__ int pos_s[kGradTokens * kRopeAxes];
  static_assert(4 * kGradTable >= kRopeThreads / 32 * 512, "the warps' shares fit");
  using Row = GradRow<T, V, HALF, WIDE, K>;
  constexpr bool kAsync = grad_async<T, V, HALF, WIDE, K>(), kFew = few<T, V, HALF, K>();
  const int rot = a.r.rot, half = rot / 2, tid = threadIdx.x;
  const int lane = tid & (a.lanes - 1), group = tid / a.lanes, groups = kRopeThreads / a.lanes;
  const bool isq = (int)blockIdx.x < a.q_ctas;
  const RopeSide s = isq ? a.q : a.k, sg = isq ? a.gq : a.gk;
  const int first = isq ? blockIdx.x : blockIdx.x - a.q_ctas, ctas = isq ? a.q_ctas : gridDim.x - a.q_ctas;
  const long long step = (long long)ctas * a.tokens;
  const Place<T, V, HALF, K> p(lane, a.lanes, a.dim, rot);
  Unit<T, V, V, HALF, WIDE> w[K];
  Values<V, HALF> dw[K] = {};
#pragma unroll
  for (int k = 0; k < K; ++k)
    w[k] = p.there[k] ? weights<T, V, HALF, WIDE>(isq ? a.qw : a.kw, p.at[k], half, p.rotary[k]) : zeros<T, V, HALF, WIDE>();
  const float inv_dim = 1.f / (float)a.dim;
  // A group's next rows are on their way while it works on one, also across the CTA's tokens.
  const RopeSide both = {s.in, const_cast<void*>(sg.in), s.in_tok, s.in_head, sg.in_tok, sg.in_head, s.heads};
  Ahead<T> ahead(both, (long long)first * a.tokens, step, a.r.n, a.tokens, group, groups);
  const uint32_t slots = smem_addr(smem) + 16 * kGradTable + 16 * tid;
  int slot = 0;                                    // of the row that is worked on
  Row next;
  auto fetch = [&](int to) {
    if constexpr (kAsync) {
      if (ahead.there()) Row::copy(slots + to * (Row::kChunks * 16 * kRopeThreads), p, ahead.row.in, ahead.row.out, half);
      asm volatile("cp.async.commit_group;" ::: "memory");
    } else {
      next.clear();
      if (ahead.there()) next.load(p, ahead.row.in, ahead.row.out, half);
    }
    ahead.next();
  };
#pragma unroll 1
  for (int i = 0; i < (kAsync ? kSlots - 1 : 1); ++i) fetch(i);
#pragma unroll 1
  for (long long t0 = (long long)first * a.tokens; t0 < a.r.n; t0 += step) {
    const int nt = (int)min((long long)a.tokens, a.r.n - t0), items = nt * s.heads;
    Walk<T> row(s, t0, group, groups);
    __syncthreads();                               // the last tokens' angles have been read
    load_positions(a.r, (int)t0, nt, pos_s, tid, kRopeThreads);
    __syncthreads();
    for (int i = tid; i < nt * half; i += kRopeThreads) {
      const int t = i / half, j = i - t * half;
      put_turn<V, HALF>(table + t * 2 * rot, p.rot_units, j, rope_turn(a.r, pos_s + t * kRopeAxes, j, -1.f), 1.f, 1.f);
    }
    __syncthreads();
#pragma unroll 1
    for (int i0 = 0; i0 < items; i0 += groups) {
      const bool live = row.t < nt && pos_s[row.t * kRopeAxes] >= 0;
      Row now;
      now.clear();
      if constexpr (kAsync) {
        // the row worked on before is read: its slot is the next to fill
        asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 2) : "memory");
        if (live) now.take(slots + slot * (Row::kChunks * 16 * kRopeThreads), p);
        fetch(slot == 0 ? kSlots - 1 : slot - 1);
        slot = slot == kSlots - 1 ? 0 : slot + 1;
      } else {
        if (live) now = next;
        fetch(0);
      }
      T* const out = row.out;
      const float* const turns = table + (live ? row.t : 0) * 2 * rot;
      row.next();
      float2 ss = make_float2(0.f, 0.f), ux = ss;
      Values<V, HALF> fh[K], fu[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!kFew && !p.there[k]) continue;
        const Values<V, HALF> fx = values_of<T, V, HALF, WIDE>(now.x[k]), fw = values_of<T, V, HALF, WIDE>(w[k]);
        fh[k] = values_of<T, V, HALF, WIDE>(now.g[k]);
        if (p.rotary[k]) turn<V, HALF>(fh[k], turns, p.rot_units, p.unit[k]);
        mul(fu[k].a, fh[k].a, fw.a);
        dot(ss, fx.a, fx.a);
        dot(ux, fu[k].a, fx.a);
        if (HALF && (kFew || p.rotary[k])) {
          mul(fu[k].b, fh[k].b, fw.b);
          dot(ss, fx.b, fx.b);
          dot(ux, fu[k].b, fx.b);
        }
      }
      const float2 both_sums = group_sum(make_float2(ss.x + ss.y, ux.x + ux.y), a.lanes);
      const float r = rsqrtf(both_sums.x * inv_dim + a.eps), along = -both_sums.y * inv_dim * r * r;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!kFew && !p.there[k]) continue;
        const Values<V, HALF> fx = values_of<T, V, HALF, WIDE>(now.x[k]);
        Values<V, HALF> xr, dx;
        mul(xr.a, fx.a, r);
        fma(dw[k].a, fh[k].a, xr.a, dw[k].a);
        fma(dx.a, fx.a, along, fu[k].a);
        mul(dx.a, dx.a, r);
        if (HALF && (kFew || p.rotary[k])) {
          mul(xr.b, fx.b, r);
          fma(dw[k].b, fh[k].b, xr.b, dw[k].b);
          fma(dx.b, fx.b, along, fu[k].b);
          mul(dx.b, dx.b, r);
        }
        if (live && p.there[k]) store<T, V, HALF, WIDE>(out, dx, p.at[k], half, p.rotary[k]);
      }
    }
  }
  if constexpr (kAsync) asm volatile("cp.async.wait_all;" ::: "memory");
  if (a.partials == nullptr) return;
  // the groups of a warp, then the warps, in a fixed order
  const int warp = tid >> 5;
  float* sums = table + warp * 512;
  __syncthreads();                                 // the last angles have been read
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float da = dw[k].a[e], db = HALF ? dw[k].b[e] : 0.f;
      for (int m = a.lanes; m < 32; m <<= 1) {
        da += __shfl_xor_sync(0xffffffffu, da, m);
        if (HALF) db += __shfl_xor_sync(0xffffffffu, db, m);
      }
      if (p.there[k] && (tid & 31) < a.lanes) {
        sums[p.at[k] + e] = da;
        if (HALF && p.rotary[k]) sums[p.at[k] + half + e] = db;
      }
    }
  }
  __syncthreads();
  for (int c = tid; c < a.dim; c += kRopeThreads) {
    float s8 = 0.f;
#pragma unroll
    for (int i = 0; i < kRopeThreads / 32; ++i) s8 += table[i * 512 + c];
    a.partials[(size_t)blockIdx.x * a.dim + c] = s8;
  }
}

// blockIdx.y: the weight of q or of k; a warp's lanes are channels, warp y adds the CTAs y, y + 8, ...
__global__ void __launch_bounds__(32 * kSumRows) k_norm_rope_sum(const float* partials, int dim, int q_ctas, int ctas, float* dqw,
                                                                 float* dkw) {
  __shared__ float part[kSumRows][32];
  const int c = blockIdx.x * 32 + threadIdx.x, y = threadIdx.y;
  const bool isq = blockIdx.y == 0;
  float* out = isq ? dqw : dkw;
  if (out == nullptr) return;
  const int lo = isq ? 0 : q_ctas, hi = isq ? q_ctas : ctas;
  float s = 0.f;
  if (c < dim) {
#pragma unroll 8
    for (int i = lo + y; i < hi; i += kSumRows) s += partials[(size_t)i * dim + c];
  }
  part[y][threadIdx.x] = s;
  __syncthreads();
  if (y != 0 || c >= dim) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kSumRows; ++i) s += part[i][threadIdx.x];
  out[c] = s;
}

int sm_count(int* sms) {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess
             ? OSCAR_OK
             : OSCAR_ERR_CUDA;
}

template <typename T, int V, bool HALF, bool WIDE, int K>
int launch_as(NormArgs a, bool grad, float* dqw, float* dkw, cudaStream_t st) {
  const int rot = a.r.rot, half = rot / 2, units = (HALF ? half / V : rot / V) + (a.dim - rot) / V;
  a.lanes = 1;
  while (a.lanes < 32 && a.lanes * K < units) a.lanes *= 2;
  int sms = 0;
  if (int rc = sm_count(&sms); rc != OSCAR_OK) return rc;
  if (!grad) {
    a.tokens = std::max(1, std::min(std::min(kRopeTable / half, kRopeTokens), a.r.n / (4 * sms)));
    k_norm_rope<T, V, HALF, WIDE, K><<<(a.r.n - 1) / a.tokens + 1, kRopeThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
  }
  a.tokens = std::max(1, std::min(std::min(kGradTable / half, kGradTokens), a.r.n / (2 * sms)));
  // CTAs are shared between q and k by their heads
  const int tiles = (a.r.n - 1) / a.tokens + 1, heads = a.q.heads + a.k.heads;
  const int most_q = std::max(1, std::min(kGradCtas - 1, (int)((long long)kGradCtas * a.q.heads / heads)));
  a.q_ctas = a.q.heads == 0 ? 0 : std::min(tiles, a.k.heads == 0 ? kGradCtas : most_q);
  const int k_ctas = a.k.heads == 0 ? 0 : std::min(tiles, a.q.heads == 0 ? kGradCtas : kGradCtas - most_q);
  const int ctas = a.q_ctas + k_ctas;
  constexpr int smem = grad_smem<T, V, HALF, WIDE, K>();
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(k_norm_rope_grad<T, V, HALF, WIDE, K>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return OSCAR_ERR_CUDA;
  k_norm_rope_grad<T, V, HALF, WIDE, K><<<ctas, kRopeThreads, smem, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return OSCAR_ERR_CUDA;
  if (a.partials == nullptr) return OSCAR_OK;
  k_norm_rope_sum<<<dim3((a.dim + 31) / 32, 2), dim3(32, kSumRows), 0, st>>>(a.partials, a.dim, a.q_ctas, ctas, dqw, dkw);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

// bytes: the widest access (16, 8 or single elements) that every row, half and remainder starts on a multiple of
template <typename T, bool HALF>
int launch_layout(const NormArgs& a, int bytes, bool grad, float* dqw, float* dkw, cudaStream_t st) {
  constexpr int V16 = 16 / sizeof(T), V8 = 8 / sizeof(T), kLeast = HALF ? 1 : 2;
  const int rot = a.r.rot;
  if (bytes == 16) {
    const int units = (HALF ? rot / 2 : rot) / V16 + (a.dim - rot) / V16;
    // 32 bytes a lane: a unit of the half layout with its partners, two of the pairs layout (one: PAIRS_MEASURED)
    constexpr int kFew = HALF ? 1 : 2;
    if (units <= 32 * kFew) return launch_as<T, V16, HALF, true, kFew>(a, grad, dqw, dkw, st);
    return launch_as<T, V16, HALF, true, 128 / (32 * V16 / 4)>(a, grad, dqw, dkw, st);
  }
  if (bytes == 8) return launch_as<T, V8, HALF, true, 16 / V8>(a, grad, dqw, dkw, st);
  return launch_as<T, kLeast, HALF, false, 16 / kLeast>(a, grad, dqw, dkw, st);
}
template <typename T>
int launch_typed(const NormArgs& a, bool half_layout, int bytes, bool grad, float* dqw, float* dkw, cudaStream_t st) {
  return half_layout ? launch_layout<T, true>(a, bytes, grad, dqw, dkw, st) : launch_layout<T, false>(a, bytes, grad, dqw, dkw, st);
}

}  // namespace

size_t norm_rope_workspace_bytes(int dim) { return (size_t)kGradCtas * dim * sizeof(float); }

int launch_norm_rope(const oscar_rope_tensor& q, const oscar_rope_tensor& k, const oscar_rope_tensor* grad, int n, int dim,
                     int dtype, const int* positions, const oscar_rotary& r, const oscar_head_norm& norm, float* dqw, float* dkw,
                     float* partials, cudaStream_t st) {
  NormArgs a = {};
  a.q = side(q);
  a.k = side(k);
  if (grad != nullptr) {
    a.gq = side(grad[0]);
    a.gk = side(grad[1]);
  }
  a.qw = norm.q_weight;
  a.kw = norm.k_weight;
  a.r = rotary_of(r, positions, n);
  a.dim = dim;
  a.eps = norm.eps;
  a.partials = dqw != nullptr || dkw != nullptr ? partials : nullptr;
  const bool half_layout = r.layout == OSCAR_ROPE_HALF;
  const int size = dtype == OSCAR_DTYPE_FP32 ? 4 : 2, rot = r.rotary_dim;
  int bytes = 16;
  for (; bytes >= 8; bytes /= 2) {
    const int v = bytes / size;
    const bool rows = fits(q, size, v) && fits(k, size, v) && (grad == nullptr || (fits(grad[0], size, v) && fits(grad[1], size, v)));
    const uintptr_t w = reinterpret_cast<uintptr_t>(a.qw) | reinterpret_cast<uintptr_t>(a.kw);
    if (rows && w % bytes == 0 && (half_layout ? rot / 2 : rot) % v == 0 && (dim - rot) % v == 0) break;
  }
  const bool g = grad != nullptr;
  if (dtype == OSCAR_DTYPE_FP32) return launch_typed<float>(a, half_layout, bytes, g, dqw, dkw, st);
  if (dtype == OSCAR_DTYPE_FP16) return launch_typed<__half>(a, half_layout, bytes, g, dqw, dkw, st);
  return launch_typed<__nv_bfloat16>(a, half_layout, bytes, g, dqw, dkw, st);
}

}  // namespace oscar
