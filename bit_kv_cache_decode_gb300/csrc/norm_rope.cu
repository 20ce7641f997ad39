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
// Measured, 128 channels, all turned in halves, bf16: 32,769 tokens x (64 + 8) heads, 1.208 GB, 197 us (6.1 TB/s, 92 % of the
// copy rate); one token 4.2 us in a graph.
//
// Gradient: the weights' sums are held in registers over all rows of a CTA, which walks tokens of q or of k; CTAs'
// partial sums go to the workspace and are added in a fixed order by a second kernel, so results do not depend on timing.
// Registers allow two CTAs an SM, too few loads to fill the memory's latency: rows come by asynchronous copies, two rows ahead.
// 32,769 tokens x (32 + 8) heads, 1.007 GB: 169 to 173 us (5.9 TB/s, 88 %; 62 % of the issue slots); 301 tokens 7.6 us in a graph.
#include <algorithm>
#include <mutex>
#include <set>
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

// Units of a row. Half layout: two chunks of V channels, those of the first half that turn and their partners; pairs layout:
// one chunk. Behind the rotated channels a unit of either layout is as many channels in a row. A lane holds K units.
template <bool HALF> constexpr int kParts = HALF ? 2 : 1;
// whether a lane holds no more than 32 bytes of a row: all but odd alignments and the longest float32 rows
template <typename T, int V, bool HALF, int K>
constexpr bool few() {
  return sizeof(T) * V * K * kParts<HALF> <= 32;
}
template <int V, bool HALF>
__host__ __device__ inline int units_of(int dim, int rot) {
  constexpr int n = V * kParts<HALF>;
  return (HALF ? rot / 2 / V : rot / V) + (dim - rot + n - 1) / n;
}

template <int V, bool HALF, int K>
struct Place {
  int rot_units, unit[K], at[K], second[K];        // first channel of a unit, and from it to its second chunk
  bool there[K][kParts<HALF>], rotary[K];
  __device__ __forceinline__ Place(int lane, int lanes, int dim, int rot) {
    rot_units = HALF ? rot / 2 / V : rot / V;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      unit[k] = lane + k * lanes;
      rotary[k] = unit[k] < rot_units;
      at[k] = rotary[k] ? unit[k] * V : rot + (unit[k] - rot_units) * V * kParts<HALF>;
      second[k] = rotary[k] ? rot / 2 : V;
#pragma unroll
      for (int p = 0; p < kParts<HALF>; ++p) there[k][p] = at[k] + p * second[k] + V <= dim;
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
// each element is touched once: streaming accesses where they are wide
template <typename T, int V, bool WIDE>
__device__ __forceinline__ void get(Vec<T, V, WIDE>& x, const T* at) {
  if constexpr (WIDE) {
    using Bits = typename AccessOf<sizeof(T) * V>::type;
    *reinterpret_cast<Bits*>(x.v) = __ldcs(reinterpret_cast<const Bits*>(at));
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) x.v[e] = at[e];
  }
}
template <typename T, int V, bool WIDE>
__device__ __forceinline__ void put(T* at, const Vec<T, V, WIDE>& x) {
  if constexpr (WIDE) {
    using Bits = typename AccessOf<sizeof(T) * V>::type;
    __stcs(reinterpret_cast<Bits*>(at), *reinterpret_cast<const Bits*>(x.v));
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) at[e] = x.v[e];
  }
}
// What a lane has of a row, as it is loaded and in float32.
template <typename T, int V, bool HALF, bool WIDE, int K>
struct Raw {
  Vec<T, V, WIDE> x[K][kParts<HALF>];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int p = 0; p < kParts<HALF>; ++p)
#pragma unroll
        for (int e = 0; e < V; ++e) x[k][p].v[e] = from_f<T>(0.f);
  }
  __device__ __forceinline__ void load(const Place<V, HALF, K>& pl, const T* in) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int p = 0; p < kParts<HALF>; ++p)
        if (pl.there[k][p]) get<T, V, WIDE>(x[k][p], in + pl.at[k] + p * pl.second[k]);
  }
};
template <int V, bool HALF, int K>
struct Values {
  float f[K][kParts<HALF>][V];
  template <typename T, bool WIDE>
  __device__ __forceinline__ explicit Values(const Raw<T, V, HALF, WIDE, K>& r) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int p = 0; p < kParts<HALF>; ++p) widen<T, V, WIDE>(f[k][p], r.x[k][p].v);
  }
  __device__ __forceinline__ explicit Values(float x) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int p = 0; p < kParts<HALF>; ++p)
#pragma unroll
        for (int e = 0; e < V; ++e) f[k][p][e] = x;
  }
  template <typename T, bool WIDE>
  __device__ __forceinline__ void store(const Place<V, HALF, K>& pl, T* out) const {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int p = 0; p < kParts<HALF>; ++p) {
        Vec<T, V, WIDE> x;
        narrow<T, V, WIDE>(x.v, f[k][p]);
        if (pl.there[k][p]) put<T, V, WIDE>(out + pl.at[k] + p * pl.second[k], x);
      }
  }
};

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
__device__ __forceinline__ void turn(float (&f)[kParts<HALF>][V], const float* token, int rot_units, int u) {
  constexpr int kFloats = HALF ? 4 * V : 2 * V;
  float t[kFloats / V][V], swapped[V];
#pragma unroll
  for (int i = 0; i < kFloats / 4; ++i) {
    const float4 c = *reinterpret_cast<const float4*>(token + (i * rot_units + u) * 4);
    t[4 * i / V][4 * i % V] = c.x;
    t[(4 * i + 1) / V][(4 * i + 1) % V] = c.y;
    t[(4 * i + 2) / V][(4 * i + 2) % V] = c.z;
    t[(4 * i + 3) / V][(4 * i + 3) % V] = c.w;
  }
#pragma unroll
  for (int e = 0; e < V; ++e) swapped[e] = f[0][HALF ? e : e ^ 1];
  mul<V>(f[0], f[0], t[0]);
  if constexpr (HALF) {
    fma<V>(f[0], f[1], t[1], f[0]);
    mul<V>(f[1], f[1], t[2]);
    fma<V>(f[1], swapped, t[3], f[1]);
  } else {
    fma<V>(f[0], swapped, t[1], f[0]);
  }
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

// Rows are zeros where a lane has nothing of them, so that the arithmetic of the usual rows needs no conditions.
template <typename T, int V, bool HALF, bool WIDE, int K>
__global__ void __launch_bounds__(kRopeThreads, few<T, V, HALF, K>() ? 4 : 2) k_norm_rope(NormArgs a) {
  __shared__ __align__(16) float table[2][4 * kRopeTable];   // of q, of k: [token][4 rot / 2]
  __shared__ __align__(16) float rest[2][512];     // the weights of the channels behind the rotated ones
  __shared__ int pos_s[kRopeTokens * kRopeAxes];
  constexpr bool kFew = few<T, V, HALF, K>();
  constexpr int kBatch = kFew ? 2 : 1;             // rows a group has in flight
  using Data = Raw<T, V, HALF, WIDE, K>;
  const int rot = a.r.rot, half = rot / 2, t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.r.n - t0), tid = threadIdx.x;
  const int lane = tid & (a.lanes - 1), group = tid / a.lanes, groups = kRopeThreads / a.lanes;
  const Place<V, HALF, K> pl(lane, a.lanes, a.dim, rot);
  load_positions(a.r, t0, nt, pos_s, tid, kRopeThreads);
  __syncthreads();
  for (int i = tid; i < nt * half; i += kRopeThreads) {
    const int t = i / half, j = i - t * half, ca = HALF ? j : 2 * j, cb = HALF ? j + half : 2 * j + 1;
    const float2 cs = rope_turn(a.r, pos_s + t * kRopeAxes, j, 1.f);
    put_turn<V, HALF>(table[0] + t * 2 * rot, pl.rot_units, j, cs, weight_at<T>(a.qw, ca), weight_at<T>(a.qw, cb));
    put_turn<V, HALF>(table[1] + t * 2 * rot, pl.rot_units, j, cs, weight_at<T>(a.kw, ca), weight_at<T>(a.kw, cb));
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
      Data x[kBatch];
      T* out[kBatch];
      const float* turns[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const bool live = row.t < nt && pos_s[row.t * kRopeAxes] >= 0;   // a padded row is left as it is
        out[b] = live ? row.out : nullptr;
        turns[b] = table[isk] + (live ? row.t : 0) * 2 * rot;
        x[b].clear();
        if (live) x[b].load(pl, row.in);
        row.next();
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        Values<V, HALF, K> f(x[b]);
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int p = 0; p < kParts<HALF>; ++p)
            if (kFew || pl.there[k][p]) dot(ss, f.f[k][p], f.f[k][p]);
        const float r = rsqrtf(group_sum(ss.x + ss.y, a.lanes) * inv_dim + a.eps);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (!kFew && !pl.there[k][0]) continue;
#pragma unroll
          for (int p = 0; p < kParts<HALF>; ++p) mul(f.f[k][p], f.f[k][p], r);
          if (pl.rotary[k]) {
            turn<V, HALF>(f.f[k], turns[b], pl.rot_units, pl.unit[k]);
          } else {
#pragma unroll
            for (int p = 0; p < kParts<HALF>; ++p)
              if (pl.there[k][p])
#pragma unroll
                for (int e = 0; e < V; ++e) f.f[k][p][e] *= rest[isk][pl.at[k] + p * V - rot + e];
          }
        }
        if (out[b] != nullptr) f.template store<T, WIDE>(pl, out[b]);
      }
    }
  }
}

// A group's rows, some trips ahead of those it works on: trip by trip, tokens by tokens as the CTA walks them.
template <typename T>
struct Ahead {
  RopeSide s;
  Walk<T> row;                                     // out: the row of the gradient that is given
  long long t0, end;
  int tokens, group, groups, i0, nt;
  __device__ __forceinline__ Ahead(const RopeSide& s_, long long begin, long long end_, int tokens_, int group_, int groups_)
      : s(s_), row(s_, begin, group_, groups_), t0(begin), end(end_), tokens(tokens_), group(group_), groups(groups_), i0(0),
        nt((int)min((long long)tokens_, end_ - begin)) {}
  __device__ __forceinline__ bool there() const { return row.t < nt; }     // behind the last tokens nt is 0
  __device__ __forceinline__ void next() {
    i0 += groups;
    if (i0 < nt * s.heads) {
      row.next();
    } else {
      t0 = min(t0 + tokens, end);
      i0 = 0;
      nt = (int)min((long long)tokens, end - t0);
      row = Walk<T>(s, t0, group, groups);
    }
  }
};

// Rows on their way: x and g of a row by asynchronous copies into slots of the thread's own in shared memory, chunk j of all
// threads side by side (no bank conflicts, no registers). Single elements, and rows of more than 32 bytes a lane, wait in registers.
constexpr int kSlots = 3;                          // one row worked on, two on their way
template <typename T, int V, bool HALF, bool WIDE, int K>
struct Slots {
  static constexpr bool kAsync = WIDE && few<T, V, HALF, K>();
  static constexpr int kBytes = sizeof(T) * V, kChunk = kBytes * kRopeThreads, kSlot = 2 * K * kParts<HALF> * kChunk;
  static constexpr int kSmem = kAsync ? kSlots * kSlot : 0;
  static __device__ __forceinline__ void copy(uint32_t slot, const Place<V, HALF, K>& pl, const T* in, const T* gin) {
    if constexpr (kAsync) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int p = 0; p < kParts<HALF>; ++p)
          if (pl.there[k][p]) {
            const int c = pl.at[k] + p * pl.second[k];
            const uint32_t to = slot + 2 * (k * kParts<HALF> + p) * kChunk;
            if constexpr (kBytes == 16) {
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(in + c) : "memory");
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + kChunk), "l"(gin + c) : "memory");
            } else {
              asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(in + c) : "memory");
              asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to + kChunk), "l"(gin + c) : "memory");
            }
          }
    }
  }
  // chunks that a lane does not have stay the zeros of the start
  static __device__ __forceinline__ void clear(uint32_t slots) {
    if constexpr (kAsync)
      for (int i = 0; i < kSlots * kSlot / kChunk; ++i)
        for (int b = 0; b < kBytes; b += 4) sts32(slots + i * kChunk + b, 0u);
  }
  static __device__ __forceinline__ void take(uint32_t slot, Raw<T, V, HALF, WIDE, K>& x, Raw<T, V, HALF, WIDE, K>& g) {
    if constexpr (kAsync) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int p = 0; p < kParts<HALF>; ++p) {
          const uint32_t at = slot + 2 * (k * kParts<HALF> + p) * kChunk;
          if constexpr (kBytes == 16) {
            *reinterpret_cast<uint4*>(x.x[k][p].v) = lds128(at);
            *reinterpret_cast<uint4*>(g.x[k][p].v) = lds128(at + kChunk);
          } else {
            *reinterpret_cast<uint2*>(x.x[k][p].v) = lds64(at);
            *reinterpret_cast<uint2*>(g.x[k][p].v) = lds64(at + kChunk);
          }
        }
    }
  }
};

template <typename T, int V, bool HALF, bool WIDE, int K>
__global__ void __launch_bounds__(kRopeThreads, few<T, V, HALF, K>() ? 2 : 1) k_norm_rope_grad(NormArgs a) {
  extern __shared__ __align__(16) float smem[];
  float* const table = smem;                       // [token][4 rot / 2]; at the end a warp's share of dw: [8][512]
  __shared__ int pos_s[kGradTokens * kRopeAxes];
  static_assert(4 * kGradTable >= kRopeThreads / 32 * 512, "the warps' shares fit");
  using Data = Raw<T, V, HALF, WIDE, K>;
  using Ring = Slots<T, V, HALF, WIDE, K>;
  using Floats = Values<V, HALF, K>;
  constexpr bool kFew = few<T, V, HALF, K>();
  const int rot = a.r.rot, half = rot / 2, tid = threadIdx.x;
  const int lane = tid & (a.lanes - 1), group = tid / a.lanes, groups = kRopeThreads / a.lanes;
  const bool isq = (int)blockIdx.x < a.q_ctas;
  const RopeSide s = isq ? a.q : a.k, sg = isq ? a.gq : a.gk;
  const int first = isq ? blockIdx.x : blockIdx.x - a.q_ctas, ctas = isq ? a.q_ctas : gridDim.x - a.q_ctas;
  // a range of the tokens, a few at a time (every ctas-th few: a fifth of the time in CTAs that had one more to do)
  const long long begin = (long long)a.r.n * first / ctas, end = (long long)a.r.n * (first + 1) / ctas;
  const Place<V, HALF, K> pl(lane, a.lanes, a.dim, rot);
  Floats fw(0.f), dw(0.f);
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int p = 0; p < kParts<HALF>; ++p)
      if (pl.there[k][p])
#pragma unroll
        for (int e = 0; e < V; ++e) fw.f[k][p][e] = weight_at<T>(isq ? a.qw : a.kw, pl.at[k] + p * pl.second[k] + e);
  const float inv_dim = 1.f / (float)a.dim;
  // A group's next rows are on their way while it works on one, also across the CTA's tokens.
  const RopeSide both = {s.in, const_cast<void*>(sg.in), s.in_tok, s.in_head, sg.in_tok, sg.in_head, s.heads};
  Ahead<T> ahead(both, begin, end, a.tokens, group, groups);
  const uint32_t slots = smem_addr(smem) + 16 * kGradTable + Ring::kBytes * tid;
  int slot = 0;                                    // of the row that is worked on
  Ring::clear(slots);
  Data next_x, next_g;
  auto fetch = [&](int to) {
    if constexpr (Ring::kAsync) {
      if (ahead.there()) Ring::copy(slots + to * Ring::kSlot, pl, ahead.row.in, ahead.row.out);
      asm volatile("cp.async.commit_group;" ::: "memory");
    } else {
      next_x.clear();
      next_g.clear();
      if (ahead.there()) {
        next_x.load(pl, ahead.row.in);
        next_g.load(pl, ahead.row.out);
      }
    }
    ahead.next();
  };
#pragma unroll 1
  for (int i = 0; i < (Ring::kAsync ? kSlots - 1 : 1); ++i) fetch(i);
#pragma unroll 1
  for (long long t0 = begin; t0 < end; t0 += a.tokens) {
    const int nt = (int)min((long long)a.tokens, end - t0), items = nt * s.heads;
    Walk<T> row(s, t0, group, groups);
    __syncthreads();                               // the last tokens' angles have been read
    load_positions(a.r, (int)t0, nt, pos_s, tid, kRopeThreads);
    __syncthreads();
    for (int i = tid; i < nt * half; i += kRopeThreads) {
      const int t = i / half, j = i - t * half;
      put_turn<V, HALF>(table + t * 2 * rot, pl.rot_units, j, rope_turn(a.r, pos_s + t * kRopeAxes, j, -1.f), 1.f, 1.f);
    }
    __syncthreads();
#pragma unroll 1
    for (int i0 = 0; i0 < items; i0 += groups) {
      const bool live = row.t < nt && pos_s[row.t * kRopeAxes] >= 0;
      Data x, g;
      if constexpr (Ring::kAsync) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 2) : "memory");
        Ring::take(slots + slot * Ring::kSlot, x, g);
        fetch(slot == 0 ? kSlots - 1 : slot - 1);  // the row before this one is done with
        slot = slot == kSlots - 1 ? 0 : slot + 1;
      } else {
        x = next_x;
        g = next_g;
        fetch(0);
      }
      if (!__all_sync(0xffffffffu, live) && !live) {   // no row, or a padded one: it adds nothing, whatever it holds
        x.clear();
        g.clear();
      }
      T* const out = row.out;
      const float* const turns = table + (live ? row.t : 0) * 2 * rot;
      row.next();
      const Floats fx(x);
      Floats h(g), u(0.f);
      float2 ss = make_float2(0.f, 0.f), ux = ss;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!kFew && !pl.there[k][0]) continue;
        if (pl.rotary[k]) turn<V, HALF>(h.f[k], turns, pl.rot_units, pl.unit[k]);
#pragma unroll
        for (int p = 0; p < kParts<HALF>; ++p) {
          mul(u.f[k][p], h.f[k][p], fw.f[k][p]);
          dot(ss, fx.f[k][p], fx.f[k][p]);
          dot(ux, u.f[k][p], fx.f[k][p]);
        }
      }
      const float2 sums = group_sum(make_float2(ss.x + ss.y, ux.x + ux.y), a.lanes);
      const float r = rsqrtf(sums.x * inv_dim + a.eps), along = -sums.y * inv_dim * r * r;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!kFew && !pl.there[k][0]) continue;
#pragma unroll
        for (int p = 0; p < kParts<HALF>; ++p) {
          float xr[V];
          mul(xr, fx.f[k][p], r);
          fma(dw.f[k][p], h.f[k][p], xr, dw.f[k][p]);
          fma(u.f[k][p], fx.f[k][p], along, u.f[k][p]);
          mul(u.f[k][p], u.f[k][p], r);
        }
      }
      if (live) u.template store<T, WIDE>(pl, out);
    }
  }
  if constexpr (Ring::kAsync) asm volatile("cp.async.wait_all;" ::: "memory");
  if (a.partials == nullptr) return;
  // the groups of a warp, then the warps, in a fixed order
  float* share = table + (tid >> 5) * 512;
  __syncthreads();                                 // the last angles have been read
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int p = 0; p < kParts<HALF>; ++p)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float d = dw.f[k][p][e];
        for (int m = a.lanes; m < 32; m <<= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
        if (pl.there[k][p] && (tid & 31) < a.lanes) share[pl.at[k] + p * pl.second[k] + e] = d;
      }
  __syncthreads();
  for (int c = tid; c < a.dim; c += kRopeThreads) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kRopeThreads / 32; ++i) sum += table[i * 512 + c];
    a.partials[(size_t)blockIdx.x * a.dim + c] = sum;
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

// a kernel's dynamic shared memory, allowed once on each device
int allow_smem(void (*kernel)(NormArgs), int bytes) {
  static std::mutex mu;
  static std::set<std::pair<int, void (*)(NormArgs)>> allowed;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return OSCAR_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  if (allowed.count({dev, kernel})) return OSCAR_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return OSCAR_ERR_CUDA;
  try {
    allowed.insert({dev, kernel});
  } catch (...) {                                  // no memory to note it in: it is done again
  }
  return OSCAR_OK;
}
int sm_count(int* sms) {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess
             ? OSCAR_OK
             : OSCAR_ERR_CUDA;
}

template <typename T, int V, bool HALF, bool WIDE, int K>
int launch_as(NormArgs a, bool grad, float* dqw, float* dkw, cudaStream_t st) {
  const int half = a.r.rot / 2, units = units_of<V, HALF>(a.dim, a.r.rot);
  a.lanes = 1;
  while (a.lanes < 32 && a.lanes * K < units) a.lanes *= 2;
  int sms = 0;
  if (int rc = sm_count(&sms); rc != OSCAR_OK) return rc;
  if (!grad) {
    a.tokens = std::max(1, std::min(std::min(kRopeTable / half, kRopeTokens), a.r.n / (4 * sms)));
    k_norm_rope<T, V, HALF, WIDE, K><<<(a.r.n - 1) / a.tokens + 1, kRopeThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
  }
  a.tokens = std::min(kGradTable / half, kGradTokens);
  // CTAs are shared between q and k by their heads; each of a token's angles counts as half of a lane's row (32,769 tokens
  // x 32 and 8 heads: 173 us; a quarter: 180, not at all: 202)
  const long long cost_q = 2ll * a.lanes * a.q.heads + half, cost_k = 2ll * a.lanes * a.k.heads + half;
  const int most_q = std::max(1, std::min(kGradCtas - 1, (int)(kGradCtas * cost_q / (cost_q + cost_k))));
  a.q_ctas = a.q.heads == 0 ? 0 : std::min(a.r.n, a.k.heads == 0 ? kGradCtas : most_q);
  const int k_ctas = a.k.heads == 0 ? 0 : std::min(a.r.n, a.q.heads == 0 ? kGradCtas : kGradCtas - most_q);
  const int ctas = a.q_ctas + k_ctas;
  constexpr int smem = 16 * kGradTable + Slots<T, V, HALF, WIDE, K>::kSmem;
  if (int rc = allow_smem(k_norm_rope_grad<T, V, HALF, WIDE, K>, smem); rc != OSCAR_OK) return rc;
  k_norm_rope_grad<T, V, HALF, WIDE, K><<<ctas, kRopeThreads, smem, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return OSCAR_ERR_CUDA;
  if (a.partials == nullptr) return OSCAR_OK;
  k_norm_rope_sum<<<dim3((a.dim + 31) / 32, 2), dim3(32, kSumRows), 0, st>>>(a.partials, a.dim, a.q_ctas, ctas, dqw, dkw);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

// bytes: the widest access (16, 8 or single elements) that every row, half and remainder starts on a multiple of
template <typename T, bool HALF>
int launch_layout(const NormArgs& a, int bytes, bool grad, float* dqw, float* dkw, cudaStream_t st) {
  constexpr int V16 = 16 / sizeof(T), V8 = 8 / sizeof(T), V1 = HALF ? 1 : 2;
  // 32 bytes a lane where 32 lanes hold a row so; K16, K8: units of a lane then (16 bytes a lane, pairs layout: 32,769 tokens
  // x 40 heads 152 us instead of 120)
  constexpr int K16 = 2 / kParts<HALF>, K8 = 4 / kParts<HALF>;
  if (bytes == 16) {
    if constexpr (sizeof(T) == 4)
      if (units_of<V16, HALF>(a.dim, a.r.rot) > 32 * K16) return launch_as<T, V16, HALF, true, 2 * K16>(a, grad, dqw, dkw, st);
    return launch_as<T, V16, HALF, true, K16>(a, grad, dqw, dkw, st);
  }
  if (bytes == 8) {
    if constexpr (sizeof(T) == 4)
      if (units_of<V8, HALF>(a.dim, a.r.rot) > 32 * K8) return launch_as<T, V8, HALF, true, 2 * K8>(a, grad, dqw, dkw, st);
    return launch_as<T, V8, HALF, true, K8>(a, grad, dqw, dkw, st);
  }
  return launch_as<T, V1, HALF, false, 8>(a, grad, dqw, dkw, st);
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
