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

#include "rope.cuh"

namespace oscar {
namespace {

constexpr int kGradCtas = 608;                     // partial sums of the weights' gradients, at most: four CTAs per SM of 152
constexpr int kSumRows = 8;                        // threads that share a channel's partial sums

struct NormArgs {
  RopeSide q, k;
  RopeSide gq, gk;                                 // gradient: dL/dy (in); q, k: x (in) and dL/dx (out)
  const void *qw, *kw;                             // weights of the rows' type, or null: ones
  Rotary r;
  int dim, tokens, lanes;                          // tokens per CTA (forward), lanes per row
  int q_ctas;                                      // gradient: the first CTAs walk q, the others k
  float eps;
  float* partials;                                 // gradient: [CTA][dim], or null
};

// What a lane holds of a row: K units.
template <typename T, int V, bool HALF, int K>
struct Place {
  int at[K];                                       // first channel of unit k
  bool there[K], rotary[K];
  __device__ __forceinline__ Place(int lane, int lanes, int dim, int rot) {
    const int rot_units = HALF ? rot / 2 / V : rot / V, units = rot_units + (dim - rot) / V;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int u = lane + k * lanes;
      there[k] = u < units;
      rotary[k] = u < rot_units;
      at[k] = rotary[k] ? u * V : rot + (u - rot_units) * V;
    }
  }
};

// A unit's values in float32: V channels and, for a rotary unit of the half layout, their V partners (else zeros).
template <int V, bool HALF> struct Values {
  float a[V], b[HALF ? V : 1];
};
template <typename T, int V, bool HALF, bool WIDE>
__device__ __forceinline__ Values<V, HALF> values_of(const Unit<T, V, V, HALF, WIDE>& x, bool rotary) {
  Values<V, HALF> f;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    f.a[e] = to_f(x.a.v[e]);
    if (HALF) f.b[e] = rotary ? to_f(x.b.v[e]) : 0.f;
  }
  return f;
}
// turned by the unit's angles (cs[0] belongs to its first pair)
template <int V, bool HALF>
__device__ __forceinline__ void turn(Values<V, HALF>& f, const float2* cs) {
  if constexpr (HALF) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float x = f.a[e], y = f.b[e];
      const float2 t = cs[e];
      f.a[e] = x * t.x - y * t.y;
      f.b[e] = y * t.x + x * t.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      const float x = f.a[2 * e], y = f.a[2 * e + 1];
      const float2 t = cs[e];
      f.a[2 * e] = x * t.x - y * t.y;
      f.a[2 * e + 1] = y * t.x + x * t.y;
    }
  }
}
template <typename T, int V, bool HALF, bool WIDE>
__device__ __forceinline__ void store(T* out, const Values<V, HALF>& f, int at, int half, bool rotary) {
  Unit<T, V, V, HALF, WIDE> x;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    x.a.v[e] = from_f<T>(f.a[e]);
    if (HALF) x.b.v[e] = from_f<T>(f.b[e]);
  }
  x.store(out, at, half, rotary);
}
template <typename T, int V, bool HALF, bool WIDE>
__device__ __forceinline__ Unit<T, V, V, HALF, WIDE> weights(const void* w, int at, int half, bool rotary) {
  Unit<T, V, V, HALF, WIDE> x;
  if (w != nullptr) {
    x.load(static_cast<const T*>(w), at, half, rotary);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) x.a.v[e] = x.b.v[e] = from_f<T>(1.f);
  }
  return x;
}
__device__ __forceinline__ float group_sum(float s, int lanes) {
  for (int m = 1; m < lanes; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  return s;
}

template <typename T, int V, bool HALF, bool WIDE, int K>
__global__ void __launch_bounds__(kRopeThreads, K == 1 ? 4 : 2) k_norm_rope(NormArgs a) {
  __shared__ float2 table[kRopeTable];
  __shared__ int pos_s[kRopeTokens * kRopeAxes];
  constexpr int kBatch = K == 1 ? 2 : 1;           // rows a group has in flight
  const int rot = a.r.rot, half = rot / 2, t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.r.n - t0), tid = threadIdx.x;
  const int lane = tid & (a.lanes - 1), group = tid / a.lanes, groups = kRopeThreads / a.lanes;
  const Place<T, V, HALF, K> p(lane, a.lanes, a.dim, rot);
  Unit<T, V, V, HALF, WIDE> wq[K], wk[K];
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (p.there[k]) {
      wq[k] = weights<T, V, HALF, WIDE>(a.qw, p.at[k], half, p.rotary[k]);
      wk[k] = weights<T, V, HALF, WIDE>(a.kw, p.at[k], half, p.rotary[k]);
    }
  load_positions(a.r, t0, nt, pos_s, tid, kRopeThreads);
  __syncthreads();
  load_turns(a.r, nt, pos_s, 1.f, table, tid, kRopeThreads);
  __syncthreads();
  const int heads = a.q.heads + a.k.heads, items = nt * heads;
  const float inv_dim = 1.f / (float)a.dim;
  // the same trips for every lane of a warp: the row's sum is a shuffle
  for (int i0 = 0; i0 < items; i0 += kBatch * groups) {
    Unit<T, V, V, HALF, WIDE> x[kBatch][K];
    T* out[kBatch];
    int tok[kBatch];
    bool isq[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * groups + group;       // (token, head)
      const int t = min(i, items - 1) / heads, h = min(i, items - 1) - t * heads;
      isq[b] = h < a.q.heads;
      const RopeSide& s = isq[b] ? a.q : a.k;
      const int hh = isq[b] ? h : h - a.q.heads;
      const T* in = static_cast<const T*>(s.in) + (t0 + t) * s.in_tok + hh * s.in_head;
      out[b] = static_cast<T*>(s.out) + (t0 + t) * s.out_tok + hh * s.out_head;
      tok[b] = t;
      if (i >= items || pos_s[t * kRopeAxes] < 0) out[b] = nullptr;       // a padded row is left as it is
      if (out[b] != nullptr)
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (p.there[k]) x[b][k].load(in, p.at[k], half, p.rotary[k]);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      float ss = 0.f;
      Values<V, HALF> f[K];
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (p.there[k] && out[b] != nullptr) {
          f[k] = values_of<T, V, HALF, WIDE>(x[b][k], p.rotary[k]);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            ss = fmaf(f[k].a[e], f[k].a[e], ss);
            if (HALF) ss = fmaf(f[k].b[e], f[k].b[e], ss);
          }
        }
      const float r = rsqrtf(group_sum(ss, a.lanes) * inv_dim + a.eps);
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (p.there[k] && out[b] != nullptr) {
          const Values<V, HALF> w = values_of<T, V, HALF, WIDE>(isq[b] ? wq[k] : wk[k], p.rotary[k]);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            f[k].a[e] *= r * w.a[e];
            if (HALF) f[k].b[e] *= r * w.b[e];
          }
          if (p.rotary[k]) turn<V, HALF>(f[k], table + tok[b] * half + (HALF ? p.at[k] : p.at[k] / 2));
          store<T, V, HALF, WIDE>(out[b], f[k], p.at[k], half, p.rotary[k]);
        }
    }
  }
}

template <typename T, int V, bool HALF, bool WIDE, int K>
__global__ void __launch_bounds__(kRopeThreads, K == 1 ? 3 : 1) k_norm_rope_grad(NormArgs a) {
  __shared__ float2 table[kRopeTable];
  __shared__ int pos_s[kRopeTokens * kRopeAxes];
  __shared__ float sums[kRopeThreads / 32][512];   // a warp's share of the weights' gradient
  const int rot = a.r.rot, half = rot / 2, tid = threadIdx.x;
  const int lane = tid & (a.lanes - 1), group = tid / a.lanes, groups = kRopeThreads / a.lanes;
  const bool isq = (int)blockIdx.x < a.q_ctas;
  const RopeSide s = isq ? a.q : a.k, sg = isq ? a.gq : a.gk;
  const int first = isq ? blockIdx.x : blockIdx.x - a.q_ctas, step = isq ? a.q_ctas : gridDim.x - a.q_ctas;
  const Place<T, V, HALF, K> p(lane, a.lanes, a.dim, rot);
  Unit<T, V, V, HALF, WIDE> w[K];
  Values<V, HALF> dw[K] = {};
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (p.there[k]) w[k] = weights<T, V, HALF, WIDE>(isq ? a.qw : a.kw, p.at[k], half, p.rotary[k]);
  const float inv_dim = 1.f / (float)a.dim;
  for (long long t0 = (long long)first * a.tokens; t0 < a.r.n; t0 += (long long)step * a.tokens) {
    const int nt = (int)min((long long)a.tokens, a.r.n - t0), items = nt * s.heads;
    __syncthreads();                               // the last tokens' angles have been read
    load_positions(a.r, (int)t0, nt, pos_s, tid, kRopeThreads);
    __syncthreads();
    load_turns(a.r, nt, pos_s, -1.f, table, tid, kRopeThreads);
    __syncthreads();
    for (int i0 = 0; i0 < items; i0 += groups) {
      const int i = i0 + group, t = min(i, items - 1) / s.heads, h = min(i, items - 1) - t * s.heads;
      const bool live = i < items && pos_s[t * kRopeAxes] >= 0;
      const T* in = static_cast<const T*>(s.in) + (t0 + t) * s.in_tok + h * s.in_head;
      const T* gin = static_cast<const T*>(sg.in) + (t0 + t) * sg.in_tok + h * sg.in_head;
      T* out = static_cast<T*>(s.out) + (t0 + t) * s.out_tok + h * s.out_head;
      Unit<T, V, V, HALF, WIDE> x[K], g[K];
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (p.there[k] && live) {
          x[k].load(in, p.at[k], half, p.rotary[k]);
          g[k].load(gin, p.at[k], half, p.rotary[k]);
        }
      float ss = 0.f, ux = 0.f;
      Values<V, HALF> fx[K], fh[K];
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (p.there[k] && live) {
          fx[k] = values_of<T, V, HALF, WIDE>(x[k], p.rotary[k]);
          fh[k] = values_of<T, V, HALF, WIDE>(g[k], p.rotary[k]);
          if (p.rotary[k]) turn<V, HALF>(fh[k], table + t * half + (HALF ? p.at[k] : p.at[k] / 2));
          const Values<V, HALF> fw = values_of<T, V, HALF, WIDE>(w[k], p.rotary[k]);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            ss = fmaf(fx[k].a[e], fx[k].a[e], ss);
            ux = fmaf(fh[k].a[e] * fw.a[e], fx[k].a[e], ux);
            if (HALF) {
              ss = fmaf(fx[k].b[e], fx[k].b[e], ss);
              ux = fmaf(fh[k].b[e] * fw.b[e], fx[k].b[e], ux);
            }
          }
        }
      const float r = rsqrtf(group_sum(ss, a.lanes) * inv_dim + a.eps);
      const float along = group_sum(ux, a.lanes) * inv_dim * r * r;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (p.there[k] && live) {
          const Values<V, HALF> fw = values_of<T, V, HALF, WIDE>(w[k], p.rotary[k]);
          Values<V, HALF> dx;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            dw[k].a[e] = fmaf(fh[k].a[e], fx[k].a[e] * r, dw[k].a[e]);
            dx.a[e] = r * (fh[k].a[e] * fw.a[e] - fx[k].a[e] * along);
            if (HALF) {
              dw[k].b[e] = fmaf(fh[k].b[e], fx[k].b[e] * r, dw[k].b[e]);
              dx.b[e] = r * (fh[k].b[e] * fw.b[e] - fx[k].b[e] * along);
            }
          }
          store<T, V, HALF, WIDE>(out, dx, p.at[k], half, p.rotary[k]);
        }
    }
  }
  if (a.partials == nullptr) return;
  // the groups of a warp, then the warps, in a fixed order
  const int warp = tid >> 5;
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
        sums[warp][p.at[k] + e] = da;
        if (HALF && p.rotary[k]) sums[warp][p.at[k] + half + e] = db;
      }
    }
  }
  __syncthreads();
  for (int c = tid; c < a.dim; c += kRopeThreads) {
    float s8 = 0.f;
#pragma unroll
    for (int i = 0; i < kRopeThreads / 32; ++i) s8 += sums[i][c];
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
  while (a.lanes < 32 && a.lanes < units) a.lanes *= 2;
  int sms = 0;
  if (int rc = sm_count(&sms); rc != OSCAR_OK) return rc;
  a.tokens = std::max(1, std::min(std::min(kRopeTable / half, kRopeTokens), a.r.n / (4 * sms)));
  if (!grad) {
    k_norm_rope<T, V, HALF, WIDE, K><<<(a.r.n - 1) / a.tokens + 1, kRopeThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
  }
  // CTAs are shared between q and k by their heads
  const int tiles = (a.r.n - 1) / a.tokens + 1, heads = a.q.heads + a.k.heads;
  const int most_q = std::max(1, std::min(kGradCtas - 1, (int)((long long)kGradCtas * a.q.heads / heads)));
  a.q_ctas = a.q.heads == 0 ? 0 : std::min(tiles, a.k.heads == 0 ? kGradCtas : most_q);
  const int k_ctas = a.k.heads == 0 ? 0 : std::min(tiles, a.q.heads == 0 ? kGradCtas : kGradCtas - most_q);
  const int ctas = a.q_ctas + k_ctas;
  k_norm_rope_grad<T, V, HALF, WIDE, K><<<ctas, kRopeThreads, 0, st>>>(a);
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
    if (units <= 32) return launch_as<T, V16, HALF, true, 1>(a, grad, dqw, dkw, st);
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
