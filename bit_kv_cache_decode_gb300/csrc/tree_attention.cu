// Attention of a tree of drafted tokens over the mixed cache (sm_103a: tcgen05.mma, TMEM accumulators).
//
// Query row (node i, head) of a request attends to all committed tokens, read where they are (INT2 history in
// the rotated basis, BF16 sink and recent rows), and to the drafted nodes of its mask word i:
//   logits  history: s (q R_K) . khat   BF16, drafted: s q . k,   one softmax, o = sum p v.
// The T gq query rows of a kv head are the M = 128 rows of a tensor-core tile, so a page is read and unpacked
// once for all of them.
//
// Grid (slot, kv head x row tile, request), one CTA per SM. A slot is a range of the request's history pages in
// tiles of two pages (128 tokens), or of its BF16 and draft pages in tiles of one (64 tokens). Per tile:
//  * S = Q K^T, A = the rows in TMEM (history: q R_K as fp16, rotated by this CTA at its start; else q as bf16),
//    B = the keys in shared memory: history keys dequantised to fp16 (zero + scale code, one rounding).
//  * row threads (thread = row = TMEM lane): running maximum, weights p = 2^(x - m), their sum in float32. The
//    maximum moves only when it grows by more than 2^8, so O is seldom rescaled; history weights are fp16 and
//    carry 2^7 more, so that weights down to 2^-31 of the row's largest still count.
//  * O += P V, A = P in TMEM, B = the values in shared memory, dequantised like the keys; BF16 tiles take P as two
//    bf16 parts, since their tokens often carry most of the weight.
// Values are rounded with their zero point in place: with scale * code alone, the rounding of the products and of
// the zero point's sum would no longer cancel where many tokens average out.
//
// The M128 N128 K16 MMA takes 89 cycles with A in TMEM whatever N up to 128 is (138 for N = 256, 108 with A in
// shared memory), so a 128-token tile is 16 MMAs, 1,424 cycles; everything else is arranged to fit beside them.
// TMEM is full: S of two tiles (2 x 128 columns), O (128), P (64), Q (64). Roles: warps 0-3 rows, 4-7 unpack
// keys, 8-11 unpack values (all double-buffered), 12 issues the MMAs in the order S(i+1), O(i), so that S of the
// next tile runs while the rows work on this one, 13 streams the pages through a ring of bulk copies.
// Every wait is bounded; a CTA whose wait expires flags OSCAR_STATUS_TIMEOUT and writes empty partials.
#include <algorithm>

#include "tcgen05.cuh"
#include "tma.cuh"
#include "tree.cuh"

namespace oscar {
namespace {

constexpr int kRowWarps = 4, kKWarp0 = 4, kVWarp0 = 8, kMmaWarp = 12, kLoadWarp = 13;
constexpr int kTreeThreads = 14 * 32;
constexpr int kRows = 128;                         // query rows of a CTA
constexpr int kTok = 2 * kP;                       // tokens of a history tile
constexpr int kStages = 4;                         // ring stages of one tile (two page blocks)
constexpr int kStageBytes = 2 * kBlockBytes;
constexpr int kOpBytes = kTok * kD * 2;            // a tile's unpacked keys or values: 32 KB
constexpr int kSbo = (kD / 8) * 128;               // K-major, no swizzle: 2,048 B between 8-row blocks
static_assert(kTok == kD, "keys (rows = tokens) and values (rows = channels) have one geometry");
constexpr int kSboV64 = (kP / 8) * 128 + 16;       // values of a BF16 tile: 64 tokens, padded against bank conflicts
constexpr int kOffK = 0, kOffV = kOffK + 2 * kOpBytes, kOffRing = kOffV + 2 * kOpBytes;
constexpr int kPids = 4096;                        // page ids of a slot kept in shared memory
constexpr int kOffPid = kOffRing + kStages * kStageBytes;
constexpr int kOffBar = kOffPid + kPids * 4;
// BF16 slots keep no page ids; the same bytes hold a bit set per tile of the value rows that are not finite
constexpr int kPoisonTiles = kPids / 2;
static_assert(kMaxTreeBf16Pages + kMaxDraft / kP <= kPoisonTiles, "a set for every BF16 and draft tile");
constexpr int kBFull = 0, kBEmpty = kBFull + kStages, kBKFull = kBEmpty + kStages, kBVFull = kBKFull + 2,
              kBSDone = kBVFull + 2, kBSFree = kBSDone + 2, kBODone = kBSFree + 2, kBPReady = kBODone + 2,
              kBImg = kBPReady + 1, kBQ = kBImg + 1, kBFinal = kBQ + 1, kNumBars = kBFinal + 1;
constexpr int kTreeSmem = kOffBar + kNumBars * 8 + 16 + 1024;   // + TMEM address, flag, alignment slack
constexpr uint32_t kColS = 0, kColO = 256, kColP = 384, kColQ = 448, kTmemCols = 512;
constexpr uint32_t kIdescF16 = idesc_f16(128, 128);
constexpr uint32_t kBf16Bits = (1u << 7) | (1u << 10);              // A and B bf16
constexpr uint32_t kIdescBf16 = idesc_f16(128, 128) | kBf16Bits, kIdescBf16N64 = idesc_f16(128, 64) | kBf16Bits;
constexpr float kLazy = 8.f;                       // log2 growth of a maximum that forces a rescale
constexpr float kBias = 7.f;                       // log2 of the factor of history weights: 2^(8 + 7) fits fp16
constexpr uint32_t kMagic = 0x64006400u;           // fp16 1024.0 in both halves

// K-major operand with the 128-byte swizzle (the rotation images)
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}
// the code at position p (0 .. 3) of both 16-bit halves as exact fp16 values: (1024 + c 4^p) 4^-p - 1024 4^-p
__device__ __forceinline__ uint32_t codes_at(uint32_t x, int p) {
  return hfma2_u(and_or(x, 0x00030003u << (2 * p), kMagic), 0x3C003C00u - (uint32_t)(p * 0x08000800u),
                 0xE400E400u - (uint32_t)(p * 0x08000800u));
}
// codebook format: the level k_c / 256 of the code at position p of both halves (lut: the codebook's bytes)
__device__ __forceinline__ uint32_t levels_at(uint32_t x, int p, uint32_t lut) {
  const uint32_t y = (x >> (2 * p)) & 0x00030003u;
  const uint32_t v = __byte_perm(lut, 0x64646464u, ((y | (y >> 8)) & 0x0303u) | 0x4040u);   // 1024 + k_c
  return hfma2_u(v, 0x1C001C00u, 0xC400C400u);
}
template <int FMT>
__device__ __forceinline__ uint32_t value_at(uint32_t x, int p, uint32_t lut, uint32_t s2, uint32_t z2) {
  return hfma2_u(FMT == kFmtCB ? levels_at(x, p, lut) : codes_at(x, p), s2, z2);
}
// (scale, zero) of the two groups of a row as fp16 pairs {s0, z0}, {s1, z1}
template <int FMT>
__device__ __forceinline__ uint2 scale_zero(const uint8_t* blk, int kind, int row, const float* mc) {
  if (FMT == kFmtU8) {
    const uint32_t m = *reinterpret_cast<const uint32_t*>(blk + (kind ? kVMetaOffU8 : kKMetaOff) + 4 * row);
    const float* c = mc + 8 * kind;
    const float2 a = u8_scale_zero(m & 0xffu, (m >> 8) & 0xffu, c[0], c[1], c[2]);
    const float2 b = u8_scale_zero((m >> 16) & 0xffu, m >> 24, c[4], c[5], c[6]);
    return make_uint2(pack_f16x2(a.x, a.y), pack_f16x2(b.x, b.y));
  }
  uint2 m = *reinterpret_cast<const uint2*>(blk + (kind ? kVMetaOff : kKMetaOff) + 8 * row);
  if (FMT == kFmtCB) {                             // range 256 / 255: the levels are k_c / 256
    const float f = 256.f / 255.f;
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&m.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&m.y));
    m = make_uint2(pack_f16x2(a.x * f, a.y), pack_f16x2(b.x * f, b.y));
  }
  return m;
}
__device__ __forceinline__ uint32_t lut_of(const LayerView& lv, int h, int kind) {
  const float* c = cb_consts(lv, h, kind);
  uint32_t lut = 0;
  for (int i = 0; i < 4; ++i) lut |= (uint32_t)c[i] << (8 * i);
  return lut;
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// What the roles share.
struct Ctx {
  uint8_t* smem;
  uint32_t bar0, tmem;
  volatile int* failed;
  __device__ uint32_t bar(int k) const { return bar0 + 8u * (uint32_t)k; }
  // one wait of a whole warp; false ends its work
  __device__ bool wait(int k, int phase) const {
    const bool ok = *failed == 0 && mbar_wait(bar(k), (uint32_t)phase & 1u);
    return __all_sync(0xffffffffu, ok);
  }
  __device__ void arrive(int k) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar(k));
  }
};

// O of this warp's rows times al
__device__ __forceinline__ void rescale_o(uint32_t trow, float al) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    float o[32];
    tmem_ld32(trow + kColO + 32 * c, o);
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] *= al;
    tmem_st32(trow + kColO + 32 * c, o);
  }
}

// ---- row threads, history tiles ------------------------------------------------------------------------
// tokens(k): valid tokens of page k of the slot
template <typename Tokens>
__device__ __forceinline__ bool rows_history(const Ctx& c, int n, float F, Tokens tokens, float& m, float& lsum) {
  const uint32_t trow = c.tmem + ((uint32_t)(32 * (threadIdx.x >> 5)) << 16);
  float2 l2 = make_float2(0.f, 0.f);
  const float2 F2 = make_float2(F, F);
  for (int i = 0; i < n; ++i) {
    const int b = i & 1;
    if (!c.wait(kBSDone + b, i >> 1)) return false;
    tc_fence_after();
    const int nv[2] = {tokens(2 * i), tokens(2 * i + 1)};
    const bool whole = nv[0] == kP && nv[1] == kP;
    float mx = -INFINITY;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float s[32];
      tmem_ld32(trow + kColS + 128 * b + 32 * q, s);
      if (whole) {
#pragma unroll
        for (int e = 0; e < 32; ++e) mx = fmaxf(mx, s[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) mx = fmaxf(mx, 32 * (q & 1) + e < nv[q >> 1] ? s[e] : -INFINITY);
      }
    }
    float al = 1.f;
    const bool grow = (mx - m) * F > kLazy;
    if (grow) {
      al = m == -INFINITY ? 0.f : exp2f((m - mx) * F);
      m = mx;
    }
    bool free_o = i == 0;                          // O(i - 1) is complete
    if (__any_sync(0xffffffffu, grow)) {
      l2 = __fmul2_rn(l2, make_float2(al, al));
      if (i > 0) {
        if (!c.wait(kBODone + ((i - 1) & 1), (i - 1) >> 1)) return false;
        tc_fence_after();
        rescale_o(trow, al);
        free_o = true;
      }
    }
    const float mF = m == -INFINITY ? 0.f : fmaf(m, F, -kBias);
    const float2 nm2 = make_float2(-mF, -mF);
#pragma unroll
    for (int pi = 0; pi < 2; ++pi) {
      float s[2][32];
      tmem_ld32x2(trow + kColS + 128 * b + 64 * pi, trow + kColS + 128 * b + 64 * pi + 32, s[0], s[1]);
      if (pi == 1) {
        tc_fence_before();
        c.arrive(kBSFree + b);
      }
      if (!whole) {
#pragma unroll
        for (int e = 0; e < kP; ++e)
          if (e >= nv[pi]) s[e >> 5][e & 31] = -INFINITY;
      }
      uint32_t r[32];                              // column 8w + p: the weights of tokens t, t + 1
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const int t = 16 * (p >> 1) + 2 * w + 8 * (p & 1);
          const float2 x = __ffma2_rn(make_float2(s[t >> 5][t & 31], s[t >> 5][(t & 31) + 1]), F2, nm2);
          const float2 v = make_float2(fast_exp2(x.x), fast_exp2(x.y));
          l2 = __fadd2_rn(l2, v);
          r[8 * w + p] = pack_f16x2(v.x, v.y);
        }
      if (!free_o) {
        if (!c.wait(kBODone + ((i - 1) & 1), (i - 1) >> 1)) return false;
        tc_fence_after();
        free_o = true;
      }
      tmem_st32u(trow + kColP + 32 * pi, r);
    }
    tmem_wait_st();
    tc_fence_before();
    c.arrive(kBPReady);
  }
  lsum = l2.x + l2.y;
  return true;
}

// ---- row threads, BF16 and draft tiles -----------------------------------------------------------------
// bits(i): the tokens of tile i that this row sees
template <typename Bits>
__device__ __forceinline__ bool rows_bf16(const Ctx& c, int n, float F, Bits bits, float& m, float& lsum) {
  const uint32_t trow = c.tmem + ((uint32_t)(32 * (threadIdx.x >> 5)) << 16);
  const volatile unsigned long long* poison = reinterpret_cast<const unsigned long long*>(c.smem + kOffPid);
  float l = 0.f;
  for (int i = 0; i < n; ++i) {
    const int b = i & 1;
    const unsigned long long see = bits(i);
    if (!c.wait(kBSDone + b, i >> 1) || !c.wait(kBVFull + b, i >> 1)) return false;
    tc_fence_after();
    if (see & poison[i]) l = NAN;                  // a NaN or infinity among the values the row sees
    float s[2][32];
    tmem_ld32x2(trow + kColS + 128 * b, trow + kColS + 128 * b + 32, s[0], s[1]);
    tc_fence_before();
    c.arrive(kBSFree + b);
    float mx = -INFINITY;
#pragma unroll
    for (int e = 0; e < kP; ++e) {
      if (!(see >> e & 1)) s[e >> 5][e & 31] = -INFINITY;
      mx = fmaxf(mx, s[e >> 5][e & 31]);
    }
    float al = 1.f;
    const bool grow = (mx - m) * F > kLazy;
    if (grow) {
      al = m == -INFINITY ? 0.f : exp2f((m - mx) * F);
      m = mx;
    }
    if (i > 0) {
      if (!c.wait(kBODone + ((i - 1) & 1), (i - 1) >> 1)) return false;
      tc_fence_after();
      if (__any_sync(0xffffffffu, grow)) rescale_o(trow, al);
    }
    l *= al;
    const float mF = m == -INFINITY ? 0.f : m * F;
    uint32_t hi[32], lo[32];                       // p = hi + lo, pairs of tokens 2j, 2j + 1
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float x = fast_exp2(fmaf(s[j >> 4][2 * (j & 15)], F, -mF)), y = fast_exp2(fmaf(s[j >> 4][2 * (j & 15) + 1], F, -mF));
      l += x + y;
      hi[j] = pack_bf16x2(x, y);
      lo[j] = pack_bf16x2(x - __uint_as_float(hi[j] << 16), y - __uint_as_float(hi[j] & 0xffff0000u));
    }
    tmem_st32u(trow + kColP, hi);
    tmem_st32u(trow + kColP + 32, lo);
    tmem_wait_st();
    tc_fence_before();
    c.arrive(kBPReady);
  }
  lsum = l;
  return true;
}

// ---- key warps, history tiles --------------------------------------------------------------------------
// Key row t of the tile: the 16-channel block u is one word of codes; k positions 2q, 2q + 1 of the block are
// channels 16u + q, 16u + 8 + q (the rows' fragments use the same order).
template <int FMT>
__device__ __forceinline__ bool keys_history(const Ctx& c, const LayerView& lv, int h, int n) {
  const int lane = threadIdx.x & 31, kw = (threadIdx.x >> 5) - kKWarp0;
  const float* mc = meta_consts(lv, h, 0);
  const uint32_t lut = FMT == kFmtCB ? lut_of(lv, h, OSCAR_KIND_K) : 0u;
  for (int i = 0; i < n; ++i) {
    const int b = i & 1, st = i % kStages;
    if (!c.wait(kBFull + st, i / kStages)) return false;
    if (i >= 2 && !c.wait(kBSDone + b, (i - 2) >> 1)) return false;
    uint8_t* dst = c.smem + kOffK + b * kOpBytes;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = (lane & 7) + 8 * (kw + 4 * k), row = t & 63;
      const uint8_t* blk = c.smem + kOffRing + st * kStageBytes + (t >> 6) * kBlockBytes;
      const uint2 sz = scale_zero<FMT>(blk, 0, row, mc);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int u = (lane >> 3) + 4 * g;
        const uint32_t m = g ? sz.y : sz.x, s2 = __byte_perm(m, m, 0x1010), z2 = __byte_perm(m, m, 0x3232);
        const uint32_t x = *reinterpret_cast<const uint32_t*>(blk + kKCodesOff + 32 * row + 4 * u), y = x >> 8;
        uint8_t* d = dst + (t >> 3) * kSbo + (2 * u) * 128 + (t & 7) * 16;
        *reinterpret_cast<uint4*>(d) = make_uint4(value_at<FMT>(x, 0, lut, s2, z2), value_at<FMT>(x, 1, lut, s2, z2),
                                                  value_at<FMT>(x, 2, lut, s2, z2), value_at<FMT>(x, 3, lut, s2, z2));
        *reinterpret_cast<uint4*>(d + 128) = make_uint4(value_at<FMT>(y, 0, lut, s2, z2), value_at<FMT>(y, 1, lut, s2, z2),
                                                        value_at<FMT>(y, 2, lut, s2, z2), value_at<FMT>(y, 3, lut, s2, z2));
      }
    }
    fence_async();
    c.arrive(kBKFull + b);
    if (lane == 0) mbar_arrive(c.bar(kBEmpty + st));
  }
  return true;
}

// ---- value warps, history tiles ------------------------------------------------------------------------
// Value channel c: word w of its codes holds tokens 16 (p >> 1) + 2w + 8 (p & 1) + e at k positions 16w + 2p + e of
// the page (the order of the weights' columns). Tokens past the end get scale and zero 0: the block's bytes there
// may be anything, and 0 times a NaN would reach O.
template <int FMT, typename Tokens>
__device__ __forceinline__ bool values_history(const Ctx& c, const LayerView& lv, int h, int n, Tokens tokens) {
  const int lane = threadIdx.x & 31, vw = (threadIdx.x >> 5) - kVWarp0, w = lane >> 3, cl = lane & 7;
  const float* mc = meta_consts(lv, h, 0);
  const uint32_t lut = FMT == kFmtCB ? lut_of(lv, h, OSCAR_KIND_V) : 0u;
  for (int i = 0; i < n; ++i) {
    const int b = i & 1, st = i % kStages;
    if (!c.wait(kBFull + st, i / kStages)) return false;
    if (i >= 2 && !c.wait(kBODone + b, (i - 2) >> 1)) return false;
    uint8_t* dst = c.smem + kOffV + b * kOpBytes;
#pragma unroll
    for (int pi = 0; pi < 2; ++pi) {
      const uint8_t* blk = c.smem + kOffRing + st * kStageBytes + pi * kBlockBytes;
      const int nv = tokens(2 * i + pi);
      uint32_t s2[2][8], z2[2][8];
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const int t = 16 * (p >> 1) + 2 * w + 8 * (p & 1);
        uint2 a, d;
        if (FMT == kFmtU8) {
          a = scale_zero<FMT>(blk, 1, t, mc);
          d = scale_zero<FMT>(blk, 1, t + 1, mc);
        } else if (FMT == kFmtCB) {
          a = scale_zero<FMT>(blk, 1, t, mc);
          d = scale_zero<FMT>(blk, 1, t + 1, mc);
        } else {
          const uint4 m = *reinterpret_cast<const uint4*>(blk + kVMetaOff + 8 * t);
          a = make_uint2(m.x, m.y);
          d = make_uint2(m.z, m.w);
        }
        if (t >= nv) a = make_uint2(0u, 0u);
        if (t + 1 >= nv) d = make_uint2(0u, 0u);
        s2[0][p] = __byte_perm(a.x, d.x, 0x5410);
        z2[0][p] = __byte_perm(a.x, d.x, 0x7632);
        s2[1][p] = __byte_perm(a.y, d.y, 0x5410);
        z2[1][p] = __byte_perm(a.y, d.y, 0x7632);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int ch = cl + 8 * (vw + 4 * j), g = j >> 1;
        const uint32_t x = *reinterpret_cast<const uint32_t*>(blk + v_chan_off(ch) + 4 * w), y = x >> 8;
        uint8_t* d = dst + (ch >> 3) * kSbo + (8 * pi + 2 * w) * 128 + (ch & 7) * 16;
        *reinterpret_cast<uint4*>(d) =
            make_uint4(value_at<FMT>(x, 0, lut, s2[g][0], z2[g][0]), value_at<FMT>(x, 1, lut, s2[g][1], z2[g][1]),
                       value_at<FMT>(x, 2, lut, s2[g][2], z2[g][2]), value_at<FMT>(x, 3, lut, s2[g][3], z2[g][3]));
        *reinterpret_cast<uint4*>(d + 128) =
            make_uint4(value_at<FMT>(y, 0, lut, s2[g][4], z2[g][4]), value_at<FMT>(y, 1, lut, s2[g][5], z2[g][5]),
                       value_at<FMT>(y, 2, lut, s2[g][6], z2[g][6]), value_at<FMT>(y, 3, lut, s2[g][7], z2[g][7]));
      }
    }
    fence_async();
    c.arrive(kBVFull + b);
    if (lane == 0) mbar_arrive(c.bar(kBEmpty + st));
  }
  return true;
}

// A BF16 or draft tile: rows 0 .. rows - 1 of K and V at k0, v0, `step` elements apart.
struct Near {
  const __nv_bfloat16 *k, *v;
  size_t step;
  int rows;
  bool draft;
};

// ---- key warps, BF16 tiles (natural channel order) -----------------------------------------------------
template <typename Page>
__device__ __forceinline__ bool keys_bf16(const Ctx& c, int* status, int n, Page page) {
  const int lane = threadIdx.x & 31, kw = (threadIdx.x >> 5) - kKWarp0;
  for (int i = 0; i < n; ++i) {
    const int b = i & 1;
    const Near p = page(i);
    uint4 x[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = (lane & 7) + 8 * (kw + 4 * k), ck = (lane >> 3) + 4 * j;
        x[k][j] = t < p.rows ? *reinterpret_cast<const uint4*>(p.k + t * p.step + 8 * ck) : make_uint4(0u, 0u, 0u, 0u);
        if (p.draft && (bf16x2_nonfinite(x[k][j].x) || bf16x2_nonfinite(x[k][j].y) || bf16x2_nonfinite(x[k][j].z) ||
                        bf16x2_nonfinite(x[k][j].w)))
          flag(status, OSCAR_STATUS_NONFINITE);
      }
    if (i >= 2 && !c.wait(kBSDone + b, (i - 2) >> 1)) return false;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = (lane & 7) + 8 * (kw + 4 * k), ck = (lane >> 3) + 4 * j;
        *reinterpret_cast<uint4*>(c.smem + kOffK + b * kOpBytes + (t >> 3) * kSbo + ck * 128 + (t & 7) * 16) = x[k][j];
      }
    fence_async();
    c.arrive(kBKFull + b);
  }
  return true;
}

// ---- value warps, BF16 tiles: transposed, non-finite values replaced by 0 and their rows noted ----------
template <typename Page>
__device__ __forceinline__ bool values_bf16(const Ctx& c, int* status, int n, Page page) {
  const int lane = threadIdx.x & 31, vw = (threadIdx.x >> 5) - kVWarp0;
  unsigned long long* poison = reinterpret_cast<unsigned long long*>(c.smem + kOffPid);
  for (int i = 0; i < n; ++i) {
    const int b = i & 1;
    const Near p = page(i);
    uint32_t x[4][8];                              // [octet, channel half][token]: channels 2 cp, 2 cp + 1
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = 8 * (vw + 4 * (k >> 1)) + e, cp = lane + 32 * (k & 1);
        x[k][e] = t < p.rows ? *reinterpret_cast<const uint32_t*>(p.v + t * p.step + 2 * cp) : 0u;
      }
    if (i >= 2 && !c.wait(kBODone + b, (i - 2) >> 1)) return false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (bf16x2_nonfinite(x[k][e])) {
          if (p.draft) flag(status, OSCAR_STATUS_NONFINITE);
          atomicOr(poison + i, 1ull << (8 * (vw + 4 * (k >> 1)) + e));
          x[k][e] = 0u;
        }
      const int o = vw + 4 * (k >> 1), ch = 2 * (lane + 32 * (k & 1));
      uint8_t* d = c.smem + kOffV + b * kOpBytes + (ch >> 3) * kSboV64 + o * 128 + (ch & 7) * 16;
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo[e] = __byte_perm(x[k][2 * e], x[k][2 * e + 1], 0x5410);
        hi[e] = __byte_perm(x[k][2 * e], x[k][2 * e + 1], 0x7632);
      }
      *reinterpret_cast<uint4*>(d) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      *reinterpret_cast<uint4*>(d + 16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
    fence_async();
    c.arrive(kBVFull + b);
  }
  return true;
}

template <int FMT>
__global__ void __launch_bounds__(kTreeThreads, 1) k_tree_attention(LayerView lv, TreeArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const int slot = blockIdx.x, h = blockIdx.y % lv.hkv, qt = blockIdx.y / lv.hkv, b = blockIdx.z;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int gq = lv.hq / lv.hkv;
  const bool hist = slot < a.nsplit;
  pdl_wait();
  pdl_launch_dependents();
  const int nodes = live_nodes(a, b);
  if (a.n_draft != nullptr && a.n_draft[b] != nodes && tid == 0 && slot == 0) flag(lv.status, OSCAR_STATUS_BAD_TREE);
  const int live = min(kRows, nodes * gq - qt * kRows);   // this tile's query rows
  if (live <= 0) return;

  Ctx c;
  c.smem = smem;
  c.bar0 = smem_addr(smem + kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + kNumBars * 8);
  c.failed = reinterpret_cast<volatile int*>(smem + kOffBar + kNumBars * 8 + 4);
  int* pids = reinterpret_cast<int*>(smem + kOffPid);   // BF16 slots: see kPoisonTiles

  // ---- the slot's tokens -----------------------------------------------------------------------------------
  int L = a.seq_lens[b];
  if (L < 0) {
    if (tid == 0 && slot == 0) flag(lv.status, OSCAR_STATUS_BAD_SEQLEN);
    L = 0;
  }
  int Lh = max(0, L - lv.sink - lv.recent), np = (Lh + kP - 1) / kP;
  if (np > a.max_hist_pages) {
    if (tid == 0 && slot == 0) flag(lv.status, OSCAR_STATUS_BAD_SEQLEN);
    np = a.max_hist_pages;
    Lh = np * kP;
  }
  const int nbf = (lv.sink + lv.recent) / kP, near_pages = nbf + (nodes + kP - 1) / kP;
  int p0, cnt;                                     // first page and number of pages of the slot
  if (hist) {
    p0 = (int)((long long)slot * np / a.nsplit);
    cnt = (int)((long long)(slot + 1) * np / a.nsplit) - p0;
  } else {
    p0 = (slot - a.nsplit) * near_pages / a.nb;
    cnt = (slot - a.nsplit + 1) * near_pages / a.nb - p0;
  }
  const int n = hist ? (cnt + 1) / 2 : cnt;        // tiles
  const int* pt = a.hist_pt + (size_t)b * a.max_hist_pages + p0;
  auto checked = [&](int id) { return id >= 0 && id < lv.n_int2 ? id : -1; };
  auto page_id = [&](int k) { return k < kPids ? pids[k] : checked(__ldg(pt + k)); };
  auto tokens = [&](int k) { return k < cnt && page_id(k) >= 0 ? min(kP, Lh - (p0 + k) * kP) : 0; };

  const int active = (live + 31) / 32;             // row warps with rows
  if (w == kMmaWarp) {
    if (lane == 0) {
      for (int s = 0; s < kStages; ++s) {
        mbar_init_n(c.bar(kBFull + s), 1);
        mbar_init_n(c.bar(kBEmpty + s), 8);
      }
      for (int j = 0; j < 2; ++j) {
        mbar_init_n(c.bar(kBKFull + j), 4);
        mbar_init_n(c.bar(kBVFull + j), 4);
        mbar_init_n(c.bar(kBSDone + j), 1);
        mbar_init_n(c.bar(kBSFree + j), active);
        mbar_init_n(c.bar(kBODone + j), 1);
      }
      mbar_init_n(c.bar(kBPReady), active);
      mbar_init_n(c.bar(kBImg), 1);
      mbar_init_n(c.bar(kBQ), 1);
      mbar_init_n(c.bar(kBFinal), 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      *c.failed = 0;
    }
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (hist && w >= kKWarp0) {
    // page ids, those out of range as -1
    const int step = kTreeThreads - 32 * (kKWarp0 + 1);          // the threads of warps 4 .. 11 and 13
    const int at = w == kLoadWarp ? 8 * 32 + lane : tid - 32 * kKWarp0;
    for (int k = at; k < cnt && k < kPids; k += step) {
      const int id = checked(__ldg(pt + k));
      if (id < 0) flag(lv.status, OSCAR_STATUS_BAD_PAGE);
      pids[k] = id;
    }
  } else if (w >= kKWarp0 && w < kMmaWarp) {
    for (int k = tid - 32 * kKWarp0; k < 2 * n; k += 32 * 8) pids[k] = 0;   // the tiles' sets of non-finite rows
  }
  // ---- the rows: history tiles stage q for the rotation, BF16 tiles keep it -------------------------------
  const int row = tid, Q = qt * kRows + row, node = Q / gq, hq = h * gq + Q % gq;   // row threads
  uint4 q4[16];
  if (w < kRowWarps && n > 0) {
    const uint4* src = reinterpret_cast<const uint4*>(a.q + (((size_t)b * a.T + node) * lv.hq + hq) * kD);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      q4[j] = row < live ? src[j] : make_uint4(0u, 0u, 0u, 0u);
      if (bf16x2_nonfinite(q4[j].x) || bf16x2_nonfinite(q4[j].y) || bf16x2_nonfinite(q4[j].z) || bf16x2_nonfinite(q4[j].w))
        flag(lv.status, OSCAR_STATUS_NONFINITE);
    }
    if (hist) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        *reinterpret_cast<uint4*>(smem + kOffV + (row >> 3) * kSbo + j * 128 + (row & 7) * 16) = q4[j];
      fence_async();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  c.tmem = *tmem_slot;

  auto issue_tile = [&](int i) {                   // tile i into ring stage i % kStages (one thread)
    const int st = i % kStages;
    int id[2];
    uint32_t bytes = 0;
    for (int j = 0; j < 2; ++j) {
      id[j] = 2 * i + j < cnt ? page_id(2 * i + j) : -1;
      if (id[j] >= 0) bytes += (uint32_t)lv.blk_bytes;
    }
    mbar_expect_tx(c.bar(kBFull + st), bytes);     // also with no page: the phase completes
    const uint64_t pol = l2_evict_first();
    for (int j = 0; j < 2; ++j)
      if (id[j] >= 0)
        bulk_copy_hint(smem_addr(smem + kOffRing + st * kStageBytes + j * kBlockBytes), int2_block(lv, id[j], h),
                       (uint32_t)lv.blk_bytes, c.bar(kBFull + st), pol);
  };

  // ---- the rows' A operand in TMEM -------------------------------------------------------------------------
  float F = a.scale_log2;
  bool ok = true;
  if (n > 0 && hist) {
    if (w == kLoadWarp) {
      if (lane == 0) {
        const uint8_t* img = reinterpret_cast<const uint8_t*>(lv.params + (size_t)h * kParamFloats + kRKImgOff);
        mbar_expect_tx(c.bar(kBImg), 2 * kOpBytes);
        for (int p = 0; p < 2; ++p)                // R = b1 + b2 to about 17 bits
          bulk_copy_hint(smem_addr(smem + kOffK + p * kOpBytes), img + p * kOpBytes, kOpBytes, c.bar(kBImg), l2_evict_last());
        for (int i = 0; i < min(n, kStages); ++i) issue_tile(i);
      }
      __syncwarp();
    } else if (w == kMmaWarp) {
      ok = c.wait(kBImg, 0);
      if (ok && lane == 0) {
        tc_fence_after();
        const uint32_t a0 = smem_addr(smem + kOffV), b0 = smem_addr(smem + kOffK);
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma(c.tmem + kColS, umma_desc(a0 + kk * 256, 128, kSbo),
                 desc_sw128(b0 + p * kOpBytes + (kk >> 2) * (kOpBytes / 2) + (kk & 3) * 32), kIdescBf16, (p | kk) != 0);
        umma_commit(c.bar(kBQ));
      }
      __syncwarp();
    } else if (w < kRowWarps) {
      ok = c.wait(kBQ, 0);
      if (ok) {
        tc_fence_after();
        const uint32_t trow = c.tmem + ((uint32_t)(32 * w) << 16);
        float y[32], mx = 0.f;
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          tmem_ld32(trow + kColS + 32 * k, y);
#pragma unroll
          for (int e = 0; e < 32; ++e) mx = fmaxf(mx, fabsf(y[e]));
        }
        int e2 = 0;                                // 2^sigma brings the largest channel near 2^10
        if (mx > 0.f && mx < INFINITY) frexpf(mx, &e2);
        const int sigma = min(max(10 - e2, -60), 60);
        const float sc = exp2f((float)sigma);
        F *= exp2f((float)-sigma);
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          tmem_ld32(trow + kColS + 32 * k, y);
          uint32_t r[16];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) r[8 * u + j] = pack_f16x2(y[16 * u + j] * sc, y[16 * u + 8 + j] * sc);
          tmem_st16(trow + kColQ + 16 * k, r);
        }
        tmem_wait_st();
      }
    }
  } else if (n > 0 && w < kRowWarps) {
    const uint32_t trow = c.tmem + ((uint32_t)(32 * w) << 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t r[16] = {q4[4 * k].x, q4[4 * k].y, q4[4 * k].z, q4[4 * k].w, q4[4 * k + 1].x, q4[4 * k + 1].y,
                              q4[4 * k + 1].z, q4[4 * k + 1].w, q4[4 * k + 2].x, q4[4 * k + 2].y, q4[4 * k + 2].z,
                              q4[4 * k + 2].w, q4[4 * k + 3].x, q4[4 * k + 3].y, q4[4 * k + 3].z, q4[4 * k + 3].w};
      tmem_st16(trow + kColQ + 16 * k, r);
    }
    tmem_wait_st();
  }
  if (!ok) *c.failed = 1;
  tc_fence_before();
  __syncthreads();                                 // Q is in; the rotation's operands may be overwritten
  tc_fence_after();

  auto near = [&](int i) {
    const int u = p0 + i;
    Near r = {nullptr, nullptr, (size_t)kD, 0, u >= nbf};
    if (u >= nbf) {
      const size_t at = (((size_t)b * a.T + (u - nbf) * kP) * lv.hkv + h) * kD;
      r.k = a.kd + at;
      r.v = a.vd + at;
      r.step = (size_t)lv.hkv * kD;
      r.rows = min(kP, nodes - (u - nbf) * kP);
      return r;
    }
    const int rows = u < lv.sink / kP ? min(L, lv.sink) - u * kP : min(max(L - lv.sink, 0), lv.recent) - (u - lv.sink / kP) * kP;
    if (rows <= 0) return r;
    const int id = a.bf16_pt[(size_t)b * nbf + u];
    if (id < 0 || id >= lv.n_bf16) {
      if (lane == 0) flag(lv.status, OSCAR_STATUS_BAD_PAGE);
      return r;
    }
    r.k = bf16_row(lv, id, h, 0, 0);
    r.v = bf16_row(lv, id, h, 1, 0);
    r.rows = min(kP, rows);
    return r;
  };

  float m = -INFINITY, lsum = 0.f;
  ok = *c.failed == 0;
  if (ok) {
    if (w < kRowWarps) {
      if (w < active) {
        if (hist) {
          ok = rows_history(c, n, F, tokens, m, lsum);
        } else {
          auto bits = [&](int i) -> unsigned long long {
            const Near p = near(i);
            unsigned long long see = p.rows >= kP ? ~0ull : (1ull << p.rows) - 1ull;
            if (p.draft) see &= row < live ? a.mask[((size_t)b * a.T + node) * a.W + (p0 + i - nbf)] : 0ull;
            return see;
          };
          ok = rows_bf16(c, n, F, bits, m, lsum);
        }
        if (ok && n > 0) ok = c.wait(kBODone + ((n - 1) & 1), (n - 1) >> 1);
      }
    } else if (w < kVWarp0) {
      ok = hist ? keys_history<FMT>(c, lv, h, n) : keys_bf16(c, lv.status, n, near);
    } else if (w < kMmaWarp) {
      ok = hist ? values_history<FMT>(c, lv, h, n, tokens) : values_bf16(c, lv.status, n, near);
    } else if (w == kLoadWarp) {
      if (hist)
        for (int i = kStages; i < n && ok; ++i) {
          ok = c.wait(kBEmpty + i % kStages, i / kStages - 1);
          if (ok && lane == 0) issue_tile(i);
          __syncwarp();
        }
    } else {
      // ---- the MMAs: S(0), then S(i + 1) and O(i) ----
      const uint32_t k0 = smem_addr(smem + kOffK), v0 = smem_addr(smem + kOffV);
      auto issue_s = [&](int i) {
        const uint32_t kb = k0 + (i & 1) * kOpBytes, d = c.tmem + kColS + 128 * (i & 1);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_ta(d, c.tmem + kColQ + 8 * kk, umma_desc(kb + kk * 256, 128, kSbo), hist ? kIdescF16 : kIdescBf16N64, kk > 0);
        umma_commit(c.bar(kBSDone + (i & 1)));
      };
      auto issue_o = [&](int i) {
        const uint32_t vb = v0 + (i & 1) * kOpBytes;
        if (hist) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ta(c.tmem + kColO, c.tmem + kColP + 8 * kk, umma_desc(vb + kk * 256, 128, kSbo), kIdescF16, (i | kk) != 0);
        } else {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)           // high parts, then low parts
            umma_ta(c.tmem + kColO, c.tmem + kColP + 8 * kk, umma_desc(vb + (kk & 3) * 256, 128, kSboV64), kIdescBf16,
                    (i | kk) != 0);
        }
        umma_commit(c.bar(kBODone + (i & 1)));
      };
      for (int i = -1; i < n && ok; ++i) {
        if (i + 1 < n) {
          const int j = i + 1;
          ok = c.wait(kBKFull + (j & 1), j >> 1);
          if (ok && j >= 2) ok = c.wait(kBSFree + (j & 1), (j - 2) >> 1);
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) issue_s(j);
          __syncwarp();
        }
        if (i >= 0) {
          ok = c.wait(kBVFull + (i & 1), i >> 1) && c.wait(kBPReady, i);
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) issue_o(i);
          __syncwarp();
        }
      }
    }
  }
  if (!ok) {
    if (*c.failed == 0) flag(lv.status, OSCAR_STATUS_TIMEOUT);
    *c.failed = 1;
  }
  if (w == kMmaWarp && lane == 0) {                // every MMA completes before TMEM is read or released
    umma_commit(c.bar(kBFinal));
    mbar_wait(c.bar(kBFinal), 0);
  }
  if (w == kLoadWarp && lane == 0 && hist && n > 0 && *c.failed != 0) {
    // copies still in flight land before the CTA leaves: each stage's newest (bounded waits)
    mbar_wait(c.bar(kBImg), 0);
    for (int s = 0; s < kStages; ++s)
      for (int ph = 0; ph < 2; ++ph) mbar_wait(c.bar(kBFull + s), ph);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // ---- partials: thread = row ------------------------------------------------------------------------------
  if (w < active) {
    const bool good = *c.failed == 0 && n > 0;     // block-uniform after the barrier
    float* part = tree_part(a, lv.hq, b, min(node, a.T - 1), hq, slot);
    const uint32_t trow = c.tmem + ((uint32_t)(32 * w) << 16);
    const float M = m == -INFINITY ? -INFINITY : hist ? fmaf(m, F, -kBias) : m * F;
    if (row < live) *reinterpret_cast<float2*>(part) = good ? make_float2(M, lsum) : make_float2(-INFINITY, 0.f);
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      float o[32];
      if (good) tmem_ld32(trow + kColO + 32 * k, o);
      if (row < live) {
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<float4*>(part + 4 + 32 * k + e) =
              good ? make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (w == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(c.tmem), "r"(kTmemCols) : "memory");
  }
}

template <int FMT>
int launch_fmt(const LayerView& lv, const TreeArgs& a, int B, cudaStream_t st) {
  const int tiles = (a.T * (lv.hq / lv.hkv) + kRows - 1) / kRows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.nsplit + a.nb, lv.hkv * tiles, B);
  cfg.blockDim = dim3(kTreeThreads);
  cfg.dynamicSmemBytes = kTreeSmem;
  cfg.stream = st;
  return cudaLaunchKernelEx(&cfg, k_tree_attention<FMT>, lv, a) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

template <int FMT>
int configure_fmt() {
  if (cudaFuncSetAttribute(k_tree_attention<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTreeSmem) != cudaSuccess)
    return OSCAR_ERR_CUDA;
  return set_max_shared_carveout(reinterpret_cast<const void*>(k_tree_attention<FMT>));
}

}  // namespace

// Slots of a query row: the history over nsplit of them, the BF16 and draft pages over nb. One CTA runs on an SM at a
// time; its start (rotation of the rows, first pages) and its end cost about as much as kFixed history tiles, a BF16
// tile, which is not pipelined as deeply, about as much as two. The counts that need the fewest waves times tiles
// win, and of equal ones those with the fewest slots, which the merge reads.
void tree_splits(int B, int T, int hkv, int gq, int nbf, int max_hist_pages, int sms, int max_slots, int* nsplit,
                 int* nb) {
  constexpr double kFixed = 6.0;
  const long units = (long)B * hkv * ((T * gq + kRows - 1) / kRows);
  const int near = nbf + (T + kP - 1) / kP, tiles = std::max(1, (max_hist_pages + 1) / 2);
  double best = 0.0;
  *nsplit = *nb = 1;
  for (int m = 1; m <= near && m < max_slots; ++m)
    for (int s = 1; s <= std::min(tiles, 2 * sms) && s + m <= max_slots; ++s) {
      const long waves = (units * (s + m) + sms - 1) / sms;
      const int work = std::max((tiles + s - 1) / s, 2 * ((near + m - 1) / m));
      const double cost = (double)waves * (work + kFixed) + 0.05 * (s + m);
      if (best == 0.0 || cost < best) {
        best = cost;
        *nsplit = s;
        *nb = m;
      }
    }
}

int launch_tree_attention(const LayerView& lv, const TreeArgs& a, int B, cudaStream_t st) {
  const int rc = lv.meta_cb ? launch_fmt<kFmtCB>(lv, a, B, st)
                            : lv.meta_u8 ? launch_fmt<kFmtU8>(lv, a, B, st) : launch_fmt<kFmtF16>(lv, a, B, st);
  return rc == OSCAR_OK ? launch_tree_merge(lv, a, B, st) : rc;
}

int configure_tree_kernels() {
  if (configure_fmt<kFmtF16>() != OSCAR_OK || configure_fmt<kFmtU8>() != OSCAR_OK) return OSCAR_ERR_CUDA;
  return configure_fmt<kFmtCB>();
}

}  // namespace oscar
