// Attention of a tree of drafted tokens over the mixed cache (sm_103a: tcgen05.mma, TMEM accumulators).
//
// Query row (node i, head) of a request attends to all committed tokens, read where they are (INT2 history in
// the rotated basis, BF16 sink and recent rows), and to the drafted nodes of its mask word i:
//   logits  history: s (q R_K) . khat   BF16, drafted: s q . k,   one softmax, o = sum p v.
// The T gq query rows of a kv head are the M = 128 rows of a tensor-core tile, so a page is read and unpacked
// once for all of them.
//
// Grid (slot, kv head x row tiles, request), one CTA per SM. A slot is a range of the request's history pages, or of
// its BF16 and draft pages. A page (64 tokens) is a tile:
//  * S = Q K^T, A = the rows in TMEM (history: q R_K as fp16, rotated by this CTA at its start; else q as bf16),
//    B = the keys in shared memory: history keys dequantised to fp16 (zero + scale code, one rounding).
//  * row threads (thread = row = TMEM lane): weights p = 2^(x - m) and their sum in float32. m is a reference near
//    the running maximum, not the maximum: a page whose weights sum to at most 2^15 keeps it (fp16 holds them), any
//    other sets it to the row's maximum, rescales O and redoes its weights. So no page but the first looks for a
//    maximum. History weights carry 2^7, so that weights down to 2^-31 of the largest still count.
//  * O += P V, A = P in TMEM, B = the values in shared memory, dequantised like the keys; BF16 pages take P as two
//    bf16 parts, since their tokens often carry most of the weight.
// Values are rounded with their zero point in place: with scale * code alone, the rounding of the products and of
// the zero point's sum would no longer cancel where many tokens average out.
//
// Two streams with an S, P and O, a reference and a sum each keep the tensor pipe and the row threads busy beside each
// other. With at most 128 query rows they are the even and the odd pages, joined when the slot ends. With more, a CTA
// takes two tiles of rows (WIDE), a stream each, and every page is unpacked once for both: 136 rows over 2 x 33K tokens
// 80 us (a CTA per tile: 105 us), 256 rows over 102,400 tokens 98 us (115 us). TMEM is full: O (2 x 128 columns), S
// (2 x 64), P (2 x 32), the rows (64; a second tile's are an operand in shared memory).
// Warpgroups: 0-1 rows of the two streams, 2-3 unpack keys, 4-5 unpack values (even and odd pages), 6: warp 24 issues
// S, warp 25 streams the pages through a ring of bulk copies, warp 26 turns the values' scales and zeros into the pairs
// the value warps multiply by, warp 27 issues O. A row thread reads a page's 64 logits at once and so frees S for the
// stream's next product; it keeps them until its weights stand, in case it has to raise the reference.
// A history page of one tile is 8 MMAs of M128 N64 K16 (32 cycles each) and 4 of M128 N128 K16 (64): 512 cycles of the
// tensor pipe. The CUDA cores issue about 725 warp instructions per scheduler beside them (rows 250, keys 190, values
// 190, control 95) and take 915 cycles a page, 1,770 for two tiles (1,000 instructions): the exponentials take 4 cycles a
// warp, the packed multiplies, adds and half-precision products 2 each, and the bit operations 2. Neither is full (two
// tiles over 102,400 tokens: tensor pipe 49 % of the cycles, issue slots 56 %; one, 8 requests: 24 and 47 %): what is
// left is the time the roles wait for one another, page by page. Two threads to a row, half of a page's tokens each,
// measured 15 % slower: the same instructions and more hand-overs.
// Every wait is bounded; a CTA whose wait expires flags OSCAR_STATUS_TIMEOUT and writes empty partials.
#include <algorithm>

#include "tcgen05.cuh"
#include "tma.cuh"
#include "tree.cuh"

namespace oscar {
namespace {

constexpr int kRowWarps = 8, kKWarp0 = 8, kVWarp0 = 16, kMmaWarp = 24, kLoadWarp = 25, kMetaWarp = 26,
              kMmaOWarp = 27;
constexpr int kTreeThreads = 28 * 32;
// registers per thread: at launch, then of the rows, the unpacking and the control warpgroups; the shares stay within
// what the CTA was launched with
constexpr int kRegsLaunch = 72, kRegsRows = 112, kRegsUnpack = 56, kRegsCtl = 56;
static_assert(2 * kRegsRows + 4 * kRegsUnpack + kRegsCtl <= 7 * kRegsLaunch, "register shares");
constexpr int kRows = kTreeRows;                   // query rows of a tile
constexpr int kStages = 8;                         // ring stages of one page block
constexpr int kBufs = 4;                           // unpacked pages: keys, and values
constexpr int kSboK = (kD / 8) * 128;              // keys: rows = tokens, 128 channels: 2,048 B between 8-row blocks
constexpr int kSboV = (kP / 8) * 128;              // values: rows = channels, 64 tokens
constexpr int kSboVNear = kSboV + 16;              // values of a BF16 page, padded against bank conflicts
constexpr int kKBytes = kP * kD * 2, kVBytes = kD / 8 * kSboVNear + 256;
static_assert(kVBytes % 256 == 0, "operand alignment");
constexpr int kImgBytes = kD * kD * 2;             // one part of the rotation
constexpr int kOffK = 0, kOffV = kOffK + kBufs * kKBytes, kOffRing = kOffV + kBufs * kVBytes;
static_assert(kBufs * kKBytes >= 2 * kImgBytes && kBufs * kVBytes >= kRows * kD * 2, "the rotation's operands fit");
constexpr int kPids = 4096;                        // page ids of a slot kept in shared memory
constexpr int kOffPid = kOffRing + kStages * kBlockBytes;
// BF16 slots keep no page ids; the same bytes hold a bit set per page of the value rows that are not finite
constexpr int kPoisonTiles = kPids / 2;
static_assert(kMaxTreeBf16Pages + kMaxDraft / kP <= kPoisonTiles, "a set for every BF16 and draft page");
// and the ring holds those slots' page descriptors: page id, or -1 - draft page, and rows
constexpr int kOffNear = kOffRing;
static_assert(8 * kPoisonTiles <= kStages * kBlockBytes, "a descriptor for every BF16 and draft page");
constexpr int kWarm = 8;                           // BF16 and draft pages that are asked for at the start
// [stage][group][scale, zero][32 token pairs in the order of the values' k positions], fp16 pairs
constexpr int kMetaStage = 2 * 2 * 32 * 4;
constexpr int kOffMeta = kOffPid + kPids * 4;
constexpr int kOffJoin = kOffMeta + kStages * kMetaStage;   // [2 streams][128 rows] (M, l)
constexpr int kOffF = kOffJoin + 2 * kRows * 8;    // [256 rows] factor of a row's logits
constexpr int kOffInfo = kOffF + 2 * kRows * 4;    // what the roles read about the slot: kI*
constexpr int kIPages = 0, kIRest = 4, kILive = 8;
constexpr int kOffBar = kOffInfo + 32;
constexpr int kBFull = 0, kBEmpty = kBFull + kStages, kBMeta = kBEmpty + kStages, kBKFull = kBMeta + kStages,
              kBVFull = kBKFull + kBufs, kBKFree = kBVFull + kBufs, kBVFree = kBKFree + kBufs, kBSDone = kBVFree + kBufs,
              kBSFree = kBSDone + 2, kBPReady = kBSFree + 2, kBODone = kBPReady + 2, kBImg = kBODone + 2, kBQ = kBImg + 1,
              kBFinal = kBQ + 1, kNumBars = kBFinal + 1;
constexpr int kOffTmem = kOffBar + kNumBars * 8, kOffFailed = kOffTmem + 4;   // TMEM address, failure flag
constexpr int kOffQ = (kOffTmem + 16 + 127) / 128 * 128;   // two tiles: the second one's rows, an A operand
// with alignment slack
template <bool WIDE> constexpr int kTreeSmem = (WIDE ? kOffQ + kRows * kD * 2 : kOffTmem + 16) + 1024;
constexpr uint32_t kColO = 0, kColS = 256, kColP = 384, kColQ = 448, kTmemCols = 512;   // stream e: + 128 e, 64 e, 32 e
constexpr uint32_t kIdescS = idesc_f16(128, 64), kIdescO = idesc_f16(128, 128);
constexpr uint32_t kBf16Bits = (1u << 7) | (1u << 10);              // A and B bf16
constexpr float kLazy = 8.f;                       // BF16 pages: log2 growth of a maximum that forces a rescale
constexpr float kBias = 7.f;                       // log2 of the factor of history weights
constexpr float kMostSum = 32768.f;                // a page's weights may sum to this: each fits fp16
constexpr uint32_t kMagic = 0x64006400u;           // fp16 1024.0 in both halves

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
// shared memory by 32-bit address: the roles' pointers stay one register each
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t x;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 x;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ void sts32(uint32_t at, uint32_t x) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t at, uint4 x) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}
// (scale, zero) of the two groups of a row as fp16 pairs {s0, z0}, {s1, z1}; blk: shared address of the page block.
// Codebook format: the levels k / 256 are exact fp16 numbers, 255ths are not; the range takes the factor 256 / 255 and is
// rounded to fp16 once more, so a key or value has two roundings of 2^-11, of scale times level and of the sum.
// Compact format: a value is mn8 D - T + code (mx8 - mn8) E with D = 3 E and T = 127.5 D, that is E times
// 3 mn8 - 382.5 + code (mx8 - mn8), which fp16 holds exactly. The group's E goes into the query rows and, for values,
// into the partials. (Scale and zero rounded to fp16 tripled the outputs' error.)
template <int FMT>
__device__ __forceinline__ uint2 scale_zero(uint32_t blk, int kind, int row) {
  if (FMT == kFmtU8) {
    const uint32_t m = lds32(blk + (kind ? kVMetaOffU8 : kKMetaOff) + 4 * row);   // mn8, mx8 of group 0, of group 1
    const uint32_t mn = hfma2_u(__byte_perm(m, kMagic, 0x5250), 0x3C003C00u, 0xE400E400u);   // (1024 + mn8) - 1024
    const uint32_t mx = hfma2_u(__byte_perm(m, kMagic, 0x5351), 0x3C003C00u, 0xE400E400u);
    const uint32_t s = hfma2_u(mn, 0xBC00BC00u, mx), z = hfma2_u(mn, 0x42004200u, 0xDDFADDFAu);   // 3 mn8 - 382.5
    return make_uint2(__byte_perm(s, z, 0x5410), __byte_perm(s, z, 0x7632));
  }
  uint2 m = lds64(blk + (kind ? kVMetaOff : kKMetaOff) + 8 * row);
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
  uint32_t base;                                   // shared memory, 1,024-byte aligned
  int rest;                                        // history: tokens from the slot's first page on
  // all 512 columns are allocated: they start at column 0 (checked). A constant address keeps the MMAs' operands uniform.
  static constexpr uint32_t tmem = 0;
  __device__ __forceinline__ uint32_t bar(int k) const { return base + kOffBar + 8u * (uint32_t)k; }
  __device__ __forceinline__ bool failed() const { return lds32(base + kOffFailed) != 0u; }
  __device__ __forceinline__ void fail() const { sts32(base + kOffFailed, 1u); }
  // one wait of a whole warp; false (the CTA has failed, or the wait expired) ends its work
  __device__ __forceinline__ bool wait(int k, int phase) const {
    const uint32_t parity = (uint32_t)phase & 1u;
    bool ok = mbar_try(bar(k), parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    const unsigned long long t0 = global_ns();     // a small loop: the roles' code shares the instruction caches
#pragma unroll 1
    while (!ok && !failed() && global_ns() - t0 <= kWaitNs) ok = mbar_try(bar(k), parity);
    return __all_sync(0xffffffffu, ok);
  }
  __device__ __forceinline__ void arrive(int k) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar(k));
  }
  __device__ __forceinline__ void arrive(int j, int k) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      mbar_arrive(bar(j));
      mbar_arrive(bar(k));
    }
  }
  // valid tokens of history page i of the slot
  __device__ __forceinline__ int tokens(int i) const {
    return (int)lds32(base + kOffPid + 4 * i) >= 0 ? min(kP, rest - i * kP) : 0;
  }
};

// O of this warp's rows, of one stream, times al
__device__ __forceinline__ void rescale_o(uint32_t to, float al) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    float o[32];
    tmem_ld32(to + 32 * c, o);
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] *= al;
    tmem_st32(to + 32 * c, o);
  }
}

// ---- row threads, history pages ------------------------------------------------------------------------
// Weights of 32 tokens from their S columns as fp16 pairs in the k order of the values: pair 4w + p holds tokens
// 16 (p >> 1) + 2w + 8 (p & 1) and the next. Their sum is added to t2.
__device__ __forceinline__ void weights32(const float (&s)[32], float2 F2, float2 nm2, uint32_t (&r)[16], float2& t2) {
#pragma unroll
  for (int w = 0; w < 4; ++w)
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int t = 16 * (p >> 1) + 2 * w + 8 * (p & 1);
      const float2 x = __ffma2_rn(make_float2(s[t], s[t + 1]), F2, nm2);
      const float2 v = make_float2(fast_exp2(x.x), fast_exp2(x.y));
      t2 = __fadd2_rn(t2, v);
      r[4 * w + p] = pack_f16x2(v.x, v.y);
    }
}

// The stream's pages: e, e + 2, ... of the slot, or with two tiles all of them.
template <bool WIDE>
__device__ __forceinline__ bool rows_history(const Ctx c, int e, int n, float F, float& m, float& lsum) {
  const uint32_t lane0 = (uint32_t)(32 * ((threadIdx.x >> 5) & 3)) << 16;
  const uint32_t to = c.tmem + lane0 + kColO + 128 * e, ts = c.tmem + lane0 + kColS + 64 * e, tp = c.tmem + lane0 + kColP + 32 * e;
  float l = 0.f;
#pragma unroll 1
  for (int i = WIDE ? 0 : e; i < n; i += WIDE ? 1 : 2) {
    const int ph = WIDE ? i : i >> 1, live = c.tokens(i);
    if (!c.wait(kBSDone + e, ph)) return false;
    tc_fence_after();
    float s0[32], s1[32];                          // kept until the weights stand: S itself is free for the next page
    tmem_ld32x2(ts, ts + 32, s0, s1);
    tc_fence_before();
    c.arrive(kBSFree + e);
    if (live < kP) {                               // the end of the history
#pragma unroll
      for (int x = 0; x < 32; ++x) {
        s0[x] = x < live ? s0[x] : -INFINITY;
        s1[x] = 32 + x < live ? s1[x] : -INFINITY;
      }
    }
    uint32_t r0[16], r1[16];
    float sum = 0.f;
    bool free_o = ph == 0;                         // O of the stream's last page is complete
    bool redo = __any_sync(0xffffffffu, m == -INFINITY);
    // Twice at most: the first pass may be for a row of the warp that has no reference yet while the others keep theirs,
    // so its sums are looked at like any other's; what they raise in the second pass is at the page's maximum.
#pragma unroll 1
    for (int pass = 0;; ++pass) {
      if (redo) {                                  // a reference at the rows' maxima: the first page, or weights too large
        float mx = -INFINITY;
#pragma unroll
        for (int x = 0; x < 32; ++x) mx = fmaxf(mx, fmaxf(s0[x], s1[x]));
        float al = 1.f;
        if ((m == -INFINITY || sum > kMostSum) && mx > m) {
          al = m == -INFINITY ? 0.f : exp2f((m - mx) * F);
          m = mx;
        }
        l *= al;
        if (!free_o) {
          if (!c.wait(kBODone + e, ph - 1)) return false;
          tc_fence_after();
          free_o = true;
        }
        if (ph > 0) rescale_o(to, al);
      }
      // the page's weights against the reference m
      const float mF = m == -INFINITY ? 0.f : fmaf(m, F, -kBias);
      const float2 F2 = make_float2(F, F), nm2 = make_float2(-mF, -mF);
      float2 t2 = make_float2(0.f, 0.f);
      weights32(s0, F2, nm2, r0, t2);
      weights32(s1, F2, nm2, r1, t2);
      sum = t2.x + t2.y;
      if (pass > 0) break;
      redo = __any_sync(0xffffffffu, sum > kMostSum);
      if (!redo) break;
    }
    l += sum;
    if (!free_o) {                                 // the stream's last O has read the weights before these
      if (!c.wait(kBODone + e, ph - 1)) return false;
      tc_fence_after();
    }
    tmem_st16(tp, r0);
    tmem_st16(tp + 16, r1);
    tmem_wait_st();
    tc_fence_before();
    c.arrive(kBPReady + e);
  }
  lsum = l;
  return true;
}

// ---- row threads, BF16 and draft pages -----------------------------------------------------------------
// bits(i): the tokens of page i that this row sees. The low parts of the weights go where S was: the stream's next S waits for
// this O.
template <bool WIDE, typename Bits>
__device__ __forceinline__ bool rows_bf16(const Ctx c, int e, int n, float F, Bits bits, float& m, float& lsum) {
  const uint32_t lane0 = (uint32_t)(32 * ((threadIdx.x >> 5) & 3)) << 16;
  const uint32_t to = c.tmem + lane0 + kColO + 128 * e, ts = c.tmem + lane0 + kColS + 64 * e, tp = c.tmem + lane0 + kColP + 32 * e;
  float l = 0.f;
#pragma unroll 1
  for (int i = WIDE ? 0 : e; i < n; i += WIDE ? 1 : 2) {
    const int ph = WIDE ? i : i >> 1;
    const unsigned long long see = bits(i);
    if (!c.wait(kBSDone + e, ph)) return false;
    tc_fence_after();
    float mx = -INFINITY;
#pragma unroll 1
    for (int q = 0; q < 2; ++q) {
      float s[32];
      tmem_ld32(ts + 32 * q, s);
      const uint32_t mine = (uint32_t)(see >> (32 * q));
#pragma unroll
      for (int x = 0; x < 32; ++x) mx = fmaxf(mx, mine >> x & 1u ? s[x] : -INFINITY);
    }
    float al = 1.f;
    const bool grow = (mx - m) * F > kLazy;
    if (grow) {
      al = m == -INFINITY ? 0.f : exp2f((m - mx) * F);
      m = mx;
    }
    if (__any_sync(0xffffffffu, grow) && ph > 0) { // O of the stream's last page is complete: S(i) waited for it
      rescale_o(to, al);
    }
    l *= al;
    const float mF = m == -INFINITY ? 0.f : m * F;
#pragma unroll 1
    for (int q = 0; q < 2; ++q) {                  // p = hi + lo, pairs of tokens 2j, 2j + 1; lo over logits already read
      float s[32];
      uint32_t hi[16], lo[16];
      tmem_ld32(ts + 32 * q, s);
      const uint32_t mine = (uint32_t)(see >> (32 * q));
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float x = mine >> (2 * j) & 1u ? fast_exp2(fmaf(s[2 * j], F, -mF)) : 0.f;
        const float y = mine >> (2 * j + 1) & 1u ? fast_exp2(fmaf(s[2 * j + 1], F, -mF)) : 0.f;
        l += x + y;
        hi[j] = pack_bf16x2(x, y);
        lo[j] = pack_bf16x2(x - __uint_as_float(hi[j] << 16), y - __uint_as_float(hi[j] & 0xffff0000u));
      }
      tmem_st16(tp + 16 * q, hi);
      tmem_st16(ts + 16 * q, lo);
    }
    if (!c.wait(kBVFull + i % kBufs, i / kBufs)) return false;   // last: the values take longer than the keys
    const uint2 bad = lds64(c.base + kOffPid + 8 * i);
    if ((uint32_t)see & bad.x || (uint32_t)(see >> 32) & bad.y) l = NAN;   // a NaN or infinity among the values the row sees
    tmem_wait_st();
    tc_fence_before();
    c.arrive(kBPReady + e);
  }
  lsum = l;
  return true;
}

// ---- key warps, history pages --------------------------------------------------------------------------
// Key row t: the 16-channel block u is one word of codes; k positions 2q, 2q + 1 of the block are channels 16u + q,
// 16u + 8 + q (the rows' fragments use the same order).
template <int FMT>
__device__ __forceinline__ bool keys_history(const Ctx c, const LayerView& lv, int h, int e, int n) {
  const int lane = threadIdx.x & 31, kw = (threadIdx.x >> 5) & 3, t0 = (lane & 7) + 8 * kw, u0 = lane >> 3;
  const uint32_t lut = FMT == kFmtCB ? lut_of(lv, h, OSCAR_KIND_K) : 0u;
  const uint32_t dst0 = c.base + kOffK + kw * kSboK + 2 * u0 * 128 + (t0 & 7) * 16;
#pragma unroll 1
  for (int i = e; i < n; i += 2) {
    const int b = i % kBufs, st = i % kStages;
    if (!c.wait(kBFull + st, i / kStages)) return false;
    if (i >= kBufs && !c.wait(kBKFree + b, i / kBufs - 1)) return false;
    const uint32_t blk = c.base + kOffRing + st * kBlockBytes, codes = blk + kKCodesOff + 32 * t0 + 4 * u0;
    const uint32_t dst = dst0 + b * kKBytes;
    // tokens t0, t0 + 32 (k) and the 16-channel blocks u0, u0 + 4 (g), one of each group; all loads first
    uint2 sz[2];
    uint32_t x[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      sz[k] = scale_zero<FMT>(blk, 0, t0 + 32 * k);
#pragma unroll
      for (int g = 0; g < 2; ++g) x[k][g] = lds32(codes + 1024 * k + 16 * g);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint32_t m = g ? sz[k].y : sz[k].x, s2 = __byte_perm(m, m, 0x1010), z2 = __byte_perm(m, m, 0x3232);
        const uint32_t lo = x[k][g], hi = lo >> 8;
        const uint32_t d = dst + 4 * k * kSboK + 8 * g * 128;
        sts128(d, make_uint4(value_at<FMT>(lo, 0, lut, s2, z2), value_at<FMT>(lo, 1, lut, s2, z2),
                             value_at<FMT>(lo, 2, lut, s2, z2), value_at<FMT>(lo, 3, lut, s2, z2)));
        sts128(d + 128, make_uint4(value_at<FMT>(hi, 0, lut, s2, z2), value_at<FMT>(hi, 1, lut, s2, z2),
                                   value_at<FMT>(hi, 2, lut, s2, z2), value_at<FMT>(hi, 3, lut, s2, z2)));
      }
    fence_async();
    c.arrive(kBKFull + b, kBEmpty + st);
  }
  return true;
}

// ---- value warps, history pages ------------------------------------------------------------------------
// Value channel c: word w of its codes holds tokens 16 (p >> 1) + 2w + 8 (p & 1) + e at code positions p. Positions
// p < 4 are tokens 0 .. 31 of the page, the others tokens 32 .. 63, so token half hf takes the k positions
// 32 hf + 8w + 2 (p & 3) + e: 16 bytes a word, and the rows store the weights of 32 tokens as 16 columns.

// Warp 26: the scales and zeros of a page as fp16 pairs in that order. Tokens past the end get 0 and 0: the block's
// bytes there may be anything, and 0 times a NaN would reach O.
template <int FMT>
__device__ __forceinline__ bool value_pairs(const Ctx c, int n) {
  const int lane = threadIdx.x & 31;
  const int w = (lane >> 2) & 3, p = (lane & 3) + 4 * (lane >> 4), t = 16 * (p >> 1) + 2 * w + 8 * (p & 1);
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    const int st = i % kStages, nv = c.tokens(i);
    if (!c.wait(kBFull + st, i / kStages)) return false;
    const uint32_t blk = c.base + kOffRing + st * kBlockBytes, to = c.base + kOffMeta + st * kMetaStage + 4 * lane;
    uint2 a = scale_zero<FMT>(blk, 1, t), d = scale_zero<FMT>(blk, 1, t + 1);
    if (t >= nv) a = make_uint2(0u, 0u);
    if (t + 1 >= nv) d = make_uint2(0u, 0u);
    sts32(to, __byte_perm(a.x, d.x, 0x5410));
    sts32(to + 128, __byte_perm(a.x, d.x, 0x7632));
    sts32(to + 256, __byte_perm(a.y, d.y, 0x5410));
    sts32(to + 384, __byte_perm(a.y, d.y, 0x7632));
    c.arrive(kBMeta + st, kBEmpty + st);
  }
  return true;
}

template <int FMT>
__device__ __forceinline__ bool values_history(const Ctx c, const LayerView& lv, int h, int e, int n) {
  // a thread has one word position w and the channels cl + 8 (vw + 4 j + 8 g); their 16-byte slots (v_chan_off) swap
  // the low three bits of the channel with (channel >> 4) & 7 = (vw >> 1) + 2 j + 4 g
  const int lane = threadIdx.x & 31, vw = (threadIdx.x >> 5) & 3, w = lane >> 3, cl = lane & 7;
  const uint32_t lut = FMT == kFmtCB ? lut_of(lv, h, OSCAR_KIND_V) : 0u;
  const uint32_t slot0 = kVCodesOff + vw * 128 + (cl ^ (vw >> 1)) * 16 + 4 * w;
  const uint32_t dst0 = c.base + kOffV + vw * kSboV + w * 128 + cl * 16, meta0 = c.base + kOffMeta + 16 * w;
#pragma unroll 1
  for (int i = e; i < n; i += 2) {
    const int b = i % kBufs, st = i % kStages;
    if (!c.wait(kBMeta + st, i / kStages)) return false;   // after the page itself
    if (i >= kBufs && !c.wait(kBVFree + b, i / kBufs - 1)) return false;
    const uint32_t codes = c.base + kOffRing + st * kBlockBytes + slot0, meta = meta0 + st * kMetaStage;
    const uint32_t dst = dst0 + b * kVBytes;
    uint32_t x[2][2];
    uint4 s2[2][2], z2[2][2];                      // [group][positions 0-3 (tokens 0-31), 4-7] of word w
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        x[g][j] = lds32((codes ^ (32 * j + 64 * g)) + 512 * j + 1024 * g);
        s2[g][j] = lds128(meta + 256 * g + 64 * j);
        z2[g][j] = lds128(meta + 256 * g + 128 + 64 * j);
      }
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t lo = x[g][j], hi = lo >> 8;
        const uint32_t d = dst + (4 * j + 8 * g) * kSboV;
        sts128(d, make_uint4(value_at<FMT>(lo, 0, lut, s2[g][0].x, z2[g][0].x), value_at<FMT>(lo, 1, lut, s2[g][0].y, z2[g][0].y),
                             value_at<FMT>(lo, 2, lut, s2[g][0].z, z2[g][0].z), value_at<FMT>(lo, 3, lut, s2[g][0].w, z2[g][0].w)));
        sts128(d + 4 * 128,
               make_uint4(value_at<FMT>(hi, 0, lut, s2[g][1].x, z2[g][1].x), value_at<FMT>(hi, 1, lut, s2[g][1].y, z2[g][1].y),
                          value_at<FMT>(hi, 2, lut, s2[g][1].z, z2[g][1].z), value_at<FMT>(hi, 3, lut, s2[g][1].w, z2[g][1].w)));
      }
    fence_async();
    c.arrive(kBVFull + b, kBEmpty + st);
  }
  return true;
}

// A BF16 or draft page: rows 0 .. rows - 1 of K and V at k0, v0, `step` elements apart.
struct Near {
  const __nv_bfloat16 *k, *v;
  size_t step;
  int rows;
  int draft;                                       // the page of the drafts, -1: a BF16 page
};
// bits 15 and 31: the bf16 value of that half is a NaN or an infinity (its exponent carries)
__device__ __forceinline__ uint32_t exponents(uint32_t x) { return (x & 0x7F807F80u) + 0x00800080u; }
constexpr uint32_t kNonfinite = 0x80008000u;

// ---- key warps, BF16 pages (natural channel order) -----------------------------------------------------
template <typename Page>
__device__ __forceinline__ bool keys_bf16(const Ctx c, int* status, int e, int n, Page page) {
  const int lane = threadIdx.x & 31, kw = (threadIdx.x >> 5) & 3, t0 = (lane & 7) + 8 * kw;
  const uint32_t dst0 = c.base + kOffK + kw * kSboK + (lane & 7) * 16 + (lane >> 3) * 128;
#pragma unroll 1
  for (int i = e; i < n; i += 2) {
    const int b = i % kBufs;
    const Near p = page(i);
    uint4 x[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint4* src = reinterpret_cast<const uint4*>(p.k + (t0 + 32 * k) * p.step) + (lane >> 3);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[k][j] = t0 + 32 * k < p.rows ? src[4 * j] : make_uint4(0u, 0u, 0u, 0u);
    }
    if (i >= kBufs && !c.wait(kBKFree + b, i / kBufs - 1)) return false;
    if (p.draft >= 0) {
      uint32_t bad = 0u;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) bad |= exponents(x[k][j].x) | exponents(x[k][j].y) | exponents(x[k][j].z) | exponents(x[k][j].w);
      if ((bad & kNonfinite) != 0u) flag(status, OSCAR_STATUS_NONFINITE);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        sts128(dst0 + b * kKBytes + 4 * k * kSboK + 4 * j * 128, x[k][j]);
    fence_async();
    c.arrive(kBKFull + b);
  }
  return true;
}

// ---- value warps, BF16 pages: transposed, non-finite values replaced by 0 and their rows noted ----------
template <typename Page>
__device__ __forceinline__ bool values_bf16(const Ctx c, int* status, int e, int n, Page page) {
  const int lane = threadIdx.x & 31, vw = (threadIdx.x >> 5) & 3;
#pragma unroll 1
  for (int i = e; i < n; i += 2) {
    const int b = i % kBufs;
    const Near p = page(i);
    bool mine = i < kBufs;                         // the buffer is free
#pragma unroll 1
    for (int o = vw; o < kP / 8; o += 4) {         // token octets; a small loop: a slot runs it a few times only
      uint32_t x[2][8];                            // [channel half][token]: channels 2 cp, 2 cp + 1
      const uint32_t* src = reinterpret_cast<const uint32_t*>(p.v + 8 * o * p.step) + lane;
      uint32_t bad = 0u;
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const bool in = 8 * o + t < p.rows;
        x[0][t] = in ? src[0] : 0u;
        x[1][t] = in ? src[32] : 0u;
        src += p.step >> 1;
      }
#pragma unroll
      for (int t = 0; t < 8; ++t) bad |= exponents(x[0][t]) | exponents(x[1][t]);
      if ((bad & kNonfinite) != 0u) {
        uint32_t rows = 0u;
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if ((exponents(x[k][t]) & kNonfinite) != 0u) {
              rows |= 1u << t;
              x[k][t] = 0u;
            }
        asm volatile("red.shared.or.b32 [%0], %1;" ::"r"(c.base + kOffPid + 8 * i + 4 * (o >> 2)), "r"(rows << (8 * (o & 3))) : "memory");
        if (p.draft >= 0) flag(status, OSCAR_STATUS_NONFINITE);
      }
      if (!mine && !c.wait(kBVFree + b, i / kBufs - 1)) return false;
      mine = true;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int ch = 2 * (lane + 32 * k);
        const uint32_t d = c.base + kOffV + b * kVBytes + (ch >> 3) * kSboVNear + o * 128 + (ch & 7) * 16;
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          lo[t] = __byte_perm(x[k][2 * t], x[k][2 * t + 1], 0x5410);
          hi[t] = __byte_perm(x[k][2 * t], x[k][2 * t + 1], 0x7632);
        }
        sts128(d, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        sts128(d + 16, make_uint4(hi[0], hi[1], hi[2], hi[3]));
      }
    }
    fence_async();
    c.arrive(kBVFull + b);
  }
  return true;
}

// Page i of the slot into ring stage i % kStages (one thread).
__device__ __forceinline__ void issue_page(const Ctx c, const LayerView& lv, int h, int i) {
  const int st = i % kStages, id = (int)lds32(c.base + kOffPid + 4 * i);
  mbar_expect_tx(c.bar(kBFull + st), id >= 0 ? (uint32_t)lv.blk_bytes : 0u);   // also for no page: the phase completes
  if (id >= 0)
    bulk_copy_hint(c.base + kOffRing + st * kBlockBytes, int2_block(lv, id, h), (uint32_t)lv.blk_bytes, c.bar(kBFull + st),
                   l2_evict_first());
}

// The control warps: page stream, scale pairs, MMAs.
template <int FMT, bool WIDE>
__device__ __forceinline__ bool control(const Ctx c, const LayerView& lv, int w, int h, bool hist, int n, bool second) {
  const int lane = threadIdx.x & 31;
  if (w == kLoadWarp) {
    if (!hist) return true;
#pragma unroll 1
    for (int i = kStages; i < n; ++i) {
      if (!c.wait(kBEmpty + i % kStages, i / kStages - 1)) return false;
      if (lane == 0) issue_page(c, lv, h, i);
      __syncwarp();
    }
    return true;
  }
  if (w == kMetaWarp) return !hist || value_pairs<FMT>(c, n);
  // the MMAs, each kind issued by a warp of its own; page i is in buffer i % 4. One tile: page i belongs to stream i & 1.
  // Two tiles: to both streams, the second one's rows are an operand in shared memory.
  static_assert(kBufs == 4, "two pages of each stream");
  const uint32_t more = hist ? 0u : kBf16Bits;
  if (w == kMmaWarp) {
    const uint32_t kd = desc_lo(c.base + kOffK, 128), qd = desc_lo(c.base + kOffQ, 128);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int b = i % kBufs;
      if (!c.wait(kBKFull + b, i / kBufs)) return false;
#pragma unroll
      for (int k = 0; k < (WIDE ? 2 : 1); ++k) {
        if (k == 1 && !second) break;
        const int e = WIDE ? k : i & 1, ph = WIDE ? i : i >> 1;
        // the stream's last S is out of the way: read, or (BF16 pages, whose weights' low parts follow it there) used by O
        if (ph > 0 && !c.wait((hist ? kBSFree : kBODone) + e, ph - 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t keys = kd + b * (kKBytes >> 4) + 16 * kk;
          if (k == 1)
            umma_warp(c.tmem + kColS + 64, qd + 16 * kk, desc_hi(kSboK), keys, desc_hi(kSboK), kIdescS | more, kk > 0);
          else
            umma_ta_warp(c.tmem + kColS + 64 * e, c.tmem + kColQ + 8 * kk, keys, desc_hi(kSboK), kIdescS | more, kk > 0);
        }
        umma_commit_warp(c.bar(kBSDone + e));
      }
      umma_commit_warp(c.bar(kBKFree + b));
    }
  } else {
    const uint32_t vd = desc_lo(c.base + kOffV, 128), vh = hist ? desc_hi(kSboV) : desc_hi(kSboVNear);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int b = i % kBufs;
      if (!c.wait(kBVFull + b, i / kBufs)) return false;
#pragma unroll 1
      for (int k = 0; k < (WIDE && second ? 2 : 1); ++k) {
        const int e = WIDE ? k : i & 1, ph = WIDE ? i : i >> 1;
        if (!c.wait(kBPReady + e, ph)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_ta_warp(c.tmem + kColO + 128 * e, c.tmem + kColP + 32 * e + 8 * kk, vd + b * (kVBytes >> 4) + 16 * kk, vh,
                       kIdescO | more, ph > 0 || kk > 0);
        if (!hist) {                               // the weights' low parts
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ta_warp(c.tmem + kColO + 128 * e, c.tmem + kColS + 64 * e + 8 * kk, vd + b * (kVBytes >> 4) + 16 * kk, vh,
                         kIdescO | more, true);
        }
        umma_commit_warp(c.bar(kBODone + e));
      }
      umma_commit_warp(c.bar(kBVFree + b));
    }
  }
  return true;
}

// The sink and the recent pages that hold tokens of a request.
__device__ __forceinline__ int near_sink(const LayerView& lv, int L) { return (min(L, lv.sink) + kP - 1) / kP; }
__device__ __forceinline__ int near_recent(const LayerView& lv, int L) { return (min(max(L - lv.sink, 0), lv.recent) + kP - 1) / kP; }

// The BF16 and draft pages of a slot, by the descriptors that the start has left in shared memory.
struct NearPages {
  const LayerView& lv;
  const TreeArgs& a;
  uint32_t base;
  int b, h;
  __device__ __forceinline__ Near operator()(int i) const {
    const uint2 d = lds64(base + kOffNear + 8 * i);
    const int id = (int)d.x;
    Near r = {nullptr, nullptr, (size_t)kD, (int)d.y, id < 0 ? -1 - id : -1};
    if (id < 0) {
      const size_t at = (((size_t)b * a.T + r.draft * kP) * lv.hkv + h) * kD;
      r.k = a.kd + at;
      r.v = a.vd + at;
      r.step = (size_t)lv.hkv * kD;
    } else {
      r.k = bf16_row(lv, id, h, 0, 0);
      r.v = bf16_row(lv, id, h, 1, 0);
    }
    return r;
  }
};
// Descriptor of page i of n; p0: the slot's first page, seen: its draft pages, the last of the n.
__device__ __forceinline__ uint2 describe_page(const LayerView& lv, const TreeArgs& a, int b, int i, int n, int p0, int seen, int L,
                                               int nodes) {
  const int held = n - __popc(seen);
  if (i >= held) {
    int bits = seen;
    for (int k = i - held; k > 0; --k) bits &= bits - 1;
    const int d = __ffs(bits) - 1;
    return make_uint2((uint32_t)(-1 - d), (uint32_t)min(kP, nodes - d * kP));
  }
  const int ns = near_sink(lv, L), u = p0 + i, page = u < ns ? u : lv.sink / kP + u - ns, nbf = (lv.sink + lv.recent) / kP;
  const int rows = u < ns ? min(L, lv.sink) - u * kP : min(L - lv.sink, lv.recent) - (u - ns) * kP;
  const int id = a.bf16_pt[(size_t)b * nbf + page];
  if (id >= 0 && id < lv.n_bf16) return make_uint2((uint32_t)id, (uint32_t)min(kP, rows));
  flag(lv.status, OSCAR_STATUS_BAD_PAGE);
  return make_uint2(0u, 0u);                       // no rows of it are read
}

// Partials of a slot, thread = row. One tile: the streams' O joined, a warpgroup per half of the channels; both streams'
// row warps meet first (each has waited for its stream's last product). Two tiles: a warpgroup each. A CTA that failed
// writes empty ones. ref, l: the row's reference and sum of its stream. unit: what the values of a group were in units of.
template <bool WIDE>
__device__ __forceinline__ void write_partials(const Ctx c, const LayerView& lv, const TreeArgs& a, int h, int qt, int n, int live,
                                               float ref, float l, float2 unit) {
  const int tid = threadIdx.x, w = tid >> 5, row = tid & (kRows - 1), half = (tid >> 7) & 1;
  float M = ref, w0 = 1.f, w1 = 0.f;
  if (!WIDE) {
    sts32(c.base + kOffJoin + 8 * (half * kRows + row), __float_as_uint(ref));
    sts32(c.base + kOffJoin + 8 * (half * kRows + row) + 4, __float_as_uint(l));
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"r"(64 * ((live + 31) / 32)) : "memory");
    tc_fence_after();
    const uint2 u0 = lds64(c.base + kOffJoin + 8 * row), u1 = lds64(c.base + kOffJoin + 8 * (kRows + row));
    const float m0 = __uint_as_float(u0.x), m1 = n > 1 ? __uint_as_float(u1.x) : -INFINITY;
    M = fmaxf(m0, m1);
    w0 = m0 == -INFINITY ? 0.f : exp2f(m0 - M);
    w1 = m1 == -INFINITY ? 0.f : exp2f(m1 - M);
    l = w0 * __uint_as_float(u0.y) + (n > 1 ? w1 * __uint_as_float(u1.y) : 0.f);
  } else if (M == -INFINITY) {
    w0 = 0.f;
  }
  const bool good = __all_sync(0xffffffffu, !c.failed() && n > 0);
  float* part = tree_part(lv, a, blockIdx.z, qt, h, blockIdx.x);
  const uint32_t to = c.tmem + ((uint32_t)(32 * (w & 3)) << 16) + kColO + (WIDE ? 128 * half : 0);
  if (row < live && (WIDE || half == 0))
    *reinterpret_cast<float2*>(part + a.rows * kD + 2 * row) = good ? make_float2(M, l) : make_float2(-INFINITY, 0.f);
#pragma unroll 1
  for (int k = WIDE ? 0 : 2 * half; k < (WIDE ? 4 : 2 * half + 2); ++k) {
    float x[32], y[32];
    const float u = k < 2 ? unit.x : unit.y, u0 = w0 * u, u1 = w1 * u;
    if (!good) {
#pragma unroll
      for (int t = 0; t < 32; ++t) x[t] = 0.f;
    } else if (!WIDE && n > 1) {
      tmem_ld32x2(to + 32 * k, to + 128 + 32 * k, x, y);
#pragma unroll
      for (int t = 0; t < 32; ++t) x[t] = u0 * x[t] + u1 * y[t];
    } else {
      tmem_ld32(to + 32 * k, x);
#pragma unroll
      for (int t = 0; t < 32; ++t) x[t] *= u0;
    }
    if (row < live) {
      float4* dst = reinterpret_cast<float4*>(part) + 8 * k * a.rows + row;
#pragma unroll
      for (int t = 0; t < 8; ++t) dst[t * a.rows] = make_float4(x[4 * t], x[4 * t + 1], x[4 * t + 2], x[4 * t + 3]);
    }
  }
}

template <int FMT, bool WIDE>
__device__ __forceinline__ void run_roles(const LayerView& lv, const TreeArgs& a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Ctx c;
  c.base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t info = c.base + kOffInfo;
  const int w = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int h = blockIdx.y % lv.hkv, e = (w >> 2) & 1;   // e: the warpgroup's stream
  const int qt = WIDE ? 2 * (blockIdx.y / lv.hkv) + e : blockIdx.y / lv.hkv;
  const bool hist = (int)blockIdx.x < a.nsplit;
  const int n = (int)lds32(info + kIPages), all = (int)lds32(info + kILive);
  c.rest = (int)lds32(info + kIRest);
  const NearPages near = {lv, a, c.base, (int)blockIdx.z, h};
  bool ok = !c.failed();
  if (w < kRowWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRows));
    const int live = WIDE ? min(kRows, all - e * kRows) : all, row = threadIdx.x & (kRows - 1);
    if (32 * (w & 3) < live) {
      const float F = __uint_as_float(lds32(c.base + kOffF + 4 * (WIDE ? e * kRows + row : row)));
      // a row whose q is not finite (F is NaN) has NaN weights, whatever the reference: it asks for none
      float m = hist && F != F ? 0.f : -INFINITY, lsum = 0.f;
      if (ok && hist) {
        ok = rows_history<WIDE>(c, e, n, F, m, lsum);
      } else if (ok) {
        const int node = (qt * kRows + row) >> a.gq_log2;
        auto bits = [&](int i) -> unsigned long long {
          const Near p = near(i);
          unsigned long long see = p.rows >= kP ? ~0ull : (1ull << p.rows) - 1ull;
          if (p.draft >= 0) see &= row < live ? a.mask[((size_t)blockIdx.z * a.T + node) * a.W + p.draft] : 0ull;
          return see;
        };
        ok = rows_bf16<WIDE>(c, e, n, F, bits, m, lsum);
      }
      // the stream's last product
      if (WIDE) {
        if (ok && n > 0) ok = c.wait(kBODone + e, n - 1);
      } else {
        if (ok && e < n) ok = c.wait(kBODone + e, (n - 1 - e) >> 1);
      }
      if (!ok) c.fail();
      const float ref = m == -INFINITY ? -INFINITY : hist ? fmaf(m, F, -kBias) : m * F;
      float2 unit = make_float2(1.f, 1.f);
      if (FMT == kFmtU8 && hist) {
        const float* mc = meta_consts(lv, h, OSCAR_KIND_V);
        unit = make_float2(mc[2], mc[6]);
      }
      write_partials<WIDE>(c, lv, a, h, qt, n, live, ref, lsum, unit);
    }
  } else if (w < kVWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsUnpack));
    if (ok) ok = hist ? keys_history<FMT>(c, lv, h, e, n) : keys_bf16(c, lv.status, e, n, near);
  } else if (w < kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsUnpack));
    if (ok) ok = hist ? values_history<FMT>(c, lv, h, e, n) : values_bf16(c, lv.status, e, n, near);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
    if (ok) ok = control<FMT, WIDE>(c, lv, w, h, hist, n, all > kRows);
  }
  if (!ok) {
    if (lane == 0) flag(lv.status, OSCAR_STATUS_TIMEOUT);
    c.fail();
  }
  if (w == kMmaWarp || w == kMmaOWarp) {           // every MMA completes before TMEM is released
    umma_commit_warp(c.bar(kBFinal));
    mbar_wait(c.bar(kBFinal), 0);
    __syncwarp();
  }
  if (w == kLoadWarp && lane == 0 && hist && n > 0 && c.failed()) {
    // copies still in flight land before the CTA leaves: each stage's newest (bounded waits)
    mbar_wait(c.bar(kBImg), 0);
    for (int s = 0; s < kStages; ++s)
      for (int ph = 0; ph < 2; ++ph) mbar_wait(c.bar(kBFull + s), ph);
  }
}

template <int FMT, bool WIDE>
__global__ void __launch_bounds__(kTreeThreads, 1) k_tree_attention(LayerView lv, TreeArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  constexpr int kCtaRows = WIDE ? 2 * kRows : kRows;
  const int slot = blockIdx.x, h = blockIdx.y % lv.hkv, Q0 = (blockIdx.y / lv.hkv) * kCtaRows, b = blockIdx.z;
  const int tid = threadIdx.x, w = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int gq_log2 = a.gq_log2, gq = 1 << gq_log2;
  const bool hist = slot < a.nsplit;
  Ctx c;
  c.base = smem_addr(smem);
  c.rest = 0;
  // the barriers but those whose count depends on the request, before the kernel before this one is waited for
  if (w == kLoadWarp) {
    for (int k = lane; k < kNumBars; k += 32) {
      if (k >= kBSFree && k < kBODone) continue;
      // kBEmpty: a key and a value warpgroup, warp 26; unpacked pages: a warpgroup; kBFinal: both issuing warps
      mbar_init_n(c.bar(k), k >= kBEmpty && k < kBMeta ? 9 : k >= kBKFull && k < kBKFree ? 4 : k == kBFinal ? 2 : 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
    if (lane == 0 && hist) {                       // the rotation; the parameters come from no kernel
      const uint8_t* img = reinterpret_cast<const uint8_t*>(lv.params + (size_t)h * kParamFloats + kRKImgOff);
      mbar_expect_tx(c.bar(kBImg), 2 * kImgBytes);
      for (int p = 0; p < 2; ++p)                  // R = b1 + b2 to 2^-16; the rotated row is rounded to 2^-11 next
        bulk_copy_hint(c.base + kOffK + p * kImgBytes, img + p * kImgBytes, kImgBytes, c.bar(kBImg), l2_evict_last());
    }
    __syncwarp();
  }
  pdl_wait();
  pdl_launch_dependents();

  // ---- the rows' q: a warp takes 8 rows (lane & 7), loaded before anything is known about the request -------------
  constexpr int kStagers = kMmaWarp;               // warps
  auto load_q = [&](int blk, uint4 (&x)[4]) {
    const int Q = Q0 + 8 * blk + (lane & 7), node = Q >> gq_log2, hq = (h << gq_log2) + (Q & (gq - 1));
    const uint4* src = reinterpret_cast<const uint4*>(a.q + (((size_t)b * a.T + node) * lv.hq + hq) * kD);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = node < a.T ? src[(lane >> 3) + 4 * j] : make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 x[4];
  if (w < kStagers && w < kCtaRows / 8) load_q(w, x);
  const int asked = a.n_draft != nullptr ? a.n_draft[b] : a.T;
  int L = a.seq_lens[b];
  const int nodes = min(max(asked, 0), a.T);
  if (asked != nodes && tid == 0 && slot == 0) flag(lv.status, OSCAR_STATUS_BAD_TREE);
  const int live = min(kCtaRows, nodes * gq - Q0);  // this CTA's query rows
  auto leave = [&]() {                             // nothing to do here: the copies requested above land first
    if (w == kLoadWarp && lane == 0 && hist) mbar_wait(c.bar(kBImg), 0);
  };
  if (live <= 0) return leave();

  // ---- the slot's tokens -----------------------------------------------------------------------------------
  if (L < 0) {
    if (tid == 0 && slot == 0) flag(lv.status, OSCAR_STATUS_BAD_SEQLEN);
    L = 0;
  }
  int Lh = max(0, L - lv.sink - lv.recent);
  const int np = tree_pages(lv, a, L);
  if (Lh > np * kP) {
    if (tid == 0 && slot == 0) flag(lv.status, OSCAR_STATUS_BAD_SEQLEN);
    Lh = np * kP;
  }
  int p0, n, seen = 0;                             // first page and number of pages of the slot; draft pages: a bit each
  if (hist) {
    const int slots = tree_hist_slots(a, np);
    if (slot >= slots) return leave();             // a shorter request: the merge knows
    n = tree_div(np, slots);
    p0 = slot * n + min(slot, np - slots * n);
    n += slot < np - slots * n;
  } else {
    // a share of the BF16 and draft pages that hold tokens; of the draft pages those that some row of this CTA sees
    const int held = near_sink(lv, L) + near_recent(lv, L), pages = held + (nodes + kP - 1) / kP;
    p0 = (slot - a.nsplit) * pages / a.nb;
    const int p1 = (slot - a.nsplit + 1) * pages / a.nb, d0 = max(p0 - held, 0), d1 = max(p1 - held, 0);
    const int node = (Q0 >> gq_log2) + tid;
    const bool mine = node <= (Q0 + live - 1) >> gq_log2;
    unsigned long long words[kMaxDraft / kP];
#pragma unroll
    for (int d = 0; d < kMaxDraft / kP; ++d) words[d] = mine && d >= d0 && d < d1 ? a.mask[((size_t)b * a.T + node) * a.W + d] : 0ull;
    n = max(min(p1, held) - p0, 0);
#pragma unroll
    for (int d = 0; d < kMaxDraft / kP; ++d) {
      if (d < d0 || d >= d1) continue;
      const int rows = nodes - d * kP;             // bits from n_draft on are ignored
      if (__syncthreads_or((words[d] & (rows >= kP ? ~0ull : (1ull << rows) - 1ull)) != 0ull)) {
        seen |= 1 << d;
        ++n;
      }
    }
  }

  if (w == kLoadWarp) {
    if (lane < 2) {                                // row warps that have rows, of a stream
      const int active = ((WIDE ? min(kRows, live - lane * kRows) : live) + 31) / 32;
      mbar_init_n(c.bar(kBSFree + lane), max(active, 1));
      mbar_init_n(c.bar(kBPReady + lane), max(active, 1));
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
  } else if (w == kMmaWarp) {
    // only now: the kernel before this one may still have been about to allocate its own
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(c.base + kOffTmem),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (w == kMetaWarp) {
    if (lane == 0) {
      sts32(c.base + kOffFailed, 0u);
      const uint32_t info = c.base + kOffInfo;
      sts32(info + kIPages, (uint32_t)n);
      sts32(info + kIRest, (uint32_t)(Lh - p0 * kP));
      sts32(info + kILive, (uint32_t)live);
    }
    __syncwarp();
  } else if (w >= kKWarp0 && w < kMmaWarp) {
    const int at = tid - 32 * kKWarp0, step = 32 * (kMmaWarp - kKWarp0);
    if (hist) {                                    // page ids, those out of range as -1
      const int* pt = a.hist_pt + (size_t)b * a.max_hist_pages + p0;
      for (int k = at; k < n; k += step) {         // at most kPids, see tree_splits
        int id = __ldg(pt + k);
        if (id < 0 || id >= lv.n_int2) {
          flag(lv.status, OSCAR_STATUS_BAD_PAGE);
          id = -1;
        }
        sts32(c.base + kOffPid + 4 * k, (uint32_t)id);
      }
    } else {                                       // the pages' descriptors and sets of non-finite rows
      for (int k = at; k < n; k += step) {
        const uint2 d = describe_page(lv, a, b, k, n, p0, seen, L, nodes);
        sts32(c.base + kOffNear + 8 * k, d.x);
        sts32(c.base + kOffNear + 8 * k + 4, d.y);
        sts32(c.base + kOffPid + 8 * k, 0u);
        sts32(c.base + kOffPid + 8 * k + 4, 0u);
      }
    }
  }
  // q staged where the values go, the rotation's A operand (BF16 pages: the second tile where it is used); each row's
  // largest magnitude, as bf16 bits, where the join will be
  if (w < kStagers && n > 0) {
#pragma unroll 1
    for (int blk = w; blk < kCtaRows / 8; blk += kStagers) {
      if (blk >= kStagers) load_q(blk, x);
      const int r = 8 * blk + (lane & 7), rr = r & (kRows - 1);
      const uint32_t dst = c.base + (!WIDE || r < kRows ? kOffV : hist ? kOffV + kRows * kD * 2 : kOffQ) +
                           (rr >> 3) * kSboK + (rr & 7) * 16 + (lane >> 3) * 128;
      uint32_t mx = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (r >= live) x[j] = make_uint4(0u, 0u, 0u, 0u);
        mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(x[j].x & 0x7FFF7FFFu, x[j].y & 0x7FFF7FFFu),
                                   __vmaxu2(x[j].z & 0x7FFF7FFFu, x[j].w & 0x7FFF7FFFu)));
        sts128(dst + 4 * j * 128, x[j]);
      }
      mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = __vmaxu2(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      mx = max(mx & 0xffffu, mx >> 16);
      if (lane < 8) {
        sts32(c.base + kOffJoin + 4 * r, mx);
        if (mx >= 0x7F80u) flag(lv.status, OSCAR_STATUS_NONFINITE);
      }
    }
    fence_async();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  bool ok = lds32(c.base + kOffTmem) == c.tmem;

  // ---- the rows' A operand in TMEM (a second tile's in shared memory) -----------------------------------------
  // thread = row; one tile: the second warpgroup takes the upper half of the channels
  const int row = tid & (kRows - 1), half = (tid >> 7) & 1;
  float F = a.scale_log2;
  if (ok && n > 0 && hist) {
    if (w == kLoadWarp) {
      if (lane == 0)
        for (int i = 0; i < min(n, kStages); ++i) issue_page(c, lv, h, i);
      __syncwarp();
    } else if (w == kMmaWarp) {
      ok = c.wait(kBImg, 0);
      if (ok) {
        tc_fence_after();
        const uint32_t a0 = c.base + kOffV, b0 = c.base + kOffK;
#pragma unroll 1
        for (int t = 0; t < (WIDE && live > kRows ? 2 : 1); ++t)
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_warp(c.tmem + kColO + 128 * t, desc_lo(a0, 128) + t * (kRows * kD * 2 / 16) + 16 * kk, desc_hi(kSboK),
                        desc_lo(b0, 16) + (p * kImgBytes + (kk >> 2) * (kImgBytes / 2) + (kk & 3) * 32) / 16,
                        desc_hi(1024, true), kIdescO | kBf16Bits, (p | kk) != 0);
        umma_commit_warp(c.bar(kBQ));
      }
    } else if (w < kRowWarps) {
      // q R_K has no channel above sqrt(128) max |q|, and one above max |q| / sqrt(128): 2^sigma brings that range to
      // 2^7.5 .. 2^14.5, away from both ends of fp16, the type the dequantised keys need (bf16 would keep 8 bits of them)
      const int ex = (int)(lds32(c.base + kOffJoin + 4 * (WIDE ? tid : row)) >> 7), sigma = min(max(137 - ex, -120), 100);
      const float sc = __int_as_float((127 + sigma) << 23);
      F *= __int_as_float((127 - sigma) << 23);
      float unit[2] = {1.f, 1.f};                  // compact format: what the keys of a group are in units of
      if (FMT == kFmtU8) {
        const float* mc = meta_consts(lv, h, OSCAR_KIND_K);
        const float most = fmaxf(mc[2], mc[6]), all = most > 0.f ? most : 1.f;
        unit[0] = mc[2] / all;
        unit[1] = mc[6] / all;
        F *= all;
      }
      ok = c.wait(kBQ, 0);
      if (ok) {
        tc_fence_after();
        const uint32_t trow = c.tmem + ((uint32_t)(32 * (w & 3)) << 16), from = trow + kColO + (WIDE ? 128 * half : 0);
#pragma unroll 1
        for (int k = WIDE ? 0 : 2 * half; k < (WIDE ? 4 : 2 * half + 2); ++k) {
          float y[32];
          tmem_ld32(from + 32 * k, y);
          uint32_t r[16];
          const float u_sc = FMT == kFmtU8 ? sc * (k < 2 ? unit[0] : unit[1]) : sc;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 8; ++j) r[8 * u + j] = pack_f16x2(y[16 * u + j] * u_sc, y[16 * u + 8 + j] * u_sc);
          if (WIDE && half == 1) {
            const uint32_t dst = c.base + kOffQ + (row >> 3) * kSboK + (row & 7) * 16 + 4 * k * 128;
#pragma unroll
            for (int j = 0; j < 4; ++j) sts128(dst + j * 128, make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]));
          } else {
            tmem_st16(trow + kColQ + 16 * k, r);
          }
        }
        tmem_wait_st();
        if (WIDE) fence_async();
      }
    }
  } else if (ok && n > 0 && w >= kKWarp0 && w < kMmaWarp) {
    // the first pages' rows on their way to L2, and their addresses known to the SM, before the unpacking loads them
    const NearPages near = {lv, a, c.base, b, h};
    for (int k = (tid - 32 * kKWarp0) >> 2; k < min(n, kWarm) * 2 * kP; k += 8 * (kMmaWarp - kKWarp0)) {
      const Near p = near(k / (2 * kP));
      const int t = k & (kP - 1);
      const __nv_bfloat16* at = ((k & kP) != 0 ? p.v : p.k) + t * p.step + 32 * (tid & 3);
      if (t < p.rows) asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
    }
  } else if (ok && n > 0 && w < (WIDE ? kRowWarps / 2 : kRowWarps)) {
    const uint32_t trow = c.tmem + ((uint32_t)(32 * (w & 3)) << 16);
    const uint32_t qs = c.base + kOffV + (row >> 3) * kSboK + (row & 7) * 16;
#pragma unroll 1
    for (int k = WIDE ? 0 : 2 * half; k < (WIDE ? 4 : 2 * half + 2); ++k) {
      uint32_t r[16];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 y = lds128(qs + (4 * k + j) * 128);
        r[4 * j] = y.x;
        r[4 * j + 1] = y.y;
        r[4 * j + 2] = y.z;
        r[4 * j + 3] = y.w;
      }
      tmem_st16(trow + kColQ + 16 * k, r);
    }
    tmem_wait_st();
  }
  if (w < kRowWarps && (WIDE || half == 0)) {
    // Not 0, which times a masked logit's -inf would be NaN: a sum of products is below 2^40, so a factor this small or
    // smaller gives weights of exactly 1 either way.
    if (hist) F = fmaxf(F, 1.17549435e-38f);
    // a NaN or infinity in q: the whole row is NaN, as its formula's softmax is
    if (n > 0 && lds32(c.base + kOffJoin + 4 * (WIDE ? tid : row)) >= 0x7F80u) F = NAN;
    sts32(c.base + kOffF + 4 * (WIDE ? tid : row), __float_as_uint(F));
  }
  if (!ok) c.fail();
  tc_fence_before();
  __syncthreads();                                 // Q is in; the rotation's operands may be overwritten
  tc_fence_after();

  // ---- the roles. What they need is read back from shared memory: nothing of the start is kept in registers ----
  run_roles<FMT, WIDE>(lv, a);
  tc_fence_before();
  __syncthreads();
  if (w == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(lds32(c.base + kOffTmem)), "r"(kTmemCols)
                 : "memory");
  }
}

template <int FMT, bool WIDE>
int launch_as(const LayerView& lv, const TreeArgs& a, int B, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  const int tiles = tree_tiles(a.T, lv.hq / lv.hkv);
  cfg.gridDim = dim3(a.nsplit + a.nb, lv.hkv * (WIDE ? (tiles + 1) / 2 : tiles), B);
  cfg.blockDim = dim3(kTreeThreads);
  cfg.dynamicSmemBytes = kTreeSmem<WIDE>;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_tree_attention<FMT, WIDE>, lv, a) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}
template <int FMT>
int launch_fmt(const LayerView& lv, const TreeArgs& a, int B, cudaStream_t st) {
  return tree_wide(a.T, lv.hq / lv.hkv) ? launch_as<FMT, true>(lv, a, B, st) : launch_as<FMT, false>(lv, a, B, st);
}

template <int FMT, bool WIDE>
int configure_as() {
  cudaFuncAttributes at;                           // the register shares assume what the CTA is launched with
  if (cudaFuncGetAttributes(&at, k_tree_attention<FMT, WIDE>) != cudaSuccess) return OSCAR_ERR_CUDA;
  if (at.numRegs < kRegsLaunch) return OSCAR_ERR_UNSUPPORTED;   // a compiler that gives fewer: the shares would wait forever
  if (cudaFuncSetAttribute(k_tree_attention<FMT, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTreeSmem<WIDE>) !=
      cudaSuccess)
    return OSCAR_ERR_CUDA;
  return set_max_shared_carveout(reinterpret_cast<const void*>(k_tree_attention<FMT, WIDE>));
}
template <int FMT>
int configure_fmt() {
  const int rc = configure_as<FMT, false>();
  return rc == OSCAR_OK ? configure_as<FMT, true>() : rc;
}

}  // namespace

// Slots of a query row: the history over nsplit of them, the BF16 and draft pages over nb. One CTA runs on an SM at a
// time; its start (rotation of the rows, first pages) and its end cost about as much as kFixed history pages, a BF16
// page, which is not pipelined as deeply, about as much as kNear. If the CTAs fit the SMs at once, the longest of them is
// the time; else the work of an SM and, since CTAs come whole, one more of the longest. The host knows the page tables'
// width only (a request shorter than that is spread over as many slots as its own pages fill, *pps each), so the time
// counts for kFull with all of several requests as long as the tables are wide, and else with kFill of that. The counts
// of least time win, and of equal ones those with the fewest slots, which the merge reads. (Counting full waves of the
// longest CTA: 4 requests x 5 nodes over 5K-30K tokens 78 us instead of 66, 5 x 60 over 3K-9K 85 instead of 69, 8 x 133
// over 98 80 instead of 61; kFull 1: 95, 86, 60; kFull 0: 2 x 17 over 33K 107 instead of 80.)
// The tensor cores' sums truncate, so an accumulator's error grows with the products summed into it. Measured with equal
// weights over values of one sign, relative to their mean, pages to a slot: 256 0, 512 8e-6, 1,024 2.7e-5, 2,048 1.5e-4,
// 4,096 5e-4 (two tiles, whose streams take every page: 1.3e-3). A slot therefore takes pages for kProducts MMAs of an
// accumulator at most (a history page is 4, a BF16 page 8), as far as max_slots allows.
void tree_splits(int B, int T, int hkv, int gq, int nbf, int max_hist_pages, int sms, int max_slots, int* nsplit,
                 int* nb, int* pps) {
  constexpr double kFixed = 20.0, kNear = 5.0, kFull = 0.35, kFill = 0.75;
  constexpr int kProducts = 1024;
  const int tiles = tree_tiles(T, gq), streams = tree_wide(T, gq) ? 1 : 2;   // that share a slot's pages
  const long units = std::max(1L, (long)B * hkv * (tree_wide(T, gq) ? (tiles + 1) / 2 : tiles));   // B may be 0
  const int near = nbf + (T + kP - 1) / kP, pages = std::max(1, max_hist_pages);
  double best = 0.0;
  *nsplit = *nb = 0;                               // stays 0 when max_slots is too small
  *pps = 1;
  auto parts = [](int n, int most) { return (n + most - 1) / most; };
  const int exact_s = parts(pages, streams * kProducts / 4), exact_m = parts(near, streams * kProducts / 8);
  // at least: a slot's page ids fit shared memory, and what the exact sums take of max_slots
  const int least_s = std::min(exact_s, std::max(parts(pages, kPids), max_slots - exact_m));
  const int least_m = std::min(exact_m, std::max(1, max_slots - least_s));
  // more than four waves of CTAs gain nothing
  const int most_s = std::max(least_s, std::min(pages, (int)std::min<long>(2 * sms, 4 * sms / units + 1)));
  // More slots of the same length cost more, so only counts that shorten the longest are looked at: about 2 sqrt(pages) of
  // each kind. The search runs in every call (one request and kv
  // head over 1,600 pages: 1.5 us with 5 BF16 pages, 6 with 67, 32 with 2,040; all counts: 7, 84 and 2,519).
  auto next = [&](int n, int x) {                  // the next count after x with shorter parts of n; beyond n: none
    const int longest = parts(n, x);
    return longest == 1 ? n + 1 : parts(n, longest - 1);
  };
  for (int m = least_m; m <= near && m < max_slots; m = next(near, m))
    for (int s = least_s; s <= most_s && s + m <= max_slots; s = next(pages, s)) {
      const double h = (pages + s - 1) / s + kFixed, g = kNear * ((near + m - 1) / m) + kFixed, longest = std::max(h, g);
      auto more = [&](double fill) { return units * (fill * s + m) <= sms ? 0.0 : units * (fill * s * h + m * g) / sms; };
      const double cost = longest + (B > 1 ? kFull * more(1.0) + (1.0 - kFull) * more(kFill) : more(1.0)) + 0.1 * (s + m);
      if (best == 0.0 || cost < best) {
        best = cost;
        *nsplit = s;
        *nb = m;
        *pps = (pages + s - 1) / s;
      }
    }
}

int launch_tree_attention(const LayerView& lv, const TreeArgs& a, int B, int sms, cudaStream_t st) {
  const int rc = lv.meta_cb ? launch_fmt<kFmtCB>(lv, a, B, st)
                            : lv.meta_u8 ? launch_fmt<kFmtU8>(lv, a, B, st) : launch_fmt<kFmtF16>(lv, a, B, st);
  return rc == OSCAR_OK ? launch_tree_merge(lv, a, B, sms, st) : rc;
}

int configure_tree_kernels() {
  int rc = configure_tree_merge();
  if (rc == OSCAR_OK) rc = configure_fmt<kFmtF16>();
  if (rc == OSCAR_OK) rc = configure_fmt<kFmtU8>();
  return rc == OSCAR_OK ? configure_fmt<kFmtCB>() : rc;
}

}  // namespace oscar
