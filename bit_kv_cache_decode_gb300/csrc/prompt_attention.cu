// Causal attention over whole prompts, packed one behind the other (sm_103a: tcgen05.mma, TMEM accumulators, TMA).
//
//   o_i = sum_{j <= i} p_ij v_j / sum_j p_ij,  p_ij = 2^(F (q_i . k_j) - m_i),  F = scale log2(e)
//
// for every query head; gq query heads share a key head. A tile is M = 128 rows: 128 / gq tokens times the gq heads of
// a key head, so that short prompts fill tiles too and a tile's diagonal is narrow. A CTA takes two tiles of neighbouring
// tokens and streams the keys and values they see through shared memory, 128 tokens (a block) at a time:
//  * S = Q K^T, M128 N128 K16 x 8, A and B in shared memory, into the tile's 128 TMEM columns;
//  * row threads (thread = row = TMEM lane) turn 64 logits at a time into weights and their sum (float32), rounded once to
//    BF16 and written over their logits. m is a reference near the running maximum, not the maximum: 64 weights that sum
//    to at most 2^10 keep it, others set it to the row's maximum, rescale O and redo the 64. So only few blocks look for a
//    maximum, and O is hardly ever rescaled;
//  * O += P V, M128 N128 K16 x 4 for 64 tokens, A = P in TMEM, B = V as it lies in shared memory (channels contiguous).
// The tensor pipe takes 1,024 cycles for a block of one tile (512 for S, 512 for O); while it works for one tile, the row
// threads of the other have its logits. Products run in issue order, so an S may be issued over weights whose O is issued.
// Warps: 0-3 and 4-7 rows of the two tiles, 8 finds the work and loads, 9 issues the products, 12-15 write the results: the
// row threads are at the next item's weights by then.
// TMEM is full: O (2 x 128 columns), S and P (2 x 128).
//
// Work. The grid has a CTA for every item (prompt, key head, two tiles), the long ones of a head first. A CTA that runs
// takes over CTAs that have not started yet (clusterlaunchcontrol), so that the loads and the first S of an item overlap
// the end of the one before it; nothing is counted in memory that calls could share.
//
// Masked places hold whatever the packed buffer holds: logits are replaced by -inf before anything looks at them. Values
// that some row of the CTA does not see would reach it as 0 times a NaN; before the products of those last blocks the row
// threads look at their values, note rows that are not finite, replace them by zeros, and make the rows that do see them NaN.
#include <algorithm>

#include "quant_tile.cuh"
#include "smem.cuh"

namespace oscar {
namespace {

using qtile::tma_load_3d;

constexpr int kTile = 128;                         // rows of a tile
constexpr int kBlock = 128, kSub = 64;             // tokens of a block, and of what the row threads take at a time
constexpr int kLoadWarp = 8, kMmaWarp = 9, kOutWarp = 12, kWarps = 16;
// registers per thread: at launch, then of the rows' and the other warpgroups; the shares are what the CTA was launched with
constexpr int kRegsLaunch = 128, kRegsRows = 144, kRegsOther = 112;
static_assert(2 * kRegsRows + 2 * kRegsOther <= 4 * kRegsLaunch, "register shares");
constexpr int kStages = 4;                         // ring of blocks: keys and values in turn
constexpr int kHalfBytes = 128 * 128;              // 128 rows of 64 channels, 128-byte swizzle
constexpr int kTileBytes = 2 * kHalfBytes;         // 32 KB: Q of a tile, K or V of a block
constexpr int kOutBytes = 32 * 128;                // a warp's rows on their way out, 128 bytes of each
constexpr int kItems = 3;                          // items found ahead
constexpr int kMasks = 8;                          // 64-token groups at an item's end that not all rows see: 5 at most
constexpr int kItemBytes = 16 + 8 * kMasks;        // start, len, h, q0; a bit set of each such group
constexpr int kOffQ = 0, kOffRing = 2 * kTileBytes, kOffOut = kOffRing + kStages * kTileBytes, kOffStat = kOffOut + 4 * kOutBytes,
              kOffItem = kOffStat + 2 * kTile * 8;   // [tile][row] (reference, sum)
constexpr int kOffNext = kOffItem + kItems * kItemBytes;   // the CTA that was taken over, 16 bytes
constexpr int kOffBar = kOffNext + 16;
// two barriers for a tile's weights and products: both halves of a block may be there before the first is used
constexpr int kBFull = 0, kBEmpty = kBFull + kStages, kBQ = kBEmpty + kStages, kBQFree = kBQ + 1, kBS = kBQFree + 1, kBP = kBS + 2,
              kBC = kBP + 4, kBOFree = kBC + 2, kBStat = kBOFree + 2, kBO = kBStat + 2, kBItem = kBO + 4, kBItemFree = kBItem + kItems,
              kBNext = kBItemFree + kItems, kBFinal = kBNext + 1, kNumBars = kBFinal + 1;
constexpr int kOffTmem = kOffBar + 8 * kNumBars, kOffFailed = kOffTmem + 4;
constexpr int kSmem = kOffFailed + 4 + 1024;       // with alignment slack
static_assert(kOffItem % 16 == 0 && kItemBytes % 16 == 0 && kOffBar % 16 == 0, "alignment");
static_assert(kSmem <= 232448, "shared memory of a CTA");
constexpr uint32_t kColO = 0, kColS = 256, kTmemCols = 512;   // tile t: + 128 t
constexpr uint32_t kBf16Bits = (1u << 7) | (1u << 10);        // A and B bf16
constexpr uint32_t kIdescS = idesc_f16(128, 128) | kBf16Bits, kIdescO = kIdescS | (1u << 16);   // V: channels contiguous
constexpr float kMostSum = 1024.f;

struct PromptArgs {
  const int* cu;
  int B, total, hq, hkv, gq_log2;
  float F;
  void* out;                                       // [total][hq][kD]
  int out_fp32;
  float* lse;                                      // [total][hq], or null
  int* status;
};

struct Item {
  int start, len;                                  // the prompt's tokens
  int h, q0;                                       // key head, first token of the CTA's tiles (len <= q0: nothing to do)
};

// Item i of prompt-major, then key head, then tiles from the last (which sees most) to the first; one warp. A prompt's
// bounds are taken within [0, total] and in order, whatever cu holds.
__device__ __forceinline__ Item find_item(const PromptArgs& a, long long i) {
  const int lane = threadIdx.x & 31, tokens = 2 * kTile >> a.gq_log2;
  long long before = 0;
  bool bad = false;
  Item it = {0, 0, 0, 0};
  bool found = false;
  for (int c = 0; c < a.B; c += 32) {
    const int r = min(c + lane, a.B - 1), lo = a.cu[r], hi = a.cu[r + 1];
    const int start = min(max(lo, 0), a.total), end = min(max(hi, start), a.total);
    bad |= start != lo || end != hi;
    const int tiles = c + lane < a.B ? (end - start + tokens - 1) / tokens : 0;
    long long sum = (long long)tiles * a.hkv;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, sum, m);
      if (lane >= m) sum += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, i < before + sum);
    if (hit != 0u && !found) {
      const int src = __ffs(hit) - 1, n = __shfl_sync(0xffffffffu, tiles, src);
      const long long first = before + __shfl_sync(0xffffffffu, sum, src) - (long long)n * a.hkv;
      it.start = __shfl_sync(0xffffffffu, start, src);
      it.len = __shfl_sync(0xffffffffu, end, src) - it.start;
      const int at = (int)(i - first);
      it.h = at / n;
      it.q0 = (n - 1 - (at - it.h * n)) * tokens;
      found = true;
      if (i != 0) break;                           // the first item's finder looks at all bounds
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  if (i == 0 && __any_sync(0xffffffffu, bad) && lane == 0) flag(a.status, OSCAR_STATUS_BAD_SEQLEN);
  return it;
}

struct Ctx {
  uint32_t base;                                   // shared memory, 1,024-byte aligned
  // all 512 columns are allocated: they start at column 0 (checked)
  static constexpr uint32_t tmem = 0;
  __device__ __forceinline__ uint32_t bar(int k) const { return base + kOffBar + 8u * (uint32_t)k; }
  __device__ __forceinline__ bool failed() const { return lds32(base + kOffFailed) != 0u; }
  __device__ __forceinline__ void fail() const { sts32(base + kOffFailed, 1u); }
  // one wait of a whole warp; false (the CTA has failed, or the wait expired) ends its work
  __device__ __forceinline__ bool wait(int k, int phase) const {
    const uint32_t parity = (uint32_t)phase & 1u;
    bool ok = mbar_try(bar(k), parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    const unsigned long long t0 = global_ns();
#pragma unroll 1
    while (!ok && !failed() && global_ns() - t0 <= kWaitNs) ok = mbar_try(bar(k), parity);
    return __all_sync(0xffffffffu, ok);
  }
  __device__ __forceinline__ void arrive(int k) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar(k));
  }
  // tokens that some row of tile t sees
  __device__ __forceinline__ int seen(const Item& it, int t, int tokens) const {
    return it.q0 + t * tokens >= it.len ? 0 : min(it.len, it.q0 + (t + 1) * tokens);
  }
};

// O of this warp's rows times al
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

// weights of 32 logits as BF16 pairs of neighbouring tokens; their sum is added to t2
__device__ __forceinline__ void weights32(const float (&s)[32], float2 F2, float2 nm2, uint32_t (&r)[16], float2& t2) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 x = __ffma2_rn(make_float2(s[2 * i], s[2 * i + 1]), F2, nm2);
    const float2 v = make_float2(fast_exp2(x.x), fast_exp2(x.y));
    t2 = __fadd2_rn(t2, v);
    r[i] = pack_bf16x2(v.x, v.y);
  }
}

// The values of 64 tokens, two threads a token: rows that are not finite are noted in the mask at `mask` and replaced by
// zeros. Both tiles may look at the same rows: the note stands before the zeros do, and a noted row is zeroed again.
__device__ __forceinline__ void clean_values(uint32_t rows, uint32_t mask) {
  const int x = threadIdx.x & (kTile - 1), row = x >> 1;
  const uint32_t at = rows + (x & 1) * kHalfBytes + row * 128;
  __nv_bfloat162 acc = __floats2bfloat162_rn(0.f, 0.f);
  const __nv_bfloat162 zero = acc;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint4 v = lds128(at + 16 * (j ^ (row & 7)));   // chunks in an order without bank conflicts
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]), zero, acc);
  }
  const float2 f = __bfloat1622float2(acc);
  const uint32_t word = mask + 4 * (row >> 5), bit = 1u << (row & 31);
  const bool bad = f.x != 0.f || f.y != 0.f;         // 0 times a NaN or an infinity is NaN
  if (__any_sync(0xffffffffu, bad || (lds32(mask) | lds32(mask + 4)) != 0u)) {
    if (bad) asm volatile("red.shared.or.b32 [%0], %1;" ::"r"(word), "r"(bit) : "memory");
    __threadfence_block();
    __syncwarp();                                    // a token's two threads are in one warp
    if (lds32(word) & bit) {
#pragma unroll
      for (int j = 0; j < 8; ++j) sts128(at + 16 * j, make_uint4(0u, 0u, 0u, 0u));
    }
    fence_async();
  }
}

// An item as the roles read it; false: there is none any more. The shuffles tell the compiler that a warp's lanes have the same
// numbers: operands of products that follow from them stay in uniform registers (without: 32,769 tokens 8.1 ms instead of ITEM_MS).
__device__ __forceinline__ bool read_item(const Ctx c, int slot, Item& it) {
  const uint4 x = lds128(c.base + kOffItem + slot * kItemBytes);
  it.start = __shfl_sync(0xffffffffu, (int)x.x, 0);
  it.len = __shfl_sync(0xffffffffu, (int)x.y, 0);
  it.h = __shfl_sync(0xffffffffu, (int)x.z, 0);
  it.q0 = __shfl_sync(0xffffffffu, (int)x.w, 0);
  return it.len >= 0;
}

// ---- row threads of tile t ------------------------------------------------------------------------------
// What has gone before in this CTA, by which the barriers' phases go.
struct RowCount {
  int s = 0, half0 = 0, half1 = 0, cleaned = 0, ring = 0, tiles = 0;
  __device__ __forceinline__ int half(int h) const { return h ? half1 : half0; }
};

__device__ __forceinline__ bool rows_item(const Ctx c, const PromptArgs& a, const Item& it, int slot, int t, int tokens,
                                          RowCount& k) {
  const int row = threadIdx.x & (kTile - 1), w = (threadIdx.x >> 5) & 3;
  const uint32_t lane0 = (uint32_t)(32 * w) << 16, to = c.tmem + lane0 + kColO + 128 * t, ts = c.tmem + lane0 + kColS + 128 * t;
  const int token = it.q0 + t * tokens + (row >> a.gq_log2);
  const int n = (c.seen(it, t, tokens) + kSub - 1) / kSub, masked = it.q0 / kSub;   // from group `masked` on not all rows see all
  float m = -INFINITY, l = 0.f;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    if (!(i & 1)) {
      if (!c.wait(kBS + t, k.s + (i >> 1))) return false;
      tc_fence_after();
    }
    float s0[32], s1[32];
    const uint32_t at = ts + 64 * (i & 1);
    tmem_ld32x2(at, at + 32, s0, s1);
    const int live = token + 1 - i * kSub;         // of the 64 tokens
    if (i >= masked) {
#pragma unroll
      for (int x = 0; x < 32; ++x) {
        s0[x] = x < live ? s0[x] : -INFINITY;
        s1[x] = 32 + x < live ? s1[x] : -INFINITY;
      }
    }
    uint32_t r0[16], r1[16];
    float sum = 0.f;
    bool redo = __any_sync(0xffffffffu, m == -INFINITY);
    // Twice at most: the first pass may be for a row of the warp that has no reference yet while the others keep theirs,
    // so its sums are looked at like any other's; what they raise in the second pass is at the rows' maxima.
#pragma unroll 1
    for (int pass = 0;; ++pass) {
      if (redo) {
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < 32; ++x) mx4[x & 3] = qtile::max3f(mx4[x & 3], s0[x], s1[x]);
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        float al = 1.f;
        if ((m == -INFINITY || sum > kMostSum) && mx > m) {
          al = m == -INFINITY ? 0.f : exp2f((m - mx) * a.F);
          m = mx;
        }
        l *= al;
        if (i > 0) {
          const int h = (i - 1) & 1;
          if (!c.wait(kBO + 2 * t + h, k.half(h) + ((i - 1) >> 1))) return false;
          tc_fence_after();
          rescale_o(to, al);
        }
      }
      const float mF = m == -INFINITY ? 0.f : m * a.F;
      const float2 F2 = make_float2(a.F, a.F), nm2 = make_float2(-mF, -mF);
      float2 t2 = make_float2(0.f, 0.f);
      weights32(s0, F2, nm2, r0, t2);
      weights32(s1, F2, nm2, r1, t2);
      sum = t2.x + t2.y;
      if (pass > 0) break;
      if (redo && sum != sum && m == -INFINITY) m = 0.f;   // a row of NaN logits asks for no more references
      redo = __any_sync(0xffffffffu, sum > kMostSum);
      if (!redo) break;
    }
    l += sum;
    tmem_st16(at, r0);
    tmem_st16(at + 16, r1);
    if (i >= masked) {
      const int v = k.ring + (i >> 1) * 2 + 1;     // the block's values in the ring
      if (!c.wait(kBFull + v % kStages, v / kStages)) return false;
      const uint32_t mask = c.base + kOffItem + slot * kItemBytes + 16 + 8 * (i - masked);
      clean_values(c.base + kOffRing + (v % kStages) * kTileBytes + (i & 1) * kSub * 128, mask);
      c.arrive(kBC + t);                           // all four warps have looked
      if (!c.wait(kBC + t, k.cleaned + i - masked)) return false;
      const uint2 bad = lds64(mask);
      const uint32_t lo = live >= 32 ? ~0u : live <= 0 ? 0u : (1u << live) - 1u;
      const uint32_t hi = live >= 64 ? ~0u : live <= 32 ? 0u : (1u << (live - 32)) - 1u;
      if ((bad.x & lo) | (bad.y & hi)) l = NAN;
    }
    tmem_wait_st();
    tc_fence_before();
    c.arrive(kBP + 2 * t + (i & 1));
  }
  if (n > 0) {
    if (k.tiles > 0 && !c.wait(kBOFree + t, k.tiles - 1)) return false;   // the last item's sums are read
    const uint32_t stat = c.base + kOffStat + 8 * (t * kTile + row);
    sts32(stat, __float_as_uint(m));
    sts32(stat + 4, __float_as_uint(l));
    c.arrive(kBStat + t);
    ++k.tiles;
  }
  const int most = max(c.seen(it, 0, tokens), c.seen(it, 1, tokens));
  k.s += (n + 1) / 2;
  k.half0 += (n + 1) / 2;
  k.half1 += n / 2;
  k.cleaned += max(n - masked, 0);
  k.ring += 2 * ((most + kBlock - 1) / kBlock);
  return true;
}

// ---- the results: warps 12-15, a quarter of a tile's rows each -----------------------------------------------
struct OutCount {
  int half[2][2] = {{0, 0}, {0, 0}}, tiles[2] = {0, 0};
};
// 128 bytes of each row at a time go through shared memory, so that eight lanes write a row's 128 bytes
__device__ __forceinline__ bool out_tile(const Ctx c, const PromptArgs& a, const Item& it, int t, int tokens, int n, OutCount& k) {
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, first = 32 * warp, row = first + lane;
  const uint32_t buf = c.base + kOffOut + warp * kOutBytes, to = c.tmem + ((uint32_t)first << 16) + kColO + 128 * t;
  const int gq = 1 << a.gq_log2, chunks = a.out_fp32 ? 4 : 2, h = (n - 1) & 1;
  if (!c.wait(kBStat + t, k.tiles[t]) || !c.wait(kBO + 2 * t + h, (h ? k.half[t][1] : k.half[t][0]) + ((n - 1) >> 1))) return false;
  tc_fence_after();
  const uint2 stat = lds64(c.base + kOffStat + 8 * (t * kTile + row));
  const float l = __uint_as_float(stat.y), inv = 1.f / l;
  float bad = 0.f;
#pragma unroll 1
  for (int q = 0; q < chunks; ++q) {
    if (a.out_fp32) {
      float o[32];
      tmem_ld32(to + 32 * q, o);
#pragma unroll
      for (int x = 0; x < 32; ++x) {
        o[x] *= inv;
        bad = fmaf(o[x], 0.f, bad);
      }
#pragma unroll
      for (int x = 0; x < 8; ++x)
        sts128(buf + lane * 128 + ((x ^ (lane & 7)) << 4), make_uint4(__float_as_uint(o[4 * x]), __float_as_uint(o[4 * x + 1]),
                                                                      __float_as_uint(o[4 * x + 2]), __float_as_uint(o[4 * x + 3])));
    } else {
#pragma unroll 1
      for (int p = 0; p < 2; ++p) {
        float o[32];
        tmem_ld32(to + 64 * q + 32 * p, o);
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          o[x] *= inv;
          bad = fmaf(o[x], 0.f, bad);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
          sts128(buf + lane * 128 + (((x + 4 * p) ^ (lane & 7)) << 4),
                 make_uint4(pack_bf16x2(o[8 * x], o[8 * x + 1]), pack_bf16x2(o[8 * x + 2], o[8 * x + 3]),
                            pack_bf16x2(o[8 * x + 4], o[8 * x + 5]), pack_bf16x2(o[8 * x + 6], o[8 * x + 7])));
      }
    }
    if (q == chunks - 1) {                         // O and the sums are read: the next item's may be written
      tc_fence_before();
      c.arrive(kBOFree + t);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3), tr = first + r, token = it.q0 + t * tokens + (tr >> a.gq_log2);
      const uint4 x = lds128(buf + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
      if (token < it.len) {
        const long long at = (long long)(it.start + token) * a.hq + (it.h << a.gq_log2) + (tr & (gq - 1));
        char* dst = static_cast<char*>(a.out) + at * (a.out_fp32 ? 4 * kD : 2 * kD) + 128 * q + 16 * (lane & 7);
        *reinterpret_cast<uint4*>(dst) = x;
      }
    }
    __syncwarp();
  }
  const int token = it.q0 + t * tokens + (row >> a.gq_log2);
  if (token < it.len) {
    if (bad != 0.f) flag(a.status, OSCAR_STATUS_NONFINITE);
    if (a.lse != nullptr)
      a.lse[(long long)(it.start + token) * a.hq + (it.h << a.gq_log2) + (row & (gq - 1))] =
          (__uint_as_float(stat.x) * a.F + log2f(l)) * 0.69314718055994531f;
  }
  return true;
}
__device__ __forceinline__ bool out_item(const Ctx c, const PromptArgs& a, const Item& it, int tokens, OutCount& k) {
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int n = (c.seen(it, t, tokens) + kSub - 1) / kSub;
    if (n == 0) continue;
    if (!out_tile(c, a, it, t, tokens, n, k)) return false;
    k.half[t][0] += (n + 1) / 2;
    k.half[t][1] += n / 2;
    ++k.tiles[t];
  }
  return true;
}

// ---- finding and loading: an item's first keys, Q of its tiles, then values and keys of each block ------------
struct LoadCount {
  int ring = 0, items = 0, asked = 0;
};
__device__ __forceinline__ bool load_block(const Ctx c, const Item& it, const CUtensorMap* map, int j, LoadCount& k, uint64_t keep) {
  const int s = k.ring % kStages;
  if (k.ring >= kStages && !c.wait(kBEmpty + s, k.ring / kStages - 1)) return false;
  if ((threadIdx.x & 31) == 0) {
    const uint32_t dst = c.base + kOffRing + s * kTileBytes;
    mbar_expect_tx(c.bar(kBFull + s), kTileBytes);
    for (int p = 0; p < 2; ++p)
      tma_load_3d(dst + p * kHalfBytes, map, 64 * p, it.h, it.start + j * kBlock, c.bar(kBFull + s), keep);
  }
  ++k.ring;
  __syncwarp();
  return true;
}
__device__ __forceinline__ bool load_role(const Ctx c, const PromptArgs& a, const CUtensorMap* mq, const CUtensorMap* mk,
                                          const CUtensorMap* mv, int tokens, LoadCount& k) {
  const uint64_t keep = qtile::l2_evict_normal();
  const int lane = threadIdx.x & 31;
  unsigned index = blockIdx.x;
  for (bool more = true; more;) {
    __syncwarp();                                  // the last answer is read
    if (lane == 0) {                               // ask for the CTA after this one
      fence_async();
      mbar_expect_tx(c.bar(kBNext), 16);
      asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                       c.base + kOffNext),
                   "r"(c.bar(kBNext))
                   : "memory");
    }
    ++k.asked;
    const Item it = find_item(a, index);
    if (it.q0 < it.len) {                          // the grid holds room for the prompts' last tiles
      const int slot = k.items % kItems;
      if (k.items >= kItems && !c.wait(kBItemFree + slot, k.items / kItems - 1)) return false;
      const uint32_t at = c.base + kOffItem + slot * kItemBytes;
      if (lane < 2 * kMasks) sts32(at + 16 + 4 * lane, 0u);
      if (lane == 0) sts128(at, make_uint4((uint32_t)it.start, (uint32_t)it.len, (uint32_t)it.h, (uint32_t)it.q0));
      c.arrive(kBItem + slot);
      const int blocks = (max(c.seen(it, 0, tokens), c.seen(it, 1, tokens)) + kBlock - 1) / kBlock;
      if (!load_block(c, it, mk, 0, k, keep)) return false;
      if (k.items > 0 && !c.wait(kBQFree, k.items - 1)) return false;
      if (lane == 0) {
        mbar_expect_tx(c.bar(kBQ), 2 * kTileBytes);
        for (int t = 0; t < 2; ++t)
          for (int p = 0; p < 2; ++p)
            tma_load_3d(c.base + kOffQ + t * kTileBytes + p * kHalfBytes, mq, 64 * p, it.h << a.gq_log2,
                        it.start + it.q0 + t * tokens, c.bar(kBQ), keep);
      }
      __syncwarp();
      ++k.items;
#pragma unroll 1
      for (int j = 0; j < blocks; ++j) {
        if (!load_block(c, it, mv, j, k, keep)) return false;
        if (j + 1 < blocks && !load_block(c, it, mk, j + 1, k, keep)) return false;
      }
    }
    if (!c.wait(kBNext, k.asked - 1)) return false;
    const uint4 x = lds128(c.base + kOffNext);
    uint32_t taken;
    asm volatile(
        "{\n.reg .b128 r;\n.reg .b64 lo, hi;\n.reg .pred p;\nmov.b64 lo, {%2, %3};\nmov.b64 hi, {%4, %5};\nmov.b128 r, {lo, hi};\n"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\nselp.u32 %0, 1, 0, p;\nmov.u32 %1, 0;\n"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}"
        : "=r"(taken), "=r"(index)
        : "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w));
    more = taken != 0u;
  }
  const int slot = k.items % kItems;               // no more items
  if (k.items >= kItems && !c.wait(kBItemFree + slot, k.items / kItems - 1)) return false;
  if (lane == 0) sts32(c.base + kOffItem + slot * kItemBytes + 4, 0xffffffffu);
  c.arrive(kBItem + slot);
  return true;
}

// ---- products ---------------------------------------------------------------------------------------------
struct MmaCount {
  int half[2][2] = {{0, 0}, {0, 0}}, tiles[2] = {0, 0}, ring = 0;
};
__device__ __forceinline__ bool mma_item(const Ctx c, const Item& it, int tokens, int items, MmaCount& k) {
  const int n0 = (c.seen(it, 0, tokens) + kSub - 1) / kSub, n1 = (c.seen(it, 1, tokens) + kSub - 1) / kSub;
  const int blocks = (max(n0, n1) + 1) / 2;
  if (!c.wait(kBQ, items)) return false;
#pragma unroll 1
  for (int j = 0; j <= blocks; ++j)
#pragma unroll 1
    for (int t = 0; t < 2; ++t) {
      const int n = t ? n1 : n0;
      const uint32_t ts = c.tmem + kColS + 128 * t, to = c.tmem + kColO + 128 * t;
      const int tiles = t ? k.tiles[1] : k.tiles[0], h0 = t ? k.half[1][0] : k.half[0][0], h1 = t ? k.half[1][1] : k.half[0][1];
      const int kk0 = k.ring + 2 * j, vv0 = kk0 - 1;   // this block's keys and the last one's values in the ring
#pragma unroll 1
      for (int i = 2 * (j - 1); i >= 0 && i < min(n, 2 * j); ++i) {   // O of the block before
        if (i == 0 && tiles > 0 && !c.wait(kBOFree + t, tiles - 1)) return false;
        if (!c.wait(kBFull + vv0 % kStages, vv0 / kStages) || !c.wait(kBP + 2 * t + (i & 1), (i & 1 ? h1 : h0) + (i >> 1))) return false;
        tc_fence_after();
        const uint32_t v = desc_lo(c.base + kOffRing + (vv0 % kStages) * kTileBytes + (i & 1) * kSub * 128, kHalfBytes);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_ta_warp(to, ts + 64 * (i & 1) + 8 * kk, v + kk * (16 * 128 / 16), desc_hi(1024, true), kIdescO, i > 0 || kk > 0);
        umma_commit_warp(c.bar(kBO + 2 * t + (i & 1)));
      }
      if (j > 0 && t == 1) umma_commit_warp(c.bar(kBEmpty + vv0 % kStages));   // both tiles are done with the values
      if (2 * j < n) {                             // S of this one
        if (!c.wait(kBFull + kk0 % kStages, kk0 / kStages)) return false;
        tc_fence_after();
        const uint32_t q = desc_lo(c.base + kOffQ + t * kTileBytes, 16);
        const uint32_t key = desc_lo(c.base + kOffRing + (kk0 % kStages) * kTileBytes, 16);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t step = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) / 16;
          umma_warp(ts, q + step, desc_hi(1024, true), key + step, desc_hi(1024, true), kIdescS, kk > 0);
        }
        umma_commit_warp(c.bar(kBS + t));
      }
      if (j < blocks && t == 1) umma_commit_warp(c.bar(kBEmpty + kk0 % kStages));
      if (j == blocks - 1 && t == 1) umma_commit_warp(c.bar(kBQFree));
    }
  k.ring += 2 * blocks;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int n = t ? n1 : n0;
    k.half[t][0] += (n + 1) / 2;
    k.half[t][1] += n / 2;
    k.tiles[t] += n > 0;
  }
  return true;
}

__global__ void __launch_bounds__(32 * kWarps, 1)
    k_prompt_attention(PromptArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Ctx c;
  c.base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int tid = threadIdx.x, w = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int tokens = kTile >> a.gq_log2;           // of a tile
  if (w == kLoadWarp) {
    for (int k = lane; k < kNumBars; k += 32)
      mbar_init_n(c.bar(k), k >= kBP && k < kBO ? 4 : k >= kBItemFree && k < kBNext ? 13 : 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (lane == 0) sts32(c.base + kOffFailed, 0u);
  } else if (w == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(c.base + kOffTmem),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  bool ok = lds32(c.base + kOffTmem) == c.tmem;
  if (w < kLoadWarp) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRows));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
  LoadCount loads;
  if (ok && w == kLoadWarp) {
    ok = load_role(c, a, &mq, &mk, &mv, tokens, loads);
  } else if (ok && w == kMmaWarp) {
    MmaCount products;
#pragma unroll 1
    for (int i = 0;; ++i) {
      const int slot = i % kItems;
      Item it;
      ok = c.wait(kBItem + slot, i / kItems);
      if (!ok || !read_item(c, slot, it)) break;
      ok = mma_item(c, it, tokens, i, products);
      if (!ok) break;
      c.arrive(kBItemFree + slot);
    }
  } else if (ok && w >= kOutWarp) {
    OutCount results;
#pragma unroll 1
    for (int i = 0;; ++i) {
      const int slot = i % kItems;
      Item it;
      ok = c.wait(kBItem + slot, i / kItems);
      if (!ok || !read_item(c, slot, it)) break;
      ok = out_item(c, a, it, tokens, results);
      if (!ok) break;
      c.arrive(kBItemFree + slot);
    }
  } else if (ok && w < kLoadWarp) {
    RowCount rows;
#pragma unroll 1
    for (int i = 0;; ++i) {
      const int slot = i % kItems;
      Item it;
      ok = c.wait(kBItem + slot, i / kItems);
      if (!ok || !read_item(c, slot, it)) break;
      ok = rows_item(c, a, it, slot, w >> 2, tokens, rows);
      if (!ok) break;
      c.arrive(kBItemFree + slot);
    }
  }
  if (!ok) {
    if (lane == 0) flag(a.status, OSCAR_STATUS_TIMEOUT);
    c.fail();
  }
  if (w == kMmaWarp) {                             // every MMA completes before TMEM is released
    umma_commit_warp(c.bar(kBFinal));
    mbar_wait(c.bar(kBFinal), 0);
  }
  if (w == kLoadWarp) {                            // and every copy and answer lands before the CTA leaves
    if (loads.asked > 0) mbar_wait(c.bar(kBNext), (loads.asked - 1) & 1);
    if (loads.items > 0) mbar_wait(c.bar(kBQ), (loads.items - 1) & 1);
    for (int i = max(0, loads.ring - kStages); i < loads.ring; ++i) mbar_wait(c.bar(kBFull + i % kStages), (i / kStages) & 1);
  }
  tc_fence_before();
  __syncthreads();
  if (w == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(lds32(c.base + kOffTmem)), "r"(kTmemCols)
                 : "memory");
  }
}

// [tokens][heads][128] bf16 with free token and head strides as a 3-D tensor (channel, head, token); boxes of 64 channels x
// `heads_box` heads x `tokens_box` tokens land 128-byte swizzled, a token's heads one behind the other; tokens past the end
// read as zero
bool rows_map(CUtensorMap* map, const oscar_heads& x, int heads, int total, int heads_box, int tokens_box) {
  qtile::EncodeTiledFn enc = qtile::encode_tiled();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)heads, (cuuint64_t)total};
  const cuuint64_t strides[2] = {(cuuint64_t)x.head * 2, (cuuint64_t)x.token * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)heads_box, (cuuint32_t)tokens_box};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x.ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int launch_prompt_attention(int hq, int hkv, int B, const oscar_heads& q, const oscar_heads& k, const oscar_heads& v,
                            const int* cu_seqlens, int total, float sm_scale, void* out, int out_dtype, float* lse, int* status,
                            cudaStream_t st) {
  const int gq = hq / hkv, tokens = 2 * kTile / gq;
  PromptArgs a = {cu_seqlens, B, total, hq, hkv, 0, sm_scale * kLog2e, out, out_dtype == OSCAR_OUT_FP32, lse, status};
  while (1 << a.gq_log2 < gq) ++a.gq_log2;
  CUtensorMap mq, mk, mv;
  if (!rows_map(&mq, q, hq, total, gq, kTile / gq) || !rows_map(&mk, k, hkv, total, 1, kBlock) ||
      !rows_map(&mv, v, hkv, total, 1, kBlock))
    return OSCAR_ERR_CUDA;
  // a prompt of n tokens has ceil(n / tokens) items a head
  const long long items = hkv * (((long long)total + (long long)B * (tokens - 1)) / tokens);
  if (items >= 1ll << 31) return OSCAR_ERR_UNSUPPORTED;
  k_prompt_attention<<<(int)items, 32 * kWarps, kSmem, st>>>(a, mq, mk, mv);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

int configure_prompt_kernel() {
  cudaFuncAttributes at;                           // the register shares assume what the CTA is launched with
  if (cudaFuncGetAttributes(&at, k_prompt_attention) != cudaSuccess) return OSCAR_ERR_CUDA;
  if (at.numRegs < kRegsLaunch) return OSCAR_ERR_UNSUPPORTED;   // a compiler that gives fewer: the shares would wait forever
  if (cudaFuncSetAttribute(k_prompt_attention, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
    return OSCAR_ERR_CUDA;
  return set_max_shared_carveout(reinterpret_cast<const void*>(k_prompt_attention));
}

}  // namespace oscar
