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
// Warps: 0-3 and 4-7 rows of the two tiles, 8 loads, 9 issues the products, 10 looks at values that are not finite,
// 11 finds the work, 12-15 write the results: the row threads are at the next item's weights by then.
// TMEM is full: O (2 x 128 columns), S and P (2 x 128).
// Measured: 32,769 tokens, 32 query and 8 key heads, 5.05 to 5.3 ms, 2 prompts of 8,192 with 64 and 8, 1.22 ms (1.74 to 1.66 and
// 1.76 PFLOP/s of products that count): the tensor pipe works in 77 % of the cycles, the rest is the chain of a tile (two times 64
// weights, 1,870 cycles, O of the last 64 and the next S, 768, and three hand-overs), which the other tile covers but for that.
// Halves of S that are asked for by themselves would take the chain apart, but N = 64 takes as long as N = 128 (6.2 ms); a warp
// of its own for each tile's products mixes the tiles' products in the pipe (5.6 ms); logits loaded under the stores of the
// weights before them change nothing. 64 prompts of 1-901 tokens 150 us (0.95 PFLOP/s; 49 %): half of a diagonal block is
// masked, and a tile's first and masked weights and its end cost as much as two more groups of 64. One prompt of 777 tokens
// 15.5 us in a graph: a CTA's chain of up to seven blocks, and the launch.
//
// Work. The grid has a CTA for every item (prompt, key head, two tiles), the long ones of a head first. A CTA that runs
// takes over CTAs that have not started yet (clusterlaunchcontrol), so that the loads and the first S of an item overlap
// the end of the one before it; nothing is counted in memory that calls could share.
//
// Masked places hold whatever the packed buffer holds: logits are replaced by -inf before anything looks at them. Values
// that a row does not see could reach it as 0 times a NaN. So an item with a result that is not finite is done once more, and then
// warp 10 looks at the values that not all rows see before they are used, notes tokens with values that are not finite and
// replaces those values by zeros; rows that do see such a token get its values added to their results, channel by channel, so
// that a value does the same wherever it lies in the item, and nothing to the sum of the weights. (Looking at all items' last
// blocks took a tenth of the time of short prompts.)
#include <algorithm>

#include "quant_tile.cuh"
#include "smem.cuh"

namespace oscar {
namespace {

using qtile::tma_load_3d;

constexpr int kTile = 128;                         // rows of a tile
constexpr int kBlock = 128, kSub = 64;             // tokens of a block, and of what the row threads take at a time
constexpr int kLoadWarp = 8, kMmaWarp = 9, kCheckWarp = 10, kFindWarp = 11, kOutWarp = 12, kWarps = 16;
// registers per thread: at launch, then of the rows' and the other warpgroups; the shares are what the CTA was launched with
constexpr int kRegsLaunch = 128, kRegsRows = 136, kRegsOther = 120;
static_assert(2 * kRegsRows + 2 * kRegsOther <= 4 * kRegsLaunch, "register shares");
// Two pairs of places for a block's keys (0, 2) and values (1, 3), taken in turn.
constexpr int kStages = 4;
constexpr int kHalfBytes = 128 * 128;              // 128 rows of 64 channels, 128-byte swizzle
constexpr int kTileBytes = 2 * kHalfBytes;         // 32 KB: Q of a tile, K or V of a block
constexpr int kOutBytes = 32 * 128;                // a warp's rows on their way out, 128 bytes of each
constexpr int kItems = 3;                          // worked on, loaded, found
constexpr int kNear = 4;                           // blocks before the end of an item's loads at which the next one is looked for
// 64-token groups at an item's end that not all rows see: an item is 2 kTile / gq tokens from a multiple of as many on
constexpr int kMasks = 2 * kTile / kSub;
static_assert(2 * kTile % kSub == 0, "an item of one head begins at a group");
constexpr int kItemMasks = 32, kItemBytes = kItemMasks + 8 * kMasks;   // start, len, h, q0; clean, bad; a bit set of each such group
constexpr int kOffQ = 0, kOffRing = 2 * kTileBytes, kOffOut = kOffRing + kStages * kTileBytes, kOffStat = kOffOut + 4 * kOutBytes,
              kOffItem = kOffStat + 2 * kTile * 8;   // [tile][row] (reference, sum)
constexpr int kOffNext = kOffItem + kItems * kItemBytes;   // the CTA that was taken over, 16 bytes
constexpr int kOffBar = kOffNext + 16;
// two barriers for a tile's weights and products: both halves of a block may be there before the first is used
constexpr int kBFull = 0, kBEmpty = kBFull + kStages, kBQ = kBEmpty + kStages, kBQFree = kBQ + 2, kBS = kBQFree + 2, kBP = kBS + 2,
              kBOFree = kBP + 4, kBStat = kBOFree + 2, kBO = kBStat + 2, kBItem = kBO + 4, kBItemFree = kBItem + kItems,
              kBGo = kBItemFree + kItems, kBCheck = kBGo + 1, kBNear = kBCheck + 1, kBNext = kBNear + 1, kBFinal = kBNext + 1, kNumBars = kBFinal + 1;
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
  float* lse;                                      // [total][hq], or null
  int* status;
  const __nv_bfloat16* v;                          // what the map of v covers
  long long v_token, v_head;
};

struct Item {
  int start, len;                                  // the prompt's tokens
  int h, q0;                                       // key head, first token of the CTA's tiles (len <= q0: nothing to do)
  bool clean;                                      // values that not all rows see are looked at
};

// Item i of prompt-major, then key head, then tiles from the last (which sees most) to the first; one warp. A prompt's
// bounds are taken within [0, total] and in order, whatever cu holds. from, before: the 32 prompts that held the last item
// and the items before them, where the search starts unless i is further in front; once a number was behind the last item,
// the end and all items.
struct Finder {
  int from = 0;
  unsigned before = 0;
};
__device__ __forceinline__ Item find_item(const PromptArgs& a, unsigned i, Finder& f) {
  const int lane = threadIdx.x & 31, tokens = 2 * kTile >> a.gq_log2;
  if (i < f.before) f = Finder();
  Item it = {0, 0, 0, 0, false};
  bool bad = false, found = false;
  unsigned before = f.before;
  for (int c = f.from; c < a.B; c += 32) {
    const int r = min(c + lane, a.B - 1), lo = a.cu[r], hi = a.cu[r + 1];
    const int start = min(max(lo, 0), a.total), end = min(max(hi, start), a.total);
    bad |= start != lo || end != hi;
    const int tiles = c + lane < a.B ? (end - start + tokens - 1) / tokens : 0;
    unsigned sum = (unsigned)tiles * a.hkv;        // below 2^31 in all where the bounds are in order
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, sum, m);
      if (lane >= m) sum += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, i - before < sum);
    if (hit != 0u && !found) {
      const int src = __ffs(hit) - 1, n = __shfl_sync(0xffffffffu, tiles, src);
      const unsigned at = i - before - (__shfl_sync(0xffffffffu, sum, src) - (unsigned)n * a.hkv);
      it.start = __shfl_sync(0xffffffffu, start, src);
      it.len = __shfl_sync(0xffffffffu, end, src) - it.start;
      if (n > 0 && at < (unsigned)n * a.hkv) {
        it.h = at / n;
        it.q0 = (n - 1 - ((int)at - it.h * n)) * tokens;
      } else {
        it.len = 0;
      }
      found = true;
      f.from = c;
      f.before = before;
      if (i != 0) break;                           // the first item's finder looks at all bounds
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  if (!found) {                                    // behind the last item: so are all numbers from `before` on, without a look
    f.from = a.B;
    f.before = before;
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
  // One wait of a whole warp; false (the CTA has failed, or the wait expired) ends its work. The loads' and the finder's waits are
  // bounded in time; the other roles', whose code is to be small, end once one of those has failed (and by their tries).
  __device__ __forceinline__ bool wait(int k, int phase) const {
#pragma unroll 1
    for (unsigned i = 0; !__all_sync(0xffffffffu, mbar_try(bar(k), (uint32_t)phase & 1u)); ++i)
      if (failed() || i == kWaitLimit) return false;
    return true;
  }
  __device__ __forceinline__ bool timed_wait(int k, int phase) const {
    const unsigned long long t0 = global_ns();
#pragma unroll 1
    while (!__all_sync(0xffffffffu, mbar_try(bar(k), (uint32_t)phase & 1u)))
      if (failed() || __any_sync(0xffffffffu, global_ns() - t0 > kWaitNs)) return false;
    return true;
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

// An item as the roles read it; false: there is none any more. The shuffles tell the compiler that a warp's lanes have the same
// numbers.
__device__ __forceinline__ bool read_item(const Ctx c, int slot, Item& it) {
  const uint4 x = lds128(c.base + kOffItem + slot * kItemBytes);
  it.start = __shfl_sync(0xffffffffu, (int)x.x, 0);
  it.len = __shfl_sync(0xffffffffu, (int)x.y, 0);
  it.h = __shfl_sync(0xffffffffu, (int)x.z, 0);
  it.q0 = __shfl_sync(0xffffffffu, (int)x.w, 0);
  it.clean = __shfl_sync(0xffffffffu, (int)lds32(c.base + kOffItem + slot * kItemBytes + 16), 0) != 0;
  return it.len >= 0;
}

// ---- row threads of tile t ------------------------------------------------------------------------------
// What has gone before in this CTA, by which the barriers' phases go.
struct RowCount {
  int s = 0, half0 = 0, half1 = 0, tiles = 0;
  __device__ __forceinline__ int half(int h) const { return h ? half1 : half0; }
};

__device__ __forceinline__ bool rows_item(const Ctx c, const PromptArgs& a, const Item& it, int t, int tokens, RowCount& k) {
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
    if (i >= masked) {
      const int live = token + 1 - i * kSub;       // of the 64 tokens
      if (__any_sync(0xffffffffu, live < 32)) {
#pragma unroll
        for (int x = 0; x < 32; ++x) s0[x] = x < live ? s0[x] : -INFINITY;
      }
#pragma unroll
      for (int x = 0; x < 32; ++x) s1[x] = 32 + x < live ? s1[x] : -INFINITY;
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
        for (int x = 0; x < 32; x += 2) mx4[x >> 1 & 3] = qtile::max3f(mx4[x >> 1 & 3], s0[x], s0[x + 1]);
#pragma unroll
        for (int x = 0; x < 32; x += 2) mx4[x >> 1 & 3] = qtile::max3f(mx4[x >> 1 & 3], s1[x], s1[x + 1]);
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
  k.s += (n + 1) / 2;
  k.half0 += (n + 1) / 2;
  k.half1 += n / 2;
  return true;
}

// ---- values that not all rows see: warp 10 ---------------------------------------------------------------------
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {   // two BF16 values
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xffff0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xffffu;
  return w;
}
// 64 tokens, two a lane: tokens with values that are not finite are noted in the bit set at `mask`, those values replaced by zeros.
__device__ __forceinline__ void clean_values(uint32_t rows, uint32_t mask) {
  const int lane = threadIdx.x & 31;
  const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
  __nv_bfloat162 acc[2][4];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[k][e] = zero;
#pragma unroll
  for (int j = 0; j < 16; ++j)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint4 v = lds128(rows + (j >> 3) * kHalfBytes + (32 * k + lane) * 128 + 16 * ((j ^ lane) & 7));   // no bank conflicts
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[k][e] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]), zero, acc[k][e]);
    }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float2 f = __bfloat1622float2(__hadd2(__hadd2(acc[k][0], acc[k][1]), __hadd2(acc[k][2], acc[k][3])));
    const bool bad = f.x != 0.f || f.y != 0.f;     // 0 times a NaN or an infinity is NaN
    const unsigned set = __ballot_sync(0xffffffffu, bad);
    if (set != 0u) {
      if (lane == 0) sts32(mask + 4 * k, set);
      if (bad)
        for (int j = 0; j < 16; ++j) {
          const uint32_t at = rows + (j >> 3) * kHalfBytes + (32 * k + lane) * 128 + 16 * (j & 7);
          const uint4 v = lds128(at);
          sts128(at, make_uint4(finite_only(v.x), finite_only(v.y), finite_only(v.z), finite_only(v.w)));
        }
      fence_async();
    }
  }
}
__device__ __forceinline__ bool check_item(const Ctx c, const Item& it, int slot, int tokens, int& seen_blocks, int& checked) {
  const int masked = it.q0 / kSub, most = max(c.seen(it, 0, tokens), c.seen(it, 1, tokens));
  const int blocks = (most + kBlock - 1) / kBlock;
#pragma unroll 1
  for (int j = masked / 2; it.clean && j < blocks; ++j) {
    if (!c.wait(kBGo, checked)) return false;      // the values are there, and no product uses them yet
#pragma unroll 1
    for (int i = max(2 * j, masked); i < 2 * j + 2 && i * kSub < most; ++i)
      clean_values(c.base + kOffRing + (2 * ((seen_blocks + j) & 1) + 1) * kTileBytes + (i & 1) * kSub * 128,
                   c.base + kOffItem + slot * kItemBytes + kItemMasks + 8 * (i - masked));
    c.arrive(kBCheck);
    ++checked;
  }
  seen_blocks += blocks;
  return true;
}

// ---- the results: warps 12-15, a quarter of a tile's rows each -----------------------------------------------
struct OutCount {                                  // of a tile
  int half0 = 0, half1 = 0, tiles = 0;
};
// 128 bytes of each row at a time go through shared memory, so that eight lanes write a row's 128 bytes
template <bool FP32>
__device__ __forceinline__ bool out_tile(const Ctx c, const PromptArgs& a, const Item& it, int slot, int t, int tokens, int n,
                                         const OutCount& k) {
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, first = 32 * warp, row = first + lane;
  const uint32_t buf = c.base + kOffOut + warp * kOutBytes, to = c.tmem + ((uint32_t)first << 16) + kColO + 128 * t;
  const int gq = 1 << a.gq_log2, h = (n - 1) & 1;
  if (!c.wait(kBStat + t, k.tiles) || !c.wait(kBO + 2 * t + h, (h ? k.half1 : k.half0) + ((n - 1) >> 1))) return false;
  tc_fence_after();
  const uint2 stat = lds64(c.base + kOffStat + 8 * (t * kTile + row));
  const int token = it.q0 + t * tokens + (row >> a.gq_log2);
  const float l = __uint_as_float(stat.y);
  const float inv = 1.f / l;
  const int left = it.len - it.q0 - t * tokens;    // tokens of the tile
  const long long base = ((long long)(it.start + it.q0 + t * tokens) * a.hq + (it.h << a.gq_log2)) * kD;
  float bad4[4] = {0.f, 0.f, 0.f, 0.f};            // stays 0 while all is finite
  auto write = [&](int q) {                        // 128 bytes of each row
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3), tr = first + r, tok = tr >> a.gq_log2;
      const uint4 x = lds128(buf + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
      if (tok < left) {
        const int at = (tok * a.hq + (tr & (gq - 1))) * kD;   // in the tile
        char* dst = static_cast<char*>(a.out) + (base + at) * (FP32 ? 4 : 2) + 128 * q + 16 * (lane & 7);
        *reinterpret_cast<uint4*>(dst) = x;
      }
    }
    __syncwarp();
  };
  auto free_o = [&] {                              // O and the sums are read: the next item's may be written
    tc_fence_before();
    c.arrive(kBOFree + t);
  };
  if constexpr (FP32) {
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      float o[32];
      tmem_ld32(to + 32 * q, o);
#pragma unroll
      for (int x = 0; x < 32; ++x) {
        o[x] *= inv;
        bad4[x & 3] = fmaf(o[x], 0.f, bad4[x & 3]);
      }
#pragma unroll
      for (int x = 0; x < 8; ++x)
        sts128(buf + lane * 128 + ((x ^ (lane & 7)) << 4), make_uint4(__float_as_uint(o[4 * x]), __float_as_uint(o[4 * x + 1]),
                                                                      __float_as_uint(o[4 * x + 2]), __float_as_uint(o[4 * x + 3])));
      if (q == 3) free_o();
      write(q);
    }
  } else {
#pragma unroll 1
    for (int q = 0; q < 2; ++q) {
#pragma unroll 1
      for (int p = 0; p < 2; ++p) {
        float o[32];
        tmem_ld32(to + 64 * q + 32 * p, o);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t r[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = __fmul2_rn(make_float2(o[8 * x + 2 * e], o[8 * x + 2 * e + 1]), make_float2(inv, inv));
            bad4[e] = fmaf(v.x, 0.f, fmaf(v.y, 0.f, bad4[e]));
            r[e] = pack_bf16x2(v.x, v.y);
          }
          sts128(buf + lane * 128 + (((x + 4 * p) ^ (lane & 7)) << 4), make_uint4(r[0], r[1], r[2], r[3]));
        }
      }
      if (q == 1) free_o();
      write(q);
    }
  }
  if (token < it.len) {
    if (bad4[0] + bad4[1] + bad4[2] + bad4[3] != 0.f) {
      if (it.clean) flag(a.status, OSCAR_STATUS_NONFINITE);
      else sts32(c.base + kOffItem + slot * kItemBytes + 20, 1u);   // once more
    }
    if (a.lse != nullptr)
      a.lse[(long long)(it.start + token) * a.hq + (it.h << a.gq_log2) + (row & (gq - 1))] =
          (__uint_as_float(stat.x) * a.F + log2f(l)) * 0.69314718055994531f;
  }
  return true;
}
template <bool FP32>
__device__ __forceinline__ bool out_item(const Ctx c, const PromptArgs& a, const Item& it, int slot, int tokens, OutCount& k0,
                                         OutCount& k1) {
#pragma unroll 1
  for (int t = 0; t < 2; ++t) {
    const int n = (c.seen(it, t, tokens) + kSub - 1) / kSub;
    if (n == 0) continue;
    OutCount k = t ? k1 : k0;
    if (!out_tile<FP32>(c, a, it, slot, t, tokens, n, k)) return false;
    k.half0 += (n + 1) / 2;
    k.half1 += n / 2;
    ++k.tiles;
    (t ? k1 : k0) = k;
  }
  return true;
}

// Values that were left out of an item's products, into the results of a warp's rows that see them: infinities and NaN, which no
// weight changes. A lane has a channel, and needs the first token of each kind.
template <bool FP32>
__device__ __forceinline__ void add_left_out(const Ctx c, const PromptArgs& a, const Item& it, int slot, int tokens) {
  const int first = threadIdx.x & 96, groups = (min(it.len, it.q0 + 2 * tokens) - it.q0 / kSub * kSub + kSub - 1) / kSub;
  bool any = false;
  __syncwarp();                                    // the rows are written
#pragma unroll 1
  for (int channel = threadIdx.x & 31; channel < kD; channel += 32) {
    int up = it.len, down = it.len, nan = it.len;
#pragma unroll 1
    for (int i = 0; i < 2 * groups; ++i)
#pragma unroll 1
      for (uint32_t set = lds32(c.base + kOffItem + slot * kItemBytes + kItemMasks + 4 * i); set != 0u; set &= set - 1u) {
        const int j = it.q0 / kSub * kSub + 32 * i + __ffs(set) - 1;
        const float v = __bfloat162float(a.v[(it.start + j) * a.v_token + it.h * a.v_head + channel]);
        if (v != v) nan = min(nan, j);
        if (v == INFINITY) up = min(up, j);
        if (v == -INFINITY) down = min(down, j);
      }
    nan = min(nan, max(up, down));
#pragma unroll 1
    for (int r = first; r < 2 * kTile; r += (r & 31) == 31 ? kTile - 31 : 1) {   // rows first .. first + 31 of both tiles
      const int tok = r >> a.gq_log2, token = it.q0 + tok;
      const float v = nan <= token ? NAN : up <= token ? INFINITY : down <= token ? -INFINITY : 0.f;
      if (token >= it.len || v == 0.f) continue;
      any = true;
      const long long at = (((long long)(it.start + token)) * a.hq + (it.h << a.gq_log2) + (r & ((1 << a.gq_log2) - 1))) * kD + channel;
      if constexpr (FP32) {
        static_cast<float*>(a.out)[at] += v;
      } else {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + at;
        *o = __float2bfloat16_rn(__bfloat162float(*o) + v);
      }
    }
  }
  if (any) flag(a.status, OSCAR_STATUS_NONFINITE);
}

// ---- finding ------------------------------------------------------------------------------------------------------
// Each item once, and once more if its results ask for it; the next one is looked for when the loads of the one before near their
// end. (Two found ahead whatever their lengths: CTAs that are done wait for items others hold, 2 x 8K tokens 1.44 ms instead of 1.32.)
__device__ __forceinline__ bool find_role(const Ctx c, const PromptArgs& a, int& asked) {
  const int lane = threadIdx.x & 31;
  Finder f;
  int items = 0, done = 0, near = 0;               // given out; of which the results are known; of which the loads near their end
  unsigned index = blockIdx.x;
  bool more = true, first = true;
  auto wait_near = [&] {                           // a barrier's phases can be told apart only one by one
    for (; near < items; ++near)
      if (!c.timed_wait(kBNear, near)) return false;
    return true;
  };
  for (;;) {
    Item it = {0, -1, 0, 0, false};                // the end
    if (items - done == kItems || (!more && done < items)) {
      const int slot = done % kItems;
      if (!c.timed_wait(kBItemFree + slot, done / kItems)) return false;
      ++done;
      Item old;
      read_item(c, slot, old);
      const bool bad = __shfl_sync(0xffffffffu, (int)lds32(c.base + kOffItem + slot * kItemBytes + 20), 0) != 0;
      if (!bad) continue;
      it = old;
      it.clean = true;
      if (!wait_near()) return false;
    } else if (more) {
      if (!first) {                                // the next CTA that has not started
        if (!wait_near()) return false;
        __syncwarp();                              // the last answer is read
        if (lane == 0) {
          fence_async();
          mbar_expect_tx(c.bar(kBNext), 16);
          asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                           c.base + kOffNext),
                       "r"(c.bar(kBNext))
                       : "memory");
        }
        if (!c.timed_wait(kBNext, asked++)) return false;
        const uint4 x = lds128(c.base + kOffNext);
        uint32_t taken;
        asm volatile(
            "{\n.reg .b128 r;\n.reg .b64 lo, hi;\n.reg .pred p;\nmov.b64 lo, {%2, %3};\nmov.b64 hi, {%4, %5};\nmov.b128 r, {lo, hi};\n"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\nselp.u32 %0, 1, 0, p;\nmov.u32 %1, 0;\n"
            "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}"
            : "=r"(taken), "=r"(index)
            : "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w));
        more = __shfl_sync(0xffffffffu, taken, 0) != 0u;
        if (!more) continue;
      }
      first = false;
      it = find_item(a, index, f);
      if (it.q0 >= it.len) continue;               // the grid holds room for the prompts' last tiles
    }
    const int slot = items % kItems;
    const uint32_t at = c.base + kOffItem + slot * kItemBytes;
    if (lane < 2 * kMasks) sts32(at + kItemMasks + 4 * lane, 0u);
    if (lane == 0) {
      sts128(at, make_uint4((uint32_t)it.start, (uint32_t)it.len, (uint32_t)it.h, (uint32_t)it.q0));
      sts128(at + 16, make_uint4((uint32_t)it.clean, 0u, 0u, 0u));
    }
    c.arrive(kBItem + slot);
    if (it.len < 0) return true;
    ++items;
  }
}

// ---- loading: an item's first keys, Q of its tiles, then values and keys of each block -------------------------
struct LoadCount {
  int items = 0, queries = 0, ring = 0;            // items; loads of Q, of keys and values
};
__device__ __forceinline__ bool load_item(const Ctx c, const Item& it, const CUtensorMap* mq, const CUtensorMap* mk,
                                          const CUtensorMap* mv, int gq_log2, int tokens, LoadCount& k) {
  const uint64_t keep = qtile::l2_evict_normal();
  const int blocks = (max(c.seen(it, 0, tokens), c.seen(it, 1, tokens)) + kBlock - 1) / kBlock;
  // the first keys, Q, then the values and the next keys of each block
#pragma unroll 1
  for (int i = 0; i < 2 * blocks + 2; ++i) {
    const bool query = i == 1 || i == 2;
    const int t = i - 1, x = i == 0 ? 0 : i - 2, s = k.ring % kStages;   // tile; keys or values of block x / 2
    if (query) {
      if (k.items > 0 && !c.timed_wait(kBQFree + t, k.items - 1)) return false;
    } else {
      if (k.ring >= kStages && !c.timed_wait(kBEmpty + s, k.ring / kStages - 1)) return false;
      if (i == 0 ? blocks <= kNear : (x & 1) == 1 && blocks - (x >> 1) - 1 == kNear) c.arrive(kBNear);
    }
    if ((threadIdx.x & 31) == 0) {
      const uint32_t dst = c.base + (query ? kOffQ + t * kTileBytes : kOffRing + s * kTileBytes);
      const uint32_t bar = c.bar(query ? kBQ + t : kBFull + s);
      const CUtensorMap* map = query ? mq : x & 1 ? mv : mk;
      const int head = query ? it.h << gq_log2 : it.h, token = it.start + (query ? it.q0 + t * tokens : (x >> 1) * kBlock);
      mbar_expect_tx(bar, kTileBytes);
#pragma unroll 1
      for (int p = 0; p < 2; ++p) tma_load_3d(dst + p * kHalfBytes, map, 64 * p, head, token, bar, keep);
    }
    k.queries += query;
    k.ring += !query;
    __syncwarp();
  }
  ++k.items;
  return true;
}

// ---- products ---------------------------------------------------------------------------------------------
// One elected lane issues the eight (four) products of a batch from one set of operands: issued one by one in a loop, each
// takes about 90 cycles instead of 64 (2 prompts of 8K: 1.35 ms instead of 1.27). Both tiles in one loop body, places as numbers:
// one copy of the code for each place is 20 % slower on short prompts, one for both tiles 10 % (8 and 4 % on long ones).
// Eight products over 128 channels, A and B in shared memory: one elected lane issues them all (see umma_warp).
__device__ __forceinline__ void umma_channels(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc) {
  asm volatile(
      "{\n.reg .pred p, q, t;\n.reg .b64 a, b;\n.reg .b32 x, y;\nelect.sync _|q, 0xffffffff;\nsetp.ne.u32 p, 0, 0;\nsetp.eq.u32 t, 0, 0;\n"
      "add.u32 x, %1, 0;\nadd.u32 y, %2, 0;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n"
      "add.u32 x, %1, 2;\nadd.u32 y, %2, 2;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      "add.u32 x, %1, 4;\nadd.u32 y, %2, 4;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      "add.u32 x, %1, 6;\nadd.u32 y, %2, 6;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      "add.u32 x, %1, 1024;\nadd.u32 y, %2, 1024;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      "add.u32 x, %1, 1026;\nadd.u32 y, %2, 1026;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      "add.u32 x, %1, 1028;\nadd.u32 y, %2, 1028;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      "add.u32 x, %1, 1030;\nadd.u32 y, %2, 1030;\nmov.b64 a, {x, %3};\nmov.b64 b, {y, %3};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n"
      "}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc)
      : "memory");
}
// Four products over 64 tokens, A in tensor memory.
__device__ __forceinline__ void umma_tokens(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n.reg .pred p, q, t;\n.reg .b64 b;\n.reg .b32 x, y;\nelect.sync _|q, 0xffffffff;\nsetp.ne.u32 p, %5, 0;\nsetp.eq.u32 t, 0, 0;\n"
      "add.u32 x, %1, 0;\nadd.u32 y, %2, 0;\nmov.b64 b, {y, %3};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, p;\n"
      "add.u32 x, %1, 8;\nadd.u32 y, %2, 128;\nmov.b64 b, {y, %3};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n"
      "add.u32 x, %1, 16;\nadd.u32 y, %2, 256;\nmov.b64 b, {y, %3};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n"
      "add.u32 x, %1, 24;\nadd.u32 y, %2, 384;\nmov.b64 b, {y, %3};\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n"
      "}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
// Whether a barrier's phase is over, without waiting as a try does.
__device__ __forceinline__ bool mbar_done(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// What the products need of an item.
struct Work {
  int n0, n1, blocks, checked;                     // 64-token groups of the tiles, blocks, the first block to look at
  bool clean;
  __device__ __forceinline__ Work(const Ctx& c, const Item& it, int tokens)
      : n0((c.seen(it, 0, tokens) + kSub - 1) / kSub), n1((c.seen(it, 1, tokens) + kSub - 1) / kSub),
        blocks((max(n0, n1) + 1) / 2), checked(it.q0 / kBlock), clean(it.clean) {}
};
// In each step and for each tile, O of a block and S of the next one, which may be the next item's first: its logits are
// then there when the rows' threads come to them. (Item by item: 64 prompts of 1-901 tokens 155 us instead of 150.)
__device__ __forceinline__ bool mma_role(const Ctx c, int tokens) {
  int half[2][2] = {{0, 0}, {0, 0}}, tiles[2] = {0, 0}, blocks = 0, looked = 0;   // what has gone before
  Item it;
  if (!c.wait(kBItem, 0)) return false;
  if (!read_item(c, 0, it)) return true;
  Work x(c, it, tokens), y = x;
  bool ahead = false;                              // the item's first S have been issued
#pragma unroll 1
  for (int item = 0;; ++item) {
    bool next = false;
#pragma unroll 1
    for (int j = ahead; j <= x.blocks; ++j)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int b = blocks + j, pk = 2 * (b & 1), pv = 3 - pk;   // places of this block's keys, the last one's values
        const uint32_t ts = c.tmem + kColS + 128 * t, to = c.tmem + kColO + 128 * t;
        if (j > 0) {                               // O of the block before
          // both tiles' wait at once: a wait that is over costs 64 cycles, which the few products in the queue do not cover
          if (t == 0 && !c.wait(kBFull + pv, (b - 1) >> 1)) return false;
#pragma unroll 1
          for (int i = 2 * (j - 1); i < min(t ? x.n1 : x.n0, 2 * j); ++i) {
            const int h = i & 1;
            if (i == 0 && tiles[t] > 0 && !c.wait(kBOFree + t, tiles[t] - 1)) return false;
            if (!c.wait(kBP + 2 * t + h, (h ? half[t][1] : half[t][0]) + (i >> 1))) return false;
            if (x.clean && j - 1 >= x.checked && h == 0 && (t == 0 || x.n0 <= i)) {   // the block's first product
              c.arrive(kBGo);
              if (!c.wait(kBCheck, looked++)) return false;
            }
            tc_fence_after();
            umma_tokens(to, ts + 64 * h, desc_lo(c.base + kOffRing + pv * kTileBytes + h * kSub * 128, kHalfBytes),
                        desc_hi(1024, true), kIdescO, i > 0);
            umma_commit_warp(c.bar(kBO + 2 * t + h));
          }
          if (t == 1) umma_commit_warp(c.bar(kBEmpty + pv));   // both tiles are done with the values
        }
        int n = t ? x.n1 : x.n0, at = j, last = x.blocks - 1;   // S of block `at`
        if (j == x.blocks) {
          if (t == 0) {                            // not waited for: there may be no item until this one's results are known
            const int slot = (item + 1) % kItems;
            next = __all_sync(0xffffffffu, mbar_done(c.bar(kBItem + slot), (uint32_t)((item + 1) / kItems) & 1u)) &&
                   read_item(c, slot, it);
            if (next) y = Work(c, it, tokens);
          }
          if (!next) continue;
          n = t ? y.n1 : y.n0;
          at = 0;
          last = y.blocks - 1;
        }
        // Q is waited for also by a tile without rows: its place is filled again
        if (at == 0 && !c.wait(kBQ + t, item + (j > 0))) return false;
        if (t == 0 && !c.wait(kBFull + pk, b >> 1)) return false;
        if (2 * at < n) {
          tc_fence_after();
          umma_channels(ts, desc_lo(c.base + kOffQ + t * kTileBytes, 16), desc_lo(c.base + kOffRing + pk * kTileBytes, 16),
                        desc_hi(1024, true), kIdescS);
          umma_commit_warp(c.bar(kBS + t));
        }
        if (t == 1) umma_commit_warp(c.bar(kBEmpty + pk));
        if (at == last) umma_commit_warp(c.bar(kBQFree + t));   // the tile's last S
      }
    blocks += x.blocks;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int n = t ? x.n1 : x.n0;
      half[t][0] += (n + 1) / 2;
      half[t][1] += n / 2;
      tiles[t] += n > 0;
    }
    c.arrive(kBItemFree + item % kItems);
    ahead = next;
    if (next) {
      x = y;
      continue;
    }
    const int slot = (item + 1) % kItems;
    if (!c.wait(kBItem + slot, (item + 1) / kItems)) return false;
    if (!read_item(c, slot, it)) return true;
    x = Work(c, it, tokens);
  }
}

template <bool FP32>
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
      mbar_init_n(c.bar(k), k >= kBP && k < kBO ? 4 : k >= kBItemFree && k < kBGo ? 15 : 1);
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
  // Each role walks the items by itself. (One loop around all of them made the products wait for their operands: 32,769
  // tokens 8.1 ms.)
  LoadCount loads;
  int asked = 0;
  if (ok && w == kFindWarp) {
    ok = find_role(c, a, asked);
  } else if (ok && w == kLoadWarp) {
#pragma unroll 1
    for (int i = 0;; ++i) {
      const int slot = i % kItems;
      Item it;
      ok = c.timed_wait(kBItem + slot, i / kItems);
      if (!ok || !read_item(c, slot, it)) break;
      ok = load_item(c, it, &mq, &mk, &mv, a.gq_log2, tokens, loads);
      if (!ok) break;
      c.arrive(kBItemFree + slot);
    }
  } else if (ok && w == kMmaWarp) {
    ok = mma_role(c, tokens);
  } else if (ok && w == kCheckWarp) {
    int checked = 0, seen_blocks = 0;
#pragma unroll 1
    for (int i = 0;; ++i) {
      const int slot = i % kItems;
      Item it;
      ok = c.wait(kBItem + slot, i / kItems);
      if (!ok || !read_item(c, slot, it)) break;
      ok = check_item(c, it, slot, tokens, seen_blocks, checked);
      if (!ok) break;
      c.arrive(kBItemFree + slot);
    }
  } else if (ok && w >= kOutWarp) {
    OutCount results0, results1;
#pragma unroll 1
    for (int i = 0;; ++i) {
      const int slot = i % kItems;
      Item it;
      ok = c.wait(kBItem + slot, i / kItems);
      if (!ok || !read_item(c, slot, it)) break;
      ok = out_item<FP32>(c, a, it, slot, tokens, results0, results1);
      if (!ok) break;
      if (it.clean) add_left_out<FP32>(c, a, it, slot, tokens);
      c.arrive(kBItemFree + slot);
    }
  } else if (ok) {
    RowCount rows;
#pragma unroll 1
    for (int i = 0;; ++i) {
      const int slot = i % kItems;
      Item it;
      ok = c.wait(kBItem + slot, i / kItems);
      if (!ok || !read_item(c, slot, it)) break;
      ok = rows_item(c, a, it, w >> 2, tokens, rows);
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
  if (w == kFindWarp && asked > 0) mbar_wait(c.bar(kBNext), (asked - 1) & 1);   // and every answer and copy lands before the CTA leaves
  if (w == kLoadWarp) {
    for (int t = 0; t < 2; ++t) {
      const int n = (loads.queries + 1 - t) / 2;
      if (n > 0) mbar_wait(c.bar(kBQ + t), (n - 1) & 1);
    }
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
  PromptArgs a = {cu_seqlens, B, total, hq, hkv, 0, sm_scale * kLog2e, out, lse, status,
                  static_cast<const __nv_bfloat16*>(v.ptr), v.token, v.head};
  while (1 << a.gq_log2 < gq) ++a.gq_log2;
  CUtensorMap mq, mk, mv;
  if (!rows_map(&mq, q, hq, total, gq, kTile / gq) || !rows_map(&mk, k, hkv, total, 1, kBlock) ||
      !rows_map(&mv, v, hkv, total, 1, kBlock))
    return OSCAR_ERR_CUDA;
  // a prompt of n tokens has ceil(n / tokens) items a head
  const long long items = hkv * (((long long)total + (long long)B * (tokens - 1)) / tokens);
  if (items >= 1ll << 31) return OSCAR_ERR_UNSUPPORTED;
  const auto kernel = out_dtype == OSCAR_OUT_FP32 ? k_prompt_attention<true> : k_prompt_attention<false>;
  kernel<<<(int)items, 32 * kWarps, kSmem, st>>>(a, mq, mk, mv);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

int configure_prompt_kernel() {
  for (auto fn : {k_prompt_attention<false>, k_prompt_attention<true>}) {
    cudaFuncAttributes at;                         // the register shares assume what the CTA is launched with
    if (cudaFuncGetAttributes(&at, fn) != cudaSuccess) return OSCAR_ERR_CUDA;
    if (at.numRegs < kRegsLaunch) return OSCAR_ERR_UNSUPPORTED;   // a compiler that gives fewer: the shares would wait forever
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) return OSCAR_ERR_CUDA;
    if (int rc = set_max_shared_carveout(reinterpret_cast<const void*>(fn)); rc != OSCAR_OK) return rc;
  }
  return OSCAR_OK;
}

}  // namespace oscar
