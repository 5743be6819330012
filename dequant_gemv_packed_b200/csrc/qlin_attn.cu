// qlin_attn_decode: attention of one new token per sequence over the paged,
// quantised key/value cache (layout in qlin_kv.cuh).
//
// Mathematics.  With the codes q, scales s and zeros z of a token t and a query x
// (rotated once, fp16),
//   score_t = c s_k (sum_d q_k x - z_k sum_d x),   c = scale log2(e),
//   out_d   = sum_t w_t s_v (q_v - z_v) / sum_t w_t,   w_t = 2^(score_t - m).
// Scores of 4- and 8-bit keys are integer products, m16n8k32 of u8 codes and s8
// digits: per query and group x is xi 2^(E-21), E the exponent of the largest
// |x|, xi = 2^16 hi + 2^8 mid + lo (fp16 values within a factor 2^11 of the largest
// are exact, others rounded at 2^-22 of it, the rounding of an fp32 sum); each digit's
// sum of products and sum xi are exact in int32, and the digits' sums meet in fp32.
// Two digits, 2^-14 of the largest, would lose the small channels of a query with a large
// one and move every output by 0.8e-4; the third costs four products a tile and group: 32 x
// 8,000 tokens take 62.9 us at 4 bits and 57.0 with two, and at 8 bits, where HBM binds, 88.7
// and 88.3.  The codes are the operand as stored (8 bits) or masked in place (4 bits; the odd
// codes are 16 q in accumulators of their own).
// Values: a nibble or byte masked into the low bits of an fp16 word is the
// subnormal fp16 number q 2^-24 (a nibble at bits 4-7: q 2^-20), and one packed
// multiplication makes a pair q 2^-9, exact.  (The subnormals would be exact
// operands too, but the tensor cores align products by the operands' exponent
// fields: their sums were off by 2^-16 of the products.)  The value's scale joins
// the exponent, P_t = 2^(score_t + log2 s_v - m) = w_t s_v, so that
//   out_d = (sum_t P_t q_v - z_v P_t) / sum_t P_t / s_v,
// and m follows the maximum of score + log2 s_v: P is the weight that the sum is
// really made of, whatever the sizes of the scales.  m is kept 7 to 15 binary orders
// below the maximum (4 to 12 where lo 2^15 has to stay within fp16) and moved only when
// a score exceeds it by 15 (12), which a vote decides: after the first tile that is rare.
//
// The eight columns of the products.  S^T = K Q^T has the tile's 16 tokens as rows,
// O^T = V^T P^T 16 dimensions; lane (g, t) of an accumulator has columns 2t, 2t + 1.
// Up to four queries (NT = 1): the columns are (query, digit) pairs in both (the keys'
// lowest digits take a second set, every other column unused), so a lane has the scores of
// query t for tokens g and g + 8 (none is padding at the usual four queries a key), and P
// enters the value sums as two fp16 digits, hi + 2^-11 lo (22 bits), packed as they are.
// Five to eight queries (NT = 2): the keys' products take two sets of (query, digit)
// columns and one of the eight lowest digits (16-bit keys: one set of eight queries), with
// queries 2t and 2t + 1 in lane t, and the columns of the value sums are the eight queries:
// P's two digits, hi = fp16(P) and lo = P - hi, take a product each into the same sums.  hi meets
// the codes as q 2^-9; lo, times 2^15, meets them as masked, q 2^-24 (nibbles at bits 4-7: lo 2^11
// and q 2^-20; the last bits that subnormal operands cost lie far below hi's).  Scaled, lo stays
// clear of fp16's own subnormals, and a small weight keeps its bits down to 2^-40 of the largest;
// unscaled it ended at 2^-32, too little where the largest is a token with a scale 2^20 times the
// others' and zeros in some dimensions.  One digit, 11 bits, would move every output by 1.2e-4.
// 24 x 9000 tokens of 8 kv heads at 4 bits take 75.3 us, 73.4 with lo unscaled, 70.0 with one digit.
// In both movmatrix turns the packed pair into the next product's operand, and a
// query's statistics live in the lanes that scale its sums.  More than eight queries
// take another pass over the cache.
//
// Split.  A tile is 16 tokens of one (sequence, kv head, block of queries), an item
// all tiles of one.  Items in order, each its tiles plus a constant for what an item
// costs beside them, are cut into equal shares, one a team of warps, whatever the
// lengths (which only the device knows).  If some item has more than kWholeTiles
// tiles, the eight (or four) warps of a CTA are a team and items are cut; each team
// writes its piece of a cut item to the workspace (at most two: its first and last)
// and the team of an item's first piece a record of it, and a dependent kernel joins
// the pieces in order, a block a query.  (The last team to arrive joining them by
// itself was measured slower: one CTA then reads them all, 3.7 us more at 1 x 32773
// tokens.)  Otherwise items stay whole, nothing is joined, and a team has the two, four
// or eight warps that an estimate says end first.  A team's warps take every T-th tile
// of its piece, each with its own statistics, joined in shared memory.
//
// A tile is brought in by its warp alone: 16-byte asynchronous copies into the
// warp's own ring of stages, swizzled so that both the K reads (rows g, g + 8,
// 16 bytes a lane) and the transposed V reads (rows 2t, 2t + 1, 2t + 8, 2t + 9)
// are free of bank conflicts; no barrier is needed but the warp's.  The copies run
// ahead across items, so the stream does not pause where one is finished; its sums
// pass through the ring's one free stage.
#include <atomic>

#include "qlin_kv.cuh"
#include "qlin_sm100.cuh"

namespace qlin {
namespace {

__device__ unsigned int g_attn_error;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = kPageUnit;  // tokens
constexpr int kQ = 8;             // queries a pass over the cache, at most
constexpr int kSms = 148;
constexpr float kNone = -1e30f;   // running maximum of a warp that has seen no token
constexpr int kWholeTiles = 32;   // items up to here are not cut
constexpr int kMinShare = 16;     // tiles a team when they are
// An item's cost beside its tiles, in tiles, for a team of T warps, fitted to short sequences (200 of
// up to 509 tokens, 4 bits: 25.8 us; half the slope takes 6 % more, 2 + 4 T 4 % more) and to long ones
// (24 of up to 9,000 tokens, eight queries on each of 8 kv heads, 4 bits: 35.3 us; 19 and 1 % more).
__device__ __forceinline__ int item_extra(int lt) { return 4 + (4 << lt); }
// A warp's sums in shared memory: 16 values every 20 floats, which spreads both the lanes that
// write (16 dimensions of a query each) and those that read over the banks.
constexpr int kDumpRow = 8 * 20 + 8;  // of a query
constexpr int kMaxTeams = 3 * kSms;  // teams when items are cut: one a CTA
// Up to here records are of items and not of teams, which spares the join its empty blocks: 28 items
// cut among 148 teams take 1 % less, 8 take 8 % less, 128 items 2 % more: a team begins at most one cut item, so there are blocks without work either way.
constexpr int kItemRecords = 64;
static_assert(kItemRecords <= kMaxTeams);
constexpr int kRecordBytes = kMaxTeams * 16;  // of the workspace: the item that each team is the first to cut

// log2 of the least team's warps.  Without a team of two, 400 sequences of up to 60 tokens take 25.5 us
// and not 19.4, 1,000 of up to 130 at 4 bits 76.1 and not 59.5 (where a team's size then is a constant,
// with 4 warps, 100 x 500 tokens of 256 dimensions take 27.1 and not 28.2).  A team of one: 20.2 at
// 400 x 60, 54.4 at 1,000 x 130, for a longer code.
constexpr int kMinTeam = 1;

template <int KB, int VB, int NG, int NT>
struct Cfg {
  static constexpr int kDim = NG * kGroup;
  static constexpr int kRowK = 16 * KB * NG, kRowV = 16 * VB * NG;  // bytes a token
  static constexpr int kPar = KB == 16 ? 0 : 8 * NG;
  static constexpr int kOffV = kTile * kRowK, kOffPar = kOffV + kTile * kRowV;
  static constexpr int kRowQ = 4 * NT;                  // queries
  // log2 of the largest weight over m: below 2^12 half a step of fp16 is at most 1, and lo 2^15 no more than 2^15
  static constexpr float kTop = NT == 2 && VB < 16 ? 12.f : 15.f;
  static constexpr int kTileBytes = kOffPar + kTile * kPar, kDump = 4 * kDumpRow * 4;
  // and a word: the tile's tokens; multiples of the longest row, so that swizzles apply to addresses
  static constexpr int kAlign = KB == 16 ? 256 : 128;
  static constexpr int kStage = ((kTileBytes > kDump ? kTileBytes : kDump) + 16 + kAlign - 1) / kAlign * kAlign;
  // 32 sums a lane (one group) leave room for 16 warps an SM at 128 registers; 64 (two) for 12 at
  // 168, or 8 at 255 with eight queries (7 x 20,011 tokens at most, 8/4 bits: 29.1 us; when it was
  // chosen 31.0, at 168 with spills 44.1, by two passes of four queries 33.0).  16-bit rows fill the rings: 8 warps.
  static constexpr int kSets = NG;
  static constexpr int kWarps = (kSets > 1 || KB == 16) ? 4 : 8;
  static constexpr int kPlanes = 1024 * NT * NG;                // halves of the queries, or their two upper digits
  static constexpr int kOperand = KB == 16 ? kPlanes : kPlanes + kPlanes / 2;  // and the lowest digits
  // Whether the lowest digits stay in registers through the tiles: 32 x 8,000 tokens at 4 bits take 62.9 us
  // and not 64.8; the other shapes would spill.  (As it is, 12 to 25 words a thread spill with eight queries
  // on one group of 8-bit keys or values, at 128 registers, and 12 with four on two groups, at 168.)
  static constexpr bool kLowHeld = KB < 16 && NT == 1 && NG == 1;
  static constexpr int kSmemQ = (kWarps >> kMinTeam) * kOperand;          // of each team
  static constexpr int kSmemX = (kWarps >> kMinTeam) * kRowQ * NG * 8;    // (scale, sum) of each query, a team
  static constexpr int kSmemMl = kWarps * 4 * 8;                // (m, l) of four queries, a warp
  static constexpr int kOther = kSmemQ + kSmemX + kSmemMl + kAlign;  // and room to align it
  static constexpr int fit(int ctas) { return (226 * 1024 / ctas - 4096 - kOther) / (kWarps * kStage); }
  static constexpr int kCtas = kSets == 2 && NT == 1 && KB < 16 && fit(3) >= 2 ? 3 : fit(2) >= 2 ? 2 : 1;  // per SM
  // One stage to read and one to fill are enough once a row has 8-bit codes: 32 x 8,000 tokens at 8 bits take
  // 88.6 us and not 93.6 with three, 8 x 8,192 at 8/4 bits 14.1 and not 14.4, the call of 7 above 0.7 us
  // less.  At 4 bits four take 62.9 us and two 63.7, 16-bit rows 80.6 with three and 81.0 with two (48 x 2,500).
  static constexpr int kMostStages = KB < 16 && KB + VB > 8 ? 2 : 6;
  static constexpr int kStages = fit(kCtas) > kMostStages ? kMostStages : fit(kCtas);
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kSmem = kRing + kOther;
  static constexpr int kGrid = kSms * kCtas;
  static_assert(kStages >= 2, "a stage to fill and one to read");
};

struct AttnArgs {
  KvView c;
  const __half* q;
  int64_t q_stride;
  const int32_t *table, *lens;
  const uint32_t* sign_bits;
  __half* out;
  // (first output row, queries, first team, last team) of cut items, 0 queries: none: of every item if
  // there are at most kItemRecords, else of the item that each team begins and cuts
  int4* records;
  float* ws;  // [teams][2] slots of [qper][dim + 4]: sums, then maximum and denominator per group
  float scale_log2e;
  int32_t q_heads, max_pages, batch, cap;  // cap: tokens the table can hold
  int32_t group, items, nqb, qper;  // queries a kv head; (head, query block) pairs of a sequence; blocks; queries a block
  int32_t page_shift;                      // log2 of a page's tiles; -1: no power of two
  int32_t by_item;                         // records are of items
  int32_t may_cut;                         // the table has room for more than kWholeTiles tiles
};

constexpr int kLensCached = 512;

// Tokens and tiles of sequence b; `lens` holds the first kLensCached of a block's.
__device__ __forceinline__ int clamp_len(const AttnArgs& a, int n) { return min(max(n, 0), a.cap); }
__device__ __forceinline__ int len_of(const AttnArgs& a, const int* lens, int b) {
  return b < kLensCached ? lens[b] : clamp_len(a, a.lens[b]);
}
__device__ __forceinline__ int tiles_in(int n) { return (n + kTile - 1) / kTile; }

// How the items are dealt out; the same in every warp.
struct Plan {
  int cut;    // whether items are cut
  int lt;     // log2 of a team's warps
  int extra;  // cost of an item beside its tiles, in tiles of its team
  int total, share;
};

template <int kThreads>
__device__ __forceinline__ Plan make_plan(const AttnArgs& a, int* lens, int grid) {
  __shared__ int part[3][kThreads / 32];
  const int lane = threadIdx.x & 31;
  constexpr int warps = kThreads / 32;
  int n = 0, top = 0, live = 0;
#pragma unroll 2
  for (int b = threadIdx.x; b < a.batch; b += kThreads) {
    const int len = clamp_len(a, a.lens[b]), t = tiles_in(len);
    if (b < kLensCached) lens[b] = len;
    n += t;
    top = max(top, t);
    live += t > 0;
  }
  n = __reduce_add_sync(0xffffffffu, n);
  top = __reduce_max_sync(0xffffffffu, top);
  live = __reduce_add_sync(0xffffffffu, live);
  if (lane == 0) part[0][threadIdx.x >> 5] = n, part[1][threadIdx.x >> 5] = top, part[2][threadIdx.x >> 5] = live;
  __syncthreads();
  n = top = live = 0;
#pragma unroll
  for (int i = 0; i < warps; ++i) n += part[0][i], top = max(top, part[1][i]), live += part[2][i];
  live *= a.items;
  Plan p;
  p.cut = a.may_cut && top > kWholeTiles;
  p.lt = 31 - __clz(warps);
  if (!p.cut) {
    // the longest item on one team, or as many as a team gets of the average one, in tiles of a
    // warp: the least.  Whole numbers of items: 64 sequences of up to 300 tokens take 10.7 us, 26 % more
    // by the sum of the costs over all warps.
    const float mean = live ? (float)(n * a.items) * rcp((float)live) : 0.f;
    float best = INFINITY;
#pragma unroll
    for (int lt = 31 - __builtin_clz(warps); lt >= kMinTeam; --lt) {
      const int e = item_extra(lt);
      const float each = ceilf((float)live * rcp((float)(grid * (warps >> lt))));
      const float cost = fmaxf((float)(top + e), each * (mean + (float)e)) / (float)(1 << lt);
      if (cost < best) best = cost, p.lt = lt;
    }
  }
  p.extra = item_extra(p.lt);
  static_assert(4 + 4 * warps <= kItemExtra, "positions are counted in an int");
  p.total = n * a.items + live * p.extra;
  const int teams = grid * (warps >> p.lt);
  p.share = (int)((float)p.total * rcp((float)teams)) + 1 + (p.total >> 21);  // teams * share >= total
  p.share = max(p.share, p.cut ? kMinShare : 1);
  return p;
}

// The sequence that position u (< total) belongs to, and its first position.
__device__ __forceinline__ void find_pos(const AttnArgs& a, const Plan& p, const int* lens, int lane, int u,
                                         int& b, int& first) {
  b = first = 0;
  if (a.batch == 1) return;
  const auto cost = [&](int i) {
    const int t = i < a.batch ? tiles_in(len_of(a, lens, i)) : 0;
    return t ? (t + p.extra) * a.items : 0;
  };
  // the lane whose run of sequences holds u, then 32 of that run at a time
  int before = 0, from = 0, to = a.batch;
  if (a.batch > 32) {
    const int run = (a.batch + 31) / 32;
    int n = 0;
    for (int i = 0; i < run; ++i) n += cost(lane * run + i);
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const int l = __ffs(__ballot_sync(0xffffffffu, sum > u)) - 1;  // u < total: there is one
    before = __shfl_sync(0xffffffffu, sum - n, l);
    from = l * run;
    to = from + run;
  }
  for (int b0 = from; b0 < to; b0 += 32) {
    const int n = b0 + lane < to ? cost(b0 + lane) : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + sum > u);
    if (past) {
      const int l = __ffs(past) - 1;
      b = b0 + l;
      first = before + __shfl_sync(0xffffffffu, sum - n, l);
      return;
    }
    before += __shfl_sync(0xffffffffu, sum, 31);
  }
  b = a.batch - 1;  // not reached for u < total
  first = before;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, bool load) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(load ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 ld128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
  return v;
}
__device__ __forceinline__ uint2 ld64(uint32_t p) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p));
  return v;
}
__device__ __forceinline__ uint4 ldmatrix_x4_trans(uint32_t p) {
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(p));
  return v;
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Pairs of codes masked into bits 0-7 (q 2^-24) or 4-7 (q 2^-20), times a power of two: q 2^-9.
__device__ __forceinline__ uint32_t scaled(uint32_t pair, uint32_t mul) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(pair), "r"(mul));
  return d;
}
constexpr uint32_t kLow = 0x78007800u, kHigh = 0x68006800u;  // 2^15, 2^11
constexpr uint32_t kLow4 = 0x000F000Fu, kHigh4 = 0x00F000F0u, kLow8 = 0x00FF00FFu;
__device__ __forceinline__ uint32_t low4(uint32_t w) { return scaled(w & kLow4, kLow); }
__device__ __forceinline__ uint32_t high4(uint32_t w) { return scaled(w & kHigh4, kHigh); }
__device__ __forceinline__ uint32_t low8(uint32_t w) { return scaled(w & kLow8, kLow); }
// Integer products: u8 codes, s8 digits.
__device__ __forceinline__ void imma(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A team's piece of one item.
struct Segment {
  int b, hq0, nq, h;  // sequence, first query head and how many, kv head
  int tile0, n, nt;   // tiles [tile0, tile0 + n) of nt
  int len, from;      // tokens of the sequence; position of the item's first tile
  int item;           // in all
};

// A team's place in its share: position, sequence, the sequence's first position and tiles.
__device__ __forceinline__ bool next_segment(const AttnArgs& a, const Plan& p, const int* lens, int4& cur, int end,
                                             Segment& s) {
  int u = cur.x, b = cur.y, first = cur.z, nt = cur.w;
  while (u < end) {
    while (nt == 0 || u - first >= (nt + p.extra) * a.items) {  // the next sequence that has tokens
      if (nt) first += (nt + p.extra) * a.items;
      ++b;
      nt = tiles_in(len_of(a, lens, b));
    }
    const int cost = nt + p.extra, item = div_pos(u - first, cost), at = (u - first) - item * cost;
    const int until = p.cut ? min(cost, at + end - u) : cost;
    u += until - at;
    s.tile0 = max(at - p.extra, 0);
    s.n = max(until - p.extra, 0) - s.tile0;
    if (s.n <= 0) continue;
    s.b = b, s.nt = nt;
    s.len = len_of(a, lens, b);
    s.h = a.nqb == 1 ? item : div_pos(item, a.nqb);
    const int q0 = (item - s.h * a.nqb) * a.qper;
    s.nq = min(a.qper, a.group - q0);
    s.hq0 = s.h * a.group + q0;
    s.from = first + item * cost + p.extra;
    s.item = b * a.items + item;
    cur = make_int4(u, b, first, nt);
    return true;
  }
  return false;
}

// Byte offset of 16-byte piece c (of a group's row) of tile row r, for the K reads:
// eight lanes read pieces t, t + 4, ... of rows 2j and 2j + 1.
template <int KB>
__host__ __device__ constexpr int k_at(int r, int c) {
  return r * 16 * KB + 16 * (KB == 4 ? c : c ^ ((r & 1) << 2));
}
// The same for the V reads: 4 bits, 16 lanes read 8 bytes of pieces 0, 1 (or 2, 3)
// of rows 2t; 8 bits, 8 lanes read pieces 2i, 2i + 1 of rows 2t; 16 bits, one piece
// of eight consecutive rows.
template <int VB>
__host__ __device__ constexpr int v_at(int r, int c) {
  if (VB == 4) return (r >> 1) * 128 + ((r ^ (r >> 1)) & 1) * 64 + 16 * (c ^ ((r >> 1) & 2));
  if (VB == 8) return r * 128 + 16 * (c ^ (r & 6));
  return r * 256 + 16 * (c ^ (r & 7));
}

// Rotation (or its inverse) of the four values 4 lane .. 4 lane + 3 of group g on a warp.
__device__ __forceinline__ void rotate4(float (&v)[4], const uint32_t* sign_bits, int g, int lane, bool inverse) {
  const uint32_t sw = sign_bits[g * 4 + (lane >> 3)] >> (4 * (lane & 7));
  if (!inverse)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((sw >> i) & 1u) v[i] = -v[i];
  fwht128_warp(v, lane);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] *= kInvSqrt128;
  if (inverse)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((sw >> i) & 1u) v[i] = -v[i];
}

// One group of one head's finished sums on a warp: rotated back and stored.
__device__ __forceinline__ void store_out(const AttnArgs& a, const uint32_t* signs, int row, int dim, int g, int lane,
                                           float (&r)[4], float den) {
  const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = fmaf(r[i], 0.f, r[i]) * inv;  // infinite: a value is, at 16 bits; NaN
  if (a.sign_bits) rotate4(r, signs, g, lane, true);
  const __half2 h0 = __floats2half2_rn(r[0], r[1]), h1 = __floats2half2_rn(r[2], r[3]);
  uint2 w;
  w.x = *reinterpret_cast<const uint32_t*>(&h0);
  w.y = *reinterpret_cast<const uint32_t*>(&h1);
  *reinterpret_cast<uint2*>(a.out + (int64_t)row * dim + g * kGroup + 4 * lane) = w;
}

// Sums of query j, dimensions 4 lane .. 4 lane + 3 of a group, over a team's T of at most W warps.
// Unrolled, so that the loads do not wait for one another: the call of 1 x 32,773 tokens takes 0.9 us
// less, that of 7 of 256 dimensions and eight queries 3.7.
template <int W>
__device__ __forceinline__ void gather(const uint8_t* smem, const int* dump_at, const float2* sml, int T, int j,
                                        int lane, float (&r)[4], float& top, float& den) {
  top = kNone, den = 0.f;
  r[0] = r[1] = r[2] = r[3] = 0.f;
#pragma unroll
  for (int w = 0; w < W; ++w)
    if (w < T) top = fmaxf(top, sml[w * 4 + j].x);
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w >= T) break;
    const float2 ml = sml[w * 4 + j];
    const float f = ex2(ml.x - top);
    const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + dump_at[w]) + j * kDumpRow +
                                                      20 * (lane >> 2) + 4 * (lane & 3));
    den = fmaf(f, ml.y, den);
    r[0] = fmaf(f, v.x, r[0]), r[1] = fmaf(f, v.y, r[1]), r[2] = fmaf(f, v.z, r[2]), r[3] = fmaf(f, v.w, r[3]);
  }
}

// Prepares group g of a query (rotation, fp16, digits or halves) in its team's shared operand, on a
// warp (lane: dimensions 4 lane .. 4 lane + 3).
//   16-bit keys: halves of query q at [q][dim]; below: digit planes [2 q + digit][dim] of the two
//   upper digits, then [q][dim] of the lowest, at 4 bits the dimensions of each eight in the order
//   0 2 4 6 1 3 5 7 (a word's even codes, its odd).  The lowest digits of odd queries change places
//   in blocks of 64 (4 bits: 16) bytes, so that the lanes that read them meet no bank conflict.
template <int KB, int NG, int NT>
__device__ __forceinline__ void prepare_query(const AttnArgs& a, const uint32_t* signs, uint2 r, int q, int g, int lane, uint8_t* sq,
                                               float2* sx) {
  constexpr int D = NG * kGroup;
  float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&r.x));
  float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
  float v[4] = {f0.x, f0.y, f1.x, f1.y};
  if (a.sign_bits) {
    rotate4(v, signs, g, lane, false);
    const __half2 h0 = __floats2half2_rn(v[0], v[1]), h1 = __floats2half2_rn(v[2], v[3]);
    r.x = *reinterpret_cast<const uint32_t*>(&h0);
    r.y = *reinterpret_cast<const uint32_t*>(&h1);
    f0 = __half22float2(h0), f1 = __half22float2(h1);
    v[0] = f0.x, v[1] = f0.y, v[2] = f1.x, v[3] = f1.y;
  }
  if (KB == 16) {
    *reinterpret_cast<uint2*>(sq + (q * D + g * kGroup + 4 * lane) * 2) = r;
    if (lane == 0) sx[q * NG + g] = make_float2(a.scale_log2e, 0.f);
    return;
  }
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) big = max(big, __float_as_uint(v[i]) & 0x7fffffffu);
  big = __reduce_max_sync(0xffffffffu, big);
  const int e = (int)(big >> 23) - 127;
  const float down = big ? __uint_as_float((uint32_t)(127 + 21 - e) << 23) : 0.f;
  int sum = 0;
  uint32_t hi = 0, mid = 0, lo = 0;  // digits of -128 .. 127, |hi| <= 64
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int xi = __float2int_rn(v[i] * down), up = xi + 128, upper = (up >> 8) + 128;
    sum += xi;  // at most 128 2^22
    hi |= (uint32_t)((upper >> 8) & 255) << (8 * i);
    mid |= (uint32_t)((upper & 255) ^ 128) << (8 * i);
    lo |= (uint32_t)((up & 255) ^ 128) << (8 * i);
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  uint8_t* row = sq + (2 * q) * D + g * kGroup;
  uint8_t* low = sq + 1024 * NT * NG + q * D + g * kGroup;
  if (KB == 8) {
    *reinterpret_cast<uint32_t*>(row + 4 * lane) = hi;
    *reinterpret_cast<uint32_t*>(row + D + 4 * lane) = mid;
    *reinterpret_cast<uint32_t*>(low + ((4 * lane) ^ (64 * (q & 1)))) = lo;
  } else {  // dimensions 4l .. 4l+3 of an eight: its bytes 2 (l & 1), + 1 (even) and 4 bytes on (odd)
    row += 8 * (lane >> 1) + 2 * (lane & 1);
    *reinterpret_cast<uint16_t*>(row) = (uint16_t)__byte_perm(hi, 0, 0x4420);
    *reinterpret_cast<uint16_t*>(row + 4) = (uint16_t)__byte_perm(hi, 0, 0x4431);
    *reinterpret_cast<uint16_t*>(row + D) = (uint16_t)__byte_perm(mid, 0, 0x4420);
    *reinterpret_cast<uint16_t*>(row + D + 4) = (uint16_t)__byte_perm(mid, 0, 0x4431);
    low += (8 * (lane >> 1) + 2 * (lane & 1)) ^ (16 * (q & 1));
    *reinterpret_cast<uint16_t*>(low) = (uint16_t)__byte_perm(lo, 0, 0x4420);
    *reinterpret_cast<uint16_t*>(low + 4) = (uint16_t)__byte_perm(lo, 0, 0x4431);
  }
  const float unit = KB == 4 ? 0.0625f : 1.f, step = __uint_as_float((uint32_t)(127 - 21 + e) << 23);
  const float f = big >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : big ? a.scale_log2e * step * unit : 0.f;
  if (lane == 0) sx[q * NG + g] = make_float2(f, (float)sum / unit);
}

template <int KB, int VB, int NG, int NT>
__global__ void __launch_bounds__(Cfg<KB, VB, NG, NT>::kWarps * 32, Cfg<KB, VB, NG, NT>::kCtas)
    attn_kernel(const __grid_constant__ AttnArgs a) {
  using C = Cfg<KB, VB, NG, NT>;
  constexpr int NW = C::kWarps, S = C::kStages, D = C::kDim;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + (-smem_addr(smem_raw) & (C::kAlign - 1u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
  const int grid = gridDim.x, page_tiles = a.c.page / kTile;
  uint8_t* const ring_ptr = smem + warp * S * C::kStage;
  const uint32_t ring = smem_addr(ring_ptr);

  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ int lens[kLensCached];
  __shared__ uint32_t signs[4 * NG];
  if (a.sign_bits && threadIdx.x < 4 * NG) signs[threadIdx.x] = a.sign_bits[threadIdx.x];
  const Plan plan = make_plan<NW * 32>(a, lens, grid);
  const int lt = plan.lt, T = 1 << lt, team = warp >> lt, tw = warp & (T - 1);
  const int teams = NW >> lt, worker = blockIdx.x * teams + team;
  uint8_t* sq = smem + C::kRing + team * C::kOperand;
  float2* sx = reinterpret_cast<float2*>(smem + C::kRing + C::kSmemQ) + team * C::kRowQ * NG;
  float2* sml = reinterpret_cast<float2*>(smem + C::kRing + C::kSmemQ + C::kSmemX) + (warp - tw) * 4;
  auto team_barrier = [&]() {
    named_barrier(1 + team, 32 << lt);
  };

  const int64_t begin = (int64_t)worker * plan.share;
  const int end = (int)min((int64_t)plan.total, begin + plan.share);
  __shared__ int4 place[NW][2];      // a warp's places: of its copies, of its sums
  __shared__ int dump_at[NW];        // where a warp's sums are, in bytes
  __shared__ Segment held[NW];       // a warp's segment, out of the registers while it reads the tiles
  int4 record = make_int4(0, 0, 0, 0);
  bool more = begin < plan.total;
  Segment seg = {};
  if (more) {
    int4 cur = make_int4((int)begin, 0, 0, 0);
    find_pos(a, plan, lens, lane, cur.x, cur.y, cur.z);
    cur.w = tiles_in(len_of(a, lens, cur.y));
    if (!plan.cut) {  // items that start in the share
      const int cost = cur.w + plan.extra, at = cur.x - cur.z - div_pos(cur.x - cur.z, cost) * cost;
      if (at) cur.x += cost - at;
    }
    more = next_segment(a, plan, lens, cur, end, seg);
    if (lane == 0) place[warp][0] = place[warp][1] = cur;
  }
  bool have = more;
  // the warp's part of a segment's queries, a (query, group) at a time
  uint2 qr = make_uint2(0u, 0u);
  const auto load_query = [&](int i) {
    const int q = i / NG;
    return q < seg.nq ? reinterpret_cast<const uint2*>(a.q + (int64_t)seg.b * a.q_stride + (int64_t)(seg.hq0 + q) * D +
                                                       (i % NG) * kGroup)[lane]
                      : make_uint2(0u, 0u);
  };
  if (have) qr = load_query(tw);

  // ---- copies: tile ik of icnt of the warp's piece of the segment that they have reached
  int ik = 0, icnt = have && tw < seg.n ? (seg.n - tw + T - 1) >> lt : 0;
  int itile = seg.tile0 + tw, ilen = seg.len, ih = seg.h, istage = 0;
  uint32_t src_lo = 0, src_hi = 0, meta = 0;  // of 32 tiles, one a lane: address of the K rows; tile in the page, tokens
  // where the lane's first piece goes; piece j goes to (first ^ swizzle(j)) + pitch(j), a constant each
  constexpr int RK = KB * NG, RV = VB * NG;
  const uint32_t k_dst = ring + (lane % RK) / KB * (kTile * 16 * KB) + k_at<KB>(lane / RK, lane % KB);
  const uint32_t v_dst = ring + C::kOffV + (lane % RV) / VB * (kTile * 16 * VB) + v_at<VB>(lane / RV, lane % VB);
  const int32_t* itable = a.table + (int64_t)seg.b * a.max_pages;
  __syncwarp();
  auto issue = [&]() {
    while (more && ik >= icnt) {
      int4 cur = place[warp][0];
      __syncwarp();
      Segment s;
      more = next_segment(a, plan, lens, cur, end, s);
      if (more) {
        if (lane == 0) place[warp][0] = cur;
        __syncwarp();
        ik = 0;
        icnt = tw < s.n ? (s.n - tw + T - 1) >> lt : 0;
        itile = s.tile0 + tw;
        ilen = s.len;
        ih = s.h;
        itable = a.table + (int64_t)s.b * a.max_pages;
      }
    }
    if (more) {
      if ((ik & 31) == 0) {
        const int kk = ik + lane;
        if (kk < icnt) {
          const int tile = itile + (kk << lt), page = a.page_shift >= 0 ? tile >> a.page_shift : tile / page_tiles;
          int p = itable[page], valid = min(kTile, ilen - tile * kTile);
          if ((unsigned)p >= (unsigned)a.c.pages) {
            atomicOr(&g_attn_error, kKvBadPage);
            p = 0;
            valid = 0;
          }
          const int at = tile - page * page_tiles;  // below 2^27: a page has fewer than 2^31 tokens
          const uint64_t src = reinterpret_cast<uint64_t>(a.c.block(p, ih)) + (int64_t)at * (kTile * C::kRowK);
          src_lo = (uint32_t)src, src_hi = (uint32_t)(src >> 32);
          meta = (uint32_t)at << 5 | (uint32_t)valid;
        }
      }
      const uint32_t lo = __shfl_sync(0xffffffffu, src_lo, ik & 31), hi = __shfl_sync(0xffffffffu, src_hi, ik & 31);
      const uint32_t mt = __shfl_sync(0xffffffffu, meta, ik & 31), valid = mt & 31u;
      const int64_t in_page = mt >> 5;  // tiles; a page may hold more than 2^31 bytes
      const uint8_t* src = reinterpret_cast<const uint8_t*>((uint64_t)hi << 32 | lo) + 16 * lane;
      const uint32_t at = istage * C::kStage;
#pragma unroll
      for (int j = 0; j < RK / 2; ++j) {
        constexpr int pitch = 16 * KB;
        const int r = 32 * j / RK;
        cp16(((k_dst + at) ^ (uint32_t)(k_at<KB>(r, 0) - r * pitch)) + r * pitch, src + 512 * j);
      }
      const uint8_t* v_src = src + a.c.v_offset;
      if (RV != RK) v_src += in_page * (kTile * (C::kRowV - C::kRowK));
#pragma unroll
      for (int j = 0; j < RV / 2; ++j) {
        constexpr int pitch = 16 * VB;
        const int r = 32 * j / RV;
        const uint32_t dst = ((v_dst + at) ^ (uint32_t)(v_at<VB>(r, 0) - r * pitch)) + r * pitch;
        // 16-bit values past the length could be NaN, which a weight of zero would not hide
        if (VB == 16)
          cp16_or_zero(dst, v_src + 512 * j, (unsigned)(lane / RV + r) < valid);
        else
          cp16(dst, v_src + 512 * j);
      }
      if (C::kPar) {
        if (lane < kTile * C::kPar / 16)
          cp16(ring + at + C::kOffPar + 16 * lane, src + a.c.par_offset + in_page * (kTile * (C::kPar - C::kRowK)));
      }
      if (lane == 0) *reinterpret_cast<uint32_t*>(ring_ptr + at + C::kStage - 16) = valid;
      ++ik;
      istage = istage + 1 == S ? 0 : istage + 1;
    }
    cp_commit();
  };
#pragma unroll 1
  for (int k = 0; k < S - 1; ++k) issue();

  int stage_no = 0;  // of the tile to be read next
  const uint32_t k_src = ring + k_at<KB>(g8, t4);  // rows g8 and g8 + 8, pieces t4, t4 + 4 (at ^ 64), ...
  const uint32_t v_src = ring + C::kOffV +
                         (VB == 4   ? v_at<VB>(2 * t4, g8 >> 1) + 8 * (g8 & 1)
                          : VB == 8 ? v_at<VB>(2 * t4, g8)
                                    : v_at<VB>((lane & 7) + 8 * (lane >> 4), (lane >> 3) & 1));
  // the lowest digits of column g8's query: the second piece at ^ (KB == 4 ? 16 : 64)
  const int low_q = NT == 1 ? g8 >> 1 : g8;
  const uint32_t low_src = smem_addr(sq) + C::kPlanes + low_q * D +
                           (KB == 4 ? 32 * t4 + 16 * (low_q & 1) : 16 * t4 + 64 * (low_q & 1));
  while (have) {
    const int cnt = tw < seg.n ? (seg.n - tw + T - 1) >> lt : 0;
    // ---- the queries, and the lane's operand: column g8 = (query g8 / 2, digit g8 % 2), the
    // dimensions of the codes that lanes of column t4 hold
    for (int i = tw; i < C::kRowQ * NG; i += T) {
      const uint2 r = qr;
      if (i + T < C::kRowQ * NG) qr = load_query(i + T);
      prepare_query<KB, NG, NT>(a, signs, r, i / NG, i % NG, lane, sq, sx);
    }
    team_barrier();
    constexpr int NB = KB == 16 ? 16 : 8;  // operand registers a group
    constexpr int NS = KB == 16 ? 1 : NT;  // column sets of the keys' products
    uint32_t qf[NS][NG][NB];
    uint4 qlow[2];
    if (C::kLowHeld) qlow[0] = ld128(low_src), qlow[1] = ld128(low_src ^ (KB == 4 ? 16 : 64));
    float xs[NT][NG], sc[NT][NG];  // sum and scale of query(s, t4)
    const auto query = [](int s, int t) { return NT == 1 ? t : 2 * t + s; };
#pragma unroll
    for (int s = 0; s < NT; ++s)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t base = smem_addr(sq);
        if (s < NS) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (KB == 16) {  // piece t4 + 4 j of query g8 / 2 (the odd columns are zero), or of query g8
              uint4 p = ld128(base + ((NT == 1 ? g8 >> 1 : g8) * D + g * kGroup + 32 * j + 8 * t4) * 2);
              if (NT == 1 && (g8 & 1)) p = make_uint4(0u, 0u, 0u, 0u);
              qf[s % NS][g][(4 * j) % NB] = p.x, qf[s % NS][g][(4 * j + 1) % NB] = p.y;
              qf[s % NS][g][(4 * j + 2) % NB] = p.z, qf[s % NS][g][(4 * j + 3) % NB] = p.w;
            } else {  // eight dimensions: 4 bits, word j of piece t4; 8 bits, words 2 (j & 1), + 1 of piece t4 + 4 (j / 2)
              const int d0 = KB == 4 ? 32 * t4 + 8 * j : 64 * (j >> 1) + 16 * t4 + 8 * (j & 1);
              const uint2 p = ld64(base + (2 * query(s, g8 >> 1) + (g8 & 1)) * D + g * kGroup + d0);
              qf[s % NS][g][2 * j] = p.x, qf[s % NS][g][2 * j + 1] = p.y;
            }
          }
        }
        const float2 x = sx[query(s, t4) * NG + g];
        sc[s][g] = x.x, xs[s][g] = x.y;
      }

    float o[NG][8][4], m[NT][NG], l[NT][NG], zc[NT][NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[g][j][0] = o[g][j][1] = o[g][j][2] = o[g][j][3] = 0.f;
#pragma unroll
      for (int s = 0; s < NT; ++s) {
        m[s][g] = kNone;
        l[s][g] = zc[s][g] = 0.f;
      }
    }

    if (lane == 0) held[warp] = seg;
    for (int k = 0; k < cnt; ++k) {
      cp_wait<S - 2>();
      __syncwarp();
      issue();  // into the stage that the previous tile has left
      const int stage = stage_no * C::kStage;
      stage_no = stage_no + 1 == S ? 0 : stage_no + 1;
      const uint32_t st = ring + stage;
      const int valid = *reinterpret_cast<const volatile int*>(ring_ptr + stage + C::kStage - 16);

      // scores in units of log2: query(s, t4), tokens g8 and g8 + 8
      float w[NT][2];
      float lv[NG][2], rv[NG][2], vz[NG][2];
#pragma unroll
      for (int s = 0; s < NT; ++s) w[s][0] = w[s][1] = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float dot[NT][2];
        const uint32_t kb = k_src + stage + g * (kTile * 16 * KB);
        if (KB == 4) {
          const uint4 wa = ld128(kb), wb = ld128(kb + 128 * KB);
          const uint32_t ra[4] = {wa.x, wa.y, wa.z, wa.w}, rb[4] = {wb.x, wb.y, wb.z, wb.w};
          int c0[NT][4], c1[NT][4], e0[4] = {0, 0, 0, 0}, e1[4] = {0, 0, 0, 0};
#pragma unroll
          for (int s = 0; s < NT; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) c0[s][i] = c1[s][i] = 0;
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            constexpr uint32_t lo = 0x0F0F0F0Fu, hi = 0xF0F0F0F0u;
            const uint4 x = C::kLowHeld ? qlow[j / 2] : ld128((low_src + g * kGroup) ^ (8 * j));
            imma(e0, ra[j] & lo, rb[j] & lo, ra[j + 1] & lo, rb[j + 1] & lo, x.x, x.z);
            imma(e1, ra[j] & hi, rb[j] & hi, ra[j + 1] & hi, rb[j + 1] & hi, x.y, x.w);
#pragma unroll
            for (int s = 0; s < NT; ++s) {
              imma(c0[s], ra[j] & lo, rb[j] & lo, ra[j + 1] & lo, rb[j + 1] & lo, qf[s % NS][g][2 * j], qf[s % NS][g][2 * j + 2]);
              imma(c1[s], ra[j] & hi, rb[j] & hi, ra[j + 1] & hi, rb[j + 1] & hi, qf[s % NS][g][2 * j + 1],
                   qf[s % NS][g][2 * j + 3]);
            }
          }
#pragma unroll
          for (int s = 0; s < NT; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              dot[s][i] = fmaf((float)((16 * c0[s][2 * i] + c1[s][2 * i]) * 256 + (16 * c0[s][2 * i + 1] + c1[s][2 * i + 1])),
                               256.f, (float)(16 * e0[2 * i + s] + e1[2 * i + s]));
        } else if (KB == 8) {
          int c0[NT][4], c1[NT][4], e[4] = {0, 0, 0, 0};
#pragma unroll
          for (int s = 0; s < NT; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) c0[s][i] = c1[s][i] = 0;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 wa = ld128(kb ^ (64 * j)), wb = ld128((kb ^ (64 * j)) + 128 * KB);
            const uint4 x = C::kLowHeld ? qlow[j] : ld128((low_src + g * kGroup) ^ (64 * j));
            imma(e, wa.x, wb.x, wa.y, wb.y, x.x, x.y);
            imma(e, wa.z, wb.z, wa.w, wb.w, x.z, x.w);
#pragma unroll
            for (int s = 0; s < NT; ++s) {
              imma(c0[s], wa.x, wb.x, wa.y, wb.y, qf[s % NS][g][4 * j], qf[s % NS][g][4 * j + 1]);
              imma(c1[s], wa.z, wb.z, wa.w, wb.w, qf[s % NS][g][4 * j + 2], qf[s % NS][g][4 * j + 3]);
            }
          }
#pragma unroll
          for (int s = 0; s < NT; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              dot[s][i] = fmaf((float)((c0[s][2 * i] + c1[s][2 * i]) * 256 + (c0[s][2 * i + 1] + c1[s][2 * i + 1])), 256.f,
                               (float)e[2 * i + s]);
        } else {
          float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 wa = ld128(kb ^ (64 * j)), wb = ld128((kb ^ (64 * j)) + 128 * KB);
            mma(c0, wa.x, wb.x, wa.y, wb.y, qf[0][g][(4 * j) % NB], qf[0][g][(4 * j + 1) % NB]);
            mma(c1, wa.z, wb.z, wa.w, wb.w, qf[0][g][(4 * j + 2) % NB], qf[0][g][(4 * j + 3) % NB]);
          }
#pragma unroll
          for (int s = 0; s < NT; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) dot[s][i] = c0[2 * i + s] + c1[2 * i + s];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // tokens g8, g8 + 8
          if (C::kPar) {
            const uint2 p = ld64(st + C::kOffPar + (g8 + 8 * i) * C::kPar + 8 * g);
            const float2 pk = __half22float2(*reinterpret_cast<const __half2*>(&p.x));
            const float2 pv = __half22float2(*reinterpret_cast<const __half2*>(&p.y));
#pragma unroll
            for (int s = 0; s < NT; ++s)
              w[s][i] = fmaf(fmaf(-pk.y, xs[s][g], dot[s][i]), pk.x * sc[s][g], w[s][i]);
            // a scale of 0 (a slot that was cleared, never written) is 2^-64 here: its token has a
            // share of the denominator and none of the sums.  The denominator of 2^31 such tokens
            // stays below 2^(15 + 64 + 31), and beside a scale of 2^16 weights down to 2^-53 count.
            lv[g][i] = fmaxf(lg2(pv.x), -64.f);
            rv[g][i] = fminf(rcp(pv.x), 0x1p64f);
            vz[g][i] = pv.y;
          } else {
#pragma unroll
            for (int s = 0; s < NT; ++s) w[s][i] = fmaf(dot[s][i], sc[s][g], w[s][i]);
            lv[g][i] = vz[g][i] = 0.f;
            rv[g][i] = 1.f;
          }
        }
      }
      // An infinite score is an infinity among the query's or the key's values: NaN, and not a weight of zero.
      // (Of 4- and 8-bit codes it comes as NaN, by the group's zero or the query's scale.)
      if (KB == 16)
#pragma unroll
        for (int s = 0; s < NT; ++s) w[s][0] = fmaf(w[s][0], 0.f, w[s][0]), w[s][1] = fmaf(w[s][1], 0.f, w[s][1]);
      if (valid < kTile) {  // masked tokens: no weight, and nothing kept of their parameters
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (g8 + 8 * i >= valid) {
#pragma unroll
            for (int s = 0; s < NT; ++s) w[s][i] = -INFINITY;
#pragma unroll
            for (int g = 0; g < NG; ++g) lv[g][i] = rv[g][i] = vz[g][i] = 0.f;
          }
      }

      uint32_t pb[NG][2], pl[NG][2], ph[NG][2];  // weights as operand; with NT = 2 lo for codes at q 2^-24, at q 2^-20
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float y[NT][2], top[NT];
        bool past = false;
#pragma unroll
        for (int s = 0; s < NT; ++s) {
          y[s][0] = w[s][0] + lv[g][0], y[s][1] = w[s][1] + lv[g][1];
          top[s] = fmaxf(y[s][0], y[s][1]);
          past |= top[s] > m[s][g] + C::kTop;
        }
        if (__any_sync(0xffffffffu, past)) {
          float f[NT];
#pragma unroll
          for (int s = 0; s < NT; ++s) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top[s] = fmaxf(top[s], __shfl_xor_sync(0xffffffffu, top[s], d));
            const float next = fmaxf(m[s][g], top[s] - (C::kTop - 8.f));
            f[s] = ex2(m[s][g] - next);
            m[s][g] = next;
            l[s][g] *= f[s], zc[s][g] *= f[s];
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[g][j][i] *= f[(i & 1) % NT];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          __half2 pair;
          if (NT == 1) {
            const float p = ex2(y[0][i] - m[0][g]), hi = __half2float(__float2half_rn(p));
            pair = __floats2half2_rn(p, (p - hi) * 2048.f);
            l[0][g] = fmaf(p, rv[g][i], l[0][g]);
            if (C::kPar) zc[0][g] = fmaf(p, vz[g][i], zc[0][g]);
          } else {
            float p[NT];
#pragma unroll
            for (int s = 0; s < NT; ++s) p[s] = ex2(y[s][i] - m[s][g]);
            pair = __floats2half2_rn(p[0], p[NT - 1]);
            const float r0 = p[0] - __low2float(pair), r1 = p[NT - 1] - __high2float(pair);
            constexpr float low = VB == 16 ? 1.f : 0x1p15f, high = 0x1p11f;
            const __half2 rest = __floats2half2_rn(r0 * low, r1 * low);
            pl[g][i] = movmatrix(*reinterpret_cast<const uint32_t*>(&rest));
            if (VB == 4) {
              const __half2 rest4 = __floats2half2_rn(r0 * high, r1 * high);
              ph[g][i] = movmatrix(*reinterpret_cast<const uint32_t*>(&rest4));
            }
#pragma unroll
            for (int s = 0; s < NT; ++s) {
              l[s][g] = fmaf(p[s], rv[g][i], l[s][g]);
              if (C::kPar) zc[s][g] = fmaf(p[s], vz[g][i], zc[s][g]);
            }
          }
          pb[g][i] = movmatrix(*reinterpret_cast<const uint32_t*>(&pair));
        }
      }

      // values: the lane's tokens 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9, dimensions 16 g8 .. 16 g8 + 15
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t vb = v_src + stage + g * (kTile * 16 * VB);
        if (VB == 4) {
          uint2 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = ld64((vb ^ (64 * (i & 1))) + 512 * (i >> 1));
#pragma unroll
          for (int half = 0; half < 4; ++half) {  // four dimensions: a half-word of each token
            const uint32_t sel = (half & 1) ? 0x7632u : 0x5410u;
            const uint32_t x = half < 2 ? __byte_perm(v[0].x, v[1].x, sel) : __byte_perm(v[0].y, v[1].y, sel);
            const uint32_t y = half < 2 ? __byte_perm(v[2].x, v[3].x, sel) : __byte_perm(v[2].y, v[3].y, sel);
            const uint32_t x0 = low4(x), x2 = low4(x >> 8), y0 = low4(y), y2 = low4(y >> 8);
            const uint32_t x1 = high4(x), x3 = high4(x >> 8), y1 = high4(y), y3 = high4(y >> 8);
            mma(o[g][2 * half], x0, x2, y0, y2, pb[g][0], pb[g][1]);
            mma(o[g][2 * half + 1], x1, x3, y1, y3, pb[g][0], pb[g][1]);
            if (NT == 2) {
              mma(o[g][2 * half], x & kLow4, (x >> 8) & kLow4, y & kLow4, (y >> 8) & kLow4, pl[g][0], pl[g][1]);
              mma(o[g][2 * half + 1], x & kHigh4, (x >> 8) & kHigh4, y & kHigh4, (y >> 8) & kHigh4, ph[g][0], ph[g][1]);
            }
          }
        } else if (VB == 8) {
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = ld128(vb + 128 * (i & 1) + 1024 * (i >> 1));
          const uint32_t v0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, v1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
          const uint32_t v2[4] = {v[2].x, v[2].y, v[2].z, v[2].w}, v3[4] = {v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
          for (int j = 0; j < 8; ++j) {  // two dimensions: a half-word of each token
            const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
            const uint32_t x = __byte_perm(v0[j >> 1], v1[j >> 1], sel), y = __byte_perm(v2[j >> 1], v3[j >> 1], sel);
            const uint32_t x0 = low8(x), x1 = low8(x >> 8), y0 = low8(y), y1 = low8(y >> 8);
            mma(o[g][j], x0, x1, y0, y1, pb[g][0], pb[g][1]);
            if (NT == 2) mma(o[g][j], x & kLow8, (x >> 8) & kLow8, y & kLow8, (y >> 8) & kLow8, pl[g][0], pl[g][1]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 v = ldmatrix_x4_trans(vb ^ (32 * j));
            mma(o[g][j], v.x, v.y, v.z, v.w, pb[g][0], pb[g][1]);
            if (NT == 2) mma(o[g][j], v.x, v.y, v.z, v.w, pl[g][0], pl[g][1]);
          }
        }
      }
    }
    __syncwarp();  // every lane has read the last tile, and its stage is free
    seg = held[warp];

    // ---- the sums of four queries and one group at a time: each warp's into its free stage, then the
    // team's
    float* dump = reinterpret_cast<float*>(ring_ptr + istage * C::kStage);
    if (lane == 0) dump_at[warp] = warp * S * C::kStage + istage * C::kStage;
    const int slot = seg.tile0 == 0;  // 0: the item began in an earlier share
    // query(s, t4)'s sum from a lane's two columns
    const auto column = [](float a, float b, int s) { return NT == 1 ? fmaf(b, 0x1p-11f, a) : s ? b : a; };
    if (a.may_cut && slot) {
      int4 rec = make_int4(0, 0, 0, 0);
      if (seg.n != seg.nt)
        record = rec = make_int4(seg.b * a.q_heads + seg.hq0, seg.nq, worker, (seg.from + seg.nt - 1) / plan.share);
      if (a.by_item && tw == 0 && lane == 0) a.records[seg.item] = rec;
    }
#pragma unroll
    for (int s = 0; s < NT; ++s)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          l[s][g] += __shfl_xor_sync(0xffffffffu, l[s][g], d);
          zc[s][g] += __shfl_xor_sync(0xffffffffu, zc[s][g], d);
        }
        float* row = dump + t4 * kDumpRow;
#pragma unroll
        for (int j = 0; j < 8; j += (VB == 16 ? 1 : 2)) {
          const float(&e)[4] = o[g][j];
          const float e0 = column(e[0], e[1], s), e1 = column(e[2], e[3], s);
          if (VB == 16) {
            row[20 * j + g8] = e0, row[20 * j + 8 + g8] = e1;
          } else {
            const float(&f)[4] = o[g][(j + 1) & 7];
            const float f0 = column(f[0], f[1], s), f1 = column(f[2], f[3], s), z = -zc[s][g];
            const float r0 = fmaf(e0, 512.f, z), r1 = fmaf(e1, 512.f, z), r2 = fmaf(f0, 512.f, z), r3 = fmaf(f1, 512.f, z);
            // 4 bits: rows (0, 2) and (1, 3) of four dimensions; 8 bits: (0, 1) and (2, 3)
            *reinterpret_cast<float4*>(row + 20 * g8 + 2 * j) =
                VB == 4 ? make_float4(r0, r2, r1, r3) : make_float4(r0, r1, r2, r3);
          }
        }
        if (g8 == 0) sml[tw * 4 + t4] = make_float2(m[s][g], l[s][g]);
        team_barrier();
        for (int j = tw; j < 4; j += T)
          if (query(s, j) < seg.nq) {
            float r[4], top, den;
            gather<NW>(smem, dump_at + warp - tw, sml, T, j, lane, r, top, den);
            if (seg.n == seg.nt) {
              store_out(a, signs, seg.b * a.q_heads + seg.hq0 + query(s, j), D, g, lane, r, den);
            } else {
              float* to = a.ws + (((int64_t)worker * 2 + slot) * a.qper + query(s, j)) * (D + 4);
              __stcg(reinterpret_cast<float4*>(to + g * kGroup + 4 * lane), make_float4(r[0], r[1], r[2], r[3]));
              if (lane == 0) __stcg(reinterpret_cast<float2*>(to + D + 2 * g), make_float2(top, den));
            }
          }
        team_barrier();  // the stage, the statistics and the queries may be overwritten
      }

    int4 cur = place[warp][1];
    __syncwarp();
    have = next_segment(a, plan, lens, cur, end, seg);
    if (lane == 0) place[warp][1] = cur;
    __syncwarp();
    if (have) qr = load_query(tw);
  }
  cp_wait<0>();

  // sequences without tokens
  for (int b = blockIdx.x; b < a.batch; b += grid) {
    const int n = a.lens[b];
    if (n > a.cap && threadIdx.x == 0) atomicOr(&g_attn_error, kKvBadLength);
    if (n <= 0) {
      for (int i = threadIdx.x; i < a.q_heads * (D / 8); i += NW * 32)  // q_heads < 2^31 / kItemExtra
        reinterpret_cast<uint4*>(a.out + (int64_t)b * a.q_heads * D)[i] = make_uint4(0u, 0u, 0u, 0u);
      if (a.may_cut && a.by_item && threadIdx.x < a.items) a.records[b * a.items + threadIdx.x] = make_int4(0, 0, 0, 0);
    }
  }

  if (a.may_cut && !a.by_item && threadIdx.x == 0) a.records[blockIdx.x] = record;  // a team that cuts is the CTA
}

// Joins the pieces of query blockIdx.y of the cut item of record blockIdx.x, W warps over the pieces.
// What it costs is latency (3 to 4 us of a call that cuts, its launch among them): a record, its
// pieces, the sums of the warps, and each stretch of code that runs for the first time.  So the code
// is short: a piece or two a warp at a time and not four, 1.0 us less for one query head of 18 pieces.
template <int NG, int W>
__global__ void __launch_bounds__(W * 32) attn_join_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int D = NG * kGroup;
  constexpr int N = W == 4 ? 2 : 1;  // pieces that a warp loads at a time
  __shared__ __align__(16) float sums[NG][W][kGroup];
  __shared__ float2 sml[NG][W];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = blockIdx.y;
  grid_dependency_wait();  // every block: this grid's end stands for the first one's too
  grid_launch_dependents();
  const int4 rec = __ldcg(a.records + blockIdx.x);
  if (q >= rec.y) return;
  float top[NG], den[NG], r[NG][4];
#pragma unroll
  for (int g = 0; g < NG; ++g) top[g] = kNone, den[g] = r[g][0] = r[g][1] = r[g][2] = r[g][3] = 0.f;
  for (int c = rec.z + warp; c <= rec.w; c += N * W) {
    float4 v[N][NG];
    float2 ml[N][NG];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int k = c + i * W;
      const float* p = a.ws + (((int64_t)k * 2 + (k == rec.z)) * a.qper + q) * (D + 4);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const bool live = k <= rec.w;
        ml[i][g] = live ? __ldcg(reinterpret_cast<const float2*>(p + D + 2 * g)) : make_float2(kNone, 0.f);
        v[i][g] = live ? __ldcg(reinterpret_cast<const float4*>(p + g * kGroup + 4 * lane)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float next = fmaxf(top[g], ml[i][g].x), f = ex2(top[g] - next), e = ex2(ml[i][g].x - next);
        top[g] = next;
        den[g] = den[g] * f + e * ml[i][g].y;
        r[g][0] = r[g][0] * f + e * v[i][g].x, r[g][1] = r[g][1] * f + e * v[i][g].y;
        r[g][2] = r[g][2] * f + e * v[i][g].z, r[g][3] = r[g][3] * f + e * v[i][g].w;
      }
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    *reinterpret_cast<float4*>(&sums[g][warp][4 * lane]) = make_float4(r[g][0], r[g][1], r[g][2], r[g][3]);
    if (lane == 0) sml[g][warp] = make_float2(top[g], den[g]);
  }
  __syncthreads();
  for (int g = warp; g < NG; g += W) {
    float t = kNone, d = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < W; ++w) t = fmaxf(t, sml[g][w].x);
#pragma unroll 4
    for (int w = 0; w < W; ++w) {
      const float2 ml = sml[g][w];
      const float f = ex2(ml.x - t);
      const float4 s = *reinterpret_cast<const float4*>(&sums[g][w][4 * lane]);
      d = fmaf(f, ml.y, d);
      v[0] = fmaf(f, s.x, v[0]), v[1] = fmaf(f, s.y, v[1]), v[2] = fmaf(f, s.z, v[2]), v[3] = fmaf(f, s.w, v[3]);
    }
    store_out(a, a.sign_bits, rec.x + q, D, g, lane, v, d);
  }
}

template <int KB, int VB, int NG, int NT>
qlin_status launch(const AttnArgs& a, cudaStream_t s) {
  using C = Cfg<KB, VB, NG, NT>;
  static_assert(C::kSmem <= 226 * 1024 && C::kGrid <= kMaxTeams, "launch bounds");
  static std::atomic<unsigned long long> configured{0};  // per-device attribute, set once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return record_cuda(e);
  if (dev >= 64 || !((configured.load(std::memory_order_acquire) >> dev) & 1ull)) {
    e = cudaFuncSetAttribute(attn_kernel<KB, VB, NG, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return record_cuda(e);
    if (dev < 64) configured.fetch_or(1ull << dev, std::memory_order_release);
  }
  const qlin_status r = launch_dependent(attn_kernel<KB, VB, NG, NT>, C::kGrid, C::kWarps * 32, C::kSmem, s, a);
  if (r != QLIN_OK || !a.may_cut) return r;
  // Few items have many pieces.  16 warps a block and not 8: 0.7 us less at 8 items of 18 pieces;
  // 4 and not 8: 0.7 us less at 64 items of 2 or 3.
  const int64_t items = (int64_t)a.batch * a.items;
  if (items <= 8) return launch_dependent(attn_join_kernel<NG, 16>, dim3(items, a.qper), 16 * 32, 0, s, a);
  if (items <= 32) return launch_dependent(attn_join_kernel<NG, 8>, dim3(items, a.qper), 8 * 32, 0, s, a);
  return launch_dependent(attn_join_kernel<NG, 4>, dim3(a.by_item ? items : C::kGrid - 1, a.qper), 4 * 32, 0, s, a);
}

template <int NG, int NT>
qlin_status launch_widths(const AttnArgs& a, cudaStream_t s) {
  if (a.c.k_bits == 16) return launch<16, 16, NG, NT>(a, s);
  if (a.c.k_bits == 8) return a.c.v_bits == 8 ? launch<8, 8, NG, NT>(a, s) : launch<8, 4, NG, NT>(a, s);
  return a.c.v_bits == 8 ? launch<4, 8, NG, NT>(a, s) : launch<4, 4, NG, NT>(a, s);
}

struct Split {
  int nqb, qper, may_cut;
};

Split split_of(int page, int kv_heads, int q_heads, int max_pages) {
  Split s;
  const int group = q_heads / kv_heads;
  s.nqb = (group + kQ - 1) / kQ;
  s.qper = (group + s.nqb - 1) / s.nqb;
  s.may_cut = (int64_t)max_pages * page > kWholeTiles * kTile;
  return s;
}

}  // namespace

unsigned take_attn_error() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_attn_error, sizeof(v)) != cudaSuccess) return ~0u;
  if (v) cudaMemcpyToSymbol(g_attn_error, &zero, sizeof(zero));
  return v;
}

size_t attn_workspace_bytes(const qlin_kv_desc* d, int q_heads, int, int max_pages) {
  const Split s = split_of(d->page_size, d->kv_heads, q_heads, max_pages);
  if (!s.may_cut) return 0;
  return kRecordBytes + (size_t)kMaxTeams * 2 * s.qper * (d->head_dim + 4) * sizeof(float);
}

qlin_status launch_attn_decode(const KvView& c, const __half* q, int64_t q_stride, int q_heads,
                               const int32_t* block_table, int max_pages, const int32_t* seq_lens, int batch,
                               const uint32_t* sign_bits, float scale, __half* out, void* workspace, cudaStream_t s) {
  const Split sp = split_of(c.page, c.heads, q_heads, max_pages);
  AttnArgs a;
  a.c = c;
  a.q = q;
  a.q_stride = q_stride;
  a.table = block_table;
  a.lens = seq_lens;
  a.sign_bits = sign_bits;
  a.out = out;
  a.records = static_cast<int4*>(workspace);
  a.ws = sp.may_cut ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kRecordBytes) : nullptr;
  const int page_tiles = c.page / kTile;
  a.page_shift = page_tiles & (page_tiles - 1) ? -1 : __builtin_ctz(page_tiles);
  a.scale_log2e = scale * kLog2e;
  a.q_heads = q_heads;
  a.max_pages = max_pages;
  a.batch = batch;
  a.cap = max_pages * c.page;
  a.group = q_heads / c.heads;
  a.items = c.heads * sp.nqb;
  a.nqb = sp.nqb;
  a.qper = sp.qper;
  a.may_cut = sp.may_cut;
  a.by_item = (int64_t)batch * a.items <= kItemRecords;
  if (sp.qper > 4) return c.dim == kGroup ? launch_widths<1, 2>(a, s) : launch_widths<2, 2>(a, s);
  return c.dim == kGroup ? launch_widths<1, 1>(a, s) : launch_widths<2, 1>(a, s);
}

}  // namespace qlin
