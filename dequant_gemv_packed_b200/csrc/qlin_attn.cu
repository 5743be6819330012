// qlin_attn_decode: attention of one new token per sequence over the paged,
// quantised key/value cache (layout in qlin_kv.cuh).
//
// Mathematics.  With the codes q, scales s and zeros z of a token t and a query x
// (rotated once, fp16),
//   score_t = c s_k (sum_d q_k x - z_k sum_d x),   c = scale log2(e),
//   out_d   = sum_t w_t s_v (q_v - z_v) / sum_t w_t,   w_t = 2^(score_t - m).
// Scores of 4- and 8-bit keys are integer products, m16n8k32 of u8 codes and s8
// digits: per query and group x is xi 2^(E-13), E the exponent of the largest
// |x|, xi = 256 hi + lo (values within a factor 8 of the largest are exact, others
// rounded at 2^-14 of it, as in the M = 1 integer GEMV); sum q xi and sum xi are
// exact in int32.  The codes are the operand as stored (8 bits) or masked in place
// (4 bits; the odd codes are 16 q in accumulators of their own).
// Values: a nibble or byte masked into the low bits of an fp16 word is the
// subnormal fp16 number q 2^-24 (a nibble at bits 4-7: q 2^-20), and one packed
// multiplication makes a pair q 2^-9, exact.  (The subnormals would be exact
// operands too, but the tensor cores align products by the operands' exponent
// fields: their sums were off by 2^-16 of the products.)  The value's scale joins
// the exponent, P_t = 2^(score_t + log2 s_v - m) = w_t s_v, so that
//   out_d = (sum_t P_t q_v - z_v P_t) / sum_t P_t / s_v,
// and m follows the maximum of score + log2 s_v: P is the weight that the sum is
// really made of, whatever the sizes of the scales.  P enters the products as two
// fp16 digits, hi + 2^-11 lo (22 bits).  m is kept 7 to 15 binary orders below the
// maximum and moved only when a score exceeds it by 15, which a vote decides: after
// the first tile that is rare.
//
// The columns of both products are (query, digit) pairs, four queries in eight
// columns: lane (g, t) of an accumulator holds both digits of query t, so each lane
// has the scores of one query for tokens g and g + 8 (none is padding at the usual
// four queries a key), packs (hi, lo) of P as it is, and movmatrix turns that into
// the next product's operand; a query's statistics live in the lanes that scale its
// sums.  S^T = K Q^T has the tile's 16 tokens as rows, O^T = V^T P^T 16 dimensions.
// More than four queries take a second set of columns on the same decoded codes
// (kNt = 2), more than eight a second pass over the cache.
//
// Split.  A tile is 16 tokens of one (sequence, kv head, block of queries), an item
// all tiles of one.  Items in order, each its tiles plus a constant for what an item
// costs beside them, are cut into equal shares, one a team of warps, whatever the
// lengths (which only the device knows).  If some item has more than kWholeTiles
// tiles, the eight (or four) warps of a CTA are a team and items are cut; the pieces
// go to the workspace (at most two a team: its first and last) and a dependent
// kernel joins them in order.  Otherwise items stay whole and a team has as few
// warps as keep all teams busy, down to one: nothing is joined, no barrier is
// needed.  A team's warps take every T-th tile of its piece, each with its own
// statistics, joined in shared memory.
//
// A tile is brought in by its warp alone: 16-byte asynchronous copies into the
// warp's own ring of stages, swizzled so that both the K reads (rows g, g + 8,
// 16 bytes a lane) and the transposed V reads (rows 2t, 2t + 1, 2t + 8, 2t + 9)
// are free of bank conflicts; no barrier is needed but the warp's.
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
constexpr int kExtra = 2;          // an item's cost beside its tiles, in tiles of one warp
constexpr int kMaxTeams = 3 * kSms;  // teams when items are cut: one a CTA

template <int KB, int VB, int NG, int NT>
struct Cfg {
  static constexpr int kDim = NG * kGroup;
  static constexpr int kRowK = 16 * KB * NG, kRowV = 16 * VB * NG;  // bytes a token
  static constexpr int kPar = KB == 16 ? 0 : 8 * NG;
  static constexpr int kOffV = kTile * kRowK, kOffPar = kOffV + kTile * kRowV;
  static constexpr int kStage = kOffPar + kTile * kPar + 16;  // and a word: the tile's tokens
  // 32 accumulators a warp (one group, four queries) leave room for 16 warps an SM at 128
  // registers; 64 for 12 at 168, 128 for 8 at 255.  16-bit rows fill the rings: 8 warps.
  static constexpr int kSets = NG * NT;
  static constexpr int kWarps = (kSets > 1 || KB == 16) ? 4 : 8;
  static constexpr int kRowQ = 4 * NT;                          // queries
  static constexpr int kSmemQ = kWarps * NT * NG * 1024;        // operand of the queries, a team
  static constexpr int kSmemX = kWarps * kRowQ * NG * 8;        // (scale, sum) of each, a team
  static constexpr int kSmemMl = kWarps * kRowQ * NG * 8;       // (m, l), a warp
  static constexpr int kOther = kSmemQ + kSmemX + kSmemMl;
  static constexpr int fit(int ctas) { return (226 * 1024 / ctas - 1024 - kOther) / (kWarps * kStage); }
  static constexpr int kCtas = kSets == 2 && KB < 16 && fit(3) >= 2 ? 3 : fit(2) >= 2 ? 2 : 1;  // per SM
  static constexpr int kStages = fit(kCtas) > 6 ? 6 : fit(kCtas);
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kSmem = kRing + kOther;
  static constexpr int kGrid = kSms * kCtas;
  static constexpr int kDumpRow = kDim + 8;  // floats; over the warp's idle ring
  static_assert(kStages >= 2, "a stage to fill and one to read");
  static_assert(kRowQ * kDumpRow * 4 <= kStages * kStage, "sums fit the ring");
};

struct AttnArgs {
  KvView c;
  const __half* q;
  int64_t q_stride;
  const int32_t *table, *lens;
  const uint32_t* sign_bits;
  __half* out;
  float* ws;  // [teams][2] slots of [qper][dim + 4]: sums, then maximum and denominator per group
  float scale_log2e;
  int32_t q_heads, max_pages, batch, cap;  // cap: tokens the table can hold
  int32_t items, nqb, qper;                // (head, query block) pairs of a sequence; blocks; queries a block
  int32_t may_cut;                         // the table has room for more than kWholeTiles tiles
};

__device__ __forceinline__ int tiles_of(const AttnArgs& a, int b) {
  const int n = min(max(a.lens[b], 0), a.cap);
  return (n + kTile - 1) / kTile;
}

// How the items are dealt out; the same in every warp of both kernels.
struct Plan {
  int cut;    // whether items are cut
  int lt;     // log2 of a team's warps
  int extra;  // cost of an item beside its tiles, in tiles of its team
  int total, share;
};

__device__ __forceinline__ Plan make_plan(const AttnArgs& a, int lane, int grid, int warps) {
  int n = 0, top = 0, live = 0;
  for (int b = lane; b < a.batch; b += 32) {
    const int t = tiles_of(a, b);
    n += t;
    top = max(top, t);
    live += t > 0;
  }
  n = __reduce_add_sync(0xffffffffu, n);
  top = __reduce_max_sync(0xffffffffu, top);
  live = __reduce_add_sync(0xffffffffu, live) * a.items;
  Plan p;
  p.cut = a.may_cut && top > kWholeTiles;
  p.lt = 31 - __clz(warps);
  if (!p.cut)
    while (p.lt > 0 && live > grid * (warps >> p.lt)) --p.lt;
  p.extra = min(kExtra << p.lt, kItemExtra);
  p.total = n * a.items + live * p.extra;
  const int teams = grid * (warps >> p.lt);
  p.share = (int)(((int64_t)p.total + teams - 1) / teams);
  p.share = max(p.share, p.cut ? kMinShare : 1);
  return p;
}

// The sequence that position u (< total) belongs to, and its first position.
__device__ __forceinline__ void find_pos(const AttnArgs& a, const Plan& p, int lane, int u, int& b, int& first) {
  int before = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int t = b0 + lane < a.batch ? tiles_of(a, b0 + lane) : 0;
    const int n = t ? (t + p.extra) * a.items : 0;
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
__device__ __forceinline__ uint32_t low4(uint32_t w) { return scaled(w & 0x000F000Fu, kLow); }
__device__ __forceinline__ uint32_t high4(uint32_t w) { return scaled(w & 0x00F000F0u, kHigh); }
__device__ __forceinline__ uint32_t low8(uint32_t w) { return scaled(w & 0x00FF00FFu, kLow); }
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
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Byte offset of 16-byte piece c (of a group's row) of tile row r, for the K reads:
// eight lanes read pieces t, t + 4, ... of rows 2j and 2j + 1.
template <int KB>
__device__ __forceinline__ int k_at(int r, int c) {
  return r * 16 * KB + 16 * (KB == 4 ? c : c ^ ((r & 1) << 2));
}
// The same for the V reads: 4 bits, 16 lanes read 8 bytes of pieces 0, 1 (or 2, 3)
// of rows 2t; 8 bits, 8 lanes read pieces 2i, 2i + 1 of rows 2t; 16 bits, one piece
// of eight consecutive rows.
template <int VB>
__device__ __forceinline__ int v_at(int r, int c) {
  if (VB == 4) return (r >> 1) * 128 + ((r ^ (r >> 1)) & 1) * 64 + 16 * (c ^ ((r >> 1) & 2));
  if (VB == 8) return r * 128 + 16 * (c ^ (r & 6));
  return r * 256 + 16 * (c ^ (r & 7));
}

// Rotation (or its inverse) of the four values 4 lane .. 4 lane + 3 of block g.
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

// One head's finished sums, group g: four values a lane, rotated back and stored.
__device__ __forceinline__ void store_out(const AttnArgs& a, int b, int hq, int dim, int g, int lane, float (&r)[4],
                                          float den) {
  const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] *= inv;
  if (a.sign_bits) rotate4(r, a.sign_bits, g, lane, true);
  const __half2 h0 = __floats2half2_rn(r[0], r[1]), h1 = __floats2half2_rn(r[2], r[3]);
  uint2 w;
  w.x = *reinterpret_cast<const uint32_t*>(&h0);
  w.y = *reinterpret_cast<const uint32_t*>(&h1);
  *reinterpret_cast<uint2*>(a.out + ((int64_t)b * a.q_heads + hq) * dim + g * kGroup + 4 * lane) = w;
}

// Prepares query `q` of a team (rotation, fp16, digits or halves) in its shared operand.
//   16-bit keys: halves of query q at [q][dim]; below: digit planes [2 q + digit][dim], at 4
//   bits the dimensions of each eight in the order 0 2 4 6 1 3 5 7 (a word's even codes, its odd).
template <int KB, int NG>
__device__ __forceinline__ void prepare_query(const AttnArgs& a, const __half* src, bool live, int q, int lane,
                                              uint8_t* sq, float2* sx) {
  constexpr int D = NG * kGroup;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) {
      const uint2 r = *reinterpret_cast<const uint2*>(src + g * kGroup + 4 * lane);
      const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&r.x));
      const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
      v[0] = f0.x, v[1] = f0.y, v[2] = f1.x, v[3] = f1.y;
      if (a.sign_bits) rotate4(v, a.sign_bits, g, lane, false);
    }
    const __half2 h0 = __floats2half2_rn(v[0], v[1]), h1 = __floats2half2_rn(v[2], v[3]);
    if (KB == 16) {
      uint2 w;
      w.x = *reinterpret_cast<const uint32_t*>(&h0);
      w.y = *reinterpret_cast<const uint32_t*>(&h1);
      *reinterpret_cast<uint2*>(sq + (q * D + g * kGroup + 4 * lane) * 2) = w;
      if (lane == 0) sx[q * NG + g] = make_float2(a.scale_log2e, 0.f);
      continue;
    }
    v[0] = __low2float(h0), v[1] = __high2float(h0), v[2] = __low2float(h1), v[3] = __high2float(h1);
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) big = max(big, __float_as_uint(v[i]) & 0x7fffffffu);
    big = __reduce_max_sync(0xffffffffu, big);
    const int e = (int)(big >> 23) - 127;  // exponent of the largest (a half is a normal float, or 0)
    const float down = __uint_as_float((uint32_t)(127 + 13 - e) << 23), up = __uint_as_float((uint32_t)(127 - 13 + e) << 23);
    int xi[4], sum = 0;
    uint32_t hi = 0, lo = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      xi[i] = big ? __float2int_rn(v[i] * down) : 0;
      sum += xi[i];
      const int l = ((xi[i] + 128) & 255) - 128;
      hi |= (uint32_t)(((xi[i] - l) >> 8) & 255) << (8 * i);
      lo |= (uint32_t)(l & 255) << (8 * i);
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    uint8_t* row = sq + (2 * q) * D + g * kGroup;
    if (KB == 8) {
      *reinterpret_cast<uint32_t*>(row + 4 * lane) = hi;
      *reinterpret_cast<uint32_t*>(row + D + 4 * lane) = lo;
    } else {  // dimensions 4l .. 4l+3 of an eight: its bytes 2 (l & 1), + 1 (even) and 4 bytes on (odd)
      row += 8 * (lane >> 1) + 2 * (lane & 1);
      *reinterpret_cast<uint16_t*>(row) = (uint16_t)__byte_perm(hi, 0, 0x4420);
      *reinterpret_cast<uint16_t*>(row + 4) = (uint16_t)__byte_perm(hi, 0, 0x4431);
      *reinterpret_cast<uint16_t*>(row + D) = (uint16_t)__byte_perm(lo, 0, 0x4420);
      *reinterpret_cast<uint16_t*>(row + D + 4) = (uint16_t)__byte_perm(lo, 0, 0x4431);
    }
    // the sums of 4-bit codes are kept times 16; a query with an infinity or NaN has no scale
    const float unit = KB == 4 ? 0.0625f : 1.f;
    const float f = big >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : big ? a.scale_log2e * up * unit : 0.f;
    if (lane == 0) sx[q * NG + g] = make_float2(f, (float)sum / unit);
  }
}

template <int KB, int VB, int NG, int NT>
__global__ void __launch_bounds__(Cfg<KB, VB, NG, NT>::kWarps * 32, Cfg<KB, VB, NG, NT>::kCtas)
    attn_kernel(const __grid_constant__ AttnArgs a) {
  using C = Cfg<KB, VB, NG, NT>;
  constexpr int NW = C::kWarps, S = C::kStages, D = C::kDim;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
  const int grid = gridDim.x, page_tiles = a.c.page / kTile;
  uint8_t* const ring_ptr = smem + warp * S * C::kStage;
  const uint32_t ring = smem_addr(ring_ptr);

  if (a.may_cut && threadIdx.x == 0) grid_launch_dependents();
  // sequences without tokens
  for (int b = blockIdx.x; b < a.batch; b += grid) {
    const int n = a.lens[b];
    if (n > a.cap && threadIdx.x == 0) atomicOr(&g_attn_error, kKvBadLength);
    if (n <= 0)
      for (int i = threadIdx.x; i < a.q_heads * D / 8; i += NW * 32)
        reinterpret_cast<uint4*>(a.out + (int64_t)b * a.q_heads * D)[i] = make_uint4(0u, 0u, 0u, 0u);
  }

  const Plan plan = make_plan(a, lane, grid, NW);
  const int lt = plan.lt, T = 1 << lt, team = warp >> lt, tw = warp & (T - 1);
  const int teams = NW >> lt, worker = blockIdx.x * teams + team;
  uint8_t* sq = smem + C::kRing + team * (NT * NG * 1024);
  float2* sx = reinterpret_cast<float2*>(smem + C::kRing + C::kSmemQ) + team * C::kRowQ * NG;
  float2* sml = reinterpret_cast<float2*>(smem + C::kRing + C::kSmemQ + C::kSmemX) + (warp - tw) * C::kRowQ * NG;
  auto team_barrier = [&]() {
    if (lt)
      named_barrier(1 + team, 32 << lt);
    else
      __syncwarp();
  };

  const int64_t begin = (int64_t)worker * plan.share;
  if (begin >= plan.total) return;
  int u = (int)begin;
  const int end = (int)min((int64_t)plan.total, begin + plan.share);
  int b, first;
  find_pos(a, plan, lane, u, b, first);
  int nt = tiles_of(a, b), cost = nt + plan.extra;
  if (!plan.cut && (u - first) % cost) u += cost - (u - first) % cost;  // items that start in the share
  const int group = a.q_heads / a.c.heads;
  while (u < end) {
    while (nt == 0 || u - first >= cost * a.items) {  // the next sequence that has tokens
      if (nt) first += cost * a.items;
      ++b;
      nt = tiles_of(a, b);
      cost = nt + plan.extra;
    }
    const int item = (u - first) / cost, at = (u - first) % cost;
    const int until = plan.cut ? min(cost, at + end - u) : cost;
    u += until - at;
    const int tile0 = max(at - plan.extra, 0), n = max(until - plan.extra, 0) - tile0;
    if (n <= 0) continue;
    const int len = min(a.lens[b], a.cap);
    const int h = item / a.nqb, q0 = (item % a.nqb) * a.qper;
    const int nq = min(a.qper, group - q0);
    const int hq0 = h * group + q0;

    // ---- the warp's tiles: tile0 + tw + T k, k < cnt; pages of 32 of them in registers
    const int cnt = tw < n ? (n - tw + T - 1) >> lt : 0;
    int pages = 0, offs = 0;
    auto issue = [&](int k) {
      if (k < cnt) {
        if ((k & 31) == 0) {
          const int kk = k + lane;
          pages = -1;
          if (kk < cnt) {
            const int tile = tile0 + tw + (kk << lt);
            pages = a.table[(int64_t)b * a.max_pages + tile / page_tiles];
            offs = (tile % page_tiles) * kTile;
          }
        }
        int p = __shfl_sync(0xffffffffu, pages, k & 31);
        const int off = __shfl_sync(0xffffffffu, offs, k & 31);
        int valid = min(kTile, len - (tile0 + tw + (k << lt)) * kTile);
        if ((unsigned)p >= (unsigned)a.c.pages) {
          if (lane == 0) atomicOr(&g_attn_error, kKvBadPage);
          p = 0;
          valid = 0;
        }
        const int stage = (k % S) * C::kStage;
        const uint32_t st = ring + stage;
        const uint8_t* blk = a.c.block(p, h);
        const uint8_t* src = blk + (int64_t)off * C::kRowK + 16 * lane;
#pragma unroll
        for (int j = 0; j < KB * NG / 2; ++j) {
          const int i = lane + 32 * j, r = i / (KB * NG), c = i % (KB * NG);
          cp16(st + (c / KB) * (kTile * 16 * KB) + k_at<KB>(r, c % KB), src + 512 * j);
        }
        src = blk + a.c.v_offset() + (int64_t)off * C::kRowV + 16 * lane;
#pragma unroll
        for (int j = 0; j < VB * NG / 2; ++j) {
          const int i = lane + 32 * j, r = i / (VB * NG), c = i % (VB * NG);
          const uint32_t dst = st + C::kOffV + (c / VB) * (kTile * 16 * VB) + v_at<VB>(r, c % VB);
          // 16-bit values past the length could be NaN, which a weight of zero would not hide
          if (VB == 16)
            cp16_or_zero(dst, src + 512 * j, r < valid);
          else
            cp16(dst, src + 512 * j);
        }
        if (C::kPar) {
          if (lane < kTile * C::kPar / 16)
            cp16(st + C::kOffPar + 16 * lane, blk + a.c.par_offset() + (int64_t)off * C::kPar + 16 * lane);
        }
        if (lane == 0) *reinterpret_cast<int*>(ring_ptr + stage + C::kStage - 16) = valid;
      }
      cp_commit();
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) issue(k);

    // ---- the queries, and the lane's operand: column g8 = (query g8 / 2, digit g8 % 2), the
    // dimensions of the codes that lanes of column t4 hold
    for (int q = tw; q < C::kRowQ; q += T)
      prepare_query<KB, NG>(a, a.q + (int64_t)b * a.q_stride + (int64_t)(hq0 + q) * D, q < nq, q, lane, sq, sx);
    team_barrier();
    constexpr int NB = KB == 16 ? 16 : 8;  // operand registers a group
    uint32_t qf[NT][NG][NB];
    float xs[NT][NG], sc[NT][NG];  // sum and scale of query t4
#pragma unroll
    for (int s = 0; s < NT; ++s)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t base = smem_addr(sq);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (KB == 16) {  // piece t4 + 4 j of query g8 / 2; the odd columns are zero
            uint4 p = ld128(base + ((4 * s + (g8 >> 1)) * D + g * kGroup + 32 * j + 8 * t4) * 2);
            if (g8 & 1) p = make_uint4(0u, 0u, 0u, 0u);
            qf[s][g][(4 * j) % NB] = p.x, qf[s][g][(4 * j + 1) % NB] = p.y;
            qf[s][g][(4 * j + 2) % NB] = p.z, qf[s][g][(4 * j + 3) % NB] = p.w;
          } else {  // eight dimensions: 4 bits, word j of piece t4; 8 bits, words 2 (j & 1), + 1 of piece t4 + 4 (j / 2)
            const int d0 = KB == 4 ? 32 * t4 + 8 * j : 64 * (j >> 1) + 16 * t4 + 8 * (j & 1);
            const uint2 p = ld64(base + (8 * s + g8) * D + g * kGroup + d0);
            qf[s][g][2 * j] = p.x, qf[s][g][2 * j + 1] = p.y;
          }
        }
        const float2 x = sx[(4 * s + t4) * NG + g];
        sc[s][g] = x.x, xs[s][g] = x.y;
      }

    float o[NT][NG][8][4], m[NT][NG], l[NT][NG], zc[NT][NG];
#pragma unroll
    for (int s = 0; s < NT; ++s)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[s][g][j][0] = o[s][g][j][1] = o[s][g][j][2] = o[s][g][j][3] = 0.f;
        m[s][g] = kNone;
        l[s][g] = zc[s][g] = 0.f;
      }

    for (int k = 0; k < cnt; ++k) {
      cp_wait<S - 2>();
      __syncwarp();
      issue(k + S - 1);  // into the stage that the previous tile has left
      const int stage = (k % S) * C::kStage;
      const uint32_t st = ring + stage;
      const int valid = *reinterpret_cast<const volatile int*>(ring_ptr + stage + C::kStage - 16);

      // scores in units of log2: query t4 (+ 4 s), tokens g8 and g8 + 8
      float w[NT][2];
      float lv[NG][2], rv[NG][2], vz[NG][2];
#pragma unroll
      for (int s = 0; s < NT; ++s) w[s][0] = w[s][1] = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float dot[NT][2];
        const uint32_t kb = st + g * (kTile * 16 * KB);
        if (KB == 4) {
          const uint4 wa = ld128(kb + k_at<KB>(g8, t4)), wb = ld128(kb + k_at<KB>(g8 + 8, t4));
          const uint32_t ra[4] = {wa.x, wa.y, wa.z, wa.w}, rb[4] = {wb.x, wb.y, wb.z, wb.w};
          int c0[NT][4], c1[NT][4];
#pragma unroll
          for (int s = 0; s < NT; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) c0[s][i] = c1[s][i] = 0;
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            constexpr uint32_t lo = 0x0F0F0F0Fu, hi = 0xF0F0F0F0u;
#pragma unroll
            for (int s = 0; s < NT; ++s) {
              imma(c0[s], ra[j] & lo, rb[j] & lo, ra[j + 1] & lo, rb[j + 1] & lo, qf[s][g][2 * j], qf[s][g][2 * j + 2]);
              imma(c1[s], ra[j] & hi, rb[j] & hi, ra[j + 1] & hi, rb[j + 1] & hi, qf[s][g][2 * j + 1],
                   qf[s][g][2 * j + 3]);
            }
          }
#pragma unroll
          for (int s = 0; s < NT; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              dot[s][i] = (float)((16 * c0[s][2 * i] + c1[s][2 * i]) * 256 + (16 * c0[s][2 * i + 1] + c1[s][2 * i + 1]));
        } else if (KB == 8) {
          int c0[NT][4], c1[NT][4];
#pragma unroll
          for (int s = 0; s < NT; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) c0[s][i] = c1[s][i] = 0;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 wa = ld128(kb + k_at<KB>(g8, t4 + 4 * j)), wb = ld128(kb + k_at<KB>(g8 + 8, t4 + 4 * j));
#pragma unroll
            for (int s = 0; s < NT; ++s) {
              imma(c0[s], wa.x, wb.x, wa.y, wb.y, qf[s][g][4 * j], qf[s][g][4 * j + 1]);
              imma(c1[s], wa.z, wb.z, wa.w, wb.w, qf[s][g][4 * j + 2], qf[s][g][4 * j + 3]);
            }
          }
#pragma unroll
          for (int s = 0; s < NT; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              dot[s][i] = (float)((c0[s][2 * i] + c1[s][2 * i]) * 256 + (c0[s][2 * i + 1] + c1[s][2 * i + 1]));
        } else {
          float c0[NT][4], c1[NT][4];
#pragma unroll
          for (int s = 0; s < NT; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) c0[s][i] = c1[s][i] = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 wa = ld128(kb + k_at<KB>(g8, t4 + 4 * j)), wb = ld128(kb + k_at<KB>(g8 + 8, t4 + 4 * j));
#pragma unroll
            for (int s = 0; s < NT; ++s) {
              mma(c0[s], wa.x, wb.x, wa.y, wb.y, qf[s][g][(4 * j) % NB], qf[s][g][(4 * j + 1) % NB]);
              mma(c1[s], wa.z, wb.z, wa.w, wb.w, qf[s][g][(4 * j + 2) % NB], qf[s][g][(4 * j + 3) % NB]);
            }
          }
#pragma unroll
          for (int s = 0; s < NT; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) dot[s][i] = c0[s][2 * i] + c1[s][2 * i];
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
            // a scale of 0 (a slot that was cleared, never written) is 2^-100 here: its token has a
            // share of the denominator and none of the sums
            lv[g][i] = fmaxf(lg2(pv.x), -100.f);
            rv[g][i] = fminf(rcp(pv.x), 0x1p100f);
            vz[g][i] = pv.y;
          } else {
#pragma unroll
            for (int s = 0; s < NT; ++s) w[s][i] = fmaf(dot[s][i], sc[s][g], w[s][i]);
            lv[g][i] = vz[g][i] = 0.f;
            rv[g][i] = 1.f;
          }
        }
      }
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

      uint32_t pb[NT][NG][2];
#pragma unroll
      for (int s = 0; s < NT; ++s)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float y[2] = {w[s][0] + lv[g][0], w[s][1] + lv[g][1]};
          float top = fmaxf(y[0], y[1]);
          if (__any_sync(0xffffffffu, top > m[s][g] + 15.f)) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float next = fmaxf(m[s][g], top - 7.f), f = ex2(m[s][g] - next);
            m[s][g] = next;
            l[s][g] *= f, zc[s][g] *= f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[s][g][j][i] *= f;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float p = ex2(y[i] - m[s][g]), hi = __half2float(__float2half_rn(p));
            const __half2 both = __floats2half2_rn(p, (p - hi) * 2048.f);
            pb[s][g][i] = movmatrix(*reinterpret_cast<const uint32_t*>(&both));
            l[s][g] = fmaf(p, rv[g][i], l[s][g]);
            if (C::kPar) zc[s][g] = fmaf(p, vz[g][i], zc[s][g]);
          }
        }

      // values: the lane's tokens 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9, dimensions 16 g8 .. 16 g8 + 15
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t vb = st + C::kOffV + g * (kTile * 16 * VB);
        if (VB == 4) {
          uint2 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = ld64(vb + v_at<VB>(2 * t4 + (i & 1) + 8 * (i >> 1), g8 >> 1) + 8 * (g8 & 1));
#pragma unroll
          for (int half = 0; half < 4; ++half) {  // four dimensions: a half-word of each token
            const uint32_t sel = (half & 1) ? 0x7632u : 0x5410u;
            const uint32_t x = half < 2 ? __byte_perm(v[0].x, v[1].x, sel) : __byte_perm(v[0].y, v[1].y, sel);
            const uint32_t y = half < 2 ? __byte_perm(v[2].x, v[3].x, sel) : __byte_perm(v[2].y, v[3].y, sel);
            const uint32_t x0 = low4(x), x2 = low4(x >> 8), y0 = low4(y), y2 = low4(y >> 8);
            const uint32_t x1 = high4(x), x3 = high4(x >> 8), y1 = high4(y), y3 = high4(y >> 8);
#pragma unroll
            for (int s = 0; s < NT; ++s) {
              mma(o[s][g][2 * half], x0, x2, y0, y2, pb[s][g][0], pb[s][g][1]);
              mma(o[s][g][2 * half + 1], x1, x3, y1, y3, pb[s][g][0], pb[s][g][1]);
            }
          }
        } else if (VB == 8) {
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = ld128(vb + v_at<VB>(2 * t4 + (i & 1) + 8 * (i >> 1), g8));
          const uint32_t v0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, v1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
          const uint32_t v2[4] = {v[2].x, v[2].y, v[2].z, v[2].w}, v3[4] = {v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
          for (int j = 0; j < 8; ++j) {  // two dimensions: a half-word of each token
            const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
            const uint32_t x = __byte_perm(v0[j >> 1], v1[j >> 1], sel), y = __byte_perm(v2[j >> 1], v3[j >> 1], sel);
            const uint32_t x0 = low8(x), x1 = low8(x >> 8), y0 = low8(y), y1 = low8(y >> 8);
#pragma unroll
            for (int s = 0; s < NT; ++s) mma(o[s][g][j], x0, x1, y0, y1, pb[s][g][0], pb[s][g][1]);
          }
        } else {
          const int r = (lane & 7) + 8 * (lane >> 4), c = (lane >> 3) & 1;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 v = ldmatrix_x4_trans(vb + v_at<VB>(r, 2 * j + c));
#pragma unroll
            for (int s = 0; s < NT; ++s) mma(o[s][g][j], v.x, v.y, v.z, v.w, pb[s][g][0], pb[s][g][1]);
          }
        }
      }
    }
    cp_wait<0>();
    __syncwarp();  // the warp has left its ring

    // ---- the warp's sums [query][dim] over its ring, then the team's
#pragma unroll
    for (int s = 0; s < NT; ++s)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          l[s][g] += __shfl_xor_sync(0xffffffffu, l[s][g], d);
          zc[s][g] += __shfl_xor_sync(0xffffffffu, zc[s][g], d);
        }
        float* row = reinterpret_cast<float*>(ring_ptr) + (4 * s + t4) * C::kDumpRow + g * kGroup;
#pragma unroll
        for (int j = 0; j < 8; j += (VB == 16 ? 1 : 2)) {
          const float(&e)[4] = o[s][g][j];
          const float e0 = fmaf(e[1], 0x1p-11f, e[0]), e1 = fmaf(e[3], 0x1p-11f, e[2]);
          if (VB == 16) {
            row[16 * j + g8] = e0, row[16 * j + 8 + g8] = e1;
          } else {
            const float(&f)[4] = o[s][g][(j + 1) & 7];
            const float f0 = fmaf(f[1], 0x1p-11f, f[0]), f1 = fmaf(f[3], 0x1p-11f, f[2]), z = -zc[s][g];
            const float r0 = fmaf(e0, 512.f, z), r1 = fmaf(e1, 512.f, z), r2 = fmaf(f0, 512.f, z), r3 = fmaf(f1, 512.f, z);
            // 4 bits: rows (0, 2) and (1, 3) of four dimensions; 8 bits: (0, 1) and (2, 3)
            *reinterpret_cast<float4*>(row + 16 * g8 + 2 * j) =
                VB == 4 ? make_float4(r0, r2, r1, r3) : make_float4(r0, r1, r2, r3);
          }
        }
        if (g8 == 0) sml[(tw * C::kRowQ + 4 * s + t4) * NG + g] = make_float2(m[s][g], l[s][g]);
      }
    team_barrier();
    const bool whole = n == nt;
    for (int q = tw; q < nq; q += T)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float top = kNone, den = 0.f, r[4] = {0.f, 0.f, 0.f, 0.f};
        for (int i = 0; i < T; ++i) top = fmaxf(top, sml[(i * C::kRowQ + q) * NG + g].x);
        for (int i = 0; i < T; ++i) {
          const float2 ml = sml[(i * C::kRowQ + q) * NG + g];
          const float f = ex2(ml.x - top);
          const float4 v = *reinterpret_cast<const float4*>(
              reinterpret_cast<const float*>(smem + (warp - tw + i) * S * C::kStage) + q * C::kDumpRow + g * kGroup +
              4 * lane);
          den = fmaf(f, ml.y, den);
          r[0] = fmaf(f, v.x, r[0]), r[1] = fmaf(f, v.y, r[1]), r[2] = fmaf(f, v.z, r[2]), r[3] = fmaf(f, v.w, r[3]);
        }
        if (whole) {
          store_out(a, b, hq0 + q, D, g, lane, r, den);
        } else {  // slot 0: the item began in an earlier team's share; slot 1: here
          float* slot = a.ws + ((int64_t)worker * 2 + (tile0 == 0)) * a.qper * (D + 4) + q * (D + 4);
          *reinterpret_cast<float4*>(slot + g * kGroup + 4 * lane) = make_float4(r[0], r[1], r[2], r[3]);
          if (lane == 0) slot[D + 2 * g] = top, slot[D + 2 * g + 1] = den;
        }
      }
    team_barrier();  // rings and queries may be overwritten
  }
}

// Joins the pieces of the item that is cut between shares blockIdx.x and
// blockIdx.x + 1, if no earlier cut is inside it; one query a block, four warps over
// its pieces.
template <int NG>
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ AttnArgs a, int grid, int warps) {
  constexpr int D = NG * kGroup;
  __shared__ float so[4][D], sm[4][NG], sl[4][NG];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Plan plan = make_plan(a, lane, grid, warps);
  const int64_t cut64 = (int64_t)(blockIdx.x + 1) * plan.share;
  bool mine = plan.cut && cut64 < plan.total;
  const int cut = (int)cut64, group = a.q_heads / a.c.heads, q = blockIdx.y;
  int b = 0, h = 0, q0 = 0, last = 0;
  if (mine) {
    int first = 0;
    find_pos(a, plan, lane, cut, b, first);
    const int nt = tiles_of(a, b), cost = nt + plan.extra, item = (cut - first) / cost;
    const int from = first + item * cost + plan.extra;  // position of the item's first tile
    last = from + nt - 1;
    h = item / a.nqb, q0 = (item % a.nqb) * a.qper;
    // inside the tiles, and the first cut there
    mine = cut > from && cut - plan.share <= from && q < min(a.qper, group - q0);
  }
  grid_dependency_wait();  // every block: this grid's end stands for the first one's too
  if (!mine) return;
  const int c0 = blockIdx.x, c1 = last / plan.share;  // its teams
  float top[NG], den[NG], r[NG][4];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    top[g] = kNone, den[g] = 0.f;
    r[g][0] = r[g][1] = r[g][2] = r[g][3] = 0.f;
  }
#pragma unroll 4
  for (int c = c0 + warp; c <= c1; c += 4) {
    const float* slot = a.ws + ((int64_t)c * 2 + (c == c0)) * a.qper * (D + 4) + q * (D + 4);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const float2 ml = *reinterpret_cast<const float2*>(slot + D + 2 * g);
      const float4 v = *reinterpret_cast<const float4*>(slot + g * kGroup + 4 * lane);
      const float n = fmaxf(top[g], ml.x), f = ex2(top[g] - n), e = ex2(ml.x - n);
      top[g] = n;
      den[g] = den[g] * f + e * ml.y;
      r[g][0] = r[g][0] * f + e * v.x, r[g][1] = r[g][1] * f + e * v.y;
      r[g][2] = r[g][2] * f + e * v.z, r[g][3] = r[g][3] * f + e * v.w;
    }
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    *reinterpret_cast<float4*>(&so[warp][g * kGroup + 4 * lane]) = make_float4(r[g][0], r[g][1], r[g][2], r[g][3]);
    if (lane == 0) sm[warp][g] = top[g], sl[warp][g] = den[g];
  }
  __syncthreads();
  if (warp >= NG) return;
  const int g = warp;
  float t = kNone, d = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int w = 0; w < 4; ++w) t = fmaxf(t, sm[w][g]);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float f = ex2(sm[w][g] - t);
    d = fmaf(f, sl[w][g], d);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fmaf(f, so[w][g * kGroup + 4 * lane + i], v[i]);
  }
  store_out(a, b, h * group + q0 + q, D, g, lane, v, d);
}

template <int KB, int VB, int NG, int NT>
qlin_status launch(const AttnArgs& a, cudaStream_t s) {
  using C = Cfg<KB, VB, NG, NT>;
  static_assert(C::kSmem <= 227 * 1024 && C::kGrid <= kMaxTeams, "launch bounds");
  static std::atomic<unsigned long long> configured{0};  // per-device attribute, set once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return record_cuda(e);
  if (dev >= 64 || !((configured.load(std::memory_order_acquire) >> dev) & 1ull)) {
    e = cudaFuncSetAttribute(attn_kernel<KB, VB, NG, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return record_cuda(e);
    if (dev < 64) configured.fetch_or(1ull << dev, std::memory_order_release);
  }
  attn_kernel<KB, VB, NG, NT><<<C::kGrid, C::kWarps * 32, C::kSmem, s>>>(a);
  const qlin_status r = record_cuda(cudaGetLastError());
  if (r != QLIN_OK || !a.may_cut) return r;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C::kGrid - 1, a.qper);
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return record_cuda(cudaLaunchKernelEx(&cfg, attn_join_kernel<NG>, a, (int)C::kGrid, (int)C::kWarps));
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
  return (size_t)kMaxTeams * 2 * s.qper * (d->head_dim + 4) * sizeof(float);
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
  a.ws = static_cast<float*>(workspace);
  a.scale_log2e = scale * kLog2e;
  a.q_heads = q_heads;
  a.max_pages = max_pages;
  a.batch = batch;
  a.cap = max_pages * c.page;
  a.items = c.heads * sp.nqb;
  a.nqb = sp.nqb;
  a.qper = sp.qper;
  a.may_cut = sp.may_cut;
  if (sp.qper > 4) return c.dim == kGroup ? launch_widths<1, 2>(a, s) : launch_widths<2, 2>(a, s);
  return c.dim == kGroup ? launch_widths<1, 1>(a, s) : launch_widths<2, 1>(a, s);
}

}  // namespace qlin
