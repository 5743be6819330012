// qlin_attn_decode: attention of one new token per sequence over the paged,
// quantised key/value cache (layout in qlin_kv.cuh).
//
// Mathematics.  With the codes q, scales s and zeros z of a token t and a query x
// (rotated once, fp16),
//   score_t = c s_k (sum_d q_k x - z_k sum_d x),   c = scale log2(e),
//   out_d   = sum_t w_t s_v (q_v - z_v) / sum_t w_t,   w_t = 2^(score_t - m).
// The codes enter the tensor cores unconverted: a nibble or byte masked into the low
// bits of an fp16 word IS the subnormal fp16 number q 2^-24 (a nibble at bits 4-7:
// q 2^-20), and one packed multiplication makes a pair q 2^-9, exact, with no offset
// to cancel.  (The subnormals themselves would be exact operands too, but the
// tensor cores align the products by the operands' exponent fields: sums of
// subnormals carried errors of 2^-16 of the products, measured against 64 bits.)
// The value's scale joins
// the exponent, P_t = 2^(score_t + log2 s_v - m) = w_t s_v, so that
//   out_d = (sum_t P_t q_v - sum_t P_t z_v) / sum_t P_t / s_v,
// and m is the running maximum of score + log2 s_v: P is the weight that the sum
// is really made of, whatever the sizes of the scales.  P is rounded to fp16 (the
// tensor cores' operand); the same rounded P stands in the zero's share and in the
// denominator, so a rounding moves the weights but not their normalisation (a
// subnormal P, 2^21 below the largest, enters the denominator unrounded: a token
// with a tiny scale may hold most of the weight).  m is kept 7 to 15 binary
// orders below the maximum and only moved when a score exceeds it by 15, which a
// vote decides: after the first tile that is rare, and the 2^15 of room keeps the
// weights above fp16's subnormals down to 2^-21..2^-29 of the largest.
//
// Split.  The unit is a tile of 16 tokens of one (sequence, kv head, up to 8
// queries); the tiles of all sequences in order are cut into equal shares, one a
// CTA, whatever the lengths (which only the device knows).  A share's piece of one
// (sequence, head) is a segment; a CTA's warps take every NW-th tile of a segment,
// each with its own statistics, and are joined in shared memory.  A segment that
// is a whole sequence is finished there; pieces are written to the workspace (at
// most two a CTA: its first and last) and a second, dependent kernel joins them in
// order.  If no sequence can hold more than kWholeTiles tiles (the block table's
// width tells), sequences are not cut and the second kernel is not launched.
//
// A tile is brought in by its warp alone: 16-byte asynchronous copies into the
// warp's own ring of stages, swizzled so that both the K reads (rows g, g + 8,
// 16 bytes a lane) and the transposed V reads (rows 2t, 2t + 1, 2t + 8, 2t + 9)
// are free of bank conflicts; no barrier is needed but the warp's.
//
// Products (m16n8k16, fp32 accumulation): S^T = K Q^T with the tile's 16 tokens as
// rows and 8 queries as columns, O^T = V^T P^T with 16 dimensions as rows.  The
// accumulator layout of S^T, packed to fp16 and transposed by movmatrix, is the
// operand P^T; both accumulators have queries 2t, 2t + 1 in lane (g, t), so a
// query's statistics live in the lanes that scale its sums.
#include <atomic>

#include "qlin_kv.cuh"
#include "qlin_sm100.cuh"

namespace qlin {
namespace {

__device__ unsigned int g_attn_error;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = kPageUnit;  // tokens
constexpr int kQ = 8;             // queries a segment: columns of one product
constexpr int kSms = 148;
constexpr float kNone = -1e30f;   // running maximum of a warp that has seen no token
constexpr int kWholeTiles = 32;   // sequences up to here are not cut
constexpr int kMinShare = 16;     // tiles a CTA when they are

template <int KB, int VB, int NG>
struct Cfg {
  static constexpr int kDim = NG * kGroup;
  static constexpr int kRowK = 16 * KB * NG, kRowV = 16 * VB * NG;  // bytes a token
  static constexpr int kPar = KB == 16 ? 0 : 8 * NG;
  static constexpr int kOffV = kTile * kRowK, kOffPar = kOffV + kTile * kRowV;
  static constexpr int kStage = kOffPar + kTile * kPar + 16;  // and a word: the tile's tokens
  static constexpr int kWarps = (NG == 2 || KB == 16) ? 4 : 8;
  static constexpr int kFit = (104 * 1024) / (kWarps * kStage);  // two CTAs an SM
  static constexpr int kStages = kFit < 3 ? 3 : kFit > 6 ? 6 : kFit;
  static constexpr int kJoinRow = kDim + 4;  // floats; the padding spreads the warps' rows over the banks
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kJoin = kWarps * kQ * kJoinRow * 4;  // over the idle ring
  static constexpr int kBuf = kRing > kJoin ? kRing : kJoin;
  static constexpr int kSmemQ = kQ * kDim * 2, kSmemX = kQ * NG * 4, kSmemMl = kWarps * kQ * NG * 8;
  static constexpr int kSmem = kBuf + kSmemQ + kSmemX + kSmemMl;
  static constexpr int kCtas = kSmem <= 113 * 1024 ? 2 : 1;  // per SM
  static constexpr int kGrid = kSms * kCtas;
};

struct AttnArgs {
  KvView c;
  const __half* q;
  int64_t q_stride;
  const int32_t *table, *lens;
  const uint32_t* sign_bits;
  __half* out;
  float* ws;  // [grid][2] slots of [qper][dim + 4]: sums, then maximum and denominator per group
  float scale_log2e;
  int32_t q_heads, max_pages, batch, cap;  // cap: tokens the table can hold
  int32_t items, nqb, qper;                // (head, query block) pairs of a sequence; blocks; queries a block
  int32_t split;
};

__device__ __forceinline__ int tiles_of(const AttnArgs& a, int b) {
  const int n = min(max(a.lens[b], 0), a.cap);
  return (n + kTile - 1) / kTile;
}

// Tiles of all sequences and items; every lane gets the sum.
__device__ __forceinline__ int total_tiles(const AttnArgs& a, int lane) {
  int n = 0;
  for (int b = lane; b < a.batch; b += 32) n += tiles_of(a, b);
#pragma unroll
  for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n * a.items;
}

// The sequence that tile u (< total) belongs to, and its first tile.
__device__ __forceinline__ void find_tile(const AttnArgs& a, int lane, int u, int& b, int& first) {
  int before = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int n = b0 + lane < a.batch ? tiles_of(a, b0 + lane) * a.items : 0;
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int p = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += p;
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

__device__ __forceinline__ int share_of(const AttnArgs& a, int total, int grid) {
  const int s = (int)(((int64_t)total + grid - 1) / grid);
  return a.split ? max(s, kMinShare) : max(s, 1);
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

template <int KB, int VB, int NG>
__global__ void __launch_bounds__(Cfg<KB, VB, NG>::kWarps * 32, Cfg<KB, VB, NG>::kCtas)
    attn_kernel(const __grid_constant__ AttnArgs a) {
  using C = Cfg<KB, VB, NG>;
  constexpr int NW = C::kWarps, S = C::kStages, D = C::kDim;
  extern __shared__ __align__(128) uint8_t smem[];
  __half* sq = reinterpret_cast<__half*>(smem + C::kBuf);                           // [kQ][D] queries
  float* sx = reinterpret_cast<float*>(smem + C::kBuf + C::kSmemQ);                 // [kQ][NG] their sums
  float2* sml = reinterpret_cast<float2*>(smem + C::kBuf + C::kSmemQ + C::kSmemX);  // [NW][kQ][NG] (m, l)
  float* sj = reinterpret_cast<float*>(smem);                                       // [NW][kQ][kJoinRow]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, t4 = lane & 3;
  const uint32_t ring = smem_addr(smem) + warp * S * C::kStage;
  const int grid = gridDim.x, page_tiles = a.c.page / kTile;

  if (a.split && threadIdx.x == 0) grid_launch_dependents();
  // sequences without tokens
  for (int b = blockIdx.x; b < a.batch; b += grid) {
    const int n = a.lens[b];
    if (n > a.cap && threadIdx.x == 0) atomicOr(&g_attn_error, kKvBadLength);
    if (n <= 0)
      for (int i = threadIdx.x; i < a.q_heads * D / 8; i += NW * 32)
        reinterpret_cast<uint4*>(a.out + (int64_t)b * a.q_heads * D)[i] = make_uint4(0u, 0u, 0u, 0u);
  }

  const int total = total_tiles(a, lane), share = share_of(a, total, grid);
  const int64_t begin = (int64_t)blockIdx.x * share;
  if (begin >= total) return;
  int u = (int)begin;
  const int end = (int)min((int64_t)total, begin + share);
  int b, first;
  find_tile(a, lane, u, b, first);
  int nt = tiles_of(a, b);
  if (!a.split && (u - first) % nt) {  // whole segments only: those that start in the share
    u += nt - (u - first) % nt;
  }
  while (u < end) {
    while (u - first >= nt * a.items) {  // the next sequence that has tokens
      first += nt * a.items;
      ++b;
      nt = tiles_of(a, b);
    }
    const int item = (u - first) / nt, tile0 = (u - first) % nt;
    const int n = a.split ? min(nt - tile0, end - u) : nt;
    const int len = min(a.lens[b], a.cap);
    const int h = item / a.nqb, q0 = (item % a.nqb) * a.qper;
    const int group = a.q_heads / a.c.heads;
    const int nq = min(a.qper, group - q0);
    const int hq0 = h * group + q0;

    // ---- the warp's tiles: tile0 + warp + NW k, k < cnt; pages of 32 of them in registers
    const int cnt = warp < n ? (n - warp + NW - 1) / NW : 0;
    int pages = 0, offs = 0;
    auto issue = [&](int k) {
      if (k < cnt) {
        if ((k & 31) == 0) {
          const int kk = k + lane;
          pages = -1;
          if (kk < cnt) {
            const int tile = tile0 + warp + NW * kk;
            pages = a.table[(int64_t)b * a.max_pages + tile / page_tiles];
            offs = (tile % page_tiles) * kTile;
          }
        }
        int p = __shfl_sync(0xffffffffu, pages, k & 31);
        const int off = __shfl_sync(0xffffffffu, offs, k & 31);
        int valid = min(kTile, len - (tile0 + warp + NW * k) * kTile);
        if ((unsigned)p >= (unsigned)a.c.pages) {
          if (lane == 0) atomicOr(&g_attn_error, kKvBadPage);
          p = 0;
          valid = 0;
        }
        const uint32_t st = ring + (k % S) * C::kStage;
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
        if (lane == 0) *reinterpret_cast<int*>(smem + (st - smem_addr(smem)) + C::kStage - 16) = valid;
      }
      cp_commit();
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) issue(k);

    // ---- the queries: rotated, rounded, with the sum of each group
    for (int q = warp; q < kQ; q += NW)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (q < nq) {
          const uint2 r = *reinterpret_cast<const uint2*>(a.q + (int64_t)b * a.q_stride + (int64_t)(hq0 + q) * D +
                                                          g * kGroup + 4 * lane);
          const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&r.x));
          const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
          v[0] = f0.x, v[1] = f0.y, v[2] = f1.x, v[3] = f1.y;
        }
        if (a.sign_bits) rotate4(v, a.sign_bits, g, lane, false);
        const __half2 h0 = __floats2half2_rn(v[0], v[1]), h1 = __floats2half2_rn(v[2], v[3]);
        reinterpret_cast<__half2*>(sq + q * D + g * kGroup)[2 * lane] = h0;
        reinterpret_cast<__half2*>(sq + q * D + g * kGroup)[2 * lane + 1] = h1;
        float s = (__low2float(h0) + __high2float(h0)) + (__low2float(h1) + __high2float(h1));
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) sx[q * NG + g] = s;
      }
    __syncthreads();

    // ---- the lane's operand: query g8, the dimensions of the codes that lanes of column t4 hold
    uint32_t qf[NG][16];
    float xs[NG][2];  // sums of queries 2 t4, 2 t4 + 1 in the codes' units
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint32_t base = smem_addr(sq + g8 * D + g * kGroup);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // 8 consecutive dimensions: 4 bits, word j of piece t; 8 bits, words 2(j & 1), + 1 of
        // piece t + 4 (j >> 1); 16 bits, piece t + 4 j
        const int d0 = KB == 4 ? 32 * t4 + 8 * j : KB == 8 ? 64 * (j >> 1) + 16 * t4 + 8 * (j & 1) : 32 * j + 8 * t4;
        const uint4 p = ld128(base + 2 * d0);
        if (KB == 4) {
          qf[g][4 * j] = __byte_perm(p.x, p.z, 0x5410);
          qf[g][4 * j + 1] = __byte_perm(p.y, p.w, 0x5410);
          qf[g][4 * j + 2] = __byte_perm(p.x, p.z, 0x7632);
          qf[g][4 * j + 3] = __byte_perm(p.y, p.w, 0x7632);
        } else if (KB == 8) {
          qf[g][4 * j] = __byte_perm(p.x, p.y, 0x5410);
          qf[g][4 * j + 1] = __byte_perm(p.x, p.y, 0x7632);
          qf[g][4 * j + 2] = __byte_perm(p.z, p.w, 0x5410);
          qf[g][4 * j + 3] = __byte_perm(p.z, p.w, 0x7632);
        } else {
          qf[g][4 * j] = p.x, qf[g][4 * j + 1] = p.y, qf[g][4 * j + 2] = p.z, qf[g][4 * j + 3] = p.w;
        }
      }
      xs[g][0] = sx[2 * t4 * NG + g] * 0x1p-9f;
      xs[g][1] = sx[(2 * t4 + 1) * NG + g] * 0x1p-9f;
    }

    float o[NG][8][4], m[NG][2], l[NG][2], zc[NG][2];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[g][j][0] = o[g][j][1] = o[g][j][2] = o[g][j][3] = 0.f;
      m[g][0] = m[g][1] = kNone;
      l[g][0] = l[g][1] = zc[g][0] = zc[g][1] = 0.f;
    }

    for (int k = 0; k < cnt; ++k) {
      cp_wait<S - 2>();
      __syncwarp();
      issue(k + S - 1);  // into the stage that the previous tile has left
      const uint32_t st = ring + (k % S) * C::kStage;
      const int valid = *reinterpret_cast<const volatile int*>(smem + (st - smem_addr(smem)) + C::kStage - 16);

      // scores in units of log2: lane holds tokens g8 (s[0], s[1]) and g8 + 8, queries 2 t4, 2 t4 + 1
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      float lv[NG][2], rv[NG][2], vz[NG][2];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t kb = st + g * (kTile * 16 * KB);
        if (KB == 4) {
          const uint4 wa = ld128(kb + k_at<KB>(g8, t4)), wb = ld128(kb + k_at<KB>(g8 + 8, t4));
          const uint32_t ra[4] = {wa.x, wa.y, wa.z, wa.w}, rb[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t ha = ra[j] >> 8, hb = rb[j] >> 8;
            mma(c0, low4(ra[j]), low4(rb[j]), low4(ha), low4(hb), qf[g][4 * j], qf[g][4 * j + 1]);
            mma(c1, high4(ra[j]), high4(rb[j]), high4(ha), high4(hb), qf[g][4 * j + 2], qf[g][4 * j + 3]);
          }
        } else if (KB == 8) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 wa = ld128(kb + k_at<KB>(g8, t4 + 4 * j)), wb = ld128(kb + k_at<KB>(g8 + 8, t4 + 4 * j));
            const uint32_t ra[4] = {wa.x, wa.y, wa.z, wa.w}, rb[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma((i & 1) ? c1 : c0, low8(ra[i]), low8(rb[i]), low8(ra[i] >> 8), low8(rb[i] >> 8),
                  qf[g][8 * j + 2 * i], qf[g][8 * j + 2 * i + 1]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 wa = ld128(kb + k_at<KB>(g8, t4 + 4 * j)), wb = ld128(kb + k_at<KB>(g8 + 8, t4 + 4 * j));
            mma(c0, wa.x, wb.x, wa.y, wb.y, qf[g][4 * j], qf[g][4 * j + 1]);
            mma(c1, wa.z, wb.z, wa.w, wb.w, qf[g][4 * j + 2], qf[g][4 * j + 3]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) c0[i] += c1[i];
        if (C::kPar) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {  // tokens g8, g8 + 8
            const uint2 p = ld64(st + C::kOffPar + (g8 + 8 * i) * C::kPar + 8 * g);
            const float2 pk = __half22float2(*reinterpret_cast<const __half2*>(&p.x));
            const float2 pv = __half22float2(*reinterpret_cast<const __half2*>(&p.y));
            const float f = pk.x * (a.scale_log2e * 512.f);
            s[2 * i] = fmaf(fmaf(-pk.y, xs[g][0], c0[2 * i]), f, s[2 * i]);
            s[2 * i + 1] = fmaf(fmaf(-pk.y, xs[g][1], c0[2 * i + 1]), f, s[2 * i + 1]);
            // a scale of 0 (a slot that was cleared, never written) is 2^-100 here: its token has a
            // share of the denominator and none of the sums
            lv[g][i] = fmaxf(lg2(pv.x), -100.f);
            rv[g][i] = fminf(rcp(pv.x), 0x1p100f);
            vz[g][i] = pv.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i] = fmaf(c0[i], a.scale_log2e, s[i]);
          lv[g][0] = lv[g][1] = vz[g][0] = vz[g][1] = 0.f;
          rv[g][0] = rv[g][1] = 1.f;
        }
      }
      if (valid < kTile) {  // masked tokens: no weight, and nothing read from their parameters
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (g8 + 8 * i >= valid) {
            s[2 * i] = s[2 * i + 1] = -INFINITY;
#pragma unroll
            for (int g = 0; g < NG; ++g) lv[g][i] = rv[g][i] = vz[g][i] = 0.f;
          }
      }

      uint32_t pb[NG][2];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float w[4] = {s[0] + lv[g][0], s[1] + lv[g][0], s[2] + lv[g][1], s[3] + lv[g][1]};
        float top0 = fmaxf(w[0], w[2]), top1 = fmaxf(w[1], w[3]);
        if (__any_sync(0xffffffffu, top0 > m[g][0] + 15.f || top1 > m[g][1] + 15.f)) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, d));
            top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, d));
          }
          const float n0 = fmaxf(m[g][0], top0 - 7.f), n1 = fmaxf(m[g][1], top1 - 7.f);
          const float f0 = ex2(m[g][0] - n0), f1 = ex2(m[g][1] - n1);
          m[g][0] = n0, m[g][1] = n1;
          l[g][0] *= f0, l[g][1] *= f1, zc[g][0] *= f0, zc[g][1] *= f1;
#pragma unroll
          for (int j = 0; j < 8; ++j) o[g][j][0] *= f0, o[g][j][1] *= f1, o[g][j][2] *= f0, o[g][j][3] *= f1;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float p0 = ex2(w[2 * i] - m[g][0]), p1 = ex2(w[2 * i + 1] - m[g][1]);
          const __half2 p = __floats2half2_rn(p0, p1);
          const float2 r = __half22float2(p);
          pb[g][i] = movmatrix(*reinterpret_cast<const uint32_t*>(&p));
          l[g][0] = fmaf(p0 < 0x1p-14f ? p0 : r.x, rv[g][i], l[g][0]);
          l[g][1] = fmaf(p1 < 0x1p-14f ? p1 : r.y, rv[g][i], l[g][1]);
          if (C::kPar) {
            zc[g][0] = fmaf(r.x, vz[g][i], zc[g][0]);
            zc[g][1] = fmaf(r.y, vz[g][i], zc[g][1]);
          }
        }
      }

      // values: the lane's tokens 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9, dimensions 16 g8 .. 16 g8 + 15
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t vb = st + C::kOffV + g * (kTile * 16 * VB);
        const uint32_t b0 = pb[g][0], b1 = pb[g][1];
        if (VB == 4) {
          uint2 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = ld64(vb + v_at<VB>(2 * t4 + (i & 1) + 8 * (i >> 1), g8 >> 1) + 8 * (g8 & 1));
#pragma unroll
          for (int half = 0; half < 4; ++half) {  // four dimensions: a half-word of each token
            const uint32_t sel = (half & 1) ? 0x7632u : 0x5410u;
            const uint32_t x = half < 2 ? __byte_perm(w[0].x, w[1].x, sel) : __byte_perm(w[0].y, w[1].y, sel);
            const uint32_t y = half < 2 ? __byte_perm(w[2].x, w[3].x, sel) : __byte_perm(w[2].y, w[3].y, sel);
            const uint32_t hx = x >> 8, hy = y >> 8;
            mma(o[g][2 * half], low4(x), low4(hx), low4(y), low4(hy), b0, b1);
            mma(o[g][2 * half + 1], high4(x), high4(hx), high4(y), high4(hy), b0, b1);
          }
        } else if (VB == 8) {
          uint4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = ld128(vb + v_at<VB>(2 * t4 + (i & 1) + 8 * (i >> 1), g8));
          const uint32_t w0[4] = {w[0].x, w[0].y, w[0].z, w[0].w}, w1[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
          const uint32_t w2[4] = {w[2].x, w[2].y, w[2].z, w[2].w}, w3[4] = {w[3].x, w[3].y, w[3].z, w[3].w};
#pragma unroll
          for (int j = 0; j < 8; ++j) {  // two dimensions: a half-word of each token
            const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
            const uint32_t x = __byte_perm(w0[j >> 1], w1[j >> 1], sel), y = __byte_perm(w2[j >> 1], w3[j >> 1], sel);
            mma(o[g][j], low8(x), low8(x >> 8), low8(y), low8(y >> 8), b0, b1);
          }
        } else {
          const int r = (lane & 7) + 8 * (lane >> 4), c = (lane >> 3) & 1;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 w = ldmatrix_x4_trans(vb + v_at<VB>(r, 2 * j + c));
            mma(o[g][j], w.x, w.y, w.z, w.w, b0, b1);
          }
        }
      }
    }
    cp_wait<0>();

    // ---- join the warps' sums
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          l[g][i] += __shfl_xor_sync(0xffffffffu, l[g][i], d);
          zc[g][i] += __shfl_xor_sync(0xffffffffu, zc[g][i], d);
        }
    __syncthreads();  // every warp has left its ring
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float* row = sj + (warp * kQ + 2 * t4 + i) * C::kJoinRow + g * kGroup;
        if (VB == 16) {
#pragma unroll
          for (int j = 0; j < 8; ++j) row[16 * j + g8] = o[g][j][i], row[16 * j + 8 + g8] = o[g][j][2 + i];
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float(&e)[4] = o[g][2 * j], (&f)[4] = o[g][2 * j + 1];
            // 4 bits: rows (0, 2) and (1, 3) of four dimensions; 8 bits: (0, 1) and (2, 3)
            const float v0 = fmaf(e[i], 512.f, -zc[g][i]), v1 = fmaf(e[2 + i], 512.f, -zc[g][i]);
            const float v2 = fmaf(f[i], 512.f, -zc[g][i]), v3 = fmaf(f[2 + i], 512.f, -zc[g][i]);
            *reinterpret_cast<float4*>(row + 16 * g8 + 4 * j) =
                VB == 4 ? make_float4(v0, v2, v1, v3) : make_float4(v0, v1, v2, v3);
          }
        }
        if (g8 == 0) sml[(warp * kQ + 2 * t4 + i) * NG + g] = make_float2(m[g][i], l[g][i]);
      }
    __syncthreads();
    const bool whole = tile0 == 0 && n == nt;
    for (int q = warp; q < nq; q += NW)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float top = kNone, den = 0.f, r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; ++w) top = fmaxf(top, sml[(w * kQ + q) * NG + g].x);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float2 ml = sml[(w * kQ + q) * NG + g];
          const float f = ex2(ml.x - top);
          const float4 v = *reinterpret_cast<const float4*>(sj + (w * kQ + q) * C::kJoinRow + g * kGroup + 4 * lane);
          den = fmaf(f, ml.y, den);
          r[0] = fmaf(f, v.x, r[0]), r[1] = fmaf(f, v.y, r[1]), r[2] = fmaf(f, v.z, r[2]), r[3] = fmaf(f, v.w, r[3]);
        }
        if (whole) {
          store_out(a, b, hq0 + q, D, g, lane, r, den);
        } else {  // slot 0: the piece began in an earlier CTA; slot 1: here
          float* slot = a.ws + ((int64_t)blockIdx.x * 2 + (tile0 == 0)) * a.qper * (D + 4) + q * (D + 4);
          *reinterpret_cast<float4*>(slot + g * kGroup + 4 * lane) = make_float4(r[0], r[1], r[2], r[3]);
          if (lane == 0) slot[D + 2 * g] = top, slot[D + 2 * g + 1] = den;
        }
      }
    __syncthreads();  // the ring and the queries may be overwritten
    u += n;
  }
}

// Joins the pieces of the sequence that crosses the boundary between CTAs
// blockIdx.x and blockIdx.x + 1, if no earlier boundary cuts it; one query a block,
// four warps over its pieces.
template <int NG>
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ AttnArgs a, int grid) {
  constexpr int D = NG * kGroup;
  __shared__ float so[4][D], sm[4][NG], sl[4][NG];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int total = total_tiles(a, lane), share = share_of(a, total, grid);
  const int64_t cut64 = (int64_t)(blockIdx.x + 1) * share;
  bool mine = cut64 < total;
  const int cut = (int)cut64, group = a.q_heads / a.c.heads, q = blockIdx.y;
  int b = 0, first = 0, h = 0, q0 = 0, to = 0;
  if (mine) {
    find_tile(a, lane, cut, b, first);
    const int nt = tiles_of(a, b), item = (cut - first) / nt, from = first + item * nt;
    to = from + nt;
    h = item / a.nqb, q0 = (item % a.nqb) * a.qper;
    // inside a sequence, and the first boundary there
    mine = from != cut && from >= cut - share && q < min(a.qper, group - q0);
  }
  grid_dependency_wait();  // every block: this grid's end stands for the first one's too
  if (!mine) return;
  const int c0 = blockIdx.x, c1 = (to - 1) / share;  // its CTAs
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

template <int KB, int VB, int NG>
qlin_status launch(const AttnArgs& a, cudaStream_t s) {
  using C = Cfg<KB, VB, NG>;
  static_assert(C::kSmem <= 227 * 1024, "shared memory");
  static std::atomic<unsigned long long> configured{0};  // per-device attribute, set once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return record_cuda(e);
  if (dev >= 64 || !((configured.load(std::memory_order_acquire) >> dev) & 1ull)) {
    e = cudaFuncSetAttribute(attn_kernel<KB, VB, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return record_cuda(e);
    if (dev < 64) configured.fetch_or(1ull << dev, std::memory_order_release);
  }
  attn_kernel<KB, VB, NG><<<C::kGrid, C::kWarps * 32, C::kSmem, s>>>(a);
  const qlin_status r = record_cuda(cudaGetLastError());
  if (r != QLIN_OK || !a.split) return r;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C::kGrid - 1, a.qper);
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return record_cuda(cudaLaunchKernelEx(&cfg, attn_join_kernel<NG>, a, (int)C::kGrid));
}

template <int NG>
qlin_status launch_widths(const AttnArgs& a, cudaStream_t s) {
  if (a.c.k_bits == 16) return launch<16, 16, NG>(a, s);
  if (a.c.k_bits == 8) return a.c.v_bits == 8 ? launch<8, 8, NG>(a, s) : launch<8, 4, NG>(a, s);
  return a.c.v_bits == 8 ? launch<4, 8, NG>(a, s) : launch<4, 4, NG>(a, s);
}

struct Split {
  int nqb, qper, split;
};

Split split_of(int page, int kv_heads, int q_heads, int max_pages) {
  Split s;
  const int group = q_heads / kv_heads;
  s.nqb = (group + kQ - 1) / kQ;
  s.qper = (group + s.nqb - 1) / s.nqb;
  s.split = (int64_t)max_pages * page > kWholeTiles * kTile;
  return s;
}

}  // namespace

unsigned take_attn_error() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_attn_error, sizeof(v)) != cudaSuccess) return ~0u;
  if (v) cudaMemcpyToSymbol(g_attn_error, &zero, sizeof(zero));
  return v;
}

size_t attn_workspace_bytes(const qlin_kv_desc* d, int q_heads, int batch, int max_pages) {
  const Split s = split_of(d->page_size, d->kv_heads, q_heads, max_pages);
  if (!s.split) return 0;
  return (size_t)(2 * kSms) * 2 * s.qper * (d->head_dim + 4) * sizeof(float);
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
  a.split = sp.split;
  return c.dim == kGroup ? launch_widths<1>(a, s) : launch_widths<2>(a, s);
}

}  // namespace qlin
