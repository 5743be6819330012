// The paged key/value cache: layout of one (page, head) block, shared by the
// kernels that write it, read it back and attend to it.
//
// A vector is one row of head_dim codes in qlin_pack's bit stream (4 or 8 bits),
// or its fp16 values (16 bits).  The block of a page and a head holds the K rows
// of the page's tokens, then their V rows, then (below 16 bits) four fp16
// parameters per token and group of 128: scale and zero of K, scale and zero of V.
// Rows of one head are contiguous over a page, so 16 tokens are one run of whole
// 128-byte lines for every width; a token's four parameters are one 8-byte load.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "qlin_internal.cuh"

namespace qlin {

constexpr int kPageUnit = 16;  // tokens: pages are multiples of this, tiles never cross a page
constexpr int kItemExtra = 36; // most that attention adds to an item's tiles when it deals them out

struct KvView {
  uint8_t* pool;
  int64_t block_bytes;        // one (page, head) block
  int64_t v_offset, par_offset;  // of its V rows and parameters
  int32_t pages, page, heads, dim;
  int32_t k_bits, v_bits;
  int32_t k_row, v_row;  // bytes of a row
  int32_t par;           // bytes of a token's parameters (0 at 16 bits)
  int32_t page_shift;    // log2 of the page's tokens; -1: no power of two

  __host__ __device__ const uint8_t* block(int p, int h) const {
    return pool + ((int64_t)p * heads + h) * block_bytes;
  }
};

__host__ inline KvView make_kv_view(const qlin_kv_desc* d, const void* cache) {
  KvView v;
  v.pool = const_cast<uint8_t*>(static_cast<const uint8_t*>(cache));
  v.pages = d->num_pages;
  v.page = d->page_size;
  v.heads = d->kv_heads;
  v.dim = d->head_dim;
  v.page_shift = d->page_size & (d->page_size - 1) ? -1 : __builtin_ctz(d->page_size);
  v.k_bits = d->k_bits;
  v.v_bits = d->v_bits;
  v.k_row = d->head_dim * d->k_bits / 8;
  v.v_row = d->head_dim * d->v_bits / 8;
  v.par = d->k_bits == 16 ? 0 : 8 * (d->head_dim / kGroup);
  v.v_offset = (int64_t)d->page_size * v.k_row;
  v.par_offset = v.v_offset + (int64_t)d->page_size * v.v_row;
  v.block_bytes = v.par_offset + (int64_t)d->page_size * v.par;
  return v;
}

// Bits of the cache kernels' error word (bits 24-31 of qlin_device_error).
constexpr unsigned kKvBadSlot = 1u;    // a slot at or past num_pages * page_size
constexpr unsigned kKvBadPage = 2u;    // a page outside the pool within a sequence's length
constexpr unsigned kKvBadLength = 4u;  // a length beyond the sequence's row of the block table
unsigned take_kv_error();              // each file's own word, read and cleared
unsigned take_attn_error();

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// n / d for 0 <= n < 2^31, d > 0: two estimates in fp32 (the second of a remainder below 2^9 d),
// each at most one off, and a correction; shorter than the integer division.
__device__ __forceinline__ int div_pos(int n, int d) {
  const float r = rcp((float)d) * 0.9999995f;  // from below
  int q = (int)((float)n * r);
  int rest = n - q * d;
  const int more = (int)((float)rest * r);
  q += more;
  rest -= more * d;
  return q + (rest >= d);
}

// A group of 128 values on L = 8 or 4 lanes: lane t = lane % L has the values 8 L c + 8 t ..
// 8 L c + 8 t + 7, c = 0 .. 16 / L - 1, as pairs v[4 c + i], so that 16-byte pieces of halves are
// contiguous over the lanes.

// Two fp32 values in one register pair; each operation rounds both to nearest, like two single ones.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair2(float lo, float hi) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void split2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Butterflies of strides 1..64 (1, 2, 4 in the lane, then across the L lanes, then over c), then the
// scaling.  A difference a - b is the multiply-add b (-1) + a, and across lanes both halves are
// v (+-1) + p: one rounding each, as the definition has it.
template <int L>
__device__ __forceinline__ void fwht128(f32x2 (&p)[64 / L], int t) {
  constexpr int N = 64 / L;
  const f32x2 minus = pair2(-1.f, -1.f);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    float a, b;
    split2(p[j], a, b);
    p[j] = pair2(__fadd_rn(a, b), __fsub_rn(a, b));
  }
#pragma unroll
  for (int h = 1; h < 4; h <<= 1)
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (!(j & h)) {
        const f32x2 a = p[j], b = p[j + h];
        p[j] = add2(a, b);
        p[j + h] = fma2(b, minus, a);
      }
#pragma unroll
  for (int o = 1; o < L; o <<= 1) {
    const float sign = (t & o) ? -1.f : 1.f;
    const f32x2 s = pair2(sign, sign);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float lo, hi;
      split2(p[j], lo, hi);
      p[j] = fma2(p[j], s, pair2(__shfl_xor_sync(0xffffffffu, lo, o), __shfl_xor_sync(0xffffffffu, hi, o)));
    }
  }
#pragma unroll
  for (int h = 4; h < N; h <<= 1)
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (!(j & h)) {
        const f32x2 a = p[j], b = p[j + h];
        p[j] = add2(a, b);
        p[j + h] = fma2(b, minus, a);
      }
  const f32x2 scale = pair2(kInvSqrt128, kInvSqrt128);
#pragma unroll
  for (int j = 0; j < N; ++j) p[j] = mul2(p[j], scale);
}

// Sign masks of the lane's piece c as four pairs of halves; `words` are the group's four.
template <int L>
__device__ __forceinline__ uint4 sign_mask(const uint32_t* words, int t, int c) {
  const int at = 8 * L * c + 8 * t;
  const uint32_t sw = words[at >> 5] >> (at & 31);
  uint32_t m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = ((sw >> (2 * i)) & 1u) << 15 | ((sw >> (2 * i + 1)) & 1u) << 31;
  return make_uint4(m[0], m[1], m[2], m[3]);
}

__device__ __forceinline__ void flip(uint4& r, const uint4& m) { r.x ^= m.x, r.y ^= m.y, r.z ^= m.z, r.w ^= m.w; }

template <int C>
__device__ __forceinline__ void halves_to_float(const uint4 (&r)[C], f32x2 (&v)[4 * C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const uint32_t w[4] = {r[c].x, r[c].y, r[c].z, r[c].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[4 * c + i] = pair2(f.x, f.y);
    }
  }
}

template <int C>
__device__ __forceinline__ void float_to_halves(const f32x2 (&v)[4 * C], uint4 (&r)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      split2(v[4 * c + i], a, b);
      const __half2 h = __floats2half2_rn(a, b);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    r[c] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace qlin
