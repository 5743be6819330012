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
constexpr int kItemExtra = 32; // most that attention adds to an item's tiles when it deals them out

struct KvView {
  uint8_t* pool;
  int64_t block_bytes;  // one (page, head) block
  int32_t pages, page, heads, dim;
  int32_t k_bits, v_bits;
  int32_t k_row, v_row;  // bytes of a row
  int32_t par;           // bytes of a token's parameters (0 at 16 bits)
  int32_t page_shift;    // log2 of the page's tokens; -1: no power of two

  __host__ __device__ const uint8_t* block(int p, int h) const {
    return pool + ((int64_t)p * heads + h) * block_bytes;
  }
  __host__ __device__ int64_t v_offset() const { return (int64_t)page * k_row; }
  __host__ __device__ int64_t par_offset() const { return (int64_t)page * (k_row + v_row); }
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
  v.block_bytes = (int64_t)d->page_size * (v.k_row + v.v_row + v.par);
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

// A group of 128 values on eight lanes, lane t = lane % 8 with values 16 t .. 16 t + 15.

// Butterflies of strides 1..64 over the 16 values of each of a group's eight lanes.
__device__ __forceinline__ void fwht128_oct(float (&v)[16], int t) {
#pragma unroll
  for (int h = 1; h < 16; h <<= 1)
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (!(j & h)) {
        const float a = v[j], b = v[j + h];
        v[j] = __fadd_rn(a, b);
        v[j + h] = __fsub_rn(a, b);
      }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const bool upper = (t & o) != 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float p = __shfl_xor_sync(0xffffffffu, v[j], o);
      v[j] = upper ? __fsub_rn(p, v[j]) : __fadd_rn(v[j], p);
    }
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = __fmul_rn(v[j], kInvSqrt128);
}

// Changes the signs of the lane's values of group g.
__device__ __forceinline__ void flip16(float (&v)[16], uint32_t sw) {
#pragma unroll
  for (int j = 0; j < 16; ++j)
    v[j] = __uint_as_float(__float_as_uint(v[j]) ^ (((sw >> j) & 1u) << 31));
}

__device__ __forceinline__ void halves_to_float(const uint4& r0, const uint4& r1, float (&v)[16]) {
  const uint32_t raw[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&raw[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ void float_to_halves(const float (&v)[16], uint4& r0, uint4& r1) {
  uint32_t raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    raw[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  r0 = make_uint4(raw[0], raw[1], raw[2], raw[3]);
  r1 = make_uint4(raw[4], raw[5], raw[6], raw[7]);
}

}  // namespace qlin
