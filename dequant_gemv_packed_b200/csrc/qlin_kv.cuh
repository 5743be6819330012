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
constexpr int kItemExtra = 16; // most that attention adds to an item's tiles when it deals them out

struct KvView {
  uint8_t* pool;
  int64_t block_bytes;  // one (page, head) block
  int32_t pages, page, heads, dim;
  int32_t k_bits, v_bits;
  int32_t k_row, v_row;  // bytes of a row
  int32_t par;           // bytes of a token's parameters (0 at 16 bits)

  __host__ __device__ const uint8_t* block(int p, int h) const {
    return pool + ((int64_t)p * heads + h) * block_bytes;
  }
  __host__ __device__ uint8_t* block(int p, int h) { return pool + ((int64_t)p * heads + h) * block_bytes; }
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

}  // namespace qlin
