// qlin_attn_decode: attention of one new token per sequence over the paged,
// quantised key/value cache.
//
// One CTA per (sequence, query head): each warp takes every eighth token, with a
// running maximum and sum; the warps' states are joined in shared memory, the sum
// is rotated back and rounded once.
#include "qlin_kv.cuh"

namespace qlin {
namespace {

__device__ unsigned int g_attn_error;

constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;

struct AttnArgs {
  KvView c;
  const __half* q;
  int64_t q_stride;
  const int32_t *table, *lens;
  const uint32_t* sign_bits;
  __half* out;
  float scale_log2e;
  int32_t q_heads, max_pages;
};

// Rotation (or its inverse) of the four values 4 lane .. 4 lane + 3 of a block.
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

// The lane's four values of group g of a stored row.
__device__ __forceinline__ void values4(const uint8_t* row, const uint8_t* par, int bits, int side, int g, int lane,
                                        float (&v)[4]) {
  if (bits == 16) {
    const uint2 r = *reinterpret_cast<const uint2*>(row + 256 * g + 8 * lane);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&r.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    return;
  }
  const float2 p = __half22float2(*reinterpret_cast<const __half2*>(par + 8 * g + 4 * side));
  const uint32_t w = bits == 8 ? *reinterpret_cast<const uint32_t*>(row + 128 * g + 4 * lane)
                               : *reinterpret_cast<const uint16_t*>(row + 64 * g + 2 * lane);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = p.x * ((float)((w >> (bits * i)) & ((1u << bits) - 1u)) - p.y);
}

template <int NG>
__global__ void __launch_bounds__(kWarps * 32) attn_kernel(const AttnArgs a) {
  __shared__ float so[kWarps][NG * kGroup], sm[kWarps], sl[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / a.q_heads, hq = blockIdx.x % a.q_heads;
  const int h = hq / (a.q_heads / a.c.heads);
  const int dim = NG * kGroup, page = a.c.page;
  int len = a.lens[b];
  if (len > a.max_pages * page) {
    len = a.max_pages * page;
    if (threadIdx.x == 0) atomicOr(&g_attn_error, kKvBadLength);
  }
  float x[NG][4], o[NG][4];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const __half* q = a.q + (int64_t)b * a.q_stride + (int64_t)hq * dim + g * kGroup + 4 * lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[g][i] = __half2float(q[i]), o[g][i] = 0.f;
    if (a.sign_bits) {
      rotate4(x[g], a.sign_bits, g, lane, false);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[g][i] = __half2float(__float2half_rn(x[g][i]));
    }
  }
  float m = -INFINITY, l = 0.f;
  for (int t = warp; t < len; t += kWarps) {
    const int p = a.table[(int64_t)b * a.max_pages + t / page], off = t % page;
    if (p < 0 || p >= a.c.pages) {
      if (lane == 0) atomicOr(&g_attn_error, kKvBadPage);
      continue;
    }
    const uint8_t* blk = a.c.block(p, h);
    const uint8_t* par = blk + a.c.par_offset() + (int64_t)off * a.c.par;
    float s = 0.f, v[NG][4];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      values4(blk + (int64_t)off * a.c.k_row, par, a.c.k_bits, 0, g, lane, v[g]);
#pragma unroll
      for (int i = 0; i < 4; ++i) s += x[g][i] * v[g][i];
      values4(blk + a.c.v_offset() + (int64_t)off * a.c.v_row, par, a.c.v_bits, 1, g, lane, v[g]);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale_log2e;
    const float top = s != s ? s : fmaxf(m, s), old = m == -INFINITY ? 0.f : exp2f(m - top), e = exp2f(s - top);
    m = top;
    l = l * old + e;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[g][i] = o[g][i] * old + e * v[g][i];
  }
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i) so[warp][g * kGroup + 4 * lane + i] = o[g][i];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  __syncthreads();
  if (warp >= NG) return;  // warp g joins group g
  float top = -INFINITY, sum = 0.f, r[4] = {0.f, 0.f, 0.f, 0.f};
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  for (int w = 0; w < kWarps; ++w) {
    if (sm[w] == -INFINITY) continue;
    const float f = exp2f(sm[w] - top);
    sum += f * sl[w];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] += f * so[w][warp * kGroup + 4 * lane + i];
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] *= inv;
  if (a.sign_bits) rotate4(r, a.sign_bits, warp, lane, true);
  __half* out = a.out + ((int64_t)b * a.q_heads + hq) * dim + warp * kGroup + 4 * lane;
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = __float2half_rn(r[i]);
}

}  // namespace

unsigned take_attn_error() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_attn_error, sizeof(v)) != cudaSuccess) return ~0u;
  if (v) cudaMemcpyToSymbol(g_attn_error, &zero, sizeof(zero));
  return v;
}

size_t attn_workspace_bytes(const qlin_kv_desc*, int, int, int) { return 0; }

qlin_status launch_attn_decode(const KvView& c, const __half* q, int64_t q_stride, int q_heads,
                               const int32_t* block_table, int max_pages, const int32_t* seq_lens, int batch,
                               const uint32_t* sign_bits, float scale, __half* out, void*, cudaStream_t s) {
  const AttnArgs a = {c, q, q_stride, block_table, seq_lens, sign_bits, out, scale * kLog2e, q_heads, max_pages};
  const unsigned grid = (unsigned)((int64_t)batch * q_heads);
  if (c.dim == kGroup)
    attn_kernel<1><<<grid, kWarps * 32, 0, s>>>(a);
  else
    attn_kernel<2><<<grid, kWarps * 32, 0, s>>>(a);
  return record_cuda(cudaGetLastError());
}

}  // namespace qlin
