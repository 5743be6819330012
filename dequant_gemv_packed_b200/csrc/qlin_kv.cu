// qlin_kv_write and qlin_kv_read: quantising keys and values into the paged
// cache as they are written, and reading them back.
//
// Per group of 128 values (one Hadamard block, one scale and zero): the vector
// is rotated like an activation ("24B0978-Week01-Track2_20-Submission01",
// paragraph "Random Hadamard transform"), then quantised by the affine form of
// "Group-wise affine integer quantisation" on a grid that contains zero,
//   lo = min(v, 0), hi = max(v, 0), s = fp16 up((hi - lo) / qmax),
//   z = fp16(-lo / s), q = clamp(rint(v / s + z), 0, qmax),  value = s (q - z).
// Zero on the grid keeps z inside [0, qmax] for every input, so fp16 holds it to
// 1/16 of a step or better (a group far from zero would otherwise overflow z);
// rounding s up keeps hi on the grid where s is subnormal (values of 1e-4 and
// below, where rounding to nearest could drop several per cent of the range).
// Every step is one IEEE fp32 operation and the butterfly strides run 1, 2, ...,
// 64, so the stored bytes are a function of the input alone.
//
// Four lanes a group, 32 values each (eight and 16 while there are few groups):
// strides 1, 2, 4, 32 and 64 in the lane, 8 and 16 over lane distances 1, 2; a warp
// has eight groups of one side (K or V, which may differ in width) and strides over
// the tokens, the next group's data and the slot after it in flight.
// The quotients v / s share one correctly rounded reciprocal r and take three
// multiply-adds each, q0 = v r, q0 + (v - q0 s) r: correctly rounded by Markstein's
// theorem (IBM Journal of Research and Development 34, 1990), s having 11
// significant bits and nothing here nearing the ends of the exponent range.
// Bound by HBM's writes and by issue slots, which add up: reading 30,001 rotated
// tokens of 8 heads at 4/8 bits takes 53.6 us; 31 with the rotation and the cache's
// loads left out (a plain fill of the 123 MB it writes takes 32), 41 with the stores
// left out.  With 574 instructions a warp of four groups it took 84; two-
// value operations, constants in place of divisions and four lanes a group brought
// it here.  Four lanes against eight: 16,384 unrotated wide tokens written and read
// 41.2 us against 48.8; eight are 0.7 us better at 16 tokens (5.2).  A write alone:
// 16 tokens 2.3 us; 16,384 tokens of 8 heads at 8 bits 22.3 not rotated, 33.2 rotated,
// at 16 bits 23.7 (a read of those 24.5).
#include "qlin_kv.cuh"
#include "qlin_sm100.cuh"

namespace qlin {
namespace {

__device__ unsigned int g_kv_error;

constexpr int kThreads = 256;
constexpr int units_per_cta(int lanes) { return kThreads / (2 * lanes); }  // groups of each side
constexpr int ctas(int lanes) { return lanes == 8 ? 4 : 2; }                 // an SM

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Sign masks of every lane's values, in shared memory: [group][lane][piece].
template <int L>
__device__ __forceinline__ void fill_masks(uint4* masks, const uint32_t* sign_bits, int groups) {
  constexpr int C = 16 / L;
  for (int i = threadIdx.x; i < groups * L * C; i += kThreads)
    masks[i] = sign_mask<L>(sign_bits + 4 * (i / (L * C)), i / C % L, i % C);
  __syncthreads();
}

struct KvArgs {
  KvView c;
  const __half *k_in, *v_in;  // write: token rows
  __half *k_out, *v_out;      // read: token rows
  int64_t k_stride, v_stride; // elements between tokens
  const int32_t* slots;
  const uint32_t* sign_bits;  // null: not rotated
  int32_t tokens;
};

// A lane's walk over the groups (units) of its side: unit = (token, head, group), the group of 128
// within the head fixed.
template <int L>
struct Walk {
  int side, g, bits, t;
  int tok, r;         // token, and head * groups + group
  int dtok, dr;       // a step
  int unit, lg;       // units a token; log2 of the groups a head
  int row_bytes;
  int64_t row0, par0; // of the group in a block, at offset 0

  __device__ __forceinline__ Walk(const KvArgs& a, int lane, int warp) {
    lg = a.c.dim == kGroup ? 0 : 1;
    unit = a.c.heads << lg;
    const unsigned u = blockIdx.x * units_per_cta(L) + (warp >> 1) * (32 / L) + lane / L, step = gridDim.x * units_per_cta(L);
    t = lane % L;
    side = warp & 1;
    bits = side ? a.c.v_bits : a.c.k_bits;
    tok = (int)(u / (unsigned)unit);
    r = (int)(u % (unsigned)unit);
    dtok = (int)(step / (unsigned)unit);
    dr = (int)(step % (unsigned)unit);
    g = r & ((1 << lg) - 1);  // steps are even
    row_bytes = side ? a.c.v_row : a.c.k_row;
    row0 = (side ? a.c.v_offset : 0) + g * (kGroup / 8) * bits;
    par0 = a.c.par_offset + 8 * g + 4 * side;
  }
  __device__ __forceinline__ void next() {
    tok += dtok;
    r += dr;
    if (r >= unit) r -= unit, ++tok;
  }
  __device__ __forceinline__ int head() const { return r >> lg; }
  // The group's codes in the cache, and its (scale, zero), for a slot inside the pool.
  __device__ __forceinline__ void place(const KvArgs& a, int slot, uint8_t*& row, uint8_t*& par) const {
    const int page = a.c.page_shift >= 0 ? slot >> a.c.page_shift : slot / a.c.page, off = slot - page * a.c.page;
    uint8_t* b = a.c.pool + ((int64_t)page * a.c.heads + head()) * a.c.block_bytes;
    row = b + row0 + (int64_t)off * row_bytes;
    par = b + par0 + (int64_t)off * a.c.par;
  }
};

// The slot of a token as given, -1 past the last; it is looked at (checked_slot) one step later, so
// that no step waits for this load.
__device__ __forceinline__ int slot_of(const KvArgs& a, int tok) { return tok < a.tokens ? a.slots[tok] : -1; }

// A slot inside the pool, or -1 where there is nothing to do.
__device__ __forceinline__ int checked_slot(const KvArgs& a, int s, int t) {
  if (s < a.c.pages * a.c.page) return max(s, -1);
  if (t == 0) atomicOr(&g_kv_error, kKvBadSlot);
  return -1;
}

// The loops below keep the next unit's data and the slot of the one after it in flight.

template <int L>
__global__ void __launch_bounds__(kThreads, ctas(L)) kv_write_kernel(const __grid_constant__ KvArgs a) {
  constexpr int C = 16 / L;  // pieces of eight values a lane
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ uint4 masks[2 * L * C];
  if (a.sign_bits) fill_masks<L>(masks, a.sign_bits, a.c.dim / kGroup);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Walk<L> w(a, lane, warp);
  const int64_t stride = w.side ? a.v_stride : a.k_stride;
  const uint4* src = reinterpret_cast<const uint4*>((w.side ? a.v_in : a.k_in) + w.g * kGroup) + w.t;
  const uint4* mask = masks + (w.g * L + w.t) * C;
  uint4 next[C];
  auto load = [&]() {
    const uint4* in = src + (((int64_t)min(w.tok, a.tokens - 1) * stride + (int64_t)w.head() * a.c.dim) >> 3);
#pragma unroll
    for (int c = 0; c < C; ++c) next[c] = in[L * c];
  };
  int next_slot = slot_of(a, w.tok);
  load();
  while (__any_sync(0xffffffffu, w.tok < a.tokens)) {
    const int slot = checked_slot(a, next_slot, w.t);
    uint4 r[C];
#pragma unroll
    for (int c = 0; c < C; ++c) r[c] = next[c];
    uint8_t *row, *par;
    w.place(a, max(slot, 0), row, par);
    w.next();
    next_slot = slot_of(a, w.tok);
    load();
    f32x2 v[4 * C];
    if (a.sign_bits) {
#pragma unroll
      for (int c = 0; c < C; ++c) flip(r[c], mask[c]);
      halves_to_float(r, v);
      fwht128<L>(v, w.t);
      if (w.bits == 16) float_to_halves(v, r);
    } else {
      halves_to_float(r, v);
    }
    if (w.bits == 16) {
      if (slot >= 0)
#pragma unroll
        for (int c = 0; c < C; ++c) reinterpret_cast<uint4*>(row)[w.t + L * c] = r[c];
      continue;
    }
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int j = 0; j < 4 * C; ++j) {
      float x, y;
      split2(v[j], x, y);
      lo = min_nan(lo, min_nan(x, y));
      hi = max_nan(hi, max_nan(x, y));
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    lo = __fadd_rn(lo, 0.f);  // a zero bound is +0 whichever zero the reduction kept
    const float qmax = (float)((1 << w.bits) - 1);
    const float span = __fdiv_rn(__fsub_rn(hi, lo), qmax);
    const bool finite = span < INFINITY;  // false for NaN too
    __half s16 = __float2half_ru(fminf(span, 65504.f));
    if (!(span > 0.f) || !finite) s16 = __float2half_rn(1.f);
    const float s = __half2float(s16);
    // a group that holds an infinity or NaN reads back as NaN throughout
    const __half z16 = finite ? __float2half_rn(__fdiv_rn(-lo, s)) : __ushort_as_half(0x7fff);
    const float z = __half2float(z16), inv = __frcp_rn(s);
    // v / s + z lies within 1/16 of [0, qmax] unless the scale was cut or the group is not finite
    const bool clamp = !(span <= 65504.f);
    const f32x2 s2 = pair2(-s, -s), inv2 = pair2(inv, inv), z2 = pair2(z, z), round2 = pair2(8388608.f, 8388608.f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      uint32_t q[8];  // the code in the low byte: adding 2^23 rounds to an integer, ties to even
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2 x = v[4 * c + i], q0 = mul2(x, inv2);
        f32x2 y = add2(fma2(fma2(q0, s2, x), inv2, q0), z2);
        float y0, y1;
        if (clamp) {
          split2(y, y0, y1);
          y = pair2(fminf(fmaxf(y0, 0.f), qmax), fminf(fmaxf(y1, 0.f), qmax));
        }
        split2(add2(y, round2), y0, y1);
        q[2 * i] = __float_as_uint(y0);
        q[2 * i + 1] = __float_as_uint(y1);
      }
      if (slot < 0) continue;
      if (w.bits == 8) {
        uint32_t b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          b[i] = __byte_perm(__byte_perm(q[4 * i], q[4 * i + 1], 0x0040), __byte_perm(q[4 * i + 2], q[4 * i + 3], 0x0040),
                             0x5410);
        reinterpret_cast<uint2*>(row)[w.t + L * c] = make_uint2(b[0], b[1]);
      } else {
        uint32_t b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) b[k] = q[2 * k] + (q[2 * k + 1] << 4);
        reinterpret_cast<uint32_t*>(row)[w.t + L * c] =
            __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
      }
    }
    if (w.t == 0 && slot >= 0) *reinterpret_cast<__half2*>(par) = __halves2half2(s16, z16);
  }
}

// s (q - z) of two codes a 2^23 + q U, U = 16^k the weight of the bits they sit on: taking 2^23 off
// is exact, the multiply-add with 1 / U rounds q - z once, the product with s once.
__device__ __forceinline__ f32x2 dequant2(uint32_t a, uint32_t b, f32x2 inv_unit, f32x2 z, f32x2 s) {
  const f32x2 x = add2(pair2(__uint_as_float(a), __uint_as_float(b)), pair2(-8388608.f, -8388608.f));
  return mul2(s, fma2(x, inv_unit, z));
}

template <int L>
__global__ void __launch_bounds__(kThreads, ctas(L)) kv_read_kernel(const __grid_constant__ KvArgs a) {
  constexpr int C = 16 / L;  // pieces of eight values a lane
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ uint4 masks[2 * L * C];
  if (a.sign_bits) fill_masks<L>(masks, a.sign_bits, a.c.dim / kGroup);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Walk<L> w(a, lane, warp);
  const int64_t stride = (int64_t)a.c.heads * a.c.dim;
  uint4* dst = reinterpret_cast<uint4*>((w.side ? a.v_out : a.k_out) + w.g * kGroup) + w.t;
  const uint4* mask = masks + (w.g * L + w.t) * C;
  uint4 next[C];
#pragma unroll
  for (int c = 0; c < C; ++c) next[c] = make_uint4(0u, 0u, 0u, 0u);
  uint32_t next_par = 0;
  auto load = [&](int slot) {
    uint8_t *row, *par;
    w.place(a, max(slot, 0), row, par);
    if (w.bits == 16) {
#pragma unroll
      for (int c = 0; c < C; ++c) next[c] = reinterpret_cast<const uint4*>(row)[w.t + L * c];
    } else {
      next_par = *reinterpret_cast<const uint32_t*>(par);
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (w.bits == 8) {
          const uint2 x = reinterpret_cast<const uint2*>(row)[w.t + L * c];
          next[c].x = x.x, next[c].y = x.y;
        } else {
          next[c].x = reinterpret_cast<const uint32_t*>(row)[w.t + L * c];
        }
    }
  };
  int next_slot = checked_slot(a, slot_of(a, w.tok), w.t);
  load(next_slot);
  int tok = w.tok, head = w.head();  // of the unit in `next`
  w.next();
  int after = slot_of(a, w.tok);
  while (__any_sync(0xffffffffu, tok < a.tokens)) {
    const int slot = next_slot;
    uint4 r[C];
#pragma unroll
    for (int c = 0; c < C; ++c) r[c] = next[c];
    const uint32_t pp = next_par;
    uint4* out = dst + (((int64_t)tok * stride + (int64_t)head * a.c.dim) >> 3);
    const bool live = tok < a.tokens;
    next_slot = checked_slot(a, after, w.t);
    load(next_slot);
    tok = w.tok, head = w.head();
    w.next();
    after = slot_of(a, w.tok);
    f32x2 v[4 * C];
    if (w.bits == 16) {
      if (a.sign_bits) halves_to_float(r, v);
    } else {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&pp));
      const f32x2 s = pair2(p.x, p.x), z = pair2(-p.y, -p.y);
      if (w.bits == 8) {
        const f32x2 one = pair2(1.f, 1.f);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const uint32_t x[2] = {r[c].x, r[c].y};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[4 * c + i] = dequant2(__byte_perm(x[i >> 1], 0x4B000000u, 0x7440 + 2 * (i & 1)),
                                    __byte_perm(x[i >> 1], 0x4B000000u, 0x7441 + 2 * (i & 1)), one, z, s);
        }
      } else {
        const f32x2 u0 = pair2(1.f, 0.0625f), u2 = pair2(0x1p-8f, 0x1p-12f);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t y = r[c].x >> (16 * k);
            v[4 * c + 2 * k] = dequant2((y & 0xFu) | 0x4B000000u, (y & 0xF0u) | 0x4B000000u, u0, z, s);
            v[4 * c + 2 * k + 1] = dequant2((y & 0xF00u) | 0x4B000000u, (y & 0xF000u) | 0x4B000000u, u2, z, s);
          }
      }
    }
    if (a.sign_bits) fwht128<L>(v, w.t);
    if (a.sign_bits || w.bits != 16) float_to_halves(v, r);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (a.sign_bits) flip(r[c], mask[c]);
      if (slot < 0) r[c] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (live)
#pragma unroll
      for (int c = 0; c < C; ++c) out[L * c] = r[c];
  }
}

}  // namespace

unsigned take_kv_error() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_kv_error, sizeof(v)) != cudaSuccess) return ~0u;
  if (v) cudaMemcpyToSymbol(g_kv_error, &zero, sizeof(zero));
  return v;
}

// Four lanes a group once every CTA has two rounds of them, else eight.
static int lanes_for(int64_t units) { return units >= 2 * 148 * ctas(4) * units_per_cta(4) ? 4 : 8; }

// Blocks for the units (a token's groups of one side), counted with a step beyond them in 31 bits.
static qlin_status kv_grid(const KvArgs& a, int& lanes, unsigned& grid) {
  const int64_t units = (int64_t)a.tokens * a.c.heads * (a.c.dim / kGroup);
  if (units > 0x7fffffffLL - (1 << 20)) return QLIN_ERR_SHAPE;
  lanes = lanes_for(units);
  const int64_t need = (units + units_per_cta(lanes) - 1) / units_per_cta(lanes), most = 148 * ctas(lanes);
  grid = (unsigned)(need < most ? need : most);
  return QLIN_OK;
}

qlin_status launch_kv_write(const KvView& c, const __half* k, const __half* v, int64_t k_stride, int64_t v_stride,
                            const int32_t* slots, int tokens, const uint32_t* sign_bits, cudaStream_t s) {
  const KvArgs a = {c, k, v, nullptr, nullptr, k_stride, v_stride, slots, sign_bits, tokens};
  int lanes;
  unsigned grid;
  const qlin_status r = kv_grid(a, lanes, grid);
  if (r != QLIN_OK) return r;
  return launch_dependent(lanes == 4 ? kv_write_kernel<4> : kv_write_kernel<8>, grid, kThreads, 0, s, a);
}

qlin_status launch_kv_read(const KvView& c, __half* k, __half* v, const int32_t* slots, int tokens,
                           const uint32_t* sign_bits, cudaStream_t s) {
  const KvArgs a = {c, nullptr, nullptr, k, v, 0, 0, slots, sign_bits, tokens};
  int lanes;
  unsigned grid;
  const qlin_status r = kv_grid(a, lanes, grid);
  if (r != QLIN_OK) return r;
  return launch_dependent(lanes == 4 ? kv_read_kernel<4> : kv_read_kernel<8>, grid, kThreads, 0, s, a);
}

}  // namespace qlin
