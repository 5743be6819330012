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
// Eight lanes a group, 16 consecutive values each: strides 1 to 8 in the lane,
// 16 to 64 over lane distances 1, 2, 4.  The quotients v / s share one correctly
// rounded reciprocal r and take three multiply-adds each, q0 = v r,
// q0 + (v - q0 s) r: correctly rounded by Markstein's theorem (IBM Journal of
// Research and Development 34, 1990), s having 11 significant bits and nothing
// here nearing the ends of the exponent range.
#include "qlin_kv.cuh"

namespace qlin {
namespace {

__device__ unsigned int g_kv_error;

constexpr int kThreads = 256;
constexpr int kTasksPerCta = kThreads / 8;

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

struct KvArgs {
  KvView c;
  const __half *k_in, *v_in;  // write: token rows
  __half *k_out, *v_out;      // read: token rows
  int64_t k_stride, v_stride; // elements between tokens
  const int32_t* slots;
  const uint32_t* sign_bits;  // null: not rotated
  int32_t tokens;
};

// A task is one group of one token, head and side: order (token, head, side, group).
struct Task {
  bool live;
  int side, g, bits, slot;
  int64_t in;     // element offset of the group in the token rows (without the lane's 16 t)
  uint8_t* row;   // the group's codes in the cache
  uint8_t* par;   // the group's (scale, zero) pair of this side
};

__device__ __forceinline__ Task find_task(const KvArgs& a, int t, int64_t stride_k, int64_t stride_v) {
  Task k;
  const int lg = a.c.dim == kGroup ? 0 : 1, groups = 1 << lg, unit = a.c.heads * 2 * groups;  // tasks a token
  // the block's first task by one division, the block's others by a short one
  const unsigned base = blockIdx.x * (unsigned)kTasksPerCta, tok0 = base / (unsigned)unit;
  const int x = (int)(base - tok0 * unit) + (int)(threadIdx.x >> 3), ahead = div_pos(x, unit);
  int tok = (int)tok0 + ahead, r = x - ahead * unit;
  k.live = tok < a.tokens;
  if (!k.live) tok = a.tokens - 1, r = 0;
  k.g = r & (groups - 1);
  k.side = (r >> lg) & 1;
  const int h = r >> (lg + 1);
  k.bits = k.side ? a.c.v_bits : a.c.k_bits;
  k.in = (int64_t)tok * (k.side ? stride_v : stride_k) + (int64_t)h * a.c.dim + (int64_t)k.g * kGroup;
  k.slot = a.slots[tok];
  if (k.slot >= a.c.pages * a.c.page) {
    if (t == 0) atomicOr(&g_kv_error, kKvBadSlot);
    k.slot = -1;
  }
  const int s = k.slot < 0 ? 0 : k.slot;
  const int page = a.c.page_shift >= 0 ? s >> a.c.page_shift : s / a.c.page, off = s - page * a.c.page;
  uint8_t* b = const_cast<uint8_t*>(a.c.block(page, h));
  k.row = b + (k.side ? a.c.v_offset() + (int64_t)off * a.c.v_row : (int64_t)off * a.c.k_row) + k.g * (kGroup / 8) * k.bits;
  k.par = b + a.c.par_offset() + (int64_t)off * a.c.par + 8 * k.g + 4 * k.side;
  return k;
}

__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvArgs a) {
  const int t = threadIdx.x & 7;
  const Task k = find_task(a, t, a.k_stride, a.v_stride);
  const __half* src = (k.side ? a.v_in : a.k_in) + k.in + 16 * t;
  uint4 r0 = reinterpret_cast<const uint4*>(src)[0];
  uint4 r1 = reinterpret_cast<const uint4*>(src)[1];
  float v[16];
  halves_to_float(r0, r1, v);
  if (a.sign_bits) {
    flip16(v, a.sign_bits[k.g * 4 + (t >> 1)] >> (16 * (t & 1)));
    fwht128_oct(v, t);
  }
  const bool store = k.live && k.slot >= 0;
  if (k.bits == 16) {  // both sides, or neither: uniform over the grid
    if (a.sign_bits) float_to_halves(v, r0, r1);
    if (store) {
      reinterpret_cast<uint4*>(k.row)[2 * t] = r0;
      reinterpret_cast<uint4*>(k.row)[2 * t + 1] = r1;
    }
    return;
  }
  float lo = 0.f, hi = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    lo = min_nan(lo, v[j]);
    hi = max_nan(hi, v[j]);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  lo = __fadd_rn(lo, 0.f);  // a zero bound is +0 whichever zero the reduction kept
  const float qmax = (float)((1 << k.bits) - 1);
  const float span = __fdiv_rn(__fsub_rn(hi, lo), qmax);
  const bool finite = span < INFINITY;  // false for NaN too
  __half s16 = __float2half_ru(fminf(span, 65504.f));
  if (!(span > 0.f) || !finite) s16 = __float2half_rn(1.f);
  const float s = __half2float(s16);
  // a group that holds an infinity or NaN reads back as NaN throughout
  const __half z16 = finite ? __float2half_rn(__fdiv_rn(-lo, s)) : __ushort_as_half(0x7fff);
  const float z = __half2float(z16);
  const float inv = __frcp_rn(s);
  uint32_t q[16];  // the code in the low byte: adding 2^23 rounds to an integer, ties to even
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float q0 = __fmul_rn(v[j], inv), d = __fmaf_rn(__fmaf_rn(-q0, s, v[j]), inv, q0);
    q[j] = __float_as_uint(__fadd_rn(fminf(fmaxf(__fadd_rn(d, z), 0.f), qmax), 8388608.f));
  }
  if (!store) return;
  if (k.bits == 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __byte_perm(__byte_perm(q[4 * i], q[4 * i + 1], 0x0040), __byte_perm(q[4 * i + 2], q[4 * i + 3], 0x0040), 0x5410);
    reinterpret_cast<uint4*>(k.row)[t] = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t b[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) b[c] = q[8 * i + 2 * c] + (q[8 * i + 2 * c + 1] << 4);
      w[i] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
    reinterpret_cast<uint2*>(k.row)[t] = make_uint2(w[0], w[1]);
  }
  if (t == 0) *reinterpret_cast<__half2*>(k.par) = __halves2half2(s16, z16);
}

__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvArgs a) {
  const int t = threadIdx.x & 7;
  const int64_t row = (int64_t)a.c.heads * a.c.dim;
  const Task k = find_task(a, t, row, row);
  uint4 r0 = make_uint4(0u, 0u, 0u, 0u), r1 = r0;
  float v[16];
  if (k.bits == 16) {
    r0 = reinterpret_cast<const uint4*>(k.row)[2 * t];
    r1 = reinterpret_cast<const uint4*>(k.row)[2 * t + 1];
    halves_to_float(r0, r1, v);
  } else {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(k.par));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (k.bits == 8) {
      const uint4 c = reinterpret_cast<const uint4*>(k.row)[t];
      w[0] = c.x, w[1] = c.y, w[2] = c.z, w[3] = c.w;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        v[j] = __fmul_rn(p.x, __fsub_rn((float)((w[j >> 2] >> (8 * (j & 3))) & 255u), p.y));
    } else {
      const uint2 c = reinterpret_cast<const uint2*>(k.row)[t];
      w[0] = c.x, w[1] = c.y;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        v[j] = __fmul_rn(p.x, __fsub_rn((float)((w[j >> 3] >> (4 * (j & 7))) & 15u), p.y));
    }
  }
  if (a.sign_bits) {
    fwht128_oct(v, t);
    flip16(v, a.sign_bits[k.g * 4 + (t >> 1)] >> (16 * (t & 1)));
  }
  if (a.sign_bits || k.bits != 16) float_to_halves(v, r0, r1);
  if (k.slot < 0) r0 = r1 = make_uint4(0u, 0u, 0u, 0u);
  if (!k.live) return;
  uint4* dst = reinterpret_cast<uint4*>((k.side ? a.v_out : a.k_out) + k.in + 16 * t);
  dst[0] = r0;
  dst[1] = r1;
}

}  // namespace

unsigned take_kv_error() {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_kv_error, sizeof(v)) != cudaSuccess) return ~0u;
  if (v) cudaMemcpyToSymbol(g_kv_error, &zero, sizeof(zero));
  return v;
}

// Tasks are counted in 31 bits.
static qlin_status kv_grid(const KvArgs& a, unsigned* grid) {
  const int64_t tasks = (int64_t)a.tokens * a.c.heads * 2 * (a.c.dim / kGroup);
  if (tasks > 0x7fffffffLL - kTasksPerCta) return QLIN_ERR_SHAPE;
  *grid = (unsigned)((tasks + kTasksPerCta - 1) / kTasksPerCta);
  return QLIN_OK;
}

qlin_status launch_kv_write(const KvView& c, const __half* k, const __half* v, int64_t k_stride, int64_t v_stride,
                            const int32_t* slots, int tokens, const uint32_t* sign_bits, cudaStream_t s) {
  const KvArgs a = {c, k, v, nullptr, nullptr, k_stride, v_stride, slots, sign_bits, tokens};
  unsigned grid;
  const qlin_status r = kv_grid(a, &grid);
  if (r != QLIN_OK) return r;
  kv_write_kernel<<<grid, kThreads, 0, s>>>(a);
  return record_cuda(cudaGetLastError());
}

qlin_status launch_kv_read(const KvView& c, __half* k, __half* v, const int32_t* slots, int tokens,
                           const uint32_t* sign_bits, cudaStream_t s) {
  const KvArgs a = {c, nullptr, nullptr, k, v, 0, 0, slots, sign_bits, tokens};
  unsigned grid;
  const qlin_status r = kv_grid(a, &grid);
  if (r != QLIN_OK) return r;
  kv_read_kernel<<<grid, kThreads, 0, s>>>(a);
  return record_cuda(cudaGetLastError());
}

}  // namespace qlin
