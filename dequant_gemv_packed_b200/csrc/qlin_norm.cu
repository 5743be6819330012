// qlin_rmsnorm: residual addition and root-mean-square norm in front of a linear
// layer, y = fp16(h / sqrt(mean h^2 + eps) * weight), h = fp16(x + residual).
//
// A row stays in registers between its two uses: `warps` warps a row, up to eight
// 16-byte pieces (64 values) a lane.  Bound by HBM: x and the residual in, y and
// the residual out, each once (8,191 x 2,560 takes 26.2 us, 98 % of the copy rate).
// Above 32,768 values a row has eight pieces in each of up to 1,024 threads, whose 64
// registers do not hold row, residual and weight: 45 (plain) and 126 words spill, and
// 256 x 65,536 takes 41.8 us, half the copy rate.
#include "qlin_internal.cuh"
#include "qlin_sm100.cuh"

namespace qlin {
namespace {

constexpr int kMaxWarps = 32;

struct NormArgs {
  const uint4 *x, *residual, *weight;
  uint4 *y, *residual_out;
  float eps, inv_k;
  int rows, pieces;  // of 8 values a row
};

__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = p.x, f[2 * i + 1] = p.y;
  }
}

__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One row a block (blockDim.y = 1) or a warp (blockDim.x = 32); NP pieces a thread.
template <int NP, bool kResidual>
__global__ void __launch_bounds__(kMaxWarps * 32) rmsnorm_kernel(const NormArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();  // a dependent (a GEMV that overlaps) may fetch its weights meanwhile
  __shared__ float part[kMaxWarps];
  const unsigned row = blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= (unsigned)a.rows) return;  // whole warps: blocks of several rows have one warp each
  const int64_t base = (int64_t)row * a.pieces;
  uint4 h[NP], r[NP], w[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int p = threadIdx.x + i * blockDim.x;
    h[i] = r[i] = w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p < a.pieces) {
      h[i] = a.x[base + p];
      if (kResidual) r[i] = a.residual[base + p];
    }
  }
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int p = threadIdx.x + i * blockDim.x;
    if (p < a.pieces) w[i] = __ldg(a.weight + p);
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    float f[8];
    unpack(h[i], f);
    if (kResidual) {
      float g[8];
      unpack(r[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += g[j];
      h[i] = pack(f);
      unpack(h[i], f);
      const int p = threadIdx.x + i * blockDim.x;
      if (p < a.pieces) a.residual_out[base + p] = h[i];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (blockDim.x > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = (threadIdx.x & 31) < (blockDim.x >> 5) ? part[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  const float scale = 1.f / sqrtf(fmaf(sum, a.inv_k, a.eps));
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int p = threadIdx.x + i * blockDim.x;
    if (p < a.pieces) {
      float f[8], g[8];
      unpack(h[i], f);
      unpack(w[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] * scale * g[j];
      a.y[base + p] = pack(f);
    }
  }
}

template <bool kResidual>
qlin_status launch(const NormArgs& a, cudaStream_t s) {
  // A warp a row up to 1,024 values (four rows a block); longer rows a block, two pieces a thread
  // (8 lines in flight each) until the block is full.
  if (a.pieces <= 128) {
    const dim3 block(32, 4);
    const unsigned grid = ((unsigned)a.rows + 3) / 4;
    if (a.pieces <= 32)
      return launch_dependent(rmsnorm_kernel<1, kResidual>, grid, block, 0, s, a);
    else if (a.pieces <= 64)
      return launch_dependent(rmsnorm_kernel<2, kResidual>, grid, block, 0, s, a);
    else
      return launch_dependent(rmsnorm_kernel<4, kResidual>, grid, block, 0, s, a);
  }
  const unsigned grid = (unsigned)a.rows;
  const auto threads = [&](int np) { return dim3((unsigned)(((a.pieces + np - 1) / np + 31) / 32 * 32)); };
  if (a.pieces <= 2048)
    return launch_dependent(rmsnorm_kernel<2, kResidual>, grid, threads(2), 0, s, a);
  else if (a.pieces <= 4096)
    return launch_dependent(rmsnorm_kernel<4, kResidual>, grid, threads(4), 0, s, a);
  else
    return launch_dependent(rmsnorm_kernel<8, kResidual>, grid, threads(8), 0, s, a);
}

}  // namespace

qlin_status launch_rmsnorm(const __half* x, const __half* residual, const __half* weight, float eps, __half* y,
                           __half* residual_out, int M, int K, cudaStream_t s) {
  NormArgs a;
  a.x = reinterpret_cast<const uint4*>(x);
  a.residual = reinterpret_cast<const uint4*>(residual);
  a.weight = reinterpret_cast<const uint4*>(weight);
  a.y = reinterpret_cast<uint4*>(y);
  a.residual_out = reinterpret_cast<uint4*>(residual_out);
  a.eps = eps;
  a.inv_k = 1.f / (float)K;
  a.rows = M;
  a.pieces = K / 8;
  return residual ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace qlin
