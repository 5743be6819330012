// qlin_rmsnorm: residual addition and root-mean-square norm in front of a linear
// layer, y = fp16(h / sqrt(mean h^2 + eps) * weight), h = fp16(x + residual).
//
// One CTA a row; bound by HBM (x, residual in; y, residual out).
#include "qlin_internal.cuh"

namespace qlin {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) rmsnorm_kernel(const __half* __restrict__ x, const __half* residual,
                                                           const __half* __restrict__ weight, float eps,
                                                           __half* __restrict__ y, __half* residual_out, int K) {
  __shared__ float part[kThreads / 32];
  const int64_t row = (int64_t)blockIdx.x * K;
  float sum = 0.f;
  for (int i = threadIdx.x; i < K; i += kThreads) {
    float h = __half2float(x[row + i]);
    if (residual) {
      const __half r = __float2half_rn(h + __half2float(residual[row + i]));
      residual_out[row + i] = r;
      h = __half2float(r);
    }
    sum += h * h;
  }
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = 0.f;
  for (int i = 0; i < kThreads / 32; ++i) sum += part[i];
  const float inv = 1.f / sqrtf(sum / (float)K + eps);
  const __half* h = residual ? residual_out : x;  // each thread reads back what it wrote
  for (int i = threadIdx.x; i < K; i += kThreads)
    y[row + i] = __float2half_rn(__half2float(h[row + i]) * inv * __half2float(weight[i]));
}

}  // namespace

qlin_status launch_rmsnorm(const __half* x, const __half* residual, const __half* weight, float eps, __half* y,
                           __half* residual_out, int M, int K, cudaStream_t s) {
  rmsnorm_kernel<<<M, kThreads, 0, s>>>(x, residual, weight, eps, y, residual_out, K);
  return record_cuda(cudaGetLastError());
}

}  // namespace qlin
