// C ABI of the qlin library: argument validation, status codes, dispatch.
// Nothing here computes the layer; it checks arguments and enqueues kernels.
#include <atomic>
#include <cmath>
#include <cstring>
#include <vector>

#include "qlin_internal.cuh"
#include "qlin_kv.cuh"

namespace qlin {

static thread_local int g_last_cuda_error = 0;
static std::atomic<int> g_overlap{0};

bool overlap_enabled() { return g_overlap.load(std::memory_order_relaxed) != 0; }

qlin_status record_cuda(cudaError_t e) {
  if (e == cudaSuccess) return QLIN_OK;
  g_last_cuda_error = (int)e;
  return QLIN_ERR_CUDA;
}

static bool width_ok(int b) { return b == 3 || b == 4 || b == 6 || b == 8; }

static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Validates a descriptor; QLIN_OK if it describes a packed matrix we can read.
static qlin_status check_desc(const qlin_desc* d) {
  if (!d) return QLIN_ERR_INVALID_ARG;
  if (d->N < 1 || d->K < kGroup || d->K % kGroup) return QLIN_ERR_SHAPE;
  if (d->bits == 0) {
    if (d->N % kBlockRows) return QLIN_ERR_SHAPE;
    if (!d->block_bits) return QLIN_ERR_INVALID_ARG;
    for (int j = 0; j < d->N / kBlockRows; ++j)
      if (!width_ok(d->block_bits[j])) return QLIN_ERR_UNSUPPORTED;
    return QLIN_OK;
  }
  return width_ok(d->bits) ? QLIN_OK : QLIN_ERR_UNSUPPORTED;
}

size_t code_bytes(const qlin_desc* d) {
  if (d->bits) return (size_t)d->N * (size_t)d->K * (size_t)d->bits / 8u;
  size_t sum_bits = 0;
  for (int j = 0; j < d->N / kBlockRows; ++j) sum_bits += d->block_bits[j];
  return 8u * (size_t)d->K * sum_bits;
}

size_t table_offset(const qlin_desc* d) { return (code_bytes(d) + 15u) & ~(size_t)15u; }

static size_t packed_bytes(const qlin_desc* d) {
  if (d->bits) return (code_bytes(d) + 15u) & ~(size_t)15u;
  const size_t nb = (size_t)d->N / kBlockRows;
  const size_t t = table_offset(d) + 4u * (nb + 1) + nb;
  return (t + 15u) & ~(size_t)15u;
}

PackedView make_view(const qlin_desc* d, const void* packed) {
  PackedView v;
  v.codes = static_cast<const uint8_t*>(packed);
  v.N = d->N;
  v.K = d->K;
  v.bits = d->bits;
  v.row_bytes_uniform = d->bits ? (int64_t)d->K * d->bits / 8 : 0;
  if (d->bits == 0) {
    const size_t t = table_offset(d);
    v.start16 = reinterpret_cast<const uint32_t*>(v.codes + t);
    v.widths = v.codes + t + 4u * ((size_t)d->N / kBlockRows + 1);
  } else {
    v.start16 = nullptr;
    v.widths = nullptr;
  }
  return v;
}

}  // namespace qlin

using namespace qlin;

extern "C" {

const char* qlin_status_string(qlin_status s) {
  switch (s) {
    case QLIN_OK: return "QLIN_OK";
    case QLIN_ERR_INVALID_ARG: return "QLIN_ERR_INVALID_ARG: null pointer or inconsistent descriptor";
    case QLIN_ERR_UNSUPPORTED: return "QLIN_ERR_UNSUPPORTED: code width must be 3, 4, 6 or 8 (cache: 4 or 8 each side, or 16 both)";
    case QLIN_ERR_SHAPE: return "QLIN_ERR_SHAPE: K must be a positive multiple of 128, N >= 1 (mixed: N % 64 == 0), M in range (cache and norm: see their sizes in qlin.h)";
    case QLIN_ERR_ALIGNMENT: return "QLIN_ERR_ALIGNMENT: buffers must be 16-byte aligned";
    case QLIN_ERR_CUDA: return "QLIN_ERR_CUDA: a CUDA call failed (see qlin_last_cuda_error)";
    case QLIN_ERR_WORKSPACE: return "QLIN_ERR_WORKSPACE: workspace missing or too small";
  }
  return "unknown qlin_status";
}

int qlin_last_cuda_error(void) { return g_last_cuda_error; }

int qlin_set_overlap(int enable) { return g_overlap.exchange(enable ? 1 : 0); }

size_t qlin_packed_bytes(const qlin_desc* d) {
  return check_desc(d) == QLIN_OK ? packed_bytes(d) : 0;
}

size_t qlin_code_bytes(const qlin_desc* d) {
  return check_desc(d) == QLIN_OK ? code_bytes(d) : 0;
}

qlin_status qlin_pack(const qlin_desc* d, const uint8_t* codes, void* packed, qlin_stream_t st) {
  qlin_status r = check_desc(d);
  if (r != QLIN_OK) return r;
  if (!codes || !packed) return QLIN_ERR_INVALID_ARG;
  if (!aligned16(packed)) return QLIN_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(st);
  PackedView v = make_view(d, packed);
  if (d->bits == 0) {
    // Block table: start of each block in 16-byte units, then the widths.
    const int nb = d->N / kBlockRows;
    const size_t tbytes = 4u * (size_t)(nb + 1) + (size_t)nb;
    std::vector<uint8_t> table(tbytes);
    uint32_t* start = reinterpret_cast<uint32_t*>(table.data());
    uint64_t acc16 = 0;  // a block holds 64 * K * b / 8 = 8*K*b bytes = K*b/2 sixteen-byte units
    for (int j = 0; j < nb; ++j) {
      start[j] = (uint32_t)acc16;
      acc16 += (uint64_t)d->K * d->block_bits[j] / 2;
    }
    if (acc16 > 0xFFFFFFFFull) return QLIN_ERR_SHAPE;
    start[nb] = (uint32_t)acc16;
    std::memcpy(table.data() + 4u * (nb + 1), d->block_bits, (size_t)nb);
    uint8_t* dst = static_cast<uint8_t*>(packed) + table_offset(d);
    r = record_cuda(cudaMemcpyAsync(dst, table.data(), tbytes, cudaMemcpyHostToDevice, s));
    if (r != QLIN_OK) return r;
  }
  return launch_pack(v, codes, static_cast<uint8_t*>(packed), s);
}

qlin_status qlin_unpack(const qlin_desc* d, const void* packed, uint8_t* codes, qlin_stream_t st) {
  qlin_status r = check_desc(d);
  if (r != QLIN_OK) return r;
  if (!codes || !packed) return QLIN_ERR_INVALID_ARG;
  if (!aligned16(packed)) return QLIN_ERR_ALIGNMENT;
  return launch_unpack(make_view(d, packed), codes, reinterpret_cast<cudaStream_t>(st));
}

qlin_status qlin_dequant(const qlin_desc* d, const void* packed, const uint16_t* scales,
                         const uint16_t* zeros, uint16_t* w, qlin_stream_t st) {
  qlin_status r = check_desc(d);
  if (r != QLIN_OK) return r;
  if (!packed || !scales || !zeros || !w) return QLIN_ERR_INVALID_ARG;
  if (!aligned16(packed) || !aligned16(scales) || !aligned16(zeros) || !aligned16(w))
    return QLIN_ERR_ALIGNMENT;
  return launch_dequant(make_view(d, packed), reinterpret_cast<const __half*>(scales),
                        reinterpret_cast<const __half*>(zeros), reinterpret_cast<__half*>(w),
                        reinterpret_cast<cudaStream_t>(st));
}

qlin_status qlin_quantize_rtn(const qlin_desc* d, const uint16_t* w, const uint32_t* sign_bits, uint8_t* codes,
                              uint16_t* scales, uint16_t* zeros, qlin_stream_t st) {
  qlin_status r = check_desc(d);
  if (r != QLIN_OK) return r;
  if (!w || !sign_bits || !codes || !scales || !zeros) return QLIN_ERR_INVALID_ARG;
  if (!aligned16(w) || !aligned16(sign_bits) || !aligned16(codes) || !aligned16(scales) || !aligned16(zeros))
    return QLIN_ERR_ALIGNMENT;
  return launch_quantize_rtn(reinterpret_cast<const __half*>(w), sign_bits, d->block_bits, d->bits, d->N, d->K,
                             codes, reinterpret_cast<__half*>(scales), reinterpret_cast<__half*>(zeros),
                             reinterpret_cast<cudaStream_t>(st));
}

size_t qlin_gptq_workspace_bytes(const qlin_desc* d) {
  return check_desc(d) == QLIN_OK ? gptq_workspace_bytes(d->N, d->K) : 0;
}

qlin_status qlin_quantize_gptq(const qlin_desc* d, const uint16_t* w, const uint32_t* sign_bits,
                               const float* hinv_factor, uint8_t* codes, uint16_t* scales, uint16_t* zeros,
                               void* workspace, size_t workspace_bytes, qlin_stream_t st) {
  qlin_status r = check_desc(d);
  if (r != QLIN_OK) return r;
  if (!w || !sign_bits || !hinv_factor || !codes || !scales || !zeros) return QLIN_ERR_INVALID_ARG;
  if (!aligned16(w) || !aligned16(sign_bits) || !aligned16(hinv_factor) || !aligned16(codes) ||
      !aligned16(scales) || !aligned16(zeros))
    return QLIN_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < gptq_workspace_bytes(d->N, d->K)) return QLIN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return QLIN_ERR_ALIGNMENT;
  return launch_quantize_gptq(reinterpret_cast<const __half*>(w), sign_bits, hinv_factor, d->block_bits, d->bits,
                              d->N, d->K, codes, reinterpret_cast<__half*>(scales), reinterpret_cast<__half*>(zeros),
                              workspace, reinterpret_cast<cudaStream_t>(st));
}

qlin_status qlin_rht(const uint16_t* x, uint16_t* xr, const uint32_t* sign_bits, int32_t M,
                     int32_t K, qlin_stream_t st) {
  if (!x || !xr || !sign_bits) return QLIN_ERR_INVALID_ARG;
  if (M < 1 || K < kHadamard || K % kHadamard) return QLIN_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(xr) || !aligned16(sign_bits)) return QLIN_ERR_ALIGNMENT;
  if (x == xr) return QLIN_ERR_INVALID_ARG;
  return launch_rht(reinterpret_cast<const __half*>(x), reinterpret_cast<__half*>(xr), sign_bits,
                    M, K, reinterpret_cast<cudaStream_t>(st));
}

static qlin_status check_linear(const qlin_desc* d, const void* packed, const uint16_t* scales,
                                const uint16_t* zeros, const uint32_t* sign_bits,
                                const uint16_t* x, uint16_t* y) {
  qlin_status r = check_desc(d);
  if (r != QLIN_OK) return r;
  if (!packed || !scales || !zeros || !sign_bits || !x || !y) return QLIN_ERR_INVALID_ARG;
  if (!aligned16(packed) || !aligned16(scales) || !aligned16(zeros) || !aligned16(sign_bits) ||
      !aligned16(x) || !aligned16(y))
    return QLIN_ERR_ALIGNMENT;
  return QLIN_OK;
}

qlin_status qlin_gemv_plan(const qlin_desc* d, int32_t M, qlin_gemv_plan_info* info) {
  qlin_status r = check_desc(d);
  if (r != QLIN_OK) return r;
  if (!info) return QLIN_ERR_INVALID_ARG;
  if (M < 1 || M > 16) return QLIN_ERR_SHAPE;
  gemv_plan_info(d->bits, d->N, d->K, M, info);
  return QLIN_OK;
}

size_t qlin_gemv_workspace_bytes(const qlin_desc* d, int32_t M) {
  if (check_desc(d) != QLIN_OK || M < 1 || M > 16) return 0;
  return gemv_workspace_bytes(d->bits, d->N, d->K, M);
}

qlin_status qlin_gemv(const qlin_desc* d, const void* packed, const uint16_t* scales,
                      const uint16_t* zeros, const uint32_t* sign_bits, const uint16_t* x,
                      uint16_t* y, int32_t M, void* workspace, size_t workspace_bytes,
                      qlin_stream_t st) {
  qlin_status r = check_linear(d, packed, scales, zeros, sign_bits, x, y);
  if (r != QLIN_OK) return r;
  if (M < 1 || M > 16) return QLIN_ERR_SHAPE;
  const size_t ws = gemv_workspace_bytes(d->bits, d->N, d->K, M);
  if (ws && (!workspace || workspace_bytes < ws)) return QLIN_ERR_WORKSPACE;
  if (ws && !aligned16(workspace)) return QLIN_ERR_ALIGNMENT;
  return launch_gemv(make_view(d, packed), reinterpret_cast<const __half*>(scales),
                     reinterpret_cast<const __half*>(zeros), sign_bits,
                     reinterpret_cast<const __half*>(x), reinterpret_cast<__half*>(y), M,
                     workspace, reinterpret_cast<cudaStream_t>(st));
}

size_t qlin_gemm_workspace_bytes(const qlin_desc* d, int32_t M) {
  if (check_desc(d) != QLIN_OK || M < 1) return 0;
  return gemm_workspace_bytes(M, d->K);
}

qlin_status qlin_device_error(uint32_t* code) {
  if (!code) return QLIN_ERR_INVALID_ARG;
  const unsigned a = take_gemv_error(), b = take_gemm_error(), c = take_imma_error(), d = take_tc_error();
  const unsigned e = take_kv_error(), f = take_attn_error();
  if (a == ~0u || b == ~0u || c == ~0u || d == ~0u || e == ~0u || f == ~0u) return QLIN_ERR_CUDA;
  *code = a | c | (b << 8) | (d << 16) | ((e | f) << 24);
  return QLIN_OK;
}

qlin_status qlin_gemm(const qlin_desc* d, const void* packed, const uint16_t* scales,
                      const uint16_t* zeros, const uint32_t* sign_bits, const uint16_t* x,
                      uint16_t* y, int32_t M, void* workspace, size_t workspace_bytes,
                      qlin_stream_t st) {
  qlin_status r = check_linear(d, packed, scales, zeros, sign_bits, x, y);
  if (r != QLIN_OK) return r;
  if (M < 1) return QLIN_ERR_SHAPE;
  if (!workspace || workspace_bytes < gemm_workspace_bytes(M, d->K)) return QLIN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return QLIN_ERR_ALIGNMENT;
  return launch_gemm(make_view(d, packed), reinterpret_cast<const __half*>(scales),
                     reinterpret_cast<const __half*>(zeros), sign_bits,
                     reinterpret_cast<const __half*>(x), reinterpret_cast<__half*>(y), M,
                     workspace, reinterpret_cast<cudaStream_t>(st));
}

qlin_status qlin_linear_host(const qlin_desc* d, const void* packed, const uint16_t* scales,
                             const uint16_t* zeros, const uint32_t* sign_bits, const uint16_t* x_host,
                             uint16_t* y_host, uint16_t* x_dev, uint16_t* y_dev, int32_t M, void* workspace,
                             size_t workspace_bytes, qlin_stream_t st) {
  if (!x_host || !y_host) return QLIN_ERR_INVALID_ARG;
  qlin_status r = check_linear(d, packed, scales, zeros, sign_bits, x_dev, y_dev);
  if (r != QLIN_OK) return r;
  if (M < 1) return QLIN_ERR_SHAPE;
  // every check before the first enqueue: an error enqueues nothing
  const bool gemv = M <= 16;
  const size_t ws = gemv ? gemv_workspace_bytes(d->bits, d->N, d->K, M) : gemm_workspace_bytes(M, d->K);
  if (ws && (!workspace || workspace_bytes < ws)) return QLIN_ERR_WORKSPACE;
  if (ws && !aligned16(workspace)) return QLIN_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(st);
  cudaError_t e = cudaMemcpyAsync(x_dev, x_host, (size_t)M * (size_t)d->K * 2, cudaMemcpyHostToDevice, s);
  if (e != cudaSuccess) return record_cuda(e);
  const PackedView v = make_view(d, packed);
  const __half* xs = reinterpret_cast<const __half*>(x_dev);
  __half* ys = reinterpret_cast<__half*>(y_dev);
  r = gemv ? launch_gemv(v, reinterpret_cast<const __half*>(scales), reinterpret_cast<const __half*>(zeros),
                         sign_bits, xs, ys, M, workspace, s)
           : launch_gemm(v, reinterpret_cast<const __half*>(scales), reinterpret_cast<const __half*>(zeros),
                         sign_bits, xs, ys, M, workspace, s);
  if (r != QLIN_OK) return r;
  return record_cuda(cudaMemcpyAsync(y_host, y_dev, (size_t)M * (size_t)d->N * 2, cudaMemcpyDeviceToHost, s));
}

static qlin_status check_kv(const qlin_kv_desc* d) {
  if (!d) return QLIN_ERR_INVALID_ARG;
  if (d->num_pages < 1 || d->page_size < kPageUnit || d->page_size % kPageUnit || d->kv_heads < 1)
    return QLIN_ERR_SHAPE;
  if (d->head_dim != kGroup && d->head_dim != 2 * kGroup) return QLIN_ERR_SHAPE;
  if ((int64_t)d->num_pages * d->page_size > 0x7fffffffLL) return QLIN_ERR_SHAPE;  // a slot is an int32
  // values of a token; at 4 bytes each (key and value) the pool's size then fits in 64 bits
  if ((int64_t)d->kv_heads * d->head_dim > 0x7fffffffLL) return QLIN_ERR_SHAPE;
  const int k = d->k_bits, v = d->v_bits;
  const bool coded = (k == 4 || k == 8) && (v == 4 || v == 8);
  return coded || (k == 16 && v == 16) ? QLIN_OK : QLIN_ERR_UNSUPPORTED;
}

size_t qlin_kv_cache_bytes(const qlin_kv_desc* d) {
  if (check_kv(d) != QLIN_OK) return 0;
  return (size_t)make_kv_view(d, nullptr).block_bytes * (size_t)d->num_pages * (size_t)d->kv_heads;
}

// Token rows of k, v or q: at least the heads' width apart, 16-byte aligned.
static bool row_stride_ok(int64_t stride, int64_t width) { return stride >= width && stride % 8 == 0; }

qlin_status qlin_kv_write(const qlin_kv_desc* d, void* cache, const uint16_t* k, const uint16_t* v, int64_t k_stride,
                          int64_t v_stride, const int32_t* slots, int32_t T, const uint32_t* sign_bits,
                          qlin_stream_t st) {
  qlin_status r = check_kv(d);
  if (r != QLIN_OK) return r;
  if (!cache || !k || !v || !slots) return QLIN_ERR_INVALID_ARG;
  const int64_t width = (int64_t)d->kv_heads * d->head_dim;
  if (T < 1 || !row_stride_ok(k_stride, width) || !row_stride_ok(v_stride, width)) return QLIN_ERR_SHAPE;
  if (!aligned16(cache) || !aligned16(k) || !aligned16(v) || !aligned4(slots) || !aligned16(sign_bits))
    return QLIN_ERR_ALIGNMENT;
  return launch_kv_write(make_kv_view(d, cache), reinterpret_cast<const __half*>(k),
                         reinterpret_cast<const __half*>(v), k_stride, v_stride, slots, T, sign_bits,
                         reinterpret_cast<cudaStream_t>(st));
}

qlin_status qlin_kv_read(const qlin_kv_desc* d, const void* cache, const int32_t* slots, int32_t T,
                         const uint32_t* sign_bits, uint16_t* k, uint16_t* v, qlin_stream_t st) {
  qlin_status r = check_kv(d);
  if (r != QLIN_OK) return r;
  if (!cache || !k || !v || !slots || k == v) return QLIN_ERR_INVALID_ARG;
  if (T < 1) return QLIN_ERR_SHAPE;
  if (!aligned16(cache) || !aligned16(k) || !aligned16(v) || !aligned4(slots) || !aligned16(sign_bits))
    return QLIN_ERR_ALIGNMENT;
  return launch_kv_read(make_kv_view(d, cache), reinterpret_cast<__half*>(k), reinterpret_cast<__half*>(v), slots, T,
                        sign_bits, reinterpret_cast<cudaStream_t>(st));
}

// Sizes of an attention call; the tiles of 16 tokens over all heads and
// sequences, and a constant for each, are counted in an int32.
static qlin_status check_attn(const qlin_kv_desc* d, int32_t q_heads, int32_t B, int32_t max_pages) {
  qlin_status r = check_kv(d);
  if (r != QLIN_OK) return r;
  if (B < 1 || max_pages < 1 || q_heads < 1 || q_heads % d->kv_heads) return QLIN_ERR_SHAPE;
  const int64_t tokens = (int64_t)max_pages * d->page_size;
  if (tokens > 0x7fffffffLL || (int64_t)B * q_heads > 0x7fffffffLL) return QLIN_ERR_SHAPE;
  if ((double)(tokens / kPageUnit + kItemExtra) * (double)B * (double)q_heads > 2147483647.0) return QLIN_ERR_SHAPE;
  return QLIN_OK;
}

size_t qlin_attn_workspace_bytes(const qlin_kv_desc* d, int32_t q_heads, int32_t B, int32_t max_pages) {
  return check_attn(d, q_heads, B, max_pages) == QLIN_OK ? attn_workspace_bytes(d, q_heads, B, max_pages) : 0;
}

qlin_status qlin_attn_decode(const qlin_kv_desc* d, const void* cache, const uint16_t* q, int64_t q_stride,
                             int32_t q_heads, const int32_t* block_table, int32_t max_pages, const int32_t* seq_lens,
                             int32_t B, const uint32_t* sign_bits, float scale, uint16_t* out, void* workspace,
                             size_t workspace_bytes, qlin_stream_t st) {
  qlin_status r = check_attn(d, q_heads, B, max_pages);
  if (r != QLIN_OK) return r;
  if (!cache || !q || !block_table || !seq_lens || !out || q == out) return QLIN_ERR_INVALID_ARG;
  // Scores of finite values then stay below 256 * 65504 * (255 * 65504) * 2^40 = 2^89, within the kernel's
  // range (running maxima start at -1e30) and far from fp32's.
  if (!(std::fabs(scale) <= 0x1p40f)) return QLIN_ERR_INVALID_ARG;
  if (!row_stride_ok(q_stride, (int64_t)q_heads * d->head_dim)) return QLIN_ERR_SHAPE;
  if (!aligned16(cache) || !aligned16(q) || !aligned4(block_table) || !aligned4(seq_lens) || !aligned16(out) ||
      !aligned16(sign_bits))
    return QLIN_ERR_ALIGNMENT;
  const size_t ws = attn_workspace_bytes(d, q_heads, B, max_pages);
  if (ws && (!workspace || workspace_bytes < ws)) return QLIN_ERR_WORKSPACE;
  if (ws && !aligned16(workspace)) return QLIN_ERR_ALIGNMENT;
  return launch_attn_decode(make_kv_view(d, cache), reinterpret_cast<const __half*>(q), q_stride, q_heads,
                            block_table, max_pages, seq_lens, B, sign_bits, scale, reinterpret_cast<__half*>(out),
                            workspace, reinterpret_cast<cudaStream_t>(st));
}

qlin_status qlin_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps, uint16_t* y,
                         uint16_t* residual_out, int32_t M, int32_t K, qlin_stream_t st) {
  if (!x || !weight || !y || (residual == nullptr) != (residual_out == nullptr)) return QLIN_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return QLIN_ERR_INVALID_ARG;
  if (M < 1 || K < 8 || K % 8 || K > 65536) return QLIN_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(y) || !aligned16(residual_out))
    return QLIN_ERR_ALIGNMENT;
  if (y == x || y == weight || (residual && (y == residual || y == residual_out || residual_out == x || residual_out == weight)))
    return QLIN_ERR_INVALID_ARG;
  return launch_rmsnorm(reinterpret_cast<const __half*>(x), reinterpret_cast<const __half*>(residual),
                        reinterpret_cast<const __half*>(weight), eps, reinterpret_cast<__half*>(y),
                        reinterpret_cast<__half*>(residual_out), M, K, reinterpret_cast<cudaStream_t>(st));
}

}  // extern "C"
