// mixllm.cu -- the C ABI declared in include/mixllm.h.  One translation unit:
// it includes the kernels so that they share the device status word.
//
// Host code here only validates arguments, encodes TMA descriptors and
// launches kernels; every step of the layer's arithmetic runs on the GPU.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "../../include/mixllm.h"
#include "gemm_w4w8a8.cuh"
#include "gemm_small_m.cuh"
#include "search.cuh"
#include "kv4_attention.cuh"
#include "kv4_cache.cuh"
#include "kv4_prompt.cuh"
#include "head_norm.cuh"
#include "kv8_attention.cuh"
#include "kv8_cache.cuh"
#include "launch.h"
#include "norm.cuh"
#include "pack_host.cuh"
#include "quant.cuh"
#include "w8a8.cuh"

namespace {

thread_local char g_last_error[512] = "";

mixllm_status fail(mixllm_status st, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return st;
}

mixllm_status ok() {
  g_last_error[0] = '\0';
  return MIXLLM_OK;
}

mixllm_status cuda_fail(cudaError_t e, const char *what) {
  return fail(MIXLLM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Shape checks shared by the entry points.
mixllm_status check_k(int64_t K, int32_t group) {
  if (group != MIXLLM_GROUP) return fail(MIXLLM_ERR_UNSUPPORTED, "group size %d is not supported (only 128)", group);
  if (K <= 0 || K % MIXLLM_GROUP != 0)
    return fail(MIXLLM_ERR_UNSUPPORTED, "K = %lld must be a positive multiple of 128", static_cast<long long>(K));
  if (K > (1ll << 30)) return fail(MIXLLM_ERR_INVALID_ARG, "K = %lld is too large", static_cast<long long>(K));
  return MIXLLM_OK;
}

mixllm_status check_device() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  static std::atomic<unsigned long long> known{0};  // one bit per device ordinal that is sm_100
  if (dev < 64 && (known.load(std::memory_order_relaxed) >> dev & 1)) return MIXLLM_OK;
  int major = 0, minor = 0;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  if (major != 10 || minor != 0)
    return fail(MIXLLM_ERR_UNSUPPORTED, "device %d is sm_%d%d; this library is built for sm_100a only", dev, major,
                minor);
  if (dev < 64) known.fetch_or(1ull << dev);
  return MIXLLM_OK;
}

// Argument checks of the GEMM entry points.  Returns MIXLLM_OK with *empty
// set when there is nothing to compute.
mixllm_status check_gemm(const int8_t *A_q, const float *s_a, int64_t M, int64_t K, const uint8_t *W4,
                         const uint8_t *z4, const void *s_w4, const int32_t *idx4, int64_t N4, const int8_t *W8,
                         const void *s_w8, const int32_t *idx8, int64_t N8, void *Y, int32_t *P, bool *empty) {
  *empty = false;
  mixllm_status st = check_k(K, MIXLLM_GROUP);
  if (st != MIXLLM_OK) return st;
  if (M < 0 || N4 < 0 || N8 < 0) return fail(MIXLLM_ERR_INVALID_ARG, "negative size");
  if (M > 0x7FFFFFFF || N4 + N8 > 0x7FFFFFF0)
    return fail(MIXLLM_ERR_INVALID_ARG, "M or N beyond the supported 2^31 range");
  if (M == 0 || N4 + N8 == 0) {
    *empty = true;
    return MIXLLM_OK;
  }
  if (!A_q || !s_a || !(Y || P)) return fail(MIXLLM_ERR_INVALID_ARG, "null A_q, s_a or output");
  if (!aligned(A_q, 16)) return fail(MIXLLM_ERR_INVALID_ARG, "A_q must be 16-byte aligned");
  if (!aligned(s_a, 4)) return fail(MIXLLM_ERR_INVALID_ARG, "s_a must be 4-byte aligned");
  if (Y && !aligned(Y, 2)) return fail(MIXLLM_ERR_INVALID_ARG, "Y must be 2-byte aligned");
  if (P && !aligned(P, 4)) return fail(MIXLLM_ERR_INVALID_ARG, "P must be 4-byte aligned");
  if (N4 > 0) {
    if (!W4 || !z4 || !s_w4 || !idx4) return fail(MIXLLM_ERR_INVALID_ARG, "null 4-bit set buffer");
    if (!aligned(W4, 16) || !aligned(z4, 16) || !aligned(s_w4, 16) || !aligned(idx4, 4))
      return fail(MIXLLM_ERR_INVALID_ARG, "4-bit set buffers must be 16-byte aligned (idx4: 4)");
  }
  if (N8 > 0) {
    if (!W8 || !s_w8 || !idx8) return fail(MIXLLM_ERR_INVALID_ARG, "null 8-bit set buffer");
    if (!aligned(W8, 16) || !aligned(s_w8, 16) || !aligned(idx8, 4))
      return fail(MIXLLM_ERR_INVALID_ARG, "8-bit set buffers must be 16-byte aligned (idx8: 4)");
  }
  return check_device();
}

mixllm_status gemm_common(const int8_t *A_q, const float *s_a, int64_t M, int64_t K, const uint8_t *W4,
                          const uint8_t *z4, const void *s_w4, const int32_t *idx4, int64_t N4, const int8_t *W8,
                          const void *s_w8, const int32_t *idx8, int64_t N8, void *Y, int32_t *P, void *stream,
                          bool cvt_i2f = false) {
  bool empty = false;
  mixllm_status st = check_gemm(A_q, s_a, M, K, W4, z4, s_w4, idx4, N4, W8, s_w8, idx8, N8, Y, P, &empty);
  if (st != MIXLLM_OK) return st;
  if (empty) return ok();
  mixllm::GemmArgs a{A_q, s_a, M, K, W4, z4, s_w4, idx4, N4, W8, s_w8, idx8, N8, Y, P};
  a.cvt_i2f = cvt_i2f;
  const char *msg = "";
  cudaError_t e = mixllm::launch_gemm_w4w8a8(a, static_cast<cudaStream_t>(stream), &msg);
  if (e == cudaErrorNotSupported) return fail(MIXLLM_ERR_UNSUPPORTED, "%s", msg);
  if (e != cudaSuccess) return fail(MIXLLM_ERR_CUDA, "%s: %s", msg, cudaGetErrorString(e));
  return ok();
}

int page_log2_of(int32_t page_size) {
  for (int l = 4; l <= 8; ++l)
    if (page_size == 1 << l) return l;
  return -1;
}

// The cache's shape and buffers (a cache of no pages may have null buffers).
template <typename Cache, typename Meta>
mixllm_status check_cache(uint8_t *codes, Meta *meta, int64_t pages, int32_t kv_heads, int32_t head_dim,
                          int32_t page_size, Cache *cache) {
  const int page_log2 = page_log2_of(page_size);
  if (page_log2 < 0) return fail(MIXLLM_ERR_UNSUPPORTED, "page size %d is not 16, 32, 64, 128 or 256", page_size);
  if (head_dim != 64 && head_dim != 128)
    return fail(MIXLLM_ERR_UNSUPPORTED, "head size %d is not 64 or 128", head_dim);
  if (kv_heads < 1 || kv_heads > 65536) return fail(MIXLLM_ERR_INVALID_ARG, "%d key heads", kv_heads);
  if (pages < 0 || pages > 0x7FFFFFFF) return fail(MIXLLM_ERR_INVALID_ARG, "bad number of pages");
  if (pages > 0 && (!codes || !meta)) return fail(MIXLLM_ERR_INVALID_ARG, "null cache buffer");
  if (!aligned(codes, 16) || !aligned(meta, 16))
    return fail(MIXLLM_ERR_INVALID_ARG, "the cache's buffers must be 16-byte aligned");
  *cache = Cache{codes, meta, pages, kv_heads, head_dim, page_log2};
  return MIXLLM_OK;
}

mixllm_status check_kv4(uint8_t *codes, uint32_t *meta, int64_t pages, int32_t kv_heads, int32_t head_dim,
                        int32_t page_size, mixllm::Kv4Cache *cache) {
  return check_cache(codes, meta, pages, kv_heads, head_dim, page_size, cache);
}

mixllm_status check_kv_heads(int64_t requests, int64_t max_q, int32_t q_heads, int64_t table_width,
                              int H, int page_log2) {
  if (q_heads < H || q_heads % H != 0 || q_heads > 65536)
    return fail(MIXLLM_ERR_INVALID_ARG, "%d query heads are no multiple of the %d key heads", q_heads, H);
  if (requests < 0 || max_q < 0 || table_width < 0) return fail(MIXLLM_ERR_INVALID_ARG, "negative size");
  if (requests > mixllm::kKv4MaxRequests)
    return fail(MIXLLM_ERR_UNSUPPORTED, "%lld requests are beyond %d", static_cast<long long>(requests),
                mixllm::kKv4MaxRequests);
  if (max_q > 0x7FFFFF00 / (q_heads / H) || table_width > 0x7FFFFF00 >> page_log2)
    return fail(MIXLLM_ERR_INVALID_ARG, "queries or cached tokens of a request beyond the supported 2^31 range");
  return MIXLLM_OK;
}

// The attention over either cache, whose shape and heads have been checked.
template <typename Cache>
mixllm_status attend(const Cache &cache, const void *q_f16, int64_t q_stride, int64_t n_tokens, int32_t q_heads,
                     const int32_t *block_table, int64_t table_stride, int64_t table_width, const int32_t *seq_lens,
                     const int32_t *cu_q, int64_t requests, int64_t max_q, float scale, int32_t causal, void *out_f16,
                     int64_t out_stride, float *lse, void *workspace, size_t workspace_bytes, size_t need,
                     cudaError_t (*launch)(const mixllm::AttendArgsOf<Cache> &, void *, cudaStream_t, const char **),
                     void *stream) {
  if (n_tokens < 0 || n_tokens > 0x7FFFFFFF) return fail(MIXLLM_ERR_INVALID_ARG, "bad number of query tokens");
  if (!std::isfinite(scale)) return fail(MIXLLM_ERR_INVALID_ARG, "scale must be finite");
  if (n_tokens == 0 || requests == 0 || max_q == 0) return ok();
  if (!q_f16 || !out_f16 || !seq_lens || !cu_q || (table_width > 0 && !block_table))
    return fail(MIXLLM_ERR_INVALID_ARG, "null pointer");
  if (!aligned(q_f16, 16) || !aligned(out_f16, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(cu_q, 4) || !aligned(lse, 4))
    return fail(MIXLLM_ERR_INVALID_ARG, "q and out must be 16-byte aligned, the other buffers 4-byte aligned");
  if (q_stride % 8 != 0 || out_stride % 8 != 0)
    return fail(MIXLLM_ERR_INVALID_ARG, "token strides must be multiples of 8 elements");
  if (n_tokens > 1 && out_stride < static_cast<int64_t>(q_heads) * cache.D)
    return fail(MIXLLM_ERR_INVALID_ARG, "rows of out overlap");
  if (workspace_bytes < need)
    return fail(MIXLLM_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu this shape needs",
                workspace_bytes, need);
  if (!workspace || !aligned(workspace, 256))
    return fail(MIXLLM_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device buffer");
  mixllm_status st = check_device();
  if (st != MIXLLM_OK) return st;
  mixllm::AttendArgsOf<Cache> a{cache,
                       static_cast<const __half *>(q_f16),
                       q_stride,
                       n_tokens,
                       q_heads,
                       static_cast<int>(requests),
                       static_cast<int>(max_q),
                       block_table,
                       table_stride,
                       static_cast<int>(table_width),
                       seq_lens,
                       cu_q,
                       scale,
                       causal != 0,
                       static_cast<__half *>(out_f16),
                       out_stride,
                       lse};
  const char *msg = "";
  cudaError_t e = launch(a, workspace, static_cast<cudaStream_t>(stream), &msg);
  if (e == cudaErrorNotSupported) return fail(MIXLLM_ERR_UNSUPPORTED, "%s", msg);
  if (e != cudaSuccess) return fail(MIXLLM_ERR_CUDA, "%s: %s", msg, cudaGetErrorString(e));
  return ok();
}

// The tokens, rotation and norms of the entry points that write heads.
mixllm_status check_turn(int64_t n_tokens, int32_t q_heads, int32_t head_dim, const void *w_q, const void *w_k, float eps,
                         const int32_t *positions, const float *rope, int64_t max_pos, int32_t rotary) {
  if (n_tokens < 0 || n_tokens > 0x7FFFFFFF || q_heads < 0 || q_heads > 65536)
    return fail(MIXLLM_ERR_INVALID_ARG, "bad number of tokens or heads");
  if (rotary < 0 || rotary > head_dim || rotary % 16 != 0)
    return fail(MIXLLM_ERR_UNSUPPORTED, "%d rotated channels: need a multiple of 16 up to the head's %d", rotary, head_dim);
  if (!(eps >= 0.0f)) return fail(MIXLLM_ERR_INVALID_ARG, "eps must not be negative");
  if (n_tokens == 0) return MIXLLM_OK;
  if (rotary > 0 && (!rope || !positions || max_pos <= 0))
    return fail(MIXLLM_ERR_INVALID_ARG, "a rotation needs the table and the positions");
  if (!aligned(w_q, 16) || !aligned(w_k, 16) || !aligned(rope, 16) || !aligned(positions, 4))
    return fail(MIXLLM_ERR_INVALID_ARG, "weights and rope must be 16-byte aligned, positions 4");
  return MIXLLM_OK;
}

// One tensor of heads that is read or written: token stride and alignment.
mixllm_status check_heads(const char *name, const void *p, int64_t stride, int64_t n_tokens, int64_t row, bool written) {
  if (!p) return fail(MIXLLM_ERR_INVALID_ARG, "null %s", name);
  if (!aligned(p, 16)) return fail(MIXLLM_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  if (stride % 8 != 0) return fail(MIXLLM_ERR_INVALID_ARG, "the token stride of %s must be a multiple of 8", name);
  if (written && n_tokens > 1 && stride < row) return fail(MIXLLM_ERR_INVALID_ARG, "rows of %s overlap", name);
  return MIXLLM_OK;
}

mixllm_status check_w8a8(int64_t rows, int64_t K, const char *what) {
  if (K <= 0 || K % 16 != 0 || K > 131056)
    return fail(MIXLLM_ERR_UNSUPPORTED, "K = %lld must be a positive multiple of 16 up to 131056", static_cast<long long>(K));
  if (rows < 0 || rows > 0x7FFFFFFF - 256) return fail(MIXLLM_ERR_INVALID_ARG, "need 0 <= %s < 2^31 - 256", what);
  return MIXLLM_OK;
}

// The product's arguments apart from the activations.  *empty: nothing to compute.
mixllm_status check_w8a8_product(int64_t M, int64_t K, const int8_t *W, const float *s_w, int64_t N, const void *bias,
                                 const void *Y, bool *empty) {
  *empty = false;
  mixllm_status st = check_w8a8(M, K, "M");
  if (st == MIXLLM_OK) st = check_w8a8(N, K, "N");
  if (st != MIXLLM_OK) return st;
  if (M == 0 || N == 0) {
    *empty = true;
    return MIXLLM_OK;
  }
  if (!W || !s_w || !Y) return fail(MIXLLM_ERR_INVALID_ARG, "null W, s_w or Y");
  if (!aligned(W, 16) || !aligned(s_w, 4) || !aligned(bias, 2) || !aligned(Y, 2))
    return fail(MIXLLM_ERR_INVALID_ARG, "W must be 16-byte aligned, s_w 4, bias and Y 2");
  return MIXLLM_OK;
}

mixllm_status w8a8_done(cudaError_t e, const char *msg) {
  if (e == cudaErrorNotSupported) return fail(MIXLLM_ERR_UNSUPPORTED, "%s", msg);
  if (e != cudaSuccess) return fail(MIXLLM_ERR_CUDA, "%s: %s", msg, cudaGetErrorString(e));
  return ok();
}

}  // namespace

extern "C" {

int mixllm_version(void) { return 200; }

const char *mixllm_last_error(void) { return g_last_error; }

mixllm_status mixllm_packed_sizes(int64_t N, int64_t K, int64_t N8, int32_t group, size_t out_bytes[7]) {
  mixllm_status st = check_k(K, group);
  if (st != MIXLLM_OK) return st;
  if (!out_bytes) return fail(MIXLLM_ERR_INVALID_ARG, "null out_bytes");
  if (N < 0 || N8 < 0 || N8 > N) return fail(MIXLLM_ERR_INVALID_ARG, "need 0 <= N8 <= N");
  const int64_t N4 = N - N8, G = K / MIXLLM_GROUP;
  const int64_t N4p = mixllm::padded_channels(N4), N8p = mixllm::padded_channels(N8);
  out_bytes[0] = static_cast<size_t>((N4 + 127) / 128 * 128 * (K / 2));  // whole 128-channel tiles
  out_bytes[1] = static_cast<size_t>(G * (N4p / 2));
  out_bytes[2] = static_cast<size_t>(G * N4p * 2);
  out_bytes[3] = static_cast<size_t>(N4 * 4);
  out_bytes[4] = static_cast<size_t>(N8 * K);
  out_bytes[5] = static_cast<size_t>(G * N8p * 2);
  out_bytes[6] = static_cast<size_t>(N8 * 4);
  return ok();
}

mixllm_status mixllm_quantize_act(const void *X_f16, int64_t M, int64_t K, int32_t group, int8_t *A_q, float *s_a,
                                  void *stream) {
  mixllm_status st = check_k(K, group);
  if (st != MIXLLM_OK) return st;
  if (M < 0) return fail(MIXLLM_ERR_INVALID_ARG, "M < 0");
  if (M == 0) return ok();
  if (!X_f16 || !A_q || !s_a) return fail(MIXLLM_ERR_INVALID_ARG, "null pointer");
  if (!aligned(X_f16, 16) || !aligned(A_q, 16) || !aligned(s_a, 4))
    return fail(MIXLLM_ERR_INVALID_ARG, "X and A_q must be 16-byte aligned, s_a 4-byte aligned");
  st = check_device();
  if (st != MIXLLM_OK) return st;
  cudaError_t e = mixllm::launch_quantize_act(X_f16, M, K, A_q, s_a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "quantize_act launch");
  return ok();
}

mixllm_status mixllm_pack_weights(const float *W, int64_t N, int64_t K, const uint8_t *is8, int64_t N8,
                                  int32_t group, uint8_t *W4, uint8_t *z4, void *s_w4_f16, int32_t *idx4,
                                  int8_t *W8, void *s_w8_f16, int32_t *idx8, void *stream) {
  mixllm_status st = check_k(K, group);
  if (st != MIXLLM_OK) return st;
  if (N < 0 || N8 < 0 || N8 > N) return fail(MIXLLM_ERR_INVALID_ARG, "need 0 <= N8 <= N");
  if (N > 0x7FFFFFF0) return fail(MIXLLM_ERR_INVALID_ARG, "N beyond the supported range");
  if (N == 0) return ok();
  const int64_t N4 = N - N8;
  if (!W || !is8) return fail(MIXLLM_ERR_INVALID_ARG, "null W or is8");
  if (!aligned(W, 16)) return fail(MIXLLM_ERR_INVALID_ARG, "W must be 16-byte aligned");
  if (N4 > 0 && (!W4 || !z4 || !s_w4_f16 || !idx4)) return fail(MIXLLM_ERR_INVALID_ARG, "null 4-bit output");
  if (N8 > 0 && (!W8 || !s_w8_f16 || !idx8)) return fail(MIXLLM_ERR_INVALID_ARG, "null 8-bit output");
  if ((W4 && !aligned(W4, 16)) || (z4 && !aligned(z4, 16)) || (s_w4_f16 && !aligned(s_w4_f16, 16)) ||
      (W8 && !aligned(W8, 16)) || (s_w8_f16 && !aligned(s_w8_f16, 16)) || (idx4 && !aligned(idx4, 4)) ||
      (idx8 && !aligned(idx8, 4)))
    return fail(MIXLLM_ERR_INVALID_ARG, "packed outputs must be 16-byte aligned (idx: 4)");
  st = check_device();
  if (st != MIXLLM_OK) return st;
  // clear any stale status first so a bad bit map is attributed to this call
  st = mixllm_sync_status(stream);
  if (st != MIXLLM_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = mixllm::launch_split_channels(is8, N, N8, idx4, idx8, s);
  if (e != cudaSuccess) return cuda_fail(e, "split_channels launch");
  if (N4 > 0) {
    e = mixllm::launch_pack_w4(W, N, K, idx4, N4, mixllm::padded_channels(N4), W4, z4, s_w4_f16, s);
    if (e != cudaSuccess) return cuda_fail(e, "pack_w4 launch");
  }
  if (N8 > 0) {
    e = mixllm::launch_pack_w8(W, N, K, idx8, N8, mixllm::padded_channels(N8), W8, s_w8_f16, s);
    if (e != cudaSuccess) return cuda_fail(e, "pack_w8 launch");
  }
  e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "pack synchronize");
  int status = 0;
  e = cudaMemcpyFromSymbol(&status, mixllm::g_status, sizeof(int));
  if (e != cudaSuccess) return cuda_fail(e, "status read");
  if (status != 0) {
    const int zero = 0;
    cudaMemcpyToSymbol(mixllm::g_status, &zero, sizeof(int));
    if (status == mixllm::kStatusBadBitmap)
      return fail(MIXLLM_ERR_INVALID_ARG, "the bit map does not flag exactly N8 = %lld channels",
                  static_cast<long long>(N8));
    return fail(MIXLLM_ERR_TIMEOUT, "a device wait gave up during the pack");
  }
  return ok();
}

mixllm_status mixllm_pack_weights_host(const float *W, int64_t N, int64_t K, const uint8_t *is8, int64_t N8,
                                       int32_t group, uint8_t *W4, uint8_t *z4, void *s_w4_f16, int32_t *idx4,
                                       int8_t *W8, void *s_w8_f16, int32_t *idx8) {
  mixllm_status st = check_k(K, group);
  if (st != MIXLLM_OK) return st;
  if (N < 0 || N8 < 0 || N8 > N) return fail(MIXLLM_ERR_INVALID_ARG, "need 0 <= N8 <= N");
  if (N > 0x7FFFFFF0) return fail(MIXLLM_ERR_INVALID_ARG, "N beyond the supported range");
  if (N == 0) return ok();
  const int64_t N4 = N - N8;
  if (!W || !is8) return fail(MIXLLM_ERR_INVALID_ARG, "null W or is8");
  if (N4 > 0 && (!W4 || !z4 || !s_w4_f16 || !idx4)) return fail(MIXLLM_ERR_INVALID_ARG, "null 4-bit output");
  if (N8 > 0 && (!W8 || !s_w8_f16 || !idx8)) return fail(MIXLLM_ERR_INVALID_ARG, "null 8-bit output");
  // the channel lists go to the caller's buffers only once the map is known to be consistent
  int64_t n8 = 0;
  for (int64_t n = 0; n < N; ++n) n8 += is8[n] != 0;
  if (n8 != N8)
    return fail(MIXLLM_ERR_INVALID_ARG, "the bit map flags %lld channels, not N8 = %lld", static_cast<long long>(n8),
                static_cast<long long>(N8));
  (void)mixllm::host_split_channels(is8, N, N8, idx4, idx8);
  if (N4 > 0)
    mixllm::host_pack_w4(W, K, idx4, N4, mixllm::padded_channels(N4), W4, z4, static_cast<__half *>(s_w4_f16));
  if (N8 > 0) mixllm::host_pack_w8(W, K, idx8, N8, mixllm::padded_channels(N8), W8, static_cast<__half *>(s_w8_f16));
  return ok();
}

mixllm_status mixllm_gemm_w4w8a8(const int8_t *A_q, const float *s_a, int64_t M, int64_t K, const uint8_t *W4,
                                 const uint8_t *z4, const void *s_w4_f16, const int32_t *idx4, int64_t N4,
                                 const int8_t *W8, const void *s_w8_f16, const int32_t *idx8, int64_t N8,
                                 void *Y_f16, void *stream) {
  if (!Y_f16 && M > 0 && N4 + N8 > 0) return fail(MIXLLM_ERR_INVALID_ARG, "null Y");
  return gemm_common(A_q, s_a, M, K, W4, z4, s_w4_f16, idx4, N4, W8, s_w8_f16, idx8, N8, Y_f16, nullptr, stream);
}

mixllm_status mixllm_gemm_w4w8a8_plain_i2f(const int8_t *A_q, const float *s_a, int64_t M, int64_t K,
                                           const uint8_t *W4, const uint8_t *z4, const void *s_w4_f16,
                                           const int32_t *idx4, int64_t N4, const int8_t *W8, const void *s_w8_f16,
                                           const int32_t *idx8, int64_t N8, void *Y_f16, void *stream) {
  if (!Y_f16 && M > 0 && N4 + N8 > 0) return fail(MIXLLM_ERR_INVALID_ARG, "null Y");
  return gemm_common(A_q, s_a, M, K, W4, z4, s_w4_f16, idx4, N4, W8, s_w8_f16, idx8, N8, Y_f16, nullptr, stream,
                     true);
}

mixllm_status mixllm_gemm_debug_partials(const int8_t *A_q, const float *s_a, int64_t M, int64_t K,
                                         const uint8_t *W4, const uint8_t *z4, const void *s_w4_f16,
                                         const int32_t *idx4, int64_t N4, const int8_t *W8, const void *s_w8_f16,
                                         const int32_t *idx8, int64_t N8, int32_t *P, void *stream) {
  if (!P && M > 0 && N4 + N8 > 0) return fail(MIXLLM_ERR_INVALID_ARG, "null P");
  return gemm_common(A_q, s_a, M, K, W4, z4, s_w4_f16, idx4, N4, W8, s_w8_f16, idx8, N8, nullptr, P, stream);
}

mixllm_status mixllm_small_m_workspace_bytes(int64_t M, int64_t K, int64_t N4, int64_t N8, size_t *bytes) {
  mixllm_status st = check_k(K, MIXLLM_GROUP);
  if (st != MIXLLM_OK) return st;
  if (!bytes) return fail(MIXLLM_ERR_INVALID_ARG, "null bytes");
  if (M < 1 || M > 64) return fail(MIXLLM_ERR_INVALID_ARG, "the small-M path takes 1 <= M <= 64");
  if (N4 < 0 || N8 < 0 || N4 + N8 > 0x7FFFFFF0) return fail(MIXLLM_ERR_INVALID_ARG, "bad N4 / N8");
  *bytes = mixllm::small_m_workspace_bytes(M, N4, N8, K);
  return ok();
}

mixllm_status mixllm_small_m_kernel(int64_t M, int64_t K, int64_t N4, int64_t N8, int32_t *kind) {
  mixllm_status st = check_k(K, MIXLLM_GROUP);
  if (st != MIXLLM_OK) return st;
  if (!kind) return fail(MIXLLM_ERR_INVALID_ARG, "null kind");
  if (M < 1 || M > 64) return fail(MIXLLM_ERR_INVALID_ARG, "the small-M path takes 1 <= M <= 64");
  if (N4 < 0 || N8 < 0 || N4 + N8 > 0x7FFFFFF0) return fail(MIXLLM_ERR_INVALID_ARG, "bad N4 / N8");
  *kind = mixllm::small_m_kernel_kind(M, N4, N8, K);
  return ok();
}

mixllm_status mixllm_gemm_w4w8a8_small_m(const int8_t *A_q, const float *s_a, int64_t M, int64_t K,
                                         const uint8_t *W4, const uint8_t *z4, const void *s_w4_f16,
                                         const int32_t *idx4, int64_t N4, const int8_t *W8, const void *s_w8_f16,
                                         const int32_t *idx8, int64_t N8, void *Y_f16, void *workspace,
                                         size_t workspace_bytes, void *stream) {
  if (M > 64) return fail(MIXLLM_ERR_INVALID_ARG, "the small-M path takes M <= 64 (M = %lld)", static_cast<long long>(M));
  if (!Y_f16 && M > 0 && N4 + N8 > 0) return fail(MIXLLM_ERR_INVALID_ARG, "null Y");
  bool empty = false;
  mixllm_status st =
      check_gemm(A_q, s_a, M, K, W4, z4, s_w4_f16, idx4, N4, W8, s_w8_f16, idx8, N8, Y_f16, nullptr, &empty);
  if (st != MIXLLM_OK) return st;
  if (empty) return ok();
  const size_t need = mixllm::small_m_workspace_bytes(M, N4, N8, K);
  if (workspace_bytes < need)
    return fail(MIXLLM_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu this shape needs",
                workspace_bytes, need);
  if (need > 0 && (!workspace || !aligned(workspace, 16)))
    return fail(MIXLLM_ERR_INVALID_ARG, "workspace must be a 16-byte aligned device buffer");
  mixllm::GemmArgs a{A_q, s_a, M, K, W4, z4, s_w4_f16, idx4, N4, W8, s_w8_f16, idx8, N8, Y_f16, nullptr};
  const char *msg = "";
  cudaError_t e = mixllm::launch_gemm_small_m(a, workspace, workspace_bytes, static_cast<cudaStream_t>(stream), &msg);
  if (e == cudaErrorNotSupported) return fail(MIXLLM_ERR_UNSUPPORTED, "%s", msg);
  if (e != cudaSuccess) return fail(MIXLLM_ERR_CUDA, "%s: %s", msg, cudaGetErrorString(e));
  return ok();
}

mixllm_status mixllm_small_m_debug_workspace_bytes(int64_t M, int64_t K, int64_t N4, int64_t N8, int32_t kind,
                                                   size_t *bytes) {
  mixllm_status st = check_k(K, MIXLLM_GROUP);
  if (st != MIXLLM_OK) return st;
  if (!bytes) return fail(MIXLLM_ERR_INVALID_ARG, "null bytes");
  if (M < 1 || M > 64) return fail(MIXLLM_ERR_INVALID_ARG, "the small-M path takes 1 <= M <= 64");
  if (N4 < 0 || N8 < 0 || N4 + N8 > 0x7FFFFFF0) return fail(MIXLLM_ERR_INVALID_ARG, "bad N4 / N8");
  if (!mixllm::small_m_kernel_allowed(M, N4, N8, K, kind))
    return fail(MIXLLM_ERR_UNSUPPORTED, "few-token kernel %d cannot take M = %lld, K = %lld", static_cast<int>(kind),
                static_cast<long long>(M), static_cast<long long>(K));
  *bytes = mixllm::small_m_debug_workspace_bytes(M, N4, N8, K, kind);
  return ok();
}

mixllm_status mixllm_small_m_debug_partials(const int8_t *A_q, const float *s_a, int64_t M, int64_t K,
                                            const uint8_t *W4, const uint8_t *z4, const void *s_w4_f16,
                                            const int32_t *idx4, int64_t N4, const int8_t *W8,
                                            const void *s_w8_f16, const int32_t *idx8, int64_t N8, int32_t kind,
                                            int32_t *P, void *Y_f16, void *workspace, size_t workspace_bytes,
                                            void *stream) {
  if (M < 1 || M > 64) return fail(MIXLLM_ERR_INVALID_ARG, "the small-M path takes 1 <= M <= 64");
  if (N4 + N8 > 0 && (!Y_f16 || !P)) return fail(MIXLLM_ERR_INVALID_ARG, "null Y or P");
  bool empty = false;
  mixllm_status st =
      check_gemm(A_q, s_a, M, K, W4, z4, s_w4_f16, idx4, N4, W8, s_w8_f16, idx8, N8, Y_f16, nullptr, &empty);
  if (st != MIXLLM_OK) return st;
  if (empty) return ok();
  if (!mixllm::small_m_kernel_allowed(M, N4, N8, K, kind))
    return fail(MIXLLM_ERR_UNSUPPORTED, "few-token kernel %d cannot take M = %lld, K = %lld", static_cast<int>(kind),
                static_cast<long long>(M), static_cast<long long>(K));
  if (!aligned(P, 4)) return fail(MIXLLM_ERR_INVALID_ARG, "P must be 4-byte aligned");
  const size_t need = mixllm::small_m_debug_workspace_bytes(M, N4, N8, K, kind);
  if (workspace_bytes < need)
    return fail(MIXLLM_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu this shape needs",
                workspace_bytes, need);
  if (need > 0 && (!workspace || !aligned(workspace, 16)))
    return fail(MIXLLM_ERR_INVALID_ARG, "workspace must be a 16-byte aligned device buffer");
  mixllm::GemmArgs a{A_q, s_a, M, K, W4, z4, s_w4_f16, idx4, N4, W8, s_w8_f16, idx8, N8, Y_f16, P};
  const char *msg = "";
  cudaError_t e = mixllm::launch_small_m_debug_partials(a, kind, workspace, workspace_bytes,
                                                        static_cast<cudaStream_t>(stream), &msg);
  if (e == cudaErrorNotSupported) return fail(MIXLLM_ERR_UNSUPPORTED, "%s", msg);
  if (e != cudaSuccess) return fail(MIXLLM_ERR_CUDA, "%s: %s", msg, cudaGetErrorString(e));
  return ok();
}

mixllm_status mixllm_gemm_w4w8a8_small_m_noalloc(const int8_t *A_q, const float *s_a, int64_t M, int64_t K,
                                                 const uint8_t *W4, const uint8_t *z4, const void *s_w4_f16,
                                                 const int32_t *idx4, int64_t N4, const int8_t *W8,
                                                 const void *s_w8_f16, const int32_t *idx8, int64_t N8, void *Y_f16,
                                                 void *stream) {
  if (M > 64) return fail(MIXLLM_ERR_INVALID_ARG, "the small-M path takes M <= 64 (M = %lld)", static_cast<long long>(M));
  if (!Y_f16 && M > 0 && N4 + N8 > 0) return fail(MIXLLM_ERR_INVALID_ARG, "null Y");
  bool empty = false;
  mixllm_status st =
      check_gemm(A_q, s_a, M, K, W4, z4, s_w4_f16, idx4, N4, W8, s_w8_f16, idx8, N8, Y_f16, nullptr, &empty);
  if (st != MIXLLM_OK) return st;
  if (empty) return ok();
  const size_t need = mixllm::small_m_workspace_bytes(M, N4, N8, K);
  if (need > mixllm::small_m_scratch_capacity())
    return fail(MIXLLM_ERR_UNSUPPORTED, "this shape needs %zu bytes of scratch; the static buffer holds %zu", need,
                mixllm::small_m_scratch_capacity());
  mixllm::GemmArgs a{A_q, s_a, M, K, W4, z4, s_w4_f16, idx4, N4, W8, s_w8_f16, idx8, N8, Y_f16, nullptr};
  const char *msg = "";
  cudaError_t e = mixllm::launch_gemm_small_m_noalloc(a, static_cast<cudaStream_t>(stream), &msg);
  if (e == cudaErrorNotSupported) return fail(MIXLLM_ERR_UNSUPPORTED, "%s", msg);
  if (e != cudaSuccess) return fail(MIXLLM_ERR_CUDA, "%s: %s", msg, cudaGetErrorString(e));
  return ok();
}

mixllm_status mixllm_linear_small_m_workspace_bytes(int64_t M, int64_t K, int64_t N4, int64_t N8, size_t *bytes) {
  mixllm_status st = check_k(K, MIXLLM_GROUP);
  if (st != MIXLLM_OK) return st;
  if (!bytes) return fail(MIXLLM_ERR_INVALID_ARG, "null bytes");
  if (M < 1 || M > 64) return fail(MIXLLM_ERR_INVALID_ARG, "the small-M path takes 1 <= M <= 64");
  if (N4 < 0 || N8 < 0 || N4 + N8 > 0x7FFFFFF0) return fail(MIXLLM_ERR_INVALID_ARG, "bad N4 / N8");
  *bytes = mixllm::linear_small_m_workspace_bytes(M, N4, N8, K);
  return ok();
}

mixllm_status mixllm_linear_small_m(const void *X_f16, int64_t M, int64_t K, const uint8_t *W4, const uint8_t *z4,
                                    const void *s_w4_f16, const int32_t *idx4, int64_t N4, const int8_t *W8,
                                    const void *s_w8_f16, const int32_t *idx8, int64_t N8, void *Y_f16,
                                    void *workspace, size_t workspace_bytes, void *stream) {
  if (M > 64) return fail(MIXLLM_ERR_INVALID_ARG, "the small-M path takes M <= 64 (M = %lld)", static_cast<long long>(M));
  if (M > 0 && N4 + N8 > 0) {
    if (!X_f16 || !Y_f16) return fail(MIXLLM_ERR_INVALID_ARG, "null X or Y");
    if (!aligned(X_f16, 16)) return fail(MIXLLM_ERR_INVALID_ARG, "X must be 16-byte aligned");
  }
  bool empty = false;
  // the weight and size checks of the GEMM (X stands in for A_q / s_a, whose checks it passes)
  mixllm_status st = check_gemm(static_cast<const int8_t *>(X_f16), static_cast<const float *>(X_f16), M, K, W4, z4,
                                s_w4_f16, idx4, N4, W8, s_w8_f16, idx8, N8, Y_f16, nullptr, &empty);
  if (st != MIXLLM_OK) return st;
  if (empty) return ok();
  const size_t need = mixllm::linear_small_m_workspace_bytes(M, N4, N8, K);
  if (workspace_bytes < need)
    return fail(MIXLLM_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu this shape needs",
                workspace_bytes, need);
  if (need > 0 && (!workspace || !aligned(workspace, 256)))
    return fail(MIXLLM_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device buffer");
  mixllm::GemmArgs a{nullptr, nullptr, M, K, W4, z4, s_w4_f16, idx4, N4, W8, s_w8_f16, idx8, N8, Y_f16, nullptr};
  a.X = X_f16;
  const char *msg = "";
  cudaError_t e = mixllm::launch_linear_small_m(a, workspace, workspace_bytes, static_cast<cudaStream_t>(stream), &msg);
  if (e == cudaErrorNotSupported) return fail(MIXLLM_ERR_UNSUPPORTED, "%s", msg);
  if (e != cudaSuccess) return fail(MIXLLM_ERR_CUDA, "%s: %s", msg, cudaGetErrorString(e));
  return ok();
}

mixllm_status mixllm_linear_workspace_bytes(int64_t M, int64_t K, int64_t N4, int64_t N8, size_t *bytes) {
  mixllm_status st = check_k(K, MIXLLM_GROUP);
  if (st != MIXLLM_OK) return st;
  if (!bytes) return fail(MIXLLM_ERR_INVALID_ARG, "null bytes");
  if (M < 0) return fail(MIXLLM_ERR_INVALID_ARG, "M < 0");
  if (N4 < 0 || N8 < 0 || N4 + N8 > 0x7FFFFFF0) return fail(MIXLLM_ERR_INVALID_ARG, "bad N4 / N8");
  *bytes = M == 0 ? 0 : mixllm::linear_workspace_bytes(M, N4, N8, K);
  return ok();
}

static mixllm_status linear_entry(const void *X_f16, int64_t M, int64_t K, const uint8_t *W4, const uint8_t *z4,
                                  const void *s_w4_f16, const int32_t *idx4, int64_t N4, const int8_t *W8,
                                  const void *s_w8_f16, const int32_t *idx8, int64_t N8, void *Y_f16,
                                  void *workspace, size_t workspace_bytes, void *stream, bool one_launch) {
  if (one_launch && M > 0 && M <= 64)
    return fail(MIXLLM_ERR_INVALID_ARG, "the one-launch tiled form takes M > 64 (M = %lld)", static_cast<long long>(M));
  if (M > 0 && M <= 64)
    return mixllm_linear_small_m(X_f16, M, K, W4, z4, s_w4_f16, idx4, N4, W8, s_w8_f16, idx8, N8, Y_f16, workspace,
                                 workspace_bytes, stream);
  if (M > 0 && N4 + N8 > 0) {
    if (!X_f16 || !Y_f16) return fail(MIXLLM_ERR_INVALID_ARG, "null X or Y");
    if (!aligned(X_f16, 16)) return fail(MIXLLM_ERR_INVALID_ARG, "X must be 16-byte aligned");
  }
  bool empty = false;
  // the weight and size checks of the GEMM (X stands in for A_q / s_a, whose checks it passes)
  mixllm_status st = check_gemm(static_cast<const int8_t *>(X_f16), static_cast<const float *>(X_f16), M, K, W4, z4,
                                s_w4_f16, idx4, N4, W8, s_w8_f16, idx8, N8, Y_f16, nullptr, &empty);
  if (st != MIXLLM_OK) return st;
  if (empty) return ok();
  const size_t need = mixllm::linear_workspace_bytes(M, N4, N8, K);
  if (workspace_bytes < need)
    return fail(MIXLLM_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu this shape needs",
                workspace_bytes, need);
  if (!workspace || !aligned(workspace, 256))
    return fail(MIXLLM_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device buffer");
  mixllm::GemmArgs a{nullptr, nullptr, M, K, W4, z4, s_w4_f16, idx4, N4, W8, s_w8_f16, idx8, N8, Y_f16, nullptr};
  a.X = X_f16;
  const char *msg = "";
  cudaError_t e =
      mixllm::launch_linear(a, workspace, workspace_bytes, one_launch, static_cast<cudaStream_t>(stream), &msg);
  if (e == cudaErrorNotSupported) return fail(MIXLLM_ERR_UNSUPPORTED, "%s", msg);
  if (e != cudaSuccess) return fail(MIXLLM_ERR_CUDA, "%s: %s", msg, cudaGetErrorString(e));
  return ok();
}

mixllm_status mixllm_linear(const void *X_f16, int64_t M, int64_t K, const uint8_t *W4, const uint8_t *z4,
                            const void *s_w4_f16, const int32_t *idx4, int64_t N4, const int8_t *W8,
                            const void *s_w8_f16, const int32_t *idx8, int64_t N8, void *Y_f16, void *workspace,
                            size_t workspace_bytes, void *stream) {
  return linear_entry(X_f16, M, K, W4, z4, s_w4_f16, idx4, N4, W8, s_w8_f16, idx8, N8, Y_f16, workspace,
                      workspace_bytes, stream, false);
}

mixllm_status mixllm_linear_one_launch(const void *X_f16, int64_t M, int64_t K, const uint8_t *W4, const uint8_t *z4,
                                       const void *s_w4_f16, const int32_t *idx4, int64_t N4, const int8_t *W8,
                                       const void *s_w8_f16, const int32_t *idx8, int64_t N8, void *Y_f16,
                                       void *workspace, size_t workspace_bytes, void *stream) {
  return linear_entry(X_f16, M, K, W4, z4, s_w4_f16, idx4, N4, W8, s_w8_f16, idx8, N8, Y_f16, workspace,
                      workspace_bytes, stream, true);
}

mixllm_status mixllm_channel_salience(const float *W, int64_t N, int64_t K, const float *G, int64_t D, float *S,
                                      void *stream) {
  mixllm_status st = check_k(K, MIXLLM_GROUP);
  if (st != MIXLLM_OK) return st;
  if (K > 56832) return fail(MIXLLM_ERR_UNSUPPORTED, "K = %lld is beyond 56832", static_cast<long long>(K));
  if (N < 0 || D < 1) return fail(MIXLLM_ERR_INVALID_ARG, "need N >= 0 and D >= 1");
  if (N > 0x7FFFFFFF) return fail(MIXLLM_ERR_INVALID_ARG, "N beyond the supported 2^31 range");
  if (N == 0) return ok();
  if (!W || !G || !S) return fail(MIXLLM_ERR_INVALID_ARG, "null pointer");
  if (!aligned(W, 16) || !aligned(G, 16) || !aligned(S, 4))
    return fail(MIXLLM_ERR_INVALID_ARG, "W and G must be 16-byte aligned, S 4-byte aligned");
  st = check_device();
  if (st != MIXLLM_OK) return st;
  const char *msg = "";
  cudaError_t e = mixllm::launch_channel_salience(W, N, K, G, D, S, static_cast<cudaStream_t>(stream), &msg);
  if (e != cudaSuccess) return fail(MIXLLM_ERR_CUDA, "%s: %s", msg, cudaGetErrorString(e));
  return ok();
}

mixllm_status mixllm_select_top_t_workspace_bytes(int64_t n, size_t *bytes) {
  if (!bytes) return fail(MIXLLM_ERR_INVALID_ARG, "null bytes");
  if (n < 0 || n > (1ll << 40)) return fail(MIXLLM_ERR_INVALID_ARG, "bad n");
  *bytes = mixllm::select_top_t_workspace_bytes(n);
  return ok();
}

mixllm_status mixllm_select_top_t(const float *S, int64_t n, int64_t T, uint8_t *is8, void *workspace,
                                  size_t workspace_bytes, void *stream) {
  if (n < 0 || n > (1ll << 40)) return fail(MIXLLM_ERR_INVALID_ARG, "bad n");
  if (T < 0 || T > n) return fail(MIXLLM_ERR_INVALID_ARG, "need 0 <= T <= n");
  if (n == 0) return ok();
  if (!S || !is8) return fail(MIXLLM_ERR_INVALID_ARG, "null pointer");
  if (!aligned(S, 4)) return fail(MIXLLM_ERR_INVALID_ARG, "S must be 4-byte aligned");
  const size_t need = mixllm::select_top_t_workspace_bytes(n);
  if (workspace_bytes < need || !workspace || !aligned(workspace, 16))
    return fail(MIXLLM_ERR_INVALID_ARG, "workspace must be a 16-byte aligned device buffer of %zu bytes", need);
  mixllm_status st = check_device();
  if (st != MIXLLM_OK) return st;
  const char *msg = "";
  cudaError_t e = mixllm::launch_select_top_t(S, n, T, is8, workspace, static_cast<cudaStream_t>(stream), &msg);
  if (e != cudaSuccess) return fail(MIXLLM_ERR_CUDA, "%s: %s", msg, cudaGetErrorString(e));
  return ok();
}

mixllm_status mixllm_dequantize_act(const int8_t *A_q, const float *s_a, int64_t M, int64_t K, int32_t group,
                                    void *X_f16, void *stream) {
  mixllm_status st = check_k(K, group);
  if (st != MIXLLM_OK) return st;
  if (M < 0) return fail(MIXLLM_ERR_INVALID_ARG, "M < 0");
  if (M > (1ll << 40)) return fail(MIXLLM_ERR_INVALID_ARG, "M is too large");
  if (M == 0) return ok();
  if (!X_f16 || !A_q || !s_a) return fail(MIXLLM_ERR_INVALID_ARG, "null pointer");
  if (!aligned(X_f16, 16) || !aligned(A_q, 8) || !aligned(s_a, 4))
    return fail(MIXLLM_ERR_INVALID_ARG, "X must be 16-byte aligned, A_q 8-byte and s_a 4-byte aligned");
  st = check_device();
  if (st != MIXLLM_OK) return st;
  cudaError_t e = mixllm::launch_dequantize_act(A_q, s_a, M, K, X_f16, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "dequantize_act launch");
  return ok();
}

mixllm_status mixllm_residual_norm(const void *r, int64_t r_stride, int32_t r_is_f32, const void *x_f16,
                                   int64_t x_stride, const void *w_post_f16, const void *gate_f16,
                                   int64_t gate_stride, float scale, void *r_out, int64_t r_out_stride,
                                   const void *w_f16, float eps, int64_t M, int64_t K, void *y_f16, int8_t *A_q,
                                   float *s_a, void *stream) {
  mixllm_status st = check_k(K, MIXLLM_GROUP);
  if (st != MIXLLM_OK) return st;
  if (K > 32768) return fail(MIXLLM_ERR_UNSUPPORTED, "K = %lld is beyond 32768", static_cast<long long>(K));
  if (M < 0 || M > 0x7FFFFFFF) return fail(MIXLLM_ERR_INVALID_ARG, "need 0 <= M < 2^31");
  if (!(eps >= 0.0f)) return fail(MIXLLM_ERR_INVALID_ARG, "eps must not be negative");
  if (M == 0) return ok();
  if (!r || !w_f16) return fail(MIXLLM_ERR_INVALID_ARG, "null r or w");
  if (!y_f16 && !A_q) return fail(MIXLLM_ERR_INVALID_ARG, "null output");
  if (!A_q != !s_a) return fail(MIXLLM_ERR_INVALID_ARG, "A_q and s_a go together");
  if (!x_f16 && (w_post_f16 || gate_f16 || r_out))
    return fail(MIXLLM_ERR_INVALID_ARG, "w_post, gate and r_out need x");
  if (!aligned(r, 16) || !aligned(x_f16, 16) || !aligned(w_post_f16, 16) || !aligned(gate_f16, 16) ||
      !aligned(r_out, 16) || !aligned(w_f16, 16) || !aligned(y_f16, 16) || !aligned(A_q, 8) || !aligned(s_a, 4))
    return fail(MIXLLM_ERR_INVALID_ARG, "buffers must be 16-byte aligned (A_q: 8, s_a: 4)");
  const int64_t run = r_is_f32 ? 4 : 8;  // elements of 16 bytes
  if (r_stride % run != 0 || (r_out && r_out_stride % run != 0) || (x_f16 && x_stride % 8 != 0) ||
      (gate_f16 && gate_stride % 8 != 0))
    return fail(MIXLLM_ERR_INVALID_ARG, "row strides must be multiples of 16 bytes");
  if (M > 1 && r_out && r_out_stride < K) return fail(MIXLLM_ERR_INVALID_ARG, "rows of r_out overlap");
  st = check_device();
  if (st != MIXLLM_OK) return st;
  mixllm::NormArgs a{M,
                     K,
                     static_cast<const __half *>(x_f16),
                     x_stride,
                     static_cast<const __half *>(w_post_f16),
                     static_cast<const __half *>(gate_f16),
                     gate_stride,
                     scale,
                     r,
                     r_stride,
                     r_is_f32 != 0,
                     r_out,
                     r_out_stride,
                     static_cast<const __half *>(w_f16),
                     eps,
                     static_cast<__half *>(y_f16),
                     A_q,
                     s_a};
  cudaError_t e = mixllm::launch_residual_norm(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "residual_norm launch");
  return ok();
}

mixllm_status mixllm_kv4_assign(const int32_t *ctx_lens, const int32_t *new_lens, int64_t requests,
                                int32_t *block_table, int64_t table_stride, int64_t table_width,
                                const int32_t *free_pages, int64_t n_free, const int32_t *free_count,
                                int32_t page_size, int32_t *seq_lens, int32_t *cu_new, int64_t *slots,
                                int32_t *positions, int64_t n_slots, int32_t *free_left, int32_t *status,
                                void *stream) {
  const int page_log2 = page_log2_of(page_size);
  if (page_log2 < 0) return fail(MIXLLM_ERR_UNSUPPORTED, "page size %d is not 16, 32, 64, 128 or 256", page_size);
  if (requests < 0 || table_width < 0 || n_free < 0 || n_slots < 0)
    return fail(MIXLLM_ERR_INVALID_ARG, "negative size");
  if (requests > mixllm::kKv4MaxRequests)
    return fail(MIXLLM_ERR_UNSUPPORTED, "%lld requests are beyond %d", static_cast<long long>(requests),
                mixllm::kKv4MaxRequests);
  if (n_slots > 0x7FFFFFF0 || n_free > 0x7FFFFFF0 || table_width > 0x7FFFFFF0 >> page_log2)
    return fail(MIXLLM_ERR_INVALID_ARG, "slots, pages or a request's tokens beyond the supported 2^31 range");
  if (requests > 1 && table_stride < table_width) return fail(MIXLLM_ERR_INVALID_ARG, "rows of the table overlap");
  if (!cu_new || !free_count || !free_left || !status || (requests > 0 && (!ctx_lens || !new_lens || !seq_lens)) ||
      (requests > 0 && table_width > 0 && !block_table) || (n_free > 0 && !free_pages) ||
      (n_slots > 0 && (!slots || !positions)))
    return fail(MIXLLM_ERR_INVALID_ARG, "null pointer");
  if (!aligned(ctx_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4) || !aligned(free_pages, 4) ||
      !aligned(free_count, 4) || !aligned(seq_lens, 4) || !aligned(cu_new, 4) || !aligned(slots, 8) ||
      !aligned(positions, 4) || !aligned(free_left, 4) || !aligned(status, 4))
    return fail(MIXLLM_ERR_INVALID_ARG, "buffers must be 4-byte aligned (slots: 8)");
  mixllm_status st = check_device();
  if (st != MIXLLM_OK) return st;
  mixllm::AssignArgs a{ctx_lens, new_lens, static_cast<int>(requests), block_table, table_stride,
                       static_cast<int>(table_width), free_pages, static_cast<int>(n_free), free_count, page_log2,
                       seq_lens, cu_new, slots, positions, n_slots, free_left, status};
  const char *msg = "";
  cudaError_t e = mixllm::launch_kv4_assign(a, static_cast<cudaStream_t>(stream), &msg);
  if (e != cudaSuccess) return fail(MIXLLM_ERR_CUDA, "%s: %s", msg, cudaGetErrorString(e));
  return ok();
}

mixllm_status mixllm_kv4_append(uint8_t *codes, uint32_t *meta, int64_t pages, int32_t kv_heads, int32_t head_dim,
                                int32_t page_size, const int64_t *slots, int64_t n_slots, const void *k_f16,
                                int64_t k_stride, const void *v_f16, int64_t v_stride, const void *q_f16,
                                int64_t q_stride, int32_t q_heads, void *q_out_f16, int64_t q_out_stride,
                                const int32_t *positions, const float *rope, int64_t max_pos, int32_t rotary,
                                void *stream) {
  mixllm::Kv4Cache cache;
  mixllm_status st = check_kv4(codes, meta, pages, kv_heads, head_dim, page_size, &cache);
  if (st != MIXLLM_OK) return st;
  if (n_slots < 0 || n_slots > 0x7FFFFFFF || q_heads < 0 || q_heads > 65536)
    return fail(MIXLLM_ERR_INVALID_ARG, "bad number of tokens or heads");
  if (rotary < 0 || rotary > head_dim || rotary % 16 != 0)
    return fail(MIXLLM_ERR_UNSUPPORTED, "%d rotated channels: need a multiple of 16 up to the head's %d", rotary, head_dim);
  if (n_slots == 0) return ok();
  if (!slots || !k_f16 || !v_f16) return fail(MIXLLM_ERR_INVALID_ARG, "null slots, k or v");
  if (q_heads > 0 && (!q_f16 || !q_out_f16)) return fail(MIXLLM_ERR_INVALID_ARG, "null q or q_out");
  if (rotary > 0 && (!rope || !positions || max_pos <= 0))
    return fail(MIXLLM_ERR_INVALID_ARG, "a rotation needs the table and the positions");
  if (!aligned(slots, 8) || !aligned(k_f16, 16) || !aligned(v_f16, 16) || !aligned(q_f16, 16) ||
      !aligned(q_out_f16, 16) || !aligned(rope, 16) || !aligned(positions, 4))
    return fail(MIXLLM_ERR_INVALID_ARG, "k, v, q, q_out and rope must be 16-byte aligned, slots 8, positions 4");
  if (k_stride % 8 != 0 || v_stride % 8 != 0 || (q_heads > 0 && (q_stride % 8 != 0 || q_out_stride % 8 != 0)))
    return fail(MIXLLM_ERR_INVALID_ARG, "token strides must be multiples of 8 elements");
  if (n_slots > 1 && q_heads > 0 && q_out_stride < static_cast<int64_t>(q_heads) * head_dim)
    return fail(MIXLLM_ERR_INVALID_ARG, "rows of q_out overlap");
  st = check_device();
  if (st != MIXLLM_OK) return st;
  mixllm::AppendArgs a{cache,
                       n_slots,
                       slots,
                       static_cast<const __half *>(k_f16),
                       static_cast<const __half *>(v_f16),
                       static_cast<const __half *>(q_f16),
                       k_stride,
                       v_stride,
                       q_stride,
                       q_heads,
                       static_cast<__half *>(q_out_f16),
                       q_out_stride,
                       max_pos > 0 ? positions : nullptr,  // (a rotation has them)
                       rotary > 0 ? rope : nullptr,
                       max_pos,
                       rotary};
  cudaError_t e = mixllm::launch_kv4_append(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv4_append launch");
  return ok();
}

mixllm_status mixllm_kv4_read(const uint8_t *codes, const uint32_t *meta, int64_t pages, int32_t kv_heads,
                              int32_t head_dim, int32_t page_size, const int64_t *slots, int64_t n_slots,
                              void *k_f16, void *v_f16, void *stream) {
  mixllm::Kv4Cache cache;
  mixllm_status st = check_kv4(const_cast<uint8_t *>(codes), const_cast<uint32_t *>(meta), pages, kv_heads, head_dim,
                               page_size, &cache);
  if (st != MIXLLM_OK) return st;
  if (n_slots < 0 || n_slots > 0x7FFFFFFF) return fail(MIXLLM_ERR_INVALID_ARG, "bad number of tokens");
  if (n_slots == 0) return ok();
  if (!slots || !k_f16 || !v_f16) return fail(MIXLLM_ERR_INVALID_ARG, "null slots, k or v");
  if (!aligned(slots, 8) || !aligned(k_f16, 16) || !aligned(v_f16, 16))
    return fail(MIXLLM_ERR_INVALID_ARG, "k and v must be 16-byte aligned, slots 8");
  st = check_device();
  if (st != MIXLLM_OK) return st;
  cudaError_t e = mixllm::launch_kv4_read(cache, slots, n_slots, k_f16, v_f16, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv4_read launch");
  return ok();
}

mixllm_status mixllm_kv4_attention_workspace_bytes(int64_t requests, int64_t max_q, int32_t q_heads, int32_t kv_heads,
                                                   int32_t head_dim, int32_t page_size, int64_t table_width,
                                                   size_t *bytes) {
  if (!bytes) return fail(MIXLLM_ERR_INVALID_ARG, "null bytes");
  mixllm::Kv4Cache cache;
  mixllm_status st = check_kv4(nullptr, nullptr, 0, kv_heads, head_dim, page_size, &cache);
  if (st == MIXLLM_OK) st = check_kv_heads(requests, max_q, q_heads, table_width, cache.H, cache.page_log2);
  if (st != MIXLLM_OK) return st;
  *bytes = mixllm::kv4_attention_workspace_bytes(static_cast<int>(requests), static_cast<int>(max_q), q_heads,
                                                 kv_heads, head_dim);
  return ok();
}

mixllm_status mixllm_kv4_attention(const void *q_f16, int64_t q_stride, int64_t n_tokens, int32_t q_heads,
                                   const uint8_t *codes, const uint32_t *meta, int64_t pages, int32_t kv_heads,
                                   int32_t head_dim, int32_t page_size, const int32_t *block_table,
                                   int64_t table_stride, int64_t table_width, const int32_t *seq_lens,
                                   const int32_t *cu_q, int64_t requests, int64_t max_q, float scale, int32_t causal,
                                   void *out_f16, int64_t out_stride, float *lse, void *workspace,
                                   size_t workspace_bytes, void *stream) {
  mixllm::Kv4Cache cache;
  mixllm_status st = check_kv4(const_cast<uint8_t *>(codes), const_cast<uint32_t *>(meta), pages, kv_heads, head_dim,
                               page_size, &cache);
  if (st == MIXLLM_OK) st = check_kv_heads(requests, max_q, q_heads, table_width, cache.H, cache.page_log2);
  if (st != MIXLLM_OK) return st;
  const size_t need = mixllm::kv4_attention_workspace_bytes(static_cast<int>(requests), static_cast<int>(max_q),
                                                            q_heads, kv_heads, head_dim);
  return attend(cache, q_f16, q_stride, n_tokens, q_heads, block_table, table_stride, table_width, seq_lens, cu_q,
                requests, max_q, scale, causal, out_f16, out_stride, lse, workspace, workspace_bytes, need,
                mixllm::launch_kv4_attention, stream);
}

mixllm_status mixllm_w8a8_pack(const float *W, int64_t N, int64_t K, int8_t *codes, float *s_w, void *stream) {
  mixllm_status st = check_w8a8(N, K, "N");
  if (st != MIXLLM_OK) return st;
  if (N == 0) return ok();
  if (!W || !codes || !s_w) return fail(MIXLLM_ERR_INVALID_ARG, "null pointer");
  if (!aligned(W, 16) || !aligned(codes, 16) || !aligned(s_w, 4))
    return fail(MIXLLM_ERR_INVALID_ARG, "W and codes must be 16-byte aligned, s_w 4");
  st = check_device();
  if (st != MIXLLM_OK) return st;
  cudaError_t e = mixllm::launch_w8a8_pack(W, N, K, codes, s_w, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "w8a8_pack launch");
  return ok();
}

mixllm_status mixllm_w8a8_quantize(const void *X_f16, int64_t x_stride, int64_t M, int64_t K, int8_t *A_q, float *s_a,
                                   void *stream) {
  mixllm_status st = check_w8a8(M, K, "M");
  if (st != MIXLLM_OK) return st;
  if (M == 0) return ok();
  if (!A_q || !s_a) return fail(MIXLLM_ERR_INVALID_ARG, "null pointer");
  st = check_heads("X", X_f16, x_stride, M, K, false);
  if (st != MIXLLM_OK) return st;
  if (!aligned(A_q, 16) || !aligned(s_a, 4)) return fail(MIXLLM_ERR_INVALID_ARG, "A_q must be 16-byte aligned, s_a 4");
  st = check_device();
  if (st != MIXLLM_OK) return st;
  cudaError_t e = mixllm::launch_w8a8_quantize(static_cast<const __half *>(X_f16), x_stride, M, K, A_q, s_a,
                                               static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "w8a8_quantize launch");
  return ok();
}

mixllm_status mixllm_w8a8_linear_workspace_bytes(int64_t M, int64_t K, int64_t N, size_t *bytes) {
  if (!bytes) return fail(MIXLLM_ERR_INVALID_ARG, "null bytes");
  mixllm_status st = check_w8a8(M, K, "M");
  if (st == MIXLLM_OK) st = check_w8a8(N, K, "N");
  if (st != MIXLLM_OK) return st;
  *bytes = mixllm::w8a8_linear_workspace_bytes(M, N, K);
  return ok();
}

mixllm_status mixllm_w8a8_gemm(const int8_t *A_q, const float *s_a, int64_t M, int64_t K, const int8_t *W,
                               const float *s_w, int64_t N, const void *bias_f16, void *Y_f16, void *stream) {
  bool empty = false;
  mixllm_status st = check_w8a8_product(M, K, W, s_w, N, bias_f16, Y_f16, &empty);
  if (st != MIXLLM_OK) return st;
  if (empty) return ok();
  if (!A_q || !s_a) return fail(MIXLLM_ERR_INVALID_ARG, "null A_q or s_a");
  if (!aligned(A_q, 16) || !aligned(s_a, 4)) return fail(MIXLLM_ERR_INVALID_ARG, "A_q must be 16-byte aligned, s_a 4");
  st = check_device();
  if (st != MIXLLM_OK) return st;
  const mixllm::W8A8Args a{A_q, s_a, W, s_w, static_cast<const __half *>(bias_f16), static_cast<__half *>(Y_f16), M, N, K};
  const char *msg = "";
  const cudaError_t e = mixllm::launch_w8a8_gemm(a, static_cast<cudaStream_t>(stream), &msg);
  return w8a8_done(e, msg);
}

mixllm_status mixllm_w8a8_linear(const void *X_f16, int64_t x_stride, int64_t M, int64_t K, const int8_t *W,
                                 const float *s_w, int64_t N, const void *bias_f16, void *Y_f16, void *workspace,
                                 size_t workspace_bytes, void *stream) {
  bool empty = false;
  mixllm_status st = check_w8a8_product(M, K, W, s_w, N, bias_f16, Y_f16, &empty);
  if (st != MIXLLM_OK) return st;
  if (empty) return ok();
  const size_t need = mixllm::w8a8_linear_workspace_bytes(M, N, K);
  if (workspace_bytes < need)
    return fail(MIXLLM_ERR_INVALID_ARG, "workspace of %zu bytes is smaller than the %zu this shape needs",
                workspace_bytes, need);
  if (!workspace || !aligned(workspace, 256))
    return fail(MIXLLM_ERR_INVALID_ARG, "workspace must be a 256-byte aligned device buffer");
  st = check_heads("X", X_f16, x_stride, M, K, false);
  if (st == MIXLLM_OK) st = check_device();
  if (st != MIXLLM_OK) return st;
  const mixllm::W8A8Args a{nullptr, nullptr, W, s_w, static_cast<const __half *>(bias_f16), static_cast<__half *>(Y_f16),
                           M, N, K};
  const char *msg = "";
  const cudaError_t e = mixllm::launch_w8a8_linear(static_cast<const __half *>(X_f16), x_stride, a, workspace,
                                                   static_cast<cudaStream_t>(stream), &msg);
  return w8a8_done(e, msg);
}

mixllm_status mixllm_head_norm_rope(const void *q_f16, int64_t q_stride, int32_t q_heads, void *q_out_f16,
                                    int64_t q_out_stride, const void *w_q_f16, const void *k_f16, int64_t k_stride,
                                    int32_t kv_heads, void *k_out_f16, int64_t k_out_stride, const void *w_k_f16,
                                    int64_t n_tokens, int32_t head_dim, float eps, const int32_t *positions,
                                    const float *rope, int64_t max_pos, int32_t rotary, void *stream) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(MIXLLM_ERR_UNSUPPORTED, "head size %d is not 64, 128 or 256", head_dim);
  if (kv_heads < 0 || kv_heads > 65536) return fail(MIXLLM_ERR_INVALID_ARG, "%d key heads", kv_heads);
  mixllm_status st = check_turn(n_tokens, q_heads, head_dim, w_q_f16, w_k_f16, eps, positions, rope, max_pos, rotary);
  if (st != MIXLLM_OK) return st;
  if (n_tokens == 0 || (q_heads == 0 && kv_heads == 0)) return ok();
  const int64_t q_row = static_cast<int64_t>(q_heads) * head_dim, k_row = static_cast<int64_t>(kv_heads) * head_dim;
  if (q_heads > 0) st = check_heads("q", q_f16, q_stride, n_tokens, q_row, false);
  if (st == MIXLLM_OK && q_heads > 0) st = check_heads("q_out", q_out_f16, q_out_stride, n_tokens, q_row, true);
  if (st == MIXLLM_OK && kv_heads > 0) st = check_heads("k", k_f16, k_stride, n_tokens, k_row, false);
  if (st == MIXLLM_OK && kv_heads > 0) st = check_heads("k_out", k_out_f16, k_out_stride, n_tokens, k_row, true);
  if (st == MIXLLM_OK) st = check_device();
  if (st != MIXLLM_OK) return st;
  mixllm::HeadArgs a{};
  a.T = n_tokens;
  a.q = static_cast<const __half *>(q_f16), a.k = static_cast<const __half *>(k_f16);
  a.q_stride = q_stride, a.k_stride = k_stride;
  a.Hq = q_heads, a.H = kv_heads;
  a.q_out = static_cast<__half *>(q_out_f16), a.k_out = static_cast<__half *>(k_out_f16);
  a.q_out_stride = q_out_stride, a.k_out_stride = k_out_stride;
  a.w_q = static_cast<const __half *>(w_q_f16), a.w_k = static_cast<const __half *>(w_k_f16);
  a.positions = positions, a.rope = rotary > 0 ? rope : nullptr;
  a.max_pos = max_pos, a.rotary = rotary, a.eps = eps;
  cudaError_t e = mixllm::launch_head_norm_rope(a, head_dim, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "head_norm_rope launch");
  return ok();
}

mixllm_status mixllm_kv8_append(uint8_t *codes, float *scales, int64_t pages, int32_t kv_heads, int32_t head_dim,
                                int32_t page_size, const int64_t *slots, int64_t n_slots, const void *k_f16,
                                int64_t k_stride, const void *v_f16, int64_t v_stride, const void *q_f16,
                                int64_t q_stride, int32_t q_heads, void *q_out_f16, int64_t q_out_stride,
                                const void *w_q_f16, const void *w_k_f16, float eps, const int32_t *positions,
                                const float *rope, int64_t max_pos, int32_t rotary, void *stream) {
  mixllm::Kv8AppendArgs a{};
  mixllm_status st = check_cache(codes, scales, pages, kv_heads, head_dim, page_size, &a.cache);
  if (st == MIXLLM_OK)
    st = check_turn(n_slots, q_heads, head_dim, w_q_f16, w_k_f16, eps, positions, rope, max_pos, rotary);
  if (st != MIXLLM_OK) return st;
  if (n_slots == 0) return ok();
  if (!slots || !aligned(slots, 8)) return fail(MIXLLM_ERR_INVALID_ARG, "slots must be an 8-byte aligned device buffer");
  const int64_t q_row = static_cast<int64_t>(q_heads) * head_dim, k_row = static_cast<int64_t>(kv_heads) * head_dim;
  st = check_heads("k", k_f16, k_stride, n_slots, k_row, false);
  if (st == MIXLLM_OK) st = check_heads("v", v_f16, v_stride, n_slots, k_row, false);
  if (st == MIXLLM_OK && q_heads > 0) st = check_heads("q", q_f16, q_stride, n_slots, q_row, false);
  if (st == MIXLLM_OK && q_heads > 0) st = check_heads("q_out", q_out_f16, q_out_stride, n_slots, q_row, true);
  if (st == MIXLLM_OK) st = check_device();
  if (st != MIXLLM_OK) return st;
  a.slots = slots;
  mixllm::HeadArgs heads{};
  heads.T = n_slots;
  heads.q = static_cast<const __half *>(q_f16), heads.k = static_cast<const __half *>(k_f16);
  heads.v = static_cast<const __half *>(v_f16);
  heads.q_stride = q_stride, heads.k_stride = k_stride, heads.v_stride = v_stride;
  heads.Hq = q_heads, heads.H = kv_heads;
  heads.q_out = static_cast<__half *>(q_out_f16), heads.q_out_stride = q_out_stride;
  heads.w_q = static_cast<const __half *>(w_q_f16), heads.w_k = static_cast<const __half *>(w_k_f16);
  heads.positions = positions, heads.rope = rotary > 0 ? rope : nullptr;
  heads.max_pos = max_pos, heads.rotary = rotary, heads.eps = eps;
  cudaError_t e = mixllm::launch_kv8_append(a, heads, static_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported) return fail(MIXLLM_ERR_UNSUPPORTED, "more than 2^31 blocks of tokens and heads");
  if (e != cudaSuccess) return cuda_fail(e, "kv8_append launch");
  return ok();
}

mixllm_status mixllm_kv8_read(const uint8_t *codes, const float *scales, int64_t pages, int32_t kv_heads,
                              int32_t head_dim, int32_t page_size, const int64_t *slots, int64_t n_slots, void *k_f16,
                              void *v_f16, void *stream) {
  mixllm::Kv8Cache cache;
  mixllm_status st = check_cache(const_cast<uint8_t *>(codes), const_cast<float *>(scales), pages, kv_heads, head_dim,
                                 page_size, &cache);
  if (st != MIXLLM_OK) return st;
  if (n_slots < 0 || n_slots > 0x7FFFFFFF) return fail(MIXLLM_ERR_INVALID_ARG, "bad number of tokens");
  if (n_slots == 0) return ok();
  if (!slots || !k_f16 || !v_f16) return fail(MIXLLM_ERR_INVALID_ARG, "null slots, k or v");
  if (!aligned(slots, 8) || !aligned(k_f16, 16) || !aligned(v_f16, 16))
    return fail(MIXLLM_ERR_INVALID_ARG, "k and v must be 16-byte aligned, slots 8");
  st = check_device();
  if (st != MIXLLM_OK) return st;
  cudaError_t e = mixllm::launch_kv8_read(cache, slots, n_slots, k_f16, v_f16, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "kv8_read launch");
  return ok();
}

mixllm_status mixllm_kv8_attention_workspace_bytes(int64_t requests, int64_t max_q, int32_t q_heads, int32_t kv_heads,
                                                   int32_t head_dim, int32_t page_size, int64_t table_width,
                                                   size_t *bytes) {
  if (!bytes) return fail(MIXLLM_ERR_INVALID_ARG, "null bytes");
  mixllm::Kv8Cache cache;
  mixllm_status st = check_cache<mixllm::Kv8Cache, float>(nullptr, nullptr, 0, kv_heads, head_dim, page_size, &cache);
  if (st == MIXLLM_OK) st = check_kv_heads(requests, max_q, q_heads, table_width, cache.H, cache.page_log2);
  if (st != MIXLLM_OK) return st;
  *bytes = mixllm::kv8_attention_workspace_bytes(static_cast<int>(requests), static_cast<int>(max_q), q_heads, kv_heads,
                                                 head_dim);
  return ok();
}

mixllm_status mixllm_kv8_attention(const void *q_f16, int64_t q_stride, int64_t n_tokens, int32_t q_heads,
                                   const uint8_t *codes, const float *scales, int64_t pages, int32_t kv_heads,
                                   int32_t head_dim, int32_t page_size, const int32_t *block_table,
                                   int64_t table_stride, int64_t table_width, const int32_t *seq_lens,
                                   const int32_t *cu_q, int64_t requests, int64_t max_q, float scale, int32_t causal,
                                   void *out_f16, int64_t out_stride, float *lse, void *workspace,
                                   size_t workspace_bytes, void *stream) {
  mixllm::Kv8Cache cache;
  mixllm_status st = check_cache(const_cast<uint8_t *>(codes), const_cast<float *>(scales), pages, kv_heads, head_dim,
                                 page_size, &cache);
  if (st == MIXLLM_OK) st = check_kv_heads(requests, max_q, q_heads, table_width, cache.H, cache.page_log2);
  if (st != MIXLLM_OK) return st;
  const size_t need = mixllm::kv8_attention_workspace_bytes(static_cast<int>(requests), static_cast<int>(max_q),
                                                            q_heads, kv_heads, head_dim);
  return attend(cache, q_f16, q_stride, n_tokens, q_heads, block_table, table_stride, table_width, seq_lens, cu_q,
                requests, max_q, scale, causal, out_f16, out_stride, lse, workspace, workspace_bytes, need,
                mixllm::launch_kv8_attention, stream);
}

mixllm_status mixllm_sync_status(void *stream) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "stream synchronize");
  int status = 0;
  e = cudaMemcpyFromSymbol(&status, mixllm::g_status, sizeof(int));
  if (e != cudaSuccess) return cuda_fail(e, "status read");
  if (status != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(mixllm::g_status, &zero, sizeof(int));
    if (e != cudaSuccess) return cuda_fail(e, "status clear");
    if (status == mixllm::kStatusTimeout) return fail(MIXLLM_ERR_TIMEOUT, "a device-side wait gave up");
    if (status == mixllm::kStatusBounds)
      return fail(MIXLLM_ERR_BOUNDS,
                  "a KV-cache kernel met a page, slot, position or length out of range, or a range check of the "
                  "checked build failed (the access was skipped)");
    return fail(MIXLLM_ERR_INVALID_ARG, "device reported status %d", status);
  }
  return ok();
}

int mixllm_checked_build(void) { return MIXLLM_CHECKED ? 1 : 0; }

mixllm_status mixllm_selftest_bounds(void *stream) {
  if (!MIXLLM_CHECKED) return fail(MIXLLM_ERR_UNSUPPORTED, "the release build has no range checks");
  mixllm_status st = check_device();
  if (st != MIXLLM_OK) return st;
  cudaError_t e = mixllm::launch_selftest_bounds(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "selftest launch");
  return ok();
}

mixllm_status mixllm_selftest_wait_timeout(uint32_t limit_us, void *stream) {
  if (limit_us < 1 || limit_us > 1000000) return fail(MIXLLM_ERR_INVALID_ARG, "limit_us must be in 1..1000000");
  mixllm_status st = check_device();
  if (st != MIXLLM_OK) return st;
  cudaError_t e = mixllm::launch_selftest_wait_timeout(limit_us, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "selftest launch");
  return ok();
}

}  // extern "C"
