// launch.h -- host-side launchers of the library's kernels (internal).
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace mixllm {

cudaError_t launch_quantize_act(const void *X, int64_t M, int64_t K, int8_t *A_q, float *s_a,
                                cudaStream_t stream);

cudaError_t launch_split_channels(const uint8_t *is8, int64_t N, int64_t N8, int32_t *idx4, int32_t *idx8,
                                  cudaStream_t stream);

cudaError_t launch_pack_w4(const float *W, int64_t N, int64_t K, const int32_t *idx4, int64_t N4, int64_t N4p,
                           uint8_t *W4, uint8_t *z4, void *s_w4, cudaStream_t stream);

cudaError_t launch_pack_w8(const float *W, int64_t N, int64_t K, const int32_t *idx8, int64_t N8, int64_t N8p,
                           int8_t *W8, void *s_w8, cudaStream_t stream);

struct GemmArgs {
  const int8_t *A_q;
  const float *s_a;
  int64_t M, K;
  const uint8_t *W4;
  const uint8_t *z4;
  const void *s_w4;
  const int32_t *idx4;
  int64_t N4;
  const int8_t *W8;
  const void *s_w8;
  const int32_t *idx8;
  int64_t N8;
  void *Y;     // fp16 [M, N4 + N8]
  int32_t *P;  // debug partials [M, N, G] or null
  const void *X = nullptr;  // fp16 [M, K] activations: the fused few-token path quantizes them itself
  bool cvt_i2f = false;     // tiled GEMM only: plain int -> float convert instead of the bias trick (measurement)
  uint32_t *qcnt = nullptr; // fused tiled layer: two counters in the workspace (pairs quantized, CTAs done)
};

// Returns a CUDA error, or cudaErrorNotSupported when the tensor-map encoder
// is unavailable.  *msg receives a static description on failure.
cudaError_t launch_gemm_w4w8a8(const GemmArgs &a, cudaStream_t stream, const char **msg);

// The tiled layer from fp16 X (M > 64) into a.A_q / a.s_a (workspace): the
// quantizer, then the GEMM; or (one_launch) the GEMM quantizing the
// activations itself and publishing them through a.qcnt (two counters, zero
// before the call and again after it; cudaErrorNotSupported for shapes that
// form does not take).
bool linear_tiled_fuses(int64_t M, int64_t K);
cudaError_t launch_linear_tiled(const GemmArgs &a, bool one_launch, cudaStream_t stream, const char **msg);
// Any M: the few-token layer (launch_linear_small_m) for M <= 64, else the
// tiled one, each with its workspace layout (linear_workspace_bytes()).
size_t linear_workspace_bytes(int64_t M, int64_t N4, int64_t N8, int64_t K);
cudaError_t launch_linear(const GemmArgs &a, void *ws, size_t ws_bytes, bool one_launch, cudaStream_t stream,
                          const char **msg);

// Few-token variant (M <= 64): split-K over the groups with a workspace of
// small_m_workspace_bytes() bytes: fp32 partial sums, then one int32 counter
// per tile (zero before the first call; every call returns them to zero).
// Y only (the debug partials: launch_small_m_debug_partials).
cudaError_t launch_gemm_small_m(const GemmArgs &a, void *ws, size_t ws_bytes, cudaStream_t stream, const char **msg);
size_t small_m_workspace_bytes(int64_t M, int64_t N4, int64_t N8, int64_t K);
// 0: tensor-core kernel, 1: split GEMV, 2: persistent GEMV (mixllm_small_m_kind)
int small_m_kernel_kind(int64_t M, int64_t N4, int64_t N8, int64_t K);
// Debug form of one named few-token kernel (kind as above, whatever the plan
// would pick): Y, and the int32 group partials into a.P [M, N, G].
bool small_m_kernel_allowed(int64_t M, int64_t N4, int64_t N8, int64_t K, int kind);
size_t small_m_debug_workspace_bytes(int64_t M, int64_t N4, int64_t N8, int64_t K, int kind);
cudaError_t launch_small_m_debug_partials(const GemmArgs &a, int kind, void *ws, size_t ws_bytes,
                                          cudaStream_t stream, const char **msg);
// The few-token layer from fp16 X (quantization included): the split GEMV
// quantizes in its prologue when its slice of X fits a ring slot; otherwise
// the quantizer writes A_q / s_a into the workspace first.  a.X is required,
// a.A_q / a.s_a are ignored.  Workspace: linear_small_m_workspace_bytes().
size_t linear_small_m_workspace_bytes(int64_t M, int64_t N4, int64_t N8, int64_t K);
bool linear_small_m_fused(int64_t M, int64_t N4, int64_t N8, int64_t K);
cudaError_t launch_linear_small_m(const GemmArgs &a, void *ws, size_t ws_bytes, cudaStream_t stream,
                                  const char **msg);
// The same with a static device scratch instead of a workspace (no allocation);
// fails with cudaErrorInvalidValue when the shape needs more than it holds.
cudaError_t launch_gemm_small_m_noalloc(const GemmArgs &a, cudaStream_t stream, const char **msg);
size_t small_m_scratch_capacity();

cudaError_t launch_selftest_wait_timeout(uint32_t limit_us, cudaStream_t stream);
cudaError_t launch_selftest_bounds(cudaStream_t stream);

// Global mixed-precision search (search.cuh).
cudaError_t launch_channel_salience(const float *W, int64_t N, int64_t K, const float *G, int64_t D, float *S,
                                    cudaStream_t stream, const char **msg);
size_t select_top_t_workspace_bytes(int64_t n);
cudaError_t launch_select_top_t(const float *S, int64_t n, int64_t T, uint8_t *is8, void *ws, cudaStream_t stream,
                                const char **msg);

// The norms around a block (norm.cuh).
struct NormArgs {
  int64_t M, K;
  const __half *x;  // the block's output, or null: r is only normalized
  int64_t x_stride;
  const __half *w_post;  // the norm after the block, or null
  const __half *gate;    // or null; gate_stride 0: one row for all tokens
  int64_t gate_stride;
  float scale;
  const void *r;  // the residual stream, fp16 or fp32
  int64_t r_stride;
  bool r_fp32;
  void *r_out;  // or null
  int64_t r_out_stride;
  const __half *w;
  float eps;
  __half *y;   // fp16 [M, K], or null
  int8_t *A_q;  // codes and scales of y, or null
  float *s_a;
};
cudaError_t launch_residual_norm(const NormArgs &a, cudaStream_t stream);
cudaError_t launch_dequantize_act(const int8_t *A_q, const float *s_a, int64_t M, int64_t K, void *X,
                                  cudaStream_t stream);

// The paged 4-bit KV cache (kv4_cache.cuh) and the attention over it
// (kv4_attention.cuh).
constexpr int kKv4MaxRequests = 16384;

struct Kv4Cache {
  uint8_t *codes;
  uint32_t *meta;
  int64_t pages;
  int H, D, page_log2;
};

struct AssignArgs {
  const int32_t *ctx_lens, *new_lens;
  int B;
  int32_t *table;
  int64_t table_stride;
  int W;
  const int32_t *free_pages;
  int n_free;
  const int32_t *count;
  int page_log2;
  int32_t *seq_lens, *cu_new;
  int64_t *slots;
  int32_t *positions;
  int64_t T;
  int32_t *left, *status;
};
cudaError_t launch_kv4_assign(const AssignArgs &a, cudaStream_t stream, const char **msg);

struct AppendArgs {
  Kv4Cache cache;
  int64_t T;
  const int64_t *slots;
  const __half *k, *v, *q;  // q or null (Hq = 0)
  int64_t k_stride, v_stride, q_stride;
  int Hq;
  __half *q_out;
  int64_t q_out_stride;
  const int32_t *positions;
  const float *rope;  // [max_pos][rotary]: cosines, then sines; or null
  int64_t max_pos;
  int rotary;
};
cudaError_t launch_kv4_append(const AppendArgs &a, cudaStream_t stream);
cudaError_t launch_kv4_read(const Kv4Cache &c, const int64_t *slots, int64_t T, void *k, void *v,
                            cudaStream_t stream);

struct AttendArgs {
  Kv4Cache cache;
  const __half *q;
  int64_t q_stride, T;
  int Hq, B, max_q;
  const int32_t *table;
  int64_t table_stride;
  int W;
  const int32_t *kv_lens, *cu_q;
  float scale;
  int causal;
  __half *out;
  int64_t out_stride;
  float *lse;  // [T][Hq], or null
};
size_t kv4_attention_workspace_bytes(int B, int max_q, int Hq, int H, int D);
cudaError_t launch_kv4_attention(const AttendArgs &a, void *ws, cudaStream_t stream, const char **msg);

int64_t padded_channels(int64_t n);  // n rounded up to a multiple of 256

}  // namespace mixllm
