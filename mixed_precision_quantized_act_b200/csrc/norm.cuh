// norm.cuh -- the norms around a block: the norm after it with its gate and
// residual scale, the residual update, and the norm before the next linear,
// in one pass, with that linear's int8 codes as output where wanted; and the
// codes' way back to fp16.
#pragma once

#include <cuda_fp16.h>
#include <cstdint>

#include "launch.h"
#include "ptx_sm100.cuh"
#include "quant.cuh"

namespace mixllm {

// Sum of v over the block, on every thread.  Fixed order: the result does not
// depend on timing.  `part` holds one float per warp.
__device__ __forceinline__ float block_sum(float v, float *part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  v = lane < warps ? part[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

__device__ __forceinline__ void load8(const __half *p, float (&f)[8]) {
  const uint4 raw = *reinterpret_cast<const uint4 *>(p);
  const __half2 *h = reinterpret_cast<const __half2 *>(&raw);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(h[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint4 raw;
  __half2 *h = reinterpret_cast<__half2 *>(&raw);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
  return raw;
}
// Stores f rounded to the residual stream's type and leaves the rounded
// values in f: the norm that follows sees what is stored.
__device__ __forceinline__ void store8_rounded(__half *p, float (&f)[8]) {
  const uint4 raw = pack8(f);
  if (p) *reinterpret_cast<uint4 *>(p) = raw;
  const __half2 *h = reinterpret_cast<const __half2 *>(&raw);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(h[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
__device__ __forceinline__ void store8_rounded(float *p, float (&f)[8]) {
  if (!p) return;
  *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

// ---------------------------------------------------------------------------
// One block per token; a thread holds V runs of eight channels, 8 * blockDim
// apart, in fp32 registers, so each input is read once:
//   u  = x, or x * rsqrt(mean(x^2) + eps) * w_post
//   r' = r + scale * gate * u, rounded to the residual stream's type
//   y  = r' * rsqrt(mean(r'^2) + eps) * w, rounded to fp16 (the activations'
//        type, so the codes below are those of quantizing y in a pass of its own)
//   and, where A_q is given, y's int8 codes and scales per 128 channels.
// The sums of squares are held in fp32: a thread adds at most 8 V squares and
// the block adds the threads' sums as a tree.  Without x, r' = r.
// HBM-bound: 2 + 2 |r| bytes a channel and 2 (y), 1 (codes) or both out; with an
// fp32 residual, a gate and both norms, 1024 x 8192 took 20.6 us, 4.9 TB/s on
// B200 (75 % of the measured copy rate): two blocks of 512 threads fit an SM, and a
// row's loads, its two block-wide sums and its stores come one after the other.
// Threads hold one run up to 4096
// channels and two up to 16384, which keeps every load of a row in registers.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void widen8(const uint4 raw, float (&f)[8]) {
  const __half2 *h = reinterpret_cast<const __half2 *>(&raw);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(h[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

template <typename R, int V>
__global__ void __launch_bounds__(V == 1 ? 512 : 1024) residual_norm_kernel(const NormArgs a) {
  __shared__ float part[2][32];
  const int64_t m = blockIdx.x;
  const int K = static_cast<int>(a.K);
  const int step = blockDim.x * 8;
  // every load of the row is issued before the first sum, as far as the registers go
  constexpr bool kAhead = V < 4;
  float r[V][8];
  uint4 x[V], gate[V], w_post[V], w[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int k = threadIdx.x * 8 + v * step;
    if (k < K) {
      if (a.x) x[v] = *reinterpret_cast<const uint4 *>(a.x + m * a.x_stride + k);
      load8(static_cast<const R *>(a.r) + m * a.r_stride + k, r[v]);
      if constexpr (kAhead) {
        if (a.gate) gate[v] = *reinterpret_cast<const uint4 *>(a.gate + m * a.gate_stride + k);
        if (a.w_post) w_post[v] = *reinterpret_cast<const uint4 *>(a.w_post + k);
        w[v] = *reinterpret_cast<const uint4 *>(a.w + k);
      }
    } else {
      x[v] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[v][i] = 0.0f;
    }
  }
  if (a.x) {
    float inv = 1.0f;
    if (a.w_post) {
      float ss = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float u[8];
        widen8(x[v], u);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(u[i], u[i], ss);
      }
      inv = rsqrtf(block_sum(ss, part[0]) / static_cast<float>(K) + a.eps);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int k = threadIdx.x * 8 + v * step;
      if (k >= K) continue;
      float u[8], f[8];
      widen8(x[v], u);
      if (a.w_post) {
        widen8(kAhead ? w_post[v] : *reinterpret_cast<const uint4 *>(a.w_post + k), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = u[i] * inv * f[i];
      }
      if (a.gate) {
        widen8(kAhead ? gate[v] : *reinterpret_cast<const uint4 *>(a.gate + m * a.gate_stride + k), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] *= f[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) r[v][i] = fmaf(a.scale, u[i], r[v][i]);
      store8_rounded(a.r_out ? static_cast<R *>(a.r_out) + m * a.r_out_stride + k : static_cast<R *>(nullptr), r[v]);
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(r[v][i], r[v][i], ss);
  const float inv = rsqrtf(block_sum(ss, part[1]) / static_cast<float>(K) + a.eps);
  const unsigned mask = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int k = threadIdx.x * 8 + v * step;
    if (k >= K) continue;  // 16 lanes together: K and the runs of 16 lanes are multiples of 128 channels
    float f[8];
    widen8(kAhead ? w[v] : *reinterpret_cast<const uint4 *>(a.w + k), f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = r[v][i] * inv * f[i];
    const uint4 y = pack8(f);
    if (a.y) *reinterpret_cast<uint4 *>(a.y + m * a.K + k) = y;
    if (a.A_q) {
      uint32_t packed[2];
      const float s = quant_act_8x16(y, mask, packed);
      *reinterpret_cast<uint2 *>(a.A_q + m * a.K + k) = make_uint2(packed[0], packed[1]);
      if ((threadIdx.x & 15) == 0) a.s_a[m * (a.K >> 7) + (k >> 7)] = s;
    }
  }
}

// X = fp16(A_q * s_a): what the GEMM takes the activations to be.  One thread
// per eight codes.
__global__ void __launch_bounds__(256) dequantize_act_kernel(const int8_t *__restrict__ A_q,
                                                             const float *__restrict__ s_a, int64_t runs,
                                                             __half *__restrict__ X) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < runs; i += stride) {
    const uint2 raw = *reinterpret_cast<const uint2 *>(A_q + i * 8);
    const float s = s_a[i >> 4];
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      f[j] = static_cast<float>(static_cast<int8_t>((j < 4 ? raw.x : raw.y) >> (8 * (j & 3)))) * s;
    *reinterpret_cast<uint4 *>(X + i * 8) = pack8(f);
  }
}

template <typename R>
static void launch_residual_norm_type(const NormArgs &a, cudaStream_t stream) {
  const int64_t runs = a.K / 8;
  const unsigned M = static_cast<unsigned>(a.M);
  auto threads = [&](int v) { return static_cast<unsigned>(((runs + v - 1) / v + 31) / 32 * 32); };
  if (runs <= 512) residual_norm_kernel<R, 1><<<M, threads(1), 0, stream>>>(a);
  else if (runs <= 2048) residual_norm_kernel<R, 2><<<M, threads(2), 0, stream>>>(a);
  else residual_norm_kernel<R, 4><<<M, threads(4), 0, stream>>>(a);
}

cudaError_t launch_residual_norm(const NormArgs &a, cudaStream_t stream) {
  if (a.r_fp32) launch_residual_norm_type<float>(a, stream);
  else launch_residual_norm_type<__half>(a, stream);
  return cudaGetLastError();
}

cudaError_t launch_dequantize_act(const int8_t *A_q, const float *s_a, int64_t M, int64_t K, void *X,
                                  cudaStream_t stream) {
  const int64_t runs = M * (K / 8);
  const int64_t blocks = (runs + 255) / 256;
  dequantize_act_kernel<<<static_cast<unsigned>(blocks < 148 * 64 ? blocks : 148 * 64), 256, 0, stream>>>(
      A_q, s_a, runs, static_cast<__half *>(X));
  return cudaGetLastError();
}

}  // namespace mixllm
