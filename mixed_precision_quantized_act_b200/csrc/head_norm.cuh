// head_norm.cuh -- the norms of query and key heads (one RMS norm per token and
// head, over the head's channels) and the rotation by position, in one pass.
#pragma once

#include <cuda_fp16.h>
#include <cstdint>

#include "gemm_w4w8a8.cuh"  // device_sm_count
#include "kv4_ptx.cuh"      // pairs of floats
#include "launch.h"
#include "norm.cuh"
#include "ptx_sm100.cuh"

namespace mixllm {

// ---------------------------------------------------------------------------
// A row (one head of one token, D channels) is held by D / 8 lanes, eight
// channels each:
//   y = x * rsqrt(mean(x^2) + eps) * w            (w null: y = x)
//   y_i cos_i - y_j sin_i,  y_j cos_i + y_i sin_i   for j = i + rotary/2
// in fp32, rounded to fp16 once.  The weight goes into the rotation's
// factors, which all heads of a token share, and the norm's own factor comes off
// the sum: inv * (x own + x_far far).  Without weights inv = 1 and own, far are
// the cosine and the signed sine: every product and sum rounded on its own, the
// bits of the 4-bit cache's rotation.
//
// HBM-bound: 4 bytes a channel, and the table's 8 bytes a channel of a token once
// for sixteen heads.  4099 tokens of 64 + 8 heads of 128, half of their channels
// rotated: 29.2 us on B200, 5.2 TB/s (80 % of the measured copy rate).  With floats one
// by one and a way of their own for the lanes that are not rotated, 143 instructions
// a warp and row kept the issue slots 71 % busy, and it took 30.9.  40 warps an SM
// instead of 32 take 37 us (48 registers), 24 take 33, six heads ahead 31.8.
// ---------------------------------------------------------------------------
// kNorm: 0 and 1 where the compiler may know whether there is a norm, 2 where `w` says.
template <int D, int kNorm = 2>
struct HeadTurn {
  static constexpr int kLanes = D / 8;
  uint64_t own[4], far[4];  // of pairs of this lane's channels; far is -0 for channels that are not rotated
  int other;                // lane of the row that holds the channels paired with this one's
  bool norm, any, turned;   // turned: this lane's channels are rotated; any: some lane's are
  unsigned mask;

  // `angle`: the position's rotary/2 cosines, then its sines, or null; `w`: fp16 [D], or null
  __device__ __forceinline__ void start(const float *angle, int rotary, const __half *w) {
    const int sub = threadIdx.x % kLanes, c0 = sub * 8, half = rotary / 2;  // half is a multiple of 8
    mask = (kLanes == 32 ? 0xFFFFFFFFu : ((1u << (kLanes & 31)) - 1u)) << (threadIdx.x & 31 & ~(kLanes - 1));
    const bool second = c0 >= half;
    norm = kNorm == 2 ? w != nullptr : kNorm == 1, any = angle != nullptr && half > 0, turned = any && c0 < rotary;
    other = second ? sub - half / 8 : sub + half / 8;
    float o[8], f[8], w8[8];
    if (turned) {
      const float *at = angle + (second ? c0 - half : c0);
      load8(at, o);
      load8(at + half, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = second ? f[j] : -f[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = 1.0f, f[j] = -0.0f;
    }
    if (norm) {
      load8(w + c0, w8);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] *= w8[j];
      if (turned) {
        load8(w + other * 8, w8);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= w8[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) own[j] = pack_f2(o[2 * j], o[2 * j + 1]), far[j] = pack_f2(f[2 * j], f[2 * j + 1]);
  }

  // All lanes of a row together.  Channels that are not rotated meet a far of -0 and a partner of +0: what they add is
  // -0, which changes no bit, and no lane goes a way of its own.
  __device__ __forceinline__ uint4 apply(const uint4 raw, float eps) const {
    if (!norm && !any) return raw;
    uint64_t x[4], y[4];
    widen_pairs(raw, x);
    if (any) {
      uint4 far_raw;
      far_raw.x = __shfl_sync(mask, raw.x, other, kLanes);
      far_raw.y = __shfl_sync(mask, raw.y, other, kLanes);
      far_raw.z = __shfl_sync(mask, raw.z, other, kLanes);
      far_raw.w = __shfl_sync(mask, raw.w, other, kLanes);
      widen_pairs(turned ? far_raw : make_uint4(0, 0, 0, 0), y);
    }
    float out[8];
    if (norm) {
      uint64_t ss2 = mul_f2(x[0], x[0]);
#pragma unroll
      for (int j = 1; j < 4; ++j) ss2 = fma_f2(x[j], x[j], ss2);
      const float2 s = unpack_f2(ss2);
      float ss = s.x + s.y;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
      const float inv = rsqrtf(fmaf(ss, 1.0f / D, eps));
      const uint64_t inv2 = pack_f2(inv, inv);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = mul_f2(x[j], own[j]);
        if (any) x[j] = fma_f2(y[j], far[j], x[j]);
        const float2 f = unpack_f2(mul_f2(x[j], inv2));
        out[2 * j] = f.x, out[2 * j + 1] = f.y;
      }
    } else {
      // one float at a time: ptxas joins a product and a sum of pairs
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 u = unpack_f2(x[j]), v = unpack_f2(y[j]), o = unpack_f2(own[j]), f = unpack_f2(far[j]);
        out[2 * j] = __fadd_rn(__fmul_rn(u.x, o.x), __fmul_rn(v.x, f.x));
        out[2 * j + 1] = __fadd_rn(__fmul_rn(u.y, o.y), __fmul_rn(v.y, f.y));
      }
    }
    return pack8(out);
  }
  static __device__ __forceinline__ void widen_pairs(const uint4 raw, uint64_t (&x)[4]) {
    const __half2 *h = reinterpret_cast<const __half2 *>(&raw);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(h[j]);
      x[j] = pack_f2(f.x, f.y);
    }
  }
};

// One block takes 256 / (D / 8) tokens and `per` heads of queries or of keys; a
// lane loads four heads ahead, the first ones before it knows its position.
constexpr int kHeadThreads = 256, kHeadsAhead = 4;

template <int D>
struct HeadRows {
  const __half *src;
  __half *dst;
  int left;
  uint4 ahead[kHeadsAhead];

  // heads h0 .. end of one token, rows of src into dst
  __device__ __forceinline__ void start(const __half *from, __half *to, int h0, int end) {
    const int at = h0 * D + threadIdx.x % (D / 8) * 8;
    src = from + at, dst = to + at, left = end - h0;
    load();
  }
  __device__ __forceinline__ void load() {
#pragma unroll
    for (int x = 0; x < kHeadsAhead; ++x)
      if (x < left) ahead[x] = *reinterpret_cast<const uint4 *>(src + x * D);
  }
  __device__ __forceinline__ void run(const HeadTurn<D> &turn, float eps) {
    for (; left > kHeadsAhead; left -= kHeadsAhead) {
#pragma unroll
      for (int x = 0; x < kHeadsAhead; ++x) *reinterpret_cast<uint4 *>(dst + x * D) = turn.apply(ahead[x], eps);
      src += kHeadsAhead * D, dst += kHeadsAhead * D;
#pragma unroll
      for (int x = 0; x < kHeadsAhead; ++x)
        if (x + kHeadsAhead < left) ahead[x] = *reinterpret_cast<const uint4 *>(src + x * D);
    }
#pragma unroll
    for (int x = 0; x < kHeadsAhead; ++x)
      if (x < left) *reinterpret_cast<uint4 *>(dst + x * D) = turn.apply(ahead[x], eps);
  }
};

template <int D>
__global__ void __launch_bounds__(kHeadThreads, 4) head_norm_rope_kernel(const HeadArgs a, int per, int q_groups) {
  constexpr int kLanes = D / 8;
  pdl_launch_dependents();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kHeadThreads / kLanes) + threadIdx.x / kLanes;
  if (t >= a.T) return;
  const bool key = static_cast<int>(blockIdx.y) >= q_groups;
  const int g = key ? blockIdx.y - q_groups : blockIdx.y, heads = key ? a.H : a.Hq;
  HeadRows<D> rows;
  rows.start(key ? a.k + t * a.k_stride : a.q + t * a.q_stride,
             key ? a.k_out + t * a.k_out_stride : a.q_out + t * a.q_out_stride, g * per, min(heads, (g + 1) * per));
  if (a.slots) {  // the cache's append: what it skips for keys
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.limit) return;
  }
  const float *angle = nullptr;
  if (a.rope) {
    const int64_t pos = a.positions[t];
    if (pos < 0) return;  // padding
    if (pos >= a.max_pos) {
      if (threadIdx.x % kLanes == 0) record_status(kStatusBounds);
      return;
    }
    angle = a.rope + pos * a.rotary;
  }
  HeadTurn<D> turn;
  turn.start(angle, a.rotary, key ? a.w_k : a.w_q);
  rows.run(turn, a.eps);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Heads of one lane: sixteen where the call fills the GPU all the same, one where it is latency that counts.
static int turn_heads_per_lane(int64_t T, int heads, int D) {
  int per = T * heads * (D / 8) >= 8ll * device_sm_count() * 2048 ? 16 : 1;
  while ((heads + per - 1) / per > 65535 / 2) ++per;
  return per;
}

template <int D>
static void launch_head_norm_rope_type(const HeadArgs &a, cudaStream_t stream) {
  const int per = turn_heads_per_lane(a.T, a.Hq > a.H ? a.Hq : a.H, D);
  const int q_groups = (a.Hq + per - 1) / per, k_groups = (a.H + per - 1) / per;
  constexpr int kTokens = kHeadThreads / (D / 8);
  const dim3 grid(static_cast<unsigned>((a.T + kTokens - 1) / kTokens), static_cast<unsigned>(q_groups + k_groups));
  head_norm_rope_kernel<D><<<grid, kHeadThreads, 0, stream>>>(a, per, q_groups);
}

cudaError_t launch_head_norm_rope(const HeadArgs &a, int D, cudaStream_t stream) {
  if (D == 64) launch_head_norm_rope_type<64>(a, stream);
  else if (D == 128) launch_head_norm_rope_type<128>(a, stream);
  else launch_head_norm_rope_type<256>(a, stream);
  return cudaGetLastError();
}

}  // namespace mixllm
