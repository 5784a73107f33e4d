// head_norm.cuh -- the norms of query and key heads (one RMS norm per token and
// head, over the head's channels) and the rotation by position, in one pass.
#pragma once

#include <cuda_fp16.h>
#include <cstdint>

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
// bits of the 4-bit cache's rotation.  (Pairs of floats would need a third of the
// instructions fewer, but ptxas joins their products and sums; the time is the same.)
//
// HBM-bound: 4 bytes a channel, and the table's 8 bytes a channel of a token once
// for sixteen heads.  4099 tokens of 64 + 8 heads of 128, half of their channels
// rotated: 30.9 us on B200, 4.9 TB/s (75 % of the measured copy rate).  A block's
// latencies follow one another (heads and position, table, stores); more warps an SM
// (40 or 48 for 32, with two heads ahead) took 34 to 40 us, eight heads ahead 33.6,
// the first heads loaded behind the position 35.
// ---------------------------------------------------------------------------
template <int D>
struct HeadTurn {
  static constexpr int kLanes = D / 8;
  float own[8], far[8];
  int other;      // lane of the row that holds the channels paired with this one's
  bool norm, any, turned;  // turned: this lane's channels are rotated; any: some lane's are
  unsigned mask;

  // `angle`: the position's rotary/2 cosines, then its sines, or null; `w`: fp16 [D], or null
  __device__ __forceinline__ void start(const float *angle, int rotary, const __half *w) {
    const int sub = threadIdx.x % kLanes, c0 = sub * 8, half = rotary / 2;  // half is a multiple of 8
    mask = (kLanes == 32 ? 0xFFFFFFFFu : ((1u << (kLanes & 31)) - 1u)) << (threadIdx.x & 31 & ~(kLanes - 1));
    const bool second = c0 >= half;
    norm = w != nullptr, any = angle != nullptr && half > 0, turned = any && c0 < rotary;
    other = second ? sub - half / 8 : sub + half / 8;
    if (turned) {
      const float *at = angle + (second ? c0 - half : c0);
      load8(at, own);
      load8(at + half, far);
#pragma unroll
      for (int j = 0; j < 8; ++j) far[j] = second ? far[j] : -far[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) own[j] = 1.0f, far[j] = 0.0f;
    }
    if (norm) {
      float f[8];
      load8(w + c0, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) own[j] *= f[j];
      if (turned) {
        load8(w + other * 8, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) far[j] *= f[j];
      }
    }
  }

  __device__ __forceinline__ uint4 apply(const uint4 raw, float eps) const {
    if (!norm && !any) return raw;
    float x[8], inv = 1.0f;
    widen8(raw, x);
    if (norm) {
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
      inv = rsqrtf(fmaf(ss, 1.0f / D, eps));
    }
    if (any) {
      uint4 far_raw;
      far_raw.x = __shfl_sync(mask, raw.x, other, kLanes);
      far_raw.y = __shfl_sync(mask, raw.y, other, kLanes);
      far_raw.z = __shfl_sync(mask, raw.z, other, kLanes);
      far_raw.w = __shfl_sync(mask, raw.w, other, kLanes);
      float y[8];
      widen8(far_raw, y);
      if (turned) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fadd_rn(__fmul_rn(x[j], own[j]), __fmul_rn(y[j], far[j]));
      }
    }
    if (!turned) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= own[j];
    }
    if (norm) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= inv;
    }
    return pack8(x);
  }
};

// One block takes 256 / (D / 8) tokens and `per` heads of queries or of keys; a
// lane loads four heads ahead, the first ones before it knows its position.
constexpr int kHeadThreads = 256, kHeadsAhead = 4;

template <int D>
struct HeadRows {
  const __half *src;
  __half *dst;
  int h, h_end;
  uint4 ahead[kHeadsAhead];

  // heads h0 .. end of one token, rows of src into dst
  __device__ __forceinline__ void start(const __half *from, __half *to, int h0, int end) {
    const int c0 = threadIdx.x % (D / 8) * 8;
    src = from + c0, dst = to + c0, h = h0, h_end = end;
    load();
  }
  __device__ __forceinline__ void load() {
#pragma unroll
    for (int x = 0; x < kHeadsAhead; ++x)
      if (h + x < h_end) ahead[x] = *reinterpret_cast<const uint4 *>(src + (h + x) * D);
  }
  __device__ __forceinline__ void run(const HeadTurn<D> &turn, float eps) {
    while (true) {
#pragma unroll
      for (int x = 0; x < kHeadsAhead; ++x)
        if (h + x < h_end) *reinterpret_cast<uint4 *>(dst + (h + x) * D) = turn.apply(ahead[x], eps);
      h += kHeadsAhead;
      if (h >= h_end) return;
      load();
    }
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
    int per = T * heads * (D / 8) >= 8ll * 148 * 2048 ? 16 : 1;
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
