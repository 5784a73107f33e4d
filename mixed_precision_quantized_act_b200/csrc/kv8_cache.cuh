// kv8_cache.cuh -- the write side of the paged 8-bit KV cache: the normalized,
// rotated and quantized keys and values into their slots, and the cached rows
// back as fp16.
//
// Layout: codes uint8 [pages][2][H][page][D] (key, value), 128 + the whole
// number; scales fp32 [pages][2][H][page / 16], one for each block of 16 tokens
// of a head.  One head's rows of one page are one contiguous range.
#pragma once

#include <cuda_fp16.h>
#include <cstdint>

#include "head_norm.cuh"
#include "launch.h"
#include "ptx_sm100.cuh"
#include "quant.cuh"

namespace mixllm {

constexpr int kKv8Block = 16;  // tokens of one scale

// ---------------------------------------------------------------------------
// Append.  A block of 16 tokens shares a scale, so its tokens are one warp's
// work: the warp takes a run of new tokens of one block (neighbours in the list
// of slots) for one head, key or value, keeps their rows in registers, and
//   s = max(s before, amax / 127)   (before: 0 where the run holds the block's first row)
//   code = 128 + rne(x / s), and where s has grown the block's other rows are
//   re-coded: 128 + rne((code - 128) * (s before / s)).
// A NaN or an infinity makes s NaN; it stays so until the block's first row is
// written again.  Queries are rows on their own, in blocks of their own.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int64_t kv8_row(const Kv8Cache &c, int64_t slot, int kv, int h) {
  const int64_t page = slot >> c.page_log2;
  return (((page * 2 + kv) * c.H + h) << c.page_log2) + (slot & ((1 << c.page_log2) - 1));
}

// Four codes of an older row by the block's new scale.
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = static_cast<int>(w >> (8 * i) & 0xFFu) - 128;
    const int n = max(-127, min(127, __float2int_rn(__fmul_rn(static_cast<float>(c), ratio))));
    r |= static_cast<uint32_t>(n + 128) << (8 * i);
  }
  return r;
}

// One run's rows of one head, key (kv = 0) or value: the whole warp.  Lane i's
// `slot` is that of token t0 + i, or -1.
template <int D>
__device__ __forceinline__ void kv8_write_run(const Kv8AppendArgs &a, const HeadArgs &heads, int64_t t0, int64_t slot,
                                              int first, int count, int kv, int h) {
  constexpr int kLanes = D / 8, kTogether = 32 / kLanes, kPasses = kKv8Block / kTogether;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, in = lane / kLanes;
  const int64_t block = __shfl_sync(0xFFFFFFFFu, slot, first) >> 4;
  // ---- the rows, normalized and rotated
  uint4 x[kPasses];
  uint32_t rows = 0;  // of the block, bit by row, that are written
  int row_of[kPasses];
  float amax = 0.0f;
  bool odd = false;
  const __half *src = kv ? heads.v + t0 * heads.v_stride : heads.k + t0 * heads.k_stride;
  const int64_t stride = kv ? heads.v_stride : heads.k_stride;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int j = p * kTogether + in;
    row_of[p] = static_cast<int>(__shfl_sync(0xFFFFFFFFu, slot, (first + j) & 31)) & (kKv8Block - 1);
    x[p] = make_uint4(0, 0, 0, 0);
    if (j < count) x[p] = *reinterpret_cast<const uint4 *>(src + (first + j) * stride + h * D + sub * 8);
    else row_of[p] = -1;
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    if (p * kTogether >= count) continue;  // the same for the whole warp
    if (kv == 0 && (heads.rope || heads.w_k)) {
      const int j = p * kTogether + in;
      const float *angle = nullptr;
      if (heads.rope && row_of[p] >= 0) {
        const int64_t pos = heads.positions[t0 + first + j];
        if (pos < 0 || pos >= heads.max_pos) {
          if (sub == 0) record_status(kStatusBounds);
          row_of[p] = -1;
          x[p] = make_uint4(0, 0, 0, 0);
        } else {
          angle = heads.rope + pos * heads.rotary;
        }
      }
      HeadTurn<D> turn;
      turn.start(angle, heads.rotary, heads.w_k);
      turn.any = heads.rope != nullptr;  // every lane takes part in the exchange
      x[p] = turn.apply(x[p], heads.eps);
    } else if (heads.rope && row_of[p] >= 0) {  // a value is skipped where its key is
      const int64_t pos = heads.positions[t0 + first + p * kTogether + in];
      if (pos < 0 || pos >= heads.max_pos) row_of[p] = -1;
    }
    if (row_of[p] >= 0) {
      rows |= 1u << row_of[p];
      float f[8];
      widen8(x[p], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        amax = fmaxf(amax, fabsf(f[i]));
        odd |= !(fabsf(f[i]) <= 65504.0f);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  rows = __reduce_or_sync(0xFFFFFFFFu, rows);
  odd = __any_sync(0xFFFFFFFFu, odd);
  if (rows == 0) return;
  // ---- the scale
  const int64_t base = kv8_row(a.cache, block << 4, kv, h);
  float *scale = a.cache.scales + (base >> 4);
  const bool anew = rows & 1u;
  const float before = anew ? 0.0f : *scale;
  float s = fmaxf(before, __fdiv_rn(amax, 127.0f));
  if (odd || before != before) s = __int_as_float(0x7FFFFFFF);
  __syncwarp();  // every lane has read the scale
  if (lane == 0) *scale = s;
  uint8_t *codes = a.cache.codes + base * D;
  if (s > before && !anew) {
    // the older rows: 16 bytes a lane and step
    const float ratio = __fdiv_rn(before, s);
#pragma unroll
    for (int i = 0; i < kKv8Block * D / 512; ++i) {
      const int at = (i * 32 + lane) * 16;
      if (rows >> (at / D) & 1u) continue;
      uint4 *p = reinterpret_cast<uint4 *>(codes + at);
      const uint4 c = *p;
      *p = make_uint4(recode4(c.x, ratio), recode4(c.y, ratio), recode4(c.z, ratio), recode4(c.w, ratio));
    }
  }
  // ---- the new rows
  const bool none = !(s >= 0x1p-100f);  // nothing but zeros, or a NaN
  const QuantStep step = QuantStep::of(none ? 1.0f : s);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    if (row_of[p] < 0) continue;
    uint32_t packed[2] = {0x80808080u, 0x80808080u};
    if (!none) {
      float f[8];
      widen8(x[p], f);
      step.codes(f, packed);
      packed[0] ^= 0x80808080u, packed[1] ^= 0x80808080u;
    }
    *reinterpret_cast<uint2 *>(codes + row_of[p] * D + sub * 8) = make_uint2(packed[0], packed[1]);
  }
}

struct Kv8Grid {
  unsigned q_blocks, q_groups;  // blocks of queries; groups of `per` heads
  int per;
  unsigned groups;  // of `pairs` (head, kind) pairs
  int pairs;
};

template <int D>
__global__ void __launch_bounds__(kHeadThreads) kv8_append_kernel(const Kv8AppendArgs a, const HeadArgs heads,
                                                                  const Kv8Grid grid) {
  constexpr int kLanes = D / 8;
  const int64_t limit = a.cache.pages << a.cache.page_log2;
  if (blockIdx.x < grid.q_blocks) {
    // ------------------------------------------------------------ queries
    const unsigned tile = blockIdx.x / grid.q_groups, g = blockIdx.x - tile * grid.q_groups;
    const int64_t t = static_cast<int64_t>(tile) * (kHeadThreads / kLanes) + threadIdx.x / kLanes;
    if (t >= heads.T) return;
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= limit) return;  // recorded with the keys
    const float *angle = nullptr;
    if (heads.rope) {
      const int64_t pos = heads.positions[t];
      if (pos < 0 || pos >= heads.max_pos) return;  // likewise
      angle = heads.rope + pos * heads.rotary;
    }
    HeadTurn<D> turn;
    turn.start(angle, heads.rotary, heads.w_q);
    turn_heads<D>(turn, heads.q + t * heads.q_stride, heads.q_out + t * heads.q_out_stride, static_cast<int>(g) * grid.per,
                  min(heads.Hq, static_cast<int>(g + 1) * grid.per), heads.eps);
    return;
  }
  // ------------------------------------------------------------ keys and values: the runs that begin in 16 tokens
  const unsigned id = blockIdx.x - grid.q_blocks, tile = id / grid.groups, g = id - tile * grid.groups;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t0 = static_cast<int64_t>(tile) * kKv8Block;
  const auto slot_of = [&](int64_t t) {
    int64_t s = t >= 0 && t < heads.T ? a.slots[t] : -1;
    if (s >= limit) {
      record_status(kStatusBounds);
      s = -1;
    }
    return s;
  };
  const int64_t slot = slot_of(t0 + lane);
  int64_t prev = __shfl_up_sync(0xFFFFFFFFu, slot, 1);
  if (lane == 0) prev = slot_of(t0 - 1);
  const bool begins = slot >= 0 && (prev < 0 || prev >> 4 != slot >> 4);
  const uint32_t begin = __ballot_sync(0xFFFFFFFFu, begins);
  const uint32_t ends = begin | __ballot_sync(0xFFFFFFFFu, slot < 0);  // no run goes on here
  const int pair0 = g * grid.pairs, pairs = min(2 * a.cache.H - pair0, grid.pairs);
  int item = 0;
  for (uint32_t left = begin & 0xFFFFu; left; left &= left - 1) {
    const int first = __ffs(left) - 1;
    const uint32_t behind = ends & ~((2u << first) - 1u);
    int count = (behind ? __ffs(behind) - 1 : 32) - first;
    if (count > kKv8Block) {  // a slot that is there twice
      if (lane == 0) record_status(kStatusBounds);
      count = kKv8Block;
    }
    for (int p = 0; p < pairs; ++p, ++item) {
      if ((item & (kHeadThreads / 32 - 1)) != warp) continue;
      const int pair = pair0 + p, kv = pair >= a.cache.H;
      kv8_write_run<D>(a, heads, t0, slot, first, count, kv, pair - kv * a.cache.H);
    }
  }
}

// The cached rows of the given slots as fp16: s * (code - 128), rounded once and
// kept within the finite fp16 values.
template <int D>
__global__ void __launch_bounds__(kHeadThreads) kv8_read_kernel(const Kv8Cache c, const int64_t *__restrict__ slots,
                                                                int64_t T, __half *__restrict__ k,
                                                                __half *__restrict__ v, int per) {
  constexpr int kLanes = D / 8;
  const int sub = threadIdx.x % kLanes;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kHeadThreads / kLanes) + threadIdx.x / kLanes;
  if (t >= T) return;
  const int64_t slot = slots[t];
  if (slot < 0) return;
  if (slot >= c.pages << c.page_log2) {
    if (sub == 0) record_status(kStatusBounds);
    return;
  }
  const int h_end = min(2 * c.H, static_cast<int>(blockIdx.y + 1) * per);
#pragma unroll 4
  for (int h = blockIdx.y * per; h < h_end; ++h) {
    const int kv = h >= c.H, head = kv ? h - c.H : h;
    const int64_t row = kv8_row(c, slot, kv, head);
    const uint2 code = *reinterpret_cast<const uint2 *>(c.codes + row * D + sub * 8);
    const float s = c.scales[row >> 4];
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = (static_cast<float>((j < 4 ? code.x : code.y) >> (8 * (j & 3)) & 0xFFu) - 128.0f) * s;
      f[j] = x > 65504.0f ? 65504.0f : (x < -65504.0f ? -65504.0f : x);  // a NaN stays one
    }
    *reinterpret_cast<uint4 *>((kv ? v : k) + (t * c.H + head) * D + sub * 8) = pack8(f);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

cudaError_t launch_kv8_append(const Kv8AppendArgs &a, const HeadArgs &heads, cudaStream_t stream) {
  const int D = a.cache.D, H = a.cache.H;
  Kv8Grid g;
  g.per = heads.Hq > 0 ? turn_heads_per_lane(heads.T, heads.Hq, D) : 1;
  g.q_groups = static_cast<unsigned>((heads.Hq + g.per - 1) / g.per);
  const int tokens = kHeadThreads / (D / 8);
  g.q_blocks = static_cast<unsigned>((heads.T + tokens - 1) / tokens) * g.q_groups;
  // a warp's work is a run's pair: few tokens may be a run each, many are long runs
  g.pairs = heads.T <= 512 ? 1 : kHeadThreads / 32;
  g.groups = static_cast<unsigned>((2 * H + g.pairs - 1) / g.pairs);
  const unsigned blocks = g.q_blocks + static_cast<unsigned>((heads.T + kKv8Block - 1) / kKv8Block) * g.groups;
  if (g.q_groups == 0) g.q_groups = 1;
  if (D == 128) kv8_append_kernel<128><<<blocks, kHeadThreads, 0, stream>>>(a, heads, g);
  else kv8_append_kernel<64><<<blocks, kHeadThreads, 0, stream>>>(a, heads, g);
  return cudaGetLastError();
}

cudaError_t launch_kv8_read(const Kv8Cache &c, const int64_t *slots, int64_t T, void *k, void *v, cudaStream_t stream) {
  const int per = turn_heads_per_lane(T, 2 * c.H, c.D), tokens = kHeadThreads / (c.D / 8);
  const dim3 grid(static_cast<unsigned>((T + tokens - 1) / tokens), static_cast<unsigned>((2 * c.H + per - 1) / per));
  __half *kh = static_cast<__half *>(k), *vh = static_cast<__half *>(v);
  if (c.D == 128) kv8_read_kernel<128><<<grid, kHeadThreads, 0, stream>>>(c, slots, T, kh, vh, per);
  else kv8_read_kernel<64><<<grid, kHeadThreads, 0, stream>>>(c, slots, T, kh, vh, per);
  return cudaGetLastError();
}

}  // namespace mixllm
