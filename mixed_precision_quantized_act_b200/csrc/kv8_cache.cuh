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
// Append.  A block of 16 tokens shares a scale, so its tokens are two warps'
// work: they take a run of new tokens of one block (within 16 places of the list
// of slots, skipped ones among them) for one head, key or value, keep their rows
// in registers, and
//   s = max(s before, amax / 127)   (before: 0 where the run holds the block's first row)
//   code = 128 + rne(x / s), and where s has grown the block's other rows are
//   re-coded: 128 + rne((code - 128) * (s before / s)).
// A NaN or an infinity makes s NaN; it stays so until the block's first row is
// written again.  Queries are rows on their own: in blocks of their own, and for many
// tokens in a kernel of their own that runs beside this one.
//
// HBM-bound by its bytes, in fact by latency: slots, then rows, table and scale
// together, then the write.  4101 tokens of 64 + 16 heads of 128: 40.5 us (queries 25,
// keys and values 18.1, overlapping) and 8.7 us to read back, for 28.6 us of traffic;
// one warp a run took 24 us for keys and values (128 registers, 16 warps an SM; now 24),
// queries in this kernel 37.  32 tokens: 8.7 us.  Which places of a run hold a token is
// one mask for the warp: a row number for every lane spills (51.2 us with the read-back
// instead of 49.5).
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

// What the two warps of a run tell each other: the largest magnitude of their rows
// (infinity where one is not finite) and the rows themselves, bit by row.
struct Kv8Half {
  float amax;
  uint32_t rows;
};

// One run's rows of one head, key (kv = 0) or value: the 16 places of the list from
// t0 + first on, two warps, eight places each; bit j of `places`: there is a token of
// the run at the j-th.  Lane i's `slot` and `pos` are those of place t0 + i.  What
// depends on slot and position alone is loaded before anything is used.
template <int D, int kNorm>
__device__ __forceinline__ void kv8_write_run(const Kv8AppendArgs &a, const HeadArgs &heads, int64_t t0, int64_t slot,
                                              int pos, int first, uint32_t places, int kv, int h, Kv8Half *halves) {
  constexpr int kLanes = D / 8, kTogether = 32 / kLanes, kPasses = kKv8Block / 2 / kTogether;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % kLanes;
  const int mine = (warp & 1) * (kKv8Block / 2) + lane / kLanes;  // of the run's places, this lane's first
  const int64_t block = __shfl_sync(0xFFFFFFFFu, slot, first) >> 4;
  const int64_t base = kv8_row(a.cache, block << 4, kv, h);
  float *scale = a.cache.scales + (base >> 4);
  const float old_scale = *scale;
  const __half *src = kv ? heads.v + t0 * heads.v_stride : heads.k + t0 * heads.k_stride;
  const int64_t stride = kv ? heads.v_stride : heads.k_stride;
  uint4 x[kPasses];
  int row_of[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int j = mine + p * kTogether;
    row_of[p] = static_cast<int>(__shfl_sync(0xFFFFFFFFu, slot, (first + j) & 31)) & (kKv8Block - 1);
    x[p] = make_uint4(0, 0, 0, 0);
    if (places >> j & 1u) x[p] = *reinterpret_cast<const uint4 *>(src + (first + j) * stride + h * D + sub * 8);
    else row_of[p] = -1;
  }
  // ---- the rows, normalized and rotated
  uint32_t rows = 0;
  float amax = 0.0f;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    if (places >> ((warp & 1) * (kKv8Block / 2) + p * kTogether) == 0) continue;  // the same for the whole warp
    const int at = __shfl_sync(0xFFFFFFFFu, pos, (first + mine + p * kTogether) & 31);
    if (heads.rope && row_of[p] >= 0 && (at < 0 || at >= heads.max_pos)) {
      if (kv == 0 && sub == 0) record_status(kStatusBounds);
      row_of[p] = -1;  // a value is skipped where its key is
    }
    if (kv == 0 && (heads.rope || kNorm)) {
      HeadTurn<D, kNorm> turn;
      turn.start(heads.rope && row_of[p] >= 0 ? heads.rope + static_cast<int64_t>(at) * heads.rotary : nullptr,
                 heads.rotary, heads.w_k);
      turn.any = heads.rope != nullptr;  // every lane takes part in the exchange
      x[p] = turn.apply(x[p], heads.eps);
    }
    if (row_of[p] >= 0) {
      rows |= 1u << row_of[p];
      const __half2 *h2 = reinterpret_cast<const __half2 *>(&x[p]);
      const __half2 m = __hmax2_nan(__hmax2_nan(__habs2(h2[0]), __habs2(h2[1])), __hmax2_nan(__habs2(h2[2]), __habs2(h2[3])));
      const float top = __half2float(__hmax_nan(__low2half(m), __high2half(m)));
      amax = fmaxf(amax, top <= 65504.0f ? top : INFINITY);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  rows = __reduce_or_sync(0xFFFFFFFFu, rows);
  if (lane == 0) halves[warp] = Kv8Half{amax, rows};
  named_bar_sync(1 + (warp >> 1), 64);  // also: both have read the scale
  const Kv8Half other = halves[warp ^ 1];
  named_bar_sync(1 + (warp >> 1), 64);  // before either writes its next run's
  amax = fmaxf(amax, other.amax);
  rows |= other.rows;
  if (rows == 0) return;
  // ---- the scale
  const bool anew = rows & 1u;
  const float before = anew ? 0.0f : old_scale;
  float s = fmaxf(before, __fdiv_rn(amax, 127.0f));
  if (amax == INFINITY || before != before) s = __int_as_float(0x7FFFFFFF);
  if (lane == 0 && (warp & 1) == 0) *scale = s;
  uint8_t *codes = a.cache.codes + base * D;
  if (s > before && !anew) {
    // the older rows, eight a warp: 16 bytes a lane and step
    const float ratio = __fdiv_rn(before, s);
    constexpr int kSteps = kKv8Block / 2 * D / 512;
    const int from = (warp & 1) * (kKv8Block / 2 * D);
    uint4 old[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int at = from + (i * 32 + lane) * 16;
      if (!(rows >> (at / D) & 1u)) old[i] = *reinterpret_cast<const uint4 *>(codes + at);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int at = from + (i * 32 + lane) * 16;
      if (rows >> (at / D) & 1u) continue;
      *reinterpret_cast<uint4 *>(codes + at) = make_uint4(recode4(old[i].x, ratio), recode4(old[i].y, ratio),
                                                          recode4(old[i].z, ratio), recode4(old[i].w, ratio));
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

// The last slot of a cached token before place `end` of the list, or -1: for lists with long runs of skipped ones.
// The whole warp.
__device__ __forceinline__ int64_t kv8_last_before(const int64_t *slots, int64_t end, int64_t limit) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (; end > 0; end -= 128) {
    int64_t s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = end - 32 * (i + 1) + lane;
      s[i] = at >= 0 ? slots[at] : -1;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t there = __ballot_sync(0xFFFFFFFFu, s[i] >= 0 && s[i] < limit);
      if (there) return __shfl_sync(0xFFFFFFFFu, s[i], 31 - __clz(there));
    }
  }
  return -1;
}

// A run is 16 places.  Records tokens of places t0 .. t0 + 15 whose run began before t0 and that lie behind those: the
// first such token of a block has another of its block in the 16 places before it, whose run began in the 32 before t0
// then, or it has none.  The whole warp.
__device__ __forceinline__ void kv8_record_far(const int64_t *slots, int64_t t0, int64_t T, int64_t limit) {
  const int lane = threadIdx.x & 31;
  const int64_t slot = lane < kKv8Block && t0 + lane < T ? slots[t0 + lane] : -1;
  const int64_t back = t0 + lane >= 32 ? slots[t0 + lane - 32] : -1;  // of the 32 places before t0
  const bool is = slot >= 0 && slot < limit, is_back = back >= 0 && back < limit;
  const uint32_t there = __ballot_sync(0xFFFFFFFFu, is), there_back = __ballot_sync(0xFFFFFFFFu, is_back);
  if (!there) return;
  const int64_t block = __shfl_sync(0xFFFFFFFFu, slot, __ffs(there) - 1) >> 4;
  const uint32_t another = __ballot_sync(0xFFFFFFFFu, is && slot >> 4 != block);
  const int far = 31 - __clz(there & (another ? (another & -another) - 1u : ~0u));  // the first block's last token here
  const uint32_t same = __ballot_sync(0xFFFFFFFFu, is_back && back >> 4 == block), other = there_back & ~same;
  const uint32_t chain = other ? same & ~((2u << (31 - __clz(other))) - 1u) : same;
  if (chain) {
    if (far + 32 - (__ffs(chain) - 1) >= kKv8Block) record_status(kStatusBounds);
  } else if (!there_back) {
    const int64_t last = kv8_last_before(slots, t0 - 32, limit);
    if (last >= 0 && last >> 4 == block) record_status(kStatusBounds);
  }
}

struct Kv8Grid {
  unsigned q_blocks, q_groups;  // blocks of queries; groups of `per` heads
  int per;
  unsigned groups;  // of `pairs` (head, kind) pairs
  int pairs, split;  // split: blocks that share a group's runs
};

// kNorm: whether there are norms of keys
template <int D, int kNorm>
__global__ void __launch_bounds__(kHeadThreads, 3) kv8_append_kernel(const Kv8AppendArgs a, const HeadArgs heads,
                                                                  const Kv8Grid grid) {
  constexpr int kLanes = D / 8;
  const int64_t limit = a.cache.pages << a.cache.page_log2;
  if (blockIdx.x < grid.q_blocks) {
    // ------------------------------------------------------------ queries
    const unsigned tile = blockIdx.x / grid.q_groups, g = blockIdx.x - tile * grid.q_groups;
    const int64_t t = static_cast<int64_t>(tile) * (kHeadThreads / kLanes) + threadIdx.x / kLanes;
    if (t >= heads.T) return;
    HeadRows<D> rows;
    rows.start(heads.q + t * heads.q_stride, heads.q_out + t * heads.q_out_stride, static_cast<int>(g) * grid.per,
               min(heads.Hq, static_cast<int>(g + 1) * grid.per));
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
    rows.run(turn, heads.eps);
    return;
  }
  // ------------------------------------------------------------ keys and values: the runs that begin in 16 tokens
  const unsigned id = (blockIdx.x - grid.q_blocks) / grid.split, part = blockIdx.x - grid.q_blocks - id * grid.split;
  const unsigned tile = id / grid.groups, g = id - tile * grid.groups;
  constexpr int kTeams = kHeadThreads / 64;  // of two warps
  __shared__ Kv8Half halves[kHeadThreads / 32];
  const int lane = threadIdx.x & 31, team = threadIdx.x >> 6;
  const int64_t t0 = static_cast<int64_t>(tile) * kKv8Block;
  int64_t slot = t0 + lane < heads.T ? a.slots[t0 + lane] : -1, last = t0 > 0 ? a.slots[t0 - 1] : -1;
  const int pos = heads.rope && t0 + lane < heads.T ? heads.positions[t0 + lane] : 0;
  if (slot >= limit) {
    record_status(kStatusBounds);
    slot = -1;
  }
  if (last >= limit) last = -1;
  // A token begins a run unless the last one before it is of the same block, however many skipped ones stand between.
  const uint32_t there = __ballot_sync(0xFFFFFFFFu, slot >= 0);
  if (last < 0 && t0 > 0 && (there & 0xFFFFu)) last = kv8_last_before(a.slots, t0 - 1, limit);
  const uint32_t below = there & ((1u << lane) - 1u);
  const int64_t left_of = __shfl_sync(0xFFFFFFFFu, slot, below ? 31 - __clz(below) : 0);
  const int64_t prev = below ? left_of : last;
  const uint32_t begin = __ballot_sync(0xFFFFFFFFu, slot >= 0 && (prev < 0 || prev >> 4 != slot >> 4));
  const int pair0 = g * grid.pairs, pairs = min(2 * a.cache.H - pair0, grid.pairs);
  int item = 0;
  for (uint32_t left = begin & 0xFFFFu; left; left &= left - 1) {
    const int first = __ffs(left) - 1;
    const uint32_t later = begin & ~((2u << first) - 1u);
    const uint32_t rest = there & ~((1u << first) - 1u) & (later ? (later & -later) - 1u : ~0u);  // of its block
    const uint32_t run = rest & (0xFFFFu << first);  // what is farther behind is left out, and recorded
    if (rest != run) record_status(kStatusBounds);
    for (int p = 0; p < pairs; ++p, ++item) {
      if (item % (grid.split * kTeams) != static_cast<int>(part) * kTeams + team) continue;
      const int pair = pair0 + p, kv = pair >= a.cache.H;
      kv8_write_run<D, kNorm>(a, heads, t0, slot, pos, first, run >> first, kv, pair - kv * a.cache.H, halves);
    }
  }
  if (g == 0 && part == 0 && threadIdx.x < 32) kv8_record_far(a.slots, t0, heads.T, limit);
  pdl_wait();  // the queries' kernel, where there is one, runs beside this one: who waits for this waits for it
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
  const bool few = heads.T <= 512;
  Kv8Grid g;
  g.per = heads.Hq > 0 ? turn_heads_per_lane(heads.T, heads.Hq, D) : 1;
  g.q_groups = static_cast<unsigned>((heads.Hq + g.per - 1) / g.per);
  const int tokens = kHeadThreads / (D / 8);
  if (!few) g.q_groups = 0;
  g.q_blocks = static_cast<unsigned>((heads.T + tokens - 1) / tokens) * g.q_groups;
  // two warps' work is a run's pair: few tokens may be a run each, many are long runs
  g.pairs = few ? 1 : kHeadThreads / 64;
  g.split = few ? 4 : 1;
  g.groups = static_cast<unsigned>((2 * H + g.pairs - 1) / g.pairs);
  const int64_t blocks = g.q_blocks + (heads.T + kKv8Block - 1) / kKv8Block * g.groups * g.split;
  if (blocks > 0x7FFFFFFF) return cudaErrorNotSupported;
  if (!few && heads.Hq > 0) {
    // The runs' registers leave an SM 24 warps, too few for the queries' traffic: those take a kernel of their own,
    // which many tokens do not notice.
    HeadArgs q = heads;
    q.H = 0, q.slots = a.slots, q.limit = a.cache.pages << a.cache.page_log2;
    const cudaError_t e = launch_head_norm_rope(q, D, stream);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kHeadThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = !few && heads.Hq > 0 ? 1 : 0;  // behind the queries' kernel, which it does not depend on
  if (g.q_groups == 0) g.q_groups = 1;
  const bool norm = heads.w_k != nullptr;
  const auto kern = D == 128 ? (norm ? kv8_append_kernel<128, 1> : kv8_append_kernel<128, 0>)
                             : (norm ? kv8_append_kernel<64, 1> : kv8_append_kernel<64, 0>);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, heads, g);
  return e == cudaSuccess ? cudaGetLastError() : e;
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
