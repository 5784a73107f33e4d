// kv_split.cuh -- how a decode step's attention over a paged cache is shared
// among warps and blocks, whatever the cache's format: units of 32 tokens of one
// request and key head, an even run of them for every block and warp, the
// fetching of their pages, and the joining of the parts of segments that the
// ends of a run cut.
#pragma once

#include <cuda_fp16.h>
#include <cstdint>

#include "kv4_ptx.cuh"
#include "launch.h"
#include "ptx_sm100.cuh"

namespace mixllm {

constexpr int kKvTile = 32;  // tokens per unit
constexpr float kKvNoMax = -3.0e38f;
constexpr int kKvMaxGrid = 148;

// One request's share of the work.
struct KvReq {
  int q0, n, kv, tiles, row_tiles;
};

// Reads and checks one request's lengths.  Anything out of range (a device
// value the host cannot see) is recorded and the request skipped.
template <typename A>
__device__ __forceinline__ KvReq kv_req(const A &a, int b, int rows_per_tile) {
  KvReq r;
  r.q0 = a.cu_q[b];
  r.n = a.cu_q[b + 1] - r.q0;
  r.kv = a.kv_lens[b];
  if (r.q0 < 0 || r.n < 0 || r.n > a.max_q || static_cast<int64_t>(r.q0) + r.n > a.T || r.kv < 0 ||
      r.kv > static_cast<int64_t>(a.W) << a.cache.page_log2) {
    record_status(kStatusBounds);
    r.n = 0;
  }
  r.tiles = r.n > 0 ? max(1, (r.kv + kKvTile - 1) / kKvTile) : 0;  // a request without keys still writes its rows
  r.row_tiles = (r.n * (a.Hq / a.cache.H) + rows_per_tile - 1) / rows_per_tile;
  return r;
}

// Walks a warp's units as segments: runs of units of one request and key head.
struct KvWalk {
  int b, h, tile, count;  // the segment: its first unit's tile and its units in this warp
  int left;               // units of the warp from the segment's first on
  int seg_first;          // unit index of the whole segment's first tile
  KvReq r;

  template <typename A>
  __device__ __forceinline__ void next(const A &a, int rows_per_tile) {
    left -= count;
    seg_first += r.tiles;
    tile = 0;
    if (++h == a.cache.H) {
      h = 0;
      while (left > 0 && ++b < a.B) {
        r = kv_req(a, b, rows_per_tile);
        if (r.tiles > 0) break;
      }
      if (b >= a.B) left = 0;
    }
    count = min(left, r.tiles);
  }
};

// A warp's fetching: the 32 tokens of its units in turn, codes and
// metadata, into the next stage of its ring.  Half a warp copies 16 tokens:
// a page holds a multiple of 16, so they lie in one.
template <typename C>
struct KvFetch {
  uint32_t ring;     // shared address of this lane's first bytes in stage 0
  uint32_t present;  // bits 2s, 2s + 1: the halves of stage s are tokens of a page that exists
  int stage;
  int b, h, tile, batch, id, left;
  KvReq r;

  __device__ __forceinline__ void start(const KvWalk &w, int lane, const uint8_t *to) {
    ring = smem_u32(to) + C::lane_bytes(lane);
    present = 0;
    stage = 0;
    b = w.b, h = w.h, tile = w.tile, r = w.r;
    left = w.left;
    batch = -1;
  }

  template <typename A>
  __device__ __forceinline__ void unit(const A &a, int lane) {
    if (left > 0) {
      const int page_log2 = a.cache.page_log2;
      if ((tile >> 4) != batch) {
        // the pages of 16 units: lane 2u + i has unit u's half i
        batch = tile >> 4;
        const int64_t token = (static_cast<int64_t>(batch) * 32 + lane) * 16;
        id = -1;
        if (token < r.kv) {
          id = a.table[static_cast<int64_t>(b) * a.table_stride + (token >> page_log2)];
          if (id < 0 || id >= a.cache.pages) {
            record_status(kStatusBounds);
            id = -1;
          }
        }
      }
      const int page = __shfl_sync(0xFFFFFFFFu, id, (tile & 15) * 2 + (lane >> 4));
      const uint32_t halves = __ballot_sync(0xFFFFFFFFu, page >= 0);
      present = (present & ~(3u << 2 * stage)) | ((halves & 1u) | (halves >> 30 & 2u)) << 2 * stage;
      if (page >= 0) {
        const int row = (tile * kKvTile + (lane & 16)) & ((1 << page_log2) - 1);
        const int64_t at = static_cast<int64_t>(page) * (2 * a.cache.H << page_log2) + ((h << page_log2) + row);
        const int64_t to_value = static_cast<int64_t>(a.cache.H) << page_log2;  // rows from a key to its value
        C::copy(a.cache, lane, at, to_value, ring + stage * C::kStage);
      }
      --left;
      if (++tile == r.tiles) {
        tile = 0;
        batch = -1;
        if (++h == a.cache.H) {
          h = 0;
          while (left > 0 && ++b < a.B) {
            r = kv_req(a, b, C::kRows);
            if (r.tiles > 0) break;
          }
          if (b >= a.B) left = 0;
        }
      }
    }
    cp_async_commit();  // one group per unit, empty or not, so that waiting counts units
    if (++stage == C::kStages) stage = 0;
  }
};

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// A segment's place, for who joins its parts.
struct KvSeg {
  int h, tiles, q0, n;
};

// Joining parts: a warp takes a row, a lane four (or two) of its channels, and
// lane i holds the weight of part i.  A part's row holds channel D/8 g + 2k + e
// at 16k + 2g + e: the order in which the lanes of an accumulator can write it
// without conflicts of shared-memory banks.
template <int D>
struct KvRow {
  static constexpr int kCh = D / 32;
  float top, sum, plain, acc[kCh];  // sum: of the weights as rounded; plain: before

  __device__ __forceinline__ void clear() {
    top = kKvNoMax;
    sum = plain = 0.0f;
#pragma unroll
    for (int k = 0; k < kCh; ++k) acc[k] = 0.0f;
  }
  static __device__ __forceinline__ float max_lanes(float v) {
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, x));
    return v;
  }
  static __device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, x);
    return v;
  }
  // `from`: this lane's channels of the row in a part
  template <bool kGlobal>
  static __device__ __forceinline__ void load(const float *from, float (&v)[kCh]) {
    if constexpr (kCh == 4) {
      const float4 *f = reinterpret_cast<const float4 *>(from);
      const float4 u = kGlobal ? __ldcg(f) : *f;
      v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
    } else {
      const float2 *f = reinterpret_cast<const float2 *>(from);
      const float2 u = kGlobal ? __ldcg(f) : *f;
      v[0] = u.x, v[1] = u.y;
    }
  }
  __device__ __forceinline__ void add(const float (&v)[kCh], float f) {
#pragma unroll
    for (int k = 0; k < kCh; ++k) acc[k] = fmaf(v[k], f, acc[k]);
  }
  template <typename A>
  __device__ __forceinline__ void write(const A &a, const KvSeg &s, int row, int lane) {
    const int group = a.Hq / a.cache.H;
    if (row >= s.n * group) return;
    const int tok = row / group, head = s.h * group + row - tok * group;
    const int64_t token = static_cast<int64_t>(s.q0) + tok;
    const float inv = plain == 0.0f ? 0.0f : 1.0f / sum;  // a row that saw no key is zero
    __half *dst = a.out + token * a.out_stride + static_cast<int64_t>(head) * D;
#pragma unroll
    for (int j = 0; j < kCh; j += 2) {
      const int at = lane * kCh + j;  // 16k + 2g
      *reinterpret_cast<__half2 *>(dst + (at % 16 / 2) * (D / 8) + at / 16 * 2) =
          __floats2half2_rn(acc[j] * inv, acc[j + 1] * inv);
    }
    if (a.lse && lane == 0)
      a.lse[token * a.Hq + head] = plain == 0.0f ? -INFINITY : (top + log2f(plain)) * 0.6931471805599453f;
  }
};

// What a block's warps tell each other.  part_first: the segment (its first
// unit) of a part that a warp left, or -1: [0] in the workspace (behind its first
// segment), [1] in shared memory (its last one).
template <int kWarps>
struct KvShared {
  int part_first[kWarps][2], cut_first[2], join_blocks[2][2], warp_units[kWarps];
  KvSeg part_at[kWarps][2], cut_at[2];
};

// A block's share: units start .. start + mine of the U that P blocks share.
struct KvShare {
  int P, U, start, mine;
};

// This block's share and this warp's first segment (w.left units from there
// on); false when there is none for the block.
template <typename C, typename A>
__device__ __forceinline__ bool kv_first_units(const A &a, KvShared<C::kWarps> &shared, KvShare &my, KvWalk &w0) {
  // ---- this warp's units, by a prefix sum of the requests' units
  constexpr int kRows = C::kRows, kWarps = C::kWarps, kThreads = C::kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
  int P = gridDim.x;
  const auto units_of = [&](int b) {
    const KvReq r = kv_req(a, b, kRows);
    return r.tiles * a.cache.H;
  };
  const auto scan = [&](int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  constexpr int kFew = 4;  // requests per lane that a warp scans for itself, with no barrier
  const bool few = a.B <= 32 * kFew;
  int incl[kFew], U = 0;  // of requests 32 i + lane
  if (few) {
    int u[kFew];
#pragma unroll
    for (int i = 0; i < kFew; ++i) u[i] = 32 * i + lane < a.B ? units_of(32 * i + lane) : 0;
#pragma unroll
    for (int i = 0; i < kFew; ++i) {
      incl[i] = scan(u[i]) + U;
      U = __shfl_sync(0xFFFFFFFFu, incl[i], 31);
    }
  } else {
    for (int b = tid; b < a.B; b += kThreads) U += units_of(b);
    U = __reduce_add_sync(0xFFFFFFFFu, U);
    if (lane == 0) shared.warp_units[warp] = U;
    __syncthreads();
    U = 0;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) U += shared.warp_units[x];
  }
  if (C::kWholeHeads && a.B == 1 && U < P * kWarps * 4 && P >= a.cache.H) {
    // a single request's heads are alike: the same number of blocks to each, one where two units a warp do
    const int tiles = U / a.cache.H;
    P = a.cache.H * (tiles <= 2 * kWarps ? 1 : min((tiles + kWarps - 1) / kWarps, P / a.cache.H));
  } else if (U < P * kWarps * C::kLeast) {
    // at least kLeast units a warp: fewer blocks share a short context, whose joining would cost more than a unit
    P = (U + kWarps * C::kLeast - 1) / (kWarps * C::kLeast);
  }
  if (c >= P) return false;  // every other block has a unit
  const int share = U / P, rest = U - share * P;
  const auto block_start = [&](int b) { return share * b + rest * b / P; };  // rest, b < 2^8
  const int start = block_start(c), mine = block_start(c + 1) - start;
  const int my_start = start + mine * warp / kWarps, my_end = start + mine * (warp + 1) / kWarps;
  w0.left = my_end - my_start;
  w0.b = a.B;
  int before = 0;  // units before request w0.b
  if (few) {
#pragma unroll
    for (int i = kFew - 1; i >= 0; --i) {
      const uint32_t beyond = __ballot_sync(0xFFFFFFFFu, incl[i] > my_start);
      if (beyond) w0.b = 32 * i + __ffs(beyond) - 1;
    }
#pragma unroll
    for (int i = 0; i < kFew; ++i) {
      const int v = __shfl_sync(0xFFFFFFFFu, incl[i], (w0.b - 1) & 31);
      if (w0.b > 0 && (w0.b - 1) / 32 == i) before = v;
    }
  } else {
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int end = scan(b0 + lane < a.B ? units_of(b0 + lane) : 0) + before;
      const uint32_t beyond = __ballot_sync(0xFFFFFFFFu, end > my_start);
      if (beyond) {
        const int i = __ffs(beyond) - 1;
        const int v = __shfl_sync(0xFFFFFFFFu, end, i > 0 ? i - 1 : 0);
        if (i > 0) before = v;
        w0.b = b0 + i;
        break;
      }
      before = __shfl_sync(0xFFFFFFFFu, end, 31);
    }
  }
  w0.r = KvReq{0, 0, 0, 0, 0};
  w0.h = w0.tile = 0;
  if (w0.b >= a.B) w0.left = 0;
  if (w0.left > 0) {
    w0.r = kv_req(a, w0.b, kRows);
    w0.h = (my_start - before) / w0.r.tiles;
    w0.tile = my_start - before - w0.h * w0.r.tiles;
  }
  w0.seg_first = my_start - w0.tile;
  w0.count = min(w0.left, w0.r.tiles - w0.tile);
  my = KvShare{P, U, start, mine};
  return true;
}

// Joins the block's parts, and with the last block to arrive those of segments
// cut between blocks.  last_parts: the warps' last ones, in shared memory;
// warp_parts, block_parts: the workspace's.
template <int D, typename C, typename A>
__device__ __forceinline__ void kv_join_parts(const A &a, KvShared<C::kWarps> &shared, const KvShare &my,
                                              const float *last_parts, const float *warp_parts, float *block_parts,
                                              uint32_t *counters) {
  constexpr int kRows = C::kRows, kWarps = C::kWarps;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
  const int P = my.P, U = my.U, start = my.start, mine = my.mine;
  // ---- the block's parts, segment by segment; lane i looks after part i.  A
  // segment's parts are neighbours among those that there are.  A warp takes
  // one row of one segment at a time.
  const int part_seg = lane < 2 * kWarps ? shared.part_first[lane >> 1 & (kWarps - 1)][lane & 1] : -1;
  const uint32_t there = __ballot_sync(0xFFFFFFFFu, part_seg >= 0);
  const uint32_t before_me = there & ((1u << lane) - 1u);
  const int seg_before = __shfl_sync(0xFFFFFFFFu, part_seg, before_me ? 31 - __clz(before_me) : 0);
  uint32_t firsts = __ballot_sync(0xFFFFFFFFu, part_seg >= 0 && (!before_me || seg_before != part_seg));
  const int my_warp = lane >> 1 & (kWarps - 1);
  const float *my_part = lane & 1 ? last_parts + my_warp * C::kPart : warp_parts + (c * kWarps + my_warp) * C::kPart;
  KvRow<D> row;
  for (int item = 0; firsts; firsts &= firsts - 1) {
    const int first = __ffs(firsts) - 1;
    const uint32_t rest_of = firsts & (firsts - 1);
    uint32_t these = there & ~((1u << first) - 1u);
    if (rest_of) these &= (rest_of & -rest_of) - 1u;
    const int seg_first = shared.part_first[first >> 1][first & 1];
    const KvSeg seg = shared.part_at[first >> 1][first & 1];
    const bool whole = seg_first >= start && seg_first + seg.tiles <= start + mine;
    const int side = start <= seg_first ? 1 : 0;  // the block's end cuts it, or its beginning
    if (!whole && tid == 0) {
      shared.cut_first[side] = seg_first;
      shared.cut_at[side] = seg;
    }
    const int rows = min(kRows, seg.n * (a.Hq / a.cache.H));  // that there are
    for (int r = 0; r < rows; ++r, ++item) {
      if (item % kWarps != warp) continue;
      row.clear();
      const bool in = these >> lane & 1u;
      const float4 ml = in ? *reinterpret_cast<const float4 *>(my_part + kRows * C::kPitch + 4 * r)
                           : make_float4(kKvNoMax, 0.0f, 0.0f, 0.0f);
      row.top = row.max_lanes(ml.x);
      const float f = in ? ex2(ml.x - row.top) : 0.0f;
      row.sum = row.sum_lanes(ml.y * f);
      row.plain = row.sum_lanes(ml.z * f);
      const int at = r * C::kPitch + lane * KvRow<D>::kCh;
      // the warps' last parts, in shared memory, then the few that a warp left behind before going on (any fixed
      // order will do: a sum's terms are the same whoever was first)
      constexpr int kTogether = 8;
      for (uint32_t some = these & 0xAAAAAAAAu; some;) {
        float v[kTogether][KvRow<D>::kCh], fx[kTogether];
#pragma unroll
        for (int x = 0; x < kTogether; ++x) {
          const int i = some ? __ffs(some) - 1 : 0;
          fx[x] = some ? __shfl_sync(0xFFFFFFFFu, f, i) : 0.0f;
          row.template load<false>(last_parts + (some ? (i >> 1) * C::kPart : 0) + at, v[x]);
          some &= some - 1;
        }
#pragma unroll
        for (int x = 0; x < kTogether; ++x)
          if (fx[x] != 0.0f) row.add(v[x], fx[x]);
      }
      for (uint32_t some = these & 0x55555555u; some; some &= some - 1) {
        const int i = __ffs(some) - 1;
        float v[KvRow<D>::kCh];
        row.template load<true>(warp_parts + (c * kWarps + (i >> 1)) * C::kPart + at, v);
        row.add(v, __shfl_sync(0xFFFFFFFFu, f, i));
      }
      if (whole) {
        row.write(a, seg, r, lane);
      } else {
        float *part = block_parts + (c * 2 + side) * C::kPart;
#pragma unroll
        for (int k = 0; k < KvRow<D>::kCh; k += 2)
          *reinterpret_cast<float2 *>(part + at + k) = make_float2(row.acc[k], row.acc[k + 1]);
        if (lane == 0)
          *reinterpret_cast<float4 *>(part + kRows * C::kPitch + 4 * r) = make_float4(row.top, row.sum, row.plain, 0.0f);
      }
    }
  }

  // ---- segments cut between blocks: the last block to get here joins the parts
  __syncthreads();
  if (tid < 2) {
    shared.join_blocks[tid][1] = -1;
    if (shared.cut_first[tid] >= 0) {
      // blocks that hold units of the segment: the one with unit x is ((x + 1) P - 1) / U
      const int c0 = static_cast<int>((static_cast<int64_t>(shared.cut_first[tid] + 1) * P - 1) / U);
      const int c1 = static_cast<int>((static_cast<int64_t>(shared.cut_first[tid] + shared.cut_at[tid].tiles) * P - 1) / U);
      // A block's end cuts one segment at most, so the first block of a segment names its counter.  The barrier
      // before and after makes the release and the acquire the whole block's.
      const uint32_t arrived = atom_add_acq_rel_gpu_u32(counters + c0, 1u);
      if (arrived == static_cast<uint32_t>(c1 - c0)) {
        counters[c0] = 0;
        shared.join_blocks[tid][0] = c0;
        shared.join_blocks[tid][1] = c1;
      }
    }
  }
  __syncthreads();
  for (int item = warp; item < 2 * kRows; item += kWarps) {
    const int side = item / kRows, r = item % kRows;
    const int c0 = shared.join_blocks[side][0], c1 = shared.join_blocks[side][1];
    if (c1 < 0 || r >= shared.cut_at[side].n * (a.Hq / a.cache.H)) continue;
    // the segment is the first block's last one and every other's first one
    const auto part_of = [&](int b) { return block_parts + (b * 2 + (b == c0 ? 1 : 0)) * C::kPart; };
    const int at = r * C::kPitch + lane * KvRow<D>::kCh, n = c1 - c0 + 1;
    const auto ml_of = [&](int i) {
      return i < n ? __ldcg(reinterpret_cast<const float4 *>(part_of(c0 + i) + kRows * C::kPitch + 4 * r))
                   : make_float4(kKvNoMax, 0.0f, 0.0f, 0.0f);
    };
    constexpr int kTogether = 4;  // the first parts' loads are under way with the weights'
    float v[kTogether][KvRow<D>::kCh];
    float4 ml = ml_of(lane);
#pragma unroll
    for (int x = 0; x < kTogether; ++x)
      if (x < n) row.template load<true>(part_of(c0 + x) + at, v[x]);
    row.clear();
    float top = ml.x;
    for (int i = 32; i < n; i += 32) top = fmaxf(top, ml_of(i + lane).x);
    row.top = row.max_lanes(top);
    float f = ex2(ml.x - row.top), sum = ml.y * f, plain = ml.z * f;
#pragma unroll
    for (int x = 0; x < kTogether; ++x) {
      const float fx = __shfl_sync(0xFFFFFFFFu, f, x);
      if (x < n) row.add(v[x], fx);
    }
    for (int i0 = 0; i0 < n; i0 += 32) {
      if (i0 > 0) {
        ml = ml_of(i0 + lane);
        f = ex2(ml.x - row.top);
        sum = fmaf(ml.y, f, sum);
        plain = fmaf(ml.z, f, plain);
      }
#pragma unroll 8
      for (int i = i0 > 0 ? i0 : kTogether; i < min(n, i0 + 32); ++i) {
        float u[KvRow<D>::kCh];
        row.template load<true>(part_of(c0 + i) + at, u);
        row.add(u, __shfl_sync(0xFFFFFFFFu, f, i & 31));
      }
    }
    row.sum = row.sum_lanes(sum);
    row.plain = row.sum_lanes(plain);
    row.write(a, shared.cut_at[side], r, lane);
  }
}

}  // namespace mixllm
