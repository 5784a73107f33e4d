// kv4_attention.cuh -- attention over the paged 4-bit KV cache.
//
//   o[i] = sum_t softmax_t(scale * q[i] . k[t]) v[t],  k = s (code - z), v alike,
// over the cached tokens t that query i sees.  Scale and zero point are per
// token and head, so both products run on the integers code - z (exact in
// fp16): the key's scale multiplies the score after the product, the value's
// scale the probability before it.
#pragma once

#include <cuda_fp16.h>
#include <atomic>
#include <cstdint>

#include "gemm_w4w8a8.cuh"  // device_sm_count
#include "kv4_cache.cuh"
#include "launch.h"
#include "ptx_sm100.cuh"

namespace mixllm {

// ---------------------------------------------------------------------------
// Few queries per request (decode).  HBM-bound: 2 * (D/2 + 4) bytes per cached
// token and head.
//
// Work is cut into units of 128 tokens of one (request, row tile, key head);
// block c takes the units [c U / P, (c + 1) U / P) of their concatenation, so
// requests of any lengths load every SM alike, and the lengths stay on the
// device.  A row tile is 8 NT rows (query token, query head of the group).
// Within a block a producer warp copies each unit's codes and metadata into a
// ring of stages by bulk copies, one per page and array, and eight warps take
// 16 tokens each.  Tokens are the 16-row side of m16n8k16 and the query rows
// its 8-column side, so that a group of 8 heads fills the instruction and
// smaller ones waste only tensor work: S^T = K Q^T with K as the A operand,
// then O^T = V^T P^T with V^T as A.  The codes go from shared memory to the A
// registers without a shuffle:
//   * K: any permutation of the channels serves as long as Q has the same, so
//     a lane takes D/4 consecutive channels of a token and pairs nibbles i and
//     i + 4 of a word, which one AND brings to fp16 form (0x6400 | n is
//     1024 + n; a high nibble gives 1024 + 16 n and is scaled by 1/16 in the
//     FMA that subtracts the zero point);
//   * V: lane (g, t) takes channels g D/8 .. of four tokens; a byte permute
//     joins the halves of two tokens' words into (token, token') pairs.  The
//     output channel of an accumulator is then the lane's own channel range.
// P^T goes from accumulator to B layout by movmatrix.
//
// Softmax per warp with lazy rescaling: the running maximum m moves only when
// a score passes it by more than 8 (in log2 units), so p <= 2^8.  The values'
// scales pass through fp16 together with p, as p * s_v / S with S the running
// maximum of s_v (moved when passed by a factor of 4); the accumulators hold
// O / S.  p s_v is rounded once, to fp16's 11 bits; sums stay in fp32.
//
// At a segment's end the eight warps' (m, S, l, O) are joined in shared
// memory; a segment cut between blocks leaves its parts in the workspace and
// the last block to arrive adds them in the order of the tokens, so the result
// does not depend on timing.
// ---------------------------------------------------------------------------
constexpr int kKvTile = 128;       // tokens per unit
constexpr int kKvWarps = kKvTile / 16;
constexpr int kKvThreads = 32 * (kKvWarps + 1);
constexpr int kKvMaxPieces = kKvTile / 16;  // pages of a unit at the smallest page
constexpr float kKvNoMax = -3.0e38f;

template <int D, int NT>
struct KvCfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kRowBytes = D / 2;
  static constexpr int kCodes = kKvTile * kRowBytes;  // bytes of one unit's key (or value) codes
  static constexpr int kMeta = kKvTile * 4;
  static constexpr int kStage = 2 * (kCodes + kMeta);
  static constexpr int kPitch = D + 4;  // floats per row of the join buffer
  static constexpr int kJoin = kKvWarps * kRows * kPitch * 4;
  static constexpr int kStages = NT == 1 ? 4 : 5;
  static constexpr int kBlocksPerSm = NT == 1 ? 2 : 1;
  static constexpr int kSmem = kStages * kStage + kJoin + 2 * kKvWarps * kRows * 4;
};
constexpr int kKvMaxGrid = 2 * 148;

// One request's share of the work.
struct KvReq {
  int q0, n, kv, tiles, row_tiles;
};

// Reads and checks one request's lengths.  Anything out of range (a device
// value the host cannot see) is recorded and the request skipped.
__device__ __forceinline__ KvReq kv_req(const AttendArgs &a, int b, int rows_per_tile) {
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

// Walks a block's units as segments: runs of units of one (request, row tile,
// key head).
struct KvWalk {
  int b, rt, h, tile, count;  // the segment: its first unit's tile and its units in this block
  int64_t left;               // units of the block from the segment's first on
  int64_t seg_first;          // unit index of the whole segment's first tile
  KvReq r;

  __device__ __forceinline__ void settle(const AttendArgs &a, int rows_per_tile) {
    while (left > 0 && r.tiles == 0 && ++b < a.B) r = kv_req(a, b, rows_per_tile);
    if (b >= a.B) left = 0;
    count = static_cast<int>(left < r.tiles - tile ? left : r.tiles - tile);
  }
  __device__ __forceinline__ void next(const AttendArgs &a, int rows_per_tile) {
    left -= count;
    seg_first += r.tiles;
    tile = 0;
    if (++h == a.cache.H) {
      h = 0;
      if (++rt == r.row_tiles) {
        rt = 0;
        if (++b < a.B && left > 0) r = kv_req(a, b, rows_per_tile);
      }
    }
    settle(a, rows_per_tile);
  }
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// Two nibbles of w at bits 0 and 16 (low) or 4 and 20 (high) as fp16 integers
// minus the zero points in c: exact (integers below 2048, and multiples of
// 1/16 below 128).
__device__ __forceinline__ uint32_t nib_lo(uint32_t w, uint32_t c) {
  const uint32_t x = (w & 0x000F000Fu) | 0x64006400u;
  uint32_t r;
  asm("add.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t nib_hi(uint32_t w, uint32_t c) {
  const uint32_t x = (w & 0x00F000F0u) | 0x64006400u;
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0x2C002C00u), "r"(c));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float meta_scale(uint32_t m) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(m & 0xFFFFu)));
}

template <int D, int NT>
__global__ void __launch_bounds__(kKvThreads, KvCfg<D, NT>::kBlocksPerSm) kv4_decode_kernel(const AttendArgs a,
                                                                                          uint32_t *__restrict__ counters,
                                                                                          float *__restrict__ parts) {
  using C = KvCfg<D, NT>;
  constexpr int kRows = C::kRows;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *ring = smem;
  float *join = reinterpret_cast<float *>(smem + C::kStages * C::kStage);
  float *join_m = join + kKvWarps * kRows * C::kPitch, *join_l = join_m + kKvWarps * kRows;
  __shared__ uint64_t full[C::kStages], empty[C::kStages];
  __shared__ uint32_t present[C::kStages];  // bit j: piece j of the stage was copied
  __shared__ volatile int abort_flag;
  __shared__ int first_b, last_here;
  __shared__ long long first_rem, warp_units[kKvWarps + 1];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = a.Hq / a.cache.H, page_log2 = a.cache.page_log2;
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kKvWarps);
    }
    fence_mbar_init();
    abort_flag = 0;
    first_b = a.B;
  }
  __syncthreads();

  // ---- this block's units
  int P = gridDim.x;
  const int c = blockIdx.x;
  int64_t U = 0, start = 0;
  auto units_of = [&](const KvReq &r) { return static_cast<long long>(r.tiles) * r.row_tiles * a.cache.H; };
  for (int pass = 0; pass < 2; ++pass) {
    int64_t base = 0;
    for (int b0 = 0; b0 < a.B; b0 += kKvThreads) {
      const int b = b0 + tid;
      const long long u = b < a.B ? units_of(kv_req(a, b, kRows)) : 0;
      long long incl = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) warp_units[warp] = incl;
      __syncthreads();
      long long before = base;
      for (int w = 0; w <= kKvWarps; ++w) {
        if (w < warp) before += warp_units[w];
        base += warp_units[w];
      }
      incl += before;
      if (pass == 1 && u > 0 && start >= incl - u && start < incl) {
        first_b = b;
        first_rem = start - (incl - u);
      }
      __syncthreads();
      if (pass == 1 && base > start) break;
    }
    if (pass == 0) {
      U = base;
      if (U < P) P = static_cast<int>(U);  // every block that takes part has a unit
      if (c >= P) return;
      start = U / P * c + U % P * c / P;
    }
  }
  const int64_t end = U / P * (c + 1) + U % P * (c + 1) / P;
  KvWalk w0;
  w0.b = first_b;
  w0.left = end - start;
  if (w0.left <= 0 || w0.b >= a.B) return;
  w0.r = kv_req(a, w0.b, kRows);
  {
    const int64_t per_rt = static_cast<int64_t>(w0.r.tiles) * a.cache.H;
    w0.rt = static_cast<int>(first_rem / per_rt);
    const int64_t rem = first_rem - w0.rt * per_rt;
    w0.h = static_cast<int>(rem / w0.r.tiles);
    w0.tile = static_cast<int>(rem - static_cast<int64_t>(w0.h) * w0.r.tiles);
  }
  w0.seg_first = start - w0.tile;
  w0.settle(a, kRows);

  if (warp == kKvWarps) {
    // ------------------------------------------------------------ producer
    const int page = 1 << page_log2;
    const int piece = page < kKvTile ? page : kKvTile;  // tokens per copy
    const int pieces = kKvTile / piece;
    const uint32_t piece_bytes = 2u * piece * (C::kRowBytes + 4);
    const int64_t page_rows = static_cast<int64_t>(a.cache.H) << page_log2;
    int stage = 0;
    uint32_t phase = 0, issued = 0;
    for (KvWalk w = w0; w.left > 0; w.next(a, kRows)) {
      const int used = (w.r.kv + page - 1) >> page_log2;
      const int32_t *table = a.table + static_cast<int64_t>(w.b) * a.table_stride;
      // the page numbers of 32 pieces at a time, one per lane
      int batch = -1, id = -1;
      for (int i = 0; i < w.count; ++i) {
        const int tile = w.tile + i;
        const int first = tile * pieces;  // in pieces of the segment
        if (first / 32 != batch) {
          batch = first / 32;
          const int64_t token = (static_cast<int64_t>(batch) * 32 + lane) * piece;
          const int64_t entry = token >> page_log2;
          id = -1;
          if (entry < used) {
            id = table[entry];
            if (id < 0 || id >= a.cache.pages) {
              record_status(kStatusBounds);
              id = -1;
            }
          }
        }
        warp_wait(&empty[stage], phase ^ 1, &abort_flag);
        // pieces divides 32, so a unit's pieces lie in one batch
        const int src_lane = (first & 31) + (lane >> 2);
        const int my_id = __shfl_sync(0xFFFFFFFFu, id, src_lane & 31);
        const bool mine = (lane >> 2) < pieces && my_id >= 0 && !abort_flag;
        const uint32_t have = __ballot_sync(0xFFFFFFFFu, mine);  // four lanes per piece
        if (lane == 0) {
          uint32_t bits = 0;
          for (int j = 0; j < kKvMaxPieces; ++j) bits |= (have >> (4 * j) & 1u) << j;
          present[stage] = bits;
          mbar_arrive_expect_tx(&full[stage], piece_bytes * __popc(bits));
        }
        __syncwarp();
        if (mine) {
          const int j = lane >> 2, what = lane & 3;  // key codes, value codes, key meta, value meta
          const int kv = what & 1;
          const int row = static_cast<int>((static_cast<int64_t>(tile) * kKvTile + j * piece) & (page - 1));
          const int64_t at = (static_cast<int64_t>(my_id) * 2 + kv) * page_rows + (static_cast<int64_t>(w.h) << page_log2) + row;
          uint8_t *dst = ring + stage * C::kStage;
          if (what < 2)
            bulk_load(dst + kv * C::kCodes + j * piece * C::kRowBytes, a.cache.codes + at * C::kRowBytes,
                      piece * C::kRowBytes, &full[stage]);
          else
            bulk_load(dst + 2 * C::kCodes + kv * C::kMeta + j * piece * 4, a.cache.meta + at, piece * 4, &full[stage]);
        }
        ++issued;
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (abort_flag) {  // a wait gave up: let the copies in flight land before the block ends
      for (uint32_t i = issued > C::kStages ? issued - C::kStages : 0; i < issued; ++i)
        mbar_wait_drain(&full[i % C::kStages], (i / C::kStages) & 1, 1ll << 28);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = lane >> 2, t = lane & 3;
  // accumulator row r of the score tile is token r ^ (r >> 1 & 1): the value
  // rows that four lanes read together then alternate in the 32 banks
  const int row_a = 16 * warp + (g ^ (g >> 1 & 1)), row_b = row_a + 8;
  const int vr0 = 16 * warp + ((2 * t) ^ (t & 1)), vr1 = 16 * warp + ((2 * t + 1) ^ (t & 1));
  constexpr int kWords = D / 32;   // words of a lane's key chunk
  constexpr int kMTiles = D / 16;  // 16-channel tiles of O^T
  const float scale2 = a.scale * 1.4426950408889634f;
  int stage = 0;
  uint32_t phase = 0;

  for (KvWalk w = w0; w.left > 0; w.next(a, kRows)) {
    const int rows = w.r.n * group;
    const int row0 = w.rt * kRows;
    // ---- the query rows' B fragments, channels permuted as the keys' nibbles
    uint32_t qf[NT][kWords * 4];
    int lim[NT][2];  // keys seen by columns 2t and 2t + 1
#pragma unroll
    for (int ni = 0; ni < NT; ++ni) {
      const int r = row0 + ni * 8 + g;
      const __half *src = nullptr;
      if (r < rows) {
        const int tok = r / group;
        src = a.q + (static_cast<int64_t>(w.r.q0) + tok) * a.q_stride + (w.h * group + (r - tok * group)) * D + t * (D / 4);
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (src) v = *reinterpret_cast<const uint4 *>(src + 8 * i);
        qf[ni][4 * i + 0] = __byte_perm(v.x, v.z, 0x5410);
        qf[ni][4 * i + 1] = __byte_perm(v.x, v.z, 0x7632);
        qf[ni][4 * i + 2] = __byte_perm(v.y, v.w, 0x5410);
        qf[ni][4 * i + 3] = __byte_perm(v.y, v.w, 0x7632);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int rj = row0 + ni * 8 + 2 * t + j;
        lim[ni][j] = a.causal && rj < rows ? w.r.kv - w.r.n + rj / group + 1 : w.r.kv;
      }
    }
    // keys seen by the tile's first row (the fewest) and last row (the most)
    const int lim_min = a.causal ? w.r.kv - w.r.n + row0 / group + 1 : w.r.kv;
    const int last_row = min(rows, row0 + kRows) - 1;
    const int lim_max = a.causal ? w.r.kv - w.r.n + last_row / group + 1 : w.r.kv;

    float o[NT][kMTiles][4];
    float m[NT][2], l[NT][2];
    float S = 0x1p-24f, inv_S = 0x1p24f;
#pragma unroll
    for (int ni = 0; ni < NT; ++ni) {
      m[ni][0] = m[ni][1] = kKvNoMax;
      l[ni][0] = l[ni][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < kMTiles; ++i) o[ni][i][0] = o[ni][i][1] = o[ni][i][2] = o[ni][i][3] = 0.0f;
    }

    for (int i = 0; i < w.count; ++i) {
      const int base = (w.tile + i) * kKvTile;
      warp_wait(&full[stage], phase, &abort_flag);
      const uint8_t *st = ring + stage * C::kStage;
      const uint8_t *vs = st + C::kCodes;
      const uint32_t *km = reinterpret_cast<const uint32_t *>(st + 2 * C::kCodes), *vm = km + kKvTile;
      const uint32_t have = present[stage];
      uint32_t ka[kWords], kb[kWords], v0[kWords / 2], v1[kWords / 2], v2[kWords / 2], v3[kWords / 2];
      if constexpr (D == 128) {
        *reinterpret_cast<uint4 *>(ka) = *reinterpret_cast<const uint4 *>(st + row_a * C::kRowBytes + t * 16);
        *reinterpret_cast<uint4 *>(kb) = *reinterpret_cast<const uint4 *>(st + row_b * C::kRowBytes + t * 16);
        *reinterpret_cast<uint2 *>(v0) = *reinterpret_cast<const uint2 *>(vs + vr0 * C::kRowBytes + g * 8);
        *reinterpret_cast<uint2 *>(v1) = *reinterpret_cast<const uint2 *>(vs + vr1 * C::kRowBytes + g * 8);
        *reinterpret_cast<uint2 *>(v2) = *reinterpret_cast<const uint2 *>(vs + (vr0 + 8) * C::kRowBytes + g * 8);
        *reinterpret_cast<uint2 *>(v3) = *reinterpret_cast<const uint2 *>(vs + (vr1 + 8) * C::kRowBytes + g * 8);
      } else {
        *reinterpret_cast<uint2 *>(ka) = *reinterpret_cast<const uint2 *>(st + row_a * C::kRowBytes + t * 8);
        *reinterpret_cast<uint2 *>(kb) = *reinterpret_cast<const uint2 *>(st + row_b * C::kRowBytes + t * 8);
        v0[0] = *reinterpret_cast<const uint32_t *>(vs + vr0 * C::kRowBytes + g * 4);
        v1[0] = *reinterpret_cast<const uint32_t *>(vs + vr1 * C::kRowBytes + g * 4);
        v2[0] = *reinterpret_cast<const uint32_t *>(vs + (vr0 + 8) * C::kRowBytes + g * 4);
        v3[0] = *reinterpret_cast<const uint32_t *>(vs + (vr1 + 8) * C::kRowBytes + g * 4);
      }
      const uint32_t kma = km[row_a], kmb = km[row_b], vma = vm[row_a], vmb = vm[row_b];
      const uint32_t z0 = vm[vr0] >> 16 & 15u, z1 = vm[vr1] >> 16 & 15u;
      const uint32_t z2 = vm[vr0 + 8] >> 16 & 15u, z3 = vm[vr1 + 8] >> 16 & 15u;
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1;
      }
      if (base + 16 * warp >= lim_max) continue;  // nothing of these 16 tokens is seen

      // ---- scores
      float sc[NT][4];
#pragma unroll
      for (int ni = 0; ni < NT; ++ni) sc[ni][0] = sc[ni][1] = sc[ni][2] = sc[ni][3] = 0.0f;
      {
        const uint32_t za = kma >> 16 & 15u, zb = kmb >> 16 & 15u;
        const uint32_t la = 0xE400E400u | za * 0x00010001u, ha = 0xD400D400u | za * 0x00100010u;
        const uint32_t lb = 0xE400E400u | zb * 0x00010001u, hb = 0xD400D400u | zb * 0x00100010u;
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          const uint32_t a0 = nib_lo(ka[j], la), a2 = nib_hi(ka[j], ha);
          const uint32_t a1 = nib_lo(kb[j], lb), a3 = nib_hi(kb[j], hb);
          const uint32_t xa = ka[j] >> 8, xb = kb[j] >> 8;
          const uint32_t b0 = nib_lo(xa, la), b2 = nib_hi(xa, ha);
          const uint32_t b1 = nib_lo(xb, lb), b3 = nib_hi(xb, hb);
#pragma unroll
          for (int ni = 0; ni < NT; ++ni) {
            mma_f16(sc[ni], a0, a1, a2, a3, qf[ni][4 * j], qf[ni][4 * j + 1]);
            mma_f16(sc[ni], b0, b1, b2, b3, qf[ni][4 * j + 2], qf[ni][4 * j + 3]);
          }
        }
      }
      const float fa = meta_scale(kma) * scale2, fb = meta_scale(kmb) * scale2;
      float sva = meta_scale(vma), svb = meta_scale(vmb);
#pragma unroll
      for (int ni = 0; ni < NT; ++ni) {
        sc[ni][0] *= fa, sc[ni][1] *= fa;
        sc[ni][2] *= fb, sc[ni][3] *= fb;
      }
      const bool whole = base + kKvTile <= lim_min && have == (1u << (kKvTile >> min(page_log2, 7))) - 1u;
      if (!whole) {
        const int ta = base + row_a, tb = base + row_b;
        const int shift = min(page_log2, 7);
        const bool pa = have >> (row_a >> shift) & 1u, pb = have >> (row_b >> shift) & 1u;
#pragma unroll
        for (int ni = 0; ni < NT; ++ni)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (!pa || ta >= lim[ni][j]) sc[ni][j] = -INFINITY;
            if (!pb || tb >= lim[ni][j]) sc[ni][2 + j] = -INFINITY;
          }
        // rows that no query may see hold anything: keep their scales out of S and of 0 * NaN
        if (!pa || ta >= lim_max) sva = 0.0f;
        if (!pb || tb >= lim_max) svb = 0.0f;
      }
      // ---- running maximum
      bool move = fmaxf(sva, svb) > 4.0f * S;
#pragma unroll
      for (int ni = 0; ni < NT; ++ni)
#pragma unroll
        for (int j = 0; j < 2; ++j) move |= fmaxf(sc[ni][j], sc[ni][2 + j]) > m[ni][j] + 8.0f;
      if (__any_sync(0xFFFFFFFFu, move)) {
        float s_new = fmaxf(S, fmaxf(sva, svb));
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) s_new = fmaxf(s_new, __shfl_xor_sync(0xFFFFFFFFu, s_new, x));
        const float down = __fdividef(S, s_new);
        S = s_new;
        inv_S = __fdividef(1.0f, S);
#pragma unroll
        for (int ni = 0; ni < NT; ++ni)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float mx = fmaxf(m[ni][j], fmaxf(sc[ni][j], sc[ni][2 + j]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, x));
            const float keep = ex2(m[ni][j] - mx);
            m[ni][j] = mx;
            l[ni][j] *= keep;
#pragma unroll
            for (int k = 0; k < kMTiles; ++k) {
              o[ni][k][j] *= keep * down;
              o[ni][k][2 + j] *= keep * down;
            }
          }
      }
      // ---- probabilities
      const float wa = sva * inv_S, wb = svb * inv_S;
      uint32_t pf[NT][2];
#pragma unroll
      for (int ni = 0; ni < NT; ++ni) {
        float p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = ex2(sc[ni][j] - m[ni][j & 1]);
        l[ni][0] += p[0] + p[2];
        l[ni][1] += p[1] + p[3];
        p[0] *= wa, p[1] *= wa;
        p[2] *= wb, p[3] *= wb;
        if (!whole) {  // a scale may be NaN: no product with the zero of a key that is not seen
#pragma unroll
          for (int j = 0; j < 4; ++j) p[j] = sc[ni][j] == -INFINITY ? 0.0f : p[j];
        }
        pf[ni][0] = transpose8x8(half2_bits(p[0], p[1]));
        pf[ni][1] = transpose8x8(half2_bits(p[2], p[3]));
      }
      // ---- values
      {
        const uint32_t l01 = 0xE400E400u | z0 | z1 << 16, h01 = 0xD400D400u | z0 << 4 | z1 << 20;
        const uint32_t l23 = 0xE400E400u | z2 | z3 << 16, h23 = 0xD400D400u | z2 << 4 | z3 << 20;
#pragma unroll
        for (int j = 0; j < kWords / 2; ++j) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t x01 = __byte_perm(v0[j], v1[j], half ? 0x7632 : 0x5410);
            uint32_t x23 = __byte_perm(v2[j], v3[j], half ? 0x7632 : 0x5410);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint32_t a0 = nib_lo(x01, l01), a1 = nib_hi(x01, h01);
              const uint32_t a2 = nib_lo(x23, l23), a3 = nib_hi(x23, h23);
              const int k = 4 * j + 2 * half + q;
#pragma unroll
              for (int ni = 0; ni < NT; ++ni) mma_f16(o[ni][k], a0, a1, a2, a3, pf[ni][0], pf[ni][1]);
              x01 >>= 8;
              x23 >>= 8;
            }
          }
        }
      }
    }

    // ---- join the warps: each brings (m, l, S O) per row
#pragma unroll
    for (int ni = 0; ni < NT; ++ni)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float sum = l[ni][j];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
        const int r = ni * 8 + 2 * t + j;
        if (g == 0) {
          join_m[warp * kRows + r] = m[ni][j];
          join_l[warp * kRows + r] = sum;
        }
        float *dst = join + (warp * kRows + r) * C::kPitch + g * (D / 8);
#pragma unroll
        for (int k = 0; k < kMTiles; k += 2)
          *reinterpret_cast<float4 *>(dst + 2 * k) =
              make_float4(o[ni][k][j] * S, o[ni][k][2 + j] * S, o[ni][k + 1][j] * S, o[ni][k + 1][2 + j] * S);
      }
    named_bar_sync(1, 32 * kKvWarps);
    const bool cut = w.count < w.r.tiles;
    const int64_t seg_end = w.seg_first + w.r.tiles;
    // parts of the segment: the blocks that hold units of it
    const auto block_of = [&](int64_t u) { return static_cast<int>(((u + 1) * P - 1) / U); };
    const auto block_start = [&](int b) { return U / P * b + U % P * b / P; };
    const int part_floats = kRows * (D + 2);
    const auto part_of = [&](int b) {
      return parts + (static_cast<int64_t>(b) * 2 + (block_start(b) <= w.seg_first ? 1 : 0)) * part_floats;
    };
    constexpr int kLanesPerRow = 32 * kKvWarps / kRows;  // threads of one row
    constexpr int kCh = D / kLanesPerRow;                // channels of one thread
    const int r = tid / kLanesPerRow, d0 = (tid % kLanesPerRow) * kCh;
    float mx = kKvNoMax, sum = 0.0f, acc[kCh];
#pragma unroll
    for (int k = 0; k < kCh; ++k) acc[k] = 0.0f;
    for (int x = 0; x < kKvWarps; ++x) mx = fmaxf(mx, join_m[x * kRows + r]);
    for (int x = 0; x < kKvWarps; ++x) {
      const float f = ex2(join_m[x * kRows + r] - mx);
      sum += join_l[x * kRows + r] * f;
#pragma unroll
      for (int k = 0; k < kCh; ++k) acc[k] += join[(x * kRows + r) * C::kPitch + d0 + k] * f;
    }
    bool writes = true;
    if (cut) {
      float *mine = part_of(c);
#pragma unroll
      for (int k = 0; k < kCh; ++k) mine[r * D + d0 + k] = acc[k];
      if (d0 == 0) mine[kRows * D + 2 * r] = mx, mine[kRows * D + 2 * r + 1] = sum;
      const int c0 = block_of(w.seg_first), c1 = block_of(seg_end - 1);
      __threadfence();
      named_bar_sync(1, 32 * kKvWarps);
      if (tid == 0) {
        // a block's end cuts one segment at most, so the first block of a segment names its counter
        const uint32_t before = atom_add_acq_rel_gpu_u32(counters + c0, 1u);
        last_here = before == static_cast<uint32_t>(c1 - c0);
        if (last_here) counters[c0] = 0;
      }
      named_bar_sync(1, 32 * kKvWarps);
      writes = last_here;
      if (writes) {
        __threadfence();
        mx = kKvNoMax, sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kCh; ++k) acc[k] = 0.0f;
        for (int b = c0; b <= c1; ++b) mx = fmaxf(mx, __ldcg(part_of(b) + kRows * D + 2 * r));
        for (int b = c0; b <= c1; ++b) {
          const float *p = part_of(b);
          const float f = ex2(__ldcg(p + kRows * D + 2 * r) - mx);
          sum += __ldcg(p + kRows * D + 2 * r + 1) * f;
#pragma unroll
          for (int k = 0; k < kCh; ++k) acc[k] += __ldcg(p + r * D + d0 + k) * f;
        }
      }
    }
    if (writes && row0 + r < rows) {
      const int tok = (row0 + r) / group, head = w.h * group + (row0 + r) % group;
      const int64_t token = static_cast<int64_t>(w.r.q0) + tok;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // a row that saw no key is zero
      __half *dst = a.out + token * a.out_stride + static_cast<int64_t>(head) * D + d0;
#pragma unroll
      for (int k = 0; k < kCh; k += 2)
        *reinterpret_cast<__half2 *>(dst + k) = __floats2half2_rn(acc[k] * inv, acc[k + 1] * inv);
      if (a.lse && d0 == 0)
        a.lse[token * a.Hq + head] = sum == 0.0f ? -INFINITY : (mx + log2f(sum)) * 0.6931471805599453f;
    }
    named_bar_sync(1, 32 * kKvWarps);  // the join buffer is free again
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Two n-tiles of rows when a request's rows do not fit one.
static int kv4_decode_nt(int max_q, int group) { return static_cast<int64_t>(max_q) * group > 8 ? 2 : 1; }

// Workspace: one counter per block, always in the same place, then the parts
// of cut segments (two per block), which need no initial value.
constexpr size_t kKvCounterBytes = 4096;
static_assert(kKvMaxGrid * sizeof(uint32_t) <= kKvCounterBytes, "one counter per block");

size_t kv4_attention_workspace_bytes(int, int max_q, int Hq, int H, int D, int, int) {
  const int rows = 8 * kv4_decode_nt(max_q, Hq / H);
  return kKvCounterBytes + static_cast<size_t>(kKvMaxGrid) * 2 * rows * (D + 2) * sizeof(float);
}

template <int D, int NT>
static cudaError_t launch_kv4_decode(const AttendArgs &a, void *ws, cudaStream_t stream,
                                     const char **msg) {
  using C = KvCfg<D, NT>;
  auto kern = kv4_decode_kernel<D, NT>;
  static std::atomic<unsigned long long> configured{0};  // one bit per device ordinal
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !(configured.load() & (1ull << dev))) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) {
      *msg = "cudaFuncSetAttribute(MaxDynamicSharedMemorySize) failed";
      return e;
    }
    if (dev < 64) configured.fetch_or(1ull << dev);
  }
  // one wave of blocks, fewer when even the longest contexts have fewer units
  const int64_t tiles = ((static_cast<int64_t>(a.W) << a.cache.page_log2) + kKvTile - 1) / kKvTile;
  const int64_t row_tiles = (static_cast<int64_t>(a.max_q) * (a.Hq / a.cache.H) + C::kRows - 1) / C::kRows;
  const int64_t units = a.B * row_tiles * a.cache.H * (tiles > 0 ? tiles : 1);
  int64_t grid = static_cast<int64_t>(device_sm_count()) * C::kBlocksPerSm;
  if (grid > kKvMaxGrid) grid = kKvMaxGrid;
  if (grid > units) grid = units;
  kern<<<static_cast<unsigned>(grid), kKvThreads, C::kSmem, stream>>>(
      a, static_cast<uint32_t *>(ws), reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kKvCounterBytes));
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) *msg = "launch of the decode attention failed";
  return e;
}

cudaError_t launch_kv4_attention(const AttendArgs &a, void *ws, cudaStream_t stream, const char **msg) {
  const bool one = kv4_decode_nt(a.max_q, a.Hq / a.cache.H) == 1;
  if (a.cache.D == 128)
    return one ? launch_kv4_decode<128, 1>(a, ws, stream, msg) : launch_kv4_decode<128, 2>(a, ws, stream, msg);
  return one ? launch_kv4_decode<64, 1>(a, ws, stream, msg) : launch_kv4_decode<64, 2>(a, ws, stream, msg);
}

}  // namespace mixllm
