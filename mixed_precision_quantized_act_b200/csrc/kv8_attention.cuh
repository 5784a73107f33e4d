// kv8_attention.cuh -- attention over the paged 8-bit KV cache.
//
//   o[i] = sum_t softmax_t(scale * q[i] . k[t]) v[t],  k = s (code - 128), v alike,
// over the cached tokens t that query i sees.  A block of 16 tokens of a head has
// one scale for its keys and one for its values, so both products run on the
// whole numbers code - 128 (exact in fp16): the keys' scale multiplies the scores
// after the product, the values' scale the probabilities before it.
#pragma once

#include <cuda_fp16.h>
#include <atomic>
#include <cstdint>

#include "gemm_w4w8a8.cuh"  // device_sm_count
#include "kv4_prompt.cuh"
#include "kv4_ptx.cuh"
#include "kv8_cache.cuh"
#include "kv_split.cuh"
#include "launch.h"
#include "ptx_sm100.cuh"

namespace mixllm {

// ---------------------------------------------------------------------------
// Few queries per request (decode: up to 16 rows of query token and query head
// per key head).  HBM-bound: 2 (D + 1/4) bytes per cached token and head.
//
// Units of 32 tokens, two blocks of 16, shared among warps and blocks as
// kv_split.cuh says.  Tokens are the 16-row side of m16n8k16 and the query rows
// its 8-column side (NT such tiles): S^T = K Q^T with K as the A operand, then
// O^T = V^T P^T with V^T as A.
//
// Unpacking: a byte permute puts a code behind 0x64, which is 1024 + code as
// fp16, and a half-precision add takes 1152 off: exact.
//   * K: any permutation of the channels serves as long as Q has the same: a
//     lane takes D/4 consecutive channels of a token, a word's four codes in order.
//   * V: lane (g, t) takes channels g D/8 .. of four tokens; byte permutes join the
//     words of two tokens into (token, token') pairs first.
// P^T goes from accumulator to B layout by movmatrix.  The stages in shared
// memory keep a row's 16-byte chunks permuted, so that the lanes that read
// together meet every bank once.
//
// Softmax per warp with lazy rescaling.  The values' scales pass through fp16
// together with p, as weights p s_v = 2^(score + log2 s_v - m).  A row's reference m
// is 7 (in log2 units) below its largest weight so far among the keys that it
// sees, a scale counting as 2^-40 at least so that the sum of p stays finite, and
// moves only when a weight passes 2^15: weights down to 2^-21 of the largest are
// normal numbers.  A weight is rounded once, to fp16's 11 bits, and O is divided
// by the sum of p as that rounding leaves it, where the block's scale is not far
// below the largest, S (a weight that is an fp16 subnormal says little about p).
// Sums stay in fp32.
//
// Measured on B200 (as a CUDA graph): 64 requests of 100 to 8100 tokens, 32 query and
// 8 key heads of 128: 102 us, 5.3 TB/s (81 % of the measured copy rate; the loops take
// 82 us of it, at that rate, the rest is the first loads, SMs that end 10 us apart, and
// the joins); 4 requests of 100000 to 131071 tokens, 64 and 8 heads: 164 us, 5.9 TB/s
// (90 %); one request of 1003 tokens: 9.4 us.
// ---------------------------------------------------------------------------
constexpr float kKv8LeastScale = 0x1p-40f;

template <int D, int NT>
struct Kv8Cfg {
  static constexpr int kWarps = 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRows = 8 * NT;
  static constexpr int kLeast = 1;  // units of a warp
  static constexpr bool kWholeHeads = true;
  static constexpr int kCodes = 32 * D;  // bytes of 32 tokens' key (or value) codes
  static constexpr int kStage = 2 * kCodes + 16;  // and two blocks' (key, value) scales
  // One unit a warp under way beside the one at work (64 KB a block), with 64 channels two.  With twice that the memory
  // system serves some SMs (always the same ones) 15 % slower than others, and their blocks end last: 4 requests of
  // 100000 to 131071 tokens took 175 us then, 164 so; 64 of 100 to 8100 109 and 102.
  static constexpr int kStages = D == 128 ? 2 : 3;
  static constexpr int kRing = kStages * kStage;  // of one warp
  static constexpr int kPitch = D + 8;            // floats of a part's row: two rows further, 16 banks further
  static constexpr int kPart = kRows * (kPitch + 4);  // floats of one part: sums, then m, the two sums of p per row
  static constexpr int kSmem = kWarps * kRing;

  // Row r of a block keeps its chunk c of 16 bytes at c ^ key_at(r), c ^ value_at(r).
  static __device__ __forceinline__ constexpr int key_at(int r) { return D == 128 ? r & 1 : 0; }
  static __device__ __forceinline__ constexpr int value_at(int r) { return D == 128 ? r & 6 : r >> 1 & 2; }
  // Half a warp copies a block of 16 tokens, which lies in one page.
  static __device__ __forceinline__ uint32_t lane_bytes(int lane) { return (lane >> 4) * (16 * D); }
  static __device__ __forceinline__ void copy(const Kv8Cache &c, int lane, int64_t at, int64_t to_value, uint32_t dst) {
    constexpr int kChunks = D / 16;
    const int i = lane & 15;
    const uint8_t *k = c.codes + at * D + i * 16, *v = k + to_value * D;
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
      const int r = j * (16 / kChunks) + i / kChunks, chunk = i % kChunks;
      cp_async_16_u32(dst + r * D + ((chunk ^ key_at(r)) << 4), k + j * 256);
      cp_async_16_u32(dst + kCodes + r * D + ((chunk ^ value_at(r)) << 4), v + j * 256);
    }
    if (i < 2) {
      const uint32_t to = dst - lane_bytes(lane) + 2 * kCodes + (lane >> 4) * 8 + i * 4;
      cp_async_4_u32(to, c.scales + ((at + (i ? to_value : 0)) >> 4));
    }
  }
  static_assert(kWarps * kPart * 4 <= kSmem, "the warps' last parts take the ring's place");
  static_assert(kSmem + 4096 <= 227 * 1024, "shared memory of a block");
};

// Two codes, bytes 2i and 2i + 1 of w, as fp16 whole numbers code - 128.
__device__ __forceinline__ uint32_t codes_f16(uint32_t w, uint32_t bytes) {
  uint32_t r;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(__byte_perm(w, 0x64646464u, bytes)), "r"(0x64806480u));
  return r;
}
constexpr uint32_t kLowPair = 0x4140u, kHighPair = 0x4342u;

template <int D, int NT>
__global__ void __launch_bounds__(Kv8Cfg<D, NT>::kThreads, 1) kv8_decode_kernel(const Attend8Args a, uint32_t *counters,
                                                                                float *block_parts, float *warp_parts) {
  using C = Kv8Cfg<D, NT>;
  constexpr int kRows = C::kRows, kWarps = C::kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ KvShared<kWarps> shared;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = blockIdx.x;
  const int group = a.Hq / a.cache.H;
  pdl_launch_dependents();
  if (tid < 2) shared.cut_first[tid] = -1;
  if (lane < 2) shared.part_first[warp][lane] = -1;
  pdl_wait();

  KvShare my;
  KvWalk w0;
  if (!kv_first_units<C>(a, shared, my, w0)) return;
  KvFetch<C> fetch;
  fetch.start(w0, lane, smem + warp * C::kRing);
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) fetch.unit(a, lane);

  const int g = lane >> 2, t = lane & 3;
  // accumulator row r of the score tile is token r ^ (r >> 1 & 1): with 64 channels, the value rows that four lanes
  // read together then lie in both halves of the 32 banks
  const int row_a = g ^ (g >> 1 & 1);
  const int vr0 = (2 * t) ^ (t & 1), vr1 = (2 * t + 1) ^ (t & 1);
  constexpr int kWords = D / 16;   // words of a lane's key chunk
  constexpr int kMTiles = D / 16;  // 16-channel tiles of O^T
  // this lane's 16 (or 8) bytes of a value row, the same place in all four
  const int v_at = D == 128 ? (g ^ C::value_at(vr0)) << 4 : (((g >> 1) ^ C::value_at(vr0)) << 4) + (g & 1) * 8;
  const float scale2 = a.scale * 1.4426950408889634f;  // to log2 units
  const uint8_t *ring = smem + warp * C::kRing;
  int stage = 0;

  float o[NT][kMTiles][4];
  float m[NT][2], l[NT][2], off[NT][2];  // off: by how much rounding the weights moved l
  float S;  // largest scale of a value met, within a factor of 4
  // this warp's part of a segment: O, and (m, l) per row
  const auto leave = [&](float *part) {
#pragma unroll
    for (int ni = 0; ni < NT; ++ni)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = ni * 8 + 2 * t + j;
        float *dst = part + r * C::kPitch + g * 2;
#pragma unroll
        for (int k = 0; k < kMTiles; ++k)
          *reinterpret_cast<float2 *>(dst + 16 * k) = make_float2(o[ni][k][j], o[ni][k][2 + j]);
        if (g == 0)
          *reinterpret_cast<float4 *>(part + kRows * C::kPitch + 4 * r) = make_float4(m[ni][j], l[ni][j] + off[ni][j], l[ni][j], 0.0f);
      }
  };
  bool in_registers = false;  // the last segment's part, cut at one of the warp's ends
  for (KvWalk w = w0; w.left > 0; w.next(a, kRows)) {
    const int rows = w.r.n * group;
    // ---- the query rows' B fragments
    uint32_t qf[NT][kWords * 2];
    int lim[NT][2];  // keys seen by columns 2t and 2t + 1
#pragma unroll
    for (int ni = 0; ni < NT; ++ni) {
      const int r = ni * 8 + g;
      const __half *src = nullptr;
      if (r < rows) {
        const int tok = r / group;
        src = a.q + (static_cast<int64_t>(w.r.q0) + tok) * a.q_stride + (w.h * group + (r - tok * group)) * D + t * (D / 4);
      }
#pragma unroll
      for (int i = 0; i < kWords / 2; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (src) v = *reinterpret_cast<const uint4 *>(src + 8 * i);
        qf[ni][4 * i] = v.x, qf[ni][4 * i + 1] = v.y, qf[ni][4 * i + 2] = v.z, qf[ni][4 * i + 3] = v.w;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int rj = ni * 8 + 2 * t + j;
        lim[ni][j] = a.causal && rj < rows ? w.r.kv - w.r.n + rj / group + 1 : w.r.kv;
      }
    }
    // keys seen by the first row (the fewest) and the last one (the most)
    const int lim_min = a.causal ? w.r.kv - w.r.n + 1 : w.r.kv;
    const int last_row = min(rows, kRows) - 1;
    const int lim_max = a.causal ? w.r.kv - w.r.n + last_row / group + 1 : w.r.kv;

    S = kKv8LeastScale;
#pragma unroll
    for (int ni = 0; ni < NT; ++ni) {
      m[ni][0] = m[ni][1] = kKvNoMax;
      l[ni][0] = l[ni][1] = off[ni][0] = off[ni][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < kMTiles; ++i) o[ni][i][0] = o[ni][i][1] = o[ni][i][2] = o[ni][i][3] = 0.0f;
    }

    for (int i = 0; i < w.count; ++i) {
      const int base = (w.tile + i) * kKvTile;
      cp_async_wait<C::kStages - 2>();
      __syncwarp();  // every lane's copies of this stage are here, and every lane is done with the stage before
      const uint32_t have = fetch.present >> 2 * stage & 3u;
      fetch.unit(a, lane);
      const uint8_t *st = ring + stage * C::kStage;
      if (++stage == C::kStages) stage = 0;
      if (base >= lim_max || have == 0) continue;  // nothing of these 32 tokens is seen

      // ---- scores of the two blocks, as log2 of the weights
      float sc[2][NT][4], sv[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint8_t *kr = st + (16 * x + row_a) * D;
        uint32_t ka[kWords], kb[kWords];
#pragma unroll
        for (int j = 0; j < kWords / 4; ++j) {
          const int at = (D == 128 ? (2 * t + j) ^ C::key_at(row_a) : t) << 4;
          *reinterpret_cast<uint4 *>(ka + 4 * j) = *reinterpret_cast<const uint4 *>(kr + at);
          *reinterpret_cast<uint4 *>(kb + 4 * j) = *reinterpret_cast<const uint4 *>(kr + 8 * D + at);
        }
        const float2 scales = *reinterpret_cast<const float2 *>(st + 2 * C::kCodes + 8 * x);
        sv[x] = scales.y;
        float s[NT][4];
#pragma unroll
        for (int ni = 0; ni < NT; ++ni)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[ni][j] = 0.0f;
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          const uint32_t a0 = codes_f16(ka[j], kLowPair), a1 = codes_f16(kb[j], kLowPair);
          const uint32_t a2 = codes_f16(ka[j], kHighPair), a3 = codes_f16(kb[j], kHighPair);
#pragma unroll
          for (int ni = 0; ni < NT; ++ni) mma_f16(s[ni], a0, a1, a2, a3, qf[ni][2 * j], qf[ni][2 * j + 1]);
        }
        const float f = scales.x * scale2;
        const float ls = lg2(scales.y < kKv8LeastScale ? kKv8LeastScale : scales.y);  // of a NaN, a NaN
#pragma unroll
        for (int ni = 0; ni < NT; ++ni)
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[x][ni][j] = fmaf(s[ni][j], f, ls);
      }
      const bool whole = base + 32 <= lim_min && have == 3u;
      if (!whole) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int ta = have >> x & 1u ? base + 16 * x + row_a : 0x7FFFFF00, tb = ta + 8;
#pragma unroll
          for (int ni = 0; ni < NT; ++ni)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if ((j < 2 ? ta : tb) >= lim[ni][j & 1]) sc[x][ni][j] = -INFINITY;
          // blocks that no query may see hold anything: keep their scales out of S
          if (!(have >> x & 1u) || base + 16 * x >= lim_max) sv[x] = 0.0f;
        }
      }
      // ---- running maximum of the weights
      const float sv_max = fmaxf(sv[0], sv[1]);
      bool move = sv_max > 4.0f * S;
      float top[NT][2];
#pragma unroll
      for (int ni = 0; ni < NT; ++ni)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          top[ni][j] = fmaxf(fmaxf(sc[0][ni][j], sc[0][ni][2 + j]), fmaxf(sc[1][ni][j], sc[1][ni][2 + j]));
          move |= top[ni][j] > m[ni][j] + (kKvLift + 8.0f);
        }
      if (__any_sync(0xFFFFFFFFu, move)) {
        S = fmaxf(S, sv_max);
#pragma unroll
        for (int ni = 0; ni < NT; ++ni)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float mx = top[ni][j] - kKvLift;
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, x));
            mx = fmaxf(mx, m[ni][j]);
            const float keep = ex2(m[ni][j] - mx);
            m[ni][j] = mx;
            l[ni][j] *= keep, off[ni][j] *= keep;
#pragma unroll
            for (int k = 0; k < kMTiles; ++k) {
              o[ni][k][j] *= keep;
              o[ni][k][2 + j] *= keep;
            }
          }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        // ---- weights
        // A NaN scale counts as the least one here: the weights of the rows that see a key of the block are NaN (ls),
        // those of a row that sees none are zero and add nothing.
        const float rp = __fdividef(1.0f, fmaxf(sv[x], kKv8LeastScale));
        const float rr = sv[x] >= 0.125f * S ? rp : 0.0f;
        uint32_t pf[NT][2];
#pragma unroll
        for (int ni = 0; ni < NT; ++ni) {
          float p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) p[j] = ex2(sc[x][ni][j] - m[ni][j & 1]);
          if (!whole) {  // a scale may be NaN: nothing of it for a key that is not seen
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = sc[x][ni][j] == -INFINITY ? 0.0f : p[j];
          }
          const __half2 ha = __floats2half2_rn(p[0], p[1]), hb = __floats2half2_rn(p[2], p[3]);
          // how far the rounding moved the weights' sum
          const float2 fa = __half22float2(ha), fb = __half22float2(hb);
          l[ni][0] = fmaf(p[0] + p[2], rp, l[ni][0]);
          l[ni][1] = fmaf(p[1] + p[3], rp, l[ni][1]);
          off[ni][0] = fmaf((fa.x - p[0]) + (fb.x - p[2]), rr, off[ni][0]);
          off[ni][1] = fmaf((fa.y - p[1]) + (fb.y - p[3]), rr, off[ni][1]);
          pf[ni][0] = transpose8x8(*reinterpret_cast<const uint32_t *>(&ha));
          pf[ni][1] = transpose8x8(*reinterpret_cast<const uint32_t *>(&hb));
          if (sv[x] == 0.0f) pf[ni][0] = pf[ni][1] = 0u;  // values of zero, whatever their codes
        }
        // ---- values
        const uint8_t *vs = st + C::kCodes + 16 * x * D + v_at;
        uint32_t v0[D / 32], v1[D / 32], v2[D / 32], v3[D / 32];
        if constexpr (D == 128) {
          *reinterpret_cast<uint4 *>(v0) = *reinterpret_cast<const uint4 *>(vs + vr0 * D);
          *reinterpret_cast<uint4 *>(v1) = *reinterpret_cast<const uint4 *>(vs + vr1 * D);
          *reinterpret_cast<uint4 *>(v2) = *reinterpret_cast<const uint4 *>(vs + (vr0 + 8) * D);
          *reinterpret_cast<uint4 *>(v3) = *reinterpret_cast<const uint4 *>(vs + (vr1 + 8) * D);
        } else {
          *reinterpret_cast<uint2 *>(v0) = *reinterpret_cast<const uint2 *>(vs + vr0 * D);
          *reinterpret_cast<uint2 *>(v1) = *reinterpret_cast<const uint2 *>(vs + vr1 * D);
          *reinterpret_cast<uint2 *>(v2) = *reinterpret_cast<const uint2 *>(vs + (vr0 + 8) * D);
          *reinterpret_cast<uint2 *>(v3) = *reinterpret_cast<const uint2 *>(vs + (vr1 + 8) * D);
        }
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t x01 = __byte_perm(v0[j], v1[j], half ? 0x7362 : 0x5140);
            const uint32_t x23 = __byte_perm(v2[j], v3[j], half ? 0x7362 : 0x5140);
            const uint32_t a0 = codes_f16(x01, kLowPair), a1 = codes_f16(x01, kHighPair);
            const uint32_t a2 = codes_f16(x23, kLowPair), a3 = codes_f16(x23, kHighPair);
#pragma unroll
            for (int ni = 0; ni < NT; ++ni) mma_f16(o[ni][2 * j + half], a0, a1, a2, a3, pf[ni][0], pf[ni][1]);
          }
        }
      }
    }

    // ---- the segment's end, or the warp's
#pragma unroll
    for (int ni = 0; ni < NT; ++ni)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          l[ni][j] += __shfl_xor_sync(0xFFFFFFFFu, l[ni][j], x);
          off[ni][j] += __shfl_xor_sync(0xFFFFFFFFu, off[ni][j], x);
        }
    if (w.count == w.r.tiles) {
#pragma unroll
      for (int ni = 0; ni < NT; ++ni)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = ni * 8 + 2 * t + j;
          if (r >= rows) continue;
          const int tok = r / group, head = w.h * group + r - tok * group;
          const int64_t token = static_cast<int64_t>(w.r.q0) + tok;
          const float inv = l[ni][j] == 0.0f ? 0.0f : 1.0f / (l[ni][j] + off[ni][j]);  // a row that saw no key is zero
          uint32_t packed[kMTiles];
#pragma unroll
          for (int k = 0; k < kMTiles; ++k) packed[k] = half2_bits(o[ni][k][j] * inv, o[ni][k][2 + j] * inv);
          uint4 *dst = reinterpret_cast<uint4 *>(a.out + token * a.out_stride + static_cast<int64_t>(head) * D + g * (D / 8));
#pragma unroll
          for (int k = 0; k < kMTiles; k += 4) dst[k / 4] = make_uint4(packed[k], packed[k + 1], packed[k + 2], packed[k + 3]);
          if (a.lse && g == 0)
            a.lse[token * a.Hq + head] = l[ni][j] == 0.0f ? -INFINITY : (m[ni][j] + log2f(l[ni][j])) * 0.6931471805599453f;
        }
    } else {
      in_registers = w.count == w.left;
      const int side = in_registers ? 1 : 0;
      if (!in_registers) leave(warp_parts + (c * kWarps + warp) * C::kPart);
      if (lane == 0) {
        shared.part_first[warp][side] = w.seg_first;
        shared.part_at[warp][side] = KvSeg{w.h, w.r.tiles, w.r.q0, w.r.n};
      }
    }
  }
  float *last_parts = reinterpret_cast<float *>(smem);
  __threadfence_block();
  __syncthreads();  // no warp needs its ring any more
  if (in_registers) leave(last_parts + warp * C::kPart);
  __syncthreads();
  kv_join_parts<D, C>(a, shared, my, last_parts, warp_parts, block_parts, counters);
}

// ---------------------------------------------------------------------------
// Prompts: the 4-bit cache's kernel (kv4_prompt.cuh) with these rows.  A block's
// scales are taken once for 16 columns, the values' as a summand of the exponent.
// 1024 and 866 new tokens behind contexts of 8192 and 6354, 32 query and 8 key heads
// of 128: 250 to 270 us, 845 to 785 TFLOP/s (52 to 48 % of the measured bf16 burst rate); 16 and 4 heads
// of 64: 120 us.  The softmax bounds it: 64 columns take its warps some 2200 clocks, of
// which the exponentials of both tiles need 1024.
// ---------------------------------------------------------------------------
template <int D>
struct Pm8 {
  using Args = Attend8Args;
  static constexpr int kVec = D / 16;  // 16-byte loads of a row's codes
  static constexpr int kIssueRegs = 48, kUnpackRegs = 112;  // a key's and a value's codes are held at once
  static constexpr bool kBlocks = true;  // one scale for 16 tokens
  // A row's 16-byte pieces are neighbouring lanes' (each lane a row of its own took 32 lines a load): lane l has
  // piece l % kVec of rows l / kVec, + 32 / kVec, .. of the warp's 32.  `row` is the lane's token's, or -1; a block of
  // 16 tokens lies in one page, so its rows follow on its first one's, seen or not.
  static __device__ __forceinline__ uint32_t load(const Kv8Cache &c, int64_t r, uint4 (&codes)[kVec]) {
    const int lane = threadIdx.x & 31;
    const int64_t first[2] = {__shfl_sync(0xFFFFFFFFu, r, 0), __shfl_sync(0xFFFFFFFFu, r, 16)};
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int64_t from = first[i >= kVec / 2];
      const int row = (i % (kVec / 2)) * (32 / kVec) + lane / kVec;
      codes[i] = from >= 0 ? *reinterpret_cast<const uint4 *>(c.codes + (from + row) * D + lane % kVec * 16)
                           : make_uint4(0, 0, 0, 0);
    }
    return r >= 0 ? __float_as_uint(c.scales[r >> 4]) : 0u;
  }
  static __device__ __forceinline__ float scale(uint32_t meta) { return __uint_as_float(meta); }
  // (a scale of zero makes zeros of any codes: the softmax does not multiply by it)
  static __device__ __forceinline__ void store(uint8_t *to, const uint4 (&held)[kVec], uint32_t meta) {
    const int lane = threadIdx.x & 31, piece = lane % kVec;
    const bool zero[2] = {__shfl_sync(0xFFFFFFFFu, meta, 0) == 0, __shfl_sync(0xFFFFFFFFu, meta, 16) == 0};
    uint4 codes[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      codes[i] = zero[i >= kVec / 2] ? make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u) : held[i];
      const int tk = (threadIdx.x & 96) + i * (32 / kVec) + lane / kVec;
      const uint4 low = make_uint4(codes_f16(codes[i].x, kLowPair), codes_f16(codes[i].x, kHighPair),
                                   codes_f16(codes[i].y, kLowPair), codes_f16(codes[i].y, kHighPair));
      const uint4 high = make_uint4(codes_f16(codes[i].z, kLowPair), codes_f16(codes[i].z, kHighPair),
                                    codes_f16(codes[i].w, kLowPair), codes_f16(codes[i].w, kHighPair));
      // the second panel's lanes begin with their second half: eight lanes then meet all banks
      const bool swap = piece >= 4;
      uint8_t *line = to + tk * 128 + (piece >> 2) * PmCfg<D>::kPanel;
      const int chunk = (2 * piece & 7) ^ (tk & 7);
      *reinterpret_cast<uint4 *>(line + ((chunk ^ (swap ? 1 : 0)) << 4)) = swap ? high : low;
      *reinterpret_cast<uint4 *>(line + ((chunk ^ (swap ? 0 : 1)) << 4)) = swap ? low : high;
    }
  }
  static __device__ __forceinline__ uint4 order(const uint4 v) { return v; }
  static __host__ __device__ constexpr int place(int x) { return x; }
};

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// The decode workspace: as the 4-bit cache's, with eight warps a block.
static size_t kv8_decode_workspace_bytes(int max_q, int group, int D) {
  const int rows = 8 * kv4_decode_nt(max_q, group);
  return kKvCounterBytes + static_cast<size_t>(kKvMaxGrid) * (2 + 8) * rows * (D + 8 + 4) * sizeof(float);
}

template <int D, int NT>
static cudaError_t launch_kv8_decode_type(const Attend8Args &a, void *ws, cudaStream_t stream, const char **msg) {
  using C = Kv8Cfg<D, NT>;
  auto kern = kv8_decode_kernel<D, NT>;
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
  const int64_t units = static_cast<int64_t>(a.B) * a.cache.H * (tiles > 0 ? tiles : 1);
  if (units > 0x7FFFFFFF) {
    *msg = "requests x key heads x 32-token blocks of a table row pass 2^31";
    return cudaErrorNotSupported;
  }
  int64_t grid = device_sm_count();
  if (grid > kKvMaxGrid) grid = kKvMaxGrid;
  if (grid > (units + C::kWarps - 1) / C::kWarps) grid = (units + C::kWarps - 1) / C::kWarps;
  float *parts = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kKvCounterBytes);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // starts while the kernel before it ends
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, static_cast<uint32_t *>(ws), parts, parts + kKvMaxGrid * 2 * C::kPart);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) *msg = "launch of the decode attention failed";
  return e;
}

size_t kv8_attention_workspace_bytes(int B, int max_q, int Hq, int H, int D) {
  return kv4_is_decode(max_q, Hq / H) ? kv8_decode_workspace_bytes(max_q, Hq / H, D)
                                      : kv4_prompt_workspace_bytes(B, max_q, Hq / H, D);
}

cudaError_t launch_kv8_attention(const Attend8Args &a, void *ws, cudaStream_t stream, const char **msg) {
  const int group = a.Hq / a.cache.H;
  if (!kv4_is_decode(a.max_q, group))
    return a.cache.D == 128 ? launch_kv4_prompt<Pm8<128>, 128>(a, ws, stream, msg)
                            : launch_kv4_prompt<Pm8<64>, 64>(a, ws, stream, msg);
  const bool one = kv4_decode_nt(a.max_q, group) == 1;
  if (a.cache.D == 128)
    return one ? launch_kv8_decode_type<128, 1>(a, ws, stream, msg) : launch_kv8_decode_type<128, 2>(a, ws, stream, msg);
  return one ? launch_kv8_decode_type<64, 1>(a, ws, stream, msg) : launch_kv8_decode_type<64, 2>(a, ws, stream, msg);
}

}  // namespace mixllm
