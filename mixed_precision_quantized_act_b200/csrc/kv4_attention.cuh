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
#include "kv4_ptx.cuh"
#include "kv_split.cuh"
#include "launch.h"
#include "ptx_sm100.cuh"

namespace mixllm {

// ---------------------------------------------------------------------------
// Few queries per request (decode: up to 16 rows of query token and query head
// per key head).  HBM-bound: 2 * (D/2 + 4) bytes per cached token and head.
//
// Work is cut into units of 32 tokens of one (request, key head); block c takes
// the units [c U / P, (c + 1) U / P) of their concatenation and its warps an
// even share of them each, so requests of any lengths load every SM alike, and
// the lengths stay on the device.  A warp fetches its tokens itself, by
// cp.async into stages of its own (bulk copies of 2 KB, with less address
// arithmetic, took 7 % longer), and meets the others only when all of the
// block's units are done: the latencies where one request or head ends and the
// next begins are then one warp's in sixteen.  Tokens are the 16-row side of
// m16n8k16 and the query rows its 8-column side (NT such tiles), so that a group
// of 8 heads fills the instruction and smaller ones waste only tensor work:
// S^T = K Q^T with K as the A operand, then O^T = V^T P^T with V^T as A.
//
// Measured on B200 (as a CUDA graph): 64 requests of 100 to 8100 tokens, 32 query
// and 8 key heads of 128: 84.0 us, 3.4 TB/s; 4 requests of 100000 to 131071
// tokens, 64 and 8 heads: 120 us, 4.3 TB/s (65 % of the measured copy rate);
// one request of 1003 tokens: 11.6 us.  With the products left out the second
// took 96 us, with the loads left out 114: neither hides the other wholly.
// Above 128 requests a warp no longer holds all their lengths, and the walk to its
// first unit is a chain of loads: 262144 tokens as 128 requests take 83 us, as 256
// 92, as 1024 105.
//
// What bounds the loop on the way to HBM speed is the unpacking: integer
// instructions issue at half rate.  So one AND per pair of codes makes fp16
// subnormals of them, n 2^-24 (low nibbles) or 16 n 2^-24 (high nibbles), which
// the tensor cores multiply exactly, and nothing is subtracted per code.  The
// tensor cores align products by their operands' exponents, of which a
// subnormal has the smallest normal one, so n 2^-24 would lose 10 bits of
// the fp32 sum; a half-precision multiply on the otherwise idle FMA pipe makes
// it n 2^-10.  The high nibbles lose 6 bits, 2^-18 of the largest product, and
// stay as they are.
//   * K: any permutation of the channels serves as long as Q has the same, so
//     a lane takes D/4 consecutive channels of a token and pairs nibbles i and
//     i + 4 of a word.  Low and high nibbles go into accumulators of their own,
//     joined with their factor; the zero point comes off as z * sum(q).
//   * V: lane (g, t) takes channels g D/8 .. of four tokens; a byte permute
//     joins the halves of two tokens' words into (token, token') pairs.  Low
//     and high nibbles are different accumulator rows, scaled at the end.  One
//     more product, with the zero points in the place of codes, gives the sum of
//     p z that comes off every channel.
// The differences are taken in fp32 of sums of at most 15 |q| and 15 p: no more
// is lost than in the sums themselves.  P^T goes from accumulator to B layout
// by movmatrix.
//
// Softmax per warp with lazy rescaling.  The values' scales pass through fp16
// together with p, as weights p s_v.  The exponents' reference m of a row is 7
// (in log2 units) below its largest weight so far among the keys that it sees (a
// scale of zero counting as 2^-24, so that the sum of p stays finite), and moves
// only when a weight passes 2^15: what a row does not see, or gives no weight,
// costs it no bits, and weights down to 2^-21 of the largest are normal numbers.
// A weight is rounded once, to fp16's 11 bits, and O is divided by the sum of p as
// that rounding leaves it (the logarithm of the denominator is that of the
// unrounded sum): where one token has nearly all the weight, its error cancels.
// The correction is left out for values much smaller than the largest, S, that
// the warp has met: a weight that is an fp16 subnormal, or zero, says little
// about p.  Without it a single request's error against 64 bits was up to 1.6
// times that of rounding the result alone, with it 1.4; it costs 3 to 6 % of the
// time.  Sums stay in fp32.
//
// A segment (the units of one request and head) that one warp holds
// whole is written by it.  Parts of one that is cut between warps are joined by
// the block at its end, and those cut between blocks left in the workspace,
// where the last block to arrive adds them; always in the order of the tokens,
// so the result does not depend on timing.
// ---------------------------------------------------------------------------
constexpr float kKvLift = 7.0f;  // log2 of a row's largest weight where its reference is set: 2^15, 8 more, is in range

template <int D, int NT>
struct KvCfg {
  static constexpr int kWarps = D * NT <= 128 ? 16 : 8;  // by registers: 128 and 255 a thread
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRows = 8 * NT;
  static constexpr int kLeast = 2;  // units of a warp
  static constexpr bool kWholeHeads = false;
  static constexpr int kRowBytes = D / 2;
  static constexpr int kCodes = 32 * kRowBytes;  // bytes of 32 tokens' key (or value) codes
  static constexpr int kStage = 2 * (kCodes + 32 * 4);
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr int kRing = kStages * kStage;  // of one warp
  static constexpr int kPitch = D + 8;            // floats of a part's row: two rows further, 16 banks further
  static constexpr int kPart = kRows * (kPitch + 4);  // floats of one part: sums, then m, the two sums of p per row
  static constexpr int kSmem = kWarps * kRing;
  // Half a warp copies 16 tokens of a unit: this lane's first bytes in a stage, and its copies of the codes and of
  // the metadata of 16 rows from row `at` of the cache on (`to_value` rows from a key to its value).
  static __device__ __forceinline__ uint32_t lane_bytes(int lane) { return (lane >> 4) * (16 * kRowBytes) + (lane & 15) * 16; }
  static __device__ __forceinline__ void copy(const Kv4Cache &c, int lane, int64_t at, int64_t to_value, uint32_t dst) {
    const uint8_t *k = c.codes + at * kRowBytes + (lane & 15) * 16;
    const uint8_t *v = k + to_value * kRowBytes;
#pragma unroll
    for (int i = 0; i < 16 * kRowBytes; i += 256) {
      cp_async_16_u32(dst + i, k + i);
      cp_async_16_u32(dst + kCodes + i, v + i);
    }
    if ((lane & 15) < 8) {  // key metadata of 16 tokens, then value metadata
      const int part = lane & 3, kv = lane >> 2 & 1;
      const uint32_t to = dst - lane_bytes(lane) + 2 * kCodes + kv * 128 + (lane >> 4) * 64 + part * 16;
      cp_async_16_u32(to, c.meta + at + (kv ? to_value : 0) + part * 4);
    }
  }
  static_assert(kWarps * kPart * 4 <= kSmem, "the warps' last parts take the ring's place");
  static_assert(kSmem + 4096 <= 227 * 1024, "shared memory of a block");
};
// A row's scale, and its zero point as the subnormal z 2^-24 (the bits above it left out).
constexpr uint32_t kKvMetaBits = 0x000FFFFFu;
__device__ __forceinline__ float2 meta_pair(uint32_t m) { return __half22float2(*reinterpret_cast<const __half2 *>(&m)); }
// Pairs of codes as fp16: low nibbles as n 2^-10, high ones as n 2^-20.
__device__ __forceinline__ uint32_t low_codes(uint32_t w) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w & 0x000F000Fu), "r"(0x74007400u));  // by 2^14
  return r;
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w) { return w & 0x00F000F0u; }
constexpr float kHighToLow = 0x1p10f;

template <int D, int NT>
__global__ void __launch_bounds__(KvCfg<D, NT>::kThreads, 1) kv4_decode_kernel(const AttendArgs a,
                                                                                          uint32_t *counters,
                                                                                          float *block_parts,
                                                                                          float *warp_parts) {
  using C = KvCfg<D, NT>;
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
  // accumulator row r of the score tile is token r ^ (r >> 1 & 1): the value
  // rows that four lanes read together then alternate in the 32 banks
  const int row_a = g ^ (g >> 1 & 1);
  const int vr0 = (2 * t) ^ (t & 1), vr1 = (2 * t + 1) ^ (t & 1);
  const uint32_t z_order = t & 1 ? 0x3276u : 0x7632u;  // zero points of tokens (vr0, vr1) from those of (2t, 2t + 1)
  constexpr int kWords = D / 32;   // words of a lane's key chunk
  constexpr int kMTiles = D / 16;  // 16-channel tiles of O^T
  const float scale2 = a.scale * 1.4426950408889634f * 0x1p10f;  // to log2 units, from products with n 2^-10
  const uint8_t *ring = smem + warp * C::kRing;
  int stage = 0;

  float o[NT][kMTiles][4], oz[NT][4];  // oz: sums of p z, the same in every row
  float m[NT][2], l[NT][2], off[NT][2];  // off: by how much rounding the weights moved l
  float S;  // largest scale of a value met, within a factor of 4
  // this warp's part of a segment: O, and (m, l) per row
  const auto leave = [&](float *part) {
#pragma unroll
    for (int ni = 0; ni < NT; ++ni)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = ni * 8 + 2 * t + j;
        const float z = oz[ni][j];
        float *dst = part + r * C::kPitch + g * 2;
#pragma unroll
        for (int k = 0; k < kMTiles; ++k)
          *reinterpret_cast<float2 *>(dst + 16 * k) =
              make_float2((o[ni][k][j] - z) * 0x1p10f, fmaf(o[ni][k][2 + j], kHighToLow, -z) * 0x1p10f);
        if (g == 0)
          *reinterpret_cast<float4 *>(part + kRows * C::kPitch + 4 * r) = make_float4(m[ni][j], l[ni][j] + off[ni][j], l[ni][j], 0.0f);
      }
  };
  bool in_registers = false;  // the last segment's part, cut at one of the warp's ends
  for (KvWalk w = w0; w.left > 0; w.next(a, kRows)) {
    const int rows = w.r.n * group;
    // ---- the query rows' B fragments, channels permuted as the keys' nibbles, and their sums
    uint32_t qf[NT][kWords * 4];
    float qs[NT][2];
    int lim[NT][2];  // keys seen by columns 2t and 2t + 1
#pragma unroll
    for (int ni = 0; ni < NT; ++ni) {
      const int r = ni * 8 + g;
      const __half *src = nullptr;
      if (r < rows) {
        const int tok = r / group;
        src = a.q + (static_cast<int64_t>(w.r.q0) + tok) * a.q_stride + (w.h * group + (r - tok * group)) * D + t * (D / 4);
      }
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (src) v = *reinterpret_cast<const uint4 *>(src + 8 * i);
        qf[ni][4 * i + 0] = __byte_perm(v.x, v.z, 0x5410);  // channels 0, 4: low nibbles
        qf[ni][4 * i + 1] = __byte_perm(v.y, v.w, 0x5410);  // 2, 6
        qf[ni][4 * i + 2] = __byte_perm(v.x, v.z, 0x7632);  // 1, 5: high nibbles
        qf[ni][4 * i + 3] = __byte_perm(v.y, v.w, 0x7632);  // 3, 7
        const uint32_t h2[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2[j]));
          sum += f.x + f.y;
        }
      }
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        qs[ni][j] = __shfl_sync(0xFFFFFFFFu, sum, (2 * t + j) * 4) * 0x1p14f;  // meets z 2^-24
        const int rj = ni * 8 + 2 * t + j;
        lim[ni][j] = a.causal && rj < rows ? w.r.kv - w.r.n + rj / group + 1 : w.r.kv;
      }
    }
    // keys seen by the first row (the fewest) and the last one (the most)
    const int lim_min = a.causal ? w.r.kv - w.r.n + 1 : w.r.kv;
    const int last_row = min(rows, kRows) - 1;
    const int lim_max = a.causal ? w.r.kv - w.r.n + last_row / group + 1 : w.r.kv;

    S = 0x1p-24f;
#pragma unroll
    for (int ni = 0; ni < NT; ++ni) {
      m[ni][0] = m[ni][1] = kKvNoMax;
      l[ni][0] = l[ni][1] = off[ni][0] = off[ni][1] = 0.0f;
      oz[ni][0] = oz[ni][1] = oz[ni][2] = oz[ni][3] = 0.0f;
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

      // ---- scores of two 16-token blocks
      float sc[2][NT][4];
      float sv[2][2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint8_t *kr = st + (16 * x + row_a) * C::kRowBytes + t * (D / 8);
        uint32_t ka[kWords], kb[kWords];
        if constexpr (D == 128) {
          *reinterpret_cast<uint4 *>(ka) = *reinterpret_cast<const uint4 *>(kr);
          *reinterpret_cast<uint4 *>(kb) = *reinterpret_cast<const uint4 *>(kr + 8 * C::kRowBytes);
        } else {
          *reinterpret_cast<uint2 *>(ka) = *reinterpret_cast<const uint2 *>(kr);
          *reinterpret_cast<uint2 *>(kb) = *reinterpret_cast<const uint2 *>(kr + 8 * C::kRowBytes);
        }
        const uint32_t *km = reinterpret_cast<const uint32_t *>(st + 2 * C::kCodes) + 16 * x + row_a;
        const float2 ma = meta_pair(km[0] & kKvMetaBits), mb = meta_pair(km[8] & kKvMetaBits);
        sv[x][0] = meta_pair(km[32]).x;
        sv[x][1] = meta_pair(km[40]).x;
        float lo[NT][4], hi[NT][4];
#pragma unroll
        for (int ni = 0; ni < NT; ++ni)
#pragma unroll
          for (int j = 0; j < 4; ++j) lo[ni][j] = hi[ni][j] = 0.0f;
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          const uint32_t xa = ka[j] >> 8, xb = kb[j] >> 8;
#pragma unroll
          for (int ni = 0; ni < NT; ++ni) {
            mma_f16(lo[ni], low_codes(ka[j]), low_codes(kb[j]), low_codes(xa), low_codes(xb), qf[ni][4 * j],
                    qf[ni][4 * j + 1]);
            mma_f16(hi[ni], high_codes(ka[j]), high_codes(kb[j]), high_codes(xa), high_codes(xb), qf[ni][4 * j + 2],
                    qf[ni][4 * j + 3]);
          }
        }
        const float fa = ma.x * scale2, fb = mb.x * scale2;
#pragma unroll
        for (int ni = 0; ni < NT; ++ni)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            sc[x][ni][j] =
                fmaf(-(j < 2 ? ma.y : mb.y), qs[ni][j & 1], fmaf(hi[ni][j], kHighToLow, lo[ni][j])) * (j < 2 ? fa : fb);
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
          // rows that no query may see hold anything: keep their scales out of S
          if (ta >= lim_max) sv[x][0] = 0.0f;
          if (tb >= lim_max) sv[x][1] = 0.0f;
        }
      }
      // ---- running maximum of the weights
      float ls[2][2];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 2; ++i) ls[x][i] = lg2(sv[x][i] + 0x1p-24f);
      const float sv_max = fmaxf(fmaxf(sv[0][0], sv[0][1]), fmaxf(sv[1][0], sv[1][1]));
      bool move = sv_max > 4.0f * S;
      float top[NT][2];
#pragma unroll
      for (int ni = 0; ni < NT; ++ni)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          top[ni][j] = fmaxf(fmaxf(sc[0][ni][j] + ls[0][0], sc[0][ni][2 + j] + ls[0][1]),
                             fmaxf(sc[1][ni][j] + ls[1][0], sc[1][ni][2 + j] + ls[1][1]));
          move |= top[ni][j] > m[ni][j] + (kKvLift + 8.0f);
        }
      if (__any_sync(0xFFFFFFFFu, move)) {
        S = fmaxf(S, sv_max);
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) S = fmaxf(S, __shfl_xor_sync(0xFFFFFFFFu, S, x));
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
            oz[ni][j] *= keep;
#pragma unroll
            for (int k = 0; k < kMTiles; ++k) {
              o[ni][k][j] *= keep;
              o[ni][k][2 + j] *= keep;
            }
          }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        // ---- probabilities
        const float wa = sv[x][0], wb = sv[x][1];
        const float ra = wa >= 0.125f * S ? __fdividef(1.0f, wa) : 0.0f, rb = wb >= 0.125f * S ? __fdividef(1.0f, wb) : 0.0f;
        uint32_t pf[NT][2];
#pragma unroll
        for (int ni = 0; ni < NT; ++ni) {
          float p[4], pw[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            p[j] = ex2(sc[x][ni][j] - m[ni][j & 1]);
            pw[j] = p[j] * (j < 2 ? wa : wb);
          }
          if (!whole) {  // a scale may be NaN: no product with the zero of a key that is not seen
#pragma unroll
            for (int j = 0; j < 4; ++j) pw[j] = sc[x][ni][j] == -INFINITY ? 0.0f : pw[j];
          }
          const __half2 ha = __floats2half2_rn(pw[0], pw[1]), hb = __floats2half2_rn(pw[2], pw[3]);
          // how far the rounding moved the weights' sum
          const float2 fa = __half22float2(ha), fb = __half22float2(hb);
          l[ni][0] += p[0] + p[2];
          l[ni][1] += p[1] + p[3];
          off[ni][0] = fmaf(fa.x - pw[0], ra, fmaf(fb.x - pw[2], rb, off[ni][0]));
          off[ni][1] = fmaf(fa.y - pw[1], ra, fmaf(fb.y - pw[3], rb, off[ni][1]));
          pf[ni][0] = transpose8x8(*reinterpret_cast<const uint32_t *>(&ha));
          pf[ni][1] = transpose8x8(*reinterpret_cast<const uint32_t *>(&hb));
        }
        // ---- values
        const uint8_t *vs = st + C::kCodes + 16 * x * C::kRowBytes + g * (D / 16);
        uint32_t v0[kWords / 2], v1[kWords / 2], v2[kWords / 2], v3[kWords / 2];
        if constexpr (D == 128) {
          *reinterpret_cast<uint2 *>(v0) = *reinterpret_cast<const uint2 *>(vs + vr0 * C::kRowBytes);
          *reinterpret_cast<uint2 *>(v1) = *reinterpret_cast<const uint2 *>(vs + vr1 * C::kRowBytes);
          *reinterpret_cast<uint2 *>(v2) = *reinterpret_cast<const uint2 *>(vs + (vr0 + 8) * C::kRowBytes);
          *reinterpret_cast<uint2 *>(v3) = *reinterpret_cast<const uint2 *>(vs + (vr1 + 8) * C::kRowBytes);
        } else {
          v0[0] = *reinterpret_cast<const uint32_t *>(vs + vr0 * C::kRowBytes);
          v1[0] = *reinterpret_cast<const uint32_t *>(vs + vr1 * C::kRowBytes);
          v2[0] = *reinterpret_cast<const uint32_t *>(vs + (vr0 + 8) * C::kRowBytes);
          v3[0] = *reinterpret_cast<const uint32_t *>(vs + (vr1 + 8) * C::kRowBytes);
        }
        const uint2 *vm = reinterpret_cast<const uint2 *>(st + 2 * C::kCodes + 128 + 64 * x) + t;
        const uint2 m01 = vm[0], m23 = vm[4];
        const uint32_t z01 = low_codes(__byte_perm(m01.x, m01.y, z_order));
        const uint32_t z23 = low_codes(__byte_perm(m23.x, m23.y, z_order));
#pragma unroll
        for (int ni = 0; ni < NT; ++ni) mma_f16(oz[ni], z01, z01, z23, z23, pf[ni][0], pf[ni][1]);
#pragma unroll
        for (int j = 0; j < kWords / 2; ++j) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t x01 = __byte_perm(v0[j], v1[j], half ? 0x7632 : 0x5410);
            uint32_t x23 = __byte_perm(v2[j], v3[j], half ? 0x7632 : 0x5410);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
#pragma unroll
              for (int ni = 0; ni < NT; ++ni)
                mma_f16(o[ni][4 * j + 2 * half + q], low_codes(x01), high_codes(x01), low_codes(x23), high_codes(x23),
                        pf[ni][0], pf[ni][1]);
              x01 >>= 8;
              x23 >>= 8;
            }
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
          const float inv = l[ni][j] == 0.0f ? 0.0f : 0x1p10f / (l[ni][j] + off[ni][j]);  // a row that saw no key is zero
          const float z = oz[ni][j];
          uint32_t packed[kMTiles];
#pragma unroll
          for (int k = 0; k < kMTiles; ++k)
            packed[k] = half2_bits((o[ni][k][j] - z) * inv, fmaf(o[ni][k][2 + j], kHighToLow, -z) * inv);
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
// host side
// ---------------------------------------------------------------------------

// Two n-tiles of rows when a request's rows do not fit one.
static int kv4_decode_nt(int max_q, int group) { return static_cast<int64_t>(max_q) * group > 8 ? 2 : 1; }

// Workspace: one counter per block, always in the same place, then the parts
// of cut segments (two per block, one per warp), which need no initial value.
constexpr size_t kKvCounterBytes = 4096;
static_assert(kKvMaxGrid * sizeof(uint32_t) <= kKvCounterBytes, "one counter per block");

static size_t kv4_decode_workspace_bytes(int max_q, int group, int D) {
  const int rows = 8 * kv4_decode_nt(max_q, group);
  return kKvCounterBytes + static_cast<size_t>(kKvMaxGrid) * (2 + 16) * rows * (D + 8 + 4) * sizeof(float);
}

template <int D, int NT>
static cudaError_t launch_kv4_decode_type(const AttendArgs &a, void *ws, cudaStream_t stream,
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

static cudaError_t launch_kv4_decode(const AttendArgs &a, void *ws, cudaStream_t stream, const char **msg) {
  const bool one = kv4_decode_nt(a.max_q, a.Hq / a.cache.H) == 1;
  if (a.cache.D == 128)
    return one ? launch_kv4_decode_type<128, 1>(a, ws, stream, msg) : launch_kv4_decode_type<128, 2>(a, ws, stream, msg);
  return one ? launch_kv4_decode_type<64, 1>(a, ws, stream, msg) : launch_kv4_decode_type<64, 2>(a, ws, stream, msg);
}

}  // namespace mixllm
