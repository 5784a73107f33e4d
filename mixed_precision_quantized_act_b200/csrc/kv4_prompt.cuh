// kv4_prompt.cuh -- attention of prompts (many query rows per request and key
// head) over the paged 4-bit KV cache, on tcgen05.
#pragma once

#include <cuda_fp16.h>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "gemm_w4w8a8.cuh"  // device_sm_count
#include "kv4_attention.cuh"
#include "kv4_ptx.cuh"
#include "launch.h"
#include "ptx_sm100.cuh"

namespace mixllm {

// ---------------------------------------------------------------------------
// Rows of a request and key head are (query token, query head of the group),
// token by token.  A block takes 256 of them as two tiles of 128 and runs over
// the cached tokens in tiles of 128:
//   S = Q K^T      two 128 x 128 products, fp32 in tensor memory
//   P = softmax    one thread per row; fp16, over S in tensor memory
//   O += P V       A from tensor memory, accumulated there in fp32
// Warp 0 issues the products, warps 4-7 unpack keys and values, warps 8-11 and
// 12-15 are the softmax of either tile (in this order because the scheduler
// prefers older warps, and the tensor core waits for warp 0's every
// instruction).
//
// The softmax works on 64 columns at a time: while it is at one half of S, the
// tensor core multiplies the other half's weights into O and puts the next
// tile's scores in their place (whole tiles left a tile's softmax waiting for
// its own products, 1800 of 5000 clocks).  The two tiles do so independently.
//
// Unpacking: one thread per token.  A word's nibbles i and i + 4 become fp16
// integers 1024 + n (or 1024 + 16 n) by one AND-OR, and code - z by one add (or
// FMA with 1/16): exact.  Both operands are stored with the channels of each
// eight in the order 0 4 1 5 2 6 3 7; Q is laid out in the same order, and the
// output's columns are put back by the epilogue.  Keys are a K-major operand
// (channels along K), values an MN-major one (channels along N), so both are rows
// of tokens in the same 128-byte swizzle and nothing is transposed.
//
// Scales: a key's scale multiplies its column of S in the softmax, a value's
// scale its column of P before the rounding to fp16 (the one rounding of the
// weights).  The exponent's reference R is the row's own, 7 (in log2 units)
// below its largest weight p s_v so far among the columns that it sees, and moved
// only when a weight passes 2^15: what a row does not see, or gives no weight,
// costs it no bits, and weights down to 2^-21 of the largest are normal numbers.
// Where R moves, O is rescaled in tensor memory, which is rare.
//
// Bound by the tensor core (4 D flops per row and token) and, close behind, by
// the exponentials: 16 a clock and SM make a 128 x 128 tile 1024 clocks, its two
// products at D = 128 take 1024.  Blocks take equal shares of all (tile
// pair, head, token tile) units in one sequence; where the ends of a share cut a
// pair's tokens, the parts go to the workspace and a third kernel joins them in
// the order of the tokens (joined by the last block to arrive, 25 us of one SM's
// work stood behind everything).  The sequence depends on lengths that only the
// device knows: a small kernel before this one lists the pairs and the running
// sum of their tiles.
//
// Measured on B200: 1024 and 866 new tokens behind contexts of 8192 and 6354, 32
// query and 8 key heads of 128: 248 us for the three kernels, 850 TFLOP/s (51 %
// of the measured bf16 burst rate); 16 and 4 heads of 64: 122 us, 431 TFLOP/s.  A
// pair's tile takes some 4900 clocks at heads of 128, of which the exponentials
// need 2048.
// ---------------------------------------------------------------------------
constexpr int kPmThreads = 512;
constexpr int kPmTile = 128;
constexpr int kPmRows = 256;
constexpr int kPmMaxGrid = 148;
constexpr int kPmScaleRing = 4;
constexpr float kPmLift = 7.0f;        // log2 of a row's largest weight where its reference is set
constexpr float kPmTopWeight = 0x1p15f;  // and the largest before it is moved
constexpr float kPmTopSum = 0x1p80f;   // sum of p: larger ones are zero-valued tokens' alone, and move it too

template <int D>
struct PmCfg {
  static constexpr int kPanel = 128 * 128;  // bytes of 128 rows of 64 channels
  static constexpr int kOperand = D / 64 * kPanel;
  static constexpr int kSmem = 6 * kOperand + kPmScaleRing * 3 * kPmTile * 4 + 1024;
  static constexpr int64_t kPart = static_cast<int64_t>(kPmRows) * (D + 2);  // floats
  static_assert(kSmem + 1024 <= 227 * 1024, "shared memory of a block");
};

// A segment that the end of a block cuts: the blocks first .. last hold parts
// of it (last < first: none).
struct PmCut {
  int last, pair, h, q0, n;
};

// The list of tile pairs: (request, pair), and the token tiles before each; and
// the blocks' cuts.
struct PmPlan {
  int *entries;
  int64_t *cum;  // [entries + 1]
  int2 *ent;     // [entries]
  PmCut *cuts;   // [blocks]
};

constexpr int kPmPlanThreads = 1024;

__global__ void __launch_bounds__(kPmPlanThreads) kv4_prompt_plan_kernel(const AttendArgs a, const PmPlan plan) {
  extern __shared__ int pair_base[];  // pairs before each request
  pdl_launch_dependents();
  __shared__ long long warp_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = a.Hq / a.cache.H;
  // exclusive sum of v over the block, plus `base`; moves base on by the block's sum
  auto scan = [&](long long v, long long &base) {
    long long incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    long long before = base + incl - v;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += warp_sum[w];
      base += warp_sum[w];
    }
    __syncthreads();
    return before;
  };
  long long pairs = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPmPlanThreads) {
    const int b = b0 + tid;
    const long long n = b < a.B ? kv_req(a, b, kPmRows).row_tiles : 0;
    const long long before = scan(n, pairs);
    if (b < a.B) pair_base[b] = static_cast<int>(before);
  }
  __syncthreads();
  const int E = static_cast<int>(pairs);
  long long tiles = 0;
  for (int e0 = 0; e0 < E; e0 += kPmPlanThreads) {
    const int e = e0 + tid;
    long long n = 0;
    if (e < E) {
      const int b = owner_of(pair_base, a.B, e), p = e - pair_base[b];
      const KvReq r = kv_req(a, b, kPmRows);
      const int last = min(r.n * group, (p + 1) * kPmRows) - 1;
      const int seen = a.causal ? r.kv - r.n + last / group + 1 : r.kv;  // by the pair's last row, which sees most
      n = max(1, (seen + kPmTile - 1) / kPmTile);
      plan.ent[e] = make_int2(b, p);
    }
    const long long before = scan(n, tiles);
    if (e < E) plan.cum[e] = before;
  }
  if (tid == 0) {
    plan.cum[E] = tiles;
    *plan.entries = E;
  }
}

// Walks a block's units as segments: runs of token tiles of one pair and head.
struct PmWalk {
  int e, h, tile, count, tiles, pair, b;
  int left;           // units of the block from the segment's first on
  int64_t seg_first;  // unit index of the whole segment's first tile
  int q0, n, kv;

  __device__ __forceinline__ void load(const AttendArgs &a, const PmPlan &plan) {
    const int2 v = plan.ent[e];
    b = v.x, pair = v.y;
    tiles = static_cast<int>(plan.cum[e + 1] - plan.cum[e]);
    q0 = a.cu_q[b];
    n = a.cu_q[b + 1] - q0;
    kv = a.kv_lens[b];
  }
  __device__ __forceinline__ void next(const AttendArgs &a, const PmPlan &plan) {
    left -= count;
    seg_first += tiles;
    tile = 0;
    if (++h == a.cache.H) {
      h = 0;
      ++e;
      if (left > 0) load(a, plan);
    }
    count = min(left, tiles);
  }
  __device__ __forceinline__ int rows(int group) const { return min(kPmRows, n * group - pair * kPmRows); }
};

__device__ __forceinline__ ulonglong2 lds_2x2f(const float *p) { return *reinterpret_cast<const ulonglong2 *>(p); }

// Codes minus zero point of eight channels (order 0 4 1 5 2 6 3 7), exact.
__device__ __forceinline__ uint4 unpack_codes(uint32_t w, uint32_t zlo, uint32_t zhi) {
  const uint32_t x = w >> 8;
  uint4 r;
  asm("add.f16x2 %0, %1, %2;" : "=r"(r.x) : "r"((w & 0x000F000Fu) | 0x64006400u), "r"(zlo));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r.y) : "r"((w & 0x00F000F0u) | 0x64006400u), "r"(0x2C002C00u), "r"(zhi));
  asm("add.f16x2 %0, %1, %2;" : "=r"(r.z) : "r"((x & 0x000F000Fu) | 0x64006400u), "r"(zlo));
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r.w) : "r"((x & 0x00F000F0u) | 0x64006400u), "r"(0x2C002C00u), "r"(zhi));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kPmThreads, 1) kv4_prompt_kernel(const AttendArgs a, const PmPlan plan,
                                                                 float *parts) {
  using C = PmCfg<D>;
  constexpr int kPanel = C::kPanel, kOperand = C::kOperand;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t *q_s = smem, *k_s = smem + 2 * kOperand, *v_s = smem + 4 * kOperand;
  float *k_scale = reinterpret_cast<float *>(smem + 6 * kOperand);  // [ring][128], to log2 units
  float *v_scale = k_scale + kPmScaleRing * kPmTile;
  float *v_log = v_scale + kPmScaleRing * kPmTile;  // log2 of it, of 2^-24 at least
  __shared__ uint64_t q_full[2], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2][2], p_full[2][2];  // s, p: [tile][half]
  __shared__ __align__(16) uint32_t seen[kPmScaleRing][4];  // bit t: token t's page exists; read in pairs
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ int first_e;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = a.Hq / a.cache.H, H = a.cache.H;
  const int c = blockIdx.x;
  if (tid == 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 128);
      mbar_init(&k_full[i], 128);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 128);
      mbar_init(&v_empty[i], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&s_full[i][h], 2);
        mbar_init(&p_full[i][h], 128);
      }
    }
    fence_mbar_init();
    abort_flag = 0;
  }
  pdl_wait();  // the plan, and with it all that came before it
  const int E = *plan.entries;
  const int64_t U = plan.cum[E] * H;
  const int P = U < gridDim.x ? static_cast<int>(U) : static_cast<int>(gridDim.x);
  if (tid == 0) plan.cuts[c].last = -1;
  if (c >= P) return;  // every other block has a unit
  const int64_t share = U / P;
  const int rest = static_cast<int>(U - share * P);
  const auto block_start = [&](int b) { return share * b + rest * b / P; };
  const int64_t start = block_start(c), end = block_start(c + 1);

  if (warp == 15) {  // the pair that holds unit `start`: the last e with cum[e] H <= start
    int lo = 0, hi = E;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, at = lo + lane * step;
      const uint32_t below = __ballot_sync(0xFFFFFFFFu, at < hi && plan.cum[at] * H <= start);
      lo += (31 - __clz(below)) * step;
      hi = min(hi, lo + step);
    }
    if (lane == 0) first_e = lo;
  }
  if (warp == 0) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();  // only now: a dependent may take tensor memory as it starts
  const uint32_t tmem = tmem_slot;
  PmWalk w;
  w.e = first_e;
  w.left = static_cast<int>(end - start);
  w.load(a, plan);
  {
    const int64_t in = start - plan.cum[w.e] * H;
    w.h = static_cast<int>(in / w.tiles);
    w.tile = static_cast<int>(in - static_cast<int64_t>(w.h) * w.tiles);
  }
  w.seg_first = start - w.tile;
  w.count = min(w.left, w.tiles - w.tile);

  if (warp < 4) {
    // ------------------------------------------------------------ products
    regs_dec<64>();
    if (warp == 0) {
      // The whole warp walks and waits; one elected lane issues.  (With the
      // walk itself inside a one-lane branch a product cost about 300 clocks to
      // issue, ten times the tensor core's: its operands were not known to be
      // uniform.)
      constexpr uint32_t kQk = idesc_f16(128, 64, false), kPv = idesc_f16(128, D, true);
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const uint64_t q_desc = sw128_kmajor_desc(smem_u32(q_s)), k_desc = sw128_kmajor_desc(smem_u32(k_s));
      const uint64_t v_desc = sw128_mnmajor_desc(smem_u32(v_s), D > 64 ? kPanel : 16);
      uint32_t it = 0, q_phase = 0, p_phase = 0;  // bit i: tile i; p: bit 2i + h
      bool ok = true;
      const auto qk = [&](int i, int h, int s) {  // elected lane
        const uint64_t qa = q_desc + i * (kOperand >> 4), ka = k_desc + (s * kOperand + h * 64 * 128 >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * kPanel + (k & 3) * 32) >> 4;
          mma_f16_ss(tm + i * 128 + h * 64, qa + off, ka + off, kQk, k > 0);
        }
      };
      const auto s_ready = [&](int i, int h) {
        mma_commit(&s_full[i][h]);
        mbar_arrive(&s_full[i][h]);  // passes on what this thread saw of the unpacking warps' scales
      };
      for (; w.left > 0 && ok; w.next(a, plan)) {
        const int tiles = w.rows(group) > 128 ? 2 : 1;
        ok = warp_wait(&k_full[it & 1], it >> 1 & 1, &abort_flag);
        for (int i = 0; i < tiles && ok; ++i) {
          ok = warp_wait(&q_full[i], q_phase >> i & 1, &abort_flag);
          if (!ok) break;
          q_phase ^= 1u << i;
          tc_fence_after();
          if (elect_one()) {
            for (int h = 0; h < 2; ++h) {
              qk(i, h, it & 1);
              s_ready(i, h);
            }
            if (i + 1 == tiles) mma_commit(&k_empty[it & 1]);
          }
          __syncwarp();
        }
        for (int j = 0; j < w.count && ok; ++j, ++it) {
          const int s = it & 1;
          const bool more = j + 1 < w.count;
          for (int x = 0; x < 2 * tiles; ++x) {
            const int h = x >= tiles, i = h ? x - tiles : x;
            ok = warp_wait(&p_full[i][h], p_phase >> (2 * i + h) & 1, &abort_flag);
            if (x == 0) ok = ok && warp_wait(&v_full[s], it >> 1 & 1, &abort_flag);
            if (x == 0 && more) ok = ok && warp_wait(&k_full[s ^ 1], (it + 1) >> 1 & 1, &abort_flag);
            if (!ok) break;
            p_phase ^= 1u << (2 * i + h);
            tc_fence_after();
            if (elect_one()) {
              const uint64_t va = v_desc + (s * kOperand + h * 64 * 128 >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_f16_ts(tm + 256 + i * D, tm + i * 128 + h * 64 + k * 8, va + k * (2048 >> 4), kPv, x >= tiles || j > 0 || k > 0);
              if (more) qk(i, h, s ^ 1);
              s_ready(i, h);  // after the last tile: O has taken this half's weights
              if (x + 1 == 2 * tiles) {
                mma_commit(&v_empty[s]);
                if (more) mma_commit(&k_empty[s ^ 1]);
              }
            }
            __syncwarp();
          }
        }
      }
      if (!ok && elect_one()) {  // let the products in flight end before tensor memory goes
        mma_commit(&v_empty[0]);
        mbar_wait_drain(&v_empty[0], 0, 1ll << 24);
        __nanosleep(100000);
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------ unpacking: thread = token of the tile
    regs_dec<96>();
    const int tk = tid - 128;
    const float scale2 = a.scale * 1.4426950408889634f;
    const int page_log2 = a.cache.page_log2;
    const int64_t to_value = static_cast<int64_t>(H) << page_log2;
    constexpr int kVec = D / 32;  // 16-byte loads of a row's codes
    PmWalk n = w;  // one unit ahead of w
    int left = w.left;
    uint4 kr[kVec], vr[kVec];
    uint32_t km, vm;
    int64_t row;   // of the token whose codes are loaded next, or -1
    bool page_ok;  // false: the table names a page that does not exist
    const auto look_up = [&] {
      const int64_t token = static_cast<int64_t>(n.tile) * kPmTile + tk;
      row = -1;
      page_ok = true;
      if (token < n.kv) {
        const int id = a.table[static_cast<int64_t>(n.b) * a.table_stride + (token >> page_log2)];
        page_ok = id >= 0 && id < a.cache.pages;
        if (page_ok)
          row = ((static_cast<int64_t>(id) * 2 * H + n.h) << page_log2) + (token & ((1 << page_log2) - 1));
        else
          record_status(kStatusBounds);
      }
    };
    const auto load = [&](int64_t r, uint4 (&codes)[kVec], uint32_t &meta) {
      meta = 0;
#pragma unroll
      for (int i = 0; i < kVec; ++i) codes[i] = make_uint4(0, 0, 0, 0);
      if (r >= 0) {
        meta = a.cache.meta[r];
        const uint4 *src = reinterpret_cast<const uint4 *>(a.cache.codes + r * (D / 2));
#pragma unroll
        for (int i = 0; i < kVec; ++i) codes[i] = src[i];
      }
    };
    const auto store = [&](uint8_t *to, const uint4 (&codes)[kVec], uint32_t meta) {
      const uint32_t z = meta >> 16 & 15u;
      const uint32_t zlo = 0xE400E400u | z * 0x00010001u, zhi = 0xD400D400u | z * 0x00100010u;
      uint8_t *line = to + tk * 128;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const uint32_t words[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int chunk = 4 * i + j;
          *reinterpret_cast<uint4 *>(line + (chunk >> 3) * kPanel + (((chunk & 7) ^ (tk & 7)) << 4)) =
              unpack_codes(words[j], zlo, zhi);
        }
      }
      fence_proxy_async_smem();
    };
    look_up();
    load(row, kr, km);
    load(row < 0 ? row : row + to_value, vr, vm);
    bool ok_now = page_ok;
    for (uint32_t it = 0; left > 0; --left, ++it) {
      const int s = it & 1;
      const uint32_t phase = it >> 1 & 1;
      // the next unit
      if (left > 1) {
        if (++n.tile == n.tiles) {
          n.tile = 0;
          if (++n.h == H) {
            n.h = 0;
            ++n.e;
            n.load(a, plan);
          }
        }
        look_up();
      }
      const bool next_ok = page_ok;
      if (!mbar_wait(&k_empty[s], phase ^ 1, &abort_flag)) break;
      const int at = it & (kPmScaleRing - 1);
      {
        const float2 ks = __half22float2(*reinterpret_cast<const __half2 *>(&km));
        const float2 vs = __half22float2(*reinterpret_cast<const __half2 *>(&vm));
        k_scale[at * kPmTile + tk] = ks.x * scale2;
        v_scale[at * kPmTile + tk] = vs.x;
        v_log[at * kPmTile + tk] = __log2f(fmaxf(vs.x, 0x1p-24f));
        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, ok_now);
        if (lane == 0) seen[at][warp - 4] = bits;
      }
      store(k_s + s * kOperand, kr, km);
      mbar_arrive(&k_full[s]);
      if (left > 1) load(row, kr, km);
      if (!mbar_wait(&v_empty[s], phase ^ 1, &abort_flag)) break;
      store(v_s + s * kOperand, vr, vm);
      mbar_arrive(&v_full[s]);
      if (left > 1) load(row < 0 ? row : row + to_value, vr, vm);
      ok_now = next_ok;
    }
  } else {
    // ------------------------------------------------------------ softmax: thread = row of a tile
    regs_inc<176>();
    const int i = (warp >> 2) - 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + i * 128, o_at = tmem + lanes + 256 + i * D;
    uint32_t it = 0, s_phase = 0;  // bit h: half h
    bool ok = true;
    for (; w.left > 0 && ok; it += w.count, w.next(a, plan)) {
      const int rows = w.rows(group);
      if (i * 128 >= rows) continue;
      const int row = w.pair * kPmRows + i * 128 + r;
      const bool valid = i * 128 + r < rows;
      const int tok = row / group, head = w.h * group + row - tok * group;
      const int64_t token = static_cast<int64_t>(w.q0) + tok;
      // Q: D / 8 lanes copy a row of the warp's 32, channels in the unpacked codes' order
      uint8_t *tile_s = q_s + i * kOperand;
      constexpr int kChunks = D / 8, kTogether = 32 / kChunks;
      const int chunk = lane % kChunks, first_rr = (warp & 3) * 32 + lane / kChunks;
      const int first_tok = (w.pair * kPmRows + i * 128 + first_rr) / group;
      const int first_head = w.pair * kPmRows + i * 128 + first_rr - first_tok * group;
      int tok2 = first_tok, head2 = first_head;  // of the row that this lane copies next
      const auto next_row = [&] {
        for (head2 += kTogether; head2 >= group; head2 -= group) ++tok2;
      };
#pragma unroll 8
      for (int k = 0; k < 32 / kTogether; ++k, next_row()) {
        const int rr = first_rr + k * kTogether;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (i * 128 + rr < rows)
          v = *reinterpret_cast<const uint4 *>(a.q + (static_cast<int64_t>(w.q0) + tok2) * a.q_stride +
                                               static_cast<int64_t>(w.h * group + head2) * D + chunk * 8);
        *reinterpret_cast<uint4 *>(tile_s + rr * 128 + (chunk >> 3) * kPanel + (((chunk & 7) ^ (rr & 7)) << 4)) =
            make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                       __byte_perm(v.y, v.w, 0x7632));
      }
      fence_proxy_async_smem();
      mbar_arrive(&q_full[i]);
      // keys this row sees; rows behind the last one see what the request has
      const int lim = valid && a.causal ? w.kv - w.n + tok + 1 : w.kv;
      const int lim_min = __shfl_sync(0xFFFFFFFFu, lim, 0);
      float ref = kKvNoMax;  // of the exponents; the first column that the row sees sets it
      uint64_t sum2 = 0;
      for (int jh = 0; jh < 2 * w.count; ++jh) {
        const int h = jh & 1, at = (it + (jh >> 1)) & (kPmScaleRing - 1);
        const int base = (w.tile + (jh >> 1)) * kPmTile + 64 * h;
        const uint32_t sh_at = s_at + 64 * h;
        ok = mbar_wait(&s_full[i][h], s_phase >> h & 1, &abort_flag);
        s_phase ^= 1u << h;
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float *ks = k_scale + at * kPmTile + 64 * h, *vs = v_scale + at * kPmTile + 64 * h,
                    *vl = v_log + at * kPmTile + 64 * h;
        const uint2 there = *reinterpret_cast<const uint2 *>(&seen[at][2 * h]);
        const bool whole = base + 64 <= lim_min && (there.x & there.y) == 0xFFFFFFFFu;
        // bit k: column 32 b + k is seen by this row
        const auto visible = [&](int b) {
          const int n = lim - base - 32 * b;
          return (b == 0 ? there.x : there.y) &
                 (n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u));
        };
        // the logarithm of the row's largest weight; a value scale of zero counts as 2^-24, so that the sum of
        // p stays finite, too
        const auto maximum = [&] {
          float top = -INFINITY;
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            uint32_t c[32];
            tmem_ld_32x32b_x32(sh_at + 32 * b, c);
            tmem_ld_wait();
            reg_fence(c);
            const uint32_t see = visible(b);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float v = fmaf(__uint_as_float(c[k]), ks[32 * b + k], vl[32 * b + k]);
              top = fmaxf(top, see >> k & 1u ? v : -INFINITY);
            }
          }
          return top;
        };
        // the row's weights p s_v, relative to the reference; adds sum p to sum2 and returns the largest weight
        uint32_t p[32];
        const auto weights = [&](auto all) {
          constexpr bool kAll = decltype(all)::value;
          const uint64_t ref2 = pack_f2(-ref, -ref);
          uint32_t x[2][32];
          float hi[2] = {0.0f, 0.0f};
          tmem_ld_32x32b_x32(sh_at, x[0]);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            uint32_t(&c)[32] = x[b];
            tmem_ld_wait();
            reg_fence(c);
            if (b == 0) tmem_ld_32x32b_x32(sh_at + 32, x[1]);
            const uint32_t see = kAll ? 0xFFFFFFFFu : visible(b);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const ulonglong2 f = lds_2x2f(ks + 32 * b + 4 * k), g = lds_2x2f(vs + 32 * b + 4 * k);
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const int at2 = 4 * k + 2 * q;
                float2 v = unpack_f2(
                    fma_f2(pack_f2(__uint_as_float(c[at2]), __uint_as_float(c[at2 + 1])), q ? f.y : f.x, ref2));
                if constexpr (!kAll) v.x = see >> at2 & 1u ? v.x : -INFINITY, v.y = see >> (at2 + 1) & 1u ? v.y : -INFINITY;
                const uint64_t e2 = pack_f2(ex2(v.x), ex2(v.y));
                sum2 = add_f2(sum2, e2);
                float2 pv = unpack_f2(mul_f2(e2, q ? g.y : g.x));
                // a value's scale may be NaN: select, not multiply
                if constexpr (!kAll) pv.x = see >> at2 & 1u ? pv.x : 0.0f, pv.y = see >> (at2 + 1) & 1u ? pv.y : 0.0f;
                hi[q] = fmaxf(fmaxf(hi[q], pv.x), pv.y);
                p[16 * b + 2 * k + q] = half2_bits(pv.x, pv.y);
              }
            }
          }
          return fmaxf(hi[0], hi[1]);
        };
        // moves the reference there, and takes the sums along
        const auto move_to = [&](float to) {
          const float keep = ex2(ref - to);
          ref = to;
          sum2 = mul_f2(sum2, pack_f2(keep, keep));
          if (jh > 0) {
            // no product into O may be under way: this half's last one came before its s_full, the other
            // half's before the s_full that this thread waits for next
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&s_full[i][h ^ 1], s_phase >> (h ^ 1) & 1, &abort_flag))) return;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < D / 32; ++b) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(o_at + b * 32, o);
              tmem_ld_wait();
              reg_fence(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * keep);
              tmem_st_32x32b_x32(o_at + b * 32, o);
            }
          }
        };
        // A row's first scores set its reference before they are used.  Later ones are used with the reference
        // that there is, and once more where a weight passes it by too much, which is rare.
        for (bool set = __any_sync(0xFFFFFFFFu, ref == kKvNoMax);; set = true) {
          if (set) {
            const float to = maximum() - kPmLift;
            const bool move = to > ref + 8.0f;
            if (__any_sync(0xFFFFFFFFu, move)) move_to(move ? to : ref);
          }
          const uint64_t sum_before = sum2;
          const float top = whole ? weights(std::true_type{}) : weights(std::false_type{});
          const float2 s2 = unpack_f2(sum2);
          const bool over = top > kPmTopWeight || s2.x + s2.y > kPmTopSum;
          if (set || !__any_sync(0xFFFFFFFFu, over)) break;
          sum2 = sum_before;
        }
        tmem_st_32x32b_x32(sh_at, p);  // over the half's first columns
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[i][h]);
      }
      if (!ok) break;
      ok = mbar_wait(&s_full[i][0], s_phase & 1, &abort_flag) && mbar_wait(&s_full[i][1], s_phase >> 1 & 1, &abort_flag);
      ok = __all_sync(0xFFFFFFFFu, ok);
      s_phase ^= 3u;
      if (!ok) break;
      tc_fence_after();
      const float2 both = unpack_f2(sum2);
      const float sum = both.x + both.y;
      const bool cut = w.count < w.tiles;
      const int side = start <= w.seg_first ? 1 : 0;  // the block's end cuts it, or its beginning
      float *part = parts + (static_cast<int64_t>(c) * 2 + side) * C::kPart;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // a row that saw no key is zero
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(o_at + b * 32, o);
        tmem_ld_wait();
        reg_fence(o);
#pragma unroll
        for (int k = 0; k < 32; k += 8) {  // columns 0 4 1 5 2 6 3 7 back in order
          float v[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) v[x] = __uint_as_float(o[k + (x < 4 ? 2 * x : 2 * x - 7)]);
          const int ch = 4 * b + k / 8;
          if (cut) {  // four channels of all rows together: neighbouring rows are neighbouring lanes
            float4 *dst = reinterpret_cast<float4 *>(part) + 2 * ch * kPmRows + i * 128 + r;
            dst[0] = make_float4(v[0], v[1], v[2], v[3]);
            dst[kPmRows] = make_float4(v[4], v[5], v[6], v[7]);
          } else {  // by way of Q's place, which no product reads any more
            *reinterpret_cast<uint4 *>(tile_s + r * 128 + (ch >> 3) * kPanel + (((ch & 7) ^ (r & 7)) << 4)) =
                make_uint4(half2_bits(v[0] * inv, v[1] * inv), half2_bits(v[2] * inv, v[3] * inv),
                           half2_bits(v[4] * inv, v[5] * inv), half2_bits(v[6] * inv, v[7] * inv));
          }
        }
      }
      if (!cut) {
        __syncwarp();
        tok2 = first_tok, head2 = first_head;
#pragma unroll 8
        for (int k = 0; k < 32 / kTogether; ++k, next_row()) {
          const int rr = first_rr + k * kTogether;
          if (i * 128 + rr >= rows) continue;
          *reinterpret_cast<uint4 *>(a.out + (static_cast<int64_t>(w.q0) + tok2) * a.out_stride +
                                     static_cast<int64_t>(w.h * group + head2) * D + chunk * 8) =
              *reinterpret_cast<const uint4 *>(tile_s + rr * 128 + (chunk >> 3) * kPanel + (((chunk & 7) ^ (rr & 7)) << 4));
        }
        __syncwarp();
      }
      tc_fence_before();
      if (cut) {
        *reinterpret_cast<float2 *>(part + static_cast<int64_t>(kPmRows) * D + 2 * (i * 128 + r)) = make_float2(ref, sum);
        if (tid == 256 && side == 1)  // the segment's last block: unit x is in block ((x + 1) P - 1) / U
          plan.cuts[c] = PmCut{static_cast<int>(((w.seg_first + w.tiles) * P - 1) / U), w.pair, w.h, w.q0, w.n};
      } else if (valid && a.lse) {
        a.lse[token * a.Hq + head] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
      }
    }
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Joins a cut segment's parts, 32 rows a block: lane = row, a warp an eighth of
// the channels.  Block x's parts are those of the segment that block x of the
// kernel before was the first to hold.
template <int D>
__global__ void __launch_bounds__(256) kv4_prompt_join_kernel(const AttendArgs a, const PmPlan plan,
                                                              const float *__restrict__ parts) {
  pdl_wait();
  using C = PmCfg<D>;
  const int c0 = blockIdx.x, group = a.Hq / a.cache.H;
  const PmCut cut = plan.cuts[c0];
  const int r = blockIdx.y * 32 + (threadIdx.x & 31), row = cut.pair * kPmRows + r;
  if (cut.last < c0 || row >= cut.n * group) return;
  constexpr int kVec = D / 32;  // of four channels
  const int k0 = (threadIdx.x >> 5) * kVec;
  // the segment is the first block's last one and every other's first one
  const auto part_of = [&](int b) { return parts + (static_cast<int64_t>(b) * 2 + (b == c0 ? 1 : 0)) * C::kPart; };
  const auto ref_of = [&](int b) {
    return *reinterpret_cast<const float2 *>(part_of(b) + static_cast<int64_t>(kPmRows) * D + 2 * r);
  };
  float top = -INFINITY, sum = 0.0f;
#pragma unroll 4
  for (int b = c0; b <= cut.last; ++b) top = fmaxf(top, ref_of(b).x);
  float4 acc[kVec];
#pragma unroll
  for (int k = 0; k < kVec; ++k) acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
  for (int b = c0; b <= cut.last; ++b) {
    const float2 rl = ref_of(b);
    const float f = ex2(rl.x - top);
    sum = fmaf(rl.y, f, sum);
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      const float4 v = reinterpret_cast<const float4 *>(part_of(b))[(k0 + k) * kPmRows + r];
      acc[k].x = fmaf(v.x, f, acc[k].x), acc[k].y = fmaf(v.y, f, acc[k].y);
      acc[k].z = fmaf(v.z, f, acc[k].z), acc[k].w = fmaf(v.w, f, acc[k].w);
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int tok = row / group, head = cut.h * group + row - tok * group;
  const int64_t token = static_cast<int64_t>(cut.q0) + tok;
  uint4 *dst = reinterpret_cast<uint4 *>(a.out + token * a.out_stride + static_cast<int64_t>(head) * D + 4 * k0);
#pragma unroll
  for (int k = 0; k < kVec; k += 2) {
    const float4 u = acc[k], v = acc[k + 1];
    dst[k / 2] = make_uint4(half2_bits(u.x * inv, u.y * inv), half2_bits(u.z * inv, u.w * inv),
                            half2_bits(v.x * inv, v.y * inv), half2_bits(v.z * inv, v.w * inv));
  }
  if (a.lse && k0 == 0) a.lse[token * a.Hq + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

// Most tile pairs a call can have.
static int64_t pm_max_entries(int B, int max_q, int group) {
  return static_cast<int64_t>(B) * ((static_cast<int64_t>(max_q) * group + kPmRows - 1) / kPmRows);
}
constexpr size_t kPmPlanHead = 4096;  // entries, then the blocks' cuts from byte 256
static_assert(256 + kPmMaxGrid * sizeof(PmCut) <= kPmPlanHead, "room for the cuts");
static size_t pm_plan_bytes(int64_t entries) { return (kPmPlanHead + (entries + 1) * 8 + entries * 8 + 255) / 256 * 256; }

static size_t kv4_prompt_workspace_bytes(int B, int max_q, int group, int D) {
  return kKvCounterBytes + pm_plan_bytes(pm_max_entries(B, max_q, group)) +
         static_cast<size_t>(kPmMaxGrid) * 2 * kPmRows * (D + 2) * sizeof(float);
}

template <int D>
static cudaError_t launch_kv4_prompt(const AttendArgs &a, void *ws, cudaStream_t stream, const char **msg) {
  using C = PmCfg<D>;
  auto kern = kv4_prompt_kernel<D>;
  static std::atomic<unsigned long long> configured{0};  // one bit per device ordinal
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !(configured.load() & (1ull << dev))) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kv4_prompt_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kKv4MaxRequests * static_cast<int>(sizeof(int)));
    if (e != cudaSuccess) {
      *msg = "cudaFuncSetAttribute(MaxDynamicSharedMemorySize) failed";
      return e;
    }
    if (dev < 64) configured.fetch_or(1ull << dev);
  }
  const int group = a.Hq / a.cache.H;
  const int64_t entries = pm_max_entries(a.B, a.max_q, group);
  uint8_t *at = static_cast<uint8_t *>(ws) + kKvCounterBytes;
  PmPlan plan;
  plan.entries = reinterpret_cast<int *>(at);
  plan.cuts = reinterpret_cast<PmCut *>(at + 256);
  plan.cum = reinterpret_cast<int64_t *>(at + kPmPlanHead);
  plan.ent = reinterpret_cast<int2 *>(at + kPmPlanHead + (entries + 1) * 8);
  float *parts = reinterpret_cast<float *>(at + pm_plan_bytes(entries));
  const int64_t tiles = ((static_cast<int64_t>(a.W) << a.cache.page_log2) + kPmTile - 1) / kPmTile;
  const int64_t units = entries * a.cache.H * (tiles > 0 ? tiles : 1);
  int64_t grid = device_sm_count();
  if (grid > kPmMaxGrid) grid = kPmMaxGrid;
  if (grid > units) grid = units;
  kv4_prompt_plan_kernel<<<1, kPmPlanThreads, a.B * sizeof(int), stream>>>(a, plan);
  cudaError_t e = cudaGetLastError();
  // the other two start while the one before them ends, and wait for its results themselves
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kPmThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kern, a, plan, parts);
  cfg.gridDim = dim3(static_cast<unsigned>(grid), kPmRows / 32);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kv4_prompt_join_kernel<D>, a, plan, static_cast<const float *>(parts));
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) *msg = "launch of the prompt attention failed";
  return e;
}

// ---------------------------------------------------------------------------
// Which kernel: the decode kernel takes requests of up to 16 rows per key head
// (its second 8-row tile costs a quarter more than one), above that the tensor
// core's 128-row tiles.
// ---------------------------------------------------------------------------
static bool kv4_is_decode(int max_q, int group) { return static_cast<int64_t>(max_q) * group <= 16; }

size_t kv4_attention_workspace_bytes(int B, int max_q, int Hq, int H, int D) {
  return kv4_is_decode(max_q, Hq / H) ? kv4_decode_workspace_bytes(max_q, Hq / H, D)
                                      : kv4_prompt_workspace_bytes(B, max_q, Hq / H, D);
}

cudaError_t launch_kv4_attention(const AttendArgs &a, void *ws, cudaStream_t stream, const char **msg) {
  if (kv4_is_decode(a.max_q, a.Hq / a.cache.H)) return launch_kv4_decode(a, ws, stream, msg);
  return a.cache.D == 128 ? launch_kv4_prompt<128>(a, ws, stream, msg) : launch_kv4_prompt<64>(a, ws, stream, msg);
}

}  // namespace mixllm
