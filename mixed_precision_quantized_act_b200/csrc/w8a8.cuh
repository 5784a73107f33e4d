// w8a8.cuh -- the linear layer in 8-bit integers with one scale per token and
// one per output channel:
//   Y[m, n] = fp16( float(sum_k A[m, k] W[n, k]) * s_a[m] * s_w[n] + bias[n] ),
// its quantizers (activations and weights alike: one scale per row) and the
// product on the int8 tensor cores.
#pragma once

#include <cuda_fp16.h>
#include <atomic>
#include <cstdint>

#include "gemm_w4w8a8.cuh"  // device_sm_count, tensor maps
#include "kv4_ptx.cuh"      // elect_one
#include "launch.h"
#include "norm.cuh"
#include "ptx_sm100.cuh"
#include "quant.cuh"

namespace mixllm {

// ---------------------------------------------------------------------------
// One scale per row: amax over the row's K values, s = amax / 127 (IEEE fp32),
// codes rne(x / s) by the fp32 quotient, within +-127; a row of zeros gets s = 0
// and codes 0, one with a NaN or an infinity s = NaN and codes 0.  A block takes
// a row, which stays in registers up to V runs of eight a thread and is read
// again from there on.
// ---------------------------------------------------------------------------
template <typename T>
struct RowRun;  // eight values as loaded; top(): their largest magnitude, NaN or infinity if one is
template <>
struct RowRun<__half> {
  uint4 raw;
  __device__ __forceinline__ void load(const __half *p) { raw = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void widen(float (&f)[8]) const { widen8(raw, f); }
  __device__ __forceinline__ float top() const {
    const __half2 *h = reinterpret_cast<const __half2 *>(&raw);
    const __half2 m = __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])), __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
    return __half2float(__hmax_nan(__low2half(m), __high2half(m)));
  }
};
template <>
struct RowRun<float> {
  float4 lo, hi;
  __device__ __forceinline__ void load(const float *p) {
    lo = *reinterpret_cast<const float4 *>(p);
    hi = *reinterpret_cast<const float4 *>(p + 4);
  }
  __device__ __forceinline__ void widen(float (&f)[8]) const {
    f[0] = lo.x, f[1] = lo.y, f[2] = lo.z, f[3] = lo.w, f[4] = hi.x, f[5] = hi.y, f[6] = hi.z, f[7] = hi.w;
  }
  __device__ __forceinline__ float top() const {
    float f[8], m = 0.0f;
    widen(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fabsf(f[i]) <= 3.4028234663852886e38f ? fmaxf(m, fabsf(f[i])) : INFINITY;
    return m;
  }
};

template <typename T, int V>
__global__ void __launch_bounds__(1024) row_quantize_kernel(const T *__restrict__ X, int64_t stride, int K,
                                                            int8_t *__restrict__ codes, float *__restrict__ scales) {
  __shared__ float warp_max[32];
  pdl_wait();
  pdl_launch_dependents();  // behind all that came before this kernel: a dependent may read the weights at once
  const int64_t m = blockIdx.x;
  const T *row = X + m * stride;
  const int step = blockDim.x * 8, k0 = threadIdx.x * 8, lane = threadIdx.x & 31;
  RowRun<T> run[V];
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (k0 + v * step < K) run[v].load(row + k0 + v * step);
  float amax = 0.0f;
  const auto look = [&](const RowRun<T> &r) {
    const float top = r.top();
    amax = fmaxf(amax, top == top ? top : INFINITY);
  };
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (k0 + v * step < K) look(run[v]);
  for (int k = k0 + V * step; k < K; k += step) {
    RowRun<T> r;
    r.load(row + k);
    look(r);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  if (lane == 0) warp_max[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = lane < (blockDim.x >> 5) ? warp_max[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  const float s = amax == INFINITY ? __int_as_float(0x7FFFFFFF) : __fdiv_rn(amax, 127.0f);
  if (threadIdx.x == 0) scales[m] = s;
  const bool none = !(s > 0.0f);
  const QuantStep q = QuantStep::of(none ? 1.0f : s);
  const auto store = [&](const RowRun<T> &r, int k) {
    uint32_t packed[2] = {0u, 0u};
    if (!none) {
      float f[8];
      r.widen(f);
      if constexpr (sizeof(T) == 2) {
        q.codes(f, packed);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = max(-127, min(127, __float2int_rn(__fdiv_rn(f[i], s))));
          packed[i >> 2] |= (static_cast<uint32_t>(c) & 0xFFu) << ((i & 3) * 8);
        }
      }
    }
    *reinterpret_cast<uint2 *>(codes + m * K + k) = make_uint2(packed[0], packed[1]);
  };
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (k0 + v * step < K) store(run[v], k0 + v * step);
  for (int k = k0 + V * step; k < K; k += step) {
    RowRun<T> r;
    r.load(row + k);
    store(r, k);
  }
}

template <typename T>
static cudaError_t launch_row_quantize(const T *X, int64_t stride, int64_t M, int64_t K, int8_t *codes, float *scales,
                                       cudaStream_t stream) {
  // Few rows: a run a thread, for latency (above K = 8192 a block has not the threads).  Many: four or six, so that what a block does once costs each value less
  // (2047 rows of 14336: two a thread 36 us, four 24, six 21; 4096 of 4096: two 14.7, four 12.0, six 12.7).
  const int64_t runs = K / 8;
  const int each = M < 512 && runs <= 1024 ? 1 : runs <= 1024 ? 4 : 6;
  int64_t threads = ((runs + each - 1) / each + 31) / 32 * 32;
  if (threads > 1024) threads = 1024;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // starts while the kernel before it ends
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(M));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kern = each == 1 ? row_quantize_kernel<T, 1> : each == 4 ? row_quantize_kernel<T, 4> : row_quantize_kernel<T, 6>;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, X, stride, static_cast<int>(K), codes, scales);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

// ---------------------------------------------------------------------------
// The product.  Channels are the tensor core's 128-row side and tokens its
// column side (NT of them, 16 to 64 here), so that a few tokens cost no more than
// their columns and the weights stream through shared memory at any number of
// tokens.  A tile's K is cut into S even shares, one for each block of a cluster
// (S = 1: none), so that few tiles still use every SM; a block of no cluster
// takes tiles in turn, an even run of them.
//
// Warp 0 loads both operands by TMA (128-byte swizzle), warp 1 issues
// tcgen05.mma kind::i8, warps 4-11 are the epilogue: thread = channel, four warps
// to one half of the tokens.  They scale the accumulator and write Y by way of
// shared memory, 16 bytes a lane, while the next tile's products run (two
// accumulators in tensor memory).  The blocks of a cluster give each other their
// parts through distributed shared memory, each block adding four tokens at a time
// of its own share: whole numbers, so the sum does not depend on who was first.
//
// A few tokens are bound by the weights' bytes.  Two blocks an SM with 90 KB of
// copies under way each serve that better than one with 200 (224 tiles would load the
// SMs unevenly), but for few tiles (w8a8_plan); the first copies of the weights start while the quantizer still runs.  Measured on B200 (graph of quantizer and
// product, weights from HBM): 1 token, 4096 -> 6144: 9.0 us (weights alone 3.8; the
// product by itself 7.7: its blocks run 7 us, 5 of them for the weights, 0.8 for the
// exchange of parts), 37 tokens, 4096 -> 28672: 23 us, 5.2 TB/s.  Parts left in global
// memory for the last block to join them took 14.7 and 31 us.
// ---------------------------------------------------------------------------
constexpr int kW8Threads = 384;
constexpr int kW8Rows = 128;   // channels of a tile
constexpr int kW8Chunk = 128;  // values of K of a chunk

// Walks a block's chunks: tile by tile, tokens innermost, n chunks of K from k0 on.
struct W8Walk {
  int rt, tt, chunk, TT, k0, k1;

  __device__ __forceinline__ W8Walk(int tile, int token_tiles, int first, int end) : chunk(first), TT(token_tiles), k0(first), k1(end) {
    rt = tile / TT, tt = tile - rt * TT;
  }
  __device__ __forceinline__ void next() {
    if (++chunk == k1) {
      chunk = k0;
      if (++tt == TT) tt = 0, ++rt;
    }
  }
};

// kAlone: one block an SM, with a deeper ring of stages.  kApart: a cluster's parts have a place of their own, not that
// of the operands (a barrier of the cluster less: 1 token, 4096 -> 4096, 8.5 against 8.0 us); two blocks of 32
// or 64 tokens have no room for it.
template <int NT, bool kAlone = false>
struct W8Cfg {
  static constexpr int kStageW = kW8Rows * kW8Chunk, kStageA = NT * kW8Chunk, kStage = kStageW + kStageA;
  static constexpr int kCols = NT / 2 < 32 ? NT / 2 : 32;  // tokens of one load from tensor memory
  static constexpr int kOutCols = kCols < 16 ? kCols : 16;  // and of one round through shared memory
  static constexpr int kOut = 8 * kOutCols * 32 * 2;       // bytes: eight warps' tokens x 32 channels, fp16
  static constexpr int kGroups = NT / 4;  // of four tokens
  // parts that a block receives: of each block of the cluster, its groups' tokens x channels, int32
  static constexpr int received(int S) { return S * ((kGroups + S - 1) / S) * 4 * kW8Rows * 4; }
  static constexpr bool kApart = kAlone || NT == 16;
  static constexpr int kParts = !kApart ? 0 : received(3) > received(4) ? received(3) : received(4);
  static constexpr int kRoom = (kAlone ? 224 : 112) * 1024 - kOut - kParts - 1024 - 2 * NT * 4;
  static constexpr int kMost = kAlone ? 12 : 8;
  static constexpr int kStages = kRoom / kStage < kMost ? kRoom / kStage : kMost;
  static constexpr int kSmem = kStages * kStage + kOut + kParts + 1024;
  // Chunks of weights that are asked for while the quantizer runs: more would make its own loads wait (1 token,
  // 4096 -> 4096: none 8.65 us, three 8.45, five 8.7; a block alone, 14336 -> 4096, 64 tokens: none 18.8, three
  // 18.1, four 18.5).
  static constexpr int kEarly = 3;
  static_assert(kEarly < kStages, "the early chunks lie in the ring");
  static constexpr int kTmem = 2 * NT < 32 ? 32 : 2 * NT;
  static_assert(kApart || (received(2) <= kStages * kStage && received(4) <= kStages * kStage), "parts in the operands' place");
  static_assert((kAlone ? 1 : 2) * (kSmem + 2048) <= 227 * 1024, "the blocks of an SM");
};

struct W8Job {
  const float *s_a, *s_w;
  const __half *bias;  // or null
  __half *Y;
  int64_t M, N;
  int KC;      // chunks along K
  int TT;      // token tiles
  int tiles;   // S = 1: of the run that the blocks share
  int S;
  bool early;  // the kernel before this one does not write W: its loads need not wait
  bool wide;   // Y may be written 16 bytes at a time
};

// A whole tile's accumulator (128 channels from ch0 x NT tokens from m0) once `full` completes: scaled, and written
// by way of `out`.  Warps 4-11, which go on together or not at all (false).
template <typename C, int NT>
__device__ __forceinline__ bool w8_write_tile(const W8Job &a, int64_t ch0, int64_t m0, uint32_t tmem, uint64_t *full,
                                              uint32_t parity, float *token_scale, uint8_t *out, volatile int *abort) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int half = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
  const int64_t ch = ch0 + r, ch8 = ch0 + (warp & 3) * 32 + (lane & 3) * 8;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(NT), a.M - m0));
  out += (warp - 4) * (C::kOutCols * 64);
  for (int j = tid - 128; j < NT; j += 256) token_scale[j] = j < tokens ? a.s_a[m0 + j] : 0.0f;
  const float sw = ch < a.N ? a.s_w[ch] : 0.0f;
  const float bias = a.bias && ch < a.N ? __half2float(a.bias[ch]) : 0.0f;
  if (!named_bar_and(1, 256, warp_wait(full, parity, abort))) return false;  // also publishes the scales; warps arrive whole
  tc_fence_after();
  const uint32_t at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
#pragma unroll 1
  for (int j0 = half * (NT / 2); j0 < (half + 1) * (NT / 2) && j0 < tokens; j0 += C::kCols) {
    uint32_t v[C::kCols];
    tmem_ld_cols(at + j0, v);
    tmem_ld_wait();
    reg_fence(v);
    const float *scale = token_scale + j0;
#pragma unroll
    for (int j = 0; j < C::kCols; j += 4) {
      const float4 sa = *reinterpret_cast<const float4 *>(scale + j);
      const float f[4] = {sa.x, sa.y, sa.z, sa.w};
#pragma unroll
      for (int x = 0; x < 4; ++x)
        v[j + x] = __float_as_uint(fmaf(static_cast<float>(static_cast<int32_t>(v[j + x])) * f[x], sw, bias));
    }
    if (a.wide) {
      // 32 channels of kOutCols tokens at a time; lane = 8 channels of every eighth token
#pragma unroll
      for (int j1 = 0; j1 < C::kCols; j1 += C::kOutCols) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < C::kOutCols; ++j)
          *reinterpret_cast<__half *>(out + j * 64 + lane * 2) = __float2half_rn(__uint_as_float(v[j1 + j]));
        __syncwarp();
        __half *to = a.Y + (m0 + j0 + j1 + (lane >> 2)) * a.N + ch8;
#pragma unroll
        for (int j = 0; j < C::kOutCols; j += 8)
          if (j0 + j1 + j + (lane >> 2) < tokens && ch8 < a.N)
            *reinterpret_cast<uint4 *>(to + j * a.N) =
                *reinterpret_cast<const uint4 *>(out + (j + (lane >> 2)) * 64 + (lane & 3) * 16);
      }
    } else if (ch < a.N) {
      __half *to = a.Y + (m0 + j0) * a.N + ch;
#pragma unroll
      for (int j = 0; j < C::kCols; ++j)
        if (j0 + j < tokens) to[j * a.N] = __float2half_rn(__uint_as_float(v[j]));
    }
  }
  return true;
}

template <int NT, bool kAlone>
__global__ void __launch_bounds__(kW8Threads, 2)
    w8a8_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a, const W8Job a) {
  using C = W8Cfg<NT, kAlone>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ uint64_t full[C::kStages], empty[C::kStages], acc_full[2], acc_empty[2], drained;
  __shared__ __align__(16) float token_scale[2][NT];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // ---- this block's tiles, and its share of their K
  int tile0, tile1, k0 = 0, k1 = a.KC;
  if (a.S > 1) {
    const int r = static_cast<int>(cluster_rank());
    tile0 = static_cast<int>(blockIdx.x) / a.S, tile1 = tile0 + 1;
    k0 = a.KC * r / a.S, k1 = a.KC * (r + 1) / a.S;
  } else {
    const int P = gridDim.x, share = a.tiles / P, rest = a.tiles - share * P, c = blockIdx.x;
    tile0 = share * c + min(c, rest), tile1 = tile0 + share + (c < rest ? 1 : 0);
  }
  const int chunks = (tile1 - tile0) * (k1 - k0);
  const auto weights = [&](int s, const W8Walk &w) {
    mbar_arrive_expect_tx(&full[s], C::kStage);
    tma_load_2d(smem + s * C::kStage, &tm_w, &full[s], w.chunk * kW8Chunk, w.rt * kW8Rows);
  };
  int ahead = 0;  // chunks whose weights are under way
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 256);
    }
    mbar_init(&drained, 1);
    fence_mbar_init();
    fence_proxy_async_smem();
    abort_flag = 0;
  }
  __syncwarp();
  if (warp == 0 && a.early) {
    for (W8Walk w(tile0, a.TT, k0, k1); ahead < C::kEarly && ahead < chunks; ++ahead, w.next()) {
      if (elect_one()) weights(ahead, w);
      __syncwarp();
    }
  }
  if (warp == 2) {
    tmem_alloc(&tmem_slot, C::kTmem);
    tmem_relinquish();
  }
  if (tid == 96) prefetch_tmap(&tm_a);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();  // only now: a dependent may take tensor memory as it starts
  const uint32_t tmem = tmem_slot;
  // This block runs: others may write to its shared memory.  Relaxed: a release would wait for this warp's copies
  // of weights (9.8 instead of 9.0 us, 1 token, 4096 -> 6144).
  if (C::kApart && a.S > 1) cluster_arrive_relaxed();

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    // The whole warp walks and waits, an elected lane issues: from a one-lane branch 512 tokens x 4096 x 4096 took
    // 13.1 us instead of 12.4.
    pdl_wait();
    const auto tokens = [&](int s, const W8Walk &w) {
      tma_load_2d(smem + s * C::kStage + C::kStageW, &tm_a, &full[s], w.chunk * kW8Chunk, w.tt * NT);
    };
    int s = 0, issued = 0;
    uint32_t phase = 1;
    W8Walk w(tile0, a.TT, k0, k1);
    for (; issued < ahead; ++issued, ++s, w.next()) {
      if (elect_one()) tokens(s, w);
      __syncwarp();
    }
    for (; issued < chunks; ++issued, w.next()) {
      if (issued >= C::kStages && !warp_wait(&empty[s], phase, &abort_flag)) break;
      if (elect_one()) {
        weights(s, w);
        tokens(s, w);
      }
      __syncwarp();
      if (++s == C::kStages) s = 0, phase ^= 1;
    }
    if (abort_flag) {  // the last copies into each stage land before the block's memory goes to another
      for (int i = 0; i < C::kStages && i < issued; ++i)
        mbar_wait_drain(&full[i], static_cast<uint32_t>((issued - 1 - i) / C::kStages & 1), 1ll << 24);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    constexpr uint32_t kIdesc = idesc_i8(kW8Rows, NT);
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    const uint64_t w_desc = sw128_kmajor_desc(smem_u32(smem)), a_desc = sw128_kmajor_desc(smem_u32(smem) + C::kStageW);
    int s = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = 0; i < tile1 - tile0 && ok; ++i) {
      const int acc = i & 1;
      ok = warp_wait(&acc_empty[acc], (i >> 1 & 1) ^ 1, &abort_flag);
      for (int k = k0; k < k1 && ok; ++k) {
        ok = warp_wait(&full[s], phase, &abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t off = static_cast<uint64_t>(s * C::kStage >> 4);
#pragma unroll
          for (int j = 0; j < kW8Chunk / 32; ++j)
            mma_i8(tm + acc * NT, w_desc + off + 2 * j, a_desc + off + 2 * j, kIdesc, k > k0 || j > 0);
          mma_commit(&empty[s]);
          if (k + 1 == k1) mma_commit(&acc_full[acc]);
        }
        __syncwarp();
        if (++s == C::kStages) s = 0, phase ^= 1;
      }
    }
    if (!ok && elect_one()) {  // let the products in flight end before tensor memory goes
      mma_commit(&drained);
      mbar_wait_drain(&drained, 0, 1ll << 24);
    }
    __syncwarp();
  } else if (warp >= 4 && a.S == 1) {
    // ------------------------------------------------------------ scales and Y
    pdl_wait();  // s_a
    for (int tile = tile0, i = 0; tile < tile1; ++tile, ++i) {
      const int rt = tile / a.TT, tt = tile - rt * a.TT, acc = i & 1;
      if (!w8_write_tile<C, NT>(a, static_cast<int64_t>(rt) * kW8Rows, static_cast<int64_t>(tt) * NT, tmem + acc * NT,
                                &acc_full[acc], i >> 1 & 1, token_scale[acc], smem + C::kStages * C::kStage, &abort_flag))
        break;
      tc_fence_before();
      mbar_arrive(&acc_empty[acc]);
    }
  }
  if (a.S > 1) {
    // ------------------------------------------------------------ a cluster's parts: thread = channel
    const int S = a.S, me = static_cast<int>(cluster_rank()), half = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
    const int most = (C::kGroups + S - 1) / S;  // groups of a block
    uint8_t *parts = smem + (C::kApart ? C::kStages * C::kStage + C::kOut : 0);
    const auto first_group = [&](int b) { return (C::kGroups * b + S - 1) / S; };  // owner of group g: g S / kGroups
    const int rt = tile0 / a.TT, tt = tile0 - rt * a.TT;
    const int64_t ch = static_cast<int64_t>(rt) * kW8Rows + r, m0 = static_cast<int64_t>(tt) * NT;
    const int groups = static_cast<int>((min(static_cast<int64_t>(NT), a.M - m0) + 3) / 4);  // with tokens in them
    bool there = true;
    if (warp >= 4) there = mbar_wait(&acc_full[0], 0, &abort_flag);
    __syncwarp();
    tc_fence_after();
    if (!C::kApart) cluster_arrive();  // every block is done with its operands: parts take their place
    cluster_wait();
    if (warp >= 4 && __all_sync(0xFFFFFFFFu, there)) {
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t mine = smem_u32(parts) + static_cast<uint32_t>(me * most * kW8Rows + r) * 16;
#pragma unroll 1
      for (int j0 = half * (NT / 2); j0 < (half + 1) * (NT / 2) && j0 < groups * 4; j0 += C::kCols) {
        uint32_t v[C::kCols];
        tmem_ld_cols(tmem + lanes + j0, v);
        tmem_ld_wait();
        reg_fence(v);
#pragma unroll
        for (int j = 0; j < C::kCols; j += 4) {
          const int g = (j0 + j) / 4, owner = g * S / C::kGroups;
          const uint32_t at = mine + static_cast<uint32_t>((g - first_group(owner)) * kW8Rows) * 16;
          st_cluster_v4(cluster_map(at, owner), v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
      }
    }
    tc_fence_before();
    cluster_arrive();
    cluster_wait();
    if (warp >= 4) {
      pdl_wait();  // s_a, and Y's earlier readers
      const float sw = ch < a.N ? a.s_w[ch] : 0.0f;
      const float bias = a.bias && ch < a.N ? __half2float(a.bias[ch]) : 0.0f;
      const int g0 = first_group(me), g1 = min(first_group(me + 1), groups);
      for (int g = g0 + half; g < g1; g += 2) {
        const int64_t m = m0 + g * 4;
        float sa[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) sa[x] = m + x < a.M ? a.s_a[m + x] : 0.0f;
        int4 sum = make_int4(0, 0, 0, 0);
        const int4 *part = reinterpret_cast<const int4 *>(parts) + (g - g0) * kW8Rows + r;
        for (int b = 0; b < S; ++b) {
          const int4 v = part[b * most * kW8Rows];
          sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
        const int p[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (m + x < a.M && ch < a.N) a.Y[(m + x) * a.N + ch] = __float2half_rn(fmaf(static_cast<float>(p[x]) * sa[x], sw, bias));
      }
    }
  }
  __syncthreads();
  if (warp == 2) tmem_dealloc(tmem, C::kTmem);
}

// ---------------------------------------------------------------------------
// The same with two blocks on one product (cta_group::2): a tile is 256 channels
// x NT tokens, each block of a pair loads its 128 channels and half of the
// tokens, and the pair's tensor cores read both halves.  What bounds it is shared
// memory: a chunk of 256 tokens writes 32 KB and reads 64 KB of operands in some 660
// clocks, its products alone would take 512; one block's tiles of 128 x 256 write 48 KB.
// The loads of both complete on the first block's barriers, its warp 1 issues the
// products and frees the stages of both.
//
// Measured on B200: 2047 tokens, 14336 -> 4096: 80 us, 3.0 POP/s, 95 % of cuBLAS's
// int8 rate (one block a tile: 89 us; 128 tiles on 74 pairs are 2 rounds of 1.7); 4096
// tokens, 4096 -> 28672: 350 to 390 us; 512 tokens, 4096 -> 4096: 12.3 us.
// ---------------------------------------------------------------------------
template <int NT>
struct W8PairCfg {
  static constexpr int kStageW = kW8Rows * kW8Chunk, kStageA = NT / 2 * kW8Chunk, kStage = kStageW + kStageA;
  static constexpr int kCols = 32, kOutCols = 16, kOut = 8 * kOutCols * 32 * 2;
  static constexpr int kRoom = 224 * 1024 - kOut - 1024 - 2 * NT * 4;
  static constexpr int kStages = kRoom / kStage < 8 ? kRoom / kStage : 8;
  // Chunks of weights ahead of the quantizer's codes: none for tiles of 128 tokens (300 tokens, 4096 -> 6144: 14.5
  // against 15.0 us with three, 15.4 with all of the ring; 512 tokens, 4096 -> 4096: 15.8, 16.1, 16.3), three for 256
  // (130 tokens, 4096 -> 28672: 29.8, 29.6, 30.2).
  static constexpr int kEarly = NT == 128 ? 0 : 3;
  static_assert(kEarly < kStages, "the early chunks lie in the ring");
  static constexpr int kSmem = kStages * kStage + kOut + 1024;
  static constexpr int kTmem = 2 * NT;
};

template <int NT>
__global__ void __launch_bounds__(kW8Threads, 1)
    w8a8_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a, const W8Job a) {
  using C = W8PairCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ uint64_t full[C::kStages], empty[C::kStages], acc_full[2], acc_empty[2], drained;
  __shared__ __align__(16) float token_scale[2][NT];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5;
  const int side = static_cast<int>(cluster_rank());
  const int P = gridDim.x / 2, c = blockIdx.x / 2, share = a.tiles / P, rest = a.tiles - share * P;
  const int tile0 = share * c + min(c, rest), tile1 = tile0 + share + (c < rest ? 1 : 0);
  const int chunks = (tile1 - tile0) * a.KC;
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 512);
    }
    mbar_init(&drained, 1);
    fence_mbar_init();
    abort_flag = 0;
  }
  if (tid == 96) {
    prefetch_tmap(&tm_w);
    prefetch_tmap(&tm_a);
  }
  __syncwarp();
  cluster_arrive();
  if (warp == 2) {
    tmem_alloc_pair(&tmem_slot, C::kTmem);
    tmem_relinquish_pair();
  }
  cluster_wait();  // both blocks' barriers exist
  const auto weights = [&](int s, const W8Walk &w) {
    if (side == 0) mbar_arrive_expect_tx(&full[s], 2 * C::kStage);
    tma_load_2d_pair(smem + s * C::kStage, &tm_w, cluster_map(smem_u32(&full[s]), 0), w.chunk * kW8Chunk,
                     (2 * w.rt + side) * kW8Rows);
  };
  int ahead = 0;  // chunks whose weights are under way
  if (warp == 0 && a.early) {
    for (W8Walk w(tile0, a.TT, 0, a.KC); ahead < C::kEarly && ahead < chunks; ++ahead, w.next()) {
      if (elect_one()) weights(ahead, w);
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();  // only now: a dependent may take tensor memory as it starts
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ loads, each block's own
    pdl_wait();
    const auto tokens = [&](int s, const W8Walk &w) {
      tma_load_2d_pair(smem + s * C::kStage + C::kStageW, &tm_a, cluster_map(smem_u32(&full[s]), 0),
                       w.chunk * kW8Chunk, w.tt * NT + side * (NT / 2));
    };
    int s = 0;
    uint32_t phase = 1;
    W8Walk w(tile0, a.TT, 0, a.KC);
    for (; s < ahead; ++s, w.next()) {
      if (elect_one()) tokens(s, w);
      __syncwarp();
    }
    for (int issued = ahead; issued < chunks; ++issued, w.next()) {
      if (issued >= C::kStages && !warp_wait(&empty[s], phase, &abort_flag)) break;
      if (elect_one()) {
        weights(s, w);
        tokens(s, w);
      }
      __syncwarp();
      if (++s == C::kStages) s = 0, phase ^= 1;
    }
    __syncwarp();
  } else if (warp == 1 && side == 0) {
    // ------------------------------------------------------------ products, for both blocks
    constexpr uint32_t kIdesc = idesc_i8(2 * kW8Rows, NT);
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    const uint64_t w_desc = sw128_kmajor_desc(smem_u32(smem)), a_desc = sw128_kmajor_desc(smem_u32(smem) + C::kStageW);
    int s = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = 0; i < tile1 - tile0 && ok; ++i) {
      const int acc = i & 1;
      ok = warp_wait(&acc_empty[acc], (i >> 1 & 1) ^ 1, &abort_flag);
      for (int k = 0; k < a.KC && ok; ++k) {
        ok = warp_wait(&full[s], phase, &abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t off = static_cast<uint64_t>(s * C::kStage >> 4);
#pragma unroll
          for (int j = 0; j < kW8Chunk / 32; ++j)
            mma_i8_pair(tm + acc * NT, w_desc + off + 2 * j, a_desc + off + 2 * j, kIdesc, k > 0 || j > 0);
          mma_commit_pair(&empty[s], 3);
          if (k + 1 == a.KC) mma_commit_pair(&acc_full[acc], 3);
        }
        __syncwarp();
        if (++s == C::kStages) s = 0, phase ^= 1;
      }
    }
    if (!ok && elect_one()) {  // let the products in flight end before tensor memory goes
      mma_commit_pair(&drained, 1);
      mbar_wait_drain(&drained, 0, 1ll << 24);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ scales and Y, each block's own channels
    pdl_wait();  // s_a
    for (int tile = tile0, i = 0; tile < tile1; ++tile, ++i) {
      const int rt = tile / a.TT, tt = tile - rt * a.TT, acc = i & 1;
      if (!w8_write_tile<C, NT>(a, static_cast<int64_t>(2 * rt + side) * kW8Rows, static_cast<int64_t>(tt) * NT,
                                tmem + acc * NT, &acc_full[acc], i >> 1 & 1, token_scale[acc],
                                smem + C::kStages * C::kStage, &abort_flag))
        break;
      tc_fence_before();
      mbar_arrive_cluster(cluster_map(smem_u32(&acc_empty[acc]), 0));
    }
  }
  __syncwarp();
  if (abort_flag) __nanosleep(1000000);  // copies in flight land before the block's memory goes to another
  __syncthreads();
  cluster_arrive();  // neither block's barriers and tensor memory are in use any more
  cluster_wait();
  if (warp == 2) tmem_dealloc_pair(tmem, C::kTmem);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

struct W8Plan {
  int NT, KC, TT, S, tiles, grid;
  bool pair, alone;
};

// The clusters of S blocks of the kernels with one block an SM that fit on the current device at once (0 where the
// runtime cannot say): asked for the one of 64 tokens, the others are as large.
static int w8a8_clusters(int S) {
  using C = W8Cfg<64, true>;
  const auto kern = w8a8_kernel<64, true>;
  static std::atomic<int> known[64][5];  // by device ordinal and S, 1 + the number: what a device holds does not change
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && known[dev][S].load() > 0) return known[dev][S].load() - 1;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(S));
  cfg.blockDim = dim3(kW8Threads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (dev < 64) known[dev][S].store(n + 1);
  return n;
}

// False where the tiles and chunks pass 32 bits.
static bool w8a8_plan(int64_t M, int64_t N, int64_t K, W8Plan *plan) {
  W8Plan p{};
  const int64_t sms = device_sm_count();
  const int64_t rows = (N + kW8Rows - 1) / kW8Rows, pairs = (rows + 1) / 2;
  p.KC = static_cast<int>((K + kW8Chunk - 1) / kW8Chunk);
  p.NT = M <= 16 ? 16 : M <= 32 ? 32 : 64;
  // Two blocks on a tile where there are more tiles of 64 tokens and 128 channels than SMs (one tile an SM
  // is faster: 256 tokens, N = 4096 12.6 against 13.7 us, 128 tokens, N = 8192 12.9 against 13.9; more
  // than that: 100 tokens, N = 10240 15.7 against 14.3, 256 tokens, N = 6144 15.4 against 14.2).  A chunk of 128 tokens
  // takes some 250 ns, one of 256 some 350: whichever needs less for its rounds (N = 4096, the product by itself:
  // 512 tokens 12.4 against 15.1 us, 1024 tokens 19.8 against 15.9).
  const int64_t narrow = pairs * ((M + 127) / 128), broad = pairs * ((M + 255) / 256), slots = sms / 2;
  p.pair = M > 64 && rows * ((M + 63) / 64) > sms;
  if (p.pair) p.NT = M > 128 && (broad + slots - 1) / slots * 7 < (narrow + slots - 1) / slots * 5 ? 256 : 128;
  const int64_t TT = (M + p.NT - 1) / p.NT, tiles = (p.pair ? pairs : rows) * TT;
  if (tiles * p.KC > 0x7FFFFFFF) return false;
  p.TT = static_cast<int>(TT), p.tiles = static_cast<int>(tiles);
  p.S = 1;  // shares of K: as many as leave every cluster an SM to be on (N = 6144, one token: 4 8.2 us, 6 11.9 us)
  if (p.pair) {
    p.grid = static_cast<int>(tiles < sms / 2 ? tiles : sms / 2) * 2;
  } else {
    // One block an SM.  17 to 64 tokens: where that gives five eighths of the SMs a block and every cluster a place
    // (4096 -> 4096, 64 tokens: 9.6 against 10.5 us, 32 tokens: 8.7 against 9.1; 14336 -> 4096, 64 tokens: 18.1
    // against 20.2; 4096 -> 12288, 32 tokens: 12.4 against 14.9, 4096 -> 11904, 93 blocks: 12.3 against 14.8; with fewer,
    // 14336 -> 5888, 32 tokens, 92 blocks: 20.7 against 20.2).  Up to 16: where K then is not cut, but would be for
    // two blocks an SM (4096 -> 14336, 1 token: 13.8 against 14.4); with K cut both ways two blocks an SM are
    // better (4096 -> 6144: 9.0 against 9.4), and with neither (4096 -> 18432: 15.7 against 16.5).
    // K is cut while the shares leave an eighth of the places (two an SM) free, which clusters cannot all take, in
    // whole clusters of four (1 token, 4096 -> 16384, 256 shares: 16.4 us, not cut 15.0, of one block an SM 15.2;
    // 4096 -> 8192, 256 shares: 9.9; 4096 -> 8320, 130 shares: 10.7).
    const int64_t most = sms * 7 / 4 / 4 * 4;
    for (int S = 4; S >= 1 && !p.alone; --S)
      if ((p.NT > 16 || (S == 1 && tiles * 2 <= most)) && tiles * S <= sms && tiles * S * 8 >= sms * 5 &&
          S * 2 <= p.KC && (S == 1 || tiles <= w8a8_clusters(S)))
        p.alone = true, p.S = S;
    while (!p.alone && p.S < 4 && tiles * p.S * 2 <= most && p.S * 2 <= p.KC) p.S *= 2;
    p.grid = static_cast<int>(p.S > 1 ? tiles * p.S : tiles < 2 * sms ? tiles : 2 * sms);
  }
  *plan = p;
  return true;
}

// The layer from fp16 keeps the codes and scales of its activations.
size_t w8a8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M == 0 || N == 0) return 0;
  return (static_cast<size_t>(M) * K + 255) / 256 * 256 + (static_cast<size_t>(M) * 4 + 255) / 256 * 256;
}

template <typename C, typename Kernel>
static cudaError_t launch_w8a8_type(Kernel kern, const W8A8Args &a, const W8Plan &p, const CUtensorMap &tm_w,
                                    const CUtensorMap &tm_a, bool early, cudaStream_t stream, const char **msg) {
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
  const bool wide = a.N % 8 == 0 && (reinterpret_cast<uintptr_t>(a.Y) & 15) == 0;
  const W8Job job{a.s_a, a.s_w, a.bias, a.Y, a.M, a.N, p.KC, p.TT, p.tiles, p.S, early, wide};
  const int cluster = p.pair ? 2 : p.S;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // starts while the kernel before it ends
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.grid));
  cfg.blockDim = dim3(kW8Threads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tm_w, tm_a, job);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) *msg = "launch of the 8-bit product failed";
  return e;
}

template <int NT>
static cudaError_t launch_w8a8_tokens(const W8A8Args &a, const W8Plan &p, const CUtensorMap &tm_w,
                                      const CUtensorMap &tm_a, bool early, cudaStream_t stream, const char **msg) {
  return p.alone ? launch_w8a8_type<W8Cfg<NT, true>>(w8a8_kernel<NT, true>, a, p, tm_w, tm_a, early, stream, msg)
                 : launch_w8a8_type<W8Cfg<NT>>(w8a8_kernel<NT, false>, a, p, tm_w, tm_a, early, stream, msg);
}

// `early`: the kernel before this one on the stream is the quantizer, which starts behind all that came before.
static cudaError_t launch_w8a8(const W8A8Args &a, bool early, cudaStream_t stream, const char **msg) {
  auto enc = get_encode_fn();
  if (!enc) {
    *msg = "cuTensorMapEncodeTiled is not available from the driver";
    return cudaErrorNotSupported;
  }
  W8Plan p;
  if (!w8a8_plan(a.M, a.N, a.K, &p)) {
    *msg = "the product's tiles x chunks of K pass 2^31";
    return cudaErrorNotSupported;
  }
  CUtensorMap tm_w, tm_a;
  if (!encode_2d_u8_uncached(enc, &tm_w, a.W, a.K, a.N, kW8Chunk, kW8Rows, true) ||
      !encode_2d_u8_uncached(enc, &tm_a, a.A_q, a.K, a.M, kW8Chunk, p.pair ? p.NT / 2 : p.NT, true)) {
    *msg = "tensor map encoding of W or A_q failed";
    return cudaErrorInvalidValue;
  }
  if (p.pair)
    return p.NT == 256
               ? launch_w8a8_type<W8PairCfg<256>>(w8a8_pair_kernel<256>, a, p, tm_w, tm_a, early, stream, msg)
               : launch_w8a8_type<W8PairCfg<128>>(w8a8_pair_kernel<128>, a, p, tm_w, tm_a, early, stream, msg);
  if (p.NT == 16) return launch_w8a8_tokens<16>(a, p, tm_w, tm_a, early, stream, msg);
  if (p.NT == 32) return launch_w8a8_tokens<32>(a, p, tm_w, tm_a, early, stream, msg);
  return launch_w8a8_tokens<64>(a, p, tm_w, tm_a, early, stream, msg);
}

cudaError_t launch_w8a8_pack(const float *W, int64_t N, int64_t K, int8_t *codes, float *s_w, cudaStream_t stream) {
  return launch_row_quantize(W, K, N, K, codes, s_w, stream);
}
cudaError_t launch_w8a8_quantize(const __half *X, int64_t stride, int64_t M, int64_t K, int8_t *A_q, float *s_a,
                                 cudaStream_t stream) {
  return launch_row_quantize(X, stride, M, K, A_q, s_a, stream);
}
cudaError_t launch_w8a8_gemm(const W8A8Args &a, cudaStream_t stream, const char **msg) {
  return launch_w8a8(a, false, stream, msg);
}
cudaError_t launch_w8a8_linear(const __half *X, int64_t stride, W8A8Args a, void *ws, cudaStream_t stream,
                               const char **msg) {
  int8_t *codes = static_cast<int8_t *>(ws);
  float *s_a = reinterpret_cast<float *>(codes + (static_cast<size_t>(a.M) * a.K + 255) / 256 * 256);
  a.A_q = codes;
  a.s_a = s_a;
  cudaError_t e = launch_w8a8_quantize(X, stride, a.M, a.K, codes, s_a, stream);
  if (e != cudaSuccess) {
    *msg = "launch of the activations' quantizer failed";
    return e;
  }
  return launch_w8a8(a, true, stream, msg);
}

}  // namespace mixllm
