// w8a8.cuh -- the linear layer in 8-bit integers with one scale per token and
// one per output channel:
//   Y[m, n] = fp16( float(sum_k A[m, k] W[n, k]) * s_a[m] * s_w[n] + bias[n] ),
// its quantizers (activations and weights alike: one scale per row) and the
// product on the int8 tensor cores.
#pragma once

#include <cuda_fp16.h>
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
// and codes 0, one with a NaN or an infinity s = NaN and codes 0.  One block per
// row, which stays in registers up to V runs of eight a thread and is read
// again from there on.
// ---------------------------------------------------------------------------
template <typename T>
struct RowRun;  // eight values as loaded
template <>
struct RowRun<__half> {
  uint4 raw;
  __device__ __forceinline__ void load(const __half *p) { raw = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void widen(float (&f)[8]) const { widen8(raw, f); }
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
};

constexpr int kRowQuantRuns = 4;  // of eight values, a thread's registers

template <typename T>
__global__ void __launch_bounds__(1024) row_quantize_kernel(const T *__restrict__ X, int64_t stride, int K,
                                                            int8_t *__restrict__ codes, float *__restrict__ scales) {
  __shared__ float warp_max[32];
  pdl_launch_dependents();
  const int64_t m = blockIdx.x;
  const T *row = X + m * stride;
  const int step = blockDim.x * 8, k0 = threadIdx.x * 8;
  RowRun<T> run[kRowQuantRuns];
  float amax = 0.0f;
  bool odd = false;
  const auto look = [&](const RowRun<T> &r) {
    float f[8];
    r.widen(f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      amax = fmaxf(amax, fabsf(f[i]));
      odd |= !(fabsf(f[i]) <= 3.4028234663852886e38f);
    }
  };
#pragma unroll
  for (int v = 0; v < kRowQuantRuns; ++v)
    if (k0 + v * step < K) run[v].load(row + k0 + v * step);
#pragma unroll
  for (int v = 0; v < kRowQuantRuns; ++v)
    if (k0 + v * step < K) look(run[v]);
  for (int k = k0 + kRowQuantRuns * step; k < K; k += step) {
    RowRun<T> r;
    r.load(row + k);
    look(r);
  }
  if (odd) amax = INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = (threadIdx.x & 31) < (blockDim.x >> 5) ? warp_max[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  const float s = amax == INFINITY ? __int_as_float(0x7FFFFFFF) : __fdiv_rn(amax, 127.0f);
  if (threadIdx.x == 0) scales[m] = s;
  const bool none = !(s > 0.0f);
  const auto store = [&](const RowRun<T> &r, int k) {
    uint32_t packed[2] = {0u, 0u};
    if (!none) {
      float f[8];
      r.widen(f);
      if constexpr (sizeof(T) == 2) {
        const QuantStep q = QuantStep::of(s);
#pragma unroll
        for (int i = 0; i < 8; ++i) packed[i >> 2] |= (q.code(f[i]) & 0xFFu) << ((i & 3) * 8);
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
  for (int v = 0; v < kRowQuantRuns; ++v)
    if (k0 + v * step < K) store(run[v], k0 + v * step);
  for (int k = k0 + kRowQuantRuns * step; k < K; k += step) {
    RowRun<T> r;
    r.load(row + k);
    store(r, k);
  }
}

template <typename T>
static cudaError_t launch_row_quantize(const T *X, int64_t stride, int64_t M, int64_t K, int8_t *codes, float *scales,
                                       cudaStream_t stream) {
  const int64_t runs = K / 8;
  // a thread per run up to 512, then up to four runs a thread
  int64_t threads = runs <= 512 ? runs : (runs + kRowQuantRuns - 1) / kRowQuantRuns;
  threads = threads < 256 && runs > 512 ? 256 : threads;
  threads = threads > 1024 ? 1024 : (threads + 31) / 32 * 32;
  row_quantize_kernel<T><<<static_cast<unsigned>(M), static_cast<unsigned>(threads), 0, stream>>>(
      X, stride, static_cast<int>(K), codes, scales);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// The product.  Channels are the tensor core's 128-row side and tokens its
// column side (NT of them, 16 to 256), so that a few tokens cost no more than
// their columns and the weights stream through shared memory at any number of
// tokens.  Work is cut into chunks of 128 channels x NT tokens x 128 values of K;
// block c takes the units (runs of `per` chunks) [c U / P, (c + 1) U / P) of
// their sequence, K innermost, tokens next.  With `per` the whole of K a block
// has whole tiles; with 1 the ends of its share may cut a tile, whose int32 parts
// go to the workspace, and the last block to arrive adds them: integers, so the
// result is the same whoever is last.
//
// Warp 0 loads both operands by TMA (128-byte swizzle), warp 1 issues
// tcgen05.mma kind::i8, warps 4-7 scale the accumulators and write Y while the
// next tile's products run (two accumulators in tensor memory).
// ---------------------------------------------------------------------------
constexpr int kW8Threads = 256;
constexpr int kW8Rows = 128;   // channels of a tile
constexpr int kW8Chunk = 128;  // values of K of a chunk
constexpr int kW8MaxGrid = 148;

template <int NT>
struct W8Cfg {
  static constexpr int kStageW = kW8Rows * kW8Chunk, kStageA = NT * kW8Chunk, kStage = kStageW + kStageA;
  static constexpr int kStages = 200 * 1024 / kStage < 10 ? 200 * 1024 / kStage : 10;
  static constexpr int kSmem = kStages * kStage + 1024;
  static constexpr int kTmem = 2 * NT < 32 ? 32 : 2 * NT;
  static constexpr int kStep = NT < 32 ? 16 : 32;  // columns of one load from tensor memory
  static constexpr int kPart = kW8Rows * NT;       // int32 values of a part
  static_assert(kSmem + 4096 <= 227 * 1024, "shared memory of a block");
};

struct W8Job {
  const float *s_a, *s_w;
  const __half *bias;  // or null
  __half *Y;
  int64_t M, N;
  int KC;       // chunks along K
  int TT;       // token tiles
  int64_t U;    // units
  int per;      // chunks of a unit: 1 or KC
  bool early;   // the kernel before this one does not write W: its loads need not wait
  bool pairs;   // Y may be written two channels at a time
  uint32_t *counters;
  int32_t *parts;
};

template <int NT>
__global__ void __launch_bounds__(kW8Threads, 1) w8a8_kernel(const __grid_constant__ CUtensorMap tm_w,
                                                             const __grid_constant__ CUtensorMap tm_a, const W8Job a) {
  using C = W8Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ uint64_t full[C::kStages], empty[C::kStages], acc_full[2], acc_empty[2], drained;
  __shared__ __align__(16) float token_scale[NT];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ int join_first, join_last;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 128);
    }
    mbar_init(&drained, 1);
    fence_mbar_init();
    abort_flag = 0;
  }
  if (warp == 2) {
    tmem_alloc(&tmem_slot, C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();  // only now: a dependent may take tensor memory as it starts
  const uint32_t tmem = tmem_slot;

  const int P = gridDim.x, c = blockIdx.x;
  const int64_t share = a.U / P;
  const int rest = static_cast<int>(a.U - share * P);
  const auto block_start = [&](int b) { return (share * b + static_cast<int64_t>(rest) * b / P) * a.per; };
  const int64_t start = block_start(c), end = block_start(c + 1);

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      prefetch_tmap(&tm_w);
      prefetch_tmap(&tm_a);
      const int64_t tile0 = start / a.KC;
      int row_tile = static_cast<int>(tile0 / a.TT), token_tile = static_cast<int>(tile0 - static_cast<int64_t>(row_tile) * a.TT);
      int kc = static_cast<int>(start - tile0 * a.KC);
      const auto weights = [&](int s, int rt, int k) {
        mbar_arrive_expect_tx(&full[s], C::kStage);
        tma_load_2d(smem + s * C::kStage, &tm_w, &full[s], k * kW8Chunk, rt * kW8Rows);
      };
      int ahead = 0;  // chunks whose weights are under way
      if (a.early) {
        int rt = row_tile, tt = token_tile, k = kc;
        for (; ahead < C::kStages && start + ahead < end; ++ahead) {
          weights(ahead, rt, k);
          if (++k == a.KC) {
            k = 0;
            if (++tt == a.TT) tt = 0, ++rt;
          }
        }
      }
      pdl_wait();
      int s = 0;
      uint32_t phase = 1;
      int64_t issued = 0;
      for (int64_t x = start; x < end; ++x, ++issued) {
        if (issued >= C::kStages && !mbar_wait(&empty[s], phase, &abort_flag)) break;
        if (issued >= ahead) weights(s, row_tile, kc);
        tma_load_2d(smem + s * C::kStage + C::kStageW, &tm_a, &full[s], kc * kW8Chunk, token_tile * NT);
        if (++s == C::kStages) s = 0, phase ^= 1;
        if (++kc == a.KC) {
          kc = 0;
          if (++token_tile == a.TT) token_tile = 0, ++row_tile;
        }
      }
      if (abort_flag) {  // the last copies into each stage land before the block's memory goes to another
        for (int i = 0; i < C::kStages && i < issued; ++i) {
          const int64_t last = (issued - 1 - i) / C::kStages;  // uses of stage i before this one
          mbar_wait_drain(&full[i], static_cast<uint32_t>(last & 1), 1ll << 24);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    constexpr uint32_t kIdesc = idesc_i8(kW8Rows, NT);
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    const uint64_t w_desc = sw128_kmajor_desc(smem_u32(smem)), a_desc = sw128_kmajor_desc(smem_u32(smem) + C::kStageW);
    int s = 0;
    uint32_t phase = 0, piece = 0;
    bool ok = true;
    for (int64_t x = start; x < end && ok; ++piece) {
      const int k0 = static_cast<int>(x % a.KC);
      const int n = static_cast<int>(min(static_cast<int64_t>(a.KC - k0), end - x));
      x += n;
      const int acc = piece & 1;
      ok = warp_wait(&acc_empty[acc], (piece >> 1 & 1) ^ 1, &abort_flag);
      for (int k = 0; k < n && ok; ++k) {
        ok = warp_wait(&full[s], phase, &abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t off = static_cast<uint64_t>(s * C::kStage >> 4);
#pragma unroll
          for (int j = 0; j < kW8Chunk / 32; ++j)
            mma_i8(tm + acc * NT, w_desc + off + 2 * j, a_desc + off + 2 * j, kIdesc, k > 0 || j > 0);
          mma_commit(&empty[s]);
          if (k + 1 == n) mma_commit(&acc_full[acc]);
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
  } else if (warp >= 4) {
    // ------------------------------------------------------------ scales and Y: thread = channel of the tile
    pdl_wait();  // s_a, and the parts' counters
    const int r = tid - 128;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t piece = 0;
    for (int64_t x = start; x < end; ++piece) {
      const int64_t tile = x / a.KC;
      const int k0 = static_cast<int>(x - tile * a.KC);
      const int n = static_cast<int>(min(static_cast<int64_t>(a.KC - k0), end - x));
      x += n;
      const int row_tile = static_cast<int>(tile / a.TT), token_tile = static_cast<int>(tile - static_cast<int64_t>(row_tile) * a.TT);
      const int64_t ch = static_cast<int64_t>(row_tile) * kW8Rows + r, m0 = static_cast<int64_t>(token_tile) * NT;
      const int tokens = static_cast<int>(min(static_cast<int64_t>(NT), a.M - m0));
      named_bar_sync(1, 128);  // everyone is done with the last piece's scales
      for (int j = r; j < tokens; j += 128) token_scale[j] = a.s_a[m0 + j];
      const float sw = ch < a.N ? a.s_w[ch] : 0.0f;
      const float bias = a.bias && ch < a.N ? __half2float(a.bias[ch]) : 0.0f;
      const int acc = piece & 1;
      // the four warps go on together or not at all: they meet at barriers below
      if (!named_bar_and(1, 128, mbar_wait(&acc_full[acc], piece >> 1 & 1, &abort_flag))) break;
      tc_fence_after();
      const uint32_t at = tmem + lanes + acc * NT;
      const bool cut = n < a.KC;
      bool write = true;
      int first = c, last = c;
      if (cut) {
        // this block's part, then whether it is the last one to arrive
        int32_t *mine = a.parts + (static_cast<int64_t>(c) * 2 + (k0 == 0 ? 1 : 0)) * C::kPart + r;
#pragma unroll 1
        for (int j0 = 0; j0 < tokens; j0 += C::kStep) {
          uint32_t v[C::kStep];
          tmem_ld_cols(at + j0, v);
          tmem_ld_wait();
          reg_fence(v);
#pragma unroll
          for (int j = 0; j < C::kStep; ++j) __stcg(mine + (j0 + j) * kW8Rows, static_cast<int32_t>(v[j]));
        }
        named_bar_sync(1, 128);
        if (r == 0) {
          // chunk x is in block ((x + 1) P - 1) / U of those with a unit of one chunk each
          const int64_t t0 = tile * a.KC;
          join_first = static_cast<int>(((t0 + 1) * P - 1) / a.U);
          join_last = static_cast<int>(((t0 + a.KC) * P - 1) / a.U);
          // a block's end cuts one tile at most: the first block of a tile names its counter
          const uint32_t arrived = atom_add_acq_rel_gpu_u32(a.counters + join_first, 1u);
          if (arrived == static_cast<uint32_t>(join_last - join_first)) a.counters[join_first] = 0;
          else join_last = -1;
        }
        named_bar_sync(1, 128);
        first = join_first, last = join_last;
        write = last >= 0;
      }
      if (write) {
#pragma unroll 1
        for (int j0 = 0; j0 < tokens; j0 += C::kStep) {
          uint32_t v[C::kStep];
          tmem_ld_cols(at + j0, v);
          tmem_ld_wait();
          reg_fence(v);
          for (int b = first; b <= last; ++b) {
            if (b == c) continue;
            const int32_t *part = a.parts + (static_cast<int64_t>(b) * 2 + (b == first ? 1 : 0)) * C::kPart + r;
#pragma unroll
            for (int j = 0; j < C::kStep; ++j) v[j] += static_cast<uint32_t>(__ldcg(part + (j0 + j) * kW8Rows));
          }
          float f[C::kStep];
#pragma unroll
          for (int j = 0; j < C::kStep; ++j)
            f[j] = fmaf(static_cast<float>(static_cast<int32_t>(v[j])) * token_scale[j0 + j], sw, bias);
          __half *to = a.Y + (m0 + j0) * a.N + ch;
          if (a.pairs) {
            // neighbouring lanes swap, so that each writes two channels of every other token
            const bool odd = lane & 1;
#pragma unroll
            for (int j = 0; j < C::kStep; j += 2) {
              const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? f[j] : f[j + 1], 1);
              const __half2 h = odd ? __floats2half2_rn(got, f[j + 1]) : __floats2half2_rn(f[j], got);
              if (j0 + j + odd < tokens && ch < a.N)
                *reinterpret_cast<__half2 *>(to + (j + odd) * a.N - odd) = h;
            }
          } else {
#pragma unroll
            for (int j = 0; j < C::kStep; ++j)
              if (j0 + j < tokens && ch < a.N) to[j * a.N] = __float2half_rn(f[j]);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&acc_empty[acc]);
    }
  }
  __syncthreads();
  if (warp == 2) tmem_dealloc(tmem, C::kTmem);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

struct W8Plan {
  int NT, KC, TT, per, grid;
  int64_t U;
};

static W8Plan w8a8_plan(int64_t M, int64_t N, int64_t K) {
  W8Plan p;
  const int64_t sms = kW8MaxGrid;
  const int64_t rows = (N + kW8Rows - 1) / kW8Rows;
  p.KC = static_cast<int>((K + kW8Chunk - 1) / kW8Chunk);
  p.NT = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : rows * ((M + 255) / 256) >= sms ? 256 : 128;
  p.TT = static_cast<int>((M + p.NT - 1) / p.NT);
  const int64_t tiles = rows * p.TT;
  // Whole tiles where they fill the GPU in nearly whole rounds, else even shares of chunks.
  const int64_t rounds = (tiles + sms - 1) / sms;
  p.per = tiles * 10 >= rounds * sms * 9 ? p.KC : 1;
  p.U = tiles * p.KC / p.per;
  p.grid = static_cast<int>(p.U < sms ? p.U : sms);
  return p;
}

constexpr size_t kW8CounterBytes = 4096;
static_assert(kW8MaxGrid * sizeof(uint32_t) <= kW8CounterBytes, "one counter per block");

// Room for two parts of every block at the widest tile that up to M tokens take: enough for fewer tokens, too.
size_t w8a8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M == 0 || N == 0) return 0;
  const int64_t widest = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : M <= 128 ? 128 : 256;
  return kW8CounterBytes + static_cast<size_t>(kW8MaxGrid) * 2 * kW8Rows * widest * sizeof(int32_t);
}

// The layer from fp16 adds the codes and scales of its activations.
size_t w8a8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M == 0 || N == 0) return 0;
  const size_t codes = (static_cast<size_t>(M) * K + 255) / 256 * 256;
  return w8a8_gemm_workspace_bytes(M, N, K) + codes + (static_cast<size_t>(M) * 4 + 255) / 256 * 256;
}

template <int NT>
static cudaError_t launch_w8a8_type(const W8A8Args &a, const W8Plan &p, const CUtensorMap &tm_w, const CUtensorMap &tm_a,
                                    bool early, cudaStream_t stream, const char **msg) {
  using C = W8Cfg<NT>;
  auto kern = w8a8_kernel<NT>;
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
  const bool pairs = a.N % 2 == 0 && (reinterpret_cast<uintptr_t>(a.Y) & 3) == 0;
  const W8Job job{a.s_a, a.s_w, a.bias, a.Y, a.M, a.N, p.KC, p.TT, p.U, p.per, early, pairs,
                  static_cast<uint32_t *>(a.ws), reinterpret_cast<int32_t *>(static_cast<uint8_t *>(a.ws) + kW8CounterBytes)};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // starts while the kernel before it ends
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.grid));
  cfg.blockDim = dim3(kW8Threads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tm_w, tm_a, job);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) *msg = "launch of the 8-bit product failed";
  return e;
}

// `early`: the kernel before this one on the stream is the quantizer, behind everything that came before.
static cudaError_t launch_w8a8(const W8A8Args &a, bool early, cudaStream_t stream, const char **msg) {
  auto enc = get_encode_fn();
  if (!enc) {
    *msg = "cuTensorMapEncodeTiled is not available from the driver";
    return cudaErrorNotSupported;
  }
  const W8Plan p = w8a8_plan(a.M, a.N, a.K);
  CUtensorMap tm_w, tm_a;
  if (!encode_2d_u8_uncached(enc, &tm_w, a.W, a.K, a.N, kW8Chunk, kW8Rows, true) ||
      !encode_2d_u8_uncached(enc, &tm_a, a.A_q, a.K, a.M, kW8Chunk, p.NT, true)) {
    *msg = "tensor map encoding of W or A_q failed";
    return cudaErrorInvalidValue;
  }
  switch (p.NT) {
    case 16: return launch_w8a8_type<16>(a, p, tm_w, tm_a, early, stream, msg);
    case 32: return launch_w8a8_type<32>(a, p, tm_w, tm_a, early, stream, msg);
    case 64: return launch_w8a8_type<64>(a, p, tm_w, tm_a, early, stream, msg);
    case 128: return launch_w8a8_type<128>(a, p, tm_w, tm_a, early, stream, msg);
    default: return launch_w8a8_type<256>(a, p, tm_w, tm_a, early, stream, msg);
  }
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
cudaError_t launch_w8a8_linear(const __half *X, int64_t stride, W8A8Args a, cudaStream_t stream, const char **msg) {
  uint8_t *codes = static_cast<uint8_t *>(a.ws) + w8a8_gemm_workspace_bytes(a.M, a.N, a.K);
  float *s_a = reinterpret_cast<float *>(codes + (static_cast<size_t>(a.M) * a.K + 255) / 256 * 256);
  a.A_q = reinterpret_cast<const int8_t *>(codes);
  a.s_a = s_a;
  cudaError_t e = launch_w8a8_quantize(X, stride, a.M, a.K, reinterpret_cast<int8_t *>(codes), s_a, stream);
  if (e != cudaSuccess) {
    *msg = "launch of the activations' quantizer failed";
    return e;
  }
  return launch_w8a8(a, true, stream, msg);
}

}  // namespace mixllm
