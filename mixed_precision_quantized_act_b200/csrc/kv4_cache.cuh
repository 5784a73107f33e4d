// kv4_cache.cuh -- the write side of the paged 4-bit KV cache: pages and slots
// of a step's tokens from the requests' lengths, the rotated and quantized
// keys and values into their slots, and the cached rows back as fp16.
//
// Layout: codes uint8 [pages][2][H][page][D/2] (key, value), code 2i in the
// low and 2i + 1 in the high nibble of byte i; meta uint32 [pages][2][H][page],
// the fp16 scale in the low half and the zero point above it.  One head's
// rows of one page are one contiguous block, for bulk copies.
#pragma once

#include <cuda_fp16.h>
#include <atomic>
#include <cstdint>

#include "launch.h"
#include "norm.cuh"
#include "ptx_sm100.cuh"
#include "quant.cuh"

namespace mixllm {

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Index of the last entry of start[0..n) that is <= i (start[0] = 0 <= i,
// ascending): the request that item i belongs to; empty requests are passed
// over.
__device__ __forceinline__ int owner_of(const int *start, int n, int i) {
  int lo = 0, hi = n;  // start[lo] <= i < start[hi], start[n] taken as infinite
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// Pages and slots.  One cluster: every block of it scans all requests'
// lengths (two prefix sums: new tokens and new pages), then the blocks share
// the tokens and the new pages, each found by a binary search in the sums.
// The cluster barrier between the scan and the first write lets seq_lens be
// ctx_lens and left be count.  Latency-bound: one load round trip, the scan,
// the search and a second trip for the page's number.
// ---------------------------------------------------------------------------
constexpr int kAssignThreads = 1024;
constexpr int kAssignCluster = 8;

__global__ void __launch_bounds__(kAssignThreads) kv4_assign_kernel(const AssignArgs a) {
  extern __shared__ int assign_smem[];
  __shared__ long long warp_sum[2][32];
  __shared__ int bad_bits;
  const int B = a.B, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int *cu = assign_smem, *off = cu + B, *ctx = off + B;
  const int per = (B + kAssignThreads - 1) / kAssignThreads;  // requests of one thread, consecutive
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  const int count = *a.count;
  auto pages = [&](long long n) { return (n + (1ll << a.page_log2) - 1) >> a.page_log2; };
  if (tid == 0) bad_bits = 0;

  long long tokens = 0, added = 0;
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    const long long c = a.ctx_lens[b], n = a.new_lens[b];
    ctx[b] = static_cast<int>(c);
    if (c < 0 || n < 0) {
      bad |= 8;
      continue;
    }
    if (pages(c + n) > a.W) bad |= 2;
    tokens += n;
    added += pages(c + n) - pages(c);
  }
  long long t_base = tokens, p_base = added;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xFFFFFFFFu, t_base, o), p = __shfl_up_sync(0xFFFFFFFFu, p_base, o);
    if (lane >= o) t_base += t, p_base += p;
  }
  if (lane == 31) warp_sum[0][warp] = t_base, warp_sum[1][warp] = p_base;
  t_base -= tokens, p_base -= added;
  __syncthreads();
  long long t_all = 0, p_all = 0;
#pragma unroll
  for (int w = 0; w < 32; ++w) {
    if (w < warp) t_base += warp_sum[0][w], p_base += warp_sum[1][w];
    t_all += warp_sum[0][w], p_all += warp_sum[1][w];
  }
  if (t_all > a.T) bad |= 4;
  if (p_all > count || count > a.n_free) bad |= 1;
  if (bad) atomicOr(&bad_bits, bad);
  for (int b = b0; b < b1; ++b) {  // where a total is out of range these wrap, and are not used
    const long long c = a.ctx_lens[b], n = a.new_lens[b];
    cu[b] = static_cast<int>(t_base);
    off[b] = static_cast<int>(p_base);
    if (c >= 0 && n >= 0) t_base += n, p_base += pages(c + n) - pages(c);
  }
  cluster_sync();  // every input is read; also publishes cu, off, ctx and bad_bits within the block

  bad = bad_bits;
  const int total = bad ? 0 : static_cast<int>(t_all), fresh = bad ? 0 : static_cast<int>(p_all);
  const int first = blockIdx.x * kAssignThreads + tid, stride = gridDim.x * kAssignThreads;
  if (first == 0) {
    *a.left = count - fresh;
    *a.status = bad;
    a.cu_new[B] = total;
  }
  for (int b = first; b < B; b += stride) {
    a.cu_new[b] = bad ? 0 : cu[b];
    const int next = b + 1 < B ? cu[b + 1] : total;
    a.seq_lens[b] = bad ? ctx[b] : ctx[b] + (next - cu[b]);
  }
  for (int e = first; e < fresh; e += stride) {
    const int b = owner_of(off, B, e);
    a.table[static_cast<int64_t>(b) * a.table_stride + pages(ctx[b]) + (e - off[b])] = a.free_pages[count - 1 - e];
  }
  for (int64_t t = first; t < a.T; t += stride) {
    int64_t slot = -1;
    int pos = -1;
    if (t < total) {
      const int b = owner_of(cu, B, static_cast<int>(t));
      pos = ctx[b] + (static_cast<int>(t) - cu[b]);
      const int j = pos >> a.page_log2, have = static_cast<int>(pages(ctx[b]));
      // a page of this call is read where it came from: its table entry may still be on its way
      const int page = j < have ? a.table[static_cast<int64_t>(b) * a.table_stride + j]
                                : a.free_pages[count - 1 - (off[b] + j - have)];
      if (page < 0) record_status(kStatusBounds);
      else slot = (static_cast<int64_t>(page) << a.page_log2) + (pos & ((1 << a.page_log2) - 1));
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }
}

// ---------------------------------------------------------------------------
// Append: D / 8 lanes per row (one head of one token), eight channels a lane.
// The first `rotary` channels of queries and keys are rotated in pairs
// (i, i + rotary / 2) in fp32 with every product and sum rounded on its own,
// and rounded to fp16 -- the value the codes are made of.  Keys and values
// then take the weights' 4-bit asymmetric quantizer over the head's D
// channels (w4_params, w4_code).  A row that holds a NaN or an infinity is
// stored with a NaN scale: it reads back as NaN instead of as something
// finite.  HBM-bound: reads 2 bytes and writes 0.5 (keys, values) or 2
// (queries) a channel.
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;

// Where row `h` of kind `kv` (0 key, 1 value) at `slot` lives: code bytes and meta words.
__device__ __forceinline__ int64_t kv4_row(const Kv4Cache &c, int64_t slot, int kv, int h) {
  const int64_t page = slot >> c.page_log2;
  return (((page * 2 + kv) * c.H + h) << c.page_log2) + (slot & ((1 << c.page_log2) - 1));
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads) kv4_append_kernel(const AppendArgs a) {
  constexpr int kLanes = D / 8;
  const int sub = threadIdx.x % kLanes;
  const unsigned mask = (kLanes == 32 ? 0xFFFFFFFFu : ((1u << kLanes) - 1u)) << (threadIdx.x & 31 & ~(kLanes - 1));
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kAppendThreads / kLanes);
  const int rows = a.Hq + 2 * a.cache.H;
  const int half = a.rotary / 2;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / kLanes) + threadIdx.x / kLanes;
       i < a.T * rows; i += stride) {
    const int64_t t = i / rows;
    const int h = static_cast<int>(i - t * rows);
    const int64_t slot = a.slots[t];
    if (slot < 0) continue;  // padding behind the last token
    int64_t pos = a.rope ? a.positions[t] : 0;
    if (slot >= a.cache.pages << a.cache.page_log2 || pos < 0 || (a.rope && pos >= a.max_pos)) {
      if (sub == 0) record_status(kStatusBounds);
      continue;
    }
    const int kind = h < a.Hq ? 0 : (h < a.Hq + a.cache.H ? 1 : 2);  // query, key, value
    const int head = kind == 0 ? h : (kind == 1 ? h - a.Hq : h - a.Hq - a.cache.H);
    const __half *src = kind == 0 ? a.q + t * a.q_stride : (kind == 1 ? a.k + t * a.k_stride : a.v + t * a.v_stride);
    uint4 raw = *reinterpret_cast<const uint4 *>(src + head * D + sub * 8);
    if (kind < 2 && half > 0) {
      const int c0 = sub * 8;  // half is a multiple of 8: a lane lies in one half, or behind both
      const bool second = c0 >= half;
      const int other = second ? sub - half / 8 : sub + half / 8;
      uint4 far;
      far.x = __shfl_sync(mask, raw.x, other, kLanes);
      far.y = __shfl_sync(mask, raw.y, other, kLanes);
      far.z = __shfl_sync(mask, raw.z, other, kLanes);
      far.w = __shfl_sync(mask, raw.w, other, kLanes);
      if (c0 < a.rotary) {
        const float *angle = a.rope + pos * a.rotary + (second ? c0 - half : c0);
        float cs[8], sn[8], own[8], oth[8];
        load8(angle, cs);
        load8(angle + half, sn);
        const __half2 *h0 = reinterpret_cast<const __half2 *>(&raw), *h1 = reinterpret_cast<const __half2 *>(&far);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 u = __half22float2(h0[j]), w = __half22float2(h1[j]);
          own[2 * j] = u.x, own[2 * j + 1] = u.y, oth[2 * j] = w.x, oth[2 * j + 1] = w.y;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float near_part = __fmul_rn(own[j], cs[j]), far_part = __fmul_rn(oth[j], sn[j]);
          own[j] = second ? __fadd_rn(near_part, far_part) : __fsub_rn(near_part, far_part);
        }
        raw = pack8(own);
      }
    }
    if (kind == 0) {
      *reinterpret_cast<uint4 *>(a.q_out + t * a.q_out_stride + head * D + sub * 8) = raw;
      continue;
    }
    const __half2 *h2 = reinterpret_cast<const __half2 *>(&raw);
    float x[8], lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(h2[j]);
      x[2 * j] = f.x, x[2 * j + 1] = f.y;
    }
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      lo = fminf(lo, x[j]), hi = fmaxf(hi, x[j]);
      odd |= !(fabsf(x[j]) <= 65504.0f);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      lo = fminf(lo, __shfl_xor_sync(mask, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(mask, hi, o));
    }
    uint32_t code = 0, meta = 0x7FFFu;
    if (!__any_sync(mask, odd)) {
      const W4Params p = w4_params(lo, hi);
#pragma unroll
      for (int j = 0; j < 8; ++j) code |= static_cast<uint32_t>(w4_code(x[j], p)) << (4 * j);
      meta = static_cast<uint32_t>(__half_as_ushort(p.sh)) | static_cast<uint32_t>(p.z) << 16;
    }
    const int64_t row = kv4_row(a.cache, slot, kind - 1, head);
    *reinterpret_cast<uint32_t *>(a.cache.codes + row * (D / 2) + sub * 4) = code;
    if (sub == 0) a.cache.meta[row] = meta;
  }
}

// The cached rows of the given slots as fp16: s * (code - z), rounded once and
// kept within the finite fp16 values (15 steps of a scale rounded up can pass
// the largest one).
template <int D>
__global__ void __launch_bounds__(kAppendThreads) kv4_read_kernel(const Kv4Cache c, const int64_t *__restrict__ slots,
                                                                  int64_t T, __half *__restrict__ k,
                                                                  __half *__restrict__ v) {
  constexpr int kLanes = D / 8;
  const int sub = threadIdx.x % kLanes;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (kAppendThreads / kLanes);
  const int rows = 2 * c.H;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / kLanes) + threadIdx.x / kLanes; i < T * rows;
       i += stride) {
    const int64_t t = i / rows;
    const int h = static_cast<int>(i - t * rows);
    const int64_t slot = slots[t];
    if (slot < 0) continue;
    if (slot >= c.pages << c.page_log2) {
      if (sub == 0) record_status(kStatusBounds);
      continue;
    }
    const int kv = h >= c.H, head = kv ? h - c.H : h;
    const int64_t row = kv4_row(c, slot, kv, head);
    const uint32_t code = *reinterpret_cast<const uint32_t *>(c.codes + row * (D / 2) + sub * 4), meta = c.meta[row];
    const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(meta & 0xFFFFu)));
    const int z = static_cast<int>(meta >> 16 & 15u);
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = static_cast<float>(static_cast<int>(code >> (4 * j) & 15u) - z) * s;
      f[j] = x > 65504.0f ? 65504.0f : (x < -65504.0f ? -65504.0f : x);  // a NaN stays one
    }
    *reinterpret_cast<uint4 *>((kv ? v : k) + (t * c.H + head) * D + sub * 8) = pack8(f);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

cudaError_t launch_kv4_assign(const AssignArgs &a, cudaStream_t stream, const char **msg) {
  const size_t smem = static_cast<size_t>(a.B) * 3 * sizeof(int);
  static std::atomic<unsigned long long> configured{0};  // one bit per device ordinal
  int dev = 0;
  cudaGetDevice(&dev);
  if (smem > 40 * 1024 && (dev >= 64 || !(configured.load() & (1ull << dev)))) {
    cudaError_t e = cudaFuncSetAttribute(kv4_assign_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kKv4MaxRequests * 3 * static_cast<int>(sizeof(int)));
    if (e != cudaSuccess) {
      *msg = "cudaFuncSetAttribute(MaxDynamicSharedMemorySize) failed";
      return e;
    }
    if (dev < 64) configured.fetch_or(1ull << dev);
  }
  cudaLaunchConfig_t cfg = {};
  // few tokens: one block, which has no other to wait for at the barrier
  cfg.gridDim = dim3(a.T > 2 * kAssignThreads ? kAssignCluster : 1);
  cfg.blockDim = dim3(kAssignThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cfg.gridDim.x;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_assign_kernel, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) *msg = "launch of the page assignment failed";
  return e;
}

static unsigned append_grid(int64_t rows, int D) {
  const int64_t blocks = (rows + kAppendThreads / (D / 8) - 1) / (kAppendThreads / (D / 8));
  return static_cast<unsigned>(blocks < 148 * 64 ? blocks : 148 * 64);
}

cudaError_t launch_kv4_append(const AppendArgs &a, cudaStream_t stream) {
  const unsigned grid = append_grid(a.T * (a.Hq + 2 * a.cache.H), a.cache.D);
  if (a.cache.D == 128) kv4_append_kernel<128><<<grid, kAppendThreads, 0, stream>>>(a);
  else kv4_append_kernel<64><<<grid, kAppendThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4Cache &c, const int64_t *slots, int64_t T, void *k, void *v,
                            cudaStream_t stream) {
  const unsigned grid = append_grid(T * 2 * c.H, c.D);
  __half *kh = static_cast<__half *>(k), *vh = static_cast<__half *>(v);
  if (c.D == 128) kv4_read_kernel<128><<<grid, kAppendThreads, 0, stream>>>(c, slots, T, kh, vh);
  else kv4_read_kernel<64><<<grid, kAppendThreads, 0, stream>>>(c, slots, T, kh, vh);
  return cudaGetLastError();
}

}  // namespace mixllm
