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
// the search and a second trip for the page's number; 5.7 us for 64 requests of
// one token on B200, 13.7 us for 256 prompts in 130304 slots.
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
  // A warp takes a run of tokens, 32 at a time: one search for the first, then the owner moves along.  Four
  // times 32 tokens' page loads are under way together.
  constexpr int kAtOnce = 4;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kAssignThreads / 32);
  const int64_t run = ((a.T + warps - 1) / warps + 31) / 32 * 32;
  const int64_t begin = (static_cast<int64_t>(blockIdx.x) * (kAssignThreads / 32) + warp) * run;
  const int64_t stop = begin + run < a.T ? begin + run : a.T;
  int b = begin + lane < total ? owner_of(cu, B, static_cast<int>(begin) + lane) : 0;
  for (int64_t t0 = begin + lane; t0 < stop; t0 += 32 * kAtOnce) {
    int page[kAtOnce], pos[kAtOnce];
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) {
      const int64_t t = t0 + 32 * x;
      page[x] = pos[x] = -1;
      if (t < total && t < stop) {
        while (b + 1 < B && cu[b + 1] <= t) ++b;
        pos[x] = ctx[b] + (static_cast<int>(t) - cu[b]);
        const int j = pos[x] >> a.page_log2, have = static_cast<int>(pages(ctx[b]));
        // a page of this call is read where it came from: its table entry may still be on its way
        page[x] = j < have ? a.table[static_cast<int64_t>(b) * a.table_stride + j]
                           : a.free_pages[count - 1 - (off[b] + j - have)];
      }
    }
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) {
      const int64_t t = t0 + 32 * x;
      if (t >= stop) break;
      if (t < total && page[x] < 0) record_status(kStatusBounds);
      a.slots[t] = page[x] < 0 ? -1 : (static_cast<int64_t>(page[x]) << a.page_log2) + (pos[x] & ((1 << a.page_log2) - 1));
      a.positions[t] = pos[x];
    }
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
// (queries) a channel.  A lane takes `per` heads of its token, so that the
// table's 8 bytes a channel are read once for all of them, and loads four heads
// ahead: 4099 tokens of 64 + 16 heads of 128 took 44 us on B200, and 8 us to read
// back (both with one head at a time 78 us), for 27 us of traffic.  No unit is
// full there (issue slots 61 %, DRAM 34 %): 64 registers leave 32 warps an SM, which
// wait for their loads and, row by row, for a chain of shuffles and divisions.
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;

// Where row `h` of kind `kv` (0 key, 1 value) at `slot` lives: code bytes and meta words.
__device__ __forceinline__ int64_t kv4_row(const Kv4Cache &c, int64_t slot, int kv, int h) {
  const int64_t page = slot >> c.page_log2;
  return (((page * 2 + kv) * c.H + h) << c.page_log2) + (slot & ((1 << c.page_log2) - 1));
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads, 4) kv4_append_kernel(const AppendArgs a, int per) {
  constexpr int kLanes = D / 8, kAhead = 4;
  const int sub = threadIdx.x % kLanes;
  const unsigned mask = ((1u << kLanes) - 1u) << (threadIdx.x & 31 & ~(kLanes - 1));
  const int rows = a.Hq + 2 * a.cache.H;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / kLanes) + threadIdx.x / kLanes;
  if (t >= a.T) return;
  const int64_t slot = a.slots[t];
  if (slot < 0) return;  // padding behind the last token
  const int64_t pos = a.positions ? a.positions[t] : 0;
  if (slot >= a.cache.pages << a.cache.page_log2 || pos < 0 || (a.positions && pos >= a.max_pos)) {
    if (sub == 0) record_status(kStatusBounds);
    return;
  }
  // a lane lies in one half of the rotated channels, or behind both: half is a multiple of 8
  const int half = a.rotary / 2, c0 = sub * 8;
  const bool second = c0 >= half, turned = c0 < a.rotary;
  const int other = second ? sub - half / 8 : sub + half / 8;
  float cs[8], sn[8];  // sn negative in the first half: x cos - y sin is x cos + y (-sin), rounding and all
  if (turned) {
    const float *angle = a.rope + pos * a.rotary + (second ? c0 - half : c0);
    load8(angle, cs);
    load8(angle + half, sn);
#pragma unroll
    for (int j = 0; j < 8; ++j) sn[j] = second ? sn[j] : -sn[j];
  }
  const __half *q_row = a.q + t * a.q_stride + c0, *k_row = a.k + t * a.k_stride + c0, *v_row = a.v + t * a.v_stride + c0;
  __half *q_to = a.q_out + t * a.q_out_stride + c0;
  const int64_t first_row = kv4_row(a.cache, slot, 0, 0), to_value = static_cast<int64_t>(a.cache.H) << a.cache.page_log2;
  const int h_end = min(rows, static_cast<int>(blockIdx.y + 1) * per);
  for (int h0 = blockIdx.y * per; h0 < h_end; h0 += kAhead) {
    uint4 ahead[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int h = h0 + x;
      if (h < h_end) {
        const __half *src = h < a.Hq ? q_row + h * D
                                     : (h < a.Hq + a.cache.H ? k_row + (h - a.Hq) * D : v_row + (h - a.Hq - a.cache.H) * D);
        ahead[x] = *reinterpret_cast<const uint4 *>(src);
      }
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      const int h = h0 + x;
      if (h >= h_end) break;
      uint4 raw = ahead[x];
      if (half > 0 && h < a.Hq + a.cache.H) {
        uint4 far;
        far.x = __shfl_sync(mask, raw.x, other, kLanes);
        far.y = __shfl_sync(mask, raw.y, other, kLanes);
        far.z = __shfl_sync(mask, raw.z, other, kLanes);
        far.w = __shfl_sync(mask, raw.w, other, kLanes);
        if (turned) {
          const __half2 *n2 = reinterpret_cast<const __half2 *>(&raw), *f2 = reinterpret_cast<const __half2 *>(&far);
          float own[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 u = __half22float2(n2[j]), w = __half22float2(f2[j]);
            own[2 * j] = __fadd_rn(__fmul_rn(u.x, cs[2 * j]), __fmul_rn(w.x, sn[2 * j]));
            own[2 * j + 1] = __fadd_rn(__fmul_rn(u.y, cs[2 * j + 1]), __fmul_rn(w.y, sn[2 * j + 1]));
          }
          raw = pack8(own);
        }
      }
      if (h < a.Hq) {
        *reinterpret_cast<uint4 *>(q_to + h * D) = raw;
        continue;
      }
      const __half2 *h2 = reinterpret_cast<const __half2 *>(&raw);
      float v[8], lo = 0.0f, hi = 0.0f;
      bool odd = false;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(h2[j]);
        v[2 * j] = f.x, v[2 * j + 1] = f.y;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        lo = fminf(lo, v[j]), hi = fmaxf(hi, v[j]);
        odd |= !(fabsf(v[j]) <= 65504.0f);
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
        for (int j = 0; j < 8; ++j) code |= static_cast<uint32_t>(w4_code(v[j], p)) << (4 * j);
        meta = static_cast<uint32_t>(__half_as_ushort(p.sh)) | static_cast<uint32_t>(p.z) << 16;
      }
      const bool value = h >= a.Hq + a.cache.H;
      const int64_t row = first_row + (value ? to_value : 0) +
                          (static_cast<int64_t>(h - a.Hq - (value ? a.cache.H : 0)) << a.cache.page_log2);
      *reinterpret_cast<uint32_t *>(a.cache.codes + row * (D / 2) + sub * 4) = code;
      if (sub == 0) a.cache.meta[row] = meta;
    }
  }
}

// The cached rows of the given slots as fp16: s * (code - z), rounded once and
// kept within the finite fp16 values (15 steps of a scale rounded up can pass
// the largest one).
template <int D>
__global__ void __launch_bounds__(kAppendThreads) kv4_read_kernel(const Kv4Cache c, const int64_t *__restrict__ slots,
                                                                  int64_t T, __half *__restrict__ k,
                                                                  __half *__restrict__ v, int per) {
  constexpr int kLanes = D / 8;
  const int sub = threadIdx.x % kLanes;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / kLanes) + threadIdx.x / kLanes;
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
    const int64_t row = kv4_row(c, slot, kv, head);
    const uint32_t code = *reinterpret_cast<const uint32_t *>(c.codes + row * (D / 2) + sub * 4), meta = c.meta[row];
    const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(meta & 0xFFFFu)));
    // code + 2^23 as a float, less z + 2^23: the difference, exactly
    const float z = __uint_as_float(0x4B000000u | (meta >> 16 & 15u));
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = (__uint_as_float(0x4B000000u | (code >> (4 * j) & 15u)) - z) * s;
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

// Heads of one lane: eight where the call fills the GPU all the same, one where
// it is latency that counts.
static int heads_per_lane(int64_t T, int rows, int D) {
  const int64_t lanes = T * rows * (D / 8);
  int per = lanes >= 8ll * 148 * 2048 ? 8 : 1;
  while ((rows + per - 1) / per > 65535) ++per;
  return per;
}
static dim3 append_grid(int64_t T, int rows, int D, int per) {
  const int tokens = kAppendThreads / (D / 8);
  return dim3(static_cast<unsigned>((T + tokens - 1) / tokens), static_cast<unsigned>((rows + per - 1) / per));
}

cudaError_t launch_kv4_append(const AppendArgs &a, cudaStream_t stream) {
  const int rows = a.Hq + 2 * a.cache.H, per = heads_per_lane(a.T, rows, a.cache.D);
  const dim3 grid = append_grid(a.T, rows, a.cache.D, per);
  if (a.cache.D == 128) kv4_append_kernel<128><<<grid, kAppendThreads, 0, stream>>>(a, per);
  else kv4_append_kernel<64><<<grid, kAppendThreads, 0, stream>>>(a, per);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4Cache &c, const int64_t *slots, int64_t T, void *k, void *v,
                            cudaStream_t stream) {
  const int per = heads_per_lane(T, 2 * c.H, c.D);
  const dim3 grid = append_grid(T, 2 * c.H, c.D, per);
  __half *kh = static_cast<__half *>(k), *vh = static_cast<__half *>(v);
  if (c.D == 128) kv4_read_kernel<128><<<grid, kAppendThreads, 0, stream>>>(c, slots, T, kh, vh, per);
  else kv4_read_kernel<64><<<grid, kAppendThreads, 0, stream>>>(c, slots, T, kh, vh, per);
  return cudaGetLastError();
}

}  // namespace mixllm
