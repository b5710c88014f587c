// attn_evict.cu — eviction from K/V caches by accumulated attention weight on
// GB300 (sm_103a): keep the positions whose weight is largest and the most
// recent ones, and gather their rows into a smaller cache.
//
// Per sequence b and K/V head u, with len = lens[b] cached positions, a budget
// of N and a window of R recent positions:
//
//   len <= N   keep all;
//   len >  N   keep the last R positions and, of the len - R before them, the
//              N - R of largest weight, ties to the lowest position.
//
// The kept positions stay in order. Two kernels:
//
//   select  one cluster of 1 to 8 CTAs per (b, u). A radix select over the
//           weights' order-preserving integer keys (three passes of 11, 11 and
//           10 bits) finds the (N - R)-th largest key: each CTA counts its part
//           of the row in shared memory and sums the cluster's counts through
//           distributed shared memory. A last pass compacts the kept positions
//           in order (prefix sums over warps, CTA and cluster) and writes their
//           index and weight.
//   gather  copies the kept K and V rows, in the order of the destination, 16
//           bytes a lane; it is what the call's bytes are.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "attn_prefill.h"

namespace gb300_host {
attn_status_t device_status_word(cudaStream_t stream, int** status);
}

namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;               // 11-bit digits (the last one has 10)
constexpr int kMaxCluster = 8;
constexpr int kPartSmem = 40960;          // weights of a CTA's part held in shared memory
constexpr int kGatherThreads = 256;
constexpr int kGatherRows = 64;           // destination positions per gather CTA

struct EvictParams {
  const float* w;       // [B, n_kv, C]
  const int* lens;      // [B]
  float* w_out;         // [B, n_kv, C_out]
  int* index;           // [B, n_kv, N]
  int* lens_out;        // [B]
  int n_kv, N, R;
  int C, C_out;
  int part;             // positions per CTA of a cluster
};

// Order-preserving integer of a weight: larger weight, larger key. -0 equals
// +0 and a NaN is below everything.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct SelectSmem {
  unsigned int hist[kBins];        // this CTA's counts, read by the cluster
  unsigned int warp_sum[kSelWarps];
  unsigned int n_gt, n_eq;         // this CTA's kept and tied positions, read by the cluster
  unsigned int digit, above;       // the digit of the key sought, keys above it
  unsigned int scan_total;
};

// Inclusive sum of v over the CTA's threads; *total gets the sum of all.
__device__ __forceinline__ unsigned int block_scan(unsigned int v, SelectSmem& sm,
                                                   unsigned int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned int n = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += n;
  }
  if (lane == 31) sm.warp_sum[warp] = v;
  __syncthreads();
  if (warp == 0) {
    unsigned int s = sm.warp_sum[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const unsigned int n = __shfl_up_sync(0xffffffffu, s, off);
      if (lane >= off) s += n;
    }
    sm.warp_sum[lane] = s;
  }
  __syncthreads();
  const unsigned int base = warp ? sm.warp_sum[warp - 1] : 0u;
  *total = sm.warp_sum[kSelWarps - 1];
  __syncthreads();
  return base + v;
}

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const EvictParams p) {
  extern __shared__ __align__(16) float held[];      // the part's weights, when they fit
  __shared__ SelectSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int ncta = static_cast<int>(cluster.num_blocks());
  const int row = static_cast<int>(blockIdx.x) / ncta;      // b * n_kv + u
  const int b = row / p.n_kv;
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const int len = min(max(p.lens[b], 0), p.C);
  const int kept = min(len, p.N);
  const int old = len > p.N ? len - p.R : len;   // positions that compete (all are kept if len <= N)
  const int need = kept - (len - old);           // how many of them stay
  const float* w = p.w + static_cast<size_t>(row) * p.C;
  float* w_out = p.w_out + static_cast<size_t>(row) * p.C_out;
  int* index = p.index + static_cast<size_t>(row) * p.N;

  // what lies behind the kept positions, and the recent ones
  for (int i = kept + rank * kSelThreads + tid; i < p.C_out; i += ncta * kSelThreads) w_out[i] = 0.0f;
  for (int i = kept + rank * kSelThreads + tid; i < p.N; i += ncta * kSelThreads) index[i] = -1;
  for (int i = need + rank * kSelThreads + tid; i < kept; i += ncta * kSelThreads) {
    const int src = old + (i - need);
    w_out[i] = w[src];
    index[i] = src;
  }
  if (rank == 0 && tid == 0 && row % p.n_kv == 0) p.lens_out[b] = kept;

  const int lo = min(rank * p.part, old), hi = min(lo + p.part, old);
  if (need == old) {                             // the same for the whole cluster
    for (int i = lo + tid; i < hi; i += kSelThreads) {
      w_out[i] = w[i];
      index[i] = i;
    }
    return;
  }
  const bool in_smem = p.part <= kPartSmem;
  const float* src = w + lo;
  const int n = hi - lo;
  if (in_smem) {
    for (int i = tid; i < n; i += kSelThreads) held[i] = w[lo + i];
    src = held;
    __syncthreads();
  }

  // the need-th largest key: `prefix` holds its digits found so far, `above`
  // the number of keys larger than every key with this prefix
  uint32_t prefix = 0;
  unsigned int above = 0;
  bool all = need == 0;                          // nothing of the older part stays
  for (int pass = 0; pass < 3 && !all; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    for (int i = tid; i < kBins; i += kSelThreads) sm.hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t key = order_key(src[i]);
      if (pass == 0 || (key >> (pass == 1 ? 21 : 10)) == prefix)
        atomicAdd(&sm.hist[(key >> shift) & mask], 1u);
    }
    cluster.sync();
    // digits in descending order: thread t owns digits 2047 - 2t and 2046 - 2t
    unsigned int c0 = 0, c1 = 0;
    const int d0 = kBins - 1 - 2 * tid, d1 = d0 - 1;
    for (int r = 0; r < ncta; ++r) {
      const unsigned int* h = cluster.map_shared_rank(sm.hist, r);
      c0 += h[d0];
      c1 += h[d1];
    }
    unsigned int total;
    const unsigned int incl = block_scan(c0 + c1, sm, &total);
    const unsigned int before = above + incl - c0 - c1;       // keys above digit d0
    const unsigned int want = static_cast<unsigned int>(need);
    if (before < want && before + c0 >= want) {
      sm.digit = d0;
      sm.above = before;
    } else if (before + c0 < want && before + c0 + c1 >= want) {
      sm.digit = d1;
      sm.above = before + c0;
    }
    __syncthreads();
    prefix = (prefix << (pass == 2 ? 10 : 11)) | sm.digit;
    above = sm.above;
    cluster.sync();                              // every CTA has read the counts
  }
  // kept: keys above `prefix`, and the first `ties` of those equal to it
  const unsigned int ties = all ? 0u : static_cast<unsigned int>(need) - above;

  // this CTA's counts, then how many lie in the CTAs before it
  unsigned int gt = 0, eq = 0;
  if (!all) {
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t key = order_key(src[i]);
      gt += key > prefix;
      eq += key == prefix;
    }
  }
  unsigned int n_gt, n_eq;
  block_scan(gt, sm, &n_gt);
  block_scan(eq, sm, &n_eq);
  if (tid == 0) {
    sm.n_gt = n_gt;
    sm.n_eq = n_eq;
  }
  cluster.sync();
  unsigned int base_gt = 0, base_eq = 0;
  for (int r = 0; r < rank; ++r) {
    base_gt += *cluster.map_shared_rank(&sm.n_gt, r);
    base_eq += *cluster.map_shared_rank(&sm.n_eq, r);
  }
  // in order, kSelThreads positions at a time
  for (int i0 = 0; i0 < n && !all; i0 += kSelThreads) {
    const int i = i0 + tid;
    const float x = i < n ? src[i] : 0.0f;
    const uint32_t key = i < n ? order_key(x) : 0u;
    const bool is_gt = i < n && key > prefix, is_eq = i < n && key == prefix;
    unsigned int t;
    // both counts in one scan: at most 1024 of each
    const unsigned int s =
        block_scan((is_gt ? 1u : 0u) | (is_eq ? 1u << 16 : 0u), sm, &t);
    const unsigned int my_gt = base_gt + (s & 0xFFFFu), my_eq = base_eq + (s >> 16);   // inclusive
    if (is_gt || (is_eq && my_eq <= ties)) {
      const unsigned int at = my_gt + min(my_eq, ties) - 1u;
      w_out[at] = x;
      index[at] = lo + i;
    }
    base_gt += t & 0xFFFFu;
    base_eq += t >> 16;
  }
  cluster.sync();                                // no CTA ends while its counts are read
}

struct GatherParams {
  const uint4* k;       // [B, C, n_kv, row16] rows of row16 16-byte units
  const uint4* v;
  uint4* k_out;         // [B, C_out, n_kv, row16]
  uint4* v_out;
  const int* index;     // [B, n_kv, N]
  const int* lens_out;  // [B]
  int n_kv, N, C, C_out, row16, blocks;
};

// One CTA per (b, kGatherRows destination positions): the positions' indexes
// for every head go to shared memory, then the lanes copy the destination's
// 16-byte units in order (contiguous stores, loads of whole rows).
__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const GatherParams p) {
  extern __shared__ __align__(16) int idx[];           // [n_kv][kGatherRows]
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = static_cast<int>(blockIdx.x) / p.blocks;
  const int i0 = (static_cast<int>(blockIdx.x) - b * p.blocks) * kGatherRows;
  const int rows = min(p.lens_out[b] - i0, kGatherRows);
  if (rows <= 0) return;
  for (int t = threadIdx.x; t < p.n_kv * kGatherRows; t += kGatherThreads) {
    const int u = t / kGatherRows, i = t - u * kGatherRows;
    if (i < rows) idx[t] = p.index[(static_cast<size_t>(b) * p.n_kv + u) * p.N + i0 + i];
  }
  __syncthreads();
  const int per_pos = p.n_kv * p.row16;
  const size_t src0 = static_cast<size_t>(b) * p.C * per_pos;
  const size_t dst0 = (static_cast<size_t>(b) * p.C_out + i0) * per_pos;
  const int units = rows * per_pos;
  constexpr int kUnroll = 4;
  for (int t0 = threadIdx.x; t0 < units; t0 += kUnroll * kGatherThreads) {
    uint4 a[kUnroll], c[kUnroll];
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
      const int t = t0 + e * kGatherThreads;
      if (t >= units) break;
      const int i = t / per_pos, rest = t - i * per_pos, u = rest / p.row16;
      const size_t s = src0 + static_cast<size_t>(idx[u * kGatherRows + i]) * per_pos + rest;
      a[e] = __ldcs(p.k + s);
      c[e] = __ldcs(p.v + s);
    }
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
      const int t = t0 + e * kGatherThreads;
      if (t >= units) break;
      p.k_out[dst0 + t] = a[e];
      p.v_out[dst0 + t] = c[e];
    }
  }
}

constexpr int kMaxDevices = 64;
std::mutex g_evict_mutex;
bool g_evict_ready[kMaxDevices] = {};

attn_status_t evict_device_ready(cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_UNSUPPORTED;
  // the device check (sm_103) is the forward's
  int* status = nullptr;
  const attn_status_t ds = gb300_host::device_status_word(stream, &status);
  if (ds != ATTN_OK) return ds;
  std::lock_guard<std::mutex> lock(g_evict_mutex);
  if (g_evict_ready[dev]) return ATTN_OK;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess || cs != cudaStreamCaptureStatusNone) {
    cudaGetLastError();
    return ATTN_ERR_UNSUPPORTED;
  }
  if (cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kPartSmem * 4) != cudaSuccess)
    return ATTN_ERR_CUDA;
  g_evict_ready[dev] = true;
  return ATTN_OK;
}

bool misaligned(const void* ptr, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0;
}

struct Span {
  uintptr_t at;
  uint64_t bytes;
};
Span span(const void* ptr, int64_t bytes) {
  return {reinterpret_cast<uintptr_t>(ptr), static_cast<uint64_t>(bytes)};
}
bool overlap(const Span& a, const Span& b) {
  return a.at < b.at + b.bytes && b.at < a.at + a.bytes;
}

}  // namespace

extern "C" attn_status_t attn_cache_evict(const void* k, const void* v, const float* weights,
                                          const int32_t* lens, void* k_out, void* v_out,
                                          float* weights_out, int32_t* lens_out, int32_t* index,
                                          int64_t B, int64_t C, int64_t C_out, int64_t budget,
                                          int64_t recent, int32_t n_kv, int32_t d_h,
                                          int32_t elem_bytes, void* stream_ptr) {
  if (!k || !v || !weights || !lens || !k_out || !v_out || !weights_out || !lens_out || !index)
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || C < 1 || n_kv < 1 || budget < 1 || recent < 0 || recent > budget ||
      C_out < budget || (elem_bytes != 1 && elem_bytes != 2))
    return ATTN_ERR_INVALID_ARG;
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(k_out, 16) || misaligned(v_out, 16) ||
      misaligned(weights, 4) || misaligned(weights_out, 4) || misaligned(lens, 4) ||
      misaligned(lens_out, 4) || misaligned(index, 4))
    return ATTN_ERR_INVALID_ARG;
  if (d_h != 64 && d_h != 128) return ATTN_ERR_UNSUPPORTED;
  constexpr int64_t kMost = int64_t{1} << 30;
  const int64_t blocks = (budget + kGatherRows - 1) / kGatherRows;
  if (C > kMost || C_out > kMost || B > kMost || n_kv > 128 || B * n_kv > (int64_t{1} << 24) ||
      B * blocks > INT32_MAX)
    return ATTN_ERR_UNSUPPORTED;
  const int64_t row = static_cast<int64_t>(d_h) * elem_bytes;
  const Span in[4] = {span(k, B * C * n_kv * row), span(v, B * C * n_kv * row),
                      span(weights, B * n_kv * C * 4), span(lens, B * 4)};
  const Span out[5] = {span(k_out, B * C_out * n_kv * row), span(v_out, B * C_out * n_kv * row),
                       span(weights_out, B * n_kv * C_out * 4), span(lens_out, B * 4),
                       span(index, B * n_kv * budget * 4)};
  for (int i = 0; i < 5; ++i) {
    for (const Span& s : in)
      if (overlap(out[i], s)) return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return ATTN_ERR_INVALID_ARG;
  }
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  const attn_status_t ds = evict_device_ready(stream);
  if (ds != ATTN_OK) return ds;

  const int64_t rows = B * n_kv;
  int cluster = 1;
  while (cluster < kMaxCluster && rows * cluster * 2 <= 304 && C >= 4096 * 2 * cluster) cluster *= 2;
  EvictParams p;
  p.w = weights;
  p.lens = lens;
  p.w_out = weights_out;
  p.index = index;
  p.lens_out = lens_out;
  p.n_kv = n_kv;
  p.N = static_cast<int>(budget);
  p.R = static_cast<int>(recent);
  p.C = static_cast<int>(C);
  p.C_out = static_cast<int>(C_out);
  p.part = static_cast<int>((C + cluster - 1) / cluster);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * cluster));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = p.part <= kPartSmem ? static_cast<size_t>(p.part) * 4 : 0;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, evict_select_kernel, p) != cudaSuccess) return ATTN_ERR_CUDA;

  GatherParams g;
  g.k = static_cast<const uint4*>(k);
  g.v = static_cast<const uint4*>(v);
  g.k_out = static_cast<uint4*>(k_out);
  g.v_out = static_cast<uint4*>(v_out);
  g.index = index;
  g.lens_out = lens_out;
  g.n_kv = n_kv;
  g.N = p.N;
  g.C = p.C;
  g.C_out = p.C_out;
  g.row16 = static_cast<int>(row / 16);
  g.blocks = static_cast<int>(blocks);
  cfg.gridDim = dim3(static_cast<unsigned>(B * blocks));
  cfg.blockDim = dim3(kGatherThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(n_kv) * kGatherRows * 4;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, evict_gather_kernel, g) != cudaSuccess) return ATTN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
