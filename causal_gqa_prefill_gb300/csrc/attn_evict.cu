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
//   select  one cluster of 1 to 8 CTAs per (b, u), each with its part of the row
//           in shared memory. A radix select over the weights' order-preserving
//           integer keys, 8 bits a pass, finds the (N - R)-th largest key; it
//           ends early when a pass leaves exactly the keys that are needed, or
//           few enough to compare with one another. A
//           CTA counts into 32 histograms, one per lane, whose counters lie in
//           the lane's own bank: weights crowd into a few exponents, and with one
//           histogram the atomics on its few busy counters took most of the time
//           (39 us of a call for 6 rows of 131072). The cluster's counts are
//           summed through distributed shared memory. A last pass compacts the
//           kept positions in order and writes index and weight. Bound by the
//           latency of its steps: of 16 us for 128 rows of up to 8192, some
//           1.5 to 2.5 us a pass go to the counters' sums, the cluster's barrier
//           and the scan, 0.4 to the counting; 22 us for 6 rows of 131072.
//   gather  copies the kept K and V rows, in the order of the destination, 16
//           bytes a lane; it is what the call's bytes are: 259 MB in 39 us (6.6
//           TB/s, 98 % of a copy's) for 16 sequences of 8 heads brought to 2048.
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

constexpr int kBins = 256;                // 8-bit digits
constexpr int kMaxCluster = 8;
constexpr int kSms = 152;                 // SMs of a GB300
constexpr int kPartSmem = 32768;          // keys of a CTA's part held in shared memory
static_assert(kPartSmem < 1 << 16, "a piece's two counts share 32 bits");
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

// The weight of a key; a NaN's and a zero's bits are the original's (`at`).
__device__ __forceinline__ float weight_of(uint32_t key, const float* at) {
  if (key == 0u || key == 0x80000000u) return *at;
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

struct SelectSmem {
  unsigned int hist[kBins][32];            // [digit][lane]
  unsigned int total[2][kMaxCluster][kBins];   // a pass's counts of every CTA, written by it
  unsigned int warp_sum[32];
  unsigned long long wide_sum[kBins / 32];
  // the digit of the key sought: keys above it and at it in the row, and in
  // the parts of the CTAs before this one
  unsigned int digit, above, at, above_before, at_before;
  unsigned int listed;                     // candidates of this CTA in the list so far
};

// With at most this many keys left to choose from, they are listed (over the
// histograms) and compared with one another instead of counted digit by digit, which
// spares a pass or two (128 rows of 8192: 21 us without, 18 with 128, 20 with 256,
// whose comparisons are four times as many).
constexpr int kList = 128;
static_assert(kList <= 512, "a thread per candidate");

template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
evict_select_kernel(const EvictParams p) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint32_t held[];   // the part's keys, or those of a piece of it
  __shared__ SelectSmem sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int ncta = static_cast<int>(cluster.num_blocks());
  const int row = static_cast<int>(blockIdx.x) / ncta;      // b * n_kv + u
  const int b = row / p.n_kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the cluster's CTAs write to one another's shared memory: all must have begun
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const int len = min(max(p.lens[b], 0), p.C);
  const int kept = min(len, p.N);
  const int old = len > p.N ? len - p.R : len;   // positions that compete (all are kept if len <= N)
  const int need = kept - (len - old);           // how many of them stay
  const float* w = p.w + static_cast<size_t>(row) * p.C;
  float* w_out = p.w_out + static_cast<size_t>(row) * p.C_out;
  int* index = p.index + static_cast<size_t>(row) * p.N;

  const int lo = min(rank * p.part, old), hi = min(lo + p.part, old);
  const int n = hi - lo;
  const bool choose = need != old && need > 0;   // the same for the whole cluster
  const bool in_smem = p.part <= kPartSmem;
  // keys of positions from .. from + m - 1 to shared memory; up to the next
  // multiple of four, keys of nothing (0 is a NaN's: they are not counted)
  auto hold = [&](int from, int m) {
    constexpr int kFlight = 16;                  // loads on their way at once
    for (int i0 = tid; i0 < (m + 3) / 4 * 4; i0 += kFlight * kThreads) {
      float x[kFlight];
#pragma unroll
      for (int e = 0; e < kFlight; ++e) {
        const int i = i0 + e * kThreads;
        x[e] = i < m ? w[from + i] : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < kFlight; ++e) {
        const int i = i0 + e * kThreads;
        if (i < (m + 3) / 4 * 4) held[i] = i < m ? order_key(x[e]) : 0u;
      }
    }
  };
  if (choose && in_smem) hold(lo, n);
  // what lies behind the kept positions, and the recent ones
  for (int i = kept + rank * kThreads + tid; i < p.C_out; i += ncta * kThreads) w_out[i] = 0.0f;
  for (int i = kept + rank * kThreads + tid; i < p.N; i += ncta * kThreads) index[i] = -1;
  for (int i = need + rank * kThreads + tid; i < kept; i += ncta * kThreads) {
    const int src = old + (i - need);
    w_out[i] = w[src];
    index[i] = src;
  }
  if (rank == 0 && tid == 0 && row % p.n_kv == 0) p.lens_out[b] = kept;
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (!choose) {
    if (need > 0)                                // all of them stay
      for (int i = lo + tid; i < hi; i += kThreads) {
        w_out[i] = w[i];
        index[i] = i;
      }
    return;
  }

  // The need-th largest key: `prefix` holds its digits found so far (the key
  // shifted right by `shift`), `above` the number of keys with larger leading
  // digits, and `gt`, `eq` how many of the larger and of the equal ones lie in
  // the CTAs before this one.
  uint32_t prefix = 0;
  unsigned int above = 0, gt = 0, eq = 0;
  int shift = 32;
  for (int pass = 0; pass < 4; ++pass) {
    shift -= 8;
#pragma unroll
    for (int i = 0; i < kBins * 32 / 4 / kThreads; ++i)
      reinterpret_cast<uint4*>(&sm.hist[0][0])[tid + i * kThreads] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    auto count = [&](uint32_t key) {
      if (pass == 0 || (key >> (shift + 8)) == prefix)
        atomicAdd(&sm.hist[(key >> shift) & (kBins - 1)][lane], 1u);
    };
    if (in_smem) {
#pragma unroll 2
      for (int i = 4 * tid; i < n; i += 4 * kThreads) {
        const uint4 key = *reinterpret_cast<const uint4*>(held + i);
        count(key.x);
        if (i + 1 < n) count(key.y);
        if (i + 2 < n) count(key.z);
        if (i + 3 < n) count(key.w);
      }
    } else {
      for (int i = tid; i < n; i += kThreads) count(order_key(w[lo + i]));
    }
    __syncthreads();
    if (tid < kBins) {
      // (each thread starts at another lane's counter: all banks at once)
      unsigned int sum = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) sum += sm.hist[tid][(tid + i) & 31];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < ncta) *cluster.map_shared_rank(&sm.total[pass & 1][rank][tid], r) = sum;
    }
    cluster.sync();
    // digits in descending order, one per thread: counts of the row (low half)
    // and of the CTAs before this one (high half)
    unsigned long long c = 0, incl = 0;
    if (tid < kBins) {
      unsigned int all = 0, before = 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        const unsigned int x = r < ncta ? sm.total[pass & 1][r][kBins - 1 - tid] : 0u;
        all += x;
        before += r < rank ? x : 0u;
      }
      c = all | static_cast<unsigned long long>(before) << 32;
      incl = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
      }
      if (lane == 31) sm.wide_sum[warp] = incl;
    }
    __syncthreads();
    if (tid < kBins) {
      for (int x = 0; x < warp; ++x) incl += sm.wide_sum[x];
      const unsigned long long excl = incl - c;
      const unsigned int larger = above + static_cast<unsigned int>(excl);
      const unsigned int here = static_cast<unsigned int>(c);
      if (larger < static_cast<unsigned int>(need) && larger + here >= static_cast<unsigned int>(need)) {
        sm.digit = kBins - 1 - tid;
        sm.above = larger;
        sm.at = here;
        sm.above_before = static_cast<unsigned int>(excl >> 32);
        sm.at_before = static_cast<unsigned int>(c >> 32);
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | sm.digit;
    above = sm.above;
    gt += sm.above_before;
    eq = sm.at_before;
    const unsigned int left = sm.at;                  // keys that share the digits so far
    if (above + left == static_cast<unsigned int>(need)) break;    // all of these stay
    if (left <= kList && pass < 3) {
      // every CTA's candidates to every CTA's list, those of the CTAs before first
      const unsigned int first = eq;
      unsigned int* const list = &sm.hist[0][0];
      if (tid == 0) sm.listed = first;
      __syncthreads();
      auto put = [&](uint32_t key) {
        if ((key >> shift) != prefix) return;
        const unsigned int slot = atomicAdd(&sm.listed, 1u);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < ncta) *cluster.map_shared_rank(list + slot, r) = key;
      };
      if (in_smem) {
        for (int i = tid; i < n; i += kThreads) put(held[i]);
      } else {
        for (int i = tid; i < n; i += kThreads) put(order_key(w[lo + i]));
      }
      cluster.sync();
      const uint32_t key = tid < left ? list[tid] : 0u;
      if (tid < left) {
        unsigned int larger = 0, same = 0;
        for (unsigned int j = 0; j < left; ++j) {
          larger += list[j] > key ? 1u : 0u;
          same += list[j] == key ? 1u : 0u;
        }
        const unsigned int k = static_cast<unsigned int>(need) - above;
        if (larger < k && larger + same >= k) {       // (equal keys write the same)
          sm.digit = key;
          sm.above = above + larger;
        }
      }
      __syncthreads();
      prefix = sm.digit;
      above = sm.above;
      shift = 0;
      gt += __syncthreads_count(tid < left && tid < first && key > prefix);
      eq = __syncthreads_count(tid < left && tid < first && key == prefix);
      break;
    }
  }
  // kept: keys above `prefix`, and the first `ties` of those equal to it
  const unsigned int ties = static_cast<unsigned int>(need) - above;

  // in order, a piece of at most kPartSmem positions at a time; a warp takes a
  // run of whole rows of 32. First the warps' counts, then, with those before
  // it known, each row's kept positions next to each other.
  for (int i0 = 0; i0 < n; i0 += kPartSmem) {
    const int m = min(n - i0, kPartSmem);
    if (!in_smem) {
      __syncthreads();
      hold(lo + i0, m);
      __syncthreads();
    }
    const int run = ((m + 31) / 32 + kWarps - 1) / kWarps * 32;
    const int r0 = min(warp * run, m), r1 = min(r0 + run, m);
    unsigned int my = 0;                                     // larger | equal << 16
    for (int i = r0 + lane; i < r1; i += 32) {
      const uint32_t lead = held[i] >> shift;
      my += lead > prefix ? 1u : 0u;
      my += lead == prefix ? 1u << 16 : 0u;
    }
    my = __reduce_add_sync(0xffffffffu, my);                 // a piece has fewer than 2^16
    if (lane == 0) sm.warp_sum[warp] = my;
    __syncthreads();
    const unsigned int ws = lane < kWarps ? sm.warp_sum[lane] : 0u;
    const unsigned int before = __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0u);
    const unsigned int all = __reduce_add_sync(0xffffffffu, ws);
    unsigned int at_gt = gt + (before & 0xFFFFu), at_eq = eq + (before >> 16);
    const unsigned int lower = (1u << lane) - 1u;
    for (int i = r0; i < r1; i += 32) {
      const uint32_t key = i + lane < r1 ? held[i + lane] : 0u;
      const uint32_t lead = key >> shift;
      const bool is_gt = i + lane < r1 && lead > prefix, is_eq = i + lane < r1 && lead == prefix;
      const unsigned int mg = __ballot_sync(0xffffffffu, is_gt), me = __ballot_sync(0xffffffffu, is_eq);
      const unsigned int my_eq = at_eq + __popc(me & lower);
      if (is_gt || (is_eq && my_eq < ties)) {
        const unsigned int to = at_gt + __popc(mg & lower) + min(my_eq, ties);
        w_out[to] = weight_of(key, w + lo + i0 + i + lane);
        index[to] = lo + i0 + i + lane;
      }
      at_gt += __popc(mg);
      at_eq += __popc(me);
    }
    gt += all & 0xFFFFu;
    eq += all >> 16;
    if (!in_smem) __syncthreads();
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
  if (cudaFuncSetAttribute(evict_select_kernel<512>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kPartSmem * 4) != cudaSuccess ||
      cudaFuncSetAttribute(evict_select_kernel<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
  // CTAs per row while two fit an SM and each has 4096 positions: few long rows
  // need them (a call for 6 rows of 131072 and few kept: 96, 55, 29 and 22 us with 1, 2,
  // 4 and 8, no less with 16), for 128 rows of 8192 one or two are the same (21)
  int cluster = 1;
  while (cluster < kMaxCluster && rows * cluster * 2 <= 2 * kSms && C >= 4096 * 2 * cluster)
    cluster *= 2;
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
  // 1024 threads to a CTA, or two CTAs of 512 to an SM where there are more CTAs
  // than SMs (512 rows of 2048: 31 us, 40 with 1024) or so many large clusters that
  // some would wait for eight free SMs side by side (16 rows of 131072: 33, 40);
  // else 1024 are as fast or faster (64 rows of 8192: 16, 18)
  const bool wide = rows * cluster <= (cluster < 4 ? kSms : kSms / 2);
  cfg.blockDim = dim3(wide ? 1024 : 512);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.part <= kPartSmem ? (p.part + 3) / 4 * 4 : kPartSmem) * 4;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if ((wide ? cudaLaunchKernelEx(&cfg, evict_select_kernel<1024>, p)
            : cudaLaunchKernelEx(&cfg, evict_select_kernel<512>, p)) != cudaSuccess)
    return ATTN_ERR_CUDA;

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
