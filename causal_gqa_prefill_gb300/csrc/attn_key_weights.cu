// attn_key_weights.cu — the attention that every key of a prefill received, on
// GB300 (sm_103a): the column sums of the softmax weights, rebuilt from Q, K
// and the forward's log-sum-exps,
//
//   W[b,u,j] (+)= sum_{h in group u} sum_{i sees j} 2^(c q_ih . k_ju - lse2_ih),
//   c = scale * log2(e),  lse2 = LSE * log2(e).
//
// With the keys on the TMEM lanes (S^T = K Q^T, tcgen05, both operands in
// shared memory) a column sum is a sum over one thread's own columns: no
// reduction over threads at all, one FMA, one exponential and one addition per
// score. The columns are packed: one step of 128 columns holds nr = 128 / g
// consecutive query rows of all g heads of the group (column = row * g + head,
// which is what one TMA box of g heads x nr rows lands as), so every head
// count fills the tile, a causal step wastes at most nr rows, and masking a
// row means comparing the column with a threshold.
//
//   unit     256 keys of one (b, K/V head): two 128-key tiles that read the same
//            Q steps (at one tile the Q tiles would need 64 bytes a clock and SM
//            from L2; two halve that). A unit's steps are the row blocks that
//            see it, in order.
//   CTA      one per SM; the steps of all units, in order, are cut into equal
//            ranges (triangles need no further balancing). A unit that a range
//            border cuts is summed by a second kernel from at most one partial
//            per CTA, in CTA order: no atomics, the same bits every time.
//   warps    0-3 and 4-7 one warpgroup per key tile; 8 TMA; 9 MMA; 10 the rows'
//            -lse2 (shared memory, read by the whole warpgroup as broadcasts).
//
// S^T is double-buffered per key tile (4 x 128 TMEM columns), so the products
// of a step run under the exponentials of the one before; both take 1024
// clocks a step, the exponentials at 32 a clock and SM.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "attn_prefill.h"
#include "sm103_ptx.cuh"

namespace gb300_host {
attn_status_t device_status_word(cudaStream_t stream, int** status);
}

namespace {

using namespace gb300;

constexpr int kKeys = 128;            // keys per tile (TMEM lanes)
constexpr int kUnitKeys = 2 * kKeys;
constexpr int kCols = 128;            // columns (query rows x heads) per step
constexpr int kCtas = 152;            // one CTA per SM on a 152-SM GB300
constexpr int kThreads = 384;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kLseWarp = 10;
constexpr uint32_t kTmemCols = 512;
constexpr int kStatusTimeout = 1;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Geometry {
  static constexpr int kChunks = D * 2 / 128;              // 128-byte swizzle column chunks
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kChunkBytes = 128 * 128;
  static constexpr int kQStages = D == 128 ? 3 : 6;
  // K: two buffers of two tiles; Q ring; two steps' row statistics
  static constexpr int kSmemBytes = (4 + kQStages) * kTileBytes + 2 * kCols * 4 + 1024;
};

struct Params {
  const float* lse;      // [B, n_q, Lq]
  float* weights;        // [B, n_kv, Lk]
  float* part;           // [G][2][kUnitKeys] partial sums of cut units
  int* status;
  int Lq, Lk, off;       // off = Lk - Lq, the position of row 0
  int n_q, n_kv, g, nr;  // nr = 128 / g rows per step
  int steps;             // ceil(Lq / nr)
  int T;                 // units per (b, K/V head)
  int causal, accumulate, G;
  float c;
  long long spin_limit;
};

// Where each CTA's range starts: unit, step, and the number of steps.
struct Starts {
  int unit[kCtas], step[kCtas], count[kCtas];
};

struct Ctl {
  uint64_t k_full[2], k_empty[2];
  uint64_t q_full[6], q_empty[6];
  uint64_t l_full[2], l_empty[2];
  uint64_t s_full[2][2], s_free[2][2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

__host__ __device__ __forceinline__ int first_step(int t, int off, int nr, int causal) {
  const long long past = static_cast<long long>(t) * kUnitKeys - off;
  return causal && past > 0 ? static_cast<int>(past / nr) : 0;
}

struct Segment {
  int unit, b, kvh, key0, s0, n;
  bool first, whole;     // the range's first segment; a unit that nothing cuts
};

struct Walk {
  const Params& p;
  int unit, step, left;
  bool first;
  __device__ Walk(const Params& params, const Starts& st, int c)
      : p(params), unit(st.unit[c]), step(st.step[c]), left(st.count[c]), first(true) {}
  __device__ bool next(Segment& s) {
    if (left <= 0) return false;
    const int grp = unit / p.T, t = unit - grp * p.T;
    s.unit = unit;
    s.b = grp / p.n_kv;
    s.kvh = grp - s.b * p.n_kv;
    s.key0 = t * kUnitKeys;
    s.s0 = step;
    s.n = min(left, p.steps - step);
    s.first = first;
    s.whole = s.n == p.steps - first_step(t, p.off, p.nr, p.causal);
    left -= s.n;
    first = false;
    ++unit;
    step = unit % p.T ? first_step(unit % p.T, p.off, p.nr, p.causal) : 0;
    return true;
  }
};

// Key tile w of a segment takes part in step `step`: it has keys, and the
// step's last row sees the first of them.
__device__ __forceinline__ bool takes_part(const Params& p, int key, int step) {
  if (key >= p.Lk) return false;
  const int last = min((step + 1) * p.nr, p.Lq) - 1;
  return !p.causal || key <= last + p.off;
}

__device__ __forceinline__ bool spin_wait(uint32_t bar, uint32_t parity, Ctl& ctl,
                                          const Params& p) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = clock64_now();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&ctl.abort)) return false;
    if (static_cast<long long>(clock64_now() - t0) > p.spin_limit) {
      *reinterpret_cast<volatile int*>(&ctl.abort) = 1;
      atomicOr(p.status, kStatusTimeout);
      return false;
    }
  }
}

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, Ctl& ctl,
                                          const Params& p) {
  return __all_sync(0xffffffffu, spin_wait(bar, parity, ctl, p));
}

// Wait used while draining after an abort: ignores the abort flag.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, const Params& p) {
  const uint64_t t0 = clock64_now();
  while (!mbar_try_wait(bar, parity))
    if (static_cast<long long>(clock64_now() - t0) > p.spin_limit) return;
}

// sum over the step's columns of 2^(c s + nl) for this thread's key; kMask:
// columns below `from` are rows that do not see it.
template <bool kMask>
__device__ __forceinline__ float column_sum(const float (&s)[kCols], const float* nl, uint64_t c2,
                                            int from) {
  uint64_t a0 = f32x2_pack(0.0f, 0.0f), a1 = a0;
#pragma unroll
  for (int i = 0; i < kCols; i += 4) {
    const float4 l = *reinterpret_cast<const float4*>(nl + i);
    float x0, x1, x2, x3;
    f32x2_unpack(ffma2(f32x2_pack(s[i], s[i + 1]), c2, f32x2_pack(l.x, l.y)), x0, x1);
    f32x2_unpack(ffma2(f32x2_pack(s[i + 2], s[i + 3]), c2, f32x2_pack(l.z, l.w)), x2, x3);
    float e0 = ex2_approx(x0), e1 = ex2_approx(x1), e2 = ex2_approx(x2), e3 = ex2_approx(x3);
    if (kMask) {
      if (i < from) e0 = 0.0f;
      if (i + 1 < from) e1 = 0.0f;
      if (i + 2 < from) e2 = 0.0f;
      if (i + 3 < from) e3 = 0.0f;
    }
    a0 = fadd2(a0, f32x2_pack(e0, e1));
    a1 = fadd2(a1, f32x2_pack(e2, e3));
  }
  float lo, hi;
  f32x2_unpack(fadd2(a0, a1), lo, hi);
  return lo + hi;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
key_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ Params p, const __grid_constant__ Starts starts) {
  using G = Geometry<D>;
  extern __shared__ uint8_t dyn_smem[];
  __shared__ Ctl ctl;
  const uint32_t base = (smem_addr(dyn_smem) + 1023u) & ~1023u;   // swizzle atoms need 1 KiB
  const uint32_t sK = base, sQ = base + 4 * G::kTileBytes;
  const uint32_t sL = sQ + G::kQStages * G::kTileBytes;
  uint8_t* const generic = dyn_smem + (base - smem_addr(dyn_smem));
  float* const nl_ring = reinterpret_cast<float*>(generic + (sL - base));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = static_cast<int>(blockIdx.x);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_addr(&ctl.k_full[s]), 1);
      mbar_init(smem_addr(&ctl.k_empty[s]), 1);
      mbar_init(smem_addr(&ctl.l_full[s]), 32);
      mbar_init(smem_addr(&ctl.l_empty[s]), 8);
      for (int w = 0; w < 2; ++w) {
        mbar_init(smem_addr(&ctl.s_full[w][s]), 1);
        mbar_init(smem_addr(&ctl.s_free[w][s]), 4);
      }
    }
    for (int s = 0; s < G::kQStages; ++s) {
      mbar_init(smem_addr(&ctl.q_full[s]), 1);
      mbar_init(smem_addr(&ctl.q_empty[s]), 1);
    }
    mbar_init(smem_addr(&ctl.drain), 1);
    ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&ctl.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (p.nr * p.g < kCols && warp < 8) {
    // columns past nr * g are never loaded: zeros, so that their scores are 0
    // and their weight 2^(0 - inf) too
    uint4* z = reinterpret_cast<uint4*>(generic + (sQ - base));
    for (int i = threadIdx.x; i < G::kQStages * G::kTileBytes / 16; i += 256)
      z[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = ctl.tmem_base;
  // programmatic dependent of the kernel before it: set-up overlaps that
  // kernel, global memory is touched only after it has completed
  asm volatile("griddepcontrol.wait;" ::: "memory");

  Walk walk(p, starts, cta);
  Segment sg;
  if (warp == kLoadWarp) {
    if (lane == 0) {
      uint32_t qn = 0, kn = 0;       // Q steps and K buffers issued
      bool ok = true;
      const uint32_t q_bytes = static_cast<uint32_t>(G::kChunks * 128 * p.g * p.nr);
      while (ok && walk.next(sg)) {
        const uint32_t kb = kn & 1;
        if (kn >= 2 && !spin_wait(smem_addr(&ctl.k_empty[kb]), ((kn >> 1) - 1) & 1, ctl, p)) {
          ok = false;
          break;
        }
        const int tiles = sg.key0 + kKeys < p.Lk ? 2 : 1;
        const uint32_t kbar = smem_addr(&ctl.k_full[kb]);
        mbar_arrive_expect_tx(kbar, tiles * G::kTileBytes);
        for (int w = 0; w < tiles; ++w)
          for (int ch = 0; ch < G::kChunks; ++ch)
            tma_load_4d(sK + (2 * kb + w) * G::kTileBytes + ch * G::kChunkBytes, &tmK, kbar, ch * 64,
                        sg.kvh, sg.key0 + w * kKeys, sg.b);
        ++kn;
        for (int i = 0; i < sg.n; ++i, ++qn) {
          const uint32_t slot = qn % G::kQStages, use = qn / G::kQStages;
          if (use > 0 && !spin_wait(smem_addr(&ctl.q_empty[slot]), (use - 1) & 1, ctl, p)) {
            ok = false;
            break;
          }
          const uint32_t bar = smem_addr(&ctl.q_full[slot]);
          mbar_arrive_expect_tx(bar, q_bytes);
          for (int ch = 0; ch < G::kChunks; ++ch)
            tma_load_4d(sQ + slot * G::kTileBytes + ch * G::kChunkBytes, &tmQ, bar, ch * 64,
                        sg.kvh * p.g, (sg.s0 + i) * p.nr, sg.b);
        }
      }
      if (!ok) {
        // let every copy this thread started land before the CTA can exit
        for (uint32_t s = 0; s < 2 && s < kn; ++s)
          drain_wait(smem_addr(&ctl.k_full[s]), ((s + ((kn - 1 - s) / 2) * 2) >> 1) & 1, p);
        for (uint32_t s = 0; s < G::kQStages && s < qn; ++s)
          drain_wait(smem_addr(&ctl.q_full[s]), ((qn - 1 - s) / G::kQStages) & 1, p);
      }
    }
  } else if (warp == kMmaWarp) {
    const bool leader = elect_one();
    constexpr uint32_t idesc = idesc_bf16_f32(kKeys, kCols, false);
    uint32_t qn = 0, kn = 0, sn[2] = {0, 0};
    bool ok = true;
    while (ok && walk.next(sg)) {
      const uint32_t kb = kn & 1;
      if (!wait_warp(smem_addr(&ctl.k_full[kb]), (kn >> 1) & 1, ctl, p)) break;
      ++kn;
      for (int i = 0; i < sg.n && ok; ++i, ++qn) {
        const uint32_t slot = qn % G::kQStages;
        if (!wait_warp(smem_addr(&ctl.q_full[slot]), (qn / G::kQStages) & 1, ctl, p)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (!takes_part(p, sg.key0 + w * kKeys, sg.s0 + i)) continue;
          const uint32_t sb = sn[w] & 1;
          if (sn[w] >= 2 &&
              !wait_warp(smem_addr(&ctl.s_free[w][sb]), ((sn[w] >> 1) - 1) & 1, ctl, p)) {
            ok = false;
            break;
          }
          ++sn[w];
          tc_fence_after_sync();
          const uint64_t a0 = sdesc_sw128(sK + (2 * kb + w) * G::kTileBytes, 16, 1024);
          const uint64_t b0 = sdesc_sw128(sQ + slot * G::kTileBytes, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * G::kChunkBytes + (kk & 3) * 32) >> 4;
            if (leader)
              mma_ss(tmem + 256 * w + 128 * sb, a0 + off, b0 + off, idesc, kk > 0 ? 1u : 0u);
          }
          if (leader) mma_commit(smem_addr(&ctl.s_full[w][sb]));
        }
        if (!ok) break;
        if (leader) mma_commit(smem_addr(&ctl.q_empty[slot]));
      }
      if (leader && ok) mma_commit(smem_addr(&ctl.k_empty[kb]));
    }
    // no MMA may still be running when TMEM is released
    if (leader) mma_commit(smem_addr(&ctl.drain));
    drain_wait(smem_addr(&ctl.drain), 0, p);
    __syncwarp();
  } else if (warp == kLseWarp) {
    // lane's columns lane + 32 m: row col / g of the step, head col % g
    int row[4], head[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int col = lane + 32 * m;
      row[m] = col < p.nr * p.g ? col / p.g : p.Lq;      // past the last row: no weight
      head[m] = col % p.g;
    }
    uint32_t n = 0;
    bool ok = true;
    while (ok && walk.next(sg)) {
      const float* lse = p.lse + (static_cast<size_t>(sg.b) * p.n_q + sg.kvh * p.g) * p.Lq;
      for (int i = 0; i < sg.n; ++i, ++n) {
        const int i0 = (sg.s0 + i) * p.nr;
        float nl[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          nl[m] = -INFINITY;
          if (row[m] < p.Lq - i0) {
            const float l = lse[static_cast<size_t>(head[m]) * p.Lq + i0 + row[m]];
            if (l != -INFINITY) nl[m] = -l * kLog2e;     // a row without keys has no weight
          }
        }
        const uint32_t slot = n & 1;
        if (n >= 2 && !wait_warp(smem_addr(&ctl.l_empty[slot]), ((n >> 1) - 1) & 1, ctl, p)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) nl_ring[slot * kCols + lane + 32 * m] = nl[m];
        mbar_arrive(smem_addr(&ctl.l_full[slot]));
      }
    }
  } else if (warp < 8) {
    const int w = warp >> 2;
    const int r = (warp & 3) * 32 + lane;                // key of the tile = TMEM lane
    const uint32_t taddr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 256 * w;
    const uint64_t c2 = f32x2_pack(p.c, p.c);
    uint32_t n = 0, sn = 0;
    bool ok = true;
    while (ok && walk.next(sg)) {
      const int key = sg.key0 + w * kKeys + r;
      // the running sum with its rounding error carried along: a key of a long
      // prompt adds thousands of steps
      float sum = 0.0f, carry = 0.0f;
      for (int i = 0; i < sg.n; ++i, ++n) {
        const uint32_t slot = n & 1;
        if (!wait_warp(smem_addr(&ctl.l_full[slot]), (n >> 1) & 1, ctl, p)) {
          ok = false;
          break;
        }
        if (takes_part(p, sg.key0 + w * kKeys, sg.s0 + i)) {
          const uint32_t sb = sn & 1;
          if (!wait_warp(smem_addr(&ctl.s_full[w][sb]), (sn >> 1) & 1, ctl, p)) {
            ok = false;
            break;
          }
          ++sn;
          tc_fence_after_sync();
          float s[kCols];
          uint32_t* sr = reinterpret_cast<uint32_t*>(s);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            tmem_ld32(taddr + 128 * sb + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(sr + 32 * q));
          tmem_wait_ld(*reinterpret_cast<uint32_t(*)[32]>(sr));
          tmem_after_wait(*reinterpret_cast<uint32_t(*)[32]>(sr + 32));
          tmem_after_wait(*reinterpret_cast<uint32_t(*)[32]>(sr + 64));
          tmem_after_wait(*reinterpret_cast<uint32_t(*)[32]>(sr + 96));
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&ctl.s_free[w][sb]));
          // rows before the key's own position do not see it
          const int i0 = (sg.s0 + i) * p.nr;
          const bool diag = p.causal && sg.key0 + w * kKeys + kKeys - 1 - p.off > i0;
          const float* nl = nl_ring + slot * kCols;
          const float add = diag ? column_sum<true>(s, nl, c2, (key - p.off - i0) * p.g)
                                 : column_sum<false>(s, nl, c2, 0);
          const float y = add - carry, t = sum + y;
          carry = (t - sum) - y;
          sum = t;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&ctl.l_empty[slot]));
      }
      if (!ok) break;
      if (!sg.whole) {
        p.part[(2 * cta + (sg.first ? 0 : 1)) * kUnitKeys + w * kKeys + r] = sum;
      } else if (key < p.Lk) {
        float* out = p.weights + (static_cast<size_t>(sg.b) * p.n_kv + sg.kvh) * p.Lk + key;
        *out = p.accumulate ? *out + sum : sum;
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// CTA c sums the unit that its range starts in the middle of, if the unit
// begins in the range before: that range's last segment, then the first
// segments of ranges c, c + 1, ... up to the unit's end.
__global__ void __launch_bounds__(kUnitKeys)
key_weights_reduce_kernel(const __grid_constant__ Params p, const __grid_constant__ Starts st) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int c = static_cast<int>(blockIdx.x) + 1;
  const int unit = st.unit[c], grp = unit / p.T, t = unit - grp * p.T;
  const int first = first_step(t, p.off, p.nr, p.causal);
  if (st.step[c] == first) return;                                   // a border between units
  if (st.unit[c - 1] == unit && st.step[c - 1] > first) return;      // begins further back
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int key = t * kUnitKeys + static_cast<int>(threadIdx.x);
  if (key >= p.Lk) return;
  const float* part = p.part + threadIdx.x;
  float sum = part[(2 * (c - 1) + (st.unit[c - 1] == unit ? 0 : 1)) * kUnitKeys];
  for (int e = c; e < p.G && st.unit[e] == unit; ++e) sum += part[2 * e * kUnitKeys];
  float* out = p.weights + static_cast<size_t>(grp) * p.Lk + key;
  *out = p.accumulate ? *out + sum : sum;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr int kMaxDevices = 64;
std::mutex g_weights_mutex;
bool g_weights_ready[kMaxDevices] = {};
EncodeTiledFn g_weights_encode = nullptr;

template <int D>
bool set_smem() {
  return cudaFuncSetAttribute(key_weights_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Geometry<D>::kSmemBytes) == cudaSuccess;
}

attn_status_t weights_device_ready(cudaStream_t stream, int** status) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_UNSUPPORTED;
  const attn_status_t ds = gb300_host::device_status_word(stream, status);
  if (ds != ATTN_OK) return ds;
  std::lock_guard<std::mutex> lock(g_weights_mutex);
  if (g_weights_ready[dev]) return ATTN_OK;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess || cs != cudaStreamCaptureStatusNone) {
    cudaGetLastError();
    return ATTN_ERR_UNSUPPORTED;
  }
  if (!g_weights_encode) {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || fn == nullptr)
      return ATTN_ERR_CUDA;
    g_weights_encode = reinterpret_cast<EncodeTiledFn>(fn);
  }
  if (!set_smem<64>() || !set_smem<128>()) return ATTN_ERR_CUDA;
  g_weights_ready[dev] = true;
  return ATTN_OK;
}

// bf16 [B, L, H, D] as (D, H, L, B), boxes of 64 x heads x rows x 1 with
// 128-byte swizzle; rows past L read as zeros.
bool encode(CUtensorMap* map, const void* ptr, int D, int H, int64_t L, int64_t B, int heads,
            int rows) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H),
                              static_cast<cuuint64_t>(L), static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(H) * D * 2,
                                 static_cast<cuuint64_t>(L) * H * D * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(rows), 1};
  const cuuint32_t estride[4] = {1, 1, 1, 1};
  return g_weights_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims,
                          strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// sum_{i=0}^{n-1} floor((a i + b) / m) for n >= 0, m >= 1, a, b >= 0, by
// splitting off whole multiples and exchanging the axes of the lattice points
// below the line (the Euclidean algorithm on a and m).
int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t total = 0;
  while (n > 0) {
    total += n * (n - 1) / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const int64_t top = a * n + b;
    if (top < m) break;
    n = top / m;
    b = top % m;
    const int64_t old = m;
    m = a;
    a = old;
  }
  return total;
}

// Steps of units 0 .. t-1 of one (b, K/V head).
int64_t steps_before(const Params& p, int64_t t) {
  int64_t n = t * p.steps;
  const int64_t s0 = p.off / kUnitKeys + 1;        // first unit that starts past row 0's position
  if (p.causal && t > s0)
    n -= floor_sum(t - s0, p.nr, kUnitKeys, s0 * kUnitKeys - p.off);
  return n;
}

bool supported(int64_t B, int64_t Lq, int64_t Lk, int32_t n_q, int32_t n_kv, int32_t d_h) {
  if ((d_h != 64 && d_h != 128) || n_q / n_kv > kCols) return false;
  constexpr int64_t kMost = int64_t{1} << 30;
  if (Lq > kMost || Lk > kMost || B > kMost || B * n_kv > kMost) return false;
  // units and a CTA's steps are 32-bit; scores in all fit 64 with room
  const int64_t units = B * n_kv * ((Lk + kUnitKeys - 1) / kUnitKeys);
  const int64_t steps = (Lq * (n_q / n_kv) + kCols - 1) / kCols * 2;
  return units <= INT32_MAX - kCtas && steps <= INT64_MAX / units / kCtas &&
         units * steps / kCtas < INT32_MAX / 2 && Lk * (n_q / n_kv) <= INT32_MAX;
}

bool sizes_ok(int64_t B, int64_t Lq, int64_t Lk, int32_t n_q, int32_t n_kv, int32_t d_h) {
  return B >= 1 && Lq >= 1 && Lk >= Lq && n_q >= 1 && n_kv >= 1 && n_q % n_kv == 0 && d_h >= 1;
}

}  // namespace

extern "C" {

int64_t attn_key_weights_workspace_bytes(int64_t B, int64_t Lq, int64_t Lk, int32_t n_q,
                                         int32_t n_kv, int32_t d_h) {
  if (!sizes_ok(B, Lq, Lk, n_q, n_kv, d_h) || !supported(B, Lq, Lk, n_q, n_kv, d_h)) return -1;
  return int64_t{kCtas} * 2 * kUnitKeys * 4;
}

attn_status_t attn_key_weights_fwd(const void* q, const void* k, const float* lse, float* weights,
                                   void* workspace, int64_t workspace_bytes, int64_t B, int64_t Lq,
                                   int64_t Lk, int32_t n_q, int32_t n_kv, int32_t d_h,
                                   int32_t causal, int32_t accumulate, float scale,
                                   void* stream_ptr) {
  if (!q || !k || !lse || !weights || !workspace) return ATTN_ERR_INVALID_ARG;
  if (!sizes_ok(B, Lq, Lk, n_q, n_kv, d_h) || !std::isfinite(scale) ||
      (causal != 0 && causal != 1) || (accumulate != 0 && accumulate != 1))
    return ATTN_ERR_INVALID_ARG;
  auto misaligned = [](const void* ptr, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0;
  };
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(lse, 4) || misaligned(weights, 4) ||
      misaligned(workspace, 16))
    return ATTN_ERR_INVALID_ARG;
  if (!supported(B, Lq, Lk, n_q, n_kv, d_h)) return ATTN_ERR_UNSUPPORTED;
  if (workspace_bytes < attn_key_weights_workspace_bytes(B, Lq, Lk, n_q, n_kv, d_h))
    return ATTN_ERR_INVALID_ARG;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  int* status = nullptr;
  const attn_status_t ds = weights_device_ready(stream, &status);
  if (ds != ATTN_OK) return ds;

  Params p{};
  p.lse = lse;
  p.weights = weights;
  p.part = static_cast<float*>(workspace);
  p.status = status;
  p.Lq = static_cast<int>(Lq);
  p.Lk = static_cast<int>(Lk);
  p.off = static_cast<int>(Lk - Lq);
  p.n_q = n_q;
  p.n_kv = n_kv;
  p.g = n_q / n_kv;
  p.nr = kCols / p.g;
  p.steps = static_cast<int>((Lq + p.nr - 1) / p.nr);
  p.T = static_cast<int>((Lk + kUnitKeys - 1) / kUnitKeys);
  p.causal = causal;
  p.accumulate = accumulate;
  p.c = scale * kLog2e;
  p.spin_limit = 1ll << 31;   // about a second at 2 GHz

  // equal ranges of the steps of all units
  const int64_t per_group = steps_before(p, p.T), W = per_group * B * n_kv;
  p.G = static_cast<int>(W < kCtas ? W : kCtas);
  Starts st;
  bool cut = false;
  for (int c = 0; c < p.G; ++c) {
    const int64_t x = c * W / p.G;
    st.count[c] = static_cast<int>((c + 1) * W / p.G - x);
    const int64_t grp = x / per_group, rest = x - grp * per_group;
    int64_t lo = 0, hi = p.T;                     // the unit that holds step `rest`
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) / 2;
      (steps_before(p, mid) <= rest ? lo : hi) = mid;
    }
    const int first = first_step(static_cast<int>(lo), p.off, p.nr, causal);
    st.unit[c] = static_cast<int>(grp * p.T + lo);
    st.step[c] = first + static_cast<int>(rest - steps_before(p, lo));
    cut |= st.step[c] != first;
  }

  CUtensorMap mq, mk;
  if (!encode(&mq, q, d_h, n_q, Lq, B, p.g, p.nr) || !encode(&mk, k, d_h, n_kv, Lk, B, 1, kKeys))
    return ATTN_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.G));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (d_h == 128) {
    cfg.dynamicSmemBytes = Geometry<128>::kSmemBytes;
    e = cudaLaunchKernelEx(&cfg, key_weights_kernel<128>, mq, mk, p, st);
  } else {
    cfg.dynamicSmemBytes = Geometry<64>::kSmemBytes;
    e = cudaLaunchKernelEx(&cfg, key_weights_kernel<64>, mq, mk, p, st);
  }
  if (e != cudaSuccess) return ATTN_ERR_CUDA;
  if (cut) {
    cfg.gridDim = dim3(static_cast<unsigned>(p.G - 1));
    cfg.blockDim = dim3(kUnitKeys);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, key_weights_reduce_kernel, p, st) != cudaSuccess)
      return ATTN_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
