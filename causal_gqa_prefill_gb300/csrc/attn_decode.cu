// attn_decode.cu — decode attention (one new query token per sequence) for
// GB300 (sm_103a), split over the key range.
//
// Decode attends one query row per head to the whole K/V cache; its work per
// byte is the GQA group size g, so it is bound by HBM bandwidth, not by the
// tensor cores ("Long-Context Attention Explained" (sevydevy), prefill vs
// decode: each decode step reads the whole KV cache; "Memory-bound vs
// compute-bound" lesson (Pranay), "Attention itself": decode attention is a
// batched matrix-vector product whose time is cache size over bandwidth).
// So the kernel is built to stream K and V once at the copy rate, and it
// hands both products to the tensor cores only to keep the SM's issue slots
// free for that stream:
//
//   split kernel  persistent, one CTA per SM. The B * n_kv * T key tiles
//                 (T = ceil(Lk / 128) per K/V head) are cut into equal
//                 contiguous ranges, one per CTA; a range that crosses a head
//                 boundary becomes one segment per head. Per segment the CTA
//                 streams its K and V tiles through a 6-stage TMA ring and
//                 computes, with the keys on the TMEM lanes and the g <= 16
//                 query heads of the group as the N = 16 columns,
//                   S^T = K Q^T          (tcgen05, both operands in smem)
//                   O^T += V^T P^T       (tcgen05, V used MN-major)
//                 with an online softmax over the key lanes in between (one
//                 thread per key; the running maximum moves lazily, so the
//                 cross-thread maximum is only taken when a score exceeds it
//                 by the threshold). It writes the segment's normalised partial
//                 output and log-sum-exp to the workspace (the ragged step: its
//                 maximum, sum and undivided output). Both the scores
//                 of the next tile and the output of the segment before run
//                 across segment borders (two O^T accumulators), so many short
//                 segments go at the pace of one long one.
//   combine       one CTA per (b, query head) merges the head's segments
//                 through their log-sum-exps into bf16 O and fp32 LSE.
//
// The ragged step (caches of lens[b] positions in tensors of capacity C) is
// the same split kernel over n_kv * sum_b ceil(lens[b] / 128) key tiles. The
// lengths live on the device, so each CTA finds its range itself from their
// prefix sums; a segment's partial results go to row hd + cta (head and CTA
// both only grow along the walk, so no two segments share a row), and the
// segments that hold a head's first and last tile note their CTAs for the
// combine. Rows of K and V past a sequence's length may hold anything: their
// scores are masked, and V rows that the tensor cores would multiply by zero
// weights are overwritten with zeros in shared memory (0 * NaN is NaN).
// With weights, the split kernel also writes the scores (4 g bytes per
// position and K/V head beside the 512 of K and V), and CTAs of the combine
// turn them into softmax weights once the row's log-sum-exp is known, summed
// over the group's heads. Measured: 16 sequences of 1024 to 8192 positions, 32
// heads on 8, with weights 60 us (302 MB of K and V; split 56, combine 8 when
// timed one by one), one of 131072, 36 heads on 6, 67 us (403 MB, 6.0 TB/s): the
// stream of K and V bounds both, and the combine's latency is what is left.
//
// Behind a sliding window with sinks (kWindow: the new token sees the last W of
// lens[b] positions and the first S) the ragged step's tiles are those of the
// visible positions only: the sinks' from position 0 on, then the window's from its
// own first position on (a TMA box may start at any row), so a window of W costs
// ceil(W / 128) tiles wherever it lies. A few sinks come through maps with boxes of as
// few rows (64 steps with 4 sinks read 255 MB, 284 with whole boxes: 47 and 51 us). Hidden
// positions that share a tile with
// visible ones are masked and zeroed like those past a length.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "attn_prefill.h"
#include "decode_parts.h"
#include "sm103_ptx.cuh"

namespace gb300_host {
attn_status_t device_status_word(cudaStream_t stream, int** status);
}

namespace {

using namespace gb300;

constexpr int kDim = 128;            // head dimension handled here
constexpr int kKeys = 128;           // keys per tile (= TMEM lanes of S^T)
constexpr int kHeadsPad = 16;        // N of both products: the group's heads, padded
constexpr int kMaxG = 16;            // query heads per K/V head
constexpr int kRing = 6;             // K/V ring slots (K and V tiles alternate)
constexpr int kQBufs = 4;            // Q tiles: the ring may hold the K/V of three one-tile segments
constexpr int kTileBytes = kKeys * kDim * 2;          // 32 KiB: two 128 x 64 swizzled chunks
constexpr int kChunkBytes = kKeys * 128;              // 16 KiB
constexpr int kQBytes = kHeadsPad * kDim * 2;         // 4 KiB: two 16 x 64 chunks
constexpr int kPBytes = kHeadsPad * kKeys * 2;        // 4 KiB: P as 16 heads x 128 keys
constexpr int kSmallChunk = kHeadsPad * 128;          // 2 KiB: one 16-row swizzled chunk
constexpr int kSmemBytes = kRing * kTileBytes + kQBufs * kQBytes + 2 * kPBytes + 1024;
constexpr int kDecodeCtas = 152;     // one CTA per SM on a 152-SM GB300
constexpr int kThreads = 192;        // warps 0-3 softmax, 4 TMA producer, 5 MMA issuer
constexpr int kLoadWarp = 4, kMmaWarp = 5;
constexpr uint32_t kTmemCols = 64;
constexpr uint32_t kColS = 0;        // S^T buffers at columns 0 and 16
constexpr uint32_t kColO = 32;       // O^T accumulators at columns 32 and 48
constexpr float kRescale = 8.0f;     // lazy running-max threshold (log2 units)
constexpr int kStatusTimeout = 1;

struct DecodeParams {
  float* part_o;         // fp32 [G * P_max * g, 128] normalised partial outputs
  float* part_lse;       // fp32 [G * P_max * g] partial log-sum-exp (natural log)
  float2* part_ml;       // ragged step instead: running maximum (log2 units) and sum,
                         // part_o not normalised
  int* status;           // per-device status word (timeouts)
  int Lk, n_q, n_kv, g;
  int T;                 // key tiles per K/V head
  long long W;           // B * n_kv * T
  int G, P_max;          // CTAs and segment slots per CTA
  float c;               // scale * log2(e)
  long long spin_limit;
  // ragged step only (Lk is the capacity C there, T and W are its bounds)
  const int* lens;       // [B] cached positions
  int* ends;             // [B * n_kv][2] CTAs that hold a head's first and last tile
  float* scores;         // with weights: fp32 [B * n_q, ld] scores * scale * log2(e)
  long long ld;
  int B;
  int window, sinks;     // kWindow: W and S
  int beside;            // 1: wait for the kernel before only at the end (decode_parts.h)
};

struct DecodeCtl {
  uint64_t full[kRing], empty[kRing];
  uint64_t q_full[kQBufs], q_empty[kQBufs];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t o_done[2], o_free[2], drain;
  uint32_t tmem_base;
  int abort;
  float4 red_m[kHeadsPad];      // per head, one value per softmax warp
  float4 red_l[kHeadsPad];
  int start_b, start_u, start_t;    // ragged step: where this CTA's range starts
  long long tiles;                  // and how many tiles it has
};

// First global tile of CTA c's range, and the CTA whose range holds tile x.
__host__ __device__ __forceinline__ long long range_start(long long c, long long W, long long G) {
  return c * W / G;
}
__host__ __device__ __forceinline__ long long cta_of(long long x, long long W, long long G) {
  return ((x + 1) * G - 1) / W;
}

// Segment slots per CTA: a range of at most ceil(W / G) tiles touches at most
// this many heads.
long long segment_slots(long long W, long long G, long long T) {
  return ((W + G - 1) / G - 1) / T + 2;
}

__device__ __forceinline__ bool spin_wait(uint32_t bar, uint32_t parity, DecodeCtl& ctl,
                                          const DecodeParams& p) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = clock64_now();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&ctl.abort)) return false;
    if (static_cast<long long>(clock64_now() - t0) > p.spin_limit) {
      *reinterpret_cast<volatile int*>(&ctl.abort) = 1;
      if (p.status) atomicOr(p.status, kStatusTimeout);
      return false;
    }
  }
}

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, DecodeCtl& ctl,
                                          const DecodeParams& p) {
  return __all_sync(0xffffffffu, spin_wait(bar, parity, ctl, p));
}

// Wait used while draining after an abort: ignores the abort flag.
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, const DecodeParams& p) {
  const uint64_t t0 = clock64_now();
  while (!mbar_try_wait(bar, parity))
    if (static_cast<long long>(clock64_now() - t0) > p.spin_limit) return;
}

// Named barrier 1 over the 128 softmax threads; the OR of `v` over them.
__device__ __forceinline__ void bar_softmax() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool bar_softmax_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.or.pred po, 1, 128, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}

// Reduces GP per-head values over the warp: log2(GP) steps that each halve
// the heads a lane carries (it keeps one half and sends the other), then plain
// steps. Lane l returns the result of head l / (32 / GP): GP + 3 - log2(GP)
// shuffles or so where a butterfly per head takes 5 GP, in the same order.
template <int GP, typename Op>
__device__ __forceinline__ float reduce_heads(const float (&in)[GP], Op op) {
  const int lane = threadIdx.x & 31;
  float v[GP];
#pragma unroll
  for (int h = 0; h < GP; ++h) v[h] = in[h];
  int off = 16;
#pragma unroll
  for (int width = GP / 2; width > 0; width >>= 1, off >>= 1) {
    const bool upper = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < width; ++i) {
      const float send = upper ? v[i] : v[i + width], keep = upper ? v[i + width] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, off));
    }
  }
#pragma unroll
  for (; off > 0; off >>= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], off));
  return v[0];
}

// One segment of a CTA's tile range: K/V head `hd` (= b * n_kv + kv head),
// key tiles [t0, t0 + n) of its `len` keys (`tiles` in all), partial results in
// row `id`.
// kWindow: the first `na` of the tiles hold the positions below `sunk`, the rest
// those from `low` on.
struct Segment {
  int hd, t0, n, len, tiles;
  long long id;
  int low, sunk, na;
};

// Walks CTA c's range segment by segment (every role takes the same walk).
struct SegmentWalk {
  long long x, end, slot;
  int T, Lk;
  __device__ SegmentWalk(const DecodeParams& p, const DecodeCtl&, int c)
      : x(range_start(c, p.W, p.G)), end(range_start(c + 1, p.W, p.G)),
        slot(static_cast<long long>(c) * p.P_max), T(p.T), Lk(p.Lk) {}
  __device__ bool next(Segment& s) {
    if (x >= end) return false;
    const long long hd = x / T, base = hd * T;
    const long long t1 = (end - base < T) ? end - base : T;
    s.hd = static_cast<int>(hd);
    s.t0 = static_cast<int>(x - base);
    s.n = static_cast<int>(t1 - (x - base));
    s.len = Lk;
    s.tiles = T;
    s.id = slot++;
    x = base + t1;
    return true;
  }
};

// A sequence's length as the kernels use it, and its key tiles.
__device__ __forceinline__ int clamp_len(int len, int C) { return min(max(len, 0), C); }
__device__ __forceinline__ int key_tiles(int len) { return (len + kKeys - 1) / kKeys; }

// The positions of a sequence of `len` that its new token sees: [0, sunk) and [low, len).
template <bool kWindow>
struct Seen {
  int low, sunk, na, tiles;
  __device__ Seen(const DecodeParams& p, int len) {
    low = kWindow ? max(0, len - p.window) : 0;
    sunk = kWindow ? min(p.sinks, low) : 0;
    na = key_tiles(sunk);
    tiles = na + key_tiles(len - low);
  }
};

// First position of key tile x of a segment's list, and how many of its 128 count.
template <bool kWindow>
__device__ __forceinline__ int tile_pos(const Segment& s, int x) {
  return !kWindow || x < s.na ? x * kKeys : s.low + (x - s.na) * kKeys;
}
template <bool kWindow>
__device__ __forceinline__ int tile_end(const Segment& s, int x) {
  return kWindow && x < s.na ? s.sunk : s.len;
}

// Where CTA c's range starts, by one warp: each lane sums the tiles of a run
// of sequences, a warp scan places the runs, and the lane whose run holds the
// first tile walks it.
template <bool kWindow>
__device__ __forceinline__ void ragged_start(const DecodeParams& p, DecodeCtl& ctl, int c) {
  const int lane = threadIdx.x & 31;
  const int run = (p.B + 31) / 32, b0 = min(lane * run, p.B), b1 = min(b0 + run, p.B);
  long long sum = 0;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) sum += Seen<kWindow>(p, clamp_len(p.lens[b], p.Lk)).tiles;
  sum *= p.n_kv;
  long long incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long n = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += n;
  }
  const long long W = __shfl_sync(0xffffffffu, incl, 31);
  const long long G = min(static_cast<long long>(p.G), W);   // every range has a tile
  if (c >= G) {
    if (lane == 0) ctl.tiles = 0;
    return;
  }
  const long long x0 = range_start(c, W, G);
  long long at = incl - sum;
  if (x0 < at || x0 >= incl) return;
  for (int b = b0; b < b1; ++b) {
    const int T = Seen<kWindow>(p, clamp_len(p.lens[b], p.Lk)).tiles;
    const long long here = static_cast<long long>(T) * p.n_kv;
    if (x0 < at + here) {
      const int off = static_cast<int>(x0 - at);
      ctl.start_b = b;
      ctl.start_u = off / T;
      ctl.start_t = off - (off / T) * T;
      ctl.tiles = range_start(c + 1, W, G) - x0;
      return;
    }
    at += here;
  }
}

// The same walk over the ragged step's tiles, from the start that
// ragged_start left in `ctl`.
template <bool kWindow>
struct RaggedWalk {
  const DecodeParams& p;
  long long left;
  int cta, b, u, t, len, T, low, sunk, na;
  __device__ RaggedWalk(const DecodeParams& params, const DecodeCtl& ctl, int c)
      : p(params), left(ctl.tiles), cta(c), b(ctl.start_b), u(ctl.start_u), t(ctl.start_t) {
    if (left > 0) sequence();
  }
  __device__ void sequence() {
    len = clamp_len(p.lens[b], p.Lk);
    const Seen<kWindow> seen(p, len);
    T = seen.tiles;
    low = seen.low;
    sunk = seen.sunk;
    na = seen.na;
  }
  __device__ bool next(Segment& s) {
    if (left <= 0) return false;
    while (T == 0) {
      if (++b >= p.B) return false;
      sequence();
    }
    s.hd = b * p.n_kv + u;
    s.t0 = t;
    s.n = static_cast<int>(left < T - t ? left : T - t);
    s.len = len;
    s.tiles = T;
    s.low = low;
    s.sunk = sunk;
    s.na = na;
    s.id = static_cast<long long>(s.hd) + cta;
    left -= s.n;
    t += s.n;
    if (t == T) {
      t = 0;
      if (++u == p.n_kv) {
        u = 0;
        if (++b >= p.B) left = 0;
        else if (left > 0) sequence();
      }
    }
    return true;
  }
};

// kWindow: K and V in boxes of `rows` rows (a multiple of 8) for the sinks, where they are
// fewer than a tile.
template <bool kWindow>
struct SinkMaps {};
template <>
struct SinkMaps<true> {
  CUtensorMap k, v;
  int rows;
};

template <bool kRagged, bool kWindow>
struct WalkOf {
  using type = SegmentWalk;
};
template <bool kWindow>
struct WalkOf<true, kWindow> {
  using type = RaggedWalk<kWindow>;
};

// GP: the group's query heads padded to 4, 8 or 16 (g <= GP); the loops over
// heads unroll to GP and skip h >= g. kRagged: the ragged step; kWeights: it
// also writes the scores; kWindow: behind a window with sinks.
template <int GP, bool kRagged, bool kWeights, bool kWindow = false>
__global__ void __launch_bounds__(kThreads, 1)
attn_decode_split_kernel(const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const DecodeParams p,
                         const __grid_constant__ SinkMaps<kWindow> sinks) {
  extern __shared__ uint8_t dyn_smem[];
  __shared__ DecodeCtl ctl;
  // smem: kRing K/V tiles | Q[kQBufs] (16 heads x 128, two 2 KiB chunks) | P[2]
  const uint32_t base = (smem_addr(dyn_smem) + 1023u) & ~1023u;   // swizzle atoms need 1 KiB
  const uint32_t sRing = base, sQ = base + kRing * kTileBytes, sP = sQ + kQBufs * kQBytes;
  uint8_t* const pgen = dyn_smem + (sP - smem_addr(dyn_smem));      // generic address of P[0]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = static_cast<int>(blockIdx.x);
  // The combine kernel (launched as this grid's programmatic dependent) may
  // start now; it waits for this grid to complete before reading anything.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(smem_addr(&ctl.full[s]), 1);
      mbar_init(smem_addr(&ctl.empty[s]), 1);
    }
    for (int s = 0; s < kQBufs; ++s) {
      mbar_init(smem_addr(&ctl.q_full[s]), 1);
      mbar_init(smem_addr(&ctl.q_empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_addr(&ctl.s_full[s]), 1);
      mbar_init(smem_addr(&ctl.p_full[s]), 128);
      mbar_init(smem_addr(&ctl.pv_done[s]), 1);
      mbar_init(smem_addr(&ctl.o_done[s]), 1);
      mbar_init(smem_addr(&ctl.o_free[s]), 128);
    }
    mbar_init(smem_addr(&ctl.drain), 1);
    ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&ctl.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (warp < 4) {
    // P rows g..15 are never written again: they stay zero, so the padded
    // columns of O^T stay zero.
    uint4* pz = reinterpret_cast<uint4*>(pgen);
    for (int i = threadIdx.x; i < 2 * kPBytes / 16; i += 128) pz[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = ctl.tmem_base;
  // Launched as the programmatic dependent of the stream's previous kernel
  // (the previous call's combine, or whatever wrote Q, K and V): the set-up
  // above overlaps it; global memory is touched only after it has completed.
  if (!kRagged || !p.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
  using Walk = typename WalkOf<kRagged, kWindow>::type;
  if (kRagged) {
    if (warp == 0) ragged_start<kWindow>(p, ctl, cta);
    __syncthreads();
  }

  if (warp == kLoadWarp) {
    if (lane == 0) {
      Walk walk(p, ctl, cta);
      Segment sg;
      uint32_t it = 0;   // ring items issued (K_t and V_t alternate)
      uint32_t qn = 0;   // Q tiles issued (one per segment)
      bool ok = true;
      while (ok && walk.next(sg)) {
        const int b = sg.hd / p.n_kv, kvh = sg.hd - b * p.n_kv;
        const uint32_t qb = qn % kQBufs;
        if (qn >= kQBufs &&
            !spin_wait(smem_addr(&ctl.q_empty[qb]), (qn / kQBufs - 1) & 1, ctl, p)) {
          ok = false;
          break;
        }
        const uint32_t qbar = smem_addr(&ctl.q_full[qb]);
        mbar_arrive_expect_tx(qbar, kQBytes);
        // rows kvh*g .. kvh*g + 15: the group's heads first (rows past n_q read as zero)
        for (int ch = 0; ch < 2; ++ch)
          tma_load_3d(sQ + qb * kQBytes + ch * kSmallChunk, &tmQ, qbar, ch * 64, kvh * p.g, b);
        ++qn;
        for (int t = 0; t < sg.n && ok; ++t) {
          for (int kind = 0; kind < 2; ++kind) {
            const uint32_t slot = it % kRing, use = it / kRing;
            if (use > 0 && !spin_wait(smem_addr(&ctl.empty[slot]), (use - 1) & 1, ctl, p)) {
              ok = false;
              break;
            }
            const uint32_t bar = smem_addr(&ctl.full[slot]);
            if constexpr (kWindow) {
              // (rows of the slot past the box keep what they held: they do not count, and
              // are masked and zeroed as such)
              if (sg.t0 + t < sg.na && sinks.rows < kKeys) {
                mbar_arrive_expect_tx(bar, 2 * 128 * sinks.rows);
                for (int ch = 0; ch < 2; ++ch)
                  tma_load_4d(sRing + slot * kTileBytes + ch * kChunkBytes,
                              kind ? &sinks.v : &sinks.k, bar, ch * 64, kvh, 0, b);
                ++it;
                continue;
              }
            }
            mbar_arrive_expect_tx(bar, kTileBytes);
            for (int ch = 0; ch < 2; ++ch)
              tma_load_4d(sRing + slot * kTileBytes + ch * kChunkBytes, kind ? &tmV : &tmK, bar,
                          ch * 64, kvh, tile_pos<kWindow>(sg, sg.t0 + t), b);
            ++it;
          }
        }
      }
      // Let every copy this thread started land before the CTA can exit, also
      // where another role has given up.
      for (uint32_t s = 0; s < kQBufs && s < qn; ++s)
        drain_wait(smem_addr(&ctl.q_full[s]), ((qn - 1 - s) / kQBufs) & 1, p);
      for (uint32_t s = 0; s < kRing && s < it; ++s) {
        const uint32_t last = s + ((it - 1 - s) / kRing) * kRing;
        drain_wait(smem_addr(&ctl.full[s]), (last / kRing) & 1, p);
      }
    }
  } else if (warp == kMmaWarp) {
    // The whole warp runs the loop (warp-uniform control flow); one elected
    // lane issues every tcgen05 instruction and commit.
    const bool leader = elect_one();
    // S^T = K Q^T: M = 128 keys, N = 16 heads, both K-major (K = head dim).
    constexpr uint32_t kIdS = idesc_bf16_f32(kKeys, kHeadsPad, false);
    // O^T = V^T P^T: M = 128 dims with V read MN-major (bit 15), B = P K-major.
    constexpr uint32_t kIdO = idesc_bf16_f32(kDim, kHeadsPad, false) | (1u << 15);
    // Two cursors over the CTA's tiles: the products of tile gt are issued in
    // two parts, S^T one tile ahead (also over a segment's end, so that short
    // segments keep the same pace) and O^T once the softmax has written P.
    // Tile gt is ring items 2 gt (K) and 2 gt + 1 (V).
    struct Cursor {
      Walk walk;
      Segment sg;
      int t;
      uint32_t sn;       // segment number
      bool live;
      __device__ explicit Cursor(const Walk& w) : walk(w), t(0), sn(0) { live = walk.next(sg); }
      __device__ void advance() {
        if (++t < sg.n) return;
        t = 0;
        ++sn;
        live = walk.next(sg);
      }
    };
    Cursor ahead(Walk(p, ctl, cta));
    Cursor cur = ahead;
    auto wait_item = [&](uint32_t item) {
      const bool r = wait_warp(smem_addr(&ctl.full[item % kRing]), (item / kRing) & 1, ctl, p);
      tc_fence_after_sync();
      return r;
    };
    // S^T of the tile `ahead` is at (tile number gt); false: a wait gave up
    auto issue_s = [&](uint32_t gt) {
      const uint32_t qb = ahead.sn % kQBufs;
      if (ahead.t == 0 && !wait_warp(smem_addr(&ctl.q_full[qb]), (ahead.sn / kQBufs) & 1, ctl, p))
        return false;
      const uint32_t kitem = 2 * gt;
      if (!wait_item(kitem)) return false;
      const uint32_t k_smem = sRing + (kitem % kRing) * kTileBytes, q_smem = sQ + qb * kQBytes;
#pragma unroll
      for (int kk = 0; kk < kDim / 16; ++kk) {
        const uint64_t a = sdesc_sw128(k_smem + (kk >> 2) * kChunkBytes + (kk & 3) * 32, 16, 1024);
        const uint64_t bq = sdesc_sw128(q_smem + (kk >> 2) * kSmallChunk + (kk & 3) * 32, 16, 1024);
        if (leader) mma_ss(tmem + kColS + 16 * (gt & 1), a, bq, kIdS, kk > 0 ? 1u : 0u);
      }
      if (leader) mma_commit(smem_addr(&ctl.s_full[gt & 1]));
      if (leader) mma_commit(smem_addr(&ctl.empty[kitem % kRing]));
      if (ahead.t == ahead.sg.n - 1 && leader) mma_commit(smem_addr(&ctl.q_empty[qb]));
      ahead.advance();
      return true;
    };
    bool ok = !ahead.live || issue_s(0);
    for (uint32_t gt = 0; ok && cur.live; ++gt) {
      // scores of the next tile run while the softmax works on this one
      if (ahead.live && !issue_s(gt + 1)) break;
      // O^T of two segments ago must have been read out first
      const uint32_t ob = cur.sn & 1;
      if (cur.t == 0 && cur.sn >= 2 &&
          !wait_warp(smem_addr(&ctl.o_free[ob]), ((cur.sn >> 1) - 1) & 1, ctl, p))
        break;
      const uint32_t vitem = 2 * gt + 1;
      if (!wait_warp(smem_addr(&ctl.p_full[gt & 1]), (gt >> 1) & 1, ctl, p) || !wait_item(vitem))
        break;
      const uint32_t v_smem = sRing + (vitem % kRing) * kTileBytes;
      const uint32_t p_smem = sP + (gt & 1) * kPBytes;
#pragma unroll
      for (int kk = 0; kk < kKeys / 16; ++kk) {
        // V^T: a K step of 16 keys spans 16 rows (2 KiB); the two 64-dim
        // chunks are kChunkBytes apart. P: 32 bytes per K step.
        const uint64_t a = sdesc_sw128(v_smem + kk * 16 * 128, kChunkBytes, 1024);
        const uint64_t bp = sdesc_sw128(p_smem + (kk >> 2) * kSmallChunk + (kk & 3) * 32, 16, 1024);
        if (leader) mma_ss(tmem + kColO + 16 * ob, a, bp, kIdO, (cur.t > 0 || kk > 0) ? 1u : 0u);
      }
      if (leader) mma_commit(smem_addr(&ctl.pv_done[gt & 1]));
      if (leader) mma_commit(smem_addr(&ctl.empty[vitem % kRing]));
      if (cur.t == cur.sg.n - 1 && leader) mma_commit(smem_addr(&ctl.o_done[ob]));
      cur.advance();
    }
    // No MMA may still be running when TMEM is released.
    if (leader) mma_commit(smem_addr(&ctl.drain));
    drain_wait(smem_addr(&ctl.drain), 0, p);
    __syncwarp();
  } else if (warp < 4) {
    // softmax warps: thread r is key r of a tile (S^T lane) and dimension r
    // of the output (O^T lane)
    const int r = threadIdx.x;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    // where key r of a tile goes in a P buffer: 128-byte swizzled rows of 64
    // keys, chunk r / 64, 16-byte unit (r % 64) / 8 XOR (head % 8)
    const int p_chunk = (r >> 6) * kSmallChunk, p_unit = (r & 63) >> 3, p_byte = (r & 7) * 2;
    Walk walk(p, ctl, cta);
    Segment sg;
    uint32_t gt = 0, sn = 0;
    bool ok = true;
    // Every wait of these four warps ends in a vote over all 128 threads, so
    // they leave together when one of them gives up and none is left alone
    // at a named barrier.
    auto waited = [&](uint32_t bar, uint32_t parity) {
      const bool fail = bar_softmax_any(!spin_wait(bar, parity, ctl, p));
      tc_fence_after_sync();
      return !fail;
    };
    float m_run[GP], l_thr[GP];
    // The segment before, finished but for its output: its product is still
    // running when its last P is written, so its output waits until this
    // segment's first P is under way.
    Segment old{};
    float m_old[GP], l_old[GP];
    bool pending = false;
    // O^T / l and the log-sum-exp of segment number `num`
    auto finish = [&](uint32_t num) {
      if (!waited(smem_addr(&ctl.o_done[num & 1]), (num >> 1) & 1)) return false;
      uint32_t ov[16];
      tmem_ld16(lane_base + kColO + 16 * (num & 1), ov);
      tmem_wait_ld16(ov);
      tc_fence_before_sync();
      mbar_arrive(smem_addr(&ctl.o_free[num & 1]));
      const float part = reduce_heads<GP>(l_old, [](float a, float b) { return a + b; });
      if (lane % (32 / GP) == 0)
        reinterpret_cast<float*>(&ctl.red_l[lane / (32 / GP)])[warp] = part;
      bar_softmax();
      const size_t row0 = static_cast<size_t>(old.id) * p.g;
      if (kRagged && r == 0) {
        if (old.t0 == 0) p.ends[2 * old.hd] = cta;
        if (old.t0 + old.n == old.tiles) p.ends[2 * old.hd + 1] = cta;
      }
      if (kRagged) {
        // maximum, sum and output as they are: a division and a logarithm per
        // head would be most of a short segment's time
#pragma unroll
        for (int h = 0; h < GP; ++h)
          if (h < p.g) p.part_o[(row0 + h) * kDim + r] = __uint_as_float(ov[h]);
        if (warp == 0) {
#pragma unroll
          for (int h = 0; h < GP; ++h)
            if (lane == h && h < p.g) {
              const float4 w = ctl.red_l[h];
              p.part_ml[row0 + h] = make_float2(m_old[h], w.x + w.y + w.z + w.w);
            }
        }
      } else {
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          if (h >= p.g) break;
          const float4 w = ctl.red_l[h];
          const float l = w.x + w.y + w.z + w.w;
          p.part_o[(row0 + h) * kDim + r] = __uint_as_float(ov[h]) / l;
          if (r == h) p.part_lse[row0 + h] = (m_old[h] + log2f(l)) * 0.69314718055994530942f;
        }
      }
      return true;
    };
    while (ok && walk.next(sg)) {
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        m_run[h] = -INFINITY;
        l_thr[h] = 0.0f;
      }
      for (int t = 0; t < sg.n; ++t, ++gt) {
        if (!waited(smem_addr(&ctl.s_full[gt & 1]), (gt >> 1) & 1)) {
          ok = false;
          break;
        }
        uint32_t sv[16];
        tmem_ld16(lane_base + kColS + 16 * (gt & 1), sv);
        tmem_wait_ld16(sv);
        const int key0 = tile_pos<kWindow>(sg, sg.t0 + t), end = tile_end<kWindow>(sg, sg.t0 + t);
        const int key = key0 + r;
        const bool valid = key < end;
        float x[GP];
        bool need = false;
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          x[h] = valid ? __uint_as_float(sv[h]) * p.c : -INFINITY;
          if (h < p.g) need |= x[h] > m_run[h] + kRescale;
        }
        if (kWeights && valid) {
          float* sc = p.scores + static_cast<size_t>(sg.hd) * p.g * p.ld + key;
#pragma unroll
          for (int h = 0; h < GP; ++h)
            if (h < p.g) sc[h * p.ld] = x[h];
        }
        if (bar_softmax_any(need)) {
          // exact maximum of this tile per head, then move the running maxima
          const float top = reduce_heads<GP>(x, [](float a, float b) { return fmaxf(a, b); });
          if (lane % (32 / GP) == 0)
            reinterpret_cast<float*>(&ctl.red_m[lane / (32 / GP)])[warp] = top;
          bar_softmax();
          // (heads past the group's are computed along: no branch keeps one
          // head's chain from running beside the others')
          float alpha[GP];
          bool scaled = false;
#pragma unroll
          for (int h = 0; h < GP; ++h) {
            const float4 w = ctl.red_m[h];
            const float mn = fmaxf(m_run[h], fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w)));
            const bool moved = mn != m_run[h];
            alpha[h] = !moved ? 1.0f : (m_run[h] == -INFINITY) ? 0.0f : ex2_approx(m_run[h] - mn);
            scaled |= moved;
            m_run[h] = mn;
            l_thr[h] *= alpha[h];
          }
          if (t > 0 && scaled) {
            // rescale O^T once the previous tile's product has landed
            const uint32_t pg = gt - 1;
            if (!waited(smem_addr(&ctl.pv_done[pg & 1]), (pg >> 1) & 1)) {
              ok = false;
              break;
            }
            uint32_t ov[16];
            tmem_ld16(lane_base + kColO + 16 * (sn & 1), ov);
            tmem_wait_ld16(ov);
#pragma unroll
            for (int h = 0; h < GP; ++h) ov[h] = __float_as_uint(__uint_as_float(ov[h]) * alpha[h]);
            tmem_st16(lane_base + kColO + 16 * (sn & 1), ov);
            tmem_wait_st();
          }
        }
        // P into buffer gt & 1, free once the product of tile gt - 2 is done
        if (gt >= 2 && !waited(smem_addr(&ctl.pv_done[gt & 1]), ((gt >> 1) - 1) & 1)) {
          ok = false;
          break;
        }
        // P is rounded to bf16, as in the prefill: V is bf16 and both operands of a
        // product have one type. Two halves of 8 bits (P and what its rounding
        // leaves) would double the second product and P's stores to take the error
        // of O from 2.4e-3 to the 1.7e-3 of O's own rounding. The row sum keeps the
        // unrounded e, and so do the weights of the ragged step (from the scores).
        uint8_t* pb = pgen + (gt & 1) * kPBytes + p_chunk + p_byte;
#pragma unroll
        for (int h = 0; h < GP; ++h) {
          // (infinite keys can leave a ragged head's tiles without a finite score)
          const float m_use = kRagged && m_run[h] == -INFINITY ? 0.0f : m_run[h];
          const float e = valid ? ex2_approx(x[h] - m_use) : 0.0f;
          l_thr[h] += e;
          if (h < p.g)
            *reinterpret_cast<uint16_t*>(pb + h * 128 + ((p_unit ^ (h & 7)) << 4)) =
                static_cast<uint16_t>(pack_bf16x2(e, 0.0f) & 0xFFFFu);
        }
        if (kRagged && key0 + kKeys > end) {
          // a tile that ends past the sequence (or the sinks): zeros over what V holds there
          // (the tensor cores read V only after this tile's p_full)
          const uint32_t item = 2 * gt + 1, slot = item % kRing;
          if (!waited(smem_addr(&ctl.full[slot]), (item / kRing) & 1)) {
            ok = false;
            break;
          }
          if (!valid) {
            uint4* row = reinterpret_cast<uint4*>(dyn_smem + (sRing - smem_addr(dyn_smem)) +
                                                  slot * kTileBytes + r * 128);
#pragma unroll
            for (int e = 0; e < 8; ++e) {    // eight lanes at a time on all banks
              row[(e + r) & 7] = make_uint4(0u, 0u, 0u, 0u);
              row[((e + r) & 7) + kChunkBytes / 16] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before_sync();
        mbar_arrive(smem_addr(&ctl.p_full[gt & 1]));
        if (t == 0 && pending && !finish(sn - 1)) {
          ok = false;
          break;
        }
      }
      old = sg;
#pragma unroll
      for (int h = 0; h < GP; ++h) {
        m_old[h] = m_run[h];
        l_old[h] = l_thr[h];
      }
      pending = true;
      ++sn;
    }
    if (ok && pending) finish(sn - 1);
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (kRagged && p.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// One CTA of kCombineWarps warps per (b, query head): O = sum_s w_s O_s,
// w_s = exp(lse_s - LSE) over the head's segments (the CTAs whose tile ranges
// cover its K/V head). One pass: the warps take interleaved segments and merge
// them against a running maximum, each lane four dimensions; the warps' states
// are merged in shared memory.
constexpr int kCombineWarps = 8;

__global__ void __launch_bounds__(32 * kCombineWarps)
attn_decode_combine_kernel(uint16_t* o, float* lse, const DecodeParams p) {
  __shared__ float red_m[kCombineWarps], red_w[kCombineWarps];
  __shared__ float4 red_o[kCombineWarps][32];
  const int row = blockIdx.x;                       // b * n_q + query head
  const int b = row / p.n_q, h = row - b * p.n_q;
  const int r = h % p.g;
  const long long hd = static_cast<long long>(b) * p.n_kv + h / p.g;
  const long long c0 = cta_of(hd * p.T, p.W, p.G);
  const int ns = static_cast<int>(cta_of(hd * p.T + p.T - 1, p.W, p.G) - c0 + 1);
  // The head is segment slot `slot0` of CTA c0; every later CTA's range starts
  // inside the head (each range holds at least one tile), so it is their slot 0.
  const long long slot0 = hd - range_start(c0, p.W, p.G) / p.T;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The next kernel in the stream (the next call's split kernel) may launch
  // and set up now; it waits for this grid to complete before touching
  // global memory.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Launched early behind the split kernel: wait until it has completed and
  // its partial results are visible.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float m = -INFINITY, wsum = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int s = warp; s < ns; s += kCombineWarps) {
    const size_t sr = static_cast<size_t>(((c0 + s) * p.P_max + (s == 0 ? slot0 : 0)) * p.g + r);
    const float ls = p.part_lse[sr];
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + sr * kDim + 4 * lane);
    const float mn = fmaxf(m, ls);
    const float a = (m == -INFINITY) ? 0.0f : __expf(m - mn);
    const float w = __expf(ls - mn);
    m = mn;
    wsum = fmaf(wsum, a, w);
    acc.x = fmaf(w, v.x, acc.x * a);
    acc.y = fmaf(w, v.y, acc.y * a);
    acc.z = fmaf(w, v.z, acc.z * a);
    acc.w = fmaf(w, v.w, acc.w * a);
  }
  red_o[warp][lane] = acc;
  if (lane == 0) {
    red_m[warp] = m;
    red_w[warp] = wsum;
  }
  __syncthreads();
  if (warp == 0) {
    float mx = red_m[0];
#pragma unroll
    for (int w = 1; w < kCombineWarps; ++w) mx = fmaxf(mx, red_m[w]);
    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float ws = 0.0f;
#pragma unroll
    for (int w = 0; w < kCombineWarps; ++w) {
      const float a = (red_m[w] == -INFINITY) ? 0.0f : __expf(red_m[w] - mx);
      const float4 u = red_o[w][lane];
      t.x = fmaf(a, u.x, t.x);
      t.y = fmaf(a, u.y, t.y);
      t.z = fmaf(a, u.z, t.z);
      t.w = fmaf(a, u.w, t.w);
      ws = fmaf(a, red_w[w], ws);
    }
    const float inv = 1.0f / ws;
    const uint32_t w0 = pack_bf16x2(t.x * inv, t.y * inv);
    const uint32_t w1 = pack_bf16x2(t.z * inv, t.w * inv);
    *reinterpret_cast<uint2*>(o + static_cast<size_t>(row) * kDim + 4 * lane) = make_uint2(w0, w1);
    if (lane == 0) lse[row] = mx + logf(ws);
  }
}

// The ragged step's combine. The first `merges` CTAs merge the segments of
// eight / kPerRow rows (of one head each), segments hd + first .. hd + last CTA,
// through their maxima m and sums l:
//   O = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s.
// A sequence without a key gets O = 0 and LSE = -inf. With
// weights, `chunks` CTAs per (b, K/V head) follow, one per kWeightKeys positions:
// each rebuilds the log-sum-exps of the group's heads and adds
//   sum_h 2^(score_hj - lse2_h)
// to the weight of position j. The scores of the first four heads are on their
// way while the log-sum-exps are rebuilt.
constexpr int kWeightKeys = 1024;
constexpr int kWeightPer = kWeightKeys / (32 * kCombineWarps);   // positions per thread
constexpr int kWeightAhead = 4;

template <int kPerRow>
__global__ void __launch_bounds__(32 * kCombineWarps)
attn_decode_ragged_combine_kernel(uint16_t* o, float* lse, float* weights, int merges, int chunks,
                                  const DecodeParams p) {
  constexpr int kRows = kCombineWarps / kPerRow;
  __shared__ float red_m[kCombineWarps], red_w[kCombineWarps];
  __shared__ float4 red_o[kCombineWarps][32];
  __shared__ float lse2[kMaxG];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool merge = blockIdx.x < static_cast<unsigned>(merges);
  const long long rest = merge ? 0 : static_cast<long long>(blockIdx.x) - merges;
  const long long row = static_cast<long long>(blockIdx.x) * kRows + warp / kPerRow;   // b * n_q + h
  const bool live = !merge || row < static_cast<long long>(p.B) * p.n_q;
  const long long hd = merge ? (live ? row / p.g : 0) : rest / chunks;
  // (both loads at once: a head without keys has no ends, what is there is not used)
  const int2 ends = reinterpret_cast<const int2*>(p.ends)[hd];
  const int len = clamp_len(p.lens[hd / p.n_kv], p.Lk);
  const long long c0 = len > 0 ? ends.x : 0;
  const int ns = len > 0 ? ends.y - ends.x + 1 : 0;

  if (!merge) {
    const int first = static_cast<int>(rest - hd * chunks) * kWeightKeys, j0 = first + threadIdx.x;
    if (first >= len) return;
    const float* sc = p.scores + hd * p.g * p.ld + j0;
    float* out = weights + hd * p.Lk + j0;
    const int n = len - j0;                       // position e is live while e * 256 < n
    float x[kWeightAhead][kWeightPer], old[kWeightPer];
#pragma unroll
    for (int e = 0; e < kWeightPer; ++e) {
      const int at = e * 32 * kCombineWarps;
#pragma unroll
      for (int h = 0; h < kWeightAhead; ++h)
        x[h][e] = h < p.g && at < n ? sc[h * p.ld + at] : -INFINITY;
      old[e] = at < n ? out[at] : 0.0f;
    }
    for (int h = warp; h < p.g; h += kCombineWarps) {
      // (a lane's first segment stays in registers: there is rarely a second)
      const float2* ml = p.part_ml + (hd + c0) * p.g + h;
      const float2 own = lane < ns ? ml[lane * p.g] : make_float2(-INFINITY, 0.0f);
      float m = own.x;
      for (int s = lane + 32; s < ns; s += 32) m = fmaxf(m, ml[s * p.g].x);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      float w = exp2f(own.x - m) * own.y;
      for (int s = lane + 32; s < ns; s += 32) w += exp2f(ml[s * p.g].x - m) * ml[s * p.g].y;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) w += __shfl_xor_sync(0xffffffffu, w, off);
      if (lane == 0) lse2[h] = m + log2f(w);
    }
    __syncthreads();
    float sum[kWeightPer] = {};
#pragma unroll
    for (int h = 0; h < kWeightAhead; ++h) {
      if (h >= p.g) break;
#pragma unroll
      for (int e = 0; e < kWeightPer; ++e) sum[e] += ex2_approx(x[h][e] - lse2[h]);
    }
#pragma unroll 4
    for (int h = kWeightAhead; h < p.g; ++h) {
#pragma unroll
      for (int e = 0; e < kWeightPer; ++e)
        if (e * 32 * kCombineWarps < n)
          sum[e] += ex2_approx(sc[h * p.ld + e * 32 * kCombineWarps] - lse2[h]);
    }
#pragma unroll
    for (int e = 0; e < kWeightPer; ++e)
      if (e * 32 * kCombineWarps < n) out[e * 32 * kCombineWarps] = old[e] + sum[e];
    return;
  }

  const int r = static_cast<int>(row - hd * p.g), sub = warp % kPerRow;
  float m = -INFINITY, wsum = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (live) {
#pragma unroll 4
    for (int s = sub; s < ns; s += kPerRow) {
      const size_t sr = static_cast<size_t>((hd + c0 + s) * p.g + r);
      const float2 ml = p.part_ml[sr];
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + sr * kDim + 4 * lane);
      const float mn = fmaxf(m, ml.x);
      const float a = (m == -INFINITY) ? 0.0f : exp2f(m - mn);
      const float w = (ml.x == -INFINITY) ? 0.0f : exp2f(ml.x - mn);
      m = mn;
      wsum = fmaf(w, ml.y, wsum * a);
      acc.x = fmaf(w, v.x, acc.x * a);
      acc.y = fmaf(w, v.y, acc.y * a);
      acc.z = fmaf(w, v.z, acc.z * a);
      acc.w = fmaf(w, v.w, acc.w * a);
    }
  }
  if (kPerRow > 1) {
    red_o[warp][lane] = acc;
    if (lane == 0) {
      red_m[warp] = m;
      red_w[warp] = wsum;
    }
    __syncthreads();
    if (sub != 0) return;
    float mx = red_m[warp];
#pragma unroll
    for (int w = 1; w < kPerRow; ++w) mx = fmaxf(mx, red_m[warp + w]);
    acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    wsum = 0.0f;
#pragma unroll
    for (int w = 0; w < kPerRow; ++w) {
      const float a = (red_m[warp + w] == -INFINITY) ? 0.0f : exp2f(red_m[warp + w] - mx);
      const float4 u = red_o[warp + w][lane];
      acc.x = fmaf(a, u.x, acc.x);
      acc.y = fmaf(a, u.y, acc.y);
      acc.z = fmaf(a, u.z, acc.z);
      acc.w = fmaf(a, u.w, acc.w);
      wsum = fmaf(a, red_w[warp + w], wsum);
    }
    m = mx;
  }
  if (!live) return;
  const float inv = ns > 0 ? 1.0f / wsum : 0.0f;
  const uint32_t w0 = pack_bf16x2(acc.x * inv, acc.y * inv);
  const uint32_t w1 = pack_bf16x2(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(o + static_cast<size_t>(row) * kDim + 4 * lane) = make_uint2(w0, w1);
  if (lane == 0) lse[row] = ns > 0 ? (m + log2f(wsum)) * 0.69314718055994530942f : -INFINITY;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr int kMaxDevices = 64;
std::mutex g_decode_mutex;
bool g_decode_ready[kMaxDevices] = {};
EncodeTiledFn g_decode_encode = nullptr;

template <int GP, bool kRagged, bool kWeights, bool kWindow = false>
bool set_smem_of() {
  return cudaFuncSetAttribute(attn_decode_split_kernel<GP, kRagged, kWeights, kWindow>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kSmemBytes) == cudaSuccess;
}
template <int GP>
bool set_smem() {
  return set_smem_of<GP, false, false>() && set_smem_of<GP, true, false>() &&
         set_smem_of<GP, true, true>() && set_smem_of<GP, true, false, true>();
}

// The split kernel for groups of g query heads.
template <bool kRagged, bool kWeights, bool kWindow = false>
cudaError_t launch_split(const cudaLaunchConfig_t& cfg, const CUtensorMap& mq,
                         const CUtensorMap& mk, const CUtensorMap& mv, const DecodeParams& p,
                         const SinkMaps<kWindow>& sinks = {}) {
  if (p.g <= 4)
    return cudaLaunchKernelEx(&cfg, attn_decode_split_kernel<4, kRagged, kWeights, kWindow>, mq,
                              mk, mv, p, sinks);
  if (p.g <= 8)
    return cudaLaunchKernelEx(&cfg, attn_decode_split_kernel<8, kRagged, kWeights, kWindow>, mq,
                              mk, mv, p, sinks);
  return cudaLaunchKernelEx(&cfg, attn_decode_split_kernel<16, kRagged, kWeights, kWindow>, mq, mk,
                            mv, p, sinks);
}

attn_status_t decode_device_ready(cudaStream_t stream, int** status) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_UNSUPPORTED;
  // device check (sm_103) and the status word come from the forward's set-up
  const attn_status_t ds = gb300_host::device_status_word(stream, status);
  if (ds != ATTN_OK) return ds;
  std::lock_guard<std::mutex> lock(g_decode_mutex);
  if (g_decode_ready[dev]) return ATTN_OK;
  // one-time set-up: not inside a stream capture
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess || cs != cudaStreamCaptureStatusNone) {
    cudaGetLastError();
    return ATTN_ERR_UNSUPPORTED;
  }
  if (!g_decode_encode) {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || fn == nullptr)
      return ATTN_ERR_CUDA;
    g_decode_encode = reinterpret_cast<EncodeTiledFn>(fn);
  }
  if (!set_smem<4>() || !set_smem<8>() || !set_smem<16>()) return ATTN_ERR_CUDA;
  g_decode_ready[dev] = true;
  return ATTN_OK;
}

// K or V [B, Lk, H, 128] bf16 as (D, H, L, B): 64 x 1 x 128 x 1 boxes,
// 128-byte swizzle (the tensor cores' operand layout).
bool encode_kv(CUtensorMap* map, const void* ptr, int H, int64_t Lk, int64_t B,
               int rows = kKeys) {
  const cuuint64_t dims[4] = {kDim, static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(Lk),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {kDim * 2, static_cast<cuuint64_t>(H) * kDim * 2,
                                 static_cast<cuuint64_t>(Lk) * H * kDim * 2};
  const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(rows), 1};
  const cuuint32_t estride[4] = {1, 1, 1, 1};
  return g_decode_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims,
                         strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Q [B, 1, n_q, 128] bf16 as (D, n_q, B): 64 x 16 x 1 boxes (16 heads from
// the group's first), 128-byte swizzle.
bool encode_q(CUtensorMap* map, const void* ptr, int n_q, int64_t B) {
  const cuuint64_t dims[3] = {kDim, static_cast<cuuint64_t>(n_q), static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[2] = {kDim * 2, static_cast<cuuint64_t>(n_q) * kDim * 2};
  const cuuint32_t box[3] = {64, kHeadsPad, 1};
  const cuuint32_t estride[3] = {1, 1, 1};
  return g_decode_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims,
                         strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool decode_sizes_ok(int64_t B, int64_t Lk, int32_t n_q, int32_t n_kv, int32_t d_h) {
  return B >= 1 && Lk >= 1 && n_q >= 1 && n_kv >= 1 && n_q % n_kv == 0 && d_h >= 1;
}

// The partition of the B * n_kv * T key tiles over the split kernel's CTAs.
struct DecodeShape {
  int64_t T, W, G, P_max;
};
DecodeShape decode_shape(int64_t B, int64_t Lk, int32_t n_kv) {
  DecodeShape s;
  s.T = (Lk + kKeys - 1) / kKeys;
  s.W = B * n_kv * s.T;
  s.G = s.W < kDecodeCtas ? s.W : kDecodeCtas;
  s.P_max = segment_slots(s.W, s.G, s.T);
  return s;
}

// The ragged step's workspace: partial outputs, maxima and sums of at most
// B * n_kv + G segments, the heads' first and last CTAs, and the scores.
struct RaggedShape {
  int64_t G, ld, ml_at, ends_at, scores_at, bytes;
};
// (window > 0: a sequence has at most the tiles of its window and of its sinks)
RaggedShape ragged_shape(int64_t B, int64_t C, int32_t n_q, int32_t n_kv, bool weighted,
                         int64_t window = 0, int64_t sinks = 0) {
  RaggedShape s;
  auto tiles = [](int64_t n) { return (n + kKeys - 1) / kKeys; };
  int64_t T = tiles(C);
  if (window > 0 && window < C) {
    const int64_t seen = tiles(window) + tiles(sinks < C - window ? sinks : C - window);
    if (seen < T) T = seen;
  }
  const int64_t most = B * n_kv * T;
  s.G = most < kDecodeCtas ? most : kDecodeCtas;
  s.ld = T * kKeys;
  const int64_t rows = (B * n_kv + s.G) * (n_q / n_kv);
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  s.ml_at = up(rows * kDim * 4);
  s.ends_at = s.ml_at + up(rows * 8);
  s.scores_at = s.ends_at + up(B * n_kv * 8);
  s.bytes = s.scores_at + (weighted ? B * n_q * s.ld * 4 : 0);
  return s;
}

bool ragged_supported(int64_t B, int64_t C, int32_t n_q, int32_t n_kv, int32_t d_h) {
  if (d_h != kDim || n_q / n_kv > kMaxG) return false;
  if (C > (int64_t{1} << 30) || B > (int64_t{1} << 24) || B * n_kv > (int64_t{1} << 24)) return false;
  const int64_t chunks = (C + kWeightKeys - 1) / kWeightKeys;
  return B * n_q + B * n_kv * chunks <= INT32_MAX;
}

// Launches the ragged split kernel (arguments already validated, set-up done);
// *out gets its parameters, for the combine.
attn_status_t launch_ragged_split(const void* q, const void* k, const void* v, const int32_t* lens,
                                  void* workspace, int64_t B, int64_t C, int32_t n_q, int32_t n_kv,
                                  float scale, bool weighted, bool beside, cudaStream_t stream,
                                  int* status, DecodeParams* out, int64_t window = 0,
                                  int64_t sinks = 0) {
  const RaggedShape s = ragged_shape(B, C, n_q, n_kv, weighted, window, sinks);
  CUtensorMap mq, mk, mv;
  if (!encode_q(&mq, q, n_q, B) || !encode_kv(&mk, k, n_kv, C, B) || !encode_kv(&mv, v, n_kv, C, B))
    return ATTN_ERR_CUDA;
  char* ws = static_cast<char*>(workspace);
  DecodeParams p{};
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + s.ml_at);
  p.ends = reinterpret_cast<int*>(ws + s.ends_at);
  p.scores = weighted ? reinterpret_cast<float*>(ws + s.scores_at) : nullptr;
  p.ld = s.ld;
  p.beside = beside ? 1 : 0;
  p.window = static_cast<int>(window < C ? window : C);
  p.sinks = static_cast<int>(sinks < C ? sinks : C);
  p.status = status;
  p.lens = lens;
  p.B = static_cast<int>(B);
  p.Lk = static_cast<int>(C);
  p.n_q = n_q;
  p.n_kv = n_kv;
  p.g = n_q / n_kv;
  p.G = static_cast<int>(s.G);
  p.c = scale * 1.4426950408889634f;
  p.spin_limit = 1ll << 31;   // about a second at 2 GHz
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(s.G));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  SinkMaps<true> sm;
  sm.rows = p.sinks < kKeys ? (p.sinks + 7) / 8 * 8 : kKeys;
  if (window > 0 && p.sinks > 0 && sm.rows < kKeys &&
      (!encode_kv(&sm.k, k, n_kv, C, B, sm.rows) || !encode_kv(&sm.v, v, n_kv, C, B, sm.rows)))
    return ATTN_ERR_CUDA;
  const cudaError_t e = window > 0 ? launch_split<true, false, true>(cfg, mq, mk, mv, p, sm)
                        : weighted ? launch_split<true, true>(cfg, mq, mk, mv, p)
                                   : launch_split<true, false>(cfg, mq, mk, mv, p);
  *out = p;
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

namespace gb300_host {

attn_status_t decode_ready(cudaStream_t stream, int** status) {
  return decode_device_ready(stream, status);
}

int64_t ragged_split_bytes(int64_t B, int64_t C, int32_t n_q, int32_t n_kv, int32_t d_h) {
  if (!decode_sizes_ok(B, C, n_q, n_kv, d_h) || !ragged_supported(B, C, n_q, n_kv, d_h)) return -1;
  return ragged_shape(B, C, n_q, n_kv, false).bytes;
}

attn_status_t ragged_split_beside(const void* q, const void* k, const void* v, const int32_t* lens,
                                  void* workspace, int64_t B, int64_t C, int32_t n_q, int32_t n_kv,
                                  float scale, cudaStream_t stream, int* status,
                                  RaggedParts* parts) {
  DecodeParams p;
  const attn_status_t st = launch_ragged_split(q, k, v, lens, workspace, B, C, n_q, n_kv, scale,
                                               false, true, stream, status, &p);
  *parts = {p.part_o, p.part_ml, p.ends};
  return st;
}

}  // namespace gb300_host

extern "C" {

int64_t attn_decode_workspace_bytes(int64_t B, int64_t Lk, int32_t n_q, int32_t n_kv,
                                    int32_t d_h) {
  if (!decode_sizes_ok(B, Lk, n_q, n_kv, d_h) || d_h != kDim || n_q / n_kv > kMaxG) return -1;
  if (Lk > (int64_t{1} << 30) || B * n_kv > (int64_t{1} << 24)) return -1;
  const DecodeShape s = decode_shape(B, Lk, n_kv);
  const int64_t rows = s.G * s.P_max * (n_q / n_kv);
  return rows * kDim * 4 + rows * 4;
}

attn_status_t attn_decode_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                              void* workspace, int64_t workspace_bytes, int64_t B, int64_t Lk,
                              int32_t n_q, int32_t n_kv, int32_t d_h, float scale,
                              void* stream_ptr) {
  if (!q || !k || !v || !o || !lse || !workspace) return ATTN_ERR_INVALID_ARG;
  if (!decode_sizes_ok(B, Lk, n_q, n_kv, d_h) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  auto misaligned = [](const void* ptr, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0;
  };
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) ||
      misaligned(lse, 4) || misaligned(workspace, 16))
    return ATTN_ERR_INVALID_ARG;
  if (d_h != kDim || n_q / n_kv > kMaxG) return ATTN_ERR_UNSUPPORTED;
  if (Lk > (int64_t{1} << 30) || B * n_kv > (int64_t{1} << 24)) return ATTN_ERR_UNSUPPORTED;
  const DecodeShape s = decode_shape(B, Lk, n_kv);
  if (s.W > (int64_t{1} << 31) - 1 || B * n_q > (int64_t{1} << 31) - 1) return ATTN_ERR_UNSUPPORTED;
  const int64_t need = attn_decode_workspace_bytes(B, Lk, n_q, n_kv, d_h);
  if (workspace_bytes < need) return ATTN_ERR_INVALID_ARG;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  int* status = nullptr;
  const attn_status_t ds = decode_device_ready(stream, &status);
  if (ds != ATTN_OK) return ds;

  CUtensorMap mq, mk, mv;
  if (!encode_q(&mq, q, n_q, B) || !encode_kv(&mk, k, n_kv, Lk, B) ||
      !encode_kv(&mv, v, n_kv, Lk, B))
    return ATTN_ERR_CUDA;
  DecodeParams p{};
  const int64_t rows = s.G * s.P_max * (n_q / n_kv);
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = p.part_o + rows * kDim;
  p.status = status;
  p.Lk = static_cast<int>(Lk);
  p.n_q = n_q;
  p.n_kv = n_kv;
  p.g = n_q / n_kv;
  p.T = static_cast<int>(s.T);
  p.W = s.W;
  p.G = static_cast<int>(s.G);
  p.P_max = static_cast<int>(s.P_max);
  p.c = scale * 1.4426950408889634f;
  p.spin_limit = 1ll << 31;   // about a second at 2 GHz
  // Both kernels are launched as programmatic dependents of the kernel before
  // them in the stream: the split kernel's set-up overlaps the previous
  // kernel's end, and the combine's CTAs are scheduled while the split kernel
  // still runs. Each waits (griddepcontrol.wait) before touching memory.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(s.G));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (launch_split<false, false>(cfg, mq, mk, mv, p) != cudaSuccess) return ATTN_ERR_CUDA;
  cfg.gridDim = dim3(static_cast<unsigned>(B * n_q));
  cfg.blockDim = dim3(32 * kCombineWarps);
  cfg.dynamicSmemBytes = 0;
  uint16_t* o16 = static_cast<uint16_t*>(o);
  if (cudaLaunchKernelEx(&cfg, attn_decode_combine_kernel, o16, lse, p) != cudaSuccess)
    return ATTN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int64_t attn_decode_ragged_workspace_bytes(int64_t B, int64_t C, int32_t n_q, int32_t n_kv,
                                           int32_t d_h, int32_t weighted) {
  if (!decode_sizes_ok(B, C, n_q, n_kv, d_h) || (weighted != 0 && weighted != 1)) return -1;
  if (!ragged_supported(B, C, n_q, n_kv, d_h)) return -1;
  return ragged_shape(B, C, n_q, n_kv, weighted != 0).bytes;
}

// window > 0: behind a window with sinks, without weights. Both entry points'
// checks and launches.
static attn_status_t ragged_step(const void* q, const void* k, const void* v, const int32_t* lens,
                                 float* weights, void* o, float* lse, void* workspace,
                                 int64_t workspace_bytes, int64_t B, int64_t C, int32_t n_q,
                                 int32_t n_kv, int32_t d_h, int64_t window, int64_t sinks,
                                 float scale, void* stream_ptr) {
  if (!q || !k || !v || !lens || !o || !lse || !workspace) return ATTN_ERR_INVALID_ARG;
  if (!decode_sizes_ok(B, C, n_q, n_kv, d_h) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  auto misaligned = [](const void* ptr, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0;
  };
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) ||
      misaligned(lse, 4) || misaligned(lens, 4) || misaligned(weights, 4) ||
      misaligned(workspace, 16))
    return ATTN_ERR_INVALID_ARG;
  if (!ragged_supported(B, C, n_q, n_kv, d_h)) return ATTN_ERR_UNSUPPORTED;
  const bool weighted = weights != nullptr;
  if (workspace_bytes < ragged_shape(B, C, n_q, n_kv, weighted, window, sinks).bytes) return ATTN_ERR_INVALID_ARG;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  int* status = nullptr;
  attn_status_t st = decode_device_ready(stream, &status);
  if (st != ATTN_OK) return st;
  DecodeParams p;
  st = launch_ragged_split(q, k, v, lens, workspace, B, C, n_q, n_kv, scale, weighted, false,
                           stream, status, &p, window, sinks);
  if (st != ATTN_OK) return st;
  const int chunks = weighted ? static_cast<int>((C + kWeightKeys - 1) / kWeightKeys) : 0;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // segments per head: one, and one more for every range border inside it. Eight
  // warps per row where a head has more than nine on average (a whole step with 8
  // heads of 152: 17 us, 41 with one warp; 32 of 20: 48, 51; 64 of 10: 86, 87), one
  // where it has fewer (the combine of 16384 rows of one or two: 12, 145 with eight)
  const bool many = p.G > 8 * B * n_kv;
  const int64_t merges = many ? B * n_q : (B * n_q + kCombineWarps - 1) / kCombineWarps;
  cfg.gridDim = dim3(static_cast<unsigned>(merges + B * n_kv * chunks));
  cfg.blockDim = dim3(32 * kCombineWarps);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  uint16_t* o16 = static_cast<uint16_t*>(o);
  const int m32 = static_cast<int>(merges);
  const cudaError_t e =
      many ? cudaLaunchKernelEx(&cfg, attn_decode_ragged_combine_kernel<kCombineWarps>, o16, lse,
                                weights, m32, chunks, p)
           : cudaLaunchKernelEx(&cfg, attn_decode_ragged_combine_kernel<1>, o16, lse, weights, m32,
                                chunks, p);
  if (e != cudaSuccess) return ATTN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t attn_decode_ragged_fwd(const void* q, const void* k, const void* v,
                                     const int32_t* lens, float* weights, void* o, float* lse,
                                     void* workspace, int64_t workspace_bytes, int64_t B, int64_t C,
                                     int32_t n_q, int32_t n_kv, int32_t d_h, float scale,
                                     void* stream_ptr) {
  return ragged_step(q, k, v, lens, weights, o, lse, workspace, workspace_bytes, B, C, n_q, n_kv,
                     d_h, 0, 0, scale, stream_ptr);
}

int64_t attn_decode_window_workspace_bytes(int64_t B, int64_t C, int32_t n_q, int32_t n_kv,
                                           int32_t d_h, int64_t window, int64_t sinks) {
  if (!decode_sizes_ok(B, C, n_q, n_kv, d_h) || window < 1 || sinks < 0) return -1;
  if (!ragged_supported(B, C, n_q, n_kv, d_h)) return -1;
  return ragged_shape(B, C, n_q, n_kv, false, window, sinks).bytes;
}

attn_status_t attn_decode_window_fwd(const void* q, const void* k, const void* v,
                                     const int32_t* lens, void* o, float* lse, void* workspace,
                                     int64_t workspace_bytes, int64_t B, int64_t C, int32_t n_q,
                                     int32_t n_kv, int32_t d_h, int64_t window, int64_t sinks,
                                     float scale, void* stream_ptr) {
  if (window < 1 || sinks < 0) return ATTN_ERR_INVALID_ARG;
  return ragged_step(q, k, v, lens, nullptr, o, lse, workspace, workspace_bytes, B, C, n_q, n_kv,
                     d_h, window, sinks, scale, stream_ptr);
}

}  // extern "C"
