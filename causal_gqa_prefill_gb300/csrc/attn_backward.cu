// attn_backward.cu — gradients of the causal GQA attention forward on GB300
// (sm_103a), by recomputation from the saved log-sum-exp.
//
// The backward pass rebuilds each score tile from Q, K and the forward's row
// statistics instead of storing the L x L table ("Long-Context Attention
// Explained" (sevydevy), "What FlashAttention does not change"). With
// P = exp(scale*S - LSE), D_i = dO_i . O_i:
//
//   dV_j = sum_i P_ij dO_i        dP = dO V^T        dS = P * (dP - D)
//   dK_j = scale sum_i dS_ij Q_i  dQ_i = scale sum_j dS_ij K_j
//
// Three kernels, no atomics:
//   rowdot  per query row: -LSE*log2(e) and -D = -dO . O, padded to whole
//           128-row tiles (-inf / 0) so tiles can be fetched with bulk copies;
//   dkdv    one CTA per (b, K/V head, 128-key tile j): loops over the g query
//           heads of the group and the query tiles that see tile j; with the
//           key dimension on the TMEM lanes it computes S^T = K Q^T and
//           dP^T = V dO^T (tcgen05, both operands from shared memory, K_j and
//           V_j resident), turns them into P^T and dS^T (bf16, written back
//           into TMEM) and accumulates dV += P^T dO and dK += dS^T Q (A from
//           TMEM); dK and dV for the whole group stay in TMEM until the end.
//           Q and dO come through rings of their own, three and two tiles deep;
//   dq      persistent (one CTA per SM), walking (b, query head, 128-row
//           tile i) units longest first in snake order: S = Q K^T (Q_i in
//           TMEM) and dP = dO V^T (dO_i in shared memory), dS in its own TMEM
//           columns, dQ += dS K over the key tiles it sees; the next unit's
//           K/V tiles, Q_i and dO_i come in, and its first scores run, while the
//           current unit's last dQ product is done and stored.
// Both tile kernels step over whole 128-column score tiles (128 queries of a
// query tile in dkdv, 128 keys of a key tile in dq), so every product is
// N = 128 (or D) wide, and order their products so that the tensor cores run
// the next tile's scores while the compute warps turn this tile's into P/dS.
//
// Sliding window with sinks (kWin instances; a row at position p sees keys j <= p
// with j > p - W or j < S): a key tile meets only the query tiles whose windows
// reach it and a query tile only the sinks' and its window's key tiles. Key tiles
// that hold a sink are seen by every later row; they come first, each cut into
// `pieces` CTAs of equal runs of (head, query tile) steps, which write fp32 parts
// that a join kernel adds in order (no atomics). So are, where a call has few key
// tiles, the others (key_split). Measured: 8192 tokens, 32 heads on 8, W = 1024 and
// S = 4: rowdot 25, dkdv 220, dq 178, the join 6 us (323 GFLOP of five products: 171 at
// the burst rate; seven are run, as S and dP are rebuilt twice). A dkdv step takes
// about 2300 cycles where its four products are 2048 of the tensor pipe at its own rate
// (2600 at the burst rate), and a CTA 14000 beside its steps. A tile of dq takes 2200 for
// 1536, its exponentials' chain: 133 us for the 19040 tiles; the other 45 are the borders
// of 13.5 units an SM.
//
// Each kernel has a TMA producer warp, an MMA warp (warp-wide loop, one elected
// issuing lane) and kComputeWGs compute warpgroups that split the 128 columns
// of a tile (thread = TMEM lane = tile row; warpgroup w owns columns
// [w*C, w*C + C), C = 128 / kComputeWGs). A warpgroup writes its bf16 P (and
// in dkdv dS) back over the first C/2 of its own, already consumed, fp32
// columns, so no warpgroup ever overwrites columns another one still has to
// read; the products that consume P/dS take their A operand K-step by K-step
// from there.
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

constexpr int kT = 128;                  // rows per query tile and keys per key tile
// One bf16 tile of 128 rows x D (D = 64 or 128 head dimensions): D / 64
// chunks of 128 rows x 128 bytes, 128-byte swizzled.
template <int D>
__host__ __device__ constexpr int tile_bytes() { return kT * D * 2; }
constexpr int kComputeWGs = 2;           // compute warpgroups
constexpr int kColsQ = kT / kComputeWGs;     // dQ: key-tile columns per warpgroup
constexpr int kComputeThreads = 128 * kComputeWGs;
constexpr int kLoadWarp = 4 * kComputeWGs, kMmaWarp = kLoadWarp + 1;
// producer and MMA warps plus two idle warps: registers are granted per
// four warps, so the CTA is a whole number of warpgroups
constexpr int kThreads = kComputeThreads + 128;
constexpr long long kSpinLimit = 1ll << 31;
constexpr float kLog2e = 1.4426950408889634f;

struct BwdParams {
  int L, n_q, n_kv, g, T;   // T = 128-row tiles per sequence
  int causal;
  float c;                  // scale * log2(e)
  float scale;
  const float* nlse2;       // [B, n_q, T*128] -LSE * log2(e), -inf past L
  const float* nrowdot;     // [B, n_q, T*128] -D, 0 past L
  uint16_t* dq;             // bf16 [B, L, n_q, 128]
  uint16_t* dk;             // bf16 [B, L, n_kv, 128]
  uint16_t* dv;
  int* status;
  int q_units;              // dQ work units: B * n_q * T query tiles
  // Rows that see one key: the first `one_key_rows` (0, 1 or all L). Their weight is 1
  // whatever the score, so dS is 0; what rounding leaves of dP - D (the tensor cores' sum
  // less the row kernel's, 1e-6 of |dO| |V|) would be all that their dQ is. So is it of
  // dK where all rows are such: dk_scale, what dK is multiplied by, is then 0. (Both keep
  // what is not a number.)
  int one_key_rows;
  float dk_scale;           // else scale
  // kWin instances
  int window, sinks;        // W and S, both at most L
  int heavy, pieces;        // key tiles that hold a sink, and CTAs per such tile
  int others;               // CTAs per other key tile
  // where a tile has more than one CTA: fp32 [dV, dK][128][D] of each, [groups][heavy]
  // [pieces] and, behind them, [groups][T - heavy][others]
  float* parts;
};

// Number of the first part of key tile j of group grp.
__device__ __forceinline__ size_t first_part(const BwdParams& p, int groups, size_t grp, int j) {
  const size_t first = p.pieces > 1 ? static_cast<size_t>(groups) * p.heavy * p.pieces : 0;
  return j < p.heavy ? (grp * p.heavy + j) * p.pieces
                     : first + (grp * (p.T - p.heavy) + j - p.heavy) * p.others;
}

// The key tiles that query tile i sees, in order: tiles [0, na), which hold sinks
// before its window, then tiles lo .. i.
struct SeenTiles {
  int na, lo, n;
};
template <bool kWin>
__device__ __forceinline__ SeenTiles seen_tiles(int i, const BwdParams& p) {
  if (!kWin) return {0, 0, p.causal ? i + 1 : p.T};
  SeenTiles x;
  x.lo = max(0, i * kT - p.window + 1) / kT;
  x.na = min(p.heavy, x.lo);
  x.n = x.na + i - x.lo + 1;
  return x;
}
template <bool kWin>
__device__ __forceinline__ int seen_tile(const SeenTiles& x, int t) {
  return !kWin || t < x.na ? t : t - x.na + x.lo;
}

// One CTA's work in the dK/dV kernel: steps first .. first + n - 1 of the
// (head, query tile) pairs of key tile j, `per_head` query tiles from i0 on each.
struct KeyWork {
  int j, grp, i0, per_head, first, n, piece, pieces, groups;
};
template <bool kWin>
__device__ __forceinline__ KeyWork key_work(const BwdParams& p) {
  KeyWork w;
  if (!kWin) {
    const int groups = static_cast<int>(gridDim.x) / p.T;
    w.j = blockIdx.x / groups;                        // ascending = most work first
    w.grp = blockIdx.x - w.j * groups;
    w.i0 = p.causal ? w.j : 0;
    w.per_head = p.T - w.i0;
    w.first = 0;
    w.n = p.g * w.per_head;
    w.piece = 0;
    w.pieces = 1;
    w.groups = groups;
    return w;
  }
  const int rows = p.heavy * p.pieces + (p.T - p.heavy) * p.others;
  w.groups = static_cast<int>(gridDim.x) / rows;
  int slot = blockIdx.x / w.groups;
  w.grp = blockIdx.x - slot * w.groups;
  const bool heavy = slot < p.heavy * p.pieces;
  if (!heavy) slot -= p.heavy * p.pieces;
  w.pieces = heavy ? p.pieces : p.others;
  w.j = slot / w.pieces;
  w.piece = slot - w.j * w.pieces;
  if (!heavy) w.j += p.heavy;
  w.i0 = w.j;
  // the last row that sees the tile's last key
  const int last = heavy ? p.T - 1
                         : static_cast<int>(min(static_cast<long long>(p.T) - 1,
                               (static_cast<long long>(w.j) * kT + kT - 1 + p.window - 1) / kT));
  w.per_head = last - w.i0 + 1;
  const long long total = static_cast<long long>(p.g) * w.per_head;
  w.first = static_cast<int>(total * w.piece / w.pieces);
  w.n = static_cast<int>(total * (w.piece + 1) / w.pieces) - w.first;
  return w;
}

constexpr int kStages = 3;               // dQ: ring of streamed K/V tiles
constexpr int kStagesQ = 3, kStagesDO = 2;   // dK/dV: rings of streamed Q and dO tiles (K_j, V_j stay)

struct Sync {
  uint64_t a_ready;                 // the CTA's fixed A operands are in TMEM
  uint64_t fixed_full;              // dK/dV: V_j has landed in shared memory
  uint64_t full[kStages], empty[kStages];  // dQ: K/V tiles; dK/dV: Q tiles
  uint64_t do_full[kStagesDO], do_empty[kStagesDO];   // dK/dV: dO tiles
  uint64_t row_full[2];             // dK/dV: row statistics of a step
  uint64_t s_full[2], p_full[2];    // scores ready (commit) / P or dS ready (compute threads)
  uint64_t dp_full, ds_full;        // dP (dP^T) ready (commit) / dS (dS^T) ready (compute threads)
  uint64_t dp_free, dq_done;        // dQ: dP read out (compute threads) / dQ += dS K done (commit)
  uint64_t do_free;                 // dQ: the unit's last product with dO done (commit)
  uint64_t done, drain;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, Sync& sy,
                                             const BwdParams& p) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = clock64_now();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&sy.abort)) return false;
    if (static_cast<long long>(clock64_now() - t0) > kSpinLimit) {
      *reinterpret_cast<volatile int*>(&sy.abort) = 1;
      atomicOr(p.status, 1);
      return false;
    }
  }
}

__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = clock64_now();
  while (!mbar_try_wait(bar, parity))
    if (static_cast<long long>(clock64_now() - t0) > kSpinLimit) return;
}

// Plain (non-tensor) bulk copy global -> shared, completion on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// TMEM column (relative to the score tile's base) holding the bf16 A operand
// for K step kk (tile columns 16*kk .. 16*kk + 15): warpgroup w packs its
// columns [w*C, w*C + C) two per 32-bit column starting at column w*C.
template <int C>
__host__ __device__ constexpr uint32_t a_col(int kk) {
  return static_cast<uint32_t>((16 * kk / C) * C + (16 * kk % C) / 2);
}

// This thread's row of a bf16 [B, L, H, D] tensor into D/2 TMEM columns of
// its lane, as a tcgen05 A operand (column c = elements 2c, 2c+1, the lower in
// the low half, which is the row's memory order); rows past L become zeros.
template <int D>
__device__ __forceinline__ void row_to_tmem(uint32_t taddr, const uint16_t* src, bool valid) {
#pragma unroll
  for (int half = 0; half < D / 64; ++half) {
    uint32_t w[32];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (valid) x = reinterpret_cast<const uint4*>(src)[8 * half + q];
      w[4 * q] = x.x;
      w[4 * q + 1] = x.y;
      w[4 * q + 2] = x.z;
      w[4 * q + 3] = x.w;
    }
    tmem_st32(taddr + 32 * half, w);
  }
}

// Scores of a whole tile: D[128 x 128] = A B^T over K = 128, A a fixed operand
// in TMEM, B a [128 rows x 128] K-major tile in shared memory.
template <int D>
__device__ __forceinline__ void mma_scores_full(bool leader, uint32_t d_tmem, uint32_t a_tmem,
                                                uint32_t b_smem) {
  constexpr uint32_t idesc = idesc_bf16_f32(kT, kT, false);
  const uint64_t b0 = sdesc_sw128(b_smem, 16, 1024);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = (kk >> 2) * (kT * 128) + (kk & 3) * 32;
    if (leader) mma_ts(d_tmem, a_tmem + 8 * kk, b0 + (off >> 4), idesc, kk > 0 ? 1u : 0u);
  }
}

// D[128 x 128] (+)= A B over K = 128: A the bf16 dS of a whole tile in TMEM
// (a_col<kColsQ> layout), B a [128 rows x 128] tile used MN-major.
template <int D>
__device__ __forceinline__ void mma_accum_full(bool leader, uint32_t d_tmem, uint32_t a_tmem,
                                               uint32_t b_smem, bool accumulate) {
  constexpr uint32_t idesc = idesc_bf16_f32(kT, D, true);
  const uint64_t b0 = sdesc_sw128(b_smem, kT * 128, 1024);
#pragma unroll
  for (int kk = 0; kk < kT / 16; ++kk)
    if (leader)
      mma_ts(d_tmem, a_tmem + a_col<kColsQ>(kk), b0 + ((kk * 16 * 128) >> 4), idesc,
             (accumulate || kk > 0) ? 1u : 0u);
}

// dQ[128 x D] (+)= dS K over K = 128 keys: dS bf16 in TMEM, packed two keys
// per column (K step kk at column 8*kk), K a [128 keys x D] tile used MN-major.
template <int D>
__device__ __forceinline__ void mma_accum_dq(bool leader, uint32_t d_tmem, uint32_t a_tmem,
                                             uint32_t b_smem, bool accumulate) {
  constexpr uint32_t idesc = idesc_bf16_f32(kT, D, true);
  const uint64_t b0 = sdesc_sw128(b_smem, kT * 128, 1024);
#pragma unroll
  for (int kk = 0; kk < kT / 16; ++kk)
    if (leader)
      mma_ts(d_tmem, a_tmem + 8 * kk, b0 + ((kk * 16 * 128) >> 4), idesc,
             (accumulate || kk > 0) ? 1u : 0u);
}

// D[128 x 128] = A B^T over K = D: A a [128 rows x D] K-major tile in shared
// memory (dO), B a [128 rows x D] K-major tile (V).
template <int D>
__device__ __forceinline__ void mma_scores_full_ss(bool leader, uint32_t d_tmem, uint32_t a_smem,
                                                   uint32_t b_smem) {
  constexpr uint32_t idesc = idesc_bf16_f32(kT, kT, false);
  const uint64_t a0 = sdesc_sw128(a_smem, 16, 1024);
  const uint64_t b0 = sdesc_sw128(b_smem, 16, 1024);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = ((kk >> 2) * (kT * 128) + (kk & 3) * 32) >> 4;
    if (leader) mma_ss(d_tmem, a0 + off, b0 + off, idesc, kk > 0 ? 1u : 0u);
  }
}

__device__ __forceinline__ void setup(Sync& sy) {
  if (threadIdx.x == 0) {
    mbar_init(smem_addr(&sy.a_ready), kComputeThreads);
    mbar_init(smem_addr(&sy.fixed_full), 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(&sy.full[s]), 1);
      mbar_init(smem_addr(&sy.empty[s]), 1);
    }
    for (int s = 0; s < kStagesDO; ++s) {
      mbar_init(smem_addr(&sy.do_full[s]), 1);
      mbar_init(smem_addr(&sy.do_empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) mbar_init(smem_addr(&sy.row_full[s]), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_addr(&sy.s_full[s]), 1);
      mbar_init(smem_addr(&sy.p_full[s]), kComputeThreads);
    }
    mbar_init(smem_addr(&sy.dp_full), 1);
    mbar_init(smem_addr(&sy.ds_full), kComputeThreads);
    mbar_init(smem_addr(&sy.dp_free), kComputeThreads);
    mbar_init(smem_addr(&sy.dq_done), 1);
    mbar_init(smem_addr(&sy.do_free), 1);
    mbar_init(smem_addr(&sy.done), 1);
    mbar_init(smem_addr(&sy.drain), 1);
    sy.abort = 0;
    fence_mbar_init();
  }
  if ((threadIdx.x >> 5) == kMmaWarp) {
    tmem_alloc(smem_addr(&sy.tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
}

__device__ __forceinline__ void teardown(Sync& sy, const BwdParams& p, bool leader_mma) {
  if ((threadIdx.x >> 5) == kMmaWarp) {
    if (leader_mma) mma_commit(smem_addr(&sy.drain));
    wait_drain(smem_addr(&sy.drain), 0);
    __syncwarp();
  }
  tc_fence_before_sync();
  __syncthreads();
  if ((threadIdx.x >> 5) == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(sy.tmem_base, 512);
  }
}

// What is added to a product with `mul`: nothing (x + -0 is x), but products with 0 all
// become +0.
__device__ __forceinline__ float plus_zero(float mul) { return mul == 0.0f ? 0.0f : -0.0f; }

// 32 bf16 outputs of this thread's row from 32 fp32 TMEM columns, times `mul`.
__device__ __forceinline__ void store_chunk(uint32_t taddr, uint16_t* dst, float mul, bool valid) {
  uint32_t v[32];
  tmem_ld32(taddr, v);
  tmem_wait_ld(v);
  const float zero = plus_zero(mul);
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i)
    w[i] = pack_bf16x2(fmaf(__uint_as_float(v[2 * i]), mul, zero),
                       fmaf(__uint_as_float(v[2 * i + 1]), mul, zero));
  if (valid) {
    uint4* d4 = reinterpret_cast<uint4*>(dst);
#pragma unroll
    for (int q = 0; q < 4; ++q) d4[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  }
}

// The same 32 columns times `mul`, kept in fp32.
__device__ __forceinline__ void store_chunk_f32(uint32_t taddr, float* dst, float mul) {
  uint32_t v[32];
  tmem_ld32(taddr, v);
  tmem_wait_ld(v);
  float4* d4 = reinterpret_cast<float4*>(dst);
#pragma unroll
  for (int q = 0; q < 8; ++q)
    d4[q] = make_float4(__uint_as_float(v[4 * q]) * mul, __uint_as_float(v[4 * q + 1]) * mul,
                        __uint_as_float(v[4 * q + 2]) * mul, __uint_as_float(v[4 * q + 3]) * mul);
}

// A word whose lowest n bits are set (none for n <= 0, all from 32 on).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
}

// dK/dV phase 1 for one warpgroup: P^T = 2^(c S^T + nl) for its kColsQ query
// columns of this thread's key row (S^T read from TMEM at `taddr`, the row
// statistics nl from shared memory), kept in `pr` and written back as bf16
// over the first consumed columns. kMask: the diagonal tile, where query
// column q0 + k is masked when q0 + k < r (q_minus_r = q0 - r). kWin: or when
// it is past the last row that sees the key (q_to_end, from q0 on).
template <bool kMask, bool kWin>
__device__ __forceinline__ void pt_from_st(uint32_t taddr, const float4* nl4, uint64_t c2,
                                           int q_minus_r, int q_to_end, float (&pr)[kColsQ]) {
#pragma unroll
  for (int cc = 0; cc < kColsQ / 32; ++cc) {
    uint32_t sv[32];
    tmem_ld32(taddr + 32 * cc, sv);
    tmem_wait_ld(sv);
    // (behind a window the seen queries as bits, which cost a select each: compared with
    // both ends one by one the 8192-token layer's kernel took 5 us more)
    uint32_t seen = 0;
    if (kWin) seen = low_bits(q_to_end + 1 - 32 * cc) & ~low_bits(-q_minus_r - 32 * cc);
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float4 nl = nl4[8 * cc + e];
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        const int jj = 4 * e + 2 * h2;
        const uint64_t x = ffma2(f32x2_pack(__uint_as_float(sv[jj]), __uint_as_float(sv[jj + 1])),
                                 c2, h2 ? f32x2_pack(nl.z, nl.w) : f32x2_pack(nl.x, nl.y));
        float x0, x1;
        f32x2_unpack(x, x0, x1);
        float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
        if (kMask) {
          if (kWin ? !(seen >> jj & 1u) : q_minus_r + 32 * cc + jj < 0) p0 = 0.0f;
          if (kWin ? !(seen >> (jj + 1) & 1u) : q_minus_r + 32 * cc + jj + 1 < 0) p1 = 0.0f;
        }
        pr[32 * cc + jj] = p0;
        pr[32 * cc + jj + 1] = p1;
        pk[jj / 2] = pack_bf16x2(p0, p1);
      }
    }
    tmem_st16(taddr + 16 * cc, pk);
  }
}

// dQ phase 1 for one warpgroup: P = 2^(c S + nl) for its kColsQ key columns
// [k0, k0 + kColsQ) of this thread's query row, kept in `pr`. kMask: keys
// after in-tile index `keep` are masked (the diagonal tile, or keys past L).
// kWin: so are those up to `out` (before the window) from `sink` on.
template <bool kMask, bool kWin>
__device__ __forceinline__ void p_from_s(uint32_t taddr, uint64_t c2, uint64_t nl2, int k0,
                                         int keep, int out, int sink, float (&pr)[kColsQ]) {
#pragma unroll
  for (int c = 0; c < kColsQ / 32; ++c) {
    uint32_t sv[32];
    tmem_ld32(taddr + 32 * c, sv);
    tmem_wait_ld(sv);
    uint32_t seen = 0;
    if (kWin) {
      const int at = k0 + 32 * c;
      seen = low_bits(keep + 1 - at) & (~low_bits(out + 1 - at) | low_bits(sink - at));
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint64_t x = ffma2(
          f32x2_pack(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), c2, nl2);
      float x0, x1;
      f32x2_unpack(x, x0, x1);
      float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
      if (kMask) {
        const int at = k0 + 32 * c + 2 * e;
        if (kWin ? !(seen >> (2 * e) & 1u) : at > keep) p0 = 0.0f;
        if (kWin ? !(seen >> (2 * e + 1) & 1u) : at + 1 > keep) p1 = 0.0f;
      }
      pr[32 * c + 2 * e] = p0;
      pr[32 * c + 2 * e + 1] = p1;
    }
  }
}

// ------------------------------------------------------------------ rowdot

// Half a warp per row: 16 lanes x D / 16 dimensions. A block takes up to kRowdotH
// neighbouring heads of 8 << more positions, 64 rows or nearly, so that it reads O and dO
// in their own order, four rows (eight loads) under way per half-warp, and writes whole
// pieces of the [b, h, t] statistics out of shared memory. (One row (b, h, t) after
// another, with three divisions each, took 41 us for 134 MB, this 25; 32 positions of
// 8 heads a block took 8 us for 1000 rows of 8 heads, 8 take 5; 8 positions of a single
// head took 14 us for 32768 rows, 64 take 8.) Positions past L get -inf and 0 without
// touching O or dO. The dK/dV kernel is launched as this grid's programmatic dependent
// and waits for it before it reads the statistics.
constexpr int kRowdotH = 8;
// Doublings of a block's 8 positions: as many as keep its rows at 64.
int row_doublings(int64_t n_q) { return n_q >= 5 ? 0 : n_q >= 3 ? 1 : n_q == 2 ? 2 : 3; }
__device__ __forceinline__ float dot2_bf16(uint32_t a, uint32_t d, float acc) {
  acc = fmaf(__uint_as_float(a << 16), __uint_as_float(d << 16), acc);
  return fmaf(__uint_as_float(a & 0xFFFF0000u), __uint_as_float(d & 0xFFFF0000u), acc);
}
__device__ __forceinline__ float dot8_bf16(uint4 a, uint4 d) {
  float acc = __uint_as_float(a.x << 16) * __uint_as_float(d.x << 16);
  acc = fmaf(__uint_as_float(a.x & 0xFFFF0000u), __uint_as_float(d.x & 0xFFFF0000u), acc);
  acc = fmaf(__uint_as_float(a.y << 16), __uint_as_float(d.y << 16), acc);
  acc = fmaf(__uint_as_float(a.y & 0xFFFF0000u), __uint_as_float(d.y & 0xFFFF0000u), acc);
  acc = fmaf(__uint_as_float(a.z << 16), __uint_as_float(d.z << 16), acc);
  acc = fmaf(__uint_as_float(a.z & 0xFFFF0000u), __uint_as_float(d.z & 0xFFFF0000u), acc);
  acc = fmaf(__uint_as_float(a.w << 16), __uint_as_float(d.w << 16), acc);
  acc = fmaf(__uint_as_float(a.w & 0xFFFF0000u), __uint_as_float(d.w & 0xFFFF0000u), acc);
  return acc;
}

// Lanes of a half-warp hold D / 16 dimensions each (8 for D = 128: one
// 16-byte load; 4 for D = 64: the first half of it).
template <int D, int more>
__global__ void __launch_bounds__(256)
rowdot_kernel(const uint16_t* o, const uint16_t* dout, const float* lse, float* nlse2,
              float* nrowdot, int L, int n_q, int Lp) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int positions = 8 << more;
  __shared__ float dots[72];                            // [head][position], one more to a head
  constexpr int kAhead = 4, kHalves = 16;               // half-warps of a block
  const int t_blocks = Lp / positions, h_blocks = (n_q + kRowdotH - 1) / kRowdotH;
  const int rest = blockIdx.x / t_blocks;
  const int t0 = (blockIdx.x - rest * t_blocks) * positions, h0 = rest % h_blocks * kRowdotH;
  const int heads = min(kRowdotH, n_q - h0);
  const size_t b = rest / h_blocks;
  // row of the block's [position][head] order -> position
  auto position = [&](int row) { return heads == kRowdotH ? row / kRowdotH : row / heads; };
  const int half = threadIdx.x >> 4, l16 = threadIdx.x & 15;
  const int rows = heads * min(positions, L - t0);       // (may be none: then below zero)
  for (int r0 = half; r0 < heads * positions; r0 += kAhead * kHalves) {
    uint4 a[kAhead], d[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int row = r0 + k * kHalves;                 // position major
      const int t = position(row), h = row - t * heads;
      a[k] = d[k] = make_uint4(0u, 0u, 0u, 0u);
      if (row < rows) {
        const size_t off = ((b * L + t0 + t) * n_q + h0 + h) * D + (D / 16) * l16;
        if (D == 128) {
          a[k] = *reinterpret_cast<const uint4*>(o + off);
          d[k] = *reinterpret_cast<const uint4*>(dout + off);
        } else {
          const uint2 a2 = *reinterpret_cast<const uint2*>(o + off);
          const uint2 d2 = *reinterpret_cast<const uint2*>(dout + off);
          a[k] = make_uint4(a2.x, a2.y, 0u, 0u);
          d[k] = make_uint4(d2.x, d2.y, 0u, 0u);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int row = r0 + k * kHalves;
      float dd = (D == 128) ? dot8_bf16(a[k], d[k])
                            : dot2_bf16(a[k].y, d[k].y, dot2_bf16(a[k].x, d[k].x, 0.0f));
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) dd += __shfl_xor_sync(0xffffffffu, dd, off);
      if (l16 == 0 && row < heads * positions) {
        const int t = position(row);
        dots[(row - t * heads) * (positions + 1) + t] = row < rows ? dd : 0.0f;
      }
    }
  }
  __syncthreads();
  const int h = threadIdx.x >> (3 + more), t = threadIdx.x & (positions - 1);
  if (h < heads) {
    const size_t head = b * n_q + h0 + h;
    nrowdot[head * Lp + t0 + t] = -dots[h * (positions + 1) + t];
    nlse2[head * Lp + t0 + t] = t0 + t < L ? -lse[head * L + t0 + t] * kLog2e : -INFINITY;
  }
}

// -------------------------------------------------------------------- dK, dV

// Producer side shared by both tile kernels: drains the ring so that no copy is
// still in flight when the CTA exits; `issued` tiles were put in flight.
template <int S>
__device__ __forceinline__ void drain_ring(uint64_t* full, int issued) {
  for (int s = 0; s < S && s < issued; ++s) {
    const int last = s + ((issued - 1 - s) / S) * S;
    wait_drain(smem_addr(&full[s]), (last / S) & 1);
  }
}

// The kernel's dynamic shared memory: its tiles, statistics and barriers, and what may be
// lost to alignment as far as an SM's 227 KiB go.
template <int D>
__host__ __device__ constexpr int dkdv_smem() {
  constexpr int need = (2 + kStagesQ + kStagesDO) * tile_bytes<D>() + 2 * 1024 + sizeof(Sync);
  constexpr int most = 227 * 1024;
  static_assert(need <= most, "dK/dV's tiles do not fit");
  return need + 1024 < most ? need + 1024 : most;
}

template <int D, bool kWin>
__global__ void __launch_bounds__(kThreads, 1)
dkdv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
            const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
            const BwdParams p) {
  extern __shared__ uint8_t dyn_smem[];
  // smem: K_j | V_j | kStagesQ x Q_i | kStagesDO x dO_i | 2 x [-LSE*log2 e [128] | -D [128]] | Sync
  constexpr int kTileBytes = tile_bytes<D>();
  const uint32_t base = (smem_addr(dyn_smem) + 1023u) & ~1023u;
  const uint32_t sK = base, sV = base + kTileBytes, sQ0 = base + 2 * kTileBytes;
  const uint32_t sDO0 = sQ0 + kStagesQ * kTileBytes, sRow0 = sDO0 + kStagesDO * kTileBytes;
  Sync& sy = *reinterpret_cast<Sync*>(dyn_smem + (sRow0 + 2 * 1024 - smem_addr(dyn_smem)));
  if (sRow0 + 2 * 1024 + sizeof(Sync) > smem_addr(dyn_smem) + dkdv_smem<D>()) {
    // (at d_h = 128 all of an SM's memory, which holds if it begins on a 1 KiB boundary)
    if (threadIdx.x == 0) atomicOr(p.status, 1);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const KeyWork work = key_work<kWin>(p);
  const int j = work.j, grp = work.grp;                // key tile, (sequence, K/V head)
  const int b = grp / p.n_kv, kvh = grp - b * p.n_kv;
  const int i0 = work.i0;
  const int nsteps = work.n;                           // (head, query tile) pairs
  setup(sy);
  // Launched as the row kernel's programmatic dependent: the set-up above
  // overlaps its end; the row statistics are read only after it completed.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // The dQ kernel (this grid's programmatic dependent) reads nothing this
  // kernel writes: its CTAs may take SMs as soon as every CTA here is past
  // the wait above (so the row statistics are complete when dQ starts).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = sy.tmem_base;
  // TMEM columns: S^T 0..127 (P^T, bf16, is written over it), dP^T 128..255
  // (dS^T over it), dV at 256 and dK at 256 + D (D columns each). Each step
  // is a whole 128-query tile, so every product has N = 128 (or D): the
  // tensor cores get 64-cycle MMAs, which one issuing thread keeps up with.
  constexpr uint32_t cS = 0, cP = 128, cDV = 256, cDK = 256 + D;
  // Whether dO is waited for by itself: at d_h = 64 the products are so short that the
  // MMA warp's wait costs more than S^T gains by not waiting for dO (32768 tokens of one
  // head 483 us for the whole gradient, 465 with Q and dO on one barrier; at 128 dK/dV
  // behind a window of 4096 490 and 502).
  constexpr bool kApart = D == 128;

  if (warp == kLoadWarp) {
    if (lane == 0) {
      const uint32_t fb = smem_addr(&sy.fixed_full);
      mbar_arrive_expect_tx(fb, 2 * kTileBytes);
      for (int c = 0; c < D / 64; ++c) {
        tma_load_4d(sK + c * kT * 128, &tmK, fb, c * 64, kvh, j * kT, b);
        tma_load_4d(sV + c * kT * 128, &tmV, fb, c * 64, kvh, j * kT, b);
      }
      // Rings of their own for Q, dO and the row statistics: S^T needs Q first and dK
      // last, dO is free once dV has it. (8192 tokens, 32 heads on 8, window 1024 and 4
      // sinks: one ring of two stages for all of it 240 us, with the tensor cores
      // waiting 340 of a step's 2600 cycles for Q; two stages of each 226; this 220.)
      int nq = 0, ndo = 0, nrow = 0;                     // copies in flight so far
      for (int t = 0; t < nsteps; ++t) {
        const int h = kvh * p.g + (work.first + t) / work.per_head;
        const int i = i0 + (work.first + t) % work.per_head;
        const int sq = t % kStagesQ, sd = t % kStagesDO;
        if (t >= kStagesQ &&
            !wait_bounded(smem_addr(&sy.empty[sq]), (t / kStagesQ - 1) & 1, sy, p))
          break;
        auto do_free = [&]() {
          return t < kStagesDO ||
                 wait_bounded(smem_addr(&sy.do_empty[sd]), (t / kStagesDO - 1) & 1, sy, p);
        };
        if (!kApart && !do_free()) break;
        const uint32_t qbar = smem_addr(&sy.full[sq]);
        mbar_arrive_expect_tx(qbar, (kApart ? 1 : 2) * kTileBytes);
        for (int c = 0; c < D / 64; ++c)
          tma_load_4d(sQ0 + sq * kTileBytes + c * kT * 128, &tmQ, qbar, c * 64, h, i * kT, b);
        ++nq;
        if (kApart && !do_free()) break;
        const uint32_t dbar = kApart ? smem_addr(&sy.do_full[sd]) : qbar;
        if (kApart) {
          mbar_arrive_expect_tx(dbar, kTileBytes);
          ++ndo;
        }
        for (int c = 0; c < D / 64; ++c)
          tma_load_4d(sDO0 + sd * kTileBytes + c * kT * 128, &tmdO, dbar, c * 64, h, i * kT, b);
        // the statistics of step t - 2 have been read once its dK product was issued
        if (t >= 2 && !wait_bounded(smem_addr(&sy.empty[(t - 2) % kStagesQ]),
                                    ((t - 2) / kStagesQ) & 1, sy, p))
          break;
        const uint32_t rbar = smem_addr(&sy.row_full[t & 1]), row = sRow0 + (t & 1) * 1024;
        const size_t row0 = (static_cast<size_t>(b) * p.n_q + h) * (p.T * kT) + i * kT;
        mbar_arrive_expect_tx(rbar, 1024);
        bulk_load(row, p.nlse2 + row0, 512, rbar);
        bulk_load(row + 512, p.nrowdot + row0, 512, rbar);
        ++nrow;
      }
      wait_drain(fb, 0);
      drain_ring<kStagesQ>(sy.full, nq);
      drain_ring<kStagesDO>(sy.do_full, ndo);
      drain_ring<2>(sy.row_full, nrow);
    }
  } else if (warp == kMmaWarp) {
    const bool leader = elect_one();
    bool ok = __all_sync(0xffffffffu, wait_bounded(smem_addr(&sy.fixed_full), 0, sy, p));
    tc_fence_after_sync();
    auto q_of = [&](int t) { return sQ0 + (t % kStagesQ) * kTileBytes; };
    auto do_of = [&](int t) { return sDO0 + (t % kStagesDO) * kTileBytes; };
    auto wait_all = [&](uint64_t& bar, int use) -> bool {
      if (!__all_sync(0xffffffffu, wait_bounded(smem_addr(&bar), use & 1, sy, p))) return false;
      tc_fence_after_sync();
      return true;
    };
    auto wait_q = [&](int t) { return wait_all(sy.full[t % kStagesQ], t / kStagesQ); };
    auto wait_do = [&](int t) {
      return !kApart || wait_all(sy.do_full[t % kStagesDO], t / kStagesDO);
    };
    if (ok && (ok = wait_q(0))) {
      mma_scores_full_ss<D>(leader, tmem + cS, sK, q_of(0));                      // S^T  = K Q^T
      if (leader) mma_commit(smem_addr(&sy.s_full[0]));
      ok = wait_do(0);
      if (ok)
        mma_scores_full_ss<D>(leader, tmem + cP, sV, do_of(0));                   // dP^T = V dO^T
      if (leader) mma_commit(smem_addr(&sy.dp_full));
    }
    for (int t = 0; t < nsteps && ok; ++t) {
      const bool more = t + 1 < nsteps;
      if (more && !wait_q(t + 1)) break;
      if (!wait_all(sy.p_full[0], t)) break;
      mma_accum_full<D>(leader, tmem + cDV, tmem + cS, do_of(t), t > 0);         // dV += P^T dO
      if (leader) mma_commit(smem_addr(&sy.do_empty[t % kStagesDO]));
      // S^T(t+1) overwrites P^T(t), which the dV product issued above reads first
      if (more) {
        mma_scores_full_ss<D>(leader, tmem + cS, sK, q_of(t + 1));
        if (leader) mma_commit(smem_addr(&sy.s_full[0]));
        if (!wait_do(t + 1)) break;
      }
      if (!wait_all(sy.ds_full, t)) break;
      mma_accum_full<D>(leader, tmem + cDK, tmem + cP, q_of(t), t > 0);          // dK += dS^T Q
      if (leader) mma_commit(smem_addr(&sy.empty[t % kStagesQ]));
      if (more) {
        mma_scores_full_ss<D>(leader, tmem + cP, sV, do_of(t + 1));
        if (leader) mma_commit(smem_addr(&sy.dp_full));
      }
    }
    if (leader) mma_commit(smem_addr(&sy.done));
    teardown(sy, p, leader);
    return;
  } else if (warp < 4 * kComputeWGs) {
    // compute warpgroups: thread r = key row r of the tile = TMEM lane r;
    // warpgroup cw takes query columns [cw*kColsQ, cw*kColsQ + kColsQ) of a step
    const int cw = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const int krow = j * kT + r;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const size_t koff = ((static_cast<size_t>(b) * p.L + krow) * p.n_kv + kvh) * D;
    const uint64_t c2 = f32x2_pack(p.c, p.c);
    const int q0 = cw * kColsQ;                        // first query column (in the tile)
    bool ok = true;
    for (int t = 0; t < nsteps; ++t) {
      const int i = i0 + (work.first + t) % work.per_head;
      if (!__all_sync(0xffffffffu, wait_bounded(smem_addr(&sy.s_full[0]), t & 1, sy, p)) ||
          // the row statistics
          !__all_sync(0xffffffffu,
                      wait_bounded(smem_addr(&sy.row_full[t & 1]), (t >> 1) & 1, sy, p))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const float4* nl4 = reinterpret_cast<const float4*>(
          dyn_smem + (sRow0 + (t & 1) * 1024 - smem_addr(dyn_smem))) + q0 / 4;
      const float4* nd4 = nl4 + 32;
      const bool diag = p.causal && i == j;           // query c < key r is masked
      // phase 1: P^T from S^T, kept in registers for phase 2, and written (bf16)
      // over this warpgroup's first consumed S^T columns
      float pr[kColsQ];
      // the causal mask only touches the diagonal tile: a separate copy of the
      // loop keeps its compares and selects out of every other tile
      if (kWin && (i - j) * kT + kT - 1 >= p.window) {
        // rows that see key krow: all later ones of a sink, else those within W of it
        const int q_to_end = krow < p.sinks ? kT : krow + p.window - 1 - i * kT - q0;
        pt_from_st<true, true>(lane_base + cS + q0, nl4, c2, (i - j) * kT + q0 - r, q_to_end, pr);
      } else if (diag) {
        pt_from_st<true, false>(lane_base + cS + q0, nl4, c2, q0 - r, 0, pr);
      } else {
        pt_from_st<false, false>(lane_base + cS + q0, nl4, c2, q0 - r, 0, pr);
      }
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(smem_addr(&sy.p_full[0]));
      // phase 2: dS^T = P^T * (dP^T - D), over this warpgroup's consumed dP^T columns
      if (!__all_sync(0xffffffffu, wait_bounded(smem_addr(&sy.dp_full), t & 1, sy, p))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
#pragma unroll
      for (int cc = 0; cc < kColsQ / 32; ++cc) {
        uint32_t dpv[32];
        tmem_ld32(lane_base + cP + q0 + 32 * cc, dpv);
        tmem_wait_ld(dpv);
        uint32_t dk[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 nd = nd4[8 * cc + e];
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2) {
            const int jj = 4 * e + 2 * h2;
            const uint64_t dd = fadd2(
                f32x2_pack(__uint_as_float(dpv[jj]), __uint_as_float(dpv[jj + 1])),
                h2 ? f32x2_pack(nd.z, nd.w) : f32x2_pack(nd.x, nd.y));
            float d0, d1;
            f32x2_unpack(fmul2(f32x2_pack(pr[32 * cc + jj], pr[32 * cc + jj + 1]), dd), d0, d1);
            dk[jj / 2] = pack_bf16x2(d0, d1);
          }
        }
        tmem_st16(lane_base + cP + q0 + 16 * cc, dk);
      }
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(smem_addr(&sy.ds_full));
    }
    if (ok && __all_sync(0xffffffffu, wait_bounded(smem_addr(&sy.done), 0, sy, p))) {
      tc_fence_after_sync();
      const bool valid = krow < p.L;
      // 2*D/32 chunks of 32 columns (dV then dK) shared out over the warpgroups
      constexpr int kOut = 2 * D / 32, kPer = kOut / kComputeWGs, kHalfOut = D / 32;
#pragma unroll 1
      for (int q = cw * kPer; q < (cw + 1) * kPer; ++q) {
        const int col = (q % kHalfOut) * 32;
        if (kWin && work.pieces > 1) {
          // (rows past L are zeros: their keys are, and no row sees them)
          const size_t part = first_part(p, work.groups, grp, j) + work.piece;
          float* dst = p.parts + ((2 * part + (q < kHalfOut ? 0 : 1)) * kT + r) * D + col;
          store_chunk_f32(lane_base + (q < kHalfOut ? cDV : cDK) + col, dst, 1.0f);
          continue;
        }
        if (q < kHalfOut) store_chunk(lane_base + cDV + col, p.dv + koff + col, 1.0f, valid);
        else store_chunk(lane_base + cDK + col, p.dk + koff + col, p.dk_scale, valid);
      }
    }
  }
  teardown(sy, p, false);
}

// The parts of key tiles that several CTAs took, added in order of the pieces: a thread
// per four columns of one row of dV or dK. Tiles j0 .. j0 + tiles - 1 of each group,
// `pieces` each.
template <int D>
__global__ void __launch_bounds__(256)
join_kernel(const BwdParams p, int groups, int j0, int tiles, int pieces, long long items) {
  // (the grid before this one ends only once dK/dV has)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long item = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (item >= items) return;
  constexpr int kQuads = D / 4;
  const int col = static_cast<int>(item % kQuads) * 4;
  const int r = static_cast<int>(item / kQuads) % kT;
  const long long rest = item / (kQuads * kT);         // (tile, dV or dK)
  const int which = static_cast<int>(rest & 1);
  const long long tile = rest >> 1;
  const int j = j0 + static_cast<int>(tile % tiles);
  const long long grp = tile / tiles;
  const int row = j * kT + r;
  if (row >= p.L) return;
  const float* src = p.parts + ((2 * first_part(p, groups, grp, j) + which) * kT + r) * D + col;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int k = 0; k < pieces; ++k) {
    const float4 v = *reinterpret_cast<const float4*>(src + static_cast<size_t>(k) * 2 * kT * D);
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  const float mul = which ? p.dk_scale : 1.0f, zero = plus_zero(mul);
  const long long b = grp / p.n_kv, kvh = grp % p.n_kv;
  uint16_t* out = (which ? p.dk : p.dv) + ((b * p.L + row) * p.n_kv + kvh) * D + col;
  *reinterpret_cast<uint2*>(out) =
      make_uint2(pack_bf16x2(fmaf(sum.x, mul, zero), fmaf(sum.y, mul, zero)),
                 pack_bf16x2(fmaf(sum.z, mul, zero), fmaf(sum.w, mul, zero)));
}

// ------------------------------------------------------------------------ dQ

// dQ unit u (longest first): query tile i = T - 1 - u / groups of head
// (b, h) = u % groups, groups = B * n_q.
struct DqUnit {
  int b, h, i, n;
  SeenTiles seen;
};
template <bool kWin>
__device__ __forceinline__ DqUnit dq_unit(int u, const BwdParams& p) {
  const int groups = p.q_units / p.T;
  DqUnit x;
  x.i = p.T - 1 - u / groups;
  const int grp = u - (p.T - 1 - x.i) * groups;
  x.b = grp / p.n_q;
  x.h = grp - x.b * p.n_q;
  x.seen = seen_tiles<kWin>(x.i, p);
  x.n = x.seen.n;
  return x;
}

// Persistent: one CTA per SM walks the units in snake order (round r takes
// units r*G .. r*G+G-1, left to right on even rounds, right to left on odd
// ones), so each CTA's set-up happens once and the next unit's K/V tiles
// stream in while the current one drains.
__device__ __forceinline__ int dq_snake(int r) {
  const int G = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
  return r * G + ((r & 1) ? (G - 1 - c) : c);
}

template <int D, bool kWin>
__global__ void __launch_bounds__(kThreads, 1)
dq_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
          const __grid_constant__ CUtensorMap tmdO, const uint16_t* __restrict__ q_rows,
          const BwdParams p) {
  extern __shared__ uint8_t dyn_smem[];
  __shared__ Sync sy;
  // smem: dO_i | kStages x [K_t | V_t]
  constexpr int kTileBytes = tile_bytes<D>();
  const uint32_t base = (smem_addr(dyn_smem) + 1023u) & ~1023u;
  const uint32_t sdO = base, sRing = base + kTileBytes;
  constexpr uint32_t kStage = 2 * kTileBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = p.q_units;
  const int G = static_cast<int>(gridDim.x);
  setup(sy);
  const uint32_t tmem = sy.tmem_base;
  // TMEM columns: Q_i at 0 (D/2 columns, the A operand of S), S 64..191,
  // dP 192..319, dS 320..383 (bf16, two keys per column), dQ 384..511.
  // dP is read out before dS is formed and dS has its own columns, so per key
  // tile t the tensor cores run S(t+1) and dP(t+1) while the compute warps
  // still work on tile t, and dQ(t) as soon as dS(t) is in. Barrier phases
  // count tiles and units over the CTA's whole walk.
  constexpr uint32_t cQ = 0, cS = 64, cP = 192, cDS = 320, cDQ = 384;

  if (warp == kLoadWarp) {
    if (lane == 0) {
      const uint32_t fb = smem_addr(&sy.fixed_full);
      int it = 0, uc = 0;
      bool ok = true;
      for (int r = 0; r * G < units && ok; ++r) {
        const int u = dq_snake(r);
        if (u >= units) continue;
        const DqUnit x = dq_unit<kWin>(u, p);
        const int kvh = x.h / p.g;
        // The unit's first K/V tile, then dO_i, whose buffer is free once the last product
        // with the dO of the unit before is done (its dQ products may still run), then
        // the other tiles.
        for (int t = 0; t < x.n; ++t, ++it) {
          const int st = it % kStages, use = it / kStages;
          if (use > 0 && !wait_bounded(smem_addr(&sy.empty[st]), (use - 1) & 1, sy, p)) {
            ok = false;
            break;
          }
          const uint32_t dst = sRing + st * kStage, bar = smem_addr(&sy.full[st]);
          mbar_arrive_expect_tx(bar, 2 * kTileBytes);
          const int key0 = seen_tile<kWin>(x.seen, t) * kT;
          for (int c = 0; c < D / 64; ++c) {
            tma_load_4d(dst + c * kT * 128, &tmK, bar, c * 64, kvh, key0, x.b);
            tma_load_4d(dst + kTileBytes + c * kT * 128, &tmV, bar, c * 64, kvh, key0, x.b);
          }
          if (t == 0) {
            if (uc > 0 && !wait_bounded(smem_addr(&sy.do_free), (uc - 1) & 1, sy, p)) {
              ok = false;
              ++it;
              break;
            }
            mbar_arrive_expect_tx(fb, kTileBytes);
            for (int c = 0; c < D / 64; ++c)
              tma_load_4d(sdO + c * kT * 128, &tmdO, fb, c * 64, x.h, x.i * kT, x.b);
            ++uc;
          }
        }
      }
      if (uc > 0) wait_drain(fb, (uc - 1) & 1);
      drain_ring<kStages>(sy.full, it);
    }
  } else if (warp == kMmaWarp) {
    const bool leader = elect_one();
    int it = 0, gt = 0, uc = 0;      // ring items, tiles, units consumed so far
    bool ok = true;
    auto wait_all = [&](uint64_t& bar, int ph) -> bool {
      if (!__all_sync(0xffffffffu, wait_bounded(smem_addr(&bar), ph & 1, sy, p))) return false;
      tc_fence_after_sync();
      return true;
    };
    for (int r = 0; r * G < units && ok; ++r) {
      const int u = dq_snake(r);
      if (u >= units) continue;
      const int n = dq_unit<kWin>(u, p).n;
      auto stage_of = [&](int t) { return sRing + ((it + t) % kStages) * kStage; };
      auto wait_stage = [&](int t) -> bool {
        return wait_all(sy.full[(it + t) % kStages], (it + t) / kStages);
      };
      // Q_i in TMEM (compute threads) and dO_i in shared memory
      if (!wait_all(sy.a_ready, uc) || !wait_all(sy.fixed_full, uc) || !wait_stage(0)) {
        ok = false;
        break;
      }
      mma_scores_full<D>(leader, tmem + cS, tmem + cQ, stage_of(0));           // S  = Q K^T
      if (leader) mma_commit(smem_addr(&sy.s_full[0]));
      mma_scores_full_ss<D>(leader, tmem + cP, sdO, stage_of(0) + kTileBytes);  // dP = dO V^T
      if (leader) mma_commit(smem_addr(&sy.dp_full));
      if (leader && n == 1) mma_commit(smem_addr(&sy.do_free));
      for (int t = 0; t < n; ++t) {
        const bool more = t + 1 < n;
        // S(t) read out: the next tile's scores may overwrite it
        if (!wait_all(sy.p_full[0], gt + t)) { ok = false; break; }
        if (more) {
          if (!wait_stage(t + 1)) { ok = false; break; }
          mma_scores_full<D>(leader, tmem + cS, tmem + cQ, stage_of(t + 1));
          if (leader) mma_commit(smem_addr(&sy.s_full[0]));
        }
        // dP(t) read out: the next tile's dP may overwrite it
        if (!wait_all(sy.dp_free, gt + t)) { ok = false; break; }
        if (more) {
          mma_scores_full_ss<D>(leader, tmem + cP, sdO, stage_of(t + 1) + kTileBytes);
          if (leader) mma_commit(smem_addr(&sy.dp_full));
          if (leader && t + 2 == n) mma_commit(smem_addr(&sy.do_free));
        }
        if (!wait_all(sy.ds_full, gt + t)) { ok = false; break; }
        mma_accum_dq<D>(leader, tmem + cDQ, tmem + cDS, stage_of(t), t > 0);      // dQ += dS K
        if (leader) mma_commit(smem_addr(&sy.dq_done));
        if (leader) mma_commit(smem_addr(&sy.empty[(it + t) % kStages]));
      }
      if (!ok) break;
      if (leader) mma_commit(smem_addr(&sy.done));
      it += n;
      gt += n;
      ++uc;
    }
    teardown(sy, p, leader);
    return;
  } else if (warp < 4 * kComputeWGs) {
    // compute warpgroups: thread r = query row r of the tile = TMEM lane r;
    // warpgroup cw takes key columns [cw*kColsQ, cw*kColsQ + kColsQ)
    const int cw = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint64_t c2 = f32x2_pack(p.c, p.c);
    const int k0 = cw * kColsQ;                        // first key column (in the tile)
    int gt = 0, uc = 0, rr = 0;
    bool ok = true;
    // the CTA's next unit, if there is one
    auto next_unit = [&](DqUnit& x) {
      for (; rr * G < units; ++rr) {
        const int u = dq_snake(rr);
        if (u < units) {
          ++rr;
          x = dq_unit<kWin>(u, p);
          return true;
        }
      }
      return false;
    };
    // Q_i becomes the A operand of S in TMEM (64 channels per warpgroup); the last scores
    // with the Q there have been read by the time this is called
    float nl = 0.0f, nd = 0.0f;
    auto bring_q = [&](const DqUnit& x) {
      const int row = x.i * kT + r;
      const size_t qoff = ((static_cast<size_t>(x.b) * p.L + row) * p.n_q + x.h) * D;
      if (64 * cw < D) row_to_tmem<64>(lane_base + cQ + 32 * cw, q_rows + qoff + 64 * cw, row < p.L);
      const size_t srow = (static_cast<size_t>(x.b) * p.n_q + x.h) * (p.T * kT) + row;
      nl = p.nlse2[srow];
      // a row that sees one key: P, which is for dS alone here, is 0
      if (row < p.one_key_rows) nl -= INFINITY;
      nd = p.nrowdot[srow];
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(smem_addr(&sy.a_ready));
    };
    DqUnit x, y;
    bool more = next_unit(x);
    if (more) bring_q(x);
    while (more) {
      const int i = x.i, n = x.n;
      const int row = i * kT + r;
      const size_t qoff = ((static_cast<size_t>(x.b) * p.L + row) * p.n_q + x.h) * D;
      const uint64_t nl2 = f32x2_pack(nl, nl), nd2 = f32x2_pack(nd, nd);
      for (int t = 0; t < n; ++t) {
        // phase 1: P from S, kept in registers
        if (!__all_sync(0xffffffffu, wait_bounded(smem_addr(&sy.s_full[0]), (gt + t) & 1, sy, p))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        // keys after `keep` (in-tile) are masked: the diagonal tile, or keys past L
        const bool masked = p.causal ? (t == i) : (p.L - t * kT < kT);
        const int keep = p.causal ? r : p.L - 1 - t * kT;
        float pr[kColsQ];
        const int ahead = i - seen_tile<kWin>(x.seen, t);    // tiles from the key tile to the row's
        if (kWin && ahead * kT + kT - 1 >= p.window)
          p_from_s<true, true>(lane_base + cS + k0, c2, nl2, k0, ahead * kT + r,
                               ahead * kT + r - p.window, p.sinks - (i - ahead) * kT, pr);
        else if (kWin ? ahead == 0 : masked)
          p_from_s<true, false>(lane_base + cS + k0, c2, nl2, k0, keep, 0, 0, pr);
        else
          p_from_s<false, false>(lane_base + cS + k0, c2, nl2, k0, keep, 0, 0, pr);
        tc_fence_before_sync();
        mbar_arrive(smem_addr(&sy.p_full[0]));
        // phase 2: dP read out (its columns are then free for the next tile),
        // dS = P * (dP - D) into the dS columns once dQ(t-1) has read them
        if (!__all_sync(0xffffffffu, wait_bounded(smem_addr(&sy.dp_full), (gt + t) & 1, sy, p))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        uint32_t dk[kColsQ / 2];
#pragma unroll
        for (int c = 0; c < kColsQ / 32; ++c) {
          uint32_t dpv[32];
          tmem_ld32(lane_base + cP + k0 + 32 * c, dpv);
          tmem_wait_ld(dpv);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint64_t dd = fadd2(
                f32x2_pack(__uint_as_float(dpv[2 * e]), __uint_as_float(dpv[2 * e + 1])), nd2);
            float d0, d1;
            f32x2_unpack(fmul2(f32x2_pack(pr[32 * c + 2 * e], pr[32 * c + 2 * e + 1]), dd), d0, d1);
            dk[16 * c + e] = pack_bf16x2(d0, d1);
          }
        }
        tc_fence_before_sync();
        mbar_arrive(smem_addr(&sy.dp_free));
        if (t > 0 && !__all_sync(0xffffffffu, wait_bounded(smem_addr(&sy.dq_done), (gt + t - 1) & 1, sy, p))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
#pragma unroll
        for (int c = 0; c < kColsQ / 32; ++c)
          tmem_st16(lane_base + cDS + k0 / 2 + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(dk + 16 * c));
        tmem_wait_st();
        tc_fence_before_sync();
        mbar_arrive(smem_addr(&sy.ds_full));
      }
      if (!ok) break;
      // the next unit's Q goes in while this one's last product runs, so that its first
      // scores do while this one's dQ is stored
      more = next_unit(y);
      if (more) bring_q(y);
      if (!__all_sync(0xffffffffu, wait_bounded(smem_addr(&sy.done), uc & 1, sy, p))) break;
      tc_fence_after_sync();
      constexpr int kPer = (D / 32) / kComputeWGs;    // chunks of 32 dQ columns per warpgroup
#pragma unroll 1
      for (int q = cw * kPer; q < (cw + 1) * kPer; ++q)
        store_chunk(lane_base + cDQ + 32 * q, p.dq + qoff + 32 * q, p.scale, row < p.L);
      gt += n;
      ++uc;
      x = y;
    }
  }
  teardown(sy, p, false);
  // This grid started while dK/dV still ran (it reads nothing dK/dV writes);
  // it ends only once dK/dV has ended (one waiting thread keeps the CTA
  // alive; every thread waiting cost 1.4 %), so that a programmatic dependent
  // of this grid (the stream's next kernel) finds dK and dV complete as well.
  if (threadIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// --------------------------------------------------------------------- host

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
constexpr int kMaxDevices = 64;
std::mutex g_bwd_mutex;
bool g_bwd_ready[kMaxDevices];
EncodeTiledFn g_bwd_encode = nullptr;
template <int D>
constexpr int dq_smem() { return tile_bytes<D>() + kStages * (2 * tile_bytes<D>()) + 1024; }

template <int D, bool kWin>
bool set_smem() {
  return cudaFuncSetAttribute(dkdv_kernel<D, kWin>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              dkdv_smem<D>()) == cudaSuccess &&
         cudaFuncSetAttribute(dq_kernel<D, kWin>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              dq_smem<D>()) == cudaSuccess;
}

attn_status_t bwd_device_ready(cudaStream_t stream, int** status) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_UNSUPPORTED;
  // device check, tensor-map encoder and status word come from the forward's set-up
  const attn_status_t ds = gb300_host::device_status_word(stream, status);
  if (ds != ATTN_OK) return ds;
  std::lock_guard<std::mutex> lock(g_bwd_mutex);
  if (!g_bwd_ready[dev]) {
    // one-time set-up: not inside a stream capture
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess || cs != cudaStreamCaptureStatusNone) {
      cudaGetLastError();
      return ATTN_ERR_UNSUPPORTED;
    }
    if (!g_bwd_encode) {
      cudaDriverEntryPointQueryResult q;
      void* fn = nullptr;
      if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                           cudaEnableDefault, &q) != cudaSuccess ||
          q != cudaDriverEntryPointSuccess || fn == nullptr)
        return ATTN_ERR_CUDA;
      g_bwd_encode = reinterpret_cast<EncodeTiledFn>(fn);
    }
    if (!set_smem<128, false>() || !set_smem<64, false>() || !set_smem<128, true>() ||
        !set_smem<64, true>())
      return ATTN_ERR_CUDA;
    g_bwd_ready[dev] = true;
  }
  return ATTN_OK;
}

// dK/dV is launched as the row kernel's programmatic dependent: its CTAs set
// up while the row kernel finishes and wait for it before reading anything.
template <int D, bool kWin>
cudaError_t launch_dkdv(unsigned grid, cudaStream_t stream, const CUtensorMap& mq,
                        const CUtensorMap& mdo, const CUtensorMap& mk, const CUtensorMap& mv,
                        const BwdParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = dkdv_smem<D>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dkdv_kernel<D, kWin>, mq, mdo, mk, mv, p);
}

// dQ is launched as the dK/dV kernel's programmatic dependent: it reads only
// the inputs and the row statistics (complete once dK/dV's CTAs are past their
// wait, which is when they let dQ launch), so it needs no grid-dependency wait
// and its persistent CTAs take the SMs that dK/dV's last CTAs free.
template <int D, bool kWin>
cudaError_t launch_dq(unsigned grid, cudaStream_t stream, const CUtensorMap& mk,
                      const CUtensorMap& mv, const CUtensorMap& mdo, const uint16_t* qh,
                      const BwdParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = dq_smem<D>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dq_kernel<D, kWin>, mk, mv, mdo, qh, p);
}

// The join is dQ's programmatic dependent: it waits until that grid, and with it
// dK/dV, has ended.
template <int D>
cudaError_t launch_join(cudaStream_t stream, const BwdParams& p, int groups, int j0, int tiles,
                        int pieces) {
  const long long items = static_cast<long long>(groups) * tiles * 2 * kT * (D / 4);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((items + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D>, p, groups, j0, tiles, pieces, items);
}

bool encode_tile_map(CUtensorMap* map, const void* ptr, int D, int H, int64_t L, int64_t B) {
  const cuuint64_t d = static_cast<cuuint64_t>(D);
  const cuuint64_t dims[4] = {d, static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(L),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {d * 2, static_cast<cuuint64_t>(H) * d * 2,
                                 static_cast<cuuint64_t>(L) * H * d * 2};
  const cuuint32_t box[4] = {64, 1, kT, 1};
  const cuuint32_t estride[4] = {1, 1, 1, 1};
  return g_bwd_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims,
                      strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t row_blocks_of(int64_t B, int64_t T, int64_t n_q) {
  return B * ((n_q + kRowdotH - 1) / kRowdotH) * ((T * kT / 8) >> row_doublings(n_q));
}

// 32-bit tile indexing, and the row kernel's grid
bool sizes_fit(int64_t B, int64_t L, int32_t n_q, int32_t n_kv) {
  const int64_t T = (L + kT - 1) / kT;
  return L <= (int64_t{1} << 30) && B <= INT32_MAX && B * n_q <= INT32_MAX &&
         B * n_kv * T <= INT32_MAX && B * n_q * T <= INT32_MAX / 4 &&
         row_blocks_of(B, T, n_q) <= INT32_MAX;
}

// Row statistics of a call, in bytes: two fp32 per query row, rows padded to tiles.
int64_t row_bytes(int64_t B, int64_t L, int32_t n_q) {
  return 2 * B * n_q * ((L + kT - 1) / kT) * kT * 4;
}

// Into how many CTAs key tiles are cut. Those that hold a sink meet every later query
// tile, up to T * g steps where the others take about W / 128 * g: left whole, the
// few of them would run on long after the rest. A piece is at least as long as
// another tile's CTA, and all pieces together are about two per SM, which also
// bounds the parts' memory (128 KiB each at d_h = 128). The other tiles are cut where
// that fills SMs that would be idle: a CTA costs about nine steps beside its own, so of
// 1, 2, 3 ... pieces the number with the shortest rounds is taken (1000 rows of 8
// heads on 2 behind 256: 16 CTAs of 12 steps 22 us, 64 of 3 and the join 15). A
// rule on the shape alone, not on the device, so that the workspace's size is.
struct KeySplit {
  int64_t heavy, pieces, others, bytes;
};
KeySplit key_split(int64_t B, int64_t L, int32_t n_q, int32_t n_kv, int32_t d_h, int64_t window,
                   int64_t sinks) {
  constexpr int64_t kSms = 152, kCtaSteps = 9, kJoinSteps = 4;
  const int64_t T = (L + kT - 1) / kT, g = n_q / n_kv, groups = B * n_kv;
  window = window < L ? window : L;
  sinks = sinks < L ? sinks : L;
  KeySplit s{window < L ? (sinks + kT - 1) / kT : 0, 1, 1, 0};
  const int64_t reach = (window + kT - 2) / kT + 1, steps = g * (reach < T ? reach : T);
  if (s.heavy > 0) {
    const int64_t most = g * T / (steps > 8 ? steps : 8);
    const int64_t fill = 2 * kSms / (groups * s.heavy);
    s.pieces = most < fill ? most : fill;
    const int64_t least = g * (T - s.heavy + 1);          // steps of the shortest such tile
    if (s.pieces > least) s.pieces = least;
    if (s.pieces < 1) s.pieces = 1;
  }
  const int64_t ctas = groups * (T - s.heavy);
  if (ctas > 0 && ctas < kSms && window < L) {
    int64_t best = 0;
    for (int64_t n = 1; n <= g && n * ctas <= 2 * kSms; ++n) {   // (a tile has g steps at least)
      const int64_t rounds = (n * ctas + kSms - 1) / kSms;
      const int64_t cost = rounds * ((steps + n - 1) / n + kCtaSteps) + (n > 1 ? kJoinSteps : 0);
      if (n == 1 || cost < best) {
        best = cost;
        s.others = n;
      }
    }
  }
  const int64_t parts = (s.pieces > 1 ? groups * s.heavy * s.pieces : 0) +
                        (s.others > 1 ? ctas * s.others : 0);
  s.bytes = parts * 2 * kT * d_h * 4;
  return s;
}

template <int D, bool kWin>
attn_status_t launch_all(cudaStream_t stream, unsigned row_blocks, unsigned kv_ctas,
                         unsigned dq_grid, const uint16_t* o, const uint16_t* dout,
                         const float* lse, const uint16_t* q, float* nlse2, float* nrowdot, int B,
                         const CUtensorMap& mq, const CUtensorMap& mdo, const CUtensorMap& mk,
                         const CUtensorMap& mv, const BwdParams& p) {
  constexpr decltype(&rowdot_kernel<D, 0>) kRows[4] = {rowdot_kernel<D, 0>, rowdot_kernel<D, 1>,
                                                       rowdot_kernel<D, 2>, rowdot_kernel<D, 3>};
  kRows[row_doublings(p.n_q)]<<<row_blocks, 256, 0, stream>>>(o, dout, lse, nlse2, nrowdot, p.L,
                                                              p.n_q, p.T * kT);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  if (launch_dkdv<D, kWin>(kv_ctas, stream, mq, mdo, mk, mv, p) != cudaSuccess)
    return ATTN_ERR_CUDA;
  if (launch_dq<D, kWin>(dq_grid, stream, mk, mv, mdo, q, p) != cudaSuccess) return ATTN_ERR_CUDA;
  const int groups = B * p.n_kv;
  if (kWin && p.pieces > 1 &&
      launch_join<D>(stream, p, groups, 0, p.heavy, p.pieces) != cudaSuccess)
    return ATTN_ERR_CUDA;
  if (kWin && p.others > 1 &&
      launch_join<D>(stream, p, groups, p.heavy, p.T - p.heavy, p.others) != cudaSuccess)
    return ATTN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// window > 0: the windowed instances (causal). Both entry points' checks and launches.
attn_status_t backward(const void* q, const void* k, const void* v, const void* o,
                       const float* lse, const void* dout, void* dq, void* dk, void* dv,
                       void* workspace, int64_t workspace_bytes, int64_t B, int64_t L, int32_t n_q,
                       int32_t n_kv, int32_t d_h, int32_t causal, int64_t window, int64_t sinks,
                       float scale, void* stream_ptr) {
  if (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || !workspace)
    return ATTN_ERR_INVALID_ARG;
  if (B < 1 || L < 1 || n_q < 1 || n_kv < 1 || n_q % n_kv != 0) return ATTN_ERR_INVALID_ARG;
  if ((causal != 0 && causal != 1) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  auto misaligned = [](const void* ptr, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0;
  };
  if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) ||
      misaligned(dout, 16) || misaligned(dq, 16) || misaligned(dk, 16) || misaligned(dv, 16) ||
      misaligned(lse, 4) || misaligned(workspace, 16))
    return ATTN_ERR_INVALID_ARG;
  if (d_h != 64 && d_h != 128) return ATTN_ERR_UNSUPPORTED;
  const int64_t T = (L + kT - 1) / kT;
  if (!sizes_fit(B, L, n_q, n_kv)) return ATTN_ERR_UNSUPPORTED;
  const bool win = window > 0;
  const KeySplit split =
      win ? key_split(B, L, n_q, n_kv, d_h, window, sinks) : KeySplit{0, 1, 1, 0};
  if (workspace_bytes < row_bytes(B, L, n_q) + split.bytes) return ATTN_ERR_INVALID_ARG;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  int* status = nullptr;
  const attn_status_t ds = bwd_device_ready(stream, &status);
  if (ds != ATTN_OK) return ds;

  CUtensorMap mq, mk, mv, mdo;
  if (!encode_tile_map(&mq, q, d_h, n_q, L, B) || !encode_tile_map(&mk, k, d_h, n_kv, L, B) ||
      !encode_tile_map(&mv, v, d_h, n_kv, L, B) || !encode_tile_map(&mdo, dout, d_h, n_q, L, B))
    return ATTN_ERR_CUDA;
  BwdParams p{};
  p.L = static_cast<int>(L);
  p.n_q = n_q;
  p.n_kv = n_kv;
  p.g = n_q / n_kv;
  p.T = static_cast<int>(T);
  p.causal = causal;
  p.c = scale * kLog2e;
  p.scale = scale;
  float* nlse2 = static_cast<float*>(workspace);
  float* nrowdot = nlse2 + B * n_q * T * kT;
  p.nlse2 = nlse2;
  p.nrowdot = nrowdot;
  p.dq = static_cast<uint16_t*>(dq);
  p.dk = static_cast<uint16_t*>(dk);
  p.dv = static_cast<uint16_t*>(dv);
  p.status = status;
  p.q_units = static_cast<int>(B * n_q * T);
  const bool all_one = L == 1 || (win && window == 1 && sinks == 0);
  p.one_key_rows = all_one ? p.L : causal ? 1 : 0;
  p.dk_scale = all_one ? 0.0f : scale;
  p.window = static_cast<int>(window < L ? window : L);
  p.sinks = static_cast<int>(sinks < L ? sinks : L);
  p.heavy = static_cast<int>(split.heavy);
  p.pieces = static_cast<int>(split.pieces);
  p.others = static_cast<int>(split.others);
  p.parts = nrowdot + B * n_q * T * kT;

  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
    sms = 1;
  const unsigned row_blocks = static_cast<unsigned>(row_blocks_of(B, T, n_q));
  const uint16_t* oh = static_cast<const uint16_t*>(o);
  const uint16_t* qh = static_cast<const uint16_t*>(q);
  const uint16_t* doh = static_cast<const uint16_t*>(dout);
  const unsigned kv_ctas =
      static_cast<unsigned>(B * n_kv * ((T - split.heavy) * split.others + split.heavy * split.pieces));
  const unsigned dq_grid = static_cast<unsigned>(B * n_q * T < sms ? B * n_q * T : sms);
  const int batch = static_cast<int>(B);
  if (d_h == 128)
    return win ? launch_all<128, true>(stream, row_blocks, kv_ctas, dq_grid, oh, doh, lse, qh,
                                       nlse2, nrowdot, batch, mq, mdo, mk, mv, p)
               : launch_all<128, false>(stream, row_blocks, kv_ctas, dq_grid, oh, doh, lse, qh,
                                        nlse2, nrowdot, batch, mq, mdo, mk, mv, p);
  return win ? launch_all<64, true>(stream, row_blocks, kv_ctas, dq_grid, oh, doh, lse, qh, nlse2,
                                    nrowdot, batch, mq, mdo, mk, mv, p)
             : launch_all<64, false>(stream, row_blocks, kv_ctas, dq_grid, oh, doh, lse, qh, nlse2,
                                     nrowdot, batch, mq, mdo, mk, mv, p);
}

}  // namespace

extern "C" {

int64_t attn_prefill_bwd_workspace_bytes(int64_t B, int64_t L, int32_t n_q, int32_t n_kv,
                                         int32_t d_h) {
  if (B < 1 || L < 1 || n_q < 1 || n_kv < 1 || n_q % n_kv != 0 || (d_h != 64 && d_h != 128)) return -1;
  return row_bytes(B, L, n_q);
}

attn_status_t attn_prefill_bwd(const void* q, const void* k, const void* v, const void* o,
                               const float* lse, const void* dout, void* dq, void* dk, void* dv,
                               void* workspace, int64_t workspace_bytes, int64_t B, int64_t L,
                               int32_t n_q, int32_t n_kv, int32_t d_h, int32_t causal,
                               float scale, void* stream_ptr) {
  return backward(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes, B, L, n_q, n_kv,
                  d_h, causal, 0, 0, scale, stream_ptr);
}

int64_t attn_prefill_window_bwd_workspace_bytes(int64_t B, int64_t L, int32_t n_q, int32_t n_kv,
                                                int32_t d_h, int64_t window, int64_t sinks) {
  if (B < 1 || L < 1 || n_q < 1 || n_kv < 1 || n_q % n_kv != 0 || (d_h != 64 && d_h != 128) ||
      window < 1 || sinks < 0 || !sizes_fit(B, L, n_q, n_kv))
    return -1;
  return row_bytes(B, L, n_q) + key_split(B, L, n_q, n_kv, d_h, window, sinks).bytes;
}

attn_status_t attn_prefill_window_bwd(const void* q, const void* k, const void* v, const void* o,
                                      const float* lse, const void* dout, void* dq, void* dk,
                                      void* dv, void* workspace, int64_t workspace_bytes, int64_t B,
                                      int64_t L, int32_t n_q, int32_t n_kv, int32_t d_h,
                                      int64_t window, int64_t sinks, float scale,
                                      void* stream_ptr) {
  if (window < 1 || sinks < 0) return ATTN_ERR_INVALID_ARG;
  return backward(q, k, v, o, lse, dout, dq, dk, dv, workspace, workspace_bytes, B, L, n_q, n_kv,
                  d_h, 1, window, sinks, scale, stream_ptr);
}

}  // extern "C"
