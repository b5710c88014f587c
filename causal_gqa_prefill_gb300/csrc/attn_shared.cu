// attn_shared.cu — decode for a batch whose sequences share a long prefix, on
// GB300 (sm_103a): one new token per sequence attends to P positions that are
// stored once for the whole batch and to lens[b] positions of its own.
//
// The batch's B * g query rows of a K/V head all read the same prefix, so over
// the prefix the step is a matrix product: 4 d flops per row and position, B g
// rows for every 512 bytes of K and V. (Each sequence reading its own copy would
// be bound by memory at B times the bytes.) The own positions have g rows per
// sequence and stay bound by memory; the decode step's ragged split kernel
// takes them. The two softmaxes are joined through their maxima and sums.
//
//   prefix kernel  persistent, one CTA per SM. 128 rows of one K/V head are one
//                  tile (128 / g sequences, all heads of the group: one TMA box);
//                  a unit is two row tiles of the same head that share every K/V
//                  tile, and the key tiles of all units are cut into equal ranges,
//                  one per CTA. A range is one segment per unit it touches. Rows
//                  on the TMEM lanes, S = Q K^T and O += P V on tcgen05, P in
//                  TMEM, one softmax thread per row (no reduction over threads):
//                  the two row tiles take turns on the tensor cores. Where a unit
//                  has one row tile, its two softmax warpgroups take its even and
//                  its odd key tiles instead, so the turns stay.
//                  Every segment leaves an fp32 partial output, four dimensions of
//                  128 rows at a time (whole 512-byte stores from one-row
//                  threads), and its rows' running maxima and sums.
//   ragged split   (attn_decode.cu) starts on the SMs that the prefix kernel
//                  leaves free, without waiting for it.
//   combine        one thread per row and eight dimensions: merges the row's
//                  partials of both kernels into bf16 O and fp32 LSE.
//
// Measured, 256 sequences of 64 heads on 8 behind 32768 positions, up to 1024 own
// ones: prefix 181 us (1.52 PFLOP/s; bound by the tensor cores and the softmax's
// turns), own positions 105 (609 MB, 5.8 TB/s), merge 16; 294 for the call. 64
// sequences of 32 heads behind 8192, up to 512 own: 17, 22 and 12 when timed one
// by one, each mostly start-up, and 44 for the call. The own positions on half to
// three quarters of the SMs beside the prefix kernel on the rest were no faster
// (334 and more; the prefix reads each K/V tile for every row tile pair at another
// time, 1.06 GB from memory, so both then wait for memory).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "attn_prefill.h"
#include "decode_parts.h"
#include "sm103_ptx.cuh"

namespace {

using namespace gb300;

constexpr int kDim = 128;
constexpr int kRows = 128;            // query rows per tile (TMEM lanes)
constexpr int kKeys = 128;            // keys per tile
constexpr int kCtas = 152;            // one CTA per SM on a 152-SM GB300
constexpr int kThreads = 384;
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;   // registers per thread
constexpr int kRegBudget = 2 * 128 * kSoftmaxRegs + 128 * kOtherRegs;
static_assert(kRegBudget <= kThreads * 168, "setmaxnreg split exceeds the launch allocation");
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr int kRing = 5;              // K/V ring slots (K and V tiles alternate)
constexpr int kTileBytes = 128 * kDim * 2;    // 32 KiB: two 128 x 64 swizzled chunks
constexpr int kChunkBytes = 128 * 128;
constexpr int kSmemBytes = (2 + kRing) * kTileBytes + 1024;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescale = 8.0f;      // lazy running-max threshold (log2 units)
constexpr int kStatusTimeout = 1;
constexpr int kPartFloats = kDim * kRows;     // one row tile's partial output

struct Params {
  float* part_o;         // [2 * (units + G)][32][128][4]
  float2* part_ml;       // [2 * (units + G)][128] running maximum (log2 units) and sum
  int* status;
  int P, T;              // prefix positions and key tiles
  int B, n_q, n_kv, g;
  int nb;                // sequences per row tile: 128 / g
  int tiles, pairs;      // row tiles and units per K/V head
  int units, G;
  long long W;           // units * T
  float c;               // scale * log2(e)
  long long spin_limit;
};

struct Ctl {
  uint64_t full[kRing], empty[kRing];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

__host__ __device__ __forceinline__ long long range_start(long long c, long long W, long long G) {
  return c * W / G;
}
__host__ __device__ __forceinline__ long long cta_of(long long x, long long W, long long G) {
  return ((x + 1) * G - 1) / W;
}

// Key tiles [t0, t0 + n) of a unit; `both`: it has two row tiles.
struct Segment {
  int unit, kvh, tile0, t0, n;
  bool both;
  // how many of the key tiles warpgroup `slot` takes, and which
  __device__ int count(int slot) const { return both ? n : (n + 1 - slot) >> 1; }
  __device__ int tile(int slot, int j) const { return t0 + (both ? j : 2 * j + slot); }
};

struct Walk {
  const Params& p;
  long long x, end;
  __device__ Walk(const Params& params, int c)
      : p(params), x(range_start(c, params.W, params.G)),
        end(range_start(c + 1, params.W, params.G)) {}
  __device__ bool next(Segment& s) {
    if (x >= end) return false;
    const long long unit = x / p.T, base = unit * p.T;
    const long long t1 = end - base < p.T ? end - base : p.T;
    s.unit = static_cast<int>(unit);
    s.kvh = s.unit / p.pairs;
    s.tile0 = 2 * (s.unit - s.kvh * p.pairs);
    s.both = s.tile0 + 1 < p.tiles;
    s.t0 = static_cast<int>(x - base);
    s.n = static_cast<int>(t1 - (x - base));
    x = base + t1;
    return true;
  }
};

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

// S[128 rows x 128 keys] = Q K^T, both K-major in shared memory.
__device__ __forceinline__ void issue_qk(bool leader, uint32_t d_tmem, uint32_t q_smem,
                                         uint32_t k_smem) {
  constexpr uint32_t idesc = idesc_bf16_f32(kRows, kKeys, false);
  const uint64_t a0 = sdesc_sw128(q_smem, 16, 1024), b0 = sdesc_sw128(k_smem, 16, 1024);
#pragma unroll
  for (int kk = 0; kk < kDim / 16; ++kk) {
    const uint32_t off = ((kk >> 2) * kChunkBytes + (kk & 3) * 32) >> 4;
    if (leader) mma_ss(d_tmem, a0 + off, b0 + off, idesc, kk > 0 ? 1u : 0u);
  }
}

// O[128 rows x 128] (+)= P V: P bf16 in TMEM (two keys per column), V MN-major.
__device__ __forceinline__ void issue_pv(bool leader, uint32_t d_tmem, uint32_t p_tmem,
                                         uint32_t v_smem, bool accumulate) {
  constexpr uint32_t idesc = idesc_bf16_f32(kRows, kDim, true);
  const uint64_t b0 = sdesc_sw128(v_smem, kChunkBytes, 1024);
#pragma unroll
  for (int kk = 0; kk < kKeys / 16; ++kk)
    if (leader)
      mma_ts(d_tmem, p_tmem + 8 * kk, b0 + ((kk * 16 * 128) >> 4), idesc,
             (accumulate || kk > 0) ? 1u : 0u);
}

__device__ void load_role(const CUtensorMap* tmQ, const CUtensorMap* tmK, const CUtensorMap* tmV,
                          Ctl& ctl, const Params& p, uint32_t sQ, uint32_t sKV) {
  Walk walk(p, blockIdx.x);
  Segment sg;
  uint32_t it = 0, qn = 0;
  bool ok = true;
  const uint32_t q_bytes = static_cast<uint32_t>(2 * 128 * p.g * p.nb);
  const uint32_t qbar = smem_addr(&ctl.q_full);
  while (ok && walk.next(sg)) {
    if (qn > 0 && !spin_wait(smem_addr(&ctl.q_empty), (qn - 1) & 1, ctl, p)) {
      ok = false;
      break;
    }
    const int tiles = sg.both ? 2 : 1;
    mbar_arrive_expect_tx(qbar, tiles * q_bytes);
    for (int s = 0; s < tiles; ++s)
      for (int ch = 0; ch < 2; ++ch)
        tma_load_3d(sQ + s * kTileBytes + ch * kChunkBytes, tmQ, qbar, ch * 64, sg.kvh * p.g,
                    (sg.tile0 + s) * p.nb);
    ++qn;
    for (int t = 0; t < sg.n && ok; ++t) {
      for (int kind = 0; kind < 2; ++kind) {
        const uint32_t slot = it % kRing, use = it / kRing;
        if (use > 0 && !spin_wait(smem_addr(&ctl.empty[slot]), (use - 1) & 1, ctl, p)) {
          ok = false;
          break;
        }
        const uint32_t bar = smem_addr(&ctl.full[slot]);
        mbar_arrive_expect_tx(bar, kTileBytes);
        for (int ch = 0; ch < 2; ++ch)
          tma_load_3d(sKV + slot * kTileBytes + ch * kChunkBytes, kind ? tmV : tmK, bar, ch * 64,
                      sg.kvh, (sg.t0 + t) * kKeys);
        ++it;
      }
    }
  }
  // let every copy this thread started land before the CTA can exit, also where
  // another role has given up
  if (qn) drain_wait(qbar, (qn - 1) & 1, p);
  for (uint32_t s = 0; s < kRing && s < it; ++s)
    drain_wait(smem_addr(&ctl.full[s]), ((it - 1 - s) / kRing) & 1, p);
}

__device__ void mma_role(Ctl& ctl, const Params& p, uint32_t tmem, uint32_t sQ, uint32_t sKV) {
  const bool leader = elect_one();
  Walk walk(p, blockIdx.x);
  Segment sg;
  uint32_t it = 0, qn = 0, pn[2] = {0, 0};
  bool ok = true;
  auto landed = [&](uint32_t item) {
    const bool r = wait_warp(smem_addr(&ctl.full[item % kRing]), (item / kRing) & 1, ctl, p);
    tc_fence_after_sync();
    return r;
  };
  auto tile_at = [&](uint32_t item) { return sKV + (item % kRing) * kTileBytes; };
  auto release = [&](uint32_t item) {
    if (leader) mma_commit(smem_addr(&ctl.empty[item % kRing]));
  };
  // scores of K item `item` for slot s, from row tile `q`
  auto scores = [&](int s, int q, uint32_t item) {
    issue_qk(leader, tmem + 128 * s, sQ + q * kTileBytes, tile_at(item));
    if (leader) mma_commit(smem_addr(&ctl.s_full[s]));
  };
  // slot s's weights times V item `item`
  auto values = [&](int s, uint32_t item, bool accumulate, bool last) {
    const bool r = wait_warp(smem_addr(&ctl.p_full[s]), pn[s] & 1, ctl, p);
    if (!r) return false;
    ++pn[s];
    tc_fence_after_sync();
    issue_pv(leader, tmem + 256 + 128 * s, tmem + 128 * s, tile_at(item), accumulate);
    if (leader && last) mma_commit(smem_addr(&ctl.o_done[s]));
    return true;
  };
  while (ok && walk.next(sg)) {
    if (!wait_warp(smem_addr(&ctl.q_full), qn & 1, ctl, p)) break;
    ++qn;
    const uint32_t it0 = it;
    it += 2 * sg.n;
    for (int j = 0; j < sg.n; ++j) {
      const uint32_t k = it0 + 2 * j, v = k + 1;
      if (!landed(k)) { ok = false; break; }
      if (sg.both) {
        scores(0, 0, k);
        // the other row tile's turn: its weights of the tile before
        if (j > 0) {
          if (!values(1, v - 2, j > 1, false)) { ok = false; break; }
          release(v - 2);
        }
        scores(1, 1, k);
        release(k);
        if (leader && j == sg.n - 1) mma_commit(smem_addr(&ctl.q_empty));
        if (!landed(v) || !values(0, v, j > 0, j == sg.n - 1)) { ok = false; break; }
        if (j == sg.n - 1) {
          if (!values(1, v, j > 0, true)) { ok = false; break; }
          release(v);
        }
      } else {
        scores(j & 1, 0, k);
        release(k);
        if (leader && j == sg.n - 1) mma_commit(smem_addr(&ctl.q_empty));
        if (j > 0) {
          if (!landed(v - 2) || !values((j - 1) & 1, v - 2, j > 2, j == sg.n - 1)) {
            ok = false;
            break;
          }
          release(v - 2);
        }
        if (j == sg.n - 1) {
          if (!landed(v) || !values(j & 1, v, j > 1, true)) { ok = false; break; }
          release(v);
        }
      }
    }
  }
  // no MMA may still be running when TMEM is released
  if (leader) mma_commit(smem_addr(&ctl.drain));
  drain_wait(smem_addr(&ctl.drain), 0, p);
  __syncwarp();
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Row maximum of 128 scores with three-input max instructions.
__device__ __forceinline__ float row_max128(const float* v) {
  float m[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) m[t] = v[t];
#pragma unroll
  for (int i = 8; i < 128; i += 16)
#pragma unroll
    for (int t = 0; t < 8; ++t) m[t] = max3(m[t], v[i + t], v[i + 8 + t]);
  return max3(max3(m[0], m[1], m[2]), max3(m[3], m[4], m[5]), fmaxf(m[6], m[7]));
}

// kPos: the scale is positive and multiplies inside the exponent's FMA; any
// other is applied to the scores first, so that the maximum is of scaled ones.
template <bool kPos>
__device__ void softmax_role(int slot, Ctl& ctl, const Params& p, uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = (warp & 3) * 32 + lane;                         // row of the tile = TMEM lane
  const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
  const uint32_t tS = lane_base + 128 * slot, tO = lane_base + 256 + 128 * slot;
  const float cc = kPos ? p.c : 1.0f;
  const uint64_t cc2 = f32x2_pack(cc, cc);
  uint32_t ph_s = 0, ph_o = 0;
  Walk walk(p, blockIdx.x);
  Segment sg;
  while (walk.next(sg)) {
    const int n = sg.count(slot);
    const size_t part = 2 * (static_cast<size_t>(sg.unit) + blockIdx.x) + slot;
    if (n == 0) {
      p.part_ml[part * kRows + r] = make_float2(-INFINITY, 0.0f);
      continue;
    }
    float m_run = -INFINITY, l_run = 0.0f;
    for (int j = 0; j < n; ++j) {
      if (!wait_warp(smem_addr(&ctl.s_full[slot]), ph_s, ctl, p)) return;
      ph_s ^= 1;
      tc_fence_after_sync();
      float s[128];
      uint32_t* sr = reinterpret_cast<uint32_t*>(s);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        tmem_ld32(tS + 32 * q, *reinterpret_cast<uint32_t(*)[32]>(sr + 32 * q));
      tmem_wait_ld(*reinterpret_cast<uint32_t(*)[32]>(sr));
      tmem_after_wait(*reinterpret_cast<uint32_t(*)[32]>(sr + 32));
      tmem_after_wait(*reinterpret_cast<uint32_t(*)[32]>(sr + 64));
      tmem_after_wait(*reinterpret_cast<uint32_t(*)[32]>(sr + 96));
      if (!kPos) {
#pragma unroll
        for (int i = 0; i < 128; ++i) s[i] *= p.c;
      }
      const int live = p.P - sg.tile(slot, j) * kKeys;
      if (live < kKeys) {
#pragma unroll
        for (int i = 0; i < 128; ++i)
          if (i >= live) s[i] = -INFINITY;
      }
      const float m_new = fmaxf(m_run, row_max128(s) * cc);
      const bool need = m_new > m_run + kRescale;
      float alpha = 1.0f;
      if (need) {
        alpha = ex2_approx(m_run - m_new);
        m_run = m_new;
      }
      // P = 2^(c s - m), bf16 pairs over the scores' first columns (every score
      // of the row is in registers); the row sum keeps the unrounded values. bf16
      // because V is (both operands of a product have one type): a second product
      // with what the rounding leaves would make a kernel that the tensor cores
      // bound half as long again, to take the error of O from 2.4e-3 to the 1.7e-3
      // of O's own rounding.
      const float m_use = (m_run == -INFINITY) ? 0.0f : m_run;
      const uint64_t negm2 = f32x2_pack(-m_use, -m_use);
      uint64_t sum2 = f32x2_pack(0.0f, 0.0f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float x0, x1;
          f32x2_unpack(ffma2(f32x2_pack(s[64 * h + 2 * i], s[64 * h + 2 * i + 1]), cc2, negm2), x0,
                       x1);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          sum2 = fadd2(sum2, f32x2_pack(p0, p1));
          pk[i] = pack_bf16x2(p0, p1);
        }
        tmem_st32(tS + 32 * h, pk);
      }
      float sa, sb;
      f32x2_unpack(sum2, sa, sb);
      l_run = l_run * alpha + (sa + sb);
      // O <- O * 2^(m_old - m_new) where a row's maximum moved (rare); O holds
      // every earlier tile, since this tile's scores were issued after them
      if (j > 0 && __any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int q = 0; q < kDim; q += 32) {
          uint32_t ov[32];
          tmem_ld32(tO + q, ov);
          tmem_wait_ld(ov);
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
          tmem_st32(tO + q, ov);
        }
      }
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(smem_addr(&ctl.p_full[slot]));
    }
    if (!wait_warp(smem_addr(&ctl.o_done[slot]), ph_o, ctl, p)) return;
    ph_o ^= 1;
    tc_fence_after_sync();
    float4* out = reinterpret_cast<float4*>(p.part_o + part * kPartFloats) + r;
#pragma unroll 1
    for (int q = 0; q < kDim; q += 32) {
      uint32_t ov[32];
      tmem_ld32(tO + q, ov);
      tmem_wait_ld(ov);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        out[(q / 4 + i) * kRows] =
            make_float4(__uint_as_float(ov[4 * i]), __uint_as_float(ov[4 * i + 1]),
                        __uint_as_float(ov[4 * i + 2]), __uint_as_float(ov[4 * i + 3]));
    }
    tc_fence_before_sync();
    p.part_ml[part * kRows + r] = make_float2(m_run, l_run);
  }
}

template <bool kPos>
__global__ void __launch_bounds__(kThreads, 1)
prefix_split_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
  extern __shared__ uint8_t dyn_smem[];
  __shared__ Ctl ctl;
  const uint32_t base = (smem_addr(dyn_smem) + 1023u) & ~1023u;   // swizzle atoms need 1 KiB
  const uint32_t sQ = base, sKV = base + 2 * kTileBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRing; ++s) {
      mbar_init(smem_addr(&ctl.full[s]), 1);
      mbar_init(smem_addr(&ctl.empty[s]), 1);
    }
    mbar_init(smem_addr(&ctl.q_full), 1);
    mbar_init(smem_addr(&ctl.q_empty), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_addr(&ctl.s_full[s]), 1);
      mbar_init(smem_addr(&ctl.p_full[s]), 128);
      mbar_init(smem_addr(&ctl.o_done[s]), 1);
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
  if (p.nb * p.g < kRows && warp < 8) {
    // rows past nb * g are never loaded (nor read by the combine): zeros
    uint4* z = reinterpret_cast<uint4*>(dyn_smem + (sQ - smem_addr(dyn_smem)));
    for (int i = threadIdx.x; i < 2 * kTileBytes / 16; i += 256) z[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = ctl.tmem_base;
  // wait for everything earlier before letting the own positions' kernel
  // launch: it starts without a wait of its own
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    softmax_role<kPos>(warp >> 2, ctl, p, tmem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      if (lane == 0) load_role(&tmQ, &tmK, &tmV, ctl, p, sQ, sKV);
    } else if (warp == kMmaWarp) {
      mma_role(ctl, p, tmem, sQ, sKV);
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// 32 rows of one row tile per CTA, lane = row: the prefix partials' pieces of
// four dimensions are 512 contiguous bytes for the warp (a warp per row, lane =
// dimensions: 26 us of the 32-head case above, 12 so). Warp w of the CTA's
// eight takes dimensions 8 (8 y + w) .. + 7, y = blockIdx.y in 0 .. 1.
constexpr int kCombineRows = 32, kCombineWarps = 8, kCombineY = 2;

__global__ void __launch_bounds__(32 * kCombineWarps)
shared_combine_kernel(uint16_t* o, float* lse, const int* lens, int C,
                      const gb300_host::RaggedParts own, const Params p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int blocks = (p.nb * p.g + kCombineRows - 1) / kCombineRows;
  const int kt = blockIdx.x / blocks;                     // K/V head and row tile
  const int r = (blockIdx.x - kt * blocks) * kCombineRows + lane;
  const int kvh = kt / p.tiles, tile = kt - kvh * p.tiles;
  const int b = tile * p.nb + r / p.g, h = r % p.g;
  if (r >= p.nb * p.g || b >= p.B) return;
  const int d4 = 2 * (blockIdx.y * kCombineWarps + (threadIdx.x >> 5));   // first of two

  // where the own positions' partials are, on its way from the start
  const size_t hd = static_cast<size_t>(b) * p.n_kv + kvh;
  const int2 ends = reinterpret_cast<const int2*>(own.ends)[hd];
  const int own_len = min(lens[b], C);

  float m = -INFINITY, wsum = 0.0f;
  float4 acc[2];
  acc[0] = acc[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](const float2& ml, const float4& u, const float4& v) {
    // an empty part: u, v are not written (with NaN for a sum it has keys, none of
    // whose scores is a number)
    if (ml.x == -INFINITY && ml.y == 0.0f) return;
    const float mn = fmaxf(m, ml.x);
    const float a = (m == -INFINITY) ? 0.0f : exp2f(m - mn);
    const float w = exp2f(ml.x - mn);
    m = mn;
    wsum = fmaf(w, ml.y, wsum * a);
    acc[0].x = fmaf(w, u.x, acc[0].x * a);
    acc[0].y = fmaf(w, u.y, acc[0].y * a);
    acc[0].z = fmaf(w, u.z, acc[0].z * a);
    acc[0].w = fmaf(w, u.w, acc[0].w * a);
    acc[1].x = fmaf(w, v.x, acc[1].x * a);
    acc[1].y = fmaf(w, v.y, acc[1].y * a);
    acc[1].z = fmaf(w, v.z, acc[1].z * a);
    acc[1].w = fmaf(w, v.w, acc[1].w * a);
  };

  const int unit = kvh * p.pairs + tile / 2;
  const bool both = (tile | 1) < p.tiles;
  const long long x = static_cast<long long>(unit) * p.T;
  const int c0 = static_cast<int>(cta_of(x, p.W, p.G));
  const int c1 = static_cast<int>(cta_of(x + p.T - 1, p.W, p.G));
  // two row tiles: this tile's slot of every segment; one: both slots
  const int step = both ? 2 : 1, slots = both ? 1 : 2;
  const size_t first = 2 * (static_cast<size_t>(unit) + c0) + (both ? (tile & 1) : 0);
  const float4* part = reinterpret_cast<const float4*>(p.part_o) + d4 * kRows + r;
  const int count = (c1 - c0 + 1) * slots;
  constexpr int kBatch = 4;              // partials on their way at once
  for (int e0 = 0; e0 < count; e0 += kBatch) {
    float2 ml[kBatch];
    float4 u[kBatch], v[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      ml[e] = make_float2(-INFINITY, 0.0f);
      if (e0 + e < count) {
        const size_t at = first + static_cast<size_t>(e0 + e) * step;
        ml[e] = p.part_ml[at * kRows + r];
        u[e] = part[at * (kPartFloats / 4)];
        v[e] = part[at * (kPartFloats / 4) + kRows];
      }
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e) add(ml[e], u[e], v[e]);
  }
  if (own_len > 0) {
    for (int c = ends.x; c <= ends.y; ++c) {
      const size_t row = (hd + c) * p.g + h;
      const float4* src = reinterpret_cast<const float4*>(own.o) + row * 32 + d4;
      add(own.ml[row], src[0], src[1]);
    }
  }
  const float inv = 1.0f / wsum;
  const size_t row = static_cast<size_t>(b) * p.n_q + kvh * p.g + h;
  *reinterpret_cast<uint4*>(o + row * kDim + 4 * d4) =
      make_uint4(pack_bf16x2(acc[0].x * inv, acc[0].y * inv), pack_bf16x2(acc[0].z * inv, acc[0].w * inv),
                 pack_bf16x2(acc[1].x * inv, acc[1].y * inv), pack_bf16x2(acc[1].z * inv, acc[1].w * inv));
  if (d4 == 0) lse[row] = (m + log2f(wsum)) * 0.69314718055994530942f;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr int kMaxDevices = 64;
std::mutex g_shared_mutex;
bool g_shared_ready[kMaxDevices] = {};
EncodeTiledFn g_shared_encode = nullptr;

// The register split only works on a CTA launched with at least that many.
template <bool kPos>
bool configure() {
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, prefix_split_kernel<kPos>) != cudaSuccess ||
      fa.numRegs * kThreads < kRegBudget)
    return false;
  return cudaFuncSetAttribute(prefix_split_kernel<kPos>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kSmemBytes) == cudaSuccess;
}

attn_status_t shared_device_ready(cudaStream_t stream, int** status) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_UNSUPPORTED;
  const attn_status_t ds = gb300_host::decode_ready(stream, status);
  if (ds != ATTN_OK) return ds;
  std::lock_guard<std::mutex> lock(g_shared_mutex);
  if (g_shared_ready[dev]) return ATTN_OK;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess || cs != cudaStreamCaptureStatusNone) {
    cudaGetLastError();
    return ATTN_ERR_UNSUPPORTED;
  }
  if (!g_shared_encode) {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || fn == nullptr)
      return ATTN_ERR_CUDA;
    g_shared_encode = reinterpret_cast<EncodeTiledFn>(fn);
  }
  if (!configure<true>() || !configure<false>()) return ATTN_ERR_UNSUPPORTED;
  g_shared_ready[dev] = true;
  return ATTN_OK;
}

// bf16 [L, H, 128] as (D, H, L), boxes of 64 x heads x rows with 128-byte
// swizzle; rows past L read as zeros.
bool encode(CUtensorMap* map, const void* ptr, int H, int64_t L, int heads, int rows) {
  const cuuint64_t dims[3] = {kDim, static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(L)};
  const cuuint64_t strides[2] = {kDim * 2, static_cast<cuuint64_t>(H) * kDim * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(rows)};
  const cuuint32_t estride[3] = {1, 1, 1};
  return g_shared_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims,
                         strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Shape {
  int64_t nb, tiles, pairs, units, T, W, G, ml_at, own_at, own, bytes;
};

// False where a size is beyond the kernels' limits.
bool shape_of(int64_t B, int64_t P, int64_t C, int32_t n_q, int32_t n_kv, int32_t d_h, Shape* s) {
  s->own = gb300_host::ragged_split_bytes(B, C, n_q, n_kv, d_h);
  if (s->own < 0 || P > (int64_t{1} << 30)) return false;
  s->nb = kRows / (n_q / n_kv);
  s->tiles = (B + s->nb - 1) / s->nb;
  s->pairs = (s->tiles + 1) / 2;
  s->units = s->pairs * n_kv;
  s->T = (P + kKeys - 1) / kKeys;
  s->W = s->units * s->T;
  s->G = s->W < kCtas ? s->W : kCtas;
  const int64_t parts = 2 * (s->units + s->G);
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  s->ml_at = up(parts * kPartFloats * 4);
  s->own_at = s->ml_at + up(parts * kRows * 8);
  s->bytes = s->own_at + s->own;
  return s->units <= (int64_t{1} << 30) && s->W <= (int64_t{1} << 40) &&
         s->tiles * n_kv * (kRows / kCombineRows) <= INT32_MAX;
}

bool sizes_ok(int64_t B, int64_t P, int64_t C, int32_t n_q, int32_t n_kv, int32_t d_h) {
  return B >= 1 && P >= 1 && C >= 1 && n_q >= 1 && n_kv >= 1 && n_q % n_kv == 0 && d_h >= 1;
}

}  // namespace

extern "C" {

int64_t attn_decode_shared_workspace_bytes(int64_t B, int64_t P, int64_t C, int32_t n_q,
                                           int32_t n_kv, int32_t d_h) {
  Shape s;
  if (!sizes_ok(B, P, C, n_q, n_kv, d_h) || !shape_of(B, P, C, n_q, n_kv, d_h, &s)) return -1;
  return s.bytes;
}

attn_status_t attn_decode_shared_fwd(const void* q, const void* prefix_k, const void* prefix_v,
                                     const void* k, const void* v, const int32_t* lens, void* o,
                                     float* lse, void* workspace, int64_t workspace_bytes, int64_t B,
                                     int64_t P, int64_t C, int32_t n_q, int32_t n_kv, int32_t d_h,
                                     float scale, void* stream_ptr) {
  if (!q || !prefix_k || !prefix_v || !k || !v || !lens || !o || !lse || !workspace)
    return ATTN_ERR_INVALID_ARG;
  if (!sizes_ok(B, P, C, n_q, n_kv, d_h) || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  auto misaligned = [](const void* ptr, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0;
  };
  if (misaligned(q, 16) || misaligned(prefix_k, 16) || misaligned(prefix_v, 16) ||
      misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) || misaligned(lse, 4) ||
      misaligned(lens, 4) || misaligned(workspace, 16))
    return ATTN_ERR_INVALID_ARG;
  Shape s;
  if (!shape_of(B, P, C, n_q, n_kv, d_h, &s)) return ATTN_ERR_UNSUPPORTED;
  if (workspace_bytes < s.bytes) return ATTN_ERR_INVALID_ARG;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  int* status = nullptr;
  attn_status_t st = shared_device_ready(stream, &status);
  if (st != ATTN_OK) return st;

  Params p{};
  char* ws = static_cast<char*>(workspace);
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + s.ml_at);
  p.status = status;
  p.P = static_cast<int>(P);
  p.T = static_cast<int>(s.T);
  p.B = static_cast<int>(B);
  p.n_q = n_q;
  p.n_kv = n_kv;
  p.g = n_q / n_kv;
  p.nb = static_cast<int>(s.nb);
  p.tiles = static_cast<int>(s.tiles);
  p.pairs = static_cast<int>(s.pairs);
  p.units = static_cast<int>(s.units);
  p.G = static_cast<int>(s.G);
  p.W = s.W;
  p.c = scale * 1.4426950408889634f;
  p.spin_limit = 1ll << 31;   // about a second at 2 GHz
  CUtensorMap mq, mk, mv;
  if (!encode(&mq, q, n_q, B, p.g, p.nb) || !encode(&mk, prefix_k, n_kv, P, 1, kKeys) ||
      !encode(&mv, prefix_v, n_kv, P, 1, kKeys))
    return ATTN_ERR_CUDA;
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
  const cudaError_t e = p.c > 0.0f
                            ? cudaLaunchKernelEx(&cfg, prefix_split_kernel<true>, mq, mk, mv, p)
                            : cudaLaunchKernelEx(&cfg, prefix_split_kernel<false>, mq, mk, mv, p);
  if (e != cudaSuccess) return ATTN_ERR_CUDA;
  gb300_host::RaggedParts own;
  st = gb300_host::ragged_split_beside(q, k, v, lens, ws + s.own_at, B, C, n_q, n_kv, scale, stream,
                                       status, &own);
  if (st != ATTN_OK) return st;
  const int blocks = (p.nb * p.g + kCombineRows - 1) / kCombineRows;
  cfg.gridDim = dim3(static_cast<unsigned>(s.tiles * n_kv * blocks), kCombineY);
  cfg.blockDim = dim3(32 * kCombineWarps);
  cfg.dynamicSmemBytes = 0;
  if (cudaLaunchKernelEx(&cfg, shared_combine_kernel, static_cast<uint16_t*>(o), lse, lens,
                         static_cast<int>(C), own, p) != cudaSuccess)
    return ATTN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
