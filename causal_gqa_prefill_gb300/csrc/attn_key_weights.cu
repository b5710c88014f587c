// attn_key_weights.cu — the attention that every key of a prefill received, on
// GB300 (sm_103a): the column sums of the softmax weights, rebuilt from Q, K
// and the forward's log-sum-exps,
//
//   W[b,u,j] (+)= sum_{h in group u} sum_{i sees j} 2^(c q_ih . k_ju - lse2_ih),
//   c = scale * log2(e),  lse2 = LSE * log2(e).
//
// A step is 128 query rows against 256 keys, S = Q K^T on tcgen05 with the rows
// on the TMEM lanes. A thread owns a row and 64 keys: its lse2 is one register
// for the whole step, and it adds each weight to a register of its own per key,
// step after step, so a score costs one FMA, one exponential and one addition
// and nothing is exchanged between threads until the keys change. Only then are
// the 64 sums of a warp's 32 rows folded (62 shuffles) and the four warps' added.
// (With the keys on the lanes a column sum needs no folding at all, but then
// every score takes its row's lse2 from shared memory, whose reads queue behind
// the exponentials: 2130 clocks a step against 1600 here.)
//
//   rows     packed: a step holds nr = 128 / g consecutive query rows of all g
//            heads of the group (lane = row * g + head, which is what one TMA box
//            of g heads x nr rows lands as), so every head count fills the tile
//            and a causal step wastes at most nr rows.
//   unit     256 keys of one (b, K/V head), N = 256: at N = 128 the two operands
//            of a product are all that shared memory can read at the tensor
//            cores' rate, and the Q tiles would need 64 bytes a clock and SM from
//            L2. A unit's steps are the row blocks that see it, in order.
//   CTA      one per SM; the steps of all units, in order, are cut into equal
//            ranges (triangles need no further balancing). A unit that a range
//            border cuts is summed by a second kernel from at most one partial
//            per CTA, in CTA order: no atomics, the same bits every time.
//   warps    0-15 four warpgroups of 64 keys each (four warps a scheduler keep
//            the exponential unit fed); 16 TMA; 17 MMA; 18 the rows' -lse2.
//
// S is double-buffered (all 512 TMEM columns), so the product of a step runs
// under the exponentials of the one before; both take 1024 clocks a step, the
// exponentials at 32 a clock and SM. Measured, 8192-token 32-head layer, calls back to
// back on one set of inputs (as all times in these comments): 186 us, both pipes busy
// 66 % of it; 200 with inputs from memory. Without any sums it is 147: both operands come from
// shared memory and the next Q tile arrives in it, which fills its bandwidth (two
// products of 128 keys, which read the rows twice: 198). The rest is the latency of
// load, exponential and addition, which four warps a scheduler and 32 scores at a
// time cover in part (16 at a time: 196).
//
// K is fetched a unit ahead, and where a head's steps fit the Q ring they stay
// there from unit to unit (a prompt's last rows against a long cache: K is then
// all that is read).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "attn_prefill.h"
#include "key_weights_ranges.h"
#include "sm103_ptx.cuh"

namespace gb300_host {
attn_status_t device_status_word(cudaStream_t stream, int** status);
}

namespace {

using namespace gb300;
using namespace gb300_key_weights;    // kUnitKeys (N), kRows (TMEM lanes), kCtas

constexpr int kGroups = 4;            // warpgroups of the sums
constexpr int kCols = kUnitKeys / kGroups;    // keys per thread
constexpr int kSumWarps = 4 * kGroups;
constexpr int kThreads = 32 * kSumWarps + 128;
constexpr int kLoadWarp = kSumWarps, kMmaWarp = kSumWarps + 1, kStatWarp = kSumWarps + 2;
constexpr int kFold = kCols / 32;     // keys per lane once the rows are folded
// registers per thread: the sums of 64 keys, and their scores 32 at a time
constexpr int kSumRegs = 112, kOtherRegs = 32;
constexpr int kLaunchRegs = 96;
constexpr int kRegBudget = 32 * kSumWarps * kSumRegs + 128 * kOtherRegs;
static_assert(kRegBudget <= kThreads * kLaunchRegs, "setmaxnreg split exceeds the launch allocation");
constexpr uint32_t kTmemCols = 512;   // S at columns 0 and 256
constexpr int kStatusTimeout = 1, kStatusCheck = 2;
constexpr uint32_t kSuspendNs = 2000;
constexpr float kLog2e = 1.4426950408889634f;

// What stands for a row in the exponents: -lse2, or kNoWeight where there is no row or
// its lse is -inf (a row without keys). No other row has that value.
constexpr float kNoWeight = INFINITY;
__device__ __forceinline__ float exponent_of(float lse) {
  const float x = -lse * kLog2e;
  return lse == -INFINITY ? kNoWeight : x > FLT_MAX ? FLT_MAX : x;   // (a NaN stays one)
}

template <int D>
struct Geometry {
  static constexpr int kChunks = D * 2 / 128;              // 128-byte swizzle column chunks
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kQChunk = kRows * 128;
  static constexpr int kKBytes = kUnitKeys * D * 2;
  static constexpr int kKChunk = kUnitKeys * 128;
  static constexpr int kQStages = D == 128 ? 3 : 6;
  static constexpr int kTileBytes = 2 * kKBytes + kQStages * kQBytes;   // two K buffers, the Q ring
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

struct __align__(16) Ctl {
  uint64_t k_full[2], k_empty[2];
  uint64_t q_full[6], q_empty[6];
  uint64_t s_full[2], s_free[2];
  uint64_t fold[kGroups][3], fold_free[kGroups];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  __align__(16) float nl[2][kRows];      // -lse2 of a step's rows
  float sums[kGroups][kFold][32];        // a warpgroup's sums on their way from warp to warp
};

// Ctl, then the tiles at the next multiple of 1 KiB (swizzle atoms). With
// d_h = 128 this is all of an SM's 227 KiB: the kernel checks that it fits.
constexpr int kCtlBytes = (sizeof(Ctl) + 1023) / 1024 * 1024;
template <int D>
__host__ __device__ constexpr int smem_bytes() {
  return kCtlBytes + Geometry<D>::kTileBytes;
}
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory");

// First row of a step. The last one ends with the last row, so that every row of
// the tile is one (a zero row's product with an infinite key is NaN); the rows
// that the step before has too count there. (Lq > nr: else few rows, below.)
__device__ __forceinline__ int first_row(int step, const Params& p) {
  return min(step * p.nr, p.Lq - p.nr);
}

struct Segment {
  int head, b, kvh, key0, s0, n;   // head = b * n_kv + kvh
  bool first, whole;               // the range's first segment; a unit that nothing cuts
};

// Walks a CTA's range unit by unit; every role takes the same walk.
struct Walk {
  const Params& p;
  int head, b, kvh, t, step, first_of_unit, left;
  bool first;
  __device__ Walk(const Params& params, const Starts& st, int c)
      : p(params), step(st.step[c]), left(st.count[c]), first(true) {
    head = st.unit[c] / p.T;
    t = st.unit[c] - head * p.T;
    b = head / p.n_kv;
    kvh = head - b * p.n_kv;
    first_of_unit = first_step(t, p.off, p.nr, p.causal);
  }
  __device__ bool next(Segment& s) {
    if (left <= 0) return false;
    s.head = head;
    s.b = b;
    s.kvh = kvh;
    s.key0 = t * kUnitKeys;
    s.s0 = step;
    s.n = min(left, p.steps - step);
    s.first = first;
    s.whole = step == first_of_unit && s.n == p.steps - step;
    left -= s.n;
    first = false;
    if (++t == p.T) {
      t = 0;
      ++head;
      if (++kvh == p.n_kv) {
        kvh = 0;
        ++b;
      }
    }
    step = first_of_unit = first_step(t, p.off, p.nr, p.causal);
    return true;
  }
};

// Does any row of step `step` see `key`?
__device__ __forceinline__ bool seen(const Params& p, int key, int step) {
  if (key >= p.Lk) return false;
  const int last = min((step + 1) * p.nr, p.Lq) - 1;
  return !p.causal || key <= last + p.off;
}

// (for both kernels' control blocks and parameters)
template <typename C, typename P>
__device__ __forceinline__ bool spin_wait(uint32_t bar, uint32_t parity, C& ctl, const P& p) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = clock64_now();
  while (true) {
    if (mbar_try_wait_for(bar, parity, kSuspendNs)) return true;
    if (*reinterpret_cast<volatile int*>(&ctl.abort)) return false;
    if (static_cast<long long>(clock64_now() - t0) > p.spin_limit) {
      *reinterpret_cast<volatile int*>(&ctl.abort) = 1;
      atomicOr(p.status, kStatusTimeout);
      return false;
    }
  }
}

template <typename C, typename P>
__device__ __forceinline__ bool wait_slowly(uint32_t bar, uint32_t parity, C& ctl, const P& p) {
  return __all_sync(0xffffffffu, spin_wait(bar, parity, ctl, p));
}

template <typename C, typename P>
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, C& ctl, const P& p) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return wait_slowly(bar, parity, ctl, p);
}

// Wait used while draining after an abort: ignores the abort flag.
template <typename P>
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity, const P& p) {
  const uint64_t t0 = clock64_now();
  while (!mbar_try_wait(bar, parity))
    if (static_cast<long long>(clock64_now() - t0) > p.spin_limit) return;
}

// acc += 2^(c s + nl) for the 32 keys whose scores are in s, two at a time; with
// kMask those past key `keep` are hidden (after the product with the row's lse: one
// that is NaN reaches the keys that the row sees and no others).
template <bool kMask>
__device__ __forceinline__ void add_weights(uint64_t* acc, const uint32_t (&s)[32], uint64_t c2,
                                            uint64_t nl2, int keep) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float x0, x1;
    f32x2_unpack(ffma2(f32x2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c2, nl2), x0, x1);
    if (kMask) {
      if (i > keep) x0 = -INFINITY;
      if (i + 1 > keep) x1 = -INFINITY;
    }
    const float e0 = ex2_approx(x0), e1 = ex2_approx(x1);
    const uint64_t e = f32x2_pack(e0, e1);
    asm("add.f32x2 %0, %0, %1;" : "+l"(acc[i / 2]) : "l"(e));
  }
}

// Sums kCols values per lane over the warp's lanes: five steps that each halve
// what a lane carries. Lane l gets the sums of keys kFold l .. kFold l + kFold - 1
// in v[0 .. kFold - 1].
__device__ __forceinline__ void fold_lanes(float (&v)[kCols]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 16, width = kCols / 2; off > 0; off >>= 1, width >>= 1) {
    const bool upper = (lane & off) != 0;
#pragma unroll
    for (int i = 0; i < width; ++i) {
      const float send = upper ? v[i] : v[i + width], keep = upper ? v[i + width] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
    }
  }
}

__device__ void sum_role(Ctl& ctl, const Params& p, const Starts& starts, uint32_t tmem) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp >> 2, quarter = warp & 3;
  const int r = quarter * 32 + lane;                   // row of the step = TMEM lane
  const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + kCols * group;
  const uint64_t c2 = f32x2_pack(p.c, p.c);
  const int row = r / p.g;
  // a buffer is free once its last scores are in registers, before they are
  // summed: the next product starts half a step earlier, and a warp that is ahead
  // finds its scores (released after the sums: 203 us)
  auto release = [&](uint32_t buf) {
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&ctl.s_free[buf]));
  };
  Walk walk(p, starts, blockIdx.x);
  Segment sg;
  uint32_t n = 0, seg = 0;
  while (walk.next(sg)) {
    const int key0 = sg.key0 + kCols * group;
    // steps before `from` do not see the group's first key; in steps before
    // `until` some row does not see its last one
    const int past = p.causal ? key0 - p.off : 0;
    int from = past > 0 ? static_cast<int>(static_cast<unsigned>(past) / static_cast<unsigned>(p.nr)) : 0;
    if (key0 >= p.Lk) from = p.steps;
    int until =
        p.causal && past + kCols - 1 > 0
            ? static_cast<int>(static_cast<unsigned>(past + kCols - 2 + p.nr) / static_cast<unsigned>(p.nr))
            : 0;
    // (nor do the rows that the last step has a second time)
    if (until == p.steps - 1 && past + kCols - 1 > p.Lq - p.nr) until = p.steps;
    uint64_t acc[kCols / 2];
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) acc[i] = f32x2_pack(0.0f, 0.0f);
    const int end = sg.s0 + sg.n;
    for (int st = sg.s0; st < end; ++st, ++n) {
      const uint32_t buf = n & 1;
      if (!wait_warp(smem_addr(&ctl.s_full[buf]), (n >> 1) & 1, ctl, p)) return;
      tc_fence_after_sync();
      if (st >= from) {
        const float nl = ctl.nl[buf][r];
        const uint64_t nl2 = f32x2_pack(nl, nl);
        const uint32_t taddr = lanes + kUnitKeys * buf;
        uint32_t s[32];
        // a row without weight (lanes without rows are dropped when the rows are folded)
        // takes its warp to the sum with a mask, where it sees no key: its query may be
        // anything, and a NaN score plus -inf is NaN (a vote of the warp: 0.3 % of the
        // 8192-token layer, 1 % with a flag from the statistics' warp)
        const bool none = nl == kNoWeight;
        if (st >= until && !__any_sync(0xffffffffu, none && row < p.nr)) {
#pragma unroll
          for (int q = 0; q < kCols / 32; ++q) {
            tmem_ld32(taddr + 32 * q, s);
            tmem_wait_ld(s);
            if (q == kCols / 32 - 1) release(buf);
            add_weights<false>(acc + 16 * q, s, c2, nl2, 0);
          }
        } else {
          // this row's position sees key0 + i for i <= keep
          const int keep = none ? -1 : p.causal ? p.off + first_row(st, p) + row - key0 : kCols;
#pragma unroll
          for (int q = 0; q < kCols / 32; ++q) {
            tmem_ld32(taddr + 32 * q, s);
            tmem_wait_ld(s);
            if (q == kCols / 32 - 1) release(buf);
            add_weights<true>(acc + 16 * q, s, c2, nl2, keep - 32 * q);
          }
        }
      } else {
        release(buf);
      }
    }
    // fold the rows: over the warp's lanes, then from warp 3 of the warpgroup
    // to warp 0
    float v[kCols];
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) {
      if (row >= p.nr) acc[i] = f32x2_pack(0.0f, 0.0f);   // a lane without rows
      f32x2_unpack(acc[i], v[2 * i], v[2 * i + 1]);
    }
    fold_lanes(v);
    if (quarter == 3) {
      if (seg > 0 && !wait_warp(smem_addr(&ctl.fold_free[group]), (seg - 1) & 1, ctl, p)) return;
    } else {
      if (!wait_warp(smem_addr(&ctl.fold[group][quarter]), seg & 1, ctl, p)) return;
#pragma unroll
      for (int i = 0; i < kFold; ++i) v[i] += ctl.sums[group][i][lane];
    }
    if (quarter > 0) {
#pragma unroll
      for (int i = 0; i < kFold; ++i) ctl.sums[group][i][lane] = v[i];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&ctl.fold[group][quarter - 1]));
    } else {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&ctl.fold_free[group]));
      const int key = key0 + kFold * lane;
      float* out = sg.whole ? p.weights + static_cast<size_t>(sg.head) * p.Lk + key
                            : p.part + (2 * blockIdx.x + (sg.first ? 0 : 1)) * kUnitKeys +
                                  kCols * group + kFold * lane;
      const bool old = sg.whole && p.accumulate;
#pragma unroll
      for (int i = 0; i < kFold; ++i)
        if (!sg.whole || key + i < p.Lk) out[i] = old ? out[i] + v[i] : v[i];
    }
    ++seg;
  }
}

// One warp: -lse2 of every step's rows to shared memory, as one of the two
// arrivals that complete s_full. Lane's rows lane + 32 m; the values of the next
// kAhead steps are in registers or on their way.
__device__ void stat_role(Ctl& ctl, const Params& p, const Starts& starts) {
  const int lane = threadIdx.x & 31;
  constexpr int kAhead = 2;
  int row[4], at[4];                       // row of the step, offset of its head
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int r = lane + 32 * m;
    row[m] = r / p.g;                                    // (nr and more: none)
    at[m] = (r % p.g) * p.Lq + row[m];
  }
  Walk walk(p, starts, blockIdx.x);
  Segment sg;
  int left = 0, step = 0;
  const float* lse = nullptr;
  auto fetch = [&](float (&v)[4]) {
    if (left == 0) {
      if (!walk.next(sg)) return false;
      left = sg.n;
      step = sg.s0;
      lse = p.lse + (static_cast<size_t>(sg.b) * p.n_q + sg.kvh * p.g) * p.Lq;
    }
    const int from = first_row(step, p), again = step * p.nr - from;   // rows of the step before
#pragma unroll
    for (int m = 0; m < 4; ++m)
      v[m] = row[m] < p.nr && row[m] >= again ? lse[at[m] + from] : -INFINITY;
    --left;
    ++step;
    return true;
  };
  float l[kAhead][4];
  bool have[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) have[u] = fetch(l[u]);
  for (uint32_t n0 = 0; have[0]; n0 += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (!have[u]) return;
      const uint32_t n = n0 + u, buf = n & 1;
      // the rows of step n - 2 have been read (and its s_full phase is over)
      if (n >= 2 && !wait_warp(smem_addr(&ctl.s_free[buf]), ((n >> 1) - 1) & 1, ctl, p)) return;
      // a row without keys, like a lane without a row, has no weight
#pragma unroll
      for (int m = 0; m < 4; ++m) ctl.nl[buf][lane + 32 * m] = exponent_of(l[u][m]);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&ctl.s_full[buf]));
      have[u] = fetch(l[u]);
    }
  }
}

template <int D>
__device__ void load_role(const CUtensorMap* tmQ, const CUtensorMap* tmK, Ctl& ctl, const Params& p,
                          const Starts& starts, uint32_t sK, uint32_t sQ, bool stay) {
  using G = Geometry<D>;
  uint32_t qn = 0, kn = 0, gn = 0;         // Q steps, K buffers and heads issued
  int begun = 0;                           // steps issued of a head that a wait cut short
  const uint32_t q_bytes = static_cast<uint32_t>(G::kChunks * 128 * p.g * p.nr);
  auto load_k = [&](const Segment& s) {
    const uint32_t kb = kn & 1;
    if (kn >= 2 && !spin_wait(smem_addr(&ctl.k_empty[kb]), ((kn >> 1) - 1) & 1, ctl, p)) return false;
    const uint32_t bar = smem_addr(&ctl.k_full[kb]);
    mbar_arrive_expect_tx(bar, G::kKBytes);
    for (int ch = 0; ch < G::kChunks; ++ch)
      tma_load_4d(sK + kb * G::kKBytes + ch * G::kKChunk, tmK, bar, ch * 64, s.kvh, s.key0, s.b);
    ++kn;
    return true;
  };
  // step `step` of segment s to ring slot `slot` for the use-th time
  auto load_q = [&](const Segment& s, int step, uint32_t slot, uint32_t use) {
    if (use > 0 && !spin_wait(smem_addr(&ctl.q_empty[slot]), (use - 1) & 1, ctl, p)) return false;
    const uint32_t bar = smem_addr(&ctl.q_full[slot]);
    mbar_arrive_expect_tx(bar, q_bytes);
    for (int ch = 0; ch < G::kChunks; ++ch)
      tma_load_4d(sQ + slot * G::kQBytes + ch * G::kQChunk, tmQ, bar, ch * 64, s.kvh * p.g,
                  first_row(step, p), s.b);
    return true;
  };
  Walk walk(p, starts, blockIdx.x);
  Segment sg, nx;
  bool more = walk.next(nx);
  bool ok = more && load_k(nx);
  int head = -1;                           // whose steps are in the ring
  while (ok && more) {
    sg = nx;
    more = walk.next(nx);
    if (more && !load_k(nx)) {             // a unit ahead
      ok = false;
      break;
    }
    if (stay) {
      if (sg.head == head) continue;
      head = sg.head;
      for (begun = 0; begun < p.steps && (ok = load_q(sg, begun, begun, gn)); ++begun) {
      }
      if (!ok) break;
      begun = 0;
      ++gn;
    } else {
      for (int i = 0; i < sg.n && ok; ++i) {
        ok = load_q(sg, sg.s0 + i, qn % G::kQStages, qn / G::kQStages);
        if (ok) ++qn;
      }
    }
  }
  // let every copy this thread started land before the CTA can exit, also where
  // another role has given up: the last use of each buffer
  for (uint32_t s = 0; s < 2 && s < kn; ++s)
    drain_wait(smem_addr(&ctl.k_full[s]), ((kn - 1 - s) >> 1) & 1, p);
  for (int s = 0; s < G::kQStages; ++s) {
    const uint32_t uses = stay ? (s < p.steps ? gn + (s < begun ? 1u : 0u) : 0u)
                               : (qn + G::kQStages - 1 - s) / G::kQStages;
    if (uses > 0) drain_wait(smem_addr(&ctl.q_full[s]), (uses - 1) & 1, p);
  }
}

template <int D>
__device__ void mma_role(Ctl& ctl, const Params& p, const Starts& starts, uint32_t tmem, uint32_t sK,
                         uint32_t sQ, bool stay) {
  using G = Geometry<D>;
  const bool leader = elect_one();
  constexpr uint32_t kIdWide = idesc_bf16_f32(kRows, kUnitKeys, false);
  constexpr uint32_t kIdHalf = idesc_bf16_f32(kRows, kUnitKeys / 2, false);
  uint32_t qn = 0, seg = 0, gn = 0;
  Walk walk(p, starts, blockIdx.x);
  Segment sg, nx;
  bool more = walk.next(nx), ok = true;
  while (ok && more) {
    sg = nx;
    more = walk.next(nx);
    const bool last_of_head = !more || nx.head != sg.head;
    if (!wait_warp(smem_addr(&ctl.k_full[seg & 1]), (seg >> 1) & 1, ctl, p)) break;
    const uint64_t k0 = sdesc_sw128(sK + (seg & 1) * G::kKBytes, 16, 1024);
    for (int i = 0; i < sg.n; ++i, ++qn) {
      const uint32_t slot = stay ? sg.s0 + i : qn % G::kQStages;
      const uint32_t use = stay ? gn : qn / G::kQStages;
      const uint32_t buf = qn & 1;
      // keys that no row of the step sees are not computed, 128 at a time
      const uint32_t idesc =
          seen(p, sg.key0 + kUnitKeys / 2, sg.s0 + i) ? kIdWide : kIdHalf;
      if (!wait_warp(smem_addr(&ctl.q_full[slot]), use & 1, ctl, p) ||
          (qn >= 2 && !wait_warp(smem_addr(&ctl.s_free[buf]), ((qn >> 1) - 1) & 1, ctl, p))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint64_t q0 = sdesc_sw128(sQ + slot * G::kQBytes, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t qo = ((kk >> 2) * G::kQChunk + (kk & 3) * 32) >> 4;
        const uint32_t ko = ((kk >> 2) * G::kKChunk + (kk & 3) * 32) >> 4;
        if (leader) mma_ss(tmem + kUnitKeys * buf, q0 + qo, k0 + ko, idesc, kk > 0 ? 1u : 0u);
      }
      if (leader) mma_commit(smem_addr(&ctl.s_full[buf]));
      if (leader && !stay) mma_commit(smem_addr(&ctl.q_empty[slot]));
    }
    if (!ok) break;
    if (leader) mma_commit(smem_addr(&ctl.k_empty[seg & 1]));
    ++seg;
    if (stay && last_of_head) {
      // Steps that the range leaves out (it begins or ends inside a unit) were copied
      // to the ring all the same. Their copies have landed too before a slot is given
      // back, and before the CTA ends: the loader must not arm a barrier whose phase
      // is still open, nor a copy write to shared memory that is another CTA's by then.
      for (int i = 0; i < p.steps && ok; ++i) {
        ok = wait_warp(smem_addr(&ctl.q_full[i]), gn & 1, ctl, p);
        if (ok && leader) mma_commit(smem_addr(&ctl.q_empty[i]));
      }
      ++gn;
    }
  }
  // no MMA may still be running when TMEM is released
  if (leader) mma_commit(smem_addr(&ctl.drain));
  drain_wait(smem_addr(&ctl.drain), 0, p);
  __syncwarp();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
key_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ Params p, const __grid_constant__ Starts starts) {
  using G = Geometry<D>;
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  Ctl& ctl = *reinterpret_cast<Ctl*>(dyn_smem);
  const uint32_t start = smem_addr(dyn_smem);
  const uint32_t base = (start + static_cast<uint32_t>(sizeof(Ctl)) + 1023u) & ~1023u;
  if (base + G::kTileBytes > start + smem_bytes<D>()) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusCheck);
    return;
  }
  const uint32_t sK = base, sQ = base + 2 * G::kKBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_addr(&ctl.k_full[s]), 1);
      mbar_init(smem_addr(&ctl.k_empty[s]), 1);
      mbar_init(smem_addr(&ctl.s_full[s]), 2);       // the scores, and the rows' statistics
      mbar_init(smem_addr(&ctl.s_free[s]), kSumWarps);
    }
    for (int s = 0; s < G::kQStages; ++s) {
      mbar_init(smem_addr(&ctl.q_full[s]), 1);
      mbar_init(smem_addr(&ctl.q_empty[s]), 1);
    }
    for (int w = 0; w < kGroups; ++w) {
      for (int q = 0; q < 3; ++q) mbar_init(smem_addr(&ctl.fold[w][q]), 1);
      mbar_init(smem_addr(&ctl.fold_free[w]), 1);
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
  if (p.nr * p.g < kRows && warp < kSumWarps) {
    // rows past nr * g are never loaded: zeros (the sums of their lanes are dropped
    // when the rows are folded)
    uint4* z = reinterpret_cast<uint4*>(dyn_smem + (sQ - start));
    for (int i = threadIdx.x; i < G::kQStages * G::kQBytes / 16; i += 32 * kSumWarps)
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

  // all of a head's steps fit the Q ring: step i stays in slot i
  const bool stay = p.steps <= G::kQStages;
  if (warp < kSumWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    sum_role(ctl, p, starts, tmem);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      if (lane == 0) load_role<D>(&tmQ, &tmK, ctl, p, starts, sK, sQ, stay);
    } else if (warp == kMmaWarp) {
      mma_role<D>(ctl, p, starts, tmem, sK, sQ, stay);
    } else if (warp == kStatWarp) {
      stat_role(ctl, p, starts);
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

// ------------------------------------------------------------- few rows
//
// Where all rows of a head's group fit one tile of at most 256 columns
// (Lq * g <= 256: a prompt's last rows against a long cache), the step is a
// stream of K, and the tiles turn round: S^T = K Q^T with 128 keys on the TMEM
// lanes and every row of the group as a column. A thread owns a key, its sum is
// complete after one tile, and nothing has to be folded or cut; the rows and
// their -lse2 stay in shared memory for as long as the head stays the same.
// (The kernel above spends about as long folding 128 rows into one as on a
// unit's two steps: 32 rows of 6 heads against 131072 keys of 6 K/V heads, 70 us
// there and 38 here; K alone is 30 us at the measured copy rate. Nothing is full: 61 %
// of the memory's rate, 45 % of the tensor cores', 46 % of the exponential unit's; the
// warps wait for a tile's scores, its exponentials and one another.)
//
// The key tiles of all heads are cut into equal ranges, one per CTA. Two S^T
// buffers of 256 columns; of the four warpgroups two take each buffer's tiles,
// half of the columns each, and the second hands its sums to the first.

constexpr int kWinKeys = 128, kWinCols = 256;

template <int D>
struct WinGeometry {
  static constexpr int kChunks = D * 2 / 128;
  static constexpr int kTileBytes = kWinKeys * D * 2;
  static constexpr int kChunkBytes = kWinKeys * 128;
  static constexpr int kQBytes = kWinCols * D * 2;          // one buffer of 256 rows, or two of 128
  static constexpr int kRing = D == 128 ? 5 : 10;
  static constexpr int kTilesBytes = kQBytes + kRing * kTileBytes;
};

struct __align__(16) WinCtl {
  uint64_t k_full[10], k_empty[10];
  uint64_t q_full[2], q_empty[2], n_full[2], n_empty[2];
  uint64_t s_full[2], s_free[2], half_full[2], half_free[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  __align__(16) float nl[kWinCols];      // -lse2 of the Q buffers' columns
  float half_sum[2][kWinKeys];
  int without[2];                        // has a row of a Q buffer no weight?
};
constexpr int kWinCtlBytes = (sizeof(WinCtl) + 1023) / 1024 * 1024;    // then the tiles
template <int D>
__host__ __device__ constexpr int win_smem_bytes() {
  return kWinCtlBytes + WinGeometry<D>::kTilesBytes;
}
static_assert(win_smem_bytes<128>() <= 232448 && win_smem_bytes<64>() <= 232448, "shared memory");

struct WinParams {
  const float* lse;
  float* weights;
  int* status;
  int Lq, Lk, off, n_q, n_kv, g;
  int cols, chunks;      // Lq * g, and 32-column pieces
  int bufs;              // Q buffers: 2 where cols <= 128
  int T;                 // key tiles per (b, K/V head)
  long long W;           // B * n_kv * T
  int causal, accumulate;
  float c;
  long long spin_limit;
};

// Key tiles [t0, t0 + n) of head = b * n_kv + kvh.
struct WinSegment {
  int head, t0, n;
};

struct WinWalk {
  const WinParams& p;
  long long x, end;
  __device__ explicit WinWalk(const WinParams& params) : p(params) {
    x = blockIdx.x * params.W / gridDim.x;
    end = (blockIdx.x + 1ll) * params.W / gridDim.x;
  }
  __device__ bool next(WinSegment& s) {
    if (x >= end) return false;
    s.head = static_cast<int>(x / p.T);
    const long long first = static_cast<long long>(s.head) * p.T;
    s.t0 = static_cast<int>(x - first);
    s.n = static_cast<int>((end - first < p.T ? end - first : p.T) - s.t0);
    x += s.n;
    return true;
  }
};

// a0, a1 += 2^(c s + nl) for the 32 columns whose scores are in s. Column i of them is
// column col0 + i of those that may see the key; with kSeen or kWeighted only the first
// `seen` (from 0 on) count, with kWeighted only rows that have a weight: an infinite key
// or a query that may be anything makes the others' scores NaN. (The loop is chosen for
// 32 columns at once: branches inside it, also uniform ones that are not taken, cost the
// kernel 42 us instead of 38.)
enum Columns { kAll, kSeen, kWeighted };
template <Columns kWhich>
__device__ __forceinline__ void add_columns(uint64_t& a0, uint64_t& a1, const uint32_t (&s)[32],
                                            const float* nl, uint64_t c2, int col0,
                                            unsigned int seen) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 l = *reinterpret_cast<const float4*>(nl + i);
    float x0, x1, x2, x3;
    f32x2_unpack(ffma2(f32x2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c2,
                       f32x2_pack(l.x, l.y)), x0, x1);
    f32x2_unpack(ffma2(f32x2_pack(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), c2,
                       f32x2_pack(l.z, l.w)), x2, x3);
    float e0 = ex2_approx(x0), e1 = ex2_approx(x1), e2 = ex2_approx(x2), e3 = ex2_approx(x3);
    if (kWhich != kAll) {
      const int col = col0 + i;
      if (static_cast<unsigned int>(col) >= seen || (kWhich == kWeighted && l.x == kNoWeight))
        e0 = 0.0f;
      if (static_cast<unsigned int>(col + 1) >= seen || (kWhich == kWeighted && l.y == kNoWeight))
        e1 = 0.0f;
      if (static_cast<unsigned int>(col + 2) >= seen || (kWhich == kWeighted && l.z == kNoWeight))
        e2 = 0.0f;
      if (static_cast<unsigned int>(col + 3) >= seen || (kWhich == kWeighted && l.w == kNoWeight))
        e3 = 0.0f;
    }
    a0 = fadd2(a0, f32x2_pack(e0, e1));
    a1 = fadd2(a1, f32x2_pack(e2, e3));
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
key_weights_few_rows_kernel(const __grid_constant__ CUtensorMap tmQ,
                            const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ WinParams p) {
  using G = WinGeometry<D>;
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  WinCtl& ctl = *reinterpret_cast<WinCtl*>(dyn_smem);
  const uint32_t start = smem_addr(dyn_smem);
  const uint32_t base = (start + static_cast<uint32_t>(sizeof(WinCtl)) + 1023u) & ~1023u;
  if (base + G::kTilesBytes > start + win_smem_bytes<D>()) {     // as in the kernel above
    if (threadIdx.x == 0) atomicOr(p.status, kStatusCheck);
    return;
  }
  const uint32_t sQ = base, sK = base + G::kQBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows_per_buf = kWinCols / p.bufs;
  const uint32_t q_chunk = rows_per_buf * 128, q_buf = G::kChunks * q_chunk;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    for (int s = 0; s < G::kRing; ++s) {
      mbar_init(smem_addr(&ctl.k_full[s]), 1);
      mbar_init(smem_addr(&ctl.k_empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_addr(&ctl.q_full[s]), 1);
      mbar_init(smem_addr(&ctl.q_empty[s]), 1);
      mbar_init(smem_addr(&ctl.n_full[s]), 1);
      mbar_init(smem_addr(&ctl.n_empty[s]), kSumWarps);
      mbar_init(smem_addr(&ctl.s_full[s]), 1);
      mbar_init(smem_addr(&ctl.s_free[s]), 8);
      mbar_init(smem_addr(&ctl.half_full[s]), 4);
      mbar_init(smem_addr(&ctl.half_free[s]), 4);
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
  if (warp < kSumWarps) {
    // columns past Lq * g are never loaded: zeros, so that their scores are 0
    uint4* z = reinterpret_cast<uint4*>(dyn_smem + (sQ - start));
    for (int i = threadIdx.x; i < G::kQBytes / 16; i += 32 * kSumWarps)
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

  WinWalk walk(p);
  WinSegment sg;
  uint32_t seg = 0, it = 0;          // segments and key tiles so far
  if (warp == kLoadWarp) {
    if (lane == 0) {
      bool ok = true;
      const uint32_t q_bytes = static_cast<uint32_t>(G::kChunks * 128 * p.cols);
      while (ok && walk.next(sg)) {
        const int b = sg.head / p.n_kv, kvh = sg.head - b * p.n_kv;
        const uint32_t qb = seg % p.bufs, use = seg / p.bufs;
        if (use > 0 && !spin_wait(smem_addr(&ctl.q_empty[qb]), (use - 1) & 1, ctl, p)) {
          ok = false;
          break;
        }
        const uint32_t qbar = smem_addr(&ctl.q_full[qb]);
        mbar_arrive_expect_tx(qbar, q_bytes);
        for (int ch = 0; ch < G::kChunks; ++ch)
          tma_load_4d(sQ + qb * q_buf + ch * q_chunk, &tmQ, qbar, ch * 64, kvh * p.g, 0, b);
        ++seg;
        for (int t = 0; t < sg.n; ++t, ++it) {
          const uint32_t slot = it % G::kRing, u = it / G::kRing;
          if (u > 0 && !spin_wait(smem_addr(&ctl.k_empty[slot]), (u - 1) & 1, ctl, p)) {
            ok = false;
            break;
          }
          const uint32_t bar = smem_addr(&ctl.k_full[slot]);
          mbar_arrive_expect_tx(bar, G::kTileBytes);
          for (int ch = 0; ch < G::kChunks; ++ch)
            tma_load_4d(sK + slot * G::kTileBytes + ch * G::kChunkBytes, &tmK, bar, ch * 64, kvh,
                        (sg.t0 + t) * kWinKeys, b);
        }
      }
      // let every copy this thread started land before the CTA can exit, also where
      // another role has given up
      for (uint32_t q = 0; q < static_cast<uint32_t>(p.bufs) && q < seg; ++q)
        drain_wait(smem_addr(&ctl.q_full[q]), ((seg - 1 - q) / p.bufs) & 1, p);
      for (uint32_t s = 0; s < G::kRing && s < it; ++s)
        drain_wait(smem_addr(&ctl.k_full[s]), ((it - 1 - s) / G::kRing) & 1, p);
    }
  } else if (warp == kMmaWarp) {
    const bool leader = elect_one();
    const uint32_t idesc = idesc_bf16_f32(kWinKeys, 32 * p.chunks, false);
    bool ok = true;
    while (ok && walk.next(sg)) {
      const uint32_t qb = seg % p.bufs;
      if (!wait_warp(smem_addr(&ctl.q_full[qb]), (seg / p.bufs) & 1, ctl, p)) break;
      ++seg;
      const uint64_t q0 = sdesc_sw128(sQ + qb * q_buf, 16, 1024);
      for (int t = 0; t < sg.n; ++t, ++it) {
        const uint32_t slot = it % G::kRing, buf = it & 1;
        if (!wait_warp(smem_addr(&ctl.k_full[slot]), (it / G::kRing) & 1, ctl, p) ||
            (it >= 2 && !wait_warp(smem_addr(&ctl.s_free[buf]), ((it >> 1) - 1) & 1, ctl, p))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint64_t k0 = sdesc_sw128(sK + slot * G::kTileBytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t ko = ((kk >> 2) * G::kChunkBytes + (kk & 3) * 32) >> 4;
          const uint32_t qo = ((kk >> 2) * q_chunk + (kk & 3) * 32) >> 4;
          if (leader) mma_ss(tmem + kWinCols * buf, k0 + ko, q0 + qo, idesc, kk > 0 ? 1u : 0u);
        }
        if (leader) mma_commit(smem_addr(&ctl.s_full[buf]));
        if (leader) mma_commit(smem_addr(&ctl.k_empty[slot]));
      }
      if (leader && ok) mma_commit(smem_addr(&ctl.q_empty[qb]));
    }
    // no MMA may still be running when TMEM is released
    if (leader) mma_commit(smem_addr(&ctl.drain));
    drain_wait(smem_addr(&ctl.drain), 0, p);
    __syncwarp();
  } else if (warp == kStatWarp) {
    while (walk.next(sg)) {
      const int b = sg.head / p.n_kv, kvh = sg.head - b * p.n_kv;
      const uint32_t qb = seg % p.bufs, use = seg / p.bufs;
      const float* lse = p.lse + (static_cast<size_t>(b) * p.n_q + kvh * p.g) * p.Lq;
      float l[kWinCols / 32];
#pragma unroll
      for (int m = 0; m < kWinCols / 32; ++m) {
        const int col = lane + 32 * m, i = col / p.g;
        l[m] = col < p.cols ? lse[static_cast<size_t>(col - i * p.g) * p.Lq + i] : -INFINITY;
      }
      if (use > 0 && !wait_warp(smem_addr(&ctl.n_empty[qb]), (use - 1) & 1, ctl, p)) break;
      // a row without keys, like a column without a row, has no weight
      bool without = false;
#pragma unroll
      for (int m = 0; m < kWinCols / 32; ++m) {
        if (lane + 32 * m < rows_per_buf)
          ctl.nl[qb * rows_per_buf + lane + 32 * m] = exponent_of(l[m]);
        without |= lane + 32 * m < p.cols && l[m] == -INFINITY;
      }
      without = __any_sync(0xffffffffu, without);
      if (lane == 0) ctl.without[qb] = without;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&ctl.n_full[qb]));
      ++seg;
    }
  } else if (warp < kSumWarps) {
    const int buf = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
    const int r = quarter * 32 + lane;                     // key of the tile = TMEM lane
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + kWinCols * buf;
    const uint64_t c2 = f32x2_pack(p.c, p.c);
    const int split = (p.chunks + 1) / 2;                  // 32-column pieces of the first half
    const int c_from = half ? split : 0, c_to = half ? p.chunks : split;
    bool ok = true;
    while (ok && walk.next(sg)) {
      const uint32_t qb = seg % p.bufs;
      if (!wait_warp(smem_addr(&ctl.n_full[qb]), (seg / p.bufs) & 1, ctl, p)) break;
      ++seg;
      const float* nl_buf = ctl.nl + qb * rows_per_buf;
      const bool without = ctl.without[qb] != 0;
      for (int t = 0; t < sg.n; ++t, ++it) {
        if ((it & 1) != static_cast<uint32_t>(buf)) continue;
        const uint32_t turn = it >> 1;                     // of this buffer
        if (!wait_warp(smem_addr(&ctl.s_full[buf]), turn & 1, ctl, p)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const int key0 = (sg.t0 + t) * kWinKeys, key = key0 + r;
        // columns before `from` do not see the key; those past Lq * g are zeros,
        // and their scores NaN where the key is infinite
        const bool mask = (p.causal && key0 + kWinKeys - 1 > p.off) || p.cols % 32 != 0;
        const int from = p.causal ? max((key - p.off) * p.g, 0) : 0;
        const unsigned int seen = max(p.cols - from, 0);
        uint64_t a0 = f32x2_pack(0.0f, 0.0f), a1 = a0;
        for (int ch = c_from; ch < c_to; ++ch) {
          uint32_t s[32];
          tmem_ld32(lanes + 32 * ch, s);
          tmem_wait_ld(s);
          if (ch == c_to - 1) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&ctl.s_free[buf]));
          }
          const float* nl = nl_buf + 32 * ch;
          const int col0 = 32 * ch - from;
          if (without)
            add_columns<kWeighted>(a0, a1, s, nl, c2, col0, seen);
          else if (mask)
            add_columns<kSeen>(a0, a1, s, nl, c2, col0, seen);
          else
            add_columns<kAll>(a0, a1, s, nl, c2, col0, seen);
        }
        if (c_from == c_to) {                              // a single piece: nothing for this half
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&ctl.s_free[buf]));
        }
        float lo, hi;
        f32x2_unpack(fadd2(a0, a1), lo, hi);
        float sum = lo + hi;
        if (half == 1) {
          if (turn > 0 && !wait_warp(smem_addr(&ctl.half_free[buf]), (turn - 1) & 1, ctl, p)) {
            ok = false;
            break;
          }
          ctl.half_sum[buf][r] = sum;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&ctl.half_full[buf]));
        } else {
          float* out = p.weights + static_cast<size_t>(sg.head) * p.Lk + key;
          const float old = p.accumulate && key < p.Lk ? *out : 0.0f;
          if (!wait_warp(smem_addr(&ctl.half_full[buf]), turn & 1, ctl, p)) {
            ok = false;
            break;
          }
          sum += ctl.half_sum[buf][r];
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&ctl.half_free[buf]));
          if (key < p.Lk) *out = p.accumulate ? old + sum : sum;
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&ctl.n_empty[qb]));
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr int kMaxDevices = 64;
std::mutex g_weights_mutex;
bool g_weights_ready[kMaxDevices] = {};
EncodeTiledFn g_weights_encode = nullptr;

// The register split only works on a CTA launched with at least that many.
template <int D>
bool configure() {
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, key_weights_kernel<D>) != cudaSuccess ||
      fa.numRegs * kThreads < kRegBudget)
    return false;
  return cudaFuncSetAttribute(key_weights_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              smem_bytes<D>()) == cudaSuccess &&
         cudaFuncSetAttribute(key_weights_few_rows_kernel<D>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              win_smem_bytes<D>()) == cudaSuccess;
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
  if (!configure<64>() || !configure<128>()) return ATTN_ERR_UNSUPPORTED;
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

bool supported(int64_t B, int64_t Lq, int64_t Lk, int32_t n_q, int32_t n_kv, int32_t d_h) {
  if ((d_h != 64 && d_h != 128) || n_q / n_kv > kRows) return false;
  constexpr int64_t kMost = int64_t{1} << 30;
  if (Lq > kMost || Lk > kMost || B > kMost || B * n_kv > kMost) return false;
  // units and a CTA's steps are 32-bit; scores in all fit 64 with room
  const int64_t units = B * n_kv * ((Lk + kUnitKeys - 1) / kUnitKeys);
  const int64_t steps = (Lq * (n_q / n_kv) + kRows - 1) / kRows * 2;
  return units <= INT32_MAX - kCtas && steps <= INT64_MAX / units / kCtas &&
         units * steps / kCtas < INT32_MAX / 2 && Lk * (n_q / n_kv) <= INT32_MAX;
}

attn_status_t launch_few_rows(const void* q, const void* k, const float* lse, float* weights,
                              int* status, int64_t B, int64_t Lq, int64_t Lk, int32_t n_q,
                              int32_t n_kv, int32_t d_h, int32_t causal, int32_t accumulate,
                              float scale, cudaStream_t stream) {
  WinParams p{};
  p.lse = lse;
  p.weights = weights;
  p.status = status;
  p.Lq = static_cast<int>(Lq);
  p.Lk = static_cast<int>(Lk);
  p.off = static_cast<int>(Lk - Lq);
  p.n_q = n_q;
  p.n_kv = n_kv;
  p.g = n_q / n_kv;
  p.cols = p.Lq * p.g;
  p.chunks = (p.cols + 31) / 32;
  p.bufs = p.cols <= kWinCols / 2 ? 2 : 1;
  p.T = static_cast<int>((Lk + kWinKeys - 1) / kWinKeys);
  p.W = B * n_kv * p.T;
  p.causal = causal;
  p.accumulate = accumulate;
  p.c = scale * kLog2e;
  p.spin_limit = 1ll << 31;   // about a second at 2 GHz
  CUtensorMap mq, mk;
  if (!encode(&mq, q, d_h, n_q, Lq, B, p.g, p.Lq) || !encode(&mk, k, d_h, n_kv, Lk, B, 1, kWinKeys))
    return ATTN_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.W < kCtas ? p.W : kCtas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (d_h == 128) {
    cfg.dynamicSmemBytes = win_smem_bytes<128>();
    e = cudaLaunchKernelEx(&cfg, key_weights_few_rows_kernel<128>, mq, mk, p);
  } else {
    cfg.dynamicSmemBytes = win_smem_bytes<64>();
    e = cudaLaunchKernelEx(&cfg, key_weights_few_rows_kernel<64>, mq, mk, p);
  }
  if (e != cudaSuccess) return ATTN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
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

  if (Lq * (n_q / n_kv) <= kWinCols)
    return launch_few_rows(q, k, lse, weights, status, B, Lq, Lk, n_q, n_kv, d_h, causal, accumulate,
                           scale, stream);
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
  p.nr = kRows / p.g;
  p.steps = static_cast<int>((Lq + p.nr - 1) / p.nr);
  p.T = static_cast<int>((Lk + kUnitKeys - 1) / kUnitKeys);
  p.causal = causal;
  p.accumulate = accumulate;
  p.c = scale * kLog2e;
  p.spin_limit = 1ll << 31;   // about a second at 2 GHz

  Starts st;
  bool cut;
  p.G = cut_ranges({p.off, p.nr, p.steps, p.T, causal}, B * n_kv, &st, &cut);

  CUtensorMap mq, mk;
  if (!encode(&mq, q, d_h, n_q, Lq, B, p.g, p.nr) || !encode(&mk, k, d_h, n_kv, Lk, B, 1, kUnitKeys))
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
    cfg.dynamicSmemBytes = smem_bytes<128>();
    e = cudaLaunchKernelEx(&cfg, key_weights_kernel<128>, mq, mk, p, st);
  } else {
    cfg.dynamicSmemBytes = smem_bytes<64>();
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
