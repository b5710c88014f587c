// attn_decode4.cu — decode attention (one new token per sequence) over caches
// held in 4 bits (cache4.cuh), whole or behind a sliding window with sinks.
//
// A position costs 160 bytes per K/V head where bf16 takes 512, so at the copy
// rate every element leaves a scheduler about three instruction slots per lane:
// what bounds the step is the stream of rows and, close behind it, turning
// codes into matrix operands. So the codes never leave registers between the
// load and the product, and nothing but the products' results is kept in fp32:
//
//   * every warp streams its own run of positions of one head (the rows of a head
//     are contiguous) through a ring of kStages steps and works alone: it waits for
//     nothing but its own copies until the end. They are 16-byte asynchronous copies,
//     ten a lane and step, and not bulk ones: those cost a warp of this size some
//     sixty instructions a step in moves to uniform registers and barriers, of
//     some 350 a 16-position chunk with these;
//   * S^T = K Q^T with m16n8k16 products, 16 positions x 8 heads. A code is put
//     into the upper mantissa bits of a bf16 16 (bits 3..6: 16 + code, exact),
//     one shift and one logic instruction for two codes; a group's scale is
//     applied to the fp32 sum of its 32 channels, and the rest is a product of its
//     own, in which a position's words of (scale, lo) are the operand as they are:
//       s = sum_g scale_g (sum (16 + code) q) + (scale_g, lo_g) . (-16 sum q, sum q)
//     (the sums of q in three bf16 parts), so no value of K is rounded;
//   * O^T += V^T P^T likewise, 16 channels x 8 heads: with a position's and group's
//     center c, the code next to a value of 0, V = (lo + scale c) + scale (code - c),
//     the codes less c (exact) against scale_g P (rounded to bf16), and
//     sum_j P_j (lo_gj + scale_gj c_gj) in fp32 beside it. So a rounding counts as
//     much as one of P counts for V itself. (With c = 0 it counts for V - lo, up to 15
//     steps of one sign: over 131072 positions, a channel of each group six times the
//     others, O was 0.0056 of itself off, with c = 7.5 0.0037, now 0.0021, of which O's
//     own rounding is 0.0016.) Each lane works the centers of one position out, while
//     the scores' products run, and leaves them in shared memory (36.5 us where those
//     positions took 35.5 without; P^T in two bf16 parts, 0.0016, 40.3). P^T is
//     turned by movmatrix; the two rows that a lane's operand pairs up are brought
//     together by one byte permutation per four codes.
// (mma.sync and not tcgen05: those operands come from shared memory or tensor
// memory, and writing the bf16 values there would cost more than the product.)
//
// The list of 16-position chunks over all sequences and heads is cut into equal
// runs, one per warp. At the end the warps of a CTA that stand in the same head
// merge their results in shared memory, and a combine kernel merges what the
// CTAs left. Lengths are read on the device.
//
// Measured: 16 sequences of 1024 to 8192 positions, 32 heads on 8, 32 us (95 MB of
// rows: 14 us at the copy rate); one of 131072, 36 heads on 6, 36.5 us (126 MB: 19 us);
// 64 sequences behind a window of 1024 with 4 sinks, 32 heads on 8, 31.6 us (79 MB: 12;
// 128 heads on 8: 50).
// Longer lists cost 22 us more per 126 MB, 87 % of the copy rate; some 13 us are there
// whatever the length: finding the runs, the first step's copies, the merge and the
// combine.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "attn_prefill.h"
#include "cache4.cuh"
#include "sm103_ptx.cuh"

namespace gb300_host {
attn_status_t device_status_word(cudaStream_t stream, int** status);
}

namespace {

using namespace gb300;

constexpr int kChunk = 16;                         // positions per product, unit of the runs
constexpr int kStep = 2 * kChunk;                  // positions per step of a warp
constexpr int kStepBytes = kStep * kRow4Bytes;     // of K, and of V
constexpr int kStages = 2;                           // steps under way per warp
constexpr int kRingBytes = kStages * 2 * kStepBytes;
// Behind its ring a warp keeps, of a step's V, mid = lo + scale c [position][group] in
// fp32, and bf16 16 + c of positions t + 8 h and t + 8 h + 4 of its chunks, [h][t][group]
// [which of the two].
constexpr int kMidBytes = kStep * kRow4Groups * 4;
constexpr int kWarpBytes = kRingBytes + kMidBytes + kStep * kRow4Groups * 2;
constexpr int kCtas = 152;                         // one per SM
constexpr int kMaxG = 16;
constexpr float kRescale = 8.0f;                   // lazy running maximum (log2 units)
// A running maximum before the first score: below every one that counts, and finite,
// so that nothing has to be told apart from a maximum of -inf.
constexpr float kNoMax = -3.4028234663852886e38f;

// NT: the group's query heads in tiles of 8: one where they fit, as 12 warps of it have
// the registers, and 8 with two, whose second tile does the work of 8 heads for as few as
// there are. (16 sequences of up to 8192 positions: 8 heads a group 32.6 us in one tile,
// 42.3 in two; 9, 12 and 16 heads 43, 44 and 45. One of 131072: 36.6 and 48.4; 12 and 16
// heads 50. With two the compiler spills: 32 bytes a thread stored, 16 loaded.)
template <int NT>
constexpr int kWarpsOf = NT == 1 ? 12 : 8;
template <int NT>
constexpr int kSmemOf = kWarpsOf<NT> * kWarpBytes;
static_assert(kMaxG * kRow4Dim * 4 <= kWarpBytes, "a warp's result fits its ring");

struct Params4 {
  const uint16_t* q;       // bf16 [B, n_q, 128]
  const uint8_t *k4, *v4;
  const int* lens;
  float* part_o;           // fp32 [2 (B * n_kv + CTAs)][g][128]
  float2* part_ml;         // running maximum (log2 units) and sum (0: nothing here)
  int* ends;               // [B * n_kv][2] CTAs that hold a head's first and last chunk
  int B, C, n_q, n_kv, g;
  int window, sinks;       // window 0: everything before lens[b]
  int walkers;             // warps that may have a run
  float c;                 // scale * log2(e)
  uint32_t sixteens;       // bf16 16 twice (codes16)
};

// A sequence's visible positions, [0, sunk) and [low, len), in chunks.
struct Seen4 {
  int len, low, sunk, na, chunks;
  __device__ Seen4(const Params4& p, int b) {
    len = min(max(p.lens[b], 0), p.C);
    low = p.window > 0 ? max(0, len - p.window) : 0;
    sunk = p.window > 0 ? min(p.sinks, low) : 0;
    na = (sunk + kChunk - 1) / kChunk;
    chunks = na + (len - low + kChunk - 1) / kChunk;
  }
};

// A warp's place in the list: sequence, head, chunk; `left` chunks of its run to go.
struct Walk4 {
  int b, u, t, left;
  int len, low, sunk, na, chunks;
  __device__ void enter(const Params4& p) {
    const Seen4 s(p, b);
    len = s.len;
    low = s.low;
    sunk = s.sunk;
    na = s.na;
    chunks = s.chunks;
  }
  // Past n chunks of this head.
  __device__ void move(const Params4& p, int n) {
    t += n;
    left -= n;
    if (left == 0 || t < chunks) return;
    t = 0;
    if (++u < p.n_kv) return;
    u = 0;
    do {
      if (++b >= p.B) {     // (cannot be with chunks left)
        left = 0;
        return;
      }
      enter(p);
    } while (chunks == 0);
  }
};

// A run of neighbouring positions of one head: the next part of a walk.
struct Part4 {
  int units, pos, rows;    // chunks, first position, rows that count
  __device__ Part4(const Walk4& w) {
    const bool sink = w.t < w.na;
    const int until = sink ? w.na : w.chunks, end = sink ? w.sunk : w.len;
    pos = sink ? w.t * kChunk : w.low + (w.t - w.na) * kChunk;
    units = min(w.left, until - w.t);
    rows = w.t + units == until ? end - pos : units * kChunk;
  }
};

// What a part is to its segment, which is what one run has of one head.
constexpr int kFirst = 1, kLast = 2;            // it is its first, last part
constexpr int kHeadStart = 4, kHeadEnd = 8;     // it holds the head's first, last chunk
constexpr int kRunEnd = 16;
constexpr int kNotes = kStages + 1;             // parts that copies may be ahead by, and one

// The warp's copies: walks the run and leaves a note of each part for the products, so
// that only one place of the walk is kept.
struct Sender {
  Walk4 w;
  int rows;                    // of this part, to go
  uint32_t parts;              // begun so far
  int64_t at;                  // byte offset of the next row
  bool fresh;                  // the next part begins a segment
  __device__ void begin(const Walk4& walk) {
    w = walk;
    rows = 0;
    parts = 0;
    fresh = true;
  }
  // The next part; its note is (rows, head, flags).
  __device__ int4 next(const Params4& p) {
    const Part4 part(w);
    rows = part.rows;
    const int hd = w.b * p.n_kv + w.u;
    at = (static_cast<int64_t>(hd) * p.C + part.pos) * kRow4Bytes;
    const bool head_end = w.t + part.units == w.chunks, run_end = part.units == w.left;
    const int start = (fresh ? kFirst : 0) | (w.t == 0 ? kHeadStart : 0);
    fresh = head_end || run_end;
    w.move(p, part.units);
    ++parts;
    return make_int4(rows, hd,
                     start | (fresh ? kLast : 0) | (head_end ? kHeadEnd : 0) | (run_end ? kRunEnd : 0),
                     0);
  }
};

// w W / G, by a 32-bit division where that holds it (a 64-bit one is a hundred
// instructions of a short step).
__device__ __forceinline__ int part_of(int w, int W, int G) {
  const uint64_t x = static_cast<uint64_t>(w) * static_cast<uint32_t>(W);
  return (x >> 32) == 0 ? static_cast<int>(static_cast<uint32_t>(x) / static_cast<uint32_t>(G))
                        : static_cast<int>(x / static_cast<uint32_t>(G));
}

// Where walker w's run starts: each lane sums a run of sequences, a scan places
// them, and the lane that holds the first chunk finds it.
__device__ __forceinline__ Walk4 walk_start(const Params4& p, int w) {
  const int lane = threadIdx.x & 31;
  const int run = (p.B + 31) / 32, b0 = min(lane * run, p.B), b1 = min(b0 + run, p.B);
  int sum = 0;                                 // (all chunks together are below 2^31)
#pragma unroll 4
  for (int b = b0; b < b1; ++b) sum += Seen4(p, b).chunks;
  sum *= p.n_kv;
  int incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += n;
  }
  const int W = __shfl_sync(0xffffffffu, incl, 31);
  const int G = min(p.walkers, W);             // every run has a chunk
  Walk4 x{};
  if (w >= G) return x;
  const int x0 = part_of(w, W, G);
  int at = incl - sum;
  const bool mine = x0 >= at && x0 < incl;
  int b = 0, u = 0, t = 0;
  if (mine) {
    for (int i = b0; i < b1; ++i) {
      const int T = Seen4(p, i).chunks, here = T * p.n_kv;
      if (x0 - at < here) {
        b = i;
        u = static_cast<int>(static_cast<uint32_t>(x0 - at) / static_cast<uint32_t>(T));
        t = x0 - at - u * T;
        break;
      }
      at += here;
    }
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
  x.b = __shfl_sync(0xffffffffu, b, src);
  x.u = __shfl_sync(0xffffffffu, u, src);
  x.t = __shfl_sync(0xffffffffu, t, src);
  x.left = part_of(w + 1, W, G) - x0;
  x.enter(p);
  return x;
}

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// All but the last `kAfter` groups of this thread's copies have landed.
template <int kAfter>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kAfter) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ int4 lds_desc(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// D = A B + C, 16 x 8 x 16, bf16 operands.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                         float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Codes n and n + 4 of a word (or the n-th of its two halves) as bf16 16 + code: one
// shift and one logic instruction, which takes the 16s from a register (`sixteens`,
// from the parameters: a constant that the compiler knows becomes a second
// instruction with another immediate, 54 more a chunk).
template <int n>
__device__ __forceinline__ uint32_t codes16(uint32_t w, uint32_t sixteens) {
  const uint32_t at = n == 0 ? w << 3 : w >> (4 * n - 3);
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x00780078, %2, 0xEA;" : "=r"(r) : "r"(at), "r"(sixteens));   // (at & m) | 16s
  return r;
}
// The codes less their centers, exactly: `center` is bf16 16 + c of each.
template <int n>
__device__ __forceinline__ uint32_t codes_less(uint32_t w, uint32_t sixteens, uint32_t center) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(codes16<n>(w, sixteens)), "r"(center));
  return r;
}

// What a warp holds of one head: lane (r = lane / 4, t = lane % 4) has, for heads
// 8 n + 2 t and + 1, channels 32 g + 4 r + 2 j (o[.][0..1]) and + 1 (o[.][2..3]),
// its own share of sum_j P_j (lo_gj + scale_gj c_gj) and of the row sum, and the running
// maximum.
template <int NT>
struct Acc {
  float o[NT][4][2][4];
  float mids[NT][4][2];
  float m[NT][2], l[NT][2];
  __device__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][g][j][e] = 0.0f;
        mids[n][g][0] = mids[n][g][1] = 0.0f;
      }
      m[n][0] = m[n][1] = kNoMax;
      l[n][0] = l[n][1] = 0.0f;
    }
  }
  // Sums over the lanes; then lane (r, t) has head 8 n + 2 t + e whole.
  __device__ void finish() {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], off);
#pragma unroll
          for (int g = 0; g < 4; ++g)
            mids[n][g][e] += __shfl_xor_sync(0xffffffffu, mids[n][g][e], off);
        }
      }
  }
  // Channels 32 g + 4 r .. + 3 of head 8 n + 2 t + e.
  __device__ float4 channels(int n, int g, int e) const {
    const float mid = mids[n][g][e];
    return make_float4(o[n][g][0][e] + mid, o[n][g][0][2 + e] + mid, o[n][g][1][e] + mid,
                       o[n][g][1][2 + e] + mid);
  }
};

template <int NT>
__global__ void __launch_bounds__(32 * kWarpsOf<NT>, 1)
decode4_split_kernel(const Params4 p) {
  constexpr int kWarps = kWarpsOf<NT>;
  extern __shared__ __align__(128) uint8_t dyn_smem[];
  __shared__ __align__(16) int4 note[kWarps][kNotes];
  __shared__ int head_of[kWarps];             // head that the warp ended in, -1: had no run
  __shared__ float m_of[kWarps][8 * NT], l_of[kWarps][8 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, t = lane & 3;
  const int cta = static_cast<int>(blockIdx.x), w = cta * kWarps + warp;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const uint32_t ring = smem_addr(dyn_smem) + warp * kWarpBytes;
  Sender ahead;
  ahead.begin(walk_start(p, w));
  int slot_in = 0;                            // ring slot of the next copies
  auto send = [&]() {                         // the next step's rows of K and V
    if (ahead.rows <= 0 && ahead.w.left > 0) {
      const int4 n = ahead.next(p);
      if (lane == 0) note[warp][(ahead.parts - 1) % kNotes] = n;
    }
    if (ahead.rows > 0) {
      const uint32_t dst = ring + slot_in * 2 * kStepBytes + 16 * lane;
      const uint8_t *k = p.k4 + ahead.at + 16 * lane, *v = p.v4 + ahead.at + 16 * lane;
      const int left = min(ahead.rows, kStep) * kRow4Bytes - 16 * lane;   // bytes from the lane's on
#pragma unroll
      for (int i = 0; i < kStepBytes / 512; ++i)
        if (i * 512 < left) {
          copy16(dst + i * 512, k + i * 512);
          copy16(dst + kStepBytes + i * 512, v + i * 512);
        }
      ahead.rows -= kStep;
      ahead.at += kStepBytes;
    }
    copies_commit();
    slot_in = slot_in + 1 == kStages ? 0 : slot_in + 1;
  };

  // position of row i of a chunk's products (i < 8; the others are 8 further on): rows
  // 2 a and 2 a + 1 are positions a and a + 4, so that eight lanes' 16-byte loads of a
  // chunk's 80-byte rows, of K (two rows) and of V (four), fall into different banks
  const int kpos = (r >> 1) + 4 * (r & 1);
  const uint32_t half = (r & 1) ? 0x7632u : 0x5410u;
  const uint32_t sixteens = p.sixteens;
  const uint32_t mid_out = ring + kRingBytes + 16 * lane, mid_in = ring + kRingBytes + 16 * kpos;
  const uint32_t center_in = ring + kRingBytes + kMidBytes + 16 * t;
  const uint32_t center_out = center_in + 64 * (lane >> 3) + 2 * (r & 1);
  Acc<NT> acc;
  uint32_t qf[NT][4][4];                      // Q as the products' second operand
  uint32_t qo[NT][3];                         // (-16 sum q, sum q) of group t, three bf16 parts
  int hd = -1, where = 0;                     // the segment: head, kHeadStart and kHeadEnd

  // One step's products; kFull: all of its rows count.
  auto step = [&](auto full_step, int slot, int valid) {
    constexpr bool kFull = decltype(full_step)::value;
    const uint32_t sk = ring + slot * 2 * kStepBytes, sv = sk + kStepBytes;
    const uint32_t row0 = kpos * kRow4Bytes, row1 = row0 + 8 * kRow4Bytes;

    // S^T: rows r and r + 8 of each chunk, heads 2 t and 2 t + 1 of each tile
    float s[2][NT][4];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t at = sk + c * kChunk * kRow4Bytes;
      const uint4 k0 = lds128(at + row0 + 16 * t), k1 = lds128(at + row1 + 16 * t);
      const uint4 p0 = lds128(at + row0 + kRow4Codes), p1 = lds128(at + row1 + kRow4Codes);
      const uint32_t c0[4] = {k0.x, k0.y, k0.z, k0.w}, c1[4] = {k1.x, k1.y, k1.z, k1.w};
      const uint32_t m0[4] = {p0.x, p0.y, p0.z, p0.w}, m1[4] = {p1.x, p1.y, p1.z, p1.w};
      const uint32_t w0 = lds32(at + row0 + kRow4Codes + 4 * t);
      const uint32_t w1 = lds32(at + row1 + kRow4Codes + 4 * t);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float d[4];
        mma16816(d, w0, w1, w0, w1, qo[n][0], qo[n][1], 0.0f, 0.0f, 0.0f, 0.0f);
        mma16816(s[c][n], w0, w1, 0u, 0u, qo[n][2], 0u, d[0], d[1], d[2], d[3]);
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t a00 = codes16<0>(c0[g], sixteens), a01 = codes16<0>(c1[g], sixteens);
        const uint32_t a02 = codes16<1>(c0[g], sixteens), a03 = codes16<1>(c1[g], sixteens);
        const uint32_t a10 = codes16<2>(c0[g], sixteens), a11 = codes16<2>(c1[g], sixteens);
        const uint32_t a12 = codes16<3>(c0[g], sixteens), a13 = codes16<3>(c1[g], sixteens);
        const float s0 = row4_scale(m0[g]), s1 = row4_scale(m1[g]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float d[4], f[4];
          mma16816(d, a00, a01, a02, a03, qf[n][g][0], qf[n][g][1], 0.0f, 0.0f, 0.0f, 0.0f);
          mma16816(f, a10, a11, a12, a13, qf[n][g][2], qf[n][g][3], d[0], d[1], d[2], d[3]);
          s[c][n][0] = fmaf(s0, f[0], s[c][n][0]);
          s[c][n][1] = fmaf(s0, f[1], s[c][n][1]);
          s[c][n][2] = fmaf(s1, f[2], s[c][n][2]);
          s[c][n][3] = fmaf(s1, f[3], s[c][n][3]);
        }
      }
    }
    // the centers of V's position `lane`
    {
      const uint4 pv = lds128(sv + lane * kRow4Bytes + kRow4Codes);
      const uint32_t words[4] = {pv.x, pv.y, pv.z, pv.w};
      float mid[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float scale = row4_scale(words[g]), lo = row4_low(words[g]);
        float inv;                            // (near enough: any whole c will do)
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
        // 2^23 + c, c = -lo / scale rounded and kept in 0 .. 15 (0 where that is not a number)
        const float at = fmaf(__saturatef(lo * (-1.0f / 15.0f) * inv), 15.0f, 8388608.0f);
        mid[g] = kFull || lane < valid ? fmaf(scale, at - 8388608.0f, lo) : 0.0f;
        // bf16 16 + c is 0x4180 + 8 c
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(center_out + 4 * g),
                     "h"(static_cast<uint16_t>(__float_as_uint(at) * 8u + 0x4180u))
                     : "memory");
      }
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(mid_out), "f"(mid[0]), "f"(mid[1]),
                   "f"(mid[2]), "f"(mid[3])
                   : "memory");
    }

    bool need = false;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[c][n][e] = kFull || c * kChunk + kpos + 4 * (e & 2) < valid ? s[c][n][e] * p.c
                                                                        : -INFINITY;
          need |= s[c][n][e] > acc.m[n][e & 1] + kRescale;
        }
    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = fmaxf(fmaxf(s[0][n][e], s[0][n][2 + e]), fmaxf(s[1][n][e], s[1][n][2 + e]));
#pragma unroll
          for (int off = 4; off < 32; off <<= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
          const float m = fmaxf(acc.m[n][e], top);
          const float alpha = ex2_approx(acc.m[n][e] - m);
          acc.m[n][e] = m;
          acc.l[n][e] *= alpha;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            acc.mids[n][g][e] *= alpha;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              acc.o[n][g][j][e] *= alpha;
              acc.o[n][g][j][2 + e] *= alpha;
            }
          }
        }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[c][n][e] = ex2_approx(s[c][n][e] - acc.m[n][e & 1]);
          acc.l[n][e & 1] += s[c][n][e];
        }

    // O^T: P times the scale of its position's group, turned, against V's codes
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t at = sv + c * kChunk * kRow4Bytes;
      const uint4 p0 = lds128(at + row0 + kRow4Codes), p1 = lds128(at + row1 + kRow4Codes);
      // (rows that do not count may hold anything)
      const uint32_t keep0 = kFull || c * kChunk + kpos < valid ? ~0u : 0u;
      const uint32_t keep1 = kFull || c * kChunk + kpos + 8 < valid ? ~0u : 0u;
      const uint32_t m0[4] = {p0.x & keep0, p0.y & keep0, p0.z & keep0, p0.w & keep0};
      const uint32_t m1[4] = {p1.x & keep1, p1.y & keep1, p1.z & keep1, p1.w & keep1};
      // rows 2 t, 2 t + 1 (positions t, t + 4) and 8 further on; codes of block r / 2
      const uint32_t base = at + t * kRow4Bytes + 16 * (r >> 1);
      const uint4 va = lds128(base), vb = lds128(base + 4 * kRow4Bytes);
      const uint4 vc = lds128(base + 8 * kRow4Bytes), vd = lds128(base + 12 * kRow4Bytes);
      const uint4 l0 = lds128(mid_in + c * kChunk * 16), l1 = lds128(mid_in + (c * kChunk + 8) * 16);
      const uint32_t mid0[4] = {l0.x, l0.y, l0.z, l0.w}, mid1[4] = {l1.x, l1.y, l1.z, l1.w};
      const uint4 cl = lds128(center_in + 128 * c), ch = lds128(center_in + 128 * c + 64);
      const uint32_t cen0[4] = {cl.x, cl.y, cl.z, cl.w}, cen1[4] = {ch.x, ch.y, ch.z, ch.w};
      const uint32_t ca[4] = {va.x, va.y, va.z, va.w}, cb[4] = {vb.x, vb.y, vb.z, vb.w};
      const uint32_t cc[4] = {vc.x, vc.y, vc.z, vc.w}, cd[4] = {vd.x, vd.y, vd.z, vd.w};
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t ab = __byte_perm(ca[g], cb[g], half), gh = __byte_perm(cc[g], cd[g], half);
        const uint32_t a0 = codes_less<0>(ab, sixteens, cen0[g]), a1 = codes_less<1>(ab, sixteens, cen0[g]);
        const uint32_t a2 = codes_less<0>(gh, sixteens, cen1[g]), a3 = codes_less<1>(gh, sixteens, cen1[g]);
        const uint32_t b0 = codes_less<2>(ab, sixteens, cen0[g]), b1 = codes_less<3>(ab, sixteens, cen0[g]);
        const uint32_t b2 = codes_less<2>(gh, sixteens, cen1[g]), b3 = codes_less<3>(gh, sixteens, cen1[g]);
        const float s0 = row4_scale(m0[g]), s1 = row4_scale(m1[g]);
        const float l0 = __uint_as_float(mid0[g]), l1 = __uint_as_float(mid1[g]);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float* x = s[c][n];
          const uint32_t x0 = transpose8x8(pack_bf16x2(x[0] * s0, x[1] * s0));
          const uint32_t x1 = transpose8x8(pack_bf16x2(x[2] * s1, x[3] * s1));
          acc.mids[n][g][0] = fmaf(x[0], l0, fmaf(x[2], l1, acc.mids[n][g][0]));
          acc.mids[n][g][1] = fmaf(x[1], l0, fmaf(x[3], l1, acc.mids[n][g][1]));
          float(&d0)[4] = acc.o[n][g][0];
          float(&d1)[4] = acc.o[n][g][1];
          mma16816(d0, a0, a1, a2, a3, x0, x1, d0[0], d0[1], d0[2], d0[3]);
          mma16816(d1, b0, b1, b2, b3, x0, x1, d1[0], d1[1], d1[2], d1[3]);
        }
      }
    }
  };
  // Q of a head: on its way, and as operands.
  uint4 raw[NT][4];
  auto fetch_q = [&](int head) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        raw[n][g] = make_uint4(0u, 0u, 0u, 0u);
        if (8 * n + r < p.g)
          raw[n][g] = *reinterpret_cast<const uint4*>(
              p.q + (static_cast<int64_t>(head) * p.g + 8 * n + r) * kRow4Dim + 32 * g + 8 * t);
      }
  };
  auto turn_q = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float own = 0.0f;                       // the sum of group t
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint4 v = raw[n][g];
        // channels e and e + 4 of the lane's eight, as the codes come
        qf[n][g][0] = __byte_perm(v.x, v.z, 0x5410);
        qf[n][g][1] = __byte_perm(v.x, v.z, 0x7632);
        qf[n][g][2] = __byte_perm(v.y, v.w, 0x5410);
        qf[n][g][3] = __byte_perm(v.y, v.w, 0x7632);
        float sum = 0.0f;
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sum += __uint_as_float(u[e] << 16) + __uint_as_float(u[e] & 0xFFFF0000u);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (g == t) own = sum;
      }
      float rest[2] = {-16.0f * own, own};
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        qo[n][k] = pack_bf16x2(rest[0], rest[1]);
        rest[0] -= __uint_as_float(qo[n][k] << 16);
        rest[1] -= __uint_as_float(qo[n][k] & 0xFFFF0000u);
      }
    }
  };

  // Copies go out first, but for the first head's Q: behind them it would wait for all
  // that the other warps ask for as well.
  bool going = ahead.w.left > 0;
  if (going) fetch_q(ahead.w.b * p.n_kv + ahead.w.u);
  for (int i = 0; i < kStages; ++i) send();
  __syncwarp();
  int slot = 0;
  for (uint32_t part = 0; going; ++part) {
    const int4 now = lds_desc(smem_addr(&note[warp][part % kNotes]));
    if (now.z & kFirst) {
      hd = now.y;
      where = 0;
      acc.clear();
      if (part > 0) fetch_q(hd);
      turn_q();
    }
    where |= now.z;
    for (int rows = now.x; rows > 0; rows -= kStep) {
      copies_wait<kStages - 1>();
      __syncwarp();
      if (rows >= kStep) step(std::true_type{}, slot, kStep);
      else step(std::false_type{}, slot, rows);
      __syncwarp();
      send();
      slot = slot + 1 == kStages ? 0 : slot + 1;
    }
    going = !(now.z & kRunEnd);
    if (!(now.z & kLast) || !going) continue;

    // the head goes on in no other warp's run but earlier ones: its end goes out as it is
    acc.finish();
    if (lane == 0) {
      if (where & kHeadStart) p.ends[2 * hd] = cta;
      p.ends[2 * hd + 1] = cta;
    }
    const int64_t place = 2 * (static_cast<int64_t>(hd) + cta) + 1;
    // without a run of this CTA before it, the run's place stays empty
    const bool alone = (where & kHeadStart) || warp == 0;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 8 * n + 2 * t + e;
        if (h >= p.g) continue;
        float* out = p.part_o + (place * p.g + h) * kRow4Dim + 4 * r;
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<float4*>(out + 32 * g) = acc.channels(n, g, e);
        if (r == 0) {
          p.part_ml[place * p.g + h] = make_float2(acc.m[n][e], acc.l[n][e]);
          if (alone) p.part_ml[(place - 1) * p.g + h] = make_float2(kNoMax, 0.0f);
        }
      }
  }

  // The warps that ended in one head are neighbours: their results meet in shared memory,
  // first the maxima and then, brought to the largest, sums and outputs.
  if (hd >= 0) {
    acc.finish();
    if (r == 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m_of[warp][8 * n + 2 * t] = acc.m[n][0];
        m_of[warp][8 * n + 2 * t + 1] = acc.m[n][1];
      }
    }
    if (lane == 0) {
      if (where & kHeadStart) p.ends[2 * hd] = cta;
      if (where & kHeadEnd) p.ends[2 * hd + 1] = cta;
    }
  }
  if (lane == 0) head_of[warp] = hd;
  __syncthreads();
  int first = warp, last = warp + 1;
  while (first > 0 && head_of[first - 1] == hd) --first;
  while (last < kWarps && head_of[last] == hd) ++last;
  if (hd >= 0) {
    float* own = reinterpret_cast<float*>(dyn_smem + warp * kWarpBytes);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 8 * n + 2 * t + e;
        if (h >= p.g) continue;
        float m = kNoMax;
        for (int i = first; i < last; ++i) m = fmaxf(m, m_of[i][h]);
        const float f = ex2_approx(acc.m[n][e] - m);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float4 v = acc.channels(n, g, e);
          *reinterpret_cast<float4*>(own + h * kRow4Dim + 32 * g + 4 * r) =
              make_float4(f * v.x, f * v.y, f * v.z, f * v.w);
        }
        if (r == 0) l_of[warp][h] = f * acc.l[n][e];
      }
  }
  __syncthreads();
  if (hd < 0) return;
  const int64_t place = 2 * (static_cast<int64_t>(hd) + cta);
  // the head's end is in this CTA, in the next warp's first segment, or not here
  const bool tail = last < kWarps && head_of[last] >= 0 && !(where & kHeadEnd);
  for (int item = (warp - first) * 32 + lane; item < p.g * 32; item += (last - first) * 32) {
    const int h = item >> 5, quad = item & 31;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = first; i < last; ++i) {
      const float4 v =
          *reinterpret_cast<const float4*>(dyn_smem + i * kWarpBytes + (h * kRow4Dim + 4 * quad) * 4);
      sum.x += v.x;
      sum.y += v.y;
      sum.z += v.z;
      sum.w += v.w;
    }
    *reinterpret_cast<float4*>(p.part_o + (place * p.g + h) * kRow4Dim + 4 * quad) = sum;
    if (quad == 0) {
      float m = kNoMax, l = 0.0f;
      for (int i = first; i < last; ++i) {
        m = fmaxf(m, m_of[i][h]);
        l += l_of[i][h];
      }
      p.part_ml[place * p.g + h] = make_float2(m, l);
    }
  }
  if (warp == last - 1 && !tail && lane < p.g)
    p.part_ml[(place + 1) * p.g + lane] = make_float2(kNoMax, 0.0f);
}

// O = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s over a row's places (two per
// CTA of the head, some empty): kPerRow warps per (b, query head). A warp reads
// the maxima and sums of its share of the places at once, a lane each, and then
// only the outputs of those that hold something, four under way. A sequence without a key gets
// O = 0 and LSE = -inf.
constexpr int kCombineWarps = 8;

template <int kPerRow>
__global__ void __launch_bounds__(32 * kCombineWarps)
decode4_combine_kernel(uint16_t* o, float* lse, const Params4 p) {
  constexpr int kRows = kCombineWarps / kPerRow;
  __shared__ float red_m[kCombineWarps], red_w[kCombineWarps];
  __shared__ float4 red_o[kCombineWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % kPerRow;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + warp / kPerRow;   // b * n_q + h
  const bool live = row < static_cast<int64_t>(p.B) * p.n_q;
  float m = kNoMax, l = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  bool keys = false;
  if (live) {
    const int64_t hd = row / p.g;
    const int h = static_cast<int>(row - hd * p.g);
    keys = p.lens[hd / p.n_kv] > 0;
    const int2 ends = reinterpret_cast<const int2*>(p.ends)[hd];
    const int64_t first = 2 * (hd + ends.x);
    const int n = keys ? 2 * (ends.y - ends.x + 1) : 0;
    const int share = min(32, (n + kPerRow - 1) / kPerRow);
    for (int at = share * sub; at < n; at += share * kPerRow) {
      const float2 ml = lane < share && at + lane < n ? p.part_ml[(first + at + lane) * p.g + h]
                                                      : make_float2(kNoMax, 0.0f);
      float top = ml.x;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const float mn = fmaxf(m, top);
      const float a = ex2_approx(m - mn), f = ex2_approx(ml.x - mn);
      float part = f * ml.y;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
      l = fmaf(l, a, part);
      m = mn;
      acc.x *= a;
      acc.y *= a;
      acc.z *= a;
      acc.w *= a;
      // (a place whose scores are all NaN has no maximum, but NaN for a sum)
      unsigned some = __ballot_sync(0xffffffffu, ml.y != 0.0f);
      while (some) {
        float4 v[4];
        float fs[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int src = some ? __ffs(some) - 1 : -1;
          some &= some - 1;
          fs[k] = __shfl_sync(0xffffffffu, f, src < 0 ? 0 : src);
          v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (src >= 0)
            v[k] = *reinterpret_cast<const float4*>(
                p.part_o + ((first + at + src) * p.g + h) * kRow4Dim + 4 * lane);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          acc.x = fmaf(fs[k], v[k].x, acc.x);
          acc.y = fmaf(fs[k], v[k].y, acc.y);
          acc.z = fmaf(fs[k], v[k].z, acc.z);
          acc.w = fmaf(fs[k], v[k].w, acc.w);
        }
      }
    }
  }
  if (kPerRow > 1) {
    red_o[warp][lane] = acc;
    if (lane == 0) {
      red_m[warp] = m;
      red_w[warp] = l;
    }
    __syncthreads();
    if (sub != 0) return;
    m = red_m[warp];
#pragma unroll
    for (int k = 1; k < kPerRow; ++k) m = fmaxf(m, red_m[warp + k]);
    acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    l = 0.0f;
#pragma unroll
    for (int k = 0; k < kPerRow; ++k) {
      const float f = ex2_approx(red_m[warp + k] - m);
      const float4 v = red_o[warp + k][lane];
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
      l = fmaf(f, red_w[warp + k], l);
    }
  }
  if (!live) return;
  const float inv = keys ? 1.0f / l : 0.0f;
  *reinterpret_cast<uint2*>(o + row * kRow4Dim + 4 * lane) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0) lse[row] = keys ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

// --------------------------------------------------------------------- host

constexpr int kMaxDevices = 64;
std::mutex g_mutex;
bool g_ready[kMaxDevices];

attn_status_t device_ready(cudaStream_t stream, int** status) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_UNSUPPORTED;
  // device check (sm_103) and the status word come from the forward's set-up
  const attn_status_t ds = gb300_host::device_status_word(stream, status);
  if (ds != ATTN_OK) return ds;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (g_ready[dev]) return ATTN_OK;
  // one-time set-up: not inside a stream capture
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess || cs != cudaStreamCaptureStatusNone) {
    cudaGetLastError();
    return ATTN_ERR_UNSUPPORTED;
  }
  if (cudaFuncSetAttribute(decode4_split_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmemOf<1>) != cudaSuccess ||
      cudaFuncSetAttribute(decode4_split_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmemOf<2>) != cudaSuccess)
    return ATTN_ERR_CUDA;
  g_ready[dev] = true;
  return ATTN_OK;
}

bool sizes_ok(int64_t B, int64_t C, int32_t n_q, int32_t n_kv, int32_t d_h, int64_t window,
              int64_t sinks) {
  return B >= 1 && C >= 1 && n_q >= 1 && n_kv >= 1 && n_q % n_kv == 0 && d_h >= 1 && window >= 0 &&
         sinks >= 0 && (window > 0 || sinks == 0);
}
bool supported(int64_t B, int64_t C, int32_t n_q, int32_t n_kv, int32_t d_h) {
  return d_h == kRow4Dim && n_q / n_kv <= kMaxG && C <= (int64_t{1} << 30) &&
         B <= (int64_t{1} << 24) && B * n_kv <= (int64_t{1} << 24) &&
         B * n_kv * (C / kChunk + 2) < (int64_t{1} << 31);
}

// Grid and workspace: two places for each head and each CTA that may stand in it.
struct Shape4 {
  int64_t ctas, ml_at, ends_at, bytes;
};
Shape4 shape4(int64_t B, int64_t C, int32_t n_q, int32_t n_kv, int64_t window, int64_t sinks) {
  auto chunks = [](int64_t n) { return (n + kChunk - 1) / kChunk; };
  int64_t T = chunks(C);
  if (window > 0 && window < C) {
    const int64_t seen = chunks(window) + chunks(sinks < C - window ? sinks : C - window);
    if (seen < T) T = seen;
  }
  const int64_t g = n_q / n_kv, warps = g <= 8 ? kWarpsOf<1> : kWarpsOf<2>;
  const int64_t most = (B * n_kv * T + warps - 1) / warps;
  Shape4 s;
  s.ctas = most < kCtas ? most : kCtas;
  const int64_t rows = 2 * (B * n_kv + s.ctas) * g;
  auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
  s.ml_at = up(rows * kRow4Dim * 4);
  s.ends_at = s.ml_at + up(rows * 8);
  s.bytes = s.ends_at + up(B * n_kv * 8);
  return s;
}

}  // namespace

extern "C" {

int64_t attn_decode4_workspace_bytes(int64_t B, int64_t C, int32_t n_q, int32_t n_kv, int32_t d_h,
                                     int64_t window, int64_t sinks) {
  if (!sizes_ok(B, C, n_q, n_kv, d_h, window, sinks) || !supported(B, C, n_q, n_kv, d_h)) return -1;
  return shape4(B, C, n_q, n_kv, window, sinks).bytes;
}

attn_status_t attn_decode4_fwd(const void* q, const void* k4, const void* v4, const int32_t* lens,
                               void* o, float* lse, void* workspace, int64_t workspace_bytes,
                               int64_t B, int64_t C, int32_t n_q, int32_t n_kv, int32_t d_h,
                               int64_t window, int64_t sinks, float scale, void* stream_ptr) {
  if (!q || !k4 || !v4 || !lens || !o || !lse || !workspace) return ATTN_ERR_INVALID_ARG;
  if (!sizes_ok(B, C, n_q, n_kv, d_h, window, sinks) || !std::isfinite(scale))
    return ATTN_ERR_INVALID_ARG;
  auto misaligned = [](const void* ptr, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0;
  };
  if (misaligned(q, 16) || misaligned(k4, 16) || misaligned(v4, 16) || misaligned(o, 16) ||
      misaligned(lse, 4) || misaligned(lens, 4) || misaligned(workspace, 16))
    return ATTN_ERR_INVALID_ARG;
  if (!supported(B, C, n_q, n_kv, d_h)) return ATTN_ERR_UNSUPPORTED;
  const Shape4 s = shape4(B, C, n_q, n_kv, window, sinks);
  if (workspace_bytes < s.bytes) return ATTN_ERR_INVALID_ARG;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  int* status = nullptr;
  const attn_status_t ds = device_ready(stream, &status);
  if (ds != ATTN_OK) return ds;
  char* ws = static_cast<char*>(workspace);
  Params4 p{};
  p.q = static_cast<const uint16_t*>(q);
  p.k4 = static_cast<const uint8_t*>(k4);
  p.v4 = static_cast<const uint8_t*>(v4);
  p.lens = lens;
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + s.ml_at);
  p.ends = reinterpret_cast<int*>(ws + s.ends_at);
  p.B = static_cast<int>(B);
  p.C = static_cast<int>(C);
  p.n_q = n_q;
  p.n_kv = n_kv;
  p.g = n_q / n_kv;
  p.window = static_cast<int>(window < C ? window : C);
  p.sinks = static_cast<int>(sinks < C ? sinks : C);
  const bool two = p.g > 8;
  p.walkers = static_cast<int>(s.ctas) * (two ? kWarpsOf<2> : kWarpsOf<1>);
  p.c = scale * 1.4426950408889634f;
  p.sixteens = 0x41804180u;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(s.ctas));
  cfg.blockDim = dim3(32 * (two ? kWarpsOf<2> : kWarpsOf<1>));
  cfg.dynamicSmemBytes = two ? kSmemOf<2> : kSmemOf<1>;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = two ? cudaLaunchKernelEx(&cfg, decode4_split_kernel<2>, p)
                      : cudaLaunchKernelEx(&cfg, decode4_split_kernel<1>, p);
  if (e != cudaSuccess) return ATTN_ERR_CUDA;
  // eight warps per row where a head may have more places than a warp reads at once
  const bool many = s.ctas > 16 * B * n_kv;
  cfg.gridDim = dim3(static_cast<unsigned>(many ? B * n_q : (B * n_q + kCombineWarps - 1) / kCombineWarps));
  cfg.blockDim = dim3(32 * kCombineWarps);
  cfg.dynamicSmemBytes = 0;
  uint16_t* o16 = static_cast<uint16_t*>(o);
  e = many ? cudaLaunchKernelEx(&cfg, decode4_combine_kernel<kCombineWarps>, o16, lse, p)
           : cudaLaunchKernelEx(&cfg, decode4_combine_kernel<1>, o16, lse, p);
  if (e != cudaSuccess) return ATTN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // extern "C"
