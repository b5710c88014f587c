// attn_cache4.cu — rows of K and V into and out of caches held in 4 bits.
//
//   lo = min x,  scale = bf16((max x - lo) / 15),  code = rint((x - lo) / scale)
//
// over each group of 32 channels of a row and head. Inputs are bf16, so lo is
// one of them and exact. Both kernels move bytes (256 of bf16 and 80 of codes per
// row), but packing's arithmetic costs more than they do (18432 positions of 8 heads,
// K and V, 99 MB in and out: 29 us where the copy rate would take 15, 31.6 alone and
// cold, issue slots 71 % full; 32768 of them, 176 MB: 42 for 26.5; unpacking those 29,
// 27.3 alone and cold, 97 % of the copy rate). What keeps it at that: eight lanes take a
// row, half a group each, so that two of them work out a group's scale and not more,
// extremes on packed pairs, quotients by a reciprocal and one correction, two at once,
// rounding and joining of the codes in fp32's and integer multiply-adds.
//
// The code is the nearest integer to the exact quotient, ties to even, and the
// scale the exact quotient rounded to fp32 and then to bf16. While |x| and |lo| are
// 2^-11 scale or more, d = x - lo is a multiple of 2^-19 of the scale's power of two
// and exact, so a quotient that is not half-way is 2^-20 away from it, more than the
// corrected quotient is off (half a unit, 2^-21 below 16), and one that is half-way
// comes out exactly: rounding it is right. (Ties are common: d is often an odd
// multiple of half the scale.) A lane with a smaller value settles its codes by what
// they leave of the dividend.
#include <cuda_runtime.h>

#include <cstdint>

#include "attn_prefill.h"
#include "cache4.cuh"
#include "sm103_ptx.cuh"

namespace gb300_host {
attn_status_t device_status_word(cudaStream_t stream, int** status);
}

namespace {

using namespace gb300;

constexpr int kThreads = 128;                       // (64: 38 us of packing, 256: 32, 512: 36)
constexpr int kLanes = 8;                           // lanes per row, 16 channels each
constexpr int kRowsAtOnce = kThreads / kLanes;
constexpr int kAhead = 2;                           // rows under way per thread
constexpr int kRowsPerBlock = kRowsAtOnce * kAhead;

struct Cache4Params {
  uint16_t* x[2];          // K and V rows, bf16 [B, L, n_kv, 128]
  uint8_t* cache[2];       // their caches [B, n_kv, C, 80]
  const int* at;           // [B] position of the first row; null: 0
  const int* counts;       // [B] rows that a sequence stores; null: L (packing only)
  int L, C, n_kv;
  int blocks;              // blocks per sequence
  uint32_t div_m, div_s;   // r / n_kv = (umulhi(m, r) + r) >> s for r < 2^31
};

// Row number r (of L * n_kv) of sequence b: its place in the cache (-1: outside, or not
// to be stored).
struct Place {
  int64_t cache;
  bool live;               // r < L * n_kv
};
__device__ __forceinline__ Place place(const Cache4Params& p, int b, uint32_t r, int first,
                                       int count) {
  Place w;
  w.live = r < static_cast<uint32_t>(p.L) * static_cast<uint32_t>(p.n_kv);
  const uint32_t i = (__umulhi(p.div_m, r) + r) >> p.div_s;      // r / n_kv
  const uint32_t u = r - i * p.n_kv;
  const int64_t pos = static_cast<int64_t>(first) + i;
  w.cache = w.live && static_cast<int>(i) < count && pos >= 0 && pos < p.C
                ? ((static_cast<int64_t>(b) * p.n_kv + u) * p.C + pos) * kRow4Bytes
                : -1;
  return w;
}

// Two bf16 at once; NaN where one of two is.
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The smaller magnitude (its sign means nothing).
__device__ __forceinline__ uint32_t min_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float low_half(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_half(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// bf16 of the fp32 rounding of (hi - lo) / 15, both finite.
__device__ __forceinline__ uint32_t scale_of(float hi, float lo) {
  const float d = hi - lo;
  float q = d * (1.0f / 15.0f);
  // off by the difference's, the constant's and the product's roundings: less than four
  // units, which only matters next to the middle of two bf16 values, or where the
  // difference overflowed
  const uint32_t low = __float_as_uint(q) & 0xFFFFu;
  if (isinf(d) || (low >= 0x7FFCu && low <= 0x8004u) || (q < 0x1p-120f && d != 0.0f))
    q = static_cast<float>((static_cast<double>(hi) - static_cast<double>(lo)) / 15.0);
  return pack_bf16x2(q, 0.0f) & 0xFFFFu;
}

// The nearest code to (x - lo) / s given one of its two neighbours c and d = x - lo as
// fp32 has it. What c leaves of the dividend, d - s c, is exact (s c has 12 bits);
// where it is half a step, what d's rounding left out decides, then the even code.
__device__ __forceinline__ float settled(float c, float d, float x, float lo, float s) {
  const float h = 0.5f * s, rest = fmaf(-s, c, d);
  const float back = d - x, left = (x - (d - back)) + (-lo - back);
  const float beyond = rest > 0.0f ? left : -left, half_c = 0.5f * c;
  const bool odd = half_c != truncf(half_c);
  const bool move = fabsf(rest) > h || (fabsf(rest) == h && (beyond > 0.0f || (beyond == 0.0f && odd)));
  return move ? c + (rest > 0.0f ? 1.0f : -1.0f) : c;
}

// The code of x where 1 / s or the differences would leave fp32's range: everything
// times a power of two, exact for bf16.
__device__ __noinline__ uint32_t scaled_code(float x, float lo, float s) {
  const float unit = s < 1.0f ? 0x1p64f : 0x1p-8f;
  x *= unit;
  lo *= unit;
  s *= unit;
  const float d = x - lo;
  // (a scale of few bits may be well below a fifteenth of the span: codes stop at 15)
  return static_cast<uint32_t>(fminf(settled(rintf(d * __frcp_rn(s)), d, x, lo, s), 15.0f));
}

// Row r0 + a * kRowsAtOnce of the thread's block, for a = 0 .. kAhead - 1.
struct Rows {
  int b, l;
  int64_t x;               // element offset of row r0
  Place at[kAhead];
  __device__ Rows(const Cache4Params& p, const int* counts) {
    b = static_cast<int>(blockIdx.x) / p.blocks;
    const uint32_t r0 =
        static_cast<uint32_t>(static_cast<int>(blockIdx.x) - b * p.blocks) * kRowsPerBlock +
        threadIdx.x / kLanes;
    l = threadIdx.x % kLanes;
    const int first = p.at ? p.at[b] : 0, count = counts ? counts[b] : p.L;
    x = (static_cast<int64_t>(b) * p.L * p.n_kv + r0) * kRow4Dim;
#pragma unroll
    for (int a = 0; a < kAhead; ++a) at[a] = place(p, b, r0 + a * kRowsAtOnce, first, count);
  }
};

__global__ void __launch_bounds__(kThreads, 9)
pack4_kernel(const Cache4Params p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Rows rows(p, p.counts);
  const uint16_t* __restrict__ x = (blockIdx.y ? p.x[1] : p.x[0]) + rows.x + 16 * rows.l;
  uint8_t* __restrict__ cache = blockIdx.y ? p.cache[1] : p.cache[0];
  const int g = rows.l >> 1, t = 2 * (rows.l & 1);       // group; blocks of eight t and t + 1
  uint32_t u[kAhead][8];
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (rows.at[a].cache >= 0)
        v = *reinterpret_cast<const uint4*>(x + a * kRowsAtOnce * kRow4Dim + 8 * h);
      u[a][4 * h] = v.x;
      u[a][4 * h + 1] = v.y;
      u[a][4 * h + 2] = v.z;
      u[a][4 * h + 3] = v.w;
    }
  }
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    if (!__any_sync(0xffffffffu, rows.at[a].cache >= 0)) continue;
    auto value = [&](int e) { return e & 1 ? high_half(u[a][e >> 1]) : low_half(u[a][e >> 1]); };
    uint32_t lo2 = u[a][0], hi2 = u[a][0], near2 = u[a][0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
      lo2 = min2(lo2, u[a][e]);
      hi2 = max2(hi2, u[a][e]);
      near2 = min_abs2(near2, u[a][e]);
    }
    lo2 = min2(lo2, __shfl_xor_sync(0xffffffffu, lo2, 1));
    hi2 = max2(hi2, __shfl_xor_sync(0xffffffffu, hi2, 1));
    const float lo = fminf(low_half(lo2), high_half(lo2)), hi = fmaxf(low_half(hi2), high_half(hi2));
    // (a NaN is in both packed extremes, perhaps in one half only)
    const bool finite = (lo2 & 0x7F80u) != 0x7F80u && (lo2 & 0x7F800000u) != 0x7F800000u &&
                        (hi2 & 0x7F80u) != 0x7F80u && (hi2 & 0x7F800000u) != 0x7F800000u;
    const uint32_t s16 = finite ? scale_of(hi, lo) : 0x7FC0u;
    const float s = __uint_as_float(s16 << 16);
    uint32_t word[2] = {0u, 0u};
    if (finite && s > 0.0f) {
      float inv;                            // (within a unit; the correction takes care of it)
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
      const float smallest =
          fminf(fminf(fabsf(low_half(near2)), fabsf(high_half(near2))), fabsf(lo));
      if (s < 0x1p-100f || s > 0x1p100f) {
#pragma unroll 1
        for (int e = 0; e < 16; ++e) {
          const uint16_t bits = x[a * kRowsAtOnce * kRow4Dim + e];
          word[e >> 3] |= scaled_code(__uint_as_float(static_cast<uint32_t>(bits) << 16), lo, s)
                          << (4 * (e & 7));
        }
      } else {
        float c[16];                        // 1.5 * 2^23 + code
        // (two at once)
        const uint64_t lo_2 = f32x2_pack(-lo, -lo), inv_2 = f32x2_pack(inv, inv);
        const uint64_t s_2 = f32x2_pack(-s, -s), one_2 = f32x2_pack(12582912.0f, 12582912.0f);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const uint64_t d = fadd2(f32x2_pack(value(e), value(e + 1)), lo_2), q = fmul2(d, inv_2);
          f32x2_unpack(fadd2(ffma2(ffma2(s_2, q, d), inv_2, q), one_2), c[e], c[e + 1]);
        }
        if (smallest < 0x1p-11f * s) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float v = value(e);
            c[e] = settled(c[e] - 12582912.0f, v - lo, v, lo, s) + 12582912.0f;
          }
        }
        // sum 16^e (bits of 1.5 * 2^23 + code), less the constant part
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t sum = __float_as_uint(c[8 * h + 7]);
#pragma unroll
          for (int e = 6; e >= 0; --e) sum = sum * 16u + __float_as_uint(c[8 * h + e]);
          word[h] = sum - 0x4B400000u * 0x11111111u;
        }
      }
    }
    if (rows.at[a].cache < 0) continue;
    uint8_t* row = cache + rows.at[a].cache;
    *reinterpret_cast<uint32_t*>(row + 4 * (4 * t + g)) = word[0];
    *reinterpret_cast<uint32_t*>(row + 4 * (4 * t + 4 + g)) = word[1];
    if (t == 0)
      *reinterpret_cast<uint32_t*>(row + kRow4Codes + 4 * g) =
          s16 | (finite ? __float_as_uint(lo) : 0x7FC00000u);
  }
}

__global__ void __launch_bounds__(kThreads)
unpack4_kernel(const Cache4Params p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Rows rows(p, nullptr);
  // a lane takes block l of eight channels and block l + 8, so that a warp's stores cover
  // whole 128-byte pieces (neighbouring blocks a lane: 37 us where this takes 27.5)
  uint16_t* __restrict__ x = (blockIdx.y ? p.x[1] : p.x[0]) + rows.x + 8 * rows.l;
  const uint8_t* __restrict__ cache = blockIdx.y ? p.cache[1] : p.cache[0];
  const int g = rows.l >> 2, t = rows.l & 3;
  uint32_t word[kAhead][2], pair[kAhead][2];
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    // (positions outside the cache read as zeros)
    word[a][0] = word[a][1] = pair[a][0] = pair[a][1] = 0u;
    if (rows.at[a].cache >= 0) {
      const uint8_t* row = cache + rows.at[a].cache;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        word[a][h] = *reinterpret_cast<const uint32_t*>(row + 4 * (4 * t + g + 2 * h));
        pair[a][h] = *reinterpret_cast<const uint32_t*>(row + kRow4Codes + 4 * (g + 2 * h));
      }
    }
  }
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    if (!rows.at[a].live) continue;
    // two codes at once as bf16 16 + code (bits 3 .. 6 of each half), less 16, then
    // lo + scale * code, one rounding
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t s2 = __byte_perm(pair[a][h], 0, 0x1010), lo2 = __byte_perm(pair[a][h], 0, 0x3232);
      uint32_t f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t at = e == 0 ? word[a][h] << 3 : word[a][h] >> (4 * e - 3);
        asm("{\n\t.reg .b32 c;\n\t"
            "sub.rn.bf16x2 c, %1, %2;\n\t"
            "fma.rn.bf16x2 %0, %3, c, %4;\n\t}"
            : "=r"(f[e])
            : "r"((at & 0x00780078u) | 0x41804180u), "r"(0x41804180u), "r"(s2), "r"(lo2));
      }
      // f[e]: channels e and e + 4
      *reinterpret_cast<uint4*>(x + a * kRowsAtOnce * kRow4Dim + 64 * h) =
          make_uint4(__byte_perm(f[0], f[1], 0x5410), __byte_perm(f[2], f[3], 0x5410),
                     __byte_perm(f[0], f[1], 0x7632), __byte_perm(f[2], f[3], 0x7632));
    }
  }
}

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return x < y + nb && y < x + na;
}

// Both calls' checks and launch.
template <bool kPack>
attn_status_t run_cache4(const void* k, const void* v, const void* k4, const void* v4,
                         const int32_t* at, const int32_t* counts, int64_t B, int64_t L, int64_t C,
                         int32_t n_kv, int32_t d_h, void* stream_ptr) {
  if (!k || !v || !k4 || !v4) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || L < 1 || C < 1 || n_kv < 1) return ATTN_ERR_INVALID_ARG;
  auto misaligned = [](const void* ptr, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0;
  };
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(k4, 16) || misaligned(v4, 16) ||
      misaligned(at, 4) || misaligned(counts, 4))
    return ATTN_ERR_INVALID_ARG;
  if (d_h != kRow4Dim) return ATTN_ERR_UNSUPPORTED;
  constexpr int64_t kMost = int64_t{1} << 30;
  if (B > (1 << 24) || n_kv > (1 << 24) || L > kMost || C > kMost || B * n_kv > (1 << 24) ||
      L * n_kv > (int64_t{1} << 30))
    return ATTN_ERR_UNSUPPORTED;
  const int64_t blocks = (L * n_kv + kRowsPerBlock - 1) / kRowsPerBlock;
  if (B * blocks > INT32_MAX) return ATTN_ERR_UNSUPPORTED;
  const int64_t rows = B * L * n_kv * kRow4Dim * 2, held = B * n_kv * C * kRow4Bytes;
  const void* written[2] = {kPack ? k4 : k, kPack ? v4 : v};
  const void* read[2] = {kPack ? k : k4, kPack ? v : v4};
  const int64_t nw = kPack ? held : rows, nr = kPack ? rows : held;
  if (overlap(written[0], nw, written[1], nw)) return ATTN_ERR_INVALID_ARG;
  for (const void* w : written)
    for (const void* r : read)
      if (overlap(w, nw, r, nr)) return ATTN_ERR_INVALID_ARG;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  int* status = nullptr;
  const attn_status_t ds = gb300_host::device_status_word(stream, &status);
  if (ds != ATTN_OK) return ds;
  Cache4Params p{};
  p.x[0] = static_cast<uint16_t*>(const_cast<void*>(k));
  p.x[1] = static_cast<uint16_t*>(const_cast<void*>(v));
  p.cache[0] = static_cast<uint8_t*>(const_cast<void*>(k4));
  p.cache[1] = static_cast<uint8_t*>(const_cast<void*>(v4));
  p.at = at;
  p.counts = counts;
  p.L = static_cast<int>(L);
  p.C = static_cast<int>(C);
  p.n_kv = n_kv;
  p.blocks = static_cast<int>(blocks);
  while ((1u << p.div_s) < static_cast<uint32_t>(n_kv)) ++p.div_s;
  p.div_m = static_cast<uint32_t>(
      (((uint64_t{1} << p.div_s) - static_cast<uint64_t>(n_kv)) << 32) / n_kv + 1);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(B * blocks), 2);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = kPack ? cudaLaunchKernelEx(&cfg, pack4_kernel, p)
                              : cudaLaunchKernelEx(&cfg, unpack4_kernel, p);
  if (e != cudaSuccess) return ATTN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

extern "C" {

attn_status_t attn_cache_pack4(const void* k, const void* v, void* k4, void* v4,
                               const int32_t* at, const int32_t* counts, int64_t B, int64_t L,
                               int64_t C, int32_t n_kv, int32_t d_h, void* stream) {
  return run_cache4<true>(k, v, k4, v4, at, counts, B, L, C, n_kv, d_h, stream);
}

attn_status_t attn_cache_unpack4(const void* k4, const void* v4, void* k, void* v,
                                 const int32_t* at, int64_t B, int64_t L, int64_t C, int32_t n_kv,
                                 int32_t d_h, void* stream) {
  return run_cache4<false>(k, v, k4, v4, at, nullptr, B, L, C, n_kv, d_h, stream);
}

}  // extern "C"
