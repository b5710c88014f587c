// attn_cache4.cu — rows of K and V into and out of caches held in 4 bits.
//
//   lo = min x,  scale = bf16((max x - lo) / 15),  code = rint((x - lo) / scale)
//
// over each group of 32 channels of a row and head. Inputs are bf16, so lo is
// one of them and exact. Both kernels move bytes and little else (256 of bf16 and
// 80 of codes per row): half a warp takes a row, 16 bytes of channels or one word
// of codes a lane, so a warp's loads and stores cover whole rows, and each thread
// has kAhead rows under way.
//
// The code is the nearest integer to the exact quotient, ties to even, and the
// scale the exact quotient rounded to fp32 and then to bf16: where fp32 cannot
// tell (a quotient next to a border), what it left out decides.
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

constexpr int kThreads = 256;
constexpr int kRowsAtOnce = kThreads / 16;          // half a warp per row
constexpr int kAhead = 4;
constexpr int kRowsPerBlock = kRowsAtOnce * kAhead;

struct Cache4Params {
  uint16_t* x[2];          // K and V rows, bf16 [B, L, n_kv, 128]
  uint8_t* cache[2];       // their caches [B, n_kv, C, 80]
  const int* at;           // [B] position of the first row; null: 0
  const int* counts;       // [B] rows that a sequence stores; null: L (packing only)
  int L, C, n_kv;
  int blocks;              // blocks per sequence
};

// Row number r (of L * n_kv) of sequence b: its bf16 row, and its place in the cache
// (-1: outside, or not to be stored).
struct Place {
  int64_t x;
  int64_t cache;
  bool live;               // r < L * n_kv
};
template <bool kPack>
__device__ __forceinline__ Place place(const Cache4Params& p, int b, int64_t r, int first,
                                       int count) {
  Place w;
  w.live = r < static_cast<int64_t>(p.L) * p.n_kv;
  const int i = static_cast<int>(r / p.n_kv), u = static_cast<int>(r - static_cast<int64_t>(i) * p.n_kv);
  const int64_t pos = static_cast<int64_t>(first) + i;
  w.x = (static_cast<int64_t>(b) * p.L * p.n_kv + r) * kRow4Dim;
  w.cache = w.live && i < count && pos >= 0 && pos < p.C
                ? ((static_cast<int64_t>(b) * p.n_kv + u) * p.C + pos) * kRow4Bytes
                : -1;
  return w;
}

// bf16 of the fp32 rounding of (hi - lo) / 15, both finite.
__device__ __forceinline__ uint16_t scale_of(float hi, float lo) {
  const float d = hi - lo;
  float q = __fdiv_rn(d, 15.0f);
  // what the difference's own rounding left out (0 where it is exact) can only matter
  // next to the middle of two bf16 values, or where the difference overflowed
  const float back = d - hi, left = (hi - (d - back)) + (-lo - back);
  const uint32_t low = __float_as_uint(q) & 0xFFFFu;
  if (left != 0.0f && (isinf(d) || (low >= 0x7FFEu && low <= 0x8002u)))
    q = static_cast<float>((static_cast<double>(hi) - static_cast<double>(lo)) / 15.0);
  return static_cast<uint16_t>(pack_bf16x2(q, 0.0f) & 0xFFFFu);
}

// rint((x - lo) / s) for s > 0, inv = 1 / s.
__device__ __forceinline__ uint32_t code_of(float x, float lo, float s, float inv) {
  const float d = x - lo, t = d * inv;
  float c = rintf(t);
  // t is off by 15 * 3 * 2^-24 at most; nearer to a border the sign of what is left of
  // the dividend decides: d - s (k + 1/2) is exact (s (k + 1/2) has 13 bits and is
  // about d), and where it is zero, what d's rounding left out
  if (fabsf(t - c) > 0.4999f) {
    const float k = floorf(t);
    const float rest = fmaf(-s, k + 0.5f, d);
    const float back = d - x, left = (x - (d - back)) + (-lo - back);
    const float sign = rest != 0.0f ? rest : left;
    c = sign > 0.0f ? k + 1.0f : sign < 0.0f ? k : 2.0f * rintf(0.5f * (k + 0.5f));
  }
  return static_cast<uint32_t>(fminf(c, 15.0f));
}

__global__ void __launch_bounds__(kThreads)
pack4_kernel(const Cache4Params p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = static_cast<int>(blockIdx.x) / p.blocks;
  const int64_t r0 =
      static_cast<int64_t>(static_cast<int>(blockIdx.x) - b * p.blocks) * kRowsPerBlock +
      (threadIdx.x >> 4);
  const int l = threadIdx.x & 15, g = l >> 2, t = l & 3;
  const uint16_t* __restrict__ x = blockIdx.y ? p.x[1] : p.x[0];
  uint8_t* __restrict__ cache = blockIdx.y ? p.cache[1] : p.cache[0];
  const int first = p.at ? p.at[b] : 0, count = p.counts ? p.counts[b] : p.L;
  Place w[kAhead];
  uint4 v[kAhead];
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    w[a] = place<true>(p, b, r0 + a * kRowsAtOnce, first, count);
    v[a] = make_uint4(0u, 0u, 0u, 0u);
    if (w[a].cache >= 0) v[a] = *reinterpret_cast<const uint4*>(x + w[a].x + 8 * l);
  }
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    const uint32_t u[4] = {v[a].x, v[a].y, v[a].z, v[a].w};
    float f[8];
    uint32_t odd = 0;                       // 1: something is not finite
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(u[e] << 16);
      f[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
      odd |= (u[e] & 0x7F80u) == 0x7F80u || (u[e] & 0x7F800000u) == 0x7F800000u;
    }
    float lo = f[0], hi = f[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) {
      lo = fminf(lo, f[e]);
      hi = fmaxf(hi, f[e]);
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
      odd |= __shfl_xor_sync(0xffffffffu, odd, off);
    }
    const uint32_t s16 = odd ? 0x7FC0u : scale_of(hi, lo);
    float s = __uint_as_float(s16 << 16);
    // (powers of two, exact for bf16: 1 / s and the differences stay in fp32's range)
    const float unit = s < 0x1p-100f ? 0x1p64f : s > 0x1p100f ? 0x1p-8f : 1.0f;
    s *= unit;
    const float inv = __frcp_rn(s), base = lo * unit;
    uint32_t word = 0;
    if (!odd && s > 0.0f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) word |= code_of(f[e] * unit, base, s, inv) << (4 * e);
    }
    if (w[a].cache < 0) continue;
    uint8_t* row = cache + w[a].cache;
    *reinterpret_cast<uint32_t*>(row + 4 * (4 * t + g)) = word;
    if (t == 0)
      *reinterpret_cast<uint32_t*>(row + kRow4Codes + 4 * g) =
          s16 | (odd ? 0x7FC00000u : __float_as_uint(lo));
  }
}

__global__ void __launch_bounds__(kThreads)
unpack4_kernel(const Cache4Params p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = static_cast<int>(blockIdx.x) / p.blocks;
  const int64_t r0 =
      static_cast<int64_t>(static_cast<int>(blockIdx.x) - b * p.blocks) * kRowsPerBlock +
      (threadIdx.x >> 4);
  const int l = threadIdx.x & 15, g = l >> 2, t = l & 3;
  uint16_t* __restrict__ x = blockIdx.y ? p.x[1] : p.x[0];
  const uint8_t* __restrict__ cache = blockIdx.y ? p.cache[1] : p.cache[0];
  const int first = p.at ? p.at[b] : 0;
  Place w[kAhead];
  uint32_t word[kAhead], pair[kAhead];
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    w[a] = place<false>(p, b, r0 + a * kRowsAtOnce, first, p.L);
    word[a] = pair[a] = 0u;                 // (positions outside the cache read as zeros)
    if (w[a].cache >= 0) {
      const uint8_t* row = cache + w[a].cache;
      word[a] = *reinterpret_cast<const uint32_t*>(row + 4 * (4 * t + g));
      pair[a] = *reinterpret_cast<const uint32_t*>(row + kRow4Codes + 4 * g);
    }
  }
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    if (!w[a].live) continue;
    const float s = row4_scale(pair[a]), lo = row4_low(pair[a]);
    uint32_t out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      out[e] = pack_bf16x2(fmaf(s, static_cast<float>((word[a] >> (8 * e)) & 15u), lo),
                           fmaf(s, static_cast<float>((word[a] >> (8 * e + 4)) & 15u), lo));
    *reinterpret_cast<uint4*>(x + w[a].x + 8 * l) = make_uint4(out[0], out[1], out[2], out[3]);
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
  if (B > (1 << 24) || n_kv > (1 << 24) || L > kMost || C > kMost || B * n_kv > (1 << 24))
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
