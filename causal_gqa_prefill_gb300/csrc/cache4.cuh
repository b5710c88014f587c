// cache4.cuh — the rows of a K or V cache held in 4 bits, as attn_cache4.cu
// writes and reads them and attn_decode4.cu attends to them.
//
// A cache is uint8 [B, n_kv, C, 80]: one row of 80 bytes per sequence, K/V head
// and position, so the rows of a head lie side by side and a run of them is one
// contiguous copy. Each of the four groups of 32 channels has a scale and a
// lowest value `lo`, both bf16, and 32 codes of 0 .. 15 that stand for
// lo + scale * code.
//
//   bytes  0 .. 63   16 words of 32 bits: word 4 t + g holds the codes of
//                    channels 32 g + 8 t .. + 7, the first in the lowest bits
//   bytes 64 .. 79   four words: word g holds scale (low half) and lo of group g
//
// The order of the words puts what one lane of a matrix instruction needs of
// every group (its eight channels of each) into one 16-byte load.
#pragma once

#include <cstdint>

namespace gb300 {

constexpr int kRow4Dim = 128;
constexpr int kRow4Groups = 4;
constexpr int kRow4Codes = 64;                // bytes of codes
constexpr int kRow4Bytes = kRow4Codes + 4 * kRow4Groups;

// The two halves of a parameter word as fp32 (a bf16 is an fp32's upper half).
__device__ __forceinline__ float row4_scale(uint32_t word) { return __uint_as_float(word << 16); }
__device__ __forceinline__ float row4_low(uint32_t word) {
  return __uint_as_float(word & 0xFFFF0000u);
}

}  // namespace gb300
