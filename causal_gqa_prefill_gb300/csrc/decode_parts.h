// decode_parts.h — what attn_decode.cu offers to other kernels of the library:
// its ragged split kernel as one part of a step whose combine is elsewhere.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "attn_prefill.h"

namespace gb300_host {

// Partial results of the ragged split kernel: for K/V head hd (= b * n_kv + u)
// of a sequence with lens[b] > 0 keys, segments hd + c for the CTAs
// c = ends[2 hd] .. ends[2 hd + 1], each with g rows: the running maximum m
// (log2 units), the sum l of 2^(score - m) and the output [row][128] not yet
// divided by it.
struct RaggedParts {
  const float* o;
  const float2* ml;
  const int* ends;
};

// Set-up of the decode family on the current device, and its status word.
attn_status_t decode_ready(cudaStream_t stream, int** status);

// Workspace bytes of the split kernel alone; -1 where it does not go.
int64_t ragged_split_bytes(int64_t B, int64_t C, int32_t n_q, int32_t n_kv, int32_t d_h);

// Launches the split kernel beside the kernel before it on `stream`: it does
// not wait for that kernel before it starts (which must itself have waited for
// everything earlier before it let dependents launch), only before it ends, so
// a programmatic dependent of this one finds both complete.
attn_status_t ragged_split_beside(const void* q, const void* k, const void* v, const int32_t* lens,
                                  void* workspace, int64_t B, int64_t C, int32_t n_q, int32_t n_kv,
                                  float scale, cudaStream_t stream, int* status,
                                  RaggedParts* parts);

}  // namespace gb300_host
