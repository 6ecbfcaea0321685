// Host <-> device interface of reading rows of a 4-bit cache back in 16 bits.
// The append to one takes the 16-bit append's (rotary.cuh).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "packed.cuh"

namespace attn {

struct Read4Params {
  PackedBatch batch;
  const uint8_t* k_pages;  // [n_pages, Hkv, page, 5 D / 8]
  const uint8_t* v_pages;
  void* k;                 // [Hkv, total, D], written
  void* v;
  int Hkv, d;
  int group_heads, head_groups;  // heads (of K and V together) a thread walks, groups of them
  unsigned token_blocks;         // the blocks behind them check the batch
};

struct Read4Launch {
  Read4Params params;
  bool bf16;
  cudaStream_t stream;
};

cudaError_t launch_read4(const Read4Launch& a, int num_sms);

}  // namespace attn
