// Host <-> device interface of the rotary position kernels: the rotation of
// whole tensors (forward and backward) and the append to a paged key/value
// cache with the rotation on the way.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "packed.cuh"

namespace attn {

constexpr int kMaxAxes = 8;  // position axes

// A [B, heads, N, D] tensor with the last dimension contiguous; strides in
// elements, multiples of 8.
struct RopeTensor {
  void* p;
  int64_t sb, sh, sn;
};

struct RopeParams {
  RopeTensor x[2], y[2];   // q and k: inputs and outputs (x[1].p null: q alone)
  const int* positions;    // [n_axes, pos_batches, N]
  const int64_t* table;    // [2, rot / 2]: angle per position (2^-64 turns), axis
  int n_axes, pos_batches; // pos_batches 1: one set of positions for every batch
  int heads[2], N, d, rot;
  int group_heads, head_groups;  // heads one block turns, blocks per run of tokens
  bool inverse;
};

struct RopeLaunch {
  RopeParams params;
  int B;
  bool bf16, interleaved;
  cudaStream_t stream;
};

cudaError_t launch_rope(const RopeLaunch& a, int num_sms);

struct AppendParams {
  // packed new tokens [heads, total, D], strides in elements: 0 k, 1 v, 2 q
  const void* src[3];
  int64_t sh[3], sn[3];
  void* q_out;             // [heads, total, D] contiguous (null: no q)
  void* k_pages;           // [n_pages, Hkv, page, D]
  void* v_pages;
  PackedBatch batch;
  const int* positions;    // [n_axes, total]; null: the position in the cache on every axis
  const int64_t* table;    // null: no rotation
  int n_axes, Hq, Hkv, d, rot;
  int group_heads, head_groups;
  unsigned token_blocks;   // the blocks behind them check the batch
};

struct AppendLaunch {
  AppendParams params;
  bool bf16, interleaved;
  cudaStream_t stream;
};

cudaError_t launch_append(const AppendLaunch& a, int num_sms);

// The same into a 4-bit cache (kv4.cuh): k_pages, v_pages [n_pages, Hkv, page, 5 D / 8]
// bytes.  d in {64, 96, 128}.
cudaError_t launch_append4(const AppendLaunch& a, int num_sms);

}  // namespace attn
