// Host <-> device interface of what a paged cache retains: the weights that
// attention gives its positions, and the eviction of the light ones.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "paged.cuh"

namespace attn {

struct WeightsParams {
  PagedParams paged;   // q, k4 (a cache in 4 bits), lse (read), the batch
  const void* k_pages; // [n_pages, Hkv, page, D] of a cache in 16 bits
  float* weights;      // [n_pages, Hkv, page]
};

struct WeightsLaunch {
  WeightsParams params;
  int grid;
  cudaStream_t stream;
};

// d in {64, 96, 128}.
cudaError_t launch_kv_weights(const WeightsLaunch& a, int d, bool bf16, bool kv4);

struct EvictParams {
  uint8_t* k_pages;        // [n_pages, Hkv, page, row_bytes]
  uint8_t* v_pages;
  float* weights;          // [n_pages, Hkv, page]
  const int* block_table;  // [n_seq, max_pages]
  const int* kv_lens;      // [n_seq]
  int* kept;               // [n_seq, Hkv, budget]
  int* new_lens;           // [n_seq]
  uint32_t* status;
  int n_seq, n_pages, page_log2, max_pages, Hkv;
  int budget, sinks, recent;
};

struct EvictLaunch {
  EvictParams params;
  int row_bytes;  // 2 d or 5 d / 8
  int cluster;    // CTAs that share a sequence's key/value head
  cudaStream_t stream;
};

constexpr int kEvictCluster = 8;  // at most

cudaError_t launch_evict(const EvictLaunch& a);

}  // namespace attn
