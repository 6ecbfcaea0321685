// New tokens packed by cu_seqlens and their places in a paged cache, as the
// kernels that write or read a token's rows share them.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "attn.h"

namespace attn {

constexpr int kBadBatch = 63, kBadPage = 64;  // sites in the status word

// The batch: sequence b owns tokens cu_seqlens[b] .. cu_seqlens[b + 1], the
// last of its kv_lens[b] positions.
struct PackedBatch {
  const int* block_table;  // [n_seq, max_pages]
  const int* cu_seqlens;   // [n_seq + 1]
  const int* kv_lens;      // [n_seq]
  uint32_t* status;
  int n_seq, max_pages, n_pages, page_log2, total;
};

#ifdef __CUDACC__

__device__ __forceinline__ void report_bad(uint32_t* status, int site, int index) {
  atomicCAS(status, 0u, (uint32_t)ATTN_ERR_INVALID_ARG | ((uint32_t)site << 8) |
                            ((uint32_t)min(index, 0xFFFF) << 16));
}

// Records sequence b as invalid if its offsets or its length are out of range.
__device__ __forceinline__ void packed_check(const PackedBatch& p, int64_t b) {
  const int a = __ldg(p.cu_seqlens + b), e = __ldg(p.cu_seqlens + b + 1);
  const int k = __ldg(p.kv_lens + b);
  if ((b == 0 && a != 0) || a < 0 || e < a || e > p.total || k < 0 ||
      k > (p.max_pages << p.page_log2))
    report_bad(p.status, kBadBatch, (int)b);
}

// A token's place: its sequence (n_seq: behind the last), whether it is one of
// it and not padding, its position in the cache, and the page of that (stored:
// a page of the cache).
struct PackedPlace {
  int b;
  bool in_seq, stored;
  int64_t pos;
  int page;
};

// The token's sequence: the last b with cu[b] <= t, n_seq behind the last.  Tokens
// before the first or behind the last are padding.  The offsets need not be valid
// for the search to end in range.
__device__ __forceinline__ int packed_seq(const PackedBatch& p, int t) {
  int lo = 0, hi = p.n_seq;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(p.cu_seqlens + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The token's place in that sequence, b < n_seq.  (A call of its own: the append to
// 16 bits leaves between the two, and took 4 % longer with both in one.)
__device__ __forceinline__ PackedPlace packed_place(const PackedBatch& p, int b, int t) {
  PackedPlace s = {b, false, false, 0, -1};
  const int s0 = __ldg(p.cu_seqlens + s.b), s1 = __ldg(p.cu_seqlens + s.b + 1);
  s.in_seq = t >= s0 && t < s1;
  s.pos = (int64_t)__ldg(p.kv_lens + s.b) - s1 + t;
  const int64_t at = s.pos >> p.page_log2;
  if (s.in_seq && s.pos >= 0 && at < p.max_pages)
    s.page = __ldg(p.block_table + (int64_t)s.b * p.max_pages + at);
  s.stored = s.page >= 0 && s.page < p.n_pages;
  return s;
}

#endif  // __CUDACC__

}  // namespace attn
