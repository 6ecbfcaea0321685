// Attention over a paged key/value cache: the host <-> device interface and
// what its kernels share (the batch description, the partition of the work
// over a persistent grid, and the partial results).
//
// Work.  A sequence with new tokens gives each of its key/value heads a run
// of items; an item is a tile of query rows, and costs its key blocks plus
// one (its prologue and epilogue).  All items of the batch laid end to end
// (sequence, key/value head, tile) form one line of cost units, and CTA c of
// the grid takes units [c w, (c + 1) w): equal shares whatever the lengths
// are, so one long sequence spreads over every SM and a ragged batch
// balances itself.  The lengths live on the device (a captured graph replays
// with new ones), so each CTA finds its own start by a prefix sum over the
// sequences.
//
// An item that lies in one CTA's share is finished there.  One that crosses
// shares leaves a partial result per share: an unnormalised O and the (m, l)
// of each row, in slot 0 of the CTA that continues it and slot 1 of the CTA
// that begins it.  The beginning CTA describes the item in desc[cta], and
// the join kernel combines its parts in key order, so equal calls give equal
// bits.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace attn {

constexpr int kPagedMaxSms = 160;  // bound of the grids (two CTAs per SM at most)
// Query rows (query heads of a group x new tokens) of an item on the
// warp-level kernel: the M = 16 of its product.
constexpr int kPagedRows = 16;
// Rows of an item of the tile kernel (two query tiles).
constexpr int kPagedTileRows = 256;
// Keys of a block there (rows of the tensor-map box).
constexpr int kPagedBlock = 16;
// Query heads per key/value head at most.
constexpr int kPagedMaxGroup = 128;
// Keys of one cost unit there (16 for each of the four warps).
constexpr int kPagedUnitKeys = 64;

struct PagedParams {
  const void* q;            // [Hkv * G, total, D]
  void* o;                  // [Hkv * G, total, D]
  float* lse;               // [Hkv * G, total]
  uint32_t* status;         // device status word
  const int* block_table;   // [n_seq, max_pages]
  const int* cu_seqlens;    // [n_seq + 1]
  const int* kv_lens;       // [n_seq], new tokens included
  int4* desc;               // [grid][2] of the item the CTA began and others continue: parts
                            // (0: none), key/value head, first token; s0, qlen of its sequence
  float* part_ml;           // [grid][2][rows][2]
  float* part_o;            // [grid][2][rows][D], of the tile kernel [grid][2][D / 4][rows][4]
  int n_seq, total, max_q, n_pages, page, page_log2, max_pages, Hkv, G;
  int causal;               // query i of n sees keys j <= i + kv_len - n
  int min_share;            // least cost units per CTA
  float scale_log2;         // scale * log2(e)
  unsigned long long wait_limit_ns;
};

struct PagedLaunch {
  CUtensorMap tmQ;          // [Hkv * G, total, D] (tile kernel)
  CUtensorMap tmK, tmV;     // [n_pages * Hkv, page, D]
  PagedParams params;
  int grid;                 // CTAs of the main kernel
  int rows;                 // rows of an item at most
  cudaStream_t stream;
};

// d in {64, 96, 128}.  The decoding kernel takes at most kPagedRows query
// rows per sequence and key/value head, the tile kernel any number; the join
// follows either with the same grid.
cudaError_t launch_paged_decode(const PagedLaunch& a, int d, bool bf16);
cudaError_t launch_paged_tile(const PagedLaunch& a, int d, bool bf16);
cudaError_t launch_paged_join(const PagedLaunch& a, int d, bool bf16, bool decode);

#ifdef __CUDACC__

// One sequence of the batch, clamped so that no access leaves the tensors.
struct PagedSeq {
  int s0, qlen, klen;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int b) {
  PagedSeq s;
  const int a = __ldg(p.cu_seqlens + b), e = __ldg(p.cu_seqlens + b + 1);
  s.s0 = min(max(a, 0), p.total);
  s.qlen = min(min(max(e, s.s0), p.total) - s.s0, p.max_q);
  s.klen = min(max(__ldg(p.kv_lens + b), 0), p.max_pages << p.page_log2);
  return s;
}

// Records sequence b as invalid in the status word if what paged_seq clamps
// was out of range.
__device__ __forceinline__ void paged_check(const PagedParams& p, int b) {
  const int a = __ldg(p.cu_seqlens + b), e = __ldg(p.cu_seqlens + b + 1);
  const int k = __ldg(p.kv_lens + b);
  if ((b == 0 && a != 0) || a < 0 || e < a || e > p.total || e - a > p.max_q || k < 0 ||
      k > (p.max_pages << p.page_log2))
    atomicCAS(p.status, 0u, 1u | (63u << 8) | ((uint32_t)min(b, 0xFFFF) << 16));
}

// Where a CTA's share begins (sequence b, its item counted over the key/value
// heads, the unit in the item), its units (left 0: none), and the units of a
// full share.
struct PagedStart {
  int b;
  int item, items_per_head, unit;
  long long left;
  long long share;
};

// Every thread of the CTA calls this.  head_cost(seq) gives the cost units of
// one key/value head of a sequence (a long long); place(seq, off, start) turns
// an offset into a sequence's line into item, items_per_head and unit.  The
// threads take runs of sequences, a scan over the threads' sums places the
// share, and the thread whose run holds its start walks there.
template <int THREADS, typename HeadCost, typename Place>
__device__ __forceinline__ PagedStart paged_partition(const PagedParams& p, HeadCost head_cost,
                                                      Place place) {
  __shared__ long long warp_sum[THREADS / 32];
  __shared__ PagedStart start;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (p.n_seq + THREADS - 1) / THREADS;
  const int b0 = min(tid * run, p.n_seq), b1 = min(b0 + run, p.n_seq);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    sum += head_cost(paged_seq(p, b)) * p.Hkv;
    if (blockIdx.x == 0) paged_check(p, b);
  }
  long long incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += up;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    all += warp_sum[w];
  }
  long long share = (all + gridDim.x - 1) / gridDim.x;
  if (share < p.min_share) share = p.min_share;
  const long long s = share * blockIdx.x;
  if (tid == 0 && s >= all) start = PagedStart{0, 0, 1, 0, 0, share};
  long long at = before + incl - sum;
  if (s >= at && s < at + sum) {
    for (int b = b0; b < b1; ++b) {
      const long long c = head_cost(paged_seq(p, b)) * p.Hkv;
      if (s < at + c) {
        start = PagedStart{b, 0, 1, 0, min(share, all - s), share};
        place(paged_seq(p, b), s - at, start);
        break;
      }
      at += c;
    }
  }
  __syncthreads();
  return start;
}

#endif  // __CUDACC__

}  // namespace attn
