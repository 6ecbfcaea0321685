// What the decoding kernels over a paged cache share, whatever it is held in:
// items of at most 16 query rows (a sequence's key/value head), their keys shared
// out in blocks over the warps of a CTA and the CTAs of a cluster or of the whole
// grid, and how the warps' and the CTAs' results meet.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "dependent.cuh"
#include "mma16.cuh"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace rows {

constexpr int kUnit = kPagedBlock;  // keys that never lie in two pages
constexpr int kMeet = 4;            // rows that meet in shared memory at a time
template <int D>
constexpr int kRowStride = D + 4;  // floats of a row there

// An item is a sequence's key/value head; the W warps of a CTA take the blocks (K
// keys each) of its cost blocks (one block for each warp) in turn.  An item's borders cost
// as much as 128 keys in 16 bits, as 512 in 4 (whose keys take less; 64 single tokens with 16
// rows over up to 8192 keys 66.5 us, with 128 70.4, with 1024 69.4; 3 sequences of 16 rows
// over up to 65536 24.8, 27.2 and 24.7).
template <int W, int K>
using Cost = PagedCost<W * K, 1, 1, K == 32 ? 512 : 128, true>;
template <int W, int K>
struct Walk : PagedWalk<Cost<W, K>> {};

template <int W, int K>
__device__ __forceinline__ int warp_blocks(const Walk<W, K>& w, int warp) {
  const int keys = min(w.u1 * W * K, w.sq.klen) - w.u0 * W * K;
  const int nb = (max(keys, 0) + K - 1) / K;
  return nb > warp ? (nb - warp + W - 1) / W : 0;
}
// First key of the warp's block j.
template <int W, int K>
__device__ __forceinline__ int first_key(const Walk<W, K>& w, int warp, int j) {
  return (w.u0 * W + warp + j * W) * K;
}

// Where the CTA starts.  CLUSTER: an item is shared by the p.cluster CTAs of a
// cluster; otherwise the grid takes equal shares of the whole batch.
template <int W, int K, bool CLUSTER>
__device__ __forceinline__ Walk<W, K> start_rows(const PagedParams& p) {
  Walk<W, K> w;
  if constexpr (CLUSTER) {
    const int item = blockIdx.x / p.cluster, rank = blockIdx.x - item * p.cluster;
    w.b = item / p.Hkv;
    w.head = item - w.b * p.Hkv;
    w.sq = paged_seq(p, w.b);
    w.nb = (w.sq.klen + W * K - 1) / (W * K);
    w.u0 = (int)((long long)rank * w.nb / p.cluster);
    w.u1 = (int)((long long)(rank + 1) * w.nb / p.cluster);
    w.x0 = 0;
    w.take = 1;
    w.left = w.sq.qlen > 0 ? 1 : 0;
    if (threadIdx.x == 0 && rank == 0 && w.head == 0) paged_check(p, w.b);
    __syncthreads();
  } else {
    if (threadIdx.x == 0) paged_clear(p);
    static_cast<PagedWalk<Cost<W, K>>&>(w) = paged_start<Cost<W, K>, W * 32>(p, p.max_q);
  }
  return w;
}

// A warp's blocks in order, over the borders of pieces: it walks ahead of the
// kernel as far as the warp's ring reaches.  The lanes hold the pages of the next
// 32 units (a block has K / kUnit), so that a table read's latency is paid once for
// them.  SINGLE: the CTA has one piece.
template <int W, int K, bool SINGLE>
struct BlockStream {
  static constexpr int kUnits = K / kUnit;
  Walk<W, K> ahead;
  int key, left;  // the block's first key; blocks of the piece, this one included
  int pages, at;  // at: the lane that holds the page of the block's first unit
  uint32_t issued;

  __device__ __forceinline__ BlockStream(const PagedParams& p, const Walk<W, K>& w, int warp,
                                         int lane)
      : ahead(w), key(0), left(0), pages(-2), at(0), issued(0) {
    if (w.left > 0) begin(p, warp, lane);
  }
  // Whether there is a block to issue.
  __device__ __forceinline__ bool more() const { return left > 0; }
  // The page of unit u of the block: -1 if it is none of the cache (lane 0 reports
  // it), -2 if the unit lies past the sequence.
  __device__ __forceinline__ int page(const PagedParams& p, int u, int lane) const {
    const int page = __shfl_sync(0xffffffffu, pages, at + u);
    if (page >= p.n_pages || page == -1) {
      if (lane == 0)
        atomicCAS(p.status, 0u, 1u | (64u << 8) | ((uint32_t)min(ahead.b, 0xFFFF) << 16));
      return -1;
    }
    return page;
  }
  // The unit's first row in its page.
  __device__ __forceinline__ int row(const PagedParams& p, int u) const {
    return (key + u * kUnit) & (p.page - 1);
  }
  __device__ __forceinline__ void next(const PagedParams& p, int warp, int lane) {
    ++issued;
    key += W * K;
    at += kUnits;
    if (--left == 0) {
      if constexpr (!SINGLE) {
        ahead.advance(p, p.max_q);
        if (ahead.left > 0) begin(p, warp, lane);
      }
    } else if (at == 32) {
      read(p, lane);
    }
  }

 private:
  // Goes to the first block of the warp from the current piece on, if there is one.
  __device__ __forceinline__ void begin(const PagedParams& p, int warp, int lane) {
    while ((left = warp_blocks(ahead, warp)) == 0) {
      if constexpr (SINGLE) return;
      ahead.advance(p, p.max_q);
      if (ahead.left <= 0) return;
    }
    key = first_key(ahead, warp, 0);
    read(p, lane);
  }
  // The pages of the next 32 units, as many as the piece has blocks for.
  __device__ __forceinline__ void read(const PagedParams& p, int lane) {
    const int n = lane / kUnits, k = key + n * W * K + lane % kUnits * kUnit;
    at = 0;
    pages = n < left && k < ahead.sq.klen
                ? max(__ldg(p.block_table + (size_t)ahead.b * p.max_pages + (k >> p.page_log2)),
                      -1)
                : -2;
  }
};

// Row r of the item in q, o and lse: new token r / G, query head r % G of the group.
template <int W, int K>
__device__ __forceinline__ size_t row_of(const PagedParams& p, const Walk<W, K>& w, int r) {
  const int i = r / p.G, h = r - i * p.G;
  return (size_t)(w.head * p.G + h) * p.total + w.sq.s0 + i;
}

// Last key that row r of the item sees (-1: it comes before the first key).
__device__ __forceinline__ int last_key_of(const PagedParams& p, const PagedSeq& sq, int r) {
  return min(p.causal ? r / p.G + sq.klen - sq.qlen : sq.klen, sq.klen - 1);
}

template <int D, bool BF16>
__device__ __forceinline__ void store_row(const PagedParams& p, size_t row, int c, float4 acc,
                                          float M, float l) {
  const float inv = paged_inverse(l);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * D + c) = make_uint2(
      pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
  if (c == 0) p.lse[row] = paged_lse(M, l);
}

// Combines the warps' results (O, m, l) of rows pass * kMeet .. of the piece,
// which lie in meet and meet_ml [W][kMeet]: the item's rows, the CTA's
// part of a cluster's item (part, part_ml, by row), or a part for the join kernel.
template <int D, bool BF16, bool CLUSTER, int W, int K>
__device__ __forceinline__ void meet_rows(const PagedParams& p, const Walk<W, K>& w,
                                          const float* meet, const float2* meet_ml, float* part,
                                          float2* part_ml, int pass, int rows) {
  const bool whole = !CLUSTER && w.whole();
  const size_t slot = 2 * (size_t)blockIdx.x + (w.x0 == 0 ? 1 : 0);
  for (int idx = threadIdx.x; idx < kMeet * (D / 4); idx += W * 32) {
    const int mr = idx / (D / 4), c = idx % (D / 4) * 4;
    const int r = pass * kMeet + mr;
    if (r >= rows) break;
    float M = -INFINITY;
#pragma unroll
    for (int k = 0; k < W; ++k) M = fmaxf(M, meet_ml[k * kMeet + mr].x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float lsum = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const float2 ml = meet_ml[k * kMeet + mr];
      const float f = paged_weight(ml.x, ml.y, M);
      lsum += f * ml.y;
      const float4 x =
          *reinterpret_cast<const float4*>(meet + (k * kMeet + mr) * kRowStride<D> + c);
      acc.x += f * x.x;
      acc.y += f * x.y;
      acc.z += f * x.z;
      acc.w += f * x.w;
    }
    if constexpr (CLUSTER) {
      *reinterpret_cast<float4*>(part + r * D + c) = acc;
      if (c == 0) part_ml[r] = make_float2(M, lsum);
    } else if (whole) {
      store_row<D, BF16>(p, row_of(p, w, r), c, acc, M, lsum);
    } else {
      *reinterpret_cast<float4*>(p.part_o + (slot * kPagedRows + r) * D + c) = acc;
      if (c == 0)
        *reinterpret_cast<float2*>(p.part_ml + (slot * kPagedRows + r) * 2) =
            make_float2(M, lsum);
    }
  }
}

// Joins the parts of a cluster's item through its CTAs' shared memory.
template <int D, bool BF16, int W, int K>
__device__ __forceinline__ void join_cluster(const PagedParams& p, const Walk<W, K>& w,
                                             const float* part, const float2* part_ml,
                                             bool given_up) {
  if (w.sq.qlen == 0) return;  // the same in every CTA of the cluster
  cluster_sync();
  const int rows = min(kPagedRows, w.sq.qlen * p.G);
  const int rank = blockIdx.x % p.cluster;
  for (int e = rank * W * 32 + threadIdx.x; !given_up && e < rows * (D / 4);
       e += p.cluster * W * 32) {
    const int r = e / (D / 4), c = e % (D / 4) * 4;
    float2 ml[kPagedCluster];
    float4 x[kPagedCluster];
#pragma unroll
    for (int k = 0; k < kPagedCluster; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
      if (k >= p.cluster) continue;
      ml[k] = cluster_load2(smem_u32(part_ml + r), k);
      x[k] = cluster_load4(smem_u32(part + r * D + c), k);
    }
    float M = ml[0].x;
#pragma unroll
    for (int k = 1; k < kPagedCluster; ++k) M = fmaxf(M, ml[k].x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float lsum = 0.f;
#pragma unroll
    for (int k = 0; k < kPagedCluster; ++k) {
      if (k >= p.cluster) continue;
      const float f = paged_weight(ml[k].x, ml[k].y, M);
      lsum += f * ml[k].y;
      acc.x += f * x[k].x;
      acc.y += f * x[k].y;
      acc.z += f * x[k].z;
      acc.w += f * x[k].w;
    }
    store_row<D, BF16>(p, row_of(p, w, r), c, acc, M, lsum);
  }
  cluster_sync();  // the others have read this CTA's part
}

}  // namespace rows
}  // namespace attn
