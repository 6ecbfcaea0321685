// What the decoding kernels over a paged cache share, whatever it is held in:
// items of at most 16 query rows (a sequence's key/value head), their keys shared
// out in 16-key blocks over the warps of a CTA and the CTAs of a cluster or of
// the whole grid, and how the warps' and the CTAs' results meet.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "dependent.cuh"
#include "mma16.cuh"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace rows {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kKeys = kPagedBlock;
constexpr int kMeet = 4;  // rows that meet in shared memory at a time
template <int D>
constexpr int kRowStride = D + 4;  // floats of a row there

// An item is a sequence's key/value head; the warps take the 16-key blocks of
// its kUnit-key cost blocks in turn.
constexpr int kUnit = kWarps * kKeys;
using Cost = PagedCost<kUnit, 1, 1, 128, true>;
using Walk = PagedWalk<Cost>;

__device__ __forceinline__ int warp_blocks(const Walk& w, int warp) {
  const int keys = min(w.u1 * kUnit, w.sq.klen) - w.u0 * kUnit;
  const int nb = (max(keys, 0) + kKeys - 1) / kKeys;
  return nb > warp ? (nb - warp + kWarps - 1) / kWarps : 0;
}
// First key of the warp's block j.
__device__ __forceinline__ int first_key(const Walk& w, int warp, int j) {
  return w.u0 * kUnit + (warp + j * kWarps) * kKeys;
}

// Where the CTA starts.  CLUSTER: an item is shared by the p.cluster CTAs of a
// cluster; otherwise the grid takes equal shares of the whole batch.
template <bool CLUSTER>
__device__ __forceinline__ Walk start_rows(const PagedParams& p) {
  Walk w;
  if constexpr (CLUSTER) {
    const int item = blockIdx.x / p.cluster, rank = blockIdx.x - item * p.cluster;
    w.b = item / p.Hkv;
    w.head = item - w.b * p.Hkv;
    w.sq = paged_seq(p, w.b);
    w.nb = (w.sq.klen + kUnit - 1) / kUnit;
    w.u0 = (int)((long long)rank * w.nb / p.cluster);
    w.u1 = (int)((long long)(rank + 1) * w.nb / p.cluster);
    w.x0 = 0;
    w.take = 1;
    w.left = w.sq.qlen > 0 ? 1 : 0;
    if (threadIdx.x == 0 && rank == 0 && w.head == 0) paged_check(p, w.b);
    __syncthreads();
  } else {
    if (threadIdx.x == 0) paged_clear(p);
    w = paged_start<Cost, kThreads>(p, p.max_q);
  }
  return w;
}

// A warp's blocks in order, over the borders of pieces: it walks ahead of the
// kernel as far as the warp's ring reaches.  Lane i holds the page of the
// piece's block 32 n + i, so that a table read's latency is paid once in 32
// blocks.
struct BlockStream {
  Walk ahead;
  int j, n, pages;
  uint32_t issued;

  __device__ __forceinline__ BlockStream(const PagedParams& p, const Walk& w, int warp, int lane)
      : ahead(w), j(0), n(w.left > 0 ? warp_blocks(w, warp) : 0), pages(-1), issued(0) {
    settle(p, warp, lane);
  }
  // Goes to the next block, or to left <= 0.
  __device__ __forceinline__ void settle(const PagedParams& p, int warp, int lane) {
    while (ahead.left > 0 && j >= n) {
      ahead.advance(p, p.max_q);
      n = warp_blocks(ahead, warp);
      j = 0;
    }
    if (ahead.left > 0 && (j & 31) == 0) {
      const int i = j + lane;
      pages = i < n ? __ldg(p.block_table + (size_t)ahead.b * p.max_pages +
                            (first_key(ahead, warp, i) >> p.page_log2))
                    : -1;
    }
  }
  // Lane 0 copies the next block: copy(page, -1 if it is none of the cache;
  // head; the block's first row in the page).
  template <typename Copy>
  __device__ __forceinline__ void issue(const PagedParams& p, int warp, int lane, Copy copy) {
    if (ahead.left <= 0) return;
    const int page = __shfl_sync(0xffffffffu, pages, j & 31);
    if (lane == 0) {
      const bool ok = page >= 0 && page < p.n_pages;
      if (!ok)
        atomicCAS(p.status, 0u, 1u | (64u << 8) | ((uint32_t)min(ahead.b, 0xFFFF) << 16));
      copy(ok ? page : -1, ahead.head, first_key(ahead, warp, j) & (p.page - 1));
    }
    ++issued;
    ++j;
    settle(p, warp, lane);
  }
};

// Row r of the item in q, o and lse: new token r / G, query head r % G of the group.
__device__ __forceinline__ size_t row_of(const PagedParams& p, const Walk& w, int r) {
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
// which lie in meet and meet_ml [kWarps][kMeet]: the item's rows, the CTA's
// part of a cluster's item (part, part_ml, by row), or a part for the join kernel.
template <int D, bool BF16, bool CLUSTER>
__device__ __forceinline__ void meet_rows(const PagedParams& p, const Walk& w, const float* meet,
                                          const float2* meet_ml, float* part, float2* part_ml,
                                          int pass, int rows) {
  const bool whole = !CLUSTER && w.whole();
  const size_t slot = 2 * (size_t)blockIdx.x + (w.x0 == 0 ? 1 : 0);
  for (int idx = threadIdx.x; idx < kMeet * (D / 4); idx += kThreads) {
    const int mr = idx / (D / 4), c = idx % (D / 4) * 4;
    const int r = pass * kMeet + mr;
    if (r >= rows) break;
    float M = -INFINITY;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) M = fmaxf(M, meet_ml[k * kMeet + mr].x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float lsum = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
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
template <int D, bool BF16>
__device__ __forceinline__ void join_cluster(const PagedParams& p, const Walk& w,
                                             const float* part, const float2* part_ml,
                                             bool given_up) {
  if (w.sq.qlen == 0) return;  // the same in every CTA of the cluster
  cluster_sync();
  const int rows = min(kPagedRows, w.sq.qlen * p.G);
  const int rank = blockIdx.x % p.cluster;
  for (int e = rank * kThreads + threadIdx.x; !given_up && e < rows * (D / 4);
       e += p.cluster * kThreads) {
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
