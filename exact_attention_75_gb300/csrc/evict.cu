// Eviction from a paged cache: of each sequence longer than `budget` and each of
// its key/value heads the first `sinks` positions stay, the last `recent`, and of
// those between the heaviest by their accumulated weight, equal ones from the
// lowest position up.  What stays moves to the front of the sequence's pages, in
// order.
//
// A cluster of CTAs takes a sequence's head, in two kernels.
//
// Choice.  The n-th largest weight by its bits, most significant digits first
// (11, 11 and 10 bits): each CTA counts its part of the positions by digit in
// shared memory, the cluster adds the counts up, and the digit in which the n-th
// lies is kept.  One more pass lists what lies above it, and of what equals it
// as many as are wanted, a scan at a time.
//
// Move.  Rows go to places that other rows may still have to be read from; but a
// row only moves forward, so the rows go in order, as many at a time as the
// cluster's registers hold: all of them are read, the cluster meets, all of them
// are written.  No place written is a place still to be read, since that lies
// behind every place written so far.
#include <cuda_runtime.h>
#include <cstdint>

#include "dependent.cuh"
#include "packed.cuh"
#include "retain.cuh"
#include "sm103_ptx.cuh"

namespace attn {

namespace {

constexpr int kThreads = 512;
constexpr int kBins = 2048;

// Weights as numbers that order alike: -0 is 0, NaN the heaviest.
__device__ __forceinline__ uint32_t order(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint32_t cluster_load(uint32_t addr, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];"
               : "=r"(v)
               : "r"(cluster_addr(addr, rank))
               : "memory");
  return v;
}

// The cluster's item.
struct Item {
  int b, head, rank, n;  // n: positions, in range
  const int* table;      // of the sequence's pages

  __device__ __forceinline__ Item(const EvictParams& p, int cluster) {
    const int item = blockIdx.x / cluster;
    rank = blockIdx.x - item * cluster;
    b = item / p.Hkv;
    head = item - b * p.Hkv;
    n = min(max(__ldg(p.kv_lens + b), 0), p.max_pages << p.page_log2);
    table = p.block_table + (size_t)b * p.max_pages;
  }
  // Row of position `at` in the pages; -1: its page is none of the cache.
  __device__ __forceinline__ int64_t row(const EvictParams& p, int at) const {
    const int page = __ldg(table + (at >> p.page_log2));
    if (page < 0 || page >= p.n_pages) return -1;
    return (((int64_t)page * p.Hkv + head) << p.page_log2) + (at & ((1 << p.page_log2) - 1));
  }
};

__global__ void __launch_bounds__(kThreads, 2) evict_choose_kernel(const EvictParams p,
                                                                   int cluster) {
  __shared__ uint32_t count[kBins];  // of the CTA's positions, by digit
  __shared__ uint32_t scan[kThreads / 32];
  __shared__ uint32_t chosen, above, own[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_wait();
  const Item it(p, cluster);
  int* const kept = p.kept + ((size_t)it.b * p.Hkv + it.head) * p.budget;
  if (it.rank == 0 && it.head == 0 && tid == 0) {
    const int k = __ldg(p.kv_lens + it.b);
    if (k != it.n) report_bad(p.status, kBadBatch, it.b);
    p.new_lens[it.b] = min(it.n, p.budget);
  }
  if (it.n <= p.budget) {  // the same in the whole cluster
    for (int i = it.rank * kThreads + tid; i < p.budget; i += cluster * kThreads)
      kept[i] = i < it.n ? i : -1;
    grid_release();
    return;
  }
  const int middle = it.n - p.sinks - p.recent;
  const int m0 = p.sinks + (int)((int64_t)middle * it.rank / cluster);
  const int m1 = p.sinks + (int)((int64_t)middle * (it.rank + 1) / cluster);
  auto weight = [&](int at) {
    const int64_t row = it.row(p, at);
    if (row < 0) {
      report_bad(p.status, kBadPage, it.b);
      return 0u;
    }
    return order(p.weights[row]);
  };
  // want: positions still to be chosen among those whose first digits are `prefix`;
  // more: of the CTA's positions those that lie above it.
  uint32_t want = (uint32_t)(p.budget - p.sinks - p.recent), prefix = 0, more = 0, equal = 0;
  for (int digit = 0; digit < 3 && want > 0; ++digit) {
    const int shift = digit == 0 ? 21 : (digit == 1 ? 10 : 0), bits = digit == 2 ? 10 : 11;
    for (int i = tid; i < kBins; i += kThreads) count[i] = 0u;
    __syncthreads();
    for (int at = m0 + tid; at < m1; at += kThreads) {
      const uint32_t w = weight(at);
      if (digit == 0 || w >> (shift + bits) == prefix)
        atomicAdd(count + (w >> shift & ((1u << bits) - 1)), 1u);
    }
    cluster_sync();
    // A thread has four digits, the largest first, and scans over the cluster's counts.
    const int top = kBins - 1 - 4 * tid;
    uint32_t c[4], mine = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = 0u;
      for (int r = 0; r < cluster; ++r) c[i] += cluster_load(smem_u32(count + top - i), r);
      mine += count[top - i];
      sum += c[i];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += up;
    }
    if (lane == 31) scan[warp] = incl;
    if (tid == 0) own[0] = 0u;
    __syncthreads();
    uint32_t before = incl - sum;
    for (int w = 0; w < warp; ++w) before += scan[w];
    uint32_t here = 0;  // the CTA's positions above the chosen digit
    if (before + sum < want) {
      here = mine;
    } else if (before < want) {
      int i = 0;
      for (; before + c[i] < want; ++i) {
        before += c[i];
        here += count[top - i];
      }
      chosen = (uint32_t)(top - i);
      above = before;
      own[1] = count[top - i];
    }
    if (here > 0) atomicAdd(own, here);
    __syncthreads();
    prefix = prefix << bits | chosen;
    want -= above;
    more += own[0];
    equal = own[1];
    cluster_sync();  // the others have read this CTA's counts
  }
  if (want == 0) {  // nothing of the middle stays
    prefix = 0xFFFFFFFFu;
    more = equal = 0u;
  }
  // Of the CTAs before this one: what lies above the limit, what equals it.
  if (tid == 0) {
    count[0] = more;
    count[1] = equal;
  }
  cluster_sync();
  uint32_t gt = 0, eq = 0;
  for (int r = 0; r < it.rank; ++r) {
    gt += cluster_load(smem_u32(count), r);
    eq += cluster_load(smem_u32(count + 1), r);
  }
  cluster_sync();  // the others have read
  const uint32_t limit = prefix;
  const bool none = want == 0;
  for (int t0 = m0; t0 < m1 && !none; t0 += kThreads) {
    const int at = t0 + tid;
    const uint32_t w = at < m1 ? weight(at) : 0u;
    const bool is_gt = at < m1 && w > limit, is_eq = at < m1 && w == limit;
    const uint32_t bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
    if (lane == 0) scan[warp] = (uint32_t)__popc(bg) | (uint32_t)__popc(be) << 16;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) {
      if (k < warp) before += scan[k];
      all += scan[k];
    }
    const uint32_t under = (1u << lane) - 1;
    const uint32_t g = gt + (before & 0xFFFFu) + __popc(bg & under);
    const uint32_t e = eq + (before >> 16) + __popc(be & under);
    if (is_gt || (is_eq && e < want)) kept[p.sinks + g + min(e, want)] = at;
    gt += all & 0xFFFFu;
    eq += all >> 16;
    __syncthreads();
  }
  for (int i = it.rank * kThreads + tid; i < p.sinks + p.recent; i += cluster * kThreads) {
    if (i < p.sinks) kept[i] = i;
    else kept[p.budget - p.recent + i - p.sinks] = it.n - p.recent + i - p.sinks;
  }
  grid_release();
}

// Vec: what a row is moved in, VPR: of them a row has.  A round moves the rows that
// the cluster's threads hold UNROLL vectors of K or V each of.
template <typename Vec, int VPR>
__global__ void __launch_bounds__(kThreads, 2) evict_move_kernel(const EvictParams p, int cluster) {
  constexpr int kUnroll = 8;
  constexpr int kPerCta = kUnroll * kThreads / (2 * VPR);  // rows of a round a CTA has
  constexpr int kVecs = kPerCta * 2 * VPR;
  __shared__ int64_t from[kPerCta], to[kPerCta];
  const int tid = threadIdx.x;
  grid_wait();
  const Item it(p, cluster);
  if (it.n <= p.budget) {
    grid_release();
    return;
  }
  const int* const kept = p.kept + ((size_t)it.b * p.Hkv + it.head) * p.budget;
  for (int r0 = p.sinks; r0 < p.budget; r0 += kPerCta * cluster) {
    // The round's rows of this CTA (from -1: it stays where it is).
    for (int i = tid; i < kPerCta; i += kThreads) {
      const int dst = r0 + it.rank * kPerCta + i;
      int64_t f = -1, t = -1;
      if (dst < p.budget) {
        const int src = kept[dst];
        if (src > dst && src < it.n) {
          f = it.row(p, src);
          t = it.row(p, dst);
          if (f < 0 || t < 0) {
            report_bad(p.status, kBadPage, it.b);
            f = -1;
          }
        }
      }
      from[i] = f;
      to[i] = t;
    }
    __syncthreads();
    Vec x[kUnroll];
    float w[(kPerCta + kThreads - 1) / kThreads];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = u * kThreads + tid, i = v / (2 * VPR), c = v % (2 * VPR);
      if (v >= kVecs || from[i] < 0) continue;
      const uint8_t* pages = c < VPR ? p.k_pages : p.v_pages;
      x[u] = *(reinterpret_cast<const Vec*>(pages) + from[i] * VPR + c % VPR);
    }
#pragma unroll
    for (int j = 0; j < (kPerCta + kThreads - 1) / kThreads; ++j) {
      const int i = j * kThreads + tid;
      if (i < kPerCta && from[i] >= 0) w[j] = p.weights[from[i]];
    }
    cluster_sync();  // every row of the round has been read
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = u * kThreads + tid, i = v / (2 * VPR), c = v % (2 * VPR);
      if (v >= kVecs || from[i] < 0) continue;
      uint8_t* pages = c < VPR ? p.k_pages : p.v_pages;
      *(reinterpret_cast<Vec*>(pages) + to[i] * VPR + c % VPR) = x[u];
    }
#pragma unroll
    for (int j = 0; j < (kPerCta + kThreads - 1) / kThreads; ++j) {
      const int i = j * kThreads + tid;
      if (i < kPerCta && from[i] >= 0) p.weights[to[i]] = w[j];
    }
    __syncthreads();  // from and to are read
  }
  grid_release();
}

template <typename Vec, int VPR>
cudaError_t launch_move(const EvictLaunch& a, dim3 grid) {
  return launch_clusters(evict_move_kernel<Vec, VPR>, a.cluster, grid, kThreads, 0, a.stream,
                         a.params, a.cluster);
}

}  // namespace

cudaError_t launch_evict(const EvictLaunch& a) {
  const dim3 grid((unsigned)(a.params.n_seq * a.params.Hkv * a.cluster));
  cudaError_t e = launch_clusters(evict_choose_kernel, a.cluster, grid, kThreads, 0, a.stream,
                                  a.params, a.cluster);
  if (e != cudaSuccess) return e;
  switch (a.row_bytes) {
    case 40: return launch_move<uint2, 5>(a, grid);
    case 60: return launch_move<uint32_t, 15>(a, grid);
    case 80: return launch_move<uint4, 5>(a, grid);
    case 128: return launch_move<uint4, 8>(a, grid);
    case 192: return launch_move<uint4, 12>(a, grid);
    case 256: return launch_move<uint4, 16>(a, grid);
    case 384: return launch_move<uint4, 24>(a, grid);
    case 512: return launch_move<uint4, 32>(a, grid);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace attn
