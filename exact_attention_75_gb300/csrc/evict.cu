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
// shared memory, the CTAs add up a part of the counts each and give all of them the
// sums, and the digit in which the n-th lies is kept.  One more pass lists what
// lies above it, and of what equals it as many as are wanted.  Weights of the first
// 8192 positions of a part stay in registers for all passes.  Bound by the chain of
// these steps (two meetings of the cluster a digit), not by what it reads.
//
// Move.  Rows go to places that other rows may still have to be read from; but a
// row only moves forward, so the rows go in order, as many at a time as the
// cluster's registers hold: all of them are read, the cluster meets, all of them
// are written.  No place written is a place still to be read, since that lies
// behind every place written so far.  Bound by HBM with many items, by a round's
// latency (2.3 us) with few.
//
// 16 sequences of up to 8192 positions on 4 heads of 128 in 16 bits, half of them
// kept, cold and for the first time 57 us (alone, the choice 20, the move of 240 MB 42).
// One sequence of 65536 on 8 heads of 64 in 4 bits, a quarter kept, 45 (choice 34, five
// rounds 22).  From L2 and over a cache that was cut before, whose heavy rows lie in
// front, 33 and 35; three such caches in turn 58 and 36, of which the choice has 18 and
// 17.  Measured on the way, in that last form: every CTA reading all the CTAs' counts, 64 and 38; equal digits of a warp counted
// together, 70 and 50; 16 vectors of a row's a thread in place of 8, 45 for the move
// of the second, not 38.
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
static_assert(kBins == 4 * kThreads, "four digits a thread");

// Weights as numbers that order alike: -0 is 0, NaN the heaviest.
__device__ __forceinline__ uint32_t order(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint4 cluster_load(const uint32_t* x, int rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(cluster_addr(smem_u32(x), rank))
               : "memory");
  return v;
}

__device__ __forceinline__ void cluster_store(const uint32_t* x, int rank, uint4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                   cluster_addr(smem_u32(x), rank)),
               "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
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

// A CTA's positions in runs of kHeld x kThreads, kHeld to a thread (kThreads apart,
// so that a run is in order by (j, thread)); the first run's weights stay in
// registers.
constexpr int kHeld = 16;
constexpr int kRun = kHeld * kThreads;

__global__ void __launch_bounds__(kThreads, 2) evict_choose_kernel(const EvictParams p,
                                                                   int cluster) {
  __shared__ __align__(16) uint32_t count[kBins];  // of the CTA's positions, by digit
  __shared__ __align__(16) uint32_t total[kBins];  // of the cluster's
  __shared__ uint32_t scan[kHeld * kThreads / 32];
  __shared__ uint32_t chosen, above, own[2], all;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kThreads / 32;
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
  // The weights of a run that begins at r0, eight on their way together.
  auto read = [&](int r0, uint32_t (&w)[kHeld]) {
#pragma unroll
    for (int j0 = 0; j0 < kHeld; j0 += 8) {
      if (r0 + j0 * kThreads >= m1) break;
      int64_t row[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = r0 + (j0 + j) * kThreads + tid;
        row[j] = at < m1 ? it.row(p, at) : -2;
        if (row[j] == -1) report_bad(p.status, kBadPage, it.b);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j0 + j] = row[j] >= 0 ? order(p.weights[row[j]]) : 0u;
    }
  };
  uint32_t first[kHeld];
  read(m0, first);
  // want: positions still to be chosen among those whose first digits are `prefix`;
  // more: of the CTA's positions those that lie above it.
  uint32_t want = (uint32_t)(p.budget - p.sinks - p.recent), prefix = 0, more = 0, equal = 0;
  for (int digit = 0; digit < 3 && want > 0; ++digit) {
    const int shift = digit == 0 ? 21 : (digit == 1 ? 10 : 0), bits = digit == 2 ? 10 : 11;
    for (int i = tid; i < kBins; i += kThreads) count[i] = 0u;
    __syncthreads();
    auto add = [&](int r0, const uint32_t (&w)[kHeld]) {
#pragma unroll
      for (int j = 0; j < kHeld; ++j) {
        if (r0 + j * kThreads >= m1) break;
        if (r0 + j * kThreads + tid < m1 && (digit == 0 || w[j] >> (shift + bits) == prefix))
          atomicAdd(count + (w[j] >> shift & ((1u << bits) - 1)), 1u);
      }
    };
    add(m0, first);
    for (int r0 = m0 + kRun; r0 < m1; r0 += kRun) {
      uint32_t w[kHeld];
      read(r0, w);
      add(r0, w);
    }
    cluster_sync();
    // Each CTA adds up a part of the digits, one load of four a thread, and gives the
    // sums to all; neighbouring lanes have the same digits of different CTAs.
    {
      const int k = tid & (cluster - 1), at = (it.rank * (kThreads / cluster) + tid / cluster) * 4;
      uint4 x = cluster_load(count + at, k);
      for (int off = 1; off < cluster; off <<= 1) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, off);
        x.y += __shfl_xor_sync(0xffffffffu, x.y, off);
        x.z += __shfl_xor_sync(0xffffffffu, x.z, off);
        x.w += __shfl_xor_sync(0xffffffffu, x.w, off);
      }
      cluster_store(total + at, k, x);
    }
    cluster_sync();
    // A thread has four digits, the largest first, and scans over the cluster's counts.
    const int top = kBins - 1 - 4 * tid;
    const uint4 got = *reinterpret_cast<const uint4*>(total + top - 3);
    const uint32_t c[4] = {got.w, got.z, got.y, got.x};
    const uint32_t sum = c[0] + c[1] + c[2] + c[3];
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
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t mine = count[top - i];
      if (before + c[i] < want) {
        here += mine;
      } else if (before < want) {  // one thread, one digit
        chosen = (uint32_t)(top - i);
        above = before;
        own[1] = mine;
      }
      before += c[i];
    }
    here = __reduce_add_sync(0xffffffffu, here);
    if (lane == 0 && here > 0) atomicAdd(own, here);
    __syncthreads();
    prefix = prefix << bits | chosen;
    want -= above;
    more += own[0];
    equal = own[1];
    // (The others have read this CTA's counts before they gave it their sums.)
  }
  // Of the CTAs before this one: what lies above the limit, what equals it.
  if (tid == 0) {
    count[0] = more;
    count[1] = equal;
  }
  cluster_sync();
  uint32_t gt = 0, eq = 0;
#pragma unroll
  for (int r = 0; r < kEvictCluster; ++r) {
    if (r >= it.rank) break;
    const uint4 x = cluster_load(count, r);
    gt += x.x;
    eq += x.y;
  }
  cluster_sync();  // the others have read
  for (int r0 = m0; r0 < m1 && want > 0; r0 += kRun) {  // (want 0: nothing of the middle stays)
    if (r0 > m0) read(r0, first);
    uint32_t above_in[kHeld], equal_in[kHeld];  // ballots
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      if (r0 + j * kThreads >= m1) break;
      const bool in = r0 + j * kThreads + tid < m1;
      above_in[j] = __ballot_sync(0xffffffffu, in && first[j] > prefix);
      equal_in[j] = __ballot_sync(0xffffffffu, in && first[j] == prefix);
      if (lane == 0)
        scan[j * kWarps + warp] =
            (uint32_t)__popc(above_in[j]) | (uint32_t)__popc(equal_in[j]) << 16;
    }
    __syncthreads();
    if (warp == 0) {  // scans all counts of the run (kHeld x kWarps, in order), eight a lane
      constexpr int kEach = kHeld * kWarps / 32;
      const int n = min(kHeld, (m1 - r0 + kThreads - 1) / kThreads) * kWarps;
      uint32_t part[kEach], sum = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        part[i] = sum;
        sum += lane * kEach + i < n ? scan[lane * kEach + i] : 0u;
      }
      uint32_t incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += up;
      }
#pragma unroll
      for (int i = 0; i < kEach; ++i) scan[lane * kEach + i] = incl - sum + part[i];
      if (lane == 31) all = incl;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      if (r0 + j * kThreads >= m1) break;
      const uint32_t off = scan[j * kWarps + warp], under = (1u << lane) - 1;
      const uint32_t g = gt + (off & 0xFFFFu) + __popc(above_in[j] & under);
      const uint32_t q = eq + (off >> 16) + __popc(equal_in[j] & under);
      const bool is_gt = above_in[j] >> lane & 1, is_eq = equal_in[j] >> lane & 1;
      if (is_gt || (is_eq && q < want))
        kept[p.sinks + g + min(q, want)] = r0 + j * kThreads + tid;
    }
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
// the cluster's threads hold kUnroll vectors of K or V each of.
template <typename Vec, int VPR>
__global__ void __launch_bounds__(kThreads, 2) evict_move_kernel(const EvictParams p, int cluster) {
  constexpr int kUnroll = 8;
  constexpr int kPerCta = kUnroll * kThreads / (2 * VPR);  // rows of a round a CTA has
  constexpr int kVecs = kPerCta * 2 * VPR;
  __shared__ int64_t from[2][kPerCta], to[2][kPerCta];
  const int tid = threadIdx.x;
  grid_wait();
  const Item it(p, cluster);
  if (it.n <= p.budget) {
    grid_release();
    return;
  }
  const int* const kept = p.kept + ((size_t)it.b * p.Hkv + it.head) * p.budget;
  // The rows of the round that begins at r0 (from -1: it stays where it is).
  auto find = [&](int r0, int buf) {
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
      from[buf][i] = f;
      to[buf][i] = t;
    }
  };
  find(p.sinks, 0);
  __syncthreads();
  int buf = 0;
  for (int r0 = p.sinks; r0 < p.budget; r0 += kPerCta * cluster, buf ^= 1) {
    Vec x[kUnroll];
    float w[(kPerCta + kThreads - 1) / kThreads];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = u * kThreads + tid, i = v / (2 * VPR), c = v % (2 * VPR);
      if (v >= kVecs || from[buf][i] < 0) continue;
      const uint8_t* pages = c < VPR ? p.k_pages : p.v_pages;
      x[u] = *(reinterpret_cast<const Vec*>(pages) + from[buf][i] * VPR + c % VPR);
    }
#pragma unroll
    for (int j = 0; j < (kPerCta + kThreads - 1) / kThreads; ++j) {
      const int i = j * kThreads + tid;
      if (i < kPerCta && from[buf][i] >= 0) w[j] = p.weights[from[buf][i]];
    }
    find(r0 + kPerCta * cluster, buf ^ 1);  // the next round's, while the rows are on their way
    cluster_sync();                         // every row of the round has been read
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = u * kThreads + tid, i = v / (2 * VPR), c = v % (2 * VPR);
      if (v >= kVecs || from[buf][i] < 0) continue;
      uint8_t* pages = c < VPR ? p.k_pages : p.v_pages;
      *(reinterpret_cast<Vec*>(pages) + to[buf][i] * VPR + c % VPR) = x[u];
    }
#pragma unroll
    for (int j = 0; j < (kPerCta + kThreads - 1) / kThreads; ++j) {
      const int i = j * kThreads + tid;
      if (i < kPerCta && from[buf][i] >= 0) p.weights[to[buf][i]] = w[j];
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
