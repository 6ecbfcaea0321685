// Attention of a few new tokens per sequence (at most 16 query rows per
// key/value head) over a paged key/value cache.
//
// The mathematics is the decoding kernel's (online softmax over 16-key
// blocks on the warp-level product, 16 query rows: the group's query heads x
// the new tokens); what differs is where the keys lie and how the work is
// cut.  A block of 16 keys never crosses a page (pages hold a power of two of
// at least 16 rows), so each TMA box takes one table entry.  A page number
// outside the cache, or a box row past the cache, reads zeros.
//
// Bound by the HBM reads of the cache: each warp streams its own blocks through
// a ring (two CTAs of four warps per SM keep 192 KB in flight), and the stream
// runs on over the borders of items while their results meet in shared memory
// (64 sequences of 2048 to 8192 keys, 4 key/value heads, d = 128, bf16: 118.9 us
// with the ring drained at each border, 106.4 without).  Measured, kernel and
// join: that batch 102 us, 6.1 TB/s (0.90 of the measured copy rate; the CTAs
// end between 77 and 101 us, mean 88), 64 sequences of 8192 keys 167 us, 6.4
// TB/s (0.95), 3 x 4 drafts over up to 65536 keys, d = 64 31 us: 3.5 us to
// the first page number, 0.8 to the first key, 18 of streaming, 2 of meeting
// (16 rows), 4 of join.  Shares cut finer for the scheduler to balance cost
// more at their borders than they gain (two per CTA slot 104.7 us, three 106.5).
#include <cuda_runtime.h>
#include <cstdint>

#include "dependent.cuh"
#include "mma16.cuh"
#include "paged.cuh"
#include "sm103_ptx.cuh"
#include "smem_attr.cuh"

namespace attn {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kKeys = kPagedBlock;
constexpr int kMeet = 4;                // rows that meet in shared memory at a time
constexpr int kBoxBytes = kKeys * 128;  // one 64-column chunk of a block's K or V

template <int D>
struct PagedDecodeLayout {
  static constexpr int kChunks = (D + 63) / 64;
  static constexpr int kSlotBytes = 2 * kChunks * kBoxBytes;  // K chunks, then V chunks
  static constexpr int kSlots = D == 64 ? 6 : 3;              // ring depth of each warp
  static constexpr int kRingBytes = kWarps * kSlots * kSlotBytes;
  // Where the warps' results meet: kMeet rows of O each (padded), m and l.
  static constexpr int kRowStride = D + 4;
  static constexpr int kMeetOff = kRingBytes;
  static constexpr int kMlOff = kMeetOff + kWarps * kMeet * kRowStride * 4;
  static constexpr int kBarOff = kMlOff + kWarps * kMeet * 8;  // one mbarrier per slot
  static constexpr int kFlagOff = kBarOff + kWarps * kSlots * 8;
  static constexpr int kBytes = kFlagOff + 16 + 1024;  // + room to align the base
  static_assert(kRingBytes % 1024 == 0 && kBytes + 256 <= 113 * 1024, "two CTAs per SM");
};

// Byte offset of 16-byte piece `piece` of row `row` in a staged block.
__device__ __forceinline__ uint32_t sw_off(int row, int piece) {
  return (uint32_t)((piece >> 3) * kBoxBytes + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
}

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

// CLUSTER: an item is shared by the p.cluster CTAs of a cluster, which join
// their parts through each other's shared memory; otherwise the grid
// takes equal shares of the whole batch and leaves parts to the join kernel.
template <int D, bool BF16, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, 2)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
  using L = PagedDecodeLayout<D>;
  constexpr int KS = D / 16;      // k-steps of S = Q K^T
  constexpr int NT = kKeys / 8;   // 8-key column tiles of S
  constexpr int DN = D / 8;       // 8-column tiles of O
  constexpr int NS = L::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kFlagOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int s) { return sbase + L::kBarOff + 8u * (uint32_t)(warp * NS + s); };

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kWarps * NS; ++i) mbar_init(sbase + L::kBarOff + 8u * i, 1);
    mbar_fence_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  grid_wait();
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
  Watchdog wd{p.status, abort_flag, p.wait_limit_ns};
  const uint32_t ring = sbase + (uint32_t)(warp * NS * L::kSlotBytes);

  // The warp's stream of blocks runs over the pieces without a break: ahead
  // walks it as far as the ring reaches.  Lane i holds the page of the piece's
  // block 32 n + i, so that a table read's latency is paid once in 32 blocks.
  // issued, it: blocks issued to and taken from the ring.
  Walk ahead = w;
  int aj = 0, an = w.left > 0 ? warp_blocks(w, warp) : 0, pages = -1;
  uint32_t issued = 0, it = 0;
  auto find_next = [&]() {  // settles ahead on its next block, or on left <= 0
    while (ahead.left > 0 && aj >= an) {
      ahead.advance(p, p.max_q);
      an = warp_blocks(ahead, warp);
      aj = 0;
    }
    if (ahead.left > 0 && (aj & 31) == 0) {
      const int j = aj + lane;
      pages = j < an ? __ldg(p.block_table + (size_t)ahead.b * p.max_pages +
                             (first_key(ahead, warp, j) >> p.page_log2))
                     : -1;
    }
  };
  auto issue = [&]() {
    if (ahead.left <= 0) return;
    const int page = __shfl_sync(0xffffffffu, pages, aj & 31);
    if (lane == 0) {
      const int s = (int)(issued % NS);
      const uint32_t dk = ring + (uint32_t)(s * L::kSlotBytes);
      const uint32_t dv = dk + L::kChunks * kBoxBytes;
      const bool ok = page >= 0 && page < p.n_pages;
      if (!ok)
        atomicCAS(p.status, 0u, 1u | (64u << 8) | ((uint32_t)min(ahead.b, 0xFFFF) << 16));
      const int z = ok ? page * p.Hkv + ahead.head : -1;  // -1: the box reads zeros
      const int y = first_key(ahead, warp, aj) & (p.page - 1);
      mbar_arrive_expect_tx(bar(s), L::kSlotBytes);
#pragma unroll
      for (int c = 0; c < L::kChunks; ++c) {
        tma_load_3d(dk + c * kBoxBytes, &tmK, bar(s), c * 64, y, z);
        tma_load_3d(dv + c * kBoxBytes, &tmV, bar(s), c * 64, y, z);
      }
    }
    ++issued;
    ++aj;
    find_next();
  };
  find_next();
  for (int i = 0; i < NS; ++i) issue();

  float* meet = reinterpret_cast<float*>(smem + L::kMeetOff);
  float2* meet_ml = reinterpret_cast<float2*>(smem + L::kMlOff);  // [kWarps][kMeet]
  // The CTA's part of a cluster's item, over the idle ring: O, (m, l) by row.
  float* part = reinterpret_cast<float*>(smem);
  float2* part_ml = reinterpret_cast<float2*>(smem + kPagedRows * D * 4);
  bool given_up = false;

  for (; w.left > 0; w.advance(p, p.max_q)) {
    if (!CLUSTER && w.nothing()) continue;
    const int nbw = warp_blocks(w, warp);
    const PagedSeq sq = w.sq;
    const int rows = min(kPagedRows, sq.qlen * p.G);
    // Row r of the item: new token r / G, query head r % G of the group.
    auto grow = [&](int r) -> size_t {
      const int i = r / p.G, h = r - i * p.G;
      return (size_t)(w.head * p.G + h) * p.total + sq.s0 + i;
    };
    const int r0 = lane >> 2, cq = 2 * (lane & 3);
    const uint16_t* qa_ = static_cast<const uint16_t*>(p.q) + (r0 < rows ? grow(r0) * D : 0);
    const uint16_t* qb_ =
        static_cast<const uint16_t*>(p.q) + (r0 + 8 < rows ? grow(r0 + 8) * D : 0);
    uint32_t qa[KS][4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int c = 16 * ks + cq;
      qa[ks][0] = r0 < rows ? *reinterpret_cast<const uint32_t*>(qa_ + c) : 0u;
      qa[ks][1] = r0 + 8 < rows ? *reinterpret_cast<const uint32_t*>(qb_ + c) : 0u;
      qa[ks][2] = r0 < rows ? *reinterpret_cast<const uint32_t*>(qa_ + c + 8) : 0u;
      qa[ks][3] = r0 + 8 < rows ? *reinterpret_cast<const uint32_t*>(qb_ + c + 8) : 0u;
    }
    // Last key each of the thread's two rows sees (-1: a padding row, or one
    // before the first key).
    auto last_key = [&](int r) {
      if (r >= rows) return -1;
      return min(p.causal ? r / p.G + sq.klen - sq.qlen : sq.klen, sq.klen - 1);
    };
    const int limA = last_key(r0), limB = last_key(r0 + 8);
    const bool hiB = rows > 8;

    float o[DN][4];
#pragma unroll
    for (int dn = 0; dn < DN; ++dn) o[dn][0] = o[dn][1] = o[dn][2] = o[dn][3] = 0.f;
    float mA = -INFINITY, mB = -INFINITY, lA = 0.f, lB = 0.f;
    bool aborted = false;
#pragma unroll 1
    for (int j = 0; j < nbw; ++j) {
      const int s = (int)(it % NS);
      if (!__all_sync(0xffffffffu, mbar_wait(bar(s), (it / NS) & 1, wd, 65))) {
        aborted = true;
        break;
      }
      ++it;
      const uint32_t tk = ring + (uint32_t)(s * L::kSlotBytes);
      const uint32_t tv = tk + L::kChunks * kBoxBytes;
      const int key0 = first_key(w, warp, j);
      if (key0 + kKeys > sq.klen) {
        // Rows past the sequence's last key hold whatever the page held (P is
        // 0 there, but 0 x NaN is not): zero those rows of V.
        const int dead = key0 + kKeys - sq.klen;
        for (int i = lane; i < dead * 8 * L::kChunks; i += 32) {
          const int row = kKeys - 1 - i / (8 * L::kChunks), pc = i % (8 * L::kChunks);
          *reinterpret_cast<uint4*>(smem + (tv - sbase) + sw_off(row, pc)) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();  // before the slot's next copy
        __syncwarp();
      }

      float sc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ks += 2) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t bm[4];
          ldsm_x4(tk + sw_off(8 * nt + (lane & 7), 2 * ks + (lane >> 3)), bm);
          mma16816<BF16>(sc[nt], qa[ks], bm[0], bm[1]);
          mma16816<BF16>(sc[nt], qa[ks + 1], bm[2], bm[3]);
        }
      }

      // Online softmax.  sc[nt][e]: row r0 (e < 2) or r0 + 8, key key0 + 8 nt + cq + e % 2.
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = key0 + 8 * nt + cq + (e & 1);
          const float x = sc[nt][e] * p.scale_log2;
          sc[nt][e] = key <= (e < 2 ? limA : limB) ? x : -INFINITY;
        }
      float bA = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
      bA = fmaxf(bA, __shfl_xor_sync(0xffffffffu, bA, 1));
      bA = fmaxf(bA, __shfl_xor_sync(0xffffffffu, bA, 2));
      const float nA = fmaxf(mA, bA);
      const float alphaA = nA == mA ? 1.f : ex2_approx(mA - nA);
      const float uA = nA == -INFINITY ? 0.f : nA;
      mA = nA;
      float psA = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sc[nt][e] = ex2_approx(sc[nt][e] - uA);
          psA += sc[nt][e];
        }
      lA = lA * alphaA + psA;
      float alphaB = 1.f;
      if (hiB) {
        float bB = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
        bB = fmaxf(bB, __shfl_xor_sync(0xffffffffu, bB, 1));
        bB = fmaxf(bB, __shfl_xor_sync(0xffffffffu, bB, 2));
        const float nB = fmaxf(mB, bB);
        alphaB = nB == mB ? 1.f : ex2_approx(mB - nB);
        const float uB = nB == -INFINITY ? 0.f : nB;
        mB = nB;
        float psB = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 2; e < 4; ++e) {
            sc[nt][e] = ex2_approx(sc[nt][e] - uB);
            psB += sc[nt][e];
          }
        lB = lB * alphaB + psB;
      }
      if (__any_sync(0xffffffffu, alphaA != 1.f || alphaB != 1.f)) {
#pragma unroll
        for (int dn = 0; dn < DN; ++dn) {
          o[dn][0] *= alphaA;
          o[dn][1] *= alphaA;
          o[dn][2] *= alphaB;
          o[dn][3] *= alphaB;
        }
      }

      // O += P V.  P is rounded to the inputs' 16 bits, as in the dense kernels:
      // at most eps / 2 of sum_j P_ij |v_j| (l sums the unrounded values).  For
      // 64 sequences of up to 8192 keys in bf16 the relative error of O is 0.0022,
      // of which the output's own rounding, with P in 32 bits, makes 0.0017; two
      // 16-bit terms for P would double the products.
      uint32_t pa[4];
      pa[0] = pack2<BF16>(sc[0][0], sc[0][1]);
      pa[1] = hiB ? pack2<BF16>(sc[0][2], sc[0][3]) : 0u;
      pa[2] = pack2<BF16>(sc[1][0], sc[1][1]);
      pa[3] = hiB ? pack2<BF16>(sc[1][2], sc[1][3]) : 0u;
      const int vrow = 8 * ((lane >> 3) & 1) + (lane & 7);
#pragma unroll
      for (int dn = 0; dn < DN; dn += 2) {
        uint32_t bm[4];
        ldsm_x4_trans(tv + sw_off(vrow, dn + (lane >> 4)), bm);
        mma16816<BF16>(o[dn], pa, bm[0], bm[1]);
        mma16816<BF16>(o[dn + 1], pa, bm[2], bm[3]);
      }

      // The slot is read: refill it with the next block of the stream.
      __syncwarp();
      if (lane == 0) fence_proxy_async_smem();
      issue();
    }
    // The warps leave together when one has given up; the barrier also frees
    // the meeting place from the piece before.
    given_up = __syncthreads_or(aborted);
    if (given_up) break;

    lA += __shfl_xor_sync(0xffffffffu, lA, 1);
    lA += __shfl_xor_sync(0xffffffffu, lA, 2);
    lB += __shfl_xor_sync(0xffffffffu, lB, 1);
    lB += __shfl_xor_sync(0xffffffffu, lB, 2);

    // The warps' (O, m, l) meet in shared memory, kMeet rows at a time.
    const bool whole = !CLUSTER && w.whole();
    const size_t slot = 2 * (size_t)blockIdx.x + (w.x0 == 0 ? 1 : 0);
    if (!CLUSTER && !whole && threadIdx.x == 0) w.describe(p, 0);
    for (int pass = 0; pass * kMeet < rows; ++pass) {
      if (pass > 0) __syncthreads();
      if ((r0 >> 2) == (pass & 1)) {
        float* ro = meet + (warp * kMeet + (r0 & 3)) * L::kRowStride + cq;
#pragma unroll
        for (int dn = 0; dn < DN; ++dn)
          *reinterpret_cast<float2*>(ro + 8 * dn) =
              pass < 2 ? make_float2(o[dn][0], o[dn][1]) : make_float2(o[dn][2], o[dn][3]);
        if ((lane & 3) == 0)
          meet_ml[warp * kMeet + (r0 & 3)] = pass < 2 ? make_float2(mA, lA) : make_float2(mB, lB);
      }
      __syncthreads();
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
              *reinterpret_cast<const float4*>(meet + (k * kMeet + mr) * L::kRowStride + c);
          acc.x += f * x.x;
          acc.y += f * x.y;
          acc.z += f * x.z;
          acc.w += f * x.w;
        }
        if constexpr (CLUSTER) {
          *reinterpret_cast<float4*>(part + r * D + c) = acc;
          if (c == 0) part_ml[r] = make_float2(M, lsum);
        } else if (whole) {
          const float inv = paged_inverse(lsum);
          const size_t gr = grow(r);
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + gr * D + c) = make_uint2(
              pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
          if (c == 0) p.lse[gr] = paged_lse(M, lsum);
        } else {
          *reinterpret_cast<float4*>(p.part_o + (slot * kPagedRows + r) * D + c) = acc;
          if (c == 0)
            *reinterpret_cast<float2*>(p.part_ml + (slot * kPagedRows + r) * 2) =
                make_float2(M, lsum);
        }
      }
    }
  }
  if constexpr (CLUSTER) {
    if (w.sq.qlen > 0) {  // the same in every CTA of the cluster
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
        const float inv = paged_inverse(lsum);
        const int i = r / p.G, h = r - i * p.G;
        const size_t gr = (size_t)(w.head * p.G + h) * p.total + w.sq.s0 + i;
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + gr * D + c) = make_uint2(
            pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
        if (c == 0) p.lse[gr] = paged_lse(M, lsum);
      }
      cluster_sync();  // the others have read this CTA's part
    }
  }
  // After an abort, copies still on their way must land before the CTA exits.
  Watchdog dw = wd;
  volatile int never = 0;
  dw.abort_flag = &never;
  dw.limit_ns = drain_limit_ns(wd.limit_ns);
  for (; it < issued; ++it) mbar_wait(bar((int)(it % NS)), (it / NS) & 1, dw, 66);
  grid_release();
}

template <int D, bool BF16, bool CLUSTER>
cudaError_t launch_dbc(const PagedLaunch& a) {
  using L = PagedDecodeLayout<D>;
  static DeviceFlags configured;
  auto kern = paged_decode_kernel<D, BF16, CLUSTER>;
  cudaError_t e = ensure_dyn_smem(kern, L::kBytes, configured);
  if (e != cudaSuccess) return e;
  return launch_clusters(kern, CLUSTER ? a.params.cluster : 1, dim3((unsigned)a.grid), kThreads,
                         L::kBytes, a.stream, a.tmK, a.tmV, a.params);
}

template <int D, bool BF16>
cudaError_t launch_db(const PagedLaunch& a) {
  return a.params.cluster > 0 ? launch_dbc<D, BF16, true>(a) : launch_dbc<D, BF16, false>(a);
}

template <int D>
cudaError_t launch_d(const PagedLaunch& a, bool bf16) {
  return bf16 ? launch_db<D, true>(a) : launch_db<D, false>(a);
}

}  // namespace

cudaError_t launch_paged_decode(const PagedLaunch& a, int d, bool bf16) {
  switch (d) {
    case 64: return launch_d<64>(a, bf16);
    case 96: return launch_d<96>(a, bf16);
    default: return launch_d<128>(a, bf16);
  }
}

}  // namespace attn
