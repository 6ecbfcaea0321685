// Attention of chunks of new tokens over a paged key/value cache on the
// tensor cores: the forward kernel's pipeline (TMA-fed tcgen05 products, S and
// O in tensor memory, online softmax in base 2, two query tiles that
// ping-pong; fwd.cu) over work cut into equal shares (paged.cuh).
//
// An item is a pair of adjacent query tiles of one sequence and key/value
// head.  A tile's 128 rows are TT = 128 / G tokens x the G query heads of the
// group (row = head * TT + token: one TMA box of [G heads][TT tokens]), so a
// key block is read and multiplied once for the whole group.  A key block of
// 128 positions is 128 / page boxes of the cache (one when a page holds it),
// one lane of the producer warp per box, each with its own table entry.
//
// CTA organisation (one per SM, persistent): warps 0-3 / 4-7 softmax of query
// tile 0 / 1, warp 8 TMA producer, warp 9 tcgen05 issuer, warp 10 relay of
// the TMA completions (and of the zeroing behind a sequence's last key).
//
// Bound, like the dense forward, by the softmax and products of 128-row tiles:
// a key block of two tiles takes 1.55 to 1.75 us (d = 128; d = 96 1.65), of one
// 1.06.  Measured, kernel and join, bf16: 4096 new tokens over 16384 keys, 16
// query heads on 8, d = 128 367 us, 1.31 PFLOP/s, 0.68 of the library product
// (the dense non-causal forward 1.39); 2 x 256 tokens over up to 16384 keys, 16
// heads, d = 96 53.6 us; 4 chunks of up to 509 tokens with 12 single tokens over
// up to 4096 keys 56 us.  In those two a CTA has some 22 key blocks; 2 us go to
// finding its share, 3.5 to the first block, 3 to 4 to each border of an item.
// On the warp-level product the three took 3050, 267 and 256 us.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "dependent.cuh"
#include "mma16.cuh"
#include "paged.cuh"
#include "sm103_ptx.cuh"
#include "smem_attr.cuh"
#include "tiles.cuh"

namespace attn {

namespace {

constexpr int kThreads = 352;
constexpr int kWarpProducer = 8;
constexpr int kWarpMma = 9;
constexpr int kWarpRelay = 10;
constexpr uint32_t kBarKv = 1, kBarP = 2;  // issuer <-> relay, issuer <-> softmax t
constexpr float kRescaleThreshold = 8.0f;  // log2 units: P stays <= 2^8
constexpr int kRows = kPagedTileRows;
constexpr int kStageBytes = 32 * 128;      // a softmax warp's rows on their way out

template <int D>
struct PagedTileLayout {
  static constexpr int kTileBytes = 128 * kPaddedD<D> * 2;
  static constexpr int kSlots = D == 64 ? 8 : 4;  // K/V ring
  static constexpr int kQOff = 0;
  static constexpr int kKvOff = 2 * kTileBytes;
  static constexpr int kStageOff = kKvOff + kSlots * kTileBytes;
  static constexpr int kBarOff = kStageOff + 8 * kStageBytes;
  static constexpr int kQFull = 0, kQEmpty = 2, kSFull = 4, kOFull = 6, kDrain = 8;
  static constexpr int kKvFull = 9, kKvEmpty = 9 + kSlots;
  static constexpr int kNumBars = 9 + 2 * kSlots;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kBytes = kMiscOff + 16;
  static constexpr int kDynSmem = kBytes + 1024;  // + alignment slack
  static_assert(kDynSmem + 256 <= 232448, "shared memory budget (227 KB) exceeded");
};

// A walk along the CTA's share; an item is a pair of tiles of TT tokens each.
// Weights: a key block of one tile was measured at 1.06 us, of a pair at 1.55,
// an item's borders at 3 to 4 us; 3 : 4 and two blocks an item balance best (a
// mixed batch 58.5 us, with 2 : 3 59.8, with equal weights 60.4).
using Cost = PagedCost<128, 3, 4, 1024, false>;
struct Walk : PagedWalk<Cost> {
  int n[2];  // key blocks of the piece that tile 0 / 1 sees (two: tile 1 has rows)

  __device__ __forceinline__ void tiles(const PagedParams& p, int TT) {
    int k0 = nb;  // key blocks of tile 0: fewer than tile 1's under causal masking
    if (two && p.causal)
      k0 = (max((2 * item + 1) * TT + sq.klen - sq.qlen, 0) + 127) >> 7;
    n[0] = max(min(u1, k0) - u0, 0);
    n[1] = two ? u1 - u0 : 0;
  }
  __device__ __forceinline__ void next(const PagedParams& p, int TT) {
    advance(p, 2 * TT);
    if (left > 0) tiles(p, TT);
  }
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tile_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
  using L = PagedTileLayout<D>;
  constexpr int kChunks = kPaddedD<D> / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + L::kBarOff;
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  Watchdog wd{p.status, abort_flag, p.wait_limit_ns};
  const int TT = 128 / p.G;  // tokens of a query tile

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(L::kQFull + t), 1);
      mbar_init(bar(L::kQEmpty + t), 1);
      mbar_init(bar(L::kSFull + t), 1);
      mbar_init(bar(L::kOFull + t), 1);
    }
    mbar_init(bar(L::kDrain), 1);
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(bar(L::kKvFull + s), 1);
      mbar_init(bar(L::kKvEmpty + s), 1);
    }
    mbar_fence_init();
  }
  grid_wait();
  // Tensor memory only now: held earlier, it could be what a block of the
  // previous kernel still waits for.
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  if (threadIdx.x == 0) paged_clear(p);
  Walk w;
  static_cast<PagedWalk<Cost>&>(w) = paged_start<Cost, kThreads>(p, 2 * TT);  // a CTA barrier
  if (w.left > 0) w.tiles(p, TT);
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;

  if (warp == kWarpProducer) {
    // ------------------------------------------------------ TMA producer ---
    const int box_rows = min(p.page, 128);
    const int boxes = 128 / box_rows;
    uint32_t kv_it = 0, q_it[2] = {0, 0};
    bool ok = true;
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    for (; w.left > 0 && ok; w.next(p, TT)) {
      const int nbmax = max(w.n[0], w.n[1]);
      if (nbmax == 0) continue;
      // The page of the lane's box of key block kb, read ahead of its use: -2
      // past the sequence.
      auto box_page = [&](int kb) {
        const int key0 = kb * 128 + lane * box_rows;
        return lane < boxes && key0 < w.sq.klen
                   ? __ldg(p.block_table + (size_t)w.b * p.max_pages + (key0 >> p.page_log2))
                   : -2;
      };
      int page = box_page(w.u0);
      for (int t = 0; t < 2 && ok; ++t) {
        if (w.n[t] == 0) continue;
        ok = __all_sync(0xffffffffu,
                        mbar_wait(bar(L::kQEmpty + t), (q_it[t] & 1) ^ 1, wd, 67));
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(L::kQFull + t), (uint32_t)(kChunks * TT * p.G * 128));
          const uint32_t dst = sbase + L::kQOff + t * L::kTileBytes;
#pragma unroll
          for (int h = 0; h < kChunks; ++h)
            tma_load_3d(dst + h * 16384, &tmQ, bar(L::kQFull + t), h * 64,
                        w.sq.s0 + (2 * w.item + t) * TT, w.head * p.G);
        }
        ++q_it[t];
      }
      for (int j = 0; j < nbmax && ok; ++j) {
        const int y = (w.u0 + j) * 128 & (p.page - 1);  // 0 unless a page holds two blocks
        const int next = j + 1 < nbmax ? box_page(w.u0 + j + 1) : -2;
        // tensor-map page index; -1 (zeros) past the sequence or for a page
        // outside the cache
        const bool in_cache = page >= 0 && page < p.n_pages;
        if (!in_cache && page != -2)
          atomicCAS(p.status, 0u, 1u | (64u << 8) | ((uint32_t)min(w.b, 0xFFFF) << 16));
        const int z = in_cache ? page * p.Hkv + w.head : -1;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          const uint32_t slot = kv_it % L::kSlots;
          ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kKvEmpty + slot),
                                                 ((kv_it / L::kSlots) & 1) ^ 1, wd, 68));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(L::kKvFull + slot), L::kTileBytes);
          __syncwarp();
          if (lane < boxes) {
            const uint32_t dst = sbase + L::kKvOff + slot * L::kTileBytes + lane * box_rows * 128;
#pragma unroll
            for (int h = 0; h < kChunks; ++h)
              tma_load_3d(dst + h * 16384, which ? &tmV : &tmK, bar(L::kKvFull + slot), h * 64,
                          y, z);
          }
          ++kv_it;
        }
        page = next;
      }
    }
    // Drain: every copy this warp issued must have landed before the CTA may
    // exit (only matters after an abort; otherwise all were consumed).
    Watchdog dw = wd;
    volatile int never = 0;
    dw.abort_flag = &never;
    dw.limit_ns = drain_limit_ns(wd.limit_ns);
    const uint32_t first = kv_it > (uint32_t)L::kSlots ? kv_it - L::kSlots : 0u;
    for (uint32_t it = first; it < kv_it; ++it)
      mbar_wait(bar(L::kKvFull + it % L::kSlots), (it / L::kSlots) & 1, dw, 69);
    for (int t = 0; t < 2; ++t)
      if (q_it[t] > 0) mbar_wait(bar(L::kQFull + t), (q_it[t] - 1) & 1, dw, 70);
    __syncwarp();
  } else if (warp == kWarpRelay) {
    // ---------------------------------------------------------- TMA relay ---
    // Waits for the TMA completions the issuer needs and meets it at named
    // barrier kBarKv: per piece [Q tiles + K_0], then per block [V_j + K_{j+1}].
    // After an abort the schedule is still walked to the end (waits skipped),
    // so that every rendezvous pairs up.
    const int box_rows = min(p.page, 128);
    uint32_t kv_it = 0, q_it[2] = {0, 0};
    bool aborted = false;
    auto kv_ready = [&]() {
      const uint32_t slot = kv_it % L::kSlots;
      const uint32_t par = (kv_it / L::kSlots) & 1;
      ++kv_it;
      if (!aborted)
        aborted = !__all_sync(0xffffffffu, mbar_wait(bar(L::kKvFull + slot), par, wd, 71));
      return slot;
    };
    for (; w.left > 0; w.next(p, TT)) {
      const int nbmax = max(w.n[0], w.n[1]);
      if (!w.nothing() && !w.whole() && lane == 0) w.describe(p, 2 * w.item * TT);
      if (nbmax == 0) continue;  // the same skip in every role
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (w.n[t] == 0) continue;
        const uint32_t par = q_it[t] & 1;
        ++q_it[t];
        if (aborted) continue;
        aborted = !__all_sync(0xffffffffu, mbar_wait(bar(L::kQFull + t), par, wd, 72));
      }
      kv_ready();
      aborted = named_bar_or(kBarKv, 64, aborted);
      for (int j = 0; j < nbmax; ++j) {
        const uint32_t vslot = kv_ready();
        const int valid = w.sq.klen - (w.u0 + j) * 128;  // rows of V that are keys
        if (valid < 128 && !aborted) {
          // Rows past the sequence's last key hold whatever their page held
          // (P is 0 there, but 0 x NaN is not): zero them, up to the end of
          // the last key's box (later boxes read zeros).
          const int end = (valid + box_rows - 1) / box_rows * box_rows;
          uint8_t* tile = smem + L::kKvOff + vslot * L::kTileBytes;
          for (int i = lane; i < (end - valid) * 8 * kChunks; i += 32) {
            const int row = valid + i / (8 * kChunks), pc = i % (8 * kChunks);
            *reinterpret_cast<uint4*>(tile + (pc >> 3) * 16384 + row * 128 + (pc & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        if (j + 1 < nbmax) kv_ready();
        aborted = named_bar_or(kBarKv, 64, aborted);
      }
    }
  } else if (warp == kWarpMma) {
    // ---------------------------------------------------- tcgen05 issuer ---
    constexpr uint32_t kIdS = idesc_f16(128, 128, BF16, false, false);
    constexpr uint32_t kIdO = idesc_f16(128, D, BF16, false, true);
    uint32_t kv_it = 0;
    bool aborted = false;
    bool issued = false;
    const uint64_t qdesc0 = kmajor_base(sbase + L::kQOff);
    const uint64_t qdesc1 = kmajor_base(sbase + L::kQOff + L::kTileBytes);
    auto issue_s = [&](int t, uint32_t kaddr) {
      const uint64_t kd = kmajor_base(kaddr);
      const uint64_t qd = t ? qdesc1 : qdesc0;
      const uint32_t dcol = tbase + 128 * t;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_f16_ss(dcol, desc_plus(qd, kmajor16_off(kk)), desc_plus(kd, kmajor16_off(kk)), kIdS,
                   kk > 0);
    };
    auto issue_pv = [&](int t, uint32_t vaddr, uint32_t acc0) {
      const uint32_t ocol = tbase + 256 + kPaddedD<D> * t;
      const uint32_t pcol = tbase + 128 * t;
      const uint64_t vd = mnmajor_base(vaddr);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)  // 16 keys per MMA
        mma_f16_ts(ocol, pcol + kk * 8, desc_plus(vd, mnmajor16_off(kk)), kIdO,
                   kk > 0 ? 1u : acc0);
    };
    for (; w.left > 0; w.next(p, TT)) {
      const int nb0 = w.n[0], nb1 = w.n[1];
      const int nbmax = max(nb0, nb1);
      if (nbmax == 0) continue;  // the same skip in every role
      aborted = named_bar_or(kBarKv, 64, aborted);
      uint32_t kslot = kv_it % L::kSlots;
      ++kv_it;
      if (!aborted) {
        tc_fence_after();
        if (lane == 0) {
          const uint32_t kaddr = sbase + L::kKvOff + kslot * L::kTileBytes;
          if (nb0 > 0) {
            issue_s(0, kaddr);
            mma_commit(bar(L::kSFull + 0));
            if (nb0 == 1) mma_commit(bar(L::kQEmpty + 0));
          }
          if (nb1 > 0) {
            issue_s(1, kaddr);
            mma_commit(bar(L::kSFull + 1));
            if (nb1 == 1) mma_commit(bar(L::kQEmpty + 1));
          }
          mma_commit(bar(L::kKvEmpty + kslot));
        }
        issued = true;
        __syncwarp();
      }
      for (int j = 0; j < nbmax; ++j) {
        // V_j and (if any) K_{j+1} are in shared memory.
        aborted = named_bar_or(kBarKv, 64, aborted);
        const uint32_t vslot = kv_it % L::kSlots;
        ++kv_it;
        const bool have_next = j + 1 < nbmax;
        if (have_next) {
          kslot = kv_it % L::kSlots;
          ++kv_it;
        }
        const uint32_t vaddr = sbase + L::kKvOff + vslot * L::kTileBytes;
        const uint32_t kaddr = sbase + L::kKvOff + kslot * L::kTileBytes;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int nbt = t ? nb1 : nb0;
          if (j >= nbt) continue;
          // P_t(j) is in tensor memory.
          aborted = named_bar_or(kBarP + t, 160, aborted);
          if (aborted) continue;
          tc_fence_after();
          if (lane == 0) {
            issue_pv(t, vaddr, j > 0 ? 1u : 0u);
            if (j == nbt - 1) mma_commit(bar(L::kOFull + t));
            if (j + 1 < nbt) {
              issue_s(t, kaddr);
              mma_commit(bar(L::kSFull + t));
              if (j + 1 == nbt - 1) mma_commit(bar(L::kQEmpty + t));
            }
          }
          __syncwarp();
        }
        if (!aborted) {
          if (lane == 0) {
            mma_commit(bar(L::kKvEmpty + vslot));
            if (have_next) mma_commit(bar(L::kKvEmpty + kslot));
          }
          __syncwarp();
        }
      }
    }
    // Drain: wait until every MMA issued above has completed.
    if (lane == 0 && issued) {
      mma_commit(bar(L::kDrain));
      Watchdog dw = wd;
      volatile int never = 0;
      dw.abort_flag = &never;
      dw.limit_ns = drain_limit_ns(wd.limit_ns);
      mbar_wait(bar(L::kDrain), 0, dw, 73);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------- softmax warpgroups ---
    const int t = warp >> 2;          // query tile of the pair
    const int r = threadIdx.x & 127;  // row within the tile = TMEM lane
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_addr = tbase + lane_base + 128u * t;
    const uint32_t o_addr = tbase + lane_base + 256u + kPaddedD<D> * t;
    const float sl2 = p.scale_log2;
    const int gi = r / TT, ti = r - gi * TT;  // query head of the group, token of the tile
    uint32_t s_it = 0, o_it = 0;
    bool aborted = false;
    for (; w.left > 0; w.next(p, TT)) {
      if (w.nothing()) continue;
      const int nb = w.n[t];
      const int token = (2 * w.item + t) * TT + ti;
      const bool live = gi < p.G && token < w.sq.qlen;
      const size_t grow = (size_t)(w.head * p.G + gi) * p.total + w.sq.s0 + token;
      const bool whole = w.whole();
      const size_t slot = 2 * (size_t)blockIdx.x + (w.x0 == 0 ? 1 : 0);
      float2* const ml =
          reinterpret_cast<float2*>(p.part_ml) + slot * kRows + t * 128 + r;
      if (nb == 0) {
        // A tile without rows, or whose rows see no key of this share.
        if (live) {
          if (!whole) {
            *ml = make_float2(-INFINITY, 0.f);
          } else {
            uint4* orow = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + grow * D);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) orow[c] = make_uint4(0u, 0u, 0u, 0u);
            p.lse[grow] = -INFINITY;
          }
        }
        continue;
      }
      const int koff = p.causal ? w.sq.klen - w.sq.qlen : w.sq.klen;
      const int lim = min(token + koff, w.sq.klen - 1);  // last key the row sees
      const int lim0 = min(token - ti + koff, w.sq.klen - 1);  // of the tile's first token
      float m = -INFINITY;  // running max of the log2-scaled scores (reference value)
      float l = 0.f;        // running sum of exp2(x - m)
      for (int j = 0; j < nb; ++j) {
        const uint32_t spar = s_it & 1;
        ++s_it;
        if (!aborted)
          aborted = !__all_sync(0xffffffffu, mbar_wait(bar(L::kSFull + t), spar, wd, 74));
        if (!aborted) {
          tc_fence_after();
          uint32_t sr[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + c * 32, sr[c]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 4; ++c) reg_fence32(sr[c]);
          float s[128];
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) s[c * 32 + i] = __uint_as_float(sr[c][i]);
          const int kbase = (w.u0 + j) * 128;
          if (kbase + 127 > lim0) {
#pragma unroll
            for (int c = 0; c < 128; ++c) s[c] = (kbase + c > lim) ? -INFINITY : s[c];
          }
          const float m_blk = row_max128(s) * sl2;
          // Raise the reference max where the block's exceeds it by more than
          // the threshold; O and l of those rows are rescaled by alpha.
          bool rescale = false;
          float alpha = 1.f;
          if (j == 0) {
            m = m_blk;
          } else {
            const bool need = m_blk > m + kRescaleThreshold;
            rescale = __any_sync(0xffffffffu, need);
            if (need) {
              alpha = ex2_approx(m - m_blk);
              m = m_blk;
            }
          }
          const float mref = (m == -INFINITY) ? 0.f : m;
          const float2 nm2 = make_float2(-mref, -mref);
          float2 rs2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                           make_float2(0.f, 0.f)};
          const float2 sc2 = make_float2(sl2, sl2);
          // P goes to tensor memory in the inputs' 16 bits, what the product with
          // V takes (at most eps / 2 of sum_j P_ij |v_j|; l sums the unrounded
          // values); two 16-bit terms for P would double that product.
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 x =
                  __ffma2_rn(make_float2(s[c * 32 + 2 * i], s[c * 32 + 2 * i + 1]), sc2, nm2);
              const float p0 = ex2_approx(x.x);
              const float p1 = ex2_approx(x.y);
              rs2[i & 3] = __fadd2_rn(rs2[i & 3], make_float2(p0, p1));
              pk[i] = pack2<BF16>(p0, p1);
            }
            tmem_st16(s_addr + c * 16, pk);
          }
          const float2 rsum =
              __fadd2_rn(__fadd2_rn(rs2[0], rs2[1]), __fadd2_rn(rs2[2], rs2[3]));
          l = l * alpha + (rsum.x + rsum.y);
          if (rescale) {
            // O_row *= alpha; the previous P V into O has completed (its MMA
            // was issued before the S this block waited for).
#pragma unroll 1
            for (int c = 0; c < kChunks; ++c) {
              uint32_t ra[32], rb[32];
              tmem_ld32(o_addr + c * 64, ra);
              tmem_ld32(o_addr + c * 64 + 32, rb);
              tmem_wait_ld();
              reg_fence32(ra);
              reg_fence32(rb);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                ra[i] = __float_as_uint(__uint_as_float(ra[i]) * alpha);
                rb[i] = __float_as_uint(__uint_as_float(rb[i]) * alpha);
              }
              tmem_st32(o_addr + c * 64, ra);
              tmem_st32(o_addr + c * 64 + 32, rb);
            }
          }
          tmem_wait_st();
          tc_fence_before();
        }
        // Hand P_t(j) to the issuer (and learn whether anyone has aborted).
        aborted = named_bar_or(kBarP + t, 160, aborted);
      }
      // ------------------------------------------------------- epilogue ---
      const uint32_t opar = o_it & 1;
      ++o_it;
      if (!aborted)
        aborted = !__all_sync(0xffffffffu, mbar_wait(bar(L::kOFull + t), opar, wd, 75));
      if (aborted) continue;
      tc_fence_after();
      if (whole) {
        const float inv_l = paged_inverse(l);
        // Rows go out through the warp's stage, 64 columns at a time (swizzled
        // 16-byte pieces), so that a store covers whole 128-byte row pieces:
        // a lane per row would write 16 bytes of 32 lines.
        uint8_t* const stage = smem + L::kStageOff + warp * kStageBytes;
#pragma unroll
        for (int c0 = 0; c0 < D / 32; c0 += 2) {
          constexpr int kPieces = 8;
          const int pieces = D / 32 - c0 >= 2 ? kPieces : kPieces / 2;  // of a row
#pragma unroll
          for (int c = c0; c < c0 + pieces / 4; ++c) {
            uint32_t raw[32];
            tmem_ld32_sync(o_addr + c * 32, raw);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              uint32_t pk[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                pk[i] = pack2<BF16>(__uint_as_float(raw[8 * v + 2 * i]) * inv_l,
                                    __uint_as_float(raw[8 * v + 2 * i + 1]) * inv_l);
              const int pc = (c - c0) * 4 + v;
              *reinterpret_cast<uint4*>(stage + lane * 128 + ((pc ^ (lane & 7)) << 4)) =
                  make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < pieces; ++i) {
            const int row = i * (32 / pieces) + lane / pieces, pc = lane % pieces;
            const uint4 x =
                *reinterpret_cast<const uint4*>(stage + row * 128 + ((pc ^ (row & 7)) << 4));
            const int at = __shfl_sync(0xffffffffu, live ? (int)grow : -1, row);
            if (at >= 0)
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + (size_t)at * D + c0 * 32 +
                                        pc * 8) = x;
          }
          __syncwarp();
        }
        if (live) p.lse[grow] = paged_lse(m, l);
      } else {
        uint4* part = reinterpret_cast<uint4*>(p.part_o + slot * kRows * D);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t raw[32];
          tmem_ld32_sync(o_addr + c * 32, raw);
          if (live) {  // the join reads no other rows
#pragma unroll
            for (int v = 0; v < 8; ++v)
              part[(size_t)(c * 8 + v) * kRows + t * 128 + r] =
                  make_uint4(raw[4 * v], raw[4 * v + 1], raw[4 * v + 2], raw[4 * v + 3]);
          }
        }
        if (live) *ml = make_float2(m, l);
      }
      tc_fence_before();
    }
  }

  grid_release();
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D, bool BF16>
cudaError_t launch_db(const PagedLaunch& a) {
  using L = PagedTileLayout<D>;
  auto kern = paged_tile_kernel<D, BF16>;
  static DeviceFlags configured;
  cudaError_t e = ensure_dyn_smem(kern, L::kDynSmem, configured);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3((unsigned)a.grid), kThreads, L::kDynSmem, a.stream, a.tmQ,
                          a.tmK, a.tmV, a.params);
}

template <int D>
cudaError_t launch_d(const PagedLaunch& a, bool bf16) {
  return bf16 ? launch_db<D, true>(a) : launch_db<D, false>(a);
}

}  // namespace

cudaError_t launch_paged_tile(const PagedLaunch& a, int d, bool bf16) {
  switch (d) {
    case 64: return launch_d<64>(a, bf16);
    case 96: return launch_d<96>(a, bf16);
    default: return launch_d<128>(a, bf16);
  }
}

}  // namespace attn
