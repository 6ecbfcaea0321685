// Accumulated attention weights of a paged cache's positions: for position j of a
// sequence and one of its key/value heads
//   w_j = [j is older than the call's tokens] w_j + sum over the sequence's new
//         rows i and the head's query heads of exp(scale q_i k_j - LSE_i).
//
// The log-sum-exp is given, so each key is read once and no row waits for another:
// a warp takes 16 keys and the rows that see them, 8 at a time.  The product is
//   S^T = K Q^T  (A = 16 keys x 16 channels, B = 8 query rows),
// keys going from memory straight into the operand's registers (a lane reads 16
// bytes of keys g and g + 8; the contraction may take the channels in any order), the
// next block's while this one is multiplied.  The sum over rows stays in the lane
// that has the key, and four lanes add theirs up at the end: no atomics, the
// same bits from run to run.
//
// Queries are put in shared memory as operands, 64 rows at a time (a tile a warp): a
// warp's 8 rows of a decoding step then stay in registers, and the tiles of a longer
// run are read by all warps for all their keys.  Each 64 rows go over the keys once;
// from the second time on the keys come from L2.
//
// Of a cache in 4 bits (kv4.cuh) the product is taken with the codes in fp16, as in the
// decoding kernel, and what the groups' minima add is one more product for all of them.
//
// Work.  A block of 16 keys costs kRead + its tiles of 8 rows; the blocks of all
// sequences and heads laid end to end are shared out evenly over the grid, and
// the warps of a CTA take its blocks in turn.
//
// Single tokens are bound by HBM: 64 of them over 2048 to 8192 keys, 16 query heads on 4
// of 128, 57 us in 16 bits, 6.0 TB/s, 0.90 of a copy's rate.  In 4 bits 37, 2.1 times
// their bytes' time: a block ahead is 88 bytes a key, 22 KB on their way for an SM's 16
// warps, where HBM's rate and latency want some 35 (in 16 bits it is 67).  Windows are
// bound by the product's latencies and the operands read for it: 4 of 32 tokens over up to
// 16384 keys, 16 heads on 8, 38 us in 4 bits (49 with the minima added to the scores one by
// one), 35 in 16; of 256 tokens 235 and 203; a whole prompt of 4096, whose keys are read
// again for every 64 rows of a head, 893 and 582.
#include <cuda_runtime.h>
#include <cstdint>

#include "dependent.cuh"
#include "kv4.cuh"
#include "mma16.cuh"
#include "paged.cuh"
#include "retain.cuh"
#include "sm103_ptx.cuh"

namespace attn {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kKeys = 16;  // of a block: never past the end of a page
constexpr int kRead = 3;   // cost of reading a block, in tiles of 8 rows

// A sequence's part of the line.
struct Line {
  PagedSeq sq;
  int blocks, cost;  // key blocks of a head, cost of each
  __device__ __forceinline__ Line(const PagedParams& p, int b) : sq(paged_seq(p, b)) {
    blocks = sq.qlen > 0 ? (sq.klen + kKeys - 1) / kKeys : 0;
    cost = kRead + (int)(((long long)sq.qlen * p.G + 7) / 8);
  }
  __device__ __forceinline__ long long head() const { return (long long)blocks * cost; }
};

// The CTA's share [begin, end) of the line, the first sequence of it and where
// that one begins.
struct Share {
  long long begin, end, at;
  int b;
};

__device__ __forceinline__ Share find_share(const PagedParams& p) {
  __shared__ long long warp_sum[kWarps];
  __shared__ Share share;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (p.n_seq + kThreads - 1) / kThreads;
  const int b0 = min(tid * run, p.n_seq), b1 = min(b0 + run, p.n_seq);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    sum += Line(p, b).head() * p.Hkv;
    if (blockIdx.x == 0) paged_check(p, b);
  }
  long long incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += up;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (tid == 0) share = {0, 0, 0, 0};
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_sum[w];
    all += warp_sum[w];
  }
  const long long part = (all + gridDim.x - 1) / gridDim.x;
  const long long s = part * blockIdx.x;
  long long at = before + incl - sum;
  if (s < all && s >= at && s < at + sum) {
    int b = b0;
    for (;; ++b) {
      const long long line = Line(p, b).head() * p.Hkv;
      if (s < at + line) break;
      at += line;
    }
    share = {s, min(s + part, all), at, b};
  }
  __syncthreads();
  return share;
}

// Last key that token i of a sequence sees.
__device__ __forceinline__ int last_key(const PagedParams& p, const PagedSeq& sq, int i) {
  return min(p.causal ? i + sq.klen - sq.qlen : sq.klen, sq.klen - 1);
}

// A block's keys as operand A: register pairs of row g (h = 0) and g + 8.
template <int D, bool KV4>
struct Keys {
  static constexpr int C = D / 32;
  uint4 x[2][KV4 ? 1 : C];     // 16 bits: channels 32 c + 8 t ..
  uint32_t code[2][KV4 ? C : 1], par[2][KV4 ? C : 1];
  float old[2];                // the weights so far
  size_t slot;                 // of the block's first key in weights; valid only
  bool valid;

  // page: of the block, key0: its first key
  template <typename Params>
  __device__ __forceinline__ void load(const Params& a, int page, int head, int key0, int g,
                                       int t) {
    const PagedParams& p = a.paged;
    valid = page >= 0 && page < p.n_pages;
    if (!valid) return;
    slot = (((size_t)page * p.Hkv + head) << p.page_log2) + (key0 & (p.page - 1));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const size_t row = slot + g + 8 * h;
      if constexpr (KV4) {
        const uint32_t* k = reinterpret_cast<const uint32_t*>(p.k4 + row * kv4_row(D));
#pragma unroll
        for (int c = 0; c < C; ++c) {
          code[h][c] = __ldg(k + 4 * c + t);
          par[h][c] = __ldg(k + D / 8 + c);
        }
      } else {
        const uint4* k = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(a.k_pages) + row * D);
#pragma unroll
        for (int c = 0; c < C; ++c) x[h][c] = __ldg(k + 4 * c + t);
      }
      old[h] = a.weights[row];
    }
  }
};

// A row of queries beside its operand: what takes its products to base 2, its
// log-sum-exp in base 2, the last key it sees, and the last that all of its tile see.
struct RowInfo {
  float to2, lse;
  int lim, all;
};

template <int D, bool BF16, bool KV4>
__global__ void __launch_bounds__(kThreads, 2) kv_weights_kernel(const WeightsParams a) {
  constexpr int C = D / 32;
  __shared__ uint4 tiles[kWarps][C][32];  // operand B of 8 rows: by lane
  __shared__ uint2 minima[KV4 ? kWarps : 1][32];  // operand B of what the minima add
  __shared__ __align__(16) RowInfo info[kWarps * 8];
  const PagedParams& p = a.paged;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  grid_wait();
  const Share share = find_share(p);

  long long at = share.at;  // where sequence b begins
  for (int b = share.b; at < share.end; ++b) {
    const Line line(p, b);
    const PagedSeq sq = line.sq;
    const long long whole = line.head();
    const int rows = sq.qlen * p.G;
    for (int head = 0; head < p.Hkv && whole > 0; ++head, at += whole) {
      if (at + whole <= share.begin || at >= share.end) continue;
      // blocks whose first unit of cost lies in the share
      const int u0 = (int)((max(share.begin - at, 0LL) + line.cost - 1) / line.cost);
      const int u1 = (int)((min(share.end - at, whole) + line.cost - 1) / line.cost);
      auto page_of = [&](int u) {
        return u < u1 ? __ldg(p.block_table + (size_t)b * p.max_pages +
                              (u * kKeys >> p.page_log2))
                      : -2;
      };
      auto get = [&](Keys<D, KV4>& k, int page, int u) {
        k.load(a, page, head, u * kKeys, g, t);
        if (!k.valid && page != -2 && lane == 0)
          atomicCAS(p.status, 0u, 1u | (64u << 8) | ((uint32_t)min(b, 0xFFFF) << 16));
      };
      for (int r0 = 0; r0 < rows; r0 += 8 * kWarps) {
        // The first keys are on their way while the queries are prepared.
        int u = u0 + warp;
        Keys<D, KV4> k;
        get(k, page_of(u), u);
        int page = page_of(u + kWarps);
        const int n_tiles = min(kWarps, (rows - r0 + 7) / 8);
        __syncthreads();  // the tiles before have been read
        if (warp < n_tiles) {
          const int r = r0 + 8 * warp + g, i = r / p.G, h = r - i * p.G;
          const bool live = i < sq.qlen;
          const size_t row = live ? (size_t)(head * p.G + h) * p.total + sq.s0 + i : 0;
          const uint4* x =
              reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + row * D);
          uint4 q[C];
#pragma unroll
          for (int c = 0; c < C; ++c)
            q[c] = live ? __ldg(x + 4 * c + t) : make_uint4(0u, 0u, 0u, 0u);
          RowInfo ri = {};
          ri.to2 = p.scale_log2;
          if constexpr (KV4) {
            float sums[C];
            const float undo = kv4_query<BF16, C>(q, sums);
            minima[warp][lane] = kv4_sum_terms<BF16, C>(sums, t);
            ri.to2 = kv4_to_base2(p.scale_log2, undo);
          }
#pragma unroll
          for (int c = 0; c < C; ++c) tiles[warp][c][lane] = q[c];
          ri.lim = live ? last_key(p, sq, i) : -1;
          ri.all = ri.lim;
#pragma unroll
          for (int off = 4; off < 32; off <<= 1)
            ri.all = min(ri.all, __shfl_xor_sync(0xffffffffu, ri.all, off));
          ri.lse = live ? 1.4426950408889634f * __ldg(p.lse + row) : 0.f;
          if (t == 0) info[8 * warp + g] = ri;
        }
        __syncthreads();
        uint4 q[C];
        uint2 qm = {};
        RowInfo ri[2];
        auto load_tile = [&](int n) {
          if constexpr (KV4) qm = minima[n][lane];
#pragma unroll
          for (int c = 0; c < C; ++c) q[c] = tiles[n][c][lane];
          ri[0] = info[8 * n + 2 * t];
          ri[1] = info[8 * n + 2 * t + 1];
        };
        if (n_tiles == 1) load_tile(0);

        for (; u < u1; u += kWarps) {
          const Keys<D, KV4> cur = k;
          get(k, page, u + kWarps);
          page = page_of(u + 2 * kWarps);
          if (!cur.valid) continue;
          const int key0 = u * kKeys;
          uint32_t v[KV4 ? C : 1][2][4];  // 4 bits: the codes, and s and m
          float scale[KV4 ? C : 1][2];
          uint32_t am[4] = {};  // the minima
          if constexpr (KV4) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int c = 0; c < C; ++c) {
                scale[c][h] = unpack2<BF16>(cur.par[h][c]).x;
                kv4_halves(cur.code[h][c], v[c][h]);
              }
              am[h] = am[h + 2] = kv4_minima(cur.par[h], t);
            }
          }
          float sum[2] = {0.f, 0.f};
          for (int n = 0; n < n_tiles; ++n) {
            if (n_tiles > 1) load_tile(n);
            float x[4] = {0.f, 0.f, 0.f, 0.f};  // key g + 8 (e / 2), row 2 t + e % 2 of the tile
            if constexpr (KV4) mma16816<BF16>(x, am, qm.x, qm.y);
#pragma unroll
            for (int c = 0; c < C; ++c) {
              if constexpr (KV4) {
                const uint32_t a0[4] = {v[c][0][0], v[c][1][0], v[c][0][1], v[c][1][1]};
                const uint32_t a1[4] = {v[c][0][2], v[c][1][2], v[c][0][3], v[c][1][3]};
                float y[4] = {0.f, 0.f, 0.f, 0.f};
                mma16816<false>(y, a0, q[c].x, q[c].y);
                mma16816<false>(y, a1, q[c].z, q[c].w);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = fmaf(scale[c][e >> 1], y[e], x[e]);
              } else {
                const uint32_t a0[4] = {cur.x[0][c].x, cur.x[1][c].x, cur.x[0][c].y, cur.x[1][c].y};
                const uint32_t a1[4] = {cur.x[0][c].z, cur.x[1][c].z, cur.x[0][c].w, cur.x[1][c].w};
                mma16816<BF16>(x, a0, q[c].x, q[c].y);
                mma16816<BF16>(x, a1, q[c].z, q[c].w);
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = ex2_approx(fmaf(x[e], ri[e & 1].to2, -ri[e & 1].lse));
            // (An unseen key may hold anything.  In 16 bits a test for none costs more than
            // it saves: the window 37.7 us, not 35.2.)
            if (!KV4 || key0 + kKeys - 1 > ri[0].all) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (key0 + g + 8 * (e >> 1) > ri[e & 1].lim) x[e] = 0.f;
            }
            sum[0] += x[0] + x[1];
            sum[1] += x[2] + x[3];
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
            const int key = key0 + g + 8 * h;
            if (t == 0 && key < sq.klen)
              a.weights[cur.slot + g + 8 * h] =
                  r0 > 0 || key < sq.klen - sq.qlen ? cur.old[h] + sum[h] : sum[h];
          }
        }
      }
    }
  }
  grid_release();
}

template <int D, bool BF16>
cudaError_t launch_db(const WeightsLaunch& a, bool kv4) {
  auto kern = kv4 ? kv_weights_kernel<D, BF16, true> : kv_weights_kernel<D, BF16, false>;
  return launch_dependent(kern, dim3((unsigned)a.grid), kThreads, 0, a.stream, a.params);
}

template <int D>
cudaError_t launch_d(const WeightsLaunch& a, bool bf16, bool kv4) {
  return bf16 ? launch_db<D, true>(a, kv4) : launch_db<D, false>(a, kv4);
}

}  // namespace

cudaError_t launch_kv_weights(const WeightsLaunch& a, int d, bool bf16, bool kv4) {
  switch (d) {
    case 64: return launch_d<64>(a, bf16, kv4);
    case 96: return launch_d<96>(a, bf16, kv4);
    default: return launch_d<128>(a, bf16, kv4);
  }
}

}  // namespace attn
