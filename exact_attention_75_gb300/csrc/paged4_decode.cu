// Attention of a few new tokens per sequence (at most 16 query rows per
// key/value head) over a paged cache held in 4 bits (kv4.cuh).
//
// The work is cut and the results meet as in the 16-bit kernel (paged_rows.cuh,
// paged_decode.cu), and each warp streams its 32-key blocks through a ring, here
// as plain bulk copies of 16 rows.  Since a row is 5/8 byte a channel, the
// instructions that widen it are what competes with HBM: a card at full rate
// hands an SM a block every 111 cycles (d = 128), 444 issue slots for 4096
// values.  So the product is turned round against the 16-bit kernel's:
//   S^T = K Q^T  (A = 16 keys x 16 channels, B = 8 query rows)
//   O^T = V^T P^T  (A = 16 channels x 16 keys, B = 8 query rows),
// where the widened codes are the A operands in the registers that they were
// widened in, no shared memory between, and up to 8 rows cost half the products
// that 16 do.  Both contractions may take their index in any order and the rows
// of V^T may be any channels, so a lane takes the channels and keys whose codes
// lie side by side:
//   K: lane (g, t) = (lane / 4, lane % 4) reads channels 8 t .. of each group of 32
//      of keys g and g + 8; a word's nibbles i and i + 4 (16 bits apart) are one
//      operand register;
//   V: it reads channels g D/8 .. of keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9; two keys'
//      half words side by side give the pairs of keys that an operand holds.
// A group's product is taken with the codes in fp16, the query scaled into its range by
// a power of two, and s of its keys is applied to it in 32 bits; what m adds is one more
// product for all groups, with the query's sums in three terms: keys lose nothing.
// Values are m + c s rounded to 16 bits.  (In bf16 c s rounded by itself and m by a
// product of its own took an instruction less a pair of values, 50.1 us for the 50.5
// below, but what cancels between the two is lost: 2.5 times the error of O over a few
// keys.)
// P leaves the softmax by keys and is wanted by rows: one 8 x 8 transpose for 8
// keys.
//
// The running maximum is a reference that is raised only where a score passes
// it by 2^8 (P stays below that), so that most blocks need no maximum across lanes.
//
// No unit is full (some 370 instructions for 16 keys and 8 rows at d = 128: issue 58 % of
// the time, ALU 46 %, DRAM 50 %, tensor 17 %): what is left are waits between dependent
// instructions of 12 warps an SM, and the 15 us around them: 4 to the first key, the
// borders of items, 2 of meeting, 3 to 6 of join.  64 single tokens over 2048 to 8192 keys,
// 16 query heads on 4 of 128, 50.5 us, 196 MB, 3.9 TB/s; over up to 65536 keys 297 us,
// 5.3 TB/s, 0.79 of a copy's rate (the 16-bit cache's: 102 us and 0.90 for 3.2 times the
// bytes).  d = 96 takes 47, d = 64 37, 16 rows 68.  Drafts of 16 rows (8 warps an SM: issue
// 39 %, DRAM 20 %) are such waits altogether.  Six warps a CTA, two CTAs an
// SM; four, five and eight took 1, 9 and 7 % longer.
#include <cuda_runtime.h>
#include <cstdint>

#include "dependent.cuh"
#include "kv4.cuh"
#include "mma16.cuh"
#include "paged.cuh"
#include "paged_rows.cuh"
#include "sm103_ptx.cuh"
#include "smem_attr.cuh"

namespace attn {

using namespace rows;

namespace {

constexpr int kKeys = 2 * kUnit;  // of a block
// Warps of a CTA by 8-row tiles: what two CTAs an SM leave registers for.
template <int NT>
constexpr int kWarps = NT == 1 ? 6 : 4;
constexpr float kRaise = 8.f;  // log2 units

template <int D, int W>
struct Paged4Layout {
  static constexpr int kRow = kv4_row(D);
  static constexpr int kUnitBytes = kUnit * kRow;   // K or V of 16 keys
  static constexpr int kSlotBytes = 4 * kUnitBytes;  // K, K, V, V of a block
  static constexpr int kSlots = 100 * 1024 / (W * kSlotBytes);  // ring depth of each warp
  static constexpr int kRingBytes = W * kSlots * kSlotBytes;
  static constexpr int kMeetOff = kRingBytes;
  static constexpr int kMlOff = kMeetOff + W * kMeet * kRowStride<D> * 4;
  static constexpr int kBarOff = kMlOff + W * kMeet * 8;
  static constexpr int kFlagOff = kBarOff + W * kSlots * 8;
  static constexpr int kBytes = kFlagOff + 16 + 128;  // + room to align the base
  static_assert(kUnitBytes % 16 == 0 && kRingBytes % 128 == 0, "bulk copies");
  static_assert(kRingBytes >= kPagedRows * (D * 4 + 8), "a cluster's part lies over the ring");
  static_assert(kBytes + 256 <= 113 * 1024, "two CTAs per SM");
  static_assert(W * kKeys <= kPaged4Share, "a share holds a cost block");
};

// Bytes global -> shared (both addresses and the size multiples of 16),
// completion signalled on an mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
      : "memory");
}

// The 8 x 8 matrix of 16-bit values of which lane l holds row l / 4, columns
// 2 (l % 4) and the next, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// N 32-bit words from shared memory, at an address of that space (a generic one
// costs 64-bit arithmetic and a look at what it points to).
template <int N>
__device__ __forceinline__ void load_words(uint32_t a, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(a)
                 : "memory");
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[i]) : "r"(a + 4 * i) : "memory");
  }
}
__device__ __forceinline__ uint32_t load_word(uint32_t a) {
  uint32_t w[1];
  load_words<1>(a, w);
  return w[0];
}

// The codes of 4 C channels of two keys (at a: the first's, at b: the second's), the
// first key's in the low halves.
template <int C>
__device__ __forceinline__ void load_pairs(uint32_t a, uint32_t b, uint32_t (&w)[C]) {
  if constexpr (C == 3) {
    auto half = [](uint32_t at) {
      uint16_t x;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at) : "memory");
      return (uint32_t)x;
    };
#pragma unroll
    for (int c = 0; c < C; ++c) w[c] = half(a + 2 * c) | half(b + 2 * c) << 16;
  } else {
    uint32_t x[C / 2], y[C / 2];
    load_words<C / 2>(a, x);
    load_words<C / 2>(b, y);
#pragma unroll
    for (int c = 0; c < C; ++c) w[c] = __byte_perm(x[c / 2], y[c / 2], c & 1 ? 0x7632 : 0x5410);
  }
}

// NT: 8-row tiles of query rows.  CLUSTER as in the 16-bit kernel.
template <int D, bool BF16, int NT, bool CLUSTER>
__global__ void __launch_bounds__(kWarps<NT> * 32, 2) paged4_decode_kernel(const PagedParams p) {
  constexpr int W = kWarps<NT>;
  using L = Paged4Layout<D, W>;
  constexpr int KS = D / 16;  // k-steps of S^T, 16-channel tiles of O^T
  constexpr int C = D / 32;   // a lane's words of a key, half words of a value row
  constexpr int NS = L::kSlots;
  constexpr bool kSplit = D == 96;  // a lane's channels of V lie in more than one group
  constexpr int G = kSplit ? C : 1;  // scales and minima of them
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                             ~static_cast<uintptr_t>(127));
  const uint32_t sbase = smem_u32(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kFlagOff);
  // (the warp's number as one value, which the compiler can keep for the whole warp)
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  auto bar = [&](int s) { return sbase + L::kBarOff + 8u * (uint32_t)(warp * NS + s); };

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < W * NS; ++i) mbar_init(sbase + L::kBarOff + 8u * i, 1);
    mbar_fence_init();
  }
  grid_wait();
  Walk<W, kKeys> w = start_rows<W, kKeys, CLUSTER>(p);
  Watchdog wd{p.status, abort_flag, p.wait_limit_ns};
  const uint32_t ring = sbase + (uint32_t)(warp * NS * L::kSlotBytes);

  // Block n of the warp's stream lies in slot n % NS; the ring is full until the
  // stream ends, so the slot that is read is the one that is filled next.
  BlockStream<W, kKeys, CLUSTER> stream(p, w, warp, lane);
  uint32_t it = 0;         // blocks taken from the ring
  int slot = 0;            // it % NS
  uint32_t parity = 0;     // (it / NS) & 1
  auto issue = [&](int s) {
    if (!stream.more()) return;
    // A page outside the cache (reported): any of it.  Past the sequence a unit is
    // what its page holds, or, in a page of its own, what the slot held: numbers that
    // count nothing.
    const bool two = p.page == kUnit;  // a unit a page
    const int page0 = stream.page(p, 0, lane), page1 = two ? stream.page(p, 1, lane) : 0;
    if (lane == 0) {
      auto copy = [&](int page, int u, int units) {
        const size_t row = (((size_t)max(page, 0) * p.Hkv + stream.ahead.head) << p.page_log2) +
                           stream.row(p, u);
        const uint32_t dst = ring + (uint32_t)(s * L::kSlotBytes + u * L::kUnitBytes);
        const uint32_t bytes = (uint32_t)(units * L::kUnitBytes);
        bulk_load(dst, p.k4 + row * L::kRow, bytes, bar(s));
        bulk_load(dst + 2 * L::kUnitBytes, p.v4 + row * L::kRow, bytes, bar(s));
      };
      const int units = two && page1 == -2 ? 1 : 2;
      mbar_arrive_expect_tx(bar(s), (uint32_t)(2 * units * L::kUnitBytes));
      copy(page0, 0, two ? 1 : 2);
      if (two && units == 2) copy(page1, 1, 1);
    }
    stream.next(p, warp, lane);
  };
  for (int i = 0; i < NS; ++i) issue(i);

  float* meet = reinterpret_cast<float*>(smem + L::kMeetOff);
  float2* meet_ml = reinterpret_cast<float2*>(smem + L::kMlOff);  // [W][kMeet]
  // The CTA's part of a cluster's item, over the idle ring: O, (m, l) by row.
  float* part = reinterpret_cast<float*>(smem);
  float2* part_ml = reinterpret_cast<float2*>(smem + kPagedRows * D * 4);
  bool given_up = false;

  for (; w.left > 0; w.advance(p, p.max_q)) {
    if (!CLUSTER && w.nothing()) continue;
    const int nbw = warp_blocks(w, warp);
    const PagedSeq sq = w.sq;
    const int rows = min(kPagedRows, sq.qlen * p.G);
    // Q^T: of row 8 nt + g the channels that the lane has of the keys (kv4_query) and the
    // terms of the sums over each group; of rows 8 nt + 2 t and the next what takes
    // their products to base 2.
    uint32_t qb[NT][KS][2];
    uint2 qm[NT];
    float2 to2[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + g;
      const uint16_t* q =
          static_cast<const uint16_t*>(p.q) + (r < rows ? row_of(p, w, r) * D + 8 * t : 0);
      uint4 x[C];
#pragma unroll
      for (int c = 0; c < C; ++c)
        x[c] = r < rows ? *reinterpret_cast<const uint4*>(q + 32 * c) : make_uint4(0u, 0u, 0u, 0u);
      float sums[C];
      const float undo = kv4_query<BF16, C>(x, sums);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        qb[nt][2 * c][0] = x[c].x;
        qb[nt][2 * c][1] = x[c].y;
        qb[nt][2 * c + 1][0] = x[c].z;
        qb[nt][2 * c + 1][1] = x[c].w;
      }
      qm[nt] = kv4_sum_terms<BF16, C>(sums, t);
      const float by = kv4_to_base2(p.scale_log2, undo);
      to2[nt] = make_float2(__shfl_sync(0xffffffffu, by, 8 * t),
                            __shfl_sync(0xffffffffu, by, 8 * t + 4));
    }
    // Last key that rows 8 nt + 2 t and the next see, and the item's first row.
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) lim[nt][e] = last_key_of(p, sq, 8 * nt + 2 * t + e);
    const int lim0 = last_key_of(p, sq, 0);

    float o[NT][KS][4];
    // The reference of a row's exponentials, what it is subtracted as (0 before there
    // is one), the product beyond which it is raised; the sum of the exponentials.
    float m[NT][2], ref[NT][2], limit[NT][2];
    float2 l[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < KS; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      m[nt][0] = m[nt][1] = limit[nt][0] = limit[nt][1] = -INFINITY;
      ref[nt][0] = ref[nt][1] = 0.f;
      l[nt] = make_float2(0.f, 0.f);
    }
    bool aborted = false;
    int key0 = first_key(w, warp, 0) - W * kKeys;
#pragma unroll 1
    for (int j = 0; j < nbw; ++j) {
      if (!__all_sync(0xffffffffu, mbar_wait(bar(slot), parity, wd, 76))) {
        aborted = true;
        break;
      }
      ++it;
      const uint32_t block = ring + (uint32_t)(slot * L::kSlotBytes);
      key0 += W * kKeys;

      // S^T: x[nt][2 u + h] is rows 8 nt + 2 t and the next, key key0 + 16 u + 8 h + g.
      float2 x[NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t kw[2][C], kp[2][C];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t row = block + u * L::kUnitBytes + (g + 8 * h) * L::kRow;
#pragma unroll
          for (int c = 0; c < C; ++c) kw[h][c] = load_word(row + 16 * c + 4 * t);
          load_words<C>(row + D / 2, kp[h]);
        }
        {
          const uint32_t m0 = kv4_minima(kp[0], t), m1 = kv4_minima(kp[1], t);
          const uint32_t a[4] = {m0, m1, m0, m1};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float y[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816<BF16>(y, a, qm[nt].x, qm[nt].y);
            x[nt][2 * u] = make_float2(y[0], y[1]);
            x[nt][2 * u + 1] = make_float2(y[2], y[3]);
          }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          uint32_t v[2][4];
          float s[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            s[h] = unpack2<BF16>(kp[h][c]).x;
            kv4_halves(kw[h][c], v[h]);
          }
          const uint32_t a0[4] = {v[0][0], v[1][0], v[0][1], v[1][1]};
          const uint32_t a1[4] = {v[0][2], v[1][2], v[0][3], v[1][3]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float y[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816<false>(y, a0, qb[nt][2 * c][0], qb[nt][2 * c][1]);
            mma16816<false>(y, a1, qb[nt][2 * c + 1][0], qb[nt][2 * c + 1][1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float2& z = x[nt][2 * u + h];
              z.x = fmaf(s[h], y[2 * h], z.x);
              z.y = fmaf(s[h], y[2 * h + 1], z.y);
            }
          }
        }
      }

      // Online softmax.
      if (key0 + kKeys - 1 > lim0) {
        asm volatile("");  // few blocks: a branch, not selects in every one
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (key0 + g + 8 * i > lim[nt][0]) x[nt][i].x = -INFINITY;
            if (key0 + g + 8 * i > lim[nt][1]) x[nt][i].y = -INFINITY;
          }
      }
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          raise |= x[nt][i].x > limit[nt][0] || x[nt][i].y > limit[nt][1];
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            auto at = [&](int i) { return e ? x[nt][i].y : x[nt][i].x; };
            float b = fmaxf(fmaxf(at(0), at(1)), fmaxf(at(2), at(3)));
            b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 4));
            b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 8));
            b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 16));
            // (by the row's own scores alone: no row's bits depend on another's)
            if (!(b > limit[nt][e])) continue;
            const float by = e ? to2[nt].y : to2[nt].x, n = b * by;
            const float alpha = ex2_approx(m[nt][e] - n);
            m[nt][e] = ref[nt][e] = n;
            limit[nt][e] = b + kRaise / by;  // (infinite where no product can be that much more)
            (e ? l[nt].y : l[nt].x) *= alpha;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              o[nt][i][e] *= alpha;
              o[nt][i][e + 2] *= alpha;
            }
          }
      }
      // P is rounded to 16 bits for its product, as in the 16-bit kernel; l sums
      // the unrounded values.
      uint32_t pb[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 z = __ffma2_rn(x[nt][i], to2[nt], make_float2(-ref[nt][0], -ref[nt][1]));
          z = make_float2(ex2_approx(z.x), ex2_approx(z.y));
          l[nt] = __fadd2_rn(l[nt], z);
          pb[nt][i] = transpose8(pack2<BF16>(z.x, z.y));
        }
      }

      // O^T += V^T P^T.
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        // keys 2 t, 2 t + 1 and those 8 behind: codes, and s and m of each key
        uint32_t vw[2][C], vp[2][2][G];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a = block + (2 + u) * L::kUnitBytes + (2 * t + 8 * h) * L::kRow;
          load_pairs<C>(a + g * (D / 16), a + L::kRow + g * (D / 16), vw[h]);
#pragma unroll
          for (int n = 0; n < G; ++n) {
            const int group = (C * g + n) / 8;
            vp[h][0][n] = load_word(a + D / 2 + 4 * group);
            vp[h][1][n] = load_word(a + L::kRow + D / 2 + 4 * group);
          }
        }
        if (key0 + kKeys > sq.klen) {
          asm volatile("");
          // Rows past the sequence's last key hold whatever the page, or the slot,
          // held (P is 0 there, but 0 x NaN is not): they stand for 0.
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int n = 0; n < G; ++n)
                if (key0 + 16 * u + 2 * t + 8 * h + e >= sq.klen) vp[h][e][n] = 0u;
        }
        uint32_t sc[2][G], lo[2][G];  // scales and minima of two keys side by side
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < G; ++n) {
            sc[h][n] = __byte_perm(vp[h][0][n], vp[h][1][n], 0x5410);
            lo[h][n] = __byte_perm(vp[h][0][n], vp[h][1][n], 0x7632);
          }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          uint32_t v[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int n = kSplit ? c : 0;
            kv4_values<BF16>(vw[h][c], sc[h][n], lo[h][n], v[h]);
          }
          const uint32_t a0[4] = {v[0][0], v[0][1], v[1][0], v[1][1]};
          const uint32_t a1[4] = {v[0][2], v[0][3], v[1][2], v[1][3]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816<BF16>(o[nt][2 * c], a0, pb[nt][2 * u], pb[nt][2 * u + 1]);
            mma16816<BF16>(o[nt][2 * c + 1], a1, pb[nt][2 * u], pb[nt][2 * u + 1]);
          }
        }
      }

      // The slot is read: refill it with the next block of the stream.
      __syncwarp();
      if (lane == 0) fence_proxy_async_smem();
      issue(slot);
      if (++slot == NS) {
        slot = 0;
        parity ^= 1;
      }
    }
    // The warps leave together when one has given up; the barrier also frees
    // the meeting place from the piece before.
    given_up = __syncthreads_or(aborted);
    if (given_up) break;

#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        l[nt].x += __shfl_xor_sync(0xffffffffu, l[nt].x, off);
        l[nt].y += __shfl_xor_sync(0xffffffffu, l[nt].y, off);
      }
    }

    // The warps' (O, m, l) meet in shared memory, kMeet rows at a time.  The
    // lane's channels of row 8 nt + 2 t + e are g D/8 .. in the order of the tiles
    // (two a tile).
    if (!CLUSTER && !w.whole() && threadIdx.x == 0) w.describe(p, 0);
    for (int pass = 0; pass * kMeet < rows; ++pass) {
      if (pass > 0) __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (2 * nt + (t >> 1) != pass) continue;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int mr = warp * kMeet + 2 * (t & 1) + e;
          float4* ro = reinterpret_cast<float4*>(meet + mr * kRowStride<D> + g * (D / 8));
#pragma unroll
          for (int c = 0; c < C; ++c)
            ro[c] = make_float4(o[nt][2 * c][e], o[nt][2 * c][e + 2], o[nt][2 * c + 1][e],
                                o[nt][2 * c + 1][e + 2]);
          if (g == 0) meet_ml[mr] = make_float2(m[nt][e], e ? l[nt].y : l[nt].x);
        }
      }
      __syncthreads();
      meet_rows<D, BF16, CLUSTER>(p, w, meet, meet_ml, part, part_ml, pass, rows);
    }
  }
  if constexpr (CLUSTER) join_cluster<D, BF16>(p, w, part, part_ml, given_up);
  // After an abort, copies still on their way must land before the CTA exits.
  Watchdog dw = wd;
  volatile int never = 0;
  dw.abort_flag = &never;
  dw.limit_ns = drain_limit_ns(wd.limit_ns);
  for (; it < stream.issued; ++it) mbar_wait(bar((int)(it % NS)), (it / NS) & 1, dw, 77);
  grid_release();
}

template <int D, bool BF16, int NT, bool CLUSTER>
cudaError_t launch_dbnc(const PagedLaunch& a) {
  using L = Paged4Layout<D, kWarps<NT>>;
  static DeviceFlags configured;
  auto kern = paged4_decode_kernel<D, BF16, NT, CLUSTER>;
  cudaError_t e = ensure_dyn_smem(kern, L::kBytes, configured);
  if (e != cudaSuccess) return e;
  return launch_clusters(kern, CLUSTER ? a.params.cluster : 1, dim3((unsigned)a.grid),
                         kWarps<NT> * 32, L::kBytes, a.stream, a.params);
}

template <int D, bool BF16, int NT>
cudaError_t launch_dbn(const PagedLaunch& a) {
  return a.params.cluster > 0 ? launch_dbnc<D, BF16, NT, true>(a)
                              : launch_dbnc<D, BF16, NT, false>(a);
}

template <int D>
cudaError_t launch_d(const PagedLaunch& a, bool bf16) {
  const bool one = (int64_t)a.params.max_q * a.params.G <= 8;
  if (bf16) return one ? launch_dbn<D, true, 1>(a) : launch_dbn<D, true, 2>(a);
  return one ? launch_dbn<D, false, 1>(a) : launch_dbn<D, false, 2>(a);
}

}  // namespace

cudaError_t launch_paged4_decode(const PagedLaunch& a, int d, bool bf16) {
  switch (d) {
    case 64: return launch_d<64>(a, bf16);
    case 96: return launch_d<96>(a, bf16);
    default: return launch_d<128>(a, bf16);
  }
}

}  // namespace attn
