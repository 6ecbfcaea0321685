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
// Over a cache held in 4 bits (KV4; kv4.cuh) warps 12-15 take the producer's place
// for K and V: a thread owns a key of the block, has the next block's row on its way
// to registers, and stores the widened row where TMA would have put it.  The rest
// of the pipeline does not differ.  With 16 warps a thread has 128 registers, not the
// 168 in which a softmax thread holds a row of 128 scores: it holds half, and reads
// the other half twice, for the maximum and for the exponentials.  The channels of a
// word lie in a tile in the order in which its nibbles come out, 0, 4, 1, 5, 2, 6, 3, 7:
// queries are put in that order too, and O is put back from it.
//
// Keys of a 4-bit cache have more bits than a 16-bit operand (kv4.cuh).  Their
// scores are a product in fp16 of d + 16 columns: (c - 8) s by the query, exact, and
// behind them, for each group, m + 8 s by the query's sum over the group, both in two
// terms (three products).  The scale of an fp16 cache has 11 bits; its upper 8 and
// its lower 3 make a tile of keys each.  Powers of two bring every 32 keys, and each
// query, into fp16's range; the scores are scaled back where they are scaled anyway.
// The softmax threads prepare their queries' rows.  A pair of query tiles widens its
// keys again: with 32 pairs to a head, 2.35 us a key block for the 1.9 of 16 bits.  Widening,
// a longer softmax and what each border of an item runs once share the instruction
// cache, so the loops are kept short: with the halves of a row of scores unrolled, the
// words of a row and the preparation of queries too, the mixed batch took 84 us and the long
// chunk 463.  Measured: 4096 tokens over 16384 keys 446 us (fp16, with its two tiles of
// keys, 715), 4 chunks of up to 509 tokens with 12 single ones 71.  640 threads with
// registers moved between roles took 552 to 746 for the first, a whole row of scores
// held in 168 registers 617.
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
#include "kv4.cuh"
#include "mma16.cuh"
#include "paged.cuh"
#include "sm103_ptx.cuh"
#include "smem_attr.cuh"
#include "tiles.cuh"

namespace attn {

namespace {

template <bool KV4>
constexpr int kTileThreads = KV4 ? 512 : 352;
constexpr int kWarpProducer = 8;
constexpr int kWarpMma = 9;
constexpr int kWarpRelay = 10;
constexpr int kWarpWiden = 12;  // first of four
constexpr uint32_t kBarKv = 1, kBarP = 2;  // issuer <-> relay, issuer <-> softmax t
constexpr float kRescaleThreshold = 8.0f;  // log2 units: P stays <= 2^8
constexpr int kRows = kPagedTileRows;
constexpr int kExtraBytes = 128 * 32;      // 16 columns more of a tile (KV4)

template <int D, bool KV4>
struct PagedTileLayout {
  static constexpr int kTileBytes = 128 * kPaddedD<D> * 2;
  static constexpr int kSlots = D == 64 ? 8 : 4;  // K/V ring
  static constexpr int kQOff = 0;
  static constexpr int kKvOff = 2 * kTileBytes;
  static constexpr int kQExtraOff = kKvOff + kSlots * kTileBytes;
  static constexpr int kExtras = kSlots / 2;      // blocks of the ring at most
  static constexpr int kKExtraOff = kQExtraOff + (KV4 ? 2 * kExtraBytes : 0);
  // A softmax warp's rows on their way out, 32 or 64 columns at a time.
  static constexpr int kStageCols = KV4 ? 1 : 2;
  static constexpr int kStageBytes = 32 * 64 * kStageCols;
  static constexpr int kStageOff = kKExtraOff + (KV4 ? kExtras * kExtraBytes : 0);
  static constexpr int kBarOff = kStageOff + 8 * kStageBytes;
  static constexpr int kQFull = 0, kQEmpty = 2, kSFull = 4, kOFull = 6, kDrain = 8;
  static constexpr int kKvFull = 9, kKvEmpty = 9 + kSlots;
  static constexpr int kQReady = 9 + 2 * kSlots;  // queries for a 4-bit cache
  static constexpr int kNumBars = kQReady + 2;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  // Scales of 4 x 32 keys by block of a 4-bit cache.  The widening warps are at
  // most kSlots / 2 + 1 blocks past one whose scores are read.
  static constexpr int kScales = 8;
  static_assert(kScales > kSlots / 2 + 1, "a scale is read before it is written again");
  static constexpr int kScaleOff = (kMiscOff + 16 + 15) / 16 * 16;
  static constexpr int kBytes = kScaleOff + kScales * 16;
  static constexpr int kDynSmem = kBytes + 1024;  // + alignment slack
  static_assert(kDynSmem + 256 <= 232448, "shared memory budget (227 KB) exceeded");
};

// A walk along the CTA's share; an item is a pair of tiles of TT tokens each.
// Weights: a key block of one tile was measured at 1.06 us, of a pair at 1.55,
// an item's borders at 3 to 4 us; 3 : 4 and two blocks an item balance best (a
// mixed batch 58.5 us, with 2 : 3 59.8, with equal weights 60.4).  Over a 4-bit cache, where
// queries are prepared and the first keys widened at a border, three blocks an item (a mixed
// batch 70.6 us, 32 chunks of 24 tokens 52.4; two blocks 72.1 and 53.4, four 70.1 and 54.0).
template <bool KV4>
using Cost = PagedCost<128, 3, 4, KV4 ? 1536 : 1024, false>;
template <bool KV4>
struct Walk : PagedWalk<Cost<KV4>> {
  using Base = PagedWalk<Cost<KV4>>;
  using Base::advance, Base::item, Base::left, Base::nb, Base::sq, Base::two, Base::u0, Base::u1;
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

__device__ __forceinline__ float row_max32(const uint32_t (&s)[32]) {
  auto at = [&](int i) { return __uint_as_float(s[i]); };
  float m[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) m[a] = fmax3(at(3 * a), at(3 * a + 1), at(3 * a + 2));
#pragma unroll
  for (int i = 12; i < 28; i += 8) {
#pragma unroll
    for (int a = 0; a < 4; ++a) m[a] = fmax3(m[a], at(i + 2 * a), at(i + 2 * a + 1));
  }
  m[0] = fmax3(m[0], at(28), at(29));
  m[1] = fmax3(m[1], at(30), at(31));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// x as the sum of two fp16 numbers (22 bits of it), the first in the low half.
__device__ __forceinline__ uint32_t two_terms(float x) {
  const float hi = unpack2<false>(pack_f16x2(x, 0.f)).x;
  return pack_f16x2(x, x - hi);
}

// Shared memory by its own addresses (a pointer into the dynamic part is generic: it
// costs 64-bit arithmetic and a look at what it points to).
__device__ __forceinline__ uint4 load_smem16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void store_smem16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
// Piece c of row `row` of a tile (128-byte swizzle; the tile begins at a multiple of 1024).
__device__ __forceinline__ uint32_t tile_piece(uint32_t tile, int row, int c) {
  const uint32_t first = tile + row * 128 + ((row & 7) << 4);
  return (first ^ ((c & 7) << 4)) + (c >> 3) * 16384;
}

// Row `row` of a tile's 16 further columns (32 bytes a row, 32-byte swizzle): columns
// 0-7, then 8-11; the last four are 0.
__device__ __forceinline__ void store_extra(uint32_t extra, int row, uint4 a, uint2 b) {
  const uint32_t x = extra + row * 32, swap = (row >> 2 & 1) * 16;
  store_smem16(x + swap, a);
  store_smem16(x + (swap ^ 16), make_uint4(b.x, b.y, 0u, 0u));
}

// N words from global memory, aligned as rows of a 4-bit cache are.
template <int N, int ALIGN>
__device__ __forceinline__ void read_words(const uint8_t* x, uint32_t (&w)[N]) {
  if constexpr (ALIGN % 16 == 0 && N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(x) + i / 4);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  } else if constexpr (ALIGN % 8 == 0 && N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(x) + i / 2);
      w[i] = v.x, w[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(x) + i);
  }
}

// A row of a 4-bit cache: its code words, and its groups' scales and minima.
template <int D>
struct Row4 {
  uint32_t w[D / 8], par[D / 32];

  // Rows of 128 are widened in two turns of a loop: all roles' instructions have to fit
  // their cache.
  static constexpr int kParts = D == 128 ? 2 : 1, kGroups = D / 32 / kParts;
  // Number i of part h of x, whose parts have n.
  template <int N>
  static __device__ __forceinline__ uint32_t part(const uint32_t (&x)[N], int n, int h, int i) {
    return kParts == 1 ? x[i] : (h ? x[n + i] : x[i]);
  }

  __device__ __forceinline__ void load(const uint8_t* x) {  // null: a row of zeros
#pragma unroll
    for (int i = 0; i < D / 8; ++i) w[i] = 0u;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) par[i] = 0u;
    if (x == nullptr) return;
    read_words<D / 8, kv4_row(D)>(x, w);
    read_words<D / 32, kv4_row(D)>(x + D / 2, par);
  }
  // The bits of the largest finite number that key() has to hold.
  template <bool BF16>
  __device__ __forceinline__ uint32_t top() const {
    uint32_t b = 0u;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const float2 p = unpack2<BF16>(par[c]);
      b = max(b, max(finite_bits(8.f * p.x), finite_bits(fmaf(8.f, p.x, p.y))));
    }
    return b;
  }
  // Row `row` of a tile of keys times f: the codes less 8, times the upper 8 bits of the
  // scale or what these leave of it (LOW).
  template <bool BF16, bool LOW>
  __device__ __forceinline__ void key(uint32_t tile, int row, float f) const {
#pragma unroll 1
    for (int h = 0; h < kParts; ++h) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const float s = unpack2<BF16>(part(par, kGroups, h, g)).x * f;
        const float hi = __uint_as_float(__float_as_uint(s) & 0xFFFF0000u);
        const float by = LOW ? s - hi : hi;
        const uint32_t even = pack_f16x2(by, by), odd = pack_f16x2(by * 0.0625f, by * 0.0625f);
#pragma unroll
        for (int c = 4 * g; c < 4 * g + 4; ++c)
          store_smem16(tile_piece(tile, row, c) + h * 16384,
                       kv4_scaled_word(part(w, 4 * kGroups, h, c), even, odd));
      }
    }
  }
  // Its columns behind: m + 8 s in two terms, the first of them once more.
  template <bool BF16>
  __device__ __forceinline__ void key_extra(uint32_t extra, int row, float f) const {
    uint32_t two[4] = {0u, 0u, 0u, 0u};  // first and second term
#pragma unroll
    for (int g = 0; g < D / 32; ++g) {
      const float2 p = unpack2<BF16>(par[g]);
      two[g] = two_terms(fmaf(8.f, p.x, p.y) * f);
    }
    store_extra(extra, row, make_uint4(two[0], two[1], two[2], two[3]),
                make_uint2(__byte_perm(two[0], two[1], 0x5410),
                           __byte_perm(two[2], two[3], 0x5410)));
  }
  // Widened values.
  template <bool BF16>
  __device__ __forceinline__ void value(uint32_t tile, int row) const {
#pragma unroll 1
    for (int h = 0; h < kParts; ++h) {
#pragma unroll
      for (int c = 0; c < 4 * kGroups; ++c)
        store_smem16(tile_piece(tile, row, c) + h * 16384,
                     kv4_word<BF16, false>(part(w, 4 * kGroups, h, c),
                                           part(par, kGroups, h, c / 4)));
    }
  }
};

// Row `row` of a tile of queries as fp16, scaled into its range with room for sums
// of 32, and the sums over its groups as the columns behind: the first term twice,
// the second.  The factor that undoes the scaling.
template <int D, bool BF16>
__device__ __forceinline__ float query_row(uint32_t tile, uint32_t extra, int row) {
  // The largest of the row, by the bits of |x| two at a time; a number by number look at a
  // row that is not finite.
  uint32_t both = 0u;
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    const uint4 x = load_smem16(tile_piece(tile, row, c));
    const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("max.u16x2 %0, %0, %1;" : "+r"(both) : "r"(y[i] & 0x7FFF7FFFu));
  }
  const uint32_t most = max(both & 0xFFFFu, both >> 16);
  uint32_t top = __float_as_uint(unpack2<BF16>(most).x);
  if (most >= (BF16 ? 0x7F80u : 0x7C00u)) {
    top = 0u;
#pragma unroll 1
    for (int c = 0; c < D / 8; ++c) {
      const uint4 x = load_smem16(tile_piece(tile, row, c));
      const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = unpack2<BF16>(y[i]);
        top = max(top, max(finite_bits(v.x), finite_bits(v.y)));
      }
    }
  }
  const float2 f = to_fp16_range<9>(top);
  const uint32_t x32 = extra + row * 32, swap = (row >> 2 & 1) * 16;  // (as store_extra)
  store_smem16(x32 + swap, make_uint4(0u, 0u, 0u, 0u));
  store_smem16(x32 + (swap ^ 16), make_uint4(0u, 0u, 0u, 0u));
#pragma unroll 1
  for (int g = 0; g < D / 32; ++g) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t at = tile_piece(tile, row, 4 * g + i);
      const uint4 x = load_smem16(at);
      uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 v = unpack2<BF16>(y[e]);
        v.x *= f.x;
        v.y *= f.x;
        sum += v.x + v.y;
        y[e] = pack_f16x2(v.x, v.y);
      }
      // channels (0, 1) (2, 3) (4, 5) (6, 7) as (0, 4) (1, 5) (2, 6) (3, 7)
      store_smem16(at,
                   make_uint4(__byte_perm(y[0], y[2], 0x5410), __byte_perm(y[0], y[2], 0x7632),
                              __byte_perm(y[1], y[3], 0x5410), __byte_perm(y[1], y[3], 0x7632)));
    }
    const uint32_t two = two_terms(sum);
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(x32 + swap + 4 * g),
                 "r"(__byte_perm(two, 0u, 0x1010))
                 : "memory");
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(x32 + (swap ^ 16) + 2 * g),
                 "h"((uint16_t)(two >> 16))
                 : "memory");
  }
  return f.y;
}

// Descriptor of 16 further columns (store_extra): 8 rows of 32 bytes every 256, the
// 32-byte swizzle (bit 4 of the address changes with bit 7).
__device__ __forceinline__ uint64_t extra_desc(uint32_t addr) {
  constexpr uint64_t kSwizzles = 7ull << 61, kSwizzle32 = 6ull << 61;
  return (sdesc_sw128(addr, 16, 256) & ~kSwizzles) | kSwizzle32;
}

template <int D, bool BF16, bool KV4>
__global__ void __launch_bounds__(kTileThreads<KV4>, 1)
    paged_tile_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
  using L = PagedTileLayout<D, KV4>;
  constexpr int kChunks = kPaddedD<D> / 64;
  constexpr int kKeyTiles = KV4 && !BF16 ? 2 : 1;  // tiles of a block's keys
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
  float4* const scales = reinterpret_cast<float4*>(smem + L::kScaleOff);

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(L::kQFull + t), 1);
      mbar_init(bar(L::kQEmpty + t), 1);
      mbar_init(bar(L::kQReady + t), 4);
      mbar_init(bar(L::kSFull + t), 1);
      mbar_init(bar(L::kOFull + t), 1);
    }
    mbar_init(bar(L::kDrain), 1);
    for (int s = 0; s < L::kSlots; ++s) {
      mbar_init(bar(L::kKvFull + s), KV4 ? 4 : 1);
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
  Walk<KV4> w;
  // (a CTA barrier)
  static_cast<PagedWalk<Cost<KV4>>&>(w) =
      paged_start<Cost<KV4>, kTileThreads<KV4>>(p, 2 * TT);
  if (w.left > 0) w.tiles(p, TT);
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  if (warp >= kWarpProducer) {
    if (warp == kWarpProducer) {
      // ------------------------------------------------------ TMA producer ---
      const int box_rows = min(p.page, 128);
      const int boxes = 128 / box_rows;
      uint32_t kv_it = 0, q_it[2] = {0, 0};
      bool ok = true;
      if (lane == 0) {
        tma_prefetch_desc(&tmQ);
        if (!KV4) {
          tma_prefetch_desc(&tmK);
          tma_prefetch_desc(&tmV);
        }
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
        int page = KV4 ? -2 : box_page(w.u0);
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
        for (int j = 0; !KV4 && j < nbmax && ok; ++j) {
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
    } else if (KV4 && warp > kWarpRelay) {
      // ------------------------------------------------ widening of K and V ---
      const int row = threadIdx.x & 127;     // key of the block
      constexpr int kTiles = kKeyTiles + 1;  // of a block in the ring: keys, values
      uint32_t block = 0;
      bool ok = warp >= kWarpWiden;  // warp 11 is idle
      for (; w.left > 0 && ok; w.next(p, TT)) {
        const int nbmax = max(w.n[0], w.n[1]);
        if (nbmax == 0) continue;  // the same skip in every role
        const uint32_t page_bytes = (uint32_t)(p.page * kv4_row(D));
        // The page of the thread's key of the piece's block j: -2 past the sequence
        // or the piece.
        auto key_page = [&](int j) {
          const int key = (w.u0 + j) * 128 + row;
          return j < nbmax && key < w.sq.klen
                     ? __ldg(p.block_table + (size_t)w.b * p.max_pages + (key >> p.page_log2))
                     : -2;
        };
        // Where its row lies in the cache; -1 past the sequence and for a page outside
        // the cache, which give zeros.
        auto find = [&](int page, int j) -> int64_t {
          if (page >= 0 && page < p.n_pages)  // (n_pages Hkv is a number of 32 bits)
            return (uint64_t)(uint32_t)(page * p.Hkv + w.head) * page_bytes +
                   (uint32_t)(((w.u0 + j) * 128 + row) & (p.page - 1)) * kv4_row(D);
          if (page != -2)
            atomicCAS(p.status, 0u, 1u | (64u << 8) | ((uint32_t)min(w.b, 0xFFFF) << 16));
          return -1;
        };
        // Tile n of the block's in the ring, filled by `write`.
        auto put = [&](int n, auto write) {
          const uint32_t it = block * kTiles + n, slot = it % L::kSlots;
          ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kKvEmpty + slot),
                                                     ((it / L::kSlots) & 1) ^ 1, wd, 78));
          if (!ok) return;
          write(sbase + L::kKvOff + slot * L::kTileBytes);
          fence_proxy_async_smem();  // before the products read it
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kKvFull + slot));
        };
        // A row is asked for a block before it is widened, its page two before.
        int64_t at = find(key_page(0), 0);
        int page = key_page(1);
        Row4<D> k, v;
        k.load(at < 0 ? nullptr : p.k4 + at);
        v.load(at < 0 ? nullptr : p.v4 + at);
        for (int j = 0; j < nbmax && ok; ++j, ++block) {
          at = find(page, j + 1);
          const float2 f =
              to_fp16_range<14>(__reduce_max_sync(0xffffffffu, k.template top<BF16>()));
          put(0, [&](uint32_t tile) {
            if (lane == 0) reinterpret_cast<float*>(scales + block % L::kScales)[row >> 5] = f.y;
            k.template key_extra<BF16>(
                sbase + L::kKExtraOff + block % L::kExtras * kExtraBytes, row, f.x);
            k.template key<BF16, false>(tile, row, f.x);
          });
          if (kKeyTiles == 2 && ok)
            put(1, [&](uint32_t tile) { k.template key<BF16, true>(tile, row, f.x); });
          k.load(at < 0 ? nullptr : p.k4 + at);
          if (!ok) break;
          page = key_page(j + 2);
          put(kKeyTiles, [&](uint32_t tile) { v.template value<BF16>(tile, row); });
          v.load(at < 0 ? nullptr : p.v4 + at);
        }
      }
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
          const int full = KV4 ? L::kQReady : L::kQFull;
          aborted = !__all_sync(0xffffffffu, mbar_wait(bar(full + t), par, wd, 72));
        }
        for (int i = 0; i < kKeyTiles; ++i) kv_ready();
        aborted = named_bar_or(kBarKv, 64, aborted);
        for (int j = 0; j < nbmax; ++j) {
          const uint32_t vslot = kv_ready();
          const int valid = w.sq.klen - (w.u0 + j) * 128;  // rows of V that are keys
          if (!KV4 && valid < 128 && !aborted) {
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
          for (int i = 0; i < kKeyTiles && j + 1 < nbmax; ++i) kv_ready();
          aborted = named_bar_or(kBarKv, 64, aborted);
        }
      }
    } else if (warp == kWarpMma) {
      // ---------------------------------------------------- tcgen05 issuer ---
      constexpr uint32_t kIdS = idesc_f16(128, 128, BF16 && !KV4, false, false);
      constexpr uint32_t kIdO = idesc_f16(128, D, BF16, false, true);
      uint32_t kv_it = 0;
      bool aborted = false;
      bool issued = false;
      const uint64_t qdesc0 = kmajor_base(sbase + L::kQOff);
      const uint64_t qdesc1 = kmajor_base(sbase + L::kQOff + L::kTileBytes);
      // S_t of the block whose keys begin in ring slot kslot; its number, for the
      // columns behind.
      auto slot_addr = [&](uint32_t slot) {
        return sbase + L::kKvOff + slot % L::kSlots * L::kTileBytes;
      };
      auto issue_s = [&](int t, uint32_t kslot, uint32_t block) {
        const uint64_t qd = t ? qdesc1 : qdesc0;
        const uint32_t dcol = tbase + 128 * t;
#pragma unroll
        for (int n = 0; n < kKeyTiles; ++n) {
          const uint64_t kd = kmajor_base(slot_addr(kslot + n));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_f16_ss(dcol, desc_plus(qd, kmajor16_off(kk)), desc_plus(kd, kmajor16_off(kk)),
                       kIdS, kk > 0 || n > 0);
        }
        if constexpr (KV4)
          mma_f16_ss(dcol, extra_desc(sbase + L::kQExtraOff + t * kExtraBytes),
                     extra_desc(sbase + L::kKExtraOff + block % L::kExtras * kExtraBytes), kIdS,
                     1u);
      };
      auto free_keys = [&](uint32_t kslot) {
#pragma unroll
        for (int n = 0; n < kKeyTiles; ++n)
          mma_commit(bar(L::kKvEmpty + (kslot + n) % L::kSlots));
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
        uint32_t block = kv_it / (kKeyTiles + 1);
        kv_it += kKeyTiles;
        if (!aborted) {
          tc_fence_after();
          if (lane == 0) {
            if (nb0 > 0) {
              issue_s(0, kslot, block);
              mma_commit(bar(L::kSFull + 0));
              if (nb0 == 1) mma_commit(bar(L::kQEmpty + 0));
            }
            if (nb1 > 0) {
              issue_s(1, kslot, block);
              mma_commit(bar(L::kSFull + 1));
              if (nb1 == 1) mma_commit(bar(L::kQEmpty + 1));
            }
            free_keys(kslot);
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
            block = kv_it / (kKeyTiles + 1);
            kv_it += kKeyTiles;
          }
          const uint32_t vaddr = slot_addr(vslot);
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
                issue_s(t, kslot, block);
                mma_commit(bar(L::kSFull + t));
                if (j + 1 == nbt - 1) mma_commit(bar(L::kQEmpty + t));
              }
            }
            __syncwarp();
          }
          if (!aborted) {
            if (lane == 0) {
              mma_commit(bar(L::kKvEmpty + vslot));
              if (have_next) free_keys(kslot);
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
    }
  } else {
    // --------------------------------------------------- softmax warpgroups ---
    const int t = warp >> 2;          // query tile of the pair
    const int r = threadIdx.x & 127;  // row within the tile = TMEM lane
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_addr = tbase + lane_base + 128u * t;
    const uint32_t o_addr = tbase + lane_base + 256u + kPaddedD<D> * t;
    float sl2 = p.scale_log2;
    const int gi = r / TT, ti = r - gi * TT;  // query head of the group, token of the tile
    // The column of a word's channel i, 0 .. 7, and of channel i of 32.
    auto column = [](int i) { return KV4 ? (i & 3) * 2 + (i >> 2) : i; };
    auto at_column = [&](int i) { return (i & ~7) + column(i & 7); };
    uint32_t s_it = 0, o_it = 0, blocks = 0;  // blocks: key blocks of the pieces before
    bool aborted = false;
    for (; w.left > 0; w.next(p, TT)) {
      if (w.nothing()) continue;
      const int nb = w.n[t];
      const uint32_t block0 = blocks;
      blocks += max(w.n[0], w.n[1]);
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
      if constexpr (KV4) {
        if (!aborted)
          aborted = !__all_sync(0xffffffffu, mbar_wait(bar(L::kQFull + t), o_it & 1, wd, 79));
        if (!aborted) {
          sl2 = p.scale_log2 * query_row<D, BF16>(sbase + L::kQOff + t * L::kTileBytes,
                                                  sbase + L::kQExtraOff + t * kExtraBytes, r);
          fence_proxy_async_smem();  // before the products read it
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kQReady + t));
        }
      }
      float m = -INFINITY;  // running max of the log2-scaled scores (reference value)
      float l = 0.f;        // running sum of exp2(x - m)
      for (int j = 0; j < nb; ++j) {
        const uint32_t spar = s_it & 1;
        ++s_it;
        if (!aborted)
          aborted = !__all_sync(0xffffffffu, mbar_wait(bar(L::kSFull + t), spar, wd, 74));
        if (!aborted) {
          tc_fence_after();
          const int kbase = (w.u0 + j) * 128;
          // Scores 32 c .. of the row, those that it does not see -inf.
          constexpr int kHeld = KV4 ? 2 : 4;  // chunks of 32 in registers at a time
          // Their halves are turns of a loop where the roles' instructions do not fit their
          // cache otherwise (d = 128: the mixed batch 74 us for 84, the long chunk 443 for
          // 463; d = 96 the latter 420 for 471, but d = 64 389 for 355).
          constexpr int kTurns = D == 64 ? 2 : 1;
          uint32_t sr[kHeld][32];
          auto read_scores = [&](int c0) {
#pragma unroll
            for (int c = 0; c < kHeld; ++c) tmem_ld32(s_addr + (c0 + c) * 32, sr[c]);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < kHeld; ++c) reg_fence32(sr[c]);
            if (kbase + 127 > lim0) {
#pragma unroll
              for (int c = 0; c < kHeld; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (kbase + (c0 + c) * 32 + i > lim) sr[c][i] = 0xFF800000u;
            }
          };
          // What takes chunk c's scores to base 2: 1e-37 .. 1e37, since a masked
          // score times 0 would be NaN (a product that needs more is 0 or inf anyway).
          float to2[4] = {sl2, sl2, sl2, sl2};
          if constexpr (KV4) {
            const uint4 f = load_smem16(sbase + L::kScaleOff + (block0 + j) % L::kScales * 16);
            const uint32_t by[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int c = 0; c < 4; ++c)
              to2[c] = fminf(fmaxf(sl2 * __uint_as_float(by[c]), 1e-37f), 1e37f);
          }
          float m_blk;
          if constexpr (KV4) {
            m_blk = -INFINITY;
#pragma unroll (kTurns)
            for (int c0 = 2; c0 >= 0; c0 -= 2) {
              read_scores(c0);
              m_blk = fmaxf(m_blk, fmaxf(row_max32(sr[0]) * (c0 ? to2[2] : to2[0]),
                                         row_max32(sr[1]) * (c0 ? to2[3] : to2[1])));
            }
          } else {
            read_scores(0);
            float x[kHeld * 32];
#pragma unroll
            for (int i = 0; i < kHeld * 32; ++i) x[i] = __uint_as_float(sr[i / 32][i % 32]);
            m_blk = row_max128(x) * sl2;
          }
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
          // P goes to tensor memory in the inputs' 16 bits, what the product with
          // V takes (at most eps / 2 of sum_j P_ij |v_j|; l sums the unrounded
          // values); two 16-bit terms for P would double that product.
          // P_c lies over scores that have been read: chunks 0 and 1 over the first.
          auto exponentials = [&](int c0) {
#pragma unroll
            for (int c = 0; c < kHeld; ++c) {
              uint32_t pk[16];
              const float by = KV4 && c0 ? to2[2 + c % 2] : to2[c];
              const float2 sc2 = make_float2(by, by);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 x = __ffma2_rn(make_float2(__uint_as_float(sr[c][2 * i]),
                                                        __uint_as_float(sr[c][2 * i + 1])),
                                            sc2, nm2);
                const float p0 = ex2_approx(x.x);
                const float p1 = ex2_approx(x.y);
                rs2[i & 3] = __fadd2_rn(rs2[i & 3], make_float2(p0, p1));
                pk[i] = pack2<BF16>(p0, p1);
              }
              tmem_st16(s_addr + (c0 + c) * 16, pk);
            }
          };
          if constexpr (KV4) {
#pragma unroll (kTurns)
            for (int c0 = 0; c0 < 4; c0 += 2) {
              if (c0 > 0) read_scores(2);
              exponentials(c0);
            }
          } else {
            exponentials(0);
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
        // Rows go out through the warp's stage, so that a store covers whole row
        // pieces of 64 or 128 bytes: a lane per row would write 16 bytes of 32
        // lines.
        constexpr int kPitch = 64 * L::kStageCols;
        uint8_t* const stage = smem + L::kStageOff + warp * L::kStageBytes;
        auto place = [&](int row, int pc) {  // of a 16-byte piece, spread over the banks
          const int x = kPitch == 128 ? row & 7 : row >> 1 & 3;
          return reinterpret_cast<uint4*>(stage + row * kPitch + ((pc ^ x) << 4));
        };
#pragma unroll
        for (int c0 = 0; c0 < D / 32; c0 += L::kStageCols) {
          constexpr int kPieces = 4 * L::kStageCols;
          const int pieces = D / 32 - c0 >= L::kStageCols ? kPieces : kPieces / 2;  // of a row
#pragma unroll
          for (int c = c0; c < c0 + pieces / 4; ++c) {
            uint32_t raw[32];
            tmem_ld32_sync(o_addr + c * 32, raw);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              uint32_t pk[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                pk[i] = pack2<BF16>(__uint_as_float(raw[8 * v + column(2 * i)]) * inv_l,
                                    __uint_as_float(raw[8 * v + column(2 * i + 1)]) * inv_l);
              *place(lane, (c - c0) * 4 + v) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < pieces; ++i) {
            const int row = i * (32 / pieces) + lane / pieces, pc = lane % pieces;
            const uint4 x = *place(row, pc);
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
              part[(size_t)(c * 8 + v) * kRows + t * 128 + r] = make_uint4(
                  raw[at_column(4 * v)], raw[at_column(4 * v + 1)], raw[at_column(4 * v + 2)],
                  raw[at_column(4 * v + 3)]);
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

template <int D, bool BF16, bool KV4>
cudaError_t launch_dbk(const PagedLaunch& a) {
  using L = PagedTileLayout<D, KV4>;
  auto kern = paged_tile_kernel<D, BF16, KV4>;
  static DeviceFlags configured;
  cudaError_t e = ensure_dyn_smem(kern, L::kDynSmem, configured);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, dim3((unsigned)a.grid), kTileThreads<KV4>, L::kDynSmem, a.stream,
                          a.tmQ, a.tmK, a.tmV, a.params);
}

template <int D, bool KV4>
cudaError_t launch_dk(const PagedLaunch& a, bool bf16) {
  return bf16 ? launch_dbk<D, true, KV4>(a) : launch_dbk<D, false, KV4>(a);
}

template <bool KV4>
cudaError_t launch_k(const PagedLaunch& a, int d, bool bf16) {
  switch (d) {
    case 64: return launch_dk<64, KV4>(a, bf16);
    case 96: return launch_dk<96, KV4>(a, bf16);
    default: return launch_dk<128, KV4>(a, bf16);
  }
}

}  // namespace

cudaError_t launch_paged_tile(const PagedLaunch& a, int d, bool bf16) {
  return launch_k<false>(a, d, bf16);
}

cudaError_t launch_paged4_tile(const PagedLaunch& a, int d, bool bf16) {
  return launch_k<true>(a, d, bf16);
}

}  // namespace attn
