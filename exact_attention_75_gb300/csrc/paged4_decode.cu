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
// A group's product is taken with c - 8, and s and m + 8 s of its keys are applied to
// it and to the sum of the query's channels in 32 bits: keys lose nothing.
// P leaves the softmax by keys and is wanted by rows: one 8 x 8 transpose for 8
// keys.
//
// The running maximum is a reference that is raised only where a score passes
// it by 2^8 (P stays below that), so that most blocks need no maximum across lanes.
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

// N 32-bit words from shared memory.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* x, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(x);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(x);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint32_t*>(x)[i];
  }
}

// The codes of 4 C channels of two keys (a: the first's, b: the second's), the
// first key's in the low halves.
template <int C>
__device__ __forceinline__ void load_pairs(const uint8_t* a, const uint8_t* b, uint32_t (&w)[C]) {
  if constexpr (C == 3) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      w[c] = (uint32_t)reinterpret_cast<const uint16_t*>(a)[c] |
             (uint32_t)reinterpret_cast<const uint16_t*>(b)[c] << 16;
  } else {
    uint32_t x[C / 2], y[C / 2];
    if constexpr (C == 4) {
      load_words<2>(a, x);
      load_words<2>(b, y);
    } else {
      x[0] = *reinterpret_cast<const uint32_t*>(a);
      y[0] = *reinterpret_cast<const uint32_t*>(b);
    }
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
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                             ~static_cast<uintptr_t>(127));
  const uint32_t sbase = smem_u32(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kFlagOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  const float raise_by = kRaise / p.scale_log2;
  uint8_t* const ring = smem + warp * NS * L::kSlotBytes;
  const uint32_t ring_addr = smem_u32(ring);

  // Block n of the warp's stream lies in slot n % NS; the ring is full until the
  // stream ends, so the slot that is read is the one that is filled next.
  BlockStream<W, kKeys> stream(p, w, warp, lane);
  uint32_t it = 0;         // blocks taken from the ring
  int slot = 0;            // it % NS
  uint32_t parity = 0;     // (it / NS) & 1
  auto issue = [&](int s) {
    if (!stream.more()) return;
    // Lanes 0 to 3 copy a unit of K or V each, of a page outside the cache (reported)
    // any one; what the second unit of a block past the sequence has is not read
    // but as numbers that count nothing.
    const int page0 = stream.page(p, 0, lane), page1 = stream.page(p, 1, lane);
    const int pages = page1 == -2 ? 1 : 2;
    if (lane == 0) mbar_arrive_expect_tx(bar(s), (uint32_t)(2 * pages * L::kUnitBytes));
    __syncwarp();
    const int u = lane & 1;
    if (lane < 4 && u < pages) {
      const size_t row = (((size_t)max(u ? page1 : page0, 0) * p.Hkv + stream.ahead.head)
                          << p.page_log2) + stream.row(p, u, warp);
      bulk_load(ring_addr + (uint32_t)(s * L::kSlotBytes + lane * L::kUnitBytes),
                (lane < 2 ? p.k4 : p.v4) + row * L::kRow, L::kUnitBytes, bar(s));
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
    // Q^T: of row 8 nt + g the channels that the lane has of the keys; and the
    // sums over each group of rows 8 nt + 2 t and the next.
    uint32_t qb[NT][KS][2];
    float qsum[NT][C][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + g;
      const uint16_t* q =
          static_cast<const uint16_t*>(p.q) + (r < rows ? row_of(p, w, r) * D + 8 * t : 0);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) x = *reinterpret_cast<const uint4*>(q + 32 * c);
        qb[nt][2 * c][0] = __byte_perm(x.x, x.z, 0x5410);
        qb[nt][2 * c][1] = __byte_perm(x.x, x.z, 0x7632);
        qb[nt][2 * c + 1][0] = __byte_perm(x.y, x.w, 0x5410);
        qb[nt][2 * c + 1][1] = __byte_perm(x.y, x.w, 0x7632);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack2<BF16>(reinterpret_cast<const uint32_t*>(&x)[i]);
          sum += f.x + f.y;
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        qsum[nt][c][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
        qsum[nt][c][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
      }
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
    float m[NT][2], ref[NT][2], limit[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < KS; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      m[nt][0] = m[nt][1] = limit[nt][0] = limit[nt][1] = -INFINITY;
      ref[nt][0] = ref[nt][1] = 0.f;
      l[nt][0] = l[nt][1] = 0.f;
    }
    bool aborted = false;
#pragma unroll 1
    for (int j = 0; j < nbw; ++j) {
      if (!__all_sync(0xffffffffu, mbar_wait(bar(slot), parity, wd, 76))) {
        aborted = true;
        break;
      }
      ++it;
      const uint8_t* const block = ring + slot * L::kSlotBytes;
      const int key0 = first_key(w, warp, j);

      // S^T: x[nt][4 u + e] is row 8 nt + 2 t + e % 2, key key0 + 16 u + g + 8 (e / 2).
      float x[NT][8];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[nt][e] = 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t kw[2][C], kp[2][C];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* row = block + u * L::kUnitBytes + (g + 8 * h) * L::kRow;
#pragma unroll
          for (int c = 0; c < C; ++c) kw[h][c] = reinterpret_cast<const uint32_t*>(row)[4 * c + t];
          load_words<C>(row + D / 2, kp[h]);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          uint32_t v[2][4];
          float2 par[2];  // s, m + 8 s
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            par[h] = unpack2<BF16>(kp[h][c]);
            par[h].y = fmaf(8.f, par[h].x, par[h].y);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[h][i] = kv4_codes<BF16, 8>(kw[h][c] >> (4 * i));
          }
          const uint32_t a0[4] = {v[0][0], v[1][0], v[0][1], v[1][1]};
          const uint32_t a1[4] = {v[0][2], v[1][2], v[0][3], v[1][3]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float y[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816<BF16>(y, a0, qb[nt][2 * c][0], qb[nt][2 * c][1]);
            mma16816<BF16>(y, a1, qb[nt][2 * c + 1][0], qb[nt][2 * c + 1][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[nt][4 * u + e] = fmaf(par[e >> 1].y, qsum[nt][c][e & 1],
                                      fmaf(par[e >> 1].x, y[e], x[nt][4 * u + e]));
          }
        }
      }

      // Online softmax.
      if (key0 + kKeys - 1 > lim0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (key0 + g + 8 * (e >> 1) > lim[nt][e & 1]) x[nt][e] = -INFINITY;
      }
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 8; ++e) raise |= x[nt][e] > limit[nt][e & 1];
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float b = fmaxf(fmaxf(x[nt][e], x[nt][e + 2]), fmaxf(x[nt][e + 4], x[nt][e + 6]));
            b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 4));
            b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 8));
            b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 16));
            // (by the row's own scores alone: no row's bits depend on another's)
            if (!(b > limit[nt][e])) continue;
            const float n = b * p.scale_log2;
            const float alpha = ex2_approx(m[nt][e] - n);
            m[nt][e] = ref[nt][e] = n;
            limit[nt][e] = b + raise_by;
            l[nt][e] *= alpha;
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
        for (int e = 0; e < 8; ++e) {
          x[nt][e] = ex2_approx(fmaf(x[nt][e], p.scale_log2, -ref[nt][e & 1]));
          l[nt][e & 1] += x[nt][e];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          pb[nt][i] = transpose8(pack2<BF16>(x[nt][2 * i], x[nt][2 * i + 1]));
      }

      // O^T += V^T P^T.
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t vw[2][C], vp[2][2][kSplit ? C : 1];  // keys 2 t, 2 t + 1 and those 8 behind
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t* a = block + (2 + u) * L::kUnitBytes + (2 * t + 8 * h) * L::kRow;
          load_pairs<C>(a + g * (D / 16), a + L::kRow + g * (D / 16), vw[h]);
#pragma unroll
          for (int c = 0; c < (kSplit ? C : 1); ++c) {
            const int group = (C * g + c) / 8;
            uint32_t p0 = reinterpret_cast<const uint32_t*>(a + D / 2)[group];
            uint32_t p1 = reinterpret_cast<const uint32_t*>(a + L::kRow + D / 2)[group];
            if (key0 + kKeys > sq.klen) {
              // Rows past the sequence's last key hold whatever the page, or the slot,
              // held (P is 0 there, but 0 x NaN is not): they stand for 0.
              const int key = key0 + 16 * u + 2 * t + 8 * h;
              if (key >= sq.klen) p0 = 0u;
              if (key + 1 >= sq.klen) p1 = 0u;
            }
            vp[h][0][c] = __byte_perm(p0, p1, 0x5410);
            vp[h][1][c] = __byte_perm(p0, p1, 0x7632);
          }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
          uint32_t v[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              v[h][i] = kv4_values<BF16>(vw[h][c] >> (4 * i), vp[h][0][kSplit ? c : 0],
                                         vp[h][1][kSplit ? c : 0]);
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
      if (lane < 4) fence_proxy_async_smem();  // the lanes that copy
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
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
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
          if (g == 0) meet_ml[mr] = make_float2(m[nt][e], l[nt][e]);
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
  return launch_clusters(kern, CLUSTER ? a.params.cluster : 1, dim3((unsigned)a.grid), kWarps<NT> * 32,
                         L::kBytes, a.stream, a.params);
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
