// New keys and values into a paged cache held in 4 bits (kv4.cuh), turned by
// their positions on the way, and rows of that cache back in 16 bits.
//
// The append reads and turns like the 16-bit one (rotary.cu): a thread owns 16
// channels of a token, as two pieces of 8, and walks up to 16 heads.  What it
// would store there is what is quantized here, so keys are rounded to 16 bits
// between the turn and the groups.  A group of 32 channels is four pieces,
// which the half-split rotation leaves with up to four threads of the token:
// each piece's minimum and maximum go to shared memory, and every thread
// takes its group's from there, two heads between two barriers.
//
// The instructions for a value hold this back from the rate of its bytes (0.66 a cycle
// and scheduler beside 0.41 of DRAM's time), with what waits between two barriers, so
// extremes are taken two values at a time in 16 bits (of 16-bit values they
// are exact), and quotients by multiplying with the group's reciprocal and a
// correction (divide).  A prompt of 16384 tokens, 16 + 8 + 8 heads of 128 in bf16: 132 us
// with __fdiv_rn, 70 with divide, 60 with two heads between barriers and six blocks an SM
// (four heads and four blocks, as in the 16-bit append, 65), 56 with one loop over them,
// whose instructions fit their cache where two buffers in turn do not, and five blocks:
// 222 MB, 4.0 TB/s, 0.60 of a copy's rate (the 16-bit append takes 44 for 296 MB).  Reading it back takes 17 us.
#include <cuda_runtime.h>
#include <cstdint>

#include "append4.cuh"
#include "dependent.cuh"
#include "kv4.cuh"
#include "packed.cuh"
#include "rotary.cuh"
#include "turn.cuh"

namespace attn {

namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 2;  // heads whose rows are read together

// The larger of two pairs of 16-bit values; NaN where one is.
template <bool BF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The extremes of eight values: -min in the low half, max in the high.
template <bool BF16>
__device__ __forceinline__ uint32_t extremes(const uint4& x) {
  constexpr uint32_t kSigns = 0x80008000u;
  const uint32_t top = max2<BF16>(max2<BF16>(x.x, x.y), max2<BF16>(x.z, x.w));
  const uint32_t low = max2<BF16>(max2<BF16>(x.x ^ kSigns, x.y ^ kSigns),
                                  max2<BF16>(x.z ^ kSigns, x.w ^ kSigns));
  return max2<BF16>(__byte_perm(low, top, 0x5410), __byte_perm(low, top, 0x7632));
}

template <bool BF16>
__device__ __forceinline__ float from16(uint32_t x) {
  return BF16 ? __uint_as_float(x << 16) : __half2float(__ushort_as_half((unsigned short)x));
}
template <bool BF16>
__device__ __forceinline__ uint32_t to16(float x) {
  return BF16 ? pack_bf16x2(x, 0.f) : pack_f16x2(x, 0.f);
}

// x / y rounded to nearest, given y's correctly rounded reciprocal: the quotient by
// multiplication, corrected by its residual (Markstein's theorem, IBM Journal of
// Research and Development 34, 1990).  Holds where nothing leaves the range of the
// normal numbers: for y in 2^-60 .. 2^60 and x / y up to 2^6, and for x = 0.
__device__ __forceinline__ float divide(float x, float y, float reciprocal) {
  const float q = x * reciprocal;
  return fmaf(fmaf(-q, y, x), reciprocal, q);
}

// Outside that range, and where there is nothing to divide by.  Not inlined, as all
// that is rare here: the instructions of the way that is taken have to fit their cache.
__device__ __noinline__ float divide_any(float x, float y) { return __fdiv_rn(x, y); }
__device__ __forceinline__ bool in_range(float y) { return y > 0x1p-60f && y < 0x1p60f; }

// s in the low half, m in the high, for extremes -min, max.
template <bool BF16>
__device__ __forceinline__ uint32_t kv4_params(uint32_t ends) {
  const uint32_t m = (ends & 0xFFFFu) ^ 0x8000u;
  const float lo = from16<BF16>(m), hi = from16<BF16>(ends >> 16);
  const float range = hi - lo;
  uint32_t s =
      to16<BF16>(in_range(range) ? divide(range, 15.f, 1.f / 15.f) : divide_any(range, 15.f));
  constexpr uint32_t kInf = BF16 ? 0x7F80u : 0x7C00u;
  if (s >= kInf) return 0x7FFF7FFFu;
  // s rounded up may carry code 15 past the type's range
  if (to16<BF16>(fmaf(15.f, from16<BF16>(s), lo)) == kInf) --s;
  return s | m << 16;
}

// The bits of 1.5 2^23 at every fourth place, modulo 2^32: what they add up to below.
constexpr uint32_t magic_sum() {
  uint32_t w = 0;
  for (int i = 0; i < 8; ++i) w += 0x4B400000u << (4 * i);
  return w;
}

template <bool BF16>
__device__ __noinline__ uint32_t quantize8_any(uint4 x, float m, float s) {
  float v[8];
  unpack8<BF16>(x, v);
  uint32_t w = 0;
  const float by = s > 0.f ? s : INFINITY;  // one value: code 0
  for (int i = 7; i >= 0; --i) w = w << 4 | (uint32_t)fminf(rintf(__fdiv_rn(v[i] - m, by)), 15.f);
  return w;
}

// The code word of eight values.
template <bool BF16>
__device__ __forceinline__ uint32_t quantize8(const uint4& x, uint32_t par) {
  const float m = from16<BF16>(par >> 16), s = from16<BF16>(par & 0xFFFFu);
  // (of a normal number s no quotient passes 15.2, so that none has to be cut to 15)
  if (!in_range(s) || (!BF16 && s < 0x1p-14f)) return quantize8_any<BF16>(x, m, s);
  constexpr uint32_t kMagic = magic_sum();
  const float reciprocal = __frcp_rn(s);
  float v[8];
  unpack8<BF16>(x, v);
  uint32_t w = 0;
  // q + 1.5 2^23 has the nearest whole number in its low bits
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = divide(v[i] - m, s, reciprocal);
    w += __float_as_uint(q + 0x1.8p23f) << (4 * i);
  }
  return w - kMagic;
}

template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kThreads, 5) append4_kernel(const AppendParams p) {
  __shared__ __align__(16) uint32_t ends[2][kBatch][2 * kThreads];  // of each token's pieces
  grid_wait();
  grid_release();
  if (blockIdx.x >= p.token_blocks) {  // as in the 16-bit append
    const int64_t b = (int64_t)(blockIdx.x - p.token_blocks) * kThreads + threadIdx.x;
    if (b < p.batch.n_seq) packed_check(p.batch, b);
    return;
  }
  // A token's threads lie in one block; the threads left over, and those of
  // tokens that are not stored, walk along to the barriers.
  const int per_row = p.d / 16, tokens = kThreads / per_row;
  const int group = blockIdx.x % p.head_groups;
  const int own = threadIdx.x / per_row, c = threadIdx.x % per_row;
  const int64_t t64 = (int64_t)(blockIdx.x / p.head_groups) * tokens + own;
  const bool token = own < tokens && t64 < p.batch.total;
  const int t = token ? (int)t64 : 0;
  const Pieces s = pieces<INTER>(c, p.rot);
  // heads in the order k, v, q
  const int h0 = group * p.group_heads;
  const int count = min(p.group_heads, 2 * p.Hkv + p.Hq - h0);
  auto which = [&](int h) { return h < p.Hkv ? 0 : (h < 2 * p.Hkv ? 1 : 2); };
  uint4 lo[2][kBatch], hi[2][kBatch];
  auto load = [&](uint4 (&l)[kBatch], uint4 (&h)[kBatch], int at) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (at + i >= count || !token) break;
      const int w = which(h0 + at + i);
      const uint16_t* x = static_cast<const uint16_t*>(p.src[w]) +
                          (h0 + at + i - w * p.Hkv) * p.sh[w] + (int64_t)t * p.sn[w];
      l[i] = *reinterpret_cast<const uint4*>(x + s.lo);
      h[i] = *reinterpret_cast<const uint4*>(x + s.hi);
    }
  };
  load(lo[0], hi[0], 0);

  PackedPlace at = {p.batch.n_seq, false, false, 0, -1};
  if (token) {
    at.b = packed_seq(p.batch, t);
    if (at.b < p.batch.n_seq) at = packed_place(p.batch, at.b, t);
  }
  if (at.b < p.batch.n_seq && !at.stored && c == 0 && group == 0)
    report_bad(p.batch.status, at.in_seq ? kBadPage : kBadBatch, at.b);

  float cs[8], sn[8];
  if (s.turn && at.in_seq) {
    angles(p.table, p.rot / 2, c,
           [&](int axis) {
             return p.positions == nullptr
                        ? (int)at.pos
                        : __ldg(p.positions +
                                (int64_t)min(max(axis, 0), p.n_axes - 1) * p.batch.total + t);
           },
           cs, sn);
  }
  const int page_row = (int)at.pos & ((1 << p.batch.page_log2) - 1);
  const int row_bytes = kv4_row(p.d);
  const int base = own * 2 * per_row;  // of the token's pieces in ends: a multiple of 4
  auto store = [&](uint4 (&l)[kBatch], uint4 (&hh)[kBatch], int first, int buf) {
    if (first >= count) return;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (first + i >= count || !at.in_seq) break;
      const int w = which(h0 + first + i);
      const int h = h0 + first + i - w * p.Hkv;
      if (s.turn && w != 1) turn_pieces<BF16, INTER>(l[i], hh[i], cs, sn);
      if (w == 2) {
        uint16_t* y = static_cast<uint16_t*>(p.q_out) + ((int64_t)h * p.batch.total + t) * p.d;
        *reinterpret_cast<uint4*>(y + s.lo) = l[i];
        *reinterpret_cast<uint4*>(y + s.hi) = hh[i];
        continue;
      }
      ends[buf][i][base + s.lo / 8] = extremes<BF16>(l[i]);
      ends[buf][i][base + s.hi / 8] = extremes<BF16>(hh[i]);
    }
    if (h0 + first >= 2 * p.Hkv) return;  // queries alone
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (first + i >= count || !at.stored) break;
      const int w = which(h0 + first + i);
      if (w == 2) break;
      const int h = h0 + first + i - w * p.Hkv;
      uint8_t* y =
          static_cast<uint8_t*>(w ? p.v_pages : p.k_pages) +
          ((((int64_t)at.page * p.Hkv + h) << p.batch.page_log2) + page_row) * row_bytes;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int ch = half ? s.hi : s.lo;
        const uint4 r = *reinterpret_cast<const uint4*>(
            &ends[buf][i][base + ch / kKv4Group * 4]);
        const uint32_t par =
            kv4_params<BF16>(max2<BF16>(max2<BF16>(r.x, r.y), max2<BF16>(r.z, r.w)));
        *reinterpret_cast<uint32_t*>(y + ch / 2) = quantize8<BF16>(half ? hh[i] : l[i], par);
        if (ch % kKv4Group == 0)
          *reinterpret_cast<uint32_t*>(y + p.d / 2 + ch / kKv4Group * 4) = par;
      }
    }
  };
  // The next heads are on their way while these are stored.  The barrier of a batch also
  // says that the one before last has been read.
#pragma unroll 1
  for (int first = 0; first < count; first += kBatch) {
    load(lo[1], hi[1], first + kBatch);
    store(lo[0], hi[0], first, first / kBatch & 1);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      lo[0][i] = lo[1][i];
      hi[0][i] = hi[1][i];
    }
  }
}

// A thread owns a code word (8 channels) of a token and walks its heads.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) read4_kernel(const Read4Params p) {
  grid_wait();
  grid_release();
  if (blockIdx.x >= p.token_blocks) {
    const int64_t b = (int64_t)(blockIdx.x - p.token_blocks) * kThreads + threadIdx.x;
    if (b < p.batch.n_seq) packed_check(p.batch, b);
    return;
  }
  const int words = p.d / 8;
  const int group = blockIdx.x % p.head_groups;
  const int64_t idx = (int64_t)(blockIdx.x / p.head_groups) * kThreads + threadIdx.x;
  const int64_t t64 = idx / words;
  if (t64 >= p.batch.total) return;
  const int t = (int)t64, c = (int)(idx % words);
  const int b = packed_seq(p.batch, t);
  if (b == p.batch.n_seq) return;
  const PackedPlace at = packed_place(p.batch, b, t);
  if (!at.stored) {
    if (c == 0 && group == 0)
      report_bad(p.batch.status, at.in_seq ? kBadPage : kBadBatch, at.b);
    return;
  }
  const int page_row = (int)at.pos & ((1 << p.batch.page_log2) - 1);
  const int row_bytes = kv4_row(p.d);
  const int h0 = group * p.group_heads, h1 = min(h0 + p.group_heads, 2 * p.Hkv);
#pragma unroll 4
  for (int i = h0; i < h1; ++i) {  // heads in the order k, v
    const int w = i >= p.Hkv, h = i - w * p.Hkv;
    const uint8_t* x = (w ? p.v_pages : p.k_pages) +
                       ((((int64_t)at.page * p.Hkv + h) << p.batch.page_log2) + page_row) * row_bytes;
    const uint32_t code = __ldg(reinterpret_cast<const uint32_t*>(x) + c);
    const uint32_t par = __ldg(reinterpret_cast<const uint32_t*>(x + p.d / 2) + c / 4);
    uint16_t* y = static_cast<uint16_t*>(w ? p.v : p.k) + ((int64_t)h * p.batch.total + t) * p.d;
    reinterpret_cast<uint4*>(y)[c] = kv4_word<BF16>(code, par);
  }
}

}  // namespace

cudaError_t launch_append4(const AppendLaunch& a, int num_sms) {
  AppendParams p = a.params;
  const int heads = 2 * p.Hkv + p.Hq, tokens = kThreads / (p.d / 16);
  const int64_t bx = ((int64_t)p.batch.total + tokens - 1) / tokens;
  p.group_heads = heads_per_block(bx, heads, num_sms);
  p.head_groups = (heads + p.group_heads - 1) / p.group_heads;
  p.token_blocks = (unsigned)(bx * p.head_groups);
  const dim3 grid(p.token_blocks + ((unsigned)p.batch.n_seq + kThreads - 1) / kThreads);
  auto kern = a.bf16 ? (a.interleaved ? append4_kernel<true, true> : append4_kernel<true, false>)
                     : (a.interleaved ? append4_kernel<false, true> : append4_kernel<false, false>);
  return launch_dependent(kern, grid, kThreads, 0, a.stream, p);
}

cudaError_t launch_read4(const Read4Launch& a, int num_sms) {
  Read4Params p = a.params;
  const int64_t bx = ((int64_t)p.batch.total * (p.d / 8) + kThreads - 1) / kThreads;
  p.group_heads = heads_per_block(bx, 2 * p.Hkv, num_sms);
  p.head_groups = (2 * p.Hkv + p.group_heads - 1) / p.group_heads;
  p.token_blocks = (unsigned)(bx * p.head_groups);
  const dim3 grid(p.token_blocks + ((unsigned)p.batch.n_seq + kThreads - 1) / kThreads);
  return launch_dependent(a.bf16 ? read4_kernel<true> : read4_kernel<false>, grid, kThreads, 0,
                          a.stream, p);
}

}  // namespace attn
