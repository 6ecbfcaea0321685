// Rotary positions with one or several axes, and the append of new keys and
// values to a paged cache with the rotation on the way.
//
// Channel pair p of a row at position (pos_0, pos_1, ...) turns by the angle
// a_p = pos[axis_p] f_p:
//   y_a = x_a cos a_p - x_b sin a_p,   y_b = x_b cos a_p + x_a sin a_p
// with (a, b) = (p, p + rot/2), or (2p, 2p + 1) interleaved; channels past
// rot pass through.  The turn is orthogonal, so the backward pass is the same
// kernel with the angle's sign flipped.
//
// Angles are held in turns as 64-bit fixed point: the table's step times the
// position, modulo 2^64, is the fraction of a turn exactly (the product wraps
// where whole turns drop out), so a far position costs no accuracy and no
// argument reduction; its upper 32 bits become the fp32 argument of sincospi.
//
// One thread owns 16 channels (8 pairs) of one token and walks up to 16 heads
// with the cosines and sines in registers: per head two 16-byte reads and two
// 16-byte writes.  The kernels are bound by those HBM bytes, so the rows of
// the next four heads are always on their way while four are turned, and the
// first are asked for before the angles and the token's place in the cache
// are worked out.  Measured (bf16, in a graph): q and k of a fused projection,
// 2 x 8192 tokens x 32 heads, d = 128 (268 MB) 43.6 us, 6.2 TB/s, 0.91 of the
// measured copy rate; the backward of 20 heads with three axes (168 MB) 28.2 us,
// 6.0 TB/s; the append of ragged prompts (225 MB in 16-token pages, d = 64,
// three axes) 38.7 us, 5.8 TB/s, of one prompt of 16384 tokens (268 MB) 44.4 us.
// What else was tried: one batch of 8 heads per thread without the overlap
// took 45.9 us for the ragged prompts, two heads at a time 39.8, 32 heads per
// thread 41.3.  Blocks of 128 threads, head groups fastest (a projection's row
// is then read by neighbouring blocks): 256 threads with tokens fastest took
// 4.3 us against 3.3 for a 577-token image and were equal at the large sizes.
// Five blocks an SM (96 registers) against four: 28.2 / 29.6 us for that
// backward, but 27.9 / 24.9 for 32 interleaved heads of 8192 tokens and 40.6 /
// 38.7 for the ragged prompts, so the half-split rotation alone takes five.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "attn.h"
#include "dependent.cuh"
#include "rotary.cuh"
#include "sm103_ptx.cuh"
#include "smem_attr.cuh"

namespace attn {

namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 4;   // heads whose rows are read together
constexpr int kHeads = 16;  // heads a thread turns at most
constexpr int kBadBatch = 63, kBadPage = 64;  // sites in the status word

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      x[2 * i] = __uint_as_float(wd[i] << 16);
      x[2 * i + 1] = __uint_as_float(wd[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&wd[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = BF16 ? pack_bf16x2(x[2 * i], x[2 * i + 1]) : pack_f16x2(x[2 * i], x[2 * i + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Cosines and sines of pairs 8 c .. 8 c + 7; position_of(axis) gives the
// token's position on an axis.
template <typename Pos>
__device__ __forceinline__ void angles(const int64_t* table, int half, int c, Pos position_of,
                                       float (&cs)[8], float (&sn)[8]) {
  const longlong2* steps = reinterpret_cast<const longlong2*>(table + 8 * c);
  const longlong2* axes = reinterpret_cast<const longlong2*>(table + half + 8 * c);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const longlong2 step = __ldg(steps + i), axis = __ldg(axes + i);
    const uint64_t t0 = (uint64_t)step.x * (uint64_t)(int64_t)position_of((int)axis.x);
    const uint64_t t1 = (uint64_t)step.y * (uint64_t)(int64_t)position_of((int)axis.y);
    sincospif((float)(int32_t)(t0 >> 32) * 0x1p-31f, &sn[2 * i], &cs[2 * i]);
    sincospif((float)(int32_t)(t1 >> 32) * 0x1p-31f, &sn[2 * i + 1], &cs[2 * i + 1]);
  }
}

// The thread's two 16-byte pieces (element offsets of the row) and whether
// they turn: half-split rows pair piece c with piece c + rot/16, all others
// lie side by side.
struct Pieces {
  int lo, hi;
  bool turn;
};

template <bool INTER>
__device__ __forceinline__ Pieces pieces(int c, int rot) {
  Pieces s;
  s.turn = 16 * c < rot;
  const bool split = !INTER && s.turn;
  s.lo = split ? 8 * c : 16 * c;
  s.hi = split ? 8 * c + rot / 2 : 16 * c + 8;
  return s;
}

template <bool BF16, bool INTER>
__device__ __forceinline__ void turn_pieces(uint4& lo, uint4& hi, const float (&cs)[8],
                                            const float (&sn)[8]) {
  float a[8], b[8], u[8], v[8];
  unpack8<BF16>(lo, a);
  unpack8<BF16>(hi, b);
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[2 * i] = a[2 * i] * cs[i] - a[2 * i + 1] * sn[i];
      u[2 * i + 1] = a[2 * i + 1] * cs[i] + a[2 * i] * sn[i];
      v[2 * i] = b[2 * i] * cs[4 + i] - b[2 * i + 1] * sn[4 + i];
      v[2 * i + 1] = b[2 * i + 1] * cs[4 + i] + b[2 * i] * sn[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      u[i] = a[i] * cs[i] - b[i] * sn[i];
      v[i] = b[i] * cs[i] + a[i] * sn[i];
    }
  }
  lo = pack8<BF16>(u);
  hi = pack8<BF16>(v);
}

template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kThreads, INTER ? 4 : 5) rope_kernel(const RopeParams p) {
  grid_wait();
  grid_release();
  const int per_row = p.d / 16;
  const int group = blockIdx.x % p.head_groups;
  const int64_t idx = (int64_t)(blockIdx.x / p.head_groups) * kThreads + threadIdx.x;
  const int n = (int)(idx / per_row), c = (int)(idx % per_row);
  if (n >= p.N) return;
  const int b = blockIdx.z;
  const Pieces s = pieces<INTER>(c, p.rot);
  const int h0 = group * p.group_heads;
  const int count = min(p.group_heads, p.heads[0] + p.heads[1] - h0);
  auto row = [&](const RopeTensor (&t)[2], int h) {
    const int w = h >= p.heads[0];
    return static_cast<uint16_t*>(t[w].p) + b * t[w].sb + (h - (w ? p.heads[0] : 0)) * t[w].sh +
           n * t[w].sn;
  };
  uint4 lo[2][kBatch], hi[2][kBatch];
  auto load = [&](uint4 (&l)[kBatch], uint4 (&h)[kBatch], int at) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (at + i >= count) break;
      const uint16_t* x = row(p.x, h0 + at + i);
      l[i] = *reinterpret_cast<const uint4*>(x + s.lo);
      h[i] = *reinterpret_cast<const uint4*>(x + s.hi);
    }
  };
  load(lo[0], hi[0], 0);
  // the angles, while the rows are on their way
  float cs[8], sn[8];
  if (s.turn) {
    const int64_t axis_stride = (int64_t)p.pos_batches * p.N;
    const int* pos = p.positions + (p.pos_batches > 1 ? (int64_t)b * p.N : 0) + n;
    angles(p.table, p.rot / 2, c,
           [&](int axis) { return __ldg(pos + min(max(axis, 0), p.n_axes - 1) * axis_stride); },
           cs, sn);
    if (p.inverse) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sn[i] = -sn[i];
    }
  }
  auto store = [&](uint4 (&l)[kBatch], uint4 (&h)[kBatch], int at) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (at + i >= count) break;
      if (s.turn) turn_pieces<BF16, INTER>(l[i], h[i], cs, sn);
      uint16_t* y = row(p.y, h0 + at + i);
      *reinterpret_cast<uint4*>(y + s.lo) = l[i];
      *reinterpret_cast<uint4*>(y + s.hi) = h[i];
    }
  };
  for (int at = 0; at < count; at += 2 * kBatch) {
    load(lo[1], hi[1], at + kBatch);
    store(lo[0], hi[0], at);
    load(lo[0], hi[0], at + 2 * kBatch);
    store(lo[1], hi[1], at + kBatch);
  }
}

__device__ __forceinline__ void report_bad(uint32_t* status, int site, int index) {
  atomicCAS(status, 0u, (uint32_t)ATTN_ERR_INVALID_ARG | ((uint32_t)site << 8) |
                            ((uint32_t)min(index, 0xFFFF) << 16));
}

// Records sequence b as invalid if its offsets or its length are out of range.
__device__ __forceinline__ void append_check(const AppendParams& p, int64_t b) {
  const int a = __ldg(p.cu_seqlens + b), e = __ldg(p.cu_seqlens + b + 1);
  const int k = __ldg(p.kv_lens + b);
  if ((b == 0 && a != 0) || a < 0 || e < a || e > p.total || k < 0 ||
      k > (p.max_pages << p.page_log2))
    report_bad(p.status, kBadBatch, (int)b);
}

template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const AppendParams p) {
  grid_wait();
  grid_release();
  // The blocks behind the tokens' check the batch, a sequence a thread: what
  // the tokens' own places do not show (a last offset past the tokens,
  // sequences without any).  Without the check, with blocks of its own, and
  // behind the stores of a token's first thread: 64 single tokens 3.18, 3.28
  // and 3.30 us, a prompt of 16384 tokens 43.6, 43.6 and 43.9.
  if (blockIdx.x >= p.token_blocks) {
    const int64_t b = (int64_t)(blockIdx.x - p.token_blocks) * kThreads + threadIdx.x;
    if (b < p.n_seq) append_check(p, b);
    return;
  }
  const int per_row = p.d / 16;
  const int group = blockIdx.x % p.head_groups;
  const int64_t idx = (int64_t)(blockIdx.x / p.head_groups) * kThreads + threadIdx.x;
  const int t = (int)(idx / per_row), c = (int)(idx % per_row);
  if (t >= p.total) return;
  const Pieces s = pieces<INTER>(c, p.rot);
  // heads in the order k, v, q
  const int h0 = group * p.group_heads;
  const int count = min(p.group_heads, 2 * p.Hkv + p.Hq - h0);
  auto which = [&](int h) { return h < p.Hkv ? 0 : (h < 2 * p.Hkv ? 1 : 2); };
  uint4 lo[2][kBatch], hi[2][kBatch];
  auto load = [&](uint4 (&l)[kBatch], uint4 (&h)[kBatch], int at) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (at + i >= count) break;
      const int w = which(h0 + at + i);
      const uint16_t* x = static_cast<const uint16_t*>(p.src[w]) +
                          (h0 + at + i - w * p.Hkv) * p.sh[w] + (int64_t)t * p.sn[w];
      l[i] = *reinterpret_cast<const uint4*>(x + s.lo);
      h[i] = *reinterpret_cast<const uint4*>(x + s.hi);
    }
  };
  load(lo[0], hi[0], 0);

  // While the rows are on their way: the token's sequence, the last b with
  // cu[b] <= t.  Tokens before the first or behind the last sequence are
  // padding: nothing of theirs is written.  The offsets need not be valid for
  // the search to end in range.
  int lo_b = 0, hi_b = p.n_seq;
  while (lo_b < hi_b) {
    const int mid = (lo_b + hi_b + 1) >> 1;
    if (__ldg(p.cu_seqlens + mid) <= t) lo_b = mid;
    else hi_b = mid - 1;
  }
  const int b = lo_b;
  if (b == p.n_seq) return;
  const int s0 = __ldg(p.cu_seqlens + b), s1 = __ldg(p.cu_seqlens + b + 1);
  const bool in_seq = t >= s0 && t < s1;
  const int64_t pos64 = (int64_t)__ldg(p.kv_lens + b) - s1 + t;  // position in the cache
  const int64_t page_at = pos64 >> p.page_log2;
  int page = -1;
  if (in_seq && pos64 >= 0 && page_at < p.max_pages)
    page = __ldg(p.block_table + (int64_t)b * p.max_pages + page_at);
  const bool stored = page >= 0 && page < p.n_pages;
  if (!stored && c == 0 && group == 0)
    report_bad(p.status, in_seq ? kBadPage : kBadBatch, b);
  if (!in_seq) return;

  float cs[8], sn[8];
  if (s.turn) {
    angles(p.table, p.rot / 2, c,
           [&](int axis) {
             return p.positions == nullptr
                        ? (int)pos64
                        : __ldg(p.positions +
                                (int64_t)min(max(axis, 0), p.n_axes - 1) * p.total + t);
           },
           cs, sn);
  }
  const int page_row = (int)pos64 & ((1 << p.page_log2) - 1);
  auto store = [&](uint4 (&l)[kBatch], uint4 (&hh)[kBatch], int at) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (at + i >= count) break;
      const int w = which(h0 + at + i);
      if (w < 2 && !stored) continue;
      const int h = h0 + at + i - w * p.Hkv;
      if (s.turn && w != 1) turn_pieces<BF16, INTER>(l[i], hh[i], cs, sn);
      uint16_t* y =
          w == 2 ? static_cast<uint16_t*>(p.q_out) + ((int64_t)h * p.total + t) * p.d
                 : static_cast<uint16_t*>(w ? p.v_pages : p.k_pages) +
                       (((((int64_t)page * p.Hkv + h) << p.page_log2) + page_row)) * p.d;
      *reinterpret_cast<uint4*>(y + s.lo) = l[i];
      *reinterpret_cast<uint4*>(y + s.hi) = hh[i];
    }
  };
  for (int at = 0; at < count; at += 2 * kBatch) {
    load(lo[1], hi[1], at + kBatch);
    store(lo[0], hi[0], at);
    load(lo[0], hi[0], at + 2 * kBatch);
    store(lo[1], hi[1], at + kBatch);
  }
}

// Heads per thread: as many as leave every SM its blocks (the angles are
// computed once per thread), the same for every group.
int heads_per_block(int64_t blocks_x, int heads, int num_sms) {
  int g = kHeads;
  while (g > 1 && blocks_x * ((heads + g - 1) / g) < 4LL * num_sms) g >>= 1;
  const int groups = (heads + g - 1) / g;
  return (heads + groups - 1) / groups;
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& a, int num_sms) {
  RopeParams p = a.params;
  const int heads = p.heads[0] + p.heads[1];
  const int64_t bx = ((int64_t)p.N * (p.d / 16) + kThreads - 1) / kThreads;
  p.group_heads = heads_per_block(bx * a.B, heads, num_sms);
  p.head_groups = (heads + p.group_heads - 1) / p.group_heads;
  const dim3 grid((unsigned)(bx * p.head_groups), 1, (unsigned)a.B);
  if (a.bf16) {
    if (a.interleaved)
      return launch_dependent(rope_kernel<true, true>, grid, kThreads, 0, a.stream, p);
    return launch_dependent(rope_kernel<true, false>, grid, kThreads, 0, a.stream, p);
  }
  if (a.interleaved)
    return launch_dependent(rope_kernel<false, true>, grid, kThreads, 0, a.stream, p);
  return launch_dependent(rope_kernel<false, false>, grid, kThreads, 0, a.stream, p);
}

cudaError_t launch_append(const AppendLaunch& a, int num_sms) {
  AppendParams p = a.params;
  const int heads = 2 * p.Hkv + p.Hq;
  const int64_t bx = ((int64_t)p.total * (p.d / 16) + kThreads - 1) / kThreads;
  p.group_heads = heads_per_block(bx, heads, num_sms);
  p.head_groups = (heads + p.group_heads - 1) / p.group_heads;
  p.token_blocks = (unsigned)(bx * p.head_groups);
  const dim3 grid(p.token_blocks + ((unsigned)p.n_seq + kThreads - 1) / kThreads);
  if (a.bf16) {
    if (a.interleaved)
      return launch_dependent(append_kernel<true, true>, grid, kThreads, 0, a.stream, p);
    return launch_dependent(append_kernel<true, false>, grid, kThreads, 0, a.stream, p);
  }
  if (a.interleaved)
    return launch_dependent(append_kernel<false, true>, grid, kThreads, 0, a.stream, p);
  return launch_dependent(append_kernel<false, false>, grid, kThreads, 0, a.stream, p);
}

}  // namespace attn
