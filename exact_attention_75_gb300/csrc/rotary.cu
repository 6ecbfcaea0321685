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
// One thread owns 16 channels (8 pairs) of one token and walks group_heads
// heads with the cosines and sines in registers: per head two 16-byte reads
// and two 16-byte writes.  The kernels are bound by those HBM bytes.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "attn.h"
#include "rotary.cuh"
#include "sm103_ptx.cuh"

namespace attn {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // heads whose rows are read together
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
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t step = (uint64_t)__ldg(table + 8 * c + i);
    const int axis = (int)__ldg(table + half + 8 * c + i);
    const uint64_t turn = step * (uint64_t)(int64_t)position_of(axis);
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &sn[i], &cs[i]);
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
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  const int per_row = p.d / 16;
  const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int n = (int)(idx / per_row), c = (int)(idx % per_row);
  if (n >= p.N) return;
  const int b = blockIdx.z;
  const Pieces s = pieces<INTER>(c, p.rot);
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
  const int h0 = blockIdx.y * p.group_heads;
  const int h1 = min(h0 + p.group_heads, p.heads[0] + p.heads[1]);
  for (int h = h0; h < h1; h += kBatch) {
    uint4 lo[kBatch], hi[kBatch];
    uint16_t* yr[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (h + i >= h1) break;
      const int w = h + i >= p.heads[0];
      const int hh = h + i - (w ? p.heads[0] : 0);
      const RopeTensor x = w ? p.x[1] : p.x[0], y = w ? p.y[1] : p.y[0];
      const uint16_t* xr = static_cast<const uint16_t*>(x.p) + b * x.sb + hh * x.sh + n * x.sn;
      yr[i] = static_cast<uint16_t*>(y.p) + b * y.sb + hh * y.sh + n * y.sn;
      lo[i] = *reinterpret_cast<const uint4*>(xr + s.lo);
      hi[i] = *reinterpret_cast<const uint4*>(xr + s.hi);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (h + i >= h1) break;
      if (s.turn) turn_pieces<BF16, INTER>(lo[i], hi[i], cs, sn);
      *reinterpret_cast<uint4*>(yr[i] + s.lo) = lo[i];
      *reinterpret_cast<uint4*>(yr[i] + s.hi) = hi[i];
    }
  }
}

__device__ __forceinline__ void report_bad(uint32_t* status, int site, int index) {
  atomicCAS(status, 0u, (uint32_t)ATTN_ERR_INVALID_ARG | ((uint32_t)site << 8) |
                            ((uint32_t)min(index, 0xFFFF) << 16));
}

template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
  const int per_row = p.d / 16;
  const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int t = (int)(idx / per_row), c = (int)(idx % per_row);
  if (t >= p.total) return;
  // The token's sequence: the last b with cu[b] <= t.  Tokens before the
  // first or behind the last sequence are padding: nothing of theirs is
  // written.  The offsets need not be valid for the search to end in range.
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
  const int64_t page_at = pos64 / p.page;
  int page = -1;
  if (in_seq && pos64 >= 0 && page_at < p.max_pages)
    page = __ldg(p.block_table + (int64_t)b * p.max_pages + page_at);
  const bool stored = page >= 0 && page < p.n_pages;
  if (!stored && c == 0 && blockIdx.y == 0)
    report_bad(p.status, in_seq ? kBadPage : kBadBatch, b);
  if (!in_seq) return;

  const Pieces s = pieces<INTER>(c, p.rot);
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
  const int h0 = blockIdx.y * p.group_heads;
  const int h1 = min(h0 + p.group_heads, 2 * p.Hkv + p.Hq);
  for (int h = h0; h < h1; h += kBatch) {
    uint4 lo[kBatch], hi[kBatch];
    uint16_t* yr[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      // heads in the order k, v, q
      const int w = h + i < p.Hkv ? 0 : (h + i < 2 * p.Hkv ? 1 : 2);
      const int hh = h + i - w * p.Hkv;
      yr[i] = nullptr;
      if (h + i >= h1 || (w < 2 && !stored)) continue;
      const uint16_t* xr =
          static_cast<const uint16_t*>(p.src[w]) + hh * p.sh[w] + (int64_t)t * p.sn[w];
      if (w == 2)
        yr[i] = static_cast<uint16_t*>(p.q_out) + ((int64_t)hh * p.total + t) * p.d;
      else
        yr[i] = static_cast<uint16_t*>(w ? p.v_pages : p.k_pages) +
                (((int64_t)page * p.Hkv + hh) * p.page + (int)(pos64 % p.page)) * p.d;
      lo[i] = *reinterpret_cast<const uint4*>(xr + s.lo);
      hi[i] = *reinterpret_cast<const uint4*>(xr + s.hi);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (yr[i] == nullptr) continue;
      const bool is_v = h + i >= p.Hkv && h + i < 2 * p.Hkv;
      if (s.turn && !is_v) turn_pieces<BF16, INTER>(lo[i], hi[i], cs, sn);
      *reinterpret_cast<uint4*>(yr[i] + s.lo) = lo[i];
      *reinterpret_cast<uint4*>(yr[i] + s.hi) = hi[i];
    }
  }
}

// Heads per block: as many as leave every SM its blocks (the angles are
// computed once per block and token), at most 8.
int heads_per_block(int64_t blocks_x, int heads, int num_sms) {
  int g = 8;
  while (g > 1 && blocks_x * ((heads + g - 1) / g) < 4LL * num_sms) g >>= 1;
  return g;
}

}  // namespace

cudaError_t launch_rope(const RopeLaunch& a, int num_sms) {
  RopeParams p = a.params;
  const int heads = p.heads[0] + p.heads[1];
  const int64_t bx = ((int64_t)p.N * (p.d / 16) + kThreads - 1) / kThreads;
  p.group_heads = heads_per_block(bx * a.B, heads, num_sms);
  const dim3 grid((unsigned)bx, (unsigned)((heads + p.group_heads - 1) / p.group_heads),
                  (unsigned)a.B);
  if (a.bf16) {
    if (a.interleaved) rope_kernel<true, true><<<grid, kThreads, 0, a.stream>>>(p);
    else rope_kernel<true, false><<<grid, kThreads, 0, a.stream>>>(p);
  } else {
    if (a.interleaved) rope_kernel<false, true><<<grid, kThreads, 0, a.stream>>>(p);
    else rope_kernel<false, false><<<grid, kThreads, 0, a.stream>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_append(const AppendLaunch& a, int num_sms) {
  AppendParams p = a.params;
  const int heads = 2 * p.Hkv + p.Hq;
  const int64_t bx = ((int64_t)p.total * (p.d / 16) + kThreads - 1) / kThreads;
  p.group_heads = heads_per_block(bx, heads, num_sms);
  const dim3 grid((unsigned)bx, (unsigned)((heads + p.group_heads - 1) / p.group_heads));
  if (a.bf16) {
    if (a.interleaved) append_kernel<true, true><<<grid, kThreads, 0, a.stream>>>(p);
    else append_kernel<true, false><<<grid, kThreads, 0, a.stream>>>(p);
  } else {
    if (a.interleaved) append_kernel<false, true><<<grid, kThreads, 0, a.stream>>>(p);
    else append_kernel<false, false><<<grid, kThreads, 0, a.stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace attn
