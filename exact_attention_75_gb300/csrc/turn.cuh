// The rotation by position as the rotary and append kernels share it: angles
// from the table, 16 channels of a row as two 16-byte pieces, and their turn.
// The formulas stand in rotary.cu.
#pragma once

#include <cuda_fp16.h>
#include <cstdint>

#include "sm103_ptx.cuh"

namespace attn {

constexpr int kTurnHeads = 16;  // heads a thread turns at most

// Heads per thread: as many as leave every SM its blocks (the angles are
// computed once per thread), the same for every group.
inline int heads_per_block(int64_t blocks_x, int heads, int num_sms) {
  int g = kTurnHeads;
  while (g > 1 && blocks_x * ((heads + g - 1) / g) < 4LL * num_sms) g >>= 1;
  const int groups = (heads + g - 1) / g;
  return (heads + groups - 1) / groups;
}

#ifdef __CUDACC__

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

#endif  // __CUDACC__

}  // namespace attn
