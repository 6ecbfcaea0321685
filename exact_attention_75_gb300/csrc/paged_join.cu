// Joins the partial results of paged attention items whose keys several CTAs
// shared.  Per row, over the item's parts in key order,
//   M = max m_k,  l = sum l_k 2^(m_k - M),  O = sum O_k 2^(m_k - M) / l.
//
// A warp takes a segment of 32 (row, four columns) elements, contiguous in
// every part (512 bytes a read), four parts in flight at a time.  The
// decoding kernel's items are small and may be spread over every CTA (one
// sequence with a long cache), so four warps share the parts of a segment and
// meet in shared memory; a pair of query tiles has enough segments.  Launched
// as a programmatic dependent of the kernel that wrote the parts.
#include <cuda_runtime.h>
#include <cstdint>

#include "mma16.cuh"
#include "paged.cuh"
#include "sm103_ptx.cuh"
#include "smem_attr.cuh"

namespace attn {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kFlight = 4;  // parts read together

struct Sum {
  float m, l;
  float4 o;
};

__device__ __forceinline__ void add(Sum& s, float m, float l, const float4& o) {
  const float M = fmaxf(s.m, m);
  const float ref = M == -INFINITY ? 0.f : M;
  const float f = exp2f(s.m - ref), g = exp2f(m - ref);
  s.m = M;
  s.l = s.l * f + l * g;
  s.o.x = s.o.x * f + o.x * g;
  s.o.y = s.o.y * f + o.y * g;
  s.o.z = s.o.z * f + o.z * g;
  s.o.w = s.o.w * f + o.w * g;
}

// ROWS: rows of an item's partial result (kPagedRows: the decoding kernel;
// kPagedTileRows: a pair of query tiles).
template <int D, bool BF16, int ROWS>
__global__ void __launch_bounds__(kThreads, 4) paged_join_kernel(const PagedParams p) {
  constexpr bool kDecode = ROWS == kPagedRows;
  constexpr int kWays = kDecode ? 4 : 1;  // warps that share a segment's parts
  constexpr int kSegs = ROWS * (D / 4) / 32;
  __shared__ Sum meet[kDecode ? kThreads : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int way = warp % kWays;
  grid_wait();
  grid_release();
  const int4 item = p.desc[2 * blockIdx.x], seq = p.desc[2 * blockIdx.x + 1];
  const int parts = item.x;
  if (parts == 0) return;
  // decoding: the grid covers the live segments in one round
  const int segs = kDecode ? (int)gridDim.y * (kWarps / kWays) : kSegs;
  for (int s0 = blockIdx.y * (kWarps / kWays); s0 < segs; s0 += gridDim.y * (kWarps / kWays)) {
    const int seg = s0 + warp / kWays;
    const int e = min(seg, kSegs - 1) * 32 + lane;
    int r, c4, token, head;  // row of the item, columns; token of the sequence, head of the group
    if constexpr (kDecode) {
      r = e / (D / 4);
      c4 = e % (D / 4);
      token = r / p.G;
      head = r - token * p.G;
    } else {
      r = e % ROWS;
      c4 = e / ROWS;
      const int TT = 128 / p.G;
      head = (r & 127) / TT;
      token = item.z + (r >> 7) * TT + (r & 127) - head * TT;
    }
    const bool live = seg < kSegs && head < p.G && token < seq.y;
    Sum s = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int k0 = way * kFlight; live && k0 < parts; k0 += kWays * kFlight) {
      float2 ml[kFlight];
      float4 o[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        if (k0 + i >= parts) break;
        const int k = k0 + i;
        const size_t slot = 2 * ((size_t)blockIdx.x + k) + (k == 0 ? 1 : 0);
        ml[i] = *reinterpret_cast<const float2*>(p.part_ml + (slot * ROWS + r) * 2);
        o[i] = *reinterpret_cast<const float4*>(p.part_o + slot * ROWS * D + (size_t)e * 4);
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        if (k0 + i >= parts) break;
        // a part with no key for the row holds no O
        if (ml[i].x != -INFINITY) add(s, ml[i].x, ml[i].y, o[i]);
      }
    }
    if constexpr (kDecode) {
      if (parts > kFlight) {  // the other warps have some
        meet[threadIdx.x] = s;
        __syncthreads();
        if (way == 0) {
#pragma unroll
          for (int w = 1; w < kWays; ++w) {
            const Sum& x = meet[threadIdx.x + 32 * w];
            add(s, x.m, x.l, x.o);
          }
        }
        __syncthreads();
      }
      if (way != 0) continue;
    }
    if (!live) continue;
    const size_t gr = (size_t)(item.y * p.G + head) * p.total + seq.x + token;
    const float inv = s.l > 0.f ? 1.f / s.l : 0.f;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + gr * D + 4 * c4) = make_uint2(
        pack2<BF16>(s.o.x * inv, s.o.y * inv), pack2<BF16>(s.o.z * inv, s.o.w * inv));
    if (c4 == 0) p.lse[gr] = s.l > 0.f ? (s.m + log2f(s.l)) * 0.69314718055994531f : -INFINITY;
  }
}

template <int D, bool BF16, int ROWS>
cudaError_t launch_dbr(const PagedLaunch& a) {
  // decoding: every live segment at once, kWarps / 4 in a CTA; tiles: two
  // rounds of kWarps segments per CTA
  const unsigned y = ROWS == kPagedRows ? (unsigned)(a.rows * (D / 4) + 63) / 64 : D / 8;
  return launch_dependent(paged_join_kernel<D, BF16, ROWS>, dim3((unsigned)a.grid, y), kThreads, 0,
                          a.stream, a.params);
}

template <int D>
cudaError_t launch_d(const PagedLaunch& a, bool bf16, bool decode) {
  if (decode)
    return bf16 ? launch_dbr<D, true, kPagedRows>(a) : launch_dbr<D, false, kPagedRows>(a);
  return bf16 ? launch_dbr<D, true, kPagedTileRows>(a) : launch_dbr<D, false, kPagedTileRows>(a);
}

}  // namespace

cudaError_t launch_paged_join(const PagedLaunch& a, int d, bool bf16, bool decode) {
  switch (d) {
    case 64: return launch_d<64>(a, bf16, decode);
    case 96: return launch_d<96>(a, bf16, decode);
    default: return launch_d<128>(a, bf16, decode);
  }
}

}  // namespace attn
