// Joins the partial results of paged attention items whose keys several CTAs
// shared.  Per row, over the item's parts,
//   M = max m_k,  l = sum l_k 2^(m_k - M),  O = sum O_k 2^(m_k - M) / l,
// few parts in key order, many in strided runs whose sums are then added up:
// the number of parts alone fixes the order.
//
// A warp takes a segment of 32 (row, four columns) elements, contiguous in
// every part (512 bytes a read), up to four parts in flight at a time; where
// an item has many parts (one sequence with a long cache is spread over every
// CTA), several warps share them and meet in shared memory.  Launched as a
// programmatic dependent of the kernel that wrote the parts.
#include <cuda_runtime.h>
#include <cstdint>

#include "dependent.cuh"
#include "mma16.cuh"
#include "paged.cuh"
#include "sm103_ptx.cuh"
#include "smem_attr.cuh"

namespace attn {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

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

template <int D, bool BF16>
__device__ __forceinline__ void store(const PagedParams& p, size_t row, int c4, const Sum& s) {
  const float inv = paged_inverse(s.l);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * D + 4 * c4) = make_uint2(
      pack2<BF16>(s.o.x * inv, s.o.y * inv), pack2<BF16>(s.o.z * inv, s.o.w * inv));
  if (c4 == 0) p.lse[row] = paged_lse(s.m, s.l);
}

// Adds parts k0, k0 + 1, .. (at most FLIGHT of them) of element e (row r) of
// the item that CTA first began.
template <int D, int ROWS, int FLIGHT>
__device__ __forceinline__ void add_parts(const PagedParams& p, Sum& s, int first, int e, int r,
                                          int k0, int parts) {
  float2 ml[FLIGHT];
  float4 o[FLIGHT];
#pragma unroll
  for (int i = 0; i < FLIGHT; ++i) {
    if (k0 + i >= parts) break;
    const size_t slot = 2 * (size_t)(first + k0 + i) + (k0 + i == 0 ? 1 : 0);
    ml[i] = *reinterpret_cast<const float2*>(p.part_ml + (slot * ROWS + r) * 2);
    o[i] = *reinterpret_cast<const float4*>(p.part_o + slot * ROWS * D + (size_t)e * 4);
  }
#pragma unroll
  for (int i = 0; i < FLIGHT; ++i) {
    if (k0 + i >= parts) break;
    // a part with no key for the row holds no O
    if (ml[i].y != 0.f) add(s, ml[i].x, ml[i].y, o[i]);
  }
}

// The decoding kernel's items: rows of D columns.  Up to 4 parts a warp takes
// a segment of 32 (row, four columns) elements alone, beyond that 4 warps
// share a segment's parts, beyond 16 parts 8 warps (one item of 65536 keys,
// some 76 parts: 30.8 us of kernel and join against 32.8 with 4 warps; 64 items
// of 1024 keys: 16.4 with 4, 19.4 with 8).
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 4) paged_join_rows_kernel(const PagedParams p) {
  __shared__ Sum meet[kThreads];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_wait();
  grid_release();
  const int4* d = p.desc + 2 * (2 * blockIdx.x + blockIdx.y);
  const int4 item = d[0], seq = d[1];
  const int parts = item.x;
  if (parts == 0) return;
  const int ways = parts > 16 ? 8 : (parts > 4 ? 4 : 1), segs = kWarps / ways;
  const int way = warp % ways;
  const int elements = seq.y * p.G * (D / 4);
  for (int s0 = item.y * segs; s0 * 32 < elements; s0 += parts * segs) {
    const int e = (s0 + warp / ways) * 32 + lane;
    const int r = e / (D / 4), c4 = e % (D / 4);
    const bool live = e < elements;
    Sum s = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (live)
      for (int k0 = way * 4; k0 < parts; k0 += ways * 4)
        add_parts<D, kPagedRows, 4>(p, s, blockIdx.x - item.y, e, r, k0, parts);
    if (ways > 1) {
      meet[threadIdx.x] = s;
      __syncthreads();
      if (way == 0) {
        for (int w = 1; w < ways; ++w) {
          const Sum& x = meet[threadIdx.x + 32 * w];
          add(s, x.m, x.l, x.o);
        }
      }
      __syncthreads();
    }
    const int token = r / p.G, head = r - token * p.G;  // of the sequence, of the group
    if (live && way == 0)
      store<D, BF16>(p, (size_t)(item.z * p.G + head) * p.total + seq.x + token, c4, s);
  }
}

// The few parts (at most PARTS) of a tile's row: the weights 2^(m_k - M) once,
// then COLS groups of four columns at a time, all their reads in flight
// together.
template <int D, bool BF16, int PARTS, int COLS>
__device__ __forceinline__ void join_few(const PagedParams& p, int first, int parts, int r,
                                         size_t row, int c, int step) {
  auto slot = [&](int k) { return 2 * (size_t)(first + k) + (k == 0 ? 1 : 0); };
  float2 ml[PARTS];
#pragma unroll
  for (int k = 0; k < PARTS; ++k)
    ml[k] = k < parts ? *reinterpret_cast<const float2*>(p.part_ml +
                                                         (slot(k) * kPagedTileRows + r) * 2)
                      : make_float2(-INFINITY, 0.f);
  float M = ml[0].x, l = 0.f, f[PARTS];
#pragma unroll
  for (int k = 1; k < PARTS; ++k) M = fmaxf(M, ml[k].x);
#pragma unroll
  for (int k = 0; k < PARTS; ++k) {
    f[k] = paged_weight(ml[k].x, ml[k].y, M);
    l += f[k] * ml[k].y;
  }
  const float inv = paged_inverse(l);
  if (c == 0) p.lse[row] = paged_lse(M, l);
  for (; c < D / 4; c += step) {
    float4 x[COLS][PARTS];
#pragma unroll
    for (int h = 0; h < COLS; ++h)
#pragma unroll
      for (int k = 0; k < PARTS; ++k)
        // a part with no key for the row holds no O
        x[h][k] = f[k] == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                              : *reinterpret_cast<const float4*>(
                                    p.part_o + slot(k) * kPagedTileRows * D +
                                    ((size_t)(c + h) * kPagedTileRows + r) * 4);
#pragma unroll
    for (int h = 0; h < COLS; ++h) {
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < PARTS; ++k) {
        o.x += f[k] * x[h][k].x;
        o.y += f[k] * x[h][k].y;
        o.z += f[k] * x[h][k].z;
        o.w += f[k] * x[h][k].w;
      }
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * D + 4 * (c + h)) = make_uint2(
          pack2<BF16>(o.x * inv, o.y * inv), pack2<BF16>(o.z * inv, o.w * inv));
    }
  }
}

// The tile kernel's items, a thread a row: up to 8 parts in one go, beyond that
// four at a time, and beyond 16 parts four threads share a row's parts (a 64-token chunk of 4 key/value heads over 32768 keys,
// 38 parts an item: 29 us of kernel and join, 44 with a thread a row).
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 4) paged_join_tiles_kernel(const PagedParams p) {
  __shared__ Sum meet[kThreads];
  grid_wait();
  grid_release();
  const int4* d = p.desc + 2 * (2 * blockIdx.x + (blockIdx.y & 1));
  const int4 item = d[0], seq = d[1];
  const int parts = item.x;
  if (parts == 0) return;
  const int TT = 128 / p.G;
  // row r of the item: whether it is one, and its row of O
  auto place = [&](int r, size_t& row) {
    const int head = (r & 127) / TT;
    const int token = item.w + (r >> 7) * TT + (r & 127) - head * TT;
    row = (size_t)(item.z * p.G + head) * p.total + seq.x + token;
    return head < p.G && token < seq.y;
  };
  const int first = blockIdx.x - item.y;
  const int slices = parts * (gridDim.y / 2), slice = item.y * (gridDim.y / 2) + (blockIdx.y >> 1);
  size_t row;
  if (parts <= 8) {
    const int r = threadIdx.x;
    if (!place(r, row)) return;
    if (parts == 2)
      join_few<D, BF16, 2, 4>(p, first, parts, r, row, 4 * slice, 4 * slices);
    else if (parts <= 4)
      join_few<D, BF16, 4, 2>(p, first, parts, r, row, 2 * slice, 2 * slices);
    else
      join_few<D, BF16, 8, 1>(p, first, parts, r, row, slice, slices);
    return;
  }
  const int ways = parts > 16 ? 4 : 1, rows = kThreads / ways;  // rows at once
  const int way = threadIdx.x / rows;
  for (int u = slice; u < D / 4 * ways; u += slices) {
    const int c4 = u / ways, r = u % ways * rows + threadIdx.x % rows;
    const bool live = place(r, row);
    Sum s = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int k0 = way * 4; live && k0 < parts; k0 += ways * 4)
      add_parts<D, kPagedTileRows, 4>(p, s, first, c4 * kPagedTileRows + r, r, k0, parts);
    if (ways > 1) {
      meet[threadIdx.x] = s;
      __syncthreads();
      if (way == 0) {
        for (int w = 1; w < ways; ++w) {
          const Sum& x = meet[threadIdx.x + rows * w];
          add(s, x.m, x.l, x.o);
        }
      }
      __syncthreads();
    }
    if (live && way == 0) store<D, BF16>(p, row, c4, s);
  }
}

template <int D, bool BF16>
cudaError_t launch_db(const PagedLaunch& a, bool decode) {
  // a CTA per slot of the main kernel's, four for tiles
  const dim3 grid((unsigned)a.grid, decode ? 2 : 8);
  return decode ? launch_dependent(paged_join_rows_kernel<D, BF16>, grid, kThreads, 0, a.stream,
                                   a.params)
                : launch_dependent(paged_join_tiles_kernel<D, BF16>, grid, kThreads, 0, a.stream,
                                   a.params);
}

template <int D>
cudaError_t launch_d(const PagedLaunch& a, bool bf16, bool decode) {
  return bf16 ? launch_db<D, true>(a, decode) : launch_db<D, false>(a, decode);
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
