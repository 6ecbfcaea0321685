// Attention over a paged key/value cache: the host <-> device interface and
// what its kernels share (the batch description, the partition of the work
// over a persistent grid, and the partial results).
//
// Work.  A sequence with new tokens gives each of its key/value heads a run
// of items; an item is a tile of query rows, and costs the keys they see plus
// kPagedOverhead (its prologue and epilogue).  All items of the batch laid end
// to end (sequence, key/value head, tile) form one line, and CTA c of the grid
// takes [c w, (c + 1) w) of it: equal shares whatever the lengths are, so one
// long sequence spreads over every SM and a ragged batch balances itself.  A
// key block belongs to the share that its first key falls in.  The lengths
// live on the device (a captured graph replays with new ones), so each CTA
// finds its own start: costs in keys make an item run's cost an arithmetic
// series (no loop over tiles), and a prefix sum over the sequences does the
// rest.
//
// An item that lies in one CTA's share is finished there.  One that crosses
// shares leaves a partial result per share: an unnormalised O and the (m, l)
// of each row, in slot 0 of the CTA that continues it and slot 1 of the CTA
// that begins it.  The beginning CTA describes the item in desc[cta], and
// the join kernel combines its parts in key order, so equal calls give equal
// bits.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace attn {

constexpr int kPagedMaxSms = 160;  // bound of the grids (two CTAs per SM at most)
// Query rows (query heads of a group x new tokens) of an item on the
// warp-level kernel: the M = 16 of its product.
constexpr int kPagedRows = 16;
// Rows of an item of the tile kernel (two query tiles).
constexpr int kPagedTileRows = 256;
// Keys of a block there (rows of the tensor-map box).
constexpr int kPagedBlock = 16;
// Query heads per key/value head at most.
constexpr int kPagedMaxGroup = 128;
// Keys an item's prologue and epilogue cost as much as.
constexpr int kPagedOverhead = 128;

struct PagedParams {
  const void* q;            // [Hkv * G, total, D]
  void* o;                  // [Hkv * G, total, D]
  float* lse;               // [Hkv * G, total]
  uint32_t* status;         // device status word
  const int* block_table;   // [n_seq, max_pages]
  const int* cu_seqlens;    // [n_seq + 1]
  const int* kv_lens;       // [n_seq], new tokens included
  int4* desc;               // [grid][2] of the item the CTA began and others continue: parts
                            // (0: none), key/value head, first token; s0, qlen of its sequence
  float* part_ml;           // [grid][2][rows][2]
  float* part_o;            // [grid][2][rows][D], of the tile kernel [grid][2][D / 4][rows][4]
  int n_seq, total, max_q, n_pages, page, page_log2, max_pages, Hkv, G;
  int causal;               // query i of n sees keys j <= i + kv_len - n
  int min_share;            // least share, at least one key block
  float scale_log2;         // scale * log2(e)
  unsigned long long wait_limit_ns;
};

struct PagedLaunch {
  CUtensorMap tmQ;          // [Hkv * G, total, D] (tile kernel)
  CUtensorMap tmK, tmV;     // [n_pages * Hkv, page, D]
  PagedParams params;
  int grid;                 // CTAs of the main kernel
  int rows;                 // rows of an item at most
  cudaStream_t stream;
};

// d in {64, 96, 128}.  The decoding kernel takes at most kPagedRows query
// rows per sequence and key/value head, the tile kernel any number; the join
// follows either with the same grid.
cudaError_t launch_paged_decode(const PagedLaunch& a, int d, bool bf16);
cudaError_t launch_paged_tile(const PagedLaunch& a, int d, bool bf16);
cudaError_t launch_paged_join(const PagedLaunch& a, int d, bool bf16, bool decode);

#ifdef __CUDACC__

// One sequence of the batch, clamped so that no access leaves the tensors.
struct PagedSeq {
  int s0, qlen, klen;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int b) {
  PagedSeq s;
  const int a = __ldg(p.cu_seqlens + b), e = __ldg(p.cu_seqlens + b + 1);
  s.s0 = min(max(a, 0), p.total);
  s.qlen = min(min(max(e, s.s0), p.total) - s.s0, p.max_q);
  s.klen = min(max(__ldg(p.kv_lens + b), 0), p.max_pages << p.page_log2);
  return s;
}

// Records sequence b as invalid in the status word if what paged_seq clamps
// was out of range.
__device__ __forceinline__ void paged_check(const PagedParams& p, int b) {
  const int a = __ldg(p.cu_seqlens + b), e = __ldg(p.cu_seqlens + b + 1);
  const int k = __ldg(p.kv_lens + b);
  if ((b == 0 && a != 0) || a < 0 || e < a || e > p.total || e - a > p.max_q || k < 0 ||
      k > (p.max_pages << p.page_log2))
    atomicCAS(p.status, 0u, 1u | (63u << 8) | ((uint32_t)min(b, 0xFFFF) << 16));
}

// Items of one key/value head of a sequence: W new tokens each.
__device__ __forceinline__ int paged_items(const PagedSeq& s, int W) {
  return (s.qlen + W - 1) / W;
}

// Keys that item i's rows see: all klen in the last item (and without causal
// masking in every one), fewer by the tokens that follow in the others.
__device__ __forceinline__ int paged_keys(const PagedSeq& s, int W, int causal, int i) {
  return causal ? max(min((i + 1) * W, s.qlen) + s.klen - s.qlen, 0) : s.klen;
}

// Cost of a head's items 0 .. q-1, q at most their number.
__device__ __forceinline__ long long paged_line(const PagedSeq& s, int W, int causal, int q) {
  long long sum = (long long)q * kPagedOverhead;
  if (q == 0) return sum;
  if (!causal) return sum + (long long)q * s.klen;
  const int koff = s.klen - s.qlen;
  const int i0 = koff + W > 0 ? 0 : -koff / W;  // the first item that sees a key
  const long long n = q - 1 - i0;               // items from it up to the one before the last
  if (n > 0) sum += n * ((long long)(i0 + 1) * W + koff) + n * (n - 1) / 2 * W;
  return sum + paged_keys(s, W, causal, q - 1);
}

// A CTA's walk along its share, one piece (an item, or the part of one that
// the share holds) at a time.  UNIT: keys of a block.
template <int UNIT>
struct PagedWalk {
  long long left;     // of the share, the current piece included
  long long share;
  int b, head, item;  // sequence, key/value head, tile of rows
  PagedSeq sq;
  int x0, take;       // the piece: [x0, x0 + take) of the item's cost
  int nb;             // the item's key blocks
  int u0, u1;         // those of the piece

  __device__ __forceinline__ void piece(const PagedParams& p, int W) {
    const int keys = paged_keys(sq, W, p.causal, item);
    nb = (keys + UNIT - 1) / UNIT;
    take = (int)min((long long)(keys + kPagedOverhead - x0), left);
    u0 = min((x0 + UNIT - 1) / UNIT, nb);
    u1 = min((x0 + take + UNIT - 1) / UNIT, nb);
  }
  // The item is finished here.
  __device__ __forceinline__ bool whole() const { return x0 == 0 && u1 == nb; }
  // No block of the item starts in this share (and if it has none at all, the
  // share that begins it sees to its rows).
  __device__ __forceinline__ bool nothing() const { return u0 == u1 && (nb > 0 || x0 > 0); }
  // Parts of an item that this share begins and others continue.
  __device__ __forceinline__ int parts() const {
    return (int)((share - left + (long long)(nb - 1) * UNIT) / share) + 1;
  }
  __device__ __forceinline__ void advance(const PagedParams& p, int W) {
    left -= take;
    if (left <= 0) return;
    x0 = 0;
    if (++item * W >= sq.qlen) {
      item = 0;
      if (++head == p.Hkv) {
        head = 0;
        do {
          sq = paged_seq(p, ++b);
        } while (sq.qlen == 0 && b + 1 < p.n_seq);
      }
    }
    piece(p, W);
  }
};

// Places the CTA at the start of its share (left 0: it has none).  Every
// thread calls this.  The threads take runs of sequences, a scan over their
// sums places the share, and the thread whose run holds its start walks there.
template <int UNIT, int THREADS>
__device__ __forceinline__ PagedWalk<UNIT> paged_start(const PagedParams& p, int W) {
  __shared__ long long warp_sum[THREADS / 32];
  __shared__ PagedWalk<UNIT> start;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (p.n_seq + THREADS - 1) / THREADS;
  const int b0 = min(tid * run, p.n_seq), b1 = min(b0 + run, p.n_seq);
  long long sum = 0, line = 0;  // of the run, of a head of its last sequence
  PagedSeq sq = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    sq = paged_seq(p, b);
    line = paged_line(sq, W, p.causal, paged_items(sq, W));
    sum += line * p.Hkv;
    if (blockIdx.x == 0) paged_check(p, b);
  }
  long long incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += up;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (tid == 0) start.left = 0;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    all += warp_sum[w];
  }
  const long long share = max((all + gridDim.x - 1) / gridDim.x, (long long)p.min_share);
  const long long s = share * blockIdx.x;
  long long at = before + incl - sum;
  if (s < all && s >= at && s < at + sum) {
    int b = b1 - 1;
    if (run > 1) {  // the last sequence's line is known, the others' not
      for (b = b0; b < b1; ++b) {
        sq = paged_seq(p, b);
        line = paged_line(sq, W, p.causal, paged_items(sq, W));
        if (s < at + line * p.Hkv) break;
        at += line * p.Hkv;
      }
    }
    PagedWalk<UNIT> w;
    w.b = b;
    w.sq = sq;
    w.share = share;
    w.left = min(share, all - s);
    w.head = (int)((s - at) / line);
    const long long off = s - at - w.head * line;
    int lo = 0, hi = paged_items(sq, W) - 1;  // the last item that starts at or before off
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (paged_line(sq, W, p.causal, mid) <= off) lo = mid;
      else hi = mid - 1;
    }
    w.item = lo;
    w.x0 = (int)(off - paged_line(sq, W, p.causal, lo));
    w.piece(p, W);
    start = w;
  }
  __syncthreads();
  return start;
}

#endif  // __CUDACC__

}  // namespace attn
