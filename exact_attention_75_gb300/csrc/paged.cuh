// Attention over a paged key/value cache: the host <-> device interface and
// what its kernels share (the batch description, the partition of the work
// over a persistent grid, and the partial results).
//
// Work.  A sequence with new tokens gives each of its key/value heads a run
// of items; an item is a tile of query rows, and costs the keys they see, times
// a weight, plus an overhead (PagedCost).  All items of the batch laid end to
// end (sequence, key/value head, tile) form one line, and CTA c of the grid
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
// of each row, in slot 0 of a CTA that continues it and slot 1 of the CTA that
// begins it, each described in desc.  The join kernel combines an item's parts
// in an order that their number fixes, so equal calls give equal bits; a CTA of
// it takes a slice of the item that its counterpart had a part of, so the join
// is shared out as evenly as the parts are.
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
// Keys of a block of the warp-level kernel (rows of its tensor-map box).
constexpr int kPagedBlock = 16;
// CTAs at most that share an item of a small batch on the warp-level kernel.
constexpr int kPagedCluster = 8;
// Query heads per key/value head at most.
constexpr int kPagedMaxGroup = 128;

struct PagedParams {
  const void* q;            // [Hkv * G, total, D]
  void* o;                  // [Hkv * G, total, D]
  float* lse;               // [Hkv * G, total]
  uint32_t* status;         // device status word
  const int* block_table;   // [n_seq, max_pages]
  const int* cu_seqlens;    // [n_seq + 1]
  const int* kv_lens;       // [n_seq], new tokens included
  int4* desc;               // [grid][slot][2] of the CTA's part of an item: parts in all (0: the
                            // slot is empty), its number, key/value head, first token; s0, qlen
  float* part_ml;           // [grid][2][rows][2]
  float* part_o;            // [grid][2][rows][D], of the tile kernel [grid][2][D / 4][rows][4]
  int n_seq, total, max_q, n_pages, page, page_log2, max_pages, Hkv, G;
  int causal;               // query i of n sees keys j <= i + kv_len - n
  int min_share;            // least share, at least one key block
  int cluster;              // CTAs of an item's cluster (decoding kernel; 0: equal shares)
  float scale_log2;         // scale * log2(e)
  unsigned long long wait_limit_ns;
};

struct PagedLaunch {
  CUtensorMap tmQ;          // [Hkv * G, total, D] (tile kernel)
  CUtensorMap tmK, tmV;     // [n_pages * Hkv, page, D]
  PagedParams params;
  int grid;                 // CTAs of the main kernel
  cudaStream_t stream;
};

// d in {64, 96, 128}.  The decoding kernel takes at most kPagedRows query
// rows per sequence and key/value head, the tile kernel any number; the join
// follows either with the same grid.
cudaError_t launch_paged_decode(const PagedLaunch& a, int d, bool bf16);
cudaError_t launch_paged_tile(const PagedLaunch& a, int d, bool bf16);
cudaError_t launch_paged_join(const PagedLaunch& a, int d, bool bf16, bool decode);

#ifdef __CUDACC__

// A row's statistics: the maximum m and the sum l of its exponentials.  A row
// without a key has l = 0 (one with a key has a term of about 1); m tells
// nothing, since the maximum passes over NaN scores and stays -inf where every
// score is one, while l is NaN then.
__device__ __forceinline__ float paged_inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float paged_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}
// Weight of partial sums at maximum M.
__device__ __forceinline__ float paged_weight(float m, float l, float M) {
  return l == 0.f ? 0.f : exp2f(m - M);
}

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

// How a kernel's items are cut and what they cost.  UNIT: keys of a block.
// KEY1, KEY2: cost of a key in an item whose rows fill one query tile or
// reach into the second (the last item of a sequence may have one tile, all
// before it have two); OVERHEAD: of an item's prologue and epilogue.  SINGLE:
// an item holds all new tokens of its sequence.  The general form finds the
// same shares, and the short one saves every CTA 0.3 to 0.5 us of its start:
// three sequences of 65536 keys, d = 64, take 30.8 us with SINGLE and 31.3
// without, four of 4096 keys 7.8 and 8.2.
template <int UNIT_, int KEY1_, int KEY2_, int OVERHEAD_, bool SINGLE_>
struct PagedCost {
  static constexpr int UNIT = UNIT_, KEY1 = KEY1_, KEY2 = KEY2_, OVERHEAD = OVERHEAD_;
  static constexpr bool SINGLE = SINGLE_;
};

// Items of one key/value head of a sequence: W new tokens each.
template <typename Cost>
__device__ __forceinline__ int paged_items(const PagedSeq& s, int W) {
  return Cost::SINGLE ? s.qlen > 0 : (s.qlen + W - 1) / W;
}

// Whether item i has rows in its second half.
__device__ __forceinline__ bool paged_two(const PagedSeq& s, int W, int i) {
  return i * W + W / 2 < s.qlen;
}

// Keys that item i's rows see: all klen in the last item (and without causal
// masking in every one), fewer by the tokens that follow in the others.
__device__ __forceinline__ int paged_keys(const PagedSeq& s, int W, int causal, int i) {
  return causal ? max(min((i + 1) * W, s.qlen) + s.klen - s.qlen, 0) : s.klen;
}

// Cost of a head's items 0 .. q-1, q at most their number.
template <typename Cost>
__device__ __forceinline__ long long paged_line(const PagedSeq& s, int W, int causal, int q) {
  if (q == 0) return 0;
  if constexpr (Cost::SINGLE) return Cost::OVERHEAD + (long long)s.klen * Cost::KEY1;
  long long keys = 0;  // of the items before the last of the q
  if (!causal) {
    keys = (long long)(q - 1) * s.klen;
  } else {
    const int koff = s.klen - s.qlen;
    const int i0 = koff + W > 0 ? 0 : -koff / W;  // the first item that sees a key
    const long long n = q - 1 - i0;
    if (n > 0) keys = n * ((long long)(i0 + 1) * W + koff) + n * (n - 1) / 2 * W;
  }
  return (long long)q * Cost::OVERHEAD + keys * Cost::KEY2 +
         (long long)paged_keys(s, W, causal, q - 1) *
             (paged_two(s, W, q - 1) ? Cost::KEY2 : Cost::KEY1);
}

// A CTA's walk along its share, one piece (an item, or the part of one that
// the share holds) at a time.
template <typename Cost>
struct PagedWalk {
  long long left;     // of the share, the current piece included
  long long share;
  int b, head, item;  // sequence, key/value head, tile of rows
  PagedSeq sq;
  uint32_t x0, take;  // the piece: [x0, x0 + take) of the item's cost (keys <= 2^29, times 4)
  int nb;             // the item's key blocks
  int u0, u1;         // those of the piece
  bool two;           // rows in the item's second half

  __device__ __forceinline__ int key_cost() const { return two ? Cost::KEY2 : Cost::KEY1; }
  // Blocks that start before offset x of the item.
  __device__ __forceinline__ int blocks(uint32_t x) const {
    constexpr uint32_t c1 = Cost::UNIT * Cost::KEY1, c2 = Cost::UNIT * Cost::KEY2;
    const uint32_t n = two ? x / c2 + (x % c2 != 0) : x / c1 + (x % c1 != 0);
    return min((int)n, nb);
  }
  __device__ __forceinline__ void piece(const PagedParams& p, int W) {
    const int keys = Cost::SINGLE ? sq.klen : paged_keys(sq, W, p.causal, item);
    two = !Cost::SINGLE && paged_two(sq, W, item);
    nb = (keys + Cost::UNIT - 1) / Cost::UNIT;
    const uint32_t rest = (uint32_t)keys * key_cost() + Cost::OVERHEAD - x0;
    take = left < (long long)rest ? (uint32_t)left : rest;
    u0 = blocks(x0);
    u1 = blocks(x0 + take);
  }
  // The item is finished here.
  __device__ __forceinline__ bool whole() const { return x0 == 0 && u1 == nb; }
  // No block of the item starts in this share (and if it has none at all, the
  // share that begins it sees to its rows).
  __device__ __forceinline__ bool nothing() const { return u0 == u1 && (nb > 0 || x0 > 0); }
  // Shares between the one that begins the item and this one: the number of
  // the piece among the item's parts, and the parts in all.
  __device__ __forceinline__ int part() const { return (int)((x0 + share - 1) / share); }
  __device__ __forceinline__ int parts() const {
    const long long at = x0 == 0 ? share - left : part() * share - x0;  // in the share that begins it
    return (int)((at + (long long)(nb - 1) * Cost::UNIT * key_cost()) / share) + 1;
  }
  // Describes the piece, a part of its item, to the join; token: the item's
  // first row's.
  __device__ __forceinline__ void describe(const PagedParams& p, int token) const {
    int4* d = p.desc + 2 * (2 * blockIdx.x + (x0 == 0 ? 1 : 0));
    d[0] = make_int4(parts(), part(), head, token);
    d[1] = make_int4(sq.s0, sq.qlen, 0, 0);
  }
  __device__ __forceinline__ void advance(const PagedParams& p, int W) {
    left -= take;
    if (left <= 0) return;
    x0 = 0;
    if (Cost::SINGLE || ++item * W >= sq.qlen) {
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

// One thread of a CTA, before its pieces are described.
__device__ __forceinline__ void paged_clear(const PagedParams& p) {
  p.desc[4 * blockIdx.x] = make_int4(0, 0, 0, 0);
  p.desc[4 * blockIdx.x + 2] = make_int4(0, 0, 0, 0);
}

// Places the CTA at the start of its share (left 0: it has none).  Every
// thread calls this.  The threads take runs of sequences, a scan over their
// sums places the share, and the thread whose run holds its start walks there.
template <typename Cost, int THREADS>
__device__ __forceinline__ PagedWalk<Cost> paged_start(const PagedParams& p, int W) {
  __shared__ long long warp_sum[THREADS / 32];
  __shared__ PagedWalk<Cost> start;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (p.n_seq + THREADS - 1) / THREADS;
  const int b0 = min(tid * run, p.n_seq), b1 = min(b0 + run, p.n_seq);
  long long sum = 0, line = 0;  // of the run, of a head of its last sequence
  PagedSeq sq = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    sq = paged_seq(p, b);
    line = paged_line<Cost>(sq, W, p.causal, paged_items<Cost>(sq, W));
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
  // (a 32-bit division where it does; the 64-bit one costs three times as much)
  const long long share =
      max(all >> 31 ? (all - 1) / gridDim.x + 1
                    : (long long)(((uint32_t)all + gridDim.x - 1) / gridDim.x),
          (long long)p.min_share);
  const long long s = share * blockIdx.x;
  long long at = before + incl - sum;
  if (s < all && s >= at && s < at + sum) {
    int b = b1 - 1;
    if (run > 1) {  // the last sequence's line is known, the others' not
      for (b = b0; b < b1; ++b) {
        sq = paged_seq(p, b);
        line = paged_line<Cost>(sq, W, p.causal, paged_items<Cost>(sq, W));
        if (s < at + line * p.Hkv) break;
        at += line * p.Hkv;
      }
    }
    PagedWalk<Cost> w;
    w.b = b;
    w.sq = sq;
    w.share = share;
    w.left = min(share, all - s);
    // the head by a rounded quotient, put right by at most a few steps
    w.head = min((int)__fdividef((float)(s - at), (float)line), p.Hkv - 1);
    while (w.head * line > s - at) --w.head;
    while ((w.head + 1) * line <= s - at) ++w.head;
    const long long off = s - at - w.head * line;
    int lo = 0, hi = paged_items<Cost>(sq, W) - 1;  // the last item that starts at or before off
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (paged_line<Cost>(sq, W, p.causal, mid) <= off) lo = mid;
      else hi = mid - 1;
    }
    w.item = lo;
    w.x0 = (uint32_t)(off - paged_line<Cost>(sq, W, p.causal, lo));
    w.piece(p, W);
    start = w;
  }
  __syncthreads();
  return start;
}

#endif  // __CUDACC__

}  // namespace attn
