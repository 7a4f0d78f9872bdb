// decode_common.cuh — work plan of the split decode and the cross-range combine.
//
// Split-KV flash decoding (not on the pages; the standard exact identity of the softmax): the
// tokens of a sequence are cut into ranges; each range yields an unnormalised partial
// (O_r = sum_t e^{s_t - m_r} c_t, m_r, l_r = sum_t e^{s_t - m_r}); the partials merge exactly.
// Scores are carried in the log2 domain (scale * log2(e) folded into one factor) so the kernels
// use exp2; lse is converted back to the natural log at the end.
//
// Work plan.  Every sequence is cut into 128-token tiles (the last one ragged); T = total tiles.
// P work ranges (one CTA pair each) share them in one of two ways:
//  * per sequence (when every non-empty sequence has at least T / P tiles): sequence b gets
//    r_b = floor(P tiles_b / T) >= 1 ranges that split its tiles evenly, so every range holds one
//    piece of one sequence (pairs beyond sum r_b stay idle);
//  * balanced (otherwise): the tiles of the batch are laid end to end (sequence b owns global
//    tiles [off_b, off_b + tiles_b)) and the ranges cut that line into P pieces of equal cost,
//    where a non-empty sequence costs kSegCost + tiles_b: a range spends a few tiles' worth of
//    time at each segment it starts (the new Q, the pipeline refill, the epilogue of the previous
//    segment), so a range that meets more sequences takes fewer tiles.  On the cost line sequence
//    b spans [W_b, W_b + kSegCost + tiles_b) (W_b the sum over earlier non-empty sequences); the
//    boundary x_p = floor(p C / P) (C the total cost) falls in one such span and becomes global
//    tile off_b + max(0, x_p - W_b - kSegCost) (off_b itself when it falls in the sequence's
//    segment charge), or T when p = P.  Range p takes tiles [bound_p, bound_{p+1}) (possibly none);
//    the part of each sequence a range touches is a segment.  Tile j of sequence b sits at cost
//    y = W_b + kSegCost + j, and bound_p <= its global index exactly when x_p <= y, so the ranges
//    holding a sequence's tiles follow from W_b, tiles_b and C in closed form (the combine).
// A segment that covers its whole sequence is finished by the decode kernel; otherwise (in the
// balanced plan at most the first and the last segment of a range) its partial goes to
// workspace slot 2p (the range's first segment) or 2p + 1 (its last) and the combine merges the
// partials of the sequence in ascending range order.  The plan depends only on the sequence
// lengths and P, so paged and contiguous caches with equal lengths use the same ranges.
#pragma once

#include <cuda_bf16.h>

#include <climits>

#include "append.cuh"

namespace mla {

constexpr int kTile = 128;               // tokens per tile of the work plan and of the decode kernel
// What a segment start costs a range in the balanced plan, in tiles: about 4-5 us per segment against
// 1.6-2.2 us per steady-state tile (timestamps of 1024 chunk rows and of 128 sequences).
constexpr int kSegCost = 2;
constexpr int kMaxDecodeBatch = 16384;   // sequences per decode call (the plan's prefix fits in smem)

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Workspace layout for P work ranges and `batch` sequences:
//   O      [2P][128][512] fp32   (unnormalised partial sums of c)
//   m      [2P][128]      fp32   (running max, log2 domain)
//   l      [2P][128]      fp32   (running sum of exp2(s - m))
//   plan   [batch + 2]    int32  (balanced: cost prefix W_b of each sequence, [batch] = C;
//                                 per sequence: first range of each sequence, [batch] = ranges used;
//                                 [batch + 1] = the plan kind)
struct Workspace {
  float* o;
  float* m;
  float* l;
  int32_t* off;
};
__host__ __device__ __forceinline__ Workspace ws_carve(void* base, int P) {
  Workspace w;
  w.o = reinterpret_cast<float*>(base);
  w.m = w.o + static_cast<int64_t>(2 * P) * kHeads * kDLat;
  w.l = w.m + static_cast<int64_t>(2 * P) * kHeads;
  w.off = reinterpret_cast<int32_t*>(w.l + static_cast<int64_t>(2 * P) * kHeads);
  return w;
}
__host__ __device__ __forceinline__ size_t ws_bytes(int batch, int P) {
  const size_t partials = static_cast<size_t>(2 * P) * kHeads * (kDLat + 2) * sizeof(float);
  return partials + ((static_cast<size_t>(batch) + 2) * sizeof(int32_t) + 15) / 16 * 16;
}

// Effective length of sequence b: seq_lens[b] clamped to [0, capacity] (error word set if it
// had to be clamped).
__device__ __forceinline__ int seq_len_checked(const int32_t* seq_lens, int b, int capacity) {
  int L = seq_lens[b];
  if (L < 0 || L > capacity) {
    set_dev_error(0x4);
    L = L < 0 ? 0 : capacity;
  }
  return L;
}
__host__ __device__ __forceinline__ int tiles_of(int L) { return (L + kTile - 1) / kTile; }

// What a query row of cached length L attends to.
//
// FullRows: every token t < L.
//
// WindowRows (sliding window with sinks): the first `sinks` tokens and the last `window` ones,
//   V(L) = { t < L : t < sinks or t >= L - window };
// the tokens between them are neither copied nor scored.  The plan, the ranges and the segments
// count a row's tokens in a shortened frame: the whole 64-token boxes that hold a visible token, laid
// end to end, so frame token v stands for token v below `first` (the sinks' boxes) and v + shift
// from there on, shift a multiple of 64.  A box never crosses a page, the same boxes are used in
// paged and contiguous caches, and every box holds a visible token.  Hidden tokens that share a box
// with visible ones, [hole0, hole1), get a score of -inf and a zeroed V row (0 * inf would be NaN).
struct FullRows {
  static constexpr bool kHoles = false;
  struct Map {
    __device__ __forceinline__ int real(int v) const { return v; }
    __device__ __forceinline__ int hole0() const { return 0; }
    __device__ __forceinline__ int hole1() const { return 0; }
  };
  __device__ __forceinline__ int span(int L) const { return L; }
  __device__ __forceinline__ Map map(int) const { return {}; }
};
struct WindowRows {
  static constexpr bool kHoles = true;
  int window, sinks;
  struct Map {
    int first, shift, h0, h1;
    __device__ __forceinline__ int real(int v) const { return v < first ? v : v + shift; }
    __device__ __forceinline__ int hole0() const { return h0; }
    __device__ __forceinline__ int hole1() const { return h1; }
  };
  // Without a window only the sinks are left: a row of at most `sinks` tokens.
  __device__ __forceinline__ int visible_end(int L) const { return window > 0 ? L : min(L, sinks); }
  __device__ __forceinline__ Map map(int L) const {
    const int start = max(visible_end(L) - window, 0);
    if (start <= sinks) return {INT_MAX, 0, 0, 0};   // no gap
    const int first = (sinks + 63) & ~63;
    return {first, max((start & ~63) - first, 0), sinks, start};
  }
  __device__ __forceinline__ int span(int L) const { return visible_end(L) - map(L).shift; }
};

// floor(x y / z) for x, y >= 0 and z > 0, exact; 32-bit arithmetic when x y fits (the wide
// division is out of line: it is rarely taken and its code is long).
__host__ __device__ __noinline__ int muldiv_wide(uint64_t p, uint32_t z) { return static_cast<int>(p / z); }
__host__ __device__ __forceinline__ int muldiv(int x, int y, int z) {
  const uint64_t p = static_cast<uint64_t>(x) * static_cast<uint32_t>(y);
  if (p <= 0xffffffffull) return static_cast<int>(static_cast<uint32_t>(p) / static_cast<uint32_t>(z));
  return muldiv_wide(p, static_cast<uint32_t>(z));
}

// The (non-empty) range of the balanced plan that holds the tile at cost y (0 <= y < C): the last
// p with x_p = floor(p C / P) <= y, i.e. ceil((y + 1) P / C) - 1.
__host__ __device__ __forceinline__ int range_of_cost(int y, int P, int C) {
  const uint64_t x = static_cast<uint64_t>(y + 1) * static_cast<uint32_t>(P) + static_cast<uint32_t>(C - 1);
  if (x <= 0xffffffffull) return static_cast<int>(static_cast<uint32_t>(x) / static_cast<uint32_t>(C)) - 1;
  return muldiv_wide(x, static_cast<uint32_t>(C)) - 1;
}

constexpr int kPlanBalanced = 0;
constexpr int kPlanPerSequence = 1;

// One segment of a work range: tokens [tok_begin, tok_end) of sequence b.
struct Segment {
  int b;
  int tok_begin;
  int tok_end;
  int n_tiles;
  bool direct;   // covers the whole sequence: the decode kernel writes the final output
  int slot;      // workspace slot of the partial otherwise
  int len;       // cached tokens of the sequence ([tok_begin, tok_end) is in the frame of Rows)
};

// Walks the segments of one work range in order.  Every role of a CTA walks the same sequence.
struct SegmentCursor {
  int b;       // next sequence to look at
  int off;     // its tile offset (global in the balanced plan, 0 in the per-sequence plan)
  int start;   // the range's tiles [start, end) in the same frame
  int end;
  int b_end;   // sequences [b, b_end) may hold segments
  int pair;
  bool first;
  int len0;    // length of the first sequence b (known from the plan: no memory read on the way in)

  template <class Rows>
  __device__ bool next(const int32_t* seq_lens, int capacity, const Rows& rows, Segment& s) {
    while (b < b_end && off < end) {
      const int len = first ? len0 : seq_len_checked(seq_lens, b, capacity);
      const int L = rows.span(len);
      const int tiles = tiles_of(L);
      const int t0 = (start > off ? start : off) - off;
      const int t1 = (end < off + tiles ? end : off + tiles) - off;
      const int cur = b;
      off += tiles;
      ++b;
      if (t1 > t0) {
        s.b = cur;
        s.tok_begin = t0 * kTile;
        s.tok_end = min(t1 * kTile, L);
        s.n_tiles = t1 - t0;
        s.direct = t0 == 0 && t1 == tiles;
        s.slot = first ? 2 * pair : 2 * pair + 1;
        s.len = len;
        first = false;
        return true;
      }
    }
    return false;
  }
};

// Combine: merges the partials of split rows and writes the empty ones (out_lat = 0, lse = -inf).
//   out = sum_p 2^{m_p - M} O_p / sum_p 2^{m_p - M} l_p,   M = max_p m_p,   in ascending range order.
// kByRange: block x < P takes the row whose first piece range x holds, if it is split (fewer rows are split
// than there are ranges), looked up in the plan table, and the blocks from P on look over 32 rows each
// for empty ones; otherwise block x takes row x.  An empty row is written by the blocks y of its x, kCols
// heads each (one block a row: 4000 rows of nothing 286 us, 127 now).  A warp covers 128 kCols latent
// columns of a head (a lane kCols pieces of four), a block of four warps kCols heads: kCols = 4 where there
// are rows enough to fill the device, 1 where few rows may have many partials each.  8 / kCols partials are in flight at a time; their m and l are read by
// lane i for the row's i-th range, 32 ranges at once.
template <int kCols, bool kByRange>
__global__ void __launch_bounds__(128) combine_kernel(Workspace ws, int P, int B, __nv_bfloat16* __restrict__ out_lat,
                                                      float* __restrict__ lse) {
  constexpr int kAhead = 8 / kCols;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  auto write_empty = [&](int b) {
    const int64_t row = static_cast<int64_t>(b) * kHeads + blockIdx.y * kCols;
    for (int i = threadIdx.x; i < kCols * kDLat / 8; i += 128)
      reinterpret_cast<uint4*>(out_lat + row * kDLat)[i] = make_uint4(0, 0, 0, 0);
    if (lse != nullptr && threadIdx.x < kCols) lse[row + threadIdx.x] = -INFINITY;
  };
  const bool per_seq = ws.off[B + 1] == kPlanPerSequence;
  const int C = ws.off[B];
  int b = blockIdx.x, p0;
  if (kByRange) {
    if (blockIdx.x >= P) {
      const int b0 = 32 * (static_cast<int>(blockIdx.x) - P);
      uint32_t empty = __ballot_sync(0xffffffffu, b0 + lane < B && ws.off[b0 + lane + 1] == ws.off[b0 + lane]);
      for (; empty != 0; empty &= empty - 1) write_empty(b0 + __ffs(empty) - 1);
      return;
    }
    // The last row that starts at or before the key: range p itself, or the cost at which it ends.  (A row
    // that begins there or later has no piece in it.)  32 probes a round.
    const int key = per_seq ? static_cast<int>(blockIdx.x) : muldiv(static_cast<int>(blockIdx.x) + 1, C, P) - 1;
    if (key < 0) return;   // ends where the line of tiles begins: no piece
    int lo = 0, n = B;     // off[lo] <= key: among rows [lo, lo + n)
    while (n > 1) {
      const int step = (n + 31) / 32;
      const bool le = lane * step < n && ws.off[lo + lane * step] <= key;
      const int last = __popc(__ballot_sync(0xffffffffu, le)) - 1;   // the offsets ascend
      lo += last * step;
      n = min(step, n - last * step);
    }
    b = lo;
  }
  // Ranges [p0, p1] hold b's pieces; in the per-sequence plan each holds one (slot 2p).  In the balanced
  // plan they are those that hold its first and last tiles, at costs off + kSegCost and off + span - 1;
  // a piece is the range's last segment (slot 2p + 1) where the range began before b, x_p < W_b = off,
  // and a range with x_p = x_{p+1} is empty.
  const int off = ws.off[b], span = ws.off[b + 1] - off;
  if (span == 0) {
    if (!kByRange) write_empty(b);
    return;
  }
  p0 = per_seq ? off : range_of_cost(off + kSegCost, P, C);
  if (kByRange && p0 != blockIdx.x) return;
  const int p1 = per_seq ? off + span - 1 : range_of_cost(off + span - 1, P, C);
  if (p0 == p1) return;   // finished by the decode kernel
  const int h = blockIdx.y * kCols + (kCols == 4 ? warp : 0);
  const int col = 4 * lane + (kCols == 4 ? 0 : 128 * warp);
  float M = -INFINITY, den = 0.f;
  float4 acc[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int pc = p0; pc <= p1; pc += 32) {   // 32 ranges at a time, this lane's first
    const int p = pc + lane;
    int slot = -1;
    if (p <= p1) {
      if (per_seq) {
        slot = 2 * p;
      } else {
        const int x = muldiv(p, C, P);
        if (x < muldiv(p + 1, C, P)) slot = x < off ? 2 * p + 1 : 2 * p;
      }
    }
    float m = -INFINITY, l = 0.f;
    if (slot >= 0) {
      m = ws.m[static_cast<int64_t>(slot) * kHeads + h];
      l = ws.l[static_cast<int64_t>(slot) * kHeads + h];
    }
    float4 o[kAhead][kCols];
    auto fetch = [&](int i0) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int sl = __shfl_sync(0xffffffffu, slot, i0 + u);
        const float* src = ws.o + (static_cast<int64_t>(sl) * kHeads + h) * kDLat + col;
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          o[u][c] = sl >= 0 ? *reinterpret_cast<const float4*>(src + 128 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    fetch(0);
    float top = m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float Mn = fmaxf(M, top);   // finite: a non-empty range holds at least one valid token of b
    const float sa = M == -INFINITY ? 0.f : exp2f(M - Mn);
    const float w = slot >= 0 ? exp2f(m - Mn) : 0.f;
    float wl = w * l;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) wl += __shfl_xor_sync(0xffffffffu, wl, d);
    den = den * sa + wl;
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      acc[c].x *= sa;
      acc[c].y *= sa;
      acc[c].z *= sa;
      acc[c].w *= sa;
    }
    M = Mn;
    const int cnt = min(32, p1 - pc + 1);
#pragma unroll 1
    for (int i0 = 0;;) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float wu = __shfl_sync(0xffffffffu, w, i0 + u);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          acc[c].x = fmaf(wu, o[u][c].x, acc[c].x);
          acc[c].y = fmaf(wu, o[u][c].y, acc[c].y);
          acc[c].z = fmaf(wu, o[u][c].z, acc[c].z);
          acc[c].w = fmaf(wu, o[u][c].w, acc[c].w);
        }
      }
      if ((i0 += kAhead) >= cnt) break;
      fetch(i0);
    }
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  const int64_t bh = static_cast<int64_t>(b) * kHeads + h;
#pragma unroll
  for (int c = 0; c < kCols; ++c) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[c].x * inv, acc[c].y * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[c].z * inv, acc[c].w * inv);
    uint2 pk;
    pk.x = *reinterpret_cast<const uint32_t*>(&lo);
    pk.y = *reinterpret_cast<const uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(out_lat + bh * kDLat + col + 128 * c) = pk;
  }
  if (lse != nullptr && lane == 0 && (kCols == 4 || warp == 0))
    lse[bh] = den > 0.f ? (M + log2f(den)) * kLn2 : -INFINITY;
}

}  // namespace mla
