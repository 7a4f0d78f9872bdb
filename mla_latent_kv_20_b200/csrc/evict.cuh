// evict.cuh — eviction from the latent cache by accumulated attention weight.
//
// A sequence of L > keep tokens keeps its first `sinks`, its last `recent`, and of those between
// them the k = keep - sinks - recent with the largest weights (equal weights by the lower token, NaN
// below every number); L <= keep keeps all.  The kept tokens' rows move, in order, to slots
// 0 .. n - 1 of the same cache or of another one.
//
// The selection finds the k-th largest weight by its bits (a radix select: 8-bit digits from the top, each one
// histogram of the keys that share the digits found so far, done early when all of them are kept), then
// numbers the kept tokens in order.  A cluster of CTAs shares a long sequence: each holds the order keys of
// its slice in shared memory, and the histograms are summed through distributed shared memory.  It is bound
// by the latency of its steps: 8-12 us for 128 sequences of 1024..8192 tokens, a CTA each.
//
// The move is a copy bound by HBM, the rows' bytes read once and written once: 128 x 1024 rows (302 MB) in
// 53 us, 5.7 TB/s, 0.88 of the measured copy rate.  Few rows are moved by the selection kernel itself.
#pragma once

#include "append.cuh"
#include "decode_common.cuh"

namespace mla {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvKeys = 16384;        // order keys a CTA holds in shared memory (a longer slice is read again)
constexpr int kEvMaxCluster = 8;
constexpr int kEvCopies = 8;         // of each counter of a histogram

// Workspace: the kept tokens' weights [batch][keep] fp32 and the lengths before the eviction [batch].
// The move kernel reads these alone, so weights_out may be weights, and lens_out seq_lens.
struct EvictWorkspace {
  float* w;
  int32_t* len;
};
__host__ __device__ __forceinline__ EvictWorkspace ev_carve(void* base, int batch, int keep) {
  EvictWorkspace e;
  e.w = reinterpret_cast<float*>(base);
  e.len = reinterpret_cast<int32_t*>(e.w + static_cast<int64_t>(batch) * keep);
  return e;
}
__host__ __device__ __forceinline__ size_t ev_ws_bytes(int batch, int keep) {
  return ((static_cast<size_t>(batch) * keep + batch) * 4 + 15) / 16 * 16;
}

struct EvSmem {
  uint32_t keys[kEvKeys];
  uint32_t hist[256 * kEvCopies]; // [digit][lane % 8]: at most four lanes of a warp meet in a counter
  uint32_t total[2][256];         // this CTA's histogram, read by the cluster (two passes alternate)
  uint32_t sums[256];             // the cluster's (clusters of more than one CTA)
  uint32_t count[2];              // this CTA's keys above and at the threshold, read by the cluster
  uint32_t warp_gt[32], warp_eq[32];   // (the warps there are, then zeros)
  uint32_t digit, above, same;
};

// Weights in order as unsigned numbers: -inf < ... < -0 = 0 < ... < inf, and NaN (0) below them all.
__device__ __forceinline__ uint32_t ev_key(float w) {
  const uint32_t u = __float_as_uint(w);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;
  if ((u << 1) == 0u) return 0x80000000u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_dsmem_u32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
  return v;
}

// A cache of rows of `row_bytes` bytes (1152 bf16, 576 FP8) with, for FP8, a scale byte per row.
struct EvictCache {
  CacheView v;
  uint8_t* rows;
  uint8_t* scales;
};

// What the move writes beside the rows: the weights at their new slots, zeros in the slots that the
// eviction freed (up to the old length), and the new lengths.  By thread `me` of `all`.
__device__ __forceinline__ void ev_write_weights(const EvictWorkspace& ws, int b, int L, int keep, int capacity_out,
                                                 float* weights_out, int32_t* lens_out, int64_t me, int64_t all) {
  const int n = min(L, keep);
  float* wo = weights_out + static_cast<int64_t>(b) * capacity_out;
  const float* kw = ws.w + static_cast<int64_t>(b) * keep;
  for (int64_t j = me; j < min(L, capacity_out); j += all) wo[j] = j < n ? kw[j] : 0.f;
  if (me == 0) lens_out[b] = n;
}

// What a selection that also moves the rows needs for it.
struct EvictMove {
  EvictCache src, dst;
  int capacity_out;
  float* weights_out;
  int32_t* lens_out;
};
// At most this many kept tokens are moved by the selection itself (one CTA of the cluster does it): one launch
// instead of two, which is what a short call costs.  Its reads are all in flight at once, 18 pieces of 16 bytes
// a thread for 128 bf16 rows, which is what its registers hold.  Calls over cold inputs, alone, one launch / two:
//   sequences of 1000 tokens, bf16:   to 16          to 64          to 128
//     1                               14.3 / 15.4    15.0 / 15.4    16.3 / 15.4   (to 129..512, two: 15.4-15.6)
//     32                              14.7 / 15.4    15.7 / 17.4    16.8 / 17.4
//     148                             15.0 / 17.4    17.1 / 19.4    20.9 / 23.0
//     512                             39.3 / 33.8    45.3 / 44.0    53.1 / 55.3
//     1024                            65.1 / 54.3    76.0 / 72.7    90.7 / 95.2
// and FP8, half the bytes: to 128 15.0 / 15.4, 14.8 / 17.4, 16.8 / 19.4, 43.8 / 46.1, 74.0 / 76.8 us.  (From the second
// wave of blocks on, few rows of many sequences would take two launches: left, for such a call is rare.)
constexpr int kEvMoveRows = 128;

// One CTA moves the first n <= kEvMoveRows slots' rows of sequence b: reads them all, waits for all threads,
// writes them (in place whatever a write overwrites belongs to an evicted token or has been read).
template <int kRowBytes>
__device__ void ev_move_rows(const EvictMove& mv, int b, int n, const int32_t* kp, int64_t* rows) {
  constexpr int kPieces = kRowBytes / 16, kPer = kEvMoveRows * kPieces / kEvThreads;
  static_assert(kEvMoveRows * kPieces % kEvThreads == 0, "every thread moves as many pieces");
  if (threadIdx.x < kEvMoveRows) {
    const int j = threadIdx.x;
    int64_t s = -1, d = -1;
    if (j < n) {
      s = cache_row(mv.src.v, b, kp[j]);
      d = cache_row(mv.dst.v, b, j);
      if (s < 0 || d < 0) s = d = -1;
    }
    rows[j] = s;
    rows[kEvMoveRows + j] = d;
  }
  __syncthreads();
  uint4 x[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = u * kEvThreads + threadIdx.x, r = i / kPieces;
    if (rows[r] >= 0) x[u] = reinterpret_cast<const uint4*>(mv.src.rows + rows[r] * kRowBytes)[i - r * kPieces];
  }
  uint8_t sc = 0;
  const bool scale = threadIdx.x < kEvMoveRows && mv.src.scales != nullptr && rows[threadIdx.x] >= 0;
  if (scale) sc = mv.src.scales[rows[threadIdx.x]];
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = u * kEvThreads + threadIdx.x, r = i / kPieces;
    if (rows[r] >= 0)
      reinterpret_cast<uint4*>(mv.dst.rows + rows[kEvMoveRows + r] * kRowBytes)[i - r * kPieces] = x[u];
  }
  if (scale) mv.dst.scales[rows[kEvMoveRows + threadIdx.x]] = sc;
}

// grid = batch * C CTAs in clusters of C: cluster b selects for sequence b, and (kRowBytes > 0) moves its rows.
template <int kRowBytes>
__global__ void __launch_bounds__(kEvThreads, 1)
    evict_select_kernel(const float* weights, const int32_t* seq_lens, int capacity, int keep,
                        int sinks, int recent, int C, int32_t* kept, EvictWorkspace ws,
                        const __grid_constant__ EvictMove mv) {
  extern __shared__ __align__(16) uint8_t ev_raw[];
  EvSmem& sm = *reinterpret_cast<EvSmem*>(ev_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / C;
  const int rank = blockIdx.x - b * C;
  pdl_trigger();
  pdl_wait();
  int L = seq_lens[b];
  if (L < 0 || L > capacity) {
    if (tid == 0 && rank == 0) set_dev_error(0x4);
    L = L < 0 ? 0 : capacity;
  }
  if (tid == 0 && rank == 0) ws.len[b] = L;
  const float* w = weights + static_cast<int64_t>(b) * capacity;
  int32_t* kp = kept + static_cast<int64_t>(b) * keep;
  float* kw = ws.w + static_cast<int64_t>(b) * keep;
  const int me = rank * kEvThreads + tid, all = C * kEvThreads;
  // Every thread comes here once the kept tokens are written: rank 0 moves the rows, all write the weights.
  auto finish = [&]() {
    if constexpr (kRowBytes > 0) {
      if (C > 1) cluster_sync();
      else __syncthreads();
      ev_write_weights(ws, b, L, keep, mv.capacity_out, mv.weights_out, mv.lens_out, me, all);
      if (rank == 0) ev_move_rows<kRowBytes>(mv, b, min(L, keep), kp, reinterpret_cast<int64_t*>(sm.hist));
    }
  };
  if (L <= keep) {   // the same in every CTA of the cluster
    for (int j = me; j < keep; j += all) {
      kp[j] = j < L ? j : -1;
      kw[j] = j < L ? w[j] : 0.f;
    }
    finish();
    return;
  }
  auto write_sure = [&](int from, int step) {   // the tokens that are kept whatever they weigh
    for (int j = from; j < sinks + recent; j += step) {
      const int to = j < sinks ? j : keep - recent + (j - sinks), t = j < sinks ? j : L - recent + (j - sinks);
      kp[to] = t;
      kw[to] = w[t];
    }
  };
  const int k = keep - sinks - recent;
  if (k == 0) {
    write_sure(me, all);
    finish();
    return;
  }
  // This CTA's slice of the middle, in order: tokens first + [0, n).
  const int M = L - sinks - recent;   // > k
  const int S = (M + C - 1) / C;
  const int first = sinks + min(M, rank * S);
  const int n = min(M - min(M, rank * S), S);
  for (int i = tid; i < 256 * kEvCopies; i += kEvThreads) sm.hist[i] = 0;
  if (tid < 32) sm.warp_gt[tid] = sm.warp_eq[tid] = 0;
  const int held = min(n, kEvKeys);
  for (int i0 = tid; i0 < held; i0 += 8 * kEvThreads) {   // eight loads in flight
    float x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = i0 + u * kEvThreads < held ? w[first + i0 + u * kEvThreads] : 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i0 + u * kEvThreads < held) sm.keys[i0 + u * kEvThreads] = ev_key(x[u]);
  }
  auto key_at = [&](int i) { return i < kEvKeys ? sm.keys[i] : ev_key(w[first + i]); };

  // Digit by digit from the top.  `prefix` holds the digits found, k_rem how many of the keys that share
  // them are kept.  Done before the last digit if that is all of them.
  uint32_t prefix = 0, k_rem = static_cast<uint32_t>(k), thr = 0;
  for (int pass = 0;; ++pass) {
    const int shift = 24 - 8 * pass;
    __syncthreads();   // the counters are zero
    for (int i = tid; i < n; i += kEvThreads) {
      const uint32_t key = key_at(i);
      if (pass == 0 || (key >> (shift + 8)) == prefix)
        atomicAdd(&sm.hist[((key >> shift) & 255u) * kEvCopies + (lane & (kEvCopies - 1))], 1u);
    }
    __syncthreads();
    if (tid < 256) {   // digit tid: its copies lie in different banks for the lanes of a warp
      uint32_t s = 0;
#pragma unroll
      for (int u = 0; u < kEvCopies; ++u) s += sm.hist[tid * kEvCopies + ((u + (tid >> 2)) & (kEvCopies - 1))];
      sm.total[pass & 1][tid] = s;
    }
    if (C > 1) {
      cluster_sync();
      if (tid < 256) {
        uint32_t s = 0;
        for (int c = 0; c < C; ++c) s += ld_dsmem_u32(&sm.total[pass & 1][tid], c);
        sm.sums[tid] = s;
      }
    }
    __syncthreads();
    if (warp == 0) {   // the digit of the k-th largest: lane l takes digits 255 - 8 l .. 248 - 8 l
      const uint32_t* sums = C > 1 ? sm.sums : sm.total[pass & 1];
      uint32_t c8[8], s = 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        c8[u] = sums[255 - 8 * lane - u];
        s += c8[u];
      }
      uint32_t incl = s;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      uint32_t above = incl - s;
      if (above < k_rem && incl >= k_rem) {   // one lane
        uint32_t digit = 255u - 8u * lane, same = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (same == 0) {
            if (above + c8[u] >= k_rem) {
              same = c8[u];
              digit -= u;
            } else {
              above += c8[u];
            }
          }
        }
        sm.digit = digit;
        sm.above = above;
        sm.same = same;
      }
    } else {
      for (int i = tid - 32; i < 256 * kEvCopies; i += kEvThreads - 32) sm.hist[i] = 0;
      if (pass == 0) write_sure(rank * (kEvThreads - 32) + tid - 32, C * (kEvThreads - 32));
    }
    __syncthreads();
    prefix = (prefix << 8) | sm.digit;
    k_rem -= sm.above;
    // Keys above thr are kept, and the first k_rem of those equal to it.
    if (k_rem == sm.same) {           // all that share the digits: the ones above the largest key below these
      thr = (prefix << shift) - 1u;   // (not below 0: with k < M some key is smaller)
      k_rem = 0;
      break;
    }
    if (pass == 3) {
      thr = prefix;
      break;
    }
  }

  // Number the kept tokens: warp w walks its part of the slice in order, 32 at a time.
  const int per = ((n + kEvWarps - 1) / kEvWarps + 31) & ~31;
  const int lo = min(n, warp * per), hi = min(n, lo + per);
  uint32_t gt = 0, eq = 0;
  for (int i = lo + lane; i < hi; i += 32) {
    const uint32_t key = key_at(i);
    gt += key > thr;
    eq += key == thr;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    sm.warp_gt[warp] = gt;
    sm.warp_eq[warp] = eq;
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t g = sm.warp_gt[lane], e = sm.warp_eq[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, g, o), y = __shfl_up_sync(0xffffffffu, e, o);
      if (lane >= o) {
        g += x;
        e += y;
      }
    }
    if (lane == 31) {
      sm.count[0] = g;
      sm.count[1] = e;
    }
    sm.warp_gt[lane] = g - sm.warp_gt[lane];   // before this warp, within the slice
    sm.warp_eq[lane] = e - sm.warp_eq[lane];
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
  uint32_t g0 = sm.warp_gt[warp], e0 = sm.warp_eq[warp];
  for (int c = 0; c < rank; ++c) {
    g0 += ld_dsmem_u32(&sm.count[0], c);
    e0 += ld_dsmem_u32(&sm.count[1], c);
  }
  const uint32_t below = (1u << lane) - 1u;
  constexpr int kAhead = 4;
  for (int i0 = lo; i0 < hi; i0 += 32 * kAhead) {
    float x[kAhead];   // the weights themselves are written too
#pragma unroll
    for (int u = 0; u < kAhead; ++u) x[u] = i0 + 32 * u + lane < hi ? w[first + i0 + 32 * u + lane] : 0.f;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + 32 * u + lane;
      const uint32_t key = ev_key(x[u]);
      const bool above = i < hi && key > thr, equal = i < hi && key == thr;
      const uint32_t bg = __ballot_sync(0xffffffffu, above), be = __ballot_sync(0xffffffffu, equal);
      const uint32_t e = e0 + __popc(be & below);
      if (above || (equal && e < k_rem)) {
        const int j = sinks + static_cast<int>(g0 + __popc(bg & below) + min(e, k_rem));
        kp[j] = first + i;
        kw[j] = x[u];
      }
      g0 += __popc(bg);
      e0 += __popc(be);
    }
  }
  finish();
  if (C > 1) cluster_sync();   // no CTA leaves while another reads its counts
}

// Move into another buffer: grid = (blocks of kEvRows slots, batch).  Every row on its own, so the
// loads of a thread (nine 16-byte pieces for bf16) are all in flight together.
constexpr int kEvRows = 32;
template <int kRowBytes>
__global__ void __launch_bounds__(256) evict_copy_kernel(EvictCache src, EvictCache dst, const int32_t* __restrict__ kept,
                                                         EvictWorkspace ws, int keep, int capacity_out,
                                                         float* weights_out, int32_t* lens_out) {
  constexpr int kPieces = kRowBytes / 16;
  constexpr int kPer = (kEvRows * kPieces + 255) / 256;
  __shared__ int64_t from[kEvRows], to[kEvRows];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y;
  const int L = ws.len[b];
  const int n = min(L, keep);
  const int j0 = blockIdx.x * kEvRows;
  if (threadIdx.x < kEvRows) {
    const int j = j0 + threadIdx.x;
    int64_t s = -1, d = -1;
    if (j < n) {
      s = cache_row(src.v, b, kept[static_cast<int64_t>(b) * keep + j]);
      d = cache_row(dst.v, b, j);
      if (s < 0 || d < 0) s = d = -1;
      if (s >= 0 && src.scales != nullptr) dst.scales[d] = src.scales[s];
    }
    from[threadIdx.x] = s;
    to[threadIdx.x] = d;
  }
  __syncthreads();
  uint4 x[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = u * 256 + threadIdx.x;
    const int r = i / kPieces;
    if (r < kEvRows && from[r] >= 0) x[u] = reinterpret_cast<const uint4*>(src.rows + from[r] * kRowBytes)[i - r * kPieces];
  }
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = u * 256 + threadIdx.x;
    const int r = i / kPieces;
    if (r < kEvRows && from[r] >= 0) reinterpret_cast<uint4*>(dst.rows + to[r] * kRowBytes)[i - r * kPieces] = x[u];
  }
  ev_write_weights(ws, b, L, keep, capacity_out, weights_out, lens_out,
                   static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x,
                   static_cast<int64_t>(gridDim.x) * blockDim.x);
}

// Move within one buffer: grid = (9 column slices, batch).  A kept token never moves to a later slot,
// so a slice of the columns can be moved in order of the slots by one CTA: it reads the pieces of 256
// slots, waits until all its threads have, and writes them; whatever a write overwrites belongs to a
// token that was evicted or has been read.  The slices do not meet, so no CTA waits for another.
template <int kRowBytes>
__global__ void __launch_bounds__(256) evict_compact_kernel(EvictCache src, EvictCache dst,
                                                            const int32_t* __restrict__ kept, EvictWorkspace ws,
                                                            int keep, int capacity_out, float* weights_out,
                                                            int32_t* lens_out) {
  constexpr int kSlices = 9;
  constexpr int kPieces = kRowBytes / 16 / kSlices;   // 16-byte pieces of a row in a slice
  constexpr int kStep = 256;                          // slots at a time
  __shared__ int64_t from[kStep], to[kStep];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y;
  const int L = ws.len[b];
  const int n = min(L, keep);
  const int tid = threadIdx.x;
  const int col = blockIdx.x * kPieces + tid % kPieces;
  for (int j0 = 0; j0 < n; j0 += kStep) {
    {
      const int j = j0 + tid;
      int64_t s = -1, d = -1;
      if (j < n) {
        s = cache_row(src.v, b, kept[static_cast<int64_t>(b) * keep + j]);
        d = cache_row(dst.v, b, j);
        if (s < 0 || d < 0 || s == d) s = d = -1;
      }
      from[tid] = s;
      to[tid] = d;
    }
    __syncthreads();
    uint4 x[kPieces];
    uint8_t sc = 0;
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int64_t s = from[u * (kStep / kPieces) + tid / kPieces];
      if (s >= 0) x[u] = reinterpret_cast<const uint4*>(src.rows + s * kRowBytes)[col];
    }
    const bool scale = blockIdx.x == 0 && src.scales != nullptr && from[tid] >= 0;
    if (scale) sc = src.scales[from[tid]];
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int r = u * (kStep / kPieces) + tid / kPieces;
      if (from[r] >= 0) reinterpret_cast<uint4*>(dst.rows + to[r] * kRowBytes)[col] = x[u];
    }
    if (scale) dst.scales[to[tid]] = sc;
    __syncthreads();   // from and to are read above
  }
  ev_write_weights(ws, b, L, keep, capacity_out, weights_out, lens_out,
                   static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x,
                   static_cast<int64_t>(gridDim.x) * blockDim.x);
}

}  // namespace mla
