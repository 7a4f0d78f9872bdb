// attn_weights.cuh — attention weight accumulated per cached token, on the tcgen05 tensor cores.
//
//   weights[b, t] = decay * prev[b, t] + sum_i sum_h exp(scale * q[i, h] . row_t - lse[i, h])
// over the query rows i of sequence b that attend to token t (one row per sequence in a decode step,
// or the rows of a chunk, row i up to q_len[i] tokens).  The log-sum-exps are those the attention left,
// so one pass over the rows gives final weights: no running maximum, nothing to rescale, no value product.
//
// Mapping.  A unit of work is (256 tokens of a sequence, one query row): S = K Q^T, 256 tokens x 128
// heads over 576 dims, one pair MMA shape (cta_group::2, M = 256, N = 128) with the tokens as M: CTA r
// of the pair holds tokens [128 r, +128) of the tile and heads [64 r, +64) of the query, and its TMEM
// receives all 128 heads of its own tokens, a token per lane.  A thread therefore owns a token, and the
// sum over heads needs no exchange between lanes (heads as M would need a 128-lane reduction per token).
//
// Shared memory holds one token tile (147 KB a CTA) and one query row (74 KB), each in three parts of
// three 64-dim slabs with full / empty barriers of their own, so a part is refilled as soon as the MMAs
// of that part have read it.  A decode step keeps Q and streams token tiles (bound by HBM: 1152 bytes
// and 147,456 flops per token); a chunk of rows keeps the token tile and streams the rows' queries from
// L2 (bound by the tensor pipe).  A tile's rows are stored [8-row group][slab][8 rows][128 bytes]: one
// copy brings 64 rows x 3 slabs in whole swizzle atoms, and the operand descriptor's 8-row stride spans
// the three slabs, so two 64-token pages form one 128-row operand.
//
// TMEM: two S buffers of 128 columns, so a unit's MMAs overlap the exponentials of the one before.
//
// What bounds it.  A decode step: HBM.  128 sequences of 1024..8192 tokens in pages (670 MB, none of it in L2)
// take 127 us, 5.3 TB/s, 0.82 of the measured copy rate; of these about 7 us go before the first tile's
// scores.  A chunk: the tensor pipe; 64 rows of 74 tiles take 113 us, 2620 cycles a unit against the 2304
// of its 36 MMAs.  FP8: the bandwidth of shared memory, which the
// MMAs' operands (2304 cycles a unit), the codes' way in and out (1152) and the bf16 values written (1152)
// share: 5500 cycles a unit, 74 x 4096 in 59 us.  (Codes in two buffers of their own, refilled during the
// conversion: 64; sixteen converter warps: 29.0 -> 30.0 for 32 x 4096.)
//
// Split.  The units of all sequences (sequence, then tile, then row) are laid end to end and cut into P
// equal ranges, one per CTA pair.  A tile whose rows fall into several ranges leaves partial sums in the
// workspace, which a second kernel adds in range order (a decode step has one row per tile: no partials).
//
// FP8: the codes are expanded to bf16 in shared memory (exact) by eight converter warps; the power-of-two
// row scale multiplies the token's finished scores, so the converters need no scales.
#pragma once

#include "decode_common.cuh"
#include "decode_tc.cuh"

namespace mla {

constexpr int kAwTile = 256;                       // tokens of a unit (128 per CTA)
constexpr int kAwParts = 3;                        // parts of the K buffer
constexpr int kAwSlabs = 9 / kAwParts;             // 64-dim slabs of a part
constexpr int kAwQParts = 3;                       // parts of the Q buffer
constexpr int kAwQSlabs = 9 / kAwQParts;
constexpr int kAwQPart = kAwQSlabs * kTcSlab;      // 64 heads
static_assert(kAwQParts % kAwParts == 0, "a part of K covers whole parts of Q");
constexpr int kAwKBox = 64 * kAwSlabs * 128;       // 64 tokens x 3 slabs
constexpr int kAwKPart = 2 * kAwKBox;
constexpr int kAwOffQ = 0;
constexpr int kAwOffK = kAwOffQ + kAwQParts * kAwQPart;
constexpr int kAwOffLse = kAwOffK + kAwParts * kAwKPart;   // [2][128] -lse * log2(e)
constexpr int kAwOffRed = kAwOffLse + 2 * kHeads * 4;      // [2][128] sums over the upper heads
constexpr int kAwOffBar = kAwOffRed + 2 * 128 * 4;
constexpr int kAwOffMisc = kAwOffBar + 512;
constexpr int kAwSmemBytes = kAwOffMisc + 64;
static_assert(kAwSmemBytes <= 232448, "shared memory budget");

constexpr uint32_t kAwTmemCols = 256;              // two S buffers x 128 heads
constexpr int kAwSumWarps = 8;                     // read S, exponentiate, sum
constexpr int kAwMmaWarp = 8;
constexpr int kAwProducerWarp = 9;                 // and, bf16, the next two
constexpr int kAwConvWarp0 = 10;
constexpr int kAwConvThreads = 256;
__host__ __device__ constexpr int aw_producers(bool fp8) { return fp8 ? 1 : kAwParts; }
__host__ __device__ constexpr int aw_threads(bool fp8) {
  return 32 * (kAwProducerWarp + aw_producers(fp8)) + (fp8 ? kAwConvThreads : 0);
}

struct AwBars {
  uint64_t k_full[kAwParts];    // even CTA: both CTAs' part landed (one arrival per CTA + tx)
  uint64_t k_empty[kAwParts];   // both: the part consumed
  uint64_t q_full[kAwQParts];
  uint64_t q_empty[kAwQParts];
  uint64_t s_full[2];           // both: a unit's scores done
  uint64_t s_empty[2];          // even CTA: every summing warp of both CTAs has read them
  uint64_t kraw[kAwParts];      // FP8, per CTA: the part's codes landed (+ tx)
};
static_assert(sizeof(AwBars) <= 512, "barrier block");

struct AwArgs {
  CacheView v;
  const int32_t* seq_lens;
  const int32_t* q_start;   // [batch + 1] first query row of each sequence (kRows)
  const int32_t* q_len;     // [n_rows] tokens each row attends to (kRows)
  int n_rows;
  int batch;
  int capacity;
  int P;
  bool grouped;             // the K map's third coordinate counts 8-row groups (else: one copy per group)
  float scale_log2;
  float decay;
  const float* lse;
  const float* prev;        // or null
  float* weights;
  const uint8_t* scales;    // FP8
  float* part;              // [2 P][kAwTile] partial sums (kRows)
  int4* rec;                // [2 P] {sequence or -1, tile, first row, end row} of each partial (kRows); the sign
                            // bit of the end row marks the tile's last piece
};

// Workspace of the chunk form: partial sums, then their records.
__host__ __device__ __forceinline__ size_t aw_ws_bytes(int P) {
  return static_cast<size_t>(2 * P) * (kAwTile * sizeof(float) + sizeof(int4));
}

struct AwSeq {
  int L, tiles;
  int q0, R;   // query rows [q0, q0 + R); a sequence without rows counts as one that computes nothing
  bool has;
};
template <bool kRows>
__device__ __forceinline__ AwSeq aw_seq(const AwArgs& a, int b) {
  AwSeq s;
  s.L = seq_len_checked(a.seq_lens, b, a.capacity);
  s.tiles = s.L / kAwTile + (s.L % kAwTile != 0);
  s.q0 = b;
  s.R = 1;
  s.has = true;
  if (kRows) {
    const int q0 = a.q_start[b], q1 = a.q_start[b + 1];
    s.has = q1 > q0 && q0 >= 0 && q1 <= a.n_rows;
    if (!s.has && q1 != q0) set_dev_error(0x4);
    s.q0 = s.has ? q0 : 0;
    s.R = s.has ? q1 - q0 : 1;
  }
  return s;
}

struct AwPlan {
  int b, tile, row;   // where the range starts
  long long n;        // its units
};

// One warp: this pair's range of the line of units.
template <bool kRows>
__device__ __noinline__ AwPlan aw_make_plan(const AwArgs& a, int pair) {
  const int lane = threadIdx.x & 31;
  const int per = (a.batch + 31) / 32;
  const int lo = min(a.batch, lane * per), hi = min(a.batch, lo + per);
  long long mine = 0;
#pragma unroll 4
  for (int b = lo; b < hi; ++b) {
    const AwSeq s = aw_seq<kRows>(a, b);
    mine += static_cast<long long>(s.tiles) * s.R;
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  const long long total = __shfl_sync(0xffffffffu, incl, 31);
  const long long x0 = total * pair / a.P, x1 = total * (pair + 1) / a.P;
  AwPlan p{0, 0, 0, x1 - x0};
  const bool here = incl - mine <= x0 && x0 < incl;
  if (here) {
    long long left = x0 - (incl - mine);
    for (int b = lo; b < hi; ++b) {
      const AwSeq s = aw_seq<kRows>(a, b);
      const long long u = static_cast<long long>(s.tiles) * s.R;
      if (left < u) {
        p.b = b;
        p.tile = static_cast<int>(left / s.R);
        p.row = static_cast<int>(left % s.R);
        break;
      }
      left -= u;
    }
  }
  const uint32_t who = __ballot_sync(0xffffffffu, here);
  const int src = who != 0 ? __ffs(who) - 1 : 0;
  p.b = __shfl_sync(0xffffffffu, p.b, src);
  p.tile = __shfl_sync(0xffffffffu, p.tile, src);
  p.row = __shfl_sync(0xffffffffu, p.row, src);
  return p;
}

// Walks the segments of a range: the units of one tile, rows [r0, r1) of its sequence.  Every role
// walks the same ones.  A row that does not reach the tile is skipped by all of them.
template <bool kRows>
struct AwCursor {
  const AwArgs& a;
  AwSeq s;
  int b, tile, row;
  long long left;
  int r0, r1, t0;   // the current segment
  int seg_b;

  __device__ AwCursor(const AwArgs& args, const AwPlan& p)
      : a(args), s(aw_seq<kRows>(args, p.b)), b(p.b), tile(p.tile), row(p.row), left(p.n) {}

  __device__ bool next() {
    if (left <= 0) return false;
    while (tile >= s.tiles) {
      if (++b >= a.batch) return false;
      s = aw_seq<kRows>(a, b);
      tile = row = 0;
    }
    seg_b = b;
    t0 = tile * kAwTile;
    r0 = row;
    r1 = static_cast<int>(min(static_cast<long long>(s.R), r0 + left));
    left -= r1 - r0;
    row = r1;
    if (row == s.R) {
      row = 0;
      ++tile;
    }
    return true;
  }
  // Tokens that row r attends to; the first row from r on that reaches the segment's tile, or r1.
  __device__ int limit(int r) const { return kRows ? a.q_len[s.q0 + r] : s.L; }
  __device__ int active(int r) const {
    if (!s.has) return r1;
    if (kRows)
      while (r < r1 && a.q_len[s.q0 + r] <= t0) ++r;
    return r;
  }
};

// ------------------------------------------------------------------------------ TMA producers
// A thread needs about 0.2 us to wait for a slot, announce the bytes and issue the copy, whatever its size
// (8 KB copies from L2: 39 GB/s per SM from one thread, 137 from four), so a chunk's queries take three
// producer warps: warp i copies part i of K and the part of Q that it covers.  (Nine parts of Q, one slab each,
// would be refilled sooner, but their handshakes cost the issuer more: 124 -> 182 us for 8 x 32 rows.)
template <bool kRows, bool kFp8>
__device__ bool aw_producer(const CUtensorMap* tm_k, const CUtensorMap* tm_q, const AwArgs& a, const AwPlan& plan,
                            uint8_t* smem, AwBars* bars, int rank, int me, volatile int* abort_flag) {
  if (!elect_one()) return true;
  AwCursor<kRows> cur(a, plan);
  uint32_t kl = 0, ql = 0;   // tiles and query rows loaded
  int held = -1;             // the query row in shared memory
  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) { return mbar_wait(bar, parity, site) && !*abort_flag; };
  while (cur.next()) {
    int r = cur.active(cur.r0);
    if (r >= cur.r1) continue;
    // the cache rows of this CTA's two 64-token boxes; a box behind the sequence's end reads zeros
    int64_t row[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = cur.t0 + 128 * rank + 64 * h;
      row[h] = t < cur.s.L ? cache_row(a.v, cur.seg_b, t) : -1;
    }
    for (bool first = true; r < cur.r1; r = cur.active(r + 1), first = false) {
      const int q = cur.s.q0 + r;
      const bool new_q = q != held;
#pragma unroll 1
      for (int p = me; p < kAwParts; p += aw_producers(kFp8)) {
        if (first) {
          if (kl > 0 && !wait(&bars->k_empty[p], (kl - 1) & 1u, 0x40 + p)) return false;
          uint64_t* kraw = &bars->kraw[p];
          const uint32_t full = lbar(&bars->k_full[p]);
          uint8_t* dst = smem + kAwOffK + p * kAwKPart;
          if constexpr (kFp8) {
            mbar_arrive_expect_tx(kraw, kAwKPart / 2);
          } else {
            if (rank == 0)
              mbar_arrive_expect_tx_relaxed(full, 2u * kAwKPart);
            else
              mbar_arrive_relaxed(full);
          }
          auto copy = [&](int off, int y, int w) {   // off: bytes of bf16 rows before the box
            if constexpr (kFp8)
              tma_load_4d_local(dst + kAwKPart / 2 + off / 2, tm_k, kraw, 0, y, kAwSlabs * p, w);
            else
              tma_load_4d_pair(dst + off, tm_k, full, 0, y, kAwSlabs * p, w);
          };
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            if (a.grouped) {
              copy(h * kAwKBox, 0, row[h] < 0 ? -8 : static_cast<int>(row[h] >> 3));
            } else {
              for (int g = 0; g < 8; ++g)
                copy(h * kAwKBox + g * (kAwKBox / 8), row[h] < 0 ? -8 : static_cast<int>(row[h]) + 8 * g, 0);
            }
          }
        }
        if (new_q) {
#pragma unroll 1
          for (int i = p * (kAwQParts / kAwParts); i < (p + 1) * (kAwQParts / kAwParts); ++i) {
            if (ql > 0 && !wait(&bars->q_empty[i], (ql - 1) & 1u, 0x44)) return false;
            const uint32_t full = lbar(&bars->q_full[i]);
            if (rank == 0)
              mbar_arrive_expect_tx_relaxed(full, 2u * kAwQPart);
            else
              mbar_arrive_relaxed(full);
            tma_load_3d_pair(smem + kAwOffQ + i * kAwQPart, tm_q, full, 0, q * kHeads + 64 * rank, kAwQSlabs * i);
          }
        }
      }
      if (first) ++kl;
      if (new_q) ++ql;
      held = q;
    }
  }
  return true;
}

// ------------------------------------------------------------------------------ MMA issuer (even CTA)
// One elected thread.  A part of K is released with the last row of
// its segment, a part of Q as soon as another row of the segment follows; the last row's Q is released
// when the next segment turns out to need another one.
template <bool kRows>
__device__ bool aw_mma(uint8_t* smem, AwBars* bars, uint32_t tmem, const AwArgs& a, const AwPlan& plan,
                       volatile int* abort_flag) {
  const uint32_t idesc = idesc_bf16_f32(256, 128, false, false);
  const uint64_t dk = sdesc_sw128(smem_u32(smem + kAwOffK), 16, kAwSlabs * 1024);
  const uint64_t dq = sdesc_sw128(smem_u32(smem + kAwOffQ), 16, 1024);
  AwCursor<kRows> cur(a, plan);
  uint32_t kl = 0, ql = 0, u = 0;
  int held = -1;
  bool q_freed = true;   // the held row's parts have been released
  while (cur.next()) {
    int r = cur.active(cur.r0);
    for (bool first = true; r < cur.r1; first = false, ++u) {
      const int q = cur.s.q0 + r;
      const bool new_q = q != held;
      const int nr = cur.active(r + 1);
      const bool last = nr >= cur.r1;
      if (new_q && !q_freed)
        for (int i = 0; i < kAwQParts; ++i) umma_commit_pair_mc(&bars->q_empty[i], 3);
      // S buffer u & 1 last held unit u - 2
      if (u >= 2 && !mbar_wait_cluster(&bars->s_empty[u & 1], ((u - 2) >> 1) & 1u, 0x50)) return false;
      const uint32_t d = tmem + 128 * (u & 1);
#pragma unroll
      for (int c = 0; c < 9; ++c) {   // dim-slabs
        const int p = c / kAwSlabs, i = c / kAwQSlabs;
        const bool new_part = c % kAwSlabs == 0, new_q_part = c % kAwQSlabs == 0;
        if (first && new_part && !mbar_wait_cluster(&bars->k_full[p], kl & 1u, 0x51)) return false;
        if (new_q && new_q_part && !mbar_wait_cluster(&bars->q_full[i], ql & 1u, 0x52)) return false;
        if (new_part || new_q_part) tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16_pair(d, sdesc_add(dk, p * kAwKPart + (c % kAwSlabs) * 1024 + 32 * kk),
                         sdesc_add(dq, c * kTcSlab + 32 * kk), idesc, (c | kk) != 0 ? 1u : 0u);
        if (last && (c + 1) % kAwSlabs == 0) umma_commit_pair_mc(&bars->k_empty[p], 3);
        if (!last && (c + 1) % kAwQSlabs == 0) umma_commit_pair_mc(&bars->q_empty[i], 3);
      }
      umma_commit_pair_mc(&bars->s_full[u & 1], 3);
      if (first) ++kl;
      if (new_q) ++ql;
      held = q;
      q_freed = !last;
      r = nr;
      if (*abort_flag) return false;
    }
  }
  return true;
}

// ------------------------------------------------------------------------------ FP8 converter warps
// A part's codes wait in the upper half of its buffer, [8-row group][slab][8 rows][64 bytes] as the copies
// left them; each thread reads six 16-byte chunks, meets the others, and writes the exact bf16 values
// into the swizzle atoms of the whole buffer (chunk i: atom i / 32, row (i / 4) % 8, pieces 2 (i % 4), + 1).
template <bool kRows>
__device__ bool aw_convert(const AwArgs& a, const AwPlan& plan, uint8_t* smem, AwBars* bars, volatile int* abort_flag) {
  constexpr int kChunks = kAwKPart / 2 / 16 / kAwConvThreads;
  const int ct = static_cast<int>(threadIdx.x) - 32 * kAwConvWarp0;
  AwCursor<kRows> cur(a, plan);
  uint32_t kl = 0;
  while (cur.next()) {
    if (cur.active(cur.r0) >= cur.r1) continue;
    for (int p = 0; p < kAwParts; ++p) {
      const bool got = mbar_wait(&bars->kraw[p], kl & 1u, 0x48 + p) && !*abort_flag;
      if (!named_bar_red_and(3, kAwConvThreads, got)) return false;
      uint8_t* buf = smem + kAwOffK + p * kAwKPart;
      uint4 c[kChunks];
#pragma unroll
      for (int k = 0; k < kChunks; ++k) c[k] = reinterpret_cast<const uint4*>(buf + kAwKPart / 2)[ct + k * kAwConvThreads];
      named_bar_sync(3, kAwConvThreads);
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const int i = ct + k * kAwConvThreads;
        const int row = (i >> 2) & 7, pc = i & 3;
        uint4 lo, hi;
        e4m3x16_to_bf16<false>(c[k], __nv_bfloat162(), lo, hi);
        uint8_t* dst = buf + (i >> 5) * 1024 + row * 128;
        *reinterpret_cast<uint4*>(dst + (((2 * pc) ^ row) << 4)) = lo;
        *reinterpret_cast<uint4*>(dst + (((2 * pc + 1) ^ row) << 4)) = hi;
      }
      fence_proxy_async_smem();
      named_bar_sync(3, kAwConvThreads);
      if (ct == 0) {
        fence_release_smem_to_cluster();
        mbar_arrive_relaxed(lbar(&bars->k_full[p]));
      }
    }
    ++kl;
  }
  return true;
}

// ------------------------------------------------------------------------------ exponentials and sums
// Warp w reads TMEM lane quadrant w % 4 (its lanes' tokens) and the heads [64 (w / 4), +64).  A failed
// wait leaves the loop running without waits, so that all eight warps pass the same barriers.
template <bool kRows, bool kFp8>
__device__ void aw_sum(const AwArgs& a, const AwPlan& plan, int pair, uint8_t* smem, AwBars* bars, uint32_t tmem,
                       int rank, volatile int* abort_flag) {
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int half = warp >> 2;
  const int m = 32 * (warp & 3) + lane;   // token of this CTA's 128
  const uint32_t addr = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + 64 * half;
  float* nl = reinterpret_cast<float*>(smem + kAwOffLse);
  float* red = reinterpret_cast<float*>(smem + kAwOffRed);
  AwCursor<kRows> cur(a, plan);
  uint32_t u = 0;
  int held = -1, buf = 0, seg = 0;
  bool ok = true;
  // -lse * log2(e) of head m; a row that attends to nothing (lse = -inf) adds nothing
  auto load_lse = [&](int q) {
    const float l = a.lse[static_cast<int64_t>(q) * kHeads + m];
    return l == -INFINITY ? -INFINITY : -l * kLog2e;
  };
  if (kRows && m == 0 && half == 0 && rank == 0) a.rec[2 * pair] = a.rec[2 * pair + 1] = make_int4(-1, 0, 0, 0);
  for (; cur.next(); ++seg) {
    const int t = cur.t0 + 128 * rank + m;
    const int64_t at = static_cast<int64_t>(cur.seg_b) * a.capacity + t;
    const bool whole = cur.r0 == 0 && cur.r1 == cur.s.R;
    float before = 0.f;
    if (whole && half == 0 && a.prev != nullptr && t < cur.s.L) before = a.prev[at];
    float scale = a.scale_log2;
    if (kFp8 && t < cur.s.L) {
      const int64_t row = cache_row(a.v, cur.seg_b, t);
      if (row >= 0) scale *= e8m0_value(a.scales[row]);
    }
    float acc = 0.f;
    int r = cur.active(cur.r0);
    float ahead = 0.f;
    if (r < cur.r1 && cur.s.q0 + r != held && half == 0) ahead = load_lse(cur.s.q0 + r);
    for (; r < cur.r1; ++u) {
      const int q = cur.s.q0 + r;
      const int lim = cur.limit(r);
      const int nr = cur.active(r + 1);
      if (q != held) {
        buf ^= 1;
        if (half == 0) nl[buf * kHeads + m] = ahead;
        named_bar_sync(1, 32 * kAwSumWarps);
        held = q;
      }
      if (nr < cur.r1 && half == 0) ahead = load_lse(cur.s.q0 + nr);
      const int j = u & 1;
      if (ok && !__all_sync(0xffffffffu, mbar_wait(&bars->s_full[j], (u >> 1) & 1u, 0x54))) ok = false;
      if (ok) {
        tc_fence_after();
        const float4* l4 = reinterpret_cast<const float4*>(nl + buf * kHeads + 64 * half);
        uint32_t ra[2][16];
        tmem_ld16(addr + 128 * j, ra[0]);
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_ld_wait();
          if (c < 3) {
            tmem_ld16(addr + 128 * j + 16 * (c + 1), ra[(c + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(lbar(&bars->s_empty[j]));
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 l = l4[4 * c + e];
            const uint32_t* x = &ra[c & 1][4 * e];
            sum[0] += ex2_approx(fmaf(__uint_as_float(x[0]), scale, l.x));
            sum[1] += ex2_approx(fmaf(__uint_as_float(x[1]), scale, l.y));
            sum[2] += ex2_approx(fmaf(__uint_as_float(x[2]), scale, l.z));
            sum[3] += ex2_approx(fmaf(__uint_as_float(x[3]), scale, l.w));
          }
        }
        if (t < lim) acc += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      r = nr;
    }
    // The two halves of the heads meet; the lower half's threads write.
    float* rd = red + (seg & 1) * 128;
    if (half == 1) rd[m] = acc;
    named_bar_sync(1, 32 * kAwSumWarps);
    if (half == 0 && ok && !*abort_flag) {
      acc += rd[m];
      if (whole) {
        if (t < cur.s.L) a.weights[at] = (a.prev != nullptr ? a.decay * before : 0.f) + acc;
      } else {   // at most a range's first and last segments
        const int slot = 2 * pair + (seg > 0 ? 1 : 0);
        a.part[static_cast<int64_t>(slot) * kAwTile + 128 * rank + m] = acc;
        if (m == 0 && rank == 0)
          a.rec[slot] = make_int4(cur.seg_b, cur.t0 / kAwTile, cur.r0, cur.r1 | (cur.r1 == cur.s.R ? INT_MIN : 0));
      }
    }
  }
}

// ------------------------------------------------------------------------------ kernel
// grid = 2 P CTAs in clusters of 2: blockIdx.x = 2 * pair + rank.
template <bool kRows, bool kFp8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(aw_threads(kFp8), 1)
    attn_weights_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                        const __grid_constant__ AwArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  AwBars* bars = reinterpret_cast<AwBars*>(smem + kAwOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kAwOffMisc);
  int* abort_flag = reinterpret_cast<int*>(smem + kAwOffMisc + 16);
  AwPlan* plan = reinterpret_cast<AwPlan*>(smem + kAwOffMisc + 32);
  static_assert(sizeof(AwPlan) <= 32, "plan block");
  // The swizzle atoms need a 1024-byte aligned base (every CTA sees the same one).
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) set_dev_error(0x8);
    return;
  }
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair = blockIdx.x >> 1;
  const int warp = threadIdx.x >> 5;
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int p = 0; p < kAwParts; ++p) {
      mbar_init(&bars->k_full[p], 2);
      mbar_init(&bars->k_empty[p], 1);
      mbar_init(&bars->kraw[p], 1);
    }
    for (int i = 0; i < kAwQParts; ++i) {
      mbar_init(&bars->q_full[i], 2);
      mbar_init(&bars->q_empty[i], 1);
    }
    for (int j = 0; j < 2; ++j) {
      mbar_init(&bars->s_full[j], 1);
      mbar_init(&bars->s_empty[j], 2 * kAwSumWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kAwMmaWarp) {
    tmem_alloc_pair(tmem_slot, kAwTmemCols);
    tmem_relinquish_pair();
  }
  if (warp == kAwProducerWarp && (threadIdx.x & 31) == 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_q);
  }
  tc_fence_before();
  cluster_arrive_release();
  pdl_wait();
  if (warp == kAwProducerWarp) {
    const AwPlan p = aw_make_plan<kRows>(a, pair);
    if ((threadIdx.x & 31) == 0) *plan = p;
  }
  __syncthreads();
  cluster_wait_acquire();
  tc_fence_after();
  const AwPlan pl = *plan;
  const uint32_t tmem = *tmem_slot;
  if (warp < kAwSumWarps) {
    aw_sum<kRows, kFp8>(a, pl, pair, smem, bars, tmem, rank, abort_flag);
  } else if (warp >= kAwProducerWarp && warp < kAwProducerWarp + aw_producers(kFp8)) {
    if (!aw_producer<kRows, kFp8>(&tm_k, &tm_q, a, pl, smem, bars, rank, warp - kAwProducerWarp, abort_flag))
      *abort_flag = 1;
  } else if (kFp8 && warp >= kAwConvWarp0) {
    if (!aw_convert<kRows>(a, pl, smem, bars, abort_flag) && threadIdx.x == 32 * kAwConvWarp0) *abort_flag = 1;
  } else if (rank == 0 && elect_one()) {
    if (!aw_mma<kRows>(smem, bars, tmem, a, pl, abort_flag)) *abort_flag = 1;
  }
  __syncwarp();
  if (*reinterpret_cast<volatile int*>(abort_flag)) __nanosleep(200000);   // let stray copies land
  tc_fence_before();
  __syncwarp();
  cluster_sync();
  if (warp == kAwMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kAwTmemCols);
  }
}

// The tiles whose rows several ranges share: the block of the range that holds a tile's first row adds
// the partial sums in range order and writes the weights.  grid = P, block = 256.  The records of the next
// slots are read with the first one's (a tile's pieces lie in neighbouring ranges), so a tile shared by two
// ranges takes two round trips to memory.
__global__ void __launch_bounds__(kAwTile) attn_weights_join_kernel(const __grid_constant__ AwArgs a) {
  constexpr int kNext = 4;
  pdl_trigger();
  pdl_wait();
#pragma unroll 1
  for (int s = 2 * blockIdx.x; s < 2 * static_cast<int>(blockIdx.x) + 2; ++s) {
    int4 rec[kNext];
#pragma unroll
    for (int i = 0; i < kNext; ++i) rec[i] = a.rec[min(s + i, 2 * a.P - 1)];
    const int4 first = rec[0];
    if (first.x < 0 || first.z != 0) continue;
    const int t = first.y * kAwTile + threadIdx.x;
    const int L = seq_len_checked(a.seq_lens, first.x, a.capacity);
    const int64_t at = static_cast<int64_t>(first.x) * a.capacity + t;
    float acc = a.part[static_cast<int64_t>(s) * kAwTile + threadIdx.x];
    const float before = a.prev != nullptr && t < a.capacity ? a.prev[at] : 0.f;
    int done = first.w;
    auto add = [&](int n, const int4& r) {
      if (done < 0 || r.x != first.x || r.y != first.y || r.z != done) return;
      acc += a.part[static_cast<int64_t>(n) * kAwTile + threadIdx.x];
      done = r.w;
    };
#pragma unroll
    for (int i = 1; i < kNext; ++i)
      if (s + i < 2 * a.P) add(s + i, rec[i]);
    for (int n = s + kNext; done >= 0 && n < 2 * a.P; ++n) add(n, a.rec[n]);
    if (t < L) a.weights[at] = (a.prev != nullptr ? a.decay * before : 0.f) + acc;
  }
}

}  // namespace mla
