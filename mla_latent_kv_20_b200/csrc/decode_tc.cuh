// decode_tc.cuh — split-KV MLA decode on the tcgen05 tensor cores, one CTA pair per work range
// of 128-token tiles (the plan in decode_common.cuh: a range is one piece of one sequence, or a
// run of tiles that crosses sequences; each sequence piece it meets is a segment).
//
// What it computes (《DeepSeek-V2》深度解读报告 §2.3 Absorption, §2.4 Decoupled RoPE): for every
// head h the score of cached token t is  s = scale * q_full[h] . row_t  over the 576-wide row
// [c (512) | RoPE(k^R) (64)] (content plus position channel), an online softmax over the segment's
// tokens, and  O[h] = sum_t e^{s - m} c_t  over the 512-wide latent.  Every latent row is read from
// HBM once and shared by all 128 heads, which is what makes QK^T and PV dense contractions.
//
// B200 mapping.  The two CTAs of a cluster run "pair" MMAs (tcgen05 cta_group::2, M = 128): CTA r
// owns heads [64r, 64r+64) (its half of the A operand: Q for QK^T, P for PV) and each CTA's TMEM
// receives a 64-head slice of the accumulator folded over all 128 lanes, so
//   S tile (64 heads x 128 tokens, fp32)  = 64 TMEM columns per CTA (two buffers),
//   O      (64 heads x 512 latent, fp32)  = 256 TMEM columns per CTA.
// Per 128-token tile the B operand of QK^T is split by tokens: CTA r holds tokens [64r, 64r+64)
// with all 576 dims, as 9 swizzled slabs of 64 dims.  The B operand of PV is split by latent
// columns: CTA r holds latent [256n + 128r, +128) of all 128 tokens, a second read of the tile's
// rows that hits L2 because the pair reads them within microseconds.
//
// Staging.  A thread needs 0.2 us to wait for a slot, announce the bytes and issue a copy, whatever
// its size (8 KB copies from L2: 39 GB/s per SM from one thread, 137 from four), and a slot is refilled
// as soon as the MMAs have read it, so copies are large and K and V have a producer warp each: a CTA's K
// rows of a tile come as two boxes (5 and 4 dim-slabs, 72 KB together) with slots of their own, V rows
// (the L2 re-read) as 4-D boxes of 64 tokens x both 64-wide latent chunks x both latent halves (32 KB,
// two slots, one per half tile).  Separate producers took the batch-128 call with a 2001-token window
// from 118 to 110 us and 1024 chunk rows (window 512) from 341 to 286 us.  PV leaves out groups of 16
// tokens with nothing to see, and rows it must not see in the other groups are zeroed in shared memory
// before (rows past a sequence's end may hold anything, and 0 * NaN would poison the sum).
//
// Segments.  Every role walks the same segments of its range with a SegmentCursor.  A new segment loads
// its sequence's Q (once QK^T is done with the previous Q), restarts the softmax state, overwrites O with
// its first PV (after the previous segment's epilogue has read O), and ends with an epilogue that writes
// either the final output (a segment covering its whole sequence) or an fp32 partial for the combine.
// The epilogue runs after the next segment's first softmax, whose P waits in registers: the wait for the
// last PV and that softmax overlap.
//
// Warp roles (384 threads): warps 0-7 softmax / O correction / epilogue (two warps per TMEM lane
// quadrant, each owning half of the S columns), warp 8 work plan, then Q and K copies, warp 9 TMEM
// allocation (both CTAs) and, in the even CTA, QK^T, warp 10 PV (even CTA), warp 11 V copies.
//
// What bounds it.  At the 1.36-1.6 GHz that the power cap leaves a long call, a tile takes 2.1-2.3 us per
// pair: 3000-3400 cycles, of which the tensor pipe works 2176 (36 x 32 for QK^T, 16 x 64 for PV); the HBM
// floor is 1.7 us.  A call of 128 sequences of 1024..8192 tokens runs at 0.61 of the measured HBM rate.
//
// FP8 cache (kFp8, 640 threads).  Rows are 576 E4M3 codes with a power-of-two scale per token (an
// E8M0 exponent byte, 2^(e - 127)): code * scale is exact in bf16, so the MMAs, the softmax and
// the epilogue are those of the bf16 cache.  The producers copy a box's codes into the upper half
// of the bf16 buffer it will become, and the box's 64 scale bytes to the buffer's start, on a
// CTA-local barrier; four converter warps for K (12-15) and four for V (16-19) write the exact bf16
// values of code * scale over the buffer in the swizzled layout the MMAs read, then publish it to
// the pair barrier the MMA waits on.  The conversions bound it (about 4 us a tile): 8 + 24 conversion and
// 8 scaling instructions for 16 codes, twice per row (K and V layouts).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>

#include "decode_common.cuh"

namespace mla {

constexpr int kTcTile = 128;                 // tokens per tile
constexpr int kTcSlab = 8192;                // 64 rows x 128 bytes
// K of a tile is split along the 576 dims into two parts with a slot and barriers of their own, refilled as soon
// as QK^T has read them: part A = dim-slabs [0, 5), part B = [5, 9).  One thread issues both into one accumulator.
constexpr int kTcKSlabsA = 5;
constexpr int kTcKSlabsB = 4;
__host__ __device__ constexpr int tc_part_slab0(int part) { return part ? kTcKSlabsA : 0; }
__host__ __device__ constexpr int tc_part_slabs(int part) { return part ? kTcKSlabsB : kTcKSlabsA; }
constexpr int kTcVSlots = 2;                 // one slot per 64-token half of a tile (producer and PV rely on it)
constexpr int kTcVBox = 4 * kTcSlab;         // 64 tokens x 2 chunks x 2 latent halves
constexpr int kTcQBytes = 9 * kTcSlab;
constexpr int kTcPBytes = 2 * kTcSlab;       // 64 heads x 128 tokens bf16, two 64-token K chunks
constexpr float kTcRescaleThreshold = 8.0f;  // log2 units: rescale O only when the max grows > 2^8

constexpr int kTcOffQ = 0;
constexpr int kTcOffP = kTcOffQ + kTcQBytes;
constexpr int kTcOffK = kTcOffP + kTcPBytes;  // slot of part A, then slot of part B: 9 slabs in dim order
constexpr int kTcOffV = kTcOffK + 9 * kTcSlab;
constexpr int kTcOffBar = kTcOffV + kTcVSlots * kTcVBox;
constexpr int kTcOffMisc = kTcOffBar + 256;
constexpr int kTcSmemBytes = kTcOffMisc + 64 + 2 * 256 * 4;   // the dynamic base is 1024-aligned (checked)

// TMEM columns of each CTA (512 allocated): S (2 buffers x 64), O (256).
constexpr uint32_t kTcColS = 0;
constexpr uint32_t kTcColO = 256;

constexpr int kTcSoftmaxWarps = 8;
constexpr int kTcProducerWarp = 8;    // work plan, then Q and K copies
constexpr int kTcMmaWarp = 9;         // TMEM allocation (both CTAs); QK^T issue (even CTA)
constexpr int kTcPvWarp = 10;         // PV issue (even CTA)
constexpr int kTcVProducerWarp = 11;  // V copies
constexpr int kTcThreads = 32 * (kTcSoftmaxWarps + 4);
// FP8 cache: four converter warps for K and four for V after the others.
constexpr int kTcConvWarp0 = kTcSoftmaxWarps + 4;
constexpr int kTcConvThreads = 128;
constexpr int kTcThreadsFp8 = kTcThreads + 2 * kTcConvThreads;
__host__ __device__ constexpr int tc_threads(bool fp8) { return fp8 ? kTcThreadsFp8 : kTcThreads; }
// Where the codes of a box wait for conversion: the upper half of the bf16 buffer they become.
constexpr int kTcFp8OffA = kTcKSlabsA * kTcSlab / 2;
constexpr int kTcFp8OffB = kTcKSlabsB * kTcSlab / 2;
constexpr int kTcFp8OffV = kTcVBox / 2;

struct DecodeTcArgs {
  CacheView v;
  const int32_t* seq_lens;
  int batch;
  int capacity;        // tokens a sequence can hold (lengths are clamped to it)
  int P;               // work ranges (CTA pairs)
  float scale_log2;    // softmax_scale * log2(e)
  Workspace ws;
  __nv_bfloat16* out_lat;
  float* lse;
  const uint8_t* cache;   // the cache buffer (L2 prefetch addresses)
  int row_bytes;          // bytes of one cached row: 1152 (bf16) or 576 (FP8 codes)
  const int32_t* seq_map; // query row -> cache sequence (chunked prefill), or null: row b reads sequence b
  WindowRows win;         // the window and sinks (windowed instances)
};
template <class Rows>
__device__ __forceinline__ Rows tc_rows(const DecodeTcArgs& a) {
  if constexpr (Rows::kHoles)
    return a.win;
  else
    return {};
}

// This CTA pair's work range, computed once per CTA at entry (the cursor's starting state).
struct TcPlan {
  int start, end;   // tiles [start, end): global (balanced plan) or of sequence b0 (per sequence)
  int b0, off0;     // the first sequence of the range and its tile offset in the same frame
  int b_end;        // sequences [b0, b_end) may hold segments
  int len0;         // length of sequence b0
};

struct TcBars {
  uint64_t k_full[2];            // even CTA only, per K part: both CTAs' K boxes landed (one arrival per CTA + tx)
  uint64_t k_empty[2];           // both CTAs, per part: K box consumed by the MMAs
  uint64_t v_full[kTcVSlots];    // even CTA only: both CTAs' V box landed (one arrival per CTA + tx)
  uint64_t v_empty[kTcVSlots];   // both CTAs: V box consumed
  uint64_t fix[kTcVSlots];       // per CTA and slot: local load of a ragged V box
  uint64_t s_full[2];            // both: QK^T of a tile done
  uint64_t s_empty[2];           // even CTA only: every softmax warp of both CTAs has read S
  uint64_t p_full[2];            // even CTA only, per 64-token half: P ready in both CTAs (half 0: O corrected too)
  uint64_t p_empty[2];           // both, per half: PV of a tile done reading P
  uint64_t o_ready;              // both: PV of a tile done writing O (one phase per tile)
  uint64_t o_final;              // both: the last PV of a segment done (one phase per segment)
  uint64_t o_free;               // even CTA only: every softmax warp of both CTAs has read O of a segment
  uint64_t q_full;               // even CTA only: Q of both CTAs landed (one phase per segment)
  uint64_t q_empty;              // both: QK^T of a segment's last tile done
  uint64_t kraw[2];              // FP8, per CTA and part: this CTA's K codes and scales landed (+ tx)
  uint64_t vraw[kTcVSlots];      // FP8, per CTA and slot: this CTA's V codes and scales landed (+ tx)
};
static_assert(sizeof(TcBars) <= 256, "barrier block");
static_assert(kTcSmemBytes <= 232448, "shared memory budget");

__device__ __forceinline__ uint32_t lbar(const void* p) { return mapa_shared(smem_u32(p), 0); }

// The cache sequence that query row b reads: b itself, or seq_map[b] in a chunked prefill (where
// several query rows, one per new token, read one sequence).  A map entry outside the cache gives
// -1 (rows read as zeros); the producer also reports it through the device error word.
template <bool kMapped>
__device__ __forceinline__ int tc_cache_seq(const DecodeTcArgs& a, int b, bool report) {
  if (!kMapped) return b;
  const int s = a.seq_map[b];
  if (s >= 0 && s < a.v.num_seqs) return s;
  if (report) set_dev_error(0x2);
  return -1;
}

// 3-D TMA load (x: element in a 64-wide dim-slab, y: cache row, z: dim-slab) into this CTA's
// shared memory; completion counted on a barrier that may live in the peer CTA.
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* m, uint32_t bar_cluster_addr, int x,
                                                 int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar_cluster_addr), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// 4-D TMA load (x: element in a 64-wide chunk, y: cache row, z: chunk, w: latent half).
__device__ __forceinline__ void tma_load_4d_pair(void* dst, const CUtensorMap* m, uint32_t bar_cluster_addr, int x,
                                                 int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar_cluster_addr), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d_local(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int y, int z,
                                                  int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// ------------------------------------------------------------------------------ TMA producers
// Two warps, one lane of each issuing: one copies Q and K, one V, each as soon as its slots are free.
//  K(i): CTA r's 64 tokens [tile0 + 64r, +64) x 576 dims as two boxes, one per QK^T part
//        (5 and 4 dim-slabs).  A half-tile past the split end is loaded from a negative row
//        (zeros); its scores are masked anyway.
//  V(i): per 64-token half h of the tile, latent [256n + 128r, +128) for n = 0, 1 in one box,
//        laid out [n][chunk][64 rows][128 B].
//
// Rows of a V box that PV must not see: those at or past `valid` (past the segment's end) and the
// hidden ones [h0, h1).  PV works in groups of 16 tokens and leaves out groups with no row to see;
// in the others such rows are zeroed.
struct TcBox {
  int valid, h0, h1;
  __device__ bool whole() const { return valid == 64 && h0 >= h1; }
  __device__ bool sees(int r) const { return r < valid && !(r >= h0 && r < h1); }
  // Whether group q has a row to see: the first row of the group that is not hidden, or none.
  __device__ bool group(int q) const {
    int r = 16 * q;
    if (r >= h0 && r < h1) r = h1;
    return r < 16 * q + 16 && r < valid;
  }
};
// Zeroes the rows of the box's groups that PV must not see (each row is 4 slabs x 128 bytes: one
// 16-byte chunk per lane): behind the valid ones, and at both ends of the hidden run, to the border
// of the group.  Short loops: this code is cold whenever it runs, and its fetches cost more than its work.
__device__ __forceinline__ void tc_zero_hidden(uint8_t* box, const TcBox& bx, int lane) {
  uint4* p = reinterpret_cast<uint4*>(box + (lane >> 3) * kTcSlab) + (lane & 7);
#pragma unroll 1
  for (int u = 0; u < 3; ++u) {
    int r = bx.valid, end = (bx.valid + 15) & ~15;
    if (u > 0) {
      r = u == 1 ? bx.h0 : max(bx.h0, bx.h1 & ~15);
      end = u == 1 ? min(bx.h1, (bx.h0 + 15) & ~15) : bx.h1;
    }
#pragma unroll 1
    for (; r < end; ++r) p[r * 8] = make_uint4(0, 0, 0, 0);
  }
}

// The 64-token box whose first token is `tok0` (in the frame of the map) of a segment that ends at t_end.
template <bool kHoles, class Map>
__device__ __forceinline__ TcBox tc_box(const Map& map, int tok0, int t_end) {
  TcBox bx{min(max(t_end - tok0, 0), 64), 0, 0};
  if (kHoles) {
    const int r0 = map.real(tok0);
    bx.h0 = min(max(map.hole0() - r0, 0), 64);
    bx.h1 = min(max(map.hole1() - r0, 0), 64);
  }
  return bx;
}

// A V box with rows that PV must not see is loaded through a CTA-local barrier of its slot; once the
// copy has landed all lanes zero those rows, and the box is published: each lane's proxy fence, the
// warp barrier, and lane 0's release of shared memory and arrival on the even CTA's v_full.  Out of
// line: it runs at most twice per segment (four times with a window).  False if the wait failed.
__device__ __noinline__ bool tc_finish_ragged_v(uint8_t* box, uint64_t* fix, uint32_t fix_phase, TcBox bx,
                                                uint32_t vfull, volatile int* abort_flag) {
  const int lane = threadIdx.x & 31;
  int ok = 1;
  if (lane == 0) ok = (mbar_wait(fix, fix_phase, 0x13) && !*abort_flag) ? 1 : 0;
  if (__shfl_sync(0xffffffffu, ok, 0) == 0) return false;
  tc_zero_hidden(box, bx, lane);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    fence_release_smem_to_cluster();   // (a release arrival at cluster scope would take about 1 us)
    mbar_arrive_relaxed(vfull);
  }
  return true;
}

template <bool kV, bool kMapped, bool kFp8, class Rows>
__device__ bool tc_producer(const CUtensorMap* tm_ka, const CUtensorMap* tm_kb, const CUtensorMap* tm_v,
                            const CUtensorMap* tm_q, const CUtensorMap* tm_sc, const DecodeTcArgs& a,
                            const TcPlan& plan, uint8_t* smem, TcBars* bars, uint32_t rank, int pair,
                            volatile int* abort_flag) {
  const bool l0 = elect_one();
  const bool leader = rank == 0;
  // Every lane waits; the verdict (and an abort seen meanwhile) is shared by the warp.
  auto wait0 = [&](uint64_t* bar, uint32_t parity, uint32_t site) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, site) && !*abort_flag);
  };
  SegmentCursor cur{plan.b0, plan.off0, plan.start, plan.end, plan.b_end, pair, true, plan.len0};
  Segment sg;
  int g = 0;    // global tile index of the range (K copies)
  int vn = 0;   // V boxes issued
  int k = 0;    // segment index
  uint32_t fix_phase = 0;
  bool ok = true;
  const bool paged = a.v.page_size != 0;
  const Rows rows = tc_rows<Rows>(a);
  while (ok && cur.next(a.seq_lens, a.capacity, rows, sg)) {
    const auto map = rows.map(sg.len);
    const int b = sg.b, t_begin = sg.tok_begin, t_end = sg.tok_end, n_tiles = sg.n_tiles;
    // Q of sequence b.  The buffer is free once both QK^T parts have finished the previous segment.
    // Arrivals on the even CTA's barriers that only count (the data and its visibility come with
    // the TMA's complete_tx) are relaxed.
    if (!kV && k > 0 && !wait0(&bars->q_empty, static_cast<uint32_t>(k - 1) & 1u, 0x14)) {
      ok = false;
      break;
    }
    if (!kV && l0) {
      tma_load_3d_pair(smem + kTcOffQ, tm_q, lbar(&bars->q_full), 0, b * kHeads + 64 * static_cast<int>(rank), 0);
      if (leader)
        mbar_arrive_expect_tx_relaxed(lbar(&bars->q_full), 2u * kTcQBytes);
      else
        mbar_arrive_relaxed(lbar(&bars->q_full));
    }
    // Where the 64-token box at token t (of the frame; boxes never cross a page) lies: its block id, or its
    // row in a contiguous cache.  Fetched a tile ahead, so that neither a copy nor the wait before it
    // stands behind a dependent load of the block table; turned into the TMA row when it is used (for a bad
    // block id or map entry that of a fully out-of-bounds box, which the TMA unit fills with zeros).
    const int cb = tc_cache_seq<kMapped>(a, b, !kV);
    const int32_t* table = paged ? a.v.block_table + static_cast<int64_t>(cb < 0 ? 0 : cb) * a.v.max_blocks : nullptr;
    auto fetch = [&](int t) -> int {
      if (kMapped && cb < 0) return INT_MIN;
      const int r = map.real(t);
      return paged ? table[r / kPage] : static_cast<int>(cache_row(a.v, cb, r));
    };
    auto row_of = [&](int id) -> int {
      if (!paged || id == INT_MIN) return id < 0 ? -kTcTile : id;
      const int64_t r = static_cast<int64_t>(id) * kPage;
      if (id < 0 || r >= a.v.num_rows) {
        if (l0) set_dev_error(0x2);
        return -kTcTile;
      }
      return static_cast<int>(r);
    };
    auto k_token = [&](int i) { return t_begin + i * kTcTile + 64 * static_cast<int>(rank); };
    int k_id = 0;
    if (!kV && k_token(0) < t_end) k_id = fetch(k_token(0));
    auto issue_k = [&](int i) -> bool {
      const int gi = g + i;
      const int y = k_token(i) < t_end ? row_of(k_id) : -kTcTile;
      if (k_token(i + 1) < t_end) k_id = fetch(k_token(i + 1));
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
        if (gi >= 1 && !wait0(&bars->k_empty[part], static_cast<uint32_t>(gi - 1) & 1u, 0x10 + part)) return false;
        uint8_t* slot = smem + kTcOffK + tc_part_slab0(part) * kTcSlab;
        if (l0) {
          if constexpr (kFp8) {
            // codes to the slot's upper half, the 64 rows' scale bytes to its start (this CTA only;
            // the converter warps publish the converted slot to k_full)
            mbar_arrive_expect_tx(&bars->kraw[part], static_cast<uint32_t>(tc_part_slabs(part) * kTcSlab / 2 + 64));
            tma_load_3d(slot + (part ? kTcFp8OffB : kTcFp8OffA), part ? tm_kb : tm_ka, &bars->kraw[part], 0, y,
                        tc_part_slab0(part));
            tma_load_1d(slot, tm_sc, &bars->kraw[part], y);
          } else {
            tma_load_3d_pair(slot, part ? tm_kb : tm_ka, lbar(&bars->k_full[part]), 0, y, tc_part_slab0(part));
            if (leader)
              mbar_arrive_expect_tx_relaxed(lbar(&bars->k_full[part]), 2u * tc_part_slabs(part) * kTcSlab);
            else
              mbar_arrive_relaxed(lbar(&bars->k_full[part]));
          }
        }
      }
      return true;
    };
    int v_id[2];
    auto fetch_v = [&](int i) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int tok0 = t_begin + i * kTcTile + 64 * s;
        if (tok0 < t_end) v_id[s] = fetch(tok0);
      }
    };
    if (kV) fetch_v(0);
    auto issue_v = [&](int i) -> bool {
      TcBox bx[2];
      int rows2[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        bx[s] = tc_box<Rows::kHoles>(map, t_begin + i * kTcTile + 64 * s, t_end);
        rows2[s] = bx[s].valid > 0 ? row_of(v_id[s]) : 0;
      }
      if (i + 1 < n_tiles) fetch_v(i + 1);
#pragma unroll
      for (int s = 0; s < 2; ++s, ++vn) {   // box h of a tile sits in slot h
        const int row = rows2[s];
        if (vn >= kTcVSlots && !wait0(&bars->v_empty[s], static_cast<uint32_t>((vn / kTcVSlots) - 1) & 1u, 0x12))
          return false;
        uint8_t* box = smem + kTcOffV + s * kTcVBox;
        if constexpr (kFp8) {
          // A box with no token in the segment is not copied, its barrier completes on the arrival
          // alone.
          if (l0) {
            if (bx[s].valid > 0) {
              mbar_arrive_expect_tx(&bars->vraw[s], static_cast<uint32_t>(kTcVBox / 2 + 64));
              tma_load_4d_local(box + kTcFp8OffV, tm_v, &bars->vraw[s], 0, row, 2 * static_cast<int>(rank), 0);
              tma_load_1d(box, tm_sc, &bars->vraw[s], row);
            } else {
              mbar_arrive(&bars->vraw[s]);
            }
          }
          continue;
        }
        if (bx[s].valid == 0) {   // PV skips the box, its barrier completes on the arrivals alone
          if (l0) mbar_arrive_relaxed(lbar(&bars->v_full[s]));
        } else if (bx[s].whole()) {
          if (l0) {
            tma_load_4d_pair(box, tm_v, lbar(&bars->v_full[s]), 0, row, 2 * static_cast<int>(rank), 0);
            if (leader)
              mbar_arrive_expect_tx_relaxed(lbar(&bars->v_full[s]), 2u * kTcVBox);
            else
              mbar_arrive_relaxed(lbar(&bars->v_full[s]));
          }
        } else if (l0) {
          mbar_arrive_expect_tx(&bars->fix[s], kTcVBox);
          tma_load_4d_local(box, tm_v, &bars->fix[s], 0, row, 2 * static_cast<int>(rank), 0);
        }
      }
      if constexpr (!kFp8) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {   // with both copies on their way
          if (bx[s].valid == 0 || bx[s].whole()) continue;
          if (!tc_finish_ragged_v(smem + kTcOffV + s * kTcVBox, &bars->fix[s], (fix_phase >> s) & 1u, bx[s],
                                  lbar(&bars->v_full[s]), abort_flag))
            return false;
          fix_phase ^= 1u << s;
        }
      }
      return true;
    };
    for (int i = 0; ok && i < n_tiles; ++i) ok = kV ? issue_v(i) : issue_k(i);
    g += n_tiles;
    ++k;
  }
  return ok;
}

// ------------------------------------------------------------------------------ MMA issuers (even CTA)
// One elected thread issues QK^T and one PV.  Both shapes then run at the tensor pipe's full rate (M = 128
// pair, cycles per K step of 16: N = 128 32.6, N = 256 64.6; from a thread chosen by its lane number 52.9 and
// 64.6): QK^T of tile i + 1 shares the pipe with PV of tile i, and the softmax warps work in between.

// Advance a shared-memory descriptor by `bytes` (a multiple of 16): the start address field
// holds address / 16 in its low 14 bits, and every operand here lies below 256 KB, so the sum
// never carries out of the field.
__device__ __forceinline__ uint64_t sdesc_add(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

// S(g) = Q . K(g)^T into S buffer g & 1, for every global tile g of the range; Q is reloaded for each
// segment.  Part A's slabs come first, so its K slot is released halfway through the tile's QK^T.
template <class Rows>
__device__ bool tc_mma_qk(uint8_t* smem, TcBars* bars, uint32_t tmem, const int32_t* seq_lens, int capacity,
                          const Rows rows, SegmentCursor cur, volatile int* abort_flag) {
  const uint32_t idesc_qk = idesc_bf16_f32(128, 128, false, false);
  const uint64_t dq = sdesc_sw128(smem_u32(smem + kTcOffQ), 16, 1024);
  const uint64_t dk = sdesc_sw128(smem_u32(smem + kTcOffK), 16, 1024);
  Segment sg;
  int g = 0, k = 0;
  while (cur.next(seq_lens, capacity, rows, sg)) {
    if (!mbar_wait_cluster(&bars->q_full, static_cast<uint32_t>(k) & 1u, 0x20)) return false;
    for (int i = 0; i < sg.n_tiles; ++i, ++g) {
      const uint32_t sb = tmem + kTcColS + 64 * (g & 1);
      // S buffer g & 1 last held tile g - 2: every softmax warp of both CTAs must have read it.
      if (g >= 2 && !mbar_wait_cluster(&bars->s_empty[g & 1], static_cast<uint32_t>((g - 2) >> 1) & 1u, 0x24))
        return false;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        if (!mbar_wait_cluster(&bars->k_full[part], static_cast<uint32_t>(g) & 1u, 0x21)) return false;
        tc_fence_after();
        // Fully unrolled: every descriptor is a constant offset from the base.
#pragma unroll
        for (int c = tc_part_slab0(part); c < tc_part_slab0(part) + tc_part_slabs(part); ++c)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t off = c * kTcSlab + 32 * kk;
            umma_bf16_pair(sb, sdesc_add(dq, off), sdesc_add(dk, off), idesc_qk, (c | kk) != 0 ? 1u : 0u);
          }
        umma_commit_pair_mc(&bars->k_empty[part], 3);
      }
      umma_commit_pair_mc(&bars->s_full[g & 1], 3);
      if (*abort_flag) return false;
    }
    umma_commit_pair_mc(&bars->q_empty, 3);   // Q of this segment no longer read
    ++k;
  }
  return true;
}

// O[:, latent half n] += P(g) . V(g)[:, half n] for both halves.  The first 64-token half of the tile is
// consumed first, as soon as its P is ready, and its P and V box are released before the second's.
// The first tile of a segment overwrites O, after the previous segment's epilogue has read it.
template <class Rows>
__device__ bool tc_mma_pv(uint8_t* smem, TcBars* bars, uint32_t tmem, const int32_t* seq_lens, int capacity,
                          const Rows rows, SegmentCursor cur, volatile int* abort_flag) {
  const uint32_t idesc_pv = idesc_bf16_f32(128, 256, false, true);
  const uint64_t dp = sdesc_sw128(smem_u32(smem + kTcOffP), 16, 1024);
  const uint64_t dv = sdesc_sw128(smem_u32(smem + kTcOffV), kTcSlab, 1024);
  const uint32_t ocol = tmem + kTcColO;
  Segment sg;
  int g = 0, k = 0;
  bool ok = true;
  while (ok && cur.next(seq_lens, capacity, rows, sg)) {
    if (k > 0 && !mbar_wait_cluster(&bars->o_free, static_cast<uint32_t>(k - 1) & 1u, 0x25)) {
      ok = false;
      break;
    }
    const auto map = rows.map(sg.len);
    uint32_t acc = 0;   // the segment's first MMA overwrites O
    for (int i = 0; i < sg.n_tiles && ok; ++i, ++g) {
      // V box 2g + h sits in slot h of the 2-slot ring, in its (g + 1)-th fill.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!mbar_wait_cluster(&bars->p_full[h], static_cast<uint32_t>(g) & 1u, 0x22) ||
            !mbar_wait_cluster(&bars->v_full[h], static_cast<uint32_t>(g) & 1u, 0x23)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t pb = sdesc_add(dp, h * kTcSlab);
        const uint64_t vb = sdesc_add(dv, h * kTcVBox);
        const TcBox bx = tc_box<Rows::kHoles>(map, sg.tok_begin + i * kTcTile + 64 * h, sg.tok_end);
        auto group = [&](int g4) {   // 16 tokens, both latent halves
#pragma unroll
          for (int n = 0; n < 2; ++n)
            umma_bf16_pair(ocol + 128 * n, sdesc_add(pb, 32 * g4), sdesc_add(vb, n * 2 * kTcSlab + g4 * 2048), idesc_pv,
                           acc);
          acc = 1;
        };
        if (bx.whole()) {
#pragma unroll
          for (int g4 = 0; g4 < 4; ++g4) group(g4);
        } else {
#pragma unroll 1
          for (int g4 = 0; g4 < 4; ++g4)
            if (bx.group(g4)) group(g4);
        }
        umma_commit_pair_mc(&bars->v_empty[h], 3);
        umma_commit_pair_mc(&bars->p_empty[h], 3);
      }
      if (!ok) break;
      umma_commit_pair_mc(&bars->o_ready, 3);
      if (*abort_flag) ok = false;
    }
    // A dedicated barrier (one phase per segment) says "all PV of the segment done" to its
    // epilogue; o_ready cannot serve by parity (it may be two phases short when the epilogue starts).
    umma_commit_pair_mc(&bars->o_final, 3);
    ++k;
  }
  return ok;
}

// ------------------------------------------------------------------------------ FP8 converter warps
// 2^(e - 127) of an E8M0 scale byte (e = 255, not written by the FP8 append, is read as 2^128 = inf).
__device__ __forceinline__ float e8m0_value(uint32_t e) {
  return e == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(e << 23);
}

// A row's power-of-two scale as a pair of bf16, exact.
__device__ __forceinline__ __nv_bfloat162 e8m0_bf162(uint32_t e) { return __float2bfloat162_rn(e8m0_value(e)); }

// 16 E4M3 codes (one 16-byte chunk), times the row scale if kScaled, as 16 bf16 values in two 16-byte
// chunks (codes 0-7, codes 8-15).  Exact: four significant bits, and products with a power of two (below
// bf16's normal range rounded once).  Scaling the bf16 pairs takes half the instructions of scaling the fp32
// values they come from: 269 -> 260 us for 128 sequences of 1024..8192 tokens.  (Moving the codes' bits into
// bf16 fields and multiplying by 2^120 measured slower, for all codes, 260 -> 283, or half of them, 269.)
template <bool kScaled>
__device__ __forceinline__ void e4m3x16_to_bf16(const uint4& c, __nv_bfloat162 mult, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const uint32_t f2 = e4m3x2_to_f16x2(static_cast<uint16_t>(w[q] >> (16 * hh)));
      const __half2 h2 = *reinterpret_cast<const __half2*>(&f2);
      __nv_bfloat162 b2 = __floats2bfloat162_rn(__low2float(h2), __high2float(h2));
      if constexpr (kScaled) b2 = __hmul2(b2, mult);
      o[2 * q + hh] = *reinterpret_cast<const uint32_t*>(&b2);
    }
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// One box: wait for its codes and scale bytes (a CTA-local barrier), then, slab by slab, read this
// thread's two chunks, meet the other converter threads and write the bf16 values into the 128-byte
// swizzled slab layout of the buffer (rows at or past `bx.valid`, and hidden ones, as zeros); last,
// publish the buffer on the even CTA's barrier `done`.  The staged codes fill the buffer's upper half,
// [slab][row][64 bytes], so slab s of the result covers codes of slabs up to s only: those of s + 1 are
// safe to read before the barrier has been passed by all.  A loop, not unrolled code: the converter
// warps would stall on instruction fetches (a tile's boxes unrolled: 2.3 times the time).  Converter
// thread ct takes piece ct & 3 of rows ct >> 2 and (ct >> 2) + 32 of every slab.  False (the same in
// every converter thread) if the wait failed or the kernel is aborting.
template <int kSlabs>
__device__ __forceinline__ bool tc_convert_box(uint8_t* buf, int codes_off, const TcBox& bx, uint64_t* raw,
                                               uint32_t parity, uint32_t done, volatile int* abort_flag, int ct,
                                               int bar_id) {
  const bool got = mbar_wait(raw, parity, 0x17) && !*abort_flag;
  if (!named_bar_red_and(bar_id, kTcConvThreads, got)) return false;
  const int pc = ct & 3;
  const int rb = ct >> 2;
  const __nv_bfloat162 m0 = e8m0_bf162(buf[rb]);
  const __nv_bfloat162 m1 = e8m0_bf162(buf[rb + 32]);
  const uint4* src = reinterpret_cast<const uint4*>(buf + codes_off) + ct;
  uint4 c0 = src[0], c1 = src[kTcConvThreads];
  const bool in0 = bx.sees(rb), in1 = bx.sees(rb + 32);
  uint8_t* dst = buf + rb * 128;   // (rb + 32) & 7 == rb & 7
  const int o0 = ((2 * pc) ^ (rb & 7)) << 4, o1 = ((2 * pc + 1) ^ (rb & 7)) << 4;
#pragma unroll 1
  for (int s = 0; s < kSlabs; ++s, dst += kTcSlab) {
    named_bar_sync(bar_id, kTcConvThreads);   // every thread holds its codes of slab s
    const uint4 x0 = c0, x1 = c1;
    if (s + 1 < kSlabs) {
      src += 2 * kTcConvThreads;
      c0 = src[0];
      c1 = src[kTcConvThreads];
    }
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    if (in0) e4m3x16_to_bf16<true>(x0, m0, lo, hi);
    *reinterpret_cast<uint4*>(dst + o0) = lo;
    *reinterpret_cast<uint4*>(dst + o1) = hi;
    lo = hi = make_uint4(0, 0, 0, 0);
    if (in1) e4m3x16_to_bf16<true>(x1, m1, lo, hi);
    *reinterpret_cast<uint4*>(dst + 32 * 128 + o0) = lo;
    *reinterpret_cast<uint4*>(dst + 32 * 128 + o1) = hi;
  }
  fence_proxy_async_smem();
  named_bar_sync(bar_id, kTcConvThreads);
  if (ct == 0) {
    fence_release_smem_to_cluster();
    mbar_arrive_relaxed(done);
  }
  return true;
}

// Four converter warps walk the K boxes (both parts of each tile), four the V boxes (both 64-token
// halves of each tile).
template <class Rows>
__device__ bool tc_convert(const DecodeTcArgs& a, const TcPlan& plan, int pair, uint8_t* smem, TcBars* bars,
                           volatile int* abort_flag) {
  const int grp = static_cast<int>(threadIdx.x) / 32 >= kTcConvWarp0 + 4;
  const int ct = static_cast<int>(threadIdx.x) - 32 * kTcConvWarp0 - grp * kTcConvThreads;
  SegmentCursor cur{plan.b0, plan.off0, plan.start, plan.end, plan.b_end, pair, true, plan.len0};
  Segment sg;
  uint32_t g = 0;
  bool ok = true;
  const Rows rows = tc_rows<Rows>(a);
  while (ok && cur.next(a.seq_lens, a.capacity, rows, sg)) {
    const auto map = rows.map(sg.len);
    for (int i = 0; ok && i < sg.n_tiles; ++i, ++g) {
      const uint32_t par = g & 1u;
      if (grp == 0) {
        const TcBox all{64, 0, 0};
        ok = tc_convert_box<kTcKSlabsA>(smem + kTcOffK, kTcFp8OffA, all, &bars->kraw[0], par, lbar(&bars->k_full[0]),
                                        abort_flag, ct, 3) &&
             tc_convert_box<kTcKSlabsB>(smem + kTcOffK + kTcKSlabsA * kTcSlab, kTcFp8OffB, all, &bars->kraw[1], par,
                                        lbar(&bars->k_full[1]), abort_flag, ct, 3);
      } else {
        for (int h = 0; ok && h < 2; ++h) {
          const TcBox bx = tc_box<Rows::kHoles>(map, sg.tok_begin + i * kTcTile + 64 * h, sg.tok_end);
          ok = tc_convert_box<4>(smem + kTcOffV + h * kTcVBox, kTcFp8OffV, bx, &bars->vraw[h], par,
                                 lbar(&bars->v_full[h]), abort_flag, ct, 4);
        }
      }
    }
  }
  return ok;
}

// Each lane holds 64 bytes (w[0..15]) of its own row r = lane of a 32-row block whose rows lie
// row_stride bytes apart from row0.  Written through a 2 KB per-warp staging buffer (16-byte
// chunks XOR-swizzled by row pair, so neither pass meets bank conflicts beyond the 4 wavefronts
// a 512-byte access needs), each global store instruction covers eight whole 64-byte row
// segments instead of 32 scattered 16-byte pieces.
__device__ __forceinline__ void store_rows_64b(uint8_t* stage, const uint32_t* w, uint8_t* row0, size_t row_stride,
                                               int lane) {
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 4; ++c)
    *reinterpret_cast<uint4*>(stage + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = 8 * j + (lane >> 2);
    const int c = lane & 3;
    const uint4 v = *reinterpret_cast<const uint4*>(stage + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
    *reinterpret_cast<uint4*>(row0 + row * row_stride + c * 16) = v;
  }
}

// ------------------------------------------------------------------------------ softmax warps
// L2 prefetch of the K rows the producer will copy kTcPfDist tiles later.  A K copy is issued only
// once QK^T has released the slot it refills (a single K slot per part), so its HBM latency sits
// on the critical loop; with the rows already in L2 it shrinks to the L2 latency.  The softmax
// warps issue the prefetches: this CTA's 64 rows of the tile are one contiguous 72 KB run, 576 lines
// over 256 threads, once per tile.  Contiguous caches only.  (Bulk prefetches by the K producer, for
// both layouts: 74 x 2048 in pages 55.5 -> 53.8 us, but 4 x 131072 contiguous 158 -> 166 us and 128 mixed
// lengths in pages 194 -> 200 us.)
constexpr int kTcPfDist = 2;
template <bool kMapped, class Map>
__device__ __forceinline__ void tc_prefetch_tile(const DecodeTcArgs& a, const Map& map, int b, int tok0, int t_end) {
  if (tok0 >= t_end || a.v.page_size != 0) return;
  const int cb = tc_cache_seq<kMapped>(a, b, false);   // b is the query row
  if (kMapped && cb < 0) return;
  const int64_t r = cache_row(a.v, cb, map.real(tok0));
  if (r < 0) return;
  int n = min(64, t_end - tok0);
  if (a.v.num_rows - r < n) n = static_cast<int>(a.v.num_rows - r);   // rows of the buffer only
  const uint8_t* base = a.cache + r * a.row_bytes;
  const int lines = (n * a.row_bytes + 127) / 128;
  for (int L = threadIdx.x; L < lines; L += 32 * kTcSoftmaxWarps)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(base + 128 * L));
}

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Eight warps: warp w reads TMEM lane quadrant w % 4 and column half ch = w / 4, so thread
// (t = TMEM lane, ch) owns head 64*rank + (t & 63), the 32 tokens 64*(t >> 6) + 32*ch + [0, 32)
// of every tile, and O columns [128*ch, 128*ch + 128) of its lane (latent 256*ch + 128*(t >> 6)
// + [0, 128)).  The four threads (t, ch), (t ^ 64, ch), (t, ch ^ 1), (t ^ 64, ch ^ 1) share a
// head and exchange tile maxima and row sums through shared memory.
// Writes one segment's output for the head of this thread's TMEM lane: when the segment covers its
// sequence, O from TMEM divided by l_tot as bf16 into the head's output row `row` and its lse into
// *m_or_lse (if not null); else the unnormalised fp32 partial into the workspace row `row` with m
// and l into *m_or_lse and *l_out.  Kept out of line (it runs once per segment and its registers
// would otherwise crowd the per-tile loop) and given plain pointers, so that no argument struct
// has to be copied to the stack for it.
__device__ __noinline__ void tc_write_segment(bool direct, void* row, float* m_or_lse, float* l_out, uint8_t* smem,
                                              uint32_t tmem, float m_used, float l_tot) {
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int ch = warp >> 2;
  const int t = 32 * (warp & 3) + lane;
  const int half = t >> 6;
  const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  const int lat0 = 256 * ch + 128 * half;
  const uint32_t ocol = tmem + lane_base + kTcColO + 128 * ch;
  // PV has read the segment's last P (o_final), and the next P is written by these warps after
  // their next barrier: the P buffer gives 2 KB of staging per warp.
  uint8_t* stage = smem + kTcOffP + warp * 2048;
  if (direct) {
    const float inv = l_tot > 0.f ? 1.f / l_tot : 0.f;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(row) + lat0;
    uint8_t* row0 = reinterpret_cast<uint8_t*>(dst) - static_cast<size_t>(lane) * kDLat * 2;
    // A loop of small bodies, 32 latent columns (64 bytes of bf16) each: the code is cold at every segment.
#pragma unroll 1
    for (int qb = 0; qb < 4; ++qb) {
      uint32_t r[2][16];
#pragma unroll
      for (int q = 0; q < 2; ++q) tmem_ld16(ocol + 32 * qb + 16 * q, r[q]);
      tmem_ld_wait();
      uint32_t w[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        __nv_bfloat162 h2 = __floats2bfloat162_rn(__uint_as_float(r[e >> 3][2 * (e & 7)]) * inv,
                                                  __uint_as_float(r[e >> 3][2 * (e & 7) + 1]) * inv);
        w[e] = *reinterpret_cast<uint32_t*>(&h2);
      }
      store_rows_64b(stage, w, row0 + 64 * qb, static_cast<size_t>(kDLat) * 2, lane);
    }
    if (half == 0 && ch == 0 && m_or_lse != nullptr)
      *m_or_lse = l_tot > 0.f ? (m_used + log2f(l_tot)) * kLn2 : -INFINITY;
  } else {
    float* dst = static_cast<float*>(row) + lat0;
    uint8_t* row0 = reinterpret_cast<uint8_t*>(dst) - static_cast<size_t>(lane) * kDLat * 4;
#pragma unroll 1
    for (int qb = 0; qb < 8; ++qb) {   // 16 latent columns (64 bytes of fp32) each
      uint32_t w[16];
      tmem_ld16(ocol + 16 * qb, w);
      tmem_ld_wait();
      store_rows_64b(stage, w, row0 + 64 * qb, static_cast<size_t>(kDLat) * 4, lane);
    }
    if (half == 0 && ch == 0) {
      *m_or_lse = m_used;
      *l_out = l_tot;
    }
  }
}

// O row slice *= alpha (128 fp32 columns of this thread's TMEM lane from addr).  Out of line: the
// lazy rescale runs on few tiles, and the per-tile loop stays compact.
__device__ __noinline__ void tc_rescale_o(uint32_t addr, float alpha) {
  for (int qb = 0; qb < 4; ++qb, addr += 32) {   // 2 TMEM loads in flight per wait
    uint32_t r[2][16];
#pragma unroll
    for (int k = 0; k < 2; ++k) tmem_ld16(addr + 16 * k, r[k]);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int e = 0; e < 16; ++e) r[k][e] = __float_as_uint(__uint_as_float(r[k][e]) * alpha);
      tmem_st16(addr + 16 * k, r[k]);
    }
  }
  tmem_st_wait();
}

// How a softmax warp leaves whose bounded wait ran out.  The eight warps do not give up together (some waits
// are those of some warps only, and the limit runs out at its own time in each), and the others still meet
// at named barriers: it passes all of these, without further waits, arrivals or output.  They are
// `pending` in the current tile, one in each later tile of the segment (`tiles`), two more where a segment
// follows another, and the last epilogue's.
template <class Rows>
__device__ __noinline__ void tc_softmax_leave(SegmentCursor cur, const int32_t* seq_lens, int capacity, const Rows rows,
                                              int pending, int tiles, volatile int* abort_flag) {
  *abort_flag = 1;
  Segment sg;
  int left = pending + tiles + 1;
  while (cur.next(seq_lens, capacity, rows, sg)) left += 2 + sg.n_tiles;
  for (; left > 0; --left) named_bar_sync(1, 256);
}

template <bool kMapped, class Rows>
__device__ void tc_softmax(const DecodeTcArgs& a, const TcPlan& plan, int pair, uint8_t* smem, TcBars* bars,
                           float* red, uint32_t tmem, uint32_t rank, volatile int* abort_flag) {
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int ch = warp >> 2;
  const int t = 32 * (warp & 3) + lane;   // TMEM lane
  const int hl = t & 63;                  // head within this CTA
  const int half = t >> 6;                // token half of a tile / latent quarter of O
  const int me = ch * 128 + t;            // slot in the exchange arrays
  const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  SegmentCursor cur{plan.b0, plan.off0, plan.start, plan.end, plan.b_end, pair, true, plan.len0};
  Segment sg;
  int g = 0;   // global tile index of the range
  int k = 0;   // segment index
  const Rows rows = tc_rows<Rows>(a);
  auto wait = [&](uint64_t* bar, int n, uint32_t site) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, static_cast<uint32_t>(n) & 1u, site));
  };
  auto leave = [&](int pending, int tiles) {
    tc_softmax_leave(cur, a.seq_lens, a.capacity, rows, pending, tiles, abort_flag);
  };
  // The segment whose tiles are done but whose O has not been read.  Its epilogue runs once the next
  // segment's first P is in registers, so that the wait for the last PV overlaps that softmax.
  struct {
    int b, slot;
    bool direct;
    float m, l;
  } done = {};
  // rl: the sums exchange (a maxima buffer not in use).  False, before its barrier, if the wait ran out.
  auto epilogue = [&](int kd, float* rl) -> bool {
    if (!wait(&bars->o_final, kd, 0x33)) return false;
    tc_fence_after();
    rl[me] = done.l;
    named_bar_sync(1, 256);
    const float l_tot = (done.l + rl[me ^ 64]) + (rl[me ^ 128] + rl[me ^ 192]);
    if (__all_sync(0xffffffffu, !*abort_flag)) {   // (the same for the whole warp)
      const int64_t h = 64 * static_cast<int>(rank) + hl;
      if (done.direct) {
        const int64_t bh = static_cast<int64_t>(done.b) * kHeads + h;
        tc_write_segment(true, a.out_lat + bh * kDLat, a.lse != nullptr ? a.lse + bh : nullptr, nullptr, smem, tmem,
                         done.m, l_tot);
      } else {
        const int64_t ml = static_cast<int64_t>(done.slot) * kHeads + h;
        tc_write_segment(false, a.ws.o + ml * kDLat, a.ws.m + ml, a.ws.l + ml, smem, tmem, done.m, l_tot);
      }
    }
    return true;
  };
  bool more = cur.next(a.seq_lens, a.capacity, rows, sg);
  while (more) {
  const auto map = rows.map(sg.len);
  const int t_begin = sg.tok_begin, t_end = sg.tok_end, n_tiles = sg.n_tiles;
  float m_used = -INFINITY;
  float l_run = 0.f;
  for (int d = 1; d < kTcPfDist && d < n_tiles; ++d)
    tc_prefetch_tile<kMapped>(a, map, sg.b, t_begin + d * kTcTile + 64 * static_cast<int>(rank), t_end);
  for (int i = 0; i < n_tiles; ++i, ++g) {
    const int j = g & 1;
    if (!wait(&bars->s_full[j], g >> 1, 0x30)) return leave(i == 0 && k > 0 ? 3 : 1, n_tiles - i - 1);
    tc_fence_after();
    float sc[32];
    {
      uint32_t ra[2][16];
#pragma unroll
      for (int q = 0; q < 2; ++q) tmem_ld16(tmem + lane_base + kTcColS + 64 * j + 32 * ch + 16 * q, ra[q]);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 32; ++e) sc[e] = __uint_as_float(ra[e >> 4][e & 15]);
    }
    // S is in registers (tcgen05.wait::ld above): its TMEM buffer may take tile i + 2.  The
    // arrival orders nothing else, so it is relaxed.
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_relaxed(lbar(&bars->s_empty[j]));
    // Tokens at or past the split end (only in a ragged last tile) get a score of -inf.
    const int tok0 = t_begin + i * kTcTile + 64 * half + 32 * ch;
    const int nvalid = t_end - tok0;
    if (nvalid < 32) {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (e >= nvalid) sc[e] = -INFINITY;
    }
    if constexpr (Rows::kHoles) {   // tokens hidden behind the window
      const int r0 = map.real(tok0);
      const int lo = map.hole0() - r0, hi = map.hole1() - r0;
      if (lo < 32 && hi > 0) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (e >= lo && e < hi) sc[e] = -INFINITY;
      }
    }
    float mloc = sc[0];
#pragma unroll
    for (int e = 1; e < 32; ++e) mloc = fmaxf(mloc, sc[e]);
    mloc *= a.scale_log2;   // scale > 0, so the max commutes with the scaling
    float* rm = red + j * 256;
    rm[me] = mloc;
    named_bar_sync(1, 256);
    const float m_tile = fmaxf(fmaxf(mloc, rm[me ^ 64]), fmaxf(rm[me ^ 128], rm[me ^ 192]));
    float alpha = 1.f;
    bool need = false;
    if (m_used == -INFINITY) {
      m_used = m_tile;
      alpha = 0.f;
    } else if (m_tile > m_used + kTcRescaleThreshold) {
      alpha = ex2_approx(m_used - m_tile);
      m_used = m_tile;
      need = true;
    }
    if (__any_sync(0xffffffffu, need)) {
      // O must hold PV(g-1) before it is scaled (g-1 is in this segment: the first tile of a
      // segment never rescales).  Waiting on phase g-1 by parity is unambiguous: PV(g-2) is done (in
      // tile g-1 the second half's warps waited for all of it, p_empty[1], and every warp has met them at
      // this tile's named barrier) and PV(g) needs this tile's P, so o_ready has completed g-1 or g phases.
      if (!wait(&bars->o_ready, g - 1, 0x31)) return leave(0, n_tiles - i - 1);
      tc_fence_after();
      tc_rescale_o(tmem + lane_base + kTcColO + 128 * ch, alpha);
    }
    // P for this tile, packed to bf16 in registers before the buffer is known to be free.  PV's operands are
    // both bf16 (an fp16 P would need the rows in fp16, whose range they may leave), so each weight is
    // rounded by at most 2^-8 of itself; l sums the unrounded ones, in fp32.  Output against 64 bits: off by
    // 0.0019-0.0025 of its norm, where rounding the output to bf16 alone gives 0.0017.
    const float neg_m = -m_used;
    float psum = 0.f;
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float p0 = ex2_approx(fmaf(sc[2 * e], a.scale_log2, neg_m));
      const float p1 = ex2_approx(fmaf(sc[2 * e + 1], a.scale_log2, neg_m));
      psum += p0 + p1;
      __nv_bfloat162 h2 = __floats2bfloat162_rn(p0, p1);
      pk[e] = *reinterpret_cast<uint32_t*>(&h2);
    }
    // A half of the P buffer is free once PV(g-1) has read it.  By parity this is unambiguous: both halves'
    // warps waited in tile g-1 for their half of PV(g-2), so p_empty has completed g-1 or g phases.  PV of
    // the first half needs O corrected by every warp, so the second half's warps arrive for it too, without
    // waiting for their own half (but for the first one's: no arrival for tile g before PV(g-1) has taken
    // all of tile g-1).
    // Between segments the epilogue waits for more (all of PV), reads O and stages it through the P
    // buffer; the barrier then lets every warp write P, and PV (the even CTA) learns that O may be
    // overwritten.
    if (i == 0 && k > 0) {
      if (!epilogue(k - 1, red + (j ^ 1) * 256)) return leave(2, n_tiles - i - 1);
      tc_fence_before();
      named_bar_sync(1, 256);
      if (lane == 0) {
        fence_release_smem_to_cluster();
        mbar_arrive_relaxed(lbar(&bars->o_free));
      }
    } else if (g >= 1 && !wait(&bars->p_empty[0], g - 1, 0x32)) {
      return leave(0, n_tiles - i - 1);
    }
    if (half == 1) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(lbar(&bars->p_full[0]));
      if (g >= 1 && !wait(&bars->p_empty[1], g - 1, 0x34)) return leave(0, n_tiles - i - 1);
    }
    uint8_t* prow = smem + kTcOffP + half * kTcSlab + hl * 128;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int unit = 4 * ch + u;   // 16-byte unit (8 tokens) within the 128-byte row
      *reinterpret_cast<uint4*>(prow + ((unit ^ (hl & 7)) << 4)) =
          make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
    }
    l_run = l_run * alpha + psum;
    // Publish: P (generic-proxy writes) made visible to the tensor core, the O correction's
    // tcgen05.st ordered before the thread sync, then one release of the warp's shared-memory
    // writes (restricted to shared memory: P is all that PV reads from this thread's work)
    // followed by a relaxed arrival on the even CTA's barrier.
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      fence_release_smem_to_cluster();
      mbar_arrive_relaxed(lbar(&bars->p_full[half]));
    }
    if (i + kTcPfDist < n_tiles)
      tc_prefetch_tile<kMapped>(a, map, sg.b, t_begin + (i + kTcPfDist) * kTcTile + 64 * static_cast<int>(rank), t_end);
  }
  done.b = sg.b;
  done.slot = sg.slot;
  done.direct = sg.direct;
  done.m = m_used;
  done.l = l_run;
  ++k;
  more = cur.next(a.seq_lens, a.capacity, rows, sg);
  }
  if (k > 0 && !epilogue(k - 1, red + (g & 1) * 256)) leave(0, 0);   // (the buffer the last tile did not use)
}

// A call of one range has no split rows.  One of a few rows is not followed by a combine, and its empty
// rows are written here (each takes the pair about 1 us; a launch takes two).
constexpr int kTcOwnEmptyRows = 2;
template <class Rows>
__device__ void tc_empty_rows(const DecodeTcArgs& a, uint32_t rank) {
  const Rows rows = tc_rows<Rows>(a);
  for (int b = 0; b < a.batch; ++b) {
    if (rows.span(seq_len_checked(a.seq_lens, b, a.capacity)) != 0) continue;
    const int64_t row = static_cast<int64_t>(b) * kHeads + 64 * static_cast<int>(rank);
    for (int i = threadIdx.x; i < 64 * kDLat / 8; i += 32 * kTcSoftmaxWarps)
      reinterpret_cast<uint4*>(a.out_lat + row * kDLat)[i] = make_uint4(0, 0, 0, 0);
    if (a.lse != nullptr && threadIdx.x < 64) a.lse[row + threadIdx.x] = -INFINITY;
  }
}

// ------------------------------------------------------------------------------ work plan
// One warp computes the plan; every CTA computes it for itself (it only reads seq_lens), and the
// even CTA of range 0 also writes the table the combine reads (balanced: the cost prefix of each
// sequence and the total cost; per sequence: the first range of each and the ranges used).  Lane l
// walks the contiguous chunk of sequences [l per, (l + 1) per): three passes over it (tile totals,
// the smallest and largest sequence and the non-empty count; per-chunk sums of the prefix counts
// and, balanced, of the costs; the prefixes themselves, the table and this pair's piece), with warp
// reductions or scans between passes.  Every lane returns the same plan.  For batches of up to 128
// sequences (per <= 4) the lane's tile counts are formed once, all loads in flight together, and kept
// in registers for the three passes; for larger ones all warps have put them into shared memory before
// (tc_plan_tiles: setup and plan of 1024 rows 14.6 -> 8.1 us).
constexpr int kTcPlanCached = 4;
// Where the tile count of sequence bb lies: sequence u of lane l's chunk at [u][l], so that the lanes
// of the plan's warp read different banks.  In the Q, P and K buffers, which no copy has touched yet.
__device__ __forceinline__ int tc_plan_slot(int bb, int per) { return bb % per * 32 + bb / per; }
static_assert((kMaxDecodeBatch + 31) / 32 * 32 * 4 <= kTcOffBar, "the tile counts fit in front of the barriers");
template <class Rows>
__device__ void tc_plan_tiles(const int32_t* seq_lens, int capacity, const Rows rows, int B, int* tiles) {
  const int per = (B + 31) / 32;
  for (int bb = threadIdx.x; bb < B; bb += blockDim.x)
    tiles[tc_plan_slot(bb, per)] = tiles_of(rows.span(seq_len_checked(seq_lens, bb, capacity)));
  fence_proxy_async_smem();   // before the copies that later overwrite them
}
template <class Rows>
__device__ __noinline__ TcPlan tc_make_plan(const int32_t* seq_lens, int capacity, const Rows rows, int B, int P,
                                               int32_t* table, int pair, bool write_table, const int* tiles) {
  const int lane = threadIdx.x & 31;
  const int per = (B + 31) / 32;
  const int lo = min(B, lane * per), hi = min(B, lo + per);
  const bool cached = per <= kTcPlanCached;
  int held[kTcPlanCached];
#pragma unroll
  for (int u = 0; u < kTcPlanCached; ++u)
    held[u] = (cached && lo + u < hi) ? tiles_of(rows.span(seq_len_checked(seq_lens, lo + u, capacity))) : 0;
  // fn(bb, t) for every sequence bb of this lane's chunk, in order, with its tile count t
  auto for_chunk = [&](auto&& fn) {
    if (cached) {
#pragma unroll
      for (int u = 0; u < kTcPlanCached; ++u)
        if (lo + u < hi) fn(lo + u, held[u]);
    } else {
#pragma unroll 4
      for (int bb = lo; bb < hi; ++bb) fn(bb, tiles[(bb - lo) * 32 + lane]);
    }
  };
  // pass 1: total tiles T, the smallest non-empty sequence, the largest, the non-empty count
  int sum = 0, mn = INT_MAX, mx = 0, nne = 0;
  for_chunk([&](int, int t) {
    sum += t;
    mx = max(mx, t);
    if (t > 0) {
      mn = min(mn, t);
      ++nne;
    }
  });
  const int T = __reduce_add_sync(0xffffffffu, sum);
  mn = __reduce_min_sync(0xffffffffu, mn);
  mx = __reduce_max_sync(0xffffffffu, mx);
  const bool per_seq = T > 0 && static_cast<int64_t>(mn) * P >= T;
  if (per_seq && mx == mn && static_cast<int64_t>(mn) * B == T) {
    // Every sequence has the same tile count t (the usual case): r_b = floor(P t / (B t)) =
    // floor(P / B) for all b, so the prefix is b r and no scan is needed.  Same plan as below.
    const int t = mn;
    const int r = min(P / B, t);
    if (write_table) {
      #pragma unroll 1
      for (int bb = lo; bb < hi; ++bb) table[bb] = bb * r;
      if (lane == 0) {
        table[B] = B * r;
        table[B + 1] = kPlanPerSequence;
      }
    }
    TcPlan pl;
    pl.start = pl.end = 0;
    pl.b0 = pl.off0 = pl.b_end = pl.len0 = 0;
    const int b0 = pair / r, jj = pair - b0 * r;
    if (b0 < B) {
      pl.b0 = b0;
      pl.len0 = seq_len_checked(seq_lens, b0, capacity);
      pl.start = muldiv(jj, t, r);
      pl.end = muldiv(jj + 1, t, r);
      pl.b_end = b0 + 1;
    }
    return pl;
  }
  // what each sequence contributes to the prefix: its tiles, or (per sequence) its ranges
  // r_b = floor(P tiles_b / T), which the condition makes >= 1 and which is at most tiles_b
  auto count_of = [&](int t) -> int {
    if (!per_seq || t == 0) return t;
    const int r = muldiv(P, t, T);
    return r < t ? r : t;
  };
  // pass 2: this lane's share of the prefix, and (balanced) of the cost line
  int csum = sum;
  if (per_seq) {
    csum = 0;
    for_chunk([&](int, int t) { csum += count_of(t); });
  }
  const int wsum = sum + kSegCost * nne;
  int incl = csum, wincl = wsum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, d);
    const int uw = __shfl_up_sync(0xffffffffu, wincl, d);
    if (lane >= d) {
      incl += u;
      wincl += uw;
    }
  }
  const int total = __shfl_sync(0xffffffffu, incl, 31);
  const int C = __shfl_sync(0xffffffffu, wincl, 31);
  // pass 3: the prefixes, the table, and the piece of this pair.  Balanced: the range's cost
  // interval [x0, x1) of the cost line; the lane whose sequence span holds x0 finds the start
  // (and the first sequence), the one whose span holds x1 the end (none: x1 = C, the end is T).
  const int x0 = (T > 0 && !per_seq) ? muldiv(pair, C, P) : 0;
  const int x1 = (T > 0 && !per_seq) ? muldiv(pair + 1, C, P) : 0;
  TcPlan pl;
  pl.start = pl.end = 0;
  pl.b0 = pl.off0 = pl.b_end = pl.len0 = 0;
  bool found_start = false, found_end = false;
  int run = incl - csum;
  int W = wincl - wsum;
  for_chunk([&](int bb, int t) {
    const int v = count_of(t);
    if (write_table) table[bb] = per_seq ? run : W;
    if (per_seq) {
      if (v > 0 && run <= pair && pair < run + v) {
        const int jj = pair - run;
        pl.b0 = bb;
        pl.start = muldiv(jj, t, v);
        pl.end = muldiv(jj + 1, t, v);
        pl.b_end = bb + 1;
        found_start = found_end = true;
      }
    } else if (t > 0) {
      if (W <= x0 && x0 < W + kSegCost + t) {
        pl.b0 = bb;
        pl.off0 = run;
        pl.start = run + max(0, x0 - W - kSegCost);
        pl.b_end = B;
        found_start = true;
      }
      if (W <= x1 && x1 < W + kSegCost + t) {
        pl.end = run + max(0, x1 - W - kSegCost);
        found_end = true;
      }
      W += kSegCost + t;
    }
    run += v;
  });
  if (write_table && lane == 0) {
    table[B] = per_seq ? total : C;
    table[B + 1] = per_seq ? kPlanPerSequence : kPlanBalanced;
  }
  // the lanes that found the start and the end (at most one each) hand them to the warp;
  // otherwise the pair is idle (or, balanced, its range ends at T)
  const unsigned fs = __ballot_sync(0xffffffffu, found_start);
  const unsigned fe = __ballot_sync(0xffffffffu, found_end);
  const int ss = fs ? __ffs(fs) - 1 : 0;
  const int se = fe ? __ffs(fe) - 1 : 0;
  TcPlan r;
  r.start = __shfl_sync(0xffffffffu, pl.start, ss);
  r.end = __shfl_sync(0xffffffffu, pl.end, se);
  r.b0 = __shfl_sync(0xffffffffu, pl.b0, ss);
  r.off0 = __shfl_sync(0xffffffffu, pl.off0, ss);
  r.b_end = __shfl_sync(0xffffffffu, pl.b_end, ss);
  r.len0 = T > 0 ? seq_len_checked(seq_lens, r.b0, capacity) : 0;
  if (!per_seq) {
    if (!fe) r.end = T;
    if (!fs) r.start = r.end = 0;   // no tiles at all (T = 0)
  } else if (!fs) {
    r.start = r.end = 0;
  }
  return r;
}

// ------------------------------------------------------------------------------ kernel
// grid = 2 * P CTAs, clusters of 2 along x: blockIdx.x = 2 * pair + rank.  kMapped: query rows
// read the cache sequences of a.seq_map (chunked prefill); the decode instance carries none of it.
// kFp8: the cache holds E4M3 codes with E8M0 row scales (tm_ka, tm_kb, tm_v are byte maps of the
// codes, tm_sc the 1-D byte map of the scales; unused otherwise).  Rows: what a query row attends to
// (FullRows, or WindowRows for the sliding window with sinks).
template <bool kMapped, bool kFp8 = false, class Rows = FullRows>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(tc_threads(kFp8), 1)
    decode_tc_kernel(const __grid_constant__ CUtensorMap tm_ka, const __grid_constant__ CUtensorMap tm_kb,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_sc, const DecodeTcArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  TcBars* bars = reinterpret_cast<TcBars*>(smem + kTcOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kTcOffMisc);
  int* abort_flag = reinterpret_cast<int*>(smem + kTcOffMisc + 16);
  TcPlan* plan = reinterpret_cast<TcPlan*>(smem + kTcOffMisc + 32);
  float* red = reinterpret_cast<float*>(smem + kTcOffMisc + 64);   // [2][256] tile maxima, reused for sums

  // The 128-byte swizzle atoms need a 1024-byte aligned base; the layout above has no slack for
  // realigning, so a misaligned base is reported instead of used (every CTA sees the same base).
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) set_dev_error(0x8);
    return;
  }
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1;
  const int warp = threadIdx.x >> 5;
  // Setup that touches no global memory overlaps the previous kernel in the stream.
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int part = 0; part < 2; ++part) {
      mbar_init(&bars->k_full[part], 2);   // one arrival per CTA of the pair (plus the copies' bytes)
      mbar_init(&bars->k_empty[part], 1);
    }
    for (int s = 0; s < kTcVSlots; ++s) {
      mbar_init(&bars->v_full[s], 2);   // one arrival per CTA of the pair (plus the copies' bytes)
      mbar_init(&bars->v_empty[s], 1);
      mbar_init(&bars->fix[s], 1);
    }
    mbar_init(&bars->s_full[0], 1);
    mbar_init(&bars->s_full[1], 1);
    mbar_init(&bars->s_empty[0], 2 * kTcSoftmaxWarps);   // every softmax warp of both CTAs
    mbar_init(&bars->s_empty[1], 2 * kTcSoftmaxWarps);
    mbar_init(&bars->p_full[0], 2 * kTcSoftmaxWarps);   // every softmax warp of both CTAs
    mbar_init(&bars->p_full[1], kTcSoftmaxWarps);       // those of the second token half
    mbar_init(&bars->p_empty[0], 1);
    mbar_init(&bars->p_empty[1], 1);
    mbar_init(&bars->o_ready, 1);
    mbar_init(&bars->o_final, 1);
    mbar_init(&bars->o_free, 2 * kTcSoftmaxWarps);   // every softmax warp of both CTAs
    mbar_init(&bars->q_full, 2);
    mbar_init(&bars->q_empty, 1);
    if (kFp8) {
      for (int part = 0; part < 2; ++part) mbar_init(&bars->kraw[part], 1);   // this CTA's producer (plus bytes)
      for (int s = 0; s < kTcVSlots; ++s) mbar_init(&bars->vraw[s], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kTcMmaWarp) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  if (warp == kTcProducerWarp && (threadIdx.x & 31) == 0) {
    tma_prefetch_desc(&tm_ka);
    tma_prefetch_desc(&tm_kb);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_q);
    if (kFp8) tma_prefetch_desc(&tm_sc);
  }
  // The barrier inits and the TMEM allocation reach the peer CTA through the cluster barrier, whose
  // wait comes after the plan.
  tc_fence_before();
  cluster_arrive_release();
  // seq_lens (read by the plan) may come from the previous kernel.
  pdl_wait();
  // The producer warp computes the plan and hands it to the other warps through named barrier 2
  // (it only arrives, so its first copies need not wait for them).
  int* tiles = reinterpret_cast<int*>(smem);
  if (a.batch > 32 * kTcPlanCached) {
    tc_plan_tiles(a.seq_lens, a.capacity, tc_rows<Rows>(a), a.batch, tiles);
    __syncthreads();
  }
  if (warp == kTcProducerWarp) {
    const TcPlan w = tc_make_plan(a.seq_lens, a.capacity, tc_rows<Rows>(a), a.batch, a.P, a.ws.off, pair,
                                  pair == 0 && rank == 0, tiles);
    fence_proxy_async_smem();   // the tile counts have been read; copies may overwrite them
    if ((threadIdx.x & 31) == 0) *plan = w;
    __syncwarp();
    named_bar_arrive(2, tc_threads(kFp8));
  } else {
    named_bar_sync(2, tc_threads(kFp8));
  }
  cluster_wait_acquire();
  tc_fence_after();
  const TcPlan pl = *plan;
  const bool busy = pl.start < pl.end;   // the same in both CTAs of the pair
  const uint32_t tmem = *tmem_slot;

  if (warp < kTcSoftmaxWarps && a.P == 1 && a.batch <= kTcOwnEmptyRows) tc_empty_rows<Rows>(a, rank);
  if (!busy) {
    // an idle range: only the teardown below
  } else if (warp < kTcSoftmaxWarps) {
    tc_softmax<kMapped, Rows>(a, pl, pair, smem, bars, red, tmem, rank, abort_flag);
  } else if (warp == kTcProducerWarp || warp == kTcVProducerWarp) {
    const bool ok = warp == kTcProducerWarp
                        ? tc_producer<false, kMapped, kFp8, Rows>(&tm_ka, &tm_kb, &tm_v, &tm_q, &tm_sc, a, pl, smem,
                                                                  bars, rank, pair, abort_flag)
                        : tc_producer<true, kMapped, kFp8, Rows>(&tm_ka, &tm_kb, &tm_v, &tm_q, &tm_sc, a, pl, smem,
                                                                 bars, rank, pair, abort_flag);
    if (!ok && (threadIdx.x & 31) == 0) *abort_flag = 1;
  } else if (kFp8 && warp >= kTcConvWarp0) {
    if (!tc_convert<Rows>(a, pl, pair, smem, bars, abort_flag) && (threadIdx.x & 127) == 0) *abort_flag = 1;
  } else if (rank == 0 && elect_one()) {
    const SegmentCursor cur{pl.b0, pl.off0, pl.start, pl.end, pl.b_end, pair, true, pl.len0};
    const bool ok = warp == kTcMmaWarp
                        ? tc_mma_qk(smem, bars, tmem, a.seq_lens, a.capacity, tc_rows<Rows>(a), cur, abort_flag)
                        : tc_mma_pv(smem, bars, tmem, a.seq_lens, a.capacity, tc_rows<Rows>(a), cur, abort_flag);
    if (!ok) *abort_flag = 1;
  }
  __syncwarp();
  if (*reinterpret_cast<volatile int*>(abort_flag)) __nanosleep(200000);  // let stray copies land
  tc_fence_before();
  __syncwarp();
  cluster_sync();
  if (warp == kTcMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace mla
