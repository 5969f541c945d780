// paged_fwd.cuh -- attention of ragged chunks of new tokens over a paged KV
// cache, on tcgen05 (see paged.cuh for the formula).
//
// Long chunks are bound by the tensor cores and single tokens by the bytes of
// their cache; both come in one batch, so one kernel serves both.  Warps 0-7
// are the softmax and epilogue of two 128-row query tiles (a thread per row: scores from
// TMEM, running maximum and sum in fp32, P back to TMEM as bf16, O rescaled only where the
// maximum has grown by kRescaleThreshold), warps 8 and 10 the tiles' MMA issuers, warp 9
// the K/V producer and scheduler, warp 11 the Q loader.  What differs from the
// contiguous forward of prefill.cuh:
//   * A query tile packs the query heads of one KV head: row r of 128 is token
//     r / hc, head r mod hc of the hc <= 128 heads (all of the group where it
//     fits).  K/V are loaded once for the whole group, and a chunk of n tokens
//     fills its tiles with n * hc rows: 32 tokens of 4 heads are a full tile.
//   * A unit is two such tiles that share every K/V tile.  A unit with rows in
//     one tile only (a chunk's end) is thin: both tiles hold the same rows and
//     take key tiles in turn, so the two softmax chains still overlap, and the
//     unit's two results are merged in the epilogue (the second one's output is
//     read from its own TMEM columns).
//   * All units' keys form a line, in the order (sequence, KV head, unit), cut
//     into equal shares, one per CTA (one CTA per SM); a share may begin and end
//     inside a unit.  A key's weight depends on the unit's kind, and a unit has
//     a fixed weight besides.  A unit's visible keys are linear in its index, so
//     sums over a sequence's units are closed forms and every CTA finds its
//     place from the lengths on the device.  A unit that crosses shares leaves
//     one fp32 partial per CTA (two per CTA at most), which a second kernel, a
//     programmatic dependent, joins in share order.
//   * Cuts cost: partials, a piece more per CTA and the join, 14 us in all (d = 128).  Where
//     whole units balance as well or nearly (up to kPfRounds units a CTA, dealt in
//     the order of their weights there and back), they stay whole.
//   * What a sequence leaves behind its full units is the decode's work where it
//     is no more than kRowUnit rows (a single token of up to 16 heads): a 128-row
//     tile would load the same bytes at a lower rate.  These rows form a line of
//     their own, and the grid's last CTAs, in the proportion of the two lines'
//     times, each run as two of the decode kernel's CTAs (paged_decode.cuh): the
//     bytes stream while the other SMs multiply.  Launched in clusters of two CTAs,
//     which are neighbouring SMs, and both do the same kind of work: two SMs side by
//     side that ran units and rows each took a third longer (118 us where pairs of one
//     kind took 91, for 498 single tokens beside two chunks of 500).
//   * K/V tiles of 128 keys arrive as one TMA copy per page (or 128 rows of it)
//     and 64 columns; the producer's lanes issue them side by side, each with
//     the table entry it read one tile ahead.  Keys behind the last page read as
//     zeros (a page index behind the map's end).  The last page's rows behind
//     the last key hold anything, and 0 times infinity or NaN is NaN, so warp 11
//     zeroes them in V's last tile before the MMAs may read it.
// Measured on B200 (d = 128, 32 / 8 heads): a 16384-token prompt 2.01 ms = 1095
// TFLOP/s at full clocks (the contiguous forward: 1.83) and 2.2 in long runs under the
// power cap, 129 tokens behind 32639 keys 93 to 103 us = 740 to 670 TFLOP/s, a
// 2000-token chunk with 40 single tokens 72 to 74 us, five prompts of 3 to 150
// tokens 12.1 us.  A key step of a pair takes 2.1 us for
// 1.1 us of tensor work: the softmax chain of one row per thread bounds it, as in
// prefill.cuh.  The weights: at full clocks a step of 128 keys takes 2.1 us in a
// pair and 1.7 us in a thin unit (its ring of five slots covers one copy's latency
// per two tiles), a unit 3.2 us besides (first S, last P.V, stores).  They are
// d = 128's, and d = 64 uses them: there a pair's step takes 2.05 us, a thin unit's
// 1.0 (eight slots), so thin units end early beside pairs.
#pragma once
#include "paged_decode.cuh"
#include "piece_steps.h"
#include "prefill.cuh"

namespace sdpa {

// Weights on the line, in proportion to the times above.
constexpr int kPfPair = 8, kPfThin = 6;   // per key
constexpr int kPfUnitCost = 1600;
constexpr float kPfRowPlace = 165.f;      // a place on the rows' line: 0.34 us of an SM
// Units of this many key tiles or fewer are not split: joining costs more.
constexpr int kPfWholePair = 2, kPfWholeThin = 4;
constexpr int kPfRing = 4;         // pieces announced ahead
constexpr int kPfQWarp = 11;     // loads Q; cleans V's last tile
// Whole units are dealt where that leaves the last CTA at most this much behind a share.  Both sides measured, in us
// (d = 128): a prompt of 1300 tokens, 32 / 8 heads, 34.2 whole, 41.3 cut; 2000 tokens of 32 heads without sharing 54.0
// and 67.1; 25 chunks of 185 to 555 tokens, 16 / 2 heads, 79.6 and 88.7; 1024 tokens (4600 behind a share) 29.4 and
// 34.1; the other way round 256 tokens after 1000 (8300 behind) 33.2 and 24.1, 2000 tokens of 16 / 2 heads (9500
// behind) 48.1 and 42.6.  Whole is better up to 4650 places behind (900 tokens, 31.0 and 32.8), cut from 8100 on (3000
// tokens, 16 / 2 heads, 66.9 and 64.0).  d = 64, half the bytes a partial, uses the same limit and is better off cut
// from about 4300 on: 1300 tokens (3800 behind) 31.7 whole, 32.9 cut, 900 tokens (4650) 27.4 and 26.0, 700 (4400) 23.1
// and 20.7, 3000 tokens, 16 / 2 heads (8100) 59.0 and 52.1.  To look costs 0.6 us where the answer is no.
constexpr float kPfJoinCost = 7000.f;
constexpr int kPfRounds = 16;      // units of a CTA, at most; with more of them a cut weighs little

struct PagedFwdParams {
  PagedParams p;
  CUtensorMap tm_q;   // 4-D (d, head in group, KV head, token), box {64, hc, 1, tpt}, 128-byte swizzle
  CUtensorMap tm_k;   // 5-D (64 columns, page row, column block, head, page), box {64, min(P, 128), 1, 1, 1}
  CUtensorMap tm_v;
  int oob_page;       // a page index behind the map's last one (reads as zeros)
  int hc, chunks;     // heads per tile, tiles of heads per group
  int tpt;            // tokens per tile: 128 / hc
  FastDiv div_hc, div_chunks;  // by hc, chunks
  FastDiv div_per_seq;  // by Hkv * chunks
  float* part_o;      // [2 * CTAs][2 tiles][d][128 rows] locally normalised partial outputs
  float2* part_ml;    // [2 * CTAs][2 tiles][128] (max of scale * q.k, sum)
  int4* joins;        // [CTAs][2] {first token, first head, heads, last CTA (-1: no join)}, {tokens of tile 0, 1, -, -}
};

template <int D, int NS>
struct PagedFwdCfg {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kBlocks = D / 64;
  static constexpr int kBlockBytes = 128 * 128;
  // q_full[2] q_empty[2] kv_full[NS] kv_empty[NS] s_full[2] p_full[2] o_full[2] turn[2] drain
  // unit_full[4] unit_empty[4] merge_full merge_done tail[NS]
  static constexpr int kNumBars = 4 + 2 * NS + 8 + 1 + 2 * kPfRing + 2 + NS;
  static constexpr int kRingOffset = (kNumBars * 8 + 15) / 16 * 16;   // pieces: kPfRing x 16 ints
  static constexpr int kMergeOffset = kRingOffset + kPfRing * 64;     // thin units: (max, sum) of tile 1's rows
  static constexpr int kEnd = (2 + NS) * kTileBytes + kMergeOffset + 128 * 8;
  // a CTA that takes the rows that the units leave holds two of the decode's CTAs instead
  static constexpr int kRowsBytes = (PagedDecodeCfg<D>::kSumOffset + 1023) / 1024 * 1024;
  // above both: sums of 12 warps and two lines, prefix and first sequence of two shares, whole units, TMEM
  // base, abort flag
  static constexpr int kSumOffset = kEnd > 2 * kRowsBytes ? kEnd : 2 * kRowsBytes;
  static constexpr int kListOffset = kSumOffset + 28 * 8;  // whole units: {sequence, head tile, unit} each
  static constexpr int kSmemBytes = kListOffset + (3 * kPfRounds + 1) * 4 + 8;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per block");
};

// A sequence's place in the batch.
struct PfSeq {
  int start, n;     // first token, tokens
  int L, coff;      // keys; token i sees key j iff j <= i + coff (causal)
  int full, units;  // units whose two tiles are full, units (without one that is the decode's work)
  int64_t cost;     // weight of its units for one (KV head, head tile)
};

// Weight of a sequence's first V full units (tu tokens each): V times the fixed weight
// and kPfPair times the visible keys, which are clamp((v + 1) tu + coff, 0, L) in unit v.
__device__ __forceinline__ int64_t pf_prefix(const PagedFwdParams& a, int V, int L, int coff) {
  const int64_t fixed = static_cast<int64_t>(V) * kPfUnitCost;
  if (!a.p.causal || V == 0) return fixed + kPfPair * static_cast<int64_t>(V) * L;
  const int tu = 2 * a.tpt;
  auto div = [&](int x) { return static_cast<int>(fastdiv(static_cast<uint32_t>(x), a.p.div_tu)); };
  const int lo = min(V, div(max(-coff, 0)));                     // units that see nothing
  const int hi = min(V, max(lo, div(L - coff + tu - 1) - 1));    // first unit that sees every key
  const int64_t m = hi - lo;
  const int64_t mid = m * coff + tu * (static_cast<int64_t>(hi) * (hi + 1) - static_cast<int64_t>(lo) * (lo + 1)) / 2;
  return fixed + kPfPair * (mid + static_cast<int64_t>(V - hi) * L);
}

__device__ __forceinline__ PfSeq pf_of(const PagedFwdParams& a, const PagedSeq& q) {
  const PagedParams& p = a.p;
  PfSeq s;
  s.start = q.start;
  s.n = q.n;
  s.L = q.L;
  s.coff = p.causal == 2 ? s.L - s.n : 0;
  s.full = static_cast<int>(fastdiv(static_cast<uint32_t>(s.n), a.p.div_tu));
  const int rem = s.n - s.full * 2 * a.tpt;
  const bool more = rem > p.row_tokens;
  s.units = s.full + (more ? 1 : 0);
  s.cost = pf_prefix(a, s.full, s.L, s.coff);
  if (more)
    s.cost += kPfUnitCost + (rem > a.tpt ? kPfPair : kPfThin) * static_cast<int64_t>(paged_visible(p.causal, s.n, s.L, s.coff));
  return s;
}

__device__ __forceinline__ PfSeq pf_seq(const PagedFwdParams& a, int b) { return pf_of(a, paged_seq(a.p, b)); }

// SPLIT: whether units can be split at all, i.e. the table holds more keys than stay whole. Without the code for
// it five short prompts take 11.9 us instead of 12.6, 40 of 10 to 200 tokens 32.4 instead of 33.6.
template <int D, int NS, bool SPLIT>
__global__ void __launch_bounds__(kPrefillThreads, 1) paged_fwd_kernel(const __grid_constant__ PagedFwdParams a,
                                                                       const __grid_constant__ PagedDecodeParams rows) {
  using Cfg = PagedFwdCfg<D, NS>;
  const PagedParams& p = a.p;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's pattern repeats every 1024 bytes
  const uint32_t sQ = smem_u32(smem);
  const uint32_t sKV = sQ + 2 * Cfg::kTileBytes;
  const uint32_t bar0 = sKV + NS * Cfg::kTileBytes;
  auto q_full = [&](int t) { return bar0 + 8u * t; };
  auto q_empty = [&](int t) { return bar0 + 8u * (2 + t); };
  auto kv_full = [&](int s) { return bar0 + 8u * (4 + s); };
  auto kv_empty = [&](int s) { return bar0 + 8u * (4 + NS + s); };
  auto s_full = [&](int t) { return bar0 + 8u * (4 + 2 * NS + t); };
  auto p_full = [&](int t) { return bar0 + 8u * (6 + 2 * NS + t); };
  auto o_full = [&](int t) { return bar0 + 8u * (8 + 2 * NS + t); };
  auto turn = [&](int t) { return bar0 + 8u * (10 + 2 * NS + t); };
  const uint32_t drain = bar0 + 8u * (12 + 2 * NS);
  auto unit_full = [&](int k) { return bar0 + 8u * (13 + 2 * NS + k); };
  auto unit_empty = [&](int k) { return bar0 + 8u * (13 + 2 * NS + kPfRing + k); };
  const uint32_t merge_full = bar0 + 8u * (13 + 2 * NS + 2 * kPfRing);  // thin unit: tile 1's result is complete
  const uint32_t merge_done = merge_full + 8;                           // thin unit: it was read
  // a V tile that warp 11 has to clean landed in the slot; one barrier per slot, because a slot is not
  // filled again before it was cleaned (one for all could run two phases ahead of the cleaner)
  auto tail = [&](int s) { return merge_full + 16 + 8u * s; };
  uint8_t* const misc = smem + (2 + NS) * Cfg::kTileBytes;
  volatile int* const ring = reinterpret_cast<volatile int*>(misc + Cfg::kRingOffset);
  float2* const merge_ml = reinterpret_cast<float2*>(misc + Cfg::kMergeOffset);
  int64_t* const s_sum = reinterpret_cast<int64_t*>(smem + Cfg::kSumOffset);  // [2 lines][12 warps]
  int64_t* const s_prefix = s_sum + 24;  // [2 shares] weight of the sequences before the first one, per head
  int64_t* const s_first = s_sum + 26;   // [2 shares] that sequence
  int* const s_list = reinterpret_cast<int*>(smem + Cfg::kListOffset);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(s_list + 3 * kPfRounds + 1);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // Entries of an announced piece.
  enum { kHead, kG0, kHeads, kTok0, kCnt0, kCnt1, kLim, kKeys, kJ0, kN0, kN1, kThin, kSlot, kSteps };
  // The r-th piece of this CTA, for a whole warp: waits for it; nullptr where there is none left.  The warp
  // gives it back with `release` when each of its lanes has read what it needs: the producer may write the
  // entry again from then on.  The lanes meet in both, since a spin-wait leaves them in any order.
  auto next_piece = [&](int r, bool& ok) -> volatile int* {
    const int k = r % kPfRing;
    ok = __all_sync(0xffffffffu, ok && mbar_wait(unit_full(k), (r / kPfRing) & 1, abort_flag));
    volatile int* const e = ring + 16 * k;
    return ok && e[kHead] >= 0 ? e : nullptr;
  };
  auto release = [&](int r) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(unit_empty(r % kPfRing));
  };
  // The same for a lone thread.
  auto next_piece_lone = [&](int r) -> volatile int* {
    const int k = r % kPfRing;
    if (!mbar_wait(unit_full(k), (r / kPfRing) & 1, abort_flag)) return nullptr;
    volatile int* const e = ring + 16 * k;
    return e[kHead] >= 0 ? e : nullptr;
  };
  auto release_lone = [&](int r) { mbar_arrive(unit_empty(r % kPfRing)); };

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full(t), 1);
      mbar_init(q_empty(t), 1);
      mbar_init(s_full(t), 1);
      mbar_init(p_full(t), 4);
      mbar_init(turn(t), 1);
      mbar_init(o_full(t), 1);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 2);
      mbar_init(tail(s), 1);
    }
    mbar_init(drain, 2);
    for (int k = 0; k < kPfRing; ++k) {
      mbar_init(unit_full(k), 1);
      mbar_init(unit_empty(k), 2 + 8 + 1);  // MMA threads, softmax warps, warp 11
    }
    mbar_init(merge_full, 4);
    mbar_init(merge_done, 4);
    s_first[0] = s_first[1] = s_prefix[0] = s_prefix[1] = 0;
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  paged_warm(p);
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&a.tm_q);
    tma_prefetch_desc(&a.tm_k);
    tma_prefetch_desc(&a.tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Launched as a programmatic dependent of whatever precedes it on the stream:
  // no global memory is read or written before this wait (the lines asked for above go
  // to the L2 only).
  grid_dependency_wait();
  grid_dependency_trigger();

  // ---- the two lines, and this CTA's share of one of them
  const int cta = static_cast<int>(blockIdx.x), ctas = static_cast<int>(gridDim.x);
  const int per_seq = p.Hkv * a.chunks;  // head tiles per sequence of the units (the rows: p.Hkv)
  int64_t x0 = 0, x1 = 0, total = 0, quot = 0;
  int G = 0, rem = 0;
  auto share_begin = [&](int c) -> int64_t { return quot * c + rem * c / G; };  // floor(total * c / G)
  int row_ctas = 0;     // the last CTAs of the grid, which take the rows that the units leave
  bool takes_rows = false;
  int whole_units = -1;  // units of this CTA where whole units are dealt
  PdShare sh[2];
  {
    constexpr int kWarps = kPrefillThreads / 32;
    auto costs_of = [&](int b, int64_t (&t)[2]) -> int {  // returns its units
      t[0] = t[1] = 0;
      if (b >= p.B) return 0;
      const PagedSeq q = paged_seq(p, b);
      if (q.bad && cta == 0) atomicOr(&g_error_word, kErrSeqlen);
      if (q.n == 0) return 0;
      const PfSeq s = pf_of(a, q);
      t[0] = s.cost;
      t[1] = pd_cost(pd_of(p, q));
      return s.units;
    };
    // inclusive sums over the block's threads and their totals
    auto block_scan = [&](const int64_t (&t)[2], int64_t (&incl)[2], int64_t (&all)[2]) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        incl[q] = t[q];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int64_t u = __shfl_up_sync(0xffffffffu, incl[q], off);
          if (lane >= off) incl[q] += u;
        }
        if (lane == 31) s_sum[q * kWarps + warp] = incl[q];
      }
      __syncthreads();
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        all[q] = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) incl[q] += s_sum[q * kWarps + w];
          all[q] += s_sum[q * kWarps + w];
        }
      }
    };
    auto share = [&](const int64_t (&all)[2]) {
      total = all[0] * per_seq;
      const int64_t row_total = all[1] * p.Hkv;
      // CTAs for the rows: in proportion to the two lines' times, and in pairs
      if (row_total > 0) {
        const float wr = static_cast<float>(row_total) * kPfRowPlace, wu = static_cast<float>(total);
        const int pairs = ctas >> 1;
        row_ctas = total > 0 ? 2 * min(max(static_cast<int>(pairs * wr / (wr + wu) + 0.5f), 1), pairs - 1) : ctas;
      }
      takes_rows = cta >= ctas - row_ctas;
      if (takes_rows) {
#pragma unroll
        for (int g = 0; g < 2; ++g) sh[g] = pd_share(row_total, 2 * row_ctas, 2 * (cta - (ctas - row_ctas)) + g);
        x0 = sh[0].x0;
        x1 = max(sh[0].x1, sh[1].x1);
        return;
      }
      // a share is at least a pair step long, so each CTA between the first and the last one of a
      // unit has a key tile of it
      G = static_cast<int>(max(int64_t{1}, min(static_cast<int64_t>(ctas - row_ctas), total / (128 * kPfPair))));
      quot = div64(total, G);
      rem = static_cast<int>(total - quot * G);
      if (cta < G) {
        x0 = share_begin(cta);
        x1 = share_begin(cta + 1);
      }
    };
    auto find = [&](int b, const int64_t (&t)[2], const int64_t (&end)[2]) {  // sequence b's weights end at `end`
      if (takes_rows) {
#pragma unroll
        for (int g = 0; g < 2; ++g)
          if (t[1] > 0 && (end[1] - t[1]) * p.Hkv <= sh[g].x0 && sh[g].x0 < end[1] * p.Hkv) {
            s_first[g] = b;
            s_prefix[g] = end[1] - t[1];
          }
      } else if (t[0] > 0 && (end[0] - t[0]) * per_seq <= x0 && x0 < end[0] * per_seq) {
        s_first[0] = b;
        s_prefix[0] = end[0] - t[0];
      }
    };
    // Whole units where they balance: no partials, no join.  A thread takes one unit (of one head tile: all have
    // the same) and ranks it by weight, counting what is heavier; then they are dealt to the CTAs there and back.
    // Taken where the heaviest hand is at most kPfJoinCost above a share.  Returns this CTA's number of units (-1:
    // shares).  Loops are not unrolled: the code runs once, and cold code costs by its length.
    auto take_whole = [&](int n, int units_before) -> int {
      const int hands = ctas - row_ctas;
      const int units = n * per_seq;
      int* const s_base = reinterpret_cast<int*>(smem + 2 * Cfg::kTileBytes);  // in the K/V slots: [384] first unit
      float* const s_w = reinterpret_cast<float*>(s_base + kPrefillThreads);   // [384] weights
      int2* const s_rank = reinterpret_cast<int2*>(s_w + kPrefillThreads);     // [384] (sequence, unit) of each rank
      float* const s_load = reinterpret_cast<float*>(s_rank + kPrefillThreads);  // [384] hands
      const int tid = static_cast<int>(threadIdx.x);
      s_base[tid] = units_before;
      __syncthreads();
      int b = 0, v = 0;
      float w = 0.f;
      if (tid < n) {
#pragma unroll 1
        for (int hi = p.B; hi - b > 1;) {  // the last sequence whose units begin at or before this one
          const int mid = (b + hi) >> 1;
          if (s_base[mid] <= tid) b = mid;
          else hi = mid;
        }
        v = tid - s_base[b];
        const PagedSeq q = paged_seq(p, b);
        const int t0 = 2 * a.tpt * v, t1 = min(q.n, t0 + 2 * a.tpt);
        const int keys = paged_visible(p.causal, t1, q.L, p.causal == 2 ? q.L - q.n : 0);
        w = static_cast<float>(kPfUnitCost + (t1 - t0 > a.tpt ? kPfPair : kPfThin) * static_cast<int64_t>(keys));
      }
      s_w[tid] = w;
      const float most = static_cast<float>(total) + kPfJoinCost * G;  // G times the heaviest hand there may be
      if (__syncthreads_or(w * G > most)) {
        fence_async_shared();
        return -1;
      }
      if (tid < n) {
        int rank = 0;
#pragma unroll 1
        for (int j = 0; j < n; j += 4) {  // (behind n: weight 0)
          const float4 o = *reinterpret_cast<const float4*>(s_w + j);
          rank += (o.x > w || (o.x == w && j < tid)) + (o.y > w || (o.y == w && j + 1 < tid)) +
                  (o.z > w || (o.z == w && j + 2 < tid)) + (o.w > w || (o.w == w && j + 3 < tid));
        }
        s_rank[rank] = make_int2(b, v);
        s_load[rank] = w;
      }
      __syncthreads();
      // the k-th unit of hand c
      auto dealt = [&](int c, int k) { return k * hands + ((k & 1) ? hands - 1 - c : c); };
      float load = 0.f;
      int mine = 0;
      if (tid < hands) {
#pragma unroll 1
        for (int k = 0; k < kPfRounds; ++k) {
          const int u = dealt(tid, k);
          if (u >= units) break;
          load += s_load[fastdiv(static_cast<uint32_t>(u), a.div_per_seq)];
          ++mine;
        }
        if (tid == cta) s_list[3 * kPfRounds] = mine;
      }
      const int u = tid < kPfRounds ? dealt(cta, tid) : units;
      if (u < units) {
        const int i = static_cast<int>(fastdiv(static_cast<uint32_t>(u), a.div_per_seq));
        s_list[3 * tid] = s_rank[i].x;
        s_list[3 * tid + 1] = u - i * per_seq;
        s_list[3 * tid + 2] = s_rank[i].y;
      }
      fence_async_shared();  // the space is the K/V copies' from here on
      return __syncthreads_and(load * G <= most) ? s_list[3 * kPfRounds] : -1;
    };
    // 384 sequences at a time: once where that is all of them, else a round for the totals and one for the share.
    // The number of units rides in the upper bits of the rows' line (the fields of 384 sequences do not overflow).
    constexpr int kShift = 40, kMost = 1 << 14;
    int64_t base[2] = {0, 0};
    bool shared = false;
#pragma unroll 1
    for (int b0 = 0;;) {
      int64_t t[2], incl[2], all[2];
      const int units = costs_of(b0 + static_cast<int>(threadIdx.x), t);
      t[1] += static_cast<int64_t>(min(units, kMost)) << kShift;
      block_scan(t, incl, all);
      const int n = static_cast<int>(all[1] >> kShift);
      const int before = static_cast<int>((incl[1] - t[1]) >> kShift);
      for (int64_t* x : {&t[1], &incl[1], &all[1]}) *x &= (int64_t{1} << kShift) - 1;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        incl[q] += base[q];
        base[q] += all[q];
      }
      b0 += kPrefillThreads;
      const bool first = !shared;
      if (first && b0 >= p.B) {
        share(base);
        shared = true;
      }
      if (shared && !(first && p.B > kPrefillThreads)) find(b0 - kPrefillThreads + static_cast<int>(threadIdx.x), t, incl);
      if (SPLIT && p.B <= kPrefillThreads && !takes_rows && n > 0 && n <= kPrefillThreads) {
        // no look at them where there are too many, or where a unit of the mean weight is too heavy
        const float u = static_cast<float>(n) * per_seq;
        if (u <= kPfRounds * (ctas - row_ctas) && static_cast<float>(total) * (G - u) <= kPfJoinCost * G * u)
          whole_units = take_whole(n, before);
      }
      if (b0 >= p.B) {
        if (!first || p.B <= kPrefillThreads || x0 >= x1) break;  // block-uniform
        b0 = 0;
        base[0] = base[1] = 0;
      }
      __syncthreads();  // s_sum's contents are read
    }
    if (takes_rows && threadIdx.x == 0) {
      // the space becomes that of two decode CTAs
      for (int i = 0; i < Cfg::kNumBars; ++i) mbar_inval(bar0 + 8u * i);
      for (int g = 0; g < 2; ++g) PdSmem<D>(smem + g * Cfg::kRowsBytes).init();
    }
    __syncthreads();
  }
  // joins that nobody else writes: the units' of a CTA with rows, and the reverse
  if (SPLIT && threadIdx.x < 2) {
    if (takes_rows) a.joins[2 * cta + threadIdx.x] = make_int4(0, 0, 0, -1);
    else if (rows.joins != nullptr) rows.joins[2 * (row_ctas + cta) + threadIdx.x] = make_int4(-1, 0, 0, 0);
  }

  if (warp >= 8) {
    regs_decrease<kCtrlRegs>();
    if (takes_rows) {
      if (warp < 10) {
        const int g = warp - 8;
        PdShare my = g == 0 ? sh[0] : sh[1];
        my.first = static_cast<int>(s_first[g]);
        my.prefix = s_prefix[g];
        pd_producer<D>(rows, PdSmem<D>(smem + g * Cfg::kRowsBytes), my, 2 * (cta - (ctas - row_ctas)) + g, lane);
      }
    } else if (warp == kLoadWarp) {
      // ------------------------------------------- producer and scheduler
      const int pb_shift = min(p.page_shift, 7);
      const int pb = 1 << pb_shift;         // rows per copy
      const int nb = 128 >> pb_shift;       // copies per 64 columns of a tile
      const int blk = lane / nb, box = lane - blk * nb;
      const bool copier = blk < Cfg::kBlocks;
      const uint32_t box_dst = static_cast<uint32_t>(blk) * Cfg::kBlockBytes + static_cast<uint32_t>(box) * pb * 128u;
      const int tu = 2 * a.tpt;
      int it = 0;    // K/V tiles issued so far
      int ui = 0;    // pieces started so far
      uint32_t tail_uses = 0;    // per slot: parity of the tiles handed to warp 11
      uint32_t slot_tail = 0;    // per slot: its last tile was one of them
      bool ok = true;
      int4 join0 = make_int4(0, 0, 0, -1), join1 = make_int4(0, 0, 0, 0);  // the unit that a later share ends
      int64_t join_last = 0;                                               // its last key tile's place
      // The table entry of this lane's copy of key tile j (none behind the last
      // key).  It is looked at when the copy is issued, one tile later.
      auto has_copy = [&](int j, int L) { return copier && j * 128 + box * pb < L; };
      auto page_of = [&](int b, int j, int L) -> int {
        return has_copy(j, L)
                   ? p.table[static_cast<int64_t>(b) * p.max_pages + ((j * 128 + box * pb) >> p.page_shift)]
                   : 0;
      };
      int dealt = 0;  // whole units begun
      if (whole_units >= 0) {  // each is its own line, which one share covers
        x0 = 0;
        x1 = whole_units > 0 ? int64_t{1} << 60 : 0;
      }
      if (x0 < x1) {
        int b = whole_units > 0 ? s_list[0] : static_cast<int>(s_first[0]);
        PfSeq s = pf_seq(a, b);
        int hr, v = 0;     // KV head * chunks + head tile, unit
        int64_t xs = 0;    // where the unit begins
        if (whole_units > 0) {
          hr = s_list[1];
          v = s_list[2];
        } else {
          const int64_t in_seq = x0 - s_prefix[0] * per_seq;
          hr = static_cast<int>(div64(in_seq, s.cost));
          const int64_t in_head = in_seq - hr * s.cost;
          for (int hi = s.units; hi - v > 1;) {  // last unit that begins at or before the share
            const int mid = (v + hi) >> 1;
            if (pf_prefix(a, mid, s.L, s.coff) <= in_head) v = mid;
            else hi = mid;
          }
          xs = x0 - in_head + pf_prefix(a, v, s.L, s.coff);
        }
        while (ok && xs < x1) {
          // unit (b, hr, v): tokens v tu .. of the sequence
          const int cnt0 = min(s.n - v * tu, a.tpt);
          const int cnt1 = min(max(s.n - v * tu - a.tpt, 0), a.tpt);
          const bool thin = cnt1 == 0;
          const int w = 128 * (thin ? kPfThin : kPfPair);  // weight of a key tile
          const int64_t t0 = static_cast<int64_t>(v) * tu;
          const int keys = paged_visible(p.causal, t0 + cnt0 + cnt1, s.L, s.coff);
          const int n_u = (keys + 127) / 128;                                          // its key tiles
          const int n_0 = (paged_visible(p.causal, t0 + cnt0, s.L, s.coff) + 127) / 128;  // tile 0's
          // key tile k stands at xs + kPfUnitCost + w k
          const bool split = n_u > (thin ? kPfWholeThin : kPfWholePair);
          auto tile_at = [&](int64_t x) -> int {
            const int64_t off = x - xs - kPfUnitCost;
            if (off <= 0) return 0;
            if (!split) return n_u;
            // (a division by a constant either way)
            const uint64_t k = thin ? (static_cast<uint64_t>(off) + 128 * kPfThin - 1) / (128 * kPfThin)
                                    : (static_cast<uint64_t>(off) + 128 * kPfPair - 1) / (128 * kPfPair);
            return static_cast<int>(min(static_cast<uint64_t>(n_u), k));
          };
          const int j0 = tile_at(x0), j1 = tile_at(x1);
          const int64_t xe = xs + kPfUnitCost + static_cast<int64_t>(w / 128) * keys;
          if (j1 > j0 || (n_u == 0 && xs >= x0)) {
            const int steps = j1 - j0;
            const bool whole = !SPLIT || steps == n_u;
            const int hk = static_cast<int>(fastdiv(static_cast<uint32_t>(hr), a.div_chunks));
            const int chunk = hr - hk * a.chunks;
            const int g0 = chunk * a.hc;
            const int heads = min(a.hc, p.group - g0);
            const int tok0 = s.start + static_cast<int>(t0);
            int n0, n1;
            if (thin) {
              n0 = (steps + 1) >> 1;
              n1 = steps >> 1;
            } else {
              n0 = min(max(n_0 - j0, 0), steps);
              n1 = steps;
            }
            if (SPLIT && j0 == 0 && !whole) {
              join0 = make_int4(tok0, hk * p.group + g0, heads, 0);
              join1 = make_int4(cnt0, cnt1, 0, 0);
              join_last = xs + kPfUnitCost + static_cast<int64_t>(n_u - 1) * w;
            }
            int page = page_of(b, j0, s.L);
            // announce
            const int k = ui % kPfRing;
            ok = __all_sync(0xffffffffu,
                            ui < kPfRing || mbar_wait(unit_empty(k), ((ui / kPfRing) - 1) & 1, abort_flag));
            if (!ok) break;
            if (lane == 0) {
              volatile int* e = ring + 16 * k;
              e[kHead] = hk;
              e[kG0] = hk * p.group + g0;
              e[kHeads] = heads;
              e[kTok0] = tok0;
              e[kCnt0] = cnt0;
              e[kCnt1] = cnt1;
              e[kLim] = static_cast<int>(t0) + s.coff;
              e[kKeys] = s.L;
              e[kJ0] = j0;
              e[kN0] = n0;
              e[kN1] = n1;
              e[kThin] = thin;
              e[kSlot] = whole ? -1 : (j0 > 0 ? 2 * cta : 2 * cta + 1);
              e[kSteps] = steps;
              mbar_arrive(unit_full(k));
            }
            __syncwarp();
#pragma unroll 1
            for (int x = 0; ok && x < steps; ++x) {
              const int j = j0 + x;
              int cur = page;
              if (x + 1 < steps) page = page_of(b, j + 1, s.L);
              if (!has_copy(j, s.L)) {
                cur = a.oob_page;  // rows behind the last key: zeros
              } else if (cur < 0 || cur >= p.num_pages) {
                atomicOr(&g_error_word, kErrPage);
                cur = a.oob_page;
              }
              const int row = (j * 128 + box * pb) & ((1 << p.page_shift) - 1);
              const bool clean = (j + 1) * 128 > s.L;  // V's rows behind the last key
#pragma unroll
              for (int kv = 0; kv < 2; ++kv, ++it) {
                const int slot = it % NS;
                if (!__all_sync(0xffffffffu, mbar_wait(kv_empty(slot), ((it / NS) & 1) ^ 1, abort_flag))) {
                  ok = false;
                  break;
                }
                const bool to_clean = kv && clean;
                const uint32_t bar = to_clean ? tail(slot) : kv_full(slot);
                tail_uses ^= (to_clean ? 1u : 0u) << slot;
                slot_tail = (slot_tail & ~(1u << slot)) | ((to_clean ? 1u : 0u) << slot);
                if (lane == 0) mbar_arrive_expect_tx(bar, Cfg::kTileBytes);
                __syncwarp();
                if (copier) {
                  const uint32_t dst = sKV + slot * Cfg::kTileBytes + box_dst;
                  const CUtensorMap* const tm = kv ? &a.tm_v : &a.tm_k;
                  // a lone unit's keys are read once (see pd_producer)
                  if (s.units == 1) tma_load_5d_hint(dst, tm, 0, row, blk, hk, cur, bar, l2_evict_first());
                  else tma_load_5d(dst, tm, 0, row, blk, hk, cur, bar);
                }
              }
            }
            ++ui;
          }
          // the unit behind this one
          if (whole_units > 0) {
            if (++dealt == whole_units) break;
            b = s_list[3 * dealt];
            hr = s_list[3 * dealt + 1];
            v = s_list[3 * dealt + 2];
            s = pf_seq(a, b);
            continue;
          }
          xs = xe;
          if (++v == s.units) {
            v = 0;
            if (++hr == per_seq) {
              hr = 0;
              if (xs >= x1) break;
              // the next sequence with units
              unsigned some = 0u;
              for (++b; b < p.B && some == 0u; b += 32) {
                some = __ballot_sync(0xffffffffu, b + lane < p.B && pf_seq(a, b + lane).units > 0);
                if (some != 0u) b += __ffs(some) - 1 - 32;
              }
              if (some == 0u) break;
              s = pf_seq(a, b);
            }
          }
        }
      }
      if (SPLIT && join0.w >= 0) {  // the CTA whose share holds that place
        int c = static_cast<int>(div64(join_last, quot + 1));  // at most the right one
        while (c + 1 < G && share_begin(c + 1) <= join_last) ++c;
        join0.w = c;
      }
      if (SPLIT && lane == 0) {
        a.joins[2 * cta] = join0;
        a.joins[2 * cta + 1] = join1;
      }
      // the end of the pieces
      if (ok && __all_sync(0xffffffffu, ui < kPfRing || mbar_wait(unit_empty(ui % kPfRing), ((ui / kPfRing) - 1) & 1,
                                                                   abort_flag))) {
        if (lane == 0) {
          ring[16 * (ui % kPfRing) + kHead] = -1;
          mbar_arrive(unit_full(ui % kPfRing));
        }
      }
      // Copies still in flight must land before the CTA may exit.
      if (lane == 0) {
        for (int i = max(0, it - NS); i < it; ++i) {
          const int slot = i % NS;
          if ((slot_tail >> slot) & 1u) mbar_wait_drain(tail(slot), ((tail_uses >> slot) & 1u) ^ 1u);
          else mbar_wait_drain(kv_full(slot), (i / NS) & 1);
        }
      }
      __syncwarp();
    } else if (warp == kPfQWarp) {
      // ----------------------------- Q loader, and cleaner of V's last tile
      // Q_0, Q_1: each once the previous piece's last S MMA on that buffer is
      // done (a tile without key tiles only completes the phase).
      const uint32_t q_bytes = static_cast<uint32_t>(a.hc) * a.tpt * D * 2;
      int loaded[2] = {0, 0};  // pieces whose Q_t was loaded
      int it_base = 0;
      uint32_t tail_uses = 0;
      bool ok = true;
#pragma unroll 1
      for (int r = 0; ok; ++r) {
        volatile int* const e = next_piece(r, ok);
        if (e == nullptr) break;
        const int L = e[kKeys], steps = e[kSteps], j_last = e[kJ0] + steps - 1;
        const int hk = e[kHead], g0 = e[kG0] - hk * p.group, tok0 = e[kTok0];
        const int n[2] = {e[kN0], e[kN1]};
        const int tok1 = tok0 + (e[kThin] ? 0 : a.tpt);
        release(r);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          ok = ok && (loaded[t] == 0 ||
                      __all_sync(0xffffffffu, mbar_wait(q_empty(t), (loaded[t] - 1) & 1, abort_flag)));
          if (!ok) break;
          if (lane == 0) {
            if (n[t] > 0) {
              mbar_arrive_expect_tx(q_full(t), q_bytes);
              for (int c = 0; c < Cfg::kBlocks; ++c)
                tma_load_4d(sQ + t * Cfg::kTileBytes + c * Cfg::kBlockBytes, &a.tm_q, c * 64, g0, hk, t ? tok1 : tok0,
                            q_full(t));
            } else {
              mbar_arrive(q_full(t));
            }
          }
          ++loaded[t];
          __syncwarp();
        }
        if (!ok) break;
        if (steps > 0 && (j_last + 1) * 128 > L) {
          const int itv = it_base + 2 * steps - 1;
          const int slot = itv % NS;
          if (!__all_sync(0xffffffffu, mbar_wait(tail(slot), (tail_uses >> slot) & 1u, abort_flag))) break;
          tail_uses ^= 1u << slot;
          // rows L mod 128 .. 127 (those behind the last page are zeros already)
          const int first = L - j_last * 128;
          const int stop = min(128, (((L - 1) >> p.page_shift) + 1 << p.page_shift) - j_last * 128);
          for (int blk = 0; blk < Cfg::kBlocks; ++blk)
            for (int c = first * 8 + lane; c < stop * 8; c += 32)
              st_shared_zero16(sKV + slot * Cfg::kTileBytes + blk * Cfg::kBlockBytes + c * 16);
          fence_async_shared();  // the MMAs read shared memory through the async proxy
          __syncwarp();
          if (lane == 0) mbar_arrive(kv_full(slot));
        }
        it_base += 2 * steps;
      }
      // the last copies must land before the CTA may exit
      if (lane == 0)
        for (int t = 0; t < 2; ++t)
          if (loaded[t] > 0) mbar_wait_drain(q_full(t), (loaded[t] - 1) & 1);
      __syncwarp();
    } else {
      // ---------------------------------------------- MMA issuer of tile t
      // The two issuers' products as in prefill.cuh, in the order of piece_steps.h.
      const int t = (warp == kMmaWarp) ? 0 : 1;
      if (lane == 0) {
        const uint64_t hi = static_cast<uint64_t>(sdesc_hi(1024)) << 32;
        const uint64_t dq = hi | sdesc_lo(sQ + t * Cfg::kTileBytes, 16);
        auto dk = [&](int slot) { return hi | sdesc_lo(sKV + slot * Cfg::kTileBytes, 16); };
        auto dv = [&](int slot) { return hi | sdesc_lo(sKV + slot * Cfg::kTileBytes, Cfg::kBlockBytes); };
        // The operations of walk_piece (piece_steps.h, with the order of the waits and its reason).
        struct Ops {
          const decltype(kv_full)& full;
          const decltype(kv_empty)& empty;
          const decltype(dk)& k_desc;
          const decltype(dv)& v_desc;
          uint32_t p_bar, turn_bar, other_turn, s_bar, o_bar, q_bar, tS, tO;
          uint64_t dq;
          volatile int* abort_flag;
          int nt, pj;
          __device__ __forceinline__ bool p_ready() { return mbar_wait(p_bar, pj & 1, abort_flag); }
          __device__ __forceinline__ bool turn_ready(int s) { return mbar_wait(turn_bar, s & 1, abort_flag); }
          __device__ __forceinline__ bool tile_ready(int i, int slot) { return mbar_wait(full(slot), (i / NS) & 1, abort_flag); }
          __device__ __forceinline__ void multiply(int k, int vs, int ks) {
            tc_fence_after();
            if (k >= 1 && k - 1 < nt) {
              const uint64_t vd = v_desc(vs);
              issue_pv<D, 0>(tO, tS, vd, k > 1);
              issue_pv<D, 1>(tO, tS, vd, true);
              ++pj;
              if (k == nt) mma_commit(o_bar);
            }
            if (k < nt) {
              issue_qk<D>(tS, dq, k_desc(ks));
              mma_commit(s_bar);
              if (k == nt - 1) mma_commit(q_bar);
            }
          }
          __device__ __forceinline__ void free_tile(int slot, int times) {
            mma_commit(empty(slot));
            if (times > 1) mma_commit(empty(slot));
          }
          __device__ __forceinline__ void hand_over() { mbar_arrive(other_turn); }
        };
        Ops op = {kv_full,  kv_empty, dk, dv, p_full(t), turn(t), turn(1 - t), s_full(t), o_full(t), q_empty(t),
                  tmem + t * 128, tmem + 2 * 128 + t * D, dq, abort_flag, 0, 0};
        int it_base = 0, seg = 0, ui = 0;
        bool ok = true;
#pragma unroll 1
        for (int r = 0; ok; ++r) {
          volatile int* const e = next_piece_lone(r);
          if (e == nullptr) break;
          const PieceSteps steps = {e[kN0], e[kN1], e[kThin] != 0, it_base};
          it_base += 2 * e[kSteps];
          release_lone(r);
          op.nt = t ? steps.n1 : steps.n0;
          if (!mbar_wait(q_full(t), ui & 1, abort_flag)) break;
          if (op.nt == 0) mma_commit(q_empty(t));
          ok = walk_piece<NS>(op, steps, t, seg);
          ++ui;
        }
        mma_commit(drain);
        mbar_wait_drain(drain, 0);
      }
      __syncwarp();
    }
  } else if (takes_rows) {
    regs_increase<kSoftmaxRegs>();
    pd_consumer<D>(rows, PdSmem<D>(smem + (warp >> 2) * Cfg::kRowsBytes), warp & 3, lane, 1 + (warp >> 2));
  } else {
    // Warpgroups 0 and 1: softmax and epilogue of tile 0 and 1.
    regs_increase<kSoftmaxRegs>();
    const int t = warp >> 2;
    const int wq = warp & 3;
    const int r_in_tile = wq * 32 + lane;
    const uint32_t lane_bits = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_bits + t * 128;
    const uint32_t tO = tmem + lane_bits + 2 * 128 + t * D;
    const float c = p.scale_log2;
    const int tok_in_tile = static_cast<int>(fastdiv(static_cast<uint32_t>(r_in_tile), a.div_hc));
    const int head_in_tile = r_in_tile - tok_in_tile * a.hc;
    int sj = 0;     // S_t tiles consumed
    int ou = 0;     // pieces whose O_t was waited for
    int merges = 0; // thin pieces
    bool ok = true;
#pragma unroll 1
    for (int r = 0; ok; ++r) {
      volatile int* const e = next_piece(r, ok);
      if (e == nullptr) break;
      const int n = t ? e[kN1] : e[kN0];
      const int n_other = t ? e[kN0] : e[kN1];
      const bool thin = e[kThin] != 0;
      const int L = e[kKeys];
      const int cnt = (thin || t == 0) ? e[kCnt0] : e[kCnt1];
      const int first_lim = e[kLim] + (thin ? 0 : t * a.tpt);  // last key that the tile's first token sees
      const int j0 = e[kJ0] + (thin ? t : 0), j_step = thin ? 2 : 1;
      const bool live = tok_in_tile < cnt && head_in_tile < e[kHeads];
      const int row_lim = p.causal ? min(L - 1, first_lim + tok_in_tile) : L - 1;
      // a warp without rows takes part in the hand-offs only
      const bool idle = static_cast<int>(fastdiv(static_cast<uint32_t>(wq * 32), a.div_hc)) >= cnt;
      const int row_tok = live ? e[kTok0] + (thin ? 0 : t * a.tpt) + tok_in_tile : -1;
      const int row_head = e[kG0] + head_in_tile;
      const int slot = e[kSlot];
      release(r);
      float m_used = -INFINITY;
      float l = 0.f;

#pragma unroll 1
      for (int k = 0; k < n; ++k, ++sj) {
        ok = __all_sync(0xffffffffu, mbar_wait(s_full(t), sj & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        if (!idle) {
          uint32_t sv[128];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(tS + q * 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[q * 32]));
          tmem_wait_ld();
          const int k0 = (j0 + k * j_step) * 128;
          if (k0 + 128 > L || (p.causal && k0 + 127 > first_lim)) {
            const int lim = row_lim - k0;
#pragma unroll
            for (int i = 0; i < 128; ++i)
              if (i > lim) sv[i] = __float_as_uint(-INFINITY);
          }
          float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
          for (int i = 0; i < 128; i += 8) {
            mx0 = max3f(mx0, __uint_as_float(sv[i + 0]), __uint_as_float(sv[i + 1]));
            mx1 = max3f(mx1, __uint_as_float(sv[i + 2]), __uint_as_float(sv[i + 3]));
            mx2 = max3f(mx2, __uint_as_float(sv[i + 4]), __uint_as_float(sv[i + 5]));
            mx3 = max3f(mx3, __uint_as_float(sv[i + 6]), __uint_as_float(sv[i + 7]));
          }
          const float m_new = max3f(m_used, max3f(mx0, mx1, mx2), mx3);
          const bool rescale = (m_new - m_used) * c > kRescaleThreshold;
          float alpha = 1.f;
          if (rescale) {
            alpha = ex2_approx((m_used - m_new) * c);
            m_used = m_new;
            l *= alpha;
          }
          if (k > 0 && __any_sync(0xffffffffu, rescale)) {
            const float2 a2 = make_float2(alpha, alpha);
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[32];
              tmem_ld32(tO + q * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 rr = __fmul2_rn(make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), a2);
                o[i] = __float_as_uint(rr.x);
                o[i + 1] = __float_as_uint(rr.y);
              }
              tmem_st32(tO + q * 32, o);
            }
          }
          const float mc = (m_used == -INFINITY) ? 0.f : m_used * c;
          const float2 c2 = make_float2(c, c);
          const float2 nmc2 = make_float2(-mc, -mc);
          float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[32];
#pragma unroll
            for (int e2 = 0; e2 < 64; e2 += 4) {
              const int i = half * 64 + e2;
              const float2 y0 = __ffma2_rn(make_float2(__uint_as_float(sv[i]), __uint_as_float(sv[i + 1])), c2, nmc2);
              const float2 y1 =
                  __ffma2_rn(make_float2(__uint_as_float(sv[i + 2]), __uint_as_float(sv[i + 3])), c2, nmc2);
              const float2 p0 = make_float2(ex2_approx(y0.x), ex2_approx(y0.y));
              const float2 p1 = make_float2(ex2_approx(y1.x), ex2_approx(y1.y));
              acc0 = __fadd2_rn(acc0, p0);
              acc1 = __fadd2_rn(acc1, p1);
              // the product with V takes bf16: one rounding of every probability
              pk[e2 / 2] = pack_bf16x2(p0.x, p0.y);
              pk[e2 / 2 + 1] = pack_bf16x2(p1.x, p1.y);
            }
            tmem_st32(tS + half * 32, pk);
          }
          tmem_wait_st();
          l += (acc0.x + acc0.y) + (acc1.x + acc1.y);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(t));
      }
      if (!ok) break;

      // ---- epilogue
      if (n > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(o_full(t), ou & 1, abort_flag));
        ++ou;
      }
      tc_fence_after();
      float w0 = 1.f, w1 = 0.f;  // thin: weights of the two tiles' outputs
      bool have_other = false;
      if (thin) {
        if (t == 1) {
          // leave (max, sum) to tile 0's warps and wait until they have read O_1
          merge_ml[r_in_tile] = make_float2(m_used, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(merge_full);
          ok = __all_sync(0xffffffffu, ok && mbar_wait(merge_done, merges & 1, abort_flag));
          ++merges;
          tc_fence_after();
          continue;
        }
        ok = __all_sync(0xffffffffu, ok && mbar_wait(merge_full, merges & 1, abort_flag));
        ++merges;
        tc_fence_after();
        const float2 o = merge_ml[r_in_tile];
        const float l1 = n_other > 0 && !idle ? o.y : 0.f, m1 = n_other > 0 && !idle ? o.x : -INFINITY;
        have_other = n_other > 0;
        const float M = fmaxf(m_used, m1);
        w0 = saw_nothing(m_used, l) ? 0.f : ex2_approx((m_used - M) * c);
        w1 = saw_nothing(m1, l1) ? 0.f : ex2_approx((m1 - M) * c);
        m_used = M;
        l = l * w0 + l1 * w1;
      }
      const bool empty_row = saw_nothing(m_used, l);
      const float inv_l = empty_row ? 0.f : 1.f / l;
      const bool have_o = __all_sync(0xffffffffu, ok && n > 0);  // collective loads: warp-uniform
      have_other = __all_sync(0xffffffffu, ok && have_other);
      const float2 s0 = make_float2(w0 * inv_l, w0 * inv_l), s1 = make_float2(w1 * inv_l, w1 * inv_l);
      // 32 columns of this row, normalised
      auto load_cols = [&](int col, float2 (&f)[16]) {
        if (have_o) {
          uint32_t o[32];
          tmem_ld32(tO + col, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            f[i] = __fmul2_rn(make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), s0);
          if (have_other) {
            tmem_ld32(tO + D + col, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              f[i] = __ffma2_rn(make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), s1, f[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) f[i] = make_float2(0.f, 0.f);
        }
      };
      if (!idle && (!SPLIT || slot < 0)) {
        const int g4 = lane & 3;
        uint16_t* dst[4];  // rows of this lane's group of four
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = __shfl_sync(0xffffffffu, row_tok, (lane & ~3) + i);
          const int head = __shfl_sync(0xffffffffu, row_head, (lane & ~3) + i);
          dst[i] = tok < 0 ? nullptr : p.o + (static_cast<int64_t>(tok) * p.Hq + head) * D + g4 * 16;
        }
        const bool wide = (reinterpret_cast<uintptr_t>(p.o) & 31u) == 0u;
#pragma unroll 1
        for (int h = 0; h < D / 64; ++h) {
          uint32_t w[4][8];  // chunk q = columns 64 h + 16 q .. + 15 of this lane's row
#pragma unroll
          for (int q2 = 0; q2 < 2; ++q2) {
            float2 f[16];
            load_cols(h * 64 + q2 * 32, f);
#pragma unroll
            for (int i = 0; i < 16; ++i) w[q2 * 2 + i / 8][i % 8] = pack_bf16x2(f[i].x, f[i].y);
          }
          // 4 x 4 transpose of chunks between the lanes of a group: every store
          // of the warp then writes whole 128-byte row segments
#pragma unroll
          for (int sft = 2; sft > 0; sft >>= 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (i & sft) continue;
              const int jj = i | sft;
              const bool upper = (g4 & sft) != 0;
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const uint32_t x = upper ? w[i][q] : w[jj][q];
                const uint32_t y = __shfl_xor_sync(0xffffffffu, x, sft);
                if (upper) {
                  w[i][q] = y;
                } else {
                  w[jj][q] = y;
                }
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (dst[i] == nullptr) continue;
            if (wide) {
              st_global_v8(dst[i] + h * 64, w[i]);
            } else {
              reinterpret_cast<uint4*>(dst[i] + h * 64)[0] = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
              reinterpret_cast<uint4*>(dst[i] + h * 64)[1] = make_uint4(w[i][4], w[i][5], w[i][6], w[i][7]);
            }
          }
        }
        if (live && p.lse != nullptr)
          p.lse[static_cast<int64_t>(row_head) * p.T + row_tok] =
              empty_row ? -INFINITY : (m_used * p.scale + lg2_approx(l) * 0.69314718055994531f);
      } else if (SPLIT && !idle) {
        // a partial: columns outermost, so that a warp writes 32 rows side by side
        float* const dst = a.part_o + (static_cast<int64_t>(slot) * 2 + t) * (D * 128) + r_in_tile;
#pragma unroll 1
        for (int col = 0; col < D; col += 32) {
          float2 f[16];
          load_cols(col, f);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            dst[(col + 2 * i) * 128] = f[i].x;
            dst[(col + 2 * i + 1) * 128] = f[i].y;
          }
        }
        a.part_ml[(static_cast<int64_t>(slot) * 2 + t) * 128 + r_in_tile] =
            make_float2(empty_row ? -INFINITY : m_used * p.scale, empty_row ? 0.f : l);
      }
      // O_t (and in a thin piece O_1) is read: its next MMA waits for this group's next P
      tc_fence_before();
      if (thin) {
        __syncwarp();
        if (lane == 0) mbar_arrive(merge_done);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Join the partials of a unit that crosses shares: a block of 512 threads takes 32 columns of tile t
// of the unit that begins in CTA c's share; one thread per row and 8 columns, pieces in share order.
constexpr int kPfJoinCols = 8;
constexpr int kPfJoinThreads = 512;
constexpr int kPfJoinBlocksPerSm = 2;
static_assert(kPfJoinThreads == 128 * (32 / kPfJoinCols) && kPfJoinThreads == 32 * kPdRows, "a unit's tile, an item's rows");
static_assert(kPfJoinBlocksPerSm == kPdCtasPerSm, "a block per row share");

template <int D>
__device__ __forceinline__ void paged_fwd_join(const PagedFwdParams& a, int cta, int t, int col) {
  constexpr float kLog2e = 1.4426950408889634f;
  const PagedParams& p = a.p;
  col += (static_cast<int>(threadIdx.x) >> 7) * kPfJoinCols;
  const int4 j0 = a.joins[2 * cta], j1 = a.joins[2 * cta + 1];
  if (j0.w < 0) return;
  const int r = threadIdx.x & 127;
  const int tok = static_cast<int>(fastdiv(static_cast<uint32_t>(r), a.div_hc));
  const int head = r - tok * a.hc;
  if (tok >= (t ? j1.y : j1.x) || head >= j0.z) return;
  const int pieces = j0.w - cta + 1;
  auto slot = [&](int s) { return (static_cast<int64_t>(2 * (cta + s) + (s == 0 ? 1 : 0)) * 2 + t) * 128; };
  // one pass with a running maximum, the loads of kAhead pieces at a time
  constexpr int kAhead = 3;
  float M = -INFINITY, W = 0.f;
  bool some = false;  // whether any piece saw a key
  float acc[kPfJoinCols];
#pragma unroll
  for (int i = 0; i < kPfJoinCols; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (int s0 = 0; s0 < pieces; s0 += kAhead) {
    float2 ml[kAhead];
    float x[kAhead][kPfJoinCols];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      ml[u] = make_float2(-INFINITY, 0.f);
      if (s0 + u < pieces) {
        ml[u] = a.part_ml[slot(s0 + u) + r];
        const float* src = a.part_o + slot(s0 + u) * D + static_cast<int64_t>(col) * 128 + r;
#pragma unroll
        for (int i = 0; i < kPfJoinCols; ++i) x[u][i] = src[i * 128];
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (saw_nothing(ml[u].x, ml[u].y)) continue;
      some = true;
      const float m_new = fmaxf(M, ml[u].x);
      const float down = saw_nothing(M, W) ? 0.f : ex2_approx((M - m_new) * kLog2e);
      const float w = ml[u].y * ex2_approx((ml[u].x - m_new) * kLog2e);
      M = m_new;
      W = W * down + w;
#pragma unroll
      for (int i = 0; i < kPfJoinCols; ++i) acc[i] = fmaf(w, x[u][i], acc[i] * down);
    }
  }
  const float inv = some ? 1.f / W : 0.f;
  const int64_t token = j0.x + t * a.tpt + tok;
  uint16_t* const dst = p.o + (token * p.Hq + j0.y + head) * D + col;
#pragma unroll
  for (int i = 0; i < kPfJoinCols; i += 8)
    *reinterpret_cast<uint4*>(dst + i) =
        make_uint4(pack_bf16x2(acc[i] * inv, acc[i + 1] * inv), pack_bf16x2(acc[i + 2] * inv, acc[i + 3] * inv),
                   pack_bf16x2(acc[i + 4] * inv, acc[i + 5] * inv), pack_bf16x2(acc[i + 6] * inv, acc[i + 7] * inv));
  if (col == 0 && p.lse != nullptr)
    p.lse[static_cast<int64_t>(j0.y + head) * p.T + token] =
        some ? M + lg2_approx(W) * 0.69314718055994531f : -INFINITY;
}

// Both lines' joins in one launch of two blocks per CTA of the forward, all of which fit on the device
// at once: they are there when the grid before ends.  Blocks 2c and 2c + 1 look at the units of shares c,
// c - 1, .. (parts 2k and 2k + 1 of share c - k: a unit's tiles and 32-column blocks go to neighbouring
// blocks), block b at the rows of share b; what has nothing to join costs one look.
template <int D>
__global__ void __launch_bounds__(kPfJoinThreads, kPfJoinBlocksPerSm)
    paged_fwd_join_kernel(const __grid_constant__ PagedFwdParams a, const __grid_constant__ PagedDecodeParams d) {
  grid_dependency_trigger();
  constexpr int kSteps = D / 32;  // parts (2 tiles, d/32 column blocks) per block of the pair
  const int b = static_cast<int>(blockIdx.x), n = static_cast<int>(gridDim.x) >> 1;
  auto share = [&](int k) { return (b >> 1) >= k ? (b >> 1) - k : (b >> 1) - k + n; };
  grid_dependency_wait();
  unsigned units = 0;  // what there is to join
#pragma unroll
  for (int k = 0; k < kSteps; ++k) units |= (a.joins[2 * share(k)].w >= 0 ? 1u : 0u) << k;
  const bool item = d.joins != nullptr && d.joins[b].x >= 0;
#pragma unroll 1
  for (int k = 0; k < kSteps; ++k)
    if ((units >> k) & 1u) paged_fwd_join<D>(a, share(k), b & 1, k * 32);
  if (item) paged_decode_join<D>(d, b, 2 * n);
}

}  // namespace sdpa
