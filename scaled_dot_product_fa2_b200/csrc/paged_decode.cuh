// paged_decode.cuh -- split-KV decode attention over a paged KV cache, and what
// the paged forward's units leave of its sequences.
//
// A work item is (sequence, KV head, group of up to 16 query rows that share
// the head); its keys are walked in tiles of 64 with one running maximum,
// sum and output per row (see paged.cuh for the formula).  The kernel does
// two products per key for at most 16 rows, so its floor is the bytes of the
// valid keys and values, and all of the design serves the memory system:
//   * All items' tiles form one line, in the order (sequence, head, row
//     group), and the grid -- two CTAs per SM -- cuts it into equal shares.
//     A share may begin and end inside an item, so the longest CTA does one
//     tile more than the shortest, whatever the lengths are.  An item's fixed
//     cost takes kPdItemCost places on the line before its tiles.  The line is
//     measured on the device: every CTA sums the tile counts for itself and
//     finds its first item; nothing about the lengths is known on the host.
//   * One producer warp streams K/V tiles through a ring of kStages slots and
//     does not stop at item borders: the ring keeps the next item's tiles in
//     flight while an item's result is merged and written.  One TMA copy
//     brings a page's (at most 64) rows; the lanes issue a tile's copies side
//     by side, each with the table entry it read one tile ahead.
//   * Four consumer warps; a warp owns 16 keys of every tile and its own (max,
//     sum, output), on mma.sync m16n8k16 (the tensor pipe is idle most of the
//     time either way).  An item's end merges the four through shared memory;
//     the other CTA of the SM streams meanwhile.
//   * An item inside one share is written as it is.  One that crosses shares
//     leaves an fp32 partial row set per CTA -- at most two per CTA, one for
//     an item it ends or passes through, one for an item it begins -- and a
//     second kernel, a programmatic dependent, joins them in share order.
//     Items of at most kPdWhole tiles stay whole.
//   * K/V copies are the first to leave the L2 (each is read once): what a
//     call's start needs, the code above all, stays there.
// Measured on B200 (d = 128, 32 / 8 heads, three caches in rotation): 8 sequences
// of 8192 keys 47.9 us = 5.60 TB/s, 64 of 20 to 8192 keys 58 us = 5.69 TB/s (86
// and 87 % of a copy's rate), one of 131072 keys 88.9 us (92 %), of 32768 31.1 (66 %);
// one of 700 keys 8.5 us, which is the fixed cost of
// every call: lengths, table entry and first copy one after the other, the merge
// and the join.  One CTA of eight warps per SM took 136.9 us for the 64 sequences
// (short items leave the SM idle while they are merged), shares without an item
// cost 85.
#pragma once
#include "decode.cuh"
#include "paged.cuh"

namespace sdpa {

constexpr int kPdKeys = 64;                 // keys per tile
constexpr int kPdRows = 16;                 // query rows per item (mma M)
constexpr int kPdWarps = 4;                 // consumer warps, 16 keys of a tile each
constexpr int kPdCtasPerSm = 2;
constexpr int kPdThreads = kPdWarps * 32 + 32;
constexpr int kPdSegRing = 4;               // pieces announced ahead by the producer
constexpr int kPdItemCost = 2;              // an item's fixed cost (query loads, merge, writes) in tiles
constexpr int kPdWhole = 4;                 // items of this many tiles or fewer are not split: joining costs more

struct PagedDecodeParams {
  PagedParams p;
  // 5-D maps (64 columns, page row, column block, head, page); box {64, min(P, 64), d/64, 1, 1}, 128-byte swizzle
  CUtensorMap tm_k;
  CUtensorMap tm_v;
  int row_groups;      // ceil(group * Sq / 16)
  FastDiv div_rg;      // by row_groups
  int oob_page;        // a page index behind the map's last one (reads as zeros)
  float* part_o;       // [2 * CTAs][16][d] locally normalised partial outputs
  float2* part_ml;     // [2 * CTAs][16] (max of scale * q.k, sum)
  int4* joins;         // [CTAs] {first token, head * row_groups + row group, last CTA, tokens} of the item
                       // that begins in the CTA's share and ends in a later one; first token -1: none
  int64_t lse_tok, lse_head;  // element of the lse: lse_tok * tok0 + lse_head * head + token - tok0
};

template <int D>
struct PagedDecodeCfg {
  static constexpr int kHalfBytes = kPdKeys * D * 2;  // K or V tile
  static constexpr int kStageBytes = 2 * kHalfBytes;
  static constexpr int kStages = D == 128 ? 3 : 6;    // 96 KB in flight per CTA
  static constexpr int kMergeFloats = kPdWarps / 2 * kPdRows * (D + 2);
  static constexpr int kBarOffset = kStages * kStageBytes + kMergeFloats * 4;
  static constexpr int kSegOffset = kBarOffset + (2 * kStages + 2 * kPdSegRing) * 8;
  static constexpr int kSumOffset = kSegOffset + kPdSegRing * 32 + 16;
  static constexpr int kSmemBytes = kSumOffset + (kPdWarps + 1 + 2) * 8;
  // two CTAs on an SM's 228 KB, of which 1 KB each is the system's
  static_assert(kPdCtasPerSm * (kSmemBytes + 1024) <= 228 * 1024, "shared memory of two blocks");
};

// Tiles of an item over `len` keys; an empty one takes one as well (its rows are written).
__device__ __forceinline__ int pd_tiles(int len) { return max(1, (len + kPdKeys - 1) / kPdKeys); }

// The tokens of sequence b: all of the decode's Sq; what the full units leave of
// a ragged sequence, where it is little (kRowUnit).
struct PdSeq {
  int tok0, cnt;  // first token's row of q, tokens (0: no item)
  int L;          // keys that any of them sees
  int lim;        // last key that the first token sees (causal)
  int T;          // tiles of an item, 0 without one
};

__device__ __forceinline__ PdSeq pd_of(const PagedParams& p, const PagedSeq& q) {
  PdSeq s;
  const int left = q.n - static_cast<int>(fastdiv(static_cast<uint32_t>(q.n), p.div_tu)) * p.unit_tokens;
  s.cnt = left <= p.row_tokens ? left : 0;
  s.tok0 = q.start + q.n - s.cnt;
  const int coff = p.causal == 2 ? q.L - q.n : 0;
  s.L = paged_visible(p.causal, q.n, q.L, coff);
  s.lim = coff + q.n - s.cnt;
  s.T = s.cnt > 0 ? pd_tiles(s.L) : 0;
  return s;
}

__device__ __forceinline__ PdSeq pd_seq(const PagedParams& p, int b) {
  if (p.cu_q != nullptr) return pd_of(p, paged_seq(p, b));
  PdSeq s;
  s.tok0 = b * p.Sq;
  s.cnt = p.Sq;
  const int L = paged_clamp(p, p.lens[b]);
  s.lim = p.causal == 2 ? L - p.Sq : 0;
  s.L = paged_visible(p.causal, p.Sq, L, s.lim);
  s.T = pd_tiles(s.L);
  return s;
}

// Length of an item on the line.
__device__ __forceinline__ int pd_cost(const PdSeq& s) { return s.T > 0 ? s.T + kPdItemCost : 0; }

// Barrier `id` of a CTA's consumer warps that also tells whether `pred` holds in any thread.
__device__ __forceinline__ bool pd_any(int id, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(pred ? 1u : 0u), "r"(id), "n"(kPdWarps * 32)
      : "memory");
  return r != 0;
}

// Token of a KV head's query row.
__device__ __forceinline__ int row_token(const PagedParams& p, int row) {
  return static_cast<int>(fastdiv(static_cast<uint32_t>(row), p.div_group));
}

// Where a share of the line begins and ends.
struct PdShare {
  int64_t x0, x1, total;
  int G;           // shares
  int64_t prefix;  // places of the sequences before the share's first one, per (head, row group)
  int first;       // that sequence
};

__device__ __forceinline__ PdShare pd_share(int64_t total, int ctas, int cta) {
  PdShare s;
  // every share has a place at least; with fewer places than CTAs the last CTAs have none
  s.total = total;
  s.G = static_cast<int>(min(static_cast<int64_t>(ctas), total));
  s.x0 = cta < s.G ? div64(total * cta, s.G) : 0;
  s.x1 = cta < s.G ? div64(total * (cta + 1), s.G) : 0;
  s.prefix = 0;
  s.first = 0;
  return s;
}

// Shared memory of one CTA's producer and consumers at `smem` (1024-byte aligned: the swizzle's pattern).
template <int D>
struct PdSmem {
  using Cfg = PagedDecodeCfg<D>;
  uint32_t ring;
  float *s_o, *s_m, *s_l;  // merge: [2 warps][16][D], [2][16], [2][16]
  uint32_t bar0;
  // ring of announced pieces: {first token (-1: no more), head * row_groups + row group, first tile, tiles, keys,
  // slot of the partial (-1: whole item), tokens, last key the first token sees}
  volatile int* segs;
  volatile int* abort_flag;
  __device__ __forceinline__ explicit PdSmem(uint8_t* smem) {
    ring = smem_u32(smem);
    s_o = reinterpret_cast<float*>(smem + Cfg::kStages * Cfg::kStageBytes);
    s_m = s_o + kPdWarps / 2 * kPdRows * D;
    s_l = s_m + kPdWarps / 2 * kPdRows;
    bar0 = ring + Cfg::kBarOffset;
    segs = reinterpret_cast<volatile int*>(smem + Cfg::kSegOffset);
    abort_flag = segs + kPdSegRing * 8;
  }
  __device__ __forceinline__ uint32_t full(int s) const { return bar0 + 8u * s; }
  __device__ __forceinline__ uint32_t empty(int s) const { return bar0 + 8u * (Cfg::kStages + s); }
  __device__ __forceinline__ uint32_t seg_full(int s) const { return bar0 + 8u * (2 * Cfg::kStages + s); }
  __device__ __forceinline__ uint32_t seg_empty(int s) const { return bar0 + 8u * (2 * Cfg::kStages + kPdSegRing + s); }
  __device__ __forceinline__ void init() const {  // one thread
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kPdWarps);
    }
    for (int s = 0; s < kPdSegRing; ++s) {
      mbar_init(seg_full(s), 1);
      mbar_init(seg_empty(s), kPdWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
};

// The producer warp of share `sh`, which is CTA number `cta` of the line.
template <int D>
__device__ __forceinline__ void pd_producer(const PagedDecodeParams& a, const PdSmem<D>& sm, const PdShare& sh, int cta,
                                            int lane) {
  using Cfg = PagedDecodeCfg<D>;
  constexpr int NS = Cfg::kStages;
  const PagedParams& p = a.p;
  const int per_seq = p.Hkv * a.row_groups;
  const int pb = min(1 << p.page_shift, kPdKeys);  // rows per copy
  const int pb_shift = min(p.page_shift, 6);
  const int nb = kPdKeys >> pb_shift;              // copies per K (or V) tile
  const uint32_t box_bytes = static_cast<uint32_t>(pb) * D * 2;
  const bool is_v = lane >= nb;
  const int box = is_v ? lane - nb : lane;
  int4 join = make_int4(-1, 0, 0, 0);  // the item that a later share ends
  int64_t join_end = 0;
  int issued = 0, nseg = 0;
  // keys and values are read once (twice with two row groups): what else is in the L2, this kernel's
  // code among it, is worth more
  const uint64_t policy = l2_evict_first();
  bool ok = true;
  auto announce = [&](const PdSeq& q, int hr, int tile, int n, int slot) {
    const int k = nseg % kPdSegRing;
    ok = __all_sync(0xffffffffu, nseg < kPdSegRing ||
                                     mbar_wait(sm.seg_empty(k), ((nseg / kPdSegRing) - 1) & 1, sm.abort_flag));
    if (ok && lane == 0) {
      volatile int* s = sm.segs + 8 * k;
      s[0] = q.tok0;
      s[1] = hr;
      s[2] = tile;
      s[3] = n;
      s[4] = q.L;
      s[5] = slot;
      s[6] = q.cnt;
      s[7] = q.lim;
      mbar_arrive(sm.seg_full(k));
    }
    ++nseg;
  };
  if (sh.x0 < sh.x1) {
    int b = sh.first;
    PdSeq s = pd_seq(p, b);
    const int64_t in_seq = sh.x0 - sh.prefix * per_seq;
    int hr = static_cast<int>(div64(in_seq, s.T + kPdItemCost));
    // places of the share that lie before the item's end: an item's first kPdItemCost places stand
    // for its fixed cost, the others for its tiles
    int64_t xs = sh.prefix * per_seq + static_cast<int64_t>(hr) * (s.T + kPdItemCost);
    int tile = max(0, static_cast<int>(sh.x0 - xs) - kPdItemCost);
    // The table entry of this lane's copy of tile `tl`, or nothing (behind the
    // last key).  It is looked at when the copy is issued, one tile later.
    auto has_copy = [&](int tl, int len) { return lane < 2 * nb && tl * kPdKeys + (box << pb_shift) < len; };
    auto page_of = [&](int bb, int tl, int len) -> int {
      return has_copy(tl, len) ? p.table[static_cast<int64_t>(bb) * p.max_pages +
                                         ((tl * kPdKeys + (box << pb_shift)) >> p.page_shift)]
                               : 0;
    };
    int page = page_of(b, tile, s.L);
    while (ok && xs + kPdItemCost < sh.x1) {
      // a piece: tiles tile .. of item (b, hr), to its end or the share's; an item that is not split
      // belongs to the share that holds its first tile's place
      const bool small = s.T <= kPdWhole;
      const int n = small ? (tile == 0 ? s.T : 0)
                          : static_cast<int>(min(static_cast<int64_t>(s.T), sh.x1 - xs - kPdItemCost)) - tile;
      const bool whole = tile == 0 && n == s.T;
      const int head = static_cast<int>(fastdiv(static_cast<uint32_t>(hr), a.div_rg));
      const int nk = s.L > 0 ? n : 0;
      if (n > 0) announce(s, hr, tile, nk, whole ? -1 : (tile > 0 ? 2 * cta : 2 * cta + 1));
      {
        // the piece's query rows into the first-level cache
        const int r0 = (hr - head * a.row_groups) * kPdRows;
        constexpr int kLines = D * 2 / 128;
        const int r = r0 + lane / kLines;
        if (lane < kPdRows * kLines && r < p.group * s.cnt) {
          const int i = row_token(p, r);
          prefetch_l1(p.q + (static_cast<int64_t>(s.tok0 + i) * p.Hq + head * p.group + r - i * p.group) * D +
                      (lane % kLines) * 64);
        }
      }
      if (p.cu_q == nullptr && tile == 0 && hr == 0 && lane == 0 && p.lens[b] != paged_clamp(p, p.lens[b]))
        atomicOr(&g_error_word, kErrSeqlen);
      if (tile == 0 && n < s.T) {  // (never a small one)
        join = make_int4(s.tok0, hr, 0, s.cnt);
        join_end = xs + kPdItemCost + s.T;
      }
      const int64_t xe = xs + kPdItemCost + s.T;
      const bool more = xe + kPdItemCost < sh.x1;  // the next item has tiles in this share
      int nb2 = b, nhr = hr + 1;
      PdSeq ns = s;
      if (nhr == per_seq) {
        nhr = 0;
        if (more) {
          if (p.cu_q == nullptr) {
            ++nb2;
          } else {  // the next sequence with an item
            unsigned some = 0u;
            for (++nb2; nb2 < p.B && some == 0u; nb2 += 32) {
              some = __ballot_sync(0xffffffffu, nb2 + lane < p.B && pd_seq(p, nb2 + lane).cnt > 0);
              if (some != 0u) nb2 += __ffs(some) - 1 - 32;
            }
            if (some == 0u) break;
          }
          ns = pd_seq(p, nb2);
        }
      }
      for (int i = 0; ok && i < nk; ++i) {
        const int tl = tile + i;
        const int raw = page;
        if (i + 1 < nk) page = page_of(b, tl + 1, s.L);
        else if (more) page = page_of(nb2, 0, ns.L);
        const int st = issued % NS;
        ok = __all_sync(0xffffffffu, mbar_wait(sm.empty(st), ((issued / NS) & 1) ^ 1, sm.abort_flag));
        if (!ok) break;
        const int copies = min(nb, (s.L - tl * kPdKeys + pb - 1) >> pb_shift);
        if (lane == 0) mbar_arrive_expect_tx(sm.full(st), 2u * static_cast<uint32_t>(copies) * box_bytes);
        __syncwarp();
        if (has_copy(tl, s.L)) {
          int cur = raw;
          if (cur < 0 || cur >= p.num_pages) {
            atomicOr(&g_error_word, kErrPage);
            cur = a.oob_page;
          }
          const int row = (tl * kPdKeys + (box << pb_shift)) & ((1 << p.page_shift) - 1);
          tma_load_5d_hint(sm.ring + st * Cfg::kStageBytes + (is_v ? Cfg::kHalfBytes : 0) + box * box_bytes,
                      is_v ? &a.tm_v : &a.tm_k, 0, row, 0, head, cur, sm.full(st), policy);
        }
        ++issued;
      }
      if (nk == 0 && more) page = page_of(nb2, 0, ns.L);
      xs = xe;
      b = nb2;
      hr = nhr;
      s = ns;
      tile = 0;
    }
  }
  // the CTA whose share holds its last tile
  if (join.x >= 0) join.z = static_cast<int>(div64(join_end * sh.G - 1, sh.total));
  if (lane == 0) a.joins[cta] = join;
  if (ok) announce(PdSeq{-1, 0, 0, 0, 0}, 0, 0, 0, 0);
  // copies still in flight must land before the CTA may exit
  if (lane == 0)
    for (int it = max(0, issued - NS); it < issued; ++it) mbar_wait_drain(sm.full(it % NS), (it / NS) & 1);
  __syncwarp();
}

// A consumer warp (0 .. 3); the four meet at named barrier `bar`.
template <int D>
__device__ __forceinline__ void pd_consumer(const PagedDecodeParams& a, const PdSmem<D>& sm, int warp, int lane, int bar) {
  using Cfg = PagedDecodeCfg<D>;
  constexpr int NS = Cfg::kStages;
  const PagedParams& p = a.p;
  const int tid = warp * 32 + lane;
  const float c = p.scale_log2;
  const int kb = warp * 16;            // this warp's 16 keys of a tile
  const int qr = lane >> 2;            // fragment row (and row + 8)
  const int qc = (lane & 3) * 2;       // fragment column pair
  const int pb_shift = min(p.page_shift, 6);
  const uint32_t blk_bytes = 128u << pb_shift;          // one 64-column block of a copy
  const uint32_t box_bytes = blk_bytes * (D / 64);
  const int mi = lane >> 3;
  // Shared-memory offset of (tile key r, column c): copy r / pb, then 64-column
  // block, then row r mod pb of 128 bytes with its 16-byte chunks swizzled.
  auto tile_off = [&](int r, int col) -> uint32_t {
    const int in_box = r & ((1 << pb_shift) - 1);
    return static_cast<uint32_t>(r >> pb_shift) * box_bytes + static_cast<uint32_t>(col >> 6) * blk_bytes +
           in_box * 128u + ((((col & 63) >> 3) ^ (r & 7)) << 4);
  };
  const int k_row = kb + (mi >> 1) * 8 + (lane & 7);    // rows that ldmatrix reads of K and of V
  const int v_row = kb + (mi & 1) * 8 + (lane & 7);
  // 16 columns further on is 32 bytes under the swizzle (an exclusive or: the row starts on 128 bytes)
  const uint32_t k_base = tile_off(k_row, (mi & 1) * 8), v_base = tile_off(v_row, (mi >> 1) * 8);
  int it0 = 0;  // tiles of the CTA's earlier pieces
  for (int sg = 0;; ++sg) {
    const int sk = sg % kPdSegRing;
    bool ok = __all_sync(0xffffffffu, mbar_wait(sm.seg_full(sk), (sg / kPdSegRing) & 1, sm.abort_flag));
    int tok0 = -1, hr = 0, tile0 = 0, n = 0, L = 0, cnt = 0, lim0 = 0;
    if (ok) {
      volatile int* s = sm.segs + 8 * sk;
      tok0 = s[0];
      hr = s[1];
      tile0 = s[2];
      n = s[3];
      L = s[4];
      cnt = s[6];
      lim0 = s[7];
    }
    int head = static_cast<int>(fastdiv(static_cast<uint32_t>(hr), a.div_rg));
    int row0 = (hr - head * a.row_groups) * kPdRows;  // first of the head's query rows
    const int rows = min(kPdRows, p.group * cnt - row0);
    float o[D / 8][4];
#pragma unroll
    for (int e = 0; e < D / 8; ++e) o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY};
    float l[2] = {0.f, 0.f};
    if (ok && tok0 >= 0 && n > 0) {
      // query row r of the head: token r / group, head r mod group
      uint32_t qf[D / 16][4];
      int lim[2];  // last key that rows qr and qr + 8 see
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = qr + 8 * h;
        const bool live = r < rows;
        const int i = live ? row_token(p, row0 + r) : 0;
        const int g = live ? row0 + r - i * p.group : 0;
        lim[h] = L - 1;
        if (p.causal && live) lim[h] = min(lim[h], lim0 + i);
        const uint32_t* q = reinterpret_cast<const uint32_t*>(
            p.q + (static_cast<int64_t>(tok0 + i) * p.Hq + head * p.group + g) * D);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          qf[ks][h] = live ? q[(ks * 16 + qc) >> 1] : 0u;
          qf[ks][2 + h] = live ? q[(ks * 16 + 8 + qc) >> 1] : 0u;
        }
      }
      for (int i = 0; i < n; ++i) {
        const int it = it0 + i;
        const int st = it % NS;
        if (!__all_sync(0xffffffffu, mbar_wait(sm.full(st), (it / NS) & 1, sm.abort_flag))) {
          ok = false;
          break;
        }
        const uint32_t sK = sm.ring + st * Cfg::kStageBytes + k_base;
        const uint32_t sV = sm.ring + st * Cfg::kStageBytes + Cfg::kHalfBytes + v_base;
        const int key0 = (tile0 + i) * kPdKeys + kb;
        if (key0 < L) {  // warp-uniform
          float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t b0, b1, b2, b3;
            ldmatrix_x4((sK ^ ((ks & 3) << 5)) + (ks >> 2) * blk_bytes, b0, b1, b2, b3);
            mma_bf16_16816(sc[0], qf[ks], b0, b1);
            mma_bf16_16816(sc[1], qf[ks], b2, b3);
          }
          if (key0 + 15 > min(lim[0], lim[1])) {
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (key0 + nt * 8 + qc + (e & 1) > lim[e >> 1]) sc[nt][e] = -INFINITY;
          }
          float alpha[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float mx = fmaxf(fmaxf(sc[0][2 * h], sc[0][2 * h + 1]), fmaxf(sc[1][2 * h], sc[1][2 * h + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float m_new = fmaxf(m[h], mx);
            alpha[h] = (m[h] == -INFINITY) ? 0.f : ex2_approx((m[h] - m_new) * c);
            m[h] = m_new;
          }
          uint32_t pa[4];
          {
            const float mc0 = (m[0] == -INFINITY) ? 0.f : m[0] * c;
            const float mc1 = (m[1] == -INFINITY) ? 0.f : m[1] * c;
            const float p00 = ex2_approx(fmaf(sc[0][0], c, -mc0)), p01 = ex2_approx(fmaf(sc[0][1], c, -mc0));
            const float p02 = ex2_approx(fmaf(sc[0][2], c, -mc1)), p03 = ex2_approx(fmaf(sc[0][3], c, -mc1));
            const float p10 = ex2_approx(fmaf(sc[1][0], c, -mc0)), p11 = ex2_approx(fmaf(sc[1][1], c, -mc0));
            const float p12 = ex2_approx(fmaf(sc[1][2], c, -mc1)), p13 = ex2_approx(fmaf(sc[1][3], c, -mc1));
            l[0] = l[0] * alpha[0] + (p00 + p01 + p10 + p11);
            l[1] = l[1] * alpha[1] + (p02 + p03 + p12 + p13);
            // the product with V takes bf16: one rounding of every probability
            pa[0] = pack_bf16x2(p00, p01);
            pa[1] = pack_bf16x2(p02, p03);
            pa[2] = pack_bf16x2(p10, p11);
            pa[3] = pack_bf16x2(p12, p13);
          }
          // most tiles leave every maximum where it was
          if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
            for (int e = 0; e < D / 8; ++e) {
              o[e][0] *= alpha[0];
              o[e][1] *= alpha[0];
              o[e][2] *= alpha[1];
              o[e][3] *= alpha[1];
            }
          }
          // Rows of V behind the last key hold whatever the page holds, and 0
          // times infinity or NaN is NaN: those keys' values are zeroed.  A
          // fragment register has keys qc, qc + 1 (b0, b2) or qc + 8, qc + 9.
          const bool tail = key0 + 16 > L;  // warp-uniform
          uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
          if (tail) {
            const int left = L - key0 - qc;  // keys of this lane's pair that exist
            keep0 = left >= 2 ? 0xffffffffu : (left == 1 ? 0xffffu : 0u);
            keep1 = left >= 10 ? 0xffffffffu : (left == 9 ? 0xffffu : 0u);
          }
#pragma unroll
          for (int e = 0; e < D / 8; e += 2) {
            uint32_t b0, b1, b2, b3;
            ldmatrix_x4_trans((sV ^ (((e >> 1) & 3) << 5)) + (e >> 3) * blk_bytes, b0, b1, b2, b3);
            if (tail) {
              b0 &= keep0;
              b1 &= keep1;
              b2 &= keep0;
              b3 &= keep1;
            }
            mma_bf16_16816(o[e], pa, b0, b1);
            mma_bf16_16816(o[e + 1], pa, b2, b3);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(sm.empty(st));
      }
      it0 += n;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      }
    }
    // ---- merge of the four warps: the upper two leave their rows in shared
    // memory, the lower two add them to their own and leave the sums there.  A
    // row's columns are exchanged by eights so that four rows fill the 32 banks.
    const int mw = warp & 1;
    int x = qr;
    asm volatile("" : "+r"(x));  // the offsets below are not to be held in registers over the tiles
    const uint32_t part = smem_u32(sm.s_o) + ((mw * kPdRows + x) * D + qc) * 4;  // row qr's column qc of eight 0
    auto leave = [&]() {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = qr + 8 * h;
        if (r < rows) {
#pragma unroll
          for (int e = 0; e < D / 8; ++e)
            st_shared_f2(part + h * (8 * D * 4) + (e & ~3) * 32 + (((e ^ x) & 3) << 5), o[e][2 * h], o[e][2 * h + 1]);
          if ((lane & 3) == 0) {
            sm.s_m[mw * kPdRows + r] = m[h];
            sm.s_l[mw * kPdRows + r] = l[h];
          }
        }
      }
    };
    if (n > 0 && warp >= 2) leave();
    // every consumer meets here once per piece, and all of them leave together
    if (pd_any(bar, !ok) || tok0 < 0) break;
    if (n > 0 && warp < 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = qr + 8 * h;
        if (r < rows) {
          const float m1 = sm.s_m[mw * kPdRows + r], l1 = sm.s_l[mw * kPdRows + r];
          const float M = fmaxf(m[h], m1);  // (-inf where a warp saw nothing)
          const float w0 = saw_nothing(m[h], l[h]) ? 0.f : ex2_approx((m[h] - M) * c);
          const float w1 = saw_nothing(m1, l1) ? 0.f : ex2_approx((m1 - M) * c);
          m[h] = M;
          l[h] = l[h] * w0 + l1 * w1;
#pragma unroll
          for (int e = 0; e < D / 8; ++e) {
            const float2 y = ld_shared_f2(part + h * (8 * D * 4) + (e & ~3) * 32 + (((e ^ x) & 3) << 5));
            o[e][2 * h] = o[e][2 * h] * w0 + y.x * w1;
            o[e][2 * h + 1] = o[e][2 * h + 1] * w0 + y.y * w1;
          }
        }
      }
      __syncwarp();  // the warp has read the rows it now overwrites
      leave();
    }
    named_bar_sync(bar, kPdWarps * 32);
    // the announced piece again: it need not stay in registers over the tiles
    tok0 = sm.segs[8 * sk];
    hr = sm.segs[8 * sk + 1];
    const int slot = sm.segs[8 * sk + 5];
    head = static_cast<int>(fastdiv(static_cast<uint32_t>(hr), a.div_rg));
    row0 = (hr - head * a.row_groups) * kPdRows;
    __syncwarp();
    if (lane == 0) mbar_arrive(sm.seg_empty(sk));
    // 8 threads per row, D/8 consecutive columns each
    const int r = tid >> 3;
    if (r < rows) {
      constexpr int kCols = D / 8;
      const int c0 = (tid & 7) * kCols;
      float M = -INFINITY, sum = 0.f;
      float wt[kPdWarps / 2];
      float acc[kCols];
#pragma unroll
      for (int e = 0; e < kCols; ++e) acc[e] = 0.f;
      if (n > 0) {
#pragma unroll
        for (int w = 0; w < kPdWarps / 2; ++w) M = fmaxf(M, sm.s_m[w * kPdRows + r]);
#pragma unroll
        for (int w = 0; w < kPdWarps / 2; ++w) {
          const float lw = sm.s_l[w * kPdRows + r], mw = sm.s_m[w * kPdRows + r];
          wt[w] = saw_nothing(mw, lw) ? 0.f : ex2_approx((mw - M) * c);
          sum += wt[w] * lw;
        }
#pragma unroll
        for (int w = 0; w < kPdWarps / 2; ++w)
#pragma unroll
          for (int e = 0; e < kCols; e += 4) {
            const float4 v = *reinterpret_cast<const float4*>(&sm.s_o[(w * kPdRows + r) * D + ((c0 + e) ^ ((r & 3) * 8))]);
            acc[e] += wt[w] * v.x;
            acc[e + 1] += wt[w] * v.y;
            acc[e + 2] += wt[w] * v.z;
            acc[e + 3] += wt[w] * v.w;
          }
      }
      const bool empty = saw_nothing(M, sum);
      const float inv = empty ? 0.f : 1.f / sum;
      if (slot < 0) {
        const int i = row_token(p, row0 + r);
        const int hq = head * p.group + row0 + r - i * p.group;
        uint16_t* const dst = p.o + (static_cast<int64_t>(tok0 + i) * p.Hq + hq) * D + c0;
#pragma unroll
        for (int e = 0; e < kCols; e += 4)
          *reinterpret_cast<uint2*>(dst + e) = make_uint2(pack_bf16x2(acc[e] * inv, acc[e + 1] * inv),
                                                          pack_bf16x2(acc[e + 2] * inv, acc[e + 3] * inv));
        if (c0 == 0 && p.lse != nullptr)
          p.lse[a.lse_tok * tok0 + a.lse_head * hq + i] =
              empty ? -INFINITY : M * p.scale + lg2_approx(sum) * 0.69314718055994531f;
      } else {
        float* const dst = a.part_o + (static_cast<int64_t>(slot) * kPdRows + r) * D + c0;
#pragma unroll
        for (int e = 0; e < kCols; e += 4)
          *reinterpret_cast<float4*>(dst + e) =
              make_float4(acc[e] * inv, acc[e + 1] * inv, acc[e + 2] * inv, acc[e + 3] * inv);
        if (c0 == 0) a.part_ml[slot * kPdRows + r] = make_float2(empty ? -INFINITY : M * p.scale, sum);
      }
    }
    named_bar_sync(bar, kPdWarps * 32);  // the merge buffer is read
  }
}

template <int D>
__global__ void __launch_bounds__(kPdThreads, kPdCtasPerSm) paged_decode_kernel(const __grid_constant__ PagedDecodeParams a) {
  using Cfg = PagedDecodeCfg<D>;
  const PagedParams& p = a.p;
  extern __shared__ __align__(1024) uint8_t smem[];
  const PdSmem<D> sm(smem);
  int64_t* const s_sum = reinterpret_cast<int64_t*>(smem + Cfg::kSumOffset);  // [5]
  int64_t& s_prefix = s_sum[kPdWarps + 1];
  int64_t& s_first = s_sum[kPdWarps + 2];
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    sm.init();
    s_first = s_prefix = 0;
  }
  paged_warm(p);
  if (warp == kPdWarps && lane == 0) {
    tma_prefetch_desc(&a.tm_k);
    tma_prefetch_desc(&a.tm_v);
  }
  __syncthreads();
  // Launched as a programmatic dependent of whatever precedes it on the stream:
  // no global memory is read or written before this wait (the lines asked for above go
  // to the L2 only).
  grid_dependency_wait();
  grid_dependency_trigger();

  // ---- this CTA's share of the line
  const int per_seq = p.Hkv * a.row_groups;  // items per sequence
  const int cta = static_cast<int>(blockIdx.x);
  const int ctas = static_cast<int>(gridDim.x);
  int64_t total = 0;
  PdShare sh;
  // Inclusive sum of t over the block's threads so far, and their total.
  auto block_scan = [&](int t, int64_t& incl, int64_t& all) {
    int w_incl = t;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w_incl, off);
      if (lane >= off) w_incl += u;
    }
    if (lane == 31) s_sum[warp] = w_incl;
    __syncthreads();
    incl = w_incl;
    all = 0;
#pragma unroll
    for (int w = 0; w < kPdThreads / 32; ++w) {
      if (w < warp) incl += s_sum[w];
      all += s_sum[w];
    }
  };
  auto find = [&](int b, int t, int64_t end) {  // sequence b's places end at `end`
    if (t > 0 && (end - t) * per_seq <= sh.x0 && sh.x0 < end * per_seq) {
      s_first = b;
      s_prefix = end - t;
    }
  };
  if (p.B <= kPdThreads) {
    const int t = static_cast<int>(threadIdx.x) < p.B ? pd_cost(pd_seq(p, threadIdx.x)) : 0;
    int64_t incl;
    block_scan(t, incl, total);
    total *= per_seq;
    sh = pd_share(total, ctas, cta);
    find(threadIdx.x, t, incl);
  } else {
    int64_t mine = 0;
    for (int b = threadIdx.x; b < p.B; b += kPdThreads) mine += pd_cost(pd_seq(p, b));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, off);
    if (lane == 0) s_sum[warp] = mine;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPdThreads / 32; ++w) total += s_sum[w];
    total *= per_seq;
    sh = pd_share(total, ctas, cta);
    int64_t base = 0;
    for (int b0 = 0; b0 < p.B && sh.x0 < sh.x1 && base * per_seq <= sh.x0; b0 += kPdThreads) {  // block-uniform
      const int b = b0 + static_cast<int>(threadIdx.x);
      const int t = b < p.B ? pd_cost(pd_seq(p, b)) : 0;
      __syncthreads();  // s_sum's previous contents are read
      int64_t incl, all;
      block_scan(t, incl, all);
      find(b, t, base + incl);
      base += all;
    }
  }
  __syncthreads();

  sh.first = static_cast<int>(s_first);
  sh.prefix = s_prefix;
  if (warp == kPdWarps) pd_producer<D>(a, sm, sh, cta, lane);
  else pd_consumer<D>(a, sm, warp, lane, 1);
}

// Join the partial rows of the items that cross shares: block c takes the item
// that begins in CTA c's share, one warp per row.  With w_s = l_s exp(m_s - M),
// M = max_s m_s: o = sum_s w_s o_s / sum_s w_s, lse = M + ln sum_s w_s.  All that
// an item of up to kJoinRows pieces needs is loaded at once, before it is known
// which pieces there are (what is read beyond them is not used): one memory
// latency, not one per step.
constexpr int kJoinRows = 8;

template <int D>
__device__ __forceinline__ void paged_decode_join(const PagedDecodeParams& a, int cta, int ctas) {
  constexpr int kPer = D / 32;
  constexpr float kLog2e = 1.4426950408889634f;
  const PagedParams& p = a.p;
  const int r = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // piece 0 lies in CTA cta's slot for the item it begins, piece s in CTA cta + s's for the one it continues
  auto slot_row = [&](int s) { return (2 * min(cta + s, ctas - 1) + (s == 0 ? 1 : 0)) * kPdRows + r; };
  auto load = [&](int s, float (&x)[kPer]) {
    const float* src = a.part_o + static_cast<int64_t>(slot_row(s)) * D + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; e += 2) {
      const float2 t = *reinterpret_cast<const float2*>(src + e);
      x[e] = t.x;
      x[e + 1] = t.y;
    }
  };
  const int4 join = a.joins[cta];
  float2 ml = a.part_ml[slot_row(lane)];
  float x[kJoinRows][kPer];
#pragma unroll
  for (int u = 0; u < kJoinRows; ++u) load(u, x[u]);
  if (join.x < 0) return;
  const int head = static_cast<int>(fastdiv(static_cast<uint32_t>(join.y), a.div_rg));
  const int row = (join.y - head * a.row_groups) * kPdRows + r;  // of the head's query rows
  if (row >= p.group * join.w) return;
  const int pieces = join.z - cta + 1;
  float M = -INFINITY;
  bool some = false;  // whether any piece saw a key
  for (int s0 = 0; s0 < pieces; s0 += 32) {
    const float2 v = s0 == 0 ? ml : a.part_ml[slot_row(s0 + lane)];
    if (s0 + lane < pieces && !saw_nothing(v.x, v.y)) {
      M = fmaxf(M, v.x);
      some = true;
    }
  }
  some = __any_sync(0xffffffffu, some);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  float W = 0.f;
  if (some) {
    float w_lane = 0.f;
    for (int s0 = 0; s0 < pieces; s0 += kJoinRows) {
      if ((s0 & 31) == 0) {
        if (s0 > 0) ml = a.part_ml[slot_row(s0 + lane)];
        w_lane = s0 + lane < pieces && !saw_nothing(ml.x, ml.y) ? ml.y * ex2_approx((ml.x - M) * kLog2e) : 0.f;
      }
      if (s0 > 0) {
#pragma unroll
        for (int u = 0; u < kJoinRows; ++u) load(s0 + u, x[u]);
      }
#pragma unroll
      for (int u = 0; u < kJoinRows; ++u) {
        const float w = __shfl_sync(0xffffffffu, w_lane, (s0 + u) & 31);
        if (s0 + u < pieces) {
          W += w;
#pragma unroll
          for (int e = 0; e < kPer; ++e) acc[e] = fmaf(w, x[u][e], acc[e]);
        }
      }
    }
  }
  const float inv = some ? 1.f / W : 0.f;
  const int i = row_token(p, row);
  const int hq = head * p.group + row - i * p.group;
  uint16_t* const dst = p.o + (static_cast<int64_t>(join.x + i) * p.Hq + hq) * D + lane * kPer;
#pragma unroll
  for (int e = 0; e < kPer; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0 && p.lse != nullptr)
    p.lse[a.lse_tok * join.x + a.lse_head * hq + i] =
        some ? M + lg2_approx(W) * 0.69314718055994531f : -INFINITY;
}

template <int D>
__global__ void __launch_bounds__(kPdRows * 32) paged_decode_join_kernel(const __grid_constant__ PagedDecodeParams a) {
  grid_dependency_trigger();
  grid_dependency_wait();
  paged_decode_join<D>(a, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
}

}  // namespace sdpa
