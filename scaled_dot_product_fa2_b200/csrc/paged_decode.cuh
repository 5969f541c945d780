// paged_decode.cuh -- split-KV decode attention over a paged KV cache.
//
// A work item is (sequence, KV head, group of up to 16 query rows that share
// the head); its keys are walked in tiles of 64 with one running maximum,
// sum and output per row (see paged.cuh for the formula).  The kernel does
// two products per key for at most 16 rows, so its floor is the bytes of the
// valid keys and values, and all of the design serves the memory system:
//   * All items' tiles form one line, in the order (sequence, head, row
//     group), and the grid -- one CTA per SM -- cuts it into equal shares.
//     A share may begin and end inside an item, so the longest CTA does one
//     tile more than the shortest, whatever the lengths are.  The line is
//     measured on the device: every CTA sums the tile counts for itself and
//     finds its first item; nothing about the lengths is known on the host.
//   * One producer warp streams K/V tiles through a ring of kStages slots and
//     does not stop at item borders: the ring keeps the next item's tiles in
//     flight while an item's result is merged and written.  One TMA copy
//     brings a page's (at most 64) rows; the lanes issue a tile's copies side
//     by side, each with the table entry it read one tile ahead.
//   * Eight consumer warps, in two sets of four that take tiles in turn; a
//     warp owns 16 keys of a tile and its own (max, sum, output), on
//     mma.sync m16n8k16 (the tensor pipe is idle most of the time either
//     way).  An item's end merges the eight through shared memory.
//   * An item inside one share is written as it is.  One that crosses shares
//     leaves an fp32 partial row set per CTA -- at most two per CTA, one for
//     an item it ends or passes through, one for an item it begins -- and a
//     second kernel, a programmatic dependent, joins them in share order.
#pragma once
#include "decode.cuh"
#include "paged.cuh"

namespace sdpa {

constexpr int kPdKeys = 64;                 // keys per tile
constexpr int kPdRows = 16;                 // query rows per item (mma M)
constexpr int kPdWarps = 8;                 // consumer warps
constexpr int kPdThreads = kPdWarps * 32 + 32;
constexpr int kPdSegRing = 4;               // pieces announced ahead by the producer

struct PagedDecodeParams {
  PagedParams p;
  // 5-D maps (64 columns, page row, column block, head, page); box {64, min(P, 64), d/64, 1, 1}, 128-byte swizzle
  CUtensorMap tm_k;
  CUtensorMap tm_v;
  int row_groups;      // ceil(group * Sq / 16)
  int oob_page;        // a page index behind the map's last one (reads as zeros)
  float* part_o;       // [2 * CTAs][16][d] locally normalised partial outputs
  float2* part_ml;     // [2 * CTAs][16] (max of scale * q.k, sum)
  int4* joins;         // [CTAs] {sequence, head * row_groups + row group, last CTA, -} of the item that
                       // begins in the CTA's share and ends in a later one; sequence -1: none
};

template <int D>
struct PagedDecodeCfg {
  static constexpr int kHalfBytes = kPdKeys * D * 2;  // K or V tile
  static constexpr int kStageBytes = 2 * kHalfBytes;
  static constexpr int kStages = D == 128 ? 6 : 12;   // 192 KB in flight per SM
  // A slot belongs to one set of warps for good: a set that met a slot only every other time could
  // look at its barrier one phase too early (copies land in any order) and take the phase before
  // last for its own.
  static_assert(kStages % 2 == 0, "the sets take tiles, and with them slots, in turn");
  static constexpr int kMergeFloats = kPdWarps / 2 * kPdRows * (D + 2);
  static constexpr int kBarOffset = kStages * kStageBytes + kMergeFloats * 4;
  static constexpr int kSegOffset = kBarOffset + (2 * kStages + 2 * kPdSegRing) * 8;
  static constexpr int kSmemBytes = kSegOffset + kPdSegRing * 32 + 16 + 1024;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per block");
};

__device__ __forceinline__ int paged_len(const PagedParams& p, int b) {
  const int64_t cap = static_cast<int64_t>(p.max_pages) << p.page_shift;
  return static_cast<int>(min(static_cast<int64_t>(max(__ldg(p.lens + b), 0)), cap));
}

// Tiles of sequence b on the line; an empty one takes a place as well (its rows are written).
__device__ __forceinline__ int pd_tiles(const PagedParams& p, int b) {
  return max(1, (paged_len(p, b) + kPdKeys - 1) / kPdKeys);
}

// Barrier of the consumer warps that also tells whether `pred` holds in any thread.
__device__ __forceinline__ bool pd_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(pred ? 1u : 0u), "n"(kPdWarps * 32)
      : "memory");
  return r != 0;
}

template <int D>
__global__ void __launch_bounds__(kPdThreads, 1) paged_decode_kernel(const __grid_constant__ PagedDecodeParams a) {
  using Cfg = PagedDecodeCfg<D>;
  constexpr int NS = Cfg::kStages;
  const PagedParams& p = a.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = smem_u32(smem);
  float* const s_o = reinterpret_cast<float*>(smem + NS * Cfg::kStageBytes);  // [4 warps][16][D]
  float* const s_m = s_o + kPdWarps / 2 * kPdRows * D;                        // [4][16]
  float* const s_l = s_m + kPdWarps / 2 * kPdRows;                            // [4][16]
  const uint32_t bar0 = ring + Cfg::kBarOffset;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (NS + s); };
  auto seg_full = [&](int s) { return bar0 + 8u * (2 * NS + s); };
  auto seg_empty = [&](int s) { return bar0 + 8u * (2 * NS + kPdSegRing + s); };
  // ring of announced pieces: {sequence (-1: no more), head * row_groups + row group, first tile, tiles, keys, slot
  // of the partial (-1: whole item)}
  volatile int* const segs = reinterpret_cast<volatile int*>(smem + Cfg::kSegOffset);
  volatile int* const abort_flag = segs + kPdSegRing * 8;
  __shared__ int64_t s_sum[kPdThreads / 32];
  __shared__ int64_t s_prefix;  // tiles of the sequences before this CTA's first one
  __shared__ int s_first;       // that sequence
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kPdWarps / 2);
    }
    for (int s = 0; s < kPdSegRing; ++s) {
      mbar_init(seg_full(s), 1);
      mbar_init(seg_empty(s), kPdWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kPdWarps && lane == 0) {
    tma_prefetch_desc(&a.tm_k);
    tma_prefetch_desc(&a.tm_v);
  }
  __syncthreads();
  // Launched as a programmatic dependent of whatever precedes it on the stream:
  // no global memory is touched before this wait.
  grid_dependency_wait();
  grid_dependency_trigger();

  // ---- this CTA's share of the line
  const int per_seq = p.Hkv * a.row_groups;  // items per sequence
  int64_t mine = 0;
  for (int b = threadIdx.x; b < p.B; b += kPdThreads) mine += pd_tiles(p, b);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, off);
  if (lane == 0) s_sum[warp] = mine;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kPdThreads / 32; ++w) total += s_sum[w];
  total *= per_seq;
  // every share has a tile at least; with fewer tiles than CTAs the last CTAs have none
  const int cta = static_cast<int>(blockIdx.x);
  const int G = static_cast<int>(min(static_cast<int64_t>(gridDim.x), total));
  const int64_t x0 = cta < G ? total * cta / G : 0;
  const int64_t x1 = cta < G ? total * (cta + 1) / G : 0;
  // the sequence that holds tile x0
  int64_t base = 0;
  for (int b0 = 0; b0 < p.B && x0 < x1; b0 += kPdThreads) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    const int t = b < p.B ? pd_tiles(p, b) : 0;
    int64_t incl = t;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += u;
    }
    __syncthreads();  // s_sum's previous contents are read
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int64_t block = 0;
#pragma unroll
    for (int w = 0; w < kPdThreads / 32; ++w) {
      if (w < warp) incl += s_sum[w];
      block += s_sum[w];
    }
    if (t > 0 && (base + incl - t) * per_seq <= x0 && x0 < (base + incl) * per_seq) {
      s_first = b;
      s_prefix = base + incl - t;
    }
    base += block;
    if (base * per_seq > x0) break;  // block-uniform
  }
  __syncthreads();

  if (warp == kPdWarps) {
    // ------------------------------------------------------------ producer
    const int pb = min(1 << p.page_shift, kPdKeys);  // rows per copy
    const int pb_shift = min(p.page_shift, 6);
    const int nb = kPdKeys >> pb_shift;              // copies per K (or V) tile
    const uint32_t box_bytes = static_cast<uint32_t>(pb) * D * 2;
    const bool is_v = lane >= nb;
    const int box = is_v ? lane - nb : lane;
    int4 join = make_int4(-1, 0, 0, 0);
    int issued = 0, nseg = 0;
    bool ok = true;
    auto announce = [&](int b, int hr, int tile, int n, int L, int slot) {
      const int k = nseg % kPdSegRing;
      ok = __all_sync(0xffffffffu, nseg < kPdSegRing ||
                                       mbar_wait(seg_empty(k), ((nseg / kPdSegRing) - 1) & 1, abort_flag));
      if (ok && lane == 0) {
        volatile int* s = segs + 8 * k;
        s[0] = b;
        s[1] = hr;
        s[2] = tile;
        s[3] = n;
        s[4] = L;
        s[5] = slot;
        mbar_arrive(seg_full(k));
      }
      ++nseg;
    };
    if (x0 < x1) {
      int b = s_first;
      int L = paged_len(p, b);
      int T = max(1, (L + kPdKeys - 1) / kPdKeys);
      const int64_t in_seq = x0 - s_prefix * per_seq;
      int hr = static_cast<int>(in_seq / T);
      int tile = static_cast<int>(in_seq - static_cast<int64_t>(hr) * T);
      // the page of this lane's copy of tile `tl`: a table entry, oob_page when it is none, -1 behind the last key
      auto page_of = [&](int bb, int tl, int len) -> int {
        const int key = tl * kPdKeys + (box << pb_shift);
        if (lane >= 2 * nb || key >= len) return -1;
        int page = __ldg(p.table + static_cast<int64_t>(bb) * p.max_pages + (key >> p.page_shift));
        if (page < 0 || page >= p.num_pages) {
          atomicOr(&g_error_word, kErrPage);
          page = a.oob_page;
        }
        return page;
      };
      int page = page_of(b, tile, L);
      int64_t x = x0;
      while (ok && x < x1) {
        // a piece: tiles tile .. of item (b, hr), to its end or the share's
        const int n = static_cast<int>(min(static_cast<int64_t>(T - tile), x1 - x));
        const bool whole = tile == 0 && n == T;
        if (tile == 0 && hr == 0 && lane == 0 && __ldg(p.lens + b) != L) atomicOr(&g_error_word, kErrSeqlen);
        if (tile == 0 && n < T) {
          const int64_t last = x + T - 1;  // the item's last tile, and the CTA whose share holds it
          join = make_int4(b, hr, static_cast<int>(((last + 1) * G - 1) / total), 0);
        }
        const int nk = L > 0 ? n : 0;
        announce(b, hr, tile, nk, L, whole ? -1 : (tile > 0 ? 2 * cta : 2 * cta + 1));
        const int head = hr / a.row_groups;
        int nb2 = b, nhr = hr + 1, nL = L, nT = T;  // the item behind this one
        if (nhr == per_seq) {
          nhr = 0;
          nb2 = b + 1;
          if (x + n < x1) {
            nL = paged_len(p, nb2);
            nT = max(1, (nL + kPdKeys - 1) / kPdKeys);
          }
        }
        for (int i = 0; ok && i < nk; ++i) {
          const int tl = tile + i;
          const int cur = page;
          if (i + 1 < nk) page = page_of(b, tl + 1, L);
          else if (x + n < x1) page = page_of(nb2, 0, nL);
          const int st = issued % NS;
          ok = __all_sync(0xffffffffu, mbar_wait(empty(st), ((issued / NS) & 1) ^ 1, abort_flag));
          if (!ok) break;
          const int copies = min(nb, (L - tl * kPdKeys + pb - 1) >> pb_shift);
          if (lane == 0) mbar_arrive_expect_tx(full(st), 2u * static_cast<uint32_t>(copies) * box_bytes);
          __syncwarp();
          if (cur >= 0) {
            const int row = (tl * kPdKeys + (box << pb_shift)) & ((1 << p.page_shift) - 1);
            tma_load_5d(ring + st * Cfg::kStageBytes + (is_v ? Cfg::kHalfBytes : 0) + box * box_bytes,
                        is_v ? &a.tm_v : &a.tm_k, 0, row, 0, head, cur, full(st));
          }
          ++issued;
        }
        if (nk == 0 && x + n < x1) page = page_of(nb2, 0, nL);
        x += n;
        b = nb2;
        hr = nhr;
        L = nL;
        T = nT;
        tile = 0;
      }
    }
    if (lane == 0) a.joins[cta] = join;
    if (ok) announce(-1, 0, 0, 0, 0, 0);
    // copies still in flight must land before the CTA may exit
    if (lane == 0)
      for (int it = max(0, issued - NS); it < issued; ++it) mbar_wait_drain(full(it % NS), (it / NS) & 1);
    __syncwarp();
    return;
  }

  // ------------------------------------------------------------ consumers
  const float c = p.scale_log2;
  const int set = warp >> 2;           // which of every two tiles
  const int kb = (warp & 3) * 16;      // this warp's 16 keys of a tile
  const int qr = lane >> 2;            // fragment row (and row + 8)
  const int qc = (lane & 3) * 2;       // fragment column pair
  const int rows_total = p.group * p.Sq;
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
    bool ok = __all_sync(0xffffffffu, mbar_wait(seg_full(sk), (sg / kPdSegRing) & 1, abort_flag));
    int b = -1, hr = 0, tile0 = 0, n = 0, L = 0, slot = 0;
    if (ok) {
      volatile int* s = segs + 8 * sk;
      b = s[0];
      hr = s[1];
      tile0 = s[2];
      n = s[3];
      L = s[4];
      slot = s[5];
      __syncwarp();
      if (lane == 0) mbar_arrive(seg_empty(sk));
    }
    const int head = hr / a.row_groups;
    const int row0 = (hr - head * a.row_groups) * kPdRows;  // first of the head's query rows
    const int rows = min(kPdRows, rows_total - row0);
    float o[D / 8][4];
#pragma unroll
    for (int e = 0; e < D / 8; ++e) o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY};
    float l[2] = {0.f, 0.f};
    if (ok && b >= 0 && n > 0) {
      // query row r of the head: token r / group, head r mod group
      uint32_t qf[D / 16][4];
      int lim[2];  // last key that rows qr and qr + 8 see
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = qr + 8 * h;
        const bool live = r < rows;
        const int i = live ? (row0 + r) / p.group : 0;
        const int g = live ? row0 + r - i * p.group : 0;
        lim[h] = L - 1;
        if (p.causal && live) lim[h] = min(lim[h], p.causal == 2 ? L - p.Sq + i : i);
        const uint32_t* q = reinterpret_cast<const uint32_t*>(
            p.q + ((static_cast<int64_t>(b) * p.Sq + i) * p.Hq + head * p.group + g) * D);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          qf[ks][h] = live ? __ldg(q + ((ks * 16 + qc) >> 1)) : 0u;
          qf[ks][2 + h] = live ? __ldg(q + ((ks * 16 + 8 + qc) >> 1)) : 0u;
        }
      }
      // tile number it of the CTA goes to set it mod 2
      for (int i = (it0 ^ set) & 1; i < n; i += 2) {
        const int it = it0 + i;
        const int st = it % NS;
        if (!__all_sync(0xffffffffu, mbar_wait(full(st), (it / NS) & 1, abort_flag))) {
          ok = false;
          break;
        }
        const uint32_t sK = ring + st * Cfg::kStageBytes + k_base;
        const uint32_t sV = ring + st * Cfg::kStageBytes + Cfg::kHalfBytes + v_base;
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
#pragma unroll
          for (int e = 0; e < D / 8; ++e) {
            o[e][0] *= alpha[0];
            o[e][1] *= alpha[0];
            o[e][2] *= alpha[1];
            o[e][3] *= alpha[1];
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
        if (lane == 0) mbar_arrive(empty(st));
      }
      it0 += n;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      }
    }
    // ---- merge of the eight warps: the second set leaves its rows in shared
    // memory, the first adds them to its own and leaves the sums there.
    const int mw = warp & 3;
    auto leave = [&]() {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = qr + 8 * h;
        if (r < rows) {
#pragma unroll
          for (int e = 0; e < D / 8; ++e)
            *reinterpret_cast<float2*>(&s_o[(mw * kPdRows + r) * D + e * 8 + qc]) =
                make_float2(o[e][2 * h], o[e][2 * h + 1]);
          if ((lane & 3) == 0) {
            s_m[mw * kPdRows + r] = m[h];
            s_l[mw * kPdRows + r] = l[h];
          }
        }
      }
    };
    if (n > 0 && set == 1) leave();
    // every consumer meets here once per piece, and all of them leave together
    if (pd_any(!ok) || b < 0) break;
    if (n > 0 && set == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = qr + 8 * h;
        if (r < rows) {
          const float m1 = s_m[mw * kPdRows + r], l1 = s_l[mw * kPdRows + r];
          const float M = fmaxf(l[h] > 0.f ? m[h] : -INFINITY, l1 > 0.f ? m1 : -INFINITY);
          const float w0 = l[h] > 0.f ? ex2_approx((m[h] - M) * c) : 0.f;
          const float w1 = l1 > 0.f ? ex2_approx((m1 - M) * c) : 0.f;
          m[h] = M;
          l[h] = l[h] * w0 + l1 * w1;
#pragma unroll
          for (int e = 0; e < D / 8; ++e) {
            const float2 x = *reinterpret_cast<const float2*>(&s_o[(mw * kPdRows + r) * D + e * 8 + qc]);
            o[e][2 * h] = o[e][2 * h] * w0 + x.x * w1;
            o[e][2 * h + 1] = o[e][2 * h + 1] * w0 + x.y * w1;
          }
        }
      }
      __syncwarp();  // the warp has read the rows it now overwrites
      leave();
    }
    named_bar_sync(1, kPdWarps * 32);
    // 16 threads per row, D/16 consecutive columns each
    const int r = static_cast<int>(threadIdx.x) >> 4;
    if (r < rows) {
      constexpr int kCols = D / 16;
      const int c0 = (static_cast<int>(threadIdx.x) & 15) * kCols;
      float M = -INFINITY, sum = 0.f;
      float wt[kPdWarps / 2];
      float acc[kCols];
#pragma unroll
      for (int e = 0; e < kCols; ++e) acc[e] = 0.f;
      if (n > 0) {
#pragma unroll
        for (int w = 0; w < kPdWarps / 2; ++w)
          if (s_l[w * kPdRows + r] > 0.f) M = fmaxf(M, s_m[w * kPdRows + r]);
#pragma unroll
        for (int w = 0; w < kPdWarps / 2; ++w) {
          const float lw = s_l[w * kPdRows + r];
          wt[w] = lw > 0.f ? ex2_approx((s_m[w * kPdRows + r] - M) * c) : 0.f;
          sum += wt[w] * lw;
        }
#pragma unroll
        for (int w = 0; w < kPdWarps / 2; ++w)
#pragma unroll
          for (int e = 0; e < kCols; e += 4) {
            const float4 v = *reinterpret_cast<const float4*>(&s_o[(w * kPdRows + r) * D + c0 + e]);
            acc[e] += wt[w] * v.x;
            acc[e + 1] += wt[w] * v.y;
            acc[e + 2] += wt[w] * v.z;
            acc[e + 3] += wt[w] * v.w;
          }
      }
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      if (slot < 0) {
        const int i = (row0 + r) / p.group;
        const int hq = head * p.group + row0 + r - i * p.group;
        uint16_t* const dst = p.o + ((static_cast<int64_t>(b) * p.Sq + i) * p.Hq + hq) * D + c0;
#pragma unroll
        for (int e = 0; e < kCols; e += 4)
          *reinterpret_cast<uint2*>(dst + e) = make_uint2(pack_bf16x2(acc[e] * inv, acc[e + 1] * inv),
                                                          pack_bf16x2(acc[e + 2] * inv, acc[e + 3] * inv));
        if (c0 == 0 && p.lse != nullptr)
          p.lse[(static_cast<int64_t>(b) * p.Hq + hq) * p.Sq + i] =
              sum > 0.f ? M * p.scale + lg2_approx(sum) * 0.69314718055994531f : -INFINITY;
      } else {
        float* const dst = a.part_o + (static_cast<int64_t>(slot) * kPdRows + r) * D + c0;
#pragma unroll
        for (int e = 0; e < kCols; e += 4)
          *reinterpret_cast<float4*>(dst + e) =
              make_float4(acc[e] * inv, acc[e + 1] * inv, acc[e + 2] * inv, acc[e + 3] * inv);
        if (c0 == 0) a.part_ml[slot * kPdRows + r] = make_float2(sum > 0.f ? M * p.scale : -INFINITY, sum);
      }
    }
    named_bar_sync(1, kPdWarps * 32);  // the merge buffer is read
  }
}

// Join the partial rows of the items that cross shares: block c takes the item
// that begins in CTA c's share, one warp per row.  With w_s = l_s exp(m_s - M),
// M = max_s m_s: o = sum_s w_s o_s / sum_s w_s, lse = M + ln sum_s w_s.
template <int D>
__global__ void __launch_bounds__(kPdRows * 32) paged_decode_join_kernel(const __grid_constant__ PagedDecodeParams a) {
  constexpr int kPer = D / 32;
  constexpr float kLog2e = 1.4426950408889634f;
  const PagedParams& p = a.p;
  grid_dependency_trigger();
  grid_dependency_wait();
  const int cta = static_cast<int>(blockIdx.x);
  const int4 join = a.joins[cta];
  const int r = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (join.x < 0) return;
  const int head = join.y / a.row_groups;
  const int row = (join.y - head * a.row_groups) * kPdRows + r;  // of the head's query rows
  if (row >= p.group * p.Sq) return;
  const int pieces = join.z - cta + 1;
  // piece 0 lies in CTA cta's slot for the item it begins, piece s in CTA cta + s's for the one it continues
  auto slot_row = [&](int s) { return static_cast<int64_t>(2 * (cta + s) + (s == 0 ? 1 : 0)) * kPdRows + r; };
  float M = -INFINITY;
  for (int s = lane; s < pieces; s += 32) {
    const float2 v = a.part_ml[slot_row(s)];
    if (v.y > 0.f) M = fmaxf(M, v.x);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  float W = 0.f;
  if (M != -INFINITY) {
#pragma unroll 4
    for (int s = 0; s < pieces; ++s) {
      const float2 v = a.part_ml[slot_row(s)];
      const float w = v.y > 0.f ? v.y * ex2_approx((v.x - M) * kLog2e) : 0.f;
      W += w;
      const float* src = a.part_o + slot_row(s) * D + lane * kPer;
#pragma unroll
      for (int e = 0; e < kPer; e += 2) {
        const float2 x = *reinterpret_cast<const float2*>(src + e);
        acc[e] = fmaf(w, x.x, acc[e]);
        acc[e + 1] = fmaf(w, x.y, acc[e + 1]);
      }
    }
  }
  const float inv = W > 0.f ? 1.f / W : 0.f;
  const int i = row / p.group;
  const int hq = head * p.group + row - i * p.group;
  uint16_t* const dst = p.o + ((static_cast<int64_t>(join.x) * p.Sq + i) * p.Hq + hq) * D + lane * kPer;
#pragma unroll
  for (int e = 0; e < kPer; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0 && p.lse != nullptr)
    p.lse[(static_cast<int64_t>(join.x) * p.Hq + hq) * p.Sq + i] =
        W > 0.f ? M + lg2_approx(W) * 0.69314718055994531f : -INFINITY;
}

}  // namespace sdpa
