// paged.cuh -- attention over a paged KV cache.
//
// Key j of sequence b lives in row j mod P of page table[b][j / P] (P = page
// size, a power of two).  For query token i of the n_b tokens of sequence b
// with L_b keys, head hq, hk = hq / (Hq / Hkv):
//     x_j = scale * q . k_j   for visible j,   o = sum_j softmax(x)_j v_j,
//     lse = ln sum_j exp(x_j),
// key j being visible iff j < L_b and, under the bottom-right causal mask,
// j <= i + L_b - n_b.  Keys that are not visible are never read, so whatever a
// page holds behind a sequence's last key has no effect.
#pragma once
#include "fastdiv.h"
#include "ptx.cuh"

namespace sdpa {

struct PagedParams {
  const uint16_t* q;   // [T][Hq][d] bf16 (the decode: T = B * Sq)
  const uint16_t* k;   // element (page, head, row, c) at page*sp + head*sh + row*sr + c
  const uint16_t* v;
  int64_t sp, sh, sr;
  uint16_t* o;         // [T][Hq][d]
  float* lse;          // nullptr, [Hq][T] (ragged batch) or [B][Hq][Sq] (decode)
  const int* cu_q;     // [B + 1], or nullptr: Sq tokens per sequence
  const int* lens;     // [B] keys per sequence
  const int* table;    // [B][max_pages]
  int B, T, Sq, Hq, Hkv, group;
  int num_pages, max_pages, page_shift;
  int causal;          // 0 none, 1 top-left, 2 bottom-right
  float scale, scale_log2;
};

// One warp per (token, query head), the lanes sharing its d columns.
template <int D>
__global__ void __launch_bounds__(256) paged_rows_kernel(const __grid_constant__ PagedParams p) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t rows = static_cast<int64_t>(p.T) * p.Hq;
  if (row >= rows) return;
  const int t = static_cast<int>(row / p.Hq);
  const int hq = static_cast<int>(row - static_cast<int64_t>(t) * p.Hq);
  const int hk = hq / p.group;
  int b, i, n;
  if (p.cu_q == nullptr) {
    b = t / p.Sq;
    i = t - b * p.Sq;
    n = p.Sq;
  } else {
    // last sequence that starts at or before t
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu_q + mid) <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
    const int c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1);
    if (t < c0 || t >= c1) return;  // behind the last sequence
    i = t - c0;
    n = c1 - c0;
  }
  const int raw = __ldg(p.lens + b);
  const int64_t cap = static_cast<int64_t>(p.max_pages) << p.page_shift;
  const int L = static_cast<int>(min(static_cast<int64_t>(max(raw, 0)), cap));
  if (raw != L && lane == 0) atomicOr(&g_error_word, kErrSeqlen);
  int64_t last = L - 1;
  if (p.causal) last = min(last, static_cast<int64_t>(i) + (p.causal == 2 ? L - n : 0));
  float q[kPer], o[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    q[e] = bf16_bits_to_float(p.q[row * D + lane * kPer + e]);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j <= last; ++j) {
    const int page = __ldg(p.table + static_cast<int64_t>(b) * p.max_pages + (j >> p.page_shift));
    const bool good = page >= 0 && page < p.num_pages;
    if (!good && lane == 0) atomicOr(&g_error_word, kErrPage);
    const int64_t off = good ? page * p.sp + hk * p.sh + (j & ((1 << p.page_shift) - 1)) * p.sr + lane * kPer : 0;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) s += good ? q[e] * bf16_bits_to_float(p.k[off + e]) : 0.f;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float m_new = fmaxf(m, s);
    const float a = ex2_approx((m - m_new) * p.scale_log2);
    const float w = ex2_approx((s - m_new) * p.scale_log2);
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] = o[e] * a + (good ? w * bf16_bits_to_float(p.v[off + e]) : 0.f);
    m = m_new;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < kPer; e += 2)
    *reinterpret_cast<uint32_t*>(p.o + row * D + lane * kPer + e) = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
  if (lane == 0 && p.lse != nullptr) {
    const int64_t at = p.cu_q == nullptr ? (static_cast<int64_t>(b) * p.Hq + hq) * p.Sq + i
                                         : static_cast<int64_t>(hq) * p.T + t;
    p.lse[at] = l > 0.f ? m * p.scale + lg2_approx(l) * 0.69314718055994531f : -INFINITY;
  }
}

}  // namespace sdpa
