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

// a / b of non-negative values, by the 32-bit division where both fit.
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

}  // namespace sdpa
