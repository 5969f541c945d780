// paged.cuh -- attention over a paged KV cache.
//
// Key j of sequence b lives in row j mod P of page table[b][j / P] (P = page
// size, a power of two).  For query token i of the n_b tokens of sequence b
// with L_b keys, head hq, hk = hq / (Hq / Hkv):
//     x_j = scale * q . k_j   for visible j,   o = sum_j softmax(x)_j v_j,
//     lse = ln sum_j exp(x_j),
// key j being visible iff j < L_b and, under the bottom-right causal mask,
// j <= i + L_b - n_b.  Whatever a page holds behind a sequence's last key has no
// effect, infinities and NaN included.
#pragma once
#include "fastdiv.h"
#include "paged_ptx.cuh"

namespace sdpa {

// The forward takes a sequence's tokens in units of two 128-row tiles.  What the
// full units leave is the decode's work where it is no more query rows of a KV
// head than this: a single token's, mostly.
constexpr int kRowUnit = 16;

// Lengths, offsets, tables and q may be what the grid before has just written, and these kernels start before
// it ends (programmatic dependents): they are read with ordinary loads behind the dependency wait.  A
// non-coherent load (ld.global.nc, __ldg) is for data that nobody writes while the kernel lives, and the compiler
// may move it over the wait.
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
  FastDiv div_group;
  int row_tokens;      // ragged batch: tokens that kRowUnit rows hold, kRowUnit / group
  int unit_tokens;     // ragged batch: tokens of a full unit
  FastDiv div_tu;      // by unit_tokens
};

// A number of keys, clamped to what a row of the table can hold (2^30 at most).
__device__ __forceinline__ int paged_clamp(const PagedParams& p, int len) {
  return min(max(len, 0), p.max_pages << p.page_shift);
}

// Keys that the first `tokens` tokens of a sequence see together: token i sees
// key j iff j < L and, under a causal mask, j <= i + coff.
__device__ __forceinline__ int paged_visible(int causal, int64_t tokens, int L, int coff) {
  return causal ? static_cast<int>(min(max(tokens + coff, int64_t{0}), static_cast<int64_t>(L))) : L;
}

// A ragged sequence's first token, its tokens and its keys, clamped to the
// batch and the table (`bad`: something was).
struct PagedSeq {
  int start, n, L;
  bool bad;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int b) {
  const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1], raw = p.lens[b];
  PagedSeq s;
  s.start = min(max(c0, 0), p.T);
  const int end = min(max(c1, s.start), p.T);
  s.n = end - s.start;
  s.L = paged_clamp(p, raw);
  s.bad = s.start != c0 || end != c1 || s.L != raw;
  return s;
}

// Asks for the lengths and the table (a line per thread of the grid) while the grid before still runs: into the L2,
// where what that grid writes of them arrives as well.  64 caches of 20 to 8192 keys 58.1 -> 57.8 us, 129 tokens
// behind 32639 keys 95.9 -> 95.1.
__device__ __forceinline__ void paged_warm(const PagedParams& p) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 32;
  if (i < static_cast<int64_t>(p.B) * p.max_pages) prefetch_l2(p.table + i);
  if (i < p.B) {
    prefetch_l2(p.lens + i);
    if (p.cu_q != nullptr) prefetch_l2(p.cu_q + i);
  }
}

// Whether a row (or a piece of its keys) with this running maximum and sum saw no key.  Only then is it left out:
// a NaN score, or one of +infinity, makes the sum NaN (the maximum passes over a NaN), and that has to reach the
// row's output and lse through every merge and join.
__device__ __forceinline__ bool saw_nothing(float m, float l) { return m == -INFINITY && l == 0.f; }

// a / b of non-negative values, by the 32-bit division where both fit.
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

}  // namespace sdpa
