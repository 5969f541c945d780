// page_plan.cuh -- block tables and slot maps of a paged KV cache, built on
// the device from the requests' lengths.
//
// Request b holds past_b keys in ceil(past_b / P) pages (P = page size) and
// asks for new_b more.  With held_b = ceil(past_b / P), need_b =
// ceil((past_b + new_b) / P) - held_b and C_b the inclusive prefix sum of
// need over the requests, request b is granted iff need_b = 0 or C_b <= free;
// its pages are entries C_b - need_b .. C_b - 1 of the free list.  Token t of
// the ragged batch belongs to the request whose [cu_b, cu_{b+1}) holds it and
// goes to slot table[b][pos / P] * P + pos mod P with pos = past_b + t - cu_b.
//
// Two prefix sums and one lookup per token: a few bytes per token, so the
// kernel is bound by the latency of its dependent steps (lengths -> scan ->
// search -> table entry -> store).  Hence one launch: every CTA of a single
// thread-block cluster scans all requests for itself (no exchange through
// global memory), the cluster meets once, and the tokens are then spread over
// all of its threads.  Nothing that an output may alias is read after that
// meeting, so lengths and free range can be advanced in place.  Measured: 3.2 us
// for one token each of 8 requests, 6.5 us for 40 K tokens of 512.
#pragma once
#include <climits>

#include "paged_ptx.cuh"

namespace sdpa {

struct PlanParams {
  const int* past;        // [B]
  const int* fresh;       // [B] new tokens
  int* table;             // [B][max_pages], new entries written
  const int* free_pages;  // [num_free]
  const int* free_range;  // [2] {head, tail}
  int* cu;                // [B + 1]
  int* total;             // [B]
  int* positions;         // [T]
  int* slots;             // [T]
  int* range_out;         // [2]
  int B, max_pages, num_free, T;
  int page_shift;         // log2 P
};

constexpr int kPlanThreads = 512;
constexpr int kPlanTokens = 2;          // consecutive tokens per thread and pass (1: 2.7 / 10.4 us, 2: 3.0 / 8.5,
                                        // 4: 3.7 / 8.6 for 8 tokens of 8 requests / 40 K tokens of 512)
constexpr int kPlanMaxBatch = 16384;    // 3 ints of shared memory per request
constexpr int kPlanMaxCluster = 16;     // with more than kPlanSmallBatch requests 8, the portable size: their CTAs'
constexpr int kPlanSmallBatch = 4096;   // tables may leave room for one CTA per SM only
constexpr uint32_t kPlanCap = (1u << 30) + 1;  // prefix sums saturate here: above every legal total (T is at most 2^30)
constexpr int kPlanNotGranted = INT_MIN;

inline int plan_smem_bytes(int B) { return (3 * B + 1) * 4; }

// Saturating sum of two values <= kPlanCap (associative, cannot wrap).
__device__ __forceinline__ uint32_t plan_add(uint32_t a, uint32_t b) { return min(a + b, kPlanCap); }

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ int plan_smem[];
  int* const s_cu = plan_smem;            // [B + 1] first token of each request
  int* const s_past = s_cu + p.B + 1;     // [B] keys it holds
  int* const s_first = s_past + p.B;      // [B] free-list entry minus held pages, or kPlanNotGranted
  __shared__ uint32_t s_tok[kPlanThreads / 32], s_need[kPlanThreads / 32];
  __shared__ uint32_t s_used;             // pages granted
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = 1 << p.page_shift;
  const int64_t cap_keys = static_cast<int64_t>(p.max_pages) << p.page_shift;
  // a programmatic dependent of what precedes it, and what follows may be one of this kernel
  grid_dependency_trigger();
  grid_dependency_wait();

  const int raw_head = p.free_range[0], raw_tail = p.free_range[1];
  const int head = min(max(raw_head, 0), p.num_free);
  const int tail = min(max(raw_tail, head), p.num_free);
  const uint32_t free = static_cast<uint32_t>(tail - head);
  bool bad = head != raw_head || tail != raw_tail;
  if (tid == 0) s_used = 0;

  uint32_t tok_base = 0, need_base = 0;  // totals of the earlier requests
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int past = 0, n = 0;
    uint32_t need = 0;
    bool valid = true;
    if (b < p.B) {
      past = p.past[b];
      n = p.fresh[b];
      valid = past >= 0 && n >= 0 && static_cast<int64_t>(past) + n <= cap_keys;
      n = min(max(n, 0), static_cast<int>(kPlanCap));
      if (valid) need = ((past + n + P - 1) >> p.page_shift) - ((past + P - 1) >> p.page_shift);
    }
    uint32_t ti = static_cast<uint32_t>(n), ni = need;  // inclusive sums over the warp, then the block
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, ti, off), c = __shfl_up_sync(0xffffffffu, ni, off);
      if (lane >= off) {
        ti = plan_add(ti, a);
        ni = plan_add(ni, c);
      }
    }
    __syncthreads();  // the previous round's warp totals are read
    if (lane == 31) {
      s_tok[warp] = ti;
      s_need[warp] = ni;
    }
    __syncthreads();
    uint32_t tb = tok_base, nb = need_base;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      if (w == warp) {
        ti = plan_add(ti, tb);
        ni = plan_add(ni, nb);
      }
      tb = plan_add(tb, s_tok[w]);
      nb = plan_add(nb, s_need[w]);
    }
    tok_base = tb;
    need_base = nb;
    if (b < p.B) {
      const uint32_t T = static_cast<uint32_t>(p.T);
      // a request whose tokens do not fit the buffers gets nothing
      if (ti > T) valid = false;
      const bool granted = valid && (need == 0 || ni <= free);
      s_cu[b + 1] = static_cast<int>(min(ti, T));
      s_past[b] = past;
      const int held = static_cast<int>((static_cast<int64_t>(past) + P - 1) >> p.page_shift);
      s_first[b] = granted ? head + static_cast<int>(ni - need) - held : kPlanNotGranted;
      if (!granted) bad = true;
      if (granted && need > 0) atomicMax(&s_used, ni);
    }
  }
  if (tid == 0) s_cu[0] = 0;
  __syncthreads();
  const int ctas = static_cast<int>(gridDim.x);  // one cluster
  if (ctas > 1) cluster_sync();

  const bool wide = ((reinterpret_cast<uintptr_t>(p.positions) | reinterpret_cast<uintptr_t>(p.slots)) & 7u) == 0;
  const int live = s_cu[p.B];
  const int step = ctas * kPlanThreads * kPlanTokens;
  for (int t0 = (static_cast<int>(blockIdx.x) * kPlanThreads + tid) * kPlanTokens; t0 < p.T; t0 += step) {
    int pos[kPlanTokens], slot[kPlanTokens];
    int b = 0;
    if (t0 < live) {  // last request that starts at or before t0
      int lo = 0, hi = p.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= t0) lo = mid;
        else hi = mid;
      }
      b = lo;
    }
#pragma unroll
    for (int u = 0; u < kPlanTokens; ++u) {
      const int t = t0 + u;
      pos[u] = slot[u] = -1;
      if (t < live) {
        while (t >= s_cu[b + 1]) ++b;
        const int past = s_past[b], first = s_first[b];
        // a refused length keeps its tokens' places in the batch; their
        // positions are meaningful only where past is (wraps otherwise)
        pos[u] = static_cast<int>(static_cast<uint32_t>(past) + static_cast<uint32_t>(t - s_cu[b]));
        if (first != kPlanNotGranted) {
          const int j = pos[u] >> p.page_shift;
          const int held = (past + P - 1) >> p.page_shift;
          int* const entry = p.table + static_cast<int64_t>(b) * p.max_pages + j;
          int page;
          if (j >= held) {
            page = p.free_pages[first + j];
            if ((pos[u] & (P - 1)) == 0) *entry = page;  // the page's first token
          } else {
            page = *entry;
          }
          // an entry whose slots are no int32 gives the token no slot
          if (page >= 0 && page <= (INT_MAX >> p.page_shift))
            slot[u] = (page << p.page_shift) | (pos[u] & (P - 1));
          else
            atomicOr(&g_error_word, kErrPage);
        }
      }
    }
    if (wide && t0 + kPlanTokens <= p.T) {
      *reinterpret_cast<int2*>(p.positions + t0) = make_int2(pos[0], pos[1]);
      *reinterpret_cast<int2*>(p.slots + t0) = make_int2(slot[0], slot[1]);
    } else {
#pragma unroll
      for (int u = 0; u < kPlanTokens; ++u)
        if (t0 + u < p.T) {
          p.positions[t0 + u] = pos[u];
          p.slots[t0 + u] = slot[u];
        }
    }
  }
  if (blockIdx.x == 0) {
    for (int b = tid; b < p.B; b += kPlanThreads) {
      p.cu[b] = s_cu[b];
      const int n = s_cu[b + 1] - s_cu[b];
      p.total[b] = s_first[b] == kPlanNotGranted ? s_past[b] : s_past[b] + n;
    }
    if (tid == 0) {
      p.cu[p.B] = s_cu[p.B];
      p.range_out[0] = head + static_cast<int>(s_used);
      p.range_out[1] = tail;
    }
    if (bad) atomicOr(&g_error_word, kErrPage);
  }
}

}  // namespace sdpa
