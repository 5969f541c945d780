// paged_host.cuh -- host side of the paged KV cache's entry points: argument
// checks and launches.  Included by sdpa_b200.cu after the shared helpers.
#pragma once

namespace sdpa {
namespace {

constexpr int kMinPage = 16, kMaxPage = 256;

bool page_size_ok(int P) { return P >= kMinPage && P <= kMaxPage && (P & (P - 1)) == 0; }

int log2_of(int P) {
  int s = 0;
  while ((1 << s) < P) ++s;
  return s;
}

// Checks of a paged cache; the strides (page, head, row) in elements.
attn_status_t check_cache(const attn_paged_cache_t* c, int Hkv, int d, bool has_table, int64_t* sp, int64_t* sh,
                          int64_t* sr) {
  if (c == nullptr) return ATTN_ERR_NULL;
  if (c->num_pages < 0 || (has_table && c->max_pages < 0)) return ATTN_ERR_SHAPE;
  if (c->layout != ATTN_LAYOUT_BHSD && c->layout != ATTN_LAYOUT_BSHD) return ATTN_ERR_SHAPE;
  if (!page_size_ok(c->page_size)) return ATTN_ERR_PAGE;
  if (static_cast<int64_t>(c->num_pages) * c->page_size > (int64_t{1} << 31)) return ATTN_ERR_SHAPE;
  if (has_table && static_cast<int64_t>(c->max_pages) * c->page_size > kMaxSeq) return ATTN_ERR_SHAPE;
  const int64_t dense = static_cast<int64_t>(Hkv) * c->page_size * d;
  if (c->page_stride != 0 && (c->page_stride < dense || c->page_stride % 8 != 0)) return ATTN_ERR_PAGE;
  // a tensor map's strides are below 2^40 bytes
  if (c->page_stride >= (int64_t{1} << 38) || dense >= (int64_t{1} << 38)) return ATTN_ERR_SHAPE;
  if (c->num_pages > 0) {
    if (c->k_pages == nullptr || c->v_pages == nullptr) return ATTN_ERR_NULL;
    if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16)) return ATTN_ERR_ALIGN;
  }
  if (has_table && c->max_pages > 0) {
    if (c->block_table == nullptr) return ATTN_ERR_NULL;
    if (!aligned(c->block_table, 4)) return ATTN_ERR_ALIGN;
  }
  *sp = c->page_stride != 0 ? c->page_stride : dense;
  const Strides s = layout_strides(c->layout, Hkv, c->page_size, d);
  *sh = s.h;
  *sr = s.r;
  return ATTN_OK;
}

// Checks that attn_fwd_paged and attn_decode_splitkv_paged share, and the
// parameters that do not depend on the entry point.
attn_status_t paged_params(PagedParams* p, const void* q, const attn_paged_cache_t* cache, const int* lens, void* o,
                           float* lse, int B, int64_t T, int Hq, int Hkv, int d, float scale, int causal) {
  if (B < 0 || T < 0 || Hq <= 0 || Hkv <= 0 || d <= 0) return ATTN_ERR_SHAPE;
  if (T > kMaxSeq || B > kMaxSeq || Hq > (1 << 20)) return ATTN_ERR_SHAPE;
  if (Hq % Hkv != 0) return ATTN_ERR_GQA;
  if (d != 64 && d != 128) return ATTN_ERR_HEADDIM;
  if (causal < ATTN_CAUSAL_NONE || causal > ATTN_CAUSAL_BOTTOM_RIGHT) return ATTN_ERR_CAUSAL;
  if (!(scale >= 0.f) || std::isinf(scale)) return ATTN_ERR_SCALE;
  std::memset(p, 0, sizeof(*p));
  const attn_status_t s = check_cache(cache, Hkv, d, true, &p->sp, &p->sh, &p->sr);
  if (s != ATTN_OK) return s;
  if (B > 0 && T > 0) {
    if (q == nullptr || o == nullptr || lens == nullptr) return ATTN_ERR_NULL;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lens, 4)) return ATTN_ERR_ALIGN;
    if (lse != nullptr && !aligned(lse, 4)) return ATTN_ERR_ALIGN;
  }
  p->q = static_cast<const uint16_t*>(q);
  p->k = static_cast<const uint16_t*>(cache->k_pages);
  p->v = static_cast<const uint16_t*>(cache->v_pages);
  p->o = static_cast<uint16_t*>(o);
  p->lse = lse;
  p->lens = lens;
  p->table = cache->block_table;
  p->B = B;
  p->T = static_cast<int>(T);
  p->Hq = Hq;
  p->Hkv = Hkv;
  p->group = Hq / Hkv;
  p->num_pages = cache->num_pages;
  p->max_pages = cache->max_pages;
  p->page_shift = log2_of(cache->page_size);
  p->div_group = make_fastdiv(static_cast<uint32_t>(p->group));
  p->row_tokens = kRowUnit / p->group;
  p->causal = causal;
  p->scale = effective_scale(scale, d);
  p->scale_log2 = p->scale * 1.4426950408889634f;
  return ATTN_OK;
}

// 5-D map (64 columns, page row, 64-column block, head, page) over a pool of pages; box {64, rows,
// blocks, 1, 1}: one copy brings `rows` rows of a page as `blocks` blocks of 128-byte swizzled rows.
// Without pages the map has one (of `base`, never read: its index is not a valid one).
bool make_page_map(CUtensorMap* map, const void* base, const PagedParams& p, int d, int rows, int blocks) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[5] = {64, cuuint64_t{1} << p.page_shift, static_cast<cuuint64_t>(d / 64),
                              static_cast<cuuint64_t>(p.Hkv), static_cast<cuuint64_t>(std::max(p.num_pages, 1))};
  const cuuint64_t strides[4] = {static_cast<cuuint64_t>(p.sr) * 2, 128, static_cast<cuuint64_t>(p.sh) * 2,
                                 static_cast<cuuint64_t>(p.sp) * 2};
  const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(rows), static_cast<cuuint32_t>(blocks), 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch as a programmatic dependent of what precedes it on the stream.
struct PdlLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  PdlLaunch(unsigned grid, int threads, int smem, cudaStream_t st, unsigned cluster = 1) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 1) {
      attr[1].id = cudaLaunchAttributeClusterDimension;
      attr[1].val.clusterDim.x = cluster;
      attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
      cfg.numAttrs = 2;
    }
  }
};

// Whether an item or unit can be split at all: the table must hold more keys than those that stay whole.
static_assert(kPdWhole * kPdKeys == kPfWholePair * 128 && kPfWholeThin >= kPfWholePair, "one limit for all of them");
bool paged_can_split(const PagedParams& p) {
  return (static_cast<int64_t>(p.max_pages) << p.page_shift) > kPdWhole * kPdKeys;
}

// The decode's workspace: two partial row sets and one join per CTA of the grid.
size_t paged_decode_ws_bytes(int sms, int d) {
  return static_cast<size_t>(kPdCtasPerSm * sms) * (2 * kPdRows * (static_cast<size_t>(d) * sizeof(float) + sizeof(float2)) +
                                     sizeof(int4));
}

template <int D>
attn_status_t launch_paged_decode(const PagedDecodeParams& a, int sms, int dev, cudaStream_t st) {
  static bool smem_done[kMaxDevices] = {};
  static std::mutex mu;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!set_smem(paged_decode_kernel<D>, PagedDecodeCfg<D>::kSmemBytes, dev, smem_done)) return ATTN_ERR_CUDA;
  }
  PdlLaunch l(static_cast<unsigned>(kPdCtasPerSm * sms), kPdThreads, PagedDecodeCfg<D>::kSmemBytes, st);
  if (cudaLaunchKernelEx(&l.cfg, paged_decode_kernel<D>, a) != cudaSuccess) return ATTN_ERR_CUDA;
  if (!paged_can_split(a.p)) return ATTN_OK;
  PdlLaunch j(static_cast<unsigned>(kPdCtasPerSm * sms), kPdRows * 32, 0, st);
  return cudaLaunchKernelEx(&j.cfg, paged_decode_join_kernel<D>, a) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// What the decode kernel needs besides the parameters: tensor maps over the pages (`q` where there are
// none), and its part of the workspace.
bool paged_rows_params(PagedDecodeParams* a, int d, int sms, void* workspace) {
  const bool pages = a->p.num_pages > 0;
  a->oob_page = std::max(a->p.num_pages, 1);
  const int box = std::min(1 << a->p.page_shift, kPdKeys);
  a->part_o = static_cast<float*>(workspace);
  a->part_ml = reinterpret_cast<float2*>(a->part_o + static_cast<size_t>(2 * kPdCtasPerSm * sms) * kPdRows * d);
  a->joins = reinterpret_cast<int4*>(a->part_ml + static_cast<size_t>(2 * kPdCtasPerSm * sms) * kPdRows);
  return make_page_map(&a->tm_k, pages ? a->p.k : a->p.q, a->p, d, box, d / 64) &&
         make_page_map(&a->tm_v, pages ? a->p.v : a->p.q, a->p, d, box, d / 64);
}

// The forward's own part of its workspace: two partial row sets of two tiles and one join per CTA; the
// decode's part follows.
size_t paged_units_ws_bytes(int sms, int d) {
  return static_cast<size_t>(sms) * (2 * 2 * 128 * (static_cast<size_t>(d) * sizeof(float) + sizeof(float2)) +
                                     2 * sizeof(int4));
}

template <int D, int NS, bool SPLIT>
attn_status_t launch_paged_fwd_split(const PagedFwdParams& a, const PagedDecodeParams& r, int sms, int dev,
                                     cudaStream_t st) {
  static bool smem_done[kMaxDevices] = {};
  static std::mutex mu;
  using Cfg = PagedFwdCfg<D, NS>;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!smem_done[dev]) {
      // the register split (setmaxnreg) adds up to this launch allocation, as in launch_prefill
      cudaFuncAttributes fa;
      if (cudaFuncGetAttributes(&fa, paged_fwd_kernel<D, NS, SPLIT>) != cudaSuccess || fa.numRegs != kLaunchRegs)
        return ATTN_ERR_CUDA;
    }
    if (!set_smem(paged_fwd_kernel<D, NS, SPLIT>, Cfg::kSmemBytes, dev, smem_done)) return ATTN_ERR_CUDA;
  }
  const int ctas = sms & ~1;
  PdlLaunch l(static_cast<unsigned>(ctas), kPrefillThreads, Cfg::kSmemBytes, st, 2);
  if (cudaLaunchKernelEx(&l.cfg, paged_fwd_kernel<D, NS, SPLIT>, a, r) != cudaSuccess) return ATTN_ERR_CUDA;
  if (!SPLIT) return ATTN_OK;
  PdlLaunch j(static_cast<unsigned>(kPfJoinBlocksPerSm * ctas), kPfJoinThreads, 0, st);
  return cudaLaunchKernelEx(&j.cfg, paged_fwd_join_kernel<D>, a, r) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int D, int NS>
attn_status_t launch_paged_fwd(const PagedFwdParams& a, const PagedDecodeParams& r, int sms, int dev,
                               cudaStream_t st) {
  return paged_can_split(a.p) ? launch_paged_fwd_split<D, NS, true>(a, r, sms, dev, st)
                              : launch_paged_fwd_split<D, NS, false>(a, r, sms, dev, st);
}

// 4-D map (d, head in group, KV head, token) over q [T, Hq, d]; box {64, hc, 1, tpt}, 128-byte swizzle.
bool make_packed_q_map(CUtensorMap* map, const void* q, const PagedParams& p, int d, int hc, int tpt) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(d) * 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(p.group),
                              static_cast<cuuint64_t>(p.Hkv), static_cast<cuuint64_t>(p.T)};
  const cuuint64_t strides[3] = {row, row * static_cast<cuuint64_t>(p.group), row * static_cast<cuuint64_t>(p.Hq)};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(hc), 1, static_cast<cuuint32_t>(tpt)};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace sdpa

extern "C" {

attn_status_t attn_page_plan(const int* past_lens, const int* new_lens, int* block_table, const int* free_pages,
                             const int* free_range, int* cu_new, int* total_lens, int* positions, int* slot_map,
                             int* free_range_out, int B, int max_pages, int num_free, int page_size, int T,
                             void* stream) {
  if (B < 0 || max_pages < 0 || num_free < 0 || T < 0) return ATTN_ERR_SHAPE;
  if (B > kPlanMaxBatch || T > kMaxSeq) return ATTN_ERR_SHAPE;
  if (!page_size_ok(page_size)) return ATTN_ERR_PAGE;
  if (static_cast<int64_t>(max_pages) * page_size > kMaxSeq) return ATTN_ERR_SHAPE;
  if (cu_new == nullptr || free_range == nullptr || free_range_out == nullptr) return ATTN_ERR_NULL;
  if (B > 0 && (past_lens == nullptr || new_lens == nullptr || total_lens == nullptr)) return ATTN_ERR_NULL;
  if (B > 0 && max_pages > 0 && block_table == nullptr) return ATTN_ERR_NULL;
  if (num_free > 0 && free_pages == nullptr) return ATTN_ERR_NULL;
  if (T > 0 && (positions == nullptr || slot_map == nullptr)) return ATTN_ERR_NULL;
  for (const void* ptr : {static_cast<const void*>(past_lens), static_cast<const void*>(new_lens),
                          static_cast<const void*>(block_table), static_cast<const void*>(free_pages),
                          static_cast<const void*>(free_range), static_cast<const void*>(cu_new),
                          static_cast<const void*>(total_lens), static_cast<const void*>(positions),
                          static_cast<const void*>(slot_map), static_cast<const void*>(free_range_out)})
    if (!aligned(ptr, 4)) return ATTN_ERR_ALIGN;
  int dev = 0;
  attn_status_t s = current_device(&dev, nullptr);
  if (s != ATTN_OK) return s;
  PlanParams p;
  p.past = past_lens;
  p.fresh = new_lens;
  p.table = block_table;
  p.free_pages = free_pages;
  p.free_range = free_range;
  p.cu = cu_new;
  p.total = total_lens;
  p.positions = positions;
  p.slots = slot_map;
  p.range_out = free_range_out;
  p.B = B;
  p.max_pages = max_pages;
  p.num_free = num_free;
  p.T = T;
  p.page_shift = log2_of(page_size);
  static bool smem_done[kMaxDevices] = {};
  static std::mutex mu;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!smem_done[dev] && cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
                               cudaSuccess)
      return ATTN_ERR_CUDA;
    if (!set_smem(page_plan_kernel, plan_smem_bytes(kPlanMaxBatch), dev, smem_done)) return ATTN_ERR_CUDA;
  }
  // one cluster, just wide enough for one pass over the tokens
  int ctas = 1;
  const int most = B <= kPlanSmallBatch ? kPlanMaxCluster : 8;
  while (ctas < most && static_cast<int64_t>(ctas) * kPlanThreads * kPlanTokens < T) ctas *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(plan_smem_bytes(B));
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, page_plan_kernel, p) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t attn_rope_append_paged(const void* packed_qkv, const float* cos_table, const float* sin_table,
                                     int max_pos, const int* positions, const int* slot_map, void* q_out,
                                     const attn_paged_cache_t* cache, int T, int Hq, int Hkv, int d, void* stream) {
  if (T < 0 || Hq <= 0 || Hkv <= 0 || max_pos <= 0) return ATTN_ERR_SHAPE;
  if (T > kMaxSeq || max_pos > kMaxSeq || Hq + 2 * static_cast<int64_t>(Hkv) > INT_MAX / 128) return ATTN_ERR_SHAPE;
  if (Hq % Hkv != 0) return ATTN_ERR_GQA;
  if (d != 64 && d != 128) return ATTN_ERR_HEADDIM;
  RopeParams prm;
  std::memset(&prm, 0, sizeof(prm));
  attn_status_t s = check_cache(cache, Hkv, d, false, &prm.c_sb, &prm.c_sh, &prm.c_sr);
  if (s != ATTN_OK) return s;
  if (T == 0) return ATTN_OK;
  if (packed_qkv == nullptr || cos_table == nullptr || sin_table == nullptr || q_out == nullptr ||
      positions == nullptr || slot_map == nullptr)
    return ATTN_ERR_NULL;
  if (!aligned(packed_qkv, 16) || !aligned(cos_table, 16) || !aligned(sin_table, 16) || !aligned(q_out, 16) ||
      !aligned(positions, 4) || !aligned(slot_map, 4))
    return ATTN_ERR_ALIGN;
  int sms = 0;
  if ((s = current_device(nullptr, &sms)) != ATTN_OK) return s;
  prm.packed = static_cast<const uint16_t*>(packed_qkv);
  prm.cos_t = cos_table;
  prm.sin_t = sin_table;
  prm.q_out = static_cast<uint16_t*>(q_out);
  prm.k_cache = static_cast<uint16_t*>(cache->k_pages);
  prm.v_cache = static_cast<uint16_t*>(cache->v_pages);
  prm.q_sh = d;
  prm.q_sr = static_cast<int64_t>(Hq) * d;
  prm.tokens = T;
  prm.Hq = Hq;
  prm.Hkv = Hkv;
  prm.max_pos = max_pos;
  prm.positions = positions;
  prm.slots = slot_map;
  prm.page_shift = log2_of(cache->page_size);
  prm.num_pages = cache->num_pages;
  const int grid = static_cast<int>(std::min<int64_t>(T, static_cast<int64_t>(sms) * kRopePagedBlocksPerSm));
  PdlLaunch l(static_cast<unsigned>(grid), kRopeWarps * 32, 0, static_cast<cudaStream_t>(stream));
  return (d == 128 ? cudaLaunchKernelEx(&l.cfg, rope_append_kernel<128, true>, prm)
                   : cudaLaunchKernelEx(&l.cfg, rope_append_kernel<64, true>, prm)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

size_t attn_fwd_paged_workspace_size(int T, int Hq, int Hkv, int d) {
  if (T < 0 || T > kMaxSeq || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || (d != 64 && d != 128)) return 0;
  const int sms = sm_count_or_default();
  return paged_units_ws_bytes(sms, d) + (Hq / Hkv <= kRowUnit ? paged_decode_ws_bytes(sms, d) : 0);
}

attn_status_t attn_fwd_paged(const void* q, const attn_paged_cache_t* cache, const int* cu_q, const int* seqlens_k,
                             void* o, float* lse, int B, int T, int Hq, int Hkv, int d, float scale, int causal,
                             void* workspace, size_t workspace_bytes, void* stream) {
  PagedFwdParams a;
  std::memset(&a, 0, sizeof(a));
  attn_status_t s = paged_params(&a.p, q, cache, seqlens_k, o, lse, B, T, Hq, Hkv, d, scale, causal);
  if (s != ATTN_OK) return s;
  if (B == 0 || T == 0) return ATTN_OK;
  if (cu_q == nullptr) return ATTN_ERR_NULL;
  if (!aligned(cu_q, 4)) return ATTN_ERR_ALIGN;
  if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < attn_fwd_paged_workspace_size(T, Hq, Hkv, d))
    return ATTN_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  if ((s = current_device(&dev, &sms)) != ATTN_OK) return s;
  a.p.cu_q = cu_q;
  const int group = a.p.group;
  a.chunks = (group + 127) / 128;
  a.hc = (group + a.chunks - 1) / a.chunks;
  a.tpt = 128 / a.hc;
  a.div_hc = make_fastdiv(static_cast<uint32_t>(a.hc));
  a.p.unit_tokens = 2 * a.tpt;
  a.p.div_tu = make_fastdiv(static_cast<uint32_t>(a.p.unit_tokens));
  a.div_chunks = make_fastdiv(static_cast<uint32_t>(a.chunks));
  if (static_cast<int64_t>(Hkv) * a.chunks > INT_MAX / 2) return ATTN_ERR_SHAPE;
  a.div_per_seq = make_fastdiv(static_cast<uint32_t>(Hkv * a.chunks));
  const bool pages = a.p.num_pages > 0;
  a.oob_page = std::max(a.p.num_pages, 1);
  const int box = std::min(1 << a.p.page_shift, 128);
  if (!make_packed_q_map(&a.tm_q, q, a.p, d, a.hc, a.tpt) ||
      !make_page_map(&a.tm_k, pages ? cache->k_pages : q, a.p, d, box, 1) ||
      !make_page_map(&a.tm_v, pages ? cache->v_pages : q, a.p, d, box, 1))
    return ATTN_ERR_CUDA;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<size_t>(sms) * 4 * 128 * d);
  a.joins = reinterpret_cast<int4*>(a.part_ml + static_cast<size_t>(sms) * 4 * 128);
  PagedDecodeParams r;
  std::memset(&r, 0, sizeof(r));
  if (group <= kRowUnit) {  // else no sequence is short enough
    r.p = a.p;
    r.row_groups = 1;
    r.div_rg = make_fastdiv(1);
    r.lse_tok = 1;
    r.lse_head = T;
    if (!paged_rows_params(&r, d, sms, static_cast<uint8_t*>(workspace) + paged_units_ws_bytes(sms, d)))
      return ATTN_ERR_CUDA;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 128 ? launch_paged_fwd<128, kStagesD128>(a, r, sms, dev, st)
                  : launch_paged_fwd<64, kStagesD64>(a, r, sms, dev, st);
}

size_t attn_decode_paged_workspace_size(int B, int Hq, int Hkv, int Sq, int d) {
  if (B < 0 || Sq < 0 || static_cast<int64_t>(B) * Sq > kMaxSeq || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 ||
      (d != 64 && d != 128))
    return 0;
  return paged_decode_ws_bytes(sm_count_or_default(), d);
}

attn_status_t attn_decode_splitkv_paged(const void* q, const attn_paged_cache_t* cache, const int* seqlens_k, void* o,
                                        float* lse, int B, int Hq, int Hkv, int Sq, int d, float scale, int causal,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  if (B < 0 || Sq < 0) return ATTN_ERR_SHAPE;
  PagedDecodeParams a;
  attn_status_t s = paged_params(&a.p, q, cache, seqlens_k, o, lse, B, static_cast<int64_t>(B) * Sq, Hq, Hkv, d, scale,
                                 causal);
  if (s != ATTN_OK) return s;
  if (B == 0 || Sq == 0) return ATTN_OK;
  if (workspace == nullptr || !aligned(workspace, 16) ||
      workspace_bytes < attn_decode_paged_workspace_size(B, Hq, Hkv, Sq, d))
    return ATTN_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  if ((s = current_device(&dev, &sms)) != ATTN_OK) return s;
  a.p.Sq = Sq;
  const int64_t rows = static_cast<int64_t>(a.p.group) * Sq;
  if (rows > INT_MAX / 2) return ATTN_ERR_SHAPE;
  a.row_groups = static_cast<int>((rows + kPdRows - 1) / kPdRows);
  a.div_rg = make_fastdiv(static_cast<uint32_t>(a.row_groups));
  if (static_cast<int64_t>(Hkv) * a.row_groups > INT_MAX / 2) return ATTN_ERR_SHAPE;
  a.lse_tok = Hq;
  a.lse_head = Sq;
  if (!paged_rows_params(&a, d, sms, workspace)) return ATTN_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 128 ? launch_paged_decode<128>(a, sms, dev, st) : launch_paged_decode<64>(a, sms, dev, st);
}

}  // extern "C"
