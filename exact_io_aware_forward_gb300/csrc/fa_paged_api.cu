// C entry points of the 8-bit paged K / V cache: argument checks, tensor maps
// and workspace layout.  Nothing is allocated here.
#include <math.h>
#include <stdint.h>
#include <vector_types.h>

#include "../../include/fa_gb300.h"
#include "fa_paged.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f;

bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Sizes and types of the cache (its pointers are looked at by view()).
fa_status check_cache(const fa_paged_cache* c) {
  if (!c) return FA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->pages_per_seq < 1 || c->B < 1 || c->Hkv < 1) return FA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128 && c->d != 256) return FA_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return FA_ERR_UNSUPPORTED;
  if (c->cache_dtype != FA_E4M3 && c->cache_dtype != FA_E5M2) return FA_ERR_UNSUPPORTED;
  if ((long long)c->num_pages * c->Hkv >= (1LL << 31) || (long long)c->pages_per_seq * c->page_size > (1LL << 30) ||
      (long long)c->B * c->Hkv > 65535 || c->Hkv > 32767)
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

fa_status view(const fa_paged_cache* c, fa::PagedView* v) {
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages) || !aligned16(c->k_scale) || !aligned16(c->v_scale) ||
      !aligned16(c->page_table))
    return FA_ERR_INVALID_ARG;
  v->k_pages = static_cast<uint8_t*>(c->k_pages);
  v->v_pages = static_cast<uint8_t*>(c->v_pages);
  v->k_scale = c->k_scale;
  v->v_scale = c->v_scale;
  v->table = c->page_table;
  v->pages = c->num_pages;
  v->width = c->pages_per_seq;
  v->B = c->B;
  v->Hkv = c->Hkv;
  v->d = c->d;
  v->ps = c->page_size;
  v->ps_shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  v->e5m2 = c->cache_dtype == FA_E5M2;
  return FA_OK;
}

// Whether two arrays of n 4-byte elements share memory.
bool overlap(const void* x, const void* y, long long n) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  const uintptr_t bytes = static_cast<uintptr_t>(n) * 4;
  return a < b + bytes && b < a + bytes;
}

struct AttnPlan {
  int rows = 0, max_len = 0;
  fa::PagedPlan share;
  int score_rows = 1, score_groups = 1;
  long long score_stride = 0;
  size_t o_part = 0, lse_part = 0, shared = 0, scores = 0;  // bytes
  size_t total() const { return o_part + lse_part + shared + scores; }
};

fa_status attention_plan(const fa_paged_cache* c, int Hq, int Nq, int max_len, int num_splits, bool weights,
                         AttnPlan* p) {
  if (Hq < 1 || Nq < 1 || Hq % c->Hkv != 0) return FA_ERR_INVALID_ARG;
  const int slots = c->pages_per_seq * c->page_size;
  if (max_len < 0 || max_len > slots || num_splits < 0 || num_splits > 1024) return FA_ERR_INVALID_ARG;
  const long long rows = (long long)(Hq / c->Hkv) * Nq;
  const long long BH = (long long)c->B * c->Hkv;
  if (rows > 65535 * 8LL || BH * rows * c->d >= (1LL << 31)) return FA_ERR_UNSUPPORTED;
  p->rows = (int)rows;
  p->max_len = max_len ? max_len : slots;
  if (p->max_len > fa::kPagedMaxSlots) return FA_ERR_UNSUPPORTED;
  p->share = fa::paged_plan(c->B, c->Hkv, p->rows, c->d, c->page_size, p->max_len, num_splits);
  if (BH * rows + BH * ((p->max_len + 511) / 512) >= (1LL << 31)) return FA_ERR_UNSUPPORTED;  // blocks of the join
  if (p->share.ctas >= (1LL << 31) || p->share.parts >= (1LL << 31)) return FA_ERR_UNSUPPORTED;
  const size_t part_rows = (size_t)p->share.parts * p->share.row_tile;
  p->o_part = align256(part_rows * c->d * sizeof(float));
  p->lse_part = align256(part_rows * sizeof(float));
  if (p->share.balanced) p->shared = align256((size_t)BH * sizeof(int2));
  p->score_rows = rows == 1 ? 1 : rows == 2 ? 2 : rows <= 4 ? 4 : 8;
  p->score_groups = (int)((rows + 7) / 8);
  p->score_stride = (long long)p->max_len * p->score_rows;
  if (weights) p->scores = align256((size_t)BH * p->score_groups * p->score_stride * sizeof(float));
  return FA_OK;
}

bool page_map(CUtensorMap* m, const void* ptr, const fa_paged_cache* c) {
  const cuuint32_t row = c->d == 64 ? 64 : 128;
  const cuuint64_t dims[3] = {(cuuint64_t)c->d, (cuuint64_t)c->page_size, (cuuint64_t)c->num_pages * c->Hkv};
  const cuuint64_t strides[2] = {(cuuint64_t)c->d, (cuuint64_t)c->d * c->page_size};
  const cuuint32_t box[3] = {row, (cuuint32_t)c->page_size, 1};
  return fa::encode_tiled_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, ptr, dims, strides, box,
                              row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

size_t evict_bytes(const fa_paged_cache* c, int keep, size_t* pages, size_t* holes, size_t* movers, size_t* scales) {
  const size_t bh = (size_t)c->B * c->Hkv;
  *pages = align256(bh * sizeof(int));
  *holes = *pages + align256(bh * ((keep + c->page_size - 1) / c->page_size + 1) * sizeof(int));
  *movers = *holes + align256(bh * keep * sizeof(int));
  *scales = *movers + align256(bh * keep * sizeof(int));
  return *scales + align256(bh * 2 * sizeof(float));
}

}  // namespace

extern "C" {

fa_status fa_paged_append(const fa_paged_cache* cache, const void* k, const void* v, const int* lens,
                          const int* counts, int* new_lens, float* weight_acc, int* positions,
                          const int* first_position, int N, int dtype, void* stream) {
  fa_status st = check_cache(cache);
  if (st != FA_OK) return st;
  if (N < 1) return FA_ERR_INVALID_ARG;
  if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  fa::PagedAppendArgs a;
  if ((st = view(cache, &a.c)) != FA_OK) return st;
  if (!aligned16(k) || !aligned16(v) || !aligned4(lens) || !aligned4(new_lens) || (counts && !aligned4(counts)) ||
      (weight_acc && !aligned16(weight_acc)) || (positions && !aligned16(positions)) ||
      (first_position && !aligned4(first_position)))
    return FA_ERR_INVALID_ARG;
  if (overlap(lens, new_lens, cache->B) || (counts && overlap(counts, new_lens, cache->B)) ||
      (first_position && overlap(first_position, new_lens, cache->B)))
    return FA_ERR_INVALID_ARG;
  a.k = k;
  a.v = v;
  a.lens = lens;
  a.counts = counts;
  a.new_lens = new_lens;
  a.weight_acc = weight_acc;
  a.positions = positions;
  a.first_position = first_position;
  a.N = N;
  a.bf16 = dtype == FA_BF16;
  a.status = fa::device_status_word();
  if (!a.status) return FA_ERR_CUDA;
  return fa::launch_paged_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_paged_workspace_size(const fa_paged_cache* cache, int Hq, int Nq, int max_len, int num_splits, int weights) {
  AttnPlan p;
  if (check_cache(cache) != FA_OK || attention_plan(cache, Hq, Nq, max_len, num_splits, weights != 0, &p) != FA_OK)
    return 0;
  return p.total() ? p.total() : 256;
}

fa_status fa_forward_paged(const fa_paged_cache* cache, const void* q, const int* lens, void* o, float* lse,
                           float* weight_acc, int Hq, int Nq, int dtype, int causal, float scale, int max_len,
                           int num_splits, void* workspace, size_t workspace_bytes, void* stream) {
  fa_status st = check_cache(cache);
  if (st != FA_OK) return st;
  AttnPlan p;
  if ((st = attention_plan(cache, Hq, Nq, max_len, num_splits, weight_acc != nullptr, &p)) != FA_OK) return st;
  if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (!(isfinite(scale * kLog2e) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  fa::PagedAttnArgs a;
  if ((st = view(cache, &a.c)) != FA_OK) return st;
  if (!aligned16(q) || !aligned16(o) || !aligned16(lse) || !aligned4(lens) || (weight_acc && !aligned16(weight_acc)))
    return FA_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < p.total())
    return FA_ERR_WORKSPACE;
  if (!page_map(&a.tm_k, cache->k_pages, cache) || !page_map(&a.tm_v, cache->v_pages, cache)) return FA_ERR_CUDA;
  a.q = q;
  a.lens = lens;
  a.o = o;
  a.lse = lse;
  a.weight_acc = weight_acc;
  a.rows = p.rows;
  a.Nq = Nq;
  a.max_len = p.max_len;
  a.row_tile = p.share.row_tile;
  a.ctas = (int)p.share.ctas;
  a.splits = p.share.splits;
  a.per = p.share.per;
  a.min_tiles = p.share.min_tiles;
  a.seg_pages = p.share.seg_pages;
  a.balanced = p.share.balanced;
  a.score_rows = p.score_rows;
  a.score_groups = p.score_groups;
  a.score_stride = p.score_stride;
  a.causal = causal != 0;
  a.bf16 = dtype == FA_BF16;
  a.scale_log2 = scale * kLog2e;
  char* ws = static_cast<char*>(workspace);
  a.o_part = reinterpret_cast<float*>(ws);
  a.lse_part = reinterpret_cast<float*>(ws + p.o_part);
  a.shared = reinterpret_cast<int2*>(ws + p.o_part + p.lse_part);
  a.scores = weight_acc ? reinterpret_cast<float*>(ws + p.o_part + p.lse_part + p.shared) : nullptr;
  a.status = fa::device_status_word();
  if (!a.status) return FA_ERR_CUDA;
  return fa::launch_paged_attention(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_paged_evict_workspace_size(const fa_paged_cache* cache, int keep) {
  if (check_cache(cache) != FA_OK || keep < 1 || keep > cache->pages_per_seq * cache->page_size) return 0;
  size_t p, h, m, s;
  return evict_bytes(cache, keep, &p, &h, &m, &s);
}

fa_status fa_paged_evict(const fa_paged_cache* cache, const int* lens, int* new_lens, float* weight_acc,
                         int* positions, int keep, int recent, void* workspace, size_t workspace_bytes,
                         void* stream) {
  fa_status st = check_cache(cache);
  if (st != FA_OK) return st;
  if (keep < 1 || keep > cache->pages_per_seq * cache->page_size || recent < 0 || recent > keep)
    return FA_ERR_INVALID_ARG;
  fa::PagedEvictArgs a;
  if ((st = view(cache, &a.c)) != FA_OK) return st;
  if (!aligned4(lens) || !aligned4(new_lens) || !aligned16(weight_acc) || !aligned16(positions) ||
      overlap(lens, new_lens, cache->B))
    return FA_ERR_INVALID_ARG;
  size_t p, h, m, s;
  const size_t need = evict_bytes(cache, keep, &p, &h, &m, &s);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < need) return FA_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  a.lens = lens;
  a.new_lens = new_lens;
  a.weight_acc = weight_acc;
  a.positions = positions;
  a.keep = keep;
  a.recent = recent;
  a.plan_count = reinterpret_cast<int*>(ws);
  a.page_holes = reinterpret_cast<int*>(ws + p);
  a.holes = reinterpret_cast<int*>(ws + h);
  a.movers = reinterpret_cast<int*>(ws + m);
  a.edge_scales = reinterpret_cast<float2*>(ws + s);
  a.status = fa::device_status_word();
  if (!a.status) return FA_ERR_CUDA;
  return fa::launch_paged_evict(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
