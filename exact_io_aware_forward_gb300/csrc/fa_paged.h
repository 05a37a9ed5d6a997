// Launch interfaces of the 8-bit paged K/V cache (attention, append, evict).
// Not part of the public interface.
#pragma once

#include "fa_internal.h"

namespace fa {

// What of the cache the kernels see (fa_paged_cache of the C ABI).
struct PagedView {
  uint8_t* k_pages = nullptr;   // [pages, Hkv, ps, d] 8-bit codes
  uint8_t* v_pages = nullptr;
  float* k_scale = nullptr;     // [pages, Hkv]
  float* v_scale = nullptr;
  const int* table = nullptr;   // [B, width]
  int pages = 0, width = 0;
  int B = 0, Hkv = 0, d = 0;
  int ps = 0, ps_shift = 0;     // slots a page (a power of two) and its logarithm
  bool e5m2 = false;
};

// Status bit (beside those of fa_internal.h): a page table entry outside the pool.
constexpr unsigned int kStatusBadPages = 4u;

// Slots of one segment of attention: what can be lost of tiny weights grows
// with it, and its page list sits in shared memory.
constexpr int kPagedMaxChunk = 16384;
// Sequences whose lengths every CTA adds up to find its share.
constexpr int kPagedMaxBalanced = 1024;
// Parts that a row can have (the chunks of a head, or the CTAs that share it)
// and the slots that this allows at 127 tiles a part.
constexpr int kPagedMaxParts = 4096;
constexpr int kPagedMaxSlots = (kPagedMaxParts - 2) * 127 * 128;

// How the tiles are shared out among CTAs (see fa_paged.cu).
struct PagedPlan {
  int row_tile = 8;        // query rows of a CTA
  bool balanced = false;   // by the lengths, on the device; else `splits` chunks of `per` tiles a head
  long long ctas = 1;      // CTAs a row tile
  int splits = 1, per = 1;
  int min_tiles = 1;       // balanced: places on the line of heads that are worth a CTA
  int seg_pages = 1;       // pages of the longest segment
  long long parts = 0;     // partial results in the workspace, row_tile rows each
};

struct PagedAttnArgs {
  CUtensorMap tm_k, tm_v;    // [pages * Hkv, ps, d] bytes, box one page (of 128 or 64 bytes a row)
  PagedView c;
  const void* q;             // [B, Hkv, rows, d] 16 bit
  const int* lens;           // [B]
  void* o;                   // [B, Hkv, rows, d] 16 bit
  float* lse;                // [B, Hkv, rows]
  float* o_part;             // [parts, row_tile, d]
  float* lse_part;           // [parts, row_tile], log2 units
  int2* shared;              // [B * Hkv]: CTAs that share the head, the first of them (balanced)
  float* scores;             // [B * Hkv, score_groups, slots, score_rows], log2 units, or null
  float* weight_acc;         // [B * Hkv, width * ps], or null
  int rows, Nq;              // query rows of a K / V head, rows = group * Nq, row R is query R % Nq
  int max_len;
  int row_tile, ctas, splits, per, min_tiles, seg_pages;  // the plan
  bool balanced;
  int score_rows, score_groups;    // rows of a group (1, 2, 4 or 8) and groups of a head
  long long score_stride;          // floats of a group
  bool causal, bf16;
  float scale_log2;
  unsigned int* status;
};
PagedPlan paged_plan(int B, int Hkv, int rows, int d, int ps, int max_len, int num_splits);
cudaError_t launch_paged_attention(const PagedAttnArgs& a, cudaStream_t stream);

struct PagedAppendArgs {
  PagedView c;
  const void* k;             // [B, Hkv, N, d] 16 bit
  const void* v;
  const int* lens;           // [B] slots before
  const int* counts;         // [B] tokens to append, or null (N each)
  int* new_lens;             // [B]
  float* weight_acc;         // [B, Hkv, width * ps] or null: zeroed for the new slots
  int* positions;            // [B, Hkv, width * ps] or null
  const int* first_position; // [B] or null (the slot numbers)
  int N;
  bool bf16;
  unsigned int* status;
};
cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream);

struct PagedEvictArgs {
  PagedView c;
  const int* lens;
  int* new_lens;
  float* weight_acc;         // [B, Hkv, width * ps]
  int* positions;            // [B, Hkv, width * ps]
  int keep, recent;
  // workspace, per (b, h): holes in all and before each page, the holes, the slots that move
  int* plan_count;           // [B * Hkv]
  int* page_holes;           // [B * Hkv, pages of keep + 1]
  int* holes;                // [B * Hkv, keep]
  int* movers;               // [B * Hkv, keep]
  float2* edge_scales;       // [B * Hkv] (K, V) of the page where the kept part ends
  unsigned int* status;
};
cudaError_t launch_paged_evict(const PagedEvictArgs& a, cudaStream_t stream);

// Shared by the entry points (fa_api.cu).
unsigned int* device_status_word();
int sm_count();  // of the current device
bool encode_tiled_map(CUtensorMap* m, CUtensorMapDataType type, const void* ptr, const cuuint64_t (&dims)[3],
                      const cuuint64_t (&strides)[2], const cuuint32_t (&box)[3], CUtensorMapSwizzle swizzle);

}  // namespace fa
