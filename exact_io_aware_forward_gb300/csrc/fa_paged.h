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

// Pages one CTA of the attention kernel can list (its share of the table
// sits in shared memory), and slots of a chunk (what can be lost of tiny
// weights grows with it): bounds of a chunk.
constexpr int kPagedMaxPagesPerChunk = 1024;
constexpr int kPagedMaxChunk = 16384;

struct PagedAttnArgs {
  CUtensorMap tm_k, tm_v;    // [pages * Hkv, ps, d] bytes, box one page (of 128 or 64 bytes a row)
  PagedView c;
  const void* q;             // [B, Hkv, rows, d] 16 bit
  const int* lens;           // [B]
  void* o;                   // [B, Hkv, rows, d] 16 bit
  float* lse;                // [B, Hkv, rows]
  float* o_part;             // [splits, B * Hkv, rows, d] (splits > 1)
  float* lse_part;           // [splits, B * Hkv, rows], log2 units
  float* scores;             // [B * Hkv, rows, score_stride], log2 units, or null
  float* weight_acc;         // [B * Hkv, width * ps], or null
  int rows, Nq;              // query rows of a K / V head, rows = group * Nq, row R is query R % Nq
  int max_len, splits, chunk;
  long long score_stride;
  bool causal, bf16;
  float scale_log2;
  unsigned int* status;
};
// Rows of one CTA for `rows` query rows of a head.
int paged_row_tile(int rows);
// The chunk (a multiple of 128 slots) and the number of chunks of max_len slots.
void paged_plan(int BH, int rows, int ps, int max_len, int num_splits, int* splits, int* chunk);
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
  // workspace, per (b, h): count and status, then the holes, the slots that move, and their scales
  int* plan_count;           // [B * Hkv]
  int* holes;                // [B * Hkv, keep]
  int* movers;               // [B * Hkv, keep]
  float2* mover_scales;      // [B * Hkv, keep] (K, V)
  unsigned int* status;
};
cudaError_t launch_paged_evict(const PagedEvictArgs& a, cudaStream_t stream);

// Shared by the entry points (fa_api.cu).
unsigned int* device_status_word();
bool encode_tiled_map(CUtensorMap* m, CUtensorMapDataType type, const void* ptr, const cuuint64_t (&dims)[3],
                      const cuuint64_t (&strides)[2], const cuuint32_t (&box)[3], CUtensorMapSwizzle swizzle);

}  // namespace fa
