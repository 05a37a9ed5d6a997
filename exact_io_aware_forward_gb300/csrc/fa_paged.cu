// Attention over the 8-bit paged K/V cache: few queries a sequence against
// its slots, split over the slots, grouped query heads.
//
// A CTA takes up to R = 8 G query rows of a K / V head (its query heads' rows
// are consecutive: rows = group * Nq, row x is query x % Nq) and runs the
// online-softmax recurrence ("FlashAttention 为什么不需要存下注意力矩阵",
// jefxiong.cn, section 3.2) over tiles of 128 slots.  The tiles of all
// sequences and heads, in order, are shared out evenly among the CTAs that the
// GPU holds at once, by the lengths on the device: a CTA's run of tiles is cut
// into segments at the heads' ends, and the pipeline runs on across them.  A
// segment that is not a whole head leaves its normalised O_s (float32) and
// LSE_s (log2 units) in the workspace; paged_finish_kernel merges them
// exactly.  (With num_splits the chunks are cut from max_len instead, one a
// CTA, and a sequence's result does not depend on the others' lengths.)
//
// Both products run on the tensor core with the cache's bytes as they lie in
// memory (tcgen05 kind::f8f6f4), the cache as operand A and the few rows as
// operand B, so that work grows with the rows that there are:
//   S^T [128 slots, rows]    = K_tile [slots, d]  x  Q^T,
//   O^T [d features, rows]  += V_tile^T [d, slots]  x  P^T.
// A thread of the softmax warps owns one slot (one TMEM lane) and its column
// of scores; the running maximum is exchanged through shared memory.
//
// Operand B has to be 8 bits too.  A query row x is scaled by a power of two
// so that max |x| lies in [128, 256) and written as T e4m3 terms, each the
// rounding of what the terms before leave, scaled by 16:
//   x = t0 + t1 / 16 + t2 / 256,
// each term in columns of its own, summed after the product in float32.  An
// e4m3 has 4 significant bits, so two terms hold the 8 of bf16 exactly and
// three the 11 of fp16 (down to 2^-22 of the row's maximum).  The weights P
// are split alike: their rounding is that of P to bf16 or fp16 in the 16-bit
// kernels.
//
// Scales: page and head have one each.  S is multiplied by the slot's K scale
// in float32.  V's scale goes into the weight that is multiplied with its
// codes, w_j = 2^(s_j - m) vs_j, and the running reference m bounds
// s_j + ceil(log2 vs_j) instead of s_j, so that w lies in [0, 2] whatever the
// scales are and a page of large scale costs the others no precision; the sum
// l keeps 2^(s_j - m) in float32.
//
// Masked slots (behind the length, on a page that the table names wrongly,
// or behind a causal query's own slot): their scores are replaced by -inf
// after the product, whatever their bytes are; rows of V that no query of the
// sequence may see are overwritten with zeros in shared memory before the
// product, since a weight of 0 times a NaN would be a NaN.
//
// Roles: G groups of four softmax warps, eight rows each; a TMA warp (one copy
// a page, lane i the i-th page of a tile); a warp for TMEM and MMA issue; a
// warp that walks the segments ahead of the others and lists their pages, and
// one that turns their query rows into terms.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_paged.h"
#include "fa_pdl.cuh"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
// Weights are multiplied by 256, and the reference moves when a tile's maximum
// exceeds it by more than 0.8 (log2 units): they stay below 446, inside
// e4m3's range of 448.  The terms reach down to 2^-9 / 16 (T = 2), so a
// weight is lost only below 2^-22 of the chunk's largest: all 16384 slots of a
// chunk that one slot outweighs like that lose 2^-8 of it together.  (A lead
// of 4 and a factor of 16 would move the reference less often, at 16 times
// that loss.)
constexpr float kMaxLead = 0.8f;
constexpr float kWeightScale = 256.0f;
// The exponent of the smallest V scale that moves the reference: 2^(s - m)
// then stays below 2^100, far from overflow.
constexpr int kMinScaleExponent = -100;

// ceil(log2 |x|), at least kMinScaleExponent.  A whole number, so that the
// largest slot's 2^(s - m) is a power of two and LSE loses nothing to the scale.
__device__ __forceinline__ float scale_exponent(float x) {
  const int bits = __float_as_int(x) & 0x7fffffff;
  return (float)max((bits >> 23) - 127 + ((bits & 0x7fffff) != 0), kMinScaleExponent);
}
// m + log2(l), l > 0: the exponent of l goes to m, which it mostly cancels.
__device__ __forceinline__ float add_log2(float m, float l) {
  const int e = (__float_as_int(l) >> 23) - 127;
  const bool normal = e >= -126 && e <= 126;
  return (m + (normal ? (float)e : 0.f)) + __log2f(normal ? __int_as_float(__float_as_int(l) - (e << 23)) : l);
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000u); }

// Bounded wait with the same result on every lane of the warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned int* status) {
  const bool ok = mbar_wait(bar, parity, abort, status, kStatusTimeout);
  return __all_sync(0xffffffffu, ok);
}
// Bounded wait of the abort path: ignores the abort flag.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(a, parity))
    if (global_timer_ns() - t0 > kWaitTimeoutNs) return;
}

// D(tmem) (+)= A(smem) * B(smem), one K = 32 step of 8-bit floats, fp32 accumulation.
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f8f6f4 with fp32 accumulation: A e4m3 or
// e5m2 (codes 0, 1), B e4m3 and K-major, A K-major or (a_mn) MN-major.
__device__ __forceinline__ uint32_t idesc_f8(int M, int N, bool a_e5m2, bool a_mn) {
  return (1u << 4) | ((a_e5m2 ? 1u : 0u) << 7) | ((a_mn ? 1u : 0u) << 15) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// Shared-memory descriptor of rows of W bytes swizzled over W bytes (64 or
// 128; layout codes 4 and 2): sdesc_sw128 with the other swizzle code.
template <int W>
__device__ __forceinline__ uint64_t sdesc_w(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  uint64_t d = sdesc_sw128(saddr, lbo_bytes, sbo_bytes);
  if (W == 64) d ^= static_cast<uint64_t>(2 ^ 4) << 61;
  return d;
}
// Byte offset of byte `col` of row `row` in rows of W bytes swizzled over W
// bytes (16-byte chunks XORed with the row: 8 rows of 128, 4 pairs of rows of 64).
template <int W>
__device__ __forceinline__ uint32_t sw_offset(uint32_t row, uint32_t col) {
  if (W == 128) return row * 128u + ((((col >> 4) ^ row) & 7u) << 4) + (col & 15u);
  return row * 64u + ((((col >> 4) ^ (row >> 1)) & 3u) << 4) + (col & 15u);
}

// tma_load_3d for data that is read once: the lines leave L2 first.  K and V
// would otherwise push out what every CTA needs again and again, page
// tables, queries and the kernel's own instructions.
__device__ __forceinline__ uint64_t stream_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_stream_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int y, int z,
                                              uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8_wait(float (&v)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7])
               :
               : "memory");
}

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Two floats to two e4m3 codes (a in the low byte), and back.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
// The T terms of a pair of values: codes in out[0 .. T-1], each the rounding of
// what the terms before leave, times 16 (exact: a code is a rounding of its
// value).
template <int T>
__device__ __forceinline__ void split_terms(uint64_t v, uint32_t (&out)[T]) {
#pragma unroll
  for (int t = 0; t < T; ++t) {
    float a, b;
    f2_unpack(v, a, b);
    out[t] = to_e4m3x2(a, b);
    if (t + 1 < T) {
      const float2 c = from_e4m3x2(out[t]);
      v = f2_fma(f2_pack(c.x, c.y), f2_pack(-16.f, -16.f), f2_mul(v, f2_pack(16.f, 16.f)));
    }
  }
}
template <int T>
__device__ __forceinline__ void split_terms(float a, float b, uint32_t (&out)[T]) {
  split_terms<T>(f2_pack(a, b), out);
}
// Sum of the terms' columns: y[0] + y[1] / 16 + y[2] / 256, eight rows in pairs.
template <int T>
__device__ __forceinline__ void join_terms(const float (&y)[T][8], uint64_t (&out)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t z = f2_pack(y[T - 1][2 * i], y[T - 1][2 * i + 1]);
#pragma unroll
    for (int u = T - 2; u >= 0; --u)
      z = f2_fma(z, f2_pack(0.0625f, 0.0625f), f2_pack(y[u][2 * i], y[u][2 * i + 1]));
    out[i] = z;
  }
}

// CTAs on an SM for `rows` query rows a CTA.
constexpr int paged_occupancy(int d, int rows) { return rows <= 16 && d <= 128 ? 2 : 1; }

template <int D, int T, int G>
struct PagedCfg {
  static constexpr bool BF16 = T == 2;                // the 16-bit type: two terms hold a bf16, three an fp16
  static constexpr int R = 8 * G;                     // query rows of a CTA, eight a softmax group
  static constexpr int W = D == 64 ? 64 : 128;        // bytes of a shared-memory row
  static constexpr int HALVES = D == 256 ? 2 : 1;     // 128-feature parts of a K or V tile
  static constexpr int ITEM = 128 * W;                // one ring slot: 128 slots x W bytes
  static constexpr int NB = (T * R + 15) / 16 * 16;   // columns of operand B (multiple of 16 at M = 128)
  static constexpr uint32_t COL_S = 0;                // two score buffers
  static constexpr uint32_t COL_O = 2 * NB;           // HALVES accumulators
  static constexpr int COLS = (2 + HALVES) * NB;
  static constexpr uint32_t TMEM_COLS = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  // One or two groups: two CTAs on an SM, which fill each other's waits (16
  // rows of 16 x 8 heads of 8192 slots: 65 us with one, 56 with two).  More
  // groups, or tiles of 64 KB: one CTA.
  static constexpr int OCC = paged_occupancy(D, R);
  static constexpr int SEGS = 2;                      // segment buffers: one in use, one being prepared
  static constexpr int Q_BYTES = HALVES * NB * W;
  static constexpr int P_BYTES = NB * 128;
  static constexpr int BUDGET = (OCC == 2 ? 104 : 192) * 1024;
  static constexpr int NS_MAX = (BUDGET - SEGS * Q_BYTES - 2 * P_BYTES) / ITEM;
  // 128 KB of K and V under way on an SM are enough to keep HBM busy; more
  // (192 KB) only made everything else wait longer for memory: 4 x 32 heads of
  // 32768 slots took 180 us instead of 171, and shorter calls no less.
  static constexpr int NS_CAP = 128 * 1024 / OCC / ITEM;
  static constexpr int NS = NS_MAX < NS_CAP ? NS_MAX : NS_CAP;
  // Half of the slots for K and half for V.  The softmax waits for V of its
  // tile ahead of the MMA warp, when the products of the tile two before are
  // done: two tiles of V in the ring keep that wait within one turn of it.
  static constexpr int NSV = NS / 2 > 2 * HALVES ? NS / 2 : 2 * HALVES;
  static constexpr int NSK = NS - NSV;
  static constexpr int OFF_Q = 0;                     // SEGS segments' queries
  static constexpr int OFF_P = SEGS * Q_BYTES;        // two tiles' weights
  static constexpr int OFF_RING = OFF_P + 2 * P_BYTES;
  static constexpr int OFF_BAR = OFF_RING + NS * ITEM;
  // ring_full[NS], ring_empty[NS] (K's, then V's), s_full[2], p_full[2], pv_done[2], seg_pages[SEGS], seg_ready[SEGS],
  // seg_free[SEGS], o_free, drain, exchange[G][2]
  static constexpr int NBAR = 2 * NS + 8 + 3 * SEGS + 2 * G;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;             // TMEM address, abort flag
  static constexpr int OFF_DESC = (OFF_MISC + 8 + 15) / 16 * 16;  // segment descriptors of 8 ints
  static constexpr int OFF_ROW = OFF_DESC + 32 * SEGS;            // per segment: inverse scales, ends of the visible slots
  static constexpr int OFF_MAX = OFF_ROW + 8 * SEGS * R;          // [G][2][4][8] warp maxima
  static constexpr int OFF_SUM = OFF_MAX + 32 * R;                // [G][4][8] warp sums of l
  static constexpr int OFF_PAGES = OFF_SUM + 16 * R;              // per segment and page: id, K scale, V scale
  static constexpr int WARPS = 4 * G + 4;  // a multiple of four: the SM's four parts get equally many
  static constexpr int smem(int pages) { return OFF_PAGES + 12 * SEGS * pages + 1024; }
  static_assert(NSK >= 2 && Q_BYTES % 1024 == 0 && P_BYTES % 1024 == 0 && COLS <= 512, "layout");
};

// How the work is shared out among the CTAs of a row tile.  A head of t > 0
// tiles (of 128 slots) takes up kHeadCost + t places on a line of all heads;
// the line is cut into equal pieces, and a CTA gets the tiles whose places lie
// in its piece.  (The start and end of a head's segment take about as long as
// kHeadCost tiles.)
constexpr int kHeadCost = 4;
struct Share {
  long long total;  // places
  int ctas;         // CTAs that get some
  // 64-bit divisions are slow: 32 bits wherever they are enough
  __device__ __forceinline__ long long begin(int i) const {
    const unsigned long long x = (unsigned long long)i * (unsigned long long)total;
    return x >> 32 ? (long long)(x / (unsigned)ctas) : (long long)((unsigned)x / (unsigned)ctas);
  }
  // the CTA that place x belongs to: the largest i with begin(i) <= x
  __device__ __forceinline__ int owner(long long x) const {
    const unsigned long long y = ((unsigned long long)x + 1) * (unsigned)ctas - 1;
    int i = (int)(y >> 32 || total >> 32 ? y / (unsigned long long)total : (unsigned)y / (unsigned)total);
    while (begin(i) > x) --i;
    while (begin(i + 1) <= x) ++i;
    return i;
  }
};
__device__ __forceinline__ Share make_share(long long total, const PagedAttnArgs& a) {
  const long long want = (total + a.min_tiles - 1) / a.min_tiles;
  Share s;
  s.total = total;
  s.ctas = (int)(want < 1 ? 1 : want < a.ctas ? want : a.ctas);
  return s;
}
__device__ __forceinline__ int good_len(int len, int max_len) { return len < 0 || len > max_len ? 0 : len; }
__host__ __device__ __forceinline__ int places_of(int tiles) { return tiles > 0 ? tiles + kHeadCost : 0; }

struct Segment {
  int bh, first, n, len, part, pages;  // head, first tile, tiles, the sequence's length, part number or -1, pages
};

template <int D, int T, int G>
__global__ void __launch_bounds__(PagedCfg<D, T, G>::WARPS * 32, (PagedCfg<D, T, G>::OCC))
    paged_attention_kernel(const __grid_constant__ PagedAttnArgs a) {
  using C = PagedCfg<D, T, G>;
  constexpr int R = C::R;
  const int row0 = blockIdx.y * R;
  const int nr = min(R, a.rows - row0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch();

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sP = smem + C::OFF_P;
  uint8_t* sRing = smem + C::OFF_RING;
  uint64_t* ring_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* ring_empty = ring_full + C::NS;
  uint64_t* s_full = ring_empty + C::NS;
  uint64_t* p_full = s_full + 2;
  uint64_t* pv_done = p_full + 2;
  uint64_t* seg_pages = pv_done + 2;          // a segment's descriptor and page list are there
  uint64_t* seg_ready = seg_pages + C::SEGS;  // its scales and queries too
  uint64_t* seg_free = seg_ready + C::SEGS;   // all of them may be overwritten
  uint64_t* o_free = seg_free + C::SEGS;      // the accumulators have been read
  uint64_t* drain = o_free + 1;
  uint64_t* exchange = drain + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  const int shift = a.c.ps_shift, ps = a.c.ps;
  const int ne = a.seg_pages;  // page entries a segment buffer holds
  int* s_page = reinterpret_cast<int*>(smem + C::OFF_PAGES);
  float* s_ks = reinterpret_cast<float*>(s_page + C::SEGS * ne);
  float* s_vs = s_ks + C::SEGS * ne;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&ring_full[s], 1);
      mbar_init(&ring_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4 * G);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < C::SEGS; ++i) {
      mbar_init(&seg_pages[i], 1);
      mbar_init(&seg_ready[i], G == 1 ? 1 : 1 + 2 * G);
      mbar_init(&seg_free[i], 4 * G + 1);
    }
    mbar_init(o_free, 4 * G);
    mbar_init(drain, 1);
    for (int i = 0; i < 2 * G; ++i) mbar_init(&exchange[i], 4);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 4 * G && lane == 0) {
    tma_prefetch_desc(&a.tm_k);
    tma_prefetch_desc(&a.tm_v);
  }
  if (warp == 4 * G + 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  // The walker's state, found while the others set up.
  auto tiles_of = [&](int b) { return (good_len(a.lens[b], a.max_len) + 127) >> 7; };
  // The next segment: head h of sequence b (tb tiles), its tiles from t on; in the balanced case the head's place
  // on the line is `at` and this CTA's piece ends at `stop`.
  int b = 0, h = 0, t = 0, tb = 0, n = 0;
  long long at = 0, stop = 0;
  Share share = {1, 1};
  auto place = [&](long long from) {  // the head's tiles in [from, stop)
    const long long first = from - at - kHeadCost, last = stop - at - kHeadCost;
    t = (int)(first > 0 ? first : 0);
    n = (int)(last < tb ? last : tb) - t;
  };
  if (warp == 4 * G + 2) {
    pdl_wait();
    if (a.balanced) {
      int mine = 0;  // tiles of sequence `lane` of the last 32 looked at
      long long total = 0;
      for (int b0 = 0; b0 < a.c.B; b0 += 32) {
        const int len = b0 + lane < a.c.B ? a.lens[b0 + lane] : 0;
        if (good_len(len, a.max_len) != len && blockIdx.x == 0) atomicOr(a.status, kStatusBadSeqlens);
        mine = (good_len(len, a.max_len) + 127) >> 7;
        total += __reduce_add_sync(0xffffffffu, (unsigned)places_of(mine));
      }
      total *= a.c.Hkv;
      share = make_share(total, a);
      if (total > 0 && (int)blockIdx.x < share.ctas) {
        const long long lo = share.begin(blockIdx.x);
        stop = share.begin(blockIdx.x + 1);
        for (int b0 = 0; lo < stop; b0 += 32) {
          if (a.c.B > 32) mine = b0 + lane < a.c.B ? tiles_of(b0 + lane) : 0;
          int upto = places_of(mine);  // inclusive over the lanes
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
          }
          const unsigned past = __ballot_sync(0xffffffffu, at + (long long)upto * a.c.Hkv > lo);
          if (past) {
            const int l = __ffs(past) - 1;
            tb = __shfl_sync(0xffffffffu, mine, l);
            at += (long long)(__shfl_sync(0xffffffffu, upto, l) - places_of(tb)) * a.c.Hkv;
            b = b0 + l;
            break;
          }
          at += (long long)__shfl_sync(0xffffffffu, upto, 31) * a.c.Hkv;
        }
        if (lo < stop) {
          const long long in = lo - at;  // less than Hkv heads of 2^24 tiles each, mostly much less
          h = in >> 32 ? (int)(in / places_of(tb)) : (int)((unsigned)in / (unsigned)places_of(tb));
          at += (long long)h * places_of(tb);
          place(lo);
        }
      }
    } else {
      const int bh = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
      b = bh / a.c.Hkv;
      h = bh % a.c.Hkv;
      const int len = a.lens[b];
      if (good_len(len, a.max_len) != len && h == 0 && split == 0) atomicOr(a.status, kStatusBadSeqlens);
      tb = tiles_of(b);
      t = split * a.per;
      n = min(a.per, tb - t);
      if (tb == 0 && a.splits == 1) {  // nothing to see: O = 0, LSE = -inf
        const long long out_row = (long long)bh * a.rows + row0;
        uint16_t* o = static_cast<uint16_t*>(a.o) + out_row * D;
        for (int e = lane; e < nr * D; e += 32) o[e] = 0;
        for (int e = lane; e < nr; e += 32) a.lse[out_row + e] = neg_inf();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();  // over by now: the walker waited
  const uint32_t tmem = *tmem_slot;
  auto read_segment = [&](int k) {
    const int4 x = *reinterpret_cast<const int4*>(smem + C::OFF_DESC + 32 * (k % C::SEGS));
    const int2 y = *reinterpret_cast<const int2*>(smem + C::OFF_DESC + 32 * (k % C::SEGS) + 16);
    Segment g;
    g.bh = x.x, g.first = x.y, g.n = x.z, g.len = x.w, g.part = y.x, g.pages = y.y;
    return g;
  };

  // Turns rows r0 .. r1 - 1 of segment k's queries into e4m3 terms, four rows
  // at a time, eight lanes a row, the next four on their way; `between` is run
  // while the first are.  The row loop is kept rolled: instructions that run
  // once cost more to fetch than to run.
  auto fill_rows = [&](int k, const Segment& g, int r0, int r1, auto between) {
    constexpr int E = D / 8;  // neighbouring elements of a row a lane
    constexpr int L = E / 8;  // 16-byte loads of them
    const int buf = k % C::SEGS, sub = lane >> 3, col = (lane & 7) * E;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + ((long long)g.bh * a.rows + row0) * D + col;
    uint8_t* q8 = sQ + buf * C::Q_BYTES + (col / C::W) * (C::NB * C::W);
    float* qinv = reinterpret_cast<float*>(smem + C::OFF_ROW) + buf * 2 * R;
    int* row_end = reinterpret_cast<int*>(qinv + R);
    uint4 raw[L], then[L];
    auto load = [&](int r, uint4 (&to)[L]) {
#pragma unroll
      for (int i = 0; i < L; ++i)
        to[i] = r < nr && r < r1 ? reinterpret_cast<const uint4*>(q + (long long)r * D)[i] : make_uint4(0, 0, 0, 0);
    };
    load(r0 + sub, raw);
    between();
#pragma unroll 1
    for (int r = r0 + sub; r < r1; r += 4) {
      load(r + 4, then);
      float x[E];
      uint32_t top = 0;  // the largest magnitude's bits: infinities and NaN come out on top
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const uint4& u = raw[i / 8];
        const uint32_t two = i % 8 == 0 ? u.x : i % 8 == 2 ? u.y : i % 8 == 4 ? u.z : u.w;
        if (C::BF16) {
          x[i] = __uint_as_float(two << 16);
          x[i + 1] = __uint_as_float(two & 0xffff0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
          x[i] = f.x;
          x[i + 1] = f.y;
        }
        top = max(top, max(__float_as_uint(x[i]) & 0x7fffffffu, __float_as_uint(x[i + 1]) & 0x7fffffffu));
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const bool finite = top < 0x7f800000u;
      // 2^e with max * 2^e in [128, 256) (subnormal rows: at most 2^120)
      const int e = finite ? min(134 - static_cast<int>(top >> 23), 120) : 0;
      const float up = __int_as_float((e + 127) << 23);
      uint32_t words[T][E / 4];
#pragma unroll
      for (int i = 0; i < E; i += 4) {
        uint32_t lo[T], hi[T];
        split_terms<T>(finite ? x[i] * up : 0.f, finite ? x[i + 1] * up : 0.f, lo);
        split_terms<T>(finite ? x[i + 2] * up : 0.f, finite ? x[i + 3] * up : 0.f, hi);
#pragma unroll
        for (int u = 0; u < T; ++u) words[u][i / 4] = lo[u] | hi[u] << 16;
      }
#pragma unroll
      for (int u = 0; u < T; ++u) {
        if constexpr (E == 8) {
          *reinterpret_cast<uint2*>(q8 + sw_offset<C::W>(u * R + r, col % C::W)) = make_uint2(words[u][0], words[u][1]);
        } else {
#pragma unroll
          for (int i = 0; i < E / 16; ++i)
            *reinterpret_cast<uint4*>(q8 + sw_offset<C::W>(u * R + r, col % C::W + 16 * i)) =
                make_uint4(words[u][4 * i], words[u][4 * i + 1], words[u][4 * i + 2], words[u][4 * i + 3]);
        }
      }
      if ((lane & 7) == 0) {
        // a row that holds a NaN or an infinity has no softmax: its scores are NaN
        qinv[r] = finite ? __int_as_float((127 - e) << 23) : __int_as_float(0x7fc00000);
        row_end[r] = a.causal ? g.len - a.Nq + (row0 + r) % a.Nq + 1 : g.len;
      }
#pragma unroll
      for (int i = 0; i < L; ++i) raw[i] = then[i];
    }
  };

  if (warp == 4 * G + 2) {
    // ------------------------------------------------------------ segments
    // Walks this CTA's tiles segment by segment (a run of tiles of one head),
    // ahead of the others: where each one is, and its pages.
    // To the next head that has tiles in this CTA's piece; n = 0 when there is none.
    auto advance = [&]() {
      do {
        n = 0;
        at += places_of(tb);
        if (!a.balanced || at >= stop) return;
        if (++h == a.c.Hkv) {
          h = 0;
          do {
            if (++b >= a.c.B) return;  // only if the lengths change while they are read
            tb = tiles_of(b);
          } while (tb == 0);
        }
        place(at);
      } while (n <= 0);
    };
    if (n <= 0) {
      n = 0;
      if (a.balanced && at < stop) advance();
    }
    for (int k = 0;; ++k) {
      const int buf = k % C::SEGS;
      if (k >= C::SEGS && !warp_wait(&seg_free[buf], (k / C::SEGS - 1) & 1, abort_flag, a.status)) break;
      const int bh = b * a.c.Hkv + h;
      const int len = n > 0 ? good_len(a.lens[b], a.max_len) : 0;
      const int end = min(len, (t + n) * 128);  // one past the segment's last slot
      const int pages = n > 0 ? (end - t * 128 + ps - 1) >> shift : 0;
      if (lane == 0) {
        int* d = reinterpret_cast<int*>(smem + C::OFF_DESC + 32 * buf);
        d[0] = bh, d[1] = t, d[2] = n, d[3] = len;
        // a whole head goes to O; a CTA has at most two parts of heads: one that ends in it, one that begins
        d[4] = n == tb ? -1 : (int)(2 * (blockIdx.y * gridDim.x + blockIdx.x)) + (a.balanced && t == 0 ? 1 : 0);
        d[5] = pages;
      }
      const int* table = a.c.table + (long long)b * a.c.width + (t * 128 >> shift);
      for (int i = lane; i < pages; i += 32) {
        int id = table[i];
        if (id < 0 || id >= a.c.pages) {
          atomicOr(a.status, kStatusBadPages);
          id = -1;
        }
        s_page[buf * ne + i] = id;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_pages[buf]);
      if (n == 0) break;
      if (a.balanced && t == 0 && lane == 0 && blockIdx.y == 0) {
        // for the joining kernel: how many CTAs share the head, and the first of them
        const int count = n == tb ? 1 : share.owner(at + kHeadCost + tb - 1) - (int)blockIdx.x + 1;
        a.shared[bh] = make_int2(count, blockIdx.x);
      }
      advance();
    }
  } else if (warp == 4 * G + 3) {
    // ------------------------------------------------------------ scales (and queries of one group)
    for (int k = 0;; ++k) {
      const int buf = k % C::SEGS;
      if (!warp_wait(&seg_pages[buf], (k / C::SEGS) & 1, abort_flag, a.status)) break;
      const Segment g = read_segment(k);
      const int head = g.bh % a.c.Hkv;
      auto scales = [&]() {
        for (int i = lane; i < g.pages; i += 32) {
          const int id = s_page[buf * ne + i];
          s_ks[buf * ne + i] = id >= 0 ? a.c.k_scale[(long long)id * a.c.Hkv + head] * a.scale_log2 : 0.f;
          s_vs[buf * ne + i] = id >= 0 ? a.c.v_scale[(long long)id * a.c.Hkv + head] : 0.f;
        }
      };
      if (g.n > 0) {
        if (G == 1)
          fill_rows(k, g, 0, 8, scales);
        else
          scales();
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_ready[buf]);
      if (g.n == 0) break;
    }
  } else if (warp == 4 * G) {
    // ------------------------------------------------------------ producer
    // Tiles in the order K0, K1, V0, K2, V1, ... over all segments.
    const int per = 128 >> shift;  // pages a tile
    bool ok = true;
    struct Cursor {
      int k = -1, t = 0, n = 0, h = 0, end = 0;
    } kc, vc;
    // to the next tile: false when there is none (or on abort)
    auto next = [&](Cursor& c) {
      if (++c.t < c.n) return true;
      ++c.k;
      if (!(ok = warp_wait(&seg_pages[c.k % C::SEGS], (c.k / C::SEGS) & 1, abort_flag, a.status))) return false;
      const Segment g = read_segment(c.k);
      c.t = 0;
      c.n = g.n;
      c.h = g.bh % a.c.Hkv;
      c.end = g.pages;
      return g.n > 0;
    };
    const uint64_t policy = stream_policy();
    int pk = 0, pv = 0;  // items of K and V issued
    auto load = [&](const Cursor& c, const CUtensorMap* map, int& p, int first, int slots) {
      const int e = c.t * per + lane;
      const int id = lane < per && e < c.end ? s_page[(c.k % C::SEGS) * ne + e] : -1;
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, id >= 0)) * ps * C::W;
      for (int hf = 0; hf < C::HALVES; ++hf, ++p) {
        const int slot = first + p % slots;
        if (!(ok = warp_wait(&ring_empty[slot], ((p / slots) & 1) ^ 1, abort_flag, a.status))) return;
        if (lane == 0) mbar_arrive_expect_tx(&ring_full[slot], bytes);
        __syncwarp();
        if (id >= 0)
          tma_stream_3d(sRing + slot * C::ITEM + lane * ps * C::W, map, &ring_full[slot], hf * 128, 0,
                        id * a.c.Hkv + c.h, policy);
      }
    };
    // a segment's list is waited for only when V of the tile two before is on
    // its way: the list two segments on needs the place of that tile's
    bool more = true;
    auto load_k = [&]() {
      more = more && next(kc);
      if (more) load(kc, &a.tm_k, pk, 0, C::NSK);
    };
    load_k();
    if (ok) load_k();
    while (ok && next(vc)) {
      load(vc, &a.tm_v, pv, C::NSK, C::NSV);
      if (!ok) break;
      if (vc.t == vc.n - 1 && lane == 0) mbar_arrive(&seg_free[vc.k % C::SEGS]);
      load_k();
    }
    if (*abort_flag && lane == 0) {
      for (int x = pk - C::NSK < 0 ? 0 : pk - C::NSK; x < pk; ++x)
        drain_wait(&ring_full[x % C::NSK], (uint32_t)((x / C::NSK) & 1));
      for (int x = pv - C::NSV < 0 ? 0 : pv - C::NSV; x < pv; ++x)
        drain_wait(&ring_full[C::NSK + x % C::NSV], (uint32_t)((x / C::NSV) & 1));
    }
    __syncwarp();
  } else if (warp == 4 * G + 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t id_s = idesc_f8(128, C::NB, a.c.e5m2, false);
      const uint32_t id_pv = idesc_f8(128, C::NB, a.c.e5m2, true);
      const uint32_t q = smem_u32(sQ), pw = smem_u32(sP), ring = smem_u32(sRing);
      constexpr int GROUP = 8 * C::W;  // eight rows: the stride of the swizzle pattern
      bool ok = true;
      int pk = 0, pv = 0;
      auto take = [&](int& slot, int& p, int first, int slots) {
        slot = first + p % slots;
        ok = mbar_wait(&ring_full[slot], (p / slots) & 1, abort_flag, a.status, kStatusTimeout);
        ++p;
        tc_fence_after();
        return ok;
      };
      int sk = -1, st = 0, sn = 0, sj = 0;  // next score tile: segment, tile in it, its tiles; tile over all
      bool more = true;
      // the tiles of the segments whose scores are under way, in words of the
      // descriptors that are this thread's own: a descriptor itself may be
      // overwritten as soon as the softmax is done with the segment
      auto tiles_in = [&](int k) -> volatile int& {
        return *reinterpret_cast<volatile int*>(smem + C::OFF_DESC + 32 * (k % C::SEGS) + 24 + 4 * ((k / C::SEGS) & 1));
      };
      // S of the next tile: slots as rows (K-major A), query terms as columns
      auto issue_s = [&]() {
        if (++st >= sn) {
          ++sk;
          if (!(ok = mbar_wait(&seg_ready[sk % C::SEGS], (sk / C::SEGS) & 1, abort_flag, a.status, kStatusTimeout))) return;
          st = 0;
          sn = read_segment(sk).n;
          if (sn == 0) {
            more = false;
            return;
          }
          tiles_in(sk) = sn;
        }
        const int i = sj & 1;
        for (int hf = 0; hf < C::HALVES; ++hf) {
          int slot;
          if (!take(slot, pk, 0, C::NSK)) return;
          const uint64_t da = sdesc_w<C::W>(ring + slot * C::ITEM, 16, GROUP);
          const uint64_t db = sdesc_w<C::W>(q + (sk % C::SEGS) * C::Q_BYTES + hf * C::NB * C::W, 16, GROUP);
#pragma unroll
          for (int kk = 0; kk < C::W / 32; ++kk)
            mma_f8(tmem + C::COL_S + C::NB * i, sdesc_advance(da, 32 * kk), sdesc_advance(db, 32 * kk), id_s,
                   hf > 0 || kk > 0);
          mma_commit(&ring_empty[slot]);
        }
        mma_commit(&s_full[i]);
        ++sj;
      };
      issue_s();
      if (ok && more) issue_s();
      int vk = 0, vt = 0, vn = 0;  // segment and tile of PV
      for (int j = 0; ok && j < sj; ++j) {
        const int i = j & 1;
        if (vt == 0) vn = tiles_in(vk);
        if (!(ok = mbar_wait(&p_full[i], (j >> 1) & 1, abort_flag, a.status, kStatusTimeout))) break;
        // a segment's first product overwrites what the one before left for its epilogue
        if (vt == 0 && vk > 0 &&
            !(ok = mbar_wait(o_free, (vk - 1) & 1, abort_flag, a.status, kStatusTimeout)))
          break;
        tc_fence_after();
        for (int hf = 0; hf < C::HALVES; ++hf) {
          int slot;
          if (!take(slot, pv, C::NSK, C::NSV)) break;
          // features as rows (MN-major A: a row of memory is a slot); at
          // d = 64 both 64-feature halves of M = 128 read the same bytes
          // (offset 0 between them), lanes 64-127 repeat lanes 0-63
          const uint64_t da = sdesc_w<C::W>(ring + slot * C::ITEM, 0, GROUP);
          const uint64_t db = sdesc_w<128>(pw + i * C::P_BYTES, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f8(tmem + C::COL_O + C::NB * hf, sdesc_advance(da, 32 * C::W * kk), sdesc_advance(db, 32 * kk),
                   id_pv, vt > 0 || kk > 0);
          mma_commit(&ring_empty[slot]);
        }
        if (!ok) break;
        mma_commit(&pv_done[i]);
        if (++vt == vn) {
          vt = 0;
          ++vk;
        }
        if (more) issue_s();
      }
      if (!ok) {
        mma_commit(drain);
        drain_wait(drain, 0);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax, epilogue
    // Group g of four warps: rows 8 g .. 8 g + 7; warp w of it: slots 32 w .. 32 w + 31 of a tile.
    const int g8 = (warp >> 2) * 8, quarter = warp & 3;
    const int key = quarter * 32 + lane;  // slot of the tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    uint64_t* my_exchange = exchange + (warp >> 2) * 2;
    float* my_max = reinterpret_cast<float*>(smem + C::OFF_MAX) + (warp >> 2) * 64;
    float* my_sum = reinterpret_cast<float*>(smem + C::OFF_SUM) + (warp >> 2) * 32;
    // byte of this slot in row 0 of the group's weights; row r is at 128 r with
    // the 16-byte chunk XORed with r (the buffer begins on a 1024-byte boundary)
    const uint32_t p_byte = smem_u32(sP) + g8 * 128 + key;
    // the lowest number: no score but -inf is below it, and -inf - m is -inf
    constexpr float kNothing = -3.402823466e38f;
    int j = 0;  // tile over all segments
    int x = 0;  // exchanges so far
    bool ok = true;
    // With several groups two warps of each turn its rows into terms (one warp
    // for all would take 9 us for 40 rows).  Those of the next segment before
    // the end of this one: the MMA warp issues a tile's scores ahead of the
    // products of the two tiles before it.
    auto queries = [&](int k) {
      if (G == 1) return;
      ok = warp_wait(&seg_pages[k % C::SEGS], (k / C::SEGS) & 1, abort_flag, a.status);
      if (ok && quarter < 2) {
        const Segment g = read_segment(k);
        if (g.n > 0) fill_rows(k, g, g8 + 4 * quarter, g8 + 4 * quarter + 4, []() {});
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_ready[k % C::SEGS]);
      }
    };
    queries(0);
    for (int k = 0; ok; ++k) {
      const int buf = k % C::SEGS;
      if (!(ok = warp_wait(&seg_ready[buf], (k / C::SEGS) & 1, abort_flag, a.status))) break;
      const Segment g = read_segment(k);
      if (g.n == 0) break;
      const int* page = s_page + buf * ne;
      const float* qinv = reinterpret_cast<const float*>(smem + C::OFF_ROW) + buf * 2 * R + g8;
      const int* row_end = reinterpret_cast<const int*>(qinv + R);
      const int first_end = a.causal ? g.len - a.Nq + 1 : g.len;  // the fewest slots that a row sees
      const long long out_row = (long long)g.bh * a.rows + row0 + g8;
      const int rows_here = nr - g8;
      float* scores = a.scores + ((long long)g.bh * a.score_groups + (row0 + g8) / 8) * a.score_stride;
      uint64_t l[4];
      float m[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) m[r] = kNothing;
#pragma unroll
      for (int r = 0; r < 4; ++r) l[r] = 0;
      for (int t = 0; t < g.n; ++t, ++j) {
        const int i = j & 1;
        const uint32_t tS = lane_base + C::COL_S + C::NB * i + g8;
        const int slot = (g.first + t) * 128 + key;
        const int e = buf * ne + ((t * 128 + key) >> shift);
        const bool live = slot < g.len && page[(t * 128 + key) >> shift] >= 0;
        const float ks = live ? s_ks[e] : 0.f, vs = live ? s_vs[e] : 0.f;
        const float lv = scale_exponent(vs), wv = vs * kWeightScale;
        if (!(ok = warp_wait(&s_full[i], (j >> 1) & 1, abort_flag, a.status))) break;
        tc_fence_after();
        uint64_t s[4];
        {
          float y[T][8];
#pragma unroll
          for (int u = 0; u < T; ++u) tmem_ld8(tS + u * R, y[u]);
#pragma unroll
          for (int u = 0; u < T; ++u) tmem_ld8_wait(y[u]);
          join_terms<T>(y, s);
#pragma unroll
          for (int r = 0; r < 4; r += 2) {
            const float4 q = *reinterpret_cast<const float4*>(qinv + 2 * r);
            // the two scales first: a large one and a small one may meet
            s[r] = f2_mul(s[r], f2_mul(f2_pack(q.x, q.y), f2_pack(ks, ks)));
            s[r + 1] = f2_mul(s[r + 1], f2_mul(f2_pack(q.z, q.w), f2_pack(ks, ks)));
          }
        }
        if (!live || (g.first + t) * 128 + 128 > first_end) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float y0, y1;
            f2_unpack(s[r], y0, y1);
            if (!live || slot >= row_end[2 * r]) y0 = neg_inf();
            if (!live || slot >= row_end[2 * r + 1]) y1 = neg_inf();
            s[r] = f2_pack(y0, y1);
          }
        }
        if (a.scores != nullptr && slot < g.len && rows_here > 0) {
          float* to = scores + (long long)slot * a.score_rows;
          if (a.score_rows >= 4) {
            *reinterpret_cast<ulonglong2*>(to) = make_ulonglong2(s[0], s[1]);
            if (a.score_rows == 8) *reinterpret_cast<ulonglong2*>(to + 4) = make_ulonglong2(s[2], s[3]);
          } else if (a.score_rows == 2) {
            *reinterpret_cast<uint64_t*>(to) = s[0];
          } else {
            float y0, y1;
            f2_unpack(s[0], y0, y1);
            *to = y0;
          }
        }
        float* mine = my_max + ((x & 1) * 4 + quarter) * 8;
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
          float4 top;
          f2_unpack(f2_add(s[r], f2_pack(lv, lv)), top.x, top.y);
          f2_unpack(f2_add(s[r + 1], f2_pack(lv, lv)), top.z, top.w);
          top.x = warp_max(top.x);
          top.y = warp_max(top.y);
          top.z = warp_max(top.z);
          top.w = warp_max(top.w);
          if (lane == 0) *reinterpret_cast<float4*>(mine + 2 * r) = top;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&my_exchange[x & 1]);
        if (!(ok = warp_wait(&my_exchange[x & 1], (x >> 1) & 1, abort_flag, a.status))) break;
        // every thread derives the same new references from the four warps' maxima
        float top[8];
        const float* all = my_max + (x & 1) * 32;
        ++x;
#pragma unroll
        for (int r = 0; r < 8; r += 4) {
          const float4 y0 = *reinterpret_cast<const float4*>(all + r);
          const float4 y1 = *reinterpret_cast<const float4*>(all + 8 + r);
          const float4 y2 = *reinterpret_cast<const float4*>(all + 16 + r);
          const float4 y3 = *reinterpret_cast<const float4*>(all + 24 + r);
          top[r] = max3(fmaxf(y0.x, y1.x), y2.x, y3.x);
          top[r + 1] = max3(fmaxf(y0.y, y1.y), y2.y, y3.y);
          top[r + 2] = max3(fmaxf(y0.z, y1.z), y2.z, y3.z);
          top[r + 3] = max3(fmaxf(y0.w, y1.w), y2.w, y3.w);
        }
        bool moved = false;
#pragma unroll
        for (int r = 0; r < 8; ++r) moved |= top[r] > m[r] + kMaxLead;
        if (moved) {  // the same on every thread of the group
          uint64_t corr[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float c[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const float next = top[2 * r + z] > m[2 * r + z] + kMaxLead ? top[2 * r + z] : m[2 * r + z];
              c[z] = ex2_approx(m[2 * r + z] - next);
              m[2 * r + z] = next;
            }
            corr[r] = f2_pack(c[0], c[1]);
            l[r] = f2_mul(l[r], corr[r]);
          }
          if (t > 0) {  // PV(j - 1) may still add to O
            if (!(ok = warp_wait(&pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, abort_flag, a.status))) break;
            tc_fence_after();
#pragma unroll
            for (int hf = 0; hf < C::HALVES; ++hf) {
              float y[T][8];
#pragma unroll
              for (int u = 0; u < T; ++u) tmem_ld8(lane_base + C::COL_O + C::NB * hf + u * R + g8, y[u]);
#pragma unroll
              for (int u = 0; u < T; ++u) tmem_ld8_wait(y[u]);
#pragma unroll
              for (int u = 0; u < T; ++u) {
                uint32_t z[8];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                  float z0, z1;
                  f2_unpack(f2_mul(f2_pack(y[u][2 * r], y[u][2 * r + 1]), corr[r]), z0, z1);
                  z[2 * r] = __float_as_uint(z0);
                  z[2 * r + 1] = __float_as_uint(z1);
                }
                tmem_st8(lane_base + C::COL_O + C::NB * hf + u * R + g8, z);
              }
            }
            tmem_st_wait();
          }
        }
#pragma unroll
        for (int r = 0; r < 8; r += 2) {
          float x0, x1;
          f2_unpack(f2_add(s[r / 2], f2_pack(-m[r], -m[r + 1])), x0, x1);
          const uint64_t p = f2_pack(ex2_approx(x0), ex2_approx(x1));
          l[r / 2] = f2_add(l[r / 2], p);
          uint32_t code[T];
          split_terms<T>(f2_mul(p, f2_pack(wv, wv)), code);
          const uint32_t at = p_byte + i * C::P_BYTES;
#pragma unroll
          for (int u = 0; u < T; ++u) {
            asm volatile("st.shared.u8 [%0], %1;" ::"r"((at ^ (r << 4)) + (u * R + r) * 128), "r"(code[u]) : "memory");
            asm volatile("st.shared.u8 [%0], %1;" ::"r"((at ^ ((r + 1) << 4)) + (u * R + r + 1) * 128),
                         "r"(code[u] >> 8)
                         : "memory");
          }
        }
        if (!live && g8 == 0) {  // no bytes of this slot may reach the product
          for (int hf = 0; hf < C::HALVES; ++hf) {
            const int p = j * C::HALVES + hf, at = C::NSK + p % C::NSV;
            if (!mbar_wait(&ring_full[at], (p / C::NSV) & 1, abort_flag, a.status, kStatusTimeout)) ok = false;
            uint4* row = reinterpret_cast<uint4*>(sRing + at * C::ITEM + key * C::W);
            if (ok)
              for (int c = 0; c < C::W / 16; ++c) row[c] = make_uint4(0, 0, 0, 0);
          }
        }
        fence_async_smem();
        tc_fence_before();
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (lane == 0) mbar_arrive(&p_full[i]);
      }
      if (!ok) break;
      if (lane == 0) mbar_arrive(&seg_free[buf]);
      queries(k + 1);
      if (!ok) break;
      // l over the 128 slots of a tile: lanes, then warps
#pragma unroll 1
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < 4; ++r) l[r] = f2_add(l[r], __shfl_xor_sync(0xffffffffu, l[r], o));
      if (lane == 0) {
        *reinterpret_cast<ulonglong2*>(my_sum + quarter * 8) = make_ulonglong2(l[0], l[1]);
        *reinterpret_cast<ulonglong2*>(my_sum + quarter * 8 + 4) = make_ulonglong2(l[2], l[3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&my_exchange[x & 1]);
      if (!(ok = warp_wait(&my_exchange[x & 1], (x >> 1) & 1, abort_flag, a.status))) break;
      ++x;
      if (!(ok = warp_wait(&pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, abort_flag, a.status))) break;
      tc_fence_after();
      uint64_t inv[4];
      const long long part_row = (long long)g.part * R + g8;
#pragma unroll
      for (int r = 0; r < 8; r += 2) {
        float v[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float y = my_sum[r + z] + my_sum[8 + r + z] + my_sum[16 + r + z] + my_sum[24 + r + z];
          v[z] = y == 0.f ? 0.f : (1.f / kWeightScale) / y;
        }
        inv[r / 2] = f2_pack(v[0], v[1]);
      }
      if (key < 8 && key < rows_here) {  // a thread a row
        float mine = m[0];
#pragma unroll
        for (int r = 1; r < 8; ++r) mine = key == r ? m[r] : mine;
        const float y = my_sum[key] + my_sum[8 + key] + my_sum[16 + key] + my_sum[24 + key];
        const float lse2 = y == 0.f ? neg_inf() : add_log2(mine, y);
        if (g.part < 0)
          a.lse[out_row + key] = lse2 * kLn2;
        else
          a.lse_part[part_row + key] = lse2;
      }
#pragma unroll
      for (int hf = 0; hf < C::HALVES; ++hf) {
        float y[T][8];
#pragma unroll
        for (int u = 0; u < T; ++u) tmem_ld8(lane_base + C::COL_O + C::NB * hf + u * R + g8, y[u]);
#pragma unroll
        for (int u = 0; u < T; ++u) tmem_ld8_wait(y[u]);
        uint64_t o[4];
        join_terms<T>(y, o);
        const int f = hf * 128 + key;
        float z[8];
#pragma unroll
        for (int r = 0; r < 4; ++r) f2_unpack(f2_mul(o[r], inv[r]), z[2 * r], z[2 * r + 1]);
        if (f >= D) {
          // d = 64: the upper lanes repeat the lower ones
        } else if (g.part >= 0) {
          float* to = a.o_part + part_row * D + f;
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r < rows_here) to[r * D] = z[r];
        } else {
          uint16_t* to = static_cast<uint16_t*>(a.o) + out_row * D + f;
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r < rows_here)
              to[r * D] = C::BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(z[r]))
                                  : __half_as_ushort(__float2half_rn(z[r]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 4 * G + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Where the parts of a head are: part `first` of the CTA in which it begins,
// then parts first + 1, first + 3, ... of the next ones (balanced), or parts
// first, first + 2, ... of its chunks.  `count` parts; 1: it was not shared,
// 0: it is empty.
struct Parts {
  int count;
  long long first;
  int jump;  // from the first to the second
  __device__ __forceinline__ long long at(int s) const { return s == 0 ? first : first + jump + 2 * (s - 1); }
};
__device__ __forceinline__ Parts find_parts(const PagedAttnArgs& a, int bh, int tile_y) {
  const int tb = (good_len(a.lens[bh / a.c.Hkv], a.max_len) + 127) >> 7;
  Parts p;
  if (a.balanced) {
    const int2 x = a.shared[bh];  // written only for heads that hold something
    p.count = tb > 0 ? x.x : 0;
    p.first = 2 * ((long long)tile_y * a.ctas + x.y) + 1;
    p.jump = 1;
  } else {
    p.count = (tb + a.per - 1) / a.per;
    p.first = 2 * ((long long)tile_y * a.ctas + (long long)bh * a.splits);
    p.jump = 2;
  }
  return p;
}

// sum[k] += sum over the rows, in order, of 2^(score - z[row]) for slots slot0 + 256 k; z = +inf: a row that sees
// nothing (its scores are -inf).  W rows lie together, groups of W `stride` apart.
template <int W, int SLOTS>
__device__ __forceinline__ void load_scores(const float* from, int slot0, int len, float (&y)[SLOTS][W]) {
#pragma unroll
  for (int k = 0; k < SLOTS; ++k)
    if (slot0 + 256 * k < len) {
      const float* at = from + (long long)(slot0 + 256 * k) * W;
      if constexpr (W >= 4) {
#pragma unroll
        for (int r = 0; r < W; r += 4) {
          const float4 v = *reinterpret_cast<const float4*>(at + r);
          y[k][r] = v.x, y[k][r + 1] = v.y, y[k][r + 2] = v.z, y[k][r + 3] = v.w;
        }
      } else if constexpr (W == 2) {
        const float2 v = *reinterpret_cast<const float2*>(at);
        y[k][0] = v.x, y[k][1] = v.y;
      } else {
        y[k][0] = *at;
      }
    }
}
// `y` holds the first group's scores.
template <int W, int SLOTS>
__device__ __forceinline__ void add_weights(const float* from, long long stride, const float* z, int rows, int slot0,
                                            int len, float (&y)[SLOTS][W], float (&sum)[SLOTS]) {
  for (int g = 0; g < rows; g += W, from += stride) {
    float ref[W];
    if (g > 0) load_scores<W, SLOTS>(from, slot0, len, y);
#pragma unroll
    for (int r = 0; r < W; ++r) ref[r] = g + r < rows ? z[g + r] : __int_as_float(0x7f800000);
#pragma unroll
    for (int k = 0; k < SLOTS; ++k)
#pragma unroll
      for (int r = 0; r < W; ++r)
        if (g + r < rows) sum[k] += ex2_approx(y[k][r] - ref[r]);
  }
}

// 16 scores a thread under way
constexpr int weight_slots(int w) { return w == 8 ? 2 : 4; }

// Joins the parts of a row that several CTAs shared (the first row_blocks
// blocks; `team` warps a row): O = sum 2^(LSE_s) O_s / sum 2^(LSE_s), LSE =
// log2 of that sum, with a running maximum; the warps of a team take parts in
// turn and are added in order at the end, so the result does not depend on
// which CTA was first.  Rows of heads that one CTA had alone are in place
// already; empty sequences get O = 0 and LSE = -inf here.
// The other blocks add the weights: weight_acc[slot] += sum over the head's
// rows, in order, of 2^(score - LSE).  LSE is joined from the parts there as
// well: a launch that waited for the first blocks would take longer.
template <int D, int W>
__global__ void __launch_bounds__(256, 5) paged_finish_kernel(const __grid_constant__ PagedAttnArgs a, int row_blocks,
                                                           int team) {
  constexpr int V = D / 32;  // features a lane
  __shared__ float s_o[8][D];
  __shared__ float2 s_ml[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch();
  if ((int)blockIdx.x < row_blocks) {
    const int row = blockIdx.x * (8 / team) + warp / team, member = warp % team;
    const bool there = row < a.c.B * a.c.Hkv * a.rows;
    const int bh = there ? row / a.rows : 0, in_head = row % a.rows;
    pdl_wait();
    const Parts p = find_parts(a, bh, in_head / a.row_tile);
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    float m = neg_inf(), l = 0.f;
    const bool mine = there && p.count != 1;
    if (mine) {
#pragma unroll 2
      for (int s = member; s < p.count; s += team) {
        const long long at = p.at(s) * a.row_tile + in_head % a.row_tile;
        const float z = a.lse_part[at];
        float x[V];
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float2 two = *reinterpret_cast<const float2*>(a.o_part + at * D + lane * V + i);
          x[i] = two.x;
          x[i + 1] = two.y;
        }
        const float top = fmaxf(m, z), ref = top == neg_inf() ? 0.f : top;
        const float c = exp2f(m - ref), w = exp2f(z - ref);
        m = top;
        l = l * c + w;
        // a part that saw nothing has weight 0; a NaN goes through
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = acc[i] * c + (w == 0.f ? 0.f : w * x[i]);
      }
    }
    if (team > 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) s_o[warp][lane * V + i] = acc[i];
      if (lane == 0) s_ml[warp] = make_float2(m, l);
      __syncthreads();
      if (member == 0) {
        float top = m;
        for (int k = 1; k < team; ++k) top = fmaxf(top, s_ml[warp + k].x);
        const float ref = top == neg_inf() ? 0.f : top;
        float c = exp2f(m - ref);
        l *= c;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] *= c;
        for (int k = 1; k < team; ++k) {
          c = exp2f(s_ml[warp + k].x - ref);
          l += s_ml[warp + k].y * c;
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] += s_o[warp + k][lane * V + i] * c;
        }
        m = top;
      }
    }
    if (!mine || member != 0) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint32_t out[V / 2];
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      if (a.bf16) {
        __nv_bfloat162 x = __floats2bfloat162_rn(acc[i] * inv, acc[i + 1] * inv);
        out[i / 2] = *reinterpret_cast<uint32_t*>(&x);
      } else {
        __half2 x = __floats2half2_rn(acc[i] * inv, acc[i + 1] * inv);
        out[i / 2] = *reinterpret_cast<uint32_t*>(&x);
      }
    }
    uint32_t* o = reinterpret_cast<uint32_t*>(a.o) + ((long long)row * D + lane * V) / 2;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) o[i] = out[i];
    if (lane == 0) a.lse[row] = l == 0.f ? neg_inf() : ((m == neg_inf() ? 0.f : m) + __log2f(l)) * kLn2;
    return;
  }
  if constexpr (W > 0) {
    // ---------------------------------------------------------------- weights
    constexpr int SLOTS = weight_slots(W);  // slots a thread, 256 apart
    __shared__ float s_z[64];  // LSE of the rows at hand
    const int per_head = (a.max_len + 256 * SLOTS - 1) / (256 * SLOTS);
    const int x = blockIdx.x - row_blocks;
    const int bh = x / per_head, slot0 = (x % per_head) * (256 * SLOTS) + threadIdx.x;
    pdl_wait();
    const int len = good_len(a.lens[bh / a.c.Hkv], a.max_len);
    if ((x % per_head) * (256 * SLOTS) >= len) return;
    const Parts p = find_parts(a, bh, 0);  // the same for every row tile, but for the first part's number
    float* to = a.weight_acc + (long long)bh * a.c.width * a.c.ps;
    float was[SLOTS], sum[SLOTS];
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) {
      was[k] = slot0 + 256 * k < len ? to[slot0 + 256 * k] : 0.f;
      sum[k] = 0.f;
    }
    for (int r0 = 0; r0 < a.rows; r0 += 64) {
      const int rows = min(64, a.rows - r0);
      if (r0 > 0) __syncthreads();
      const float* from = a.scores + ((long long)bh * a.score_groups + r0 / 8) * a.score_stride;
      float y[SLOTS][W];
      load_scores<W, SLOTS>(from, slot0, len, y);  // under way while the rows' LSE are joined
      for (int r = warp; r < rows; r += 8) {  // a warp a row, its lanes the parts
        const int in_head = r0 + r;
        float m = neg_inf(), l = 0.f;
        if (p.count == 1) {
          m = a.lse[(long long)bh * a.rows + in_head] * kLog2e;
          l = m == neg_inf() ? 0.f : 1.f;
        } else {
          const long long tile = 2ll * (in_head / a.row_tile) * a.ctas;
          for (int s = lane; s < p.count; s += 32) {
            const float y = a.lse_part[(tile + p.at(s)) * a.row_tile + in_head % a.row_tile];
            const float top = fmaxf(m, y), ref = top == neg_inf() ? 0.f : top;
            l = l * exp2f(m - ref) + exp2f(y - ref);
            m = top;
          }
          const float top = warp_max(m), ref = top == neg_inf() ? 0.f : top;
          l = warp_sum(l * exp2f(m - ref));
          m = top;
        }
        if (lane == 0) s_z[r] = l == 0.f ? -neg_inf() : (m == neg_inf() ? 0.f : m) + __log2f(l);
      }
      __syncthreads();
      add_weights<W, SLOTS>(from, a.score_stride, s_z, rows, slot0, len, y, sum);
    }
#pragma unroll
    for (int k = 0; k < SLOTS; ++k)
      if (slot0 + 256 * k < len) to[slot0 + 256 * k] = was[k] + sum[k];
  }
}

template <int D, int T, int G>
cudaError_t launch_attention_t(const PagedAttnArgs& a, cudaStream_t stream) {
  using C = PagedCfg<D, T, G>;
  auto kern = paged_attention_kernel<D, T, G>;
  // the same limit in every call: another thread may be about to launch with more pages
  constexpr int kMostPages = kPagedMaxChunk / 16;
  static_assert(C::smem(kMostPages) <= 232448, "shared memory budget");
  if (a.seg_pages > kMostPages) return cudaErrorInvalidValue;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(kMostPages));
  if (e != cudaSuccess) return e;
  const int smem = C::smem(a.seg_pages);
  const dim3 grid((unsigned)a.ctas, (unsigned)((a.rows + C::R - 1) / C::R));
  return launch_pdl(kern, grid, dim3(C::WARPS * 32), smem, stream, a);
}

template <int D, int T>
cudaError_t launch_groups(const PagedAttnArgs& a, cudaStream_t stream) {
  switch (a.row_tile) {
    case 8: return launch_attention_t<D, T, 1>(a, stream);
    case 16: return launch_attention_t<D, T, 2>(a, stream);
    case 24: return launch_attention_t<D, T, 3>(a, stream);
    case 32: return launch_attention_t<D, T, 4>(a, stream);
    case 40: return launch_attention_t<D, T, 5>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

template <int D>
cudaError_t launch_d(const PagedAttnArgs& a, cudaStream_t stream) {
  cudaError_t e = a.bf16 ? launch_groups<D, 2>(a, stream) : launch_groups<D, 3>(a, stream);
  if (e != cudaSuccess) return e;
  const long long BH = (long long)a.c.B * a.c.Hkv;
  const bool join = a.balanced || a.splits > 1;
  // warps that join a row: about as many as it has parts
  int team = 1;
  if (a.balanced)
    while (team < 8 && team * BH < a.ctas) team *= 2;
  else
    while (team < 8 && team < a.splits) team *= 2;
  const long long row_blocks = join ? (BH * a.rows * team + 7) / 8 : 0;
  const int width = a.weight_acc ? a.score_rows : 0;
  const int per_block = 256 * weight_slots(width);
  const long long blocks = row_blocks + (width ? BH * ((a.max_len + per_block - 1) / per_block) : 0);
  if (blocks == 0) return cudaSuccess;
  auto kern = width == 0   ? paged_finish_kernel<D, 0>
              : width == 1 ? paged_finish_kernel<D, 1>
              : width == 2 ? paged_finish_kernel<D, 2>
              : width == 4 ? paged_finish_kernel<D, 4>
                           : paged_finish_kernel<D, 8>;
  return launch_pdl(kern, dim3((unsigned)blocks), dim3(256), 0, stream, a, (int)row_blocks, team);
}

}  // namespace

PagedPlan paged_plan(int B, int Hkv, int rows, int d, int ps, int max_len, int num_splits) {
  PagedPlan p;
  // row tiles of at most 40 rows, as even as groups of eight allow
  const int row_tiles = (rows + 39) / 40;
  p.row_tile = ((rows + row_tiles - 1) / row_tiles + 7) / 8 * 8;
  const int sms = sm_count();
  const long long resident = (long long)paged_occupancy(d, p.row_tile) * sms;
  const long long BH = (long long)B * Hkv;
  const int tiles = (max_len + 127) / 128;
  const long long all = BH * places_of(tiles);
  constexpr int kMostTiles = kPagedMaxChunk / 128;
  p.min_tiles = 6;
  int segment;  // tiles of the longest segment
  if (num_splits == 0 && tiles > 4 && B <= kPagedMaxBalanced) {
    // The device shares out what there is.  A CTA never gets more than
    // kMostTiles, whatever the lengths are.
    p.balanced = true;
    long long ctas = resident / row_tiles;
    if (ctas < 1) ctas = 1;
    const long long want = (all + p.min_tiles - 1) / p.min_tiles, need = (all + kMostTiles - 2) / (kMostTiles - 1);
    if (ctas > want) ctas = want;
    if (ctas < need) ctas = need;
    p.ctas = ctas;
    p.splits = 1;
    p.per = 0;
    // a piece of the line; where the lengths leave less than this, pieces of at most min_tiles
    long long share = (all + ctas - 1) / ctas + 1;
    if (share < p.min_tiles) share = p.min_tiles;
    segment = (int)(share < tiles ? share : tiles);
    p.parts = 2 * ctas * row_tiles;
  } else {
    const int splits = num_splits ? num_splits : 1;
    p.balanced = false;
    p.per = (tiles + splits - 1) / splits;
    if (p.per > kMostTiles) p.per = kMostTiles;
    p.splits = (tiles + p.per - 1) / p.per;
    p.ctas = BH * p.splits;
    segment = p.per;
    p.parts = p.splits > 1 ? 2 * p.ctas * row_tiles : 0;
  }
  p.seg_pages = (segment * 128 + ps - 1) / ps;
  return p;
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a, cudaStream_t stream) {
  if (a.c.d == 64) return launch_d<64>(a, stream);
  if (a.c.d == 128) return launch_d<128>(a, stream);
  if (a.c.d == 256) return launch_d<256>(a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fa
