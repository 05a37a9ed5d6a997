// Attention over the 8-bit paged K/V cache: few queries a sequence against
// its slots, split over the slots, grouped query heads.
//
// A CTA takes up to R query rows of one K / V head (its query heads' rows are
// consecutive: rows = group * Nq, row x is query x % Nq) and one chunk of the
// sequence's slots, and runs the online-softmax recurrence ("FlashAttention
// 为什么不需要存下注意力矩阵", jefxiong.cn, section 3.2) over tiles of 128 slots.
// The chunk's normalised O_s (float32) and LSE_s (log2 units) go to the
// workspace; paged_combine_kernel merges the chunks exactly.
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
// s_j + log2 vs_j instead of s_j, so that w lies in [0, 2] whatever the
// scales are and a page of large scale costs the others no precision; the sum
// l keeps 2^(s_j - m) in float32.
//
// Masked slots (behind the length, on a page that the table names wrongly,
// or behind a causal query's own slot): their scores are replaced by -inf
// after the product, whatever their bytes are; rows of V that no query of the
// sequence may see are overwritten with zeros in shared memory before the
// product, since a weight of 0 times a NaN would be a NaN.
//
// Roles (192 threads): warps 0-3 softmax and epilogue, warp 4 TMA (one copy a
// page, lane i the i-th page of a tile), warp 5 TMEM and MMA issue.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_paged.h"
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
// log2 of the smallest V scale that moves the reference: 2^(s - m) then
// stays below 2^100, far from overflow.
constexpr float kMinLogScale = -100.0f;

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

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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
// The T terms of a pair of values: codes in out[0 .. T-1].
template <int T>
__device__ __forceinline__ void split_terms(float a, float b, uint32_t (&out)[T]) {
#pragma unroll
  for (int t = 0; t < T; ++t) {
    out[t] = to_e4m3x2(a, b);
    if (t + 1 < T) {  // what is left, times 16: exact, the code is a rounding of the value
      const float2 c = from_e4m3x2(out[t]);
      a = (a - c.x) * 16.f;
      b = (b - c.y) * 16.f;
    }
  }
}

template <int D, int T, int R>
struct PagedCfg {
  static constexpr int W = D == 64 ? 64 : 128;        // bytes of a shared-memory row
  static constexpr int HALVES = D == 256 ? 2 : 1;     // 128-feature parts of a K or V tile
  static constexpr int ITEM = 128 * W;                // one ring slot: 128 slots x W bytes
  static constexpr int NB = (T * R + 15) / 16 * 16;   // columns of operand B (multiple of 16 at M = 128)
  static constexpr int SCOL = NB <= 16 ? 16 : NB <= 32 ? 32 : NB <= 64 ? 64 : 128;
  static constexpr uint32_t COL_S = 0;                // two score buffers
  static constexpr uint32_t COL_O = 2 * SCOL;         // HALVES accumulators
  static constexpr uint32_t TMEM_COLS = 4 * SCOL;
  // Two CTAs on an SM (about 96 KB of K and V in flight each), one where
  // the TMEM columns are taken up (NB = 96).
  static constexpr bool ALONE = NB == 96;
  static constexpr int Q_BYTES = HALVES * NB * W;
  static constexpr int P_BYTES = NB * 128;
  static constexpr int BUDGET = (ALONE ? 200 : 105) * 1024;
  static constexpr int NS_MAX = (BUDGET - Q_BYTES - 2 * P_BYTES) / ITEM;
  static constexpr int NS = NS_MAX < 12 ? NS_MAX : 12;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_P = Q_BYTES;
  static constexpr int OFF_RING = OFF_P + 2 * P_BYTES;
  static constexpr int OFF_BAR = OFF_RING + NS * ITEM;
  // ring_full[NS], ring_empty[NS], s_full[2], p_full[2], pv_done[2], exchange[2], o_full, drain
  static constexpr int NBAR = 2 * NS + 8 + 2;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;             // TMEM address, abort flag
  static constexpr int OFF_ROW = (OFF_MISC + 8 + 15) / 16 * 16;   // inverse scale, end of the visible slots
  static constexpr int OFF_MAX = OFF_ROW + 8 * R;                 // [2][4][R] warp maxima
  static constexpr int OFF_SUM = OFF_MAX + 32 * R;                // [4][R] warp sums of l
  static constexpr int OFF_PAGES = OFF_SUM + 16 * R;              // per page: id, K scale, V scale, log2 V scale
  static constexpr int THREADS = 192;
  static constexpr int smem(int pages) { return OFF_PAGES + 16 * pages + 1024; }
  static_assert(NS >= 4 && Q_BYTES % 1024 == 0 && P_BYTES % 1024 == 0, "shared memory layout");
};

// Ring position of item `tile` of K or V in the order K0, K1, V0, K2, V1, ...
__device__ __forceinline__ int v_position(int j, int n) {
  const int first = n < 2 ? n : 2, pairs = n - first;
  return j < pairs ? first + 2 * j : first + pairs + j;
}
__device__ __forceinline__ void ring_item(int p, int n, bool& is_v, int& tile) {
  const int first = n < 2 ? n : 2, pairs = n - first;
  if (p < first) {
    is_v = false;
    tile = p;
  } else if (p - first < 2 * pairs) {
    is_v = ((p - first) & 1) == 0;
    tile = is_v ? (p - first) / 2 : (p - first) / 2 + 2;
  } else {
    is_v = true;
    tile = p - first - pairs;
  }
}

template <int D, int T, int R>
__global__ void __launch_bounds__(192, (PagedCfg<D, T, R>::ALONE ? 1 : 2))
    paged_attention_kernel(const __grid_constant__ PagedAttnArgs a) {
  using C = PagedCfg<D, T, R>;
  const int BH = a.c.B * a.c.Hkv;
  const int bh = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  const int b = bh / a.c.Hkv, h = bh % a.c.Hkv;
  const int row0 = blockIdx.y * R;
  const int nr = min(R, a.rows - row0);
  pdl_launch();
  int len = a.lens[b];
  if (len < 0 || len > a.max_len) {  // reported; the sequence counts as empty
    if (threadIdx.x == 0 && split == 0 && h == 0) atomicOr(a.status, kStatusBadSeqlens);
    len = 0;
  }
  const int kb = split * a.chunk;
  const int ke = min(len, kb + a.chunk);
  const int n = ke > kb ? (ke - kb + 127) / 128 : 0;
  const long long out_row = (long long)bh * a.rows + row0;
  if (n == 0) {
    if (a.splits == 1) {  // nothing to see: O = 0, LSE = -inf
      uint16_t* o = static_cast<uint16_t*>(a.o) + out_row * D;
      for (int e = threadIdx.x; e < nr * D; e += blockDim.x) o[e] = 0;
      for (int e = threadIdx.x; e < nr; e += blockDim.x) a.lse[out_row + e] = neg_inf();
    }
    return;  // the merge knows from the length which chunks there are
  }

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
  uint64_t* exchange = pv_done + 2;
  uint64_t* o_full = exchange + 2;
  uint64_t* drain = o_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  float* s_qinv = reinterpret_cast<float*>(smem + C::OFF_ROW);
  int* s_end = reinterpret_cast<int*>(smem + C::OFF_ROW) + R;
  float* s_max = reinterpret_cast<float*>(smem + C::OFF_MAX);
  float* s_sum = reinterpret_cast<float*>(smem + C::OFF_SUM);
  const int ps = a.c.ps, shift = a.c.ps_shift;
  const int ne = (ke - kb + ps - 1) >> shift;  // pages of this chunk
  int* s_page = reinterpret_cast<int*>(smem + C::OFF_PAGES);
  float* s_ks = reinterpret_cast<float*>(s_page + ne);
  float* s_vs = s_ks + ne;
  float* s_lv = s_vs + ne;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&ring_full[s], 1);
      mbar_init(&ring_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
      mbar_init(&exchange[i], 4);
    }
    mbar_init(o_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 4 && lane == 0) {
    tma_prefetch_desc(&a.tm_k);
    tma_prefetch_desc(&a.tm_v);
  }
  if (warp == 5) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  {
    const int* table = a.c.table + (long long)b * a.c.width + (kb >> shift);
    for (int i = threadIdx.x; i < ne; i += blockDim.x) {
      int id = table[i];
      float ks = 0.f, vs = 0.f;
      if (id < 0 || id >= a.c.pages) {
        atomicOr(a.status, kStatusBadPages);
        id = -1;
      } else {
        ks = a.c.k_scale[(long long)id * a.c.Hkv + h];
        vs = a.c.v_scale[(long long)id * a.c.Hkv + h];
      }
      s_page[i] = id;
      s_ks[i] = ks * a.scale_log2;
      s_vs[i] = vs;
      s_lv[i] = fmaxf(__log2f(fabsf(vs)), kMinLogScale);
    }
  }
  // Query rows to e4m3 terms: a warp a row, D / 32 elements a lane.
  for (int r = warp; r < R; r += C::THREADS / 32) {
    constexpr int E = D / 32;
    float x[E];
    float top = 0.f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = 0.f;
    if (r < nr) {
      const long long at = (out_row + r) * D + lane * E;
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const uint32_t two = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + at + i);
        if (a.bf16) {
          x[i] = __uint_as_float(two << 16);
          x[i + 1] = __uint_as_float(two & 0xffff0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
          x[i] = f.x;
          x[i + 1] = f.y;
        }
      }
#pragma unroll
      for (int i = 0; i < E; ++i) {
        finite = finite && isfinite(x[i]);
        top = fmaxf(top, fabsf(x[i]));
      }
    }
    finite = __all_sync(0xffffffffu, finite);
    top = warp_max(top);
    // 2^e with top * 2^e in [128, 256) (subnormal rows: at most 2^120)
    const int e = min(134 - static_cast<int>(__float_as_uint(top) >> 23), 120);
    const float up = __int_as_float((e + 127) << 23);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
      uint32_t code[T];
      split_terms<T>(finite ? x[i] * up : 0.f, finite ? x[i + 1] * up : 0.f, code);
      const int col = lane * E + i;
#pragma unroll
      for (int t = 0; t < T; ++t)
        *reinterpret_cast<uint16_t*>(sQ + (col / C::W) * (C::NB * C::W) + sw_offset<C::W>(t * R + r, col % C::W)) =
            static_cast<uint16_t>(code[t]);
    }
    if (lane == 0) {
      // a row that holds a NaN or an infinity has no softmax: its scores are NaN
      s_qinv[r] = finite ? __int_as_float((127 - e) << 23) : __int_as_float(0x7fc00000);
      s_end[r] = a.causal ? len - a.Nq + (row0 + r) % a.Nq + 1 : len;
    }
  }
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    const int per = 128 >> shift;  // pages a tile
    const int items = 2 * n * C::HALVES;
    int issued = 0;
    for (int p = 0; p < items; ++p) {
      const int slot = p % C::NS;
      if (!warp_wait(&ring_empty[slot], ((p / C::NS) & 1) ^ 1, abort_flag, a.status)) break;
      bool is_v;
      int t;
      ring_item(p / C::HALVES, n, is_v, t);
      const int half = p % C::HALVES;
      const int e = t * per + lane;
      const int id = lane < per && e < ne ? s_page[e] : -1;
      const unsigned there = __ballot_sync(0xffffffffu, id >= 0);
      if (lane == 0) mbar_arrive_expect_tx(&ring_full[slot], __popc(there) * ps * C::W);
      __syncwarp();
      if (id >= 0)
        tma_load_3d(sRing + slot * C::ITEM + lane * ps * C::W, is_v ? &a.tm_v : &a.tm_k, &ring_full[slot], half * 128,
                    0, id * a.c.Hkv + h);
      issued = p + 1;
    }
    if (*abort_flag && lane == 0)
      for (int p = issued - C::NS < 0 ? 0 : issued - C::NS; p < issued; ++p)
        drain_wait(&ring_full[p % C::NS], (uint32_t)((p / C::NS) & 1));
    __syncwarp();
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t id_s = idesc_f8(128, C::NB, a.c.e5m2, false);
      const uint32_t id_pv = idesc_f8(128, C::NB, a.c.e5m2, true);
      const uint32_t q = smem_u32(sQ), pw = smem_u32(sP), ring = smem_u32(sRing);
      constexpr int GROUP = 8 * C::W;  // eight rows: the stride of the swizzle pattern
      int p = 0;
      auto take = [&](int& slot) {
        slot = p % C::NS;
        const bool ok = mbar_wait(&ring_full[slot], (p / C::NS) & 1, abort_flag, a.status, kStatusTimeout);
        ++p;
        tc_fence_after();
        return ok;
      };
      // S buffer i: slots as rows (K-major A), query terms as columns
      auto issue_s = [&](int i) {
        for (int hf = 0; hf < C::HALVES; ++hf) {
          int slot;
          if (!take(slot)) return false;
          const uint64_t da = sdesc_w<C::W>(ring + slot * C::ITEM, 16, GROUP);
          const uint64_t db = sdesc_w<C::W>(q + hf * C::NB * C::W, 16, GROUP);
#pragma unroll
          for (int kk = 0; kk < C::W / 32; ++kk)
            mma_f8(tmem + C::COL_S + C::SCOL * i, sdesc_advance(da, 32 * kk), sdesc_advance(db, 32 * kk), id_s,
                   hf > 0 || kk > 0);
          mma_commit(&ring_empty[slot]);
        }
        mma_commit(&s_full[i]);
        return true;
      };
      bool ok = issue_s(0);
      if (ok && n > 1) ok = issue_s(1);
      for (int j = 0; ok && j < n; ++j) {
        const int i = j & 1;
        if (!(ok = mbar_wait(&p_full[i], (j >> 1) & 1, abort_flag, a.status, kStatusTimeout))) break;
        tc_fence_after();
        for (int hf = 0; hf < C::HALVES; ++hf) {
          int slot;
          if (!(ok = take(slot))) break;
          // features as rows (MN-major A: a row of memory is a slot); at
          // d = 64 both 64-feature halves of M = 128 read the same bytes
          // (offset 0 between them), lanes 64-127 repeat lanes 0-63
          const uint64_t da = sdesc_w<C::W>(ring + slot * C::ITEM, 0, GROUP);
          const uint64_t db = sdesc_w<128>(pw + i * C::P_BYTES, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f8(tmem + C::COL_O + C::SCOL * hf, sdesc_advance(da, 32 * C::W * kk), sdesc_advance(db, 32 * kk),
                   id_pv, j > 0 || kk > 0);
          mma_commit(&ring_empty[slot]);
        }
        if (!ok) break;
        mma_commit(&pv_done[i]);
        if (j + 2 < n) ok = issue_s(i);
      }
      if (ok) {
        mma_commit(o_full);
      } else {
        mma_commit(drain);
        drain_wait(drain, 0);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax, epilogue
    const int key = warp * 32 + lane;  // slot of the tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    float l[R], m[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l[r] = 0.f;
      m[r] = neg_inf();
    }
    // bytes of P: row t * R + r of 128 slots
    uint32_t p_at[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) p_at[r] = smem_u32(sP) + sw_offset<128>(r, key);
    const int first_end = a.causal ? len - a.Nq + 1 : len;  // the fewest slots that a row sees
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int i = j & 1;
      const uint32_t tS = lane_base + C::COL_S + C::SCOL * i;
      const int slot = kb + j * 128 + key;
      const int e = (j * 128 + key) >> shift;
      const bool live = slot < ke && s_page[e] >= 0;
      const float ks = live ? s_ks[e] : 0.f, vs = live ? s_vs[e] * kWeightScale : 0.f, lv = live ? s_lv[e] : 0.f;
      if (!(ok = warp_wait(&s_full[i], (j >> 1) & 1, abort_flag, a.status))) break;
      tc_fence_after();
      const bool cut = kb + j * 128 + 128 > first_end;  // some row sees less than the tile
      float s[R];
#pragma unroll
      for (int c = 0; c < R; c += 8) {
        float x[T][8];
#pragma unroll
        for (int t = 0; t < T; ++t) tmem_ld8(tS + t * R + c, x[t]);
#pragma unroll
        for (int t = 0; t < T; ++t) tmem_ld8_wait(x[t]);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          float y = x[T - 1][r];
#pragma unroll
          for (int t = T - 2; t >= 0; --t) y = fmaf(y, 0.0625f, x[t][r]);
          s[c + r] = y * s_qinv[c + r] * ks;
        }
      }
      if (cut || !live) {
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (!live || slot >= s_end[r]) s[r] = neg_inf();
      }
      if (a.scores != nullptr && slot < ke) {
        float* to = a.scores + out_row * a.score_stride + slot;
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (r < nr) to[r * a.score_stride] = s[r];
      }
      float* mine = s_max + (i * 4 + warp) * R;
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        float4 x;
        x.x = warp_max(s[r] + lv);
        x.y = warp_max(s[r + 1] + lv);
        x.z = warp_max(s[r + 2] + lv);
        x.w = warp_max(s[r + 3] + lv);
        if (lane == 0) *reinterpret_cast<float4*>(mine + r) = x;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&exchange[i]);
      if (!(ok = warp_wait(&exchange[i], (j >> 1) & 1, abort_flag, a.status))) break;
      // every thread derives the same new references from the four warps' maxima
      float corr[R];
      bool moved = false;
      const float* all = s_max + i * 4 * R;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float x = fmaxf(fmaxf(all[r], all[R + r]), fmaxf(all[2 * R + r], all[3 * R + r]));
        corr[r] = 1.f;
        if (x > m[r] + kMaxLead) {
          corr[r] = ex2_approx(m[r] - x);
          l[r] *= corr[r];
          m[r] = x;
          moved = true;
        }
      }
      if (moved && j > 0) {  // the same on every thread; PV(j - 1) may still add to O
        if (!(ok = warp_wait(&pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, abort_flag, a.status))) break;
        tc_fence_after();
#pragma unroll
        for (int hf = 0; hf < C::HALVES; ++hf)
#pragma unroll
          for (int t = 0; t < T; ++t)
#pragma unroll
            for (int c = 0; c < R; c += 8) {
              float x[8];
              const uint32_t at = lane_base + C::COL_O + C::SCOL * hf + t * R + c;
              tmem_ld8(at, x);
              tmem_ld8_wait(x);
              uint32_t y[8];
#pragma unroll
              for (int r = 0; r < 8; ++r) y[r] = __float_as_uint(x[r] * corr[c + r]);
              tmem_st8(at, y);
            }
        tmem_st_wait();
      }
      const uint32_t pbuf = i * C::P_BYTES;
#pragma unroll
      for (int r = 0; r < R; r += 2) {
        const float p0 = ex2_approx(s[r] - (m[r] == neg_inf() ? 0.f : m[r]));
        const float p1 = ex2_approx(s[r + 1] - (m[r + 1] == neg_inf() ? 0.f : m[r + 1]));
        l[r] += p0;
        l[r + 1] += p1;
        uint32_t code[T];
        split_terms<T>(p0 * vs, p1 * vs, code);
#pragma unroll
        for (int t = 0; t < T; ++t) {
          const uint32_t at = pbuf + (t * R + (r & ~7)) * 128;
          asm volatile("st.shared.u8 [%0], %1;" ::"r"(p_at[r & 7] + at), "r"(code[t] & 0xffu) : "memory");
          asm volatile("st.shared.u8 [%0], %1;" ::"r"(p_at[(r & 7) + 1] + at), "r"(code[t] >> 8) : "memory");
        }
      }
      if (!live) {  // no bytes of this slot may reach the product
        for (int hf = 0; hf < C::HALVES; ++hf) {
          const int p = v_position(j, n) * C::HALVES + hf;
          if (!mbar_wait(&ring_full[p % C::NS], (p / C::NS) & 1, abort_flag, a.status, kStatusTimeout)) ok = false;
          uint4* row = reinterpret_cast<uint4*>(sRing + (p % C::NS) * C::ITEM + key * C::W);
          if (ok)
            for (int x = 0; x < C::W / 16; ++x) row[x] = make_uint4(0, 0, 0, 0);
        }
      }
      fence_async_smem();
      tc_fence_before();
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      if (lane == 0) mbar_arrive(&p_full[i]);
    }
    // l over the 128 slots of a tile: lanes, then warps
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float x = warp_sum(l[r]);
      if (lane == 0) s_sum[warp * R + r] = x;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&exchange[n & 1]);
    if (ok) ok = warp_wait(&exchange[n & 1], (n >> 1) & 1, abort_flag, a.status);
    if (ok) ok = warp_wait(o_full, 0, abort_flag, a.status);
    if (ok) {
      tc_fence_after();
      const long long part = ((long long)split * BH * a.rows + out_row) * D;
#pragma unroll
      for (int c = 0; c < R; c += 8) {
        if (c >= nr) break;
        float inv[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float x = s_sum[c + r] + s_sum[R + c + r] + s_sum[2 * R + c + r] + s_sum[3 * R + c + r];
          inv[r] = x == 0.f ? 0.f : (1.f / kWeightScale) / x;
          if (threadIdx.x == 0 && c + r < nr) {
            const float lse2 = x == 0.f ? neg_inf() : (m[c + r] == neg_inf() ? 0.f : m[c + r]) + __log2f(x);
            if (a.splits == 1)
              a.lse[out_row + c + r] = lse2 * kLn2;
            else
              a.lse_part[(long long)split * BH * a.rows + out_row + c + r] = lse2;
          }
        }
#pragma unroll
        for (int hf = 0; hf < C::HALVES; ++hf) {
          float x[T][8];
#pragma unroll
          for (int t = 0; t < T; ++t) tmem_ld8(lane_base + C::COL_O + C::SCOL * hf + t * R + c, x[t]);
#pragma unroll
          for (int t = 0; t < T; ++t) tmem_ld8_wait(x[t]);
          const int f = hf * 128 + key;
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            float y = x[T - 1][r];
#pragma unroll
            for (int t = T - 2; t >= 0; --t) y = fmaf(y, 0.0625f, x[t][r]);
            y *= inv[r];
            if (c + r < nr && f < D) {
              if (a.splits != 1) {
                a.o_part[part + (long long)(c + r) * D + f] = y;
              } else if (a.bf16) {
                static_cast<__nv_bfloat16*>(a.o)[(out_row + c + r) * D + f] = __float2bfloat16_rn(y);
              } else {
                static_cast<__half*>(a.o)[(out_row + c + r) * D + f] = __float2half_rn(y);
              }
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Merges the chunks of a row: LSE = log2 sum 2^LSE_s, O = sum 2^(LSE_s - LSE) O_s,
// in the chunks' order (GROUPS of threads take every GROUPS-th chunk, then
// their sums are added in order).
template <int D>
__global__ void __launch_bounds__(256) paged_combine_kernel(const float* __restrict__ o_part,
                                                            const float* __restrict__ lse_part,
                                                            const int* __restrict__ lens, void* __restrict__ o,
                                                            float* __restrict__ lse, int rows_per_seq,
                                                            long long rows_all, int splits, int chunk, int max_len,
                                                            bool bf16) {
  constexpr int PER = D / 4, GROUPS = 256 / PER;
  __shared__ float s_w[1024];
  __shared__ float4 s_o[GROUPS][PER];
  __shared__ float s_red[8];
  const long long row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch();
  pdl_wait();
  int len = lens[row / rows_per_seq];
  if (len < 0 || len > max_len) len = 0;
  const int ns = (len + chunk - 1) / chunk;  // chunks that hold something
  float mx = neg_inf();
  for (int s = threadIdx.x; s < ns; s += 256) {
    const float x = lse_part[s * rows_all + row];
    s_w[s] = x;
    mx = fmaxf(mx, x);  // a NaN reaches the output through its weight
  }
  mx = warp_max(mx);
  if (lane == 0) s_red[warp] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) mx = fmaxf(mx, s_red[w]);
  const float ref = mx == neg_inf() ? 0.f : mx;
  const int g = threadIdx.x / PER, f = threadIdx.x % PER;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll 4
  for (int s = g; s < ns; s += GROUPS) {
    const float w = exp2f(s_w[s] - ref);
    const float4 x = *reinterpret_cast<const float4*>(o_part + (s * rows_all + row) * D + 4 * f);
    sum += w;
    if (w != 0.f) {
      acc.x = fmaf(w, x.x, acc.x);
      acc.y = fmaf(w, x.y, acc.y);
      acc.z = fmaf(w, x.z, acc.z);
      acc.w = fmaf(w, x.w, acc.w);
    }
  }
  s_o[g][f] = acc;
  __syncthreads();
  if (f == 0) s_w[g] = sum;  // the weights are no longer needed
  __syncthreads();
  if (g == 0) {
    float l = 0.f;
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) l += s_w[k];
#pragma unroll
    for (int k = 1; k < GROUPS; ++k) {
      const float4 x = s_o[k][f];
      acc.x += x.x;
      acc.y += x.y;
      acc.z += x.z;
      acc.w += x.w;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint2 two;
    if (bf16) {
      __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
      __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
      two = make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
    } else {
      __half2 lo = __floats2half2_rn(acc.x * inv, acc.y * inv);
      __half2 hi = __floats2half2_rn(acc.z * inv, acc.w * inv);
      two = make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
    }
    reinterpret_cast<uint2*>(o)[row * PER + f] = two;
    if (f == 0) lse[row] = l == 0.f ? neg_inf() : (ref + __log2f(l)) * kLn2;
  }
}

// weight_acc[slot] += sum over the rows of 2^(score - LSE), in the rows'
// order: four slots a thread.
__global__ void __launch_bounds__(256) paged_weights_kernel(const float* __restrict__ scores,
                                                            const float* __restrict__ lse,
                                                            const int* __restrict__ lens,
                                                            float* __restrict__ weight_acc, int Hkv, int rows,
                                                            long long score_stride, long long acc_stride,
                                                            int max_len) {
  const int bh = blockIdx.y;
  const int slot = (blockIdx.x * 256 + threadIdx.x) * 4;
  pdl_wait();
  const int len = lens[bh / Hkv];
  if (len > max_len || slot >= len) return;
  const float* from = scores + (long long)bh * rows * score_stride + slot;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int r = 0; r < rows; ++r) {
    const float z = lse[(long long)bh * rows + r] * kLog2e;
    const float4 x = *reinterpret_cast<const float4*>(from + r * score_stride);
    if (z == neg_inf()) continue;  // the row sees nothing
    sum[0] += exp2f(x.x - z);
    sum[1] += exp2f(x.y - z);
    sum[2] += exp2f(x.z - z);
    sum[3] += exp2f(x.w - z);
  }
  float* to = weight_acc + (long long)bh * acc_stride + slot;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (slot + k < len) to[k] += sum[k];
}

template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

template <int D, int T, int R>
cudaError_t launch_attention_t(const PagedAttnArgs& a, cudaStream_t stream) {
  using C = PagedCfg<D, T, R>;
  auto kern = paged_attention_kernel<D, T, R>;
  const int smem = C::smem((a.chunk + a.c.ps - 1) / a.c.ps);
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             C::smem(kPagedMaxPagesPerChunk));
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(a.c.B * a.c.Hkv) * (unsigned)a.splits, (unsigned)((a.rows + R - 1) / R));
  kern<<<grid, C::THREADS, smem, stream>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const PagedAttnArgs& a, cudaStream_t stream) {
  const int r = paged_row_tile(a.rows);
  cudaError_t e;
  if (a.bf16)
    e = r == 8    ? launch_attention_t<D, 2, 8>(a, stream)
        : r == 16 ? launch_attention_t<D, 2, 16>(a, stream)
                  : launch_attention_t<D, 2, 32>(a, stream);
  else
    e = r == 8    ? launch_attention_t<D, 3, 8>(a, stream)
        : r == 16 ? launch_attention_t<D, 3, 16>(a, stream)
                  : launch_attention_t<D, 3, 32>(a, stream);
  if (e != cudaSuccess) return e;
  const int BH = a.c.B * a.c.Hkv;
  const long long rows_all = (long long)BH * a.rows;
  if (a.splits > 1) {
    e = launch_pdl(paged_combine_kernel<D>, dim3((unsigned)rows_all), dim3(256), stream, a.o_part, a.lse_part, a.lens,
                   a.o, a.lse, a.c.Hkv * a.rows, rows_all, a.splits, a.chunk, a.max_len, a.bf16);
    if (e != cudaSuccess) return e;
  }
  if (a.weight_acc != nullptr)
    e = launch_pdl(paged_weights_kernel, dim3((unsigned)((a.max_len + 1023) / 1024), (unsigned)BH), dim3(256), stream,
                   a.scores, a.lse, a.lens, a.weight_acc, a.c.Hkv, a.rows, a.score_stride,
                   (long long)a.c.width * a.c.ps, a.max_len);
  return e;
}

}  // namespace

int paged_row_tile(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }

void paged_plan(int BH, int rows, int ps, int max_len, int num_splits, int* splits, int* chunk) {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int r = paged_row_tile(rows);
  const long long resident = 2LL * sms;
  const long long units = (long long)BH * ((rows + r - 1) / r);
  const int tiles = (max_len + 127) / 128;
  const int most = kPagedMaxPagesPerChunk * ps;
  const int most_tiles = (most < kPagedMaxChunk ? most : kPagedMaxChunk) / 128;
  int best_per = 1;
  if (num_splits > 0) {
    best_per = (tiles + num_splits - 1) / num_splits;
  } else {
    // waves of CTAs, each as long as its tiles and about three more for its
    // start and end; several chunks cost the merge's launch, about four
    double best = 1e300;
    const int most_splits = tiles < 1024 ? tiles : 1024;
    for (int s = 1; s <= most_splits; ++s) {
      const int per = (tiles + s - 1) / s;
      if (per > most_tiles) continue;
      const int got = (tiles + per - 1) / per;
      const double waves = (double)((units * got + resident - 1) / resident);
      const double cost = waves * (per + 3.0) + (got > 1 ? 4.0 : 0.0) + 0.02 * got;
      if (cost < best) {
        best = cost;
        best_per = per;
      }
    }
  }
  if (best_per > most_tiles) best_per = most_tiles;
  if (best_per < 1) best_per = 1;
  *chunk = best_per * 128;
  *splits = (tiles + best_per - 1) / best_per;
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a, cudaStream_t stream) {
  if (a.c.d == 64) return launch_d<64>(a, stream);
  if (a.c.d == 128) return launch_d<128>(a, stream);
  if (a.c.d == 256) return launch_d<256>(a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fa
