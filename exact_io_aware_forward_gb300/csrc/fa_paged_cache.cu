// Writing to the 8-bit paged K/V cache: appending tokens, and evicting the
// slots with the smallest accumulated attention weight.
//
// Codes are e4m3 or e5m2; a page has one float32 scale a head for K and one
// for V, and code c stands for c * scale.  A scale that append chooses is the
// smallest power of two s with max |x| <= (largest code) * s (at least
// 2^-100): both types' largest code is 7/8 of a power of two, x / s is exact,
// and the type's relative precision is the same at every scale, so that
// another scale would only move the subnormal range.  A page's scale grows
// when larger values arrive; its codes are then rounded again to
// c * (s_old / s_new), exact for powers of two except where a code becomes
// subnormal.  A scale never shrinks while the page holds older slots.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>

#include "fa_paged.h"
#include "fa_pdl.cuh"

namespace fa {
namespace {

// Two codes (a in the low byte) to floats and back, rounding to nearest even.
template <bool E5M2>
__device__ __forceinline__ float2 from_codes(uint32_t two) {
  uint32_t h;
  if (E5M2)
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  else
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
template <bool E5M2>
__device__ __forceinline__ uint32_t to_codes(float a, float b) {
  uint16_t r;
  if (E5M2)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  uint32_t c = r;
  // satfinite hides infinities: e5m2 has a code for them, e4m3 only a NaN
  if (isinf(a)) c = (c & 0xff00u) | (E5M2 ? (a < 0.f ? 0xfcu : 0x7cu) : 0x7fu);
  if (isinf(b)) c = (c & 0x00ffu) | ((E5M2 ? (b < 0.f ? 0xfcu : 0x7cu) : 0x7fu) << 8);
  return c;
}

// to_codes for numbers within the type's range, and NaN.
template <bool E5M2>
__device__ __forceinline__ uint32_t to_codes_finite(float a, float b) {
  uint16_t r;
  if (E5M2)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// Four codes times `ratio` (at most 1), rounded again.
template <bool E5M2>
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float ratio) {
  const float2 a = from_codes<E5M2>(c & 0xffffu), b = from_codes<E5M2>(c >> 16);
  if (E5M2 && __vcmpeq4(c & 0x7f7f7f7fu, 0x7c7c7c7cu))  // an infinity
    return to_codes<E5M2>(a.x * ratio, a.y * ratio) | (to_codes<E5M2>(b.x * ratio, b.y * ratio) << 16);
  return to_codes_finite<E5M2>(a.x * ratio, a.y * ratio) | (to_codes_finite<E5M2>(b.x * ratio, b.y * ratio) << 16);
}
template <bool E5M2>
__device__ __forceinline__ uint4 rescale16(uint4 c, float ratio) {
  return make_uint4(rescale4<E5M2>(c.x, ratio), rescale4<E5M2>(c.y, ratio), rescale4<E5M2>(c.z, ratio),
                    rescale4<E5M2>(c.w, ratio));
}

__device__ __forceinline__ float2 unpack16(uint32_t v, bool bf16) {
  if (bf16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}

// The smallest power of two s >= 2^-100 with amax <= (7/8 * 2^top) * s.
template <bool E5M2>
__device__ __forceinline__ float scale_for(float amax) {
  constexpr int top = E5M2 ? 16 : 9;  // 57344 and 448
  const uint32_t bits = __float_as_uint(amax);
  // amax = 1.f * 2^(field - 127) = 0.1f * 2^(field - 126); subnormals land below the clamp
  int e = static_cast<int>(bits >> 23) - 126 - top + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, -100);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// ---------------------------------------------------------------- append
// One CTA (or, WARP, one warp: pages with at most 2048 new elements, eight to
// a CTA) a (sequence, page, head, K or V): the page's new rows are read
// once (16 elements a thread and step, kept in registers), their maximum
// gives the scale, and they are written as codes.  Reads 2 and writes 1
// byte an element.  A prompt is bound by memory as long as an element costs
// few instructions: the maximum is taken on the 16-bit patterns, two at a
// time, and infinities and NaN are looked at one by one only in pages that
// have some (8192 tokens for 4 x 8 heads: 46 us with every element looked at).
// One token a sequence is bound by the launch and three dependent reads.
template <bool E5M2, int NV, bool WARP>
__global__ void __launch_bounds__(256) paged_append_kernel(const __grid_constant__ PagedAppendArgs a, int reach) {
  pdl_launch();
  pdl_wait();
  int x, y, b;  // page among those that may be reached, head and K or V, sequence
  if (WARP) {
    const long long item = blockIdx.x * 8LL + (threadIdx.x >> 5);
    x = (int)(item % reach);
    const long long rest = item / reach;
    if (rest >= 2LL * a.c.Hkv * a.c.B) return;
    y = (int)(rest % (2 * a.c.Hkv));
    b = (int)(rest / (2 * a.c.Hkv));
  } else {
    x = blockIdx.x, y = blockIdx.y, b = blockIdx.z;
  }
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, threads = WARP ? 32 : blockDim.x;
  const int h = y >> 1;
  const bool is_v = y & 1;
  const int ps = a.c.ps, d = a.c.d;
  const int len = a.lens[b];
  const int cnt = a.counts ? a.counts[b] : a.N;
  const bool first = x == 0 && y == 0;
  if (len < 0 || cnt < 0 || cnt > a.N || len > a.c.width * ps || cnt > a.c.width * ps - len) {
    if (first && tid == 0) {
      atomicOr(a.status, kStatusBadSeqlens);
      a.new_lens[b] = len;
    }
    return;
  }
  if (first && tid == 0) a.new_lens[b] = len + cnt;
  const int t = (len >> a.c.ps_shift) + x;
  const int start = t * ps;
  const int lo = max(len, start), hi = min(len + cnt, start + ps);
  if (lo >= hi) return;
  const int page = a.c.table[(long long)b * a.c.width + t];
  const uint16_t* from = static_cast<const uint16_t*>(is_v ? a.v : a.k) +
                      (((long long)b * a.c.Hkv + h) * a.N + (lo - len)) * d;
  const int vecs = (hi - lo) * d / 16;
  uint4 in[NV][2];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = i * threads + tid;
    if (e < vecs) {
      in[i][0] = __ldcs(reinterpret_cast<const uint4*>(from) + 2 * e);
      in[i][1] = __ldcs(reinterpret_cast<const uint4*>(from) + 2 * e + 1);
    } else {
      in[i][0] = in[i][1] = make_uint4(0, 0, 0, 0);
    }
  }
  const long long state = ((long long)b * a.c.Hkv + h) * a.c.width * ps;
  if (!is_v) {  // bookkeeping of the new slots
    for (int s = lo + tid; s < hi; s += threads) {
      if (a.weight_acc) a.weight_acc[state + s] = 0.f;
      if (a.positions) a.positions[state + s] = (a.first_position ? a.first_position[b] : len) + (s - len);
    }
  }
  if (page < 0 || page >= a.c.pages) {
    if (tid == 0) atomicOr(a.status, kStatusBadPages);
    return;
  }
  float* scale = (is_v ? a.c.v_scale : a.c.k_scale) + (long long)page * a.c.Hkv + h;
  const float was = lo > start ? *scale : 0.f;  // read by every thread before it is written
  auto word = [&](int i, int w) {
    const uint4& u = in[i][w >> 2];
    return (w & 3) == 0 ? u.x : (w & 3) == 1 ? u.y : (w & 3) == 2 ? u.z : u.w;
  };
  // the largest magnitude as a 16-bit pattern
  const uint32_t inf16 = a.bf16 ? 0x7f80u : 0x7c00u;
  uint32_t two = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int w = 0; w < 8; ++w) two = __vmaxu2(two, word(i, w) & 0x7fff7fffu);
  __shared__ uint32_t s_top[2][8];
  auto most = [&](uint32_t mine, int turn) {
    mine = __reduce_max_sync(0xffffffffu, mine);
    if (WARP) return mine;
    if ((tid & 31) == 0) s_top[turn][tid >> 5] = mine;
    __syncthreads();
    for (int w = 0; w < (int)(threads >> 5); ++w) mine = max(mine, s_top[turn][w]);
    return mine;
  };
  uint32_t top = most(max(two & 0xffffu, two >> 16), 0);
  const bool all_finite = top < inf16;
  if (!all_finite) {  // infinities and NaN do not set the scale
    uint32_t fin = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const uint32_t m = word(i, w) & 0x7fff7fffu;
        if ((m & 0xffffu) < inf16) fin = max(fin, m & 0xffffu);
        if ((m >> 16) < inf16) fin = max(fin, m >> 16);
      }
    top = most(fin, 1);
  }
  const float now = fmaxf(was, scale_for<E5M2>(unpack16(top, a.bf16).x));
  uint8_t* codes = (is_v ? a.c.v_pages : a.c.k_pages) + ((long long)page * a.c.Hkv + h) * ps * d;
  if (lo > start && now != was) {  // the slots that were there, at the larger scale
    const float ratio = was / now;
    uint4* old = reinterpret_cast<uint4*>(codes);
    for (int e = tid; e < (lo - start) * d / 16; e += threads) old[e] = rescale16<E5M2>(old[e], ratio);
  }
  // x / now; for a power of two the product with its inverse is the same number
  const bool power = (__float_as_uint(now) & 0x7fffffu) == 0 && now >= 0x1p-126f && now <= 0x1p126f;
  const float inv = power ? 1.f / now : 0.f;
  const bool plain = power && all_finite;
  uint4* out = reinterpret_cast<uint4*>(codes + (long long)(lo - start) * d);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = i * threads + tid;
    if (e >= vecs) break;
    uint32_t half[8];
    if (plain) {
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const float2 f = unpack16(word(i, w), a.bf16);
        half[w] = to_codes_finite<E5M2>(f.x * inv, f.y * inv);
      }
    } else {
#pragma unroll 1
      for (int w = 0; w < 8; ++w) {
        const float2 f = unpack16(word(i, w), a.bf16);
        const uint32_t c = power ? to_codes<E5M2>(f.x * inv, f.y * inv) : to_codes<E5M2>(f.x / now, f.y / now);
#pragma unroll
        for (int z = 0; z < 8; ++z) half[z] = z == w ? c : half[z];
      }
    }
    out[e] = make_uint4(half[0] | half[1] << 16, half[2] | half[3] << 16, half[4] | half[5] << 16,
                        half[6] | half[7] << 16);
  }
  if (WARP) __syncwarp();
  if (tid == 0 && now != was) *scale = now;
}

template <bool E5M2>
cudaError_t launch_append_t(const PagedAppendArgs& a, cudaStream_t stream) {
  // pages that N tokens can reach, wherever the first of them lands
  const int reach = (int)((a.N + a.c.ps - 2LL) / a.c.ps + 1);
  const long long items = 2LL * reach * a.c.Hkv * a.c.B;
  if ((a.N < a.c.ps ? a.N : a.c.ps) * a.c.d <= 2048 && items <= 8LL * 0x7fffffff)
    return launch_pdl(paged_append_kernel<E5M2, 4, true>, dim3((unsigned)((items + 7) / 8)), dim3(256), 0, stream, a,
                      reach);
  const int vecs = a.c.ps * a.c.d / 16;  // of a full page: 64 to 2048
  const int threads = vecs < 256 ? vecs : 256;
  const dim3 grid((unsigned)reach, (unsigned)(2 * a.c.Hkv), (unsigned)a.c.B);
  switch (vecs / threads) {
    case 1: return launch_pdl(paged_append_kernel<E5M2, 1, false>, grid, dim3(threads), 0, stream, a, reach);
    case 2: return launch_pdl(paged_append_kernel<E5M2, 2, false>, grid, dim3(threads), 0, stream, a, reach);
    case 4: return launch_pdl(paged_append_kernel<E5M2, 4, false>, grid, dim3(threads), 0, stream, a, reach);
    case 8: return launch_pdl(paged_append_kernel<E5M2, 8, false>, grid, dim3(threads), 0, stream, a, reach);
    default: return cudaErrorInvalidValue;
  }
}

// ---------------------------------------------------------------- evict

constexpr int kSelectKeys = 20;  // sort keys a thread holds in registers

// Order of the slots as unsigned numbers: protected ones first, then NaN,
// then the weights from large to small (-0 counts as 0).
__device__ __forceinline__ uint32_t rank_key(float weight, int position, int latest, int recent) {
  if ((long long)position > (long long)latest - recent) return 0xffffffffu;
  if (weight != weight) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(weight + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Writes v to the same place of another CTA's shared memory.
__device__ __forceinline__ void store_remote(const void* mine, uint32_t rank, int v) {
  uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(mine)), there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(there), "r"(v) : "memory");
}

__device__ __forceinline__ int load_remote(const void* mine, uint32_t rank) {
  uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(mine)), there;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(there) : "memory");
  return v;
}
template <int C>
__device__ __forceinline__ void all_sync() {
  if (C > 1)
    cluster_sync();
  else
    __syncthreads();
}

struct Pair {
  int a, b;
};
// Exclusive prefix sums of two numbers over all threads of the C CTAs of a
// cluster (TH threads each), in order, and their totals.  s_warp: 32 pairs; s_cta:
// 8 pairs, used for one call only.
template <int C, int TH>
__device__ __forceinline__ Pair sum_before(Pair v, int (*s_warp)[2], int (*s_cta)[2], Pair* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int x = v.a, y = v.b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int p = __shfl_up_sync(0xffffffffu, x, o), q = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) x += p, y += q;
  }
  __syncthreads();  // the list may still be read from the call before
  if (lane == 31) s_warp[warp][0] = x, s_warp[warp][1] = y;
  __syncthreads();
  const int wa = lane < TH / 32 ? s_warp[lane][0] : 0, wb = lane < TH / 32 ? s_warp[lane][1] : 0;
  Pair r, all;
  r.a = x - v.a + __reduce_add_sync(0xffffffffu, lane < warp ? wa : 0);
  r.b = y - v.b + __reduce_add_sync(0xffffffffu, lane < warp ? wb : 0);
  all.a = __reduce_add_sync(0xffffffffu, wa);
  all.b = __reduce_add_sync(0xffffffffu, wb);
  if (C > 1) {
    const int rank = (int)cluster_rank();
    if (threadIdx.x < 2 * C)
      store_remote(s_cta[rank] + (threadIdx.x & 1), threadIdx.x >> 1, threadIdx.x & 1 ? all.b : all.a);
    cluster_sync();
    all.a = all.b = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (c < rank) r.a += s_cta[c][0], r.b += s_cta[c][1];
      all.a += s_cta[c][0];
      all.b += s_cta[c][1];
    }
  }
  *total = all;
  return r;
}

// One cluster of C CTAs a (sequence, head): which slots leave, and which of the
// kept ones move where.  A thread owns a run of consecutive slots, its keys
// in registers (up to 20; longer runs are read again in every pass).
//
// The m-th largest key lies in a window [lo, hi], at first from the smallest
// to the largest key that is not protected.  A pass sorts the window's keys
// into 256 bins of equal width, adds the bins up from the top, and the bin
// where the sum reaches m is the next window: at most four passes, fewer where
// a window's keys all stay.  The bins are integers: no order of additions
// changes them.  (Finding the key two bits at a time by counting took up to 16
// passes: 23 us for 64 heads of 16384 slots, 10.5 us for 256 heads of 2080.)
// Equal keys: the lowest slots stay.  Prefix sums over the runs then give every
// hole and every mover its place in slot order.  Reads 8 bytes a slot.
template <int C, int TH>
__global__ void __launch_bounds__(TH) paged_select_kernel(const __grid_constant__ PagedEvictArgs a) {
  constexpr int K = kSelectKeys;
  __shared__ int s_bin[2][256];  // two passes' turns
  __shared__ unsigned s_red[32][4];
  __shared__ unsigned s_cta[8][4];
  __shared__ int s_warp[32][2], s_before[2][8][2];
  __shared__ int s_pick[2][3];
  const int bh = blockIdx.x / C, b = bh / a.c.Hkv, h = bh % a.c.Hkv;
  const int rank = C > 1 ? (int)cluster_rank() : 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, ps = a.c.ps;
  const bool speaks = rank == 0 && tid == 0;
  pdl_launch();
  if (tid < 256) s_bin[0][tid] = s_bin[1][tid] = 0;
  pdl_wait();
  const int n = a.lens[b];
  if (n < 0 || n > a.c.width * ps || n <= a.keep) {  // the same for the whole cluster
    if (speaks) {
      if (h == 0) {
        if (n < 0 || n > a.c.width * ps) atomicOr(a.status, kStatusBadSeqlens);
        a.new_lens[b] = n;
      }
      a.plan_count[bh] = 0;
    }
    return;
  }
  const int m = a.keep;
  const int* table = a.c.table + (long long)b * a.c.width;
  const long long state = (long long)bh * a.c.width * ps;
  const float* weight = a.weight_acc + state;
  const int* position = a.positions + state;
  // runs of a multiple of four slots
  const int run = (int)(((n + TH * C - 1LL) / (TH * C) + 3) & ~3LL);
  const long long begin = (long long)(rank * TH + tid) * run;
  const int s0 = (int)(begin < n ? begin : n), s1 = (int)(s0 + (long long)run < n ? s0 + run : n);
  const bool cached = run <= K;

  // four slots' weights and positions (0 and the lowest number where there is none)
  auto load4 = [&](int s, float (&w)[4], int (&p)[4]) {
    if (s + 4 <= s1) {
      const float4 x = *reinterpret_cast<const float4*>(weight + s);
      const int4 y = *reinterpret_cast<const int4*>(position + s);
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
      p[0] = y.x, p[1] = y.y, p[2] = y.z, p[3] = y.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        w[k] = s + k < s1 ? weight[s + k] : 0.f;
        p[k] = s + k < s1 ? position[s + k] : INT_MIN;
      }
    }
  };
  // the largest position, and whether a page is bad
  int latest = INT_MIN, bad = 0;
  for (int s = s0; s < s1; s += 4) {
    float w[4];
    int p[4];
    load4(s, w, p);
    latest = max(max(latest, max(p[0], p[1])), max(p[2], p[3]));
  }
  for (int t = rank * TH + tid; t < (n + ps - 1) / ps; t += TH * C)
    bad |= table[t] < 0 || table[t] >= a.c.pages;
  latest = __reduce_max_sync(0xffffffffu, latest);
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) s_red[warp][0] = (unsigned)latest, s_red[warp][1] = bad;
  __syncthreads();
  latest = __reduce_max_sync(0xffffffffu, (int)s_red[lane & (TH / 32 - 1)][0]);
  bad = __any_sync(0xffffffffu, s_red[lane & (TH / 32 - 1)][1]);
  if (C > 1) {
    cluster_sync();  // all CTAs of the cluster are there
    if (tid < 2 * C) store_remote(&s_cta[rank][tid & 1], tid >> 1, tid & 1 ? bad : latest);
    cluster_sync();
#pragma unroll
    for (int r = 0; r < C; ++r) {
      latest = max(latest, (int)s_cta[r][0]);
      bad |= (int)s_cta[r][1];
    }
  }
  if (bad) {  // reported; the sequence stays as it is (every head sees the same row)
    if (speaks) {
      if (h == 0) {
        atomicOr(a.status, kStatusBadPages);
        a.new_lens[b] = n;
      }
      a.plan_count[bh] = 0;
    }
    if (C > 1) cluster_sync();  // no CTA leaves while another may still write to its shared memory
    return;
  }
  uint32_t key[K];
#pragma unroll
  for (int i = 0; i < K; i += 4) {
    key[i] = key[i + 1] = key[i + 2] = key[i + 3] = 0u;
    if (cached && i < run) {
      float w[4];
      int p[4];
      load4(s0 + i, w, p);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (s0 + i + k < s1) key[i + k] = rank_key(w[k], p[k], latest, a.recent);
    }
  }
  auto key_at = [&](int s) { return rank_key(weight[s], position[s], latest, a.recent); };
  // f(key, slot) for every slot of the run
  auto each = [&](auto f) {
    if (cached) {
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (i < run && s0 + i < s1) f(key[i], s0 + i);
    } else {
      for (int s = s0; s < s1; ++s) f(key_at(s), s);
    }
  };

  // the smallest key, the largest that is not protected, the protected ones
  uint32_t lo = 0xffffffffu, hi = 0;
  unsigned shielded = 0;
  each([&](uint32_t k, int) {
    lo = min(lo, k);
    if (k != 0xffffffffu) hi = max(hi, k);
    else ++shielded;
  });
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  shielded = __reduce_add_sync(0xffffffffu, shielded);
  __syncthreads();  // s_red has been read
  if (lane == 0) s_red[warp][0] = lo, s_red[warp][1] = hi, s_red[warp][2] = shielded;
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, s_red[lane & (TH / 32 - 1)][0]);
  hi = __reduce_max_sync(0xffffffffu, s_red[lane & (TH / 32 - 1)][1]);
  shielded = __reduce_add_sync(0xffffffffu, lane < TH / 32 ? s_red[lane][2] : 0u);
  if (C > 1) {
    cluster_sync();  // s_cta has been read
    if (tid < 3 * C) {
      const int i = tid % 3;
      store_remote(&s_cta[rank][i], tid / 3, (int)(i == 0 ? lo : i == 1 ? hi : shielded));
    }
    cluster_sync();
    shielded = 0;
#pragma unroll
    for (int r = 0; r < C; ++r) {
      lo = min(lo, s_cta[r][0]);
      hi = max(hi, s_cta[r][1]);
      shielded += s_cta[r][2];
    }
  }
  int above = (int)shielded, in = n - above;  // keys over the window, and in it
  if (above >= m) lo = hi = 0xffffffffu, in = above, above = 0;
  // each pass leaves at most 2^shift keys' width, shift <= 24, 16, 8, 0: four are enough
  for (int pass = 0; pass < 4 && in != m - above && lo != hi; ++pass) {
    const int turn = pass & 1;
    const int shift = max(0, 24 - __clz(hi - lo));  // at most 256 bins
    int* bin = s_bin[turn];
    each([&](uint32_t k, int) {
      if (k >= lo && k <= hi) {
        const uint32_t at = (k - lo) >> shift;
        // many equal weights: one addition for all lanes that are here
        const unsigned lanes = __activemask();
        int same;
        __match_all_sync(lanes, at, &same);
        if (!same) atomicAdd(bin + at, 1);
        else if ((threadIdx.x & 31) == (unsigned)(__ffs(lanes) - 1)) atomicAdd(bin + at, __popc(lanes));
      }
    });
    all_sync<C>();
    // sums from the top, a bin a thread
    int mine = 0, sum = 0;
    if (tid < 256) {
      mine = bin[tid];
      if (C > 1) {
        mine = 0;
#pragma unroll
        for (int r = 0; r < C; ++r) mine += load_remote(bin + tid, r);
      }
      sum = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_down_sync(0xffffffffu, sum, o);
        if (lane + o < 32) sum += y;
      }
      if (lane == 0) s_warp[warp][0] = sum;
    }
    __syncthreads();
    if (tid < 256) {
      for (int w = warp + 1; w < 8; ++w) sum += s_warp[w][0];
      if (sum >= m - above && sum - mine < m - above) {
        s_pick[turn][0] = tid;
        s_pick[turn][1] = sum - mine;
        s_pick[turn][2] = mine;
      }
      s_bin[turn ^ 1][tid] = 0;  // the other turn's bins have been read by all CTAs before this pass's all_sync
    }
    __syncthreads();
    lo += (uint32_t)s_pick[turn][0] << shift;
    hi = lo + min(hi - lo, (1u << shift) - 1u);  // lo + 2^shift may pass 2^32 (NaN's key is near it)
    above += s_pick[turn][1];
    in = s_pick[turn][2];
  }
  // Of the window's keys all stay, or (equal ones) the first m - above.
  const int stay = in == m - above ? INT_MAX : m - above;
  int eq = 0;
  if (stay != INT_MAX) {
    Pair mine = {0, 0}, all;
    each([&](uint32_t k, int) { mine.a += k == lo; });
    eq = sum_before<C, TH>(mine, s_warp, s_before[0], &all).a;
  }
  auto kept = [&](uint32_t k, int& e) {
    const bool yes = k > lo || (k == lo && e < stay);
    e += k == lo;
    return yes;
  };
  Pair mine = {0, 0}, all;
  {
    int e = eq;
    each([&](uint32_t k, int s) {
      const bool yes = kept(k, e);
      mine.a += !yes && s < m;
      mine.b += yes && s >= m;
    });
  }
  const Pair from = sum_before<C, TH>(mine, s_warp, s_before[1], &all);
  const long long list = (long long)bh * m;
  const int pages = (m + ps - 1) / ps;
  int* page_holes = a.page_holes + (long long)bh * (pages + 1);  // holes before each page
  int hole_at = from.a, mover_at = from.b;
  each([&](uint32_t k, int s) {
    const bool yes = kept(k, eq);
    if (s < m && (s & (ps - 1)) == 0) page_holes[s >> a.c.ps_shift] = hole_at;
    if (!yes && s < m) a.holes[list + hole_at++] = s;
    if (yes && s >= m) a.movers[list + mover_at++] = s;
  });
  if (speaks) {
    page_holes[pages] = all.a;
    a.plan_count[bh] = all.a;
    if (h == 0) a.new_lens[b] = m;
    if (m & (ps - 1)) {  // the moving kernel may change the scales of the page where the kept part ends
      const long long at = (long long)table[pages - 1] * a.c.Hkv + h;
      a.edge_scales[bh] = make_float2(a.c.k_scale[at], a.c.v_scale[at]);
    }
  }
  if (C > 1) cluster_sync();  // no CTA leaves while another may still use its shared memory
}

// One warp a (page before the new length, sequence and head): the movers that
// go into the page's holes, the page's slots that stay, at one scale.  A
// mover's own page may be the page where the kept part ends and be rewritten
// at the same time by its own warp: its rows behind the new length are not
// touched there, and its scales were noted by the kernel before.  The chain of
// dependent reads (list, table, codes) is what it waits for, so pages go to
// warps, not CTAs, and each keeps several rows under way.
constexpr int kMoveWarps = 8;
template <bool E5M2>
__global__ void __launch_bounds__(32 * kMoveWarps, 4) paged_move_kernel(const __grid_constant__ PagedEvictArgs a) {
  struct List {
    long long src[128];  // a mover's row in the pool, in elements
    float k[128], v[128];
    int to[128];  // its row in the page
    uint32_t hole[4];
  };
  __shared__ List lists[kMoveWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bh = blockIdx.y, b = bh / a.c.Hkv, h = bh % a.c.Hkv;
  const int ps = a.c.ps, d = a.c.d;
  const int m = a.keep;  // a sequence that loses slots keeps exactly `keep`
  const int pages = (m + ps - 1) / ps, t = blockIdx.x * kMoveWarps + warp;
  pdl_launch();
  pdl_wait();
  if (t >= pages) return;
  List& x = lists[warp];
  const int* table = a.c.table + (long long)b * a.c.width;
  const int* page_holes = a.page_holes + (long long)bh * (pages + 1) + t;
  const int lo = page_holes[0], cnt = page_holes[1] - lo;
  const int page = table[t];
  // nothing leaves, or the sequence was reported (the lists are not set then); no hole in this page
  if (a.plan_count[bh] == 0 || cnt == 0) return;
  const int start = t * ps, rows = min(m, start + ps) - start;
  const long long list = (long long)bh * m + lo;
  const long long state = (long long)bh * a.c.width * ps;
  const long long own_scale = (long long)page * a.c.Hkv + h;
  const bool stays = rows > cnt;  // slots of the page that stay
  const float k_was = a.c.k_scale[own_scale], v_was = a.c.v_scale[own_scale];
  if (lane < 4) x.hole[lane] = 0;
  __syncwarp();
  float k_now = stays ? k_was : 0.f, v_now = stays ? v_was : 0.f;
  for (int i = lane; i < cnt; i += 32) {
    const int to = a.holes[list + i], from = a.movers[list + i];
    const long long at = (long long)table[from >> a.c.ps_shift] * a.c.Hkv + h;
    const float2 s = from >> a.c.ps_shift == pages - 1 ? a.edge_scales[bh] : make_float2(a.c.k_scale[at], a.c.v_scale[at]);
    x.to[i] = to - start;
    x.src[i] = (at * ps + (from & (ps - 1))) * d;
    x.k[i] = s.x;
    x.v[i] = s.y;
    k_now = fmaxf(k_now, s.x);
    v_now = fmaxf(v_now, s.y);
    atomicOr(&x.hole[(to - start) >> 5], 1u << ((to - start) & 31));
    a.weight_acc[state + to] = a.weight_acc[state + from];
    a.positions[state + to] = a.positions[state + from];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    k_now = fmaxf(k_now, __shfl_xor_sync(0xffffffffu, k_now, o));
    v_now = fmaxf(v_now, __shfl_xor_sync(0xffffffffu, v_now, o));
  }
  __syncwarp();
  const int lanes = d / 16;  // 16 codes a thread: 4, 8 or 16 threads a row
  const int sub = lane % lanes, group = lane / lanes, groups = 32 / lanes;
  const long long own = own_scale * ps * d;
  uint4* own_k = reinterpret_cast<uint4*>(a.c.k_pages + own) + sub;
  uint4* own_v = reinterpret_cast<uint4*>(a.c.v_pages + own) + sub;
  if (stays && (k_now != k_was || v_now != v_was)) {
    const float kr = k_was / k_now, vr = v_was / v_now;
#pragma unroll 2
    for (int r = group; r < rows; r += groups) {
      if (x.hole[r >> 5] >> (r & 31) & 1u) continue;
      if (k_now != k_was) own_k[r * lanes] = rescale16<E5M2>(own_k[r * lanes], kr);
      if (v_now != v_was) own_v[r * lanes] = rescale16<E5M2>(own_v[r * lanes], vr);
    }
  }
  constexpr int U = 3;  // rows under way (two: 3% slower for long prompts, four: 12% slower for a few slots)
  for (int i0 = group; i0 < cnt; i0 += U * groups) {
    uint4 kc[U], vc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * groups;
      if (i < cnt) {
        kc[u] = reinterpret_cast<const uint4*>(a.c.k_pages + x.src[i])[sub];
        vc[u] = reinterpret_cast<const uint4*>(a.c.v_pages + x.src[i])[sub];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * groups;
      if (i < cnt) {
        if (x.k[i] != k_now) kc[u] = rescale16<E5M2>(kc[u], x.k[i] / k_now);
        if (x.v[i] != v_now) vc[u] = rescale16<E5M2>(vc[u], x.v[i] / v_now);
        own_k[x.to[i] * lanes] = kc[u];
        own_v[x.to[i] * lanes] = vc[u];
      }
    }
  }
  if (lane == 0) {
    if (k_now != k_was) a.c.k_scale[own_scale] = k_now;
    if (v_now != v_was) a.c.v_scale[own_scale] = v_now;
  }
}

template <int C, int TH>
cudaError_t launch_select(const PagedEvictArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.c.B * a.c.Hkv * C));
  cfg.blockDim = dim3(TH);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = C;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = C > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, paged_select_kernel<C, TH>, a);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream) {
  return a.c.e5m2 ? launch_append_t<true>(a, stream) : launch_append_t<false>(a, stream);
}

cudaError_t launch_paged_evict(const PagedEvictArgs& a, cudaStream_t stream) {
  // One CTA of 256 threads a head where its slots' keys fit in its registers
  // (5120), else 1024 threads, else a cluster of those (every barrier of a
  // cluster costs about 0.7 us).
  const int BH = a.c.B * a.c.Hkv;
  const long long slots = (long long)a.c.width * a.c.ps;
  const bool small = slots <= 256 * kSelectKeys;
  int c = 1;
  while (c < 8 && (long long)1024 * kSelectKeys * c < slots) c *= 2;
  cudaError_t e = small    ? launch_select<1, 256>(a, stream)
                  : c == 1 ? launch_select<1, 1024>(a, stream)
                  : c == 2 ? launch_select<2, 1024>(a, stream)
                  : c == 4 ? launch_select<4, 1024>(a, stream)
                           : launch_select<8, 1024>(a, stream);
  if (e != cudaSuccess) return e;
  const int pages = (a.keep + a.c.ps - 1) / a.c.ps;
  const dim3 grid((unsigned)((pages + kMoveWarps - 1) / kMoveWarps), (unsigned)BH);
  return a.c.e5m2 ? launch_pdl(paged_move_kernel<true>, grid, dim3(32 * kMoveWarps), 0, stream, a)
                  : launch_pdl(paged_move_kernel<false>, grid, dim3(32 * kMoveWarps), 0, stream, a);
}

}  // namespace fa
