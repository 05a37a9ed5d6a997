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

// to_codes for finite numbers within the type's range.
template <bool E5M2>
__device__ __forceinline__ uint32_t to_codes_finite(float a, float b) {
  uint16_t r;
  if (E5M2)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// Four codes times `ratio`, rounded again.
template <bool E5M2>
__device__ __forceinline__ uint32_t rescale4(uint32_t c, float ratio) {
  const float2 a = from_codes<E5M2>(c & 0xffffu), b = from_codes<E5M2>(c >> 16);
  return to_codes<E5M2>(a.x * ratio, a.y * ratio) | (to_codes<E5M2>(b.x * ratio, b.y * ratio) << 16);
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
// One CTA a (sequence, page, head, K or V): the page's new rows are read
// once (16 elements a thread and step, kept in registers), their maximum
// gives the scale, and they are written as codes.  Reads 2 and writes 1
// byte an element.  A prompt is bound by memory as long as an element costs
// few instructions: the maximum is taken on the 16-bit patterns, two at a
// time, and infinities and NaN are looked at one by one only in pages that
// have some (8192 tokens for 4 x 8 heads: 46 us with every element looked at).
// One token a sequence is bound by the launch and three dependent reads.
template <bool E5M2, int NV>
__global__ void __launch_bounds__(256) paged_append_kernel(const __grid_constant__ PagedAppendArgs a) {
  const int b = blockIdx.z, h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int ps = a.c.ps, d = a.c.d;
  const int len = a.lens[b];
  const int cnt = a.counts ? a.counts[b] : a.N;
  const bool first_cta = blockIdx.x == 0 && blockIdx.y == 0;
  if (len < 0 || cnt < 0 || cnt > a.N || len > a.c.width * ps || cnt > a.c.width * ps - len) {
    if (first_cta && threadIdx.x == 0) {
      atomicOr(a.status, kStatusBadSeqlens);
      a.new_lens[b] = len;
    }
    return;
  }
  if (first_cta && threadIdx.x == 0) a.new_lens[b] = len + cnt;
  const int t = (len >> a.c.ps_shift) + blockIdx.x;
  const int start = t * ps;
  const int lo = max(len, start), hi = min(len + cnt, start + ps);
  if (lo >= hi) return;
  const int page = a.c.table[(long long)b * a.c.width + t];
  const uint16_t* x = static_cast<const uint16_t*>(is_v ? a.v : a.k) +
                      (((long long)b * a.c.Hkv + h) * a.N + (lo - len)) * d;
  const int vecs = (hi - lo) * d / 16;
  uint4 in[NV][2];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = i * blockDim.x + threadIdx.x;
    if (e < vecs) {
      in[i][0] = __ldcs(reinterpret_cast<const uint4*>(x) + 2 * e);
      in[i][1] = __ldcs(reinterpret_cast<const uint4*>(x) + 2 * e + 1);
    } else {
      in[i][0] = in[i][1] = make_uint4(0, 0, 0, 0);
    }
  }
  const long long state = ((long long)b * a.c.Hkv + h) * a.c.width * ps;
  if (!is_v) {  // bookkeeping of the new slots
    for (int s = lo + threadIdx.x; s < hi; s += blockDim.x) {
      if (a.weight_acc) a.weight_acc[state + s] = 0.f;
      if (a.positions) a.positions[state + s] = (a.first_position ? a.first_position[b] : len) + (s - len);
    }
  }
  if (page < 0 || page >= a.c.pages) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusBadPages);
    return;
  }
  float* scale = (is_v ? a.c.v_scale : a.c.k_scale) + (long long)page * a.c.Hkv + h;
  const float was = lo > start ? *scale : 0.f;  // read by every thread before the barrier, written after it
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
  __shared__ uint32_t s_top[8], s_fin[8];
  const uint32_t mine = __reduce_max_sync(0xffffffffu, max(two & 0xffffu, two >> 16));
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = mine;
  __syncthreads();
  uint32_t top = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) top = max(top, s_top[w]);
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
    fin = __reduce_max_sync(0xffffffffu, fin);
    if ((threadIdx.x & 31) == 0) s_fin[threadIdx.x >> 5] = fin;
    __syncthreads();
    top = 0;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) top = max(top, s_fin[w]);
  }
  const float now = fmaxf(was, scale_for<E5M2>(unpack16(top, a.bf16).x));
  uint8_t* codes = (is_v ? a.c.v_pages : a.c.k_pages) + ((long long)page * a.c.Hkv + h) * ps * d;
  if (lo > start && now != was) {  // the slots that were there, at the larger scale
    const float ratio = was / now;
    uint4* old = reinterpret_cast<uint4*>(codes);
    for (int e = threadIdx.x; e < (lo - start) * d / 16; e += blockDim.x) old[e] = rescale16<E5M2>(old[e], ratio);
  }
  // x / now; for a power of two the product with its inverse is the same number
  const bool power = (__float_as_uint(now) & 0x7fffffu) == 0 && now >= 0x1p-126f && now <= 0x1p126f;
  const float inv = power ? 1.f / now : 0.f;
  const bool plain = power && all_finite;
  uint4* out = reinterpret_cast<uint4*>(codes + (long long)(lo - start) * d);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = i * blockDim.x + threadIdx.x;
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
  if (threadIdx.x == 0 && now != was) *scale = now;
}

template <bool E5M2>
cudaError_t launch_append_t(const PagedAppendArgs& a, cudaStream_t stream) {
  const int vecs = a.c.ps * a.c.d / 16;  // of a full page: 64 to 2048
  const int threads = vecs < 256 ? vecs : 256;
  // pages that N tokens can reach, wherever the first of them lands
  const int reach = (int)((a.N + a.c.ps - 2LL) / a.c.ps + 1);
  const dim3 grid((unsigned)reach, (unsigned)(2 * a.c.Hkv), (unsigned)a.c.B);
  switch (vecs / threads) {
    case 1: paged_append_kernel<E5M2, 1><<<grid, threads, 0, stream>>>(a); break;
    case 2: paged_append_kernel<E5M2, 2><<<grid, threads, 0, stream>>>(a); break;
    case 4: paged_append_kernel<E5M2, 4><<<grid, threads, 0, stream>>>(a); break;
    case 8: paged_append_kernel<E5M2, 8><<<grid, threads, 0, stream>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

// ---------------------------------------------------------------- evict
constexpr int kSelectThreads = 1024;
constexpr int kSelectKeys = 16;  // sort keys a thread holds in registers

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

// Sums of three numbers over the threads of the C CTAs of a cluster, known to
// every thread; `below` gets those of the CTAs before this one and of the threads
// before this one (PREFIX), in thread order.
struct Three {
  int a, b, c;
};
template <int C>
struct Gather {
  int (*s_warp)[32][3];  // [2] turns
  int (*s_cta)[8][3];    // [2] turns
  int turn = 0;
  __device__ __forceinline__ Three sum(Three v) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    v.a = __reduce_add_sync(0xffffffffu, v.a);
    v.b = __reduce_add_sync(0xffffffffu, v.b);
    v.c = __reduce_add_sync(0xffffffffu, v.c);
    int(*w)[3] = s_warp[turn];
    if (lane == 0) w[warp][0] = v.a, w[warp][1] = v.b, w[warp][2] = v.c;
    __syncthreads();
    v.a = __reduce_add_sync(0xffffffffu, w[lane][0]);
    v.b = __reduce_add_sync(0xffffffffu, w[lane][1]);
    v.c = __reduce_add_sync(0xffffffffu, w[lane][2]);
    if (C > 1) {
      int* mine = s_cta[turn][cluster_rank()];
      if (threadIdx.x < 3 * C) store_remote(mine + threadIdx.x % 3, threadIdx.x / 3, threadIdx.x % 3 == 0 ? v.a : threadIdx.x % 3 == 1 ? v.b : v.c);
      cluster_sync();
      v.a = v.b = v.c = 0;
#pragma unroll
      for (int r = 0; r < C; ++r) {
        v.a += s_cta[turn][r][0];
        v.b += s_cta[turn][r][1];
        v.c += s_cta[turn][r][2];
      }
    }
    turn ^= 1;
    return v;
  }
  // Exclusive prefix sums of a and b over all threads of the cluster, in order.
  __device__ __forceinline__ Three before(Three v, Three* total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int x = v.a, y = v.b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int p = __shfl_up_sync(0xffffffffu, x, o), q = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) x += p, y += q;
    }
    int(*w)[3] = s_warp[turn];
    if (lane == 31) w[warp][0] = x, w[warp][1] = y;
    __syncthreads();
    const int wa = w[lane][0], wb = w[lane][1];
    Three r, all;
    r.a = x - v.a + __reduce_add_sync(0xffffffffu, lane < warp ? wa : 0);
    r.b = y - v.b + __reduce_add_sync(0xffffffffu, lane < warp ? wb : 0);
    all.a = __reduce_add_sync(0xffffffffu, wa);
    all.b = __reduce_add_sync(0xffffffffu, wb);
    r.c = all.c = 0;
    if (C > 1) {
      const int rank = (int)cluster_rank();
      int* mine = s_cta[turn][rank];
      if (threadIdx.x < 2 * C) store_remote(mine + (threadIdx.x & 1), threadIdx.x >> 1, threadIdx.x & 1 ? all.b : all.a);
      cluster_sync();
      all.a = all.b = 0;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (c < rank) r.a += s_cta[turn][c][0], r.b += s_cta[turn][c][1];
        all.a += s_cta[turn][c][0];
        all.b += s_cta[turn][c][1];
      }
    }
    turn ^= 1;
    *total = all;
    return r;
  }
};

// One cluster of C CTAs a (sequence, head): which slots leave, and which of the
// kept ones move where.  A thread owns a run of consecutive slots, its keys
// in registers (up to 16; longer runs are read again in every pass).  The
// m-th largest key is found two bits at a time (three counts a step over all
// keys), at most 16 steps whatever the distribution, fewer where a count
// meets m earlier, and no atomics on data.  Equal keys: the lowest slots stay.
// Prefix sums over the runs then give every hole and every mover its place in
// slot order.  Reads 8 bytes a slot; the steps are bound by their barriers
// (2080 slots: 27 us with keys in shared memory, 1024 strided, and counts by
// atomics).
template <int C>
__global__ void __launch_bounds__(kSelectThreads) paged_select_kernel(const __grid_constant__ PagedEvictArgs a) {
  __shared__ int s_warp[2][32][3];
  __shared__ int s_cta[2][8][3];
  const int bh = blockIdx.x / C, b = bh / a.c.Hkv, h = bh % a.c.Hkv;
  const int rank = C > 1 ? (int)cluster_rank() : 0;
  const int tid = threadIdx.x, ps = a.c.ps;
  const bool speaks = rank == 0 && tid == 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
  const int run = ((n + kSelectThreads * C - 1) / (kSelectThreads * C) + 3) & ~3;
  const long long begin = (long long)(rank * kSelectThreads + tid) * run;
  const int s0 = (int)(begin < n ? begin : n), s1 = min(n, s0 + run);
  const bool cached = run <= kSelectKeys;
  Gather<C> gather = {s_warp, s_cta};

  int latest = INT_MIN, bad = 0;
  float w[kSelectKeys];
  int p[kSelectKeys];
  if (cached) {
#pragma unroll
    for (int i = 0; i < kSelectKeys; i += 4) {
      if (i < run && s0 + i + 4 <= s1) {
        const float4 x = *reinterpret_cast<const float4*>(weight + s0 + i);
        const int4 y = *reinterpret_cast<const int4*>(position + s0 + i);
        w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
        p[i] = y.x, p[i + 1] = y.y, p[i + 2] = y.z, p[i + 3] = y.w;
      } else {
#pragma unroll
        for (int k = i; k < i + 4; ++k) {
          const bool in = k < run && s0 + k < s1;
          w[k] = in ? weight[s0 + k] : 0.f;
          p[k] = in ? position[s0 + k] : INT_MIN;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kSelectKeys; ++i) latest = max(latest, p[i]);
  } else {
    for (int s = s0; s < s1; ++s) latest = max(latest, position[s]);
  }
  for (int t = rank * kSelectThreads + tid; t < (n + ps - 1) / ps; t += kSelectThreads * C)
    bad |= table[t] < 0 || table[t] >= a.c.pages;
  {  // the largest position, in two halves of 16 bits that add up; and bad pages
    latest = __reduce_max_sync(0xffffffffu, latest);
    int(*x)[3] = s_warp[1];
    if ((tid & 31) == 0) x[tid >> 5][0] = latest;
    __syncthreads();
    latest = __reduce_max_sync(0xffffffffu, x[tid & 31][0]);
    if (C > 1) {
      if (tid < C) store_remote(s_cta[1][rank], tid, latest);
      cluster_sync();
#pragma unroll
      for (int r = 0; r < C; ++r) latest = max(latest, s_cta[1][r][0]);
    }
  }
  if (gather.sum({bad, 0, 0}).a) {  // reported; the sequence stays as it is (every head sees the same row)
    if (speaks) {
      if (h == 0) {
        atomicOr(a.status, kStatusBadPages);
        a.new_lens[b] = n;
      }
      a.plan_count[bh] = 0;
    }
    return;
  }
  uint32_t key[kSelectKeys];
#pragma unroll
  for (int i = 0; i < kSelectKeys; ++i)
    key[i] = cached && i < run && s0 + i < s1 ? rank_key(w[i], p[i], latest, a.recent) : 0u;
  auto key_at = [&](int s) { return rank_key(weight[s], position[s], latest, a.recent); };

  // The largest v with at least m keys >= v (keys of slots are at least 0x007fffff, 0 is none).
  uint32_t v = 0;
  int at_least = n;  // keys >= v
  for (int step = 0; step < 16 && at_least != m; ++step) {
    const int shift = 30 - 2 * step;
    const uint32_t t1 = v | (1u << shift), t2 = v | (2u << shift), t3 = v | (3u << shift);
    Three c = {0, 0, 0};
    if (cached) {
#pragma unroll
      for (int i = 0; i < kSelectKeys; ++i) {
        c.a += key[i] >= t1;
        c.b += key[i] >= t2;
        c.c += key[i] >= t3;
      }
    } else {
      for (int s = s0; s < s1; ++s) {
        const uint32_t k = key_at(s);
        c.a += k >= t1;
        c.b += k >= t2;
        c.c += k >= t3;
      }
    }
    c = gather.sum(c);
    if (c.c >= m) v = t3, at_least = c.c;
    else if (c.b >= m) v = t2, at_least = c.b;
    else if (c.a >= m) v = t1, at_least = c.a;
  }
  // Of the keys equal to v all stay (at_least = m), or the first m - above.
  int stay = INT_MAX, eq = 0;
  if (at_least != m) {
    Three mine = {0, 0, 0}, all;
    if (cached) {
#pragma unroll
      for (int i = 0; i < kSelectKeys; ++i) mine.a += key[i] > v, mine.b += key[i] == v;
    } else {
      for (int s = s0; s < s1; ++s) {
        const uint32_t k = key_at(s);
        mine.a += k > v, mine.b += k == v;
      }
    }
    eq = gather.before(mine, &all).b;
    stay = m - all.a;
  }
  auto kept = [&](uint32_t k, int& e) {
    const bool yes = k > v || (k == v && e < stay);
    e += k == v;
    return yes;
  };
  Three mine = {0, 0, 0}, all;
  {
    int e = eq;
    if (cached) {
#pragma unroll
      for (int i = 0; i < kSelectKeys; ++i)
        if (i < run && s0 + i < s1) {
          const bool yes = kept(key[i], e);
          mine.a += !yes && s0 + i < m;
          mine.b += yes && s0 + i >= m;
        }
    } else {
      for (int s = s0; s < s1; ++s) {
        const bool yes = kept(key_at(s), e);
        mine.a += !yes && s < m;
        mine.b += yes && s >= m;
      }
    }
  }
  const Three from = gather.before(mine, &all);
  const long long list = (long long)bh * m;
  const int pages = (m + ps - 1) / ps;
  int* page_holes = a.page_holes + (long long)bh * (pages + 1);  // holes before each page
  int hole_at = from.a, mover_at = from.b;
  auto put = [&](int s, uint32_t k) {
    const bool yes = kept(k, eq);
    if (s < m && (s & (ps - 1)) == 0) page_holes[s >> a.c.ps_shift] = hole_at;
    if (!yes && s < m) a.holes[list + hole_at++] = s;
    if (yes && s >= m) a.movers[list + mover_at++] = s;
  };
  if (cached) {
#pragma unroll
    for (int i = 0; i < kSelectKeys; ++i)
      if (i < run && s0 + i < s1) put(s0 + i, key[i]);
  } else {
    for (int s = s0; s < s1; ++s) put(s, key_at(s));
  }
  if (speaks) {
    page_holes[pages] = all.a;
    a.plan_count[bh] = all.a;
    if (h == 0) a.new_lens[b] = m;
  }
  // The scales of the movers' pages: the moving kernel may change that of the page where the kept part ends.
  if (C > 1) cluster_sync();
  else __syncthreads();
  for (int i = rank * kSelectThreads + tid; i < all.b; i += kSelectThreads * C) {
    const long long at = (long long)table[__ldcg(a.movers + list + i) / ps] * a.c.Hkv + h;
    a.mover_scales[list + i] = make_float2(a.c.k_scale[at], a.c.v_scale[at]);
  }
  if (C > 1) cluster_sync();  // no CTA leaves while another may still write to its shared memory
}

// One CTA a (page before the new length, sequence and head): the movers that
// go into the page's holes, the page's slots that stay, at one scale.  A
// mover's own page may be the page where the kept part ends and be rewritten
// at the same time by its own CTA: its rows behind the new length are not
// touched there, and its scale was noted by the kernel before.
template <bool E5M2>
__global__ void __launch_bounds__(256) paged_move_kernel(const __grid_constant__ PagedEvictArgs a) {
  __shared__ uint32_t s_hole[4];
  __shared__ int s_to[128], s_from[128];  // a mover's row in the page, and its row in the pool (page * ps + row)
  __shared__ long long s_src[128];
  __shared__ float s_k[128], s_v[128];
  __shared__ float s_top[2][4];
  const int bh = blockIdx.y, b = bh / a.c.Hkv, h = bh % a.c.Hkv;
  const int ps = a.c.ps, d = a.c.d, tid = threadIdx.x;
  const int m = a.keep;  // a sequence that loses slots keeps exactly `keep`
  const int start = blockIdx.x * ps, end = min(m, start + ps);
  const int pages = (m + ps - 1) / ps;
  if (tid < 4) s_hole[tid] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int* table = a.c.table + (long long)b * a.c.width;
  const int2 at_page = make_int2(a.page_holes[(long long)bh * (pages + 1) + blockIdx.x],
                                 a.page_holes[(long long)bh * (pages + 1) + blockIdx.x + 1]);
  const int page = table[blockIdx.x];
  const int count = a.plan_count[bh];
  if (count == 0) return;  // nothing leaves, or the sequence was reported: the lists are not set
  const int lo = at_page.x, cnt = at_page.y - lo;
  if (cnt == 0) return;
  const long long list = (long long)bh * m + lo;
  const long long state = (long long)bh * a.c.width * ps;
  const long long own_scale = (long long)page * a.c.Hkv + h;
  const bool stays = end - start > cnt;  // slots of the page that stay
  const float k_was = a.c.k_scale[own_scale], v_was = a.c.v_scale[own_scale];
  __syncthreads();
  float k_now = 0.f, v_now = 0.f;
  if (tid < 128) {  // a page has at most 128 slots
    if (tid < cnt) {
      const int to = a.holes[list + tid], from = a.movers[list + tid];
      const float2 s = a.mover_scales[list + tid];
      s_to[tid] = to - start;
      s_src[tid] = (((long long)table[from / ps] * a.c.Hkv + h) * ps + from % ps) * d;
      s_k[tid] = k_now = s.x;
      s_v[tid] = v_now = s.y;
      atomicOr(&s_hole[(to - start) >> 5], 1u << ((to - start) & 31));
      a.weight_acc[state + to] = a.weight_acc[state + from];
      a.positions[state + to] = a.positions[state + from];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      k_now = fmaxf(k_now, __shfl_xor_sync(0xffffffffu, k_now, o));
      v_now = fmaxf(v_now, __shfl_xor_sync(0xffffffffu, v_now, o));
    }
    if ((tid & 31) == 0) s_top[0][tid >> 5] = k_now, s_top[1][tid >> 5] = v_now;
  }
  __syncthreads();
  k_now = fmaxf(fmaxf(s_top[0][0], s_top[0][1]), fmaxf(s_top[0][2], s_top[0][3]));
  v_now = fmaxf(fmaxf(s_top[1][0], s_top[1][1]), fmaxf(s_top[1][2], s_top[1][3]));
  if (stays) {
    k_now = fmaxf(k_now, k_was);
    v_now = fmaxf(v_now, v_was);
  }
  const int lanes = d / 16;  // 16 codes a thread: 4, 8 or 16 threads a row
  const int lane = tid % lanes, group = tid / lanes, groups = 256 / lanes;
  const long long own = own_scale * ps * d;
  if (stays && (k_now != k_was || v_now != v_was)) {
    const float kr = k_was / k_now, vr = v_was / v_now;
    for (int s = group; s < end - start; s += groups) {
      if (s_hole[s >> 5] >> (s & 31) & 1u) continue;
      uint4* kp = reinterpret_cast<uint4*>(a.c.k_pages + own + (long long)s * d) + lane;
      uint4* vp = reinterpret_cast<uint4*>(a.c.v_pages + own + (long long)s * d) + lane;
      uint4 kc = *kp, vc = *vp;
      if (k_now != k_was) *kp = rescale16<E5M2>(kc, kr);
      if (v_now != v_was) *vp = rescale16<E5M2>(vc, vr);
    }
  }
#pragma unroll 2
  for (int i = group; i < cnt; i += groups) {
    const long long src = s_src[i], dst = own + (long long)s_to[i] * d;
    uint4 kc = reinterpret_cast<const uint4*>(a.c.k_pages + src)[lane];
    uint4 vc = reinterpret_cast<const uint4*>(a.c.v_pages + src)[lane];
    if (s_k[i] != k_now) kc = rescale16<E5M2>(kc, s_k[i] / k_now);
    if (s_v[i] != v_now) vc = rescale16<E5M2>(vc, s_v[i] / v_now);
    reinterpret_cast<uint4*>(a.c.k_pages + dst)[lane] = kc;
    reinterpret_cast<uint4*>(a.c.v_pages + dst)[lane] = vc;
  }
  if (tid == 0) {
    if (k_now != k_was) a.c.k_scale[own_scale] = k_now;
    if (v_now != v_was) a.c.v_scale[own_scale] = v_now;
  }
}

template <int C>
cudaError_t launch_select(const PagedEvictArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.c.B * a.c.Hkv * C));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = C > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, paged_select_kernel<C>, a);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream) {
  return a.c.e5m2 ? launch_append_t<true>(a, stream) : launch_append_t<false>(a, stream);
}

cudaError_t launch_paged_evict(const PagedEvictArgs& a, cudaStream_t stream) {
  // CTAs a head: as many as hold its slots' keys in registers, more while
  // SMs are idle and each still has 4096 slots.
  const int BH = a.c.B * a.c.Hkv;
  const long long slots = (long long)a.c.width * a.c.ps;
  const int sms = sm_count();
  int c = 1;
  while (c < 8 && ((long long)c * kSelectThreads * kSelectKeys < slots ||
                   (2LL * c * BH <= sms && slots / (2 * c) >= 4096)))
    c *= 2;
  cudaError_t e = c == 1   ? launch_select<1>(a, stream)
                  : c == 2 ? launch_select<2>(a, stream)
                  : c == 4 ? launch_select<4>(a, stream)
                           : launch_select<8>(a, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.keep + a.c.ps - 1) / a.c.ps), (unsigned)BH);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return a.c.e5m2 ? cudaLaunchKernelEx(&cfg, paged_move_kernel<true>, a)
                  : cudaLaunchKernelEx(&cfg, paged_move_kernel<false>, a);
}

}  // namespace fa
