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
// byte an element: bound by memory for prompts, by its launch for one token.
template <bool E5M2, int NV>
__global__ void __launch_bounds__(256) paged_append_kernel(const __grid_constant__ PagedAppendArgs a) {
  const int b = blockIdx.z, h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int ps = a.c.ps, d = a.c.d;
  const int len = a.lens[b];
  int cnt = a.counts ? a.counts[b] : a.N;
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
  const long long state = ((long long)b * a.c.Hkv + h) * a.c.width * ps;
  if (!is_v) {  // bookkeeping of the new slots
    for (int s = lo + threadIdx.x; s < hi; s += blockDim.x) {
      if (a.weight_acc) a.weight_acc[state + s] = 0.f;
      if (a.positions) a.positions[state + s] = (a.first_position ? a.first_position[b] : len) + (s - len);
    }
  }
  const int page = a.c.table[(long long)b * a.c.width + t];
  if (page < 0 || page >= a.c.pages) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusBadPages);
    return;
  }
  const uint16_t* x = static_cast<const uint16_t*>(is_v ? a.v : a.k) +
                      (((long long)b * a.c.Hkv + h) * a.N + (lo - len)) * d;
  const int vecs = (hi - lo) * d / 16;
  uint4 in[NV][2];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = i * blockDim.x + threadIdx.x;
    if (e < vecs) {
      in[i][0] = reinterpret_cast<const uint4*>(x)[2 * e];
      in[i][1] = reinterpret_cast<const uint4*>(x)[2 * e + 1];
    } else {
      in[i][0] = in[i][1] = make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const uint4& u = in[i][w >> 2];
      const float2 f = unpack16((w & 3) == 0 ? u.x : (w & 3) == 1 ? u.y : (w & 3) == 2 ? u.z : u.w, a.bf16);
      const float m0 = fabsf(f.x), m1 = fabsf(f.y);
      if (m0 < INFINITY) top = fmaxf(top, m0);  // infinities and NaN do not set the scale
      if (m1 < INFINITY) top = fmaxf(top, m1);
    }
  __shared__ float s_top[8];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
  float* scale = (is_v ? a.c.v_scale : a.c.k_scale) + (long long)page * a.c.Hkv + h;
  const float was = lo > start ? *scale : 0.f;  // read by every thread before the barrier, written after it
  __syncthreads();
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) top = fmaxf(top, s_top[w]);
  const float now = fmaxf(was, scale_for<E5M2>(top));
  uint8_t* codes = (is_v ? a.c.v_pages : a.c.k_pages) + ((long long)page * a.c.Hkv + h) * ps * d;
  if (lo > start && now != was) {  // the slots that were there, at the larger scale
    const float ratio = was / now;
    uint4* old = reinterpret_cast<uint4*>(codes);
    for (int e = threadIdx.x; e < (lo - start) * d / 16; e += blockDim.x) old[e] = rescale16<E5M2>(old[e], ratio);
  }
  // x / now; for a power of two the product with its inverse is the same number
  const bool power = (__float_as_uint(now) & 0x7fffffu) == 0 && now >= 0x1p-126f && now <= 0x1p126f;
  const float inv = power ? 1.f / now : 0.f;
  uint4* out = reinterpret_cast<uint4*>(codes + (long long)(lo - start) * d);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = i * blockDim.x + threadIdx.x;
    if (e >= vecs) break;
    uint32_t half[8];
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const uint4& u = in[i][w >> 2];
      float2 f = unpack16((w & 3) == 0 ? u.x : (w & 3) == 1 ? u.y : (w & 3) == 2 ? u.z : u.w, a.bf16);
      if (power) {
        f.x *= inv;
        f.y *= inv;
      } else {
        f.x /= now;
        f.y /= now;
      }
      half[w] = to_codes<E5M2>(f.x, f.y);
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
  const int reach = (a.N + a.c.ps - 2) / a.c.ps + 1;
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
constexpr int kSelectKeys = 54000;  // sort keys that fit in shared memory

// Order of the slots as unsigned numbers: protected ones first, then NaN,
// then the weights from large to small (-0 counts as 0).
__device__ __forceinline__ uint32_t rank_key(float weight, int position, int latest, int recent) {
  if ((long long)position > (long long)latest - recent) return 0xffffffffu;
  if (weight != weight) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(weight + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum of v over the block's 1024 threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // s_warp may still be read by the scan before
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int y = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    s_warp[lane] = y;
  }
  __syncthreads();
  *total = s_warp[31];
  return x - v + (warp > 0 ? s_warp[warp - 1] : 0);
}

// One CTA a (sequence, head): which slots leave, and which of the kept ones
// move where.  The m-th largest key is found bit pair by bit pair (three
// counts a step, keys in shared memory): 16 passes over the keys whatever
// their distribution, and no atomics on data.  Equal keys: the lowest slots
// stay.  A thread then owns a run of consecutive slots, so that prefix sums
// give every hole and every mover its place in slot order.
__global__ void __launch_bounds__(kSelectThreads) paged_select_kernel(const __grid_constant__ PagedEvictArgs a) {
  extern __shared__ uint32_t s_keys[];
  __shared__ int s_warp[32];
  __shared__ int s_count[16][3];
  __shared__ int s_latest, s_bad;
  const int bh = blockIdx.x, b = bh / a.c.Hkv, h = bh % a.c.Hkv;
  const int tid = threadIdx.x, ps = a.c.ps;
  const int n = a.lens[b];
  if (n < 0 || n > a.c.width * ps) {
    if (tid == 0) {
      if (h == 0) {
        atomicOr(a.status, kStatusBadSeqlens);
        a.new_lens[b] = n;
      }
      a.plan_count[bh] = 0;
    }
    return;
  }
  const int m = min(n, a.keep);
  if (m == n) {
    if (tid == 0) {
      if (h == 0) a.new_lens[b] = n;
      a.plan_count[bh] = 0;
    }
    return;
  }
  const int* table = a.c.table + (long long)b * a.c.width;
  const long long state = (long long)bh * a.c.width * ps;
  const float* weight = a.weight_acc + state;
  const int* position = a.positions + state;
  if (tid == 0) {
    s_latest = INT_MIN;
    s_bad = 0;
  }
  if (tid < 48) s_count[tid / 3][tid % 3] = 0;
  __syncthreads();
  int latest = INT_MIN;
  for (int s = tid; s < n; s += kSelectThreads) latest = max(latest, position[s]);
  latest = __reduce_max_sync(0xffffffffu, latest);
  if ((tid & 31) == 0) atomicMax(&s_latest, latest);
  for (int t = tid; t < (n + ps - 1) / ps; t += kSelectThreads)
    if (table[t] < 0 || table[t] >= a.c.pages) s_bad = 1;
  __syncthreads();
  latest = s_latest;
  if (s_bad) {  // reported; the sequence stays as it is (every head's CTA sees the same row)
    if (tid == 0) {
      if (h == 0) {
        atomicOr(a.status, kStatusBadPages);
        a.new_lens[b] = n;
      }
      a.plan_count[bh] = 0;
    }
    return;
  }
  const bool cached = n <= kSelectKeys;
  auto key_of = [&](int s) { return cached ? s_keys[s] : rank_key(weight[s], position[s], latest, a.recent); };
  if (cached) {
    for (int s = tid; s < n; s += kSelectThreads) s_keys[s] = rank_key(weight[s], position[s], latest, a.recent);
    __syncthreads();
  }
  // the largest value v with at least m keys >= v
  uint32_t v = 0;
  for (int step = 0; step < 16; ++step) {
    const int shift = 30 - 2 * step;
    const uint32_t t1 = v | (1u << shift), t2 = v | (2u << shift), t3 = v | (3u << shift);
    int c1 = 0, c2 = 0, c3 = 0;
    for (int s = tid; s < n; s += kSelectThreads) {
      const uint32_t k = key_of(s);
      c1 += k >= t1;
      c2 += k >= t2;
      c3 += k >= t3;
    }
    c1 = __reduce_add_sync(0xffffffffu, c1);
    c2 = __reduce_add_sync(0xffffffffu, c2);
    c3 = __reduce_add_sync(0xffffffffu, c3);
    if ((tid & 31) == 0) {
      atomicAdd(&s_count[step][0], c1);
      atomicAdd(&s_count[step][1], c2);
      atomicAdd(&s_count[step][2], c3);
    }
    __syncthreads();
    if (s_count[step][2] >= m) v = t3;
    else if (s_count[step][1] >= m) v = t2;
    else if (s_count[step][0] >= m) v = t1;
  }
  // runs of consecutive slots, odd in length so that a warp's reads spread over the banks
  const int run = ((n + kSelectThreads - 1) / kSelectThreads) | 1;
  const int s0 = min(n, tid * run), s1 = min(n, s0 + run);
  int above = 0, equal = 0;
  for (int s = s0; s < s1; ++s) {
    const uint32_t k = key_of(s);
    above += k > v;
    equal += k == v;
  }
  int all_above, all_equal;
  block_scan(above, s_warp, &all_above);
  const int equal_before = block_scan(equal, s_warp, &all_equal);
  const int stay = m - all_above;  // of the equal ones, the first
  int holes = 0, movers = 0, eq = equal_before;
  for (int s = s0; s < s1; ++s) {
    const uint32_t k = key_of(s);
    const bool kept = k > v || (k == v && eq < stay);
    eq += k == v;
    holes += !kept && s < m;
    movers += kept && s >= m;
  }
  int all_holes, all_movers;
  int hole_at = block_scan(holes, s_warp, &all_holes);
  int mover_at = block_scan(movers, s_warp, &all_movers);
  eq = equal_before;
  const long long list = (long long)bh * a.keep;
  for (int s = s0; s < s1; ++s) {
    const uint32_t k = key_of(s);
    const bool kept = k > v || (k == v && eq < stay);
    eq += k == v;
    if (!kept && s < m) a.holes[list + hole_at++] = s;
    if (kept && s >= m) {
      const long long at = (long long)table[s / ps] * a.c.Hkv + h;
      a.movers[list + mover_at] = s;
      a.mover_scales[list + mover_at] = make_float2(a.c.k_scale[at], a.c.v_scale[at]);
      ++mover_at;
    }
  }
  if (tid == 0) {
    a.plan_count[bh] = all_holes;
    if (h == 0) a.new_lens[b] = m;
  }
}

// One CTA a (page before the new length, sequence and head): the movers that
// go into the page's holes, the page's slots that stay, at one scale.  A
// mover's own page may be the page where the kept part ends and be rewritten
// at the same time by its own CTA: its rows behind the new length are not
// touched there, and its scale was noted by the kernel before.
template <bool E5M2>
__global__ void __launch_bounds__(128) paged_move_kernel(const __grid_constant__ PagedEvictArgs a) {
  __shared__ uint32_t s_hole[4];
  const int bh = blockIdx.y, b = bh / a.c.Hkv, h = bh % a.c.Hkv;
  const int ps = a.c.ps, d = a.c.d, tid = threadIdx.x;
  const int count = a.plan_count[bh];
  if (count == 0) return;  // nothing leaves, or the sequence was reported
  const int m = a.keep;    // a sequence that loses slots keeps exactly `keep`
  const int start = blockIdx.x * ps, end = min(m, start + ps);
  const long long list = (long long)bh * a.keep;
  const int* holes = a.holes + list;
  auto lower = [&](int slot) {  // holes before `slot`
    int x = 0, y = count;
    while (x < y) {
      const int z = (x + y) >> 1;
      if (holes[z] < slot) x = z + 1; else y = z;
    }
    return x;
  };
  const int lo = lower(start), hi = lower(end);
  if (lo == hi) return;
  const int* table = a.c.table + (long long)b * a.c.width;
  const long long state = (long long)bh * a.c.width * ps;
  const int page = table[blockIdx.x];
  const long long at = (long long)page * a.c.Hkv + h;
  if (tid < 4) s_hole[tid] = 0;
  __syncthreads();
  for (int i = lo + tid; i < hi; i += 128) {
    const int to = holes[i], from = a.movers[list + i];
    atomicOr(&s_hole[(to - start) >> 5], 1u << ((to - start) & 31));
    a.weight_acc[state + to] = a.weight_acc[state + from];
    a.positions[state + to] = a.positions[state + from];
  }
  const bool stays = end - start > hi - lo;  // slots of the page that stay
  const float k_was = a.c.k_scale[at], v_was = a.c.v_scale[at];
  float k_now = 0.f, v_now = 0.f;
  for (int i = lo; i < hi; ++i) {
    const float2 s = a.mover_scales[list + i];
    k_now = fmaxf(k_now, s.x);
    v_now = fmaxf(v_now, s.y);
  }
  if (stays) {
    k_now = fmaxf(k_now, k_was);
    v_now = fmaxf(v_now, v_was);
  }
  __syncthreads();
  const int lanes = d / 16;  // 16 codes a thread
  const int lane = tid % lanes, group = tid / lanes, groups = 128 / lanes;
  const long long own = at * ps * d;
  if (stays && (k_now != k_was || v_now != v_was)) {
    const float kr = k_was / k_now, vr = v_was / v_now;
    for (int s = group; s < end - start; s += groups) {
      if (s_hole[s >> 5] >> (s & 31) & 1u) continue;
      uint4* kp = reinterpret_cast<uint4*>(a.c.k_pages + own + (long long)s * d) + lane;
      uint4* vp = reinterpret_cast<uint4*>(a.c.v_pages + own + (long long)s * d) + lane;
      if (k_now != k_was) *kp = rescale16<E5M2>(*kp, kr);
      if (v_now != v_was) *vp = rescale16<E5M2>(*vp, vr);
    }
  }
  for (int i = lo + group; i < hi; i += groups) {
    const int to = holes[i], from = a.movers[list + i];
    const float2 s = a.mover_scales[list + i];
    const long long src = (((long long)table[from / ps] * a.c.Hkv + h) * ps + from % ps) * d;
    const long long dst = own + (long long)(to - start) * d;
    uint4 kc = reinterpret_cast<const uint4*>(a.c.k_pages + src)[lane];
    uint4 vc = reinterpret_cast<const uint4*>(a.c.v_pages + src)[lane];
    if (s.x != k_now) kc = rescale16<E5M2>(kc, s.x / k_now);
    if (s.y != v_now) vc = rescale16<E5M2>(vc, s.y / v_now);
    reinterpret_cast<uint4*>(a.c.k_pages + dst)[lane] = kc;
    reinterpret_cast<uint4*>(a.c.v_pages + dst)[lane] = vc;
  }
  if (tid == 0) {
    if (k_now != k_was) a.c.k_scale[at] = k_now;
    if (v_now != v_was) a.c.v_scale[at] = v_now;
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendArgs& a, cudaStream_t stream) {
  return a.c.e5m2 ? launch_append_t<true>(a, stream) : launch_append_t<false>(a, stream);
}

cudaError_t launch_paged_evict(const PagedEvictArgs& a, cudaStream_t stream) {
  const int BH = a.c.B * a.c.Hkv;
  const long long slots = (long long)a.c.width * a.c.ps;
  const int smem = (int)(slots < kSelectKeys ? slots : kSelectKeys) * 4;
  cudaError_t e = cudaFuncSetAttribute(paged_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSelectKeys * 4);
  if (e != cudaSuccess) return e;
  paged_select_kernel<<<BH, kSelectThreads, smem, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const dim3 grid((unsigned)((a.keep + a.c.ps - 1) / a.c.ps), (unsigned)BH);
  if (a.c.e5m2)
    paged_move_kernel<true><<<grid, 128, 0, stream>>>(a);
  else
    paged_move_kernel<false><<<grid, 128, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
