// New keys and values into their slots, with the bounds of every touched page's keys.
//
// A CTA takes a block of tokens of one key head (heads vary fastest, so that the rows of a token are
// read together) and copies their rows in 16-byte pieces, rounded to e4m3 where the cache holds that.
// It brings the bounds up to date for every run of neighbouring tokens that share a page and begins
// in the block, to the run's end: runs of up to 16 tokens by one warp each, from L1; of longer ones every
// thread takes the minimum and maximum of the pieces that it copies (and of some of the run's tokens
// behind the block), and a warp per run joins them.  The exponent x is monotone in max |k|, and
// floor(floor(u) / 2^s) = floor(u / 2^s), so widening stored bounds step by step gives the bounds
// that all of the page's keys together would.
// Each row is written once.  For the bounds the keys of short runs, and those of a run behind its block, are read and
// rounded again, from L1 and L2 (DRAM: 68 MB read of 67): about half of all keys with pages of 64 that begin anywhere.  One
// CTA per head takes the whole of a run, so that pages much longer than a block are slow where bounds are kept.
// B200, 16384 tokens of 8 heads of width 128: 25 us in bf16 without bounds (134 MB, 85% of the copy rate), 37 with them, 43
// into e4m3 (27 without); there instructions bound it (issue slots 56% and 67% busy with 43% of the warps; a page of 64
// keys is some 1200 of them per warp of its CTA).  64 tokens, one page each: 2.6 us without, 6.5 with.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "paged.h"
#include "paged_types.cuh"

namespace thin {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMany = 64, kFew = 8;   // tokens of a block, at most and at least
constexpr int kPieces = 4;            // pieces of keys that a thread copies
constexpr int kShort = 16;            // tokens of a run that one warp takes

// x / scale by the rounded reciprocal and one correction of the remainder (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990): what is wrong with the reciprocal enters the
// remainder's share alone, so the result differs from the rounded quotient only where x / scale lies within 2^-23 of a
// step of the middle between two fp32 numbers.  Next to a border of two e4m3 values, where alone the byte would tell, there is no such x
// of 8 or 11 bits: all their mantissas, with the scales up to three steps around x / border, give the rounded quotient.
// It has no branch, so the rows' loads stay together.  Very large quotients go uncorrected (they are clamped), scales of
// unusual size by division.
struct Quotient {
  float scale, inverse;
  bool plain;
  __device__ __forceinline__ explicit Quotient(float s) : scale(s), inverse(1.f / s), plain(!(fabsf(s) > 1e-18f && fabsf(s) < 1e18f)) {}
  __device__ __forceinline__ float operator()(float x) const {
    const float q = x * inverse, better = fmaf(fmaf(-q, scale, x), inverse, q);
    return fabsf(q) < 1048576.f ? better : q;
  }
};

// Eight elements as they are given, and as a cache of type C holds them.
template <typename T>
struct Raw {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* src) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = ((const uint4*)src)[i];
  }
};
template <typename C>
struct Held {
  static constexpr int kWords = 2 * (int)sizeof(C);
  uint32_t w[kWords];
};
__device__ __noinline__ void divide8(float* x, float scale) {
  for (int i = 0; i < 8; ++i) x[i] /= scale;
}
template <typename T, typename C>
__device__ __forceinline__ Held<C> held_of(const Raw<T>& r, const Quotient& by) {
  Held<C> y;
  if constexpr (sizeof(C) == 1) {
    float x[8];
    load8((const T*)r.w, x);
    if (by.plain) {   // for the whole grid alike per head
      float z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = x[i];
      divide8(z, by.scale);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = z[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = by(x[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[i], x[i + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[i + 2], x[i + 3]), __NV_SATFINITE, __NV_E4M3);
      y.w[i / 4] = lo | hi << 16;
    }
  } else {
#pragma unroll
    for (int i = 0; i < Held<C>::kWords; i += 4) {
      y.w[i] = r.w[i / 4].x;
      y.w[i + 1] = r.w[i / 4].y;
      y.w[i + 2] = r.w[i / 4].z;
      y.w[i + 3] = r.w[i / 4].w;
    }
  }
  return y;
}
template <typename C>
__device__ __forceinline__ void put_held(C* dst, const Held<C>& y) {
  if constexpr (sizeof(C) == 1) {
    *(uint2*)dst = make_uint2(y.w[0], y.w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < Held<C>::kWords; i += 4) ((uint4*)dst)[i / 4] = make_uint4(y.w[i], y.w[i + 1], y.w[i + 2], y.w[i + 3]);
  }
}

// Minima and maxima run on the held values as they are: two 16-bit ones to a word (e4m3 as fp16, exactly),
// or one fp32.
template <typename C>
struct Lane8 {
  using M = typename std::conditional<sizeof(C) == 1, __half, C>::type;
  static constexpr int kWords = sizeof(M) == 4 ? 8 : 4;
  using V = typename std::conditional<sizeof(M) == 4, float, typename std::conditional<std::is_same<M, __half>::value, __half2, __nv_bfloat162>::type>::type;
  V v[kWords];
  static __device__ __forceinline__ V lesser(V a, V b) {
    if constexpr (sizeof(M) == 4) return fminf(a, b); else return __hmin2(a, b);
  }
  static __device__ __forceinline__ V greater(V a, V b) {
    if constexpr (sizeof(M) == 4) return fmaxf(a, b); else return __hmax2(a, b);
  }
  static __device__ __forceinline__ V everywhere(float x) {
    if constexpr (sizeof(M) == 4) return x;
    else if constexpr (std::is_same<M, __half>::value) return __half2half2(__float2half_rn(x));
    else return __bfloat162bfloat162(__float2bfloat16_rn(x));
  }
  // A NaN as 0.
  static __device__ __forceinline__ V number(V a) {
    if constexpr (sizeof(M) == 4) {
      return a == a ? a : 0.f;
    } else {
      const uint32_t w = *(const uint32_t*)&a & __heq2_mask(a, a);
      return *(const V*)&w;
    }
  }
  __device__ __forceinline__ void set(const Held<C>& y) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      V a;
      if constexpr (sizeof(C) == 1) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(y.w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
        a = __half2(h);
      } else {
        a = *(const V*)&y.w[i];
      }
      v[i] = number(a);
    }
  }
  __device__ __forceinline__ void floats(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(M) == 4) {
        x[i] = v[i];
      } else {
        float2 f;
        if constexpr (std::is_same<M, __half>::value) f = __half22float2(v[i]); else f = __bfloat1622float2(v[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
};
template <typename C>
struct Range {
  using L = Lane8<C>;
  static constexpr int kWords = L::kWords;
  L lo, hi;
  __device__ __forceinline__ Range() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      lo.v[i] = L::everywhere(INFINITY);
      hi.v[i] = L::everywhere(-INFINITY);
    }
  }
  __device__ __forceinline__ void take(const L& l, const L& h) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      lo.v[i] = L::lesser(lo.v[i], l.v[i]);
      hi.v[i] = L::greater(hi.v[i], h.v[i]);
    }
  }
  __device__ __forceinline__ void take(const Held<C>& y) {
    L x;
    x.set(y);
    take(x, x);
  }
  // with lanes l and l + per, l + 2 per ...
  __device__ __forceinline__ void join(int per) {
    for (int o = per; o < 32; o <<= 1) {
      L l, h;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        l.v[i] = __shfl_xor_sync(0xffffffffu, lo.v[i], o);
        h.v[i] = __shfl_xor_sync(0xffffffffu, hi.v[i], o);
      }
      take(l, h);
    }
  }
};
// Over tokens first, first + step, ... below last.
template <typename T, typename C>
__device__ __forceinline__ void range_of(const thin_attn_paged_append_args& a, Range<C>& g, int first, int last, int step, int h, int col, const Quotient& ks) {
  const T* src = (const T*)a.k + h * a.k_head + col;
  constexpr int U = 4;
  for (int t = first; t < last; t += U * step) {
    Raw<T> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t + u * step < last) x[u].load(src + (t + u * step) * a.k_token);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t + u * step < last) g.take(held_of<T, C>(x[u], ks));
  }
}

struct Stored {
  uint2 lo, hi;
  int exp;
};

// Whole numbers and floats by the exponent of 2^23: no conversions, which run at a quarter of the rate or less.
// floor and ceil of |x| <= 127 as the low byte of the result.
__device__ __forceinline__ uint32_t floor_byte(float x) { return __float_as_uint(__fadd_rd(x, 12582912.f)); }
__device__ __forceinline__ uint32_t ceil_byte(float x) { return __float_as_uint(__fadd_ru(x, 12582912.f)); }
// Byte i of w, a signed one with its top bit inverted.
__device__ __forceinline__ float signed_byte(uint32_t w, int i) {
  return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 | i)) - 8388736.f;
}
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// A warp writes the bounds of one page and head: of `g` alone, or the stored ones widened, which is the same as
// the bounds of both's values: floor(floor(u) / 2^s) = floor(u / 2^s).  Lanes of the same channels hold
// the same range.
template <typename C>
__device__ __forceinline__ void write_bounds(const thin_attn_paged_append_args& a, const Range<C>& g, const Stored& old, bool anew,
                                             int64_t at, int col, bool writes, int lane) {
  float m = 0.f, lo[8], hi[8];
  g.lo.floats(lo);
  g.hi.floats(hi);
  if (col < a.E) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  int x = bound_exponent(m);
  if (!anew) {
    x = max(x, min(max(old.exp, kBoundMin), kBoundMax));
    const float step = pow2f(min(max(old.exp, kBoundMin), kBoundMax));
    const uint32_t l[2] = {old.lo.x ^ 0x80808080u, old.lo.y ^ 0x80808080u}, h[2] = {old.hi.x ^ 0x80808080u, old.hi.y ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo[i] = fminf(lo[i], signed_byte(l[i >> 2], i & 3) * step);
      hi[i] = fmaxf(hi[i], signed_byte(h[i >> 2], i & 3) * step);
    }
  }
  if (lane == 0) a.exps[at] = (int8_t)x;
  if (!writes || col >= a.E) return;
  const float inv = pow2f(-x);
  uint32_t l[8], h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    l[i] = floor_byte(fminf(fmaxf(lo[i] * inv, -127.f), 127.f));
    h[i] = ceil_byte(fminf(fmaxf(hi[i] * inv, -127.f), 127.f));
  }
  int8_t* row = a.bounds + at * 2 * a.E;
  *(uint2*)(row + col) = make_uint2(low_bytes(l[0], l[1], l[2], l[3]), low_bytes(l[4], l[5], l[6], l[7]));
  *(uint2*)(row + a.E + col) = make_uint2(low_bytes(h[0], h[1], h[2], h[3]), low_bytes(h[4], h[5], h[6], h[7]));
}

template <typename T, typename C>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 2 : 4) append_kernel(thin_attn_paged_append_args a, int block, int k_shift, int v_shift) {
  // k_shift, v_shift: 2^shift threads take a row, 8 elements each
  const int h = blockIdx.x % a.H, t0 = blockIdx.x / a.H * block, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ int page_s[kMany + 2], off_s[kMany];   // page_s[0]: the token before the block, [block + 1]: none
  // the slots behind the block, for its last run's end
  int64_t behind = a.bounds && t0 + block + lane < a.N ? a.slots[t0 + block + lane] : -1;
  if (tid <= block + 1) {
    const int t = t0 + tid - 1;
    const int64_t slot = t >= 0 && t < a.N && tid <= block ? a.slots[t] : -1;
    int pg = -1;
    if (slot >= 0 && slot < (int64_t)a.n_pages * a.page) {
      pg = slot >> 32 ? (int)(slot / a.page) : (int)((uint32_t)slot / (uint32_t)a.page);
      if (tid > 0) off_s[tid - 1] = (int)(slot - (int64_t)pg * a.page);
    }
    page_s[tid] = pg;
  }
  __syncthreads();
  if (a.bounds && tid < block && page_s[tid + 1] >= 0 && page_s[tid + 1] != page_s[tid]) {
    // a run's stored bounds, wanted when its keys have been read
    const int64_t at = (int64_t)page_s[tid + 1] * a.H + h;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.exps + at));
    for (int i = 0; i < 2 * a.E; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.bounds + at * 2 * a.E + i));
  }
  const Quotient ks(a.k_scale ? a.k_scale[h] : 1.f), vs(a.v_scale ? a.v_scale[h] : 1.f);
  const int k_col = (tid & ((1 << k_shift) - 1)) * 8, v_col = (tid & ((1 << v_shift) - 1)) * 8;
  const int k_row = tid >> k_shift, v_row = tid >> v_shift, k_step = kThreads >> k_shift, v_step = kThreads >> v_shift;
  for (int r0 = v_row; r0 < block; r0 += kPieces * v_step) {
    Raw<T> raw[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int r = r0 + u * v_step;
      if (r < block && v_col < a.D && page_s[r + 1] >= 0) raw[u].load((const T*)a.v + (t0 + r) * a.v_token + h * a.v_head + v_col);
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int r = r0 + u * v_step;
      if (r < block && v_col < a.D && page_s[r + 1] >= 0)
        put_held((C*)a.v_pages + page_s[r + 1] * a.vp_page + h * a.vp_head + off_s[r] * a.vp_row + v_col, held_of<T, C>(raw[u], vs));
    }
  }
  // the host chose the block so that kPieces turns cover its keys
  Held<C> x[kPieces];
  bool has[kPieces];
  {
    Raw<T> raw[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int r = k_row + u * k_step;
      has[u] = r < block && k_col < a.E && page_s[r + 1] >= 0;
      if (has[u]) raw[u].load((const T*)a.k + (t0 + r) * a.k_token + h * a.k_head + k_col);
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) x[u] = held_of<T, C>(raw[u], ks);
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int r = k_row + u * k_step;
    if (has[u]) put_held((C*)a.k_pages + page_s[r + 1] * a.kp_page + h * a.kp_head + off_s[r] * a.kp_row + k_col, x[u]);
  }
  if (!a.bounds) return;

  // bit i: token i begins a run, or goes to its page's first slot
  uint64_t starts = 0, fresh = 0;
#pragma unroll
  for (int x2 = 0; x2 < kMany; x2 += 32) {
    const int i = x2 + lane;
    starts |= (uint64_t)__ballot_sync(0xffffffffu, i < block && (i == 0 || page_s[i + 1] != page_s[i])) << x2;
    fresh |= (uint64_t)__ballot_sync(0xffffffffu, i < block && page_s[i + 1] >= 0 && off_s[i] == 0) << x2;
  }
  // tokens behind the block that go on with a run that begins in it, and whether one of them is its
  // page's first slot: 32 at first, then kScan * 32 at a time
  int tail = 0;
  bool tail_anew = false;
  if (page_s[block] >= 0 && (starts > 1 || page_s[1] != page_s[0])) {
    const int64_t begin = (int64_t)page_s[block] * a.page;
    constexpr int kScan = 8;
    auto scan = [&](int64_t slot) {   // whether the run goes on behind these 32
      const uint32_t in = __ballot_sync(0xffffffffu, slot >= begin && slot < begin + a.page);
      const int run = in == 0xffffffffu ? 32 : __ffs(~in) - 1;
      tail_anew |= __any_sync(0xffffffffu, lane < run && slot == begin);
      tail += run;
      return run == 32;
    };
    bool on = scan(behind);
    while (on) {
      int64_t slot[kScan];
      const int from = t0 + block + tail + lane;
#pragma unroll
      for (int u = 0; u < kScan; ++u) slot[u] = from + 32 * u < a.N ? a.slots[from + 32 * u] : -1;
#pragma unroll
      for (int u = 0; u < kScan; ++u)
        if (on) on = scan(slot[u]);
    }
  }
  // of the runs that begin in a block all but the last end in it: at most four of 64 tokens have more than
  // kShort, two of 32 (keys wider than 128: kPieces turns), one of kFew
  constexpr int kLongs = 64;   // runs times threads of a row
  __shared__ __align__(16) Lane8<C> part[kLongs * 2 * kWarps];
  const int per = 1 << k_shift, col = (lane & (per - 1)) * 8, sub = lane >> k_shift, rows = 32 >> k_shift;
  int shorts = 0, longs = 0;
  // every run that begins in the block: its first token, its tokens, its page, whether it starts the page anew
  auto runs = [&](auto&& f) {
    for (uint64_t left = starts; left;) {
      const int begin = __ffsll(left) - 1;
      left &= left - 1;
      const int end = left ? __ffsll(left) - 1 : block, pg = page_s[begin + 1];
      if (pg < 0 || pg == page_s[begin]) continue;   // no token, or the rest of a run that began before the block
      const bool anew = (fresh >> begin & (~0ull >> (64 - (end - begin)))) || (end == block && tail_anew);
      f(begin, end - begin + (end == block ? tail : 0), pg, anew);
    }
  };
  auto stored = [&](int64_t at, bool anew) {
    Stored old{};
    if (!anew) {
      if (col < a.E) {
        old.lo = *(const uint2*)(a.bounds + at * 2 * a.E + col);
        old.hi = *(const uint2*)(a.bounds + at * 2 * a.E + a.E + col);
      }
      old.exp = a.exps[at];
      __syncwarp();   // before lane 0 writes the exponent
    }
    return old;
  };
  runs([&](int begin, int n, int pg, bool anew) {
    if (n <= kShort) {
      if (shorts++ % kWarps != warp) return;
      const int64_t at = (int64_t)pg * a.H + h;
      const Stored old = stored(at, anew);
      Range<C> g;
      if (col < a.E) range_of<T, C>(a, g, t0 + begin + sub, t0 + begin + n, rows, h, col, ks);
      g.join(per);
      write_bounds(a, g, old, anew, at, col, sub == 0, lane);
      return;
    }
    Range<C> g;
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int r = k_row + u * k_step;
      if (has[u] && r >= begin && r < begin + n) g.take(x[u]);
    }
    if (begin + n > block && col < a.E)
      range_of<T, C>(a, g, t0 + block + warp * rows + sub, t0 + begin + n, kWarps * rows, h, col, ks);
    g.join(per);
    if (sub == 0 && col < a.E) {
      Lane8<C>* dst = part + (longs * kWarps + warp) * 2 * per + col / 8;
      dst[0] = g.lo;
      dst[per] = g.hi;
    }
    ++longs;
  });
  if (longs == 0) return;   // for every thread of the CTA alike
  __syncthreads();
  longs = 0;
  runs([&](int begin, int n, int pg, bool anew) {
    if (n <= kShort || longs++ % kWarps != warp) return;
    const int64_t at = (int64_t)pg * a.H + h;
    const Stored old = stored(at, anew);
    Range<C> g;
    if (col < a.E) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const Lane8<C>* src = part + ((longs - 1) * kWarps + w) * 2 * per + col / 8;
        g.take(src[0], src[per]);
      }
    }
    write_bounds(a, g, old, anew, at, col, sub == 0, lane);
  });
}

int shift_of(int width) {
  int s = 0;
  while ((8 << s) < width) ++s;
  return s;
}

template <typename T, typename C>
cudaError_t launch_t(const thin_attn_paged_append_args& a, cudaStream_t st) {
  const int k_shift = shift_of(a.E), v_shift = shift_of(a.D);
  // as many tokens as kPieces turns cover, where there are such blocks for every SM (1999 tokens of 8 heads into
  // e4m3: 12.0 us, in blocks of 16 15.6); else few, so that a decode step's tokens, one page each, are spread out (64
  // tokens: 6.3 us, in one block per head 30)
  int block = kPieces * kThreads >> k_shift;
  if (block > kMany) block = kMany;
  if ((int64_t)a.N * a.H < 148 * kMany) block = kFew;
  const int64_t grid = (int64_t)((a.N + block - 1) / block) * a.H;
  append_kernel<T, C><<<(unsigned)grid, kThreads, 0, st>>>(a, block, k_shift, v_shift);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const thin_attn_paged_append_args& a, cudaStream_t st) {
  const bool q = a.cache_dtype == THIN_ATTN_E4M3;
  if (a.dtype == THIN_ATTN_FP32) return launch_t<float, float>(a, st);
  if (a.dtype == THIN_ATTN_BF16) return q ? launch_t<__nv_bfloat16, e4m3>(a, st) : launch_t<__nv_bfloat16, __nv_bfloat16>(a, st);
  return q ? launch_t<__half, e4m3>(a, st) : launch_t<__half, __half>(a, st);
}

}  // namespace thin
