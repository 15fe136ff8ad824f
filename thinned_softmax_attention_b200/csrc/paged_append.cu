// New keys and values into their slots, with the bounds of every touched page's keys.
//
// A warp takes one run of neighbouring tokens that share a page (a single token without bounds), for
// one key head: it copies the rows (rounding to e4m3 where the cache holds that) and keeps the
// channels' running minimum and maximum, so the keys are read once.  Lane l holds channels 8 l ..
// 8 l + 7 of a key row (E <= 256).  The exponent x is monotone in max |k|, and
// floor(floor(u) / 2^s) = floor(u / 2^s), so widening stored bounds step by step gives the bounds
// that all of the page's keys together would.  HBM bound: each row is read and written once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "paged.h"
#include "paged_types.cuh"

namespace thin {

namespace {

constexpr int kWarps = 8;

template <typename T, typename C>
__device__ __forceinline__ void hold(const float (&x)[8], float scale, C* dst, float (&held)[8]) {
  if constexpr (sizeof(C) == 1) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // the quotient is rounded to fp32, then to e4m3
      const uint32_t b = __nv_cvt_float_to_fp8(x[i] / scale, __NV_SATFINITE, __NV_E4M3);
      w[i >> 2] |= b << (8 * (i & 3));
      held[i] = e4m3_to_f(b);
    }
    *(uint2*)dst = make_uint2(w[0], w[1]);
  } else {
    store8(dst, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) held[i] = x[i];
  }
}

template <typename T, typename C>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(thin_attn_paged_append_args a) {
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (unit >= (int64_t)a.N * a.H) return;
  const int first = (int)(unit / a.H), h = (int)(unit % a.H);
  const int64_t slots = (int64_t)a.n_pages * a.page;
  int64_t slot = a.slots[first];
  if (slot < 0 || slot >= slots) return;
  const int64_t pg = slot / a.page;
  if (a.bounds && first > 0) {
    const int64_t before = a.slots[first - 1];
    if (before >= 0 && before < slots && before / a.page == pg) return;   // inside an earlier token's run
  }
  const float ks = a.k_scale ? a.k_scale[h] : 1.f, vs = a.v_scale ? a.v_scale[h] : 1.f;
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = INFINITY;
    hi[i] = -INFINITY;
  }
  bool anew = false;
  for (int t = first;;) {
    const int64_t off = slot - pg * a.page;
    anew |= off == 0;
    if (lane * 8 < a.E) {
      float x[8], held[8];
      load8((const T*)a.k + t * a.k_token + h * a.k_head + lane * 8, x);
      hold<T>(x, ks, (C*)a.k_pages + pg * a.kp_page + h * a.kp_head + off * a.kp_row + lane * 8, held);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = held[i] == held[i] ? held[i] : 0.f;
        lo[i] = fminf(lo[i], y);
        hi[i] = fmaxf(hi[i], y);
      }
    }
    if (lane * 8 < a.D) {
      float x[8], held[8];
      load8((const T*)a.v + t * a.v_token + h * a.v_head + lane * 8, x);
      hold<T>(x, vs, (C*)a.v_pages + pg * a.vp_page + h * a.vp_head + off * a.vp_row + lane * 8, held);
    }
    if (!a.bounds || ++t >= a.N) break;
    slot = a.slots[t];
    if (slot < pg * a.page || slot >= (pg + 1) * a.page) break;
  }
  if (!a.bounds) return;
  float m = 0.f;
  const bool mine = lane * 8 < a.E;
  if (mine) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  int x = bound_exponent(m);
  int8_t* row = a.bounds + (pg * a.H + h) * 2 * a.E;
  int8_t* exp = a.exps + pg * a.H + h;
  const int x0 = anew ? x : *exp;
  const int up = max(0, x - x0);   // the stored bounds' steps grow by 2^up
  x = max(x, x0);
  __syncwarp();                    // every lane has read the exponent
  if (lane == 0) *exp = (int8_t)x;
  if (!mine) return;
  const float inv = pow2f(-x);
  uint2 wl = make_uint2(0, 0), wh = wl, ol = wl, oh = wl;
  if (!anew) {
    ol = *(const uint2*)(row + lane * 8);
    oh = *(const uint2*)(row + a.E + lane * 8);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    int l = (int)fminf(fmaxf(floorf(lo[i] * inv), -127.f), 127.f);
    int u = (int)fminf(fmaxf(ceilf(hi[i] * inv), -127.f), 127.f);
    if (!anew) {
      const int sl = (int8_t)((i < 4 ? ol.x : ol.y) >> (8 * (i & 3))), sh = (int8_t)((i < 4 ? oh.x : oh.y) >> (8 * (i & 3)));
      l = min(l, sl >> min(up, 31));
      u = max(u, -((-sh) >> min(up, 31)));
    }
    const uint32_t bl = (uint32_t)(l & 0xFF) << (8 * (i & 3)), bu = (uint32_t)(u & 0xFF) << (8 * (i & 3));
    if (i < 4) {
      wl.x |= bl;
      wh.x |= bu;
    } else {
      wl.y |= bl;
      wh.y |= bu;
    }
  }
  *(uint2*)(row + lane * 8) = wl;
  *(uint2*)(row + a.E + lane * 8) = wh;
}

template <typename T, typename C>
cudaError_t launch_t(const thin_attn_paged_append_args& a, cudaStream_t st) {
  const int64_t units = (int64_t)a.N * a.H;
  append_kernel<T, C><<<(unsigned)((units + kWarps - 1) / kWarps), kWarps * 32, 0, st>>>(a);
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
