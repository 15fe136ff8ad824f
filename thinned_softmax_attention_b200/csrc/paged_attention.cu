// Attention of single query tokens over lists of cache pages.
//
// A CTA per (token, query head); its warps take every fourth key, each with a running maximum and sum
// (m <- max(m, z), the sums so far times 2^(m_old - m)), and are joined at the end.
#include "paged.h"
#include "paged_types.cuh"

namespace thin {

namespace {

constexpr int kWarps = 4;

template <typename T, typename C>
__global__ void __launch_bounds__(kWarps * 32) attention_kernel(PagedAttn p) {
  const thin_attn_paged_attention_args& a = p.a;
  const int n = blockIdx.x, qh = blockIdx.y, h = qh / (a.Hq / a.H);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = a.rows ? a.rows[n] : n;
  if (row < 0 || row >= a.R) return;   // padding: its outputs stay as they were
  const int32_t* ids = p.ids + (p.list_rows ? row : n) * p.ids_token + h * p.ids_head;
  const int len = min(max(p.keys[n], 0), p.list_width * a.page);
  const float sk = p.scale_log2e * (a.k_scale ? a.k_scale[h] : 1.f), sv = a.v_scale ? a.v_scale[h] : 1.f;
  float q[8], o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = o[i] = 0.f;
  if (lane * 8 < a.E) load8((const T*)a.q + n * a.q_token + qh * a.q_head + lane * 8, q);
  float m = -INFINITY, l = 0.f;
  for (int j = (a.window && len > a.window ? len - a.window : 0) + warp; j < len; j += kWarps) {
    const int id = ids[j / a.page], off = j % a.page;
    if (id < 0 || id >= a.n_pages) continue;
    float z = 0.f, v[8];
    if (lane * 8 < a.E) {
      float k[8];
      load8((const C*)a.k_pages + id * a.kp_page + h * a.kp_head + off * a.kp_row + lane * 8, k);
#pragma unroll
      for (int i = 0; i < 8; ++i) z = fmaf(q[i], k[i], z);
    }
    if (lane * 8 < a.D) load8((const C*)a.v_pages + id * a.vp_page + h * a.vp_head + off * a.vp_row + lane * 8, v);
#pragma unroll
    for (int s = 16; s; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
    z *= sk;
    const float mn = fmaxf(m, z), f = m == -INFINITY ? 0.f : exp2f(m - mn), w = z == -INFINITY ? 0.f : exp2f(z - mn);
    m = mn;
    l = l * f + w;
    if (lane * 8 < a.D) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = fmaf(w, v[i], o[i] * f);
    }
  }
  __shared__ float m_s[kWarps], l_s[kWarps], o_s[kWarps][256];
  if (lane == 0) {
    m_s[warp] = m;
    l_s[warp] = l;
  }
  if (lane * 8 < a.D) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o_s[warp][lane * 8 + i] = o[i];
  }
  __syncthreads();
  float M = -INFINITY, L = 0.f, f[kWarps];
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, m_s[w]);
  for (int w = 0; w < kWarps; ++w) {
    f[w] = m_s[w] == -INFINITY ? 0.f : exp2f(m_s[w] - M);
    L += l_s[w] * f[w];
  }
  const float inv = L == 0.f ? 0.f : sv / L;
  for (int d = threadIdx.x; d < a.D; d += kWarps * 32) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += o_s[w][d] * f[w];
    ((T*)a.out)[n * a.out_token + qh * a.out_head + d] = elem_of<T>(x * inv);
  }
  if (threadIdx.x == 0 && a.lse)
    a.lse[(int64_t)n * a.Hq + qh] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

template <typename T, typename C>
cudaError_t launch_t(const PagedAttn& p, cudaStream_t st) {
  attention_kernel<T, C><<<dim3(p.a.N, p.a.Hq), kWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t paged_attention_workspace(const thin_attn_paged_attention_args& a) { return 0; }

cudaError_t launch_paged_attention(const PagedAttn& p, void* workspace, cudaStream_t st) {
  const bool q = p.a.cache_dtype == THIN_ATTN_E4M3;
  if (p.a.dtype == THIN_ATTN_FP32) return launch_t<float, float>(p, st);
  if (p.a.dtype == THIN_ATTN_BF16) return q ? launch_t<__nv_bfloat16, e4m3>(p, st) : launch_t<__nv_bfloat16, __nv_bfloat16>(p, st);
  return q ? launch_t<__half, e4m3>(p, st) : launch_t<__half, __half>(p, st);
}

}  // namespace thin
