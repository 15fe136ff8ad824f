// Pages for each query token and key head, by a score from the pages' bounds.
//
//   score(page) = max over the head's queries of 2^(x + y) sum_e max(q8_e hi_e, q8_e lo_e)
// an upper bound of q . k over the page's keys, up to the rounding of q.  q8, lo and hi are whole
// numbers of at most seven bits, so the sum (below 2^22 for E <= 256) and its product with a power of two
// are exact in 32 bits: the choice does not depend on the order of any sum.
//
// score_kernel: a warp per page.  select_kernel: a CTA per (token, head); the top-th largest score by
// four rounds of an 8-bit radix search, then the pages in ascending order, those above the threshold
// and the first of those on it.
#include "paged.h"
#include "paged_types.cuh"

namespace thin {

namespace {

constexpr int kScoreWarps = 8;
constexpr int kScorePages = 64;    // pages per CTA
constexpr int kSelectThreads = 256;

// Token n's request and the pages its keys reach; false for padding.
__device__ __forceinline__ bool token_pages(const thin_attn_paged_attention_args& a, int n, int* row, int* len, int* pages) {
  *row = a.rows ? a.rows[n] : n;
  if (*row < 0 || *row >= a.R) return false;
  *len = min(max(a.lengths[n], 0), a.W * a.page);
  *pages = (*len + a.page - 1) / a.page;
  return true;
}

template <typename T>
__global__ void __launch_bounds__(kScoreWarps * 32) score_kernel(thin_attn_paged_attention_args a, float* scores) {
  const int n = blockIdx.z, h = blockIdx.y, j0 = blockIdx.x * kScorePages, G = a.Hq / a.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int row, len, pages;
  if (!token_pages(a, n, &row, &len, &pages) || j0 >= pages) return;
  extern __shared__ int8_t q8[];     // G x E, then G floats 2^y
  float* scale = (float*)(q8 + G * a.E);
  for (int g = warp; g < G; g += kScoreWarps) {
    float x[8], m = 0.f;
    const bool mine = lane * 8 < a.E;
    if (mine) {
      load8((const T*)a.q + n * a.q_token + (h * G + g) * a.q_head + lane * 8, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = x[i] == x[i] ? x[i] : 0.f;
        m = fmaxf(m, fabsf(x[i]));
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int y = bound_exponent(m);
    if (mine) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        q8[g * a.E + lane * 8 + i] = (int8_t)(int)fminf(fmaxf(rintf(x[i] * pow2f(-y)), -127.f), 127.f);
    }
    if (lane == 0) scale[g] = pow2f(y);
  }
  __syncthreads();
  float* out = scores + ((int64_t)n * a.H + h) * a.W;
  for (int j = j0 + warp; j < min(pages, j0 + kScorePages); j += kScoreWarps) {
    const int id = a.table[row * a.table_row + j];
    float best = -INFINITY;
    if (id >= 0 && id < a.n_pages) {
      const int8_t* lo = a.bounds + ((int64_t)id * a.H + h) * 2 * a.E;
      const int8_t* hi = lo + a.E;
      const float px = pow2f(a.exps[(int64_t)id * a.H + h]);
      for (int g = 0; g < G; ++g) {
        int dot = 0;
        for (int e = lane; e < a.E; e += 32) {
          const int q = q8[g * a.E + e];
          dot += max(q * hi[e], q * lo[e]);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        best = fmaxf(best, (float)dot * px * scale[g]);
      }
    }
    if (lane == 0) out[j] = best;
  }
}

// Larger scores give larger words; no score gives 0xFFFFFFFF, the word of a forced page.
__device__ __forceinline__ uint32_t rank_of(float s) {
  const uint32_t u = __float_as_uint(s);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelectThreads) select_kernel(thin_attn_paged_attention_args a, const float* scores,
                                                                 int32_t* ids, int32_t* keys) {
  const int n = blockIdx.y, h = blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int row, len, pages;
  if (!token_pages(a, n, &row, &len, &pages)) {
    if (tid == 0 && h == 0) keys[n] = 0;
    return;
  }
  const int take = min(a.top, pages);
  if (tid == 0 && h == 0) keys[n] = take ? (take - 1) * a.page + len - (pages - 1) * a.page : 0;
  const float* s = scores + ((int64_t)n * a.H + h) * a.W;
  const int32_t* table = a.table + row * a.table_row;
  int32_t* list = ids + ((int64_t)n * a.H + h) * a.top;
  int32_t* places = a.pages_out ? a.pages_out + ((int64_t)n * a.H + h) * a.top : nullptr;
  auto word = [&](int j) { return j < a.first || j >= pages - a.last ? 0xFFFFFFFFu : rank_of(s[j]); };
  __shared__ int hist[256];
  __shared__ uint32_t found_s;
  __shared__ int left_s;
  __shared__ int sums[kSelectThreads / 32][2];
  uint32_t threshold = 0;
  int left = take;   // of the pages whose leading digits equal the threshold's, how many are taken
  if (pages > take) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      hist[tid] = 0;
      __syncthreads();
      for (int j = tid; j < pages; j += kSelectThreads) {
        const uint32_t w = word(j);
        if (shift == 24 || (w ^ threshold) >> (shift + 8) == 0) atomicAdd(&hist[(w >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int d = 255, before = 0;
        while (before + hist[d] < left) before += hist[d--];
        found_s = d;
        left_s = left - before;
      }
      __syncthreads();
      threshold |= found_s << shift;
      left = left_s;
      __syncthreads();
    }
  }
  // pages above the threshold and the first `left` on it, in ascending order
  int placed = 0, on = 0;
  for (int j0 = 0; j0 < pages; j0 += kSelectThreads) {
    const int j = j0 + tid;
    const uint32_t w = j < pages ? word(j) : 0;
    const bool above = j < pages && (pages <= take || w > threshold), equal = j < pages && pages > take && w == threshold;
    const uint32_t eb = __ballot_sync(0xffffffffu, equal);
    if (lane == 0) sums[warp][0] = __popc(eb);
    __syncthreads();
    int rank = on + __popc(eb & ((1u << lane) - 1));
    int all = 0;
    for (int i = 0; i < kSelectThreads / 32; ++i) {
      if (i < warp) rank += sums[i][0];
      all += sums[i][0];
    }
    on += all;
    const bool got = above || (equal && rank < left);
    const uint32_t gb = __ballot_sync(0xffffffffu, got);
    if (lane == 0) sums[warp][1] = __popc(gb);
    __syncthreads();
    int at = placed + __popc(gb & ((1u << lane) - 1));
    all = 0;
    for (int i = 0; i < kSelectThreads / 32; ++i) {
      if (i < warp) at += sums[i][1];
      all += sums[i][1];
    }
    placed += all;
    if (got) {
      list[at] = table[j];
      if (places) places[at] = j;
    }
    __syncthreads();
  }
  if (places)
    for (int i = take + tid; i < a.top; i += kSelectThreads) places[i] = -1;
}

template <typename T>
cudaError_t score_t(const thin_attn_paged_attention_args& a, float* scores, cudaStream_t st) {
  const int G = a.Hq / a.H;
  const size_t smem = (size_t)G * a.E + (size_t)G * 4;
  cudaError_t e = cudaFuncSetAttribute(score_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  score_kernel<T><<<dim3((a.W + kScorePages - 1) / kScorePages, a.H, a.N), kScoreWarps * 32, smem, st>>>(a, scores);
  return cudaGetLastError();
}

}  // namespace

size_t paged_select_workspace(const thin_attn_paged_attention_args& a) { return (size_t)a.N * a.H * a.W * 4; }

cudaError_t launch_paged_select(const thin_attn_paged_attention_args& a, int32_t* ids, int32_t* keys, void* workspace,
                                cudaStream_t st) {
  float* scores = (float*)workspace;
  if (a.W > 0) {
    cudaError_t e = a.dtype == THIN_ATTN_FP32   ? score_t<float>(a, scores, st)
                    : a.dtype == THIN_ATTN_BF16 ? score_t<__nv_bfloat16>(a, scores, st)
                                                : score_t<__half>(a, scores, st);
    if (e != cudaSuccess) return e;
  }
  select_kernel<<<dim3(a.H, a.N), kSelectThreads, 0, st>>>(a, scores, ids, keys);
  return cudaGetLastError();
}

}  // namespace thin
