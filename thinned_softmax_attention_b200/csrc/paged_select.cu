// Pages for each query token and key head, by a score from the pages' bounds.
//
//   score(page) = max over the head's queries of 2^(x + y) sum_e max(q8_e hi_e, q8_e lo_e)
// an upper bound of q . k over the page's keys, up to the rounding of q.  q8, lo and hi are whole
// numbers of at most seven bits, so the sum (below 2^22 for E <= 256) and its product with a power of two
// are exact in 32 bits: the choice does not depend on the order of any sum.
//
// max(q hi, q lo) = max(q, 0) hi + min(q, 0) lo: the scores of a head's queries are one product of
// (queries x 2 E) by (2 E x pages) in 8-bit integers, mma m16n8k32 with the queries as rows.  The order
// of the summed index is free, so a lane takes its fragments as 16-byte pieces of a page's 2 E
// bytes, straight from global memory; each is read once.
//
// score_kernel: CTAs take equal runs of the pages of one (token, key head) and write the scores as words
// of the same order.  select_kernel: one CTA per (token, key head) finds the smallest word
// taken by a radix search, 10 bits a round from the leading bit of (largest - smallest word); it ends as
// soon as a bin is taken whole, mostly in the second round.  Then it writes the pages above that
// word, and the first of those on it, in ascending order.
// Latency bounds both (a scoring CTA's chain: length, page id, bounds).  B200: 32 requests of up to 2048 pages,
// 8 heads: scoring 18 us (34 MB of bounds), choice 10; one request of 1024 pages 8 and 9.  One launch with a
// cluster per (token, head) took 37 us for the batch: its meetings cost more than the second launch.
#include "paged.h"
#include "paged_types.cuh"

namespace thin {

namespace {

constexpr int kWarps = 8;          // of a scoring CTA
constexpr int kGroup = 8;          // pages of one product
constexpr int kSelectThreads = 512;
constexpr int kBins = 1024, kOwn = kBins / kSelectThreads;   // a thread adds up kOwn bins
constexpr int kHeld = 8192;        // words that the selection keeps in shared memory; more are read again

// Token n's request and the pages its keys reach; false for padding.
__device__ __forceinline__ bool token_pages(const thin_attn_paged_attention_args& a, int n, int* row, int* len, int* pages) {
  *row = a.rows ? a.rows[n] : n;
  if (*row < 0 || *row >= a.R) return false;
  *len = min(max(a.lengths[n], 0), a.W * a.page);
  *pages = (int)(((uint32_t)*len + a.page - 1) / (uint32_t)a.page);   // the sum may pass 31 bits
  return true;
}

// Larger scores give larger words.
__device__ __forceinline__ uint32_t rank_of(float s) {
  const uint32_t u = __float_as_uint(s);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ void mma_s8(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Bytes between two queries in shared memory: neighbouring rows half the banks apart.
__host__ __device__ __forceinline__ int q_stride(int E) { return 2 * E + 64; }

// The head's queries as min(q8, 0) (E bytes) and max(q8, 0) (E bytes), and 2^y; rows up to a multiple of 16
// are zero.
template <typename T>
__device__ __forceinline__ void round_queries(const thin_attn_paged_attention_args& a, int n, int h, int G, int rows, int8_t* qv,
                                              float* scale) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool mine = lane * 8 < a.E;
  for (int g = warp; g < rows; g += kWarps) {
    float x[8], m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (mine && g < G) {
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
      uint32_t lo[2] = {0, 0}, hi[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int q = (int)fminf(fmaxf(rintf(x[i] * pow2f(-y)), -127.f), 127.f);
        lo[i >> 2] |= (uint32_t)(min(q, 0) & 0xFF) << (8 * (i & 3));
        hi[i >> 2] |= (uint32_t)max(q, 0) << (8 * (i & 3));
      }
      *(uint2*)(qv + g * q_stride(a.E) + lane * 8) = make_uint2(lo[0], lo[1]);
      *(uint2*)(qv + g * q_stride(a.E) + a.E + lane * 8) = make_uint2(hi[0], hi[1]);
    }
    if (lane == 0) scale[g] = pow2f(y);
  }
}

// A page outside the pool scores lowest.
template <typename T, int KJ>   // KJ: 16-byte pieces per lane and page, 2 E <= 64 KJ
__global__ void __launch_bounds__(kWarps * 32) score_kernel(thin_attn_paged_attention_args a, uint32_t* words, int per) {
  // the selection may be launched now; it waits for this grid's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int n = blockIdx.z, h = blockIdx.y, G = a.Hq / a.H, rows = (G + 15) & ~15;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  extern __shared__ __align__(16) unsigned char smem[];
  int8_t* qv = (int8_t*)smem;                           // [rows][q_stride]
  float* scale = (float*)(qv + rows * q_stride(a.E));   // [rows]
  int row, len, pages;
  if (!token_pages(a, n, &row, &len, &pages) || pages <= a.top) return;   // no choice to make
  const int j0 = blockIdx.x * per, count = min(pages - j0, per);
  if (count <= 0) return;
  const int32_t* table = a.table + row * a.table_row + j0;
  words += ((int64_t)n * a.H + h) * a.W + j0;
  const int r = lane >> 2, c = lane & 3, chunks = a.E / 8;
  // kAhead products' pages at a time, their ids fetched a turn before
  constexpr int kAhead = KJ <= 4 ? 2 : 1, kTurn = kWarps * kGroup * kAhead;
  int next[kAhead];
  auto look = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) next[u] = i0 + u * kGroup + r < count ? table[i0 + u * kGroup + r] : -1;
  };
  look(warp * kGroup * kAhead);
  round_queries<T>(a, n, h, G, rows, qv, scale);
  __syncthreads();
  for (int i0 = warp * kGroup * kAhead; i0 < count; i0 += kTurn) {
    uint4 b[kAhead][KJ];
    float px[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const bool held = next[u] >= 0 && next[u] < a.n_pages;
      const int64_t at = (int64_t)(held ? next[u] : 0) * a.H + h;
      const uint4* src = (const uint4*)(a.bounds + at * 2 * a.E);
#pragma unroll
      for (int j = 0; j < KJ; ++j) b[u][j] = held && c + 4 * j < chunks ? src[c + 4 * j] : make_uint4(0, 0, 0, 0);
      px[u] = held ? pow2f(a.exps[at]) : 0.f;
    }
    look(i0 + kTurn);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float best[2] = {-INFINITY, -INFINITY};   // of pages 2 c and 2 c + 1
      for (int m0 = 0; m0 < G; m0 += 16) {
        int s[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
          uint4 q0 = make_uint4(0, 0, 0, 0), q1 = q0;
          if (c + 4 * j < chunks) {
            q0 = *(const uint4*)(qv + (m0 + r) * q_stride(a.E) + (c + 4 * j) * 16);
            if (m0 + 8 < G) q1 = *(const uint4*)(qv + (m0 + r + 8) * q_stride(a.E) + (c + 4 * j) * 16);
          }
          const uint32_t a0[4] = {q0.x, q1.x, q0.y, q1.y}, a1[4] = {q0.z, q1.z, q0.w, q1.w};
          mma_s8(s, a0, b[u][j].x, b[u][j].y);
          mma_s8(s, a1, b[u][j].z, b[u][j].w);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (m0 + r + 8 * x < G) {
            best[0] = fmaxf(best[0], (float)s[2 * x] * scale[m0 + r + 8 * x]);
            best[1] = fmaxf(best[1], (float)s[2 * x + 1] * scale[m0 + r + 8 * x]);
          }
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        best[0] = fmaxf(best[0], __shfl_xor_sync(0xffffffffu, best[0], o));
        best[1] = fmaxf(best[1], __shfl_xor_sync(0xffffffffu, best[1], o));
      }
      // lane 4 r' + c has page r' in `px` and pages 2 c, 2 c + 1 in `best`: lanes 0..7 take one page each
      const float b0 = __shfl_sync(0xffffffffu, best[0], (lane & 7) >> 1), b1 = __shfl_sync(0xffffffffu, best[1], (lane & 7) >> 1);
      const float mx = __shfl_sync(0xffffffffu, px[u], (lane & 7) << 2);
      const int k = i0 + u * kGroup + lane;
      if (lane < 8 && k < count) words[k] = rank_of(mx > 0.f ? (lane & 1 ? b1 : b0) * mx : -INFINITY);
    }
  }
}

__global__ void __launch_bounds__(kSelectThreads) select_kernel(thin_attn_paged_attention_args a, const uint32_t* words,
                                                                 int32_t* ids, int32_t* keys) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kThreads = kSelectThreads, kSelectWarps = kThreads / 32;
  const int n = blockIdx.y, h = blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ uint32_t held[kHeld];
  __shared__ int hist[2][kBins];
  __shared__ int sums[kSelectWarps][2];
  __shared__ uint32_t range[kSelectWarps][2];
  __shared__ int digit_s, left_s, whole_s;
  for (int i = tid; i < 2 * kBins; i += kThreads) hist[0][i] = 0;
  int row, len, pages;
  const bool live = token_pages(a, n, &row, &len, &pages);
  // for the scores; every CTA waits, so that this grid's end means the scoring's end too
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!live) {
    if (tid == 0 && h == 0) keys[n] = 0;
    return;
  }
  const int take = min(a.top, pages);
  if (tid == 0 && h == 0) keys[n] = take ? (take - 1) * a.page + len - (pages - 1) * a.page : 0;
  const int32_t* table = a.table + row * a.table_row;
  int32_t* list = ids + ((int64_t)n * a.H + h) * a.top;
  int32_t* places = a.pages_out ? a.pages_out + ((int64_t)n * a.H + h) * a.top : nullptr;
  if (places)
    for (int i = take + tid; i < a.top; i += kThreads) places[i] = -1;
  if (pages <= take) {
    for (int i = tid; i < take; i += kThreads) {
      list[i] = table[i];
      if (places) places[i] = i;
    }
    return;
  }
  words += ((int64_t)n * a.H + h) * a.W;
  auto forced = [&](int i) { return i < a.first || i >= pages - a.last; };
  uint32_t base = 0xFFFFFFFFu, most = 0;
  for (int i = tid; i < pages; i += kThreads) {
    const uint32_t w = words[i];
    if (pages <= kHeld) held[i] = w;
    if (!forced(i)) {
      base = min(base, w);
      most = max(most, w);
    }
  }
  base = __reduce_min_sync(0xffffffffu, base);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) {
    range[warp][0] = base;
    range[warp][1] = most;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSelectWarps; ++k) {
    base = min(base, range[k][0]);
    most = max(most, range[k][1]);
  }
  const uint32_t* w_of = pages <= kHeld ? held : words;

  // taken: forced pages, words >= floor, and the first `left` of the words floor - 1
  uint64_t floor = (uint64_t)1 << 32;
  int left = take - a.first - a.last;
  uint32_t prefix = 0;
  int shift = 32 - __clz(most - base);   // bits not yet decided
  for (int round = 0; left > 0; ++round) {
    const int bits = min(shift, 10), low = shift - bits;
    int* mine = hist[round & 1];
    for (int i = tid; i < pages; i += kThreads) {
      const uint32_t w = w_of[i] - base;
      if (!forced(i) && (shift >= 32 || w >> shift == prefix)) atomicAdd(&mine[(w >> low) & ((1 << bits) - 1)], 1);
    }
    __syncthreads();
    // thread t: its bins from the top down; the bin at which the running count reaches `left`
    int bin[kOwn], incl = 0;
#pragma unroll
    for (int x = 0; x < kOwn; ++x) {
      bin[x] = mine[kBins - 1 - kOwn * tid - x];
      incl += bin[x];
      hist[(round & 1) ^ 1][x * kThreads + tid] = 0;
    }
    int at = -incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sums[warp][0] = incl;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSelectWarps; ++k)
      if (k < warp) incl += sums[k][0];
    at += incl;   // in the bins above thread t's
#pragma unroll
    for (int k = 0; k < kOwn; ++k) {
      if (at < left && at + bin[k] >= left) {
        digit_s = kBins - 1 - kOwn * tid - k;
        left_s = left - at;
        whole_s = at + bin[k] == left;
      }
      at += bin[k];
    }
    __syncthreads();
    prefix = prefix << bits | (uint32_t)digit_s;
    left = left_s;
    shift = low;
    if (whole_s) {          // the bin is taken whole
      floor = (uint64_t)base + ((uint64_t)prefix << low);
      left = 0;
    } else if (low == 0) {
      floor = (uint64_t)base + prefix + 1;
      break;
    }
  }
  // each warp takes a run of pages: how many are above, and how many on the word below
  const int run = ((pages + kSelectWarps - 1) / kSelectWarps + 31) & ~31, from = min(pages, warp * run), to = min(pages, from + run);
  auto look_at = [&](int i, bool* top, bool* equal) {
    const uint64_t w = i < to ? w_of[i] : 0;
    *top = i < to && (forced(i) || w >= floor);
    *equal = i < to && !*top && left && w + 1 == floor;
  };
  int above = 0, on = 0;
  for (int i0 = from; i0 < to; i0 += 32) {
    bool top, equal;
    look_at(i0 + lane, &top, &equal);
    above += __popc(__ballot_sync(0xffffffffu, top));
    on += __popc(__ballot_sync(0xffffffffu, equal));
  }
  __syncthreads();   // the sums of the last round have been read
  if (lane == 0) {
    sums[warp][0] = above;
    sums[warp][1] = on;
  }
  __syncthreads();
  above = on = 0;   // in the pages before this warp's
#pragma unroll
  for (int k = 0; k < kSelectWarps; ++k)
    if (k < warp) {
      above += sums[k][0];
      on += sums[k][1];
    }
  for (int i0 = from; i0 < to; i0 += 32) {
    bool top, equal;
    look_at(i0 + lane, &top, &equal);
    const uint32_t tb = __ballot_sync(0xffffffffu, top), eb = __ballot_sync(0xffffffffu, equal), under = (1u << lane) - 1;
    const int order = on + __popc(eb & under);
    if (top || (equal && order < left)) {
      const int at = above + __popc(tb & under) + min(order, left), j = i0 + lane;
      list[at] = table[j];
      if (places) places[at] = j;
    }
    above += __popc(tb);
    on += __popc(eb);
  }
}

template <typename T, int KJ>
cudaError_t score_t(const thin_attn_paged_attention_args& a, uint32_t* words, cudaStream_t st) {
  const int rows = (a.Hq / a.H + 15) & ~15;
  // 128 pages per CTA, one turn, while those CTAs run at once (four per SM); four turns where there are more
  // (the batch above with its attention: 80 us at 128 pages, 77 at 512, 83 at 1024)
  int per = 128;
  if ((int64_t)((a.W + per - 1) / per) * a.N * a.H > 148 * 4) per = 512;
  const size_t smem = (size_t)rows * q_stride(a.E) + rows * 4;
  auto kernel = score_kernel<T, KJ>;
  static SharedMemory memory;
  cudaError_t e = memory.allow((const void*)kernel, kMaxGroup * (q_stride(256) + 4));
  if (e != cudaSuccess) return e;
  kernel<<<dim3((a.W + per - 1) / per, a.H, a.N), kWarps * 32, smem, st>>>(a, words, per);
  return cudaGetLastError();
}
template <typename T>
cudaError_t score_e(const thin_attn_paged_attention_args& a, uint32_t* words, cudaStream_t st) {
  if (a.E <= 64) return score_t<T, 2>(a, words, st);
  if (a.E <= 128) return score_t<T, 4>(a, words, st);
  return score_t<T, 8>(a, words, st);
}

}  // namespace

size_t paged_select_workspace(const thin_attn_paged_attention_args& a) { return a.W > a.top ? (size_t)a.N * a.H * a.W * 4 : 0; }

cudaError_t launch_paged_select(const thin_attn_paged_attention_args& a, int32_t* ids, int32_t* keys, void* workspace,
                                cudaStream_t st) {
  uint32_t* words = (uint32_t*)workspace;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  if (a.W > a.top) {   // else every page is taken
    cudaError_t e = a.dtype == THIN_ATTN_FP32   ? score_e<float>(a, words, st)
                    : a.dtype == THIN_ATTN_BF16 ? score_e<__nv_bfloat16>(a, words, st)
                                                : score_e<__half>(a, words, st);
    if (e != cudaSuccess) return e;
    cfg.numAttrs = 1;
  }
  cfg.gridDim = dim3(a.H, a.N);
  cfg.blockDim = dim3(kSelectThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, select_kernel, a, (const uint32_t*)words, ids, keys);
}

}  // namespace thin
