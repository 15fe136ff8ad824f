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
// A cluster of CTAs serves one (token, key head), each an equal run of its pages, the scores in shared
// memory as words of the same order.  The smallest word taken is found by a radix search, 10 bits a
// round from the leading bit of (largest - smallest word), with histograms that the CTAs read from
// one another; it ends as soon as a bin is taken whole, mostly in the second round.  Then each CTA writes
// its pages above that word, and the first of those on it, behind the pages of the CTAs before it, so
// the lists ascend.
#include <cooperative_groups.h>

#include "paged.h"
#include "paged_types.cuh"

namespace cg = cooperative_groups;

namespace thin {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kPerSm = 4;
constexpr int kMostPages = 4096;   // of a CTA, where a larger cluster can be had
constexpr int kGroup = 8;   // pages of one product
constexpr int kBins = 1024;

// Token n's request and the pages its keys reach; false for padding.
__device__ __forceinline__ bool token_pages(const thin_attn_paged_attention_args& a, int n, int* row, int* len, int* pages) {
  *row = a.rows ? a.rows[n] : n;
  if (*row < 0 || *row >= a.R) return false;
  *len = min(max(a.lengths[n], 0), a.W * a.page);
  *pages = (*len + a.page - 1) / a.page;
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

template <typename T, int KJ>   // KJ: 16-byte pieces per lane and page, 2 E <= 64 KJ
__global__ void __launch_bounds__(kThreads, kPerSm) select_kernel(thin_attn_paged_attention_args a, int32_t* ids, int32_t* keys,
                                                          int per) {
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int n = blockIdx.z, h = blockIdx.y, G = a.Hq / a.H, rows = (G + 15) & ~15;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  extern __shared__ __align__(16) unsigned char smem[];
  uint32_t* words = (uint32_t*)smem;                    // [per]
  int8_t* qv = (int8_t*)(words + ((per + 3) & ~3));     // [rows][q_stride]
  float* scale = (float*)(qv + rows * q_stride(a.E));   // [rows]
  __shared__ __align__(16) int hist[2][kBins];
  __shared__ int sums[kWarps][2];
  __shared__ uint32_t range_s[kWarps][2], range_all[2];
  __shared__ int digit_s, left_s, whole_s, counts_s[2];
  // the attention may be launched now; it waits for this grid's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int row, len, pages;
  if (!token_pages(a, n, &row, &len, &pages)) {   // the whole cluster returns
    if (tid == 0 && h == 0 && rank == 0) keys[n] = 0;
    return;
  }
  const int take = min(a.top, pages);
  if (tid == 0 && h == 0 && rank == 0) keys[n] = take ? (take - 1) * a.page + len - (pages - 1) * a.page : 0;
  const int32_t* table = a.table + row * a.table_row;
  int32_t* list = ids + ((int64_t)n * a.H + h) * a.top;
  int32_t* places = a.pages_out ? a.pages_out + ((int64_t)n * a.H + h) * a.top : nullptr;
  const int j0 = min(pages, rank * per), count = min(pages, j0 + per) - j0;   // this CTA's pages
  const bool all = pages <= take;   // no choice to make
  auto forced = [&](int i) { return j0 + i < a.first || j0 + i >= pages - a.last; };

  if (!all) {
    round_queries<T>(a, n, h, G, rows, qv, scale);
    for (int i = tid; i < 2 * kBins; i += kThreads) hist[0][i] = 0;
    __syncthreads();
    uint32_t smallest = 0xFFFFFFFFu, largest = 0;
    const int r = lane >> 2, c = lane & 3, chunks = a.E / 8;
    int next = warp * kGroup + r < count ? table[j0 + warp * kGroup + r] : -1;
    for (int i0 = warp * kGroup; i0 < count; i0 += kWarps * kGroup) {
      const int id = next, i = i0 + kWarps * kGroup + r;
      next = i < count ? table[j0 + i] : -1;   // a product ahead
      const bool held = id >= 0 && id < a.n_pages;
      const int64_t at = (int64_t)(held ? id : 0) * a.H + h;
      const uint4* src = (const uint4*)(a.bounds + at * 2 * a.E);
      uint4 b[KJ];
#pragma unroll
      for (int j = 0; j < KJ; ++j) b[j] = held && c + 4 * j < chunks ? src[c + 4 * j] : make_uint4(0, 0, 0, 0);
      const float px = held ? pow2f(a.exps[at]) : 0.f;
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
          mma_s8(s, a0, b[j].x, b[j].y);
          mma_s8(s, a1, b[j].z, b[j].w);
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
      const float mine0 = __shfl_sync(0xffffffffu, best[0], (lane & 7) >> 1), mine1 = __shfl_sync(0xffffffffu, best[1], (lane & 7) >> 1);
      const float mx = __shfl_sync(0xffffffffu, px, (lane & 7) << 2);
      const int k = i0 + lane;
      if (lane < 8 && k < count) {
        const uint32_t w = rank_of(mx > 0.f ? (lane & 1 ? mine1 : mine0) * mx : -INFINITY);   // a page outside the pool: last
        words[k] = w;
        if (!forced(k)) {
          smallest = min(smallest, w);
          largest = max(largest, w);
        }
      }
    }
    smallest = __reduce_min_sync(0xffffffffu, smallest);
    largest = __reduce_max_sync(0xffffffffu, largest);
    if (lane == 0) {
      range_s[warp][0] = smallest;
      range_s[warp][1] = largest;
    }
    __syncthreads();
    if (tid < 2) {
      uint32_t x = range_s[0][tid];
      for (int k = 1; k < kWarps; ++k) x = tid ? max(x, range_s[k][1]) : min(x, range_s[k][0]);
      range_all[tid] = x;
    }
  }

  // taken: forced pages, words >= floor, and the first `left` of the words floor - 1
  uint64_t floor = 0;
  int left = 0;
  if (!all) {
    cluster.sync();
    uint32_t base = 0xFFFFFFFFu, top = 0;
    for (int k = 0; k < ranks; ++k) {
      const uint32_t* other = cluster.map_shared_rank(range_all, k);
      base = min(base, other[0]);
      top = max(top, other[1]);
    }
    left = take - a.first - a.last;
    floor = (uint64_t)1 << 32;
    uint32_t prefix = 0;
    int shift = 32 - __clz(top - base);   // bits not yet decided
    for (int round = 0; left > 0; ++round) {
      const int bits = min(shift, 10), low = shift - bits;
      int* mine = hist[round & 1];
      for (int i = tid; i < count; i += kThreads) {
        const uint32_t w = words[i] - base;
        if (!forced(i) && (shift >= 32 || w >> shift == prefix)) atomicAdd(&mine[(w >> low) & ((1 << bits) - 1)], 1);
      }
      cluster.sync();
      // thread t: bins 1023 - 4 t and the three below, of all CTAs; the bin at which the running count reaches `left`
      int bin[4] = {0, 0, 0, 0};
      for (int k = 0; k < ranks; ++k) {
        const int4 v = ((const int4*)cluster.map_shared_rank(mine, k))[kBins / 4 - 1 - tid];
        bin[0] += v.w;
        bin[1] += v.z;
        bin[2] += v.y;
        bin[3] += v.x;
      }
      int incl = (bin[0] + bin[1]) + (bin[2] + bin[3]);
      int at = -incl;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) sums[warp][0] = incl;
      ((int4*)hist[(round & 1) ^ 1])[tid] = make_int4(0, 0, 0, 0);   // the other CTAs read it a round ago
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kWarps; ++k)
        if (k < warp) incl += sums[k][0];
      at += incl;   // in the bins above thread t's
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (at < left && at + bin[k] >= left) {
          digit_s = kBins - 1 - 4 * tid - k;
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
  }
  // how many of this CTA's pages are above, and how many on the word below
  int above = 0, on = 0;
  for (int i0 = 0; i0 < count; i0 += kThreads) {
    const int i = i0 + tid;
    const bool in = i < count;
    const uint64_t w = in && !all ? words[i] : 0;
    above += __syncthreads_count(in && (all || forced(i) || w >= floor));
    on += __syncthreads_count(in && !all && left && !forced(i) && w + 1 == floor);
  }
  if (tid == 0) {
    counts_s[0] = above;
    counts_s[1] = on;
  }
  cluster.sync();
  int before_above = 0, before_on = 0;
  for (int k = 0; k < rank; ++k) {
    const int* other = cluster.map_shared_rank(counts_s, k);
    before_above += other[0];
    before_on += other[1];
  }
  int placed = before_above + min(before_on, left);   // taken before this CTA's pages
  on = before_on;
  for (int i0 = 0; i0 < count; i0 += kThreads) {
    const int i = i0 + tid;
    const uint64_t w = i < count && !all ? words[i] : 0;
    const bool top = i < count && (all || forced(i) || w >= floor);
    const bool equal = i < count && !all && left && !forced(i) && w + 1 == floor;
    const uint32_t eb = __ballot_sync(0xffffffffu, equal);
    if (lane == 0) sums[warp][0] = __popc(eb);
    __syncthreads();
    int order = on + __popc(eb & ((1u << lane) - 1));
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      if (k < warp) order += sums[k][0];
      on += sums[k][0];
    }
    const bool got = top || (equal && order < left);
    const uint32_t gb = __ballot_sync(0xffffffffu, got);
    if (lane == 0) sums[warp][1] = __popc(gb);
    __syncthreads();
    int at = placed + __popc(gb & ((1u << lane) - 1));
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      if (k < warp) at += sums[k][1];
      placed += sums[k][1];
    }
    if (got) {
      list[at] = table[j0 + i];
      if (places) places[at] = j0 + i;
    }
  }
  if (places && rank == 0)
    for (int i = take + tid; i < a.top; i += kThreads) places[i] = -1;
  cluster.sync();   // no CTA ends while another reads its counts
}

template <typename T, int KJ>
cudaError_t launch_t(const thin_attn_paged_attention_args& a, int32_t* ids, int32_t* keys, cudaStream_t st) {
  const int rows = (a.Hq / a.H + 15) & ~15;
  // one CTA per 64 pages that the table can hold, as far as a cluster reaches, but no more CTAs than run
  // at once (four per SM), unless the scores need the room
  int cluster = 1;
  while (cluster < kMaxCluster && cluster * 64 < a.W &&
         ((int64_t)2 * cluster * a.N * a.H <= 148 * kPerSm || cluster * kMostPages < a.W))
    cluster *= 2;
  const int per = (a.W + cluster - 1) / cluster;
  const size_t smem = (size_t)((per + 3) & ~3) * 4 + (size_t)rows * q_stride(a.E) + rows * 4;
  auto kernel = select_kernel<T, KJ>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(cluster, a.H, a.N);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, ids, keys, per);
}
template <typename T>
cudaError_t launch_e(const thin_attn_paged_attention_args& a, int32_t* ids, int32_t* keys, cudaStream_t st) {
  if (a.E <= 64) return launch_t<T, 2>(a, ids, keys, st);
  if (a.E <= 128) return launch_t<T, 4>(a, ids, keys, st);
  return launch_t<T, 8>(a, ids, keys, st);
}

}  // namespace

bool paged_select_fits(const thin_attn_paged_attention_args& a) {
  const int64_t rows = (a.Hq / a.H + 15) & ~15, per = ((int64_t)a.W + kMaxCluster - 1) / kMaxCluster;
  return per * 4 + 16 + rows * (q_stride(a.E) + 4) <= 224 * 1024;
}

cudaError_t launch_paged_select(const thin_attn_paged_attention_args& a, int32_t* ids, int32_t* keys, cudaStream_t st) {
  if (a.dtype == THIN_ATTN_FP32) return launch_e<float>(a, ids, keys, st);
  if (a.dtype == THIN_ATTN_BF16) return launch_e<__nv_bfloat16>(a, ids, keys, st);
  return launch_e<__half>(a, ids, keys, st);
}

}  // namespace thin
