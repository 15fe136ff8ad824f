// Slots, block tables and the free-page stack of a step, from request lengths.
//
// A plan is two prefix sums over the requests (their new tokens; the fresh pages of those whose
// tokens and table rows have room), then one slot per token:
//   request  the r with cu[r] <= t < cu[r + 1], by binary search of the sums in shared memory
//   page     table[r][pos / page], or for a fresh page free[n_free - 1 - (fresh pages before it)]
//   slot     page id * page + pos % page
// Nothing here moves more than a few bytes per request and 16 per token: the time is the chain of
// dependent latencies (lengths, sums, search, page id).  Every CTA of a cluster repeats the sums
// for itself, so the only meeting is the one before lengths and n_free are overwritten in place.
#include <cooperative_groups.h>

#include "paged.h"

namespace cg = cooperative_groups;

namespace thin {

namespace {

constexpr int kThreads = 1024;
constexpr int kCluster = 8;   // the largest portable cluster

// Exclusive prefix of v over the block's threads and the total.
__device__ __forceinline__ int64_t block_prefix(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();   // the sums of an earlier call have been read
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int64_t s = lane < (int)(blockDim.x >> 5) ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  *total = warp_sums[(blockDim.x >> 5) - 1];
  return incl - v + (warp ? warp_sums[warp - 1] : 0);
}

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int page) { return (tokens + page - 1) / page; }

struct Request {
  int64_t have, want;   // pages before and after
  int32_t n, L;
  bool narrow;
};
__device__ __forceinline__ Request request(const thin_attn_paged_plan_args& a, int r) {
  Request q;
  const int32_t n = a.n_new[r];
  q.L = a.lengths[r];
  q.n = max(n, 0);
  q.have = pages_of(max(q.L, 0), a.page);
  q.want = pages_of((int64_t)max(q.L, 0) + q.n, a.page);
  q.narrow = q.want > a.W || n < 0 || q.L < 0 || (int64_t)q.L + q.n > 0x7FFFFFFF;
  return q;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(thin_attn_paged_plan_args a) {
  extern __shared__ int32_t smem[];
  __shared__ int64_t warp_sums[32];
  int32_t* cu_s = smem;              // R + 1
  int32_t* base_s = smem + a.R + 1;  // fresh pages before the request's own, -1 when it is not placed
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int per = (a.R + kThreads - 1) / kThreads;
  const int r0 = min(a.R, (int)threadIdx.x * per), r1 = min(a.R, r0 + per);
  const int64_t n_free = min(max(*a.n_free, 0), a.n_pages);
  int64_t tokens = 0;
  for (int r = r0; r < r1; ++r) tokens += request(a, r).n;
  int64_t all_tokens, all_pages;
  const int64_t first = block_prefix(tokens, warp_sums, &all_tokens);
  int64_t pages = 0, at = first;
  for (int r = r0; r < r1; ++r) {
    const Request q = request(a, r);
    at += q.n;
    if (!q.narrow && at <= a.max_tokens) pages += q.want - q.have;
  }
  int64_t base = block_prefix(pages, warp_sums, &all_pages);
  at = first;
  int64_t taken = 0;   // pages that this thread's placed requests take
  for (int r = r0; r < r1; ++r) {
    const Request q = request(a, r);
    cu_s[r] = (int32_t)min(at, (int64_t)0x7FFFFFFF);
    at += q.n;
    const bool late = !q.narrow && at > a.max_tokens;
    const int64_t need = q.narrow || late ? 0 : q.want - q.have;
    const bool dry = need > 0 && base + need > n_free;
    const int status = q.narrow ? 2 : late ? 3 : dry ? 1 : 0;
    base_s[r] = status ? -1 : (int32_t)base;
    if (!status) taken += need;
    base += need;
    if (rank == 0) {
      a.status[r] = status;
      a.cu[r] = cu_s[r];
    }
  }
  int64_t all_taken;
  block_prefix(taken, warp_sums, &all_taken);
  if (threadIdx.x == 0) {
    cu_s[a.R] = (int32_t)min(all_tokens, (int64_t)0x7FFFFFFF);
    if (rank == 0) a.cu[a.R] = cu_s[a.R];
  }
  __syncthreads();
  // fresh table entries, a warp per request
  const int warps = ranks * (kThreads / 32), warp = rank * (kThreads / 32) + (int)(threadIdx.x >> 5);
  for (int r = warp; r < a.R; r += warps) {
    if (base_s[r] < 0) continue;
    const Request q = request(a, r);
    for (int64_t j = q.have + (threadIdx.x & 31); j < q.want; j += 32)
      a.table[r * a.table_row + j] = a.free_pages[n_free - 1 - (base_s[r] + j - q.have)];
  }
  // the tokens' slots
  const int live = min(cu_s[a.R], a.max_tokens);
  for (int t = rank * kThreads + (int)threadIdx.x; t < a.max_tokens; t += ranks * kThreads) {
    int64_t slot = -1;
    int row = -1, context = 0;
    if (t < live) {
      int lo = 0, hi = a.R;   // the last r with cu[r] <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu_s[mid] <= t) lo = mid; else hi = mid;
      }
      if (base_s[lo] >= 0) {
        const int L = a.lengths[lo], pos = L + t - cu_s[lo], j = pos / a.page, have = (int)pages_of(L, a.page);
        const int id = j < have ? a.table[lo * a.table_row + j] : a.free_pages[n_free - 1 - (base_s[lo] + j - have)];
        slot = (int64_t)id * a.page + pos % a.page;
        row = lo;
        context = pos + 1;
      }
    }
    a.slots[t] = slot;
    a.rows[t] = row;
    a.context[t] = context;
  }
  cluster.sync();   // every CTA has read lengths and n_free
  if (rank != 0) return;
  for (int r = threadIdx.x; r < a.R; r += kThreads) {
    const int32_t L = a.lengths[r];
    a.lengths_out[r] = base_s[r] < 0 ? L : L + max(a.n_new[r], 0);
  }
  if (threadIdx.x == 0) *a.n_free_out = (int32_t)(n_free - all_taken);
}

// One CTA: the released pages' prefix sums give each its place on the stack.
__global__ void __launch_bounds__(kThreads) release_kernel(thin_attn_paged_release_args a) {
  __shared__ int64_t warp_sums[32];
  extern __shared__ int32_t base_s[];   // R
  const int per = (a.R + kThreads - 1) / kThreads;
  const int r0 = min(a.R, (int)threadIdx.x * per), r1 = min(a.R, r0 + per);
  const int64_t n_free = min(max(*a.n_free, 0), a.n_pages);
  auto kept = [&](int r, int64_t* from, int64_t* to) {
    const int64_t L = max(a.lengths[r], 0), keep = a.keep[r] < 0 ? L : min((int64_t)a.keep[r], L);
    *to = min(pages_of(L, a.page), (int64_t)a.W);
    *from = min(pages_of(keep, a.page), *to);
    return (int32_t)keep;
  };
  int64_t pages = 0, from, to, total;
  for (int r = r0; r < r1; ++r) {
    kept(r, &from, &to);
    pages += to - from;
  }
  int64_t base = block_prefix(pages, warp_sums, &total);
  for (int r = r0; r < r1; ++r) {
    kept(r, &from, &to);
    base_s[r] = (int32_t)min(base, (int64_t)a.n_pages);
    base += to - from;
  }
  __syncthreads();
  for (int r = threadIdx.x >> 5; r < a.R; r += kThreads / 32) {
    const int32_t keep = kept(r, &from, &to);
    for (int64_t j = from + (threadIdx.x & 31); j < to; j += 32) {
      const int64_t at = n_free + base_s[r] + j - from;
      int32_t* id = a.table + r * a.table_row + j;
      if (at < a.n_pages) a.free_pages[at] = *id;
      *id = -1;
    }
    __syncwarp();
    if ((threadIdx.x & 31) == 0 && a.lengths[r] >= 0) a.lengths[r] = keep;
  }
  __syncthreads();
  if (threadIdx.x == 0) *a.n_free = (int32_t)min(n_free + total, (int64_t)a.n_pages);
}

}  // namespace

cudaError_t launch_paged_plan(const thin_attn_paged_plan_args& a, cudaStream_t st) {
  const size_t smem = (size_t)(2 * a.R + 1) * 4;
  static SharedMemory memory;
  cudaError_t e = memory.allow((const void*)plan_kernel, (2 * kMaxRequests + 1) * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_kernel, a);
}

cudaError_t launch_paged_release(const thin_attn_paged_release_args& a, cudaStream_t st) {
  const size_t smem = (size_t)a.R * 4;
  static SharedMemory memory;
  cudaError_t e = memory.allow((const void*)release_kernel, kMaxRequests * 4);
  if (e != cudaSuccess) return e;
  release_kernel<<<1, kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace thin
