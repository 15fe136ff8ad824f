// Slots, block tables and the free-page stack of a step, from request lengths.
//
// A plan is two prefix sums over the requests (their new tokens; the fresh pages of those whose
// tokens and table rows have room), then one slot per token:
//   request  the r with cu[r] <= t < cu[r + 1], by binary search of the sums
//   page     table[r][pos / page], once the fresh pages, free[n_free - 1 - (those before it)], are in the table
//   slot     page id * page + pos % page
// Nothing here moves more than a few bytes per request and 16 per token: the time is the chain of
// dependent latencies (lengths, sums, search, page id), so one CTA takes it all while the tokens are few,
// and a second launch spreads the tokens over the GPU when they are many.  Both sums are taken at
// once, as if every token had room; only where one has not are the pages summed again.
// B200: 64 requests of one token 3.5 us, 512 of them 5.4, 65536 tokens of 512 requests 12 us.
#include "paged.h"

namespace thin {

namespace {

// Of the first launch; 64 requests with 256 threads 3.6 us, with 1024 4.6.
constexpr int kThreads = 1024, kFewThreads = 256;
// Tokens that the first launch places itself: alone and with the second launch, 64 requests 3.6 and 5.8 us for 64
// tokens, 6.4 and 7.1 for 2048, 7.5 and 7.2 for 4096; 512 requests 6.7 and 6.7 for 2048, 7.9 and 6.5 for 4096.
constexpr int kFillHere = 2048;
constexpr int kFillThreads = 256;
constexpr int kOwnPages = 2;                        // fresh pages that a request's thread enters itself

struct Sums {
  int64_t tokens, pages;
};
__device__ __forceinline__ Sums operator+(Sums a, Sums b) { return {a.tokens + b.tokens, a.pages + b.pages}; }
__device__ __forceinline__ Sums operator-(Sums a, Sums b) { return {a.tokens - b.tokens, a.pages - b.pages}; }

// Exclusive prefix of v over the block's threads, and the total.
__device__ __forceinline__ Sums block_prefix(Sums v, Sums* warp_sums, Sums* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums y = {__shfl_up_sync(0xffffffffu, incl.tokens, o), __shfl_up_sync(0xffffffffu, incl.pages, o)};
    if (lane >= o) incl = incl + y;
  }
  __syncthreads();   // the sums of an earlier call have been read
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  // every warp adds the warps' sums up for itself
  Sums w = lane < (int)(blockDim.x >> 5) ? warp_sums[lane] : Sums{0, 0};
  Sums before = lane < warp ? w : Sums{0, 0};
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    w = w + Sums{__shfl_xor_sync(0xffffffffu, w.tokens, o), __shfl_xor_sync(0xffffffffu, w.pages, o)};
    before = before + Sums{__shfl_xor_sync(0xffffffffu, before.tokens, o), __shfl_xor_sync(0xffffffffu, before.pages, o)};
  }
  *total = w;
  return incl - v + before;
}

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int page) {
  return tokens < 0x7FFF0000 ? ((uint32_t)tokens + page - 1) / (uint32_t)page : (tokens + page - 1) / page;
}

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

// Writes slot, request and context of place t, below the step's tokens or not (`held`), of the requests
// lo .. hi - 1.  cu(r): the sums; length(r): the request's length before the step, negative when it was not
// placed.
template <typename Cu, typename Length>
__device__ __forceinline__ void put_token(const thin_attn_paged_plan_args& a, int t, bool held, int lo, int hi, Cu&& cu, Length&& length) {
  int64_t slot = -1;
  int row = -1, context = 0;
  if (held) {
    while (hi - lo > 1) {   // the last r with cu[r] <= t
      const int mid = (lo + hi) >> 1;
      if (cu(mid) <= t) lo = mid; else hi = mid;
    }
    const int L = length(lo);
    if (L >= 0) {
      const int pos = L + t - cu(lo), j = (int)((uint32_t)pos / (uint32_t)a.page);
      slot = (int64_t)a.table[lo * a.table_row + j] * a.page + (pos - j * a.page);
      row = lo;
      context = pos + 1;
    }
  }
  a.slots[t] = slot;
  a.rows[t] = row;
  a.context[t] = context;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(thin_attn_paged_plan_args a) {
  extern __shared__ int32_t smem[];
  __shared__ Sums warp_sums[32];
  __shared__ int taken_s;
  int32_t* cu_s = smem;                 // R + 1
  int32_t* length_s = cu_s + a.R + 1;   // R: before the step, -1 when the request is not placed
  int32_t* base_s = length_s + a.R;     // R: fresh pages before its own
  const int threads = blockDim.x, tid = threadIdx.x, lane = tid & 31;
  // the filling launch may be set up now; it waits for this grid's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int per = (a.R + threads - 1) / threads;
  const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
  const int64_t n_free = min(max(*a.n_free, 0), a.n_pages);
  if (tid == 0) taken_s = 0;
  Sums mine = {0, 0}, all;
  for (int r = r0; r < r1; ++r) {
    const Request q = request(a, r);
    mine = mine + Sums{q.n, q.narrow ? 0 : q.want - q.have};
  }
  Sums at = block_prefix(mine, warp_sums, &all);
  if (all.tokens > a.max_tokens) {   // for every thread alike
    int64_t t = at.tokens;
    mine.pages = 0;
    for (int r = r0; r < r1; ++r) {
      const Request q = request(a, r);
      t += q.n;
      if (!q.narrow && t <= a.max_tokens) mine.pages += q.want - q.have;
    }
    at = block_prefix(mine, warp_sums, &all);
  }
  int taken = 0;   // pages taken up to this thread's last placed request
  bool many = false;
  for (int r = r0; r < r1; ++r) {
    const Request q = request(a, r);
    const int cu = (int)min(at.tokens, (int64_t)0x7FFFFFFF);
    at.tokens += q.n;
    const bool late = !q.narrow && at.tokens > a.max_tokens;
    const int64_t need = q.narrow || late ? 0 : q.want - q.have, base = at.pages;
    at.pages += need;
    const int status = q.narrow ? 2 : late ? 3 : need > 0 && at.pages > n_free ? 1 : 0;
    if (status == 0 && need > 0) {
      taken = (int)at.pages;
      many |= need > kOwnPages;
      if (need <= kOwnPages)
        for (int64_t j = 0; j < need; ++j) a.table[r * a.table_row + q.have + j] = a.free_pages[n_free - 1 - (base + j)];
    }
    cu_s[r] = cu;
    length_s[r] = status ? -1 : q.L;
    base_s[r] = (int)min(base, (int64_t)0x7FFFFFFF);
    a.status[r] = status;
    a.cu[r] = cu;
    a.lengths_out[r] = status ? q.L : q.L + q.n;   // lengths[r] is read by this thread alone
  }
  taken = __reduce_max_sync(0xffffffffu, taken);
  if (lane == 0 && taken) atomicMax(&taken_s, taken);
  if (tid == 0) cu_s[a.R] = a.cu[a.R] = (int)min(all.tokens, (int64_t)0x7FFFFFFF);
  if (__syncthreads_or(many)) {
    // the e-th page taken goes to the last request with base <= e (one that takes none shares its base with
    // the next; behind the last placed request no base is below the pages taken)
    for (int64_t e = tid; e < taken_s; e += threads) {
      int lo = 0, hi = a.R;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (base_s[mid] <= e) lo = mid; else hi = mid;
      }
      a.table[lo * a.table_row + pages_of(length_s[lo], a.page) + e - base_s[lo]] = a.free_pages[n_free - 1 - e];
    }
    __syncthreads();
  }
  if (tid == 0) *a.n_free_out = (int32_t)(n_free - taken_s);
  if (a.max_tokens <= kFillHere)
    for (int t = tid; t < a.max_tokens; t += threads)
      put_token(a, t, t < cu_s[a.R], 0, a.R, [&](int r) { return cu_s[r]; }, [&](int r) { return length_s[r]; });
}

__global__ void __launch_bounds__(kFillThreads) fill_kernel(thin_attn_paged_plan_args a) {
  // the search begins on every step-th sum, in shared memory: its reads of the others follow one another
  __shared__ int coarse[kFillThreads];
  const int t = blockIdx.x * kFillThreads + threadIdx.x, step = (a.R + kFillThreads - 1) / kFillThreads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tokens = a.cu[a.R];
  coarse[threadIdx.x] = a.cu[min((int)threadIdx.x * step, a.R)];
  __syncthreads();
  if (t >= a.max_tokens) return;
  int lo = 0, hi = kFillThreads;   // those behind the requests are the step's tokens, above t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (coarse[mid] <= t) lo = mid; else hi = mid;
  }
  put_token(a, t, t < tokens, lo * step, min((lo + 1) * step, a.R), [&](int r) { return a.cu[r]; },
            [&](int r) { return a.status[r] ? -1 : a.lengths_out[r] - (a.cu[r + 1] - a.cu[r]); });
}

// One CTA: the released pages' prefix sums give each its place on the stack.
__global__ void __launch_bounds__(kThreads) release_kernel(thin_attn_paged_release_args a) {
  __shared__ Sums warp_sums[32];
  extern __shared__ int32_t base_s[];   // R
  const int threads = blockDim.x, per = (a.R + threads - 1) / threads;
  const int r0 = min(a.R, (int)threadIdx.x * per), r1 = min(a.R, r0 + per);
  const int64_t n_free = min(max(*a.n_free, 0), a.n_pages);
  auto kept = [&](int r, int64_t* from, int64_t* to) {
    const int64_t L = max(a.lengths[r], 0), keep = a.keep[r] < 0 ? L : min((int64_t)a.keep[r], L);
    *to = min(pages_of(L, a.page), (int64_t)a.W);
    *from = min(pages_of(keep, a.page), *to);
    return (int32_t)keep;
  };
  Sums mine = {0, 0}, all;
  int64_t from, to;
  for (int r = r0; r < r1; ++r) {
    kept(r, &from, &to);
    mine.pages += to - from;
  }
  int64_t base = block_prefix(mine, warp_sums, &all).pages;
  for (int r = r0; r < r1; ++r) {
    kept(r, &from, &to);
    base_s[r] = (int32_t)min(base, (int64_t)a.n_pages);
    base += to - from;
  }
  __syncthreads();
  for (int r = threadIdx.x >> 5; r < a.R; r += threads >> 5) {
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
  if (threadIdx.x == 0) *a.n_free = (int32_t)min(n_free + all.pages, (int64_t)a.n_pages);
}

}  // namespace

cudaError_t launch_paged_plan(const thin_attn_paged_plan_args& a, cudaStream_t st) {
  static SharedMemory memory;
  cudaError_t e = memory.allow((const void*)plan_kernel, (3 * kMaxRequests + 1) * 4);
  if (e != cudaSuccess) return e;
  const int threads = a.R <= kFewThreads && a.max_tokens <= 2 * kFewThreads ? kFewThreads : kThreads;
  plan_kernel<<<1, threads, (size_t)(3 * a.R + 1) * 4, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.max_tokens <= kFillHere) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((a.max_tokens + kFillThreads - 1) / kFillThreads);
  cfg.blockDim = dim3(kFillThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fill_kernel, a);
}

cudaError_t launch_paged_release(const thin_attn_paged_release_args& a, cudaStream_t st) {
  static SharedMemory memory;
  cudaError_t e = memory.allow((const void*)release_kernel, kMaxRequests * 4);
  if (e != cudaSuccess) return e;
  release_kernel<<<1, a.R <= kFewThreads ? kFewThreads : kThreads, (size_t)a.R * 4, st>>>(a);
  return cudaGetLastError();
}

}  // namespace thin
