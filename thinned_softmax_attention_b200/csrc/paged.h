// Launchers of the paged-cache operators (internal).  The argument structs are the C ABI's, checked.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "thin_attn.h"

namespace thin {

// Lets `kernel` have up to `most` bytes of dynamic shared memory on the current device.  `most` is the same
// at every call, so that calls from several threads cannot take the room from one another; the
// runtime is asked once per device.
class SharedMemory {
 public:
  cudaError_t allow(const void* kernel, int most) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < kDevices && granted_[dev].load(std::memory_order_acquire))) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess && dev < kDevices) granted_[dev].store(true, std::memory_order_release);
    return e;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<bool> granted_[kDevices] = {};
};

constexpr int kMaxRequests = 16384;   // of a plan, which keeps its sums in shared memory
constexpr int kMaxGroup = 256;        // queries of a key head for page selection, for the same reason

cudaError_t launch_paged_plan(const thin_attn_paged_plan_args& a, cudaStream_t st);
cudaError_t launch_paged_release(const thin_attn_paged_release_args& a, cudaStream_t st);
cudaError_t launch_paged_append(const thin_attn_paged_append_args& a, cudaStream_t st);

// One launch of attention over lists of pages: token n and key head h read `ids` entries
// list(n) * ids_token + h * ids_head .. of page ids, the first keys[n] keys of them.
struct PagedAttn {
  thin_attn_paged_attention_args a;
  const int32_t* ids;
  int64_t ids_token, ids_head;
  int list_rows;          // 1: list(n) = rows[n], 0: list(n) = n
  int list_width;         // ids per list
  bool follows;           // launched behind the selection on the same stream: may be set up while that runs
  const int32_t* keys;    // (N)
  float scale_log2e;
  uint32_t page_mul;      // key / page = umulhi(key, page_mul) >> page_shift, page_mul = 0 for page = 1
  int page_shift;
};
size_t paged_attention_workspace(const thin_attn_paged_attention_args& a);
cudaError_t launch_paged_attention(const PagedAttn& p, void* workspace, cudaStream_t st);

// Page selection: per token and key head the chosen pages' ids (lists of `top`), and per token the
// keys they hold.
size_t paged_select_workspace(const thin_attn_paged_attention_args& a);
cudaError_t launch_paged_select(const thin_attn_paged_attention_args& a, int32_t* ids, int32_t* keys, void* workspace,
                                cudaStream_t st);

}  // namespace thin
