// Launchers of the paged-cache operators (internal).  The argument structs are the C ABI's, checked.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "thin_attn.h"

namespace thin {

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
