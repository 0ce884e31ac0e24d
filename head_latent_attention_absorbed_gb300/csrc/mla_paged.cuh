// Shared by the calls on the paged latent cache: the argument checks and the
// lookup of a page.
#pragma once

#include "mla_common.cuh"

namespace mla {

constexpr int kMinPage = 16, kMaxPage = 256;   // rows per page, a power of two

// page_size a power of two in [16, 256], num_pages >= 1, table_stride >= 1, and
// pool rows that fit a 32-bit TMA coordinate.
mla_status check_paging(const mla_paging* pg, const char* who);

inline int page_shift_of(const mla_paging* pg) {
  int s = 0;
  while ((1 << s) < pg->page_size) ++s;
  return s;
}

// Query and output type of the paged calls against the cache's type: fp32 with
// every cache, bf16 with a bf16 or E4M3 cache.
mla_status check_io(const mla_dims* d, int32_t io_dtype, const char* who);

// What the paged attention calls check of their sizes (mla_decode.cu).
mla_status check_paged(const char* who, const mla_dims* dims, const mla_paging* paging,
                       int32_t io_dtype, int32_t q_len);

// The workspace of the attention over a page selection (mla_decode.cu).
size_t selected_workspace_bytes(const char* who, const mla_dims* dims, const mla_paging* paging,
                                int32_t io_dtype, int32_t requested);
// Its argument checks, without a launch.
mla_status check_attn_selected(const char* who, const mla_dims* dims, const mla_paging* paging,
                            int32_t io_dtype, const void* q_abs, const void* q_pe,
                            const void* cache, const int32_t* block_table,
                            const int32_t* lengths, float softmax_scale, int32_t num_splits,
                            void* workspace, size_t ws_bytes, void* o_c);

// mla_decode_attn_paged with q_len 1 in two steps around the selection of its pages, the
// arguments checked: attn_queries makes the queries' FP8 codes (E4M3 caches; nothing
// otherwise), attn_selected does the rest, launched to start early under the kernel that
// writes sel_table and sel_lengths.
mla_status attn_queries(const char* who, const mla_dims* dims, const mla_paging* paging,
                        int32_t io_dtype, const void* q_abs, const void* q_pe,
                        const int32_t* lengths, int32_t num_splits, void* workspace,
                        size_t ws_bytes, void* stream);
mla_status attn_selected(const char* who, const mla_dims* dims, const mla_paging* paging,
                         int32_t io_dtype, const void* q_abs, const void* q_pe,
                         const void* cache, const int32_t* sel_table,
                         const int32_t* sel_lengths, float softmax_scale, int32_t num_splits,
                         void* workspace, size_t ws_bytes, void* o_c, float* lse,
                         int32_t* dev_status, void* stream);

}  // namespace mla
