// Shared by the calls on the paged latent cache: the argument checks and the
// lookup of a page.
#pragma once

#include <cuda_fp8.h>
#include <math.h>

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
// every cache, bf16 with a bf16, E4M3 or 4-bit cache.
mla_status check_io(const mla_dims* d, int32_t io_dtype, const char* who);

// The 4-bit forms of mla_cache_append_paged and mla_page_index, arguments checked (mla_q4.cu;
// `most`: pages that a request's max_new rows can touch).
mla_status append_q4(const char* who, const mla_paging* paging, int num_rows, bool f32_rows,
                     const void* rows, const int32_t* positions, const int64_t* slots,
                     double rope_base, void* cache, int32_t* status, cudaStream_t s);
mla_status page_index_q4(const char* who, const mla_paging* paging, int batch, int max_new, int most,
                         const void* cache, const int32_t* table, const int32_t* first_rows,
                         const int32_t* lengths, int8_t* codes, float* scales, int32_t* status,
                         cudaStream_t s);

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

// ------------------------------------------------------------- rows in and out
// What one lane holds of a row where a warp moves it: values 8 l .. and 256 + 8 l .., and the
// key's pair l.
struct RopeTurns {
  uint64_t t[kDr / 2];
};

// Eight values as loaded, and as fp32.
struct Raw8bf16 {
  uint4 q;
  __device__ __forceinline__ void load(const __nv_bfloat16* src) {
    q = __ldcs(reinterpret_cast<const uint4*>(src));
  }
  __device__ __forceinline__ void values(float* v) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
struct Raw8f32 {
  float4 a, b;
  __device__ __forceinline__ void load(const float* src) {
    a = __ldcs(reinterpret_cast<const float4*>(src));
    b = __ldcs(reinterpret_cast<const float4*>(src + 4));
  }
  __device__ __forceinline__ void values(float* v) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> : Raw8bf16 {};
template <>
struct Raw8<float> : Raw8f32 {};
__device__ __forceinline__ void store8(float* dst, const float* v) {
  *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(dst + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* dst, const float* v) {
  *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                              pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store8(__nv_fp8_storage_t* dst, const float* v) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {   // nearest even, saturating at +-448
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | hi << 16;
  }
  *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float2 load_pair(const __nv_bfloat16* src) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(src));
}
__device__ __forceinline__ float2 load_pair(const float* src) {
  return *reinterpret_cast<const float2*>(src);
}
__device__ __forceinline__ void store_pair(float* dst, float x, float y) {
  *reinterpret_cast<float2*>(dst) = make_float2(x, y);
}
__device__ __forceinline__ void store_pair(__nv_bfloat16* dst, float x, float y) {
  *reinterpret_cast<uint32_t*>(dst) = pack_bf16(x, y);
}
__device__ __forceinline__ void store_pair(__nv_fp8_storage_t* dst, float x, float y) {
  *reinterpret_cast<uint16_t*>(dst) =
      __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}

// The turns of each pair per position (see append_paged_kernel); a thread keeps the last base's,
// whose powers take longer than the rest of a call.
inline const RopeTurns& rope_turns(double rope_base) {
  thread_local double base = 0.0;
  thread_local RopeTurns turns;
  if (base == rope_base) return turns;
  base = rope_base;
  for (int i = 0; i < kDr / 2; ++i) {
    const double t = pow(rope_base, -2.0 * i / kDr) / 6.283185307179586476925;
    // the fraction of a turn per position; a base below 1 has whole turns to drop
    turns.t[i] = static_cast<uint64_t>(ldexp(t - floor(t), 64));
  }
  return turns;
}
__device__ __forceinline__ float2 rotated(float2 pair, int pos, uint64_t turn) {
  // half turns in [-1, 1) from the phase's top 32 bits
  const uint64_t phase = static_cast<uint64_t>(pos) * turn;
  const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
  float sn, cs;
  sincospif(half_turns, &sn, &cs);
  return make_float2(pair.x * cs - pair.y * sn, pair.x * sn + pair.y * cs);
}

}  // namespace mla
