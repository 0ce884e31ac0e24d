// The paged latent cache's bookkeeping and writes: block tables and slot maps
// from request lengths (mla_pages_extend, mla_pages_release), new rows into
// their slots (mla_cache_append_paged), and the per-page index that page
// selection scores (mla_page_index).
//
// "Transformer and KV Cache Basics": the cache is a preallocated buffer and
// overflowing it is an error.  Here the buffer is a pool of fixed-size pages,
// so that a sequence holds as many as its length needs.
#include <cuda_fp8.h>
#include <math.h>

#include "mla_paged.cuh"

namespace mla {

mla_status check_paging(const mla_paging* pg, const char* who) {
  if (!pg) {
    set_error("%s: paging is NULL", who);
    return MLA_ERR_INVALID_ARG;
  }
  if (pg->num_pages < 1 || pg->table_stride < 1) {
    set_error("%s: num_pages=%d and table_stride=%d must be >= 1", who, pg->num_pages,
              pg->table_stride);
    return MLA_ERR_INVALID_ARG;
  }
  if (pg->page_size < kMinPage || pg->page_size > kMaxPage ||
      (pg->page_size & (pg->page_size - 1)) != 0) {
    set_error("%s: page_size=%d is not a power of two in [%d, %d]", who, pg->page_size, kMinPage,
              kMaxPage);
    return MLA_ERR_UNSUPPORTED;
  }
  if (static_cast<long long>(pg->num_pages) * pg->page_size >= (1ll << 31) ||
      static_cast<long long>(pg->table_stride) * pg->page_size >= (1ll << 31)) {
    set_error("%s: num_pages or table_stride times page_size exceeds 2^31 rows", who);
    return MLA_ERR_UNSUPPORTED;
  }
  return MLA_OK;
}

mla_status check_io(const mla_dims* d, int32_t io_dtype, const char* who) {
  if (io_dtype != MLA_F32 && !(io_dtype == MLA_BF16 && d->dtype != MLA_F32)) {
    set_error("%s: io_dtype %d must be MLA_F32, or MLA_BF16 with a bf16 or FP8 cache", who,
              io_dtype);
    return MLA_ERR_UNSUPPORTED;
  }
  return MLA_OK;
}

namespace {

// ------------------------------------------------------------- tables and slots
// One cluster of CTAs.  Every CTA scans all requests itself (three words per
// request in shared memory: first token, first page taken, rows cached), so
// that only the writes are shared out; each token then finds its request by
// bisection.  Nothing is written before every CTA has read the inputs (the
// cluster barrier), so lengths may overwrite cached_lens and num_free_out
// num_free.  Bound by latency: two dependent rounds of loads (lengths, then
// free pages) and the barrier; the 12 bytes written per token are what grows.
constexpr int kTableThreads = 1024;
constexpr int kTableMaxBatch = 16384;
// Tokens per CTA from which another CTA of the cluster pays (a token costs its
// bisection and two stores; a CTA repeats the scan).
constexpr int kTableTokens = 4096;
constexpr int kTableMaxCtas = 8;

struct ExtendParams {
  const int32_t *cached, *fresh;
  int32_t *table, *lengths, *row_starts, *positions;
  const int32_t *free_list, *num_free;
  int32_t* num_free_out;
  int64_t* slots;
  int32_t* status;
  int B, max_tokens, page_shift, table_stride, num_pages;
};

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Exclusive prefix sums of (a, b) over the CTA's threads, and the totals.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long* tot_a,
                                            long long* tot_b, long long (*part)[32]) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  long long ia = a, ib = b;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long ya = __shfl_up_sync(0xffffffffu, ia, off);
    const long long yb = __shfl_up_sync(0xffffffffu, ib, off);
    if (lane >= off) {
      ia += ya;
      ib += yb;
    }
  }
  if (lane == 31) {
    part[0][warp] = ia;
    part[1][warp] = ib;
  }
  __syncthreads();
  if (warp == 0) {
    long long pa = lane < warps ? part[0][lane] : 0, pb = lane < warps ? part[1][lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long ya = __shfl_up_sync(0xffffffffu, pa, off);
      const long long yb = __shfl_up_sync(0xffffffffu, pb, off);
      if (lane >= off) {
        pa += ya;
        pb += yb;
      }
    }
    part[0][lane] = pa;
    part[1][lane] = pb;
  }
  __syncthreads();
  *tot_a = part[0][31];
  *tot_b = part[1][31];
  a = ia - a + (warp ? part[0][warp - 1] : 0);
  b = ib - b + (warp ? part[1][warp - 1] : 0);
}

// Last index i in [0, n) with starts[i] <= x (starts ascending, starts[0] <= x);
// among equal entries the last, so a request with nothing is never found.
__device__ __forceinline__ int bisect(const int32_t* starts, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTableThreads) pages_extend_kernel(const ExtendParams p) {
  extern __shared__ int32_t sm[];
  __shared__ long long part[2][32];
  int32_t* row_start = sm;            // [B]
  int32_t* page_start = sm + p.B;     // [B]
  int32_t* cached = sm + 2 * p.B;     // [B]
  const int tid = threadIdx.x, step = (p.B + kTableThreads - 1) / kTableThreads;
  const int b0 = min(tid * step, p.B), b1 = min(b0 + step, p.B);
  const int round_up = (1 << p.page_shift) - 1;
  const long long capacity = static_cast<long long>(p.table_stride) << p.page_shift;
  const int nf = *p.num_free;
  long long rows = 0, pages = 0;
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    const int c = p.cached[b], f = p.fresh[b];
    if (c < 0 || f < 0 || static_cast<long long>(c) + f > capacity) {
      bad = 1;
    } else {
      rows += f;
      pages += ((c + f + round_up) >> p.page_shift) - ((c + round_up) >> p.page_shift);
    }
    cached[b] = c;
    row_start[b] = f;
  }
  long long row0 = rows, page0 = pages, tot_rows, tot_pages;
  block_scan2(row0, page0, &tot_rows, &tot_pages, part);
  bad = __syncthreads_or(bad);
  const bool over = nf < 0 || nf > p.num_pages || tot_pages > nf;
  const bool ok = !bad && !over && tot_rows <= p.max_tokens;
  for (int b = b0; b < b1; ++b) {
    const int c = cached[b], f = row_start[b];
    row_start[b] = ok ? static_cast<int>(row0) : 0;
    page_start[b] = ok ? static_cast<int>(page0) : 0;
    if (ok) {
      row0 += f;
      page0 += ((c + f + round_up) >> p.page_shift) - ((c + round_up) >> p.page_shift);
    }
  }
  cluster_barrier();   // every CTA has read cached_lens, new_lens and num_free
  const int n_tok = ok ? static_cast<int>(tot_rows) : 0;
  const int n_page = ok ? static_cast<int>(tot_pages) : 0;
  const int first = blockIdx.x * kTableThreads + tid, stride = gridDim.x * kTableThreads;
  for (int b = first; b < p.B; b += stride) {
    const int end = b + 1 < p.B ? row_start[b + 1] : n_tok;
    p.lengths[b] = cached[b] + (ok ? end - row_start[b] : 0);
    p.row_starts[b] = row_start[b];
  }
  if (first == 0) {
    p.row_starts[p.B] = n_tok;
    *p.num_free_out = nf - n_page;
    if (!ok)
      report(p.status, (bad || tot_rows > p.max_tokens ? MLA_DEV_LENGTH_OUT_OF_RANGE : 0) |
                           (over ? MLA_DEV_POOL_EXHAUSTED : 0));
  }
  // The page taken k-th of all: free_list[nf - 1 - k], checked.
  auto taken = [&](int k) {
    const int id = p.free_list[nf - 1 - k];
    if (id >= 0 && id < p.num_pages) return id;
    report(p.status, MLA_DEV_PAGE_OUT_OF_RANGE);
    return -1;
  };
  for (int k = first; k < n_page; k += stride) {
    const int b = bisect(page_start, p.B, k);
    const int have = (cached[b] + round_up) >> p.page_shift;
    p.table[static_cast<size_t>(b) * p.table_stride + have + k - page_start[b]] = taken(k);
  }
  for (int t = first; t < p.max_tokens; t += stride) {
    int64_t slot = -1;
    int pos = 0;
    if (t < n_tok) {
      const int b = bisect(row_start, p.B, t);
      pos = cached[b] + t - row_start[b];
      const int have = (cached[b] + round_up) >> p.page_shift, j = pos >> p.page_shift;
      int id;
      if (j >= have) {
        id = taken(page_start[b] + j - have);
      } else {
        id = p.table[static_cast<size_t>(b) * p.table_stride + j];
        if (id < 0 || id >= p.num_pages) {
          report(p.status, MLA_DEV_PAGE_OUT_OF_RANGE);
          id = -1;
        }
      }
      if (id >= 0) slot = (static_cast<int64_t>(id) << p.page_shift) + (pos & round_up);
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
}

// Finished requests give their pages back: one CTA checks every entry it would
// push, then pushes request by request, page by page.
__global__ void __launch_bounds__(kTableThreads)
    pages_release_kernel(const int32_t* finished, int32_t* lengths, int32_t* table,
                         int32_t* free_list, int32_t* num_free, int32_t* status, int B,
                         int page_shift, int table_stride, int num_pages) {
  extern __shared__ int32_t page_start[];   // [B]
  __shared__ long long part[2][32];
  const int tid = threadIdx.x, step = (B + kTableThreads - 1) / kTableThreads;
  const int b0 = min(tid * step, B), b1 = min(b0 + step, B);
  const int round_up = (1 << page_shift) - 1;
  const int nf = *num_free;
  long long pages = 0, unused = 0, total, unused_total;
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    int n = 0;
    if (finished[b]) {
      const long long len = lengths[b];
      if (len < 0 || len > (static_cast<long long>(table_stride) << page_shift))
        bad |= MLA_DEV_LENGTH_OUT_OF_RANGE;
      else
        n = static_cast<int>((len + round_up) >> page_shift);
    }
    page_start[b] = n;
    pages += n;
  }
  long long at = pages;
  block_scan2(at, unused, &total, &unused_total, part);
  for (int b = b0; b < b1; ++b) {
    const int n = page_start[b];
    page_start[b] = static_cast<int>(min(at, 0x7fffffffll));
    at += n;
  }
  if (nf < 0 || nf + total > num_pages) bad |= MLA_DEV_POOL_EXHAUSTED;
  // A failure seen so far stops every thread before any entry is read.
  if (__syncthreads_or(bad)) {
    if (bad) report(status, bad);
    return;
  }
  const int n = static_cast<int>(total);
  for (int k = tid; k < n; k += kTableThreads) {
    const int b = bisect(page_start, B, k);
    const int id = table[static_cast<size_t>(b) * table_stride + k - page_start[b]];
    if (id < 0 || id >= num_pages) bad = MLA_DEV_PAGE_OUT_OF_RANGE;
  }
  if (__syncthreads_or(bad)) {
    if (bad) report(status, bad);
    return;
  }
  for (int k = tid; k < n; k += kTableThreads) {
    const int b = bisect(page_start, B, k);
    int32_t* e = table + static_cast<size_t>(b) * table_stride + k - page_start[b];
    free_list[nf + k] = *e;
    *e = -1;
  }
  for (int b = tid; b < B; b += kTableThreads)
    if (finished[b]) lengths[b] = 0;
  if (tid == 0) *num_free = nf + n;
}

// ------------------------------------------------------------- rows into slots
// cache[slot] = [c || RoPE(k, position)], rounded once to the cache's type.
// Bound by HBM (576 values read and written per row).  A thread moves eight
// values (16 or 32 bytes in, 8 to 32 out); 72 threads a row, the last eight of
// them the 32 RoPE pairs.  The angle of pair i at position p is p turns_i whole
// turns with turns_i = base^(-2i/64) / 2 pi held as a 64-bit fraction: the
// product modulo 2^64 drops whole turns exactly (an error of p 2^-65 turns),
// where fp64 products would run at GB300's small fp64 rate.
constexpr int kRowChunks = kRow / 8;
constexpr int kAppendThreads = 288;   // four rows
constexpr int kAppendRows = kAppendThreads / kRowChunks;

struct RopeTurns {
  uint64_t t[kDr / 2];
};

__device__ __forceinline__ void load8(const __nv_bfloat16* src, float* v) {
  const uint4 q = *reinterpret_cast<const uint4*>(src);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* src, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(src);
  const float4 b = *reinterpret_cast<const float4*>(src + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
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

template <typename In, typename Out>
__global__ void __launch_bounds__(kAppendThreads)
    append_paged_kernel(const In* __restrict__ rows, const int32_t* __restrict__ positions,
                        const int64_t* __restrict__ slots, Out* __restrict__ cache,
                        const __grid_constant__ RopeTurns turns, int32_t* status, int n,
                        int64_t pool_rows) {
  const int r = blockIdx.x * kAppendRows + threadIdx.x / kRowChunks;
  const int c = threadIdx.x % kRowChunks;
  if (r >= n) return;
  const int64_t slot = slots[r];
  float v[8];
  load8(rows + static_cast<size_t>(r) * kRow + 8 * c, v);
  const int pos = positions[r];
  if (slot < 0 || slot >= pool_rows || pos < 0) {
    if (c == 0 && slot != -1)
      report(status, slot < 0 || slot >= pool_rows ? MLA_DEV_PAGE_OUT_OF_RANGE
                                                   : MLA_DEV_LENGTH_OUT_OF_RANGE);
    return;
  }
  if (c >= kDc / 8) {
    const int i0 = 4 * (c - kDc / 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t phase = static_cast<uint64_t>(pos) * turns.t[i0 + i];
      // half turns in [-1, 1) from the phase's top 32 bits
      const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
      float sn, cs;
      sincospif(half_turns, &sn, &cs);
      const float x = v[2 * i], y = v[2 * i + 1];
      v[2 * i] = x * cs - y * sn;
      v[2 * i + 1] = x * sn + y * cs;
    }
  }
  store8(cache + static_cast<size_t>(slot) * kRow + 8 * c, v);
}

// ------------------------------------------------------------- the page index
// One CTA per touched page: the mean of its rows as 576 int8 codes and a scale.
// The sum runs in fixed point (each value rounded to 2^-20 of the power of two
// above the page's largest magnitude), so it does not depend on the order of
// its terms and every reader of the pages gets the same codes.  Bound by HBM
// (the page is read once): each thread keeps its 16-byte pieces of up to
// kIndexHold rows in registers between the maximum and the sum; pages with more
// rows per thread are read a second time, from L2.
// The conversion to integers is one fused multiply-add: x 2^(20-e) + 1.5 2^23
// leaves the integer, rounded to nearest even, in the low mantissa bits.
constexpr int kIndexHold = 16;
constexpr float kTiny = 1e-30f;   // below this a page or a query counts as zero

template <typename T>
struct IndexPlan {
  static constexpr int kVec = 16 / static_cast<int>(sizeof(T));   // columns per thread
  static constexpr int kCols = kRow / kVec;                       // threads across a row
  static constexpr int kGroups = sizeof(T) == 1 ? 8 : 4;          // row groups
  static constexpr int kThreads = kCols * kGroups;                // 288, 288, 576
};

template <typename T>
__device__ __forceinline__ void unpack16(const uint4& q, float* v);
template <>
__device__ __forceinline__ void unpack16<float>(const uint4& q, float* v) {
  v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y);
  v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
}
template <>
__device__ __forceinline__ void unpack16<__nv_bfloat16>(const uint4& q, float* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void unpack16<__nv_fp8_storage_t>(const uint4& q, float* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

struct IndexParams {
  const void* cache;
  const int32_t *table, *first_rows, *lengths;
  int8_t* codes;
  float* scales;
  int32_t* status;
  int page_shift, table_stride, num_pages, max_new;
};

// Max of x over the CTA (kThreads threads, a multiple of 32).
template <int kThreads, typename V>
__device__ __forceinline__ V block_max(V x, V* part) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, off));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  V m = part[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) m = max(m, part[w]);
  return m;
}

template <typename T>
__global__ void __launch_bounds__(IndexPlan<T>::kThreads)
    page_index_kernel(const IndexParams p) {
  using L = IndexPlan<T>;
  constexpr int kVec = L::kVec;
  __shared__ float part_f[L::kThreads / 32];
  __shared__ int part_i[L::kThreads / 32];
  __shared__ int sums[L::kGroups][kRow];
  const int b = blockIdx.y, tid = threadIdx.x;
  const int first = p.first_rows[b], len = p.lengths[b], page = 1 << p.page_shift;
  const bool bad =
      first < 0 || len < 0 || len > static_cast<long long>(p.table_stride) << p.page_shift;
  if (tid == 0 && blockIdx.x == 0 && (bad || static_cast<long long>(len) - first > p.max_new))
    report(p.status, MLA_DEV_LENGTH_OUT_OF_RANGE);
  if (bad) return;
  if (first >= len) return;
  const int j = (first >> p.page_shift) + blockIdx.x;
  const int n = min(page, len - min(len, j << p.page_shift));   // rows of this page
  if (n <= 0) return;
  const int id = p.table[static_cast<size_t>(b) * p.table_stride + j];
  if (id < 0 || id >= p.num_pages) {
    if (tid == 0) report(p.status, MLA_DEV_PAGE_OUT_OF_RANGE);
    return;
  }
  const int g = tid / L::kCols, c = tid % L::kCols;
  const T* base = static_cast<const T*>(p.cache) +
                  (static_cast<size_t>(id) << p.page_shift) * kRow + kVec * c;
  // This thread's rows: g, g + kGroups, ...
  const int mine = n > g ? (n - g + L::kGroups - 1) / L::kGroups : 0;
  uint4 hold[kIndexHold];
  float top = 0.f;
  for (int r0 = 0; r0 < mine; r0 += kIndexHold) {
#pragma unroll
    for (int u = 0; u < kIndexHold; ++u)
      hold[u] = r0 + u < mine ? *reinterpret_cast<const uint4*>(
                                    base + static_cast<size_t>(g + (r0 + u) * L::kGroups) * kRow)
                              : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < kIndexHold; ++u) {
      float v[kVec];
      unpack16<T>(hold[u], v);
#pragma unroll
      for (int i = 0; i < kVec; ++i) top = fmaxf(top, fabsf(v[i]));
    }
  }
  top = block_max<L::kThreads>(top, part_f);
  int ex = 0;
  frexpf(top, &ex);   // top = m 2^ex, m in [0.5, 1)
  const float unit = ldexpf(1.f, 20 - ex);
  const bool live = top >= kTiny && top <= 3.0e38f;
  constexpr float kMagic = 12582912.f;   // 1.5 2^23
  uint32_t sum[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) sum[i] = 0;
  const bool held = mine <= kIndexHold;
  for (int r0 = 0; r0 < mine; r0 += kIndexHold) {
#pragma unroll
    for (int u = 0; u < kIndexHold; ++u) {
      if (r0 + u >= mine) break;
      const uint4 q = held ? hold[u]
                           : *reinterpret_cast<const uint4*>(
                                 base + static_cast<size_t>(g + (r0 + u) * L::kGroups) * kRow);
      float v[kVec];
      unpack16<T>(q, v);
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        sum[i] += __float_as_uint(fmaf(v[i], unit, kMagic)) - __float_as_uint(kMagic);
    }
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) sums[g][kVec * c + i] = static_cast<int>(sum[i]);
  __syncthreads();
  int peak = 0;
  for (int d = tid; d < kRow; d += L::kThreads) {
    int s = 0;
#pragma unroll
    for (int k = 0; k < L::kGroups; ++k) s += sums[k][d];
    sums[0][d] = s;   // only this thread reads column d again
    peak = max(peak, abs(s));
  }
  peak = block_max<L::kThreads>(peak, part_i);
  const bool good = live && peak > 0;
  const float pf = static_cast<float>(peak), inv = good ? __frcp_rn(pf) * 127.f : 0.f;
  for (int d = tid; d < kRow; d += L::kThreads)
    p.codes[static_cast<size_t>(id) * kRow + d] =
        good ? static_cast<int8_t>(__float2int_rn(static_cast<float>(sums[0][d]) * inv)) : 0;
  if (tid == 0)
    p.scales[id] = good ? ldexpf(pf * (1.f / 127.f) / static_cast<float>(n), ex - 20) : 0.f;
}

template <typename T>
void launch_index(const IndexParams& p, dim3 grid, cudaStream_t s) {
  page_index_kernel<T><<<grid, IndexPlan<T>::kThreads, 0, s>>>(p);
}

// Dynamic shared memory beyond the 48 KB every kernel may use, set once per device.
template <typename K>
bool allow_smem(K kernel, size_t bytes, DeviceFlags& done) {
  const int dev = current_device();
  if (done.test(dev)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(bytes)) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  done.set(dev);
  return true;
}

mla_status check_batch(int32_t batch, const char* who) {
  if (batch < 1) {
    set_error("%s: batch=%d must be >= 1", who, batch);
    return MLA_ERR_INVALID_ARG;
  }
  if (batch > kTableMaxBatch) {
    set_error("%s: batch=%d exceeds %d requests", who, batch, kTableMaxBatch);
    return MLA_ERR_UNSUPPORTED;
  }
  return MLA_OK;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" mla_status mla_pages_extend(int32_t batch, const mla_paging* paging,
                                       const int32_t* cached_lens, const int32_t* new_lens,
                                       int32_t max_tokens, int32_t* block_table,
                                       const int32_t* free_list, const int32_t* num_free,
                                       int32_t* num_free_out, int32_t* lengths,
                                       int32_t* row_starts, int64_t* slots, int32_t* positions,
                                       int32_t* dev_status, void* stream) {
  const char* who = "mla_pages_extend";
  mla_status st = check_paging(paging, who);
  if (st == MLA_OK) st = check_batch(batch, who);
  if (st != MLA_OK) return st;
  if (max_tokens < 1) {
    set_error("%s: max_tokens=%d must be >= 1", who, max_tokens);
    return MLA_ERR_INVALID_ARG;
  }
  if (!cached_lens || !new_lens || !block_table || !free_list || !num_free || !num_free_out ||
      !lengths || !row_starts || !slots || !positions) {
    set_error("%s: a required pointer is NULL", who);
    return MLA_ERR_INVALID_ARG;
  }
  static DeviceFlags attr_done;
  if (!allow_smem(pages_extend_kernel, 3 * sizeof(int32_t) * kTableMaxBatch, attr_done)) {
    set_error("%s: cannot reserve shared memory", who);
    return MLA_ERR_CUDA;
  }
  ExtendParams p{cached_lens, new_lens, block_table, lengths, row_starts, positions,
                 free_list, num_free, num_free_out, slots, dev_status,
                 batch, max_tokens, page_shift_of(paging), paging->table_stride,
                 paging->num_pages};
  int ctas = 1;
  while (ctas < kTableMaxCtas && max_tokens > ctas * kTableTokens) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kTableThreads);
  cfg.dynamicSmemBytes = 3 * sizeof(int32_t) * batch;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, pages_extend_kernel, p);
  return launch_status(who);
}

extern "C" mla_status mla_pages_release(int32_t batch, const mla_paging* paging,
                                        const int32_t* finished, int32_t* lengths,
                                        int32_t* block_table, int32_t* free_list,
                                        int32_t* num_free, int32_t* dev_status, void* stream) {
  const char* who = "mla_pages_release";
  mla_status st = check_paging(paging, who);
  if (st == MLA_OK) st = check_batch(batch, who);
  if (st != MLA_OK) return st;
  if (!finished || !lengths || !block_table || !free_list || !num_free) {
    set_error("%s: a required pointer is NULL", who);
    return MLA_ERR_INVALID_ARG;
  }
  static DeviceFlags attr_done;
  if (!allow_smem(pages_release_kernel, sizeof(int32_t) * kTableMaxBatch, attr_done)) {
    set_error("%s: cannot reserve shared memory", who);
    return MLA_ERR_CUDA;
  }
  pages_release_kernel<<<1, kTableThreads, sizeof(int32_t) * batch,
                         static_cast<cudaStream_t>(stream)>>>(
      finished, lengths, block_table, free_list, num_free, dev_status, batch,
      page_shift_of(paging), paging->table_stride, paging->num_pages);
  return launch_status(who);
}

extern "C" mla_status mla_cache_append_paged(const mla_dims* dims, const mla_paging* paging,
                                             int32_t num_rows, int32_t row_dtype,
                                             const void* rows, const int32_t* positions,
                                             const int64_t* slots, double rope_base, void* cache,
                                             int32_t* dev_status, void* stream) {
  const char* who = "mla_cache_append_paged";
  mla_status st = check_dims(dims, who);
  if (st == MLA_OK) st = check_paging(paging, who);
  if (st != MLA_OK) return st;
  if (num_rows < 0 || !(rope_base > 0.0) || !isfinite(rope_base)) {
    set_error("%s: num_rows=%d must be >= 0 and rope_base finite and > 0", who, num_rows);
    return MLA_ERR_INVALID_ARG;
  }
  if (row_dtype != MLA_F32 && !(row_dtype == MLA_BF16 && dims->dtype != MLA_F32)) {
    set_error("%s: row_dtype %d must be MLA_F32, or MLA_BF16 with a bf16 or FP8 cache", who,
              row_dtype);
    return MLA_ERR_UNSUPPORTED;
  }
  if (num_rows == 0) return MLA_OK;
  if (!rows || !positions || !slots || !cache || !aligned16(rows) || !aligned16(cache)) {
    set_error("%s: pointers must not be NULL, rows and cache 16-byte aligned", who);
    return MLA_ERR_INVALID_ARG;
  }
  RopeTurns turns;
  for (int i = 0; i < kDr / 2; ++i) {
    const double t = pow(rope_base, -2.0 * i / kDr) / 6.283185307179586476925;
    // the fraction of a turn per position; a base below 1 has whole turns to drop
    turns.t[i] = static_cast<uint64_t>(ldexp(t - floor(t), 64));
  }
  const dim3 grid((num_rows + kAppendRows - 1) / kAppendRows);
  const int64_t pool = static_cast<int64_t>(paging->num_pages) * paging->page_size;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32_rows = row_dtype == MLA_F32;
  auto go = [&](auto* in, auto* out) {
    append_paged_kernel<<<grid, kAppendThreads, 0, s>>>(in, positions, slots, out, turns,
                                                        dev_status, num_rows, pool);
  };
  const float* in_f = static_cast<const float*>(rows);
  const __nv_bfloat16* in_b = static_cast<const __nv_bfloat16*>(rows);
  if (dims->dtype == MLA_F32) {
    go(in_f, static_cast<float*>(cache));
  } else if (dims->dtype == MLA_BF16) {
    f32_rows ? go(in_f, static_cast<__nv_bfloat16*>(cache))
             : go(in_b, static_cast<__nv_bfloat16*>(cache));
  } else {
    f32_rows ? go(in_f, static_cast<__nv_fp8_storage_t*>(cache))
             : go(in_b, static_cast<__nv_fp8_storage_t*>(cache));
  }
  return launch_status(who);
}

extern "C" mla_status mla_page_index(const mla_dims* dims, const mla_paging* paging,
                                     int32_t max_new, const void* cache,
                                     const int32_t* block_table, const int32_t* first_rows,
                                     const int32_t* lengths, int8_t* codes, float* scales,
                                     int32_t* dev_status, void* stream) {
  const char* who = "mla_page_index";
  mla_status st = check_dims(dims, who);
  if (st == MLA_OK) st = check_paging(paging, who);
  if (st != MLA_OK) return st;
  if (max_new < 1 || dims->batch > 65535) {
    set_error("%s: max_new=%d must be >= 1 and batch=%d <= 65535", who, max_new, dims->batch);
    return MLA_ERR_INVALID_ARG;
  }
  if (!cache || !block_table || !first_rows || !lengths || !codes || !scales ||
      !aligned16(cache) || !aligned16(codes)) {
    set_error("%s: pointers must not be NULL, cache and codes 16-byte aligned", who);
    return MLA_ERR_INVALID_ARG;
  }
  IndexParams p{cache, block_table, first_rows, lengths, codes, scales, dev_status,
                page_shift_of(paging), paging->table_stride, paging->num_pages, max_new};
  // A request's max_new rows touch at most this many pages.
  const long long most = (static_cast<long long>(max_new) + paging->page_size - 2) / paging->page_size + 1;
  const dim3 grid(static_cast<unsigned>(most < paging->table_stride ? most : paging->table_stride),
                  dims->batch);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dims->dtype == MLA_F32)
    launch_index<float>(p, grid, s);
  else if (dims->dtype == MLA_BF16)
    launch_index<__nv_bfloat16>(p, grid, s);
  else
    launch_index<__nv_fp8_storage_t>(p, grid, s);
  return launch_status(who);
}
