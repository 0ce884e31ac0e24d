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
// Steps of up to kTableSingles tokens: one cluster of CTAs, a token per thread.
// Every CTA scans all requests itself (three words per request in shared memory:
// first token, first page taken, rows cached), so that only the writes are shared
// out; each token then finds its request by bisection.  Nothing is written before
// every CTA has read the inputs (the cluster barrier), so lengths may overwrite
// cached_lens and num_free_out num_free.  Bound by latency: two dependent rounds of
// loads (lengths, then pages) and the barrier.
// More tokens: the same kernel as one CTA leaves the tokens to a second one over
// the whole GPU, which reads the finished tables (262 k tokens of 256 requests: 27.3
// us as one cluster of eight CTAs, 17.8 with four tokens a thread).
constexpr int kTableThreads = 1024;
constexpr int kTableMaxBatch = 16384;
constexpr int kTableMaxCtas = 8;
constexpr int kTableSingles = kTableThreads * kTableMaxCtas;

struct ExtendParams {
  const int32_t *cached, *fresh;
  int32_t *table, *lengths, *row_starts, *positions;
  const int32_t *free_list, *num_free;
  int32_t* num_free_out;
  int64_t* slots;
  int32_t* status;
  int B, max_tokens, page_shift, table_stride, num_pages;
  int fill;   // slots and positions this kernel writes: max_tokens, or 0
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
  for (int t = first; t < p.fill; t += stride) {
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

// Slots and positions of many tokens from the tables pages_extend_kernel left: four
// consecutive tokens a thread, which mostly share a bisection and a page lookup.
constexpr int kSlotThreads = 256, kSlotEach = 4;
__global__ void __launch_bounds__(kSlotThreads) slots_kernel(const ExtendParams p) {
  const int t0 = kSlotEach * (blockIdx.x * kSlotThreads + threadIdx.x);
  pdl_wait();   // row_starts, lengths and the table
  if (t0 >= p.max_tokens) return;
  const int n_tok = p.row_starts[p.B], mask = (1 << p.page_shift) - 1;
  int b = 0, end = 0, back = 0;   // the request of the last token, its end, and end - position
  int64_t base = -1, slot[kSlotEach];
  int pos[kSlotEach];
#pragma unroll
  for (int u = 0; u < kSlotEach; ++u) {
    const int t = t0 + u;
    slot[u] = -1;
    pos[u] = 0;
    if (t >= n_tok) continue;
    const bool other = t >= end;
    if (other) {
      b = bisect(p.row_starts, p.B, t);
      end = p.row_starts[b + 1];
      back = p.lengths[b] - end;
    }
    pos[u] = t + back;
    if (other || (pos[u] & mask) == 0) {
      const int id = p.table[static_cast<size_t>(b) * p.table_stride + (pos[u] >> p.page_shift)];
      base = id < 0 || id >= p.num_pages ? -1 : static_cast<int64_t>(id) << p.page_shift;
      if (base < 0) report(p.status, MLA_DEV_PAGE_OUT_OF_RANGE);
    }
    if (base >= 0) slot[u] = base + (pos[u] & mask);
  }
  const bool wide = ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions)) &
                     15) == 0;
  if (wide && t0 + kSlotEach <= p.max_tokens) {
    longlong2* s = reinterpret_cast<longlong2*>(p.slots + t0);
    s[0] = make_longlong2(slot[0], slot[1]);
    s[1] = make_longlong2(slot[2], slot[3]);
    *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    return;
  }
  for (int u = 0; u < kSlotEach && t0 + u < p.max_tokens; ++u) {
    p.slots[t0 + u] = slot[u];
    p.positions[t0 + u] = pos[u];
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
// Bound by HBM (576 values read and written per row).  A warp moves a row: each
// lane sixteen of the 512 latent values and one RoPE pair, so that a row costs one
// sine and cosine per lane (with 72 threads of eight values a row, the eight that
// held the pairs ran four each while their warps waited: 62281 bf16 rows into an
// E4M3 cache took 27.0 us).  kAppendEach rows' loads are in flight per warp.  The
// angle of pair i at position p is p turns_i whole turns with
// turns_i = base^(-2i/64) / 2 pi held as a 64-bit fraction: the product modulo 2^64
// drops whole turns exactly (an error of p 2^-65 turns), where fp64 products would
// run at GB300's small fp64 rate.
constexpr int kAppendWarps = 8;
constexpr int kAppendEach = 4;
constexpr int kAppendRows = kAppendWarps * kAppendEach;

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

template <typename In, typename Out>
__global__ void __launch_bounds__(32 * kAppendWarps)
    append_paged_kernel(const In* __restrict__ rows, const int32_t* __restrict__ positions,
                        const int64_t* __restrict__ slots, Out* __restrict__ cache,
                        const __grid_constant__ RopeTurns turns, int32_t* status, int n,
                        int64_t pool_rows) {
  const int lane = threadIdx.x & 31;
  const int r0 = blockIdx.x * kAppendRows + (threadIdx.x >> 5);
  int64_t slot[kAppendEach];
  int pos[kAppendEach];
  Raw8<In> raw[kAppendEach][2];
  float2 pair[kAppendEach];
#pragma unroll
  for (int u = 0; u < kAppendEach; ++u) {
    const int r = r0 + u * kAppendWarps;
    slot[u] = -1;
    pos[u] = 0;
    if (r < n) {
      const In* row = rows + static_cast<size_t>(r) * kRow;
      slot[u] = slots[r];
      pos[u] = positions[r];
      raw[u][0].load(row + 8 * lane);
      raw[u][1].load(row + 256 + 8 * lane);
      pair[u] = load_pair(row + kDc + 2 * lane);
    }
  }
  const uint64_t turn = turns.t[lane];
#pragma unroll
  for (int u = 0; u < kAppendEach; ++u) {
    if (slot[u] < 0 || slot[u] >= pool_rows || pos[u] < 0) {
      if (lane == 0 && slot[u] != -1)
        report(status, slot[u] < 0 || slot[u] >= pool_rows ? MLA_DEV_PAGE_OUT_OF_RANGE
                                                           : MLA_DEV_LENGTH_OUT_OF_RANGE);
      continue;
    }
    Out* dst = cache + static_cast<size_t>(slot[u]) * kRow;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float v[8];
      raw[u][i].values(v);
      store8(dst + 256 * i + 8 * lane, v);
    }
    // half turns in [-1, 1) from the phase's top 32 bits
    const uint64_t phase = static_cast<uint64_t>(pos[u]) * turn;
    const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
    float sn, cs;
    sincospif(half_turns, &sn, &cs);
    store_pair(dst + kDc + 2 * lane, pair[u].x * cs - pair[u].y * sn,
               pair[u].x * sn + pair[u].y * cs);
  }
}

// ------------------------------------------------------------- the page index
// Per touched page, the mean of its rows as 576 int8 codes and a scale.  The sum
// runs in fixed point (each value rounded to 2^-20 of the power of two above the
// page's largest magnitude), so it does not depend on the order of its terms and
// every reader of the pages gets the same codes.
// Bound by HBM (the page is read once).  One CTA per SM works through the pages.
// Two groups of worker warps take pages in turn, each with a stage of shared
// memory that a producer warp fills (a page is contiguous: one bulk copy): a group
// takes its stage into registers, gives it back at once, and then finds the
// maximum, sums and writes while the stage fills again and the other group works.
// (4096 pages of 64 bf16 rows: 72.7 us with a CTA per page and its pieces loaded
// straight into registers, where loads and arithmetic take turns; 62.4 with one
// group of 576 workers, whose barriers nothing fills.)
// Pages larger than a stage go through it in parts, twice: once for the maximum,
// once (from L2) for the sum.
// The conversion to integers is one fused multiply-add: x 2^(20-e) + 1.5 2^23
// leaves the integer, rounded to nearest even, in the low mantissa bits.
constexpr int kIndexHold = 16;       // 16-byte pieces of a stage per thread
constexpr int kIndexWorkers = 288;   // threads of a worker group
constexpr int kIndexTeams = 2;       // worker groups, one stage each
constexpr int kIndexThreads = kIndexTeams * kIndexWorkers + 32;
constexpr int kIndexStageBytes = kIndexHold * kIndexWorkers * 16;   // 73,728
constexpr float kTiny = 1e-30f;   // below this a page or a query counts as zero

template <typename T>
struct IndexPlan {
  static constexpr int kVec = 16 / static_cast<int>(sizeof(T));   // columns per thread
  static constexpr int kCols = kRow / kVec;                       // threads across a row
  static constexpr int kGroups = kIndexWorkers / kCols;           // row groups: 8, 4, 2
  static constexpr int kPartRows = kIndexHold * kGroups;          // rows of a stage: 128, 64, 32
  static constexpr size_t kTeamSmem = kIndexStageBytes + kGroups * kRow * sizeof(int);
  static constexpr size_t kSmem = kIndexTeams * kTeamSmem;
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

// What a stage holds: rows of page `id`, and the steps they end.
enum { kPartMax = 1, kPartSum = 2, kPartMaxDone = 4, kPartSumDone = 8 };
struct IndexPart {
  int id;      // page, -1: no more
  int rows;    // rows in the stage
  int n;       // rows of the page inside its sequence
  int steps;   // kPart bits
};

// Max of x over a worker group (named barrier `bar`).
template <typename V>
__device__ __forceinline__ V workers_max(V x, V* part, int bar) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, off));
  if ((threadIdx.x & 31) == 0) part[(threadIdx.x % kIndexWorkers) >> 5] = x;
  named_bar_sync(bar, kIndexWorkers);
  const int lane = threadIdx.x & 31;
  x = lane < kIndexWorkers / 32 ? part[lane] : part[0];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

// Whether `ok` holds for every worker of a group (named barrier `bar`).
__device__ __forceinline__ bool workers_all(bool ok, int bar) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, %3, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(ok)), "n"(kIndexWorkers), "r"(bar)
      : "memory");
  return r != 0;
}

// Items: page jj of request b's touched ones, item = b * most + jj, dealt to the
// CTAs in turn.
template <typename T>
__global__ void __launch_bounds__(kIndexThreads, 1)
    page_index_kernel(const IndexParams p, int B, int most) {
  using L = IndexPlan<T>;
  constexpr int kVec = L::kVec, kRowBytes = kRow * static_cast<int>(sizeof(T));
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float part_f[kIndexTeams][kIndexWorkers / 32];
  __shared__ int part_i[kIndexTeams][kIndexWorkers / 32];
  __shared__ IndexPart parts[kIndexTeams];
  __shared__ __align__(8) uint64_t s_bar[2 * kIndexTeams];   // full, empty
  const uint32_t bars = smem_u32(s_bar);
  const int tid = threadIdx.x, lane = tid & 31;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (kIndexTeams + s); };
  if (tid == 0) {
    for (int s = 0; s < kIndexTeams; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kIndexWorkers / 32);
    }
    fence_mbarrier_init();
  }
  __syncthreads();
  if (tid >= kIndexTeams * kIndexWorkers) {
    // ------------------------------------------------------------ producer warp
    const int page = 1 << p.page_shift;
    const long long items = static_cast<long long>(B) * most;
    int uses[kIndexTeams] = {};   // stages handed over
    int team = 0;                 // of the next page
    bool go = true;
    // One stage to `team`: `rows` rows from row `row` of page `id` (id < 0: the end).
    auto hand_over = [&](int s, int id, int row, int rows, int n, int steps) {
      if (uses[s] > 0 && !mbar_wait_bounded(empty(s), (uses[s] - 1) & 1)) {
        go = false;
        return;
      }
      parts[s] = IndexPart{id, rows, n, steps};
      const uint32_t bytes = id < 0 ? 0 : static_cast<uint32_t>(rows) * kRowBytes;
      mbar_arrive_expect_tx(full(s), bytes);
      if (id >= 0)
        bulk_g2s(smem_u32(smem) + s * static_cast<uint32_t>(L::kTeamSmem),
                 static_cast<const T*>(p.cache) +
                     ((static_cast<size_t>(id) << p.page_shift) + row) * kRow,
                 bytes, full(s));
      ++uses[s];
    };
    for (long long base = blockIdx.x; base < items && go;
         base += 32ll * gridDim.x) {
      // Lane l looks item base + l * gridDim.x up.
      const long long item = base + static_cast<long long>(lane) * gridDim.x;
      int id = -1, n = 0;
      if (item < items) {
        const int b = static_cast<int>(item / most), jj = static_cast<int>(item % most);
        const int first = p.first_rows[b], len = p.lengths[b];
        const bool bad = first < 0 || len < 0 ||
                         len > static_cast<long long>(p.table_stride) << p.page_shift;
        if (jj == 0 && (bad || static_cast<long long>(len) - first > p.max_new))
          report(p.status, MLA_DEV_LENGTH_OUT_OF_RANGE);
        const long long j = static_cast<long long>(first >> p.page_shift) + jj;
        if (!bad && first < len && (j << p.page_shift) < len) {
          n = static_cast<int>(min(static_cast<long long>(page), len - (j << p.page_shift)));
          id = p.table[static_cast<size_t>(b) * p.table_stride + j];
          if (id < 0 || id >= p.num_pages) {
            report(p.status, MLA_DEV_PAGE_OUT_OF_RANGE);
            id = -1;
          }
        }
      }
      for (int l = 0; l < 32; ++l) {
        const int the_id = __shfl_sync(0xffffffffu, id, l), the_n = __shfl_sync(0xffffffffu, n, l);
        if (the_id < 0 || lane != 0 || !go) continue;
        const int s = team;
        team = (team + 1) % kIndexTeams;
        if (the_n <= L::kPartRows) {
          hand_over(s, the_id, 0, the_n, the_n, kPartMax | kPartSum | kPartMaxDone | kPartSumDone);
          continue;
        }
        for (int half = 0; half < 2; ++half)
          for (int r = 0; r < the_n && go; r += L::kPartRows) {
            const bool last = r + L::kPartRows >= the_n;
            hand_over(s, the_id, r, min(L::kPartRows, the_n - r), the_n,
                      half == 0 ? kPartMax | (last ? kPartMaxDone : 0)
                                : kPartSum | (last ? kPartSumDone : 0));
          }
      }
      go = __shfl_sync(0xffffffffu, go, 0);
    }
    if (lane == 0) {
      for (int s = 0; s < kIndexTeams && go; ++s) hand_over(s, -1, 0, 0, 0, 0);
      // Copies still in flight land before the CTA may leave.
      for (int s = 0; s < kIndexTeams; ++s)
        if (uses[s] > 0) go = mbar_wait_bounded(full(s), (uses[s] - 1) & 1) && go;
      if (!go) report(p.status, MLA_DEV_PIPELINE_TIMEOUT);
    }
    return;
  }
  // -------------------------------------------------------------- workers
  const int team = tid / kIndexWorkers, w = tid % kIndexWorkers;
  const int g = w / L::kCols, c = w % L::kCols;
  uint8_t* stage = smem + team * L::kTeamSmem;
  int (*sums)[kRow] = reinterpret_cast<int (*)[kRow]>(stage + kIndexStageBytes);
  const int bar = 1 + team, vote = 1 + kIndexTeams + team;
  constexpr float kMagic = 12582912.f;   // 1.5 2^23
  float top = 0.f, unit = 0.f;
  int ex = 0;
  bool live = false;
  uint32_t sum[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) sum[i] = 0;
  for (int use = 0;; ++use) {
    if (!workers_all(mbar_wait_bounded(full(team), use & 1), vote)) return;
    const IndexPart part = parts[team];
    if (part.id < 0) return;
    uint4 hold[kIndexHold];   // rows g, g + kGroups, ... of the stage
#pragma unroll
    for (int u = 0; u < kIndexHold; ++u) {
      const int r = g + u * L::kGroups;
      hold[u] = r < part.rows
                    ? *reinterpret_cast<const uint4*>(stage + r * kRowBytes + 16 * c)
                    : make_uint4(0, 0, 0, 0);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty(team));
    if (part.steps & kPartMax) {
#pragma unroll
      for (int u = 0; u < kIndexHold; ++u) {
        float v[kVec];
        unpack16<T>(hold[u], v);
#pragma unroll
        for (int i = 0; i < kVec; ++i) top = fmaxf(top, fabsf(v[i]));
      }
    }
    if (part.steps & kPartMaxDone) {
      top = workers_max(top, part_f[team], bar);
      frexpf(top, &ex);   // top = m 2^ex, m in [0.5, 1)
      unit = ldexpf(1.f, 20 - ex);
      live = top >= kTiny && top <= 3.0e38f;
      top = 0.f;
    }
    if (part.steps & kPartSum) {
      // Rows past the part's end are zeros here and add none.
#pragma unroll
      for (int u = 0; u < kIndexHold; ++u) {
        float v[kVec];
        unpack16<T>(hold[u], v);
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          sum[i] += __float_as_uint(fmaf(v[i], unit, kMagic)) - __float_as_uint(kMagic);
      }
    }
    if (part.steps & kPartSumDone) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        sums[g][kVec * c + i] = static_cast<int>(sum[i]);
        sum[i] = 0;
      }
      named_bar_sync(bar, kIndexWorkers);
      int total[2] = {0, 0};   // of columns w and w + 288
#pragma unroll
      for (int k = 0; k < L::kGroups; ++k) {
        total[0] += sums[k][w];
        total[1] += sums[k][w + kIndexWorkers];
      }
      const int peak = workers_max(max(abs(total[0]), abs(total[1])), part_i[team], bar);
      const bool good = live && peak > 0;
      const float pf = static_cast<float>(peak), inv = good ? __frcp_rn(pf) * 127.f : 0.f;
      int8_t* out = p.codes + static_cast<size_t>(part.id) * kRow;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        out[w + i * kIndexWorkers] =
            good ? static_cast<int8_t>(__float2int_rn(static_cast<float>(total[i]) * inv)) : 0;
      if (w == 0)
        p.scales[part.id] =
            good ? ldexpf(pf * (1.f / 127.f) / static_cast<float>(part.n), ex - 20) : 0.f;
    }
  }
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

template <typename T>
mla_status launch_index(const IndexParams& p, int B, int most, cudaStream_t s, const char* who) {
  static DeviceFlags attr_done;
  int dev = 0, sms = 0;
  if (!allow_smem(page_index_kernel<T>, IndexPlan<T>::kSmem, attr_done) ||
      cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    set_error("%s: cannot reserve shared memory", who);
    return MLA_ERR_CUDA;
  }
  const long long items = static_cast<long long>(B) * most;
  page_index_kernel<T><<<static_cast<unsigned>(items < sms ? items : sms), kIndexThreads,
                         IndexPlan<T>::kSmem, s>>>(p, B, most);
  return launch_status(who);
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
                 paging->num_pages, max_tokens <= kTableSingles ? max_tokens : 0};
  int ctas = 1;
  while (ctas < kTableMaxCtas && p.fill > ctas * kTableThreads) ctas *= 2;
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
  if (p.fill == 0) {
    const int per_cta = kSlotThreads * kSlotEach;
    launch_pdl(slots_kernel, dim3((max_tokens + per_cta - 1) / per_cta), dim3(kSlotThreads), 0,
               cfg.stream, p);
  }
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
    append_paged_kernel<<<grid, 32 * kAppendWarps, 0, s>>>(in, positions, slots, out, turns,
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
  if (max_new < 1) {
    set_error("%s: max_new=%d must be >= 1", who, max_new);
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
  const int touched = static_cast<int>(most < paging->table_stride ? most : paging->table_stride);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dims->dtype == MLA_F32) return launch_index<float>(p, dims->batch, touched, s, who);
  if (dims->dtype == MLA_BF16) return launch_index<__nv_bfloat16>(p, dims->batch, touched, s, who);
  return launch_index<__nv_fp8_storage_t>(p, dims->batch, touched, s, who);
}
