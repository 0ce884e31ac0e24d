// Rows into a 4-bit pool and out of any: the 4-bit form of mla_cache_append_paged,
// mla_cache_read_paged for every pool, and the page index over 4-bit pages.
#include <type_traits>

#include "mla_q4.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;

// ------------------------------------------------------------- rows into slots
// 576 values read, 400 bytes written per row: bound by HBM for fp32 rows, and for bf16 rows as much
// by the instructions that quantise them.  A warp moves a row, as in append_paged_kernel,
// kAppendEach rows' loads in flight; two lanes share a block of 16 latents, so its largest
// magnitude is one exchange, and four a byte of exponents.  62281 rows: bf16 19.0 us, 0.75 of the
// measured copy bandwidth, fp32 27.0, 0.92.  (When these took 18.0 and 26.3, over one copy of the rows:
// four rows a warp and eight warps a CTA, whose last wave is long, fp32 30.4, 1000 bf16 rows 2.9 for 1.9.  bf16 values widened before they are
// compared and scaled: 19.1.  A grid that the SMs hold at once, each warp with its next row's
// loads out while it writes one: 26.7.)
constexpr int kAppendEach = 2, kAppendWarps = 4, kAppendRows = kAppendWarps * kAppendEach;

// Eight values times 2^-e (exact), as codes: to nearest even, saturating at 6.
__device__ __forceinline__ uint32_t q4_encode(const float* y) {
  uint32_t code = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    code |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(y[2 * k], y[2 * k + 1]),
                                                           __NV_E2M1, cudaRoundNearest)) << (8 * k);
  return q4_page_word(code);
}
// A lane's 2 x 8 values of a row, of two blocks that it shares with its neighbour: their codes as
// a page holds them, and (e + 5) mod 16 in a byte for each block.  A block's e is two below the
// exponent of its largest magnitude, or one where the mantissa is above 7/4, between -8 and 6; as
// integers, NaN counts above infinity, and both take the largest e.  (bf16: both blocks' magnitudes
// and exponents in halves of a word.)
__device__ __forceinline__ uint32_t q4_quantise(const Raw8bf16 (&x)[2], uint32_t* codes) {
  constexpr uint32_t kAbs = 0x7fff7fffu, kOne = 0x00010001u;
  uint32_t m[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    m[i] = __vmaxu2(__vmaxu2(x[i].q.x & kAbs, x[i].q.y & kAbs),
                    __vmaxu2(x[i].q.z & kAbs, x[i].q.w & kAbs));
  uint32_t top = __vmaxu2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
  const uint32_t e = (top + 0x1f * kOne) >> 7 & 0x1ff * kOne;   // 129 above the block's
  constexpr uint32_t kLow = 129 + kQ4ExpMin, kSpan = kQ4ExpMax - kQ4ExpMin;
  const uint32_t e8 = __vminu2(__vmaxu2(e, kLow * kOne) - kLow * kOne, kSpan * kOne);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t inv = (127 - kQ4ExpMin - (i == 0 ? e8 & 0xffffu : e8 >> 16)) * (kOne << 7);
    const uint32_t w[4] = {x[i].q.x, x[i].q.y, x[i].q.z, x[i].q.w};
    float y[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]),
                                       *reinterpret_cast<const __nv_bfloat162*>(&inv));
      y[2 * k] = __low2float(p);
      y[2 * k + 1] = __high2float(p);
    }
    codes[i] = q4_encode(y);
  }
  const uint32_t bits = (e8 + 13 * kOne) & 0xf * kOne;
  return bits | bits >> 8;
}
__device__ __forceinline__ uint32_t q4_quantise(const Raw8f32 (&x)[2], uint32_t* codes) {
  uint32_t exps = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float v[8];
    x[i].values(v);
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(v[k]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const int e = static_cast<int>((top + 0x1fffffu) >> 23) - 129;
    const int e8 = min(max(e, kQ4ExpMin), kQ4ExpMax) - kQ4ExpMin;
    const float inv = __uint_as_float((127 - kQ4ExpMin - e8) << 23);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= inv;
    codes[i] = q4_encode(v);
    exps |= static_cast<uint32_t>((e8 + 13) & 15) << (8 * i);
  }
  return exps;
}

template <typename In>
__global__ void __launch_bounds__(32 * kAppendWarps)
    append_q4_kernel(const In* __restrict__ rows, const int32_t* __restrict__ positions,
                     const int64_t* __restrict__ slots, uint8_t* __restrict__ pool,
                     const __grid_constant__ RopeTurns turns, int32_t* status, int n,
                     int64_t pool_rows, int page_shift) {
  const int lane = threadIdx.x & 31;
  const int r0 = blockIdx.x * kAppendRows + (threadIdx.x >> 5);
  int64_t slot[kAppendEach];
  int pos[kAppendEach];
  std::conditional_t<std::is_same_v<In, float>, Raw8f32, Raw8bf16> raw[kAppendEach][2];
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
    const Q4Page<uint8_t> page(pool, static_cast<int>(slot[u] >> page_shift), page_shift);
    const int r = static_cast<int>(slot[u]) & ((1 << page_shift) - 1);
    uint32_t codes[2], exps = q4_quantise(raw[u], codes);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      reinterpret_cast<uint32_t*>(page.codes(r))[32 * i + lane] = codes[i];
    // Four lanes share a byte of exponents, two blocks', in each half of the row.
    exps <<= 2 * (lane & 2);
    exps |= __shfl_xor_sync(0xffffffffu, exps, 2);
    if ((lane & 2) == 0)
      page.exps(r)[8 * (lane & 1) + (lane >> 2)] = static_cast<uint8_t>(exps >> (8 * (lane & 1)));
    const float2 k = rotated(pair[u], pos[u], turn);
    *reinterpret_cast<uint32_t*>(page.keys + q4_key_at(r, lane)) = pack_bf16(k.x, k.y);
  }
}

// ------------------------------------------------------------- rows out of pages
// Bound by HBM: a row read, 576 values written.  A warp takes up to 32 consecutive rows of the
// packed output.  Its lanes find the first one's sequence together (32 steps of the row starts a
// round), then each one row's page, so that a run of rows costs one chain of dependent loads; then
// the warp moves them, a few rows' loads out while as many are written: four, or two of the wide
// rows, whose registers would halve the warps.  4 x 16384 rows to bf16, 4-bit 20.3 us (0.74 of the
// measured copy bandwidth; 22.9 with four rows a warp, each row's page looked up on its way), bf16
// 28.6 (0.78), fp32 to fp32 54.0 (0.82).
constexpr int kReadMost = 32;
struct ReadParams {
  const void* pool;
  const int32_t *table, *lengths, *starts, *first;   // first may be NULL: zeros
  int32_t* status;
  int B, num_rows, page_shift, table_stride, num_pages;
};

// Last index i in [0, n) with starts[i] <= x, or 0; by a whole warp.
__device__ __forceinline__ int warp_search(const int32_t* starts, int n, int x, int lane) {
  int lo = 0, size = n;   // the answer lies in [lo, lo + size)
  while (size > 1) {
    const int step = (size + 31) / 32;
    const int at = lo + lane * step;
    const uint32_t hit = __ballot_sync(0xffffffffu, lane * step < size && starts[min(at, n)] <= x);
    const int k = hit ? 31 - __clz(hit) : 0;
    size = min(step, size - k * step);
    lo += k * step;
  }
  return lo;
}

template <typename T>
struct RowLane {   // of a pool of whole rows
  Raw8<T> raw[2];
  float2 key;
  __device__ __forceinline__ void load(const void* pool, int id, int r, int page_shift, int lane) {
    const T* row = static_cast<const T*>(pool) + ((static_cast<size_t>(id) << page_shift) + r) * kRow;
    raw[0].load(row + 8 * lane);
    raw[1].load(row + 256 + 8 * lane);
    key = load_pair(row + kDc + 2 * lane);
  }
  __device__ __forceinline__ void values(int i, int, float* v) const { raw[i].values(v); }
  __device__ __forceinline__ float2 pair() const { return key; }
};
template <>
struct RowLane<__nv_fp8_storage_t> {
  uint2 raw[2];
  uint16_t key;
  __device__ __forceinline__ void load(const void* pool, int id, int r, int page_shift, int lane) {
    const uint8_t* row =
        static_cast<const uint8_t*>(pool) + ((static_cast<size_t>(id) << page_shift) + r) * kRow;
    raw[0] = __ldcs(reinterpret_cast<const uint2*>(row + 8 * lane));
    raw[1] = __ldcs(reinterpret_cast<const uint2*>(row + 256 + 8 * lane));
    key = *reinterpret_cast<const uint16_t*>(row + kDc + 2 * lane);
  }
  static __device__ __forceinline__ float2 two(uint32_t v) {
    return __half22float2(__half2(
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E4M3)));
  }
  __device__ __forceinline__ void values(int i, int, float* v) const {
    const uint32_t w[2] = {raw[i].x, raw[i].y};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = two(w[k >> 1] >> (16 * (k & 1)));
      v[2 * k] = f.x;
      v[2 * k + 1] = f.y;
    }
  }
  __device__ __forceinline__ float2 pair() const { return two(key); }
};
struct FourBit {};
template <>
struct RowLane<FourBit> : Q4Lane {
  __device__ __forceinline__ void load(const void* pool, int id, int r, int page_shift, int lane) {
    Q4Lane::load(Q4Page<const uint8_t>(static_cast<const uint8_t*>(pool), id, page_shift), r, lane);
  }
};

template <typename T>
constexpr int kReadEach = std::is_same_v<T, float> || std::is_same_v<T, __nv_bfloat16> ? 2 : 4;

template <typename T, typename Out>
__global__ void __launch_bounds__(32 * kWarps)
    cache_read_kernel(const ReadParams p, Out* rows, int span) {
  const int lane = threadIdx.x & 31;
  const long long first = (static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * span;
  const int end = min(p.starts[p.B], p.num_rows);
  if (first >= end) return;
  const int t0 = static_cast<int>(first), n = min(span, end - t0);
  // Lane i: row t0 + i, page * page_size + row of the page, or -1 (there is none: zeros).
  const int b0 = warp_search(p.starts, p.B, t0, lane);
  long long slot = -1;
  if (lane < n) {
    const int t = t0 + lane;
    // From there on in doubling steps (most often none or one sequence further), then halved.
    int b = b0, step = 1;
    for (; b + step < p.B && p.starts[b + step] <= t; step <<= 1) b += step;
    for (step >>= 1; step > 0; step >>= 1)
      if (b + step < p.B && p.starts[b + step] <= t) b += step;
    const long long pos = static_cast<long long>(t) - p.starts[b] + (p.first ? p.first[b] : 0);
    if (pos < 0 || pos >= p.lengths[b] ||
        pos >= static_cast<long long>(p.table_stride) << p.page_shift) {
      report(p.status, MLA_DEV_LENGTH_OUT_OF_RANGE);
    } else {
      const int id = p.table[static_cast<size_t>(b) * p.table_stride + (pos >> p.page_shift)];
      if (id < 0 || id >= p.num_pages)
        report(p.status, MLA_DEV_PAGE_OUT_OF_RANGE);
      else
        slot = (static_cast<long long>(id) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
    }
  }
  constexpr int kEach = kReadEach<T>;
  RowLane<T> next[kEach];
  long long next_slot[kEach];
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      next_slot[u] = __shfl_sync(0xffffffffu, slot, (i0 + u) & 31);
      if (i0 + u < n && next_slot[u] >= 0)
        next[u].load(p.pool, static_cast<int>(next_slot[u] >> p.page_shift),
                     static_cast<int>(next_slot[u]) & ((1 << p.page_shift) - 1), p.page_shift, lane);
    }
  };
  load(0);
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += kEach) {
    RowLane<T> in[kEach];
    bool have[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      in[u] = next[u];
      have[u] = next_slot[u] >= 0;
    }
    if (i0 + kEach < n) load(i0 + kEach);
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      if (i0 + u >= n) break;
      Out* row = rows + static_cast<size_t>(t0 + i0 + u) * kRow;
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      float2 k = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (have[u]) in[u].values(i, lane, v);
        store8(row + 256 * i + 8 * lane, v);
      }
      if (have[u]) k = in[u].pair();
      store_pair(row + kDc + 2 * lane, k.x, k.y);
    }
  }
}

// ------------------------------------------------------------- the page index
// page_index_kernel's definition over 4-bit pages.  Items are the pages that each request's max_new
// rows could touch.  A CTA looks at a page that was touched twice: its largest magnitude, of which
// the power of two above it is all that counts (and of codes, their highest bits), then the sums.  A
// warp reads four of the page's rows together.
// Of no more items than the SMs hold CTAs at once, each has one (kEach), which knows its item sooner:
// one touched page of 64 rows for each of 4 sequences 5.3 us, the way from the lengths to the table to
// the rows and back, for 5.6 walked.  Of more, few of which may have been touched, a CTA walks its
// share, looked up 32 at a time: one of 32 for each of 256 requests 9.4 us for 16, of 9 for each of
// 128 7.6 for 9.5; 61 x 1024 rows all touched 17.9, and 4096 pages of 4 x 65536 rows 71 for 65 (1.5
// TB/s: bound by instructions, 77 % of the issue slots).
// A latent is a multiple of 2^-9 and at most 384, so the maximum is a maximum of exact values.
constexpr float kQ4Tiny = 1e-30f;
constexpr int kIndexRows = 4;
constexpr int kIndexPerSm = 4;   // CTAs
template <bool kEach>
__global__ void __launch_bounds__(32 * kWarps)
    page_index_q4_kernel(const uint8_t* __restrict__ pool, const int32_t* __restrict__ table,
                         const int32_t* __restrict__ first_rows, const int32_t* __restrict__ lengths,
                         int8_t* codes, float* scales, int32_t* status, int page_shift,
                         int table_stride, int num_pages, int max_new, int most, int batch) {
  __shared__ float tops[kWarps];
  __shared__ int sums[kWarps][kRow];
  __shared__ int peaks[kWarps];
  __shared__ int ids[32], rows_of[32];
  __shared__ uint32_t found;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // One page of n rows, by the whole CTA.
  auto page = [&](int id, int n) {
    const Q4Page<const uint8_t> at(pool, id, page_shift);
    constexpr int kBatch = kWarps * kIndexRows;
    Q4Lane x[kIndexRows];   // rows r0 + warp, r0 + kWarps + warp, ..
    auto load = [&](int r0) {
#pragma unroll
      for (int u = 0; u < kIndexRows; ++u) {
        const int r = r0 + kWarps * u + warp;
        if (r < n)
          x[u].load(at, r, lane);
        else
          x[u].zero();   // adds nothing
      }
    };
    float top = 0.f;
    int high = -100;   // latents are below 2^high
    for (int r0 = 0; r0 < n; r0 += kBatch) {
      load(r0);
#pragma unroll
      for (int u = 0; u < kIndexRows; ++u) {
        if (r0 + kWarps * u >= n) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) high = max(high, x[u].high(i, lane));
        const float2 k = x[u].pair();
        top = fmaxf(top, fmaxf(fabsf(k.x), fabsf(k.y)));
      }
    }
    if (high > -100) top = fmaxf(top, ldexpf(0.5f, high));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, tops[w]);
    int ex = 0;
    frexpf(top, &ex);   // top = m 2^ex, m in [0.5, 1)
    const float unit = ldexpf(1.f, 20 - ex);
    const bool live = top >= kQ4Tiny && top <= 3.0e38f;
    constexpr float kMagic = 12582912.f;   // 1.5 2^23: the sum's low bits are the rounded integer
    uint32_t sum[18], rows = 0;   // rows: those added, each with kMagic's bits
#pragma unroll
    for (int i = 0; i < 18; ++i) sum[i] = 0;
    for (int r0 = 0; r0 < n; r0 += kBatch) {
      if (n > kBatch) load(r0);
#pragma unroll
      for (int u = 0; u < kIndexRows; ++u) {
        if (r0 + kWarps * u >= n) break;
        ++rows;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float v[8];
          x[u].values(i, lane, v, unit);
#pragma unroll
          for (int k = 0; k < 8; ++k) sum[8 * i + k] += __float_as_uint(v[k] + kMagic);
        }
        const float2 k = x[u].pair();
        sum[16] += __float_as_uint(fmaf(k.x, unit, kMagic));
        sum[17] += __float_as_uint(fmaf(k.y, unit, kMagic));
      }
    }
#pragma unroll
    for (int i = 0; i < 18; ++i)
      sums[warp][i < 16 ? 256 * (i >> 3) + 8 * lane + (i & 7) : kDc + 2 * lane + (i & 1)] =
          static_cast<int>(sum[i] - rows * __float_as_uint(kMagic));
    __syncthreads();
    int total[3] = {0, 0, 0}, peak = 0;   // of columns tid, tid + 256 and tid + 512
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int c = tid + 32 * kWarps * i;
      if (c < kRow)
#pragma unroll
        for (int w = 0; w < kWarps; ++w) total[i] += sums[w][c];
      peak = max(peak, abs(total[i]));
    }
    peak = __reduce_max_sync(0xffffffffu, peak);
    if (lane == 0) peaks[warp] = peak;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) peak = max(peak, peaks[w]);
    const bool good = live && peak > 0;
    const float pf = static_cast<float>(peak), inv = good ? __frcp_rn(pf) * 127.f : 0.f;
    int8_t* out = codes + static_cast<size_t>(id) * kRow;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const int c = tid + 32 * kWarps * i;
      if (c < kRow)
        out[c] = good ? static_cast<int8_t>(__float2int_rn(static_cast<float>(total[i]) * inv)) : 0;
    }
    if (tid == 0)
      scales[id] = good ? ldexpf(pf * (1.f / 127.f) / static_cast<float>(n), ex - 20) : 0.f;
  };
  // Page jj of those that request b's new rows could touch, and its rows; -1: there is none.
  auto look_up = [&](int b, int jj, bool say, int& n) {
    const int first = first_rows[b], len = lengths[b];
    const bool bad =
        first < 0 || len < 0 || len > static_cast<long long>(table_stride) << page_shift;
    if (say && jj == 0 && (bad || static_cast<long long>(len) - first > max_new))
      report(status, MLA_DEV_LENGTH_OUT_OF_RANGE);
    const long long j = static_cast<long long>(first >> page_shift) + jj;
    if (bad || first >= len || (j << page_shift) >= len) return -1;
    n = static_cast<int>(min(1ll << page_shift, len - (j << page_shift)));
    const int id = table[static_cast<size_t>(b) * table_stride + j];
    if (id >= 0 && id < num_pages) return id;
    if (say) report(status, MLA_DEV_PAGE_OUT_OF_RANGE);
    return -1;
  };
  if constexpr (kEach) {
    int n = 0;
    const int id = look_up(blockIdx.x / most, blockIdx.x % most, tid == 0, n);
    if (id >= 0) page(id, n);
  } else {
    const long long items = static_cast<long long>(batch) * most;
    for (long long base = blockIdx.x; base < items; base += 32ll * gridDim.x) {
      // Lane l of the first warp looks item base + l * gridDim.x up.
      if (warp == 0) {
        const long long item = base + static_cast<long long>(lane) * gridDim.x;
        int id = -1, n = 0;
        if (item < items) {
          const int b = items < (1ll << 31) ? static_cast<int>(item) / most
                                            : static_cast<int>(item / most);
          id = look_up(b, static_cast<int>(item - static_cast<long long>(b) * most), true, n);
        }
        ids[lane] = id;
        rows_of[lane] = n;
        const uint32_t live = __ballot_sync(0xffffffffu, id >= 0);
        if (lane == 0) found = live;
      }
      __syncthreads();
      for (uint32_t todo = found; todo; todo &= todo - 1) {
        const int l = __ffs(todo) - 1;
        page(ids[l], rows_of[l]);
        __syncthreads();   // before the next page's sums
      }
      __syncthreads();   // before the next items are looked up
    }
  }
}

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    cudaGetLastError();
  return sms > 0 ? sms : 1;
}

template <typename T>
void launch_read(const ReadParams& p, int32_t out_dtype, void* rows, cudaStream_t s) {
  constexpr int kEach = kReadEach<T>;
  // As many rows a warp as leave every SM some 24 warps.
  const long long warps = 24ll * sm_count();
  const long long even = (p.num_rows + warps - 1) / warps;
  const int span = static_cast<int>(
      even > kReadMost ? kReadMost : (even + kEach - 1) / kEach * kEach);
  const long long per_cta = static_cast<long long>(span) * kWarps;
  const dim3 grid(static_cast<unsigned>((p.num_rows + per_cta - 1) / per_cta)), block(32 * kWarps);
  if (out_dtype == MLA_F32)
    cache_read_kernel<T><<<grid, block, 0, s>>>(p, static_cast<float*>(rows), span);
  else
    cache_read_kernel<T><<<grid, block, 0, s>>>(p, static_cast<__nv_bfloat16*>(rows), span);
}

}  // namespace

mla_status append_q4(const char* who, const mla_paging* paging, int num_rows, bool f32_rows,
                     const void* rows, const int32_t* positions, const int64_t* slots,
                     double rope_base, void* cache, int32_t* status, cudaStream_t s) {
  const dim3 grid((num_rows - 1) / kAppendRows + 1);
  const int64_t pool = static_cast<int64_t>(paging->num_pages) * paging->page_size;
  auto go = [&](auto* in) {
    append_q4_kernel<<<grid, 32 * kAppendWarps, 0, s>>>(in, positions, slots,
                                                  static_cast<uint8_t*>(cache), rope_turns(rope_base),
                                                  status, num_rows, pool, page_shift_of(paging));
  };
  if (f32_rows)
    go(static_cast<const float*>(rows));
  else
    go(static_cast<const __nv_bfloat16*>(rows));
  return launch_status(who);
}

mla_status page_index_q4(const char* who, const mla_paging* paging, int batch, int max_new, int most,
                         const void* cache, const int32_t* table, const int32_t* first_rows,
                         const int32_t* lengths, int8_t* codes, float* scales, int32_t* status,
                         cudaStream_t s) {
  const long long items = static_cast<long long>(batch) * most;
  auto go = [&](auto kernel, long long ctas) {
    kernel<<<static_cast<unsigned>(ctas), 32 * kWarps, 0, s>>>(
        static_cast<const uint8_t*>(cache), table, first_rows, lengths, codes, scales, status,
        page_shift_of(paging), paging->table_stride, paging->num_pages, max_new, most, batch);
  };
  const long long held = static_cast<long long>(kIndexPerSm) * sm_count();
  if (items <= held)
    go(page_index_q4_kernel<true>, items);
  else
    // An odd number: where every request touches its first page alone, those are `most` items apart,
    // often a power of two, and have to come to different CTAs.
    go(page_index_q4_kernel<false>, held - 1);
  return launch_status(who);
}

}  // namespace mla

using namespace mla;

extern "C" size_t mla_pool_bytes(const mla_dims* dims, const mla_paging* paging) {
  const char* who = "mla_pool_bytes";
  if (check_dims(dims, who, true) != MLA_OK || check_paging(paging, who) != MLA_OK) return 0;
  const size_t row = dims->dtype == MLA_FP4_E2M1   ? kQ4RowBytes
                     : dims->dtype == MLA_FP8_E4M3 ? kRow
                     : dims->dtype == MLA_BF16     ? 2 * kRow
                                                   : 4 * kRow;
  return static_cast<size_t>(paging->num_pages) * paging->page_size * row;
}

extern "C" mla_status mla_cache_read_paged(const mla_dims* dims, const mla_paging* paging,
                                           const void* cache, const int32_t* block_table,
                                           const int32_t* lengths, const int32_t* row_starts,
                                           const int32_t* first_rows, int32_t num_rows,
                                           int32_t row_dtype, void* rows, int32_t* dev_status,
                                           void* stream) {
  const char* who = "mla_cache_read_paged";
  mla_status st = check_dims(dims, who, true);
  if (st == MLA_OK) st = check_paging(paging, who);
  if (st != MLA_OK) return st;
  if (num_rows < 0) {
    set_error("%s: num_rows=%d must be >= 0", who, num_rows);
    return MLA_ERR_INVALID_ARG;
  }
  if (row_dtype != MLA_F32 && row_dtype != MLA_BF16) {
    set_error("%s: row_dtype %d must be MLA_F32 or MLA_BF16", who, row_dtype);
    return MLA_ERR_UNSUPPORTED;
  }
  if (num_rows == 0) return MLA_OK;
  if (!cache || !block_table || !lengths || !row_starts || !rows || !aligned16(cache) ||
      !aligned16(rows)) {
    set_error("%s: pointers must not be NULL, cache and rows 16-byte aligned", who);
    return MLA_ERR_INVALID_ARG;
  }
  const ReadParams p{cache, block_table, lengths, row_starts, first_rows, dev_status,
                     dims->batch, num_rows, page_shift_of(paging), paging->table_stride,
                     paging->num_pages};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (dims->dtype) {
    case MLA_F32: launch_read<float>(p, row_dtype, rows, s); break;
    case MLA_BF16: launch_read<__nv_bfloat16>(p, row_dtype, rows, s); break;
    case MLA_FP8_E4M3: launch_read<__nv_fp8_storage_t>(p, row_dtype, rows, s); break;
    default: launch_read<FourBit>(p, row_dtype, rows, s); break;
  }
  return launch_status(who);
}
