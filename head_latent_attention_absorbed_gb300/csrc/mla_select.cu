// Sparse attention over pages: a cheap score per page chooses the pages a token
// attends (mla_select_pages), and the paged decode attention runs over the
// choice (mla_decode_attn_sparse).
//
// Score of page g for a token: scales[g] max_h a_h <c_h, codes[g]>, with c_h the
// token's query of head h ([q_abs ; q_pe], "Multi-Head Latent Attention" 3.6)
// and codes[g] the page's mean row, both rounded to int8.  The pages kept are a
// discrete choice, so the score is built to be reproducible to the bit: the dot
// products are whole numbers below 576 127^2 < 2^24, exact in fp32 in any order,
// and what follows is a fixed chain of fp32 products and maxima.
//
// Three kernels:
//   select_query_kernel   int8 codes of the query, as the score's fp16 operand image
//   page_score_kernel     scores: tcgen05.mma kind::f16 on whole numbers
//   page_pick_kernel      the k-th largest score by radix selection, then the kept
//                         pages in order of position
#include <cuda_fp16.h>
#include <math.h>

#include "mla_paged.cuh"
#include "mla_split.cuh"

namespace mla {
namespace {

constexpr int kBoxes = kRow / 64;              // 64-column boxes of 128-byte rows
constexpr int kScorePages = 128;               // pages per CTA (the MMA's M)
constexpr int kScoreThreads = 256;
constexpr int kMaxGroup = 64;                  // heads per MMA (its N), at most
constexpr int kPageBox = kScorePages * 128;    // 16 KB
constexpr float kTinyQuery = 1e-30f;           // below this a query counts as zero

struct SelectParams {
  const void *q_abs, *q_pe;
  const int32_t *table, *lengths;
  const int8_t* codes;
  const float* scales;
  float* scores;        // [R, width]
  float* a;             // [R, groups * group]: max |q| (1/127) per head
  uint8_t* image;       // [R, groups][9 boxes][group rows][128 B], 128-byte swizzle
  int32_t *sel_table, *sel_lengths, *status;
  int R, H, q_len, s_max, group, groups, io_bf16;
  int width;            // pages of s_max rows
  int page_shift, table_stride, num_pages;
  int top, keep_first, keep_last;
  int early;            // the reader of the choice waits for it before it reads anything of it
};

// Rows token r attends (as the attention kernels clamp them).
__device__ __forceinline__ int token_rows(const SelectParams& p, int r, bool report_it) {
  int full = p.lengths[r / p.q_len];
  if (full < p.q_len || full > p.s_max) {
    if (report_it) report(p.status, MLA_DEV_LENGTH_OUT_OF_RANGE);
    full = full < 0 ? 0 : (full > p.s_max ? p.s_max : full);
  }
  const int n = full - (p.q_len - 1 - r % p.q_len);
  return n < 0 ? 0 : n;
}
__device__ __forceinline__ int token_pages(const SelectParams& p, int n) {
  return (n + (1 << p.page_shift) - 1) >> p.page_shift;
}

// One warp per (token, head), lane l holds the values 2l, 2l + 1 of each 64-column
// box; heads past H (padding of the last group) are rows of zeros.
__global__ void __launch_bounds__(128) select_query_kernel(const SelectParams p) {
  pdl_launch_dependents();   // the score kernel loads its pages meanwhile
  const int h = blockIdx.x * 4 + (threadIdx.x >> 5), r = blockIdx.y, lane = threadIdx.x & 31;
  const int padded = p.group * p.groups;
  pdl_wait();
  if (h >= padded || token_pages(p, token_rows(p, r, false)) <= p.top) return;
  float2 v[kBoxes];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kBoxes; ++i) {
    v[i] = make_float2(0.f, 0.f);
    if (h < p.H) {
      const size_t rh = static_cast<size_t>(r) * p.H + h;
      if (p.io_bf16) {
        const __nv_bfloat16* q =
            i < 8 ? static_cast<const __nv_bfloat16*>(p.q_abs) + rh * kDc + 64 * i
                  : static_cast<const __nv_bfloat16*>(p.q_pe) + rh * kDr;
        v[i] = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(q)[lane]);
      } else {
        const float* q = i < 8 ? static_cast<const float*>(p.q_abs) + rh * kDc + 64 * i
                               : static_cast<const float*>(p.q_pe) + rh * kDr;
        v[i] = reinterpret_cast<const float2*>(q)[lane];
      }
    }
    top = fmaxf(top, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  const bool live = top >= kTinyQuery;
  const float inv = live ? __frcp_rn(top) * 127.f : 0.f;
  if (lane == 0) p.a[static_cast<size_t>(r) * padded + h] = live ? top * (1.f / 127.f) : 0.f;
  const int g = h / p.group, n = h % p.group;
  uint8_t* img = p.image + (static_cast<size_t>(r) * p.groups + g) * (kBoxes * p.group * 128);
#pragma unroll
  for (int i = 0; i < kBoxes; ++i) {
    const __half2 c = __floats2half2_rn(rintf(v[i].x * inv), rintf(v[i].y * inv));
    *reinterpret_cast<__half2*>(img + i * p.group * 128 + sw128(n, lane >> 2) + 4 * (lane & 3)) = c;
  }
}

// Instruction descriptor of kind::f16 with fp16 A and B and an fp32 accumulator.
__device__ __forceinline__ uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Four int8 codes (biased to 0..255 by the caller's xor) to four fp16 whole
// numbers: the bytes become the low mantissa bits of 1024 + u, less 1024 + 128.
__device__ __forceinline__ uint2 codes_to_half(uint32_t biased) {
  uint32_t lo, hi;
  asm("prmt.b32 %0, %1, %2, 0x5150;" : "=r"(lo) : "r"(biased), "r"(0x64646464u));
  asm("prmt.b32 %0, %1, %2, 0x5352;" : "=r"(hi) : "r"(biased), "r"(0x64646464u));
  const __half2 k = __half2half2(__ushort_as_half(0x6480));   // 1152
  const __half2 x = __hsub2(*reinterpret_cast<__half2*>(&lo), k);
  const __half2 y = __hsub2(*reinterpret_cast<__half2*>(&hi), k);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

// grid (ceil(width / 128), R).  The CTA's 128 pages (rows of the table, so
// anywhere in the pool) are read as int8, 576 bytes a page, and written to
// shared memory as the fp16 A operand; the query image of a head group is the B
// operand, copied in one bulk copy per group.  36 MMAs (M 128, N the group, K
// 16) per group; each thread then takes the maximum over half of the group's
// heads of one page.  Bound by the index's bytes and the latency of one tile:
// codes, MMAs and epilogue follow one another in a CTA.
constexpr int kOffPages = 0;
constexpr int kOffQuery = kBoxes * kPageBox;
constexpr int kOffEnd = kOffQuery + kBoxes * kMaxGroup * 128;
constexpr size_t kScoreSmem = 1024 + kOffEnd;
static_assert(kScoreSmem + 4096 <= 232448, "shared memory");

__global__ void __launch_bounds__(kScoreThreads, 1) page_score_kernel(const SelectParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_id[kScorePages];
  __shared__ float s_scale[kScorePages], s_half[kScorePages], s_a[kMaxGroup];
  __shared__ uint32_t s_tmem;
  __shared__ __align__(8) uint64_t s_bar[2];   // query image landed; MMAs finished
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem), bars = smem_u32(s_bar);
  const int r = blockIdx.y, j0 = blockIdx.x * kScorePages;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // uniform to the compiler
  const int P = token_pages(p, token_rows(p, r, false));
  pdl_launch_dependents();        // the choice waits for this grid before it reads
  if (P <= p.top || j0 >= P) {    // every page is kept, or none of these exists
    if (j0 == 0) pdl_wait();      // the grid may not end before the queries' codes are made
    return;
  }
  if (tid < kScorePages) {
    const int j = j0 + tid;
    int id = -1;
    if (j < P) {
      id = p.table[static_cast<size_t>(r / p.q_len) * p.table_stride + j];
      if (id < 0 || id >= p.num_pages) {
        report(p.status, MLA_DEV_PAGE_OUT_OF_RANGE);
        id = -1;
      }
    }
    s_id[tid] = id;
    s_scale[tid] = id >= 0 ? p.scales[id] : 0.f;
  }
  if (tid == 0) {
    mbar_init(bars, 1);
    mbar_init(bars + 8, 1);
    fence_mbarrier_init();
  }
  if (warp == 0) {
    __syncwarp();
    tmem_alloc(smem_u32(&s_tmem), 64);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // 36 16-byte pieces of each of the 128 pages; every load of a thread in flight.
  constexpr int kPieces = kScorePages * (kRow / 16) / kScoreThreads;
  uint4 piece[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int x = u * kScoreThreads + tid, row = x / (kRow / 16), c = x % (kRow / 16);
    const int id = s_id[row];
    piece[u] = id >= 0 ? *reinterpret_cast<const uint4*>(
                             p.codes + static_cast<size_t>(id) * kRow + 16 * c)
                       : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int x = u * kScoreThreads + tid, row = x / (kRow / 16), c = x % (kRow / 16);
    uint8_t* box = smem + kOffPages + (c >> 2) * kPageBox;
    const uint2 h0 = codes_to_half(piece[u].x ^ 0x80808080u);
    const uint2 h1 = codes_to_half(piece[u].y ^ 0x80808080u);
    const uint2 h2 = codes_to_half(piece[u].z ^ 0x80808080u);
    const uint2 h3 = codes_to_half(piece[u].w ^ 0x80808080u);
    *reinterpret_cast<uint4*>(box + sw128(row, 2 * (c & 3))) = make_uint4(h0.x, h0.y, h1.x, h1.y);
    *reinterpret_cast<uint4*>(box + sw128(row, 2 * (c & 3) + 1)) =
        make_uint4(h2.x, h2.y, h3.x, h3.y);
  }
  fence_proxy_async_smem();
  __syncthreads();
  pdl_wait();   // the query image, and the last readers of scores
  const uint32_t tmem = s_tmem;
  const uint32_t image_bytes = kBoxes * p.group * 128;
  const uint8_t* img = p.image + static_cast<size_t>(r) * p.groups * image_bytes;
  const float* a = p.a + static_cast<size_t>(r) * p.group * p.groups;
  auto load_group = [&](int g) {
    mbar_arrive_expect_tx(bars, image_bytes);
    bulk_g2s(sbase + kOffQuery, img + static_cast<size_t>(g) * image_bytes, image_bytes, bars);
  };
  if (tid == 0) load_group(0);
  float best = -INFINITY;
  bool ok = true;
  const uint32_t idesc = idesc_f16(kScorePages, p.group);
  const uint64_t da0 = umma_desc_sw128(sbase + kOffPages, 16, 1024);
  const uint64_t db0 = umma_desc_sw128(sbase + kOffQuery, 16, 1024);
  for (int g = 0; g < p.groups; ++g) {
    if (warp == 0 && __all_sync(0xffffffffu, mbar_wait_bounded(bars, g & 1))) {
      // The warp issues as one (see umma_bf16_elected; kind::f16 takes fp16 as well); boxes
      // are not unrolled, so that the loop's code is fetched once.
      tc_fence_after();
#pragma unroll 1
      for (int i = 0; i < kBoxes; ++i) {
        const uint64_t da = da0 + static_cast<uint64_t>(i * (kPageBox >> 4));
        const uint64_t db = db0 + static_cast<uint64_t>(i * p.group * 8);
#pragma unroll
        for (int k = 0; k < 4; ++k)   // 16 columns (32 bytes) a step
          umma_bf16_elected(tmem, da + 2 * k, db + 2 * k, idesc, k > 0 ? 1u : (i > 0 ? 1u : 0u));
      }
      umma_commit_elected(bars + 8);
    }
    __syncwarp();
    if (tid >= 64 && tid < 64 + p.group) s_a[tid - 64] = a[g * p.group + tid - 64];
    // Every thread waits for the accumulators (bounded: a copy that never landed
    // leaves the MMAs unissued, and every thread gives up).
    ok = __syncthreads_and(mbar_wait_bounded(bars + 8, g & 1));
    if (!ok) break;
    tc_fence_after();
    if (tid == 0 && g + 1 < p.groups) load_group(g + 1);   // the MMAs have read the old one
    const int half = p.group / 2, c0 = warp < 4 ? 0 : half;
    for (int c = 0; c < half; c += 8) {
      uint32_t d[8];
      tmem_ld8_nowait(tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + c0 + c, d);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int h = g * p.group + c0 + c + i;
        if (h < p.H) best = fmaxf(best, s_a[c0 + c + i] * __uint_as_float(d[i]));
      }
    }
    tc_fence_before();
    __syncthreads();   // the accumulators are read
    tc_fence_after();
  }
  const int row = 32 * (warp & 3) + lane;
  if (warp >= 4) s_half[row] = best;
  __syncthreads();
  if (warp < 4 && j0 + row < P && ok) {
    // + 0 turns -0 into +0: the two tie
    const float s = fmaxf(best, s_half[row]) * s_scale[row] + 0.f;
    p.scores[static_cast<size_t>(r) * p.width + j0 + row] = s_id[row] >= 0 ? s : -INFINITY;
  }
  if (tid == 0 && !ok) report(p.status, MLA_DEV_PIPELINE_TIMEOUT);
  if (warp == 0) tmem_dealloc(tmem, 64);
}

// One CTA per token.  Radix selection (scores as unsigned integers in the same order),
// eight bits a pass from the highest bit in which any two differ, narrows down the score
// of the last page kept until the pages that share its leading bits are all kept, or only
// equal scores are left, of which the lowest positions are kept; one ordered pass then
// writes the kept pages.  Bound by latency; from the top byte on, with scores of similar
// size, the first passes count everything in one bin (five passes and its atomics: 7.5 us
// for 1024 pages).
constexpr int kPickThreads = 1024;
constexpr int kPickHold = 8192;   // scores kept in shared memory, else read again each pass

__device__ __forceinline__ uint32_t ordered_bits(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kPickThreads) page_pick_kernel(const SelectParams p) {
  __shared__ uint32_t keys[kPickHold];
  __shared__ int hist[256], s_found[3], s_part[32];
  __shared__ uint32_t s_differ[32];   // its own: with all keys equal no barrier parts its
                                      // readers from the first writers of s_part
  const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = token_rows(p, r, tid == 0);
  const int P = token_pages(p, n);
  const int32_t* row = p.table + static_cast<size_t>(r / p.q_len) * p.table_stride;
  int32_t* out = p.sel_table + static_cast<size_t>(r) * p.top;
  if (p.early) pdl_launch_dependents();
  pdl_wait();   // the scores; and the readers of the last choice are done
  if (P <= p.top) {
    for (int j = tid; j < p.top; j += kPickThreads) {
      const int id = j < P ? row[j] : -1;   // of a token that no score kernel has looked at
      if (j < P && static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_pages))
        report(p.status, MLA_DEV_PAGE_OUT_OF_RANGE);
      out[j] = id;
    }
    if (tid == 0) p.sel_lengths[r] = n;
    return;
  }
  const float* scores = p.scores + static_cast<size_t>(r) * p.width;
  const int lo = p.keep_first, hi = P - p.keep_last;   // scored pages: [lo, hi)
  const bool held = hi - lo <= kPickHold;
  if (held)
    for (int j = lo + tid; j < hi; j += kPickThreads) keys[j - lo] = ordered_bits(scores[j]);
  auto key = [&](int j) { return held ? keys[j - lo] : ordered_bits(scores[j]); };
  int want = p.top - p.keep_first - p.keep_last;   // of the scored pages, fewer than there are
  uint32_t prefix = 0, mask = 0;
  if (tid < 256) hist[tid] = 0;
  if (want > 0) {
    // The bits in which any key differs from the first.
    const uint32_t key0 = ordered_bits(scores[lo]);
    uint32_t differ = 0;
    for (int j = lo + tid; j < hi; j += kPickThreads) differ |= key(j) ^ key0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) differ |= __shfl_xor_sync(0xffffffffu, differ, off);
    if (lane == 0) s_differ[warp] = differ;
    __syncthreads();
    differ = s_differ[lane];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) differ |= __shfl_xor_sync(0xffffffffu, differ, off);
    const int same = __clz(differ);   // leading bits that all keys share
    mask = same > 0 ? ~(0xffffffffu >> same) : 0u;
    if (same >= 32) mask = 0xffffffffu;
    prefix = key0 & mask;
  }
  bool open = want > 0;   // pages with the prefix still to be told apart
  while (open && mask != 0xffffffffu) {
    const int shift = max(0, 24 - __popc(mask));   // eight more bits, or what is left
    for (int j = lo + tid; j < hi; j += kPickThreads) {
      const uint32_t k = key(j);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // Lane l holds bins 255 - 8l down to 248 - 8l; the bin where the running
      // count from the top reaches `want`.
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = hist[255 - 8 * lane - i];
        sum += c[i];
      }
      int above = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, above, off);
        if (lane >= off) above += y;
      }
      above -= sum;   // pages in higher bins of the lanes before
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (above < want && above + c[i] >= want) {
          s_found[0] = 255 - 8 * lane - i;
          s_found[1] = want - above;
          s_found[2] = c[i];
        }
        above += c[i];
      }
    }
    __syncthreads();
    prefix |= static_cast<uint32_t>(s_found[0]) << shift;
    mask |= 255u << shift;
    want = s_found[1];   // still wanted among the pages with this prefix
    open = s_found[2] > want;
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
  }
  // want: pages kept of those that have the prefix (0: none scored).
  const bool any = p.top > p.keep_first + p.keep_last;
  int base_more = 0, base_tie = 0;
  for (int j0 = 0; j0 < P; j0 += kPickThreads) {
    const int j = j0 + tid;
    const bool forced = j < P && (j < lo || j >= hi);
    const bool scored = any && j < P && !forced;
    const uint32_t k = scored ? key(j) : 0;
    const int more = forced || (scored && (k & mask) > prefix);
    const int tie = scored && (k & mask) == prefix;
    // Both counts in one scan: kept outright in the low half, ties in the high.
    const int packed = more | tie << 16;
    int incl = packed;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    if (lane == 31) s_part[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      int x = s_part[lane];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      s_part[lane] = x;
    }
    __syncthreads();
    const int before = incl - packed + (warp ? s_part[warp - 1] : 0);
    const int ties = base_tie + (before >> 16);
    if (more || (tie && ties < want))
      out[base_more + (before & 0xffff) + min(ties, want)] = row[j];
    base_more += s_part[31] & 0xffff;
    base_tie += s_part[31] >> 16;
    __syncthreads();
  }
  if (tid == 0) p.sel_lengths[r] = n - ((P - p.top) << p.page_shift);
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Heads per MMA, and MMA groups.
void head_groups(int H, int* group, int* groups) {
  *group = H >= kMaxGroup ? kMaxGroup : (H + 15) / 16 * 16;
  *groups = (H + *group - 1) / *group;
}

struct SelectSpace {
  size_t scores, a, image, total;
};
SelectSpace select_space(const mla_dims* d, const mla_paging* pg, int q_len) {
  int group, groups;
  head_groups(d->heads, &group, &groups);
  const size_t R = static_cast<size_t>(d->batch) * q_len;
  const size_t width = (static_cast<size_t>(d->s_max) + pg->page_size - 1) / pg->page_size;
  SelectSpace s;
  s.scores = round256(R * width * sizeof(float));
  s.a = round256(R * group * groups * sizeof(float));
  s.image = round256(R * groups * (static_cast<size_t>(kBoxes) * group * 128));
  s.total = s.scores + s.a + s.image;
  return s;
}

mla_status check_select(const char* who, const mla_dims* d, const mla_paging* pg,
                        int32_t io_dtype, int32_t q_len) {
  mla_status st = check_paged(who, d, pg, io_dtype, q_len);
  if (st != MLA_OK) return st;
  if (d->heads > 4096) {
    set_error("%s: heads=%d exceeds 4096", who, d->heads);
    return MLA_ERR_UNSUPPORTED;
  }
  return MLA_OK;
}

// Everything mla_select_pages checks on the host; fills the kernels' parameters.
mla_status prepare_select(const char* who, const mla_dims* d, const mla_paging* pg,
                          int32_t io_dtype, int32_t q_len, const void* q_abs, const void* q_pe,
                          const int32_t* table, const int32_t* lengths, const int8_t* codes,
                          const float* scales, int32_t top, int32_t keep_first,
                          int32_t keep_last, void* ws, size_t ws_bytes, int32_t* sel_table,
                          int32_t* sel_lengths, int32_t* status, SelectParams* p) {
  mla_status st = check_select(who, d, pg, io_dtype, q_len);
  if (st != MLA_OK) return st;
  if (!q_abs || !q_pe || !table || !lengths || !codes || !scales || !ws || !sel_table ||
      !sel_lengths || !aligned16(q_abs) || !aligned16(q_pe) || !aligned16(codes) ||
      !aligned16(ws)) {
    set_error("%s: pointers must not be NULL; q_abs, q_pe, codes and workspace 16-byte aligned",
              who);
    return MLA_ERR_INVALID_ARG;
  }
  if (top < 1 || keep_first < 0 || keep_last < 1 ||
      static_cast<long long>(keep_first) + keep_last > top) {
    set_error("%s: top_pages=%d, keep_first=%d (>= 0) and keep_last=%d (>= 1) must satisfy "
              "keep_first + keep_last <= top_pages", who, top, keep_first, keep_last);
    return MLA_ERR_INVALID_ARG;
  }
  const SelectSpace s = select_space(d, pg, q_len);
  if (ws_bytes < s.total) {
    set_error("%s: workspace %zu bytes < %zu needed", who, ws_bytes, s.total);
    return MLA_ERR_WORKSPACE;
  }
  uint8_t* w = static_cast<uint8_t*>(ws);
  p->q_abs = q_abs;
  p->q_pe = q_pe;
  p->table = table;
  p->lengths = lengths;
  p->codes = codes;
  p->scales = scales;
  p->scores = reinterpret_cast<float*>(w);
  p->a = reinterpret_cast<float*>(w + s.scores);
  p->image = w + s.scores + s.a;
  p->sel_table = sel_table;
  p->sel_lengths = sel_lengths;
  p->status = status;
  p->R = d->batch * q_len;
  p->H = d->heads;
  p->q_len = q_len;
  p->s_max = d->s_max;
  head_groups(d->heads, &p->group, &p->groups);
  p->io_bf16 = io_dtype == MLA_BF16 ? 1 : 0;
  p->width = (d->s_max + pg->page_size - 1) / pg->page_size;
  p->page_shift = page_shift_of(pg);
  p->table_stride = pg->table_stride;
  p->num_pages = pg->num_pages;
  p->top = top;
  p->keep_first = keep_first;
  p->keep_last = keep_last;
  p->early = 0;
  return MLA_OK;
}

mla_status launch_select(const char* who, const SelectParams& p, cudaStream_t s) {
  if (p.width > p.top) {   // otherwise every page is kept whatever its score
    static DeviceFlags attr_done;
    const int dev = current_device();
    if (!attr_done.test(dev)) {
      if (cudaFuncSetAttribute(page_score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               int(kScoreSmem)) != cudaSuccess) {
        cudaGetLastError();
        set_error("%s: cannot reserve %zu bytes of shared memory", who, kScoreSmem);
        return MLA_ERR_CUDA;
      }
      attr_done.set(dev);
    }
    launch_pdl(select_query_kernel, dim3((p.group * p.groups + 3) / 4, p.R), dim3(128), 0, s, p);
    launch_pdl(page_score_kernel, dim3((p.width + kScorePages - 1) / kScorePages, p.R),
               dim3(kScoreThreads), kScoreSmem, s, p);
  }
  launch_pdl(page_pick_kernel, dim3(p.R), dim3(kPickThreads), 0, s, p);
  return launch_status(who);
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" size_t mla_select_workspace_bytes(const mla_dims* dims, const mla_paging* paging,
                                             int32_t q_len) {
  if (check_select("mla_select_workspace_bytes", dims, paging, MLA_F32, q_len) != MLA_OK) return 0;
  return select_space(dims, paging, q_len).total;
}

extern "C" mla_status mla_select_pages(const mla_dims* dims, const mla_paging* paging,
                                       int32_t io_dtype, int32_t q_len, const void* q_abs,
                                       const void* q_pe, const int32_t* block_table,
                                       const int32_t* lengths, const int8_t* codes,
                                       const float* scales, int32_t top_pages,
                                       int32_t keep_first, int32_t keep_last, void* workspace,
                                       size_t ws_bytes, int32_t* sel_table, int32_t* sel_lengths,
                                       int32_t* dev_status, void* stream) {
  SelectParams p;
  mla_status st = prepare_select("mla_select_pages", dims, paging, io_dtype, q_len, q_abs, q_pe,
                                 block_table, lengths, codes, scales, top_pages, keep_first,
                                 keep_last, workspace, ws_bytes, sel_table, sel_lengths,
                                 dev_status, &p);
  if (st != MLA_OK) return st;
  return launch_select("mla_select_pages", p, static_cast<cudaStream_t>(stream));
}

// The dims and paging of the attention over the kept pages: one table row per
// token, as long as the kept pages of the longest sequence can be.
static void kept_view(const mla_dims* dims, const mla_paging* paging, int q_len, int top,
                      mla_dims* d, mla_paging* pg) {
  *d = *dims;
  d->batch = dims->batch * q_len;
  const long long rows = static_cast<long long>(top) * paging->page_size;
  d->s_max = static_cast<int>(rows < dims->s_max ? rows : dims->s_max);
  *pg = *paging;
  pg->table_stride = top;
}

extern "C" size_t mla_sparse_workspace_bytes(const mla_dims* dims, const mla_paging* paging,
                                             int32_t io_dtype, int32_t q_len, int32_t top_pages,
                                             int32_t requested) {
  const char* who = "mla_sparse_workspace_bytes";
  if (check_select(who, dims, paging, io_dtype, q_len) != MLA_OK) return 0;
  if (top_pages < 1) {
    set_error("%s: top_pages=%d must be >= 1", who, top_pages);
    return 0;
  }
  mla_dims d;
  mla_paging pg;
  kept_view(dims, paging, q_len, top_pages, &d, &pg);
  const size_t attn = selected_workspace_bytes(who, &d, &pg, io_dtype, requested);
  return attn ? select_space(dims, paging, q_len).total + attn : 0;
}

extern "C" mla_status mla_decode_attn_sparse(
    const mla_dims* dims, const mla_paging* paging, int32_t io_dtype, int32_t q_len,
    const void* q_abs, const void* q_pe, const void* cache, const int32_t* block_table,
    const int32_t* lengths, const int8_t* codes, const float* scales, float softmax_scale,
    int32_t top_pages, int32_t keep_first, int32_t keep_last, int32_t num_splits, void* workspace,
    size_t ws_bytes, int32_t* sel_table, int32_t* sel_lengths, void* o_c, float* lse,
    int32_t* dev_status, void* stream) {
  const char* who = "mla_decode_attn_sparse";
  SelectParams p;
  mla_status st = prepare_select(who, dims, paging, io_dtype, q_len, q_abs, q_pe, block_table,
                                 lengths, codes, scales, top_pages, keep_first, keep_last,
                                 workspace, ws_bytes, sel_table, sel_lengths, dev_status, &p);
  if (st != MLA_OK) return st;
  mla_dims d;
  mla_paging pg;
  kept_view(dims, paging, q_len, top_pages, &d, &pg);
  const size_t mine = select_space(dims, paging, q_len).total;
  uint8_t* attn_ws = static_cast<uint8_t*>(workspace) + mine;
  // The attention's arguments are checked before the first launch.
  st = check_attn_selected(who, &d, &pg, io_dtype, q_abs, q_pe, cache, sel_table, sel_lengths,
                        softmax_scale, num_splits, attn_ws, ws_bytes - mine, o_c);
  if (st != MLA_OK) return st;
  p.early = 1;
  // What the attention can do before it knows its pages goes first.
  st = attn_queries(who, &d, &pg, io_dtype, q_abs, q_pe, sel_lengths, num_splits, attn_ws,
                    ws_bytes - mine, stream);
  if (st == MLA_OK) st = launch_select(who, p, static_cast<cudaStream_t>(stream));
  if (st != MLA_OK) return st;
  return attn_selected(who, &d, &pg, io_dtype, q_abs, q_pe, cache, sel_table, sel_lengths,
                       softmax_scale, num_splits, attn_ws, ws_bytes - mine, o_c, lse, dev_status,
                       stream);
}
