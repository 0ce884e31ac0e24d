// Parameters shared by the split kernels (the per-chunk half of
// mla_decode_attn) and the kernels that read their partials.
#pragma once

#include "mla_common.cuh"

namespace mla {

struct SplitParams {
  const void* q_abs;
  const void* q_pe;
  const void* cache;        // used by the fp32 kernel
  const int32_t* lengths;
  float* part_o;            // [B, H, splits, 512]: one (b, h)'s chunks contiguous
  float* part_lse;          // [B, H, splits]
  int32_t* status;
  int B, H, s_max, splits, chunk;  // B counts query groups: cache sequences x q_len
  int q_len;                // query tokens per cache sequence (1: ordinary decode)
  int tpc;                  // bf16 kernel, 32 columns: query groups per CTA (2: two tokens
                            // x 16 heads; 1: 32 heads of one token)
  float scale_log2;         // softmax_scale * log2(e)
  uint8_t* q_img;           // FP8: the query's E4M3 image per (sequence, head group)
  int fill_early;           // bf16 kernel: issue tile 0's first boxes before the length
                            // is known (a one-wave grid)
  int persist;              // bf16 kernel, 16 heads per CTA: a persistent grid whose CTAs
                            // take several chunks each (chunk % 128 == 0)
  // Test hooks of the bf16 kernel (see mla_test_set_split_hooks), 0 in normal use:
  unsigned long long wait_ns;   // limit of each bounded wait (0: kWaitNs)
  int stop_after_tiles;         // ring A issues only this many tiles of a chunk (0: all)
  int32_t* debug;               // where timed-out CTAs record their first failed wait
  // Paged cache: row r of sequence b is pool row
  // table[b * table_stride + (r >> page_shift)] * 2^page_shift + r % 2^page_shift.
  const int32_t* table;         // NULL: a dense cache
  int table_stride, page_shift, num_pages;
  int io_bf16;                  // paged calls: q_abs, q_pe and o_c are bf16 (else fp32)
  // Paged calls with one chunk per sequence: the partial is the result, so the
  // split writes o_c (part_o, fp32 or bf16) and lse (part_lse, may be NULL) itself
  // and no combine follows.
  int direct;
  // Attention over a page selection: table and lengths come from the kernel just before
  // (which lets this one start early), so they are read after the PDL wait; the queries'
  // FP8 codes were made before the selection.
  int late;
  // Equal shares (take_share): how many partials each query group has; NULL otherwise.
  int32_t* pieces;
  void* out;                    // SM pairs, equal shares: o_c (else NULL) and lse (may be
  float* out_lse;               // NULL), where an item that is a whole set writes its result
};

// o_c = 0 and lse = -inf of `heads` heads from `row` (query group x H + head), which
// attend no row (direct calls; `threads` threads of the CTA, after the PDL wait).
__device__ __forceinline__ void write_no_rows(const SplitParams& p, size_t row, int heads,
                                              int tid, int threads) {
  const size_t bytes = p.io_bf16 ? 2 : 4;
  uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(p.part_o) + row * kDc * bytes);
  for (int i = tid; i < static_cast<int>(heads * kDc * bytes / 16); i += threads)
    o[i] = make_uint4(0, 0, 0, 0);
  if (p.part_lse)
    for (int i = tid; i < heads; i += threads) p.part_lse[row + i] = __uint_as_float(0xff800000u);
}

// The page that holds row r of cache sequence `seq`, or -1 (reported) when the
// table's entry names none.  r lies inside the sequence.
__device__ __forceinline__ int page_of(const SplitParams& p, int seq, int r) {
  const int id = p.table[static_cast<size_t>(seq) * p.table_stride + (r >> p.page_shift)];
  if (static_cast<unsigned>(id) < static_cast<unsigned>(p.num_pages)) return id;
  report(p.status, MLA_DEV_PAGE_OUT_OF_RANGE);
  return -1;
}

// First pool row of a box of rows r, r + 1, ... of one page (the box lies inside
// the page).  Boxes past the sequence's `len` rows, and boxes of pages that do
// not exist, start past the pool: TMA fills them with zeros.
__device__ __forceinline__ int paged_row(const SplitParams& p, int seq, int r, int len) {
  const int id = r < len ? page_of(p, seq, r) : -1;
  return id < 0 ? p.num_pages << p.page_shift
                : (id << p.page_shift) + (r & ((1 << p.page_shift) - 1));
}

// FP8 cache: the query of one (sequence, 16-head group) as the split kernel's
// shared memory holds it -- five 128-column boxes of 64 rows (4 E4M3 parts x
// 16 heads) x 128 bytes, 128-byte swizzled -- followed by the 16 per-head
// power-of-two scales (fp32).  Written once per step into the workspace.
constexpr size_t kFp8QBoxes = 5 * 64 * 128;
constexpr size_t kFp8QImage = kFp8QBoxes + 16 * sizeof(float);

// Query group v (one token of one sequence) reads cache sequence v / q_len.
__device__ __forceinline__ int cache_seq(const SplitParams& p, int v) { return v / p.q_len; }

// Rows query group v attends.  Token i of a q_len-token step sits at position
// lengths[b] - q_len + i (the cache already holds all q_len new rows), and a
// key past the query's own position is masked ("Transformer and KV Cache
// Basics", mask design for multi-token decoding), so the token sees the first
// lengths[b] - (q_len - 1 - i) rows.  A length outside [q_len, s_max] is
// reported and clamped.
__device__ __forceinline__ int clamp_rows(const SplitParams& p, bool report_it,
                                          int full, int back) {   // the length as given, q_len - 1 - i
  if (full < p.q_len || full > p.s_max) {
    if (report_it) report(p.status, MLA_DEV_LENGTH_OUT_OF_RANGE);
    full = full < 0 ? 0 : (full > p.s_max ? p.s_max : full);
  }
  const int len = full - back;
  return len < 0 ? 0 : len;
}
__device__ __forceinline__ int clamp_length(const SplitParams& p, int v, bool report_it, int full) {
  return clamp_rows(p, report_it, full, p.q_len == 1 ? 0 : p.q_len - 1 - v % p.q_len);
}
// The same without a branch for one token.  The persistent planner and the fused tail keep
// this form: with the branch the whole step of 4 x 65536 rows in 128 chunks takes 78.2 us
// against 76.2 and that of 8 x 4096 rows 16.93 against 16.88.  The one-item kernels gain by
// the branch: 32 x 16384 rows x 128 heads 275 us against 278.
__device__ __forceinline__ int plain_length(const SplitParams& p, int v, bool report_it) {
  return clamp_rows(p, report_it, p.lengths[v / p.q_len], p.q_len - 1 - v % p.q_len);
}
__device__ __forceinline__ int clamp_length(const SplitParams& p, int v, bool report_it) {
  return clamp_length(p, v, report_it, p.lengths[p.q_len == 1 ? v : v / p.q_len]);
}

// Eight bf16 or sixteen E4M3 values with NaN and infinities (E4M3 has none) as zeros.
template <bool kFp8>
__device__ __forceinline__ uint4 finite_only(uint4 v) {
  auto word = [](uint32_t w) {
    return w & ~(kFp8 ? __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu)
                      : __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u));
  };
  return make_uint4(word(v.x), word(v.y), word(v.z), word(v.w));
}

// Exclusive prefix sum of x over the warp's lanes, and the warp's total.
__device__ __forceinline__ int warp_exclusive_scan(int x, int lane, int* total) {
  int incl = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  *total = __shfl_sync(0xffffffffu, incl, 31);
  return incl - x;
}

// Equal shares of a paged call's tiles.  The tiles of all its rows sets -- one per query
// group, or per sequence where a kernel takes a sequence's tokens together (kSeq) -- one
// after another are cut into runs of `each`, one per CTA or pair of CTAs.  A run may end
// inside a set and start with the rest of another; each (run, set) that meet is an item and
// gives one partial.  A set of n tiles has at most ceil(n / each) + 1 of them, which `each`
// keeps within p.splits.
constexpr int kShareSets = 512;   // sets the planning warp holds, 16 a lane
struct TileShare {
  int each;    // tiles per run
  int first;   // this run's first tile among all
  int tiles;   // and how many it has
  int v, off;  // its first tile: tile `off` of set v
};
struct TileItem {
  int v, j;       // set, index of the partial among the set's own
  int r0, tiles;  // first row, 128-row tiles
  int len;        // rows of the set
};
template <bool kSeq>
__device__ __forceinline__ int set_length(const SplitParams& p, int v) {
  return clamp_length(p, kSeq ? (v + 1) * p.q_len - 1 : v, false);
}
// Run c of `runs`, by one whole warp.
template <bool kSeq>
__device__ __forceinline__ TileShare take_share(const SplitParams& p, int c, int runs, int lane,
                                                bool report_it) {
  constexpr int kEach = kShareSets / 32;
  const int sets = kSeq ? p.B / p.q_len : p.B;
  int n[kEach], sum = 0, top = 0;
  // All loads first (a report may follow each check, and no load moves above it); blocks of
  // 32 sets that are not there are skipped, not computed.
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int v = 32 * i + lane;
    n[i] = 0;
    if (32 * i < sets && v < sets) n[i] = p.lengths[kSeq || p.q_len == 1 ? v : v / p.q_len];
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (32 * i >= sets) break;
    const int v = 32 * i + lane;
    if (v < sets)
      n[i] = (clamp_length(p, kSeq ? (v + 1) * p.q_len - 1 : v, report_it, n[i]) + 127) / 128;
    sum += n[i];
    top = max(top, n[i]);
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  top = __reduce_max_sync(0xffffffffu, top);
  TileShare s;
  s.each = max(1, max((sum + runs - 1) / runs, (top + p.splits - 2) / (p.splits - 1)));
  s.first = static_cast<int>(min(static_cast<long long>(c) * s.each, static_cast<long long>(sum)));
  s.tiles = min(s.each, sum - s.first);
  s.v = s.off = 0;
  int base = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (32 * i >= sets || base > s.first) break;
    int total;
    const int at = base + warp_exclusive_scan(n[i], lane, &total);
    const uint32_t hit = __ballot_sync(0xffffffffu, s.first >= at && s.first < at + n[i]);
    if (hit) {
      const int src = __ffs(hit) - 1;
      s.v = 32 * i + src;
      s.off = s.first - __shfl_sync(0xffffffffu, at, src);
      break;
    }
    base += total;
  }
  return s;
}
// A value that all lanes hold, known to the compiler as such: what decides the loops around
// the warps' MMAs and copies has to be, or their operands are moved lane by lane.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
// The first item of run c, which has tiles; by whole warps, as next_item.
template <bool kSeq>
__device__ __forceinline__ TileItem first_item(const SplitParams& p, const TileShare& s, int c) {
  const int v = uniform(s.v), off = uniform(s.off), len = uniform(set_length<kSeq>(p, v));
  return TileItem{v, off > 0 ? c - (s.first - off) / s.each : 0, off * 128,
                  uniform(min((len + 127) / 128 - off, s.tiles)), len};
}
// The item after `it`, with `left` > 0 tiles of the run to go: the start of the next set
// that has any row.  (The bounds matter only if the lengths change under the kernel.)
template <bool kSeq>
__device__ __forceinline__ TileItem next_item(const SplitParams& p, TileItem it, int left) {
  const int sets = kSeq ? p.B / p.q_len : p.B;
  do {
    it.v = uniform(min(it.v + 1, sets - 1));
    it.len = uniform(set_length<kSeq>(p, it.v));
  } while (it.len == 0 && it.v + 1 < sets);
  it.j = it.r0 = 0;
  it.tiles = uniform(max(1, min((it.len + 127) / 128, left)));
  return it;
}
// Whether an item is its whole set.
__device__ __forceinline__ bool whole_set(const TileItem& it) {
  return it.r0 == 0 && it.tiles * 128 >= it.len;
}
// Partials of a set whose first tile is tile s of all.
__device__ __forceinline__ int count_pieces(const TileItem& it, int s, int each) {
  return (s + (it.len + 127) / 128 - 1) / each - s / each + 1;
}

// The FP8 (E4M3) cache's split kernel (mla_fp8.cu): same grid, partials and
// launch overlap as the bf16 one.
// It runs as two launches: the query's E4M3 image, then the split itself.
mla_status launch_split_fp8(const SplitParams& p, const void* cache, cudaStream_t stream,
                            const char* who);
// Runs of an equal-share grid whose rows each pass `ctas` CTAs: one CTA per SM.
int share_runs(int ctas);

// The paged split with bf16 queries as SM pairs (mla_pair.cu): the query rows of a
// sequence (heads x tokens) in groups of up to 128, two CTAs a group; same partials,
// chunks of whole tiles.  With an E4M3 cache the queries' codes go to p.q_img first.
constexpr int kPairRows = 128;
constexpr int pair_groups(int rows) { return (rows + kPairRows - 1) / kPairRows; }
mla_status launch_split_pair(const SplitParams& p, const void* cache, bool fp8,
                             cudaStream_t stream, const char* who);

// The kernels that make the queries' FP8 codes, which both calls above run first unless
// p.late is set.
mla_status launch_fp8_queries(const SplitParams& p, cudaStream_t stream, const char* who);
mla_status launch_pair_queries(const SplitParams& p, cudaStream_t stream, const char* who);

// Rows a cache view holds: B / q_len sequences of s_max rows, or a pool's pages.
inline uint64_t view_rows(const SplitParams& p) {
  return p.table ? static_cast<uint64_t>(p.num_pages) << p.page_shift
                 : static_cast<uint64_t>(p.B / p.q_len) * p.s_max;
}

// mla_absorb_q's work (named `who` in error messages), with the decode kernel's
// first cache rows prefetched into L2 when pf.cache is set, and (bf16, `early`)
// launched with programmatic stream serialization (mla_proj.cu).  `q_host`:
// whether q_nope is page-locked host memory, 1 or 0 when the caller knows it,
// -1 to ask the runtime.
mla_status absorb_q(const char* who, const mla_dims* dims, const void* q_nope, const void* q_rope,
                    const void* w_uk, const int32_t* positions, double rope_base, void* q_abs,
                    void* q_pe, void* stream, const CachePrefetch& pf, bool early,
                    int q_host = -1);

}  // namespace mla
