// The paged split for bf16 queries: a pair of SMs takes up to 128 query rows (heads, and
// the tokens of a multi-token step, which attend the same sequence) of one sequence.
//
// Per head the score of row t is q . c_t / sqrt(d_h + d_R), an online softmax over
// the chunk's rows, and o = sum_t p_t c_t ("Multi-Head Latent Attention" 3.3, 3.6;
// every head reads the same row).  At 128 heads a cached bf16 row costs 278 kFLOP,
// so what bounds the kernel is how the rows reach the tensor cores: with 64 heads
// per CTA every row crosses L2 -> SM twice per product and its MMAs (M = 128 rows,
// N = 64 heads) read it again from shared memory for every 64 heads.
//
// Here heads are the M of the MMAs and rows (or latent columns) the N, and two CTAs
// of a cluster work as one tcgen05 pair (cta_group::2): CTA i holds half of the heads
// (64 of 128) as its half of A, and each brings only half of every B operand:
//   scores  S[128 heads x 128 rows] = Q[128 x 576] . C^T     CTA i: rows 64 i ..
//   output  O[128 x 512] += P[128 x 128 rows] . C[128 x 512]  CTA i: 256 of the latent
//                                                             columns, all 128 rows
// so per tile and CTA 74 KB of score operand (from HBM) and 64 KB of output operand
// (from L2) are read for 64 x 128 x 1088 products.  The heads lie on tensor-memory
// lanes: a softmax thread holds 32 scores of one head, so row maxima are register
// maxima and one exchange of four values, where rows on lanes need a reduction over
// 128 of them per head.
//
// bf16 cache: the queries are bf16 as they are and P is rounded once to bf16 (at most
// 2^-8 relative and unbiased, so less in the weighted sum than the bf16 output's own
// rounding).  E4M3 cache (kind::f8f6f4): a query (8 significant bits) is exactly the sum
// of two E4M3 parts in units of a power of two per head (what falls below the second
// part's smallest step is 2^-17 of the head's largest value), and P is an E4M3 part and
// its remainder as E5M2 (2^-7 at most).  The parts have equal weight, so they accumulate
// in the same accumulators, as twice the K.  E5M2's exponents keep small weights: with
// the softmax's reference 2^3 below the running maximum, whose room up to 2^8.5 lets the
// maximum grow 2^5.5 before O is rescaled, the smallest step is 2^-19 of the largest
// weight.  (An E4M3 remainder is twice as exact for large weights but ends at 2^-9, which
// wants the reference at 2^7 and leaves 2^1.5: O was then rescaled in most of a chunk's
// first tiles, at 2000 cycles.)
//
// Tensor memory per CTA: S_0 and S_1 (the scores are their sum; each has its own issuing
// warp), two buffers of 64 columns each (lane l < 64: head l, rows 0-63
// of the tile; lane 64 + l: head l, rows 64-127), O two tiles of 128 columns (lane l:
// head l, latents 256 j + 0..127; lane 64 + l: 256 j + 128..255).
//
// Warps: 8 (bf16) or 16 (E4M3) softmax and epilogue; then one each for the score rows
// (TMA) and for the query and the output operand (TMA), two for the score MMAs and two
// for the output MMAs (the even CTA's issue for the pair); with equal shares one more for
// the later items' queries.  The even CTA's barriers collect both CTAs' copies and softmax
// warps; tcgen05.commit signals both CTAs.  Every wait is bounded.
#include <cuda_fp8.h>
#include <cudaTypedefs.h>

#include "mla_pair.cuh"

namespace mla {
namespace {

template <bool kFp8>
struct PairPlan {
  // Softmax warps: each thread takes kCols scores of one head.  E4M3's conversions make its
  // softmax the longest stage of a tile, so it gets twice the warps.
  static constexpr int kSoftWarps = kFp8 ? 16 : 8, kSoft = 32 * kSoftWarps;
  static constexpr int kThreads = kSoft + 6 * 32, kShareThreads = kThreads + 32;
  static constexpr int kSlices = kSoftWarps / 4, kCols = 64 / kSlices;
  static constexpr int kBoxCols = kFp8 ? 128 : 64;          // columns of a 128-byte box
  static constexpr int kBoxes = kFp8 ? 5 : 9;               // score boxes of a row
  static constexpr int kParts = kFp8 ? 2 : 1;
  static constexpr int kQBytes = kParts * kBoxes * kPBox;
  static constexpr int kUnit = kFp8 ? kPBox : 2 * kPBox;    // 64 rows x 128 latent columns
  // Even ring lengths: two issuers take alternate positions, so each meets a slot's
  // phases in order (a parity wait may not run two phases ahead).
  static constexpr int kSlotsS = 8, kSlotsV = 4;
  static constexpr int kPBufs = kFp8 ? 2 : 1;   // P buffers: what room is left
  static constexpr uint32_t kOCol = 256;   // O after S_0 and S_1, two buffers each
  static constexpr int kOffQ = 0;
  static constexpr int kOffS = kOffQ + kQBytes;
  static constexpr int kOffV = kOffS + kSlotsS * kPBox;
  static constexpr int kOffP = kOffV + kSlotsV * kUnit;
  static constexpr int kOffRed = kOffP + kPBufs * kPBufBytes;   // [2][2 kSlices][64] maxima
  static constexpr int kOffSum = kOffRed + 2 * 2 * kSlices * kPHeads * 4;   // row sums
  static constexpr int kOffBar = kOffSum + 2 * kSlices * kPHeads * 4;
  // full / empty of the rings; S and P hand-overs; the query; the units to clean; the
  // query read for the last time (kShare)
  static constexpr int FULLS = 0, EMPTYS = FULLS + kSlotsS, FULLV = EMPTYS + kSlotsS,
                       EMPTYV = FULLV + kSlotsV, SREADY = EMPTYV + kSlotsV, SFREE = SREADY + 2,
                       PREADY = SFREE + 2, PVDONE = PREADY + 2, QFULL = PVDONE + 2,
                       CLEANV = QFULL + 1, CLEANED = CLEANV + 4, QFREE = CLEANED + 4, kBars = QFREE + 1;
  static constexpr int kOffSlot = kOffBar + 8 * kBars;
  static constexpr int kOffAbort = kOffSlot + 8;
  static constexpr int kOffShare = kOffAbort + 8;   // TileShare of the pair
  static constexpr size_t kSmem = 1024 + kOffShare + 24;
  // Reference of the softmax below the running maximum, and how far a maximum may
  // pass it before O is rescaled (log2): E4M3 weights stay in [0, 2^8.5].
  static constexpr float kBias = kFp8 ? 3.f : 0.f, kGrow = kFp8 ? 5.5f : 8.f;
  // Epilogue staging (over the query, the rings and P): 64 rows of 512 values, 16 bytes
  // apart.
  static constexpr int kStageRow = kDc * 4 + 16;
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kOffRed >= kPHeads * kStageRow, "epilogue staging");
  static_assert(kPBufs * kPBufBytes == kSoftWarps * 32 * 64, "an item's output through P");
  static_assert(kSlotsS % 2 == 0 && kSlotsV == 4, "ring lengths");
  static_assert(kOffS % 1024 == 0 && kOffV % 1024 == 0 && kOffP % 1024 == 0, "swizzle atoms");
  static_assert(kOffBar % 8 == 0, "mbarriers");
};

// Two E4M3 parts of v in units of 2^(e - 8), where 2^e bounds the head's largest
// magnitude: row r H + h of part i at codes + (i R H + r H + h) 640, columns 576-639
// zero; the unit at sigma[r H + h].  One warp per (token, head).
__global__ void __launch_bounds__(128) pair_query_kernel(const SplitParams p, uint8_t* codes,
                                                         float* sigma) {
  pdl_launch_dependents();   // the split may set up meanwhile
  const int lane = threadIdx.x & 31;
  const size_t rh = static_cast<size_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const size_t rows = static_cast<size_t>(p.B) * p.H;
  pdl_wait();
  if (rh >= rows) return;
  float2 v[9];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 9; ++i) {
    const __nv_bfloat16* q = i < 8 ? static_cast<const __nv_bfloat16*>(p.q_abs) + rh * kDc + 64 * i
                                   : static_cast<const __nv_bfloat16*>(p.q_pe) + rh * kDr;
    v[i] = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(q)[lane]);
    top = fmaxf(top, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  int ex = 0;
  frexpf(top, &ex);   // top = f 2^ex, f in [0.5, 1)
  ex = max(ex, -100);   // keeps 1 / unit finite; smaller queries score as zero to 2^-100
  const float unit = ldexpf(1.f, ex - 8), inv = ldexpf(1.f, 8 - ex);
  if (lane == 0) sigma[rh] = unit;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    uint16_t hi = 0, lo = 0;
    if (i < 9) {
      const float x = v[i].x * inv, y = v[i].y * inv;
      hi = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
      const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(hi, __NV_E4M3)));
      lo = __nv_cvt_float2_to_fp8x2(make_float2(x - f.x, y - f.y), __NV_SATFINITE, __NV_E4M3);
    }
    reinterpret_cast<uint16_t*>(codes + rh * kQ8Row + 64 * i)[lane] = hi;
    reinterpret_cast<uint16_t*>(codes + (rows + rh) * kQ8Row + 64 * i)[lane] = lo;
  }
}

// kShare: one pair per two SMs takes an equal run of all sequences' tiles (take_share), an
// item per sequence it meets; the next item's rows and query are fetched and its scores
// computed while the last one's output is written (a change of item costs about 2.5 us, the
// softmax of its first tile behind that write).  Otherwise a pair has one item, its chunk.
// 64 sequences of 512 to 8192 bf16 rows x 32 heads 110 -> 77 us, x 128 heads 113 -> 91.
template <bool kFp8, bool kShare>
__global__ void __launch_bounds__(kShare ? PairPlan<kFp8>::kShareThreads
                                         : PairPlan<kFp8>::kThreads, 1)
    split_pair_kernel(const __grid_constant__ CUtensorMap tmap,
                      const __grid_constant__ CUtensorMap tmap_q,
                      const __grid_constant__ CUtensorMap tmap_qpe, const SplitParams p,
                      const float* __restrict__ sigma) {
  using L = PairPlan<kFp8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem), bars = sbase + L::kOffBar;
  float* red = reinterpret_cast<float*>(smem + L::kOffRed);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffAbort);
  uint32_t* slot_ptr = reinterpret_cast<uint32_t*>(smem + L::kOffSlot);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // uniform to the compiler
  // Query rows (tokens x heads) of the sequence, dealt evenly to its CTAs: this CTA's
  // are flat0 .. flat0 + mine - 1 of all; rows past them up to 64 are computed as well
  // (other rows of the query, or zeros) and dropped.
  const int all = p.q_len * p.H, parts = kShare ? 2 * pair_groups(all) : gridDim.x;
  const int dealt = (all + parts - 1) / parts, part = kShare ? blockIdx.x % parts : blockIdx.x;
  const int first = part * dealt, mine = min(dealt, all - first);
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  if (p.late) pdl_wait();
  // Rows of a sequence, all of which its last token attends, count.
  TileItem item0{0, 0, 0, 0, 0};   // the pair's first item (none: T = 0)
  int T = 0;        // tiles of the pair
  TileShare share;
  if (!kShare) {
    const int j = blockIdx.y, seq = blockIdx.z;
    const int len =
        clamp_length(p, (seq + 1) * p.q_len - 1, tid == 0 && blockIdx.x == 0 && j == 0);
    const int r0 = j * p.chunk;
    if (r0 >= len) {   // both CTAs of the pair: the chunk lies past the sequence
      if (p.direct || r0 == 0) pdl_wait();   // no row at all: see launch_pdl
      if (p.direct) write_no_rows(p, seq * all + first, mine, tid, L::kThreads);
      return;
    }
    T = (min(r0 + p.chunk, len) - r0 + kTileRows - 1) / kTileRows;
    item0 = TileItem{seq, j, r0, T, len};
  }
  // Rows past the sequence's end may hold anything (NaN included), and so may, for the
  // tokens that do not attend them, the rows of the step's later tokens: from the first row
  // that some token does not attend on, the output operand is cleaned.  Tiles of an item
  // before its first one to clean:
  auto clean_tiles = [&](const TileItem& it) {
    return min(it.tiles, max(it.len - (p.q_len - 1) - it.r0, 0) / kTileRows);
  };
  auto item_after = [&](const TileItem& it, int t) { return next_item<true>(p, it, T - t); };
  const uint32_t lead = mapa_shared(bars, 0);   // the even CTA's barriers
  auto bar = [&](int i) { return bars + 8 * i; };
  auto lbar = [&](int i) { return lead + 8 * i; };

  if (tid == L::kSoft) {
    for (int i = 0; i < L::kSlotsS; ++i) {
      mbar_init(bar(L::FULLS + i), 1);
      mbar_init(bar(L::EMPTYS + i), 1);
    }
    for (int i = 0; i < L::kSlotsV; ++i) {
      mbar_init(bar(L::FULLV + i), 1);
      mbar_init(bar(L::EMPTYV + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(L::SREADY + i), 2);                 // one commit per issuer
      mbar_init(bar(L::SFREE + i), 2 * L::kSoftWarps);  // both CTAs' softmax warps
      mbar_init(bar(L::PREADY + i), 2 * L::kSoftWarps);
      mbar_init(bar(L::PVDONE + i), 2);
    }
    mbar_init(bar(L::QFULL), 1);
    mbar_init(bar(L::QFREE), 2);   // one commit per score issuer
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(L::CLEANV + i), 1);
      mbar_init(bar(L::CLEANED + i), 2 * L::kSoftWarps);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
    prefetch_tmap(&tmap);
    prefetch_tmap(&tmap_q);
    if (!kFp8) prefetch_tmap(&tmap_qpe);
  }
  if (kShare && warp == L::kSoftWarps) {
    __syncwarp();
    share = take_share<true>(p, blockIdx.x / parts, gridDim.x / parts, lane, blockIdx.x == 0);
    if (lane == 0) *reinterpret_cast<TileShare*>(smem + L::kOffShare) = share;
  }
  // Role warps after the softmax warps.
  constexpr int kWarpS = L::kSoftWarps, kWarpV = kWarpS + 1, kWarpScore = kWarpS + 2,
                kWarpOut = kWarpS + 4, kWarpQuery = kWarpS + 6;   // the last of kShare only
  if (warp == kWarpScore) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(slot_ptr)),
                 "r"(kPTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // the barriers of both CTAs exist
  tc_fence_after();
  const uint32_t tmem = *slot_ptr;
  if (kShare) {
    share = *reinterpret_cast<const TileShare*>(smem + L::kOffShare);
    T = uniform(max(share.tiles, 0));   // none: more pairs than tiles
    if (T > 0)
      item0 = first_item<true>(p, share, blockIdx.x / parts);
    else
      pdl_wait();
  }
  // This CTA's half of the queries of sequence v, by a whole warp after its PDL wait.
  auto load_query = [&](int v) {
    const uint64_t stream = l2_evict_first_policy();
    const int flat0 = v * all + first;
    if (leader) expect_tx_elected(bar(L::QFULL), 2 * L::kQBytes);
#pragma unroll 1
    for (int i = 0; i < L::kParts * L::kBoxes; ++i) {
      if (kFp8)
        tma_load_pair(sbase + L::kOffQ + i * kPBox, &tmap_q, 128 * (i % L::kBoxes),
                      (i / L::kBoxes) * p.B * p.H + flat0, lbar(L::QFULL), stream);
      else
        tma_load_pair(sbase + L::kOffQ + i * kPBox, i < 8 ? &tmap_q : &tmap_qpe,
                      i < 8 ? 64 * i : 0, flat0, lbar(L::QFULL), stream);
    }
  };

  // Pieces of one page each: rows of a box, and pieces of 64 rows.
  const int brows = min(1 << p.page_shift, 64), np = 64 / brows;

  if (warp == kWarpS) {
    // ------------------------------------------------------------ score rows (HBM)
    // This CTA's 64 rows of each tile; lane i < np holds piece i's pool row.
    const uint64_t keep = l2_evict_last_policy();   // read again as the output operand
    auto rows_of = [&](const TileItem& it, int i) {
      return paged_row(p, it.v, it.r0 + i * kTileRows + 64 * rank + lane * brows,
                       lane < np ? it.len : 0);
    };
    TileItem it = item0;
    int row = T > 0 ? rows_of(it, 0) : 0, sl = 0;
    uint32_t phase = 1;   // of the slot's release before this use: the first uses pass
    for (int t0 = 0; t0 < T;) {   // items
      const int end = t0 + it.tiles;
      TileItem then = it;
      if (kShare && end < T) then = item_after(it, end);
      for (int i = 0; i < it.tiles; ++i) {
        const int next = i + 1 < it.tiles     ? rows_of(it, i + 1)
                         : kShare && end < T ? rows_of(then, 0)
                                             : 0;
        if (__any_sync(0xffffffffu, *abort_flag)) break;
#pragma unroll 1
        for (int k = 0; k < L::kBoxes; ++k) {
          warp_wait(bar(L::EMPTYS + sl), phase, abort_flag);
          if (leader) expect_tx_elected(bar(L::FULLS + sl), 2 * kPBox);
          const uint32_t dst = sbase + L::kOffS + sl * kPBox, full = lbar(L::FULLS + sl);
#pragma unroll 1
          for (int i = 0; i < np; ++i)
            tma_load_pair(dst + i * brows * 128, &tmap, L::kBoxCols * k,
                          __shfl_sync(0xffffffffu, row, i), full, keep);
          if (++sl == L::kSlotsS) {
            sl = 0;
            phase ^= 1;
          }
        }
        row = next;
      }
      t0 = end;
      it = then;
    }
  } else if (kShare && warp == kWarpQuery) {
    // ------------------------------------------------------------ the later items' queries
    // Each once the scores of the item before are done, which read the query it replaces.
    TileItem it = item0;
    for (int t = it.tiles, n = 0; 0 < t && t < T; t += it.tiles, ++n) {
      it = item_after(it, t);
      warp_wait(bar(L::QFREE), n & 1, abort_flag);
      if (__any_sync(0xffffffffu, *abort_flag)) break;
      pdl_wait();
      load_query(it.v);
    }
  } else if (warp == kWarpV) {
    // ------------------------------------------------------------ query, output operand (L2)
    const uint64_t stream = l2_evict_first_policy();
    pdl_wait();   // the query comes from the kernel before
    if (T > 0) load_query(item0.v);
    // Unit u of a tile: row half u >> 1, latent columns 256 (u & 1) + 128 rank ..;
    // lane i < 2 np holds the pool row of piece i of the tile's 128 rows.
    auto rows_of = [&](const TileItem& it, int i) {
      return paged_row(p, it.v, it.r0 + i * kTileRows + lane * brows, lane < 2 * np ? it.len : 0);
    };
    TileItem it = item0;
    int row = T > 0 ? rows_of(it, 0) : 0, sl = 0;
    uint32_t phase = 1;
    for (int t0 = 0; t0 < T;) {   // items
      const int end = t0 + it.tiles;
      const int clean = clean_tiles(it);
      TileItem then = it;
      if (kShare && end < T) then = item_after(it, end);
      for (int i = 0; i < it.tiles; ++i) {
        const bool own = i >= clean;   // these land on the CTA's own barriers
        const int next = i + 1 < it.tiles     ? rows_of(it, i + 1)
                         : kShare && end < T ? rows_of(then, 0)
                                             : 0;
        if (__any_sync(0xffffffffu, *abort_flag)) break;
#pragma unroll 1
        for (int u = 0; u < 4; ++u) {
          warp_wait(bar(L::EMPTYV + sl), phase, abort_flag);
          if (own)
            expect_tx_elected(bar(L::CLEANV + u), L::kUnit);
          else if (leader)
            expect_tx_elected(bar(L::FULLV + sl), 2 * L::kUnit);
          const uint32_t full = own ? mapa_shared(bar(L::CLEANV + u), rank) : lbar(L::FULLV + sl);
          const uint32_t dst = sbase + L::kOffV + sl * L::kUnit;
          const int x = 256 * (u & 1) + 128 * rank;
#pragma unroll 1
          for (int i = 0; i < np; ++i) {
            const int r = __shfl_sync(0xffffffffu, row, (u >> 1) * np + i);
            tma_load_pair(dst + i * brows * 128, &tmap, x, r, full, stream);
            if (!kFp8)   // a bf16 unit is two 64-column boxes
              tma_load_pair(dst + kPBox + i * brows * 128, &tmap, x + 64, r, full, stream);
          }
          if (++sl == L::kSlotsV) {
            sl = 0;
            phase ^= 1;
          }
        }
        row = next;
      }
      t0 = end;
      it = then;
    }
  } else if (warp == kWarpScore || warp == kWarpScore + 1) {
    // ------------------------------------------------------------ score MMAs (even CTA)
    // Issuer i takes the boxes of the stream with parity i (so every other ring slot)
    // into accumulators S_i, which the softmax adds.  The whole warp runs along,
    // converged at every MMA and commit; a wait that gave up shows in the abort flag,
    // looked at once a tile.  Not unrolled over boxes: these warps run each instruction
    // once a tile, and straight code for 36 MMAs is fetched anew every time.
    if (leader) {
      const int i = warp - kWarpScore;
      constexpr uint32_t idesc = (1u << 4) | (kFp8 ? 0u : (1u << 7) | (1u << 10)) |
                                 (128u >> 3 << 17) | (128u >> 4 << 24);
      const uint64_t q0 = umma_desc_sw128(sbase + L::kOffQ, 16, 1024);
      const uint64_t s0 = umma_desc_sw128(sbase + L::kOffS, 16, 1024);
      TileItem it = item0;
      for (int t0 = 0, n = 0; t0 < T; ++n) {   // items
        const int end = t0 + it.tiles;
        warp_wait(bar(L::QFULL), n & 1, abort_flag);
        if (kShare && warp == kWarpScore && blockIdx.x % parts == 0 && it.r0 == 0)
          // The run with a sequence's first tile says how many runs it spans.  (Not before a
          // query is here, fetched behind the PDL wait: the combine of the call before may
          // still be reading its own counts.)
          for (int q = lane; q < p.q_len; q += 32)
            p.pieces[it.v * p.q_len + q] = count_pieces(it, share.first + t0, share.each);
        for (int t = t0; t < end; ++t) {
          const int sb = t & 1;
          if (t >= 2) warp_wait(bar(L::SFREE + sb), ((t - 2) >> 1) & 1, abort_flag);
          if (__any_sync(0xffffffffu, *abort_flag)) break;
          const uint32_t d = tmem + 128 * i + 64 * sb;
          uint32_t more = 0;
#pragma unroll 1
          for (int k = (L::kBoxes * t + i) & 1; k < L::kBoxes; k += 2) {
            const int pos = L::kBoxes * t + k, sl = pos % L::kSlotsS;
            warp_wait(bar(L::FULLS + sl), (pos / L::kSlotsS) & 1, abort_flag);
            tc_fence_after();
            const uint64_t b = s0 + static_cast<uint64_t>(sl * (kPBox >> 4));
#pragma unroll
            for (int part = 0; part < L::kParts; ++part) {
              const uint64_t a = q0 + static_cast<uint64_t>((part * L::kBoxes + k) * (kPBox >> 4));
              // 32 bytes of K a step; the fifth E4M3 box holds 64 columns: two steps
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                if (!kFp8 || ks < 2 || k < 4)
                  mma_pair<kFp8>(d, a + 2 * ks, b + 2 * ks, idesc, part > 0 || ks > 0 ? 1u : more);
            }
            more = 1;
            commit_pair(bar(L::EMPTYS + sl));
          }
          commit_pair(bar(L::SREADY + sb));
        }
        t0 = end;
        if (kShare && t0 < T) {
          commit_pair(bar(L::QFREE));
          it = item_after(it, t0);
        }
      }
    }
  } else if (warp == kWarpOut || warp == kWarpOut + 1) {
    // ------------------------------------------------------------ output MMAs (even CTA)
    // Issuer jj takes the units of O tile jj.
    if (leader) {
      const int jj = warp - kWarpOut;
      constexpr uint32_t idesc = (1u << 4) | (kFp8 ? 0u : (1u << 7) | (1u << 10)) | (1u << 16) |
                                 (256u >> 3 << 17) | (128u >> 4 << 24);
      const uint64_t p0 = umma_desc_sw128(sbase + L::kOffP, 16, 1024);
      // rows (K) in groups of eight 1024 bytes apart; bf16: two 64-column boxes
      const uint64_t v0 = umma_desc_sw128(sbase + L::kOffV, kPBox, 1024);
      const uint32_t d = tmem + L::kOCol + 128 * jj;
      TileItem it = item0;
      int cleaned = 0;   // cleaned tiles so far
      for (int t0 = 0; t0 < T;) {   // items
        const int end = t0 + it.tiles, clean = t0 + clean_tiles(it);
        for (int t = t0; t < end; ++t) {
          const int pb = t & 1;
          warp_wait(bar(L::PREADY + pb), (t >> 1) & 1, abort_flag);
          if (__any_sync(0xffffffffu, *abort_flag)) break;
#pragma unroll 1
          for (int kh = 0; kh < 2; ++kh) {
            // A tile's four units take the ring's four slots; cleaned ones pass FULLV by.
            const int u = 2 * kh + jj, sl = u;
            if (t >= clean)
              warp_wait(bar(L::CLEANED + u), cleaned & 1, abort_flag);
            else
              warp_wait(bar(L::FULLV + sl), (t - cleaned) & 1, abort_flag);
            tc_fence_after();
            const uint64_t b = v0 + static_cast<uint64_t>(sl * (L::kUnit >> 4));
            // 64 rows: bf16 four steps of 16 (2 KB of rows, 32 bytes of P's box kh); E4M3
            // two steps of 32 (4 KB; 32 bytes of each part's row, the half at byte 64 kh)
#pragma unroll
            for (int part = 0; part < L::kParts; ++part) {
              const uint64_t a = p0 + static_cast<uint64_t>(t % L::kPBufs * (kPBufBytes >> 4)) +
                                 ((kFp8 ? part * kPBox + 64 * kh : kh * kPBox) >> 4);
#pragma unroll
              for (int ks = 0; ks < (kFp8 ? 2 : 4); ++ks)
                mma_pair<kFp8>(d, a + 2 * ks, b + ks * ((kFp8 ? 4096 : 2048) >> 4),
                               idesc | (part == 1 ? 1u << 7 : 0u),   // the remainder is E5M2
                               part > 0 || ks > 0 ? 1u : (t > t0 || kh > 0 ? 1u : 0u));
            }
            commit_pair(bar(L::EMPTYV + sl));
          }
          commit_pair(bar(L::PVDONE + pb));
          if (t >= clean) ++cleaned;
        }
        t0 = end;
        if (kShare && t0 < T) it = item_after(it, t0);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    // Warp w: lanes 32 (w & 3) .. of tensor memory, so head 32 (w & 1) + lane of the
    // tile's row half (w >> 1) & 1, and the column slice w >> 2 of those 64 rows.
    constexpr int kCols = L::kCols, kSlices = L::kSlices;
    const int qd = warp & 3, hh = warp >> 2;
    const int head = 32 * (qd & 1) + lane, row0 = 64 * (qd >> 1) + kCols * hh;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * qd) << 16);
    const int part_of = kSlices * (qd >> 1) + hh;   // which part of the tile's rows
    const int back = p.q_len - 1 - (first + min(head, mine - 1)) / p.H;   // tokens behind its own
    TileItem it = item0;
    int cleaned = 0;   // cleaned tiles so far
    for (int t0 = 0; t0 < T;) {   // items; t0: the item's first tile among the pair's
      const int flat0 = it.v * all + first, tiles = it.tiles;
      const int clean = t0 + clean_tiles(it);
      // E4M3: the head's unit, written by the kernel before (known complete once the
      // first scores are).
      float scale = p.scale_log2;
      // Rows from this thread's first on that its head's token attends: one before the last
      // token sees fewer.
      const int limit = min(tiles * kTileRows, it.len - back - it.r0) - row0 + t0 * kTileRows;
      float m = -INFINITY, l = 0.f;
      // A wait that gives up leaves the loop running (every later wait then returns at
      // once), so that all softmax warps meet at the same barriers.
      for (int t = t0; t < t0 + tiles; ++t) {
        const int sb = t & 1;
        warp_wait(bar(L::SREADY + sb), (t >> 1) & 1, abort_flag);
        if (kFp8 && t == t0)
          scale *= __ldcg(sigma + flat0 + min(head, mine - 1));
        tc_fence_after();
        float x[kCols], y[kCols];
        const uint32_t s_at = lanes + 64 * sb + kCols * hh;
        if constexpr (kCols == 32) {
          tmem_ld32(s_at, reinterpret_cast<uint32_t*>(x));
          tmem_ld32(s_at + 128, reinterpret_cast<uint32_t*>(y));
        } else {
          tmem_ld16(s_at, reinterpret_cast<uint32_t*>(x));
          tmem_ld16(s_at + 128, reinterpret_cast<uint32_t*>(y));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(lbar(L::SFREE + sb));
#pragma unroll
        for (int i = 0; i < kCols; ++i) x[i] += y[i];
        if (__any_sync(0xffffffffu, t * kTileRows + kCols > limit)) {
#pragma unroll
          for (int i = 0; i < kCols; ++i)
            if (t * kTileRows + i >= limit) x[i] = -INFINITY;
        }
        float mx = x[0];
#pragma unroll
        for (int i = 1; i < kCols; ++i) mx = fmaxf(mx, x[i]);
        float* rd = red + sb * 2 * kSlices * kPHeads;
        rd[part_of * kPHeads + head] = mx;
        named_bar_sync(1, L::kSoft);
        mx = rd[head];
#pragma unroll
        for (int i = 1; i < 2 * kSlices; ++i) mx = fmaxf(mx, rd[i * kPHeads + head]);
        mx = mx * scale - L::kBias;
        if (__any_sync(0xffffffffu, mx > m + L::kGrow)) {
          // Move the references of the warp's heads (the four warps of the same heads
          // decide alike); rescale the sum and this warp's share of O.
          const float mn = fmaxf(m, mx);
          const float alpha = m == -INFINITY ? 0.f : ex2(m - mn);
          m = mn;
          l *= alpha;
          if (t > t0) {
            warp_wait(bar(L::PVDONE + ((t - 1) & 1)), ((t - 1) >> 1) & 1, abort_flag);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8 / kSlices; ++c) {   // this warp's slice of O's 256 columns
              const uint32_t at = lanes + L::kOCol + 256 / kSlices * hh + 32 * c;
              float o[32];
              tmem_ld32(at, reinterpret_cast<uint32_t*>(o));
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= alpha;
#pragma unroll
              for (int i = 0; i < 4; ++i) tmem_st8(at + 8 * i, o + 8 * i);
            }
            tmem_wait_st();
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          x[i] = ex2(fmaf(x[i], scale, -ref));
          l += x[i];
        }
        // P's buffer was last read by the output MMAs of tile t - kPBufs.
        if (t >= L::kPBufs)
          warp_wait(bar(L::PVDONE + ((t - L::kPBufs) & 1)), ((t - L::kPBufs) >> 1) & 1, abort_flag);
        uint8_t* pb = smem + L::kOffP + (t % L::kPBufs) * kPBufBytes;
        if (kFp8) {
          // A operand, K-major: row `head` of each part's box, 128 bytes of tile rows.
#pragma unroll
          for (int c = 0; c < kCols / 16; ++c) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t a = 0, b = 0;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float y0 = x[16 * c + 4 * w + 2 * e], y1 = x[16 * c + 4 * w + 2 * e + 1];
                const uint32_t f1 =
                    __nv_cvt_float2_to_fp8x2(make_float2(y0, y1), __NV_SATFINITE, __NV_E4M3);
                const float2 g = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(
                    static_cast<__nv_fp8x2_storage_t>(f1), __NV_E4M3)));
                const uint32_t f2 = __nv_cvt_float2_to_fp8x2(make_float2(y0 - g.x, y1 - g.y),
                                                             __NV_SATFINITE, __NV_E5M2);
                a |= f1 << (16 * e);
                b |= f2 << (16 * e);
              }
              hi[w] = a;
              lo[w] = b;
            }
            const uint32_t at = sw128(head, row0 / 16 + c);
            *reinterpret_cast<uint4*>(pb + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(pb + kPBox + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        } else {
          // Row `head` of the box of this row half, 128 bytes of 64 tile rows.
#pragma unroll
          for (int c = 0; c < kCols / 8; ++c)
            *reinterpret_cast<uint4*>(pb + (qd >> 1) * kPBox + sw128(head, kCols / 8 * hh + c)) =
                make_uint4(pack_bf16(x[8 * c], x[8 * c + 1]), pack_bf16(x[8 * c + 2], x[8 * c + 3]),
                           pack_bf16(x[8 * c + 4], x[8 * c + 5]),
                           pack_bf16(x[8 * c + 6], x[8 * c + 7]));
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(lbar(L::PREADY + sb));
        if (t >= clean) {
          // As each unit of the tile lands in this CTA: rows past the end become zeros, and in
          // the rows that some token does not attend NaN and infinities do.  (The tokens that
          // attend such a row have them from its scores.)
          const int end = it.len - it.r0 - (t - t0) * kTileRows;   // behind the last row
          for (int u = 0; u < 4; ++u) {
            warp_wait(bar(L::CLEANV + u), cleaned & 1, abort_flag);
            const int from = max(0, end - (p.q_len - 1) - 64 * (u >> 1));
            uint8_t* unit = smem + L::kOffV + u * L::kUnit;
            for (int i = tid; i < (64 - from) * 8 * (L::kUnit / kPBox); i += L::kSoft) {
              const int box = i / ((64 - from) * 8), r = i % ((64 - from) * 8);
              uint4* at = reinterpret_cast<uint4*>(unit + box * kPBox + from * 128 + 16 * r);
              *at = from + (r >> 3) < end - 64 * (u >> 1) ? finite_only<kFp8>(*at)
                                                          : make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive_cluster(lbar(L::CLEANED + u));
          }
          ++cleaned;
        }
      }
      t0 += tiles;
      if (tid == 0 && t0 == T) pdl_launch_dependents();   // the combine waits for this grid anyway
      // The row sums of a head's four threads, its log-sum-exp, and O / sum through
      // shared memory (over operands that nothing reads any more) to whole rows.
      float* sums = reinterpret_cast<float*>(smem + L::kOffSum);
      sums[part_of * kPHeads + head] = l;
      warp_wait(bar(L::PVDONE + ((t0 - 1) & 1)), ((t0 - 1) >> 1) & 1, abort_flag);
      tc_fence_after();
      // Whether the CTA has given up is asked for all: some warp may raise the flag at any time,
      // and the softmax warps meet at a barrier below.
      if (!any_of(*abort_flag, 1, L::kSoft)) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * kSlices; ++i) sum += sums[i * kPHeads + head];
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        const bool whole = kShare ? whole_set(it) : p.direct != 0;   // the result itself
        const size_t stride = whole ? 1 : p.splits;
        const size_t row = static_cast<size_t>(flat0) * stride + (whole ? 0 : it.j);   // the first's
        float* o_to = kShare && whole ? static_cast<float*>(p.out) : p.part_o;
        float* lse_to = kShare && whole ? p.out_lse : p.part_lse;
        const bool bf16_out = whole && p.io_bf16;
        // Four values of row h, column x.
        auto put = [&](int h, int x, float4 o) {
          const size_t at = (row + static_cast<size_t>(h) * stride) * kDc + x;
          if (bf16_out)
            *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(o_to) + at) =
                make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
          else
            *reinterpret_cast<float4*>(o_to + at) = o;
        };
        if (part_of == 0 && head < mine && lse_to)
          lse_to[row + static_cast<size_t>(head) * stride] =
              sum > 0.f ? (m + log2f(sum)) * kLn2 : -INFINITY;
        if (kShare && t0 < T) {
          // The next item's operands are on their way to where the last one stages: each
          // warp turns its 32 heads' columns over in its part of P, 16 at a time, and
          // writes 64 bytes of eight rows at once.  (P of the next tile is written behind
          // the barrier of its maxima.)
          const int col0 = 256 / kSlices * hh;
          const int at = 256 * (col0 >> 7) + 128 * (qd >> 1) + (col0 & 127);   // latent
          float4* mine4 = reinterpret_cast<float4*>(smem + L::kOffP) + 128 * warp;
          const int h0 = 32 * (qd & 1);
#pragma unroll 1
          for (int c = 0; c < 16 / kSlices; ++c) {
            float o[16];
            tmem_ld16(lanes + L::kOCol + col0 + 16 * c, reinterpret_cast<uint32_t*>(o));
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mine4[4 * lane + (i ^ (lane >> 1 & 3))] = make_float4(
                  o[4 * i] * inv, o[4 * i + 1] * inv, o[4 * i + 2] * inv, o[4 * i + 3] * inv);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 8 * i + (lane >> 2), q = lane & 3;
              if (h0 + r < mine)
                put(h0 + r, at + 16 * c + 4 * q, mine4[4 * r + (q ^ (r >> 1 & 3))]);
            }
            __syncwarp();
          }
        } else {
          uint8_t* stage = smem;
          // This warp's slice of O's columns: in tile jj = col0 / 128 the lane's 128 columns
          // are latents 256 jj + 128 (qd >> 1) ..
          const int col0 = 256 / kSlices * hh;
          float* to = reinterpret_cast<float*>(stage + head * L::kStageRow) + 256 * (col0 >> 7) +
                      128 * (qd >> 1) + (col0 & 127);
#pragma unroll 1
          for (int c = 0; c < 8 / kSlices; ++c) {
            float o[32];
            tmem_ld32(lanes + L::kOCol + col0 + 32 * c, reinterpret_cast<uint32_t*>(o));
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(to + 32 * c + 4 * i) =
                  make_float4(o[4 * i] * inv, o[4 * i + 1] * inv, o[4 * i + 2] * inv,
                              o[4 * i + 3] * inv);
          }
          named_bar_sync(1, L::kSoft);
          for (int h = warp; h < mine; h += L::kSoftWarps) {
            const float4* src = reinterpret_cast<const float4*>(stage + h * L::kStageRow);
#pragma unroll
            for (int i = 0; i < 4; ++i) put(h, 128 * i + 4 * lane, src[32 * i + lane]);
          }
        }
      }
      if (kShare && t0 < T) it = item_after(it, t0);
    }
  }
  // A CTA that gave up may have copies in flight: they land long before this.
  if (*abort_flag) {
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 5000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // neither CTA leaves while the other's MMAs or barriers use it
  if (warp == kWarpScore) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kPTmem)
                 : "memory");
  }
  if (tid == 0 && *abort_flag) report(p.status, MLA_DEV_PIPELINE_TIMEOUT);
}

template <bool kFp8, bool kShare>
mla_status launch_pair(const CUtensorMap& cache, const CUtensorMap& q, const CUtensorMap& qpe,
                       const SplitParams& p, const float* sigma, cudaStream_t s, const char* who) {
  using L = PairPlan<kFp8>;
  static DeviceFlags attr_done;
  const int dev = current_device();
  if (!attr_done.test(dev)) {
    if (cudaFuncSetAttribute(split_pair_kernel<kFp8, kShare>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, int(L::kSmem)) != cudaSuccess) {
      cudaGetLastError();
      set_error("%s: cannot reserve %zu bytes of shared memory", who, L::kSmem);
      return MLA_ERR_CUDA;
    }
    attr_done.set(dev);
  }
  cudaLaunchConfig_t cfg = {};
  const int ctas = 2 * pair_groups(p.q_len * p.H);   // of a row
  cfg.gridDim = kShare ? dim3(share_runs(ctas) * ctas) : dim3(ctas, p.splits, p.B / p.q_len);
  cfg.blockDim = dim3(kShare ? L::kShareThreads : L::kThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = launch_overlap_enabled() ? 2 : 1;
  cudaLaunchKernelEx(&cfg, split_pair_kernel<kFp8, kShare>, cache, q, qpe, p, sigma);
  return launch_status(who);
}

}  // namespace

mla_status launch_pair_queries(const SplitParams& p, cudaStream_t stream, const char* who) {
  launch_pdl(pair_query_kernel, dim3(static_cast<unsigned>((size_t(p.B) * p.H + 3) / 4)),
             dim3(128), 0, stream, p, pair_codes(p), pair_units(p));
  return launch_status(who);
}

mla_status launch_split_pair(const SplitParams& p, const void* cache, bool fp8,
                             cudaStream_t stream, const char* who) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) {
    set_error("%s: cuTensorMapEncodeTiled is not available from the driver", who);
    return MLA_ERR_CUDA;
  }
  // 128-byte boxes (128-byte swizzle) of up to 64 rows inside a page; the queries in
  // boxes of one CTA's 64 heads.
  CUresult bad = CUDA_SUCCESS;
  auto encode = [&](CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, int elt,
                    int box_rows, CUtensorMapL2promotion promote) {
    const cuuint64_t gdim[2] = {cols, rows}, gstride[1] = {cols * elt};
    const cuuint32_t box[2] = {cuuint32_t(128 / elt), cuuint32_t(box_rows)}, estride[2] = {1, 1};
    const CUresult r = enc(m, elt == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                           2, const_cast<void*>(base), gdim, gstride, box, estride,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promote,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) bad = r;
  };
  const uint64_t rows = static_cast<uint64_t>(p.B) * p.H;
  const int page = 1 << p.page_shift;
  const float* sigma = pair_units(p);
  CUtensorMap tm, tq, tp;
  encode(&tm, cache, kRow, view_rows(p), fp8 ? 1 : 2, page < 64 ? page : 64,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  if (fp8) {
    encode(&tq, pair_codes(p), kQ8Row, 2 * rows, 1, kPHeads, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
    tp = tq;
  } else {
    encode(&tq, p.q_abs, kDc, rows, 2, kPHeads, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
    encode(&tp, p.q_pe, kDr, rows, 2, kPHeads, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
  }
  if (bad != CUDA_SUCCESS) {
    set_error("%s: cuTensorMapEncodeTiled failed (%d)", who, int(bad));
    return MLA_ERR_CUDA;
  }
  if (!fp8)
    return p.pieces ? launch_pair<false, true>(tm, tq, tp, p, nullptr, stream, who)
                    : launch_pair<false, false>(tm, tq, tp, p, nullptr, stream, who);
  if (!p.late) {
    const mla_status st = launch_pair_queries(p, stream, who);
    if (st != MLA_OK) return st;
  }
  return p.pieces ? launch_pair<true, true>(tm, tq, tp, p, sigma, stream, who)
                  : launch_pair<true, false>(tm, tq, tp, p, sigma, stream, who);
}

}  // namespace mla
