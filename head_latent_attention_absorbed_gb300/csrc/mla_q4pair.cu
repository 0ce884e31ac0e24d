// The split over a 4-bit pool for bf16 queries of many heads: a pair of SMs takes up to 128
// query rows (heads, and the tokens of a multi-token step) of one sequence.
//
// The products, their split over the pair and the softmax are those of mla_pair.cu with an
// E4M3 cache: heads are the M of the MMAs, CTA i of the pair holds 64 of them, and of every
// other operand half:
//   scores  S0[128 heads x 128 rows] = Q[128 x 512] . C^T, S1 = Qk[128 x 64] . K^T
//                                                       CTA i: rows 64 i ..
//   output  O[128 x 512] += P[128 x 128 rows] . C[128 x 512]
//                                                       CTA i: 256 of the latent columns
// Queries are two E4M3 parts in units of a power of two per head (their keys' part bf16, and
// so S1 has no unit), P an E4M3 part and its E5M2 remainder, whose unit follows the scores up and
// down (mla_q4.cuh).
//
// What differs is where the operands come from.  A tile's codes and exponents pass through both
// CTAs as they are stored, 32 rows at a time, and become E4M3 boxes of 64 rows x 128 columns.  A
// tile has four boxes in a CTA.  First they hold the CTA's own 64 rows, for the scores.  The
// output product wants, at the same place in both CTAs, box 2 jj + h with the rows of half h and
// the columns of box 2 jj + i in CTA i: where h is the CTA's own half that is what the box holds
// already, and the other two boxes are decoded again from the other CTA's rows, once the scores
// are done.  So each value is decoded where it is used, one and a half times in all, and three
// tiles' boxes fit.  Eight warps decode the scores' boxes, a tile or two ahead; the second halves
// are the softmax warps', behind their P, which would otherwise wait for the next scores.
// (32 x 16384 rows x 128 heads, earlier forms: 193 us with score boxes and output units apart, a
// tile of each, and a warp for each; 172 with all warps on the one and then the other; 169 with
// two tiles of units, decoded once and stored twice, where the one tile of score boxes made
// decoding and the tensor cores take turns; 137 with all of it on the eight warps.)
// Of the keys, stored as the tensor core wants them, each CTA copies its 64 rows.  Nothing needs
// cleaning behind a sequence's end: whatever bits a row holds, its latents are finite, and its
// scores are not looked at.
//
// Tensor memory per CTA as in mla_pair.cu: S0 and S1, two buffers of 64 columns each, and O.
//
// Warps (1024 threads): 0-15 softmax, second halves of the boxes, epilogue; 16, 22 and 23 copies
// of rows (one warp took 4200 cycles for a tile's four copies and what leads to them); 17 keys and
// queries; 18 score MMAs and 19 those of the keys, 20 and 21 output MMAs (the even CTA's issue for
// the pair); 24-31 the scores' boxes.
//
// What bounds it: a tile's way through one of the three sets of boxes (codes to E4M3 1.0 us, score
// MMAs 0.9 and their queue, softmax and second halves 1.8, output MMAs 0.9), a third of which is a
// tile's 2.0 us; and shared memory, of whose 3800 cycles in that time the tensor cores' reads take
// 1900 (both parts of Q and of P against every row), codes, boxes and copies some 1300.  The
// operations alone would take 1.4 us.
// 32 x 16384 rows x 128 heads 123 us (1.70 TB/s of cache; E4M3 cache 103, bf16 131), 64 sequences
// of 512 to 8192 rows 96.  A change of item takes 5 to 6 us, of which 4.8 are its result's way
// through P; stored straight from registers, or 128 bytes of a row at a time, it takes no less.
#include <cuda_fp8.h>
#include <cudaTypedefs.h>

#include "mla_pair.cuh"
#include "mla_q4.cuh"

namespace mla {
namespace {

struct Q4Pair {
  static constexpr int kSoftWarps = 16, kSoft = 32 * kSoftWarps, kThreads = 1024;
  static constexpr int kSlices = kSoftWarps / 4, kCols = 64 / kSlices;
  static constexpr int kParts = 2;
  static constexpr int kQKeys = kParts * 4 * kPBox;     // offset of the query's key part
  static constexpr int kQBytes = kQKeys + kPBox;
  // Rows arrive in slots of 32: two for the CTA's own half of a tile, two for the other half.
  static constexpr int kSlotRows = 32, kSlots = 4;
  static constexpr int kSlotBytes = kSlotRows * kQ4LatBytes;
  static constexpr int kKeyBytes = 64 * kQ4KeyBytes;
  static constexpr int kOffQ = 0;
  static constexpr int kTiles = 3;
  static constexpr int kOffC = kOffQ + kQBytes;         // [3][4] boxes
  static constexpr int kOffK = kOffC + kTiles * 4 * kPBox;   // keys
  static constexpr int kOffP = kOffK + kKeyBytes;
  static constexpr int kOffRaw = kOffP + kPBufBytes;
  static constexpr int kOffTable = kOffRaw + kSlots * kSlotBytes;
  static constexpr int kOffBar = kOffTable + 128;
  // Rows landed / decoded and keys landed (this CTA's); a tile's boxes decoded for the scores,
  // and free; keys handed over; S, P (with the boxes' second halves), O and the query as in
  // mla_pair.cu.
  static constexpr int RAWFULL = 0, RAWEMPTY = RAWFULL + kSlots, KEYFULL = RAWEMPTY + kSlots,
                       FULLS = KEYFULL + 1, FREE = FULLS + kTiles,
                       KREADY = FREE + kTiles, SREADY = KREADY + 1,
                       SFREE = SREADY + 2, PREADY = SFREE + 2, PVDONE = PREADY + 2,
                       QFULL = PVDONE + 2, QFREE = QFULL + 1, kBars = QFREE + 1;
  static constexpr int kOffSlot = kOffBar + 8 * kBars;
  static constexpr int kOffAbort = kOffSlot + 8;
  static constexpr int kOffShare = kOffAbort + 8;       // (flag and limit) TileShare of the pair
  static constexpr int kOffDrop = kOffShare + 24;       // [64 heads], see the softmax
  static constexpr size_t kSmem = kOffDrop + 64 * 4;
  static constexpr uint32_t kOCol = 256;
  // Where the softmax's reference goes below a tile's largest score when it moves, and how far
  // above the reference that score may then lie in later tiles (log2): weights stay in [0, 2^8.5].
  static constexpr float kBias = 4.f, kTop = 8.5f;
  static constexpr int kStageRow = kDc * 4 + 16;        // epilogue staging, over the operands
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kOffRaw >= kPHeads * kStageRow, "epilogue staging");
  // What the softmax warps exchange (maxima, sums, an item's output) goes through P when nothing
  // reads it; the eight warps of the same heads keep to those heads' rows of it: 32 rows of each
  // part, part 0 first.
  static_assert(kPBufBytes == kSoftWarps * 32 * 32, "an item's output through P");
  static_assert(2 * 2 * kSlices * 32 * 4 <= 4096, "the maxima and sums of 32 heads through P");
  static_assert(kOffC % 1024 == 0 && kOffK % 1024 == 0 && kOffP % 1024 == 0, "swizzle atoms");
  static_assert(kOffRaw % 16 == 0 && kOffBar % 8 == 0, "alignment");
};

// 8 columns of this thread's lane, loaded (one statement, as tmem_ld16).
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

// kSteps K steps of a pair's product, `sa` and `sb` (16-byte units) apart, by one elected thread
// of the converged warp; the first replaces what D holds unless `accumulate`.  (With an election
// and a predicate for every step the warp that issues the scores' 32 was what a tile waited for:
// 169 us for 32 x 16384 rows x 128 heads.)
template <bool kE4m3, int kSteps, int kSa, int kSb>
__device__ __forceinline__ void mma_pair_steps(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                               uint32_t accumulate) {
  static_assert(kSteps == 2 || kSteps == 4, "steps");
#define MLA_Q4_FIRST(KIND)                                                                    \
  "{\n\t.reg .pred p, e, t;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\t"                   \
  "setp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"                                   \
  "@e tcgen05.mma.cta_group::2.kind::" KIND " [%0], %1, %2, %3, p;\n\t"                       \
  "add.s64 a, %1, %5;\n\tadd.s64 b, %2, %6;\n\t"                                              \
  "@e tcgen05.mma.cta_group::2.kind::" KIND " [%0], a, b, %3, t;\n\t"
#define MLA_Q4_MORE(KIND)                                                                     \
  "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"                                                \
  "@e tcgen05.mma.cta_group::2.kind::" KIND " [%0], a, b, %3, t;\n\t"
#define MLA_Q4_ARGS                                                                           \
  ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(kSa), "n"(kSb) : "memory"
  if constexpr (kE4m3 && kSteps == 4)
    asm volatile(MLA_Q4_FIRST("f8f6f4") MLA_Q4_MORE("f8f6f4") MLA_Q4_MORE("f8f6f4") "}" MLA_Q4_ARGS);
  else if constexpr (kE4m3)
    asm volatile(MLA_Q4_FIRST("f8f6f4") "}" MLA_Q4_ARGS);
  else
    asm volatile(MLA_Q4_FIRST("f16") MLA_Q4_MORE("f16") MLA_Q4_MORE("f16") "}" MLA_Q4_ARGS);
#undef MLA_Q4_FIRST
#undef MLA_Q4_MORE
#undef MLA_Q4_ARGS
}

template <int kN>
struct Int {
  static constexpr int value = kN;
};

// Where the rows of a page that does not exist come from.
__device__ __align__(128) uint8_t g_q4_pair_zeros[Q4Pair::kSlotBytes];
static_assert(Q4Pair::kKeyBytes <= Q4Pair::kSlotBytes, "zeros for either plane");

// kShare: one pair per two SMs takes an equal run of all sequences' tiles (take_share), an
// item per sequence it meets; otherwise a pair has one item, its chunk.
template <bool kShare>
__global__ void __launch_bounds__(Q4Pair::kThreads, 1)
    split_q4_pair_kernel(const __grid_constant__ CUtensorMap tmap_q,
                         const __grid_constant__ CUtensorMap tmap_qpe, const SplitParams p,
                         const float* __restrict__ sigma) {
  using L = Q4Pair;
  extern __shared__ __align__(1024) uint8_t q4_pair_smem[];
  uint8_t* smem = q4_pair_smem;
  const uint32_t sbase = smem_u32(smem), bars = sbase + L::kOffBar;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffAbort);
  uint32_t* slot_ptr = reinterpret_cast<uint32_t*>(smem + L::kOffSlot);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // uniform to the compiler
  // Query rows (tokens x heads) of the sequence, dealt evenly to its CTAs: this CTA's are
  // flat0 .. flat0 + mine - 1 of all; rows past them up to 64 are computed as well and dropped.
  const int all = p.q_len * p.H, parts = kShare ? 2 * pair_groups(all) : gridDim.x;
  const int dealt = (all + parts - 1) / parts, part = kShare ? blockIdx.x % parts : blockIdx.x;
  const int first = part * dealt, mine = min(dealt, all - first);
  const int rank = uniform(static_cast<int>(cluster_ctarank()));
  const bool leader = rank == 0;
  if (p.late) pdl_wait();
  // Rows of a sequence, all of which its last token attends, count.
  TileItem item0{0, 0, 0, 0, 0};   // the pair's first item (none: T = 0)
  int T = 0;        // tiles of the pair
  TileShare share{};
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
  auto item_after = [&](const TileItem& it, int t) { return next_item<true>(p, it, T - t); };
  const uint32_t lead = mapa_shared(bars, 0);   // the even CTA's barriers
  auto bar = [&](int i) { return bars + 8 * i; };
  auto lbar = [&](int i) { return lead + 8 * i; };
  constexpr int kWarpRows = L::kSoftWarps, kWarpKeys = kWarpRows + 1, kWarpScore = kWarpRows + 2,
                kWarpOut = kWarpRows + 4, kWarpRows2 = kWarpRows + 6, kWarpDecode = kWarpRows + 8;

  if (tid == L::kSoft) {
    for (int i = 0; i < L::kSlots; ++i) {
      mbar_init(bar(L::RAWFULL + i), 1);
      mbar_init(bar(L::RAWEMPTY + i), 8);
    }
    for (int i = 0; i < L::kTiles; ++i) {
      mbar_init(bar(L::FULLS + i), 16);   // the decoding warps of both CTAs
      mbar_init(bar(L::FREE + i), 2);     // one commit per output issuer
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(L::SREADY + i), 2);                 // one commit per issuer
      mbar_init(bar(L::SFREE + i), 2 * L::kSoftWarps);  // both CTAs' softmax warps
      mbar_init(bar(L::PREADY + i), 2 * L::kSoftWarps);
      mbar_init(bar(L::PVDONE + i), 2);
    }
    mbar_init(bar(L::KEYFULL), 1);
    mbar_init(bar(L::KREADY), 2);   // both CTAs' keys
    mbar_init(bar(L::QFULL), 1);
    mbar_init(bar(L::QFREE), 2);   // one commit per score issuer
    q4_wait_init(p, abort_flag);
    fence_mbarrier_init();
    prefetch_tmap(&tmap_q);
    prefetch_tmap(&tmap_qpe);
  }
  if (warp == kWarpDecode && lane < 16) q4_table(smem + L::kOffTable, lane);
  if (kShare && warp == kWarpRows) {
    __syncwarp();
    share = take_share<true>(p, blockIdx.x / parts, gridDim.x / parts, lane, blockIdx.x == 0);
    if (lane == 0) *reinterpret_cast<TileShare*>(smem + L::kOffShare) = share;
  }
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
  const uint32_t tmem = uniform(static_cast<int>(*slot_ptr));
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
    for (int i = 0; i < L::kParts * 4; ++i)
      tma_load_pair(sbase + L::kOffQ + i * kPBox, &tmap_q, 128 * (i & 3),
                    (i >> 2) * p.B * p.H + flat0, lbar(L::QFULL), stream);
    tma_load_pair(sbase + L::kOffQ + L::kQKeys, &tmap_qpe, 0, flat0, lbar(L::QFULL), stream);
  };
  // Runs the pair's tiles, item by item: f(item, tile i of it, tile t of all) -> false: given up.
  auto for_tiles = [&](auto&& f) {
    TileItem it = item0;
    for (int t = 0, i = 0; t < T; ++t) {
      if (!f(it, i, t)) return;
      if (++i == it.tiles && t + 1 < T) {
        it = item_after(it, t + 1);
        i = 0;
      }
    }
  };
  auto given_up = [&] { return __any_sync(0xffffffffu, *abort_flag) != 0; };

  if (warp == kWarpRows || warp == kWarpKeys || warp == kWarpRows2 || warp == kWarpRows2 + 1) {
    // ------------------------------------------------------------ rows, keys
    // Pieces of one page each: of a slot's 32 rows, or of the CTA's 64 keys.
    const bool rows = warp != kWarpKeys;
    const uint8_t* pool = static_cast<const uint8_t*>(p.cache);
    const uint64_t pol = l2_evict_first_policy();
    const int piece = min(1 << p.page_shift, rows ? L::kSlotRows : 64);
    const int span = rows ? kTileRows : 64, row0 = rows ? 0 : 64 * rank;
    // Lane i: the page of piece i of a tile, or -1 (outside the pool), -2 (past the end).
    auto piece_page = [&](const TileItem& it, int i) {
      const int r = it.r0 + i * kTileRows + row0 + lane * piece;
      if (lane * piece >= span || r >= it.len) return -2;
      const int id = p.table[static_cast<size_t>(it.v) * p.table_stride + (r >> p.page_shift)];
      return id < 0 ? -1 : id;
    };
    // Copies pieces from .. to - 1, of which those below `live` lie in the sequence.
    auto copy_pieces = [&](const uint8_t* src, int from, int to, int live, uint32_t bytes,
                           uint32_t dst, uint32_t full) {
      const int n = max(min(to, live) - from, 0);
      expect_tx_elected(full, n * bytes);
#pragma unroll 1
      for (int i = 0; i < n; ++i)
        bulk_g2s_elected(dst + i * bytes,
                         reinterpret_cast<const uint8_t*>(__shfl_sync(
                             0xffffffffu, reinterpret_cast<unsigned long long>(src), from + i)),
                         bytes, full, pol);
    };
    if (warp == kWarpKeys) {
      pdl_wait();   // the query comes from the kernel before
      if (T > 0) load_query(item0.v);
    }
    const int bytes = rows ? kQ4LatBytes : kQ4KeyBytes, plane = rows ? 0 : kQ4LatBytes;
    // Where lane i's piece of tile i of `it` comes from, its page looked up before.
    const int mask = (1 << p.page_shift) - 1;
    auto piece_source = [&](int id, int r0) {
      if (id >= p.num_pages) id = -1;
      const int r = (r0 + row0 + lane * piece) & mask;
      return id < 0 ? g_q4_pair_zeros
                    : pool + (static_cast<size_t>(id) << p.page_shift) * kQ4RowBytes +
                          (static_cast<size_t>(plane) << p.page_shift) + r * bytes;
    };
    auto live_of = [&](int id) { return __popc(__ballot_sync(0xffffffffu, id != -2)); };
    // The next tile's pages and first row, looked up early.
    int ahead = T > 0 ? piece_page(item0, 0) : -2, ahead_r0 = item0.r0;
    auto look_ahead = [&](const TileItem& it, int i, int t) {
      if (ahead == -1 || ahead >= p.num_pages) report(p.status, MLA_DEV_PAGE_OUT_OF_RANGE);
      ahead = -2;
      if (t + 1 >= T) return;
      const bool more = i + 1 < it.tiles;
      const TileItem then = more ? it : item_after(it, t + 1);
      ahead = piece_page(then, more ? i + 1 : 0);
      ahead_r0 = then.r0 + (more ? i + 1 : 0) * kTileRows;
    };
    if (rows) {
      // Two warps for the slots of the CTA's own half, one for both of the other half.  (L2 asked
      // for a tile's rows one tile before: 126 us against 125 for 32 x 16384 rows x 128 heads.)
      const bool own = warp != kWarpRows2 + 1;
      const int k0 = own && warp != kWarpRows ? 1 : 0, k1 = own ? k0 + 1 : 2;
      const int per = L::kSlotRows / piece, half = own ? rank : 1 - rank;
      for_tiles([&](const TileItem& it, int i, int t) {
        if (given_up()) return false;
        if (p.stop_after_tiles > 0 && t >= p.stop_after_tiles) return false;   // test hook
        const uint8_t* src = piece_source(ahead, ahead_r0);
        const int live = live_of(ahead);
        look_ahead(it, i, t);
#pragma unroll 1
        for (int k = k0; k < k1; ++k) {
          const int slot = (own ? 0 : 2) + k, from = (2 * half + k) * per;
          if (t > 0) {
            q4_warp_wait(bar(L::RAWEMPTY + slot), (t - 1) & 1, abort_flag);
            if (given_up()) return false;
          }
          copy_pieces(src, from, from + per, live, piece * bytes,
                      sbase + L::kOffRaw + slot * L::kSlotBytes, bar(L::RAWFULL + slot));
        }
        return true;
      });
    } else {
      int queries = 0;   // later items' queries fetched
      for_tiles([&](const TileItem& it, int i, int t) {
        if (given_up()) return false;
        const uint8_t* src = piece_source(ahead, ahead_r0);
        const int live = live_of(ahead);
        look_ahead(it, i, t);
        if (t > 0) {   // the scores of the tile before have read them
          q4_warp_wait(bar(L::SREADY + ((t - 1) & 1)), ((t - 1) >> 1) & 1, abort_flag);
          if (given_up()) return false;
        }
        copy_pieces(src, 0, 64 / piece, live, piece * bytes, sbase + L::kOffK, bar(L::KEYFULL));
        if (kShare && i == 0 && t > 0) {
          // A later item's query, once the scores of the item before are done, which read the one
          // that it replaces.
          q4_warp_wait(bar(L::QFREE), queries & 1, abort_flag);
          if (given_up()) return false;
          ++queries;
          load_query(it.v);
        }
        // Handed over once they have landed: the even CTA's MMAs read both CTAs'.
        q4_warp_wait(bar(L::KEYFULL), t & 1, abort_flag);
        if (lane == 0) arrive_cluster(lbar(L::KREADY));
        return true;
      });
    }
  } else if (warp >= kWarpDecode) {
    // ------------------------------------------------------------ codes to E4M3
    // Warp d takes 32 columns, piece c = d & 3, of the CTA's own rows in boxes 2 j and 2 j + 1,
    // j = d >> 2.  A row per lane: rows are 17 times 16 bytes apart, so eight lanes read from
    // eight different pieces of the banks, and the swizzle has them write so.  All is decoded into
    // registers before the wait for the boxes: a tile's way through them, from here to the end of
    // its output product, is what bounds the kernel.
    const int d = warp - kWarpDecode, c = d & 3, j = d >> 2;
    const uint8_t* table = smem + L::kOffTable;
    const uint8_t* from = smem + L::kOffRaw + lane * kQ4LatBytes;
    uint8_t* boxes = smem + L::kOffC + 2 * j * kPBox + lane * 128;
    const uint32_t at = (2 * c << 4) ^ ((lane & 7) << 4);
    for (int t = 0; t < T; ++t) {
      const int buf = t % L::kTiles;
      if (given_up()) break;
      Q4Piece piece[2][2];
      bool plain = true;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        q4_warp_wait(bar(L::RAWFULL + k), t & 1, abort_flag);
        const uint8_t* raw = from + k * L::kSlotBytes;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int m = 2 * j + i;
          piece[k][i].load(raw + 64 * m + 16 * c, raw[kQ4CodeBytes + 4 * m + c]);
          plain = plain && q4_plain(piece[k][i].e);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::RAWEMPTY + k));
      }
      uint4 e4m3[2][2][2];
      auto decode = [&](auto is_plain) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            piece[k][i].template decode<decltype(is_plain)::value != 0>(e4m3[k][i][0],
                                                                        e4m3[k][i][1], table);
      };
      if (__all_sync(0xffffffffu, plain))
        decode(Int<1>{});
      else
        decode(Int<0>{});
      if (t >= L::kTiles) {
        q4_warp_wait(bar(L::FREE + buf), (t / L::kTiles - 1) & 1, abort_flag);
        tc_fence_after();
      }
      uint8_t* to = boxes + buf * 4 * kPBox;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint8_t* row = to + i * kPBox + k * (L::kSlotRows * 128);
          *reinterpret_cast<uint4*>(row + at) = e4m3[k][i][0];
          *reinterpret_cast<uint4*>(row + (at ^ 16)) = e4m3[k][i][1];
        }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_cluster(lbar(L::FULLS + buf));
    }
  } else if (warp == kWarpScore || warp == kWarpScore + 1) {
    // ------------------------------------------------------------ score MMAs (even CTA)
    // The whole warp runs along, converged at every MMA and commit.  Not unrolled over boxes:
    // code that runs once a tile is fetched anew each time.
    if (leader) {
      const bool keys = warp != kWarpScore;
      constexpr uint32_t idesc = (1u << 4) | (128u >> 3 << 17) | (128u >> 4 << 24);   // E4M3
      constexpr uint32_t idesc_k = idesc | (1u << 7) | (1u << 10);                    // bf16
      const uint64_t q0 = umma_desc_sw128(sbase + L::kOffQ, 16, 1024);
      const uint64_t c0 = umma_desc_sw128(sbase + L::kOffC, 16, 1024);
      const uint64_t qk0 = umma_desc_sw128(sbase + L::kOffQ + L::kQKeys, 16, 1024);
      const uint64_t k0 = umma_desc_sw128(sbase + L::kOffK, 16, 1024);
      int n = 0;   // items begun
      for_tiles([&](const TileItem& it, int i, int t) {
        const int sb = t & 1;
        if (i == 0) {
          q4_warp_wait(bar(L::QFULL), n & 1, abort_flag);
          ++n;
          if (kShare && !keys && blockIdx.x % parts == 0 && it.r0 == 0)
            // The run with a sequence's first tile says how many runs it spans.  (Not before a
            // query is here, fetched behind the PDL wait: the combine of the call before may
            // still be reading its own counts.)
            for (int q = lane; q < p.q_len; q += 32)
              p.pieces[it.v * p.q_len + q] = count_pieces(it, share.first + t, share.each);
        }
        if (t >= 2) q4_warp_wait(bar(L::SFREE + sb), ((t - 2) >> 1) & 1, abort_flag);
        if (given_up()) return false;
        if (keys) {
          q4_warp_wait(bar(L::KREADY), t & 1, abort_flag);
          if (given_up()) return false;
          tc_fence_after();
          mma_pair_steps<false, 4, 2, 2>(tmem + 128 + 64 * sb, qk0, k0, idesc_k, 0);
        } else {
          const int buf = t % L::kTiles;
          q4_warp_wait(bar(L::FULLS + buf), (t / L::kTiles) & 1, abort_flag);
          if (given_up()) return false;
          tc_fence_after();
#pragma unroll 1
          for (int m = 0; m < 4; ++m) {
            const uint64_t b = c0 + static_cast<uint64_t>((4 * buf + m) * (kPBox >> 4));
#pragma unroll
            for (int part = 0; part < L::kParts; ++part) {
              const uint64_t a = q0 + static_cast<uint64_t>((part * 4 + m) * (kPBox >> 4));
              // 32 bytes of K a step
              mma_pair_steps<true, 4, 2, 2>(tmem + 64 * sb, a, b, idesc,
                                            part > 0 ? 1u : (m > 0 ? 1u : 0u));
            }
          }
        }
        commit_pair(bar(L::SREADY + sb));
        if (kShare && i + 1 == it.tiles && t + 1 < T) commit_pair(bar(L::QFREE));
        return true;
      });
    }
  } else if (warp == kWarpOut || warp == kWarpOut + 1) {
    // ------------------------------------------------------------ output MMAs (even CTA)
    // Issuer jj takes the units of O tile jj.
    if (leader) {
      const int jj = warp - kWarpOut;
      constexpr uint32_t idesc =
          (1u << 4) | (1u << 16) | (256u >> 3 << 17) | (128u >> 4 << 24);
      const uint64_t p0 = umma_desc_sw128(sbase + L::kOffP, 16, 1024);
      const uint64_t v0 = umma_desc_sw128(sbase + L::kOffC, kPBox, 1024);   // rows (K) by eights
      const uint32_t d = tmem + L::kOCol + 128 * jj;
      for_tiles([&](const TileItem&, int i, int t) {
        const int pb = t & 1;
        const int buf = t % L::kTiles;
        q4_warp_wait(bar(L::PREADY + pb), (t >> 1) & 1, abort_flag);
        if (given_up()) return false;
        tc_fence_after();
#pragma unroll 1
        for (int kh = 0; kh < 2; ++kh) {
          const uint64_t b = v0 + static_cast<uint64_t>((4 * buf + 2 * jj + kh) * (kPBox >> 4));
          // 64 rows: two steps of 32 (4 KB; 32 bytes of each part's row, the half at byte 64 kh)
#pragma unroll
          for (int part = 0; part < L::kParts; ++part) {
            const uint64_t a = p0 + ((part * kPBox + 64 * kh) >> 4);
            mma_pair_steps<true, 2, 2, (4096 >> 4)>(
                d, a, b, idesc | (part == 1 ? 1u << 7 : 0u),   // the remainder is E5M2
                part > 0 ? 1u : (i > 0 || kh > 0 ? 1u : 0u));
          }
        }
        commit_pair(bar(L::PVDONE + pb));
        commit_pair(bar(L::FREE + buf));
        return true;
      });
    }
  } else if (warp < L::kSoftWarps) {
    // ------------------------------------------------------------ softmax
    // Warp w: lanes 32 (w & 3) .. of tensor memory, so head 32 (w & 1) + lane of the
    // tile's row half (w >> 1) & 1, and the column slice w >> 2 of those 64 rows.
    constexpr int kCols = L::kCols, kSlices = L::kSlices;
    const int qd = warp & 3, hh = warp >> 2;
    const int head = 32 * (qd & 1) + lane, row0 = 64 * (qd >> 1) + kCols * hh;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * qd) << 16);
    const int part_of = kSlices * (qd >> 1) + hh;   // which part of the tile's rows
    // The rows of P of the warp's heads: 32 of each part.
    uint8_t* mine_p = smem + L::kOffP + 4096 * (qd & 1);
    float* red = reinterpret_cast<float*>(mine_p);   // [2 kSlices][32 heads], two of them
    // A tile's boxes again: 32 of the other CTA's rows (slot), 32 columns (piece c) of box 2 j +
    // rank, into box 2 j + 1 - rank; a row per lane, as the decoding warps.
    const int slot = 2 + (warp >> 3), c = warp & 3, j = (warp >> 2) & 1;
    const uint8_t* raw = smem + L::kOffRaw + slot * L::kSlotBytes + lane * kQ4LatBytes;
    uint8_t* box = smem + L::kOffC + (2 * j + 1 - rank) * kPBox +
                   (warp >> 3) * (L::kSlotRows * 128) + lane * 128;
    const uint32_t box_at = (2 * c << 4) ^ ((lane & 7) << 4);
    // How far the head's reference lies below the highest it was: written by the first of the eight
    // warps, behind the barriers between which all read it.
    float* drop_at = reinterpret_cast<float*>(smem + L::kOffDrop) + head;
    const int back = p.q_len - 1 - (first + min(head, mine - 1)) / p.H;   // tokens behind its own
    const float scale = p.scale_log2;
    TileItem it = item0;
    for (int t0 = 0; t0 < T;) {   // items; t0: the item's first tile among the pair's
      const int flat0 = it.v * all + first, tiles = it.tiles;
      float unit = 0.f;   // the head's, of the query's codes
      // Rows from this thread's first on that its head's token attends: one before the last
      // token sees fewer.
      const int limit = min(tiles * kTileRows, it.len - back - it.r0) - row0 + t0 * kTileRows;
      float m = 0.f, l = 0.f;
      bool fresh = true;   // no score but -infinity so far: m is set by the first other
      int due = t0 + kBearsTiles;   // the next look at the sums
      // A wait that gives up leaves the loop running (every later wait then returns at
      // once), so that all softmax warps meet at the same barriers.
      for (int t = t0; t < t0 + tiles; ++t) {
        const int sb = t & 1;
        q4_warp_wait(bar(L::SREADY + sb), (t >> 1) & 1, abort_flag);
        // written by the kernel before, known complete once the first scores are
        if (t == t0) unit = __ldcg(sigma + flat0 + min(head, mine - 1)) * scale;
        tc_fence_after();
        float x[kCols], y[kCols];
        const uint32_t s_at = lanes + 64 * sb + kCols * hh;
        tmem_ld16(s_at, reinterpret_cast<uint32_t*>(x));
        tmem_ld16(s_at + 128, reinterpret_cast<uint32_t*>(y));
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(lbar(L::SFREE + sb));
        // Scores above the head's reference.
#pragma unroll
        for (int i = 0; i < kCols; ++i) x[i] = fmaf(x[i], unit, fmaf(y[i], scale, -m));
        if (__any_sync(0xffffffffu, t * kTileRows + kCols > limit)) {
#pragma unroll
          for (int i = 0; i < kCols; ++i)
            if (t * kTileRows + i >= limit) x[i] = -INFINITY;
        }
        float mx = x[0];
#pragma unroll
        for (int i = 1; i < kCols; ++i) mx = fmaxf(mx, x[i]);
        // The eight warps of the same heads go by one reference, and decide alike.
        if (any_of(fresh || mx > L::kTop || t == due, 1 + (qd & 1), L::kSoft / 2)) {
          if (t > t0) {   // P and O: the output product of the tile before is done
            q4_warp_wait(bar(L::PVDONE + ((t - 1) & 1)), ((t - 1) >> 1) & 1, abort_flag);
            tc_fence_after();
          }
          red[part_of * 32 + lane] = mx;
          if (t == due) red[(2 * kSlices + part_of) * 32 + lane] = l;
          named_bar_sync(3 + (qd & 1), L::kSoft / 2);
          mx = red[lane];
#pragma unroll
          for (int i = 1; i < 2 * kSlices; ++i) mx = fmaxf(mx, red[i * 32 + lane]);
          const float was = fresh ? 0.f : *drop_at;
          float low = 0.f, sum = 0.f;
          if (t == due) {
#pragma unroll 1
            for (int i = 0; i < 2 * kSlices; ++i) sum += red[(2 * kSlices + i) * 32 + lane];
            low = q4_floor(sum, t - t0, 0.f, was);
          }
          named_bar_sync(3 + (qd & 1), L::kSoft / 2);   // read before any P is written
          // Move the reference (up, or down after a look, or to wherever its first tile has it);
          // rescale the sum and this warp's share of O.
          float up = mx - L::kBias;
          up = !fresh ? fmaxf(up, low) : mx == -INFINITY ? 0.f : up;
          // (nothing is summed before the first tile, whose reference may go down past what
          // 2^-up can hold)
          const float alpha = fresh ? 0.f : ex2(-up);
          const float drop = fresh ? 0.f : fmaxf(was - up, 0.f);
          if (part_of == 0) *drop_at = drop;
          due = t == due ? t + __reduce_min_sync(0xffffffffu,
                                                 head < mine ? q4_bears(sum * alpha, t - t0, drop)
                                                             : 1 << 20)
                         : min(due, t + kBearsTiles);
          fresh = fresh && mx == -INFINITY;
          m += up;
          l *= alpha;
#pragma unroll
          for (int i = 0; i < kCols; ++i) x[i] -= up;
          if (t > t0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < 16 / kSlices; ++c) {   // this warp's slice of O's 256 columns
              const uint32_t at = lanes + L::kOCol + 256 / kSlices * hh + 16 * c;
              float o[16];
              tmem_ld16(at, reinterpret_cast<uint32_t*>(o));
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= alpha;
              tmem_st8(at, o);
              tmem_st8(at + 8, o + 8);
            }
            tmem_wait_st();
          }
        }
        // The scores of this tile are done: its boxes' second halves, loaded.
        q4_warp_wait(bar(L::RAWFULL + slot), t & 1, abort_flag);
        Q4Piece piece;
        const int box_m = 2 * j + rank;
        piece.load(raw + 64 * box_m + 16 * c, raw[kQ4CodeBytes + 4 * box_m + c]);
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          x[i] = ex2(x[i]);
          l += x[i];
        }
        // P was last read by the output MMAs of tile t - 1.
        if (t >= 1) q4_warp_wait(bar(L::PVDONE + ((t - 1) & 1)), ((t - 1) >> 1) & 1, abort_flag);
        {
          // A operand, K-major: row `head` of each part's box, 128 bytes of tile rows.
          uint8_t* pb = smem + L::kOffP;
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a = 0, b = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // by way of fp16, where the remainder is exact
              const __half2 y = __floats2half2_rn(x[4 * w + 2 * e], x[4 * w + 2 * e + 1]);
              const uint32_t f1 = __nv_cvt_halfraw2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
              const __half2 g = __half2(
                  __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(f1), __NV_E4M3));
              const uint32_t f2 =
                  __nv_cvt_halfraw2_to_fp8x2(__hsub2(y, g), __NV_SATFINITE, __NV_E5M2);
              a |= f1 << (16 * e);
              b |= f2 << (16 * e);
            }
            hi[w] = a;
            lo[w] = b;
          }
          const uint32_t at = sw128(head, row0 / 16);
          *reinterpret_cast<uint4*>(pb + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(pb + kPBox + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::RAWEMPTY + slot));
          uint8_t* to = box + t % L::kTiles * 4 * kPBox;
          if (__all_sync(0xffffffffu, q4_plain(piece.e)))
            piece.store<true>(to, box_at, smem + L::kOffTable);
          else
            piece.store<false>(to, box_at, smem + L::kOffTable);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(lbar(L::PREADY + sb));
      }
      t0 += tiles;
      if (tid == 0 && t0 == T) pdl_launch_dependents();   // the combine waits for this grid anyway
      // The row sums of a head's threads, its log-sum-exp, and O / sum through shared memory
      // (over operands that nothing reads any more) to whole rows.
      q4_warp_wait(bar(L::PVDONE + ((t0 - 1) & 1)), ((t0 - 1) >> 1) & 1, abort_flag);
      tc_fence_after();
      red[part_of * 32 + lane] = l;
      named_bar_sync(5, L::kSoft);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 2 * kSlices; ++i) sum += red[i * 32 + lane];
      // Read before P is written again.  Whether the CTA has given up is asked here for all: some
      // warp may raise the flag at any time, and the softmax warps meet at a barrier below.
      if (!any_of(*abort_flag, 5, L::kSoft)) {
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        const bool whole = kShare ? whole_set(it) : p.direct != 0;   // the result itself
        const size_t stride = whole ? 1 : p.splits;
        const size_t row = static_cast<size_t>(flat0) * stride + (whole ? 0 : it.j);   // the first's
        float* o_to = kShare && whole ? static_cast<float*>(p.out) : p.part_o;
        float* lse_to = kShare && whole ? p.out_lse : p.part_lse;
        // Four values of row h, column x (results are bf16, partials fp32).
        auto put = [&](int h, int x, float4 o) {
          const size_t at = (row + static_cast<size_t>(h) * stride) * kDc + x;
          if (whole)
            *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(o_to) + at) =
                make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
          else
            *reinterpret_cast<float4*>(o_to + at) = o;
        };
        if (part_of == 0 && head < mine && lse_to)
          lse_to[row + static_cast<size_t>(head) * stride] =
              sum > 0.f ? (m + log2f(sum)) * kLn2 : -INFINITY;
        // This warp's slice of O's columns: in tile jj = col0 / 128 the lane's 128 columns are
        // latents 256 jj + 128 (qd >> 1) ..
        const int col0 = 256 / kSlices * hh;
        const int latent = 256 * (col0 >> 7) + 128 * (qd >> 1) + (col0 & 127);
        if (kShare && t0 < T) {
          // The next item's operands are on their way to where the last one stages: each warp
          // turns its 32 heads' columns over in P, 8 at a time, and writes 32 bytes of sixteen
          // rows at once.  The eight warps of the same heads keep to those heads' rows of P,
          // which they write again behind a barrier of their own.
          float4* mine4 = reinterpret_cast<float4*>(smem + L::kOffP + (warp >> 3) * kPBox +
                                                    4096 * (warp & 1) + 1024 * (warp >> 1 & 3));
          const int h0 = 32 * (qd & 1);
#pragma unroll 1
          for (int c = 0; c < 32 / kSlices; ++c) {
            float o[8];
            tmem_ld8(lanes + L::kOCol + col0 + 8 * c, reinterpret_cast<uint32_t*>(o));
#pragma unroll
            for (int i = 0; i < 2; ++i)
              mine4[2 * lane + (i ^ (lane >> 2 & 1))] = make_float4(
                  o[4 * i] * inv, o[4 * i + 1] * inv, o[4 * i + 2] * inv, o[4 * i + 3] * inv);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int r = 16 * i + (lane >> 1), q = lane & 1;
              if (h0 + r < mine)
                put(h0 + r, latent + 8 * c + 4 * q, mine4[2 * r + (q ^ (r >> 2 & 1))]);
            }
            __syncwarp();
          }
        } else {
          float* to = reinterpret_cast<float*>(smem + head * L::kStageRow) + latent;
#pragma unroll 1
          for (int c = 0; c < 16 / kSlices; ++c) {
            float o[16];
            tmem_ld16(lanes + L::kOCol + col0 + 16 * c, reinterpret_cast<uint32_t*>(o));
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<float4*>(to + 16 * c + 4 * i) =
                  make_float4(o[4 * i] * inv, o[4 * i + 1] * inv, o[4 * i + 2] * inv,
                              o[4 * i + 3] * inv);
          }
          named_bar_sync(5, L::kSoft);
          for (int h = warp; h < mine; h += L::kSoftWarps) {
            const float4* src = reinterpret_cast<const float4*>(smem + h * L::kStageRow);
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

template <bool kShare>
mla_status launch_q4_pair(const CUtensorMap& q, const CUtensorMap& qpe, const SplitParams& p,
                          cudaStream_t s, const char* who) {
  using L = Q4Pair;
  static DeviceFlags attr_done;
  const int dev = current_device();
  if (!attr_done.test(dev)) {
    if (cudaFuncSetAttribute(split_q4_pair_kernel<kShare>,
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
  cfg.blockDim = dim3(L::kThreads);
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
  cudaLaunchKernelEx(&cfg, split_q4_pair_kernel<kShare>, q, qpe, p,
                     static_cast<const float*>(pair_units(p)));
  return launch_status(who);
}

}  // namespace

mla_status launch_split_q4_pair(const SplitParams& p, cudaStream_t stream, const char* who) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) {
    set_error("%s: cuTensorMapEncodeTiled is not available from the driver", who);
    return MLA_ERR_CUDA;
  }
  // The queries, in boxes of one CTA's 64 heads x 128 bytes (128-byte swizzle).
  CUresult bad = CUDA_SUCCESS;
  auto encode = [&](CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, int elt) {
    const cuuint64_t gdim[2] = {cols, rows}, gstride[1] = {cols * elt};
    const cuuint32_t box[2] = {cuuint32_t(128 / elt), kPHeads}, estride[2] = {1, 1};
    const CUresult r = enc(m, elt == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                           2, const_cast<void*>(base), gdim, gstride, box, estride,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) bad = r;
  };
  const uint64_t rows = static_cast<uint64_t>(p.B) * p.H;
  CUtensorMap tq, tp;
  encode(&tq, pair_codes(p), kQ8Row, 2 * rows, 1);
  encode(&tp, p.q_pe, kDr, rows, 2);
  if (bad != CUDA_SUCCESS) {
    set_error("%s: cuTensorMapEncodeTiled failed (%d)", who, int(bad));
    return MLA_ERR_CUDA;
  }
  if (!p.late) {
    const mla_status st = launch_pair_queries(p, stream, who);
    if (st != MLA_OK) return st;
  }
  return p.pieces ? launch_q4_pair<true>(tq, tp, p, stream, who)
                  : launch_q4_pair<false>(tq, tp, p, stream, who);
}

}  // namespace mla
