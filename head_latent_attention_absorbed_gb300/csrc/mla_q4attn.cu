// The split kernel over a 4-bit pool, 16 heads per CTA.
//
// Per head the score of row t is q_abs . c_t + q_pe . k_t over sqrt(d_h + d_R), an online
// softmax over the chunk's rows, and the normalised latent output with its log-sum-exp
// ("Multi-Head Latent Attention" 3.3, 3.6).  c_t are the pool's values: E2M1 codes times a
// power of two per 16, each of them an E4M3 number (mla_q4.cuh).
//
// So a tile of 128 rows (50 KB) is brought into shared memory as it is stored, and its codes
// are turned into E4M3 bytes there, once, by warps of their own; both products then run on
// the tensor cores as in the E4M3 cache's kernel (kind::f8f6f4, fp32 accumulators), and the
// keys, stored as the tensor core wants them, as kind::f16:
//   scores  S[128 rows x 16 parts] = C[128 x 512] . Q^T,  Sk[128 x 16] = K[128 x 64] . Qk^T
//   output  O^T[128 latent x 16 parts] += C^T[128 x 128 rows] . P^T   per 128-column block
// A bf16 query is two E4M3 parts (weights 1, 1/16; exact to 2^-21 of the head's largest
// value) in units of a power of two per head, and P two parts (at most 2^-8 relative, less in
// the weighted sum than the bf16 output's own rounding); an fp32 query is four parts, its key
// part a bf16 hi and lo, and P three (2^-12).  The parts' smallest step is 2^-13 (three: 2^-17)
// of the softmax's reference, which therefore follows the scores up and down (mla_q4.cuh): it lies
// 2^5 below the largest score of the tile where it last moved, and goes up, rescaling O, when a
// score passes it by 2^8.5.
//
// From codes to E4M3: a byte permute looks the eight magnitudes of a block's exponent up in
// two registers, four codes at a time (the selector is the codes themselves), and the signs
// lie where the bytes want them: seven operations for eight values, no conversion (which
// would run at an eighth of the rate) and no multiplication.
//
// Warp roles (640 threads, one CTA per SM):
//   warps 0-7    softmax (one tile row per thread, heads 0-7 in warps 0-3, 8-15 in 4-7),
//                P, epilogue
//   warp 8       copies of codes and exponents (and TMEM allocation)
//   warp 9       score MMAs of each tile (20 instructions)
//   warp 10      the first query image's copy, then the PV MMAs of each tile (16)
//   warp 11      copies of keys, and of the later items' query images
//   warps 12-19  codes to E4M3, two teams of four warps in turn
// (A copy takes its warp some 450 cycles among the others' work: one warp for all of a
// tile's, and exponents in a plane of their own, took 6600 cycles a tile.)
//
// What bounds it: a tile's way through its two buffers (codes to E4M3 0.6 us beyond what is done
// before the wait for the buffer, score MMAs 0.6, softmax 0.9, output MMAs 0.9 and what lies
// between), and the decoding warps, busy for nine tenths of a tile's 1.8 us, on a shared memory
// that the tensor cores' reads (1440 of 3500 cycles), the threads' (1200) and copies (400) keep
// busy; HBM would allow 1.15.
// 64 sequences of 512 to 8192 rows 39.9 us (2.8 TB/s of cache), 4 x 65536 rows 36.3, with an E4M3
// cache, whose rows are longer and need no decoding, 44.5 and 39.5.  Not kept (us of those two,
// when they took 41.4 and 37.4): four teams on 72 registers 44.7 / 40.6, the scores' operand in
// tensor memory, where the decoding warps put it too, 42.1 / 38.3 (and before they wait for the
// tile's buffer, so that scores run ahead of the output, 9 % slower), boxes handed over one by one
// 41.5 / 37.7, all of a tile decoded before the wait for its buffer 42.4 / 38.7.
#include <type_traits>

#include "mla_q4.cuh"

namespace mla {
namespace {

constexpr int kRowsT = 128;                   // rows per tile (the MMA's M)
constexpr int kBox = kRowsT * 128;            // 128 latent columns of a tile: 16 KB
constexpr int kTile = 4 * kBox;               // 64 KB of E4M3
constexpr int kKeyTile = kRowsT * kQ4KeyBytes;   // 16 KB of bf16 keys
constexpr int kSoft = 256;
constexpr int kTeam = 128, kTeams = 2;        // threads of a decoding team, and teams
constexpr int kThreads = kSoft + 4 * 32 + kTeams * kTeam;
constexpr int kHalf = kHeadGroup / 2;         // heads per softmax warp group
constexpr uint32_t kTmemCols = 512;   // S[2] at 0 / 64, O^T from 128 to 319, Sk[2] at 320 / 352
constexpr uint32_t kOCol = 128, kKCol = 320;

// The query of one (sequence, 16-head group) as shared memory holds it: four 128-column
// boxes of (parts x 16) rows x 128 bytes, the key part's (hi, or hi and lo) x 16 rows x 128
// bytes, both 128-byte swizzled, and the 16 scales.
template <bool kF32>
struct Q4Plan {
  static constexpr int kQParts = kF32 ? 4 : 2, kKParts = kF32 ? 2 : 1;
  static constexpr int kPParts = kF32 ? 3 : 2;
  static constexpr int kPN = kPParts * kHeadGroup;   // P rows of the PV MMA (part-major)
  static constexpr int kPBuf = kPN * 128;            // of 128 tile rows
  // Where the softmax's reference goes below a tile's largest score when it moves, and how far
  // above the reference that score may then lie in later tiles (log2): weights stay below E4M3's
  // 448.
  static constexpr float kBias = 5.f, kTop = 8.5f;
  static constexpr int kQN = kQParts * kHeadGroup, kKN = kKParts * kHeadGroup;
  static constexpr int kQBox = kQN * 128;
  static constexpr int kQKeys = 4 * kQBox;                  // offset of the key part
  static constexpr int kQBytes = kQKeys + kKN * 128;        // of the scales
  static_assert(size_t(kQBytes) + 64 <= kFp8QImage, "query image in the workspace");
  // Rows arrive in slots, whose length is what room is left.  Their number is a multiple of
  // the teams that decode them in turn: each team then meets every phase of its slots (a
  // parity wait that skips one passes too early).
  static constexpr int kSlotRows = kF32 ? 16 : 32, kSlots = 4;
  static_assert(kSlots % kTeams == 0 && (kRowsT / kSlotRows) % kTeams == 0 &&
                    kRowsT / kSlotRows >= 2 * kTeams && kSlots >= 2 * kTeams,
                "slots by team");
  static constexpr int kSlotBytes = kSlotRows * kQ4LatBytes;
  static constexpr int kOffTile = 0;
  static constexpr int kOffKeys = kOffTile + 2 * kTile;
  static constexpr int kOffQ = kOffKeys + 2 * kKeyTile;
  static constexpr int kOffP = kOffQ + kQBytes;
  static constexpr int kOffRaw = kOffP + 2 * kPBuf;
  static constexpr int kOffTable = kOffRaw + kSlots * kSlotBytes;   // [16] magnitudes by exponent
  static constexpr int kOffRed = kOffTable + 16 * 8;                // [16 heads][4 warps] maxima
  static constexpr int kOffLsum = kOffRed + kHeadGroup * 4 * 4;
  static constexpr int kOffBar = kOffLsum + kHeadGroup * 4 * 4;
  static constexpr int RAWFULL = 0, RAWEMPTY = RAWFULL + kSlots,   // rows landed / decoded
                       KEYFULL = RAWEMPTY + kSlots,   // [2] keys of the tile landed
                       CFULL = KEYFULL + 2,           // [2] tile decoded (both teams)
                       SFULL = CFULL + 2,             // [2] scores of the tile (keys free again)
                       SFREE = SFULL + 2,             // [2] softmax read them
                       PFULL = SFREE + 2,             // [2] P of the tile written
                       ODONE = PFULL + 2,             // [2] PV of the tile finished (tile free)
                       QREADY = ODONE + 2, DONE = QREADY + 1, kBars = DONE + 1;
  static constexpr int kOffSlot = kOffBar + 8 * kBars;
  static constexpr int kOffAbort = kOffSlot + 16;    // flag, limit of the waits
  static constexpr int kOffShare = kOffAbort + 16;   // TileShare of the CTA
  static constexpr size_t kSmem = 1024 + kOffShare + 32;
  static_assert(kSmem <= 232448, "shared memory");
  static_assert(kOffQ % 1024 == 0 && kQKeys % 1024 == 0 && kOffP % 1024 == 0, "swizzle atoms");
  static_assert(kOffRaw % 128 == 0 && kSlotBytes % 16 == 0 && kOffBar % 8 == 0, "alignment");
  static_assert(kBars <= 32, "a barrier per lane");
};

// Four K steps of a product, `sa` and `sb` (16-byte units) apart, by one elected thread of the
// converged warp; the first replaces what D holds unless `accumulate`.  (One at a time, with an
// election each, a step took its warp some 90 cycles among the others' work.)
template <bool kE4m3, int kSa, int kSb>
__device__ __forceinline__ void umma_x4(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate) {
#define MLA_Q4_STEPS(KIND)                                                                    \
  asm volatile(                                                                               \
      "{\n\t.reg .pred p, e, t;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\t"               \
      "setp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"                               \
      "@e tcgen05.mma.cta_group::1.kind::" KIND " [%0], %1, %2, %3, p;\n\t"                   \
      "add.s64 a, %1, %5;\n\tadd.s64 b, %2, %6;\n\t"                                          \
      "@e tcgen05.mma.cta_group::1.kind::" KIND " [%0], a, b, %3, t;\n\t"                     \
      "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"                                            \
      "@e tcgen05.mma.cta_group::1.kind::" KIND " [%0], a, b, %3, t;\n\t"                     \
      "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"                                            \
      "@e tcgen05.mma.cta_group::1.kind::" KIND " [%0], a, b, %3, t;\n\t}" ::"r"(tmem_d),     \
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(kSa), "n"(kSb)                         \
      : "memory")
  if constexpr (kE4m3)
    MLA_Q4_STEPS("f8f6f4");
  else
    MLA_Q4_STEPS("f16");
#undef MLA_Q4_STEPS
}
// kind::f8f6f4 with E4M3 A and B and fp32 accumulators; a_mn selects an MN-major A.
constexpr uint32_t idesc_e4m3(int M, int N, int a_mn) {
  return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ float2 from_e4m3x2(uint16_t v) {
  return __half22float2(
      __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E4M3)));
}
// Byte offset of K index k (< 128) in row n of a K-major box of 128-byte rows with the
// 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128_byte(int n, int k) {
  return static_cast<uint32_t>(n * 128 + ((((k >> 4) ^ n) & 7) << 4) + (k & 15));
}

// Of eight values a lane, over a warp's lanes: lane i's result is that of value i mod 8.  (Halves
// of the values go to and fro: nine exchanges, where a value at a time would take 40.)
template <typename Op>
__device__ __forceinline__ float over_lanes(const float (&v)[kHalf], int lane, Op op) {
  static_assert(kHalf == 8, "three steps");
  float a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float send = lane & 1 ? v[2 * i] : v[2 * i + 1], keep = lane & 1 ? v[2 * i + 1] : v[2 * i];
    a[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, 1));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float send = lane & 2 ? a[2 * i] : a[2 * i + 1], keep = lane & 2 ? a[2 * i + 1] : a[2 * i];
    b[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, 2));
  }
  const float send = lane & 4 ? b[0] : b[1], keep = lane & 4 ? b[1] : b[0];
  float r = op(keep, __shfl_xor_sync(0xffffffffu, send, 4));
  r = op(r, __shfl_xor_sync(0xffffffffu, r, 8));
  return op(r, __shfl_xor_sync(0xffffffffu, r, 16));
}

// Where the rows of a page that does not exist come from.
__device__ __align__(128) uint8_t g_q4_zeros[kRowsT * kQ4LatBytes];

// The query image of one (query group b, head h), in units of sigma, a power of two that puts
// the largest magnitude of q_abs and q_pe in [128, 256): q_abs (512 values) becomes a1 + a2 /
// 16 + ..., a_i E4M3, q_pe a bf16 value, or hi and lo.  Part i goes to row 16 i + (h mod 16) of the group's image.
// grid (H, B), 160 threads: thread t < 128 converts values 4 t .., thread 128 + u keys 4 u ..
template <bool kF32>
__global__ void __launch_bounds__(160) q4_query_kernel(const SplitParams p) {
  using L = Q4Plan<kF32>;
  __shared__ float wmax[5];
  pdl_launch_dependents();   // the split may begin its set-up and cache stream
  const int h = blockIdx.x, b = blockIdx.y, t = threadIdx.x, lane = t & 31;
  const int hh = h % kHeadGroup;
  uint8_t* img = p.q_img + (size_t(b) * (p.H / kHeadGroup) + h / kHeadGroup) * kFp8QImage;
  pdl_wait();   // the queries come from the kernel before, and one may still read the image
  const size_t bh = size_t(b) * p.H + h;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  const size_t at = t < 128 ? bh * kDc + 4 * t : bh * kDr + 4 * (t - 128);
  if (t < 144) {
    const void* src = t < 128 ? p.q_abs : p.q_pe;
    if (kF32) {
      v = *reinterpret_cast<const float4*>(static_cast<const float*>(src) + at);
    } else {
      const uint2 q2 = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(src) + at);
      v = make_float4(__uint_as_float(q2.x << 16), __uint_as_float(q2.x & 0xffff0000u),
                      __uint_as_float(q2.y << 16), __uint_as_float(q2.y & 0xffff0000u));
    }
  }
  float mx = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  if (lane == 0) wmax[t >> 5] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3])), wmax[4]);
  int ex = 0;
  frexpf(mx, &ex);   // mx = f 2^ex, f in [0.5, 1)
  ex = max(ex, -100);   // keeps 1 / sg finite; smaller queries score as zero to 2^-100
  const float sg = mx > 0.f ? ldexpf(1.f, ex - 8) : 1.f;
  const float inv = 1.f / sg;   // exact: a power of two
  if (t == 0) reinterpret_cast<float*>(img + L::kQBytes)[hh] = sg;
  if (t < 128) {
    float x0 = v.x * inv, x1 = v.y * inv, x2 = v.z * inv, x3 = v.w * inv;
    uint8_t* bx = img + (t >> 5) * L::kQBox;
#pragma unroll
    for (int part = 0; part < L::kQParts; ++part) {
      const uint16_t lo = to_e4m3x2(x0, x1), hi = to_e4m3x2(x2, x3);
      *reinterpret_cast<uint32_t*>(bx + sw128_byte(kHeadGroup * part + hh, (4 * t) & 127)) =
          static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
      const float2 f01 = from_e4m3x2(lo), f23 = from_e4m3x2(hi);
      // the residuals of a rounding are exact
      x0 = (x0 - f01.x) * 16.f;
      x1 = (x1 - f01.y) * 16.f;
      x2 = (x2 - f23.x) * 16.f;
      x3 = (x3 - f23.y) * 16.f;
    }
  } else if (t < 144) {
    uint32_t hi0, lo0, hi1, lo1;
    split_bf16(v.x * inv, v.y * inv, hi0, lo0);
    split_bf16(v.z * inv, v.w * inv, hi1, lo1);
    uint8_t* to = img + L::kQKeys;
    const int k = 8 * (t - 128);   // bytes
    *reinterpret_cast<uint2*>(to + sw128_byte(hh, k)) = make_uint2(hi0, hi1);
    if (kF32) *reinterpret_cast<uint2*>(to + sw128_byte(kHeadGroup + hh, k)) = make_uint2(lo0, lo1);
  }
}

// kShare: one CTA per SM takes an equal run of all query groups' tiles (take_share), one item
// per query group it meets, streamed back to back; otherwise a CTA has one item, its chunk.
template <bool kF32, bool kShare>
__global__ void __launch_bounds__(kThreads, 1) split_q4_kernel(const SplitParams p) {
  using L = Q4Plan<kF32>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + L::kOffBar;
  float* red = reinterpret_cast<float*>(smem + L::kOffRed);
  float* lsum = reinterpret_cast<float*>(smem + L::kOffLsum);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffAbort);
  uint32_t* slot_ptr = reinterpret_cast<uint32_t*>(smem + L::kOffSlot);
  auto bar = [&](int i) { return bars + 8 * i; };

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // uniform to the compiler
  const int groups = p.H / kHeadGroup;
  const int g = kShare ? blockIdx.x % groups : blockIdx.x, h0 = g * kHeadGroup;
  TileItem first{0, 0, 0, 0, 0};   // the CTA's first item (none: T = 0)
  int T = 0, row_end = 0;  // tiles of the CTA; the row behind its chunk
  TileShare share{};
  if (!kShare) {
    const int j = blockIdx.y, b = blockIdx.z;
    if (p.late) pdl_wait();
    const int len = clamp_length(p, b, tid == 0 && g == 0 && j == 0);
    const int r0 = j * p.chunk;
    if (r0 >= len) {   // chunk past the end of this sequence: nothing to do
      if (p.direct || r0 == 0) pdl_wait();   // no row at all: see launch_pdl
      if (p.direct) write_no_rows(p, size_t(b) * p.H + h0, kHeadGroup, tid, kThreads);
      return;
    }
    row_end = min(r0 + p.chunk, len);
    T = (row_end - r0 + kRowsT - 1) / kRowsT;
    first = TileItem{b, j, r0, T, len};
  }
  auto begin_share = [&] {
    T = uniform(share.tiles);
    first = first_item<false>(p, share, blockIdx.x / groups);
  };
  auto item_after = [&](const TileItem& it, int t) { return next_item<false>(p, it, T - t); };

  // A tile is 128 / piece pieces of rows of one page each (for the copies of latents at most a
  // slot); lane i knows the page of piece i, looked up a tile ahead: -1, outside the pool, or
  // -2, past the sequence's end.
  const uint8_t* pool = static_cast<const uint8_t*>(p.cache);
  const uint64_t pol = l2_evict_first_policy();
  auto piece_page = [&](const TileItem& it, int i, int piece) {
    const int r = it.r0 + i * kRowsT + lane * piece;
    if (lane * piece >= kRowsT || r >= it.len) return -2;
    const int id = p.table[static_cast<size_t>(cache_seq(p, it.v)) * p.table_stride + (r >> p.page_shift)];
    return id < 0 ? -1 : id;
  };
  // Where lane i's piece comes from, in the plane at `plane` bytes a row of the page and of
  // `bytes` bytes a row; r0: the tile's first row.
  auto piece_source = [&](int id, int r0, int piece, int plane, int bytes) {
    if (id >= p.num_pages) id = -1;
    if (id == -1) report(p.status, MLA_DEV_PAGE_OUT_OF_RANGE);
    const int r = (r0 + lane * piece) & ((1 << p.page_shift) - 1);
    return id < 0 ? g_q4_zeros
                  : pool + (static_cast<size_t>(id) << p.page_shift) * kQ4RowBytes +
                        (static_cast<size_t>(plane) << p.page_shift) + r * bytes;
  };
  // Copies pieces from .. to - 1, the first `live` of which lie in the sequence, to dst on.
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
  const int lat_piece = min(1 << p.page_shift, L::kSlotRows);
  const int key_piece = min(1 << p.page_shift, kRowsT);
  constexpr int kTileSlots = kRowsT / L::kSlotRows;
  // Slot n of the CTA, of the tile whose pieces come from `src`.
  auto issue_slot = [&](const uint8_t* src, int live, int n) {   // false: given up
    const int at = n % L::kSlots, per = L::kSlotRows / lat_piece, from = n % kTileSlots * per;
    if (n >= L::kSlots) {
      q4_warp_wait(bar(L::RAWEMPTY + at), (n / L::kSlots - 1) & 1, abort_flag);
      if (__any_sync(0xffffffffu, *abort_flag)) return false;
    }
    copy_pieces(src, from, from + per, live, lat_piece * kQ4LatBytes,
                sbase + L::kOffRaw + at * L::kSlotBytes, bar(L::RAWFULL + at));
    return true;
  };
  auto issue_keys = [&](int id, int r0, int t) {   // false: given up
    const int bf = t & 1;
    const uint8_t* src = piece_source(id, r0, key_piece, kQ4LatBytes, kQ4KeyBytes);
    if (t >= 2) {
      q4_warp_wait(bar(L::SFULL + bf), ((t - 2) >> 1) & 1, abort_flag);
      if (__any_sync(0xffffffffu, *abort_flag)) return false;
    }
    copy_pieces(src, 0, kRowsT / key_piece, __popc(__ballot_sync(0xffffffffu, id != -2)),
                key_piece * kQ4KeyBytes, sbase + L::kOffKeys + bf * kKeyTile, bar(L::KEYFULL + bf));
    return true;
  };
  // The query image of group v, by one thread.  (The scales stay behind: of a share this copy
  // may run ahead of the softmax, which reads them from global memory.)
  auto load_query = [&](int v) {
    const uint8_t* img = p.q_img + (size_t(v) * groups + g) * kFp8QImage;
    mbar_arrive_expect_tx(bar(L::QREADY), L::kQBytes);
    bulk_g2s(sbase + L::kOffQ, img, L::kQBytes, bar(L::QREADY));
  };
  int slots = 0;   // slots issued (warp 8)
  if (warp == 8) {
    if (kShare) {
      share = take_share<false>(p, blockIdx.x / groups, gridDim.x / groups, lane, blockIdx.x == 0);
      if (lane == 0) *reinterpret_cast<TileShare*>(smem + L::kOffShare) = share;
      if (share.tiles > 0)
        begin_share();
      else
        T = 0;
    }
    int id = -2, key_id = -2;
    if (T > 0) {
      id = piece_page(first, 0, lat_piece);
      key_id = piece_page(first, 0, key_piece);
    }
    if (lane < L::kBars)
      // counts: slots decoded by a team's warps, tiles by all teams'; S read and P written by
      // the softmax warps
      mbar_init(bar(lane), lane >= L::SFREE && lane < L::ODONE      ? kSoft / 32
                           : lane >= L::CFULL && lane < L::SFULL    ? kTeams * kTeam / 32
                           : lane >= L::RAWEMPTY && lane < L::KEYFULL ? kTeam / 32
                                                                      : 1);
    if (lane == 0) q4_wait_init(p, abort_flag);
    fence_mbarrier_init();
    __syncwarp();
    if (T > 0) {   // the stream starts before the CTA's barrier
      const uint8_t* src = piece_source(id, first.r0, lat_piece, 0, kQ4LatBytes);
      const int live = __popc(__ballot_sync(0xffffffffu, id != -2));
      for (; slots < min(L::kSlots, kTileSlots); ++slots) issue_slot(src, live, slots);
      issue_keys(key_id, first.r0, 0);
    }
    if (!kShare || T > 0) tmem_alloc(smem_u32(slot_ptr), kTmemCols);
  } else if (warp == 12 && lane < 16) {
    q4_table(smem + L::kOffTable, lane);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (kShare) {
    share = *reinterpret_cast<const TileShare*>(smem + L::kOffShare);
    if (share.tiles <= 0) {   // more CTAs than tiles
      pdl_wait();
      return;
    }
    if (warp != 8) begin_share();
  }
  const uint32_t tmem = __shfl_sync(0xffffffffu, *slot_ptr, 0);   // uniform to the compiler

  // Runs the tiles of the CTA, each with its pieces' pages: f(id, first row, t, first of a
  // later item, that item); false: given up.
  auto for_tiles = [&](int piece, auto&& f) {
    TileItem it = first;
    int i = 0, id = piece_page(it, 0, piece);
    for (int t = 0; t < T; ++t) {
      if (__any_sync(0xffffffffu, *abort_flag)) return;
      const TileItem now = it;
      const int at = i, now_id = id;
      if (t + 1 < T) {
        if (++i == it.tiles) {
          it = item_after(it, t + 1);
          i = 0;
        }
        id = piece_page(it, i, piece);
      }
      f(now_id, now.r0 + at * kRowsT, t, at == 0 && t > 0, now);
    }
  };
  if (warp == 8) {
    // ------------------------------------------------------------ codes and exponents
    for_tiles(lat_piece, [&](int id, int r0, int t, bool, const TileItem&) {
      if (p.stop_after_tiles > 0 && t >= p.stop_after_tiles) return;   // test hook
      const uint8_t* src = piece_source(id, r0, lat_piece, 0, kQ4LatBytes);
      const int live = __popc(__ballot_sync(0xffffffffu, id != -2));
      while (slots < (t + 1) * kTileSlots && issue_slot(src, live, slots)) ++slots;
    });
    // Copies still in flight land before the CTA may leave (bounded waits).
    for (int n = max(0, slots - L::kSlots); n < slots; ++n)
      if (!mbar_wait_bounded(bar(L::RAWFULL + n % L::kSlots), (n / L::kSlots) & 1)) *abort_flag = 1;
  } else if (warp == 11) {
    // ------------------------------------------------------------ keys, later queries
    int keys = T > 0 ? 1 : 0;   // tiles whose keys are on their way (the first from warp 8)
    for_tiles(key_piece, [&](int id, int r0, int t, bool later, const TileItem& now) {
      if (t > 0 && issue_keys(id, r0, t)) keys = t + 1;
      if (kShare && later) {
        // A new item's query, once the last score MMA of the one before has read its own.
        q4_warp_wait(bar(L::SFULL + ((t - 1) & 1)), ((t - 1) >> 1) & 1, abort_flag);
        if (!__any_sync(0xffffffffu, *abort_flag) && lane == 0) {
          pdl_wait();
          load_query(now.v);
        }
        __syncwarp();
      }
    });
    for (int t = max(0, keys - 2); t < keys; ++t)
      if (!mbar_wait_bounded(bar(L::KEYFULL + (t & 1)), (t >> 1) & 1)) *abort_flag = 1;
  } else if (warp > 11) {
    // ------------------------------------------------------------ codes to E4M3
    // Teams take slots in turn; warp m of a team decodes box m of a slot, a row (or, of slots
    // of 16 rows, half of one) per lane: rows are 17 times 16 bytes apart, so eight lanes read
    // from eight different pieces of the banks, and the swizzle has them write so too.
    const int team = (warp - 12) >> 2, m = (warp - 12) & 3;
    const int r = lane % L::kSlotRows, part = lane / L::kSlotRows;
    constexpr int kEach = L::kSlotRows / 8;   // 16-byte pieces of codes (32 values) a lane
    const uint8_t* from = smem + L::kOffRaw + r * kQ4LatBytes + 64 * m + 16 * kEach * part;
    const uint8_t* exps = smem + L::kOffRaw + r * kQ4LatBytes + kQ4CodeBytes + 4 * m + kEach * part;
    using Exps = std::conditional_t<kEach == 4, uint32_t, uint16_t>;   // a byte per piece
    static_assert(sizeof(Exps) == kEach, "a byte of exponents per piece");
    const uint8_t* table = smem + L::kOffTable;
    uint8_t* to = smem + L::kOffTile + m * kBox + r * 128;
    const uint32_t swz = (r & 7) << 4, unit0 = 2 * kEach * part;
    // Slot n's codes, and the slot given back; true: of plain exponents.  (Exponents by bytes:
    // four loads that meet in the same banks for one.)
    auto load = [&](Q4Piece (&piece)[kEach], int n) {
      const int slot = n % L::kSlots;
      q4_warp_wait(bar(L::RAWFULL + slot), (n / L::kSlots) & 1, abort_flag);
      const uint32_t e = *reinterpret_cast<const Exps*>(exps + slot * L::kSlotBytes);
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        piece[k].load(from + slot * L::kSlotBytes + 16 * k, e >> 8 * k);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::RAWEMPTY + slot));
      return __all_sync(0xffffffffu, q4_plain(e)) != 0;
    };
    auto store = [&](const Q4Piece (&piece)[kEach], bool plain, uint8_t* row) {
      if (plain) {
#pragma unroll
        for (int k = 0; k < kEach; ++k)
          piece[k].template store<true>(row, ((unit0 + 2 * k) << 4) ^ swz, table);
      } else {
#pragma unroll
        for (int k = 0; k < kEach; ++k)
          piece[k].template store<false>(row, ((unit0 + 2 * k) << 4) ^ swz, table);
      }
    };
    int n = team;
    for (int t = 0; t < T; ++t) {
      if (__any_sync(0xffffffffu, *abort_flag)) break;
      // A tile's way through its buffer, from here to the end of its output product, is part of
      // what bounds the kernel: the team's first slot is decoded, and the second read, before the
      // wait for the buffer.
      Q4Piece piece[kEach];
      uint4 e4m3[kEach][2];
      if (load(piece, n)) {
#pragma unroll
        for (int k = 0; k < kEach; ++k)
          piece[k].template decode<true>(e4m3[k][0], e4m3[k][1], table);
      } else {
#pragma unroll
        for (int k = 0; k < kEach; ++k)
          piece[k].template decode<false>(e4m3[k][0], e4m3[k][1], table);
      }
      n += kTeams;
      bool plain = load(piece, n);
      n += kTeams;
      if (t >= 2) {
        q4_warp_wait(bar(L::ODONE + (t & 1)), ((t - 2) >> 1) & 1, abort_flag);
        tc_fence_after();
      }
      uint8_t* rows = to + (t & 1) * kTile + team * L::kSlotRows * 128;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        *reinterpret_cast<uint4*>(rows + (((unit0 + 2 * k) << 4) ^ swz)) = e4m3[k][0];
        *reinterpret_cast<uint4*>(rows + (((unit0 + 2 * k + 1) << 4) ^ swz)) = e4m3[k][1];
      }
      constexpr int kStep = kTeams * L::kSlotRows * 128;
      store(piece, plain, rows += kStep);
#pragma unroll 1
      for (int s = 2 * kTeams; s < kTileSlots; s += kTeams, n += kTeams) {
        plain = load(piece, n);
        store(piece, plain, rows += kStep);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::CFULL + (t & 1)));
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ score MMAs
    // The whole warp runs along, converged at every MMA; boxes are not unrolled (code
    // that runs once a tile is fetched anew each time).
    constexpr uint32_t idesc_s = idesc_e4m3(128, L::kQN, 0);
    constexpr uint32_t idesc_k = umma_idesc_bf16(128, L::kKN, 0, 0);
    const uint64_t a0 = umma_desc_sw128(sbase + L::kOffTile, 16, 1024);
    const uint64_t k0 = umma_desc_sw128(sbase + L::kOffKeys, 16, 1024);
    const uint64_t q0 = umma_desc_sw128(sbase + L::kOffQ, 16, 1024);
    TileItem cur = first;
    int left = 0, n = 0;   // tiles left of the item; items begun
    for (int t = 0; t < T; ++t) {
      const int bf = t & 1;
      if (left == 0) {
        if (t > 0) cur = item_after(cur, t);
        left = cur.tiles;
        q4_warp_wait(bar(L::QREADY), n & 1, abort_flag);
        if (kShare && g == 0 && lane == 0 && cur.r0 == 0) {
          // The run with a query group's first tile says how many runs it spans.  (Not
          // before a query is here, fetched behind the PDL wait: the combine of the call
          // before may still be reading its own counts.)
          p.pieces[cur.v] = count_pieces(cur, share.first + t, share.each);
        }
        ++n;
      }
      --left;
      if (t >= 2) q4_warp_wait(bar(L::SFREE + bf), ((t - 2) >> 1) & 1, abort_flag);
      q4_warp_wait(bar(L::KEYFULL + bf), (t >> 1) & 1, abort_flag);
      if (__any_sync(0xffffffffu, *abort_flag)) break;
      tc_fence_after();
      // 16 key values (32 bytes) a step
      umma_x4<false, 2, 2>(tmem + kKCol + 32 * bf, k0 + ((bf * kKeyTile) >> 4),
                           q0 + (L::kQKeys >> 4), idesc_k, 0);
      q4_warp_wait(bar(L::CFULL + bf), (t >> 1) & 1, abort_flag);
      if (__any_sync(0xffffffffu, *abort_flag)) break;
      tc_fence_after();
#pragma unroll 1
      for (int m = 0; m < 4; ++m) {
        const uint64_t a = a0 + static_cast<uint64_t>((bf * kTile + m * kBox) >> 4);
        const uint64_t q = q0 + static_cast<uint64_t>((m * L::kQBox) >> 4);
        umma_x4<true, 2, 2>(tmem + 64 * bf, a, q, idesc_s, m > 0 ? 1u : 0u);   // 32 columns a step
      }
      umma_commit_elected(bar(L::SFULL + bf));
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------ query image, PV MMAs
    if (lane == 0) {
      pdl_wait();   // the image is written by the kernel before
      load_query(first.v);
    }
    __syncwarp();
    constexpr uint32_t idesc_o = idesc_e4m3(128, L::kPN, 1);
    const uint64_t p0 = umma_desc_sw128(sbase + L::kOffP, 16, 1024);
    const uint64_t c0 = umma_desc_sw128(sbase + L::kOffTile, kBox, 1024);
    TileItem cur = first;
    int done = 0;   // tiles of the item accumulated
    for (int t = 0; t < T; ++t, ++done) {
      const int bf = t & 1;
      if (kShare && done == cur.tiles) {
        cur = item_after(cur, t);
        done = 0;
      }
      q4_warp_wait(bar(L::PFULL + bf), (t >> 1) & 1, abort_flag);
      if (__any_sync(0xffffffffu, *abort_flag)) break;
      tc_fence_after();
      const uint64_t pd = p0 + static_cast<uint64_t>((bf * L::kPBuf) >> 4);
#pragma unroll 1
      for (int mb = 0; mb < 4; ++mb) {
        // C^T block mb: latent columns 128 mb.. (MN-major, one 128-byte
        // span), K = tile rows in 8-row groups 1024 B apart
        const uint64_t c = c0 + static_cast<uint64_t>((bf * kTile + mb * kBox) >> 4);
        // 32 tile rows per step: 4096 B of C^T, 32 B of P^T
        umma_x4<true, 4096 / 16, 32 / 16>(tmem + kOCol + L::kPN * mb, c, pd, idesc_o,
                                          done > 0 ? 1u : 0u);
      }
      umma_commit_elected(bar(L::ODONE + bf));
    }
    umma_commit_elected(bar(L::DONE));
    mbar_wait_bounded(bar(L::DONE), 0);
  } else {
    // ------------------------------------------------------------ softmax warps
    const int gp = warp >> 2, wq = warp & 3;
    const int hb = kHalf * gp;                          // first head of this group
    const int row = 32 * wq + lane;                     // tile row held by this thread
    const uint32_t lane_base = static_cast<uint32_t>(32 * wq) << 16;
    TileItem cur = first;
    float qsig[kHalf];
    auto read_scales = [&] {   // of the item
      const float4* sg = reinterpret_cast<const float4*>(
          p.q_img + (size_t(cur.v) * groups + g) * kFp8QImage + L::kQBytes + 4 * hb);
      const float4 s0 = __ldcg(sg), s1 = __ldcg(sg + 1);
      const float s[kHalf] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
      for (int h = 0; h < kHalf; ++h) qsig[h] = s[h] * p.scale_log2;
    };
    pdl_wait();   // the scales come with the query image
    read_scales();
    for (int t0 = 0; t0 < T;) {   // items; t0: the item's first tile among the CTA's
      const int tiles = cur.tiles;
      // Rows past the item's last (of a sequence, or of a chunk) get P = 0.  What they hold
      // is finite whatever their bytes are, but for the keys, whose scores are not looked at.
      const int end = kShare ? cur.len : row_end;
      const int last_valid = min(end - (cur.r0 + (tiles - 1) * kRowsT), kRowsT);
      float m[kHalf], l[kHalf];
      float ref = kNoRef, drop = 0.f;   // lane h: m[h], and how far it lies below the highest it was
      int due = t0 + kBearsTiles;       // the next look
#pragma unroll
      for (int h = 0; h < kHalf; ++h) {
        m[h] = kNoRef;
        l[h] = 0.f;
      }
      for (int t = t0; t < t0 + tiles; ++t) {
        const int sb = t & 1;
        const int valid = t == t0 + tiles - 1 ? last_valid : kRowsT;
        q4_warp_wait(bar(L::SFULL + sb), (t >> 1) & 1, abort_flag);
        tc_fence_after();
        float x[kHalf];   // scores in units of the head's scale
        {
          uint32_t s[L::kQParts][8], sk[L::kKParts][8];
#pragma unroll
          for (int i = 0; i < L::kQParts; ++i)
            tmem_ld8_nowait(tmem + lane_base + 64 * sb + kHeadGroup * i + hb, s[i]);
#pragma unroll
          for (int i = 0; i < L::kKParts; ++i)
            tmem_ld8_nowait(tmem + lane_base + kKCol + 32 * sb + kHeadGroup * i + hb, sk[i]);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < kHalf; ++h) {
            x[h] = __uint_as_float(s[L::kQParts - 1][h]);
#pragma unroll
            for (int i = L::kQParts - 2; i >= 0; --i)
              x[h] = fmaf(x[h], 0.0625f, __uint_as_float(s[i][h]));
#pragma unroll
            for (int i = 0; i < L::kKParts; ++i) x[h] += __uint_as_float(sk[i][h]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::SFREE + sb));
        float d[kHalf];   // and above the head's reference
        auto above = [&] {
#pragma unroll
          for (int h = 0; h < kHalf; ++h) d[h] = fmaf(x[h], qsig[h], -m[h]);
          if (row >= valid)
#pragma unroll
            for (int h = 0; h < kHalf; ++h) d[h] = -INFINITY;
        };
        above();
        bool need = t == due;
#pragma unroll
        for (int h = 0; h < kHalf; ++h) need |= d[h] > L::kTop;
        if (any_of(need, 1 + gp, kSoft / 2)) {
          // Some score is too far above its head's reference, or a look at the sums is due: the
          // tile's maxima (of a warp, then of the group's four) move the references of this
          // group's heads, lane h (and h + 8 ..) head h's; rescale its row sums and the O^T columns
          // it owns (in TMEM, after the previous PV finished).
          float alpha[kHalf];
#pragma unroll
          for (int h = 0; h < kHalf; ++h) alpha[h] = row < valid ? x[h] * qsig[h] : -INFINITY;
          float top = over_lanes(alpha, lane, [](float a, float b) { return fmaxf(a, b); });
          const int mine = hb + (lane & (kHalf - 1));
          if (lane < kHalf) red[mine * 4 + wq] = top;
          if (t == due) {
            const float sum = over_lanes(l, lane, [](float a, float b) { return a + b; });
            if (lane < kHalf) lsum[mine * 4 + wq] = sum;
          }
          named_bar_sync(3 + gp, kSoft / 2);
          const float4 t4 = *reinterpret_cast<const float4*>(red + mine * 4);
          top = fmaxf(fmaxf(t4.x, t4.y), fmaxf(t4.z, t4.w)) - L::kBias;
          float mn = fmaxf(top, ref), sum = 0.f;
          if (t == due) {
            const float4 s4 = *reinterpret_cast<const float4*>(lsum + mine * 4);
            sum = (s4.x + s4.y) + (s4.z + s4.w);
            mn = fmaxf(top, q4_floor(sum, t - t0, ref, drop));
          }
          const float al = ex2(ref - mn);
          drop = fmaxf(drop + (ref - mn), 0.f);
          ref = mn;
          due = t == due ? t + __reduce_min_sync(0xffffffffu, q4_bears(sum * al, t - t0, drop))
                         : min(due, t + kBearsTiles);
          const bool moved = __any_sync(0xffffffffu, al != 1.f);
#pragma unroll
          for (int h = 0; h < kHalf; ++h) {
            m[h] = __shfl_sync(0xffffffffu, ref, h);
            alpha[h] = __shfl_sync(0xffffffffu, al, h);
            l[h] *= alpha[h];
          }
          if (t > t0 && moved) {
            q4_warp_wait(bar(L::ODONE + ((t - 1) & 1)), ((t - 1) >> 1) & 1, abort_flag);
            tc_fence_after();
#pragma unroll
            for (int mb = 0; mb < 4; ++mb) {
#pragma unroll
              for (int part = 0; part < L::kPParts; ++part) {
                const uint32_t col = kOCol + L::kPN * mb + kHeadGroup * part + hb;
                uint32_t r[8];
                float o[8];
                tmem_ld8_nowait(tmem + lane_base + col, r);
                tmem_wait_ld();
#pragma unroll
                for (int h = 0; h < kHalf; ++h) o[h] = __uint_as_float(r[h]) * alpha[h];
                tmem_st8(tmem + lane_base + col, o);
              }
            }
            tmem_wait_st();
          }
          above();
        }
        // p as E4M3 parts, two heads per conversion.  Of three parts the row sum takes the
        // value that the PV uses.
        uint16_t pp[L::kPParts][kHalf / 2];
#pragma unroll
        for (int h2 = 0; h2 < kHalf / 2; ++h2) {
          float v0 = ex2(d[2 * h2]), v1 = ex2(d[2 * h2 + 1]);
          if constexpr (!kF32) {
            l[2 * h2] += v0;
            l[2 * h2 + 1] += v1;
            // By way of fp16 (2^-11 relative, a quarter of what two parts keep): two values
            // an instruction, and the remainder of a rounding is exact there.
            const __half2 v = __floats2half2_rn(v0, v1);
            pp[0][h2] = __nv_cvt_halfraw2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
            const __half2 f = __half2(__nv_cvt_fp8x2_to_halfraw2(pp[0][h2], __NV_E4M3));
            const __half2 r = __hfma2(f, __float2half2_rn(-16.f), __hmul2(v, __float2half2_rn(16.f)));
            pp[1][h2] = __nv_cvt_halfraw2_to_fp8x2(r, __NV_SATFINITE, __NV_E4M3);
          } else {
            float wgt = 1.f;
#pragma unroll
            for (int part = 0; part < L::kPParts; ++part) {
              pp[part][h2] = to_e4m3x2(v0, v1);
              const float2 f = from_e4m3x2(pp[part][h2]);
              l[2 * h2] = fmaf(f.x, wgt, l[2 * h2]);
              l[2 * h2 + 1] = fmaf(f.y, wgt, l[2 * h2 + 1]);
              v0 = (v0 - f.x) * 16.f;
              v1 = (v1 - f.y) * 16.f;
              wgt *= 0.0625f;
            }
          }
        }
        // P^T buffer sb was last read by the PV of tile t-2.
        if (t >= 2) q4_warp_wait(bar(L::ODONE + sb), ((t - 2) >> 1) & 1, abort_flag);
        {
          // P^T (B operand of the PV MMA, K-major, 128-byte swizzle): row
          // 16 part + n is part `part` of head n; the K index is the tile row.  Four
          // heads of four rows are turned over among four lanes, to four rows of a head
          // a word.  (Stored byte by byte: 64 sequences of 512 to 8192 rows 41.3 us, 256
          // of 2048 73.5; 40.0 and 68.5 so.)
          uint8_t* pbuf = smem + L::kOffP + sb * L::kPBuf;
          const uint32_t s1 = lane & 1 ? 0x3715u : 0x6240u, s2 = lane & 2 ? 0x3276u : 0x5410u;
#pragma unroll
          for (int part = 0; part < L::kPParts; ++part)
#pragma unroll
            for (int h4 = 0; h4 < kHalf / 4; ++h4) {
              uint32_t w = pp[part][2 * h4] | static_cast<uint32_t>(pp[part][2 * h4 + 1]) << 16;
              w = __byte_perm(w, __shfl_xor_sync(0xffffffffu, w, 1), s1);
              w = __byte_perm(w, __shfl_xor_sync(0xffffffffu, w, 2), s2);
              *reinterpret_cast<uint32_t*>(
                  pbuf + sw128_byte(kHeadGroup * part + hb + 4 * h4 + (lane & 3), row & ~3)) = w;
            }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::PFULL + sb));
      }
      t0 += tiles;
      // The combine may start launching: it waits for this grid anyway.
      if (tid == 0 && t0 == T) pdl_launch_dependents();
      // Softmax denominators over the chunk's rows.
      {
        const float sum = over_lanes(l, lane, [](float a, float b) { return a + b; });
        if (lane < kHalf) lsum[(hb + lane) * 4 + wq] = sum;
      }
      const TileItem out = cur;
      if (kShare && t0 < T) {   // fetched while the last PV runs
        cur = item_after(cur, t0);
        read_scales();
      }
      // O^T after the last PV: this thread's latent row is 128 mb + 32 wq + lane.
      q4_warp_wait(bar(L::ODONE + ((t0 - 1) & 1)), ((t0 - 1) >> 1) & 1, abort_flag);
      tc_fence_after();
      // (asked for all of the group: the flag may be raised at any time)
      if (!any_of(*abort_flag, 3 + gp, kSoft / 2)) {
        const size_t base = (size_t(out.v) * p.H + h0) * p.splits + out.j;
        // 1/L by the approximate reciprocal (within 2 ulp for the L > 0 reached
        // here, at most 2^(kTop + kSpan) x rows), branch-free; lane h of the first warp of
        // each group writes head h's log-sum-exp.
        float inv[kHalf], Lme = 0.f, mme = 0.f;
#pragma unroll
        for (int h = 0; h < kHalf; ++h) {
          const float4 q4 = *reinterpret_cast<const float4*>(lsum + (hb + h) * 4);
          const float L_ = (q4.x + q4.y) + (q4.z + q4.w);
          inv[h] = L_ > 0.f ? __fdividef(1.f, L_) : 0.f;
          Lme = lane == h ? L_ : Lme;
          mme = lane == h ? m[h] : mme;
        }
        if (wq == 0 && lane < kHalf && p.part_lse)
          p.part_lse[base + size_t(hb + lane) * p.splits] =
              Lme > 0.f ? (mme + log2f(Lme)) * kLn2 : -INFINITY;
        float* row0 = p.part_o + (base + size_t(hb) * p.splits) * kDc + 32 * wq + lane;
        const size_t head_stride = size_t(p.splits) * kDc;
#pragma unroll
        for (int mb = 0; mb < 4; ++mb) {
          uint32_t o[L::kPParts][8];
#pragma unroll
          for (int i = 0; i < L::kPParts; ++i)
            tmem_ld8_nowait(tmem + lane_base + kOCol + L::kPN * mb + kHeadGroup * i + hb, o[i]);
          tmem_wait_ld();
          float* at = row0 + 128 * mb;
#pragma unroll
          for (int h = 0; h < kHalf; ++h, at += head_stride) {
            float v = __uint_as_float(o[L::kPParts - 1][h]);
#pragma unroll
            for (int i = L::kPParts - 2; i >= 0; --i) v = fmaf(v, 0.0625f, __uint_as_float(o[i][h]));
            v *= inv[h];
            if (p.direct && p.io_bf16)
              reinterpret_cast<__nv_bfloat16*>(p.part_o)[at - p.part_o] = __float2bfloat16_rn(v);
            else
              *at = v;
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0 && *abort_flag) report(p.status, MLA_DEV_PIPELINE_TIMEOUT);
}

template <bool kF32, bool kShare>
mla_status launch_q4(const SplitParams& p, cudaStream_t stream, const char* who) {
  using L = Q4Plan<kF32>;
  static DeviceFlags attr_done;
  const int dev = current_device();
  if (!attr_done.test(dev)) {
    if (cudaFuncSetAttribute(split_q4_kernel<kF32, kShare>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, int(L::kSmem)) != cudaSuccess) {
      cudaGetLastError();
      set_error("%s: cannot reserve %zu bytes of shared memory", who, L::kSmem);
      return MLA_ERR_CUDA;
    }
    attr_done.set(dev);
  }
  const int groups = p.H / kHeadGroup;
  const dim3 grid = kShare ? dim3(share_runs(groups) * groups) : dim3(groups, p.splits, p.B);
  launch_pdl(split_q4_kernel<kF32, kShare>, grid, dim3(kThreads), L::kSmem, stream, p);
  return launch_status(who);
}

}  // namespace

mla_status launch_q4_queries(const SplitParams& p, cudaStream_t stream, const char* who) {
  launch_pdl(p.io_bf16 ? q4_query_kernel<false> : q4_query_kernel<true>, dim3(p.H, p.B), dim3(160),
             0, stream, p);
  return launch_status(who);
}

mla_status launch_split_q4(const SplitParams& p, cudaStream_t stream, const char* who) {
  if (!p.late) {
    const mla_status st = launch_q4_queries(p, stream, who);
    if (st != MLA_OK) return st;
  }
  if (p.pieces)
    return p.io_bf16 ? launch_q4<false, true>(p, stream, who) : launch_q4<true, true>(p, stream, who);
  return p.io_bf16 ? launch_q4<false, false>(p, stream, who) : launch_q4<true, false>(p, stream, who);
}

}  // namespace mla
