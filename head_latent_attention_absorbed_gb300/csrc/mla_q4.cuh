// The 4-bit latent cache (MLA_FP4_E2M1): how a page holds its rows, and one lane's share
// of a row in and out of that form.
//
// A row's 512 latents are E2M1 codes (sign, two exponent bits, one mantissa bit: 0, 1/2, 1,
// 3/2, 2, 3, 4, 6) times a power of two 2^e per 16 of them, -8 <= e <= 6; its 64 rotated key
// values are bf16.  The range of e is chosen so that every latent value is an E4M3 number
// (6 2^6 = 384, 2^-1 2^-8 = 2^-9, E4M3's smallest): the tensor cores' 8-bit products take a
// row without another rounding.  e is the smallest with which the block's largest magnitude
// is at most 7 2^e: what lies above 6 2^e is off by no more than 2^e, as between 4 and 6.
// (Root-mean-square error of N(0, 1) values 0.110 of their size; 0.113 with 6 2^e as the
// limit, 0.118 with 8 2^e; 0.112 with one e per 32.)
//
// A page of R rows is two planes, 400 R bytes in all, so that the rows of a tile are two
// contiguous copies:
//   latents [R][272]  256 bytes of codes, a 32-bit word for eight values: the magnitude of
//                     value k in bits 4 k .. 4 k + 2, the signs of values 0-3 in bits 7, 15,
//                     23, 31 and of 4-7 in bits 3, 11, 19, 27 (where a reader wants them);
//                     then 16 of exponents, byte i: (e + 5) mod 16 of blocks 2 i (low four
//                     bits) and 2 i + 1, so that the exponents with which every magnitude is a
//                     normal E4M3 number (-5 .. 6) are the bits 0 .. 11
//   keys    [R][128]  16-byte piece c of row r stands at piece c ^ (r & 7): as the tensor core
//                     wants it in shared memory (128-byte swizzle)
#pragma once

#include <cuda_fp4.h>

#include "mla_paged.cuh"
#include "mla_split.cuh"

namespace mla {

constexpr int kQ4Block = 16;                       // values that share an exponent
constexpr int kQ4CodeBytes = kDc / 2;              // 256
constexpr int kQ4KeyBytes = 2 * kDr;               // 128
constexpr int kQ4ExpBytes = kDc / kQ4Block / 2;    // 16
constexpr int kQ4LatBytes = kQ4CodeBytes + kQ4ExpBytes;                 // 272
constexpr int kQ4RowBytes = kQ4LatBytes + kQ4KeyBytes;                  // 400
constexpr int kQ4ExpMin = -8, kQ4ExpMax = 6;

// The planes of page `id` of a pool (const or not).
template <typename Byte>
struct Q4Page {
  Byte *latents, *keys;
  __device__ __forceinline__ Q4Page(Byte* pool, int id, int page_shift) {
    latents = pool + (static_cast<size_t>(id) << page_shift) * kQ4RowBytes;
    keys = latents + (static_cast<size_t>(kQ4LatBytes) << page_shift);
  }
  __device__ __forceinline__ Byte* codes(int r) const { return latents + r * kQ4LatBytes; }
  __device__ __forceinline__ Byte* exps(int r) const { return codes(r) + kQ4CodeBytes; }
};

// Byte offset of key pair `pair` of row r in the keys' plane.
__device__ __forceinline__ uint32_t q4_key_at(int r, int pair) {
  return static_cast<uint32_t>(r * kQ4KeyBytes + ((((pair >> 2) ^ r) & 7) << 4) + ((pair & 3) << 2));
}

// 2^e for an exponent's four bits (12 is never written; it reads as 11, e = 6, does).
__device__ __forceinline__ float q4_unit(uint32_t bits) {
  return __uint_as_float((min((bits + 3u) & 15u, 14u) + static_cast<uint32_t>(127 + kQ4ExpMin)) << 23);
}

// Eight codes, value k in bits 4 k .. 4 k + 3, as a page holds them, and back.
__device__ __forceinline__ uint32_t q4_page_word(uint32_t w) {
  const uint32_t odd = w << 4;
  return (w & 0x77777777u) | (__byte_perm(odd, w, 0x5140) & 0x80808080u) |
         (__byte_perm(odd, w, 0x7362) & 0x80808080u) >> 4;
}
__device__ __forceinline__ uint32_t q4_codes(uint32_t w) {
  const uint32_t low = w & 0x80808080u, high = (w << 4) & 0x80808080u;
  return (w & 0x77777777u) | __byte_perm(low, high, 0x6420) >> 4 | __byte_perm(low, high, 0x7531);
}

// Eight codes as loaded, to values in units of 2^e.
__device__ __forceinline__ void q4_values(uint32_t word, float unit, float* v) {
  const uint32_t codes = q4_codes(word);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(
        static_cast<__nv_fp4x2_storage_t>(codes >> (8 * i)), __NV_E2M1);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x * unit;
    v[2 * i + 1] = f.y * unit;
  }
}

// A lane's values of one row (8 l .., 256 + 8 l .. and the key pair l) as loaded.
struct Q4Lane {
  uint32_t code[2], key;
  uint8_t exp[2];
  __device__ __forceinline__ void load(const Q4Page<const uint8_t>& page, int r, int lane) {
    const uint32_t* c = reinterpret_cast<const uint32_t*>(page.codes(r));
    code[0] = c[lane];
    code[1] = c[32 + lane];
    exp[0] = page.exps(r)[lane >> 2];
    exp[1] = page.exps(r)[8 + (lane >> 2)];
    key = *reinterpret_cast<const uint32_t*>(page.keys + q4_key_at(r, lane));
  }
  __device__ __forceinline__ void zero() {
    code[0] = code[1] = key = 0;
    exp[0] = exp[1] = 0;
  }
  // Latents 8 l .. (i = 0) or 256 + 8 l .. (i = 1), times a power of two.
  __device__ __forceinline__ void values(int i, int lane, float* v, float times = 1.f) const {
    q4_values(code[i], q4_unit(exp[i] >> (lane & 2 ? 4 : 0)) * times, v);
  }
  // The power of two above their magnitudes, of 2^high; -100: they are all zero.
  __device__ __forceinline__ int high(int i, int lane) const {
    const uint32_t w = code[i];
    const int e = min(((exp[i] >> (lane & 2 ? 4 : 0)) + 3) & 15, 14) + kQ4ExpMin;   // as q4_unit
    return (w & (w << 1) & 0x44444444u) ? e + 3   // 4 and 6
           : (w & 0x44444444u)          ? e + 2   // 2 and 3
           : (w & 0x22222222u)          ? e + 1   // 1 and 1.5
           : (w & 0x11111111u)          ? e       // 0.5
                                        : -100;
  }
  __device__ __forceinline__ float2 pair() const {
    return make_float2(__uint_as_float(key << 16), __uint_as_float(key & 0xffff0000u));
  }
};

// Waits for a phase, bounded: gives up, raising the CTA's abort flag, after as many ns as the word
// behind the flag says, which is then none for the CTA's other waits.  The warp is suspended for up
// to kSuspendNs at a time: so many warps of these kernels wait that their polling would take issue
// slots from the others.  Out of line, since 20 to 32 warps share the instruction cache and a tile
// meets some 25 waits: 32 x 16384 rows x 128 heads, the same rows each time, 119 us for 125 with each
// wait's loop in place, fp32 queries of 64 x 4096 rows 51.7 for 52.3 (bf16 67.9 for 67.4 of 256 x 2048
// rows).
constexpr uint32_t kSuspendNs = 20000;
// Before any wait, by one thread, the CTA's barrier between them.
__device__ __forceinline__ void q4_wait_init(const SplitParams& p, volatile int* abort) {
  abort[0] = 0;
  abort[1] = static_cast<int>(static_cast<uint32_t>(min(p.wait_ns ? p.wait_ns : kWaitNs, 4000000000ull)));
}
static __device__ __noinline__ void q4_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  const uint32_t t0 = static_cast<uint32_t>(globaltimer_ns());
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kSuspendNs)
        : "memory");
    if (ok) return;
    if (static_cast<uint32_t>(globaltimer_ns()) - t0 > static_cast<uint32_t>(abort[1])) {
      abort[1] = 0;
      *abort = 1;
      return;
    }
  }
}
// By a whole warp, which leaves it converged (as the .aligned tensor-core instructions after it
// need).
__device__ __forceinline__ void q4_warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (!mbar_try_wait(bar, parity)) q4_wait(bar, parity, abort);
  __syncwarp();
}

// ------------------------------------------------------------- codes to E4M3
__device__ __forceinline__ uint16_t to_e4m3x2(float x0, float x1) {
  return static_cast<uint16_t>(
      __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3));
}
// Eight codes as E4M3 bytes; mag: the E4M3 magnitudes of codes 0-3 and 4-7.
__device__ __forceinline__ uint2 decode8(uint32_t w, uint2 mag) {
  const uint32_t sel = w & 0x77777777u;
  return make_uint2(__byte_perm(mag.x, mag.y, sel) | (w & 0x80808080u),
                    __byte_perm(mag.x, mag.y, sel >> 16) | ((w << 4) & 0x80808080u));
}
// Table of magnitudes by exponent bits, for q4_decode (16 entries of 8 bytes, by 16 lanes):
// 0, 1/2, 1, 3/2, 2, 3, 4, 6 times 2^e as E4M3.
__device__ __forceinline__ void q4_table(uint8_t* table, int lane) {
  const float u = q4_unit(lane);
  reinterpret_cast<uint2*>(table)[lane] =
      make_uint2(to_e4m3x2(0.f, 0.5f * u) | to_e4m3x2(u, 1.5f * u) << 16,
                 to_e4m3x2(2.f * u, 3.f * u) | to_e4m3x2(4.f * u, 6.f * u) << 16);
}

// Up to the bits 11 every magnitude is a normal E4M3 number, whose exponent field grows with
// the bits; others are looked up.  true: all of e's eight (zeros are) are such.
__device__ __forceinline__ bool q4_plain(uint32_t e) { return (e & (e << 1) & 0x88888888u) == 0; }

// 32 codes of one row and their two blocks' exponents, as loaded, and as E4M3 in the row's
// 16-byte units at `at` and at ^ 16 of a box of 128-byte rows (the caller has the 128-byte
// swizzle in `at`).
struct Q4Piece {
  uint4 w;
  uint32_t e;   // in the low byte
  __device__ __forceinline__ void load(const uint8_t* codes, uint32_t exps) {
    w = *reinterpret_cast<const uint4*>(codes);
    e = exps;
  }
  template <bool kPlain>
  __device__ __forceinline__ void decode(uint4& lo, uint4& hi, const uint8_t* table) const {
    auto magnitudes = [&](uint32_t x) {
      return kPlain ? make_uint2(x * 0x08080800u + 0x14100800u, x * 0x08080808u + 0x24201c18u)
                    : *reinterpret_cast<const uint2*>(table + 8 * x);
    };
    const uint2 m0 = magnitudes(e & 15), m1 = magnitudes(e >> 4 & 15);
    const uint2 a = decode8(w.x, m0), b = decode8(w.y, m0);
    lo = make_uint4(a.x, a.y, b.x, b.y);
    const uint2 x = decode8(w.z, m1), y = decode8(w.w, m1);
    hi = make_uint4(x.x, x.y, y.x, y.y);
  }
  template <bool kPlain>
  __device__ __forceinline__ void store(uint8_t* row, uint32_t at, const uint8_t* table) const {
    uint4 lo, hi;
    decode<kPlain>(lo, hi, table);
    *reinterpret_cast<uint4*>(row + at) = lo;
    *reinterpret_cast<uint4*>(row + (at ^ 16)) = hi;
  }
};

// ------------------------------------------------------------- softmax references
// A head's weights are 2^(score - reference) and enter the output product as parts of eight bits,
// which hold a weight to a share of it but for their smallest step: a tile's 128 rows may lose up
// to d = 2^-7 together (two parts; three 2^-11).  With a reference that only rises with the maximum
// the many rows that one far above them outweighs are lost so, however much they weigh together.
// So it also goes down: a look at the sum of a head's weights, tiles apart, finds whether the sum is
// below four for each tile so far, and then lowers the reference to where the tile at hand has its
// largest weight.  How many tiles the sum bears until the next look follows from the sum; a move to
// a tile's maximum, which adds 2^4 or more, bears kBearsTiles.  So each d comes with 1 to 4 of the
// sum, or with octaves that a move adds to it: over 512 tiles some two d of the sum are lost at
// most.  Looks are few, and so are moves, by which O is rescaled: 32 x 16384 rows x 128 heads whose
// scores spread by 1 nat 118 us, by 2, 3 and 5 131, 145 and 156 (with references that only rise 128, 134 and 143; with the weights
// of every tile looked at 159, 180 and 181).
constexpr float kNoRef = -3e38f;   // before a head's first score: below any, but finite, so that
                                   // scores of -infinity have no weight there either
constexpr float kSpan = 40.f;      // how far below the highest it was a reference may go: the rows
                                   // of a tile that lies further down count for nothing
constexpr float kPerTile = 4.f;
constexpr int kBearsTiles = 16;
// How low a look lets the reference go; drop: how far it lies below the highest it was, sum: of the
// weights of the `done` tiles before.
__device__ __forceinline__ float q4_floor(float sum, int done, float ref, float drop) {
  return sum < kPerTile * static_cast<float>(done + kBearsTiles) ? ref + (drop - kSpan) : ref;
}
// Tiles until the next look.
__device__ __forceinline__ int q4_bears(float sum, int done, float drop) {
  if (drop >= kSpan - 1.f) return 1 << 20;
  return max(static_cast<int>(fminf(sum * (1.f / kPerTile), 1e6f)) - done, kBearsTiles);
}

__device__ __forceinline__ void bulk_g2s_elected(uint32_t dst, const void* src, uint32_t bytes,
                                                 uint32_t bar, uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1], %2, [%3], %4;\n\t}" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}


// The split over a 4-bit pool (mla_q4attn.cu), and the kernel that makes the queries' images,
// which it runs first unless p.late is set.
mla_status launch_split_q4(const SplitParams& p, cudaStream_t stream, const char* who);
mla_status launch_q4_queries(const SplitParams& p, cudaStream_t stream, const char* who);
// The same for bf16 queries of many heads as SM pairs (mla_q4pair.cu), with the query codes of
// an E4M3 cache's pairs (launch_pair_queries).
mla_status launch_split_q4_pair(const SplitParams& p, cudaStream_t stream, const char* who);

}  // namespace mla
