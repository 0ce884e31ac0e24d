// The split kernel over a 4-bit pool.
#include "mla_q4.cuh"

namespace mla {
namespace {

// One CTA per (head, chunk, sequence), eight warps, a row per warp at a time: the form of
// split_f32_paged_kernel with a lane's values of a row as Q4Lane holds them.
constexpr int kWarps = 8;

__global__ void __launch_bounds__(32 * kWarps) split_q4_kernel(const SplitParams p) {
  __shared__ float wm[kWarps], wl[kWarps], wo[kWarps][kDc];
  const int h = blockIdx.x, j = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (p.late) pdl_wait();
  const int len = clamp_length(p, b, tid == 0 && h == 0 && j == 0);
  const int r0 = j * p.chunk;
  pdl_wait();   // the queries, and the readers of the workspace and of o_c
  if (r0 >= len) {
    if (p.direct) write_no_rows(p, size_t(b) * p.H + h, 1, tid, 32 * kWarps);
    return;
  }
  const int r1 = min(r0 + p.chunk, len);
  const size_t bh = size_t(b) * p.H + h;
  float q[16];
  float2 qk;
  if (p.io_bf16) {
    const __nv_bfloat16* qa = static_cast<const __nv_bfloat16*>(p.q_abs) + bh * kDc;
    for (int i = 0; i < 2; ++i)
      for (int k = 0; k < 8; ++k) q[8 * i + k] = __bfloat162float(qa[256 * i + 8 * lane + k]);
    qk = load_pair(static_cast<const __nv_bfloat16*>(p.q_pe) + bh * kDr + 2 * lane);
  } else {
    const float* qa = static_cast<const float*>(p.q_abs) + bh * kDc;
    for (int i = 0; i < 2; ++i)
      for (int k = 0; k < 8; ++k) q[8 * i + k] = qa[256 * i + 8 * lane + k];
    qk = load_pair(static_cast<const float*>(p.q_pe) + bh * kDr + 2 * lane);
  }
  const int seq = cache_seq(p, b), mask = (1 << p.page_shift) - 1;
  float m = -INFINITY, l = 0.f, acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int t = r0 + warp; t < r1; t += kWarps) {
    const int id = page_of(p, seq, t);   // rows of a page that does not exist read as zeros
    Q4Lane x;
    if (id >= 0)
      x.load(Q4Page<const uint8_t>(static_cast<const uint8_t*>(p.cache), id, p.page_shift), t & mask, lane);
    else
      x.zero();
    float c[16];
    x.values(0, lane, c);
    x.values(1, lane, c + 8);
    const float2 ck = x.pair();
    float s = fmaf(qk.y, ck.y, qk.x * ck.x);
#pragma unroll
    for (int i = 0; i < 16; ++i) s = fmaf(q[i], c[i], s);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s), alpha = exp2f(m - mn), w = exp2f(s - mn);
    l = l * alpha + w;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = fmaf(w, c[i], acc[i] * alpha);
    m = mn;
  }
  if (lane == 0) {
    wm[warp] = m;
    wl[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) wo[warp][256 * (i >> 3) + 8 * lane + (i & 7)] = acc[i];
  __syncthreads();
  float M = -INFINITY, L = 0.f, f[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w]);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    f[w] = wm[w] == -INFINITY ? 0.f : exp2f(wm[w] - M);
    L += f[w] * wl[w];
  }
  const size_t base = bh * p.splits + j;
  for (int c = tid; c < kDc; c += 32 * kWarps) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v = fmaf(f[w], wo[w][c], v);
    if (p.direct && p.io_bf16)
      reinterpret_cast<__nv_bfloat16*>(p.part_o)[base * kDc + c] = __float2bfloat16_rn(v / L);
    else
      p.part_o[base * kDc + c] = v / L;
  }
  if (tid == 0 && p.part_lse) p.part_lse[base] = (M + log2f(L)) * kLn2;
}

}  // namespace

mla_status launch_split_q4(const SplitParams& p, const void* cache, cudaStream_t stream,
                           const char* who) {
  launch_pdl(split_q4_kernel, dim3(p.H, p.splits, p.B), dim3(32 * kWarps), 0, stream, p);
  return launch_status(who);
}

}  // namespace mla
