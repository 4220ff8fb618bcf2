// moe_attn_prefill: attention over packed prompts.
//
// One warp per (query row, head): the row's key-value head's keys one after the other, each lane
// holding d / 32 of the products, with the running maximum and sum of a softmax.
#include "attn_device.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <int D>
__global__ void __launch_bounds__(32 * kWarps) attn_prefill_kernel(AttnPrefillParams p) {
  constexpr int W = D / 64;  // words of two values per lane
  const int lane = threadIdx.x & 31, t = blockIdx.x, h = blockIdx.y * kWarps + threadIdx.x / 32;
  if (h >= p.hq) return;
  if (t == 0 && h == 0) {
    check_offsets(p.cu_q, p.n_seqs, p.total_q, p.hdr, lane, 32);
    check_offsets(p.cu_k, p.n_seqs, p.total_k, p.hdr, lane, 32);
  }
  int lo = 0, hi = p.n_seqs;
  while (hi - lo > 1) {  // the last sequence that begins at or before t
    const int mid = (lo + hi) / 2;
    if (p.cu_q[mid] <= t) lo = mid; else hi = mid;
  }
  const int q0 = p.cu_q[lo], q1 = min(p.cu_q[lo + 1], p.total_q);
  const int k0 = max(p.cu_k[lo], 0), k1 = min(p.cu_k[lo + 1], p.total_k);
  if (q0 > t || q1 <= t || q0 < 0 || k1 < k0) {
    if (lane == 0) raise_bad_index(p.hdr);
    return;
  }
  int n = k1 - k0;
  if (p.causal) n = min(n, max(0, t - q0 + 1 + (k1 - k0) - (q1 - q0)));
  const int kvh = h / p.group;
  float q[2 * W], acc[2 * W], m = -INFINITY, l = 0.f;
  const uint32_t* qp = reinterpret_cast<const uint32_t*>(p.q.p + t * p.q.token_stride + h * p.q.head_stride);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    q[2 * i] = bf16_lo(qp[lane + 32 * i]) * p.scale;
    q[2 * i + 1] = bf16_hi(qp[lane + 32 * i]) * p.scale;
    acc[2 * i] = acc[2 * i + 1] = 0.f;
  }
  for (int j = 0; j < n; ++j) {
    const int64_t r = k0 + j;
    const uint32_t* kp = reinterpret_cast<const uint32_t*>(p.k.p + r * p.k.token_stride + kvh * p.k.head_stride);
    const uint32_t* vp = reinterpret_cast<const uint32_t*>(p.v.p + r * p.v.token_stride + kvh * p.v.head_stride);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      s = fmaf(q[2 * i], bf16_lo(kp[lane + 32 * i]), s);
      s = fmaf(q[2 * i + 1], bf16_hi(kp[lane + 32 * i]), s);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
    const float m2 = fmaxf(m, s), base = m2 == -INFINITY ? 0.f : m2;
    const float a = expf(m - base), e = expf(s - base);
    m = m2;
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      acc[2 * i] = fmaf(acc[2 * i], a, e * bf16_lo(vp[lane + 32 * i]));
      acc[2 * i + 1] = fmaf(acc[2 * i + 1], a, e * bf16_hi(vp[lane + 32 * i]));
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t* op = reinterpret_cast<uint32_t*>(p.o + ((int64_t)t * p.hq + h) * D);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(l == 0.f ? 0.f : acc[2 * i + 1] * inv),
        "f"(l == 0.f ? 0.f : acc[2 * i] * inv));
    op[lane + 32 * i] = w;
  }
  if (p.lse && lane == 0) p.lse[(int64_t)t * p.hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnPrefillParams& p, int d, cudaStream_t s) {
  const dim3 grid(p.total_q, (p.hq + kWarps - 1) / kWarps);
  if (d == 64) attn_prefill_kernel<64><<<grid, 32 * kWarps, 0, s>>>(p);
  if (d == 128) attn_prefill_kernel<128><<<grid, 32 * kWarps, 0, s>>>(p);
  if (d == 256) attn_prefill_kernel<256><<<grid, 32 * kWarps, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace moe
