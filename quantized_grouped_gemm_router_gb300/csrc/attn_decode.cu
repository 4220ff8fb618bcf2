// moe_attn_decode: attention of one new token per sequence over the paged cache.
//
// One warp per (sequence, query head) over the whole cache of the sequence, each lane holding
// d / 32 of the products, with the running maximum and sum of a softmax.
#include <cuda_fp8.h>

#include "attn_device.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float2 bf16x2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 e4m3x2(uint16_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(w, __NV_E4M3);
  return __half22float2(__half2(h));
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * kWarps) attn_decode_kernel(AttnDecodeParams p) {
  constexpr int W = D / 64;
  const int lane = threadIdx.x & 31, b = blockIdx.x, h = blockIdx.y * kWarps + threadIdx.x / 32;
  if (h >= p.hq) return;
  const int64_t room = (int64_t)p.table_width * p.page_size;
  int n = p.lens[b];
  bool bad = n < 0 || n > room;
  n = bad ? 0 : n;
  const int kvh = h / p.group;
  const float ks = E4M3 ? p.k_scale[kvh] * p.scale : p.scale, vs = E4M3 ? p.v_scale[kvh] : 1.f;
  float q[2 * W], acc[2 * W], m = -INFINITY, l = 0.f;
  const uint32_t* qp = reinterpret_cast<const uint32_t*>(p.q.p + b * p.q.token_stride + h * p.q.head_stride);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float2 x = bf16x2(qp[lane + 32 * i]);
    q[2 * i] = x.x * ks;
    q[2 * i + 1] = x.y * ks;
    acc[2 * i] = acc[2 * i + 1] = 0.f;
  }
  for (int j = 0; j < n; ++j) {
    const int page = p.table[(int64_t)b * p.table_width + j / p.page_size];
    if (page < 0 || page >= p.n_pages) {
      bad = true;
      continue;
    }
    const int64_t at = (((int64_t)page * p.hkv + kvh) * p.page_size + j % p.page_size) * (D / 2) + lane;
    float2 kx[W], vx[W];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      kx[i] = E4M3 ? e4m3x2(static_cast<const uint16_t*>(p.kc)[at + 32 * i])
                   : bf16x2(static_cast<const uint32_t*>(p.kc)[at + 32 * i]);
      vx[i] = E4M3 ? e4m3x2(static_cast<const uint16_t*>(p.vc)[at + 32 * i])
                   : bf16x2(static_cast<const uint32_t*>(p.vc)[at + 32 * i]);
      s = fmaf(q[2 * i], kx[i].x, s);
      s = fmaf(q[2 * i + 1], kx[i].y, s);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(~0u, s, x);
    const float m2 = fmaxf(m, s), base = m2 == -INFINITY ? 0.f : m2;
    const float a = expf(m - base), e = expf(s - base);
    m = m2;
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      acc[2 * i] = fmaf(acc[2 * i], a, e * vx[i].x);
      acc[2 * i + 1] = fmaf(acc[2 * i + 1], a, e * vx[i].y);
    }
  }
  if (bad && lane == 0) raise_bad_index(p.hdr);
  const float inv = l == 0.f ? 0.f : vs / l;
  uint32_t* op = reinterpret_cast<uint32_t*>(p.o + ((int64_t)b * p.hq + h) * D);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(l == 0.f ? 0.f : acc[2 * i + 1] * inv),
        "f"(l == 0.f ? 0.f : acc[2 * i] * inv));
    op[lane + 32 * i] = w;
  }
  if (p.lse && lane == 0) p.lse[(int64_t)b * p.hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

template <int D>
void launch(const AttnDecodeParams& p, bool e4m3, cudaStream_t s) {
  const dim3 grid(p.n_seqs, (p.hq + kWarps - 1) / kWarps);
  if (e4m3)
    attn_decode_kernel<D, true><<<grid, 32 * kWarps, 0, s>>>(p);
  else
    attn_decode_kernel<D, false><<<grid, 32 * kWarps, 0, s>>>(p);
}

}  // namespace

cudaError_t launch_attn_decode(const AttnDecodeParams& p, int d, bool e4m3, cudaStream_t s) {
  if (d == 64) launch<64>(p, e4m3, s);
  if (d == 128) launch<128>(p, e4m3, s);
  if (d == 256) launch<256>(p, e4m3, s);
  return cudaGetLastError();
}

}  // namespace moe
