// moe_kv_append: new keys and values into the paged cache, as bf16 or as e4m3 with a scale per head.
//
// A copy: 2 * total * hkv * d values read as bf16 and written in the cache's type; bound by HBM for
// long prompts and by one chain of dependent loads (offsets -> page number -> store) for the few
// rows of a decode step. One thread moves one 8-value piece of k and the same piece of v, so that
// its two row loads are in flight while it looks its sequence and page up.
#include <cuda_fp8.h>

#include "attn_device.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// The first b in [0, n) with cu[b + 1] > t (n - 1 if there is none); all lanes of a full warp with the same t.
__device__ __forceinline__ int warp_find_seq(const int32_t* cu, int n, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;  // the answer lies in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = min(lo + (lane + 1) * step, hi) - 1;  // last index of this lane's piece
    const unsigned m = __ballot_sync(~0u, __ldg(cu + i + 1) > t);
    const int first = m ? __ffs(m) - 1 : 31;
    const int at = lo + first * step;
    hi = min(at + step, hi);
    lo = min(at, hi - 1);
  }
  return lo;
}

__device__ __forceinline__ uint2 to_e4m3(uint4 x, float scale) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = make_float2(__fdiv_rn(__uint_as_float(w[i] << 16), scale),
                                 __fdiv_rn(__uint_as_float(w[i] & 0xFFFF0000u), scale));
    out[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(out[0] | (out[1] << 16), out[2] | (out[3] << 16));
}

template <bool E4M3>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(KvAppendParams p) {
  const int per_token = p.hkv * (p.d / 8);
  const int64_t idx = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t warp0 = idx - (threadIdx.x & 31);
  const int64_t end = (int64_t)p.total * per_token;
  if (blockIdx.x == 0) check_offsets(p.cu, p.n_seqs, p.total, p.hdr, threadIdx.x, kThreads);
  if (warp0 >= end) return;
  const int t0 = (int)(warp0 / per_token);
  const int64_t i = idx < end ? idx : end - 1;
  const int t = (int)(i / per_token), piece = (int)(i % per_token);
  const int h = piece / (p.d / 8), c = piece % (p.d / 8);
  const uint4 kx = __ldg(reinterpret_cast<const uint4*>(p.k.p + t * p.k.token_stride + h * p.k.head_stride + c * 8));
  const uint4 vx = __ldg(reinterpret_cast<const uint4*>(p.v.p + t * p.v.token_stride + h * p.v.head_stride + c * 8));
  int b = warp_find_seq(p.cu, p.n_seqs, t0);
  while (b + 1 < p.n_seqs && __ldg(p.cu + b + 1) <= t) ++b;
  const int row = t - __ldg(p.cu + b), first = __ldg(p.start + b);
  const int64_t pos = (int64_t)first + row;
  const int64_t at = pos / p.page_size;
  bool ok = row >= 0 && t < __ldg(p.cu + b + 1) && first >= 0 && at < p.table_width;
  int page = 0;
  if (ok) {
    page = __ldg(p.table + (int64_t)b * p.table_width + at);
    ok = page >= 0 && page < p.n_pages;
  }
  if (idx >= end) return;
  if (!ok) {
    raise_bad_index(p.hdr);
    return;
  }
  const int64_t cell = ((int64_t)page * p.hkv + h) * p.page_size + (int)(pos - at * p.page_size);
  const int64_t off = cell * p.d + c * 8;
  if (E4M3) {
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.kc) + off) = to_e4m3(kx, __ldg(p.k_scale + h));
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.vc) + off) = to_e4m3(vx, __ldg(p.v_scale + h));
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.kc) + off) = kx;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.vc) + off) = vx;
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t s) {
  const int64_t pieces = (int64_t)p.total * p.hkv * (p.d / 8);
  const int64_t grid = (pieces + kThreads - 1) / kThreads;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  if (p.e4m3)
    kv_append_kernel<true><<<(unsigned)grid, kThreads, 0, s>>>(p);
  else
    kv_append_kernel<false><<<(unsigned)grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace moe
