// moe_kv_append: new keys and values into the paged cache, as bf16 or as e4m3 with a scale per head.
//
// A copy: 2 * total * hkv * d values read as bf16 and written in the cache's type; bound by HBM for
// long prompts and by one chain of dependent loads (offsets -> page number -> store) for the few
// rows of a decode step. A thread moves one or two 8-value pieces of a token's k and the same pieces of
// its v: their loads are in flight while it looks the token's sequence and page up, with 32-bit divisions
// by multiplication (64-bit ones took two thirds of the issue slots: 13.9 us for 8192 tokens of 8 heads
// of 128, against 12.2 now, 5.5 TB/s; as e4m3, with an IEEE division per value, 14.4 us, 3.5 TB/s).
#include <cuda_fp8.h>

#include "attn_device.cuh"
#include "ptx.cuh"

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

// tpt threads to a token, kThreads / tpt tokens to a block; NP pieces to a thread, tpt apart.
template <bool E4M3, int NP>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ KvAppendParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const unsigned slot = p.div_tpt(threadIdx.x);  // token of the block
  const int t = blockIdx.x * p.tokens + slot, first_piece = threadIdx.x - slot * p.tpt;
  const bool mine = slot < p.tokens && t < p.total;
  uint4 kx[NP], vx[NP];
  int h[NP], c[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int piece = first_piece + i * p.tpt;
    h[i] = p.head0 + (piece >> p.log_dp);
    c[i] = (piece & ((1 << p.log_dp) - 1)) * 8;
    if (mine) {
      kx[i] = __ldg(reinterpret_cast<const uint4*>(p.k.p + t * p.k.token_stride + h[i] * p.k.head_stride + c[i]));
      vx[i] = __ldg(reinterpret_cast<const uint4*>(p.v.p + t * p.v.token_stride + h[i] * p.v.head_stride + c[i]));
    }
  }
  if (blockIdx.x == 0) check_offsets(p.cu, p.n_seqs, p.total, p.hdr, threadIdx.x, kThreads);
  int b = warp_find_seq(p.cu, p.n_seqs, __shfl_sync(~0u, t, 0));
  if (!mine) return;
  while (b + 1 < p.n_seqs && __ldg(p.cu + b + 1) <= t) ++b;
  const int row = t - __ldg(p.cu + b), first = __ldg(p.start + b);
  const unsigned pos = (unsigned)first + (unsigned)row;  // below 2^31 + 2^30 where both are valid
  const unsigned at = p.page_div(pos);
  bool ok = row >= 0 && t < __ldg(p.cu + b + 1) && first >= 0 && at < (unsigned)p.table_width;
  int page = 0;
  if (ok) {
    page = __ldg(p.table + (int64_t)b * p.table_width + at);
    ok = page >= 0 && page < p.n_pages;
  }
  if (!ok) {
    raise_bad_index(p.hdr);
    return;
  }
  const int in_page = (int)(pos - at * p.page_size);
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int cell = (page * p.hkv + h[i]) * p.page_size + in_page;  // a cache has fewer than 2^31 rows
    const int64_t off = (int64_t)cell * p.d + c[i];
    if (E4M3) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.kc) + off) = to_e4m3(kx[i], __ldg(p.k_scale + h[i]));
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.vc) + off) = to_e4m3(vx[i], __ldg(p.v_scale + h[i]));
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.kc) + off) = kx[i];
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.vc) + off) = vx[i];
    }
  }
}

template <bool E4M3>
cudaError_t launch(KvAppendParams& p, cudaStream_t s) {
  const int pieces = p.heads * (p.d / 8);  // of a token, two to a thread where they fill warps
  const int np = pieces >= 64 ? 2 : 1;
  p.tpt = pieces / np;
  p.tokens = kThreads / p.tpt;
  p.div_tpt = FastDiv(p.tpt);
  const int64_t grid = ((int64_t)p.total + p.tokens - 1) / p.tokens;
  const dim3 g((unsigned)grid);
  return np == 2 ? launch_pdl(kv_append_kernel<E4M3, 2>, g, kThreads, 0, 1, s, p)
                 : launch_pdl(kv_append_kernel<E4M3, 1>, g, kThreads, 0, 1, s, p);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& params, cudaStream_t s) {
  KvAppendParams p = params;
  p.log_dp = p.d == 64 ? 3 : p.d == 128 ? 4 : 5;
  // at most 2 * kThreads pieces to a token: 512 / (d / 8) heads at a time (more than 16 heads of 256, say,
  // take another launch)
  const int most = 2 * kThreads / (p.d / 8);
  for (int h0 = 0; h0 < params.hkv; h0 += most) {
    p.heads = params.hkv - h0 < most ? params.hkv - h0 : most;
    p.head0 = h0;
    const cudaError_t err = p.e4m3 ? launch<true>(p, s) : launch<false>(p, s);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace moe
