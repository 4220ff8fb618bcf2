// moe_gemm_e4m3: products of e4m3 rows with their experts' e4m3 matrices, a scale for each block of 128.
//
// The simplest form: a CTA makes 64 rows x 64 columns of one expert's output; 32 inputs at a time go
// through shared memory as floats, each thread sums 4 x 4 values, and every 128 inputs the block's sums
// are multiplied by their scales and added up.
#include <cuda_fp8.h>

#include "expert_device.cuh"

namespace moe {
namespace {

constexpr int kTile = 64, kStep = 32, kThreads = 256;

__device__ __forceinline__ float e4m3_float(uint8_t c) {
  __nv_fp8_e4m3 v;
  v.__x = c;
  return static_cast<float>(v);
}

__global__ void __launch_bounds__(kThreads) product_kernel(const __grid_constant__ ProductParams p) {
  __shared__ float sa[kStep][kTile + 1], sw[kStep][kTile + 1];
  __shared__ int s_expert, s_first, s_rows;
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    s_rows = 0;
    if (!p.offsets) {
      s_expert = 0;
      s_first = blockIdx.x * kTile;
      s_rows = min(kTile, p.rows - s_first);
    } else {
      int tile = blockIdx.x, end = 0;
      for (int e = 0; e < p.n_experts; ++e) {
        const int lo = __ldg(p.offsets + e), hi = __ldg(p.offsets + e + 1);
        const int b = min(max(lo, end), p.rows), n = min(max(hi, b), p.rows) - b, tiles = (n + kTile - 1) / kTile;
        if (blockIdx.x == 0 && blockIdx.y == 0 && (lo != b || hi != b + n || (e == 0 && lo != 0))) raise_index(p.hdr);
        end = b + n;
        if (tile >= 0 && tile < tiles) {
          s_expert = e;
          s_first = b + tile * kTile;
          s_rows = min(kTile, n - tile * kTile);
        }
        tile -= tiles;
        if (tile < 0 && (blockIdx.x || blockIdx.y)) break;
      }
    }
  }
  __syncthreads();
  if (s_rows <= 0) return;
  const int e = s_expert, first = s_first, rows = s_rows, c0 = blockIdx.y * kTile;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const uint8_t* aq = static_cast<const uint8_t*>(p.a.p);
  const uint8_t* wq = p.wq + (int64_t)e * p.n * p.k;
  const int kb = (p.k + kScaleBlock - 1) / kScaleBlock;
  const float* ws = p.wscale + (int64_t)e * p.in_blocks * p.out_blocks;
  float acc[4][4] = {};
  for (int b = 0; b < p.in_blocks; ++b) {
    float part[4][4] = {};
    for (int i0 = b * kScaleBlock; i0 < min(p.in, (b + 1) * kScaleBlock); i0 += kStep) {
      __syncthreads();
      for (int x = threadIdx.x; x < kTile * kStep; x += kThreads) {
        const int r = x / kStep, i = i0 + x % kStep;
        sa[x % kStep][r] = r < rows && i < p.in ? e4m3_float(aq[(int64_t)(first + r) * p.a.stride + i]) : 0.f;
        const int c = p.transposed ? x % kTile : x / kStep, j = p.transposed ? x / kTile : x % kStep;
        const bool there = c0 + c < p.outc && i0 + j < p.in;
        sw[j][c] = !there         ? 0.f
                   : p.transposed ? e4m3_float(wq[(int64_t)(i0 + j) * p.k + c0 + c])
                                  : e4m3_float(wq[(int64_t)(c0 + c) * p.k + i0 + j]);
      }
      __syncthreads();
      for (int j = 0; j < kStep; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int c = 0; c < 4; ++c) part[r][c] = fmaf(sa[j][ty * 4 + r], sw[j][tx * 4 + c], part[r][c]);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int row = ty * 4 + r, ob = (c0 + tx * 4 + c) / kScaleBlock;
        if (row < rows && c0 + tx * 4 + c < p.outc)
          acc[r][c] = fmaf(p.a.scale[(first + row) * p.a.scale_stride + b] * (p.transposed ? ws[b * kb + ob] : ws[ob * kb + b]),
                           part[r][c], acc[r][c]);
      }
  }
  uint16_t* o = static_cast<uint16_t*>(p.out.p);
  for (int r = 0; r < 4; ++r)
    for (int c = 0; c < 4; c += 2)  // the number of columns is even
      if (ty * 4 + r < rows && c0 + tx * 4 + c < p.outc)
        *reinterpret_cast<uint32_t*>(o + (int64_t)(first + ty * 4 + r) * p.out.stride + c0 + tx * 4 + c) =
            to_bf16x2(acc[r][c], acc[r][c + 1]);
}

}  // namespace

cudaError_t launch_product(const ProductParams& p, cudaStream_t s) {
  const int tiles = (p.rows + kTile - 1) / kTile;
  const dim3 grid(p.offsets ? tiles + p.n_experts : tiles, (p.outc + kTile - 1) / kTile);
  return launch_pdl(product_kernel, grid, kThreads, 0, 1, s, p);
}

}  // namespace moe
