// Device helpers of the 8-bit expert kernels: bf16 and e4m3 pieces of rows, quantising.
#pragma once

#include "experts.h"
#include "ptx.cuh"

namespace moe {

__device__ __forceinline__ void raise_index(WsHeader* hdr) { atomicOr(&hdr->status, status_bit(MOE_ERR_BAD_INDEX)); }

// 8 bf16 values as floats.
__device__ __forceinline__ void bf16x8_to_float(uint4 v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
// Two floats rounded to bf16, lo in the low half.
__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
__device__ __forceinline__ uint4 float_to_bf16x8(const float* x) {
  return make_uint4(to_bf16x2(x[0], x[1]), to_bf16x2(x[2], x[3]), to_bf16x2(x[4], x[5]), to_bf16x2(x[6], x[7]));
}
// Two floats rounded to nearest even e4m3, clamped to +-448, NaN as 0x7F; lo in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t w;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(w) : "f"(hi), "f"(lo));
  return w;
}

constexpr float kLeastAmax = 0x1p-100f;  // of a block: smaller ones are quantised as if it were this
constexpr float kE4m3Max = 448.f;

// The factors of a block whose largest finite magnitude is a: codes are x * inv.
struct BlockScale {
  float scale, inv;
};
__device__ __forceinline__ BlockScale block_scale(float a) {
  a = fmaxf(a, kLeastAmax);
  return {__fdiv_rn(a, kE4m3Max), __fdiv_rn(kE4m3Max, a)};
}
// The code's value before rounding: infinities become NaN (inf * 0), everything else stays x * inv.
__device__ __forceinline__ float coded(float x, float inv) { return __fmaf_rn(x, 0.f, __fmul_rn(x, inv)); }

__device__ __forceinline__ uint4 codes16(const float (&y)[16]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = to_e4m3x2(y[4 * i], y[4 * i + 1]) | to_e4m3x2(y[4 * i + 2], y[4 * i + 3]) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Quantises 16 consecutive values per lane, 8 lanes to a block of 128; a whole warp calls it.
__device__ __forceinline__ uint4 quantise16(const float (&x)[16], float* scale) {
  float a = 0.f, y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) a = fmaxf(a, fabsf(x[i]));  // NaN is passed over
  const bool fine = __all_sync(~0u, a < INFINITY);
  if (!fine) {  // rare: an infinity does not count either
    a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float m = fabsf(x[i]);
      a = fmaxf(a, m < INFINITY ? m : 0.f);
    }
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) a = fmaxf(a, __shfl_xor_sync(~0u, a, o));
  const BlockScale b = block_scale(a);
  *scale = b.scale;
  if (fine) {  // no infinities: the product alone (NaN stays NaN)
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(x[i], b.inv);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = coded(x[i], b.inv);
  }
  return codes16(y);
}

__device__ __forceinline__ const uint4* bf16_at(const moe_rows& r, int64_t row, int col) {
  return reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(r.p) + row * r.stride + col);
}
__device__ __forceinline__ void load16(const moe_rows& r, int64_t row, int col, uint4 (&v)[2]) {
  const uint4* p = bf16_at(r, row, col);
  v[0] = __ldg(p);
  v[1] = __ldg(p + 1);
}
// 16 codes of a lane, and the block's scale from the lane that begins it.
__device__ __forceinline__ void store_codes(const moe_rows& r, int64_t row, int col, uint4 codes, float scale) {
  *reinterpret_cast<uint4*>(static_cast<uint8_t*>(r.p) + row * r.stride + col) = codes;
  if (col % kScaleBlock == 0) r.scale[row * r.scale_stride + col / kScaleBlock] = scale;
}
__device__ __forceinline__ void store_bf16(const moe_rows& r, int64_t row, int col, uint4 v0, uint4 v1) {
  uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(r.p) + row * r.stride + col);
  p[0] = v0;
  p[1] = v1;
}
// 16 fp32 values of a lane (8 lanes to a block of 128) in the rows' format; a whole warp calls it,
// lanes with !mine store nothing and hold zeros.
template <bool E4M3>
__device__ __forceinline__ void store16(const moe_rows& r, int64_t row, int col, const float (&x)[16], bool mine) {
  if (E4M3) {
    float scale;
    const uint4 codes = quantise16(x, &scale);
    if (mine) store_codes(r, row, col, codes, scale);
  } else if (mine) {
    store_bf16(r, row, col, float_to_bf16x8(x), float_to_bf16x8(x + 8));
  }
}

}  // namespace moe
