// Device helpers of the 8-bit expert kernels: bf16 and e4m3 pieces of rows, quantising.
#pragma once

#include "attn_ptx.cuh"
#include "experts.h"

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
  // a / 448, correctly rounded: with the rounded reciprocal one corrected step is (Markstein, Computation of
  // Elementary Functions on the IBM RISC System/6000 Processor, 1990); nothing here is near under- or overflow.
  const float y = 1.f / kE4m3Max, q = __fmul_rn(a, y);
  return {__fmaf_rn(__fmaf_rn(-q, kE4m3Max, a), y, q), __fdiv_rn(kE4m3Max, a)};
}
// The code's value before rounding: infinities become NaN (inf * 0), everything else stays x * inv.
__device__ __forceinline__ float coded(float x, float inv) { return __fmaf_rn(x, 0.f, __fmul_rn(x, inv)); }

__device__ __forceinline__ const uint4* bf16_at(const moe_rows& r, int64_t row, int col) {
  return reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(r.p) + row * r.stride + col);
}

// A warp's piece of a row: 512 columns, lane l holds the 8 from 8 l and the 8 from 256 + 8 l on, so that
// every access of a warp is one run of memory (32 bytes to a lane in two halves cost 15% of a copy).
// A block of 128 is 16 lanes' first or second 8.
constexpr int kPiece = 512;
__device__ __forceinline__ int piece_col(int piece, int half) { return piece * kPiece + half * 256 + (threadIdx.x & 31) * 8; }

__device__ __forceinline__ void load_piece(const moe_rows& r, int64_t row, int piece, int cols, uint4 (&v)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = piece_col(piece, h);
    v[h] = c < cols ? __ldg(bf16_at(r, row, c)) : make_uint4(0, 0, 0, 0);
  }
}
__device__ __forceinline__ void piece_to_float(const uint4 (&v)[2], float (&x)[16]) {
  bf16x8_to_float(v[0], x);
  bf16x8_to_float(v[1], x + 8);
}

// Codes of a piece (zeros past the row's end), and the scale of the block that this lane's group of 8 is
// left with: of its first half's block in lanes 0-7 and 16-23, of its second half's in the others.
struct PieceCodes {
  uint2 q[2];
  float scale;
};
// A whole warp calls it.
__device__ __forceinline__ PieceCodes quantise_piece(const float (&x)[16]) {
  float a[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 16; i += 2) a[i >> 3] = max3(a[i >> 3], fabsf(x[i]), fabsf(x[i + 1]));  // NaN is passed over
  const bool fine = __all_sync(~0u, fmaxf(a[0], a[1]) < INFINITY);
  if (!fine) {  // rare: an infinity does not count either
    a[0] = a[1] = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float m = fabsf(x[i]);
      a[i >> 3] = fmaxf(a[i >> 3], m < INFINITY ? m : 0.f);
    }
  }
  // 16 lanes and two halves: lanes 8 apart trade halves, then each group of 8 finds the maximum of one
  const bool upper = threadIdx.x & 8;
  float m = fmaxf(upper ? a[1] : a[0], __shfl_xor_sync(~0u, upper ? a[0] : a[1], 8));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  const BlockScale b = block_scale(m);
  const float other = __shfl_xor_sync(~0u, b.inv, 8);
  const float inv[2] = {upper ? other : b.inv, upper ? b.inv : other};
  float y[16];
  if (fine) {  // no infinities: the product alone (NaN stays NaN)
#pragma unroll
    for (int i = 0; i < 16; i += 2)
      unpack2(mul2(pack2(x[i], x[i + 1]), pack2(inv[i >> 3], inv[i >> 3])), y[i], y[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = coded(x[i], inv[i >> 3]);
  }
  PieceCodes r;
  r.scale = b.scale;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float* z = y + 8 * h;
    r.q[h] = make_uint2(to_e4m3x2(z[0], z[1]) | to_e4m3x2(z[2], z[3]) << 16, to_e4m3x2(z[4], z[5]) | to_e4m3x2(z[6], z[7]) << 16);
  }
  return r;
}
__device__ __forceinline__ void store_codes(const moe_rows& r, int64_t row, int piece, int cols, const PieceCodes& p) {
  uint8_t* q = static_cast<uint8_t*>(r.p) + row * r.stride;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (piece_col(piece, h) < cols) *reinterpret_cast<uint2*>(q + piece_col(piece, h)) = p.q[h];
  const int lane = threadIdx.x & 31, b = piece * 4 + (lane >> 3 & 1) * 2 + (lane >> 4);
  if ((lane & 7) == 0 && b * kScaleBlock < cols) r.scale[row * r.scale_stride + b] = p.scale;
}
__device__ __forceinline__ void store_bf16(const moe_rows& r, int64_t row, int piece, int cols, const uint4 (&v)[2]) {
  uint16_t* o = static_cast<uint16_t*>(r.p) + row * r.stride;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (piece_col(piece, h) < cols) *reinterpret_cast<uint4*>(o + piece_col(piece, h)) = v[h];
}
// The fp32 values of a piece in the rows' format; a whole warp calls it, with zeros past the row's end.
template <bool E4M3>
__device__ __forceinline__ void store_piece(const moe_rows& r, int64_t row, int piece, int cols, const float (&x)[16]) {
  if (E4M3) {
    store_codes(r, row, piece, cols, quantise_piece(x));
  } else {
    const uint4 v[2] = {float_to_bf16x8(x), float_to_bf16x8(x + 8)};
    store_bf16(r, row, piece, cols, v);
  }
}

}  // namespace moe
