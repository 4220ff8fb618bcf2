// The row-wise 8-bit expert calls: moe_dispatch, moe_combine, moe_combine_grad, moe_swiglu and its
// gradient, moe_quant_weights. Each reads its rows once and writes its rows once: all are bound by HBM
// where there are many rows, by launch and one load's latency where there are few.
//
// A warp takes pieces of 512 columns, 16 to a lane; a block's largest magnitude takes four shuffles. Figures below: rows of
// 2048 columns, 8 assignments to a token, one GB300 (a copy: 6.78 TB/s).
#include "expert_device.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// kWarps warps of a CTA as rows x warps per row; each warp takes every warps-th piece of its row.
struct Split {
  int warps, rows;
};
inline Split split_of(int pieces) {
  int w = 1;
  while (w < kWarps && 2 * w <= pieces) w *= 2;
  return {w, kWarps / w};
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// The i-th pair of values of a piece.
__device__ __forceinline__ uint64_t pair_of(const uint4 (&v)[2], int i) {
  const uint32_t w = word(v[i >> 2], i & 3);
  return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// ------------------------------------------------------------------------------------ dispatch
// A token's row is read once and written top_k times: 16383 tokens take 53 us in e4m3 (6.3 TB/s), 89 us in bf16 (6.8).
template <bool E4M3>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const __grid_constant__ DispatchParams p, int warps) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * (kWarps / warps) + warp / warps;
  if (t >= p.T) return;  // the whole warp
  int place = -1;
  if (lane < p.k) place = p.inv ? __ldg(p.inv + t * p.k + lane) : (int)t;
  if (place >= p.out_rows) {
    raise_index(p.hdr);
    place = -1;
  }
  if (!__any_sync(~0u, place >= 0)) return;
  for (int piece = warp % warps; piece < p.segments; piece += warps) {
    uint4 v[2];
    load_piece(p.x, t, piece, p.d, v);
    PieceCodes codes;
    if (E4M3) {
      float x[16];
      piece_to_float(v, x);
      codes = quantise_piece(x);
    }
    for (int j = 0; j < p.k; ++j) {
      const int row = __shfl_sync(~0u, place, j);
      if (row < 0) continue;
      if (E4M3)
        store_codes(p.out, row, piece, p.d, codes);
      else
        store_bf16(p.out, row, piece, p.d, v);
    }
  }
}

// ------------------------------------------------------------------------------------ combine
// The rows of a token, scattered, summed in the order of its list: 4096 tokens take 25.6 us (5.9 TB/s; 28.2 with each token's
// places loaded only when its turn came).
constexpr int kCombinePiece = 256;  // 8 columns per lane: one 16-byte load of each row
constexpr int kTogether = 8;        // rows whose loads are in flight together

__global__ void __launch_bounds__(kThreads) combine_kernel(const __grid_constant__ CombineParams p, int warps) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, step = gridDim.x * (kWarps / warps);
  int t = blockIdx.x * (kWarps / warps) + warp / warps;
  // the places and weights of a token, loaded while the one before is worked on
  int place = -1;
  float weight = 1.f;
  auto load = [&](int t) {
    if (lane < p.k && t < p.T) {
      place = __ldg(p.inv + (int64_t)t * p.k + lane);
      if (p.w) weight = __ldg(p.w + (int64_t)t * p.k + lane);
    }
  };
  load(t);
  for (; t < p.T; t += step) {
    if (place >= p.ys_rows) {
      raise_index(p.hdr);
      place = -1;
    }
    const int now = place;
    const float w_now = now < 0 ? 0.f : weight;
    load(t + step);
    for (int piece = warp % warps; piece < p.segments; piece += warps) {
      const int c = piece * kCombinePiece + lane * 8;
      const bool mine = c < p.d;
      float acc[8] = {};
      if (mine && p.add.p) bf16x8_to_float(*bf16_at(p.add, t, c), acc);
      for (int j0 = 0; j0 < p.k; j0 += kTogether) {
        uint4 v[kTogether];
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
          const int row = __shfl_sync(~0u, now, j0 + i);  // lanes from top_k on hold -1
          v[i] = row >= 0 && mine ? __ldg(bf16_at(p.ys, row, c)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
          const float w = __shfl_sync(~0u, w_now, j0 + i);
          float x[8];
          bf16x8_to_float(v[i], x);
#pragma unroll
          for (int u = 0; u < 8; ++u) acc[u] = fmaf(w, x[u], acc[u]);
        }
      }
      if (mine)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y.p) + t * p.y.stride + c) = float_to_bf16x8(acc);
    }
  }
}

// One warp per assignment: dy's row is read by the token's top_k warps out of L1, and a weight's gradient is one warp's sum.
// 16383 tokens take 143 us in e4m3 (5.9 TB/s); 171 with one fp32 operation a value and no loads ahead.
template <bool E4M3>
__global__ void __launch_bounds__(512) combine_grad_kernel(const __grid_constant__ CombineGradParams p, int tokens) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = warp % p.k, step = gridDim.x * tokens;
  int t = blockIdx.x * tokens + warp / p.k, place = -1;
  float w = 0.f;
  auto load = [&](int t) {  // a token's place and weight, loaded while the one before is worked on
    if (t < p.T) {
      place = __ldg(p.inv + (int64_t)t * p.k + j);
      w = __ldg(p.w + (int64_t)t * p.k + j);
    }
  };
  load(t);
  for (; t < p.T; t += step) {
    const int now = place;
    const uint64_t w2 = pack2(w, w);
    float* dw = p.dw + (int64_t)t * p.k + j;
    load(t + step);
    if (now < 0 || now >= p.ys_rows) {
      if (lane == 0) {
        if (now >= 0) raise_index(p.hdr);
        *dw = 0.f;
      }
      continue;
    }
    uint64_t dot2[2] = {0, 0};
    uint4 g[2], y[2];
    load_piece(p.ys, now, 0, p.d, y);
    load_piece(p.dy, t, 0, p.d, g);
    for (int piece = 0; piece * kPiece < p.d; ++piece) {
      float x[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t g2 = pair_of(g, i);
        dot2[i & 1] = fma2(g2, pair_of(y, i), dot2[i & 1]);
        unpack2(mul2(g2, w2), x[2 * i], x[2 * i + 1]);
      }
      load_piece(p.ys, now, piece + 1, p.d, y);  // zeros past the end
      load_piece(p.dy, t, piece + 1, p.d, g);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (piece_col(piece, i) >= p.d) {  // past the row's end: zeros, not 0 * w (w may be infinite)
#pragma unroll
          for (int u = 0; u < 8; ++u) x[8 * i + u] = 0.f;
        }
      store_piece<E4M3>(p.dys, now, piece, p.d, x);
    }
    float part[4];
    unpack2(dot2[0], part[0], part[1]);
    unpack2(dot2[1], part[2], part[3]);
    float dot = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
    for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(~0u, dot, o);
    if (lane == 0) *dw = dot;
  }
}

// ------------------------------------------------------------------------------------ SwiGLU
// s = 1 / (1 + e^-g) of two values from -32 on: e^-g to a few units of the last place (its argument's rounding: |g| 2^-24).
__device__ __forceinline__ uint64_t sigmoid2(uint64_t g) {
  constexpr float c = -1.4426950408889634f;
  float x, y, r, s;
  unpack2(mul2(g, pack2(c, c)), x, y);
  unpack2(add2(pack2(ex2(x), ex2(y)), pack2(1.f, 1.f)), x, y);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(y));
  return pack2(r, s);
}

// Below -32, where s is less than 2^-46, its products are made in 64 bits: from -87 on s is no normal fp32 number, while a
// large u or dh may bring the result back into range (bf16 reaches from 2^-133 to 2^128). There s is e^g to 2^-46, taken
// as the fourth power of 2^(g log2(e) / 4), which is normal down to g = -349; below, no result is. Such values are rare: a
// piece is looked over once, and one that has any takes the longer way (a value at a time: 80 registers in the gradient,
// where calls in any order take 125).
constexpr float kFar = -32.f;
constexpr uint32_t kFarBits = 0xC200;  // in bf16; greater as an unsigned number are the values below (and NaN with a sign)
__device__ __forceinline__ bool any_far(const uint4 (&g)[2]) {
  uint32_t m = __vmaxu2(word(g[0], 0), word(g[1], 0));
#pragma unroll
  for (int i = 1; i < 4; ++i) m = __vmaxu2(m, __vmaxu2(word(g[0], i), word(g[1], i)));
  return m >> 16 > kFarBits || (m & 0xFFFFu) > kFarBits;
}
__device__ __forceinline__ double far_sigmoid(float g) {
  float x;
  asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(g * (1.4426950408889634f / 4)));  // volatile: one after the other
  const double r = x, r2 = r * r;
  return r2 * r2;
}

__device__ __forceinline__ int rows_that_count(const SwigluParams& p) {
  if (!p.total) return p.rows;
  const int n = __ldg(p.total);
  if (n < 0 || n > p.rows) {
    if (threadIdx.x == 0) raise_index(p.hdr);
    return n < 0 ? 0 : p.rows;
  }
  return n;
}

// A warp's way over the pieces of its rows, rows a grid's width apart: the next piece's loads are issued
// before the present one is worked on.
struct Walk {
  int64_t row, step;
  int piece, warps, pieces, rows;
  Walk() = default;
  __device__ __forceinline__ Walk(const SwigluParams& p, int w) {
    const int warp = threadIdx.x >> 5;
    warps = w, pieces = p.segments, rows = rows_that_count(p), piece = warp % w;
    row = (int64_t)blockIdx.x * (kWarps / w) + warp / w, step = (int64_t)gridDim.x * (kWarps / w);
  }
  __device__ __forceinline__ bool inside() const { return row < rows; }
  __device__ __forceinline__ Walk next() const {
    Walk n = *this;
    if ((n.piece += warps) >= pieces) n.piece = (threadIdx.x >> 5) % warps, n.row += step;
    return n;
  }
};

// Rows of p from column `first` on.
__device__ __forceinline__ moe_rows from_col(moe_rows r, int first) {
  r.p = static_cast<uint16_t*>(r.p) + first;
  return r;
}

// 32768 rows of 512 take 15 us in e4m3 (5.6 TB/s, 2 us of them a launch and its tail), 18.3 with a warp to a piece and no loads
// ahead. More CTAs to an SM cost registers and gain nothing.
template <bool E4M3>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(const __grid_constant__ SwigluParams p, int warps) {
  pdl_wait();
  pdl_launch_dependents();
  const moe_rows up = from_col(p.gu, p.inter);
  Walk at(p, warps), next;
  uint4 gv[2], uv[2];
  if (at.inside()) {
    load_piece(p.gu, at.row, at.piece, p.inter, gv);
    load_piece(up, at.row, at.piece, p.inter, uv);
  }
  for (; at.inside(); at = next) {
    next = at.next();
    uint64_t g[8], u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = pair_of(gv, i), u[i] = pair_of(uv, i);
    const bool far = any_far(gv);
    if (next.inside()) {
      load_piece(p.gu, next.row, next.piece, p.inter, gv);
      load_piece(up, next.row, next.piece, p.inter, uv);
    }
    float h[16];
    if (!far) {
#pragma unroll
      for (int i = 0; i < 8; ++i) unpack2(mul2(mul2(g[i], sigmoid2(g[i])), u[i]), h[2 * i], h[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x[2], y[2];
        unpack2(mul2(mul2(g[i], sigmoid2(g[i])), u[i]), h[2 * i], h[2 * i + 1]);
        unpack2(g[i], x[0], x[1]);
        unpack2(u[i], y[0], y[1]);
#pragma unroll
        for (int v = 0; v < 2; ++v)
          if (x[v] < kFar) h[2 * i + v] = (float)(far_sigmoid(x[v]) * x[v] * y[v]);
      }
    }
    store_piece<E4M3>(p.out, at.row, at.piece, p.inter, h);
  }
}

// dg and du of 16 columns; either may be left out.
template <bool FAR>
__device__ __forceinline__ void swiglu_grad16(const uint4 (&gv)[2], const uint4 (&uv)[2], const uint4 (&hv)[2],
                                              float (&dg)[16], float (&du)[16]) {
  const uint64_t one = pack2(1.f, 1.f), minus = pack2(-1.f, -1.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t g = pair_of(gv, i), s = sigmoid2(g), hs = mul2(pair_of(hv, i), s);
    unpack2(mul2(mul2(hs, pair_of(uv, i)), fma2(g, fma2(s, minus, one), one)), dg[2 * i], dg[2 * i + 1]);
    unpack2(mul2(hs, g), du[2 * i], du[2 * i + 1]);
    if (FAR) {
      float x[2], u[2], h[2];
      unpack2(g, x[0], x[1]);
      unpack2(pair_of(uv, i), u[0], u[1]);
      unpack2(pair_of(hv, i), h[0], h[1]);
#pragma unroll
      for (int v = 0; v < 2; ++v)
        if (x[v] < kFar) {
          const double s = far_sigmoid(x[v]) * h[v];
          dg[2 * i + v] = (float)(s * u[v] * (1.0 + x[v]));
          du[2 * i + v] = (float)(s * x[v]);
        }
    }
  }
}

// WHOLE: inter is a multiple of 128, so that the blocks of dg and of du begin at the same columns and a
// warp makes both from one reading. Otherwise the blocks of du straddle the two halves: the pieces run
// over the 2 inter output columns, and what du needs of g and dh is read again (out of L2). 15893 rows of 512: 13.1 us.
template <bool E4M3, bool WHOLE>
__global__ void __launch_bounds__(kThreads) swiglu_grad_kernel(const __grid_constant__ SwigluParams p, int warps) {
  pdl_wait();
  pdl_launch_dependents();
  const moe_rows up = from_col(p.gu, p.inter);
  moe_rows second = p.out;  // WHOLE: du begins with a block of its own
  second.p = static_cast<uint8_t*>(second.p) + (E4M3 ? 1 : 2) * p.inter;
  second.scale += E4M3 ? p.inter / kScaleBlock : 0;
  uint4 gv[2], uv[2], hv[2];
  auto load = [&](const Walk& at) {
    if constexpr (WHOLE) {
      load_piece(p.gu, at.row, at.piece, p.inter, gv);
      load_piece(p.dh, at.row, at.piece, p.inter, hv);
      load_piece(up, at.row, at.piece, p.inter, uv);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int o = piece_col(at.piece, h), c = o >= p.inter ? o - p.inter : o;  // output column, its g's
        gv[h] = uv[h] = hv[h] = make_uint4(0, 0, 0, 0);
        if (o < 2 * p.inter) {
          gv[h] = __ldg(bf16_at(p.gu, at.row, c));
          hv[h] = __ldg(bf16_at(p.dh, at.row, c));
          if (o < p.inter) uv[h] = __ldg(bf16_at(up, at.row, c));
        }
      }
    }
  };
  Walk at(p, warps), next;
  if (at.inside()) load(at);
  for (; at.inside(); at = next) {
    next = at.next();
    float dg[16], du[16];
    if (any_far(gv))
      swiglu_grad16<true>(gv, uv, hv, dg, du);
    else
      swiglu_grad16<false>(gv, uv, hv, dg, du);
    if (next.inside()) load(next);
    if (WHOLE) {
      store_piece<E4M3>(p.out, at.row, at.piece, p.inter, dg);
      store_piece<E4M3>(second, at.row, at.piece, p.inter, du);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) dg[i] = piece_col(at.piece, i >> 3) >= p.inter ? du[i] : dg[i];
      store_piece<E4M3>(p.out, at.row, at.piece, 2 * p.inter, dg);
    }
  }
}

// ------------------------------------------------------------------------------------ weights
// One CTA per block of 128 x 128: 16 threads to a row, 16 rows to a pass.
__global__ void __launch_bounds__(kThreads) quant_weights_kernel(const QuantWeightsParams p) {
  __shared__ float s_max[kWarps];
  const int r0 = blockIdx.y * kScaleBlock + threadIdx.x / 16, c = blockIdx.x * kScaleBlock + threadIdx.x % 16 * 8;
  const int64_t e = blockIdx.z;
  const uint16_t* w = p.w + (e * p.n) * p.k + c;
  uint4 v[8];
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    v[i] = r < p.n && c < p.k ? __ldg(reinterpret_cast<const uint4*>(w + (int64_t)r * p.k)) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float x[8];
    bf16x8_to_float(v[i], x);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float m = fabsf(x[u]);
      a = fmaxf(a, m < INFINITY ? m : 0.f);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(~0u, a, o));
  if (threadIdx.x % 32 == 0) s_max[threadIdx.x / 32] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) a = fmaxf(a, s_max[i]);
  const BlockScale b = block_scale(a);
  if (threadIdx.x == 0) p.scale[(e * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] = b.scale;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    if (r >= p.n || c >= p.k) continue;
    float x[8];
    bf16x8_to_float(v[i], x);
    uint2 o;
    o.x = to_e4m3x2(coded(x[0], b.inv), coded(x[1], b.inv)) | to_e4m3x2(coded(x[2], b.inv), coded(x[3], b.inv)) << 16;
    o.y = to_e4m3x2(coded(x[4], b.inv), coded(x[5], b.inv)) | to_e4m3x2(coded(x[6], b.inv), coded(x[7], b.inv)) << 16;
    *reinterpret_cast<uint2*>(p.q + (e * p.n + r) * p.k + c) = o;
  }
}

unsigned grid_of(int rows, int per) { return (unsigned)((rows + per - 1) / per); }
// At most as many CTAs as the SMs hold at once, `each` to an SM (by registers).
dim3 grid_within(int rows, int per, int each) {
  const unsigned need = grid_of(rows, per), most = (unsigned)(sm_count() * each);
  return dim3(need < most ? need : most);
}

}  // namespace

cudaError_t launch_dispatch(DispatchParams p, cudaStream_t s) {
  p.segments = (p.d + kPiece - 1) / kPiece;
  const Split sp = split_of(p.segments);
  const dim3 grid(grid_of(p.T, sp.rows));
  return p.out.format == MOE_ROWS_E4M3 ? launch_pdl(dispatch_kernel<true>, grid, kThreads, 0, 1, s, p, sp.warps)
                                       : launch_pdl(dispatch_kernel<false>, grid, kThreads, 0, 1, s, p, sp.warps);
}

cudaError_t launch_combine(CombineParams p, cudaStream_t s) {
  p.segments = (p.d + kCombinePiece - 1) / kCombinePiece;
  const Split sp = split_of(p.segments);
  return launch_pdl(combine_kernel, grid_within(p.T, sp.rows, 4), kThreads, 0, 1, s, p, sp.warps);
}

cudaError_t launch_combine_grad(const CombineGradParams& p, cudaStream_t s) {
  const int tokens = p.k < kWarps ? kWarps / p.k : 1;
  const dim3 grid = grid_within(p.T, tokens, 1024 / (32 * p.k * tokens));
  return p.dys.format == MOE_ROWS_E4M3
             ? launch_pdl(combine_grad_kernel<true>, grid, 32 * p.k * tokens, 0, 1, s, p, tokens)
             : launch_pdl(combine_grad_kernel<false>, grid, 32 * p.k * tokens, 0, 1, s, p, tokens);
}

cudaError_t launch_swiglu(SwigluParams p, bool grad, cudaStream_t s) {
  const bool e4m3 = p.out.format == MOE_ROWS_E4M3, whole = p.inter % kScaleBlock == 0;
  p.segments = ((grad && !whole ? 2 * p.inter : p.inter) + kPiece - 1) / kPiece;
  const Split sp = split_of(p.segments);
  const dim3 grid = grid_within(p.rows, sp.rows, grad ? 3 : 4);
  if (!grad)
    return e4m3 ? launch_pdl(swiglu_kernel<true>, grid, kThreads, 0, 1, s, p, sp.warps)
                : launch_pdl(swiglu_kernel<false>, grid, kThreads, 0, 1, s, p, sp.warps);
  if (whole)
    return e4m3 ? launch_pdl(swiglu_grad_kernel<true, true>, grid, kThreads, 0, 1, s, p, sp.warps)
                : launch_pdl(swiglu_grad_kernel<false, true>, grid, kThreads, 0, 1, s, p, sp.warps);
  return e4m3 ? launch_pdl(swiglu_grad_kernel<true, false>, grid, kThreads, 0, 1, s, p, sp.warps)
              : launch_pdl(swiglu_grad_kernel<false, false>, grid, kThreads, 0, 1, s, p, sp.warps);
}

cudaError_t launch_quant_weights(const QuantWeightsParams& p, int n_experts, cudaStream_t s) {
  const dim3 grid((p.k + kScaleBlock - 1) / kScaleBlock, (p.n + kScaleBlock - 1) / kScaleBlock, n_experts);
  quant_weights_kernel<<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace moe
