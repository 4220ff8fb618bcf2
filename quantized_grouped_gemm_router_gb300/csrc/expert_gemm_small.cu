// moe_gemm_e4m3 for few rows (a token's experts, a small decode batch): bound by the weights' bytes and by latency.
//
// A warp takes 16 columns of the output (16 rows of the weight matrix) and a slice of the inputs, for up to 8
// rows of one expert; the 8 warps of a CTA split the inputs (and, where they are short, the columns) and add their
// sums in a fixed order. mma.sync with the weights as its 16-row operand: a lane loads 16 consecutive bytes of a
// row at a time and hands them to two MMAs, rows and weights permuted alike along the inputs, so that every byte
// comes straight from memory into the register it is used from. A block of 128 is four MMAs into a fresh
// accumulator, which is then scaled and added in fp32.
#include "expert_device.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kRows = 8;     // rows of an expert to a CTA: the MMA's columns
constexpr int kCols = 16;    // output columns of a warp

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct Group {
  int expert, row0, rows;  // rows == 0: none
};

// The q-th group of up to kRows rows of one expert, counted over the experts. All threads of the CTA call it; a
// thread looks at kMaxExperts / kThreads consecutive experts at most.
__device__ __forceinline__ Group find_group(const ProductParams& p, int q, bool report) {
  __shared__ int s_sum[kWarps];
  __shared__ Group s_group;
  if (!p.offsets) return {0, q * kRows, min(kRows, p.rows - q * kRows)};
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.n_experts + kThreads - 1) / kThreads, e0 = threadIdx.x * per, e1 = min(e0 + per, p.n_experts);
  int sum = 0;
  bool bad = false;
  for (int e = e0; e < e1; ++e) {
    const int lo = __ldg(p.offsets + e), hi = __ldg(p.offsets + e + 1);
    const bool wrong = lo < 0 || hi < lo || hi > p.rows;
    bad |= wrong;
    if (!wrong) sum += (hi - lo + kRows - 1) / kRows;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_sum[warp] = incl;
  if (threadIdx.x == 0) s_group = {0, 0, 0};
  bad = __syncthreads_or(bad);  // then there are no groups at all
  if (report && bad && threadIdx.x == 0) raise_index(p.hdr);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) q -= w < warp ? s_sum[w] : 0;
  q -= incl - sum;
  if (!bad && q >= 0 && q < sum)
    for (int e = e0; e < e1; ++e) {
      const int lo = __ldg(p.offsets + e), hi = __ldg(p.offsets + e + 1), n = (hi - lo + kRows - 1) / kRows;
      if (q >= 0 && q < n) s_group = {e, lo + q * kRows, min(kRows, hi - lo - q * kRows)};
      q -= n;
    }
  __syncthreads();
  return s_group;
}

__device__ __forceinline__ uint4 load_bytes(const uint8_t* p, bool there) {
  return there ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ uint4 stream_bytes(const uint8_t* p, bool there) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (there)
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(p));
  return v;
}

// slices: warps that share a group of 16 columns, a power of two.
__global__ void __launch_bounds__(kThreads, 4) product_small_kernel(const __grid_constant__ ProductParams p, int slices) {
  __shared__ float s_part[kWarps][4][32];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const Group grp = find_group(p, blockIdx.y, blockIdx.x == 0 && blockIdx.y == 0);
  if (grp.rows <= 0) return;  // the whole CTA
  const int per_cta = kWarps / slices, slice = warp % slices;
  const int col0 = (blockIdx.x * per_cta + warp / slices) * kCols;
  float acc[4] = {};
  if (col0 < p.outc) {  // the columns are a multiple of 16
    const uint8_t* w0 = p.wq + ((int64_t)grp.expert * p.n + col0 + g) * p.k + t * 16;
    const uint8_t* w8 = w0 + (int64_t)8 * p.k;
    const float* ws = p.wscale + ((int64_t)grp.expert * p.out_blocks + col0 / kScaleBlock) * p.in_blocks;
    const bool has = g < grp.rows;
    const uint8_t* a = static_cast<const uint8_t*>(p.a.p) + (int64_t)(grp.row0 + (has ? g : 0)) * p.a.stride + t * 16;
    // scales of the two rows whose sums this lane holds
    const float* as = p.a.scale + (int64_t)(grp.row0 + min(2 * t, grp.rows - 1)) * p.a.scale_stride;
    const int64_t next = 2 * t + 1 < grp.rows ? p.a.scale_stride : 0;
    const int kb0 = (int)((int64_t)slice * p.in_blocks / slices), kb1 = (int)((int64_t)(slice + 1) * p.in_blocks / slices);
    // Two blocks of the inputs, each a set of registers of its own: one is on its way while the other is used. (With copies
    // out of one set, loads waited for the block before and registers spilled: 8.2 us where this takes 7.2.)
    struct Block {
      uint4 w0[2], w8[2], a[2];
    };
    auto load = [&](Block& b, int kb) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = kb * kScaleBlock + j * 64;
        const bool there = kb < kb1 && i + t * 16 < p.in;  // 16 bytes lie within the row or behind it
        b.w0[j] = stream_bytes(w0 + i, there);
        b.w8[j] = stream_bytes(w8 + i, there);
        b.a[j] = load_bytes(a + i, there && has);
      }
    };
    auto add = [&](const Block& b, int kb) {
      const float fw = __ldg(ws + kb), f0 = __ldg(as + kb) * fw, f1 = __ldg(as + next + kb) * fw;
      float c[4] = {};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mma_e4m3(c, b.w0[j].x, b.w8[j].x, b.w0[j].y, b.w8[j].y, b.a[j].x, b.a[j].y);
        mma_e4m3(c, b.w0[j].z, b.w8[j].z, b.w0[j].w, b.w8[j].w, b.a[j].z, b.a[j].w);
      }
      acc[0] = fmaf(f0, c[0], acc[0]);
      acc[1] = fmaf(f1, c[1], acc[1]);
      acc[2] = fmaf(f0, c[2], acc[2]);
      acc[3] = fmaf(f1, c[3], acc[3]);
    };
    Block even, odd;
    load(even, kb0);
#pragma unroll 1
    for (int kb = kb0; kb < kb1; kb += 2) {
      load(odd, kb + 1);
      add(even, kb);
      if (kb + 1 >= kb1) break;
      load(even, kb + 2);
      add(odd, kb + 1);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s_part[warp][i][lane] = acc[i];
  __syncthreads();
  // Two neighbouring columns of a row to a thread: columns c, c + 1 are MMA rows g and g + 1, lanes 4 apart.
  for (int o = threadIdx.x; o < per_cta * 8 * kRows; o += kThreads) {
    const int c = o % 8 * 2, row = o / 8 % kRows, unit = o / (8 * kRows);
    const int col = (blockIdx.x * per_cta + unit) * kCols + c;
    if (row >= grp.rows || col >= p.outc) continue;
    const int l = (c & 7) * 4 + row / 2, i = (c >= 8 ? 2 : 0) + (row & 1);
    float lo = 0.f, hi = 0.f;
    for (int s = 0; s < slices; ++s) {
      lo += s_part[unit * slices + s][i][l];
      hi += s_part[unit * slices + s][i][l + 4];
    }
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out.p) + (int64_t)(grp.row0 + row) * p.out.stride + col) =
        to_bf16x2(lo, hi);
  }
}

struct SmallGrid {
  int slices, groups;
  int64_t columns;  // CTAs side by side
};
SmallGrid small_grid(const ProductParams& p) {
  SmallGrid g;
  g.slices = 1;
  while (g.slices < kWarps && 2 * g.slices <= p.in_blocks) g.slices *= 2;
  const int per_cta = kWarps / g.slices * kCols;
  // every expert that has rows has a group that is not full, the others are full ones
  const int most = p.n_experts < p.rows ? p.n_experts : p.rows;
  g.groups = (p.rows - most) / kRows + most;
  g.columns = (p.outc + per_cta - 1) / per_cta;
  return g;
}
}  // namespace

// Up to 8 rows, while all CTAs are resident at once. Here and in the other kernel, us: 2048 x 2048 3.3 and 6.9, 8192 x 8192
// 14.4 and 19.1, 1024 x 16384 13.0 and 32.5, a token's 8 of 256 experts of 1024 x 2048 7.2 and 7.7 (of 2048 x 512 5.4 and
// 5.1, the closest call); but past that number, in waves of loads and latency, 16384 x 1024 6.7 and 5.9, 8 rows over
// 8 experts of 4096 x 2048 14.9 and 12.3.
bool product_is_small(const ProductParams& p, int sms) {
  if (p.transposed || p.rows > kRows) return false;
  const SmallGrid g = small_grid(p);
  return g.columns * g.groups <= 4 * (int64_t)sms;
}

cudaError_t launch_product_small(const ProductParams& p, cudaStream_t s) {
  const SmallGrid g = small_grid(p);
  return launch_pdl(product_small_kernel, dim3((unsigned)g.columns, g.groups), kThreads, 0, 1, s, p, g.slices);
}

}  // namespace moe
