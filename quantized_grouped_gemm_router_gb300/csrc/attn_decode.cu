// moe_attn_decode: attention of one new token per sequence over the paged cache.
//
// Every cache row is read once and used by the G query heads of its key-value head: G flops per byte
// in bf16, so HBM bounds it. Two things make it run at that rate:
//
//  * Equal work. All sequences' caches are cut into tiles of TR rows (of one head each), and the
//    tiles, in the order (sequence, head, position), into equal runs, one per warp of a grid of one CTA
//    per SM, whatever the lengths. A warp carries a running softmax (m, l, O in registers) through a
//    sequence's tiles; a sequence that it holds from its first to its last tile it finishes itself.
//    The other partial results are joined by weight 2^(m - max m), in tile order: those of one CTA
//    through shared memory, those of several CTAs through the workspace, by the CTA that finishes last.
//  * Loads in flight. Each warp has a ring of its own, filled by 16-byte asynchronous copies two tiles
//    ahead (8 warps x 2 x 8 KB per SM), with no barrier between warps. The page numbers of a tile are
//    read one tile earlier still. Rows past a sequence's end are filled with zeros, so what lies there
//    is never used.
//
// The products run on mma.sync (16 heads x 8 keys x 16): a group's heads fill at most 16 rows, and the
// matrix work is a small share of the copy's time. In e4m3 the codes become fp16 (exactly), the query
// row fp16 times a power of two, and the softmax weights fp16; in bf16 all operands are bf16.
#include <cuda_fp8.h>

#include "attn_device.cuh"
#include "attn_ptx.cuh"

namespace moe {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.f;  // O is scaled down when a maximum has grown by more than 2^8
constexpr int kMaxGroups = kAttnMaxSeqs / 32;

template <int D, bool E4M3>
struct Cfg {
  static constexpr int RB = D * (E4M3 ? 1 : 2);     // bytes of a cache row
  static constexpr int TR = RB <= 128 ? 32 : 16;    // rows of a tile
  static constexpr int NW = RB == 512 ? 4 : 8;      // warps
  static constexpr int kTile = 2 * TR * RB;         // K rows, then V rows
  static constexpr int kStages = kTile == 4096 ? 4 : 3;
  static constexpr int kRing = kStages * kTile;     // per warp
  static constexpr int kStride = D + 8;             // floats between the heads of a partial O (bank spread)
  static constexpr int kSmem = NW * kRing;
  static_assert(16 * kStride * 4 <= kRing, "a partial O fits its warp's ring");
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
// c += a b; bf16 or fp16 operands. HALF: rows 8..15 of a are zero and their sums are not kept.
template <bool FP16, bool HALF>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  float x = 0.f, y = 0.f;
  float& c2 = HALF ? x : c[2];
  float& c3 = HALF ? y : c[3];
  const uint32_t a1 = HALF ? 0u : a[1], a2 = HALF ? a[1] : a[2], a3 = HALF ? 0u : a[3];
  if (FP16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c2), "+f"(c3)
                 : "r"(a[0]), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c2), "+f"(c3)
                 : "r"(a[0]), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
// The two e4m3 codes in the low (0) or high (1) half of w as fp16.
template <int HI>
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t w) {
  uint32_t r;
  if (HI)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// The tiles in order: sequences, each with `units` (key-value head, 16 query heads of its group) in
// turn, each with the sequence's tiles. Lengths are read 32 sequences at a time, one per lane. Every
// member but len32 is the same in all lanes.
template <int TR>
struct Walk {
  int b, u, t, len, nt;  // sequence, unit, tile; the sequence's length and tiles
  int base, len32;       // this lane's length: of sequence base + lane

  __device__ __forceinline__ static int length(const AttnDecodeParams& p, int b) {
    if (b >= p.n_seqs) return 0;
    const int n = __ldg(p.lens + b);
    return n < 0 || (int64_t)n > (int64_t)p.table_width * p.page_size ? 0 : n;
  }
  __device__ __forceinline__ void group(const AttnDecodeParams& p, int g) {
    base = g * 32;
    len32 = length(p, base + (threadIdx.x & 31));
  }
  __device__ __forceinline__ void seq(int lane) {
    b = base + lane;
    len = __shfl_sync(~0u, len32, lane);
    nt = (len + TR - 1) / TR;
  }
  // the tile `at` (counted from the group's first)
  __device__ __forceinline__ void start(const AttnDecodeParams& p, int g, int64_t at, int units) {
    group(p, g);
    const int lane = threadIdx.x & 31;
    const int tiles = (len32 + TR - 1) / TR;
    int64_t sum = (int64_t)tiles * units;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int64_t y = __shfl_up_sync(~0u, sum, x);
      if (lane >= x) sum += y;
    }
    const int src = __ffs(__ballot_sync(~0u, sum > at)) - 1;
    const int64_t before = __shfl_sync(~0u, sum - (int64_t)tiles * units, src);
    seq(src);
    u = (int)((at - before) / nt);
    t = (int)((at - before) % nt);
  }
  __device__ __forceinline__ void next(const AttnDecodeParams& p, int units) {
    if (++t < nt) return;
    t = 0;
    if (++u < units) return;
    u = 0;
    unsigned rest = __ballot_sync(~0u, len32 > 0) & ~((2u << (b - base)) - 1);
    while (!rest) {
      if (base + 32 >= p.n_seqs) return;  // past the last tile
      group(p, base / 32 + 1);
      rest = __ballot_sync(~0u, len32 > 0);
    }
    seq(__ffs(rest) - 1);
  }
};

// One partial result: rows of O (unnormalised), their maxima (log2, scaled) and sums.
struct Part {
  const float* o;
  const float* ml;  // [16] m, [16] l
};

struct PartInfo {
  int64_t seg;  // b * units + u, -1: none
  int first, last, len;
  const float* o;
};

// Joins n partial results into the final rows of (b, u), or into another partial result (to != nullptr,
// to_ml). All threads of the CTA; `get(i)` gives partial i, in tile order.
template <int D, int TH, class Get>
__device__ __forceinline__ void join(const AttnDecodeParams& p, int64_t seg, int units, int nhb, int n, Get get, float* to,
                                     float* to_ml, int stride, float* s_w, float vscale_or) {
  const int b = (int)(seg / units), u = (int)(seg % units), kvh = u / nhb, h0 = (u % nhb) * 16;
  const int rows = min(16, p.group - h0);
  // thread x: row x / (TH / 16)... every thread of a row's share computes that row's statistics itself
  constexpr int kV = D / 4;  // float4 per row
  for (int e = threadIdx.x; e < rows * kV; e += TH) {
    const int r = e / kV, c = e % kV;
    float m = -INFINITY;
    for (int i = 0; i < n; ++i) m = fmaxf(m, get(i).ml[r]);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const Part q = get(i);
      const float w = ex2(q.ml[r] - base);
      const float4 x = *reinterpret_cast<const float4*>(q.o + r * stride + c * 4);
      l = fmaf(w, q.ml[16 + r], l);
      acc.x = fmaf(w, x.x, acc.x);
      acc.y = fmaf(w, x.y, acc.y);
      acc.z = fmaf(w, x.z, acc.z);
      acc.w = fmaf(w, x.w, acc.w);
    }
    if (to) {
      *reinterpret_cast<float4*>(to + r * stride + c * 4) = acc;
      if (c == 0) {
        to_ml[r] = m;
        to_ml[16 + r] = l;
      }
    } else {
      const int64_t row = (int64_t)b * p.hq + kvh * p.group + h0 + r;
      const float inv = l == 0.f ? 0.f : vscale_or / l;
      const bool none = l == 0.f;
      *reinterpret_cast<uint2*>(p.o + row * D + c * 4) =
          none ? make_uint2(0u, 0u) : make_uint2(bf16x2_rn(acc.x * inv, acc.y * inv), bf16x2_rn(acc.z * inv, acc.w * inv));
      if (c == 0 && p.lse) p.lse[row] = none ? -INFINITY : m * kLn2 + logf(l);
    }
  }
}

template <int D, bool E4M3, bool HALF>
__global__ void __launch_bounds__(32 * Cfg<D, E4M3>::NW, 1) attn_decode_kernel(const __grid_constant__ AttnDecodeParams p) {
  using C = Cfg<D, E4M3>;
  constexpr int RB = C::RB, TR = C::TR, NW = C::NW, TH = 32 * NW, NB = TR / 8, ND = D / 8;
  constexpr int AR = HALF ? 2 : 4, CR = HALF ? 2 : 4;  // registers of an A and a C fragment
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t s_before[kMaxGroups + 1];  // tiles before each group of 32 sequences
  __shared__ PartInfo s_part[NW][2];
  __shared__ float s_ml[NW][2][32];
  __shared__ int s_last;

  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int nhb = (p.group + 15) / 16, units = p.hkv * nhb;

  // ---- the tiles of all sequences
  const int groups = (p.n_seqs + 31) / 32;
  for (int g = warp; g < groups; g += NW) {
    const int b = g * 32 + lane;
    const int n = Walk<TR>::length(p, b);
    if (blockIdx.x == 0 && b < p.n_seqs && n != __ldg(p.lens + b)) raise_bad_index(p.hdr);
    int64_t tiles = (n + TR - 1) / TR;
#pragma unroll
    for (int x = 16; x; x >>= 1) tiles += __shfl_xor_sync(~0u, tiles, x);
    if (lane == 0) s_before[g + 1] = tiles * units;
  }
  // rows of empty sequences
  for (int b = blockIdx.x; b < p.n_seqs; b += gridDim.x) {
    if (Walk<TR>::length(p, b) > 0) continue;
    for (int e = threadIdx.x; e < p.hq * (D / 8); e += TH)
      *reinterpret_cast<uint4*>(p.o + (int64_t)b * p.hq * D + e * 8) = make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int h = threadIdx.x; h < p.hq; h += TH) p.lse[(int64_t)b * p.hq + h] = -INFINITY;
  }
  if (threadIdx.x < NW * 2) s_part[threadIdx.x / 2][threadIdx.x & 1].seg = -1;
  __syncthreads();
  if (warp == 0) {  // inclusive sums, four groups per lane
    int64_t v[kMaxGroups / 32], sum = 0;
#pragma unroll
    for (int i = 0; i < kMaxGroups / 32; ++i) {
      const int g = lane * (kMaxGroups / 32) + i;
      sum += g < groups ? s_before[g + 1] : 0;
      v[i] = sum;
    }
    int64_t inc = sum;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int64_t y = __shfl_up_sync(~0u, inc, x);
      if (lane >= x) inc += y;
    }
#pragma unroll
    for (int i = 0; i < kMaxGroups / 32; ++i) {
      const int g = lane * (kMaxGroups / 32) + i;
      if (g < groups) s_before[g + 1] = inc - sum + v[i];
    }
    if (lane == 0) s_before[0] = 0;
  }
  __syncthreads();
  const int64_t total = s_before[groups];
  const int64_t ctas = min((int64_t)gridDim.x, (total + NW - 1) / NW);  // a tile per warp at least
  if (blockIdx.x >= ctas) return;
  const int64_t cta_lo = total * blockIdx.x / ctas, cta_hi = total * (blockIdx.x + 1) / ctas;
  const int64_t lo = cta_lo + (cta_hi - cta_lo) * warp / NW, hi = cta_lo + (cta_hi - cta_lo) * (warp + 1) / NW;
  const int n = (int)(hi - lo);

  uint8_t* ring = smem + warp * C::kRing;
  const uint32_t ring_s = smem_u32(ring);
  float* scratch = p.scratch + (int64_t)(blockIdx.x * NW + warp) * (16 * C::kStride);

  if (n > 0) {
    int g = 0;
    for (int x = lane; x < groups; x += 32) g += s_before[x + 1] <= lo;
#pragma unroll
    for (int x = 16; x; x >>= 1) g += __shfl_xor_sync(~0u, g, x);
    Walk<TR> w, ld;
    w.start(p, g, lo - s_before[g], units);
    ld = w;

    // ---- copies: the pages of the next tile to copy are already in `page`
    const auto page_of = [&]() {
      const int pos = ld.t * TR + (lane & (TR - 1));
      return pos < ld.len ? __ldg(p.table + (int64_t)ld.b * p.table_width + (unsigned)pos / (unsigned)p.page_size) : -1;
    };
    int page = page_of();
    int left = n;  // tiles not yet copied
    const auto issue = [&](int stage) {
      if (left > 0) {
        const int pos = ld.t * TR + (lane & (TR - 1));
        int cell = -1;  // this lane's cache row
        if (pos < ld.len) {
          if (page >= 0 && page < p.n_pages)
            cell = (page * p.hkv + ld.u / nhb) * p.page_size + (int)((unsigned)pos % (unsigned)p.page_size);
          else
            raise_bad_index(p.hdr);
        }
        const uint32_t dst = ring_s + stage * C::kTile;
        constexpr int CPR = RB / 16, RPI = 32 / CPR;  // copies per row, rows per instruction
        const int chunk = lane % CPR;
#pragma unroll
        for (int i = 0; i < TR / RPI; ++i) {
          const int r = i * RPI + lane / CPR;
          const int c = __shfl_sync(~0u, cell, r);
          const int64_t off = (int64_t)max(c, 0) * RB + chunk * 16;
          const uint32_t at = dst + r * RB + ((chunk ^ (RB == 64 ? (r >> 1) & 3 : r & 7)) << 4);
          cp16(at, static_cast<const uint8_t*>(p.kc) + off, c >= 0);
          cp16(at + TR * RB, static_cast<const uint8_t*>(p.vc) + off, c >= 0);
        }
        if (--left > 0) {
          ld.next(p, units);
          page = page_of();
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int s = 0; s < C::kStages - 1; ++s) issue(s);

    uint32_t q[D / 16][AR];
    float o[ND][CR];
    float m[CR / 2], mc[CR / 2], l[CR / 2], cr[CR / 2];  // per row (lane / 4, and + 8): maximum, scaled, sum, scale
    bool fresh = true, from_start = false;
    int out = 0, stage = 0, fill = C::kStages - 1;
    for (int i = 0; i < n; ++i) {
      issue(fill);
      if (++fill == C::kStages) fill = 0;
      const int kvh = w.u / nhb, h0 = (w.u % nhb) * 16, rows = min(16, p.group - h0);
      if (fresh) {
        // ---- a new sequence or head: its query rows as A fragments
        fresh = false;
        from_start = w.t == 0;
#pragma unroll
        for (int x = 0; x < ND; ++x)
#pragma unroll
          for (int y = 0; y < CR; ++y) o[x][y] = 0.f;
#pragma unroll
        for (int y = 0; y < CR / 2; ++y) {
          m[y] = -INFINITY;
          mc[y] = 0.f;
          l[y] = 0.f;
          cr[y] = p.scale * kLog2e * (E4M3 ? __ldg(p.k_scale + kvh) : 1.f);
          const int r = lane / 4 + 8 * y;
          const uint16_t* src = p.q.p + (int64_t)w.b * p.q.token_stride + (int64_t)(kvh * p.group + h0 + r) * p.q.head_stride;
          uint32_t v[D / 16][2];
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              // bf16: k step ks holds values 16 ks + (0..15); e4m3: see the K fragments below
              const int d = E4M3 ? (ks / 4) * 64 + (lane & 3) * 16 + (ks & 3) * 4 + half * 2 : ks * 16 + (lane & 3) * 2 + half * 8;
              v[ks][half] = r < rows ? __ldg(reinterpret_cast<const uint32_t*>(src + d)) : 0u;
            }
          if (E4M3) {
            // fp16 has bf16's precision but not its range: the row times a power of two that brings its
            // largest magnitude to 2^14
            uint32_t big = 0;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                big = max(big, v[ks][half] & 0x7FFFu);
                big = max(big, (v[ks][half] >> 16) & 0x7FFFu);
              }
            big = max(big, __shfl_xor_sync(~0u, big, 1));
            big = max(big, __shfl_xor_sync(~0u, big, 2));
            const int e = (int)(big >> 7) - 127;  // exponent of the largest
            const int up = big == 0 || big >= 0x7F80u ? 0 : min(14 - e, 126);
            const float f = __uint_as_float((uint32_t)(127 + up) << 23);
            cr[y] *= __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
              for (int half = 0; half < 2; ++half)
                v[ks][half] = f16x2_rn(__uint_as_float(v[ks][half] << 16) * f, __uint_as_float(v[ks][half] & 0xFFFF0000u) * f);
          }
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            q[ks][y] = v[ks][0];
            q[ks][y + AR / 2] = v[ks][1];
          }
        }
      }

      cp_wait<C::kStages - 1>();
      __syncwarp();
      const uint32_t ks_ = ring_s + stage * C::kTile, vs_ = ks_ + TR * RB;

      // ---- scores. C fragment nb: rows lane / 4 (+ 8), columns 2 (lane % 4), + 1, that is keys
      //   bf16: 8 nb + column; e4m3: 8 nb + lane % 4 and 8 nb + lane % 4 + 4 (bank spread of the row reads)
      float s[NB][CR];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float s2[CR];
#pragma unroll
        for (int y = 0; y < CR; ++y) s[nb][y] = s2[y] = 0.f;
        if (!E4M3) {
          const int x = (lane >> 3) ^ (lane & 7);
          const uint32_t row = ks_ + (nb * 8 + (lane & 7)) * RB;
#pragma unroll
          for (int kp = 0; kp < D / 32; ++kp) {
            uint32_t b[4];
            ldsm4(row + ((kp * 64) ^ (x << 4)), b);
            mma<false, HALF>(s[nb], q[2 * kp], b[0], b[1]);
            mma<false, HALF>(s2, q[2 * kp + 1], b[2], b[3]);
          }
        } else {
          // a lane reads 16 codes of one key: values 64 i + 16 (lane % 4) + 0..15 serve four k steps
          const int r = nb * 8 + (lane >> 3) + 4 * ((lane >> 2) & 1);
#pragma unroll
          for (int i4 = 0; i4 < D / 64; ++i4) {
            const int chunk = i4 * 4 + (lane & 3);
            const uint4 b = lds128(ks_ + r * RB + ((chunk ^ (RB == 64 ? (r >> 1) & 3 : r & 7)) << 4));
            mma<true, HALF>(s[nb], q[4 * i4], e4m3x2_f16<0>(b.x), e4m3x2_f16<1>(b.x));
            mma<true, HALF>(s2, q[4 * i4 + 1], e4m3x2_f16<0>(b.y), e4m3x2_f16<1>(b.y));
            mma<true, HALF>(s[nb], q[4 * i4 + 2], e4m3x2_f16<0>(b.z), e4m3x2_f16<1>(b.z));
            mma<true, HALF>(s2, q[4 * i4 + 3], e4m3x2_f16<0>(b.w), e4m3x2_f16<1>(b.w));
          }
        }
#pragma unroll
        for (int y = 0; y < CR; ++y) s[nb][y] += s2[y];
      }
      const int lim = w.len - w.t * TR;
      if (lim < TR) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int y = 0; y < CR; ++y) {
            const int key = nb * 8 + (E4M3 ? (lane & 3) + 4 * (y & 1) : (lane & 3) * 2 + (y & 1));
            if (key >= lim) s[nb][y] = -INFINITY;
          }
      }

      // ---- running softmax
      bool grown = false;
      float mx[CR / 2];
#pragma unroll
      for (int y = 0; y < CR / 2; ++y) {
        mx[y] = -INFINITY;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mx[y] = fmaxf(mx[y], fmaxf(s[nb][2 * y], s[nb][2 * y + 1]));
        mx[y] = fmaxf(mx[y], __shfl_xor_sync(~0u, mx[y], 1));
        mx[y] = fmaxf(mx[y], __shfl_xor_sync(~0u, mx[y], 2));
        grown |= mx[y] * cr[y] > mc[y] + kRescaleLog2 || (m[y] == -INFINITY && mx[y] > m[y]);
      }
      if (__any_sync(~0u, grown)) {
#pragma unroll
        for (int y = 0; y < CR / 2; ++y) {
          const float m2 = fmaxf(m[y], mx[y]), mc2 = m2 == -INFINITY ? 0.f : m2 * cr[y];
          const float f = m[y] == -INFINITY ? 0.f : ex2(mc[y] - mc2);
          m[y] = m2;
          mc[y] = mc2;
          l[y] *= f;
#pragma unroll
          for (int x = 0; x < ND; ++x) {
            o[x][2 * y] *= f;
            o[x][2 * y + 1] *= f;
          }
        }
      }
      uint32_t a[TR / 16][AR];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int y = 0; y < CR / 2; ++y) {
          const float p0 = ex2(fmaf(s[nb][2 * y], cr[y], -mc[y])), p1 = ex2(fmaf(s[nb][2 * y + 1], cr[y], -mc[y]));
          l[y] += p0 + p1;
          a[nb / 2][(nb & 1) * (AR / 2) + y] = E4M3 ? f16x2_rn(p0, p1) : bf16x2_rn(p0, p1);
        }

      // ---- O += P V. C fragment x holds columns
      //   bf16: 8 x + 2 (lane % 4), + 1;  e4m3, D = 64: 16 (lane % 4) + x and + 8;
      //   e4m3, D >= 128: 128 (x / 16) + 16 (lane % 4) + x % 16 and + 64
#pragma unroll
      for (int kb = 0; kb < TR / 16; ++kb) {
        if (!E4M3) {
          const int x = (lane >> 4) ^ (lane & 7);
          const uint32_t row = vs_ + (kb * 16 + (lane & 15)) * RB;
#pragma unroll
          for (int dp = 0; dp < ND / 2; ++dp) {
            uint32_t b[4];
            ldsm4t(row + ((dp * 32) ^ (x << 4)), b);
            mma<false, HALF>(o[2 * dp], a[kb], b[0], b[1]);
            mma<false, HALF>(o[2 * dp + 1], a[kb], b[2], b[3]);
          }
        } else if (D == 64) {
          uint2 v[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int r = kb * 16 + (lane & 3) + 4 * y, chunk = lane >> 3;
            v[y] = lds64(vs_ + r * RB + ((chunk ^ ((r >> 1) & 3)) << 4) + ((lane >> 2) & 1) * 8);
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t r0 = x ? v[0].y : v[0].x, r1 = x ? v[1].y : v[1].x, r2 = x ? v[2].y : v[2].x, r3 = x ? v[3].y : v[3].x;
            const uint32_t e01 = __byte_perm(r0, r1, 0x5140), e23 = __byte_perm(r0, r1, 0x7362);
            const uint32_t f01 = __byte_perm(r2, r3, 0x5140), f23 = __byte_perm(r2, r3, 0x7362);
            mma<true, HALF>(o[4 * x], a[kb], e4m3x2_f16<0>(e01), e4m3x2_f16<0>(f01));
            mma<true, HALF>(o[4 * x + 1], a[kb], e4m3x2_f16<1>(e01), e4m3x2_f16<1>(f01));
            mma<true, HALF>(o[4 * x + 2], a[kb], e4m3x2_f16<0>(e23), e4m3x2_f16<0>(f23));
            mma<true, HALF>(o[4 * x + 3], a[kb], e4m3x2_f16<1>(e23), e4m3x2_f16<1>(f23));
          }
        } else {
#pragma unroll
          for (int dq = 0; dq < D / 128; ++dq) {
            uint4 v[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int r = kb * 16 + (lane & 3) + 4 * y, chunk = dq * 8 + (lane >> 3) + 4 * ((lane >> 2) & 1);
              v[y] = lds128(vs_ + r * RB + ((chunk ^ (r & 7)) << 4));
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const auto word = [&](const uint4& y) { return x == 0 ? y.x : x == 1 ? y.y : x == 2 ? y.z : y.w; };
              const uint32_t r0 = word(v[0]), r1 = word(v[1]), r2 = word(v[2]), r3 = word(v[3]);
              const uint32_t e01 = __byte_perm(r0, r1, 0x5140), e23 = __byte_perm(r0, r1, 0x7362);
              const uint32_t f01 = __byte_perm(r2, r3, 0x5140), f23 = __byte_perm(r2, r3, 0x7362);
              mma<true, HALF>(o[dq * 16 + 4 * x], a[kb], e4m3x2_f16<0>(e01), e4m3x2_f16<0>(f01));
              mma<true, HALF>(o[dq * 16 + 4 * x + 1], a[kb], e4m3x2_f16<1>(e01), e4m3x2_f16<1>(f01));
              mma<true, HALF>(o[dq * 16 + 4 * x + 2], a[kb], e4m3x2_f16<0>(e23), e4m3x2_f16<0>(f23));
              mma<true, HALF>(o[dq * 16 + 4 * x + 3], a[kb], e4m3x2_f16<1>(e23), e4m3x2_f16<1>(f23));
            }
          }
        }
      }
      if (++stage == C::kStages) stage = 0;
      __syncwarp();

      // ---- the end of a sequence's head, or of this warp's run
      const bool to_end = w.t == w.nt - 1;
      if (to_end || i == n - 1) {
        const bool whole = to_end && from_start, mid = i < n - 1;
        float* to = mid ? scratch : reinterpret_cast<float*>(ring);
        const float vs = E4M3 && whole ? __ldg(p.v_scale + kvh) : 1.f;
        if (!whole && !mid) {
          cp_wait<0>();  // the ring is idle: every copy has landed and been used
          __syncwarp();
        }
#pragma unroll
        for (int y = 0; y < CR / 2; ++y) {
          const int r = lane / 4 + 8 * y;
          float sum = l[y];
          sum += __shfl_xor_sync(~0u, sum, 1);
          sum += __shfl_xor_sync(~0u, sum, 2);
          const bool none = sum == 0.f;
          const float inv = whole ? (none ? 0.f : vs / sum) : 1.f;
          const int64_t row = (int64_t)w.b * p.hq + kvh * p.group + h0 + r;
          if (r < rows) {
            // pieces of values that lie together: 2 (bf16), 8 (e4m3)
            if (!E4M3) {
#pragma unroll
              for (int x = 0; x < ND; ++x) {
                const float u0 = whole && none ? 0.f : o[x][2 * y] * inv, u1 = whole && none ? 0.f : o[x][2 * y + 1] * inv;
                const int d = 8 * x + 2 * (lane & 3);
                if (whole)
                  *reinterpret_cast<uint32_t*>(p.o + row * D + d) = bf16x2_rn(u0, u1);
                else
                  *reinterpret_cast<float2*>(to + r * C::kStride + d) = make_float2(u0, u1);
              }
            } else {
#pragma unroll
              for (int z = 0; z < 2; ++z)
#pragma unroll
                for (int x = 0; x < ND; x += 4) {
                  const int d = D == 64 ? 16 * (lane & 3) + 8 * z + x : 128 * (x / 16) + 16 * (lane & 3) + 64 * z + x % 16;
                  float v[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k) v[k] = whole && none ? 0.f : o[x + k][2 * y + z] * inv;
                  if (whole)
                    *reinterpret_cast<uint2*>(p.o + row * D + d) = make_uint2(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]));
                  else
                    *reinterpret_cast<float4*>(to + r * C::kStride + d) = make_float4(v[0], v[1], v[2], v[3]);
                }
            }
            if ((lane & 3) == 0) {
              if (!whole) {
                s_ml[warp][out][r] = m[y] == -INFINITY ? -INFINITY : mc[y];
                s_ml[warp][out][16 + r] = sum;
              } else if (p.lse) {
                p.lse[row] = none ? -INFINITY : mc[y] * kLn2 + logf(sum);
              }
            }
          }
        }
        if (!whole) {
          if (lane == 0) s_part[warp][out] = PartInfo{(int64_t)w.b * units + w.u, from_start, to_end, w.nt, to};
          ++out;
        }
        fresh = true;
      }
      if (i < n - 1) w.next(p, units);
    }
    cp_wait<0>();
  }
  __syncthreads();

  // ---- partial results of this CTA's warps, in tile order; runs of one sequence's head are joined
  int pend = 0;
  int64_t pend_seg[2];
  int pend_first[2], pend_count[2];
  for (int x = 0; x < 2 * NW;) {
    const PartInfo a = s_part[x / 2][x & 1];
    if (a.seg < 0) {
      ++x;
      continue;
    }
    int list[2 * NW], cnt = 0, y = x;
    bool last = false;
    for (; y < 2 * NW; ++y) {
      const PartInfo b = s_part[y / 2][y & 1];
      if (b.seg < 0) continue;
      if (b.seg != a.seg) break;
      list[cnt++] = y;
      last = b.last;
    }
    x = y;
    const int kvh = (int)(a.seg % units) / nhb;
    const bool done = a.first && last;
    float* to = p.parts + (int64_t)(blockIdx.x * 2 + (a.first ? 1 : 0)) * (16 * C::kStride + 32);
    join<D, TH>(p, a.seg, units, nhb, cnt,
                [&](int i) {
                  const int z = list[i];
                  return Part{s_part[z / 2][z & 1].o, s_ml[z / 2][z & 1]};
                },
                done ? nullptr : to, to + 16 * C::kStride, C::kStride, nullptr,
                E4M3 ? __ldg(p.v_scale + kvh) : 1.f);
    if (!done) {
      // the CTAs that hold tiles of this head: its first tile is number `begin` of all
      const int b = (int)(a.seg / units), u = (int)(a.seg % units);
      int64_t begin = s_before[b / 32];
      for (int z = b & ~31; z < b; ++z) begin += (int64_t)((Walk<TR>::length(p, z) + TR - 1) / TR) * units;
      begin += (int64_t)u * a.len;
      const int64_t end = begin + a.len - 1;
      const int c0 = (int)(((begin + 1) * ctas - 1) / total), c1 = (int)(((end + 1) * ctas - 1) / total);
      pend_seg[pend] = a.seg;
      pend_first[pend] = c0;
      pend_count[pend] = c1 - c0 + 1;
      ++pend;
    }
  }
  if (pend == 0) return;
  __threadfence();
  for (int x = 0; x < pend; ++x) {
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      const int ticket = atomicAdd(p.counters + pend_first[x], 1);
      s_last = ticket == pend_count[x] - 1;
      if (s_last) p.counters[pend_first[x]] = 0;  // every CTA of this head has been here
      __threadfence();
    }
    __syncthreads();
    if (!s_last) continue;
    const int kvh = (int)(pend_seg[x] % units) / nhb, c0 = pend_first[x];
    join<D, TH>(p, pend_seg[x], units, nhb, pend_count[x],
                [&](int i) {
                  const float* at = p.parts + (int64_t)((c0 + i) * 2 + (i == 0 ? 1 : 0)) * (16 * C::kStride + 32);
                  return Part{at, at + 16 * C::kStride};
                },
                nullptr, nullptr, C::kStride, nullptr, E4M3 ? __ldg(p.v_scale + kvh) : 1.f);
  }
}

int num_sms() {
  static int n = [] {
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      v = 1;
    return v > kAttnMaxCtas ? kAttnMaxCtas : v > 0 ? v : 1;
  }();
  return n;
}

template <int D, bool E4M3, bool HALF>
cudaError_t launch(const AttnDecodeParams& p, cudaStream_t s) {
  using C = Cfg<D, E4M3>;
  static cudaError_t attr = cudaFuncSetAttribute(attn_decode_kernel<D, E4M3, HALF>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (attr != cudaSuccess) return attr;
  attn_decode_kernel<D, E4M3, HALF><<<num_sms(), 32 * C::NW, C::kSmem, s>>>(p);
  return cudaGetLastError();
}

template <int D, bool E4M3>
cudaError_t launch(const AttnDecodeParams& p, cudaStream_t s) {
  // up to 8 query heads per key-value head: half the rows of the matrix products are not kept
  return p.group <= 8 ? launch<D, E4M3, true>(p, s) : launch<D, E4M3, false>(p, s);
}

}  // namespace

cudaError_t launch_attn_decode(const AttnDecodeParams& p, int d, bool e4m3, cudaStream_t s) {
  if (d == 64) return e4m3 ? launch<64, true>(p, s) : launch<64, false>(p, s);
  if (d == 128) return e4m3 ? launch<128, true>(p, s) : launch<128, false>(p, s);
  return e4m3 ? launch<256, true>(p, s) : launch<256, false>(p, s);
}

}  // namespace moe
