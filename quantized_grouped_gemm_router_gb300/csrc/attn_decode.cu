// moe_attn_decode: attention of one new token per sequence over the paged cache.
//
// Every cache row is read once per 16 query heads of its key-value head (once for groups of up to 16, four times for
// 64) and used by all of these: up to 16 flops per byte in bf16, so HBM bounds it for groups of up to 8. Two things
// make it run at that rate:
//
//  * Equal work. All sequences' caches are cut into tiles of TR rows (of one head each), and the
//    tiles, in the order (sequence, head, position), into equal runs, one per warp of a grid of one CTA
//    per SM, whatever the lengths. A warp carries a running softmax (m, l, O in registers) through a
//    sequence's tiles; a sequence that it holds from its first to its last tile it finishes itself.
//    The other partial results are joined by weight 2^(m - max m), in tile order: those of one CTA
//    through shared memory, those of several CTAs by a second kernel, one CTA per head, which is
//    launched early (programmatic dependent launch) and waits for the first.
//  * Loads in flight. Each warp has a ring of its own, filled by 16-byte asynchronous copies a tile
//    ahead (8 warps x 8 KB per SM), with no barrier between warps. The page numbers of a tile are
//    read one tile earlier still. Rows past a sequence's end are filled with zeros, so what lies there
//    is never used.
//
// The products run on mma.sync with the cache as the 16-row operand and the heads as the 8 columns: S^T =
// K Q^T (16 keys x 8 heads), O^T = V^T P^T (16 values x 8 heads), P^T turned by movmatrix. A group of up
// to 8 heads thus wastes no rows; up to 16 heads take two column blocks over the same fragments of K
// and V, with twice the registers for q and O (heads of 256: four warps, spills of 58 bytes in bf16, 300 in
// e4m3). In e4m3 the codes become fp16 (exactly), the query row fp16 times a power of two, and the
// softmax weights fp16; in bf16 all operands are bf16.
//
// Measured (GB300): long batches add cache rows at the copy rate of HBM (75 sequences of 8300 rows, 2 heads of
// 128, bf16: 102 us, 6.2 TB/s, 92% of it); a call has 14 us beside that (18 in e4m3 at heads of 256): launch, three
// dependent loads before the first rows, SMs that end up to 5 us apart, the two joins. So 64 sequences of up to
// 16384 rows take 66 us (5.6 TB/s), one of 131071 rows 30 us (4.4 TB/s), 129 e4m3 sequences of up to 8191 rows of
// 256 75 us (4.6 TB/s), one of 511 rows 8.6 us. 32 sequences of up to 16384 rows of one head of 128 for 8, 16 and 64
// query heads: bf16 24, 29 and 74 us (floor 13.5), e4m3 19, 26 and 59 us (6.8); of 256: bf16 41, 72 and 224 us (27),
// e4m3 29, 52 and 134 us (13.5).
#include <cuda_fp8.h>

#include "attn_device.cuh"
#include "attn_ptx.cuh"

namespace moe {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.f;  // O is scaled down when a maximum has grown by more than 2^8
constexpr int kMaxGroups = kAttnMaxSeqs / 32;

template <int D, bool E4M3, int NH>
struct Cfg {
  static constexpr int RB = D * (E4M3 ? 1 : 2);     // bytes of a cache row
  static constexpr int TR = RB <= 128 ? 32 : 16;    // rows of a tile
  // Warps and ring stages: one tile ahead per warp, about 64 KB on their way per SM. More in flight is slower:
  // 75 sequences of 8300 rows (heads of 128, bf16) take 110 us with two tiles ahead, 104 with one. 64-byte rows
  // take most instructions for their bytes: 16 warps (43 against 55 us with 8).
  static constexpr int NW = RB == 512 ? (NH == 1 ? 6 : 4) : RB == 64 && NH == 1 ? 16 : 8;
  static constexpr int kTile = 2 * TR * RB;         // K rows, then V rows
  static constexpr int kStages = 2;
  // Weights are relative to 2^-kUp times the maximum's: fp16 has 11 bits down to 2^-14 only, so that e4m3 takes them
  // up to 2^15 (with the growth of 2^8) and keeps those of 2^-21 of the largest as exact as the others.
  static constexpr float kUp = E4M3 ? 7.f : 0.f;
  static constexpr int kRing = kStages * kTile;     // per warp
  static constexpr int kPartRows = 8 * NH * D;      // floats of a partial O
  static constexpr int kPart = 16 * D + 32;         // a CTA's partial result in the workspace: O, then 16 m and 16 l
  static constexpr int kSmem = NW * kRing;
  static_assert(kPartRows * 4 <= kRing, "a partial O fits its warp's ring");
};

// Where a partial O has value d of head h: heads follow each other, their columns turned so that the rows
// of a store spread over the banks; groups of four values stay together.
template <int D>
__device__ __forceinline__ int part_at(int h, int d) {
  return h * D + (d ^ ((h & 7) << 2));
}

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
// c += a b; bf16 or fp16 operands.
template <bool FP16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, const uint32_t (&b)[2]) {
  if (FP16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
}
// Transposes an 8 x 8 matrix of 16-bit values, one row's pair (lane / 4; 2 (lane % 4), + 1) per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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
// member but len32 is the same in all lanes. Work is dealt out in slots: a slot per tile, and kPad slots
// behind each unit's tiles that stand for the cost of going on to another one (query rows, a partial
// result: about as long as that many tiles take a warp), so that warps with such a change get fewer tiles.
constexpr int kPad = 2;
template <int TR>
struct Walk {
  int b, u, t, len, nt;  // sequence, unit, tile; the sequence's length and tiles
  int at;                // the tile's slot
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
  // The first tile in slots lo .. hi - 1; lo is in group g, whose slots begin at `before`. False: none.
  __device__ __forceinline__ bool start(const AttnDecodeParams& p, int g, int before, int lo, int hi, int units) {
    if (lo >= hi) return false;
    group(p, g);
    const int lane = threadIdx.x & 31;
    const int slots = unit_slots(len32) * units;
    int sum = slots;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(~0u, sum, x);
      if (lane >= x) sum += y;
    }
    int off = lo - before;
    const int src = __ffs(__ballot_sync(~0u, sum > off)) - 1;
    off -= __shfl_sync(~0u, sum - slots, src);
    seq(src);
    u = off / (nt + kPad);
    t = off % (nt + kPad);
    at = lo;
    return t < nt || skip(p, hi, units);
  }
  __device__ __forceinline__ static int unit_slots(int len) { return len > 0 ? (len + TR - 1) / TR + kPad : 0; }
  // From tile t of its unit, or a slot behind its tiles, to the next unit's first tile.
  __device__ __forceinline__ bool skip(const AttnDecodeParams& p, int hi, int units) {
    at += nt + kPad - t;
    if (at >= hi) return false;
    t = 0;
    if (++u < units) return true;
    u = 0;
    unsigned rest = __ballot_sync(~0u, len32 > 0) & ~((2u << (b - base)) - 1);
    while (!rest) {
      if (base + 32 >= p.n_seqs) return false;  // past the last tile
      group(p, base / 32 + 1);
      rest = __ballot_sync(~0u, len32 > 0);
    }
    seq(__ffs(rest) - 1);
    return true;
  }
  __device__ __forceinline__ bool next(const AttnDecodeParams& p, int hi, int units) {
    if (++t < nt) return ++at < hi;
    --t;
    return skip(p, hi, units);
  }
};

// A partial result of a warp: of the tiles of unit u of sequence b, which are nt tiles from slot
// `begin` of all on; whether the first and the last of them are in it.
struct PartInfo {
  int b, u, begin, nt, first, last;  // b = -1: none
  const float* o;
};

// Four values of one head over several partial results, with a running maximum.
struct Sum4 {
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);

  // Adds the partial results first, first + step, ... below n; kBatch of them in flight. get(i): partial i. What is
  // read past the last is a copy of it, with a weight of 0; INF: an infinity may be in it, and 0 times that is a NaN.
  // (e4m3 has none; its 129 sequences of up to 8191 rows take 75.1 us without the zeros, 76.6 with them.)
  template <bool INF, class Get>
  __device__ __forceinline__ void add(int first, int step, int n, Get get) {
    constexpr int kBatch = 8;
    for (int i0 = first; i0 < n; i0 += step * kBatch) {
      float4 x[kBatch];
      float xm[kBatch], xl[kBatch], top = m;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int j = i0 + i * step;
        get(min(j, n - 1), x[i], xm[i], xl[i]);
        if (j >= n) xm[i] = -INFINITY;
        if (INF && j >= n) {
          x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          xl[i] = 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) top = fmaxf(top, xm[i]);
      const float base = top == -INFINITY ? 0.f : top;
      scale(ex2(m - base));
      m = top;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) take(ex2(xm[i] - base), x[i], xl[i]);  // weight 0 past the last
    }
  }
  __device__ __forceinline__ void scale(float f) {
    l *= f;
    acc.x *= f;
    acc.y *= f;
    acc.z *= f;
    acc.w *= f;
  }
  __device__ __forceinline__ void take(float w, const float4& x, float xl) {
    l = fmaf(w, xl, l);
    acc.x = fmaf(w, x.x, acc.x);
    acc.y = fmaf(w, x.y, acc.y);
    acc.z = fmaf(w, x.z, acc.z);
    acc.w = fmaf(w, x.w, acc.w);
  }
  // The final four values, at c * 4 of output row `row`.
  template <int D>
  __device__ __forceinline__ void finish(const AttnDecodeParams& p, int64_t row, int c, float v_scale) const {
    const bool none = l == 0.f;
    const float inv = v_scale / l;
    *reinterpret_cast<uint2*>(p.o + row * D + c * 4) =
        none ? make_uint2(0u, 0u) : make_uint2(bf16x2_rn(acc.x * inv, acc.y * inv), bf16x2_rn(acc.z * inv, acc.w * inv));
    if (c == 0 && p.lse) p.lse[row] = none ? -INFINITY : m * kLn2 + logf(l);
  }
};

template <int D, bool E4M3, int NH>
__global__ void __launch_bounds__(32 * Cfg<D, E4M3, NH>::NW, 1) attn_decode_kernel(const __grid_constant__ AttnDecodeParams p) {
  using C = Cfg<D, E4M3, NH>;
  constexpr int RB = C::RB, TR = C::TR, NW = C::NW, TH = 32 * NW;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_before[kMaxGroups + 1];  // slots before each group of 32 sequences
  __shared__ PartInfo s_part[2 * NW];
  __shared__ float s_ml[2 * NW][32];
  __shared__ int s_order[2 * NW];  // the partial results there are, in tile order

  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int nhb = (p.group + 15) / 16, units = p.hkv * nhb;
  pdl_launch_dependents();
  pdl_wait();

  // ---- the tiles of all sequences
  const int groups = (p.n_seqs + 31) / 32;
  for (int g = warp; g < groups; g += NW) {
    const int b = g * 32 + lane;
    const int n = Walk<TR>::length(p, b);
    if (blockIdx.x == 0 && b < p.n_seqs && n != __ldg(p.lens + b)) raise_bad_index(p.hdr);
    // rows of empty sequences, the CTAs in turn
    unsigned none = __ballot_sync(~0u, b < p.n_seqs && n == 0 && b % gridDim.x == blockIdx.x);
    for (; none; none &= none - 1) {
      const int64_t e = g * 32 + __ffs(none) - 1;
      for (int x = lane; x < p.hq * (D / 8); x += 32)
        *reinterpret_cast<uint4*>(p.o + e * p.hq * D + x * 8) = make_uint4(0, 0, 0, 0);
      if (p.lse)
        for (int h = lane; h < p.hq; h += 32) p.lse[e * p.hq + h] = -INFINITY;
    }
    int slots = Walk<TR>::unit_slots(n);
#pragma unroll
    for (int x = 16; x; x >>= 1) slots += __shfl_xor_sync(~0u, slots, x);
    if (lane == 0) s_before[g + 1] = slots * units;
  }
  if (threadIdx.x < 2 * NW) s_part[threadIdx.x].b = -1;
  if (threadIdx.x == 0) s_before[0] = 0;
  __syncthreads();
  if (groups > 1) {
    if (warp == 0) {  // inclusive sums, kMaxGroups / 32 groups per lane
      int v[kMaxGroups / 32], sum = 0;
#pragma unroll
      for (int i = 0; i < kMaxGroups / 32; ++i) {
        const int g = lane * (kMaxGroups / 32) + i;
        sum += g < groups ? s_before[g + 1] : 0;
        v[i] = sum;
      }
      int inc = sum;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int y = __shfl_up_sync(~0u, inc, x);
        if (lane >= x) inc += y;
      }
#pragma unroll
      for (int i = 0; i < kMaxGroups / 32; ++i) {
        const int g = lane * (kMaxGroups / 32) + i;
        if (g < groups) s_before[g + 1] = inc - sum + v[i];
      }
    }
    __syncthreads();
  }
  const unsigned total = s_before[groups];
  // warp x of all has `base` slots, one more if x < more
  const unsigned warps = gridDim.x * NW, base = total / warps, more = total % warps;
  const auto slot_of = [&](unsigned x) { return x * base + min(x, more); };
  const auto cta_of = [&](unsigned slot) {
    const unsigned x = slot < more * (base + 1) ? slot / (base + 1) : more + (slot - more * (base + 1)) / base;
    return (int)(x / NW);
  };
  const unsigned lo = slot_of(blockIdx.x * NW + warp), hi = slot_of(blockIdx.x * NW + warp + 1);
  if (threadIdx.x == 0) p.splits[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (slot_of(blockIdx.x * NW) >= total) return;

  uint8_t* ring = smem + warp * C::kRing;
  const uint32_t ring_s = smem_u32(ring);
  float* scratch = p.scratch + (int64_t)(blockIdx.x * NW + warp) * (16 * D);

  {
    int g = 0;
    for (int x = lane; x < groups; x += 32) g += s_before[x + 1] <= (int)lo;
#pragma unroll
    for (int x = 16; x; x >>= 1) g += __shfl_xor_sync(~0u, g, x);
    Walk<TR> w, ld;
    bool any = w.start(p, g, s_before[g], (int)lo, (int)hi, units);
    ld = w;
    if (any) {

    // ---- copies: the pages of the next tile to copy are already in `page`
    const int row = lane & (TR - 1);  // the tile row whose place this lane looks up
    const auto page_of = [&]() {
      const int pos = ld.t * TR + row;
      return pos < ld.len ? __ldg(p.table + (int64_t)ld.b * p.table_width + p.page_div(pos)) : -1;
    };
    constexpr int CPR = RB / 16, RPI = 32 / CPR;  // copies per row, rows per instruction
    const auto swz = [](int r) { return RB == 64 ? (r >> 1) & 3 : r & 7; };
    const uint32_t at0 = ring_s + (lane / CPR) * RB, at_x = ((lane % CPR) ^ swz(lane / CPR)) << 4;
    const uint8_t* kc = static_cast<const uint8_t*>(p.kc) + (lane % CPR) * 16;
    const uint8_t* vc = static_cast<const uint8_t*>(p.vc) + (lane % CPR) * 16;
    int page = page_of();
    bool left = true;  // there is a tile to copy
    const auto issue = [&](int stage) {
      if (left) {
        const int pos = ld.t * TR + row;
        int cell = -1;  // this lane's cache row
        if (pos < ld.len) {
          if (page >= 0 && page < p.n_pages)
            cell = (page * p.hkv + ld.u / nhb) * p.page_size + (pos - (int)p.page_div(pos) * p.page_size);
          else
            raise_bad_index(p.hdr);
        }
        const uint32_t dst = at0 + stage * C::kTile;
        const bool all = __all_sync(~0u, cell >= 0);
#pragma unroll
        for (int i = 0; i < TR / RPI; ++i) {
          const int c = __shfl_sync(~0u, cell, i * RPI + lane / CPR);
          const int64_t off = (int64_t)max(c, 0) * RB;
          const uint32_t at = dst + i * RPI * RB + (at_x ^ (swz(i * RPI) << 4));
          cp16(at, kc + off, all || c >= 0);
          cp16(at + TR * RB, vc + off, all || c >= 0);
        }
        left = ld.next(p, (int)hi, units);
        if (left) page = page_of();
      }
      cp_commit();
    };
    for (int s = 0; s < C::kStages - 1; ++s) issue(s);

    const int g8 = lane >> 2, t4 = lane & 3;                // fragment coordinates
    const int slot = E4M3 ? (g8 >> 1) + 4 * (g8 & 1) : g8;  // e4m3: the key of A row g8 (spreads the row reads over the banks)
    uint32_t q[NH][D / 16][2];
    float o[NH][D / 16][4];
    float m[NH][2], mc[NH][2], l[NH][2], cr[NH][2];  // of heads 2 t4, + 1: maximum, scaled, this lane's sum, scale
    // the query rows of a sequence's head, as B fragments
    const auto load_q = [&](const Walk<TR>& at) {
      const int kvh = at.u / nhb, h0 = (at.u % nhb) * 16;
#pragma unroll
      for (int nh = 0; nh < NH; ++nh) {
        const int h = h0 + nh * 8 + g8;
        const uint16_t* src = p.q.p + (int64_t)at.b * p.q.token_stride + (int64_t)(kvh * p.group + h) * p.q.head_stride;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            // bf16: k step ks holds values 16 ks + (0..15); e4m3: see the K fragments below
            const int d = E4M3 ? (ks / 4) * 64 + t4 * 16 + (ks & 3) * 4 + half * 2 : ks * 16 + t4 * 2 + half * 8;
            q[nh][ks][half] = h < p.group ? __ldg(reinterpret_cast<const uint32_t*>(src + d)) : 0u;
          }
      }
    };
    load_q(w);
    bool fresh = true, from_start = false;
    int out = 0, stage = 0, fill = C::kStages - 1;
    while (any) {
      issue(fill);
      if (++fill == C::kStages) fill = 0;
      const int kvh = w.u / nhb, h0 = (w.u % nhb) * 16, heads = min(16, p.group - h0);
      if (fresh) {
        // ---- a new sequence or head; its query rows have been loaded
        fresh = false;
        from_start = w.t == 0;
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) o[nh][x][y] = 0.f;
          const float scale = p.scale * kLog2e * (E4M3 ? __ldg(p.k_scale + kvh) : 1.f);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            m[nh][y] = -INFINITY;
            mc[nh][y] = 0.f;
            l[nh][y] = 0.f;
            cr[nh][y] = scale;
          }
          if (E4M3) {
            // fp16 has bf16's precision but not its range: the row times a power of two that brings its
            // largest magnitude to 2^14
            uint32_t big = 0;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
              for (int half = 0; half < 2; ++half)
                big = max(big, max(q[nh][ks][half] & 0x7FFFu, (q[nh][ks][half] >> 16) & 0x7FFFu));
            big = max(big, __shfl_xor_sync(~0u, big, 1));
            big = max(big, __shfl_xor_sync(~0u, big, 2));
            const int up = big == 0 || big >= 0x7F80u ? 0 : min(14 - ((int)(big >> 7) - 127), 126);
            const float f = __uint_as_float((uint32_t)(127 + up) << 23);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const uint32_t v = q[nh][ks][half];
                q[nh][ks][half] = f16x2_rn(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xFFFF0000u) * f);
              }
#pragma unroll
            for (int y = 0; y < 2; ++y)
              cr[nh][y] *= __uint_as_float((uint32_t)(127 - __shfl_sync(~0u, up, (2 * t4 + y) * 4)) << 23);
          }
        }
      }

      cp_wait<C::kStages - 1>();
      __syncwarp();
      const uint32_t kt = ring_s + stage * C::kTile, vt = kt + TR * RB;

      // ---- scores. C fragment kb: keys 16 kb + slot (values 0, 1) and + 8 (2, 3) of heads 2 t4, + 1
      float s[TR / 16][NH][4];
#pragma unroll
      for (int kb = 0; kb < TR / 16; ++kb) {
        float s2[NH][4];
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int y = 0; y < 4; ++y) s[kb][nh][y] = s2[nh][y] = 0.f;
        if (!E4M3) {
          const uint32_t at = kt + (kb * 16 + (lane & 15)) * RB;
          const uint32_t x = ((lane >> 4) ^ (lane & 7)) << 4;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t a[4];
            ldsm4(at + ((ks * 32) ^ x), a);
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) mma<false>(ks & 1 ? s2[nh] : s[kb][nh], a[0], a[1], a[2], a[3], q[nh][ks]);
          }
        } else {
          // a lane reads 16 codes of two keys: values 64 i + 16 t4 + 0..15 serve four k steps
          const uint32_t at = kt + (kb * 16 + slot) * RB;
#pragma unroll
          for (int i4 = 0; i4 < D / 64; ++i4) {
            const int c = i4 * 4 + t4;
            const uint4 u = lds128(at + ((c ^ swz(slot)) << 4)), v = lds128(at + 8 * RB + ((c ^ swz(slot + 8)) << 4));
            const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t a0 = e4m3x2_f16<0>(uw[k]), a1 = e4m3x2_f16<0>(vw[k]), a2 = e4m3x2_f16<1>(uw[k]), a3 = e4m3x2_f16<1>(vw[k]);
#pragma unroll
              for (int nh = 0; nh < NH; ++nh) mma<true>(k & 1 ? s2[nh] : s[kb][nh], a0, a1, a2, a3, q[nh][4 * i4 + k]);
            }
          }
        }
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int y = 0; y < 4; ++y) s[kb][nh][y] += s2[nh][y];
      }
      const bool to_end = w.t == w.nt - 1;
      const int lim = w.len - w.t * TR;
      Walk<TR> nx = w;
      any = nx.next(p, (int)hi, units);
      if (any && to_end) load_q(nx);  // while the rest of this tile is worked on
      if (lim < TR) {
#pragma unroll
        for (int kb = 0; kb < TR / 16; ++kb)
#pragma unroll
          for (int nh = 0; nh < NH; ++nh)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (kb * 16 + slot + (y >> 1) * 8 >= lim) s[kb][nh][y] = -INFINITY;
      }

      // ---- running softmax
      bool grown = false;
      float mx[NH][2];
#pragma unroll
      for (int nh = 0; nh < NH; ++nh)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float x = -INFINITY;
#pragma unroll
          for (int kb = 0; kb < TR / 16; ++kb) x = fmaxf(x, fmaxf(s[kb][nh][y], s[kb][nh][y + 2]));
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
          x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
          mx[nh][y] = x;
          grown |= x * cr[nh][y] > mc[nh][y] + kRescaleLog2 + C::kUp || (m[nh][y] == -INFINITY && x > m[nh][y]);
        }
      if (__any_sync(~0u, grown)) {
#pragma unroll
        for (int nh = 0; nh < NH; ++nh)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float m2 = fmaxf(m[nh][y], mx[nh][y]), mc2 = m2 == -INFINITY ? 0.f : m2 * cr[nh][y] - C::kUp;
            const float f = m[nh][y] == -INFINITY ? 0.f : ex2(mc[nh][y] - mc2);
            m[nh][y] = m2;
            mc[nh][y] = mc2;
            l[nh][y] *= f;
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
              o[nh][x][y] *= f;
              o[nh][x][y + 2] *= f;
            }
          }
      }
      uint32_t b[TR / 16][NH][2];
#pragma unroll
      for (int kb = 0; kb < TR / 16; ++kb)
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
          float e[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) e[y] = ex2(fmaf(s[kb][nh][y], cr[nh][y & 1], -mc[nh][y & 1]));
          l[nh][0] += e[0] + e[2];
          l[nh][1] += e[1] + e[3];
          b[kb][nh][0] = transpose8x8(E4M3 ? f16x2_rn(e[0], e[1]) : bf16x2_rn(e[0], e[1]));
          b[kb][nh][1] = transpose8x8(E4M3 ? f16x2_rn(e[2], e[3]) : bf16x2_rn(e[2], e[3]));
        }

      // ---- O^T += V^T P^T. C fragment x holds, of heads 2 t4, + 1, the values
      //   bf16: 16 x + g8 (values 0, 1) and + 8 (2, 3);  e4m3, D = 64: 8 g8 + 2 x and + 1;
      //   e4m3, D >= 128: 128 (x / 8) + 16 slot + 2 (x % 8) and + 1
#pragma unroll
      for (int kb = 0; kb < TR / 16; ++kb) {
        if (!E4M3) {
          const uint32_t at = vt + (kb * 16 + (lane & 7) + ((lane >> 4) & 1) * 8) * RB;
          const uint32_t x8 = (((lane >> 3) & 1) ^ (lane & 7)) << 4;
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            uint32_t a[4];
            ldsm4t(at + ((x * 32) ^ x8), a);
#pragma unroll
            for (int nh = 0; nh < NH; ++nh) mma<false>(o[nh][x], a[0], a[1], a[2], a[3], b[kb][nh]);
          }
        } else {
          // keys t4, t4 + 4, t4 + 8, t4 + 12 of the 16 (the places of k 2 t4, + 1, + 8, + 9)
          const auto products = [&](int x, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {  // 4 codes of each key
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t u = __byte_perm(r0, r1, k ? 0x7362 : 0x5140), v = __byte_perm(r2, r3, k ? 0x7362 : 0x5140);
              const uint32_t a0 = e4m3x2_f16<0>(u), a1 = e4m3x2_f16<1>(u), a2 = e4m3x2_f16<0>(v), a3 = e4m3x2_f16<1>(v);
#pragma unroll
              for (int nh = 0; nh < NH; ++nh) mma<true>(o[nh][x + k], a0, a1, a2, a3, b[kb][nh]);
            }
          };
          if (D == 64) {
            uint2 v[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int r = kb * 16 + t4 + 4 * y;
              v[y] = lds64(vt + r * RB + (((g8 >> 1) ^ swz(r)) << 4) + (g8 & 1) * 8);
            }
            products(0, v[0].x, v[1].x, v[2].x, v[3].x);
            products(2, v[0].y, v[1].y, v[2].y, v[3].y);
          } else {
#pragma unroll
            for (int dq = 0; dq < D / 128; ++dq) {
              uint4 v[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int r = kb * 16 + t4 + 4 * y;
                v[y] = lds128(vt + r * RB + (((dq * 8 + slot) ^ swz(r)) << 4));
              }
              products(dq * 8, v[0].x, v[1].x, v[2].x, v[3].x);
              products(dq * 8 + 2, v[0].y, v[1].y, v[2].y, v[3].y);
              products(dq * 8 + 4, v[0].z, v[1].z, v[2].z, v[3].z);
              products(dq * 8 + 6, v[0].w, v[1].w, v[2].w, v[3].w);
            }
          }
        }
      }
      if (++stage == C::kStages) stage = 0;
      __syncwarp();

      // ---- the end of a sequence's head, or of this warp's run
      if (to_end || !any) {
        const bool whole = to_end && from_start, mid = any;
        float* to = mid ? scratch : reinterpret_cast<float*>(ring);
        if (!whole && !mid) {
          cp_wait<0>();  // the ring is idle: every copy has landed and been used
          __syncwarp();
        }
#pragma unroll
        for (int nh = 0; nh < NH; ++nh) {
          float inv[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int h = nh * 8 + 2 * t4 + y;
            float sum = l[nh][y];
            sum += __shfl_xor_sync(~0u, sum, 4);
            sum += __shfl_xor_sync(~0u, sum, 8);
            sum += __shfl_xor_sync(~0u, sum, 16);
            inv[y] = !whole || sum == 0.f ? 0.f : (E4M3 ? __ldg(p.v_scale + kvh) : 1.f) / sum;
            if (lane < 4 && h < heads) {
              if (!whole) {
                s_ml[warp * 2 + out][h] = m[nh][y] == -INFINITY ? -INFINITY : mc[nh][y];
                s_ml[warp * 2 + out][16 + h] = sum;
              } else if (p.lse) {
                p.lse[(int64_t)w.b * p.hq + kvh * p.group + h0 + h] = sum == 0.f ? -INFINITY : mc[nh][y] * kLn2 + logf(sum);
              }
            }
          }
          uint16_t* dst = p.o + ((int64_t)w.b * p.hq + kvh * p.group + h0 + nh * 8) * D;  // head 0 of this block
          const auto scaled = [&](float x, int y) { return inv[y] == 0.f ? 0.f : x * inv[y]; };
          if (!whole) {
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int h = nh * 8 + 2 * t4 + (y & 1);
                const int d = !E4M3     ? 16 * x + g8 + 8 * (y >> 1)
                              : D == 64 ? 8 * g8 + 2 * x + (y >> 1)
                                        : 128 * (x / 8) + 16 * slot + 2 * (x % 8) + (y >> 1);
                if (h < heads) to[part_at<D>(h, d)] = o[nh][x][y];
              }
          } else if (!E4M3) {
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                // turned: head g8, values 2 t4, + 1
                const uint32_t v = transpose8x8(bf16x2_rn(scaled(o[nh][x][2 * z], 0), scaled(o[nh][x][2 * z + 1], 1)));
                if (nh * 8 + g8 < heads) *reinterpret_cast<uint32_t*>(dst + g8 * D + 16 * x + 8 * z + 2 * t4) = v;
              }
          } else {
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int x = 0; x < D / 16; x += 4) {
                uint32_t v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = bf16x2_rn(scaled(o[nh][x + k][y], y), scaled(o[nh][x + k][y + 2], y));
                const int d = D == 64 ? 8 * g8 : 128 * (x / 8) + 16 * slot + 2 * (x % 8);
                if (nh * 8 + 2 * t4 + y < heads) *reinterpret_cast<uint4*>(dst + (2 * t4 + y) * D + d) = make_uint4(v[0], v[1], v[2], v[3]);
              }
          }
        }
        if (!whole) {
          if (lane == 0) s_part[warp * 2 + out] = PartInfo{w.b, w.u, w.at - w.t, w.nt, from_start, to_end, to};
          ++out;
        }
        fresh = true;
      }
      w = nx;
    }
    cp_wait<0>();
    }
  }
  __syncthreads();

  // ---- partial results of this CTA's warps, in tile order: those of one sequence's head are joined
  const PartInfo mine = lane < 2 * NW ? s_part[lane] : PartInfo{-1, 0, 0, 0, 0, 0, nullptr};
  unsigned rest = __ballot_sync(~0u, mine.b >= 0);
  if (!rest) return;
  if (warp == 0 && mine.b >= 0) s_order[__popc(rest & ((1u << lane) - 1))] = lane;
  __syncthreads();
  int at = 0;
  while (rest) {
    const int head = __ffs(rest) - 1, b = __shfl_sync(~0u, mine.b, head), u = __shfl_sync(~0u, mine.u, head);
    const unsigned same = __ballot_sync(~0u, mine.b == b && mine.u == u);
    const int cnt = __popc(same), tail = 31 - __clz(same);
    const int first = __shfl_sync(~0u, mine.first, head), last = __shfl_sync(~0u, mine.last, tail);
    const unsigned begin = __shfl_sync(~0u, mine.begin, head), end = begin + __shfl_sync(~0u, mine.nt, head) - 1;
    rest &= ~same;
    const int kvh = u / nhb, h0 = (u % nhb) * 16, heads = min(16, p.group - h0);
    float* to = p.parts + (int64_t)(blockIdx.x * 2 + (first ? 1 : 0)) * C::kPart;
    for (int e = threadIdx.x; e < heads * (D / 4); e += TH) {
      const int h = e / (D / 4), c = e % (D / 4);
      Sum4 sum;
      sum.template add<!E4M3>(0, 1, cnt, [&](int i, float4& x, float& xm, float& xl) {
        const int y = s_order[at + i];
        x = *reinterpret_cast<const float4*>(s_part[y].o + part_at<D>(h, c * 4));
        xm = s_ml[y][h];
        xl = s_ml[y][16 + h];
      });
      if (first && last) {
        sum.finish<D>(p, (int64_t)b * p.hq + kvh * p.group + h0 + h, c, E4M3 ? __ldg(p.v_scale + kvh) : 1.f);
      } else {
        *reinterpret_cast<float4*>(to + part_at<D>(h, c * 4)) = sum.acc;
        if (c == 0) {
          to[16 * D + h] = sum.m;
          to[16 * D + 16 + h] = sum.l;
        }
      }
    }
    at += cnt;
    // a head that begins here and goes on in the next CTAs, up to the one that holds its last tile
    if (threadIdx.x == 0 && first && !last) p.splits[blockIdx.x] = make_int4(b, u, cta_of(end) - (int)blockIdx.x + 1, 0);
  }
}

// Joins the partial results of the head that begins in CTA blockIdx.x of the kernel above, for query head
// blockIdx.y of its unit: 256 threads walk the partials D / 4 threads to one.
template <int D, bool E4M3, int NH>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnDecodeParams p) {
  using C = Cfg<D, E4M3, NH>;
  constexpr int V = D / 4, R = 256 / V;
  __shared__ float4 s_acc[R][V];
  __shared__ float s_ml[R][2];
  pdl_launch_dependents();
  pdl_wait();
  const int4 split = p.splits[blockIdx.x];
  const int n = split.z;
  if (n == 0) return;
  const int nhb = (p.group + 15) / 16, kvh = split.y / nhb, h0 = (split.y % nhb) * 16, h = blockIdx.y;
  if (h >= min(16, p.group - h0)) return;
  const int r = threadIdx.x / V, c = threadIdx.x % V;
  Sum4 sum;
  sum.template add<!E4M3>(r, R, n, [&](int i, float4& x, float& xm, float& xl) {
    // CTA blockIdx.x + i: its partial of a head that begins there (1) or before (0)
    const float* o = p.parts + (int64_t)((blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * C::kPart;
    x = *reinterpret_cast<const float4*>(o + part_at<D>(h, c * 4));
    xm = o[16 * D + h];
    xl = o[16 * D + 16 + h];
  });
  s_acc[r][c] = sum.acc;
  if (c == 0) {
    s_ml[r][0] = sum.m;
    s_ml[r][1] = sum.l;
  }
  __syncthreads();
  if (r) return;
  Sum4 all;
  all.template add<!E4M3>(0, 1, min(R, n), [&](int i, float4& x, float& xm, float& xl) {
    x = s_acc[i][c];
    xm = s_ml[i][0];
    xl = s_ml[i][1];
  });
  all.finish<D>(p, (int64_t)split.x * p.hq + kvh * p.group + h0 + h, c, E4M3 ? __ldg(p.v_scale + kvh) : 1.f);
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

template <int D, bool E4M3, int NH>
cudaError_t launch(const AttnDecodeParams& p, cudaStream_t s) {
  using C = Cfg<D, E4M3, NH>;
  static cudaError_t attr = cudaFuncSetAttribute(attn_decode_kernel<D, E4M3, NH>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (attr != cudaSuccess) return attr;
  const cudaError_t err =
      launch_pdl(attn_decode_kernel<D, E4M3, NH>, dim3(num_sms()), 32 * C::NW, (size_t)C::kSmem, 1, s, p);
  if (err != cudaSuccess) return err;
  return launch_pdl(attn_join_kernel<D, E4M3, NH>, dim3(num_sms(), p.group < 16 ? p.group : 16), 256, 0, 1, s, p);
}

template <int D, bool E4M3>
cudaError_t launch(const AttnDecodeParams& p, cudaStream_t s) {
  return p.group <= 8 ? launch<D, E4M3, 1>(p, s) : launch<D, E4M3, 2>(p, s);  // blocks of 8 heads
}

}  // namespace

cudaError_t launch_attn_decode(const AttnDecodeParams& p, int d, bool e4m3, cudaStream_t s) {
  if (d == 64) return e4m3 ? launch<64, true>(p, s) : launch<64, false>(p, s);
  if (d == 128) return e4m3 ? launch<128, true>(p, s) : launch<128, false>(p, s);
  return e4m3 ? launch<256, true>(p, s) : launch<256, false>(p, s);
}

}  // namespace moe
