// moe_gemm_e4m3 on the 5th-generation tensor cores: e4m3 rows times their experts' e4m3 matrices, a scale
// for each block of 128.
//
// out[p, c] = sum_b s_a[p, b] s_w[e, c / 128, b] (sum of the 128 code products of block b). The tensor cores
// sum a block's codes into a fresh accumulator in tensor memory; 8 warps then read it, multiply by the two
// scales (one factor per row and warp: a row's scale times the block's) and add to fp32 sums in registers,
// while the other accumulator takes the next block. So scales of any fp32 value cost no accuracy.
//
// A CTA makes 128 rows of one expert x BN columns, rows as the MMA's M: a thread owns a row, so that its
// factor is one register. Persistent CTAs, one per SM, walk the items (expert, row tile, column tile):
//   warp 0       copies: per block of 128 inputs the rows (32, 64 or 128 of them) and BN weight columns
//   warp 1       MMA issue: per block four MMAs of K = 32
//   warps 4-11   scaling and adding, then the output; warp w reads lane quadrant w % 4 and half of the
//                columns
// Transposed weights are read as they lie: their tile has its column axis contiguous (the other "major"
// of the MMA's B operand), so no second copy of the weights is kept.
#include "expert_device.cuh"
#include "attn_ptx.cuh"

namespace moe {
bool encode_tiled(CUtensorMap* m, CUtensorMapDataType type, cuuint32_t rank, const void* ptr, const cuuint64_t* dims,
                  const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swz);

namespace {

constexpr int kTileM = 128;
constexpr int kWarpCopy = 0, kWarpMma = 1, kWarpSum0 = 4, kSumWarps = 8;
constexpr int kThreads = (kWarpSum0 + kSumWarps) * 32;  // 384
// Registers: 168 a thread at launch; the first four warps give up 96 each, the summing ones take 48 more:
// 128 * 72 + 256 * 216 = 384 * 168.
constexpr int kFewRegs = 72, kManyRegs = 216;
constexpr int kGroupTiles = 16;  // row tiles of an expert whose column tiles run together

struct ProductMaps {
  CUtensorMap rows[3];  // boxes of 32, 64, 128 rows x 128 inputs
  CUtensorMap w;
};

template <int BN>
struct Layout {
  static constexpr int kABytes = kTileM * 128, kBBytes = BN * 128, kStage = kABytes + kBBytes;
  static constexpr int kStages = BN == 256 ? 4 : 6;
  static constexpr int bar_off = kStages * kStage;
  static constexpr int n_bars = 2 * kStages + 4;
  static constexpr int misc_off = bar_off + n_bars * 8;
  static constexpr int out_off = (misc_off + 16 + 127) / 128 * 128;  // per summing warp: 32 rows x 32 columns of bf16
  static constexpr int sa_off = out_off + kSumWarps * 2048;          // per summing warp: two slots of 4 scales x 32 rows
  static constexpr int sw_off = sa_off + kSumWarps * 1024;           // and of 4 of the weights
  static constexpr int sum_off = sw_off + kSumWarps * 32;            // the work list's partial sums
  static constexpr int table_off = sum_off + 64;                     // first item of every expert, and their number
  static constexpr int fixed = table_off + 1024;                     // and slack to align the base
  static constexpr int most = fixed + (kMaxExperts + 1) * 4;
  static_assert(most <= 232448, "shared memory");
};

// Four MMAs of K = 32 on a block of 128 inputs under one elected lane; B_STEP: descriptor units (16 bytes)
// from one K step of B to the next.
template <int B_STEP>
__device__ __forceinline__ void mma_block(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred f, t, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
      "setp.ne.b32 f, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
      "add.s64 b1, %2, %4;\n\tadd.s64 b2, %2, %5;\n\tadd.s64 b3, %2, %6;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, f;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, t;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "n"(B_STEP), "n"(2 * B_STEP), "n"(3 * B_STEP)
      : "memory");
}
// kind::f8f6f4: fp32 accumulator, A and B e4m3; trans_b: B has its N axis contiguous.
__device__ __forceinline__ uint32_t idesc_e4m3(int M, int N, bool trans_b) {
  return (1u << 4) | (trans_b ? kIdescBMn : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* m, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive_elect(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b64 st;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar)
      : "memory");
}
// Asynchronous copies of 4 or 16 bytes; nothing is read and zeros are written where !there.
__device__ __forceinline__ void copy4(uint32_t dst, const float* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const float* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ float4 lds128(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

struct Item {
  int expert, row0, rows, col0;
};

// An expert's rows, offsets out of range or descending cut to what lies inside.
struct Range {
  int lo, hi;
  bool bad;
};
__device__ __forceinline__ Range expert_rows(const ProductParams& p, int e) {
  if (!p.offsets) return {0, p.rows, false};
  const int a = __ldg(p.offsets + e), b = __ldg(p.offsets + e + 1);
  const int lo = min(max(a, 0), p.rows), hi = min(max(b, lo), p.rows);
  return {lo, hi, a != lo || b != hi};
}

// The i-th item of the work list; first[e]: the first one of expert e, in shared memory. A whole warp calls it.
// Row tiles of an expert go in groups of kGroupTiles; in a group the column tiles one after the other, each
// with all row tiles, so that the CTAs at work share both the rows' and the weights' tiles in L2.
template <int BN>
__device__ __forceinline__ Item find_item(const ProductParams& p, const int* first, int col_tiles, int i) {
  const int lane = threadIdx.x & 31;
  int a = 0, b = p.n_experts;  // first[a] <= i < first[b]
  while (b - a > 1) {          // 32 pieces at a time
    const int step = (b - a + 31) / 32, at = a + lane * step;
    const unsigned m = __ballot_sync(~0u, at < b && first[at] <= i);  // a run of ones from lane 0 on
    a += (31 - __clz(m)) * step;
    b = min(a + step, b);
  }
  const Range x = expert_rows(p, a);
  const int rows = x.hi - x.lo, tiles = (rows + kTileM - 1) / kTileM;
  int in = i - first[a], base = 0;
  if (tiles > kGroupTiles) {
    const int per = kGroupTiles * col_tiles, group = in / per;
    in -= group * per;
    base = group * kGroupTiles;
  }
  const int n = min(kGroupTiles, tiles - base);
  const int ct = (int)__fdividef((float)in + 0.5f, (float)n);  // in < 2^13 and n <= 16: never near an integer
  const int rt = base + in - ct * n;
  return {a, x.lo + rt * kTileM, min(kTileM, rows - rt * kTileM), ct * BN};
}

template <int BN, bool TRANS>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ ProductParams p, const __grid_constant__ ProductMaps maps) {
  using L = Layout<BN>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const uint32_t bars = base + L::bar_off;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (L::kStages + s); };
  auto acc_full = [&](int b) { return bars + 8u * (2 * L::kStages + b); };
  auto acc_empty = [&](int b) { return bars + 8u * (2 * L::kStages + 2 + b); };
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + L::misc_off);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + L::misc_off + 4);

  if (tid == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), kSumWarps);
    }
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(s_tmem), 2 * BN);
    tmem_relinquish();
  }
  if (warp == kWarpCopy && lane < 4) prefetch_tmap(lane < 3 ? &maps.rows[lane] : &maps.w);
  // Everything above touched shared and tensor memory alone; the offsets and rows are read after the
  // predecessor has completed.
  pdl_wait();
  pdl_launch_dependents();

  // ---------------------------------------------------------------- work list
  int* first = reinterpret_cast<int*>(smem + L::table_off);
  int* s_sum = reinterpret_cast<int*>(smem + L::sum_off);
  const int col_tiles = (p.outc + BN - 1) / BN;
  int n_items = 0;
  {
    constexpr int kPer = (kMaxExperts + kThreads - 1) / kThreads;
    int items[kPer], sum = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      items[i] = 0;
      if (e < p.n_experts) {
        const Range r = expert_rows(p, e);
        bad |= r.bad;
        items[i] = (r.hi - r.lo + kTileM - 1) / kTileM * col_tiles;
      }
      sum += items[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_sum[warp] = incl;
    if (blockIdx.x == 0 && bad) raise_index(p.hdr);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int at = incl - sum;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) at += s_sum[w];
      n_items += s_sum[w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (tid * kPer + i < p.n_experts) first[tid * kPer + i] = at;
      at += items[i];
    }
    __syncthreads();
  }
  const uint32_t tmem = *s_tmem;
  const int kb_n = p.in_blocks;

  if (warp < kWarpSum0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
  if (warp == kWarpCopy) {
    // ------------------------------------------------------------ copies
    uint32_t g = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < n_items && ok; i += gridDim.x) {
      const Item it = find_item<BN>(p, first, col_tiles, i);
      const int box = it.rows > 64 ? 2 : it.rows > 32 ? 1 : 0;
      const uint32_t bytes = (32u << box) * 128u + L::kBBytes;
      if (lane == 0)
        for (int kb = 0; kb < kb_n; ++kb, ++g) {
          const int s = g % L::kStages;
          if (!(ok = mbar_wait(empty(s), ((g / L::kStages) & 1) ^ 1, s_abort))) break;
          const uint32_t a = base + s * L::kStage, b = a + L::kABytes;
          mbar_arrive_expect_tx(full(s), bytes);
          tma_load_2d(a, &maps.rows[box], kb * 128, it.row0, full(s));
          if (TRANS) {
#pragma unroll
            for (int c = 0; c < BN / 128; ++c)
              tma_load_3d(b + c * 16384, &maps.w, it.col0 + c * 128, kb * 128, it.expert, full(s));
          } else {
            tma_load_3d(b, &maps.w, kb * 128, it.col0, it.expert, full(s));
          }
        }
      ok = __shfl_sync(~0u, ok, 0);
    }
    if (!ok && lane == 0)  // a wait gave up: the copies in flight land before the CTA ends
      for (int s = 0; s < L::kStages && (int)g - 1 - s >= 0; ++s) {
        const uint32_t h = g - 1 - s;
        const long long t0 = clock64();
        while (!mbar_try_wait(full(h % L::kStages), (h / L::kStages) & 1) && clock64() - t0 < kWaitCycles) {
        }
      }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA issue
    const uint32_t idesc = idesc_e4m3(kTileM, BN, TRANS);
    uint32_t g = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < n_items && ok; i += gridDim.x)
      for (int kb = 0; kb < kb_n; ++kb, ++g) {
        const int s = g % L::kStages, buf = g & 1;
        // one lane waits for the copies, the others for the accumulator
        ok = __all_sync(~0u, lane == 0 ? mbar_wait(full(s), (g / L::kStages) & 1, s_abort)
                                       : mbar_wait(acc_empty(buf), ((g >> 1) & 1) ^ 1, s_abort));
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = base + s * L::kStage, b = a + L::kABytes;
        if (TRANS)
          mma_block<32 * 128 / 16>(tmem + buf * BN, sw128_desc(a), sw128_mn_desc(b, 16384), idesc);
        else
          mma_block<2>(tmem + buf * BN, sw128_desc(a), sw128_desc(b), idesc);
        umma_commit_elect(empty(s));
        umma_commit_elect(acc_full(buf));
      }
    if (!ok && g) {  // a wait gave up: the MMAs in flight end before tensor memory is freed
      const long long t0 = clock64();
      while (!mbar_try_wait(empty((g - 1) % L::kStages), ((g - 1) / L::kStages) & 1) && clock64() - t0 < kWaitCycles) {
      }
    }
  } else if (warp >= kWarpSum0) {
    // ------------------------------------------------------------ scaling, adding, output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
    constexpr int kCols = BN / 2;  // columns of a warp
    const int quad = warp & 3, part = (warp - kWarpSum0) >> 2, r = quad * 32 + lane;
    const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + part * kCols;
    const uint32_t s_a = base + L::sa_off + (warp - kWarpSum0) * 1024 + lane * 16;
    const uint32_t s_w = base + L::sw_off + (warp - kWarpSum0) * 32;
    const uint32_t s_out = base + L::out_off + (warp - kWarpSum0) * 2048;
    const bool vec = kb_n % 4 == 0 && p.a.scale_stride % 4 == 0 && (reinterpret_cast<uintptr_t>(p.a.scale) & 15) == 0;
    const float *sa = nullptr, *sw = nullptr;  // scales of the item whose copies are issued next
    // Rows past the tile and columns past the matrix are computed on what lies there and not stored.
    auto scales_of = [&](const Item& it) {
      sa = p.a.scale + (it.row0 + min(r, it.rows - 1)) * p.a.scale_stride;
      const int cb = min((it.col0 + part * kCols) / kScaleBlock, p.out_blocks - 1);
      sw = p.wscale + (int64_t)it.expert * p.in_blocks * p.out_blocks + (TRANS ? cb : (int64_t)cb * p.in_blocks);
    };
    // The factors of blocks kb .. kb + 3, asynchronously, into a slot of the warp's own: a row's scales into its
    // thread's, the weights' by the first four lanes. (Loads into registers would be waited for where the loop
    // closes: 177 cycles a block.)
    auto copy_scales = [&](int kb, int slot) {
      if (vec)
        copy16(s_a + slot * 512, sa + kb, true);
      else
#pragma unroll
        for (int u = 0; u < 4; ++u) copy4(s_a + slot * 512 + u * 4, kb + u < kb_n ? sa + kb + u : sa, kb + u < kb_n);
      if (lane < 4) {
        const bool there = kb + lane < kb_n;
        copy4(s_w + slot * 16 + lane * 4, there ? sw + (int64_t)(kb + lane) * (TRANS ? p.out_blocks : 1) : sw, there);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint32_t g = 0;
    int slot = 0;
    Item nx = {0, 0, 1, 0};
    if (blockIdx.x < n_items) {
      nx = find_item<BN>(p, first, col_tiles, blockIdx.x);
      scales_of(nx);
      copy_scales(0, 0);
    }
    for (int i = blockIdx.x; i < n_items; i += gridDim.x) {
      const Item it = nx;
      const bool more = i + (int)gridDim.x < n_items;
      if (more) nx = find_item<BN>(p, first, col_tiles, i + gridDim.x);
      float acc[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
      for (int kb0 = 0; kb0 < kb_n; kb0 += 4) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncwarp();  // the other lanes' copies too; and nobody reads the other slot any more
        const float4 fa = lds128(s_a + slot * 512), fw = lds128(s_w + slot * 16);
        const float f4[4] = {fa.x * fw.x, fa.y * fw.y, fa.z * fw.z, fa.w * fw.w};
        slot ^= 1;
        if (kb0 + 4 < kb_n) {
          copy_scales(kb0 + 4, slot);
        } else if (more) {
          scales_of(nx);
          copy_scales(0, slot);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (kb0 + u < kb_n) {
            const int buf = g & 1;
            // after a wait that gave up, all later ones return at once, and what is computed is not stored
            if (!mbar_try_wait(acc_full(buf), (g >> 1) & 1)) mbar_wait(acc_full(buf), (g >> 1) & 1, s_abort);
            __syncwarp();
            tc_fence_after();
            ++g;
#pragma unroll
            for (int c = 0; c < kCols; c += 32) {
              float v[32];
              tmem_ld32(taddr + buf * BN + c, v);
              tmem_wait_ld32(v);
              if (c + 32 == kCols) {
                tc_fence_before();
                mbar_arrive_elect(acc_empty(buf));
              }
#pragma unroll
              for (int x = 0; x < 32; ++x) acc[c + x] = fmaf(f4[u], v[x], acc[c + x]);
            }
          }
        }
      }
      if (*s_abort) continue;
      // 32 rows x 32 columns at a time through shared memory, so that four lanes store 64 bytes of a row
      // (a thread's own row in 16-byte stores costs a tag lookup each: 4000 cycles an item)
      const int col0 = it.col0 + part * kCols, sub = lane & 3;
#pragma unroll
      for (int c = 0; c < kCols; c += 32) {
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 4; ++x) sts128(s_out + lane * 64 + ((x ^ (lane >> 1)) & 3) * 16, float_to_bf16x8(acc + c + 8 * x));
        __syncwarp();
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int row = y * 8 + (lane >> 2);
          const float4 v = lds128(s_out + row * 64 + ((sub ^ (row >> 1)) & 3) * 16);
          if (quad * 32 + row < it.rows && col0 + c + sub * 8 < p.outc)
            *reinterpret_cast<float4*>(static_cast<uint16_t*>(p.out.p) + (int64_t)(it.row0 + quad * 32 + row) * p.out.stride +
                                       col0 + c + sub * 8) = v;
        }
      }
    }
  }

  // ---------------------------------------------------------------- tear-down
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 2 * BN);
  }
  if (tid == 0 && *s_abort) set_device_status(p.hdr, MOE_ERR_DEVICE_TIMEOUT);
}

template <int BN, bool TRANS>
cudaError_t launch(const ProductParams& p, cudaStream_t s) {
  using L = Layout<BN>;
  static const cudaError_t attr =
      cudaFuncSetAttribute(product_kernel<BN, TRANS>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::most);
  if (attr != cudaSuccess) return attr;
  ProductMaps maps;
  const cuuint64_t adims[2] = {(cuuint64_t)p.in, (cuuint64_t)p.rows}, astr[1] = {(cuuint64_t)p.a.stride};
  for (int i = 0; i < 3; ++i) {
    const cuuint32_t box[2] = {128, 32u << i};
    if (!encode_tiled(&maps.rows[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p.a.p, adims, astr, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  const cuuint64_t wdims[3] = {(cuuint64_t)p.k, (cuuint64_t)p.n, (cuuint64_t)p.n_experts};
  const cuuint64_t wstr[2] = {(cuuint64_t)p.k, (cuuint64_t)p.n * p.k};
  const cuuint32_t wbox[3] = {128, TRANS ? 128u : (cuuint32_t)BN, 1};
  if (!encode_tiled(&maps.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, p.wq, wdims, wstr, wbox, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const int64_t tiles = (p.rows + kTileM - 1) / kTileM + (p.n_experts < p.rows ? p.n_experts : p.rows) - 1;
  const int64_t items = tiles * ((p.outc + BN - 1) / BN);
  const int grid = items < sm_count() ? (int)items : sm_count();
  return launch_pdl(product_kernel<BN, TRANS>, grid, kThreads, (size_t)(L::fixed + (p.n_experts + 1) * 4), 1, s, p, maps);
}

}  // namespace

cudaError_t launch_product(const ProductParams& p, cudaStream_t s) {
  const int64_t tiles = (p.rows + kTileM - 1) / kTileM + (p.n_experts < p.rows ? p.n_experts : p.rows) - 1;
  const bool narrow = tiles * ((p.outc + 255) / 256) < sm_count();
  if (narrow) return p.transposed ? launch<128, true>(p, s) : launch<128, false>(p, s);
  return p.transposed ? launch<256, true>(p, s) : launch<256, false>(p, s);
}

}  // namespace moe
