// moe_gemm_e4m3 on the 5th-generation tensor cores: e4m3 rows times their experts' e4m3 matrices, a scale
// for each block of 128.
//
// out[p, c] = sum_b s_a[p, b] s_w[e, c / 128, b] (sum of the 128 code products of block b). The tensor cores
// sum a block's codes into a fresh accumulator in tensor memory; 8 warps then read it, multiply by the two
// scales (one factor per row and warp: a row's scale times the block's) and add to fp32 sums in registers,
// while the next block goes into another accumulator. The factor is formed first, in fp32: it has to stay below 2^128 and
// keeps 24 bits from 2^-126 on.
//
// A CTA makes 128 rows of one expert x BN columns, rows as the MMA's M: a thread owns a row, so that its
// factor is one register. Persistent CTAs, one per SM, walk the items (expert, row tile, column tile):
//   warp 0       copies: per block of 128 inputs the rows (32, 64 or 128 of them) and BN weight columns
//   warp 1       MMA issue: per block four MMAs of K = 32
//   warps 2-3    the factors of four blocks ahead, into shared memory
//   warps 4-11   scaling and adding, then the output; warp w reads lane quadrant w % 4 and half of the
//                columns
// Transposed weights are read as they lie: their tile has its column axis contiguous (the other "major"
// of the MMA's B operand), so no second copy of the weights is kept.
//
// What bounds it. Many rows: a pair's block of 256 columns takes 0.45 us where its MMAs take 0.26 by the nominal rate (512
// cycles). Timestamps: the MMAs of a block follow each other without a gap, but last 950 cycles beside copies and sums and
// 740 beside the copies alone. Shared memory carries 64 KB a block (32 in, 32 to the MMAs), 512 cycles of it, and 96 KB
// where CTAs work alone; tensor memory hands 131 KB a block to the sums beside the MMAs' own traffic. The sums
// themselves are 32768 FMAs, 256 cycles of the FMA pipes. 8191 x 8192 x 8192 takes 394 us in pairs where calls are spaced out
// (2790 TFLOP/s) and, under the power limit, 414 to 440 back to back (2660 to 2500); single CTAs take 447. Few rows
// to an expert: the weights' bytes; 32768 rows over 256 experts of 1024 x 2048 take 114 us, 5.9 TB/s. (The single CTAs'
// kernel of 256 columns, which does that, spills 20 bytes a thread; the others spill nothing.)
// What it took to get there from 809 us: a row's scales read by one warp ahead instead of by all who use them
// (a line per lane filled L1's tag stage), plain FMAs (pairs cost a move for each register out of tensor memory),
// loads of scales that no loop waits for, output rows stored 64 bytes at a time, both of the issuing warp's
// barriers polled by the whole warp (lanes that wait for different barriers starve each other).
#include "expert_device.cuh"

namespace moe {
bool encode_tiled(CUtensorMap* m, CUtensorMapDataType type, cuuint32_t rank, const void* ptr, const cuuint64_t* dims,
                  const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swz);

namespace {

constexpr int kTileM = 128;
constexpr int kPairRows = 256;  // rows of an expert, on average, from which on CTAs work in pairs
constexpr int kWarpCopy = 0, kWarpMma = 1, kWarpScale0 = 2, kScaleWarps = 2, kWarpSum0 = 4, kSumWarps = 8;
constexpr int kThreads = (kWarpSum0 + kSumWarps) * 32;  // 384
// Registers: 168 a thread at launch; the first four warps give up 96 each, the summing ones take 48 more:
// 128 * 72 + 256 * 216 = 384 * 168.
constexpr int kFewRegs = 72, kManyRegs = 216;
constexpr int kSlots = 3, kSlotBytes = 4 * 2 * kTileM * 4;
constexpr int kGroupTiles = 16;  // row tiles of an expert whose column tiles run together

struct ProductMaps {
  CUtensorMap rows[3];  // boxes of 32, 64, 128 rows x 128 inputs
  CUtensorMap w;
};

// PAIR: two CTAs of a cluster make 256 rows x BN columns with MMAs that span both; each holds its own 128 rows
// and half of the columns' weights.
template <int BN, bool PAIR>
struct Layout {
  static constexpr int kABytes = kTileM * 128, kBCols = PAIR ? BN / 2 : BN, kBBytes = kBCols * 128;
  static constexpr int kItemM = PAIR ? 2 * kTileM : kTileM;  // rows of an item
  // Blocks to a step: what is copied, waited for and handed over together. Tensor memory holds two steps' sums.
  static constexpr int kStep = BN == 128 ? 2 : 1, kTmemCols = 2 * kStep * BN;
  static constexpr int kBlock = kABytes + kBBytes, kStage = kStep * kBlock;
  static constexpr int kStages = 196608 / kStage;
  static constexpr int bar_off = kStages * kStage;
  static constexpr int n_bars = 2 * kStages + 4 + 2 * kSlots;
  static constexpr int misc_off = bar_off + n_bars * 8;
  static constexpr int out_off = (misc_off + 16 + 127) / 128 * 128;  // per summing warp: 32 rows x 32 columns of bf16
  static constexpr int f_off = out_off + kSumWarps * 2048;           // factors: slots of 4 blocks x 2 column halves x 128 rows
  static constexpr int item_off = f_off + kSlots * kSlotBytes;       // and the item that a slot belongs to
  static constexpr int sum_off = item_off + kSlots * 16;             // the work list's partial sums
  static constexpr int table_off = sum_off + 64;                     // first item of every expert
  static constexpr int fixed = table_off + 1024;                     // and slack to align the base
  static constexpr int most = fixed + (kMaxExperts + 1) * 4;
  static_assert(most <= 232448, "shared memory");
};

// Four MMAs of K = 32 on a block of 128 inputs under one elected lane; B_STEP: descriptor units (16 bytes)
// from one K step of B to the next.
#define MOE_MMA_BLOCK(GROUP)                                                                     \
  asm volatile(                                                                                  \
      "{\n\t.reg .pred f, t, e;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"                         \
      "setp.ne.b32 f, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"                                         \
      "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"                       \
      "add.s64 b1, %2, %4;\n\tadd.s64 b2, %2, %5;\n\tadd.s64 b3, %2, %6;\n\t"                    \
      "elect.sync _|e, 0xffffffff;\n\t"                                                          \
      "@e tcgen05.mma.cta_group::" GROUP ".kind::f8f6f4 [%0], %1, %2, %3, f;\n\t"               \
      "@e tcgen05.mma.cta_group::" GROUP ".kind::f8f6f4 [%0], a1, b1, %3, t;\n\t"               \
      "@e tcgen05.mma.cta_group::" GROUP ".kind::f8f6f4 [%0], a2, b2, %3, t;\n\t"               \
      "@e tcgen05.mma.cta_group::" GROUP ".kind::f8f6f4 [%0], a3, b3, %3, t;\n\t}" ::"r"(d_tmem), \
      "l"(a), "l"(b), "r"(idesc), "n"(B_STEP), "n"(2 * B_STEP), "n"(3 * B_STEP)                  \
      : "memory")
template <int B_STEP, bool PAIR>
__device__ __forceinline__ void mma_block(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc) {
  if constexpr (PAIR)
    MOE_MMA_BLOCK("2");
  else
    MOE_MMA_BLOCK("1");
}
#undef MOE_MMA_BLOCK
// Arrives on the barrier once the MMAs issued so far are done; PAIR: on that of both CTAs.
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  if constexpr (PAIR) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(bar)
        : "memory");
  } else {
    umma_commit_elect(bar);
  }
}
// The address of a shared-memory location of this CTA in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Waits as mbar_wait for a barrier that threads of the other CTA arrive on, too.
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, "
      "p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  const long long t0 = clock64();
  while (!try_wait_cluster(bar, parity)) {
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitCycles) {
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}
// kind::f8f6f4: fp32 accumulator, A and B e4m3; trans_b: B has its N axis contiguous.
__device__ __forceinline__ uint32_t idesc_e4m3(int M, int N, bool trans_b) {
  return (1u << 4) | (trans_b ? kIdescBMn : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Tiled copies; PAIR: the barrier may be the other CTA's (an address in the cluster).
template <bool PAIR>
__device__ __forceinline__ void copy_2d(uint32_t dst, const CUtensorMap* m, int c0, int c1, uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void copy_3d(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, "
        "%4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
  else
    tma_load_3d(dst, m, c0, c1, c2, bar);
}
// One arrival of a warp; PAIR: on a barrier of either CTA. It orders tensor-memory loads alone (they are complete, and
// fenced, before it), so it need not release other memory to the cluster: .release.cluster takes 1300 cycles here.
template <bool PAIR>
__device__ __forceinline__ void arrive_elect(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b64 st;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar)
        : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void alloc_tmem(uint32_t dst, uint32_t cols) {
  if constexpr (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst, cols);
    tmem_relinquish();
  }
}
template <bool PAIR>
__device__ __forceinline__ void free_tmem(uint32_t taddr, uint32_t cols) {
  if constexpr (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
  else
    tmem_dealloc(taddr, cols);
}
// Four values of a run of n (zeros behind it), from the i-th on; vec: they are one aligned 16-byte load.
__device__ __forceinline__ float4 load4(const float* p, int i, int n, int64_t stride, bool vec) {
  if (vec) return __ldg(reinterpret_cast<const float4*>(p + i));
  float v[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) v[u] = i + u < n ? __ldg(p + (i + u) * stride) : 0.f;
  return make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ float lds32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts32(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }
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

// An expert's rows. Offsets that all ascend within the rows give runs that do not overlap.
struct Range {
  int lo, hi;
  __device__ __forceinline__ bool bad(int rows) const { return lo < 0 || hi < lo || hi > rows; }
};
__device__ __forceinline__ Range expert_rows(const ProductParams& p, int e) {
  if (!p.offsets) return {0, p.rows};
  return {__ldg(p.offsets + e), __ldg(p.offsets + e + 1)};
}

// The i-th item of the work list; first[e]: the first one of expert e, in shared memory. A whole warp calls it.
// Row tiles of an expert go in groups of kGroupTiles; in a group the column tiles one after the other, each
// with all row tiles, so that the CTAs at work share both the rows' and the weights' tiles in L2.
template <int BN, int ITEM_M>
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
  const int rows = x.hi - x.lo, tiles = (rows + ITEM_M - 1) / ITEM_M;
  int in = i - first[a], base = 0;
  if (tiles > kGroupTiles) {
    const int per = kGroupTiles * col_tiles, group = in / per;
    in -= group * per;
    base = group * kGroupTiles;
  }
  const int n = min(kGroupTiles, tiles - base);
  const int ct = (int)__fdividef((float)in + 0.5f, (float)n);  // in < 2^13 and n <= 16: never near an integer
  const int rt = base + in - ct * n;
  return {a, x.lo + rt * ITEM_M, min(ITEM_M, rows - rt * ITEM_M), ct * BN};
}

// The part of an item that this CTA makes: 128 rows of it, or fewer, or none.
__device__ __forceinline__ Item part_of(Item it, int rank) {
  it.row0 += rank * kTileM;
  it.rows = max(0, min(kTileM, it.rows - rank * kTileM));
  return it;
}
__device__ __forceinline__ int box_of(int rows) { return rows > 64 ? 2 : rows > 32 ? 1 : 0; }

template <int BN, bool TRANS, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ ProductParams p, const __grid_constant__ ProductMaps maps) {
  using L = Layout<BN, PAIR>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int rank = PAIR ? blockIdx.x & 1 : 0;  // in the pair; 0 issues the MMAs
  const int item0 = PAIR ? blockIdx.x >> 1 : blockIdx.x, item_step = PAIR ? gridDim.x >> 1 : gridDim.x;
  const uint32_t bars = base + L::bar_off;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (L::kStages + s); };
  auto acc_full = [&](int b) { return bars + 8u * (2 * L::kStages + b); };
  auto acc_empty = [&](int b) { return bars + 8u * (2 * L::kStages + 2 + b); };
  auto f_full = [&](int s) { return bars + 8u * (2 * L::kStages + 4 + s); };
  auto f_empty = [&](int s) { return bars + 8u * (2 * L::kStages + 4 + kSlots + s); };
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + L::misc_off);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + L::misc_off + 4);

  if (tid == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), PAIR ? 2 * kSumWarps : kSumWarps);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(f_full(s), kScaleWarps);
      mbar_init(f_empty(s), kSumWarps);
    }
    *s_abort = 0;
    fence_barrier_init();
  }
  if (PAIR) {
    __syncthreads();
    cluster_sync();  // the other CTA's barriers are ready, too
  }
  if (warp == kWarpMma) alloc_tmem<PAIR>(smem_u32(s_tmem), L::kTmemCols);
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
    Range r[kPer];
    int items[kPer], sum = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      r[i] = e < p.n_experts ? expert_rows(p, e) : Range{0, 0};
      bad |= r[i].bad(p.rows);
    }
    bad = __syncthreads_or(bad);  // then there are no items at all
    if (blockIdx.x == 0 && tid == 0 && bad) raise_index(p.hdr);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      items[i] = bad ? 0 : (r[i].hi - r[i].lo + L::kItemM - 1) / L::kItemM * col_tiles;
      sum += items[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_sum[warp] = incl;
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
    for (int i = item0; i < n_items && ok; i += item_step) {
      const Item whole = find_item<BN, L::kItemM>(p, first, col_tiles, i), it = part_of(whole, rank);
      const int box = box_of(it.rows), col0 = it.col0 + rank * L::kBCols;
      // what lands in this CTA, or, where a pair's first CTA counts for both, in both
      uint32_t bytes = ((32u << box) * 128u) + L::kBBytes;
      if (PAIR) {
        const int other = part_of(whole, 1).rows;
        bytes += L::kBBytes + (other > 0 ? (32u << box_of(other)) * 128u : 0u);
      }
      if (lane == 0)
        for (int kb0 = 0; kb0 < kb_n; kb0 += L::kStep, ++g) {
          const int s = g % L::kStages;
          if (!(ok = mbar_wait(empty(s), ((g / L::kStages) & 1) ^ 1, s_abort))) break;
          const uint32_t bar = PAIR ? in_cta(full(s), 0) : full(s);
          if (rank == 0) mbar_arrive_expect_tx(full(s), bytes * min(L::kStep, kb_n - kb0));
#pragma unroll
          for (int u = 0; u < L::kStep; ++u) {
            const int kb = kb0 + u;
            if (kb >= kb_n) break;
            const uint32_t a = base + s * L::kStage + u * L::kBlock, b = a + L::kABytes;
            if (it.rows > 0) copy_2d<PAIR>(a, &maps.rows[box], kb * 128, it.row0, bar);
            if (TRANS) {
#pragma unroll
              for (int c = 0; c < L::kBCols / 128; ++c)
                copy_3d<PAIR>(b + c * 16384, &maps.w, col0 + c * 128, kb * 128, it.expert, bar);
            } else {
              copy_3d<PAIR>(b, &maps.w, kb * 128, col0, it.expert, bar);
            }
          }
        }
      ok = __shfl_sync(~0u, ok, 0);
    }
    if (!ok && lane == 0 && rank == 0)  // a wait gave up: the copies in flight land before the CTAs end
      for (int s = 0; s < L::kStages && (int)g - 1 - s >= 0; ++s) {
        const uint32_t h = g - 1 - s;
        const long long t0 = clock64();
        while (!mbar_try_wait(full(h % L::kStages), (h / L::kStages) & 1) && clock64() - t0 < kWaitCycles) {
        }
      }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA issue
    const uint32_t idesc = idesc_e4m3(L::kItemM, BN, TRANS);
    uint32_t g = 0;
    bool ok = true;
    for (int i = item0; i < n_items && ok && rank == 0; i += item_step)
      for (int kb = 0; kb < kb_n; kb += L::kStep, ++g) {
        const int s = g % L::kStages, buf = g & 1;
        const uint32_t par = (g / L::kStages) & 1, acc_par = ((g >> 1) & 1) ^ 1;
        const bool ready = PAIR ? try_wait_cluster(full(s), par) & try_wait_cluster(acc_empty(buf), acc_par)
                                : mbar_try_wait(full(s), par) & mbar_try_wait(acc_empty(buf), acc_par);
        if (!__all_sync(~0u, ready)) {
          ok = __all_sync(~0u, PAIR ? wait_cluster(full(s), par, s_abort) : mbar_wait(full(s), par, s_abort)) &&
               __all_sync(~0u, PAIR ? wait_cluster(acc_empty(buf), acc_par, s_abort) : mbar_wait(acc_empty(buf), acc_par, s_abort));
          if (!ok) break;
        }
        tc_fence_after();
#pragma unroll
        for (int u = 0; u < L::kStep; ++u) {
          if (kb + u >= kb_n) break;
          const uint32_t a = base + s * L::kStage + u * L::kBlock, b = a + L::kABytes, d = tmem + (buf * L::kStep + u) * BN;
          if (TRANS)
            mma_block<32 * 128 / 16, PAIR>(d, sw128_desc(a), sw128_mn_desc(b, 16384), idesc);
          else
            mma_block<2, PAIR>(d, sw128_desc(a), sw128_desc(b), idesc);
        }
        mma_commit<PAIR>(empty(s));
        mma_commit<PAIR>(acc_full(buf));
      }
    if (!ok && g) {  // a wait gave up: the MMAs in flight end before tensor memory is freed
      const long long t0 = clock64();
      while (!mbar_try_wait(empty((g - 1) % L::kStages), ((g - 1) / L::kStages) & 1) && clock64() - t0 < kWaitCycles) {
      }
    }
  } else if (warp < kWarpSum0) {
    // ------------------------------------------------------------ factors
    // Of four blocks at a time: each row's scale times that of the weights, for either half of the columns.
    // Rows past the tile and columns past the matrix get those of the last ones; their sums are not stored.
    const bool vec = kb_n % 4 == 0, vec_a = vec && p.a.scale_stride % 4 == 0 && (reinterpret_cast<uintptr_t>(p.a.scale) & 15) == 0;
    const bool vec_w = !TRANS && vec && (reinterpret_cast<uintptr_t>(p.wscale) & 15) == 0;
    const int r0 = (warp - kWarpScale0) * 64 + lane, w_stride = TRANS ? p.out_blocks : 1;
    uint32_t g = 0;
    bool ok = true;
    for (int i = item0; i < n_items && ok; i += item_step) {
      const Item it = part_of(find_item<BN, L::kItemM>(p, first, col_tiles, i), rank);
      const float *sa[2], *sw[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sa[h] = p.a.scale + min(it.row0 + min(r0 + 32 * h, max(it.rows - 1, 0)), p.rows - 1) * p.a.scale_stride;
        const int cb = min((it.col0 + h * (BN / 2)) / kScaleBlock, p.out_blocks - 1);
        sw[h] = p.wscale + (int64_t)it.expert * p.in_blocks * p.out_blocks + (TRANS ? cb : (int64_t)cb * p.in_blocks);
      }
      for (int kb = 0; kb < kb_n; kb += 4, ++g) {
        const int s = g % kSlots;
        float4 a[2], w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          a[h] = load4(sa[h], kb, kb_n, 1, vec_a);
          w[h] = load4(sw[h], kb, kb_n, w_stride, vec_w);
        }
        if (!(ok = __all_sync(~0u, mbar_wait(f_empty(s), ((g / kSlots) & 1) ^ 1, s_abort)))) break;
        const uint32_t f = base + L::f_off + s * kSlotBytes + r0 * 4;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            sts32(f + h * 512 + x * 128, a[x].x * w[h].x);
            sts32(f + 1 * 1024 + h * 512 + x * 128, a[x].y * w[h].y);
            sts32(f + 2 * 1024 + h * 512 + x * 128, a[x].z * w[h].z);
            sts32(f + 3 * 1024 + h * 512 + x * 128, a[x].w * w[h].w);
          }
        if (threadIdx.x == kWarpScale0 * 32)
          sts128(base + L::item_off + s * 16, make_uint4(it.row0, it.rows, it.col0, 0));
        __syncwarp();
        if (lane == 0) mbar_arrive(f_full(s));
      }
    }
  } else {
    // ------------------------------------------------------------ scaling, adding, output
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
    constexpr int kCols = BN / 2;  // columns of a warp
    const int quad = warp & 3, part = (warp - kWarpSum0) >> 2;
    const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + part * kCols;
    const uint32_t s_f = base + L::f_off + part * 512 + (quad * 32 + lane) * 4;
    const uint32_t s_out = base + L::out_off + (warp - kWarpSum0) * 2048;
    // After a wait that gave up, all later ones return at once, and what is computed is not stored.
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (!mbar_try_wait(bar, parity)) mbar_wait(bar, parity, s_abort);
      __syncwarp();
    };
    uint32_t g = 0, q = 0;
    uint32_t acc_free[2];
    for (int b = 0; b < 2; ++b) acc_free[b] = PAIR ? in_cta(acc_empty(b), 0) : acc_empty(b);
    for (int i = item0; i < n_items; i += item_step) {
      Item it;
      float acc[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
      for (int kb0 = 0; kb0 < kb_n; kb0 += 4, ++q) {
        const int s = q % kSlots;
        wait(f_full(s), (q / kSlots) & 1);
        float f4[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) f4[u] = lds32(s_f + s * kSlotBytes + u * 1024);
        if (kb0 == 0) {
          const float4 x = lds128(base + L::item_off + s * 16);
          it = {0, __float_as_int(x.x), __float_as_int(x.y), __float_as_int(x.z)};
        }
        __syncwarp();
        arrive_elect<false>(f_empty(s));
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (kb0 + u < kb_n) {
            const int buf = g & 1, in_step = u % L::kStep;
            const uint32_t from = taddr + (buf * L::kStep + in_step) * BN;
            if (in_step == 0) {
              wait(acc_full(buf), (g >> 1) & 1);
              tc_fence_after();
            }
            const bool last = in_step == L::kStep - 1 || kb0 + u + 1 == kb_n;  // of the step
            float v[2][32];  // the next 32 columns arrive while these are added
            tmem_ld32(from, v[0]);
#pragma unroll
            for (int c = 0; c < kCols; c += 32) {
              const int x = c / 32 & 1;
              tmem_wait_ld32(v[x]);
              if (c + 32 < kCols) {
                tmem_ld32(from + c + 32, v[x ^ 1]);
              } else if (last) {
                tc_fence_before();
                arrive_elect<PAIR>(acc_free[buf]);
                ++g;
              }
#pragma unroll
              for (int y = 0; y < 32; ++y) acc[c + y] = fmaf(f4[u], v[x][y], acc[c + y]);
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
  if (PAIR) cluster_sync();  // the other CTA arrives on no barrier of this one any more
  if (warp == kWarpMma) {
    __syncwarp();
    tc_fence_after();
    free_tmem<PAIR>(tmem, L::kTmemCols);
  }
  if (tid == 0 && *s_abort) set_device_status(p.hdr, MOE_ERR_DEVICE_TIMEOUT);
}

// Items at most: every expert that has rows has a row tile that is not full, the others are full ones.
int64_t most_items(const ProductParams& p, int tile, int columns) {
  const int hit = p.n_experts < p.rows ? p.n_experts : p.rows;
  return (int64_t)((p.rows - hit) / tile + hit) * ((p.outc + columns - 1) / columns);
}

// Pairs that run at once: a pair needs two SMs of one group, so that not every SM may find a partner.
int most_pairs() {
  static const int n = [] {
    using L = Layout<256, true>;
    auto kernel = product_kernel<256, false, true>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::most) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (sm_count() / 2));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::most;
    cudaLaunchAttribute a;
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = 2;
    a.val.clusterDim.y = a.val.clusterDim.z = 1;
    cfg.attrs = &a;
    cfg.numAttrs = 1;
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n : 0;
  }();
  return n;
}

template <int BN, bool TRANS, bool PAIR>
cudaError_t launch(const ProductParams& p, cudaStream_t s) {
  using L = Layout<BN, PAIR>;
  auto kernel = product_kernel<BN, TRANS, PAIR>;
  static const cudaError_t attr = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::most);
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
  const cuuint32_t wbox[3] = {128, TRANS ? 128u : (cuuint32_t)L::kBCols, 1};
  if (!encode_tiled(&maps.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, p.wq, wdims, wstr, wbox, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const int64_t items = most_items(p, L::kItemM, BN);
  const int at_once = PAIR ? most_pairs() : sm_count();
  if (at_once < 1) return cudaErrorInvalidConfiguration;
  const int grid = (items < at_once ? (int)items : at_once) * (PAIR ? 2 : 1);
  return launch_pdl(kernel, grid, kThreads, (size_t)(L::fixed + (p.n_experts + 1) * 4), PAIR ? 2 : 1, s, p, maps);
}

}  // namespace

int product_form(const ProductParams& p, int sms, int pairs) {
  if (product_is_small(p, sms)) return MOE_PRODUCT_FEW_ROWS;
  // Which width: a block of 128 inputs takes 0.25 us in an item of 128 columns, 0.46 in one of 256 and 0.44 in a pair's
  // 256 x 256, times the rounds of items over the SMs; but L2 hands out 21.6 TB/s at most, 32, 48 and 64 KB to an item
  // and block (0.0015, 0.0022, 0.0030 us), and rows that begin off 128-byte lines take 1.6 times that. Times in 0.1 ns.
  // (8192 x 8192 x 8192: 483, 432 and 420 us; 3236 rows of 6896 x 4464: 134, 126, 104; 1195 rows of 8 experts of 2640 x
  // 3264: 24.5, 32.6 and none.) A pair wants rows for both its CTAs: with 128 rows to an expert it loses a fifth, with 512 5%.
  const bool off = p.k % 128 || p.a.stride % 128;
  auto time = [&](int64_t items, int at_once, int block, int l2) {
    const int64_t a = (items + at_once - 1) / at_once * block, b = items * l2 * (off ? 16 : 10) / 10;
    return a > b ? a : b;
  };
  const int64_t narrow = time(most_items(p, kTileM, 128), sms, 2500, 15);
  const int64_t wide = time(most_items(p, kTileM, 256), sms, off ? 5600 : 4600, 22);
  if (p.rows >= kPairRows * (int64_t)p.n_experts && pairs > 0) {
    const int64_t pair = time(most_items(p, 2 * kTileM, 256), pairs, p.n_experts == 1 ? 4400 : 4700, 30);
    if (pair <= wide && pair <= narrow) return MOE_PRODUCT_PAIRS;
  }
  return wide < narrow ? MOE_PRODUCT_256 : MOE_PRODUCT_128;
}

cudaError_t launch_product(const ProductParams& p, cudaStream_t s) {
  const int pairs = p.rows >= kPairRows * (int64_t)p.n_experts ? most_pairs() : 0;  // else never asked for
  switch (product_form(p, sm_count(), pairs)) {
    case MOE_PRODUCT_FEW_ROWS: return launch_product_small(p, s);
    case MOE_PRODUCT_PAIRS: return p.transposed ? launch<256, true, true>(p, s) : launch<256, false, true>(p, s);
    case MOE_PRODUCT_256: return p.transposed ? launch<256, true, false>(p, s) : launch<256, false, false>(p, s);
    default: return p.transposed ? launch<128, true, false>(p, s) : launch<128, false, false>(p, s);
  }
}

}  // namespace moe
