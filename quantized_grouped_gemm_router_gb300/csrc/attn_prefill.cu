// moe_attn_prefill: attention over packed prompts on the tensor cores.
//
// For a tile of query rows, over tiles of BN keys: S = Q K^T (tcgen05, fp32 in tensor memory), the
// running maximum m and sum l of a softmax in registers, P = 2^(c S - c m) (c = scale log2 e) rounded
// to bf16 back into tensor memory over S, O += P V (tcgen05, O in tensor memory, P its A operand). K and
// V are read once per tile of rows; nothing of size rows x keys leaves the SM.
//
//  * Rows. The G query heads of one key-value head read the same keys, so a 128-row tile is 128 / G
//    positions x G heads: a K or V tile serves all of them, and the diagonal of a causal mask spans
//    few positions.
//  * Items. One CTA per SM stays and draws items: two row tiles over the same keys (kRows); one row tile
//    whose even and odd key tiles are two streams, each with its own O, m and l, added at the end (kKeys);
//    or one row tile (kOne, D = 256). Each sequence's last rows come first: under a causal mask they see
//    the most keys. The next item's copies and first scores run while the last one's output is written.
//  * Steps. Step n's scores go to S buffer n % 2. An MMA warp issues S of its first step, then for every
//    second step n: P(n) V, S(n + 2). The tensor cores thus work on one step while the softmax of the
//    other runs. There are two MMA warps: the issue of an MMA waits for the ones before it, and a warp's
//    waits for its operands (about 400 cycles a step, against 1170 of MMAs at D = 128) pass while the
//    other warp's MMAs run. They take turns, a step each: mixed, both steps' scores would be done at the
//    same time, and both softmaxes would run while the tensor cores idle.
//  * Rescaling. O is scaled down only when a row's maximum has grown by more than 2^8 since the last
//    time (weights up to 2^8 are as exact in bf16, and l and O have fp32's range): softmax warps read O
//    back on few tiles.
//  * Masks. A tile that every row sees takes no compare. Scores a row does not see become -inf, so
//    their weight is 0; but 0 times a NaN or infinity in V is not 0, so a warp checks the V tiles that
//    some row does not see whole, and a tile with such a value is multiplied by the softmax warps,
//    seen keys only (rare, and bounded by one tile's work).
//  * K and V tiles are one ring, filled by TMA in the order in which the MMA warps free them.
//  * Long contexts. Every 32768 keys of a stream O, l and m are put aside (Softmax::put_aside), so that what the
//    tensor cores' sums lose does not add up.
//
// Bound by the chain S -> softmax -> P V of the two streams: at D = 128 a step takes about 1500 cycles, 1170 of
// them the tensor cores' own. Measured (GB300): 16384 tokens, 16/2 heads of 128, causal: 0.73 to 0.75 ms, 1.47 to 1.51
// PFLOP/s (77 to 80% of a cuBLAS bf16 GEMM's burst rate); 1021 tokens on 8192, heads of 256: 0.123 ms, 1.18 PFLOP/s (62%),
// bound by the MMAs of 64-key tiles: one of 64 columns takes 67 cycles, as one of 128 does (one of 256 takes 129),
// so that 64 keys take 1600. Short sequences: an item costs 3 to 4 us beside its steps (start,
// check, the last product, the output): 24 texts of 250 tokens, 8 heads of 64, both ways: 27 us. Many
// sequences: an item is found by a search over the sequences from the first on, 32 at a step: 1024 sequences of 16
// tokens take 142 us, 4096 of 2 tokens 1.41 ms.
#include "attn_device.cuh"
#include "attn_ptx.cuh"

namespace moe {
namespace {

// The warpgroups share the block's registers out: 168 x 384 at launch, then 72 for
// the four issuing warps and 216 for each softmax thread (2 x 128 x 216 + 128 x 72 = 168 x 384).
constexpr int kLaunchRegs = 168;
__device__ __forceinline__ void regs_for_softmax() { asm volatile("setmaxnreg.inc.sync.aligned.u32 216;"); }
__device__ __forceinline__ void regs_for_issue() { asm volatile("setmaxnreg.dec.sync.aligned.u32 72;"); }

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.f;
constexpr int kPutKeys = 32768;  // keys of a stream that are summed up in tensor memory

// What a CTA's streams of steps are: two row tiles over the same keys, two halves of one row tile's keys
// (even and odd tiles), or one row tile alone (D = 256: tensor memory holds one O). In kOne both softmax
// warpgroups work on every step, half of its keys each, and Q is copied to tensor memory: with 64 keys to a
// tile, S = Q K^T reads three bytes of shared memory for each byte of K otherwise, and waits for them. Q passes
// through the ring, so that seven K and V tiles have room, not five (2% at 4096 tokens).
enum Mode { kRows, kKeys, kOne };

// 16 values of an output row: a whole 32-byte sector at a time if the rows are aligned so. A warp's 32 rows are
// 32 lines apart, and it is their number that such stores cost.
__device__ __forceinline__ void st256(uint16_t* p, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// a + 0 x b, a pair of bf16 each.
__device__ __forceinline__ uint32_t times0_add(uint32_t b, uint32_t a) {
  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(a) : "r"(b), "r"(0));
  return a;
}

template <int D, Mode M>
struct Cfg {
  static constexpr int NT = M == kOne ? 1 : 2;         // streams of steps, O tiles
  static constexpr int NQ = M == kRows ? 2 : 1;        // row tiles
  static constexpr int BN = D == 256 ? 64 : 128;       // keys per tile
  static constexpr int kChunks = D / 64;               // 128-byte columns of a row
  static constexpr int kQTile = kChunks * 16384;       // one row tile
  static constexpr int kQBytes = M == kOne ? 0 : NQ * kQTile;  // kOne: Q passes through two entries of the ring
  static constexpr int kQEntries = M == kOne ? 2 : 0;
  static constexpr int kSlot = BN * D * 2;             // one K or V tile
  static constexpr int kRoom = 224 * 1024 - kQBytes;  // all but the last 3 KB, which the kernel's own variables take
  static constexpr int kSlots = kRoom / kSlot < 8 ? kRoom / kSlot : 8;
  static constexpr int kSmem = kQBytes + kSlots * kSlot;
  static constexpr int kSoftWarps = 8;                 // a warpgroup per stream; kOne: one per half of a tile's keys
  static constexpr int kWarpMma = kSoftWarps, kWarpTma = kSoftWarps + 2, kWarpCheck = kSoftWarps + 3;  // two MMA warps
  static constexpr int kThreads = 32 * (kSoftWarps + 4);
  static constexpr uint32_t kOCol = 2 * BN;            // S buffers at 0 and BN, O tiles behind them
  static constexpr uint32_t kQCol = kOCol + D;         // kOne: Q
  static_assert(kOCol + NT * D + (M == kOne ? D / 2 : 0) <= 512 && kSlots >= 4 && kSmem + 3072 <= 232448, "on-chip memory");
};

struct Maps {
  CUtensorMap q, k, v;
};

// mbar_wait for what may take as long as an item (2^30 keys: about 3e10 cycles): until one of the others' waits, which
// all end within a few steps, has given up.
__device__ __forceinline__ bool mbar_wait_item(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (*abort_flag || clock64() - t0 > 64 * kWaitCycles) {
      *abort_flag = 1;
      return false;
    }
  return true;
}

// What a CTA works on.
struct Item {
  int head;          // key-value head, -1: there is no item
  int q_row, n_pos;  // first query row (absolute) and positions of this CTA
  int pos0;          // the first position within the sequence
  int k_row, lk;     // first key row and keys of the sequence
  int off;           // keys that query 0 sees before its own: lk - lq
};

// Tile `slot` of all sequences' tiles of P positions, each sequence's last tile first (under a causal
// mask it has the most keys). One warp; false if there is no such tile.
__device__ __forceinline__ bool find_item(const AttnPrefillParams& p, int slot, int P, Item& it) {
  const int lane = threadIdx.x & 31;
  for (int base = 0; base < p.n_seqs; base += 32) {
    const int i = base + lane;
    int q0 = 0, n = 0, k0 = 0, k1 = 0;
    if (i < p.n_seqs) {
      q0 = __ldg(p.cu_q + i);
      n = __ldg(p.cu_q + i + 1);
      k0 = __ldg(p.cu_k + i);
      k1 = __ldg(p.cu_k + i + 1);
      q0 = min(max(q0, 0), p.total_q);
      n = min(max(n, q0), p.total_q) - q0;
      k0 = min(max(k0, 0), p.total_k);
      k1 = min(max(k1, k0), p.total_k);
    }
    const int tiles = (n + P - 1) / P;
    int sum = tiles;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(~0u, sum, x);
      if (lane >= x) sum += y;
    }
    const unsigned m = __ballot_sync(~0u, sum > slot);
    if (m) {
      const int src = __ffs(m) - 1;
      const int mine = tiles - 1 - (slot - (sum - tiles));  // meaningful in lane src only
      const int tile = __shfl_sync(~0u, mine, src), lq = __shfl_sync(~0u, n, src);
      it.pos0 = tile * P;
      it.q_row = __shfl_sync(~0u, q0, src) + it.pos0;
      it.n_pos = min(P, lq - it.pos0);
      it.k_row = __shfl_sync(~0u, k0, src);
      it.lk = __shfl_sync(~0u, k1, src) - it.k_row;
      it.off = it.lk - lq;
      return true;
    }
    slot -= __shfl_sync(~0u, sum, 31);
  }
  return false;
}

// Adds seen weights x V to this thread's row of O, key by key, for 64 keys: for V tiles that hold a NaN or
// an infinity some row does not see. p_tmem: this row's bf16 weights; chunk: bytes between the 64-value
// columns of V.
template <int D>
__device__ __forceinline__ void add_seen(uint32_t o_tmem, uint32_t p_tmem, const uint8_t* v, int chunk, int seen, bool fresh) {
#pragma unroll 1
  for (int d0 = 0; d0 < D; d0 += 16) {
    uint32_t acc[16];
    __syncwarp();
    tmem_ld16(o_tmem + d0, acc);
    tmem_wait_ld16(acc);
    if (fresh)
      for (int i = 0; i < 16; ++i) acc[i] = 0u;
#pragma unroll 1
    for (int row = 0; row < 64; ++row) {
      __syncwarp();
      const uint32_t w = tmem_ld1(p_tmem + row / 2);
      if (row >= seen) continue;
      const float x = __uint_as_float(row & 1 ? w & 0xFFFF0000u : w << 16);
      const uint8_t* at = v + (d0 / 64) * chunk + row * 128;
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const uint32_t y = *reinterpret_cast<const uint32_t*>(at + (((d0 % 64 + i) * 2) ^ ((row & 7) << 4)));
        acc[i] = __float_as_uint(fmaf(x, __uint_as_float(y << 16), __uint_as_float(acc[i])));
        acc[i + 1] = __float_as_uint(fmaf(x, __uint_as_float(y & 0xFFFF0000u), __uint_as_float(acc[i + 1])));
      }
    }
    __syncwarp();
    tmem_st16(o_tmem + d0, acc);
    tmem_wait_st();
  }
}

template <int N>
__device__ __forceinline__ void unsee(float* s, int lim) {  // of N scores those from lim on
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = i < lim ? s[i] : -INFINITY;
}
template <int N>
__device__ __forceinline__ float max_of(const float* s) {
  float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int i = 4; i < N; i += 2) m[(i / 2) & 3] = max3(m[(i / 2) & 3], s[i], s[i + 1]);
  return max3(m[0], m[1], fmaxf(m[2], m[3]));
}

// The N values of O at ot and those put aside, times f (none if first), added: OUT: put aside, O becomes 0; else into O.
template <int N, bool OUT>
__device__ __forceinline__ void add_aside(uint32_t ot, float4* at, float f, bool first) {
#pragma unroll 1
  for (int i = 0; i < N; i += 16) {
    uint32_t o[16];
    tmem_ld16(ot + i, o);
    tmem_wait_ld16(o);
#pragma unroll
    for (int x = 0; x < 16; x += 4) {
      float4* p = at + (i + x) / 4 * 128;
      float4 y = first ? make_float4(0.f, 0.f, 0.f, 0.f) : *p;
      y.x = fmaf(y.x, f, __uint_as_float(o[x]));
      y.y = fmaf(y.y, f, __uint_as_float(o[x + 1]));
      y.z = fmaf(y.z, f, __uint_as_float(o[x + 2]));
      y.w = fmaf(y.w, f, __uint_as_float(o[x + 3]));
      if (OUT) {
        *p = y;
        y = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      o[x] = __float_as_uint(y.x);
      o[x + 1] = __float_as_uint(y.y);
      o[x + 2] = __float_as_uint(y.z);
      o[x + 3] = __float_as_uint(y.w);
    }
    tmem_st16(ot + i, o);
  }
  tmem_wait_st();
}
template <int N, bool OUT>
__device__ __noinline__ void add_aside_call(uint32_t ot, float4* at, float f, bool first) {
  add_aside<N, OUT>(ot, at, f, first);
}

// One row's running softmax. Weights are relative to m, which follows the maximum only when that has
// grown by more than 2^8.
struct Softmax {
  float c, grown;            // scale log2 e; the growth of a score that m follows
  float m = -INFINITY, mc = 0.f;  // mc = c m, 0 while m = -inf
  uint64_t l[2] = {0, 0};    // the sum of the weights, four parts of it
  __device__ __forceinline__ explicit Softmax(float c_) : c(c_), grown(kRescaleLog2 / c_) {}

  // Takes mx into m; the factor by which what was summed so far shrinks.
  __device__ __forceinline__ float raise(float mx) {
    const float m2 = fmaxf(m, mx), mc2 = m2 == -INFINITY ? 0.f : m2 * c;
    const float f = m == -INFINITY ? 0.f : ex2(mc - mc2);
    m = m2;
    mc = mc2;
    const uint64_t f2 = pack2(f, f);
    l[0] = mul2(l[0], f2);
    l[1] = mul2(l[1], f2);
    return f;
  }
  template <int N>
  __device__ __forceinline__ void scale_o(uint32_t ot, float f) const {
#pragma unroll 1
    for (int i = 0; i < N; i += 16) {  // few values at a time: the scores are live; rarely run
      uint32_t o[16];
      tmem_ld16(ot + i, o);
      tmem_wait_ld16(o);
#pragma unroll
      for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
      tmem_st16(ot + i, o);
    }
  }
  // The weights of N scores, as bf16 to tensor memory.
  template <int N>
  __device__ __forceinline__ void weights(const float* s, uint32_t to) {
    const uint64_t c2 = pack2(c, c), mc2 = pack2(-mc, -mc);
#pragma unroll
    for (int i = 0; i < N; i += 32) {
      uint32_t w[16];
#pragma unroll
      for (int x = 0; x < 32; x += 2) {
        float p0, p1;
        unpack2(fma2(pack2(s[i + x], s[i + x + 1]), c2, mc2), p0, p1);
        p0 = ex2(p0);
        p1 = ex2(p1);
        l[(x / 2) & 1] = add2(l[(x / 2) & 1], pack2(p0, p1));
        w[x / 2] = bf16x2_rn(p0, p1);
      }
      tmem_st16(to + i / 2, w);
    }
  }
  // Long contexts. Each product that the tensor cores add to O takes about 2^-23 of O's size from it, always towards
  // zero: after 32768 keys with values of one sign O is 0.03% low, after 4 million it was 2.5%. So every kPutKeys keys
  // of a stream the row's O, l and m are put aside, in memory that only this thread reads, and O starts from 0 again.
  // to: the row's first four values, 128 float4 further the next four; ml: (m c, l). O is at rest.
  // CALL: not inlined, for want of registers (1024 tokens on 131072, heads of 256: 2.5% slower inlined).
  template <int N, bool CALL>
  __device__ __forceinline__ void put_aside(uint32_t ot, float4* to, float2* ml, bool first) {
    const float2 before = first ? make_float2(-INFINITY, 0.f) : *ml;
    const float f = ex2(before.x - mc);
    *ml = make_float2(m == -INFINITY ? -INFINITY : mc, fmaf(before.y, f, sum()));
    l[0] = l[1] = 0;
    CALL ? add_aside_call<N, true>(ot, to, f, first) : add_aside<N, true>(ot, to, f, first);
  }
  // Back into O and l for the output.
  template <int N, bool CALL>
  __device__ __forceinline__ void take_back(uint32_t ot, float4* from, const float2* ml) {
    const float2 before = *ml;
    const float f = ex2(before.x - mc);
    l[0] = add2(l[0], pack2(before.y * f, 0.f));
    CALL ? add_aside_call<N, false>(ot, from, f, false) : add_aside<N, false>(ot, from, f, false);
  }
  __device__ __forceinline__ float sum() const {
    float x[4];
    unpack2(l[0], x[0], x[1]);
    unpack2(l[1], x[2], x[3]);
    return (x[0] + x[1]) + (x[2] + x[3]);
  }
};

template <int D, Mode M, bool LONG>
__global__ void __launch_bounds__(Cfg<D, M>::kThreads, 1)
    attn_prefill_kernel(const __grid_constant__ AttnPrefillParams p, const __grid_constant__ Maps maps) {
  using C = Cfg<D, M>;
  constexpr int BN = C::BN, NT = C::NT, NQ = C::NQ, kSlots = C::kSlots;
  extern __shared__ __align__(1024) uint8_t smem[];  // the 128-byte swizzle repeats every 1024 bytes
  __shared__ float2 s_stat[M == kKeys ? 2 : 1][M == kKeys ? 128 : 1];  // m c and l of the streams' rows
  __shared__ float s_half[2][2][M == kOne ? 128 : 1];  // kOne: the row maxima of half a tile's keys, of two steps
  __shared__ Item s_item[2];
  __shared__ int s_abort_flag, s_bad_flag[2];
  __shared__ uint32_t s_tmem;
  __shared__ __align__(8) uint64_t s_bar[30 + (NQ == 1 ? 3 : 2) * kSlots];
  uint8_t* ring = smem + C::kQBytes;
  volatile int* s_abort = &s_abort_flag;
  volatile int* s_bad = s_bad_flag;  // [2] V tile (the count of tiles not seen whole, % 2) holds a non-finite value
  const uint32_t bars = smem_u32(s_bar);
  const uint32_t q_full = bars, q_free = bars + 8, merged = bars + 16;
  const auto pair = [&](int which, int b) { return bars + 24 + 16 * which + 8 * b; };
  const auto s_full = [&](int b) { return pair(0, b); };    // scores of a step are there
  const auto p_half = [&](int b) { return pair(1, b); };    // the first half of its weights
  const auto p_ready = [&](int b) { return pair(2, b); };   // all of them
  const auto pv_half = [&](int a) { return pair(3, a); };   // stream a's O holds the first half's product
  const auto pv_done = [&](int a) { return pair(4, a); };   // and the second's
  const auto check = [&](int b) { return pair(5, b); };     // a V tile may be checked
  const auto checked = [&](int b) { return pair(6, b); };   // s_bad[b] is set
  const auto turn = [&](int i) { return pair(7, i); };      // MMA warp i may issue
  const auto o_free = [&](int a) { return pair(8, a); };    // stream a's O has been read
  const auto item_full = [&](int x) { return pair(9, x); };
  const auto item_free = [&](int x) { return pair(10, x); };
  const uint32_t q_there = bars + 200;                              // kOne: Q is in tensor memory
  const auto halves = [&](int w) { return bars + 208 + 8 * w; };    // kOne: the two warps of 32 rows have exchanged
  const auto kv_free = [&](int s) { return bars + 240 + 8 * s; };
  // a ring slot's copy is there: for both MMA warps (two row tiles: both use every copy), else for the one
  // that uses it, which thus sees every phase of a barrier
  const auto kv_full = [&](int i, int s) { return bars + 240 + 8 * kSlots * (NQ == 1 ? 1 + i : 1) + 8 * s; };

  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int G = p.group, Ppt = 128 / G;  // positions per row tile

  const auto item_at = [&](int idx) {  // all lanes of a warp
    Item it;
    it.head = find_item(p, idx / p.hkv, NQ * Ppt, it) ? idx % p.hkv : -1;
    return it;
  };
  Item it;  // the TMA warp's first one
  if (warp == C::kWarpMma) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  } else if (warp == C::kWarpCheck && lane == 0) {
    *s_abort = 0;
    mbar_init(q_full, 1);
    mbar_init(q_free, 2);
    mbar_init(q_there, 8);
    for (int w = 0; w < 4; ++w) mbar_init(halves(w), 2);
    mbar_init(merged, 8);
    for (int b = 0; b < 2; ++b) {
      mbar_init(s_full(b), 1);
      mbar_init(p_half(b), M == kOne ? 8 : 4);
      mbar_init(p_ready(b), M == kOne ? 8 : 4);
      mbar_init(pv_half(b), 1);
      mbar_init(pv_done(b), 1);
      mbar_init(check(b), NQ);
      mbar_init(checked(b), 1);
      mbar_init(turn(b), 1);
      mbar_init(o_free(b), M == kRows ? 4 : 8);
      mbar_init(item_full(b), 1);
      mbar_init(item_free(b), C::kSoftWarps + 3);
    }
    for (int s = 0; s < kSlots; ++s) {
      for (int i = 0; i < 3 - NQ; ++i) mbar_init(kv_full(i, s), 1);
      mbar_init(kv_free(s), NQ);
    }
    fence_barrier_init();
  } else if (warp == C::kWarpTma) {
    if (lane == 0) {
      prefetch_tmap(&maps.q);
      prefetch_tmap(&maps.k);
      prefetch_tmap(&maps.v);
    }
    pdl_wait();
    it = item_at(blockIdx.x);
    if (blockIdx.x == 0) {
      check_offsets(p.cu_q, p.n_seqs, p.total_q, p.hdr, lane, 32);
      check_offsets(p.cu_k, p.n_seqs, p.total_k, p.hdr, lane, 32);
    }
  }
  pdl_wait();  // nothing of this call's data is read or written before
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  // Every role walks the same items with the same running counts: r (ring entries used), nb (steps before
  // this item: the global step number gives a step's S buffer, MMA warp, stream and barrier phases), x0
  // (V tiles checked). Step n of an item: key tile n / NQ; global number nb + n. With two row tiles the
  // ring's order is K0 V0 K1 V1 ... (each used by two steps), else K0 K1 V0 K2 V1 ...
  const auto wait = [&](uint32_t bar, int parity) { return __all_sync(~0u, mbar_wait(bar, parity & 1, s_abort)); };
  // the same for the warp that checks V tiles, which has nothing to do for most of an item
  const auto wait_item = [&](uint32_t bar, int parity) { return __all_sync(~0u, mbar_wait_item(bar, parity & 1, s_abort)); };
  // the t-th item of this CTA; the slot is handed back
  const auto take_item = [&](int t, Item& it) {
    if (!(warp == C::kWarpCheck ? wait_item(item_full(t & 1), t >> 1) : wait(item_full(t & 1), t >> 1))) return false;
    it = s_item[t & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(item_free(t & 1));
    return it.head >= 0;
  };
  struct Span {
    int nj, steps, masked, first;  // key tiles, steps, the first tile that not every row sees whole; keys every row sees
  };
  const auto span = [&](const Item& it) {
    const int first = p.causal ? min(max(it.pos0 + 1 + it.off, 0), it.lk) : it.lk;         // keys the first position sees
    const int last = p.causal ? min(max(it.pos0 + it.n_pos + it.off, 0), it.lk) : it.lk;   // and the last
    const int nj = (last + BN - 1) / BN;
    return Span{nj, NQ * nj, first / BN, first};
  };
  const auto k_at = [&](int j) { return NQ == 2 ? 2 * j : (j == 0 ? 0 : 2 * j - 1); };
  const auto v_at = [&](int j, int nj) { return NQ == 2 ? 2 * j + 1 : (j == nj - 1 ? 2 * j + 1 : 2 * j + 2); };

  struct Entry {
    bool v;
    int j;
  };
  const auto tile_at = [](int i, int nj) {  // what the i-th entry holds
    if (NQ == 2) return Entry{(i & 1) != 0, i / 2};
    if (i == 2 * nj - 1) return Entry{true, nj - 1};
    const bool v = i >= 2 && !(i & 1);
    return Entry{v, v ? i / 2 - 1 : (i + 1) / 2};
  };

  if (warp >= C::kSoftWarps) {
    regs_for_issue();
    if (warp == C::kWarpTma) {
      // ------------------------------------------------------------------ items and copies
      int r = 0, nb = 0, q_used = 0, t = 0;
      bool ok = true;
      for (;; ++t) {
        if (t >= 2 && !(ok = wait(item_free(t & 1), (t >> 1) + 1))) break;
        if (lane == 0) {
          s_item[t & 1] = it;
          mbar_arrive(item_full(t & 1));
        }
        __syncwarp();
        if (it.head < 0) break;
        int next = 0;
        if (lane == 0) {
          const Span sp = span(it);
          if (sp.nj) {
            ok = q_used == 0 || mbar_wait(q_free, (q_used & 1) ^ 1, s_abort);
            if (ok) {
              mbar_arrive_expect_tx(q_full, (uint32_t)(NQ * C::kChunks * Ppt * G * 128));
              for (int a = 0; a < NQ; ++a)
                for (int c = 0; c < C::kChunks; ++c) {
                  uint32_t to = smem_u32(smem) + a * C::kQTile + c * 16384;
                  if (M == kOne) {
                    const int s = r % kSlots;
                    if (r >= kSlots && !(ok = mbar_wait(kv_free(s), ((r / kSlots) & 1) ^ 1, s_abort))) break;
                    to = smem_u32(ring) + s * C::kSlot + (c & 1) * 16384;
                    r += c & 1;
                  }
                  tma_load_3d(to, &maps.q, c * 64, it.head * G, it.q_row + a * Ppt, q_full);
                }
              ++q_used;
            }
          }
          for (int i = 0; ok && i < 2 * sp.nj; ++i, ++r) {
            const int s = r % kSlots;
            if (r >= kSlots && !(ok = mbar_wait(kv_free(s), ((r / kSlots) & 1) ^ 1, s_abort))) break;
            const Entry en = tile_at(i, sp.nj);
            const uint32_t full = kv_full((nb + en.j) & 1, s);
            mbar_arrive_expect_tx(full, (uint32_t)C::kSlot);
            for (int c = 0; c < C::kChunks; ++c)
              tma_load_3d(smem_u32(ring) + s * C::kSlot + c * (BN * 128), en.v ? &maps.v : &maps.k, c * 64, it.head,
                          it.k_row + en.j * BN, full);
          }
          nb += sp.steps;
          next = atomicAdd(&p.hdr->pad[0], 1);  // drawn when all copies have been issued: the next free CTA's item
        }
        if (!(ok = __all_sync(~0u, ok))) break;
        it = item_at(gridDim.x + __shfl_sync(~0u, next, 0));
      }
      // The next kernel may start when every CTA has had its only item (4 tokens: 6.7 -> 6.3 us a call); in calls of
      // more items it would take SMs over one by one (1 to 10% slower).
      if (t <= 1) pdl_launch_dependents();
      // this CTA draws no more (after a wait that gave up, too): the last one to say so puts the counts back
      if (lane == 0 && atomicAdd(&p.hdr->pad[1], 1) == (int)gridDim.x - 1) {
        p.hdr->pad[0] = 0;
        p.hdr->pad[1] = 0;
      }
      if (lane == 0 && *s_abort) {
        // copies in flight must land before the CTA's memory is given up: nothing tells which barriers they
        // complete any more, so give them their time (a copy takes microseconds)
        const long long t0 = clock64();
        while (clock64() - t0 < 20000000) __nanosleep(1000);
      }
    } else if (warp < C::kWarpMma + 2) {
      // ------------------------------------------------------------------ MMA issuer of every second step
      constexpr uint32_t kSChunk = BN * 128 / 16, kQChunk = 16384 / 16;
      const int me = warp - C::kWarpMma, a = me % NT;
      const uint32_t idesc_s = idesc_f16(128, BN, false), idesc_o = idesc_f16(128, D, false) | kIdescBMn;
      const uint64_t qd = sw128_desc(smem_u32(smem) + me % NQ * C::kQTile);
      int r = 0, nb = 0, x0 = 0, used = 0;  // used: items with keys before this one
      uint32_t phases = 0;                  // of kv_full, a bit per slot
      bool ok = true;
      for (int t = 0; ok && take_item(t, it); ++t) {
        const Span sp = span(it);
        if (sp.nj == 0) continue;
        const auto have = [&](int i) {  // ring entry r + i; each of this warp's entries once
          const int s = (r + i) % kSlots;
          const bool there = wait(kv_full(me, s), phases >> s);
          phases ^= 1u << s;
          return there;
        };
        const auto scores = [&](int n) {
          const int j = n / NQ, s = (r + k_at(j)) % kSlots, b = (nb + n) & 1;
          tc_fence_after();
          const uint64_t kd = sw128_desc(smem_u32(ring) + s * C::kSlot);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            if (M == kOne)
              umma_f16_ts_k64_elect(tmem + b * BN, tmem + C::kQCol + c * 32, kd + c * kSChunk, idesc_s, c != 0);
            else
              umma_f16_ss_k64_elect(tmem + b * BN, qd + c * kQChunk, kd + c * kSChunk, idesc_s, c != 0);
          umma_commit_elect(s_full(b));
          umma_commit_elect(kv_free(s));
          if (M != kOne && n + 2 >= sp.steps) umma_commit_elect(q_free);
        };
        // V tile of step n, if not every row sees it whole, to the warp that checks it: it has arrived, and s_bad of
        // two tiles before has been read (by this warp, or before its last turn)
        const auto offer = [&](int n) {
          const int j = n / NQ;
          if (j < sp.masked) return true;
          if (!have(v_at(j, sp.nj))) return false;
          if (lane == 0) mbar_arrive(check((x0 + j - sp.masked) & 1));
          __syncwarp();
          return true;
        };
        const int n0 = (me - nb) & 1;
        if (!(ok = wait(M == kOne ? q_there : q_full, used))) break;
        if (M == kOne) {
          if (lane == 0) {
            mbar_arrive(q_free);  // (a warp without a step must not miss a phase)
            mbar_arrive(kv_free((r + me) % kSlots));
          }
          r += C::kQEntries;
        }
        __syncwarp();
        if (n0 >= sp.steps) {  // a single step, the other warp's
          if (M != kOne && lane == 0) mbar_arrive(q_free);
        } else if ((ok = have(k_at(n0 / NQ)))) {
          scores(n0);
          ok = offer(n0);
        }
        for (int n = n0; ok && n < sp.steps; n += 2) {
          const int j = n / NQ, g = nb + n, s = (r + v_at(j, sp.nj)) % kSlots;
          const bool more = n + 2 < sp.steps;
          if (!(ok = (j >= sp.masked || have(v_at(j, sp.nj))) && (!more || have(k_at((n + 2) / NQ))) &&
                     wait(p_half(g & 1), g >> 1)))
            break;
          if (n < NT && used && !(ok = wait(o_free(a), used - 1))) break;
          if (g > 0 && !(ok = wait(turn(me), me ? g >> 1 : (g >> 1) - 1))) break;
          tc_fence_after();
          const bool skip = j >= sp.masked && s_bad[(x0 + j - sp.masked) & 1];  // the softmax warps add this product
          const uint64_t vd = sw128_mn_desc(smem_u32(ring) + s * C::kSlot, BN * 128);
#pragma unroll
          for (int kb = 0; kb < BN / 64; ++kb) {
            if (kb == BN / 128) {
              if (BN == 128) umma_commit_elect(pv_half(a));
              if (!(ok = wait(p_ready(g & 1), g >> 1))) break;
              tc_fence_after();
            }
            if (!skip)
              umma_f16_ts_mn_k64_elect(tmem + C::kOCol + a * D, tmem + (g & 1) * BN + kb * 32, vd + kb * (64 * 128 / 16),
                                       idesc_o, n / NT + kb != 0);
          }
          if (!ok) break;
          umma_commit_elect(pv_done(a));
          umma_commit_elect(kv_free(s));
          if (more) scores(n + 2);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(turn(1 - me));
          __syncwarp();
          if (more && !(ok = offer(n + 2))) break;
        }
        r += 2 * sp.nj;
        nb += sp.steps;
        x0 += sp.nj - sp.masked;
        ++used;
      }
    } else if (warp == C::kWarpCheck) {
      // ------------------------------------------------------------------ V tiles not seen whole
      int r = 0, x = 0;
      bool ok = true;
      for (int t = 0; ok && take_item(t, it); ++t) {
        const Span sp = span(it);
        if (sp.nj) r += C::kQEntries;
        for (int j = sp.masked; j < sp.nj; ++j, ++x) {
          const int s = (r + v_at(j, sp.nj)) % kSlots, b = x & 1;
          if (!(ok = wait_item(check(b), x >> 1))) break;
          // 0 times a NaN or an infinity is a NaN, 0 times all else is 0; 32 keys at a time, from the first that some
          // row does not see
          uint32_t h0 = 0, h1 = 0, h2 = 0, h3 = 0;
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c) {
            const uint4* v = reinterpret_cast<const uint4*>(ring + s * C::kSlot + c * (BN * 128)) + lane;
            for (int y = max(sp.first - j * BN, 0) / 32 * 256; y < BN * 8; y += 256) {
#pragma unroll
              for (int z = 0; z < 256; z += 32) {
                const uint4 w = v[y + z];
                h0 = times0_add(w.x, h0);
                h1 = times0_add(w.y, h1);
                h2 = times0_add(w.z, h2);
                h3 = times0_add(w.w, h3);
              }
            }
          }
          const bool bad = __any_sync(~0u, ((h0 | h1 | h2 | h3) & 0x7FFF7FFFu) != 0);
          if (lane == 0) {
            s_bad[b] = bad;
            mbar_arrive(checked(b));
          }
        }
        r += 2 * sp.nj;
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax of stream a, or of half the keys
    regs_for_softmax();
    const int wg = warp / 4, a = wg % NT, row = threadIdx.x & 127;
    constexpr int kCols = M == kRows ? D : D / 2;  // of O, that this warpgroup scales (kOne) and writes
    const int col0 = M == kRows ? 0 : wg * kCols;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 TMEM lanes
    const uint32_t ot = lanes + C::kOCol + a * D;
    constexpr int kPut = kPutKeys / BN;  // steps of a stream between two times that it puts its sums aside
    constexpr int kPutCols = M == kOne ? kCols : D;
    const uint32_t put_ot = ot + (M == kOne ? col0 : 0);
    const auto put_o = [&] { return reinterpret_cast<float4*>(p.aside + (int64_t)(blockIdx.x * 2 + wg) * (128 * D)) + row; };
    const auto put_ml = [&] { return p.aside_ml + (blockIdx.x * 2 + wg) * 128 + row; };
    int r = 0, nb = 0, x0 = 0, used = 0;
    int exchanged = 0;  // kOne
    // kOne: this thread's value and the other half's of the same row
    const auto exchange = [&](float mine, float& other) {
      const int b = exchanged & 1;
      s_half[b][wg][row] = mine;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(halves(warp & 3));
      if (!wait(halves(warp & 3), exchanged)) return false;
      tc_fence_after();
      other = s_half[b][1 - wg][row];
      ++exchanged;
      return true;
    };
    bool ok = true;
    for (int t = 0; ok && take_item(t, it); ++t) {
      const Span sp = span(it);
      const int pos = a % NQ * Ppt + row / G, head = it.head * G + row % G;
      const bool valid = row < Ppt * G && pos < it.n_pos;
      // keys this row sees (rows of no position: all, so that they add no compares)
      const int seen = !valid ? sp.nj * BN : p.causal ? min(max(it.pos0 + pos + 1 + it.off, 0), it.lk) : it.lk;
      Softmax soft(p.scale * kLog2e);
      if (!valid) soft.grown = INFINITY;  // what such a row holds decides nothing for the others of its warp
      const auto grow = [&](float mx, bool first, uint32_t bar, int parity) {
        if (!__any_sync(~0u, mx > soft.m + soft.grown)) return true;
        const float f = soft.raise(mx);
        if (first) return true;
        if (!wait(bar, parity)) return false;  // O is at rest
        tc_fence_after();
        soft.template scale_o<M == kOne ? kCols : D>(ot + (M == kOne ? col0 : 0), f);
        return true;
      };
      if (M == kOne && sp.nj) {
        // Q to tensor memory (every S of the last item has been made: its last scores have been read)
        if (!(ok = wait(q_full, used))) break;
#pragma unroll
        for (int c = 0; c < C::kChunks / 2; ++c) {
          const uint8_t* q = ring + (r + wg) % kSlots * C::kSlot + c * 16384 + row * 128;
          uint4 v[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) v[x] = *reinterpret_cast<const uint4*>(q + ((x ^ (row & 7)) << 4));
          tmem_st32(lanes + C::kQCol + (wg * (C::kChunks / 2) + c) * 32, reinterpret_cast<const uint32_t*>(v));
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_there);
        r += C::kQEntries;
      }
      int last = -1;  // this stream's last step's number within the stream, over all items
      int n = NT == 2 ? (a - nb) & 1 : 0;
      const int begin = n;
      for (int end = LONG ? min(NT * kPut, sp.steps) : sp.steps;;) {  // up to where the sums are put aside, or the last step
        for (; n < end; n += NT) {
          const int j = n / NQ, g = nb + n, b = g & 1, k = NT == 2 ? g >> 1 : g;
          const bool first = n < NT;
          const uint32_t st = lanes + b * BN;
          last = k;
          if (!(ok = wait(s_full(b), g >> 1))) break;
          tc_fence_after();
          // Two halves (BN = 128): the second one's scores are on their way while the first one's weights are
          // made, the first one's product is under way while the second one's are.
          const bool masked = j >= sp.masked;
          const int lim = seen - j * BN, x = x0 + j - sp.masked;
          if constexpr (M == kOne) {
            float s[32], other;
            tmem_ld32(st + wg * 32, s);
            tmem_wait_ld32(s);
            if (masked) unsee<32>(s, lim - wg * 32);
            const float mine = max_of<32>(s);
            if (!(ok = exchange(mine, other) && grow(fmaxf(mine, other), first, pv_done(a), k - 1))) break;
            soft.template weights<32>(s, st + wg * 16);
            tmem_wait_st();
            if (masked) {
              if (!(ok = wait(checked(x & 1), x >> 1))) break;
              if (s_bad[x & 1]) {
                // both halves' weights are there, and O is at rest
                if (!(ok = exchange(0.f, other) && (first ? used == 0 || wait(o_free(a), used - 1) : wait(pv_done(a), k - 1)))) break;
                tc_fence_after();
                add_seen<kCols>(ot + col0, st, ring + (r + v_at(j, sp.nj)) % kSlots * C::kSlot + wg * (C::kChunks / 2) * (BN * 128),
                                BN * 128, lim, first);
              }
            }
            // The end of the item waits for the last product. A wait tells a phase from the next one only, and these
            // scores came after all products but the last two: the one before the last is waited for here, while
            // the last one cannot have been made.
            if (n > 0 && n == end - 1 && !(ok = wait(pv_done(a), k - 1))) break;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(p_half(b));
              mbar_arrive(p_ready(b));
            }
            continue;
          }
          float s0[64], s1[64], mx = -INFINITY;
          bool bad = false;
          tmem_ld32(st, s0);
          tmem_ld32(st + 32, s0 + 32);
          tmem_wait_ld32(s0);
          tmem_wait_ld32(s0 + 32);
          if (BN == 128) {
            tmem_ld32(st + 64, s1);
            tmem_ld32(st + 96, s1 + 32);
          }
          if (masked) unsee<64>(s0, lim);
          if (!(ok = grow(max_of<64>(s0), first, pv_done(a), k - 1))) break;
          soft.template weights<64>(s0, st);
          if (BN == 128) {
            tmem_wait_ld32(s1);
            tmem_wait_ld32(s1 + 32);
            if (masked) unsee<64>(s1, lim - 64);
            mx = max_of<64>(s1);
          }
          tmem_wait_st();
          if (masked) {
            if (!(ok = wait(checked(x & 1), x >> 1))) break;
            bad = s_bad[x & 1];
            if (bad) {
              // O at rest: its last product, or (a new item's first) read by every warp
              if (!(ok = first ? used == 0 || wait(o_free(a), used - 1) : wait(pv_done(a), k - 1))) break;
              tc_fence_after();
              add_seen<D>(ot, st, ring + (r + v_at(j, sp.nj)) % kSlots * C::kSlot, BN * 128, lim, first);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_half(b));
          if (BN == 128) {
            if (!(ok = grow(mx, false, pv_half(a), k))) break;
            soft.template weights<64>(s1, st + 32);
            tmem_wait_st();
            if (bad)
              add_seen<D>(ot, st + 32, ring + (r + v_at(j, sp.nj)) % kSlots * C::kSlot + 64 * 128, BN * 128, lim - 64, false);
            tc_fence_before();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(p_ready(b));
        }
        if (ok && last >= 0) ok = wait(pv_done(a), last);
        if (!LONG || !ok || end == sp.steps) break;
        tc_fence_after();
        if (n < sp.steps) soft.template put_aside<kPutCols, M == kOne>(put_ot, put_o(), put_ml(), end == NT * kPut);
        end = min(end + NT * kPut, sp.steps);
      }
      if (LONG && ok && sp.steps > begin + NT * kPut) {
        tc_fence_after();
        soft.template take_back<kPutCols, M == kOne>(put_ot, put_o(), put_ml());
      }
      // the factor of O (kKeys: of the even tiles' O and the odd tiles') in the output, and the row's log sum
      float f = 0.f, f2 = 0.f, lse = -INFINITY;
      float l = soft.sum(), l_other;
      if (M == kOne && sp.nj && ok && (ok = exchange(l, l_other))) l = wg ? l_other + l : l + l_other;
      if (M == kKeys && sp.nj) {
        // both streams' O belong to the same rows (the same lanes): each warpgroup writes half the columns. Which
        // stream had the even tiles depends on the items drawn before; the sums' order does not.
        const float mc = l == 0.f ? -INFINITY : soft.mc;
        if (ok && used) ok = wait(o_free(a), used - 1);  // the other warpgroup has read the last item's statistics
        s_stat[a][row] = make_float2(mc, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(merged);
        __syncwarp();
        if (ok) ok = wait(merged, used);
        const float2 even = s_stat[nb & 1][row], odd = s_stat[1 - (nb & 1)][row];  // (m c, l)
        const float top = fmaxf(even.x, odd.x);
        if (even.y != 0.f || odd.y != 0.f) {
          const float w = even.y == 0.f ? 0.f : ex2(even.x - top), w2 = odd.y == 0.f ? 0.f : ex2(odd.x - top);
          const float sum = fmaf(w, even.y, w2 * odd.y);
          f = w / sum;
          f2 = w2 / sum;
          lse = top * kLn2 + logf(sum);
        }
      } else if (l != 0.f) {
        f = 1.f / l;
        lse = soft.mc * kLn2 + logf(l);
      }
      if (!ok) break;
      tc_fence_after();
      const int64_t token = it.q_row + pos;
      const bool both = M == kKeys && sp.steps > 1;  // else the even tiles' O is all there is
      const uint32_t src = (M == kKeys ? lanes + C::kOCol + (nb & 1) * D : ot) + col0;
      const uint32_t src2 = lanes + C::kOCol + (1 - (nb & 1)) * D + col0;
      const uint64_t ff = pack2(f, f), ff2 = pack2(f2, f2);
      uint16_t* out = p.o + (token * p.hq + head) * D + col0;
      constexpr int kPiece = M == kKeys || kCols < 64 ? 32 : 64;  // columns to a wait, as many as the registers hold
#pragma unroll 1
      for (int i = 0; i < kCols; i += kPiece) {
        float o[kPiece], o2[kPiece];
        if (sp.nj) {
#pragma unroll
          for (int y = 0; y < kPiece; y += 32) {
            tmem_ld32(src + i + y, o + y);
            if (both) tmem_ld32(src2 + i + y, o2 + y);
          }
#pragma unroll
          for (int y = 0; y < kPiece; y += 32) {
            tmem_wait_ld32(o + y);
            if (both) tmem_wait_ld32(o2 + y);
          }
          if (i + kPiece == kCols) {  // O may be overwritten
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(o_free(a));
              if (M == kKeys) mbar_arrive(o_free(1 - a));
            }
          }
        }
        uint32_t w[kPiece / 2];
        if (both) {
#pragma unroll
          for (int y = 0; y < kPiece / 2; ++y) {
            float u, v;
            unpack2(fma2(pack2(o2[2 * y], o2[2 * y + 1]), ff2, mul2(pack2(o[2 * y], o[2 * y + 1]), ff)), u, v);
            w[y] = bf16x2_rn(u, v);
          }
        } else if (sp.nj) {
#pragma unroll
          for (int y = 0; y < kPiece / 2; ++y) w[y] = bf16x2_rn(o[2 * y] * f, o[2 * y + 1] * f);
        } else {
#pragma unroll
          for (int y = 0; y < kPiece / 2; ++y) w[y] = 0u;
        }
        if (valid) {
#pragma unroll
          for (int y = 0; y < kPiece / 2; y += 8) st256(out + i + 2 * y, w + y, p.o_wide);
        }
      }
      if (valid && p.lse && (M == kRows || wg == 0)) p.lse[token * p.hq + head] = lse;
      r += 2 * sp.nj;
      nb += sp.steps;
      x0 += max(sp.nj - sp.masked, 0);
      used += sp.nj > 0;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *s_abort) set_device_status(p.hdr, MOE_ERR_DEVICE_TIMEOUT);
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

// [tokens, heads, d] rows as (d, heads, tokens); one box is 64 values x box_heads x box_tokens.
bool make_map(CUtensorMap* m, const moe_heads_view& v, int d, int heads, int tokens, int box_heads, int box_tokens) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)v.head_stride * 2, (cuuint64_t)v.token_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, v.p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, Mode M, bool LONG = true>
cudaError_t launch(const AttnPrefillParams& p, cudaStream_t s) {
  using C = Cfg<D, M>;
  static cudaError_t attr = cudaFuncSetAttribute(attn_prefill_kernel<D, M, LONG>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (attr != cudaSuccess) return attr;
  // the register split waits for ever unless the launch brings what it hands out
  static int regs = [] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, attn_prefill_kernel<D, M, LONG>) == cudaSuccess ? a.numRegs : 0;
  }();
  if (regs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  const int ppt = 128 / p.group;
  Maps maps;
  // without keys no tile of K or V is read: any valid map will do
  const bool keys = p.total_k > 0;
  if (!make_map(&maps.q, p.q, D, p.hq, p.total_q, p.group, ppt) ||
      !make_map(&maps.k, keys ? p.k : p.q, D, keys ? p.hkv : p.hq, keys ? p.total_k : p.total_q, 1, C::BN) ||
      !make_map(&maps.v, keys ? p.v : p.q, D, keys ? p.hkv : p.hq, keys ? p.total_k : p.total_q, 1, C::BN))
    return cudaErrorInvalidValue;
  // every sequence has at most one ragged tile
  const int64_t items = ((int64_t)p.total_q / (C::NQ * ppt) + (p.n_seqs < p.total_q ? p.n_seqs : p.total_q)) * p.hkv;
  if (items > 0x40000000) return cudaErrorInvalidValue;
  return launch_pdl(attn_prefill_kernel<D, M, LONG>, dim3((unsigned)(items < num_sms() ? items : num_sms())), C::kThreads,
                    (size_t)C::kSmem, 1, s, p, maps);
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnPrefillParams& p, int d, cudaStream_t s) {
  // Two row tiles per CTA halve the K and V traffic and the items; one row tile with its keys split halves the
  // longest item. Measured at 16/2 heads of 128, one prompt: 2048 tokens (0.8 items of two row tiles per SM) 37.2
  // against 27.8 us split, 3000 tokens (1.2) 44.4 against 42.6, 4096 tokens (1.7) 59.4 against 67.9, 16384 tokens 729
  // against 803 us. Several sequences have shorter items, and the two streams of a split one wait for each other
  // at its end: 16 prompts in 1600 tokens (0.8) 12.5 against 13.2, 24 in 3000 (1.3) 16.3 against 20.1; below 0.75 items
  // per SM the split fills them better (8 in 1000 tokens, 0.4: 13.7 against 10.3). Under a causal mask that holds for
  // items of few positions; one of 256 works for half its time on keys that half its rows do not see (24 prompts
  // in 6001 tokens, 8/8 heads: 33.3 against 26.6).
  const int rows = 2 * (128 / p.group);  // positions of an item of two row tiles
  const int64_t sms = num_sms(), each = (p.total_q + p.n_seqs - 1) / p.n_seqs;
  const bool two = 10 * ((int64_t)p.total_q / rows * p.hkv) >= 13 * sms ||
                   (p.n_seqs > 1 && (!p.causal || rows <= 64) && 4 * ((each + rows - 1) / rows * p.n_seqs * p.hkv) >= 3 * sms);
  if (d == 64) return two ? launch<64, kRows>(p, s) : launch<64, kKeys>(p, s);
  if (d == 128) return two ? launch<128, kRows>(p, s) : launch<128, kKeys>(p, s);
  // Heads of 256: the code that puts sums aside costs registers that the softmax needs (4096 tokens: 109.9 us without
  // it, 111.9 with it), so that calls with fewer keys take a form without it.
  // 1024 tokens on 131072 keys take 1687 us with sums put aside, 1648 without.
  return p.total_k > kPutKeys ? launch<256, kOne, true>(p, s) : launch<256, kOne, false>(p, s);
}

}  // namespace moe
