// moe_attn_prefill: attention over packed prompts on the tensor cores.
//
// For a tile of query rows, over tiles of BN keys: S = Q K^T (tcgen05, fp32 in tensor memory), the
// running maximum m and sum l of a softmax in registers, P = 2^(c S - c m) (c = scale log2 e) rounded
// to bf16 back into tensor memory over S, O += P V (tcgen05, O in tensor memory, P its A operand). K and
// V are read once per tile of rows; nothing of size rows x keys leaves the SM.
//
//  * Rows. The G query heads of one key-value head read the same keys, so a 128-row tile is 128 / G
//    positions x G heads: a K or V tile serves all of them, and the diagonal of a causal mask spans
//    few positions. One CTA holds NT tiles of rows (each with its own softmax warps).
//  * Steps. Step n is (key tile n / NT, row tile n % NT); its scores go to S buffer n % 2. An MMA warp
//    issues S of its first step, then for every second step n: P(n) V, S(n + 2). The tensor cores thus
//    work on one step while the softmax of the other runs, with two row tiles (NT = 2) as with one.
//    There are two MMA warps: the issue of an MMA waits for the ones before it, and a warp's waits for
//    its operands (about 400 cycles a step, against 1024 of MMAs at D = 128) pass while the other
//    warp's MMAs run. They take turns, a step each: mixed, both steps' scores would be done at the same
//    time, and both softmaxes would run while the tensor cores idle.
//  * Rescaling. O is scaled down only when a row's maximum has grown by more than 2^8 since the last
//    time (weights up to 2^8 are as exact in bf16, and l and O have fp32's range): softmax warps read O
//    back on few tiles.
//  * Masks. A tile that every row sees takes no compare. Scores a row does not see become -inf, so
//    their weight is 0; but 0 times a NaN or infinity in V is not 0, so a warp checks the V tiles that
//    some row does not see whole, and a tile with such a value is multiplied by the softmax warps,
//    seen keys only (rare, and bounded by one tile's work).
//  * K and V tiles are one ring, filled by TMA in the order in which the MMA warp frees them.
#include "attn_device.cuh"
#include "attn_ptx.cuh"

namespace moe {
namespace {

// With two row tiles the warpgroups share the block's registers out: 168 x 384 at launch, then 72 for
// the four issuing warps and 216 for each softmax thread (2 x 128 x 216 + 128 x 72 = 168 x 384).
constexpr int kLaunchRegs = 168;
__device__ __forceinline__ void regs_for_softmax() { asm volatile("setmaxnreg.inc.sync.aligned.u32 216;"); }
__device__ __forceinline__ void regs_for_issue() { asm volatile("setmaxnreg.dec.sync.aligned.u32 72;"); }

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.f;

// What a CTA's streams of steps are: two row tiles over the same keys, two halves of one row tile's keys
// (even and odd tiles), or one row tile alone (D = 256: tensor memory holds one O).
enum Mode { kRows, kKeys, kOne };

template <int D, Mode M>
struct Cfg {
  static constexpr int NT = M == kOne ? 1 : 2;         // streams: softmax warpgroups, O tiles
  static constexpr int NQ = M == kRows ? 2 : 1;        // row tiles
  static constexpr int BN = D == 256 ? 64 : 128;       // keys per tile
  static constexpr int kChunks = D / 64;               // 128-byte columns of a row
  static constexpr int kQTile = kChunks * 16384;       // one row tile
  static constexpr int kSlot = BN * D * 2;             // one K or V tile
  static constexpr int kRoom = (M == kKeys ? 222 : 224) * 1024 - NQ * kQTile;  // kKeys: the streams' statistics
  static constexpr int kSlots = kRoom / kSlot < 8 ? kRoom / kSlot : 8;
  static constexpr int kSmem = NQ * kQTile + kSlots * kSlot + 1024 + 512;  // + alignment + barriers
  static constexpr int kSoftWarps = 4 * NT;
  static constexpr int kWarpMma = kSoftWarps, kWarpTma = kSoftWarps + 2, kWarpCheck = kSoftWarps + 3;  // two MMA warps
  static constexpr int kThreads = 32 * (kSoftWarps + 4);
  static constexpr uint32_t kOCol = 2 * BN;            // S buffers at 0 and BN, O tiles behind them
  static_assert(kOCol + NT * D <= 512 && kSlots >= 4 && kSmem <= 232448, "on-chip memory");
};

struct Maps {
  CUtensorMap q, k, v;
};

// What a CTA works on.
struct Item {
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
    int q0 = 0, n = 0;
    if (i < p.n_seqs) {
      q0 = min(max(__ldg(p.cu_q + i), 0), p.total_q);
      n = min(max(__ldg(p.cu_q + i + 1), q0), p.total_q) - q0;
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
      const int s = base + src;
      it.pos0 = tile * P;
      it.q_row = __shfl_sync(~0u, q0, src) + it.pos0;
      it.n_pos = min(P, lq - it.pos0);
      it.k_row = min(max(__ldg(p.cu_k + s), 0), p.total_k);
      it.lk = min(max(__ldg(p.cu_k + s + 1), it.k_row), p.total_k) - it.k_row;
      it.off = it.lk - lq;
      return true;
    }
    slot -= __shfl_sync(~0u, sum, 31);
  }
  return false;
}

// Adds seen weights x V to this thread's row of O, key by key: for V tiles that hold a NaN or an
// infinity some row does not see. P: this row's bf16 weights in tensor memory.
template <int D, int BN>
__device__ __forceinline__ void add_seen(uint32_t o_tmem, uint32_t p_tmem, const uint8_t* v, int seen, bool fresh) {
#pragma unroll 1
  for (int d0 = 0; d0 < D; d0 += 32) {
    float acc[32];
    tmem_ld32(o_tmem + d0, acc);
    tmem_wait_ld();
    if (fresh)
      for (int i = 0; i < 32; ++i) acc[i] = 0.f;
    for (int row = 0; row < BN; ++row) {
      __syncwarp();
      const uint32_t w = tmem_ld1(p_tmem + row / 2);
      if (row >= seen) continue;
      const float x = __uint_as_float(row & 1 ? w & 0xFFFF0000u : w << 16);
      const uint8_t* at = v + (d0 / 64) * (BN * 128) + row * 128;
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const uint32_t y = *reinterpret_cast<const uint32_t*>(at + (((d0 % 64 + i) * 2) ^ ((row & 7) << 4)));
        acc[i] = fmaf(x, __uint_as_float(y << 16), acc[i]);
        acc[i + 1] = fmaf(x, __uint_as_float(y & 0xFFFF0000u), acc[i + 1]);
      }
    }
    __syncwarp();
    tmem_st32(o_tmem + d0, reinterpret_cast<uint32_t*>(acc));
    tmem_wait_st();
  }
}

template <int N>
__device__ __forceinline__ float max_of(const float* s) {
  float m[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
  for (int i = 4; i < N; i += 2) m[(i / 2) & 3] = max3(m[(i / 2) & 3], s[i], s[i + 1]);
  return max3(m[0], m[1], fmaxf(m[2], m[3]));
}

// One row's running softmax. Weights are relative to m, which follows the maximum only when that has
// grown by more than 2^8.
template <int D>
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
  __device__ __forceinline__ void scale_o(uint32_t ot, float f) const {
#pragma unroll
    for (int i = 0; i < D; i += 16) {  // few values at a time: the scores are live
      uint32_t o[16];
      tmem_ld16(ot + i, o);
      tmem_wait_ld();
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
  __device__ __forceinline__ float sum() const {
    float x[4];
    unpack2(l[0], x[0], x[1]);
    unpack2(l[1], x[2], x[3]);
    return (x[0] + x[1]) + (x[2] + x[3]);
  }
};

template <int D, Mode M>
__global__ void __launch_bounds__(Cfg<D, M>::kThreads, 1)
    attn_prefill_kernel(const __grid_constant__ AttnPrefillParams p, const __grid_constant__ Maps maps) {
  using C = Cfg<D, M>;
  constexpr int BN = C::BN, NT = C::NT, NQ = C::NQ;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = smem + NQ * C::kQTile;
  uint8_t* misc = ring + C::kSlots * C::kSlot;
  __shared__ float2 s_stat[M == kKeys ? 2 : 1][M == kKeys ? 128 : 1];  // m c and l of the streams' rows
  volatile int* s_abort = reinterpret_cast<volatile int*>(misc);
  volatile int* s_bad = reinterpret_cast<volatile int*>(misc + 4);  // [2] V tile (counted from j_masked, % 2) holds a non-finite value
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(misc + 12);
  Item* s_item = reinterpret_cast<Item*>(misc + 16);
  int* s_found = reinterpret_cast<int*>(misc + 48);
  const uint32_t bars = smem_u32(misc + 64);
  const uint32_t q_full = bars;
  const auto s_full = [&](int b) { return bars + 8 + 8 * b; };
  const auto p_ready = [&](int b) { return bars + 24 + 8 * b; };
  const auto pv_done = [&](int a) { return bars + 40 + 8 * a; };
  const auto checked = [&](int b) { return bars + 56 + 8 * b; };
  const auto check = [&](int b) { return bars + 72 + 8 * b; };
  const auto p_half = [&](int b) { return bars + 88 + 8 * b; };
  const auto turn = [&](int a) { return bars + 104 + 8 * a; };
  const auto pv_half = [&](int a) { return bars + 120 + 8 * a; };
  const uint32_t merged = bars + 136;
  const auto kv_full = [&](int s) { return bars + 144 + 8 * s; };
  const auto kv_free = [&](int s) { return bars + 144 + 8 * C::kSlots + 8 * s; };

  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int G = p.group, Ppt = 128 / G;  // positions per row tile
  const int kvh = blockIdx.x % p.hkv, slot = blockIdx.x / p.hkv;

  if (warp == 0) {
    Item it;
    const bool found = find_item(p, slot, NQ * Ppt, it);
    if (lane == 0) {
      *s_found = found;
      if (found) *s_item = it;
    }
    if (blockIdx.x == 0) {
      check_offsets(p.cu_q, p.n_seqs, p.total_q, p.hdr, lane, 32);
      check_offsets(p.cu_k, p.n_seqs, p.total_k, p.hdr, lane, 32);
    }
  } else if (warp == C::kWarpMma) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  } else if (warp == C::kWarpTma && lane == 0) {
    *s_abort = 0;
    mbar_init(q_full, 1);
    mbar_init(merged, 8);
    for (int b = 0; b < 2; ++b) {
      mbar_init(s_full(b), 1);
      mbar_init(p_half(b), 4);
      mbar_init(p_ready(b), 4);
      mbar_init(pv_done(b), 1);
      mbar_init(checked(b), 1);
      mbar_init(turn(b), 1);
      mbar_init(pv_half(b), 1);
      mbar_init(check(b), NQ);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_free(s), NQ);
    }
    fence_barrier_init();
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const bool found = *s_found;

  if (found) {
    const Item it = *s_item;
    // keys that the first and the last position of this CTA see
    const int first_seen = p.causal ? min(max(it.pos0 + 1 + it.off, 0), it.lk) : it.lk;
    const int last_seen = p.causal ? min(max(it.pos0 + it.n_pos + it.off, 0), it.lk) : it.lk;
    const int nj = (last_seen + BN - 1) / BN, steps = NQ * nj;
    const int j_masked = first_seen / BN;  // tiles from here on are not seen whole by every row
    // Step n: key tile n / NQ, stream n % NT, the stream's step n / NT. The ring's order is the steps' order of
    // use: K0 V0 K1 V1 ... with two row tiles (each used by two steps), else K0 K1 V0 K2 V1 ...
    const auto k_idx = [&](int j) { return NQ == 2 ? 2 * j : (j == 0 ? 0 : 2 * j - 1); };
    const auto v_idx = [&](int j) { return NQ == 2 ? 2 * j + 1 : (j == nj - 1 ? 2 * j + 1 : 2 * j + 2); };

    if (warp >= C::kSoftWarps) {
    if (NT == 2) regs_for_issue();
    if (warp == C::kWarpTma) {
      // ------------------------------------------------------------------ TMA producer
      if (lane == 0 && steps) {
        mbar_arrive_expect_tx(q_full, (uint32_t)(NQ * C::kChunks * Ppt * G * 128));
        for (int a = 0; a < NQ; ++a)
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_3d(smem_u32(smem) + a * C::kQTile + c * 16384, &maps.q, c * 64, kvh * G, it.q_row + a * Ppt, q_full);
        int issued = 0;
        for (; issued < 2 * nj; ++issued) {
          const int i = issued, s = i % C::kSlots;
          if (i >= C::kSlots && !mbar_wait(kv_free(s), ((i / C::kSlots) & 1) ^ 1, s_abort)) break;
          bool is_v;
          int j;
          if (NQ == 2) {
            is_v = i & 1;
            j = i / 2;
          } else if (i == 2 * nj - 1) {
            is_v = true;
            j = nj - 1;
          } else {
            is_v = i >= 2 && !(i & 1);
            j = is_v ? i / 2 - 1 : (i + 1) / 2;
          }
          mbar_arrive_expect_tx(kv_full(s), (uint32_t)C::kSlot);
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_3d(smem_u32(ring) + s * C::kSlot + c * (BN * 128), is_v ? &maps.v : &maps.k, c * 64, kvh,
                        it.k_row + j * BN, kv_full(s));
        }
        if (*s_abort) {  // copies in flight must land before the CTA's memory is given up
          int none = 0;
          mbar_wait(q_full, 0, &none);
          for (int i = max(0, issued - C::kSlots); i < issued; ++i)
            mbar_wait(kv_full(i % C::kSlots), (i / C::kSlots) & 1, &none);
        }
      }
    } else if (warp < C::kWarpMma + 2) {
      // ------------------------------------------------------------------ MMA issuer of the steps n0, n0 + 2, ...
      constexpr uint32_t kSChunk = BN * 128 / 16, kQChunk = 16384 / 16;
      const int n0 = warp - C::kWarpMma, a = n0 % NT;
      const uint32_t idesc_s = idesc_f16(128, BN, false), idesc_o = idesc_f16(128, D, false) | kIdescBMn;
      const uint64_t qd = sw128_desc(smem_u32(smem) + n0 % NQ * C::kQTile);
      const auto wait = [&](uint32_t bar, int parity) { return __all_sync(~0u, mbar_wait(bar, parity & 1, s_abort)); };
      const auto have_k = [&](int n) {
        const int i = k_idx(n / NQ);
        return wait(kv_full(i % C::kSlots), i / C::kSlots);
      };
      const auto scores = [&](int n) {
        const int j = n / NQ, s = k_idx(j) % C::kSlots;
        tc_fence_after();
        const uint64_t kd = sw128_desc(smem_u32(ring) + s * C::kSlot);
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
          umma_f16_ss_k64_elect(tmem + (n & 1) * BN, qd + c * kQChunk, kd + c * kSChunk, idesc_s, c != 0);
        umma_commit_elect(s_full(n & 1));
        umma_commit_elect(kv_free(s));
        // every copy before V tile j's into its slot has arrived (it is an earlier one than K tile j's), and
        // this warp has read s_bad of tile j - 2: the check of V tile j may begin
        if (j >= j_masked && lane == 0) mbar_arrive(check((j - j_masked) & 1));
        __syncwarp();
      };
      bool ok = n0 < steps && wait(q_full, 0) && have_k(n0);
      if (ok) scores(n0);
      for (int n = n0; ok && n < steps; n += 2) {
        const int j = n / NQ, i = v_idx(j), s = i % C::kSlots;
        const bool more = n + 2 < steps;
        if (!(ok = wait(kv_full(s), i / C::kSlots) && (!more || have_k(n + 2)) && wait(p_half(n & 1), n >> 1))) break;
        if (n > 0 && !(ok = wait(turn(n0), n0 ? n >> 1 : (n >> 1) - 1))) break;
        tc_fence_after();
        const bool skip = j >= j_masked && s_bad[(j - j_masked) & 1];  // the softmax warps add this product
        const uint64_t vd = sw128_mn_desc(smem_u32(ring) + s * C::kSlot, BN * 128);
#pragma unroll
        for (int kb = 0; kb < BN / 64; ++kb) {
          if (kb == BN / 128) {
            if (BN == 128) umma_commit_elect(pv_half(a));
            if (!(ok = wait(p_ready(n & 1), n >> 1))) break;
            tc_fence_after();
          }
          if (!skip)
            umma_f16_ts_mn_k64_elect(tmem + C::kOCol + a * D, tmem + (n & 1) * BN + kb * 32, vd + kb * (64 * 128 / 16),
                                     idesc_o, n / NT + kb != 0);
        }
        if (!ok) break;
        umma_commit_elect(pv_done(a));
        umma_commit_elect(kv_free(s));
        if (more) scores(n + 2);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(turn(1 - n0));
      }
    } else if (warp == C::kWarpCheck) {
      // ------------------------------------------------------------------ V tiles not seen whole
      for (int j = j_masked; j < nj; ++j) {
        const int i = v_idx(j), s = i % C::kSlots, x = j - j_masked, b = x & 1;
        if (!__all_sync(~0u, mbar_wait(check(b), (x >> 1) & 1, s_abort) && mbar_wait(kv_full(s), (i / C::kSlots) & 1, s_abort))) break;
        const uint4* v = reinterpret_cast<const uint4*>(ring + s * C::kSlot);
        uint32_t hit = 0;
#pragma unroll 8
        for (int y = lane; y < C::kSlot / 16; y += 32) {
          const uint4 w = v[y];
          const uint32_t e = 0x7F807F80u, one = 0x00800080u;  // exponent 255: + 1 carries into the sign's place
          hit |= ((w.x & e) + one) | ((w.y & e) + one) | ((w.z & e) + one) | ((w.w & e) + one);
        }
        const bool bad = __any_sync(~0u, hit & 0x80008000u);
        if (lane == 0) {
          s_bad[b] = bad;
          mbar_arrive(checked(b));
        }
      }
    }
    } else {
      // ------------------------------------------------------------------ softmax of row tile a
      if (NT == 2) regs_for_softmax();
      const int a = warp / 4, row = threadIdx.x & 127;
      const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);  // this warp's 32 TMEM lanes
      const int pos = a % NQ * Ppt + row / G, head = kvh * G + row % G;
      const bool valid = row < Ppt * G && pos < it.n_pos;
      // keys this row sees (rows of no position: all, so that they add no compares)
      const int seen = !valid ? nj * BN : p.causal ? min(max(it.pos0 + pos + 1 + it.off, 0), it.lk) : it.lk;
      Softmax<D> soft(p.scale * kLog2e);
      const uint32_t ot = lanes + C::kOCol + a * D;
      const auto grow = [&](float mx, bool first, uint32_t bar, int parity) {
        if (!__any_sync(~0u, mx > soft.m + soft.grown)) return true;
        const float f = soft.raise(mx);
        if (first) return true;
        if (!__all_sync(~0u, mbar_wait(bar, parity & 1, s_abort))) return false;  // O is at rest
        tc_fence_after();
        soft.scale_o(ot, f);
        return true;
      };
      bool ok = true;
      for (int n = a; n < steps; n += NT) {
        const int j = n / NQ, k = n / NT;  // key tile, step of this stream
        const uint32_t st = lanes + (n & 1) * BN;
        if (!(ok = __all_sync(~0u, mbar_wait(s_full(n & 1), (n >> 1) & 1, s_abort)))) break;
        tc_fence_after();
        if (BN == 128 && j < j_masked) {
          // seen whole by every row: two halves, the second one's scores on their way while the first one's
          // weights are made, the first one's product under way while the second one's are
          float s0[64], s1[64];
          tmem_ld32(st, s0);
          tmem_ld32(st + 32, s0 + 32);
          tmem_wait_ld32(s0);
          tmem_wait_ld32(s0 + 32);
          tmem_ld32(st + 64, s1);
          tmem_ld32(st + 96, s1 + 32);
          if (!(ok = grow(max_of<64>(s0), k == 0, pv_done(a), k - 1))) break;
          soft.template weights<64>(s0, st);
          tmem_wait_ld32(s1);
          tmem_wait_ld32(s1 + 32);
          const float mx = max_of<64>(s1);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_half(n & 1));
          if (!(ok = grow(mx, false, pv_half(a), k))) break;
          soft.template weights<64>(s1, st + 32);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_ready(n & 1));
          continue;
        }
        const int lim = seen - j * BN;
        {
          float s[BN];
#pragma unroll
          for (int i = 0; i < BN; i += 32) tmem_ld32(st + i, s + i);
#pragma unroll
          for (int i = 0; i < BN; i += 32) tmem_wait_ld32(s + i);
          if (j >= j_masked) {
#pragma unroll
            for (int i = 0; i < BN; ++i) s[i] = i < lim ? s[i] : -INFINITY;
          }
          if (!(ok = grow(max_of<BN>(s), k == 0, pv_done(a), k - 1))) break;
          soft.template weights<BN>(s, st);
        }
        tmem_wait_st();
        if (j >= j_masked) {
          const int x = j - j_masked;
          if (!(ok = __all_sync(~0u, mbar_wait(checked(x & 1), (x >> 1) & 1, s_abort)))) break;
          if (s_bad[x & 1]) {
            const int i = v_idx(j);
            ok = mbar_wait(kv_full(i % C::kSlots), (i / C::kSlots) & 1, s_abort) &&
                 (k == 0 || mbar_wait(pv_done(a), (k - 1) & 1, s_abort));
            if (!(ok = __all_sync(~0u, ok))) break;
            tc_fence_after();
            add_seen<D, BN>(ot, st, ring + (i % C::kSlots) * C::kSlot, lim, k == 0);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(p_half(n & 1));
          mbar_arrive(p_ready(n & 1));
        }
      }
      const int mine = (steps - a + NT - 1) / NT;  // steps of this stream
      if (mine && ok) ok = __all_sync(~0u, mbar_wait(pv_done(a), (mine - 1) & 1, s_abort));
      // the factor of O (and of the other stream's O) in the output, and the row's log sum
      float f = 0.f, f2 = 0.f, lse = -INFINITY;
      const float l = soft.sum();
      if (M == kKeys) {
        // both streams' O belong to the same rows (the same lanes): each warpgroup writes half the columns
        const float mc = l == 0.f ? -INFINITY : soft.mc;
        s_stat[a][row] = make_float2(mc, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(merged);
        __syncwarp();
        if (ok) ok = __all_sync(~0u, mbar_wait(merged, 0, s_abort));
        const float2 other = s_stat[1 - a][row];
        const float top = fmaxf(mc, other.x);
        if (l != 0.f || other.y != 0.f) {
          const float w = l == 0.f ? 0.f : ex2(mc - top), w2 = other.y == 0.f ? 0.f : ex2(other.x - top);
          const float sum = fmaf(w, l, w2 * other.y);
          f = w / sum;
          f2 = w2 / sum;
          lse = top * kLn2 + logf(sum);
        }
      } else if (l != 0.f) {
        f = 1.f / l;
        lse = soft.mc * kLn2 + logf(l);
      }
      if (ok) {
        tc_fence_after();
        constexpr int kCols = M == kKeys ? D / 2 : D;
        const int col0 = M == kKeys ? a * kCols : 0;
        const int64_t t = it.q_row + pos;
        uint16_t* out = p.o + (t * p.hq + head) * D + col0;
#pragma unroll
        for (int i = 0; i < kCols; i += 32) {
          float o[32], o2[32];
          if (steps) {
            tmem_ld32(ot + col0 + i, o);
            if (M == kKeys) tmem_ld32(lanes + C::kOCol + (1 - a) * D + col0 + i, o2);
            tmem_wait_ld32(o);
            if (M == kKeys) tmem_wait_ld32(o2);
          }
          if (valid) {
#pragma unroll
            for (int x = 0; x < 32; x += 8) {
              uint32_t w[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                // a factor of 0: nothing was written there
                float u = f == 0.f ? 0.f : o[x + 2 * y] * f, v = f == 0.f ? 0.f : o[x + 2 * y + 1] * f;
                if (M == kKeys && f2 != 0.f) {
                  u = fmaf(o2[x + 2 * y], f2, u);
                  v = fmaf(o2[x + 2 * y + 1], f2, v);
                }
                w[y] = bf16x2_rn(u, v);
              }
              *reinterpret_cast<uint4*>(out + i + x) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        if (valid && p.lse && (M != kKeys || a == 0)) p.lse[t * p.hq + head] = lse;
      }
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

// [tokens, heads, d] rows as (d, heads, tokens); one box is 64 values x box_heads x box_tokens.
bool make_map(CUtensorMap* m, const moe_heads_view& v, int d, int heads, int tokens, int box_heads, int box_tokens) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)v.head_stride * 2, (cuuint64_t)v.token_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, v.p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, Mode M>
cudaError_t launch(const AttnPrefillParams& p, cudaStream_t s) {
  using C = Cfg<D, M>;
  static cudaError_t attr = cudaFuncSetAttribute(attn_prefill_kernel<D, M>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (attr != cudaSuccess) return attr;
  if (C::NT == 2) {  // the register split waits for ever unless the launch brings what it hands out
    static int regs = [] {
      cudaFuncAttributes a;
      return cudaFuncGetAttributes(&a, attn_prefill_kernel<D, M>) == cudaSuccess ? a.numRegs : 0;
    }();
    if (regs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  }
  const int ppt = 128 / p.group;
  Maps maps;
  // without keys no tile of K or V is read: any valid map will do
  const bool keys = p.total_k > 0;
  if (!make_map(&maps.q, p.q, D, p.hq, p.total_q, p.group, ppt) ||
      !make_map(&maps.k, keys ? p.k : p.q, D, keys ? p.hkv : p.hq, keys ? p.total_k : p.total_q, 1, C::BN) ||
      !make_map(&maps.v, keys ? p.v : p.q, D, keys ? p.hkv : p.hq, keys ? p.total_k : p.total_q, 1, C::BN))
    return cudaErrorInvalidValue;
  // every sequence has at most one ragged tile
  const int64_t tiles = (int64_t)p.total_q / (C::NQ * ppt) + (p.n_seqs < p.total_q ? p.n_seqs : p.total_q);
  if (tiles * p.hkv > 0x7FFFFFFF) return cudaErrorInvalidValue;
  attn_prefill_kernel<D, M><<<(unsigned)(tiles * p.hkv), C::kThreads, C::kSmem, s>>>(p, maps);
  return cudaGetLastError();
}

int num_sms() {
  static int n = [] {
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      v = 1;
    return v > 0 ? v : 1;
  }();
  return n;
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnPrefillParams& p, int d, cudaStream_t s) {
  // Two row tiles per CTA halve the K and V traffic; one row tile with its keys split halves the longest
  // CTA. Measured at 16/2 heads of 128: 2048 tokens (0.8 CTAs of two row tiles per SM) 35.6 against 26.8 us
  // split, 3000 tokens (1.2) 47.4 against 48.8 us, 16384 tokens 748 against 804 us.
  const bool two = (int64_t)p.total_q / (2 * (128 / p.group)) * p.hkv >= num_sms();
  if (d == 64) return two ? launch<64, kRows>(p, s) : launch<64, kKeys>(p, s);
  if (d == 128) return two ? launch<128, kRows>(p, s) : launch<128, kKeys>(p, s);
  return launch<256, kOne>(p, s);
}

}  // namespace moe
