// Parameter blocks and workspace layout of the attention calls (host + device).
#pragma once

#include "moe_internal.h"

namespace moe {

constexpr int kAttnMaxHeads = 1024;  // query heads
constexpr int kAttnMaxGroup = 64;    // query heads per key-value head
constexpr int kAttnMaxSeqs = 4096;
constexpr int kAttnMaxRows = 1 << 30;

struct AttnPrefillParams {
  moe_heads_view q, k, v;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int n_seqs, total_q, total_k;
  int hq, hkv, group;  // group = hq / hkv
  int causal;
  float scale;
  uint16_t* o;
  int o_wide;  // o is 32-byte aligned
  float* lse;
  WsHeader* hdr;
  float* aside;      // [kAttnMaxCtas][2][128 x d] sums put aside during long items, of 128 rows each
  float2* aside_ml;  // [kAttnMaxCtas][2][128] their (m c, l)
};

// Division by an invariant: n / d = (t + ((n - t) >> s1)) >> s2 with t = the high half of m n, for every
// 32-bit n (Granlund and Montgomery, Division by Invariant Integers using Multiplication).
struct FastDiv {
  uint32_t m;
  int s1, s2;
  explicit FastDiv(uint32_t d = 1) {
    int l = 0;
    while (((uint64_t)1 << l) < d) ++l;
    m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << l) - d)) / d + 1);
    s1 = l < 1 ? l : 1;
    s2 = l > 1 ? l - 1 : 0;
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
    const uint32_t t = __umulhi(m, n);
    return (t + ((n - t) >> s1)) >> s2;
  }
#endif
};

struct KvAppendParams {
  moe_heads_view k, v;
  const int32_t* cu;
  const int32_t* start;
  const int32_t* table;
  int table_width, n_seqs, total;
  int hkv, d, page_size, n_pages, e4m3;
  void* kc;
  void* vc;
  const float* k_scale;
  const float* v_scale;
  WsHeader* hdr;
  FastDiv page_div;
  // set at launch: heads head0 .. head0 + heads - 1, threads to a token, tokens to a block, log2(d / 8)
  int head0, heads, tpt, tokens, log_dp;
  FastDiv div_tpt;
};

struct AttnDecodeParams {
  moe_heads_view q;
  const void* kc;
  const void* vc;
  const float* k_scale;
  const float* v_scale;
  const int32_t* lens;
  const int32_t* table;
  int table_width, n_seqs;
  int hq, hkv, group;
  int page_size, n_pages;
  FastDiv page_div;
  float scale;
  uint16_t* o;
  float* lse;
  WsHeader* hdr;
  int4* splits;    // [kAttnMaxCtas] the head that begins in a CTA and ends in a later one: sequence, unit, CTAs (0: none)
  float* parts;    // [kAttnMaxCtas][2] partial results of a CTA: 16 rows of d values, 16 m, 16 l
  float* scratch;  // [kAttnMaxCtas * kAttnMaxWarps] partial rows of a warp
};

// Workspace of the attention calls: status word, then what the decode's two kernels hand over. The prompt kernel puts
// sums aside in the place of scratch, and their statistics in that of parts.
constexpr int kAttnMaxCtas = 256;
constexpr int kAttnMaxWarps = 16;
struct AttnWs {
  size_t splits, parts, scratch, total;
};
inline AttnWs attn_ws(const moe_attn_dims& d) {
  AttnWs w;
  const size_t rows = (size_t)16 * d.head_dim * 4;
  w.splits = sizeof(WsHeader);
  w.parts = w.splits + kAttnMaxCtas * sizeof(int4);
  w.scratch = w.parts + (size_t)kAttnMaxCtas * 2 * (rows + 128);
  static_assert(2 * 128 <= 16 * kAttnMaxWarps && 2 * 128 * sizeof(float2) <= 2 * (16 * 64 * 4 + 128), "a CTA's two row tiles");
  w.total = w.scratch + (size_t)kAttnMaxCtas * kAttnMaxWarps * rows;
  return w;
}

cudaError_t launch_attn_prefill(const AttnPrefillParams& p, int d, cudaStream_t s);
cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t s);
cudaError_t launch_attn_decode(const AttnDecodeParams& p, int d, bool e4m3, cudaStream_t s);

// Encodes a tiled TMA descriptor (element strides 1, out-of-bounds elements read zero).
bool encode_tiled(CUtensorMap* m, CUtensorMapDataType type, cuuint32_t rank, const void* ptr, const cuuint64_t* dims,
                  const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swz);

}  // namespace moe
