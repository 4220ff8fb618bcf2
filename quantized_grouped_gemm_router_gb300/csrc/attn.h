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
  float* lse;
  WsHeader* hdr;
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
  float scale;
  uint16_t* o;
  float* lse;
  WsHeader* hdr;
};

inline size_t attn_ws_bytes(const moe_attn_dims&) { return sizeof(WsHeader); }

cudaError_t launch_attn_prefill(const AttnPrefillParams& p, int d, cudaStream_t s);
cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t s);
cudaError_t launch_attn_decode(const AttnDecodeParams& p, int d, bool e4m3, cudaStream_t s);

// Encodes a tiled TMA descriptor (element strides 1, out-of-bounds elements read zero).
bool encode_tiled(CUtensorMap* m, CUtensorMapDataType type, cuuint32_t rank, const void* ptr, const cuuint64_t* dims,
                  const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swz);

}  // namespace moe
