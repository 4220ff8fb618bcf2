// Parameter blocks and workspace layout of the 8-bit expert calls (host + device).
#pragma once

#include "moe_internal.h"

namespace moe {

constexpr int kExpMaxRows = 1 << 26;   // rows, tokens, assignments: fewer than this
constexpr int kExpMaxCols = 65536;
constexpr int kScaleBlock = 128;       // columns (and rows of a weight matrix) to a scale
constexpr int kSortMaxChunks = 256;    // CTAs of the sort at most

// Workspace: status word, then the sort's histograms [chunk][expert, none].
struct ExpertWs {
  size_t counts, total;
};
inline ExpertWs expert_ws(int n_experts) {
  ExpertWs w;
  w.counts = sizeof(WsHeader);
  w.total = w.counts + (size_t)kSortMaxChunks * (n_experts + 1) * 4;
  return w;
}

struct SortParams {
  const int32_t* ids;
  int n, n_experts;
  int32_t* offsets;
  int32_t* perm;
  int32_t* inv;
  int32_t* counts;  // [chunks][n_experts + 1]
  int chunk, chunks;
  WsHeader* hdr;
};

struct DispatchParams {
  moe_rows x, out;
  const int32_t* inv;  // NULL: row t to row t
  int T, k, d, out_rows, segments;
  WsHeader* hdr;
};

struct CombineParams {
  moe_rows ys, add, y;  // add.p NULL: none
  const int32_t* inv;
  const float* w;  // NULL: ones
  int ys_rows, T, k, d, segments;
  WsHeader* hdr;
};

struct CombineGradParams {
  moe_rows dy, ys, dys;
  const int32_t* inv;
  const float* w;
  float* dw;
  int ys_rows, T, k, d;
  WsHeader* hdr;
};

struct SwigluParams {
  moe_rows gu, dh, out;  // dh: gradient only
  const int32_t* total;  // NULL: rows
  int rows, inter, segments;
  WsHeader* hdr;
};

struct QuantWeightsParams {
  const uint16_t* w;
  uint8_t* q;
  float* scale;
  int n, k;
};

struct ProductParams {
  moe_rows a, out;
  const uint8_t* wq;
  const float* wscale;
  const int32_t* offsets;  // NULL: one expert, all rows
  int rows, n_experts;
  int n, k;                // of the stored matrices
  int in, outc;            // columns of a and of out: k and n, or n and k when transposed
  int in_blocks, out_blocks;  // of 128
  int transposed;
  WsHeader* hdr;
};

cudaError_t launch_sort_tokens(SortParams p, cudaStream_t s);
cudaError_t launch_dispatch(DispatchParams p, cudaStream_t s);
cudaError_t launch_combine(CombineParams p, cudaStream_t s);
cudaError_t launch_combine_grad(const CombineGradParams& p, cudaStream_t s);
cudaError_t launch_swiglu(SwigluParams p, bool grad, cudaStream_t s);
cudaError_t launch_quant_weights(const QuantWeightsParams& p, int n_experts, cudaStream_t s);
cudaError_t launch_product(const ProductParams& p, cudaStream_t s);
int product_form(const ProductParams& p, int sms, int pairs);  // MOE_PRODUCT_*
bool product_is_small(const ProductParams& p, int sms);  // the kernel for few rows takes the call
cudaError_t launch_product_small(const ProductParams& p, cudaStream_t s);

int sm_count();  // of the device that was current at the first call

}  // namespace moe
