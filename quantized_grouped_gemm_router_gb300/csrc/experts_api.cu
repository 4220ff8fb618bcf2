// Host side of the 8-bit expert calls of include/moe_gb300.h: argument checks and launches.
#include "experts.h"

namespace moe {

int sm_count() {
  static const int n = [] {
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      v = 1;
    return v > 0 ? v : 1;
  }();
  return n;
}

namespace {

bool experts_ok(int n) { return n >= 1 && n <= kMaxExperts; }
bool cols_ok(int c) { return c >= 16 && c <= kExpMaxCols && c % 16 == 0; }

int check_space(void* ws, size_t ws_bytes, int n_experts) {
  if (!ws) return MOE_ERR_INVALID_ARG;
  if (!aligned(ws, 128)) return MOE_ERR_MISALIGNED;
  return ws_bytes < expert_ws(n_experts).total ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

int check_counts(int rows, int more = 0) {
  if (rows < 0 || more < 0) return MOE_ERR_INVALID_ARG;
  return rows >= kExpMaxRows || more >= kExpMaxRows ? MOE_ERR_UNSUPPORTED_SHAPE : MOE_OK;
}

// format: that of moe_rows, or -1 for either.
int check_rows(const moe_rows* r, int cols, int format) {
  if (!r || !r->p) return MOE_ERR_INVALID_ARG;
  if (r->format != MOE_ROWS_BF16 && r->format != MOE_ROWS_E4M3) return MOE_ERR_INVALID_ARG;
  if (format >= 0 && r->format != format) return MOE_ERR_INVALID_ARG;
  const bool e4m3 = r->format == MOE_ROWS_E4M3;
  const int64_t most = (int64_t)1 << 38;
  if (r->stride % (e4m3 ? 16 : 8) || r->stride < cols || r->stride >= most) return MOE_ERR_INVALID_ARG;
  if (e4m3 && (!r->scale || r->scale_stride < (cols + kScaleBlock - 1) / kScaleBlock || r->scale_stride >= most))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(r->p, 16) || (e4m3 && !aligned(r->scale, 4))) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

int check_assignments(int T, int top_k, int d) {
  if (T < 0) return MOE_ERR_INVALID_ARG;
  if (top_k < 1 || top_k > kMaxTopK || !cols_ok(d) || T >= kExpMaxRows || (int64_t)T * top_k >= kExpMaxRows)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
WsHeader* header(void* ws) { return static_cast<WsHeader*>(ws); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_expert_workspace_bytes(int32_t n_experts) { return experts_ok(n_experts) ? expert_ws(n_experts).total : 0; }

int moe_sort_tokens(const int32_t* ids, int32_t n, int32_t n_experts, int32_t* offsets, int32_t* perm, int32_t* inv,
                    void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!experts_ok(n_experts)) return MOE_ERR_UNSUPPORTED_SHAPE;
  int st = check_counts(n);
  if (st) return st;
  if (!offsets || (n && (!ids || !perm || !inv))) return MOE_ERR_INVALID_ARG;
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(perm, 4) || !aligned(inv, 4)) return MOE_ERR_MISALIGNED;
  if ((st = check_space(ws, ws_bytes, n_experts))) return st;
  SortParams p;
  p.ids = ids;
  p.n = n;
  p.n_experts = n_experts;
  p.offsets = offsets;
  p.perm = perm;
  p.inv = inv;
  p.counts = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + expert_ws(n_experts).counts);
  p.hdr = header(ws);
  return status_of(launch_sort_tokens(p, stream));
}

int moe_dispatch(const moe_rows* x, const int32_t* inv, int32_t T, int32_t top_k, int32_t d, const moe_rows* out,
                 int32_t out_rows, void* ws, size_t ws_bytes, moe_stream_t stream) {
  int st = check_assignments(T, top_k, d);
  if (st || (st = check_counts(out_rows))) return st;
  if (T && !inv && (top_k != 1 || out_rows < T)) return MOE_ERR_INVALID_ARG;
  if (!aligned(inv, 4)) return MOE_ERR_MISALIGNED;
  if ((st = check_space(ws, ws_bytes, 1))) return st;
  if (T == 0) return MOE_OK;
  if ((st = check_rows(x, d, MOE_ROWS_BF16)) || (out_rows && (st = check_rows(out, d, -1)))) return st;
  DispatchParams p;
  p.x = *x;
  p.out = out_rows ? *out : *x;  // without rows every place is out of range
  p.inv = inv;
  p.T = T;
  p.k = top_k;
  p.d = d;
  p.out_rows = out_rows;
  p.hdr = header(ws);
  return status_of(launch_dispatch(p, stream));
}

int moe_combine(const moe_rows* ys, int32_t ys_rows, const int32_t* inv, const float* w, int32_t T, int32_t top_k,
                int32_t d, const moe_rows* add, const moe_rows* y, void* ws, size_t ws_bytes, moe_stream_t stream) {
  int st = check_assignments(T, top_k, d);
  if (st || (st = check_counts(ys_rows))) return st;
  if (T && !inv) return MOE_ERR_INVALID_ARG;
  if (!aligned(inv, 4) || !aligned(w, 4)) return MOE_ERR_MISALIGNED;
  if ((st = check_space(ws, ws_bytes, 1))) return st;
  if (T == 0) return MOE_OK;
  if ((ys_rows && (st = check_rows(ys, d, MOE_ROWS_BF16))) || (st = check_rows(y, d, MOE_ROWS_BF16)) ||
      (add && (st = check_rows(add, d, MOE_ROWS_BF16))))
    return st;
  CombineParams p;
  p.ys = ys_rows ? *ys : *y;  // without rows every place is out of range
  p.y = *y;
  if (add)
    p.add = *add;
  else
    p.add.p = nullptr;
  p.inv = inv;
  p.w = w;
  p.ys_rows = ys_rows;
  p.T = T;
  p.k = top_k;
  p.d = d;
  p.hdr = header(ws);
  return status_of(launch_combine(p, stream));
}

int moe_combine_grad(const moe_rows* dy, const moe_rows* ys, int32_t ys_rows, const int32_t* inv, const float* w,
                     int32_t T, int32_t top_k, int32_t d, const moe_rows* dys, float* dw, void* ws, size_t ws_bytes,
                     moe_stream_t stream) {
  int st = check_assignments(T, top_k, d);
  if (st || (st = check_counts(ys_rows))) return st;
  if (T && (!inv || !w || !dw)) return MOE_ERR_INVALID_ARG;
  if (!aligned(inv, 4) || !aligned(w, 4) || !aligned(dw, 4)) return MOE_ERR_MISALIGNED;
  if ((st = check_space(ws, ws_bytes, 1))) return st;
  if (T == 0) return MOE_OK;
  if ((st = check_rows(dy, d, MOE_ROWS_BF16)) ||
      (ys_rows && ((st = check_rows(ys, d, MOE_ROWS_BF16)) || (st = check_rows(dys, d, -1)))))
    return st;
  CombineGradParams p;
  p.dy = *dy;
  p.ys = ys_rows ? *ys : *dy;  // without rows every place is out of range
  p.dys = ys_rows ? *dys : *dy;
  p.inv = inv;
  p.w = w;
  p.dw = dw;
  p.ys_rows = ys_rows;
  p.T = T;
  p.k = top_k;
  p.d = d;
  p.hdr = header(ws);
  return status_of(launch_combine_grad(p, stream));
}

int moe_quant_weights(const uint16_t* w, int32_t n_experts, int32_t n, int32_t k, uint8_t* q, float* scale,
                      moe_stream_t stream) {
  if (!experts_ok(n_experts) || !cols_ok(n) || !cols_ok(k)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!w || !q || !scale) return MOE_ERR_INVALID_ARG;
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(scale, 4)) return MOE_ERR_MISALIGNED;
  QuantWeightsParams p;
  p.w = w;
  p.q = q;
  p.scale = scale;
  p.n = n;
  p.k = k;
  return status_of(launch_quant_weights(p, n_experts, stream));
}

int moe_gemm_e4m3(const moe_rows* a, int32_t rows, const moe_e4m3_weights* w, const int32_t* offsets,
                  int32_t transposed, const moe_rows* out, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!w) return MOE_ERR_INVALID_ARG;
  if (!experts_ok(w->n_experts) || !cols_ok(w->n) || !cols_ok(w->k)) return MOE_ERR_UNSUPPORTED_SHAPE;
  int st = check_counts(rows);
  if (st) return st;
  if (!w->q || !w->scale || (!offsets && w->n_experts != 1)) return MOE_ERR_INVALID_ARG;
  if (!aligned(w->q, 16) || !aligned(w->scale, 4) || !aligned(offsets, 4)) return MOE_ERR_MISALIGNED;
  if ((st = check_space(ws, ws_bytes, w->n_experts))) return st;
  if (rows == 0) return MOE_OK;
  ProductParams p;
  p.transposed = transposed != 0;
  p.n = w->n;
  p.k = w->k;
  p.in = p.transposed ? w->n : w->k;
  p.outc = p.transposed ? w->k : w->n;
  if ((st = check_rows(a, p.in, MOE_ROWS_E4M3)) || (st = check_rows(out, p.outc, MOE_ROWS_BF16))) return st;
  p.a = *a;
  p.out = *out;
  p.wq = w->q;
  p.wscale = w->scale;
  p.offsets = offsets;
  p.rows = rows;
  p.n_experts = w->n_experts;
  p.in_blocks = (p.in + kScaleBlock - 1) / kScaleBlock;
  p.out_blocks = (p.outc + kScaleBlock - 1) / kScaleBlock;
  p.hdr = header(ws);
  return status_of(launch_product(p, stream));
}

int32_t moe_gemm_e4m3_form(int32_t rows, int32_t n_experts, int32_t n, int32_t k, int32_t transposed, int64_t stride, int32_t sms,
                           int32_t pairs) {
  if (rows < 1 || rows >= kExpMaxRows || !experts_ok(n_experts) || !cols_ok(n) || !cols_ok(k) || stride < 1 || sms < 1 || pairs < 0)
    return -1;
  ProductParams p = {};
  p.a.stride = stride;
  p.rows = rows;
  p.n_experts = n_experts;
  p.n = n;
  p.k = k;
  p.transposed = transposed != 0;
  p.in = p.transposed ? n : k;
  p.outc = p.transposed ? k : n;
  p.in_blocks = (p.in + kScaleBlock - 1) / kScaleBlock;
  p.out_blocks = (p.outc + kScaleBlock - 1) / kScaleBlock;
  return product_form(p, sms, pairs);
}

static int swiglu_call(const moe_rows* gu, const moe_rows* dh, int32_t rows, int32_t inter, const int32_t* total,
                       const moe_rows* out, void* ws, size_t ws_bytes, moe_stream_t stream, bool grad) {
  int st = check_counts(rows);
  if (st) return st;
  if (!cols_ok(inter) || 2 * inter > kExpMaxCols) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(total, 4)) return MOE_ERR_MISALIGNED;
  if ((st = check_space(ws, ws_bytes, 1))) return st;
  if (rows == 0) return MOE_OK;
  if ((st = check_rows(gu, 2 * inter, MOE_ROWS_BF16)) || (grad && (st = check_rows(dh, inter, MOE_ROWS_BF16))) ||
      (st = check_rows(out, grad ? 2 * inter : inter, -1)))
    return st;
  SwigluParams p;
  p.gu = *gu;
  p.dh = grad ? *dh : *gu;
  p.out = *out;
  p.total = total;
  p.rows = rows;
  p.inter = inter;
  p.hdr = header(ws);
  return status_of(launch_swiglu(p, grad, stream));
}

int moe_swiglu(const moe_rows* gu, int32_t rows, int32_t inter, const int32_t* total, const moe_rows* h, void* ws,
               size_t ws_bytes, moe_stream_t stream) {
  return swiglu_call(gu, nullptr, rows, inter, total, h, ws, ws_bytes, stream, false);
}

int moe_swiglu_grad(const moe_rows* gu, const moe_rows* dh, int32_t rows, int32_t inter, const int32_t* total,
                    const moe_rows* dgu, void* ws, size_t ws_bytes, moe_stream_t stream) {
  return swiglu_call(gu, dh, rows, inter, total, dgu, ws, ws_bytes, stream, true);
}

}  // extern "C"
