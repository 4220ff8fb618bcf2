// Host side of the attention calls of include/moe_gb300.h: argument checks and launches.
#include <cmath>

#include "attn.h"

namespace moe {
bool aligned(const void* p, size_t a);

namespace {

int check_attn_dims(const moe_attn_dims* d) {
  if (!d) return MOE_ERR_INVALID_ARG;
  if ((d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) || d->n_kv_heads < 1 ||
      d->n_q_heads < d->n_kv_heads || d->n_q_heads > kAttnMaxHeads || d->n_q_heads % d->n_kv_heads ||
      d->n_q_heads / d->n_kv_heads > kAttnMaxGroup)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

int check_view(const moe_heads_view& v, int d) {
  if (!v.p) return MOE_ERR_INVALID_ARG;
  const int64_t most = (int64_t)1 << 38;
  if (v.token_stride % 8 || v.head_stride % 8 || v.token_stride < d || v.head_stride < d || v.token_stride >= most ||
      v.head_stride >= most)
    return MOE_ERR_INVALID_ARG;
  return aligned(v.p, 16) ? MOE_OK : MOE_ERR_MISALIGNED;
}

int check_attn_ws(void* ws, size_t ws_bytes, const moe_attn_dims& d) {
  if (!ws) return MOE_ERR_INVALID_ARG;
  if (!aligned(ws, 128)) return MOE_ERR_MISALIGNED;
  return ws_bytes < attn_ws(d).total ? MOE_ERR_WORKSPACE_TOO_SMALL : MOE_OK;
}

int check_seqs(int n_seqs) {
  if (n_seqs < 1) return MOE_ERR_INVALID_ARG;
  return n_seqs > kAttnMaxSeqs ? MOE_ERR_UNSUPPORTED_SHAPE : MOE_OK;
}

int check_cache(const moe_kv_cache* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  int st = check_attn_dims(&c->dims);
  if (st) return st;
  if (c->format != MOE_KV_BF16 && c->format != MOE_KV_E4M3) return MOE_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->page_size < 1 || !c->k || !c->v) return MOE_ERR_INVALID_ARG;
  if (c->page_size > 65536 || (int64_t)c->n_pages * c->dims.n_kv_heads * c->page_size >= ((int64_t)1 << 31))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->format == MOE_KV_E4M3 && (!c->k_scale || !c->v_scale)) return MOE_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_attn_workspace_bytes(const moe_attn_dims* dims) {
  return check_attn_dims(dims) == MOE_OK ? attn_ws(*dims).total : 0;
}

int moe_attn_prefill(const moe_attn_dims* dims, moe_heads_view q, moe_heads_view k, moe_heads_view v,
                     const int32_t* cu_q, const int32_t* cu_k, int32_t n_seqs, int32_t total_q, int32_t total_k,
                     float scale, int32_t causal, uint16_t* o, float* lse, void* ws, size_t ws_bytes,
                     moe_stream_t stream) {
  int st = check_attn_dims(dims);
  if (st || (st = check_seqs(n_seqs))) return st;
  if (!cu_q || !cu_k || total_q < 0 || total_k < 0 || !(scale > 0.f) || !std::isfinite(scale)) return MOE_ERR_INVALID_ARG;
  if (total_q > kAttnMaxRows || total_k > kAttnMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(lse, 4) || !aligned(o, 16)) return MOE_ERR_MISALIGNED;
  if ((st = check_attn_ws(ws, ws_bytes, *dims))) return st;
  if (total_q == 0) return MOE_OK;
  if (!o) return MOE_ERR_INVALID_ARG;
  if ((st = check_view(q, dims->head_dim))) return st;
  if (total_k && ((st = check_view(k, dims->head_dim)) || (st = check_view(v, dims->head_dim)))) return st;
  AttnPrefillParams p;
  p.q = q;
  p.k = k;
  p.v = v;
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.n_seqs = n_seqs;
  p.total_q = total_q;
  p.total_k = total_k;
  p.hq = dims->n_q_heads;
  p.hkv = dims->n_kv_heads;
  p.group = p.hq / p.hkv;
  p.causal = causal != 0;
  p.scale = scale;
  p.o = o;
  p.o_wide = aligned(o, 32);
  p.lse = lse;
  const AttnWs w = attn_ws(*dims);
  p.hdr = static_cast<WsHeader*>(ws);
  p.aside = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + w.scratch);
  p.aside_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + w.parts);
  return launch_attn_prefill(p, dims->head_dim, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_kv_append(const moe_kv_cache* cache, moe_heads_view k, moe_heads_view v, const int32_t* cu,
                  const int32_t* start, const int32_t* page_table, int32_t table_width, int32_t n_seqs, int32_t total,
                  void* ws, size_t ws_bytes, moe_stream_t stream) {
  int st = check_cache(cache);
  if (st || (st = check_seqs(n_seqs))) return st;
  if (!cu || !start || !page_table || table_width < 1 || total < 0) return MOE_ERR_INVALID_ARG;
  if (total > kAttnMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(cu, 4) || !aligned(start, 4) || !aligned(page_table, 4)) return MOE_ERR_MISALIGNED;
  if ((st = check_attn_ws(ws, ws_bytes, cache->dims))) return st;
  if (total == 0) return MOE_OK;
  if ((st = check_view(k, cache->dims.head_dim)) || (st = check_view(v, cache->dims.head_dim))) return st;
  KvAppendParams p;
  p.k = k;
  p.v = v;
  p.cu = cu;
  p.start = start;
  p.table = page_table;
  p.table_width = table_width;
  p.n_seqs = n_seqs;
  p.total = total;
  p.hkv = cache->dims.n_kv_heads;
  p.d = cache->dims.head_dim;
  p.page_size = cache->page_size;
  p.n_pages = cache->n_pages;
  p.e4m3 = cache->format == MOE_KV_E4M3;
  p.page_div = FastDiv(cache->page_size);
  p.kc = cache->k;
  p.vc = cache->v;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.hdr = static_cast<WsHeader*>(ws);
  return launch_kv_append(p, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int moe_attn_decode(const moe_kv_cache* cache, moe_heads_view q, const int32_t* lens, const int32_t* page_table,
                    int32_t table_width, int32_t n_seqs, float scale, uint16_t* o, float* lse, void* ws,
                    size_t ws_bytes, moe_stream_t stream) {
  int st = check_cache(cache);
  if (st || (st = check_seqs(n_seqs))) return st;
  if (!lens || !page_table || table_width < 1 || !o || !(scale > 0.f) || !std::isfinite(scale))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(lens, 4) || !aligned(page_table, 4) || !aligned(lse, 4) || !aligned(o, 16)) return MOE_ERR_MISALIGNED;
  if ((st = check_attn_ws(ws, ws_bytes, cache->dims)) || (st = check_view(q, cache->dims.head_dim))) return st;
  // the kernel numbers the 16-row tiles of all sequences and heads, and a few slots more a head, in 31 bits
  const int64_t units = cache->dims.n_kv_heads * ((cache->dims.n_q_heads / cache->dims.n_kv_heads + 15) / 16);
  if (((int64_t)table_width * cache->page_size + 15) / 16 + 8 >= ((int64_t)1 << 31) / (units * n_seqs))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  AttnDecodeParams p;
  p.q = q;
  p.kc = cache->k;
  p.vc = cache->v;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.lens = lens;
  p.table = page_table;
  p.table_width = table_width;
  p.n_seqs = n_seqs;
  p.hq = cache->dims.n_q_heads;
  p.hkv = cache->dims.n_kv_heads;
  p.group = p.hq / p.hkv;
  p.page_size = cache->page_size;
  p.n_pages = cache->n_pages;
  p.page_div = FastDiv(cache->page_size);
  p.scale = scale;
  p.o = o;
  p.lse = lse;
  const AttnWs w = attn_ws(cache->dims);
  uint8_t* base = static_cast<uint8_t*>(ws);
  p.hdr = reinterpret_cast<WsHeader*>(base);
  p.splits = reinterpret_cast<int4*>(base + w.splits);
  p.parts = reinterpret_cast<float*>(base + w.parts);
  p.scratch = reinterpret_cast<float*>(base + w.scratch);
  return launch_attn_decode(p, cache->dims.head_dim, cache->format == MOE_KV_E4M3, stream) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

}  // extern "C"
