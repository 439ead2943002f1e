// C ABI of the packed-batch entry points (headq_span, headq_rows): argument checks and
// launches of headq_cache_write_ragged, headq_cache_read and headq_tree_attn.
#include "headq_internal.cuh"
#include "tree.cuh"

#define HEADQ_API extern "C" __attribute__((visibility("default")))

namespace headq {
namespace {

headq_status check_span(const headq_span* s, const headq_cache* c) {
  if (!s || s->T < 0 || s->T > c->T_cap || s->n < 0 || s->rows < 0) return HEADQ_ERR_INVALID_ARG;
  if (s->seq_lens && !aligned16(s->seq_lens)) return HEADQ_ERR_INVALID_ARG;
  if (s->cu && !aligned16(s->cu)) return HEADQ_ERR_INVALID_ARG;
  if (!s->cu && static_cast<long long>(c->B) * s->n > s->rows) return HEADQ_ERR_INVALID_ARG;
  return c->B > 65535 || c->Hkv > 65535 ? HEADQ_ERR_UNSUPPORTED : HEADQ_OK;
}

headq_status check_rows(const headq_rows* r) {
  if (!r || !r->ptr || !aligned16(r->ptr)) return HEADQ_ERR_INVALID_ARG;
  if (r->dtype != HEADQ_F32 && r->dtype != HEADQ_BF16) return HEADQ_ERR_INVALID_ARG;
  const long long m = r->dtype == HEADQ_BF16 ? 8 : 4;
  if (r->row_stride < 0 || r->head_stride < 0 || r->row_stride % m || r->head_stride % m)
    return HEADQ_ERR_INVALID_ARG;
  return HEADQ_OK;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

size_t part_rows(const headq_cache& c, int Hq, int n, const TreePlan& tp) {
  return tp.splits > 1 ? static_cast<size_t>(c.B) * Hq * n * tp.splits : 0;
}

size_t tree_ws(const headq_cache& c, int Hq, int n, int T, bool q_bf16) {
  const size_t rows = part_rows(c, Hq, n, tree_plan(c, Hq, n, T, q_bf16));
  return kWsHeaderBytes + round256(rows * c.d * sizeof(float)) + round256(rows * sizeof(float2));
}

}  // namespace
}  // namespace headq

using namespace headq;

HEADQ_API headq_status headq_cache_write_ragged(const headq_cache* cache, const headq_rows* k,
                                                const headq_rows* v, int src_rows, const int32_t* src,
                                                const headq_span* span, const float* U,
                                                headq_stream_t stream) {
  headq_status st = check_cache(cache);
  if (st != HEADQ_OK) return st;
  if (cache->kmode != HEADQ_K_TOKEN) return HEADQ_ERR_UNSUPPORTED;  // sealed key blocks
  if ((st = check_span(span, cache)) != HEADQ_OK) return st;
  if (src_rows < 0 || (src && !aligned16(src)) || (!src && src_rows != span->rows))
    return HEADQ_ERR_INVALID_ARG;
  if (span->n == 0 || span->rows == 0 || cache->B == 0) return HEADQ_OK;
  if ((st = check_rows(k)) != HEADQ_OK || (v && (st = check_rows(v)) != HEADQ_OK)) return st;
  if (v && v->dtype != k->dtype) return HEADQ_ERR_INVALID_ARG;
  if (cache->r > 0 && (!U || !aligned16(U))) return HEADQ_ERR_INVALID_ARG;
  CacheWriteParams p{};
  p.c = *cache;
  p.k = k->ptr;
  p.k_row = k->row_stride;
  p.k_head = k->head_stride;
  if (v) {
    p.v = v->ptr;
    p.v_row = v->row_stride;
    p.v_head = v->head_stride;
  }
  p.in_bf16 = k->dtype == HEADQ_BF16;
  p.U = U;
  p.span = *span;
  p.src = src;
  p.src_rows = src_rows;
  return launch_cache_write_ragged(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? HEADQ_OK
             : HEADQ_ERR_CUDA;
}

HEADQ_API headq_status headq_cache_read(const headq_cache* cache, const headq_span* span,
                                        const float* U, int corr_sign, const headq_rows* k_out,
                                        const headq_rows* v_out, void* ws, headq_stream_t stream) {
  headq_status st = check_cache(cache);
  if (st != HEADQ_OK) return st;
  if ((st = check_span(span, cache)) != HEADQ_OK) return st;
  if (corr_sign < -1 || corr_sign > 1 || (ws && !aligned16(ws))) return HEADQ_ERR_INVALID_ARG;
  if (span->n == 0 || span->rows == 0 || cache->B == 0) return HEADQ_OK;
  if (!k_out && !v_out) return HEADQ_ERR_INVALID_ARG;
  if ((k_out && (st = check_rows(k_out)) != HEADQ_OK) || (v_out && (st = check_rows(v_out)) != HEADQ_OK))
    return st;
  if (k_out && cache->r > 0 && (!U || !aligned16(U))) return HEADQ_ERR_INVALID_ARG;
  CacheReadParams p{};
  p.c = *cache;
  p.span = *span;
  p.U = U;
  p.sigma = static_cast<float>(corr_sign);
  if (k_out) p.k = *k_out;
  if (v_out) p.v = *v_out;
  p.err = static_cast<unsigned*>(ws);
  return launch_cache_read(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? HEADQ_OK
             : HEADQ_ERR_CUDA;
}

HEADQ_API size_t headq_tree_workspace_bytes(const headq_cache* cache, int Hq, int n, int T) {
  if (check_cache(cache) != HEADQ_OK || Hq <= 0 || Hq % cache->Hkv || n < 0 || T < 0) return 0;
  const size_t a = tree_ws(*cache, Hq, n, T, true), b = tree_ws(*cache, Hq, n, T, false);
  return a > b ? a : b;  // the queries' dtype is not known here
}

HEADQ_API headq_status headq_tree_attn(const headq_cache* cache, const headq_rows* q, int Hq,
                                       const uint8_t* mask, long long mask_stride,
                                       const headq_span* span, const float* U, float sm_scale,
                                       int corr_sign, const headq_rows* out, float* lse, void* ws,
                                       size_t ws_bytes, headq_stream_t stream) {
  headq_status st = check_cache(cache);
  if (st != HEADQ_OK) return st;
  if (cache->kmode != HEADQ_K_TOKEN) return HEADQ_ERR_UNSUPPORTED;
  if ((st = check_span(span, cache)) != HEADQ_OK) return st;
  if (Hq <= 0 || Hq % cache->Hkv != 0 || corr_sign < -1 || corr_sign > 1) return HEADQ_ERR_INVALID_ARG;
  if (static_cast<long long>(span->n) * Hq > (1 << 24) ||
      static_cast<long long>(cache->B) * cache->Hkv > 65535)
    return HEADQ_ERR_UNSUPPORTED;
  if (mask && mask_stride != 0 && mask_stride < static_cast<long long>(span->n) * span->n)
    return HEADQ_ERR_INVALID_ARG;
  if (lse && !aligned16(lse)) return HEADQ_ERR_INVALID_ARG;
  if (span->n == 0 || span->rows == 0 || cache->B == 0) return HEADQ_OK;
  if ((st = check_rows(q)) != HEADQ_OK || (st = check_rows(out)) != HEADQ_OK) return st;
  if (out->dtype != q->dtype) return HEADQ_ERR_INVALID_ARG;
  if (cache->r > 0 && (!U || !aligned16(U))) return HEADQ_ERR_INVALID_ARG;
  const bool qb = q->dtype == HEADQ_BF16;
  if (!ws || !aligned16(ws) || ws_bytes < tree_ws(*cache, Hq, span->n, span->T, qb))
    return HEADQ_ERR_WORKSPACE;
  const TreePlan tp = tree_plan(*cache, Hq, span->n, span->T, qb);
  TreeParams p{};
  p.c = *cache;
  p.q = *q;
  p.out = *out;
  p.Hq = Hq;
  p.G = Hq / cache->Hkv;
  p.span = *span;
  p.mask = mask;
  p.mask_stride = mask_stride;
  p.U = U;
  p.sm_scale = sm_scale;
  p.corr_sign = static_cast<float>(corr_sign);
  p.lse = lse;
  p.splits = tp.splits;
  p.chunk = tp.chunk;
  char* w = static_cast<char*>(ws);
  p.err = reinterpret_cast<unsigned*>(w);
  p.part_o = reinterpret_cast<float*>(w + kWsHeaderBytes);
  p.part_ml = reinterpret_cast<float2*>(
      w + kWsHeaderBytes +
      round256(part_rows(*cache, Hq, span->n, tp) * cache->d * sizeof(float)));
  return launch_tree(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? HEADQ_OK
                                                                              : HEADQ_ERR_CUDA;
}
