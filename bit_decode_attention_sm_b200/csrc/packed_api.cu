// C ABI of the packed-batch entry points (headq_span, headq_rows): argument checks and
// launches of headq_cache_write_ragged, headq_cache_read and headq_tree_attn.
#include <algorithm>

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
  if (s->T > 1 << 30 || s->rows > 1 << 30) return HEADQ_ERR_UNSUPPORTED;  // the kernels' indices are int
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

// Tree workspace: [error word][partial outputs][partial statistics][query images][logit
// factors][mask bits], the last three for the tensor-core kernel
struct TreeWs {
  size_t part_ml, qimg, qf, words, bytes;
};
TreeWs tree_ws(const headq_cache& c, int n, size_t part_rows, bool mma, int blocks) {
  TreeWs w{};
  const size_t units = static_cast<size_t>(c.B) * c.Hkv;
  w.part_ml = kWsHeaderBytes + round256(part_rows * c.d * sizeof(float));
  w.qimg = w.part_ml + round256(part_rows * sizeof(float4));
  w.qf = w.qimg + (mma ? round256(units * blocks * tree_mma_image_bytes(c)) : 0);
  w.words = w.qf + (mma ? round256(units * blocks * 128 * sizeof(float)) : 0);
  w.bytes = w.words + (mma ? round256(static_cast<size_t>(c.B) * n * ((n + 31) / 32) * 4) : 0);
  return w;
}

// most splits of decode_plan for any length up to T
int decode_max_splits(const headq_cache& c, int Hq, int T) {
  const int units = c.B * c.Hkv, G = Hq / c.Hkv;
  if (units <= 0 || !mma_decode_supported(c, G)) return 0;
  const int slots = mma_decode_ctas_per_sm(c, G) * sm_count();
  return std::max(1, std::min({(T + 63) / 64, kMaxMmaSplits, 4 * ((slots + units - 1) / units) + 4}));
}

// ... and of single tokens: [error word][queries][lengths][outputs][log-sum-exps][arrival
// counters, zeroed by each call][partials of the decode kernel]
struct TreeOneWs {
  size_t q, lens, out, lse, counters, part, bytes;
};
TreeOneWs tree_one_ws(const headq_cache& c, int Hq, int splits) {
  TreeOneWs w{};
  const size_t rows = static_cast<size_t>(c.B) * Hq;
  w.q = kWsHeaderBytes;
  w.lens = w.q + round256(rows * c.d * 2);
  w.out = w.lens + round256(static_cast<size_t>(c.B) * 4);
  w.lse = w.out + round256(rows * c.d * 4);
  w.counters = w.lse + round256(rows * 4);
  w.part = w.counters + round256(static_cast<size_t>(c.B) * c.Hkv * 4);
  w.bytes = w.part + round256(rows * splits * (c.d + 2) * sizeof(float));
  return w;
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
  if (src_rows < 0 || (src && !aligned16(src))) return HEADQ_ERR_INVALID_ARG;
  if (span->n == 0 || span->rows == 0 || cache->B == 0) return HEADQ_OK;
  if (!src && src_rows != span->rows) return HEADQ_ERR_INVALID_ARG;
  if (src_rows == 0) return HEADQ_OK;  // no token has a row to come from
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
  p.span.n = std::min(span->n, span->rows);  // a sequence has no more rows than there are
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
  p.span.n = std::min(span->n, span->rows);
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
  // the largest over both dtypes of the queries and every smaller n and T
  size_t most = tree_ws(*cache, n, tree_max_part_rows(*cache, Hq, n, T, false), false, 0).bytes;
  if (!tree_mma_supported(*cache) || cache->B == 0) return most;
  const long long blocks = (static_cast<long long>(n) * (Hq / cache->Hkv) + 127) / 128;
  most = std::max(most, tree_ws(*cache, n, tree_max_part_rows(*cache, Hq, n, T, true), true,
                                static_cast<int>(blocks)).bytes);
  return std::max(most, tree_one_ws(*cache, Hq, decode_max_splits(*cache, Hq, T)).bytes);
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
  const TreePlan tp = tree_plan(*cache, Hq, span->n, span->T, qb);
  const size_t part_rows =
      tp.parts > 1 ? static_cast<size_t>(cache->B) * Hq * span->n * tp.parts : 0;
  const TreeWs w = tree_ws(*cache, span->n, part_rows, tp.mma, tp.blocks);
  const TreeOneWs o = tree_one_ws(*cache, Hq, tp.one ? decode_plan(*cache, Hq, span->T).splits : 0);
  if (!ws || !aligned16(ws) || ws_bytes < (tp.one ? o.bytes : w.bytes)) return HEADQ_ERR_WORKSPACE;
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
  p.splits = tp.parts;
  p.chunk = tp.chunk;
  uint8_t* base = static_cast<uint8_t*>(ws);
  p.err = reinterpret_cast<unsigned*>(base);
  if (tp.one) {
    const TreeOne t{base + o.q,
                    reinterpret_cast<int32_t*>(base + o.lens),
                    reinterpret_cast<float*>(base + o.out),
                    reinterpret_cast<float*>(base + o.lse),
                    reinterpret_cast<unsigned*>(base + o.counters),
                    reinterpret_cast<float*>(base + o.part)};
    return launch_tree_one(p, t, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? HEADQ_OK
                                                                                        : HEADQ_ERR_CUDA;
  }
  p.part_o = reinterpret_cast<float*>(base + kWsHeaderBytes);
  p.part_ml = reinterpret_cast<float4*>(base + w.part_ml);
  TreeMma t{};
  t.qimg = base + w.qimg;
  t.qf = reinterpret_cast<float*>(base + w.qf);
  t.words = mask ? reinterpret_cast<uint32_t*>(base + w.words) : nullptr;
  t.wpr = (span->n + 31) / 32;
  t.blocks = tp.blocks;
  return launch_tree(p, t, tp, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? HEADQ_OK
             : HEADQ_ERR_CUDA;
}
