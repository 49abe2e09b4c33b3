// C-ABI entry points of the paged key/value cache: kv_cache_write, kv_cache_read, paged_attn,
// paged_attn_lists.
// Host-side validation, workspace layout and kernel launches on the caller's stream.
#include <cmath>

#include "api_paged.h"
#include "launch.h"

namespace dsa {
namespace {

struct PagedWs {
  float *part, *part_ml;
  PagedPiece *piece;
  int part_rows;
  size_t bytes;
};

PagedWs paged_layout(const dsa_paged_shape *s, void *base) {
  PagedWs w{};
  w.part_rows = paged_part_rows(s->n_tok, s->H_q / s->H_kv);
  Carve cv(base);
  w.part = cv.take<float>(static_cast<size_t>(2) * kPagedMaxCtas * w.part_rows * s->D);
  w.part_ml = cv.take<float>(static_cast<size_t>(2) * kPagedMaxCtas * w.part_rows * 2);
  w.piece = cv.take<PagedPiece>(kPagedMaxCtas);
  w.bytes = cv.bytes();
  return w;
}

// paged_attn with one table a sequence, or one for each of its KV heads
int attend(bool per_head, const void *q, long long q_stride, const void *k_pages, const void *v_pages,
           const uint8_t *k_scale, const uint8_t *v_scale, const int32_t *q_start, const int32_t *kv_len,
           const int32_t *page_table, const dsa_paged_shape *shape, int n_sink, int n_stream, float scale, void *out,
           float *lse, void *ws, size_t ws_bytes, void *stream) {
  clear_error();
  int st = check_paged_shape(shape);
  if (st) return st;
  if (n_sink < 0 || n_stream < -1)
    return fail(DSA_ERR_INVALID_ARG, "n_sink=%d must be >= 0 and n_stream=%d >= -1", n_sink, n_stream);
  if (!(scale > 0.f) || !std::isfinite(scale))
    return fail(DSA_ERR_INVALID_ARG, "scale=%g must be positive and finite", scale);
  if ((st = check_cache(shape, k_pages, v_pages, k_scale, v_scale, kv_len, page_table))) return st;
  if (!aligned(q_start, 4)) return fail(DSA_ERR_ALIGNMENT, "q_start must be non-NULL and 4-byte aligned");
  if ((st = check_stride("q_stride", q_stride, shape->H_q, shape->D))) return st;
  if (shape->n_tok == 0) return DSA_OK;
  if (!aligned(q, 16) || !aligned(out, 16))
    return fail(DSA_ERR_ALIGNMENT, "q and out must be non-NULL and 16-byte aligned");
  if (lse && !aligned(lse, 4)) return fail(DSA_ERR_ALIGNMENT, "lse must be 4-byte aligned");
  const size_t need = paged_layout(shape, nullptr).bytes;
  if (ws_bytes < need || !aligned(ws, 16))
    return fail(DSA_ERR_WORKSPACE, "workspace of %zu bytes (16-byte aligned) needed, got %zu", need, ws_bytes);
  const long long rows = static_cast<long long>(shape->n_tok) * shape->H_q;
  const Span outs[] = {{"out", out, rows * shape->D * 2}, {"lse", lse, rows * 4}, {"workspace", ws, static_cast<long long>(need)}};
  const Span ins[] = {{"q", q, token_bytes(shape, q_stride, shape->H_q)},
                      {"k_pages", k_pages, page_bytes(shape)},
                      {"v_pages", v_pages, page_bytes(shape)},
                      {"k_scale", k_scale, scale_bytes(shape)},
                      {"v_scale", v_scale, scale_bytes(shape)},
                      {"q_start", q_start, 4ll * (shape->B + 1)},
                      {"kv_len", kv_len, 4ll * shape->B},
                      {"page_table", page_table, table_bytes(shape) * (per_head ? shape->H_kv : 1)}};
  if ((st = check_apart(outs, ins))) return st;
  if ((st = paged_attn_ready())) return st;
  const PagedWs w = paged_layout(shape, ws);
  PagedAttnArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.page_table = page_table;
  a.B = shape->B;
  a.per_head = per_head;
  a.n_tok = shape->n_tok;
  a.max_pages = shape->max_pages;
  a.n_pages = shape->n_pages;
  a.page_size = shape->page_size;
  a.H_q = shape->H_q;
  a.H_kv = shape->H_kv;
  a.D = shape->D;
  a.fp8 = shape->dtype == DSA_BF16_FP8KV;
  a.n_sink = n_sink;
  a.n_stream = n_stream;
  a.scale = scale;
  a.out = static_cast<uint16_t *>(out);
  a.lse = lse;
  a.part_rows = w.part_rows;
  a.part = w.part;
  a.part_ml = w.part_ml;
  a.piece = w.piece;
  const cudaError_t e = launch_paged_attn(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "paged attention launch");
  return DSA_OK;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

int kv_cache_write(const void *k_new, const void *v_new, long long k_stride, long long v_stride,
                   const int32_t *q_start, const int32_t *kv_len, const int32_t *page_table,
                   const dsa_paged_shape *shape, void *k_pages, void *v_pages, uint8_t *k_scale, uint8_t *v_scale,
                   void *stream) {
  clear_error();
  int st = check_paged_shape(shape);
  if (st) return st;
  if ((st = check_cache(shape, k_pages, v_pages, k_scale, v_scale, kv_len, page_table))) return st;
  if (!aligned(q_start, 4)) return fail(DSA_ERR_ALIGNMENT, "q_start must be non-NULL and 4-byte aligned");
  if ((st = check_stride("k_stride", k_stride, shape->H_kv, shape->D))) return st;
  if ((st = check_stride("v_stride", v_stride, shape->H_kv, shape->D))) return st;
  if (shape->n_tok == 0) return DSA_OK;
  if (!aligned(k_new, 16) || !aligned(v_new, 16))
    return fail(DSA_ERR_ALIGNMENT, "k_new and v_new must be non-NULL and 16-byte aligned");
  const Span outs[] = {{"k_pages", k_pages, page_bytes(shape)},
                       {"v_pages", v_pages, page_bytes(shape)},
                       {"k_scale", k_scale, scale_bytes(shape)},
                       {"v_scale", v_scale, scale_bytes(shape)}};
  const Span ins[] = {{"k_new", k_new, token_bytes(shape, k_stride, shape->H_kv)},
                      {"v_new", v_new, token_bytes(shape, v_stride, shape->H_kv)},
                      {"q_start", q_start, 4ll * (shape->B + 1)},
                      {"kv_len", kv_len, 4ll * shape->B},
                      {"page_table", page_table, table_bytes(shape)}};
  if ((st = check_apart(outs, ins))) return st;
  CacheWriteArgs a{};
  a.k_new = static_cast<const uint16_t *>(k_new);
  a.v_new = static_cast<const uint16_t *>(v_new);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.page_table = page_table;
  a.B = shape->B;
  a.n_tok = shape->n_tok;
  a.max_pages = shape->max_pages;
  a.n_pages = shape->n_pages;
  a.page_size = shape->page_size;
  a.H_kv = shape->H_kv;
  a.D = shape->D;
  a.fp8 = shape->dtype == DSA_BF16_FP8KV;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  const cudaError_t e = launch_kv_write(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cache write launch");
  return DSA_OK;
}

int kv_cache_read(const void *k_pages, const void *v_pages, const uint8_t *k_scale, const uint8_t *v_scale,
                  const int32_t *kv_len, const int32_t *page_table, const dsa_paged_shape *shape, int T_max,
                  void *k_out, void *v_out, void *stream) {
  clear_error();
  int st = check_paged_shape(shape);
  if (st) return st;
  if ((st = check_cache(shape, k_pages, v_pages, k_scale, v_scale, kv_len, page_table))) return st;
  if (T_max < 1) return fail(DSA_ERR_INVALID_ARG, "T_max=%d < 1", T_max);
  if (!aligned(k_out, 16) || !aligned(v_out, 16))
    return fail(DSA_ERR_ALIGNMENT, "k_out and v_out must be non-NULL and 16-byte aligned");
  const long long rows = static_cast<long long>(shape->B) * T_max * shape->H_kv * shape->D * 2;
  const Span outs[] = {{"k_out", k_out, rows}, {"v_out", v_out, rows}};
  const Span ins[] = {{"k_pages", k_pages, page_bytes(shape)},
                      {"v_pages", v_pages, page_bytes(shape)},
                      {"k_scale", k_scale, scale_bytes(shape)},
                      {"v_scale", v_scale, scale_bytes(shape)},
                      {"kv_len", kv_len, 4ll * shape->B},
                      {"page_table", page_table, table_bytes(shape)}};
  if ((st = check_apart(outs, ins))) return st;
  CacheReadArgs a{};
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.kv_len = kv_len;
  a.page_table = page_table;
  a.B = shape->B;
  a.T_max = T_max;
  a.max_pages = shape->max_pages;
  a.n_pages = shape->n_pages;
  a.page_size = shape->page_size;
  a.H_kv = shape->H_kv;
  a.D = shape->D;
  a.fp8 = shape->dtype == DSA_BF16_FP8KV;
  a.k_out = k_out;
  a.v_out = v_out;
  const cudaError_t e = launch_kv_read(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cache read launch");
  return DSA_OK;
}

int paged_attn_workspace(const dsa_paged_shape *shape, size_t *bytes) {
  clear_error();
  int st = check_paged_shape(shape);
  if (st) return st;
  if (!bytes) return fail(DSA_ERR_ALIGNMENT, "bytes is NULL");
  *bytes = paged_layout(shape, nullptr).bytes;
  return DSA_OK;
}

int paged_attn(const void *q, long long q_stride, const void *k_pages, const void *v_pages, const uint8_t *k_scale,
               const uint8_t *v_scale, const int32_t *q_start, const int32_t *kv_len, const int32_t *page_table,
               const dsa_paged_shape *shape, int n_sink, int n_stream, float scale, void *out, float *lse, void *ws,
               size_t ws_bytes, void *stream) {
  return attend(false, q, q_stride, k_pages, v_pages, k_scale, v_scale, q_start, kv_len, page_table, shape, n_sink,
                n_stream, scale, out, lse, ws, ws_bytes, stream);
}

int paged_attn_lists(const void *q, long long q_stride, const void *k_pages, const void *v_pages,
                     const uint8_t *k_scale, const uint8_t *v_scale, const int32_t *q_start, const int32_t *kv_len,
                     const int32_t *page_table, const dsa_paged_shape *shape, int n_sink, int n_stream, float scale,
                     void *out, float *lse, void *ws, size_t ws_bytes, void *stream) {
  return attend(true, q, q_stride, k_pages, v_pages, k_scale, v_scale, q_start, kv_len, page_table, shape, n_sink,
                n_stream, scale, out, lse, ws, ws_bytes, stream);
}

}  // extern "C"
