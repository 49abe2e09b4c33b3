// C-ABI entry points around the paged cache's sparse path: kv_cache_write_rope,
// page_digest_update, page_select, kv_pages_copy.  Host-side validation and launches.
#include <algorithm>
#include <cmath>

#include "api_paged.h"
#include "launch.h"

namespace dsa {
namespace {

constexpr int kMaxBlocks = kMaxSeqs;   // query blocks: the sequences of the attention over their lists
constexpr int kMaxQueryBlock = 256;
constexpr int kMaxListed = 1 << 24;    // of each kind of listed page
constexpr int kMaxCopies = 1 << 24;

long long bounds_bytes(const dsa_paged_shape *s) { return static_cast<long long>(s->n_pages) * s->H_kv * 2 * s->D; }
long long exp_bytes(const dsa_paged_shape *s) { return static_cast<long long>(s->n_pages) * s->H_kv; }

// Token rows of one width: slices of one fused row share its stride, and lie apart where their places
// in it do.
struct Rows {
  const char *name;
  const void *p;
  long long stride, width;   // elements of two bytes
};

bool rows_apart(const Rows &x, const Rows &y, long long n) {
  const unsigned long long a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  const unsigned long long xn = ((n - 1) * x.stride + x.width) * 2, yn = ((n - 1) * y.stride + y.width) * 2;
  if (a < b ? xn <= b - a : yn <= a - b) return true;
  if (x.stride != y.stride) return false;
  const unsigned long long period = 2ull * x.stride, d = a < b ? (b - a) % period : (period - (a - b) % period) % period;
  return d >= 2ull * x.width && d + 2ull * y.width <= period;
}

int check_rope(const dsa_rope_cfg *c, const dsa_paged_shape *s) {
  if (!c) return fail(DSA_ERR_INVALID_ARG, "cfg is NULL");
  if (c->rot < 0 || c->rot > s->D || c->rot % 16)
    return fail(DSA_ERR_INVALID_ARG, "rot=%d must be a multiple of 16 in [0, %d]", c->rot, s->D);
  if (!(c->eps >= 0.f) || !std::isfinite(c->eps)) return fail(DSA_ERR_INVALID_ARG, "eps=%g must be finite and >= 0", c->eps);
  if (!std::isfinite(c->rope_scale)) return fail(DSA_ERR_INVALID_ARG, "rope_scale must be finite");
  const size_t w = c->weight_f32 ? 4 : 2;
  if ((c->q_weight && !aligned(c->q_weight, w)) || (c->k_weight && !aligned(c->k_weight, w)))
    return fail(DSA_ERR_ALIGNMENT, "q_weight and k_weight must be %zu-byte aligned", w);
  if (c->rot && !aligned(c->inv_freq, 8)) return fail(DSA_ERR_ALIGNMENT, "inv_freq must be non-NULL and 8-byte aligned");
  return DSA_OK;
}

int check_digest(const int8_t *bounds, const int8_t *exp) {
  if (!aligned(bounds, 16)) return fail(DSA_ERR_ALIGNMENT, "bounds must be non-NULL and 16-byte aligned");
  if (!exp) return fail(DSA_ERR_ALIGNMENT, "exp is NULL");
  return DSA_OK;
}

int select_sizes(const dsa_paged_shape *s, const dsa_page_select_cfg *c, int *n_blocks, int *max_list) {
  if (!c) return fail(DSA_ERR_INVALID_ARG, "cfg is NULL");
  if (c->keep < 0 || c->n_sink < 0 || c->n_local < 0 || c->keep > kMaxListed || c->n_sink > kMaxListed ||
      c->n_local > kMaxListed)
    return fail(DSA_ERR_INVALID_ARG, "keep=%d, n_sink=%d and n_local=%d must be in [0, %d]", c->keep, c->n_sink, c->n_local,
                kMaxListed);
  if (c->q_block < 1 || c->q_block > kMaxQueryBlock)
    return fail(DSA_ERR_UNSUPPORTED, "q_block=%d outside [1, %d]", c->q_block, kMaxQueryBlock);
  if (s->max_pages > kSelectMaxPages)
    return fail(DSA_ERR_UNSUPPORTED, "max_pages=%d > %d", s->max_pages, kSelectMaxPages);
  // (a call without tokens has a block too: the attention over the lists takes one sequence at least)
  const long long blocks =
      std::max(1ll, (s->n_tok + static_cast<long long>(s->B) * (c->q_block - 1)) / c->q_block);
  if (blocks > kMaxBlocks)
    return fail(DSA_ERR_UNSUPPORTED, "%lld blocks of q_block=%d queries > %d", blocks, c->q_block, kMaxBlocks);
  const long long list = static_cast<long long>(c->n_sink) + c->keep + c->n_local +
                         (c->q_block + s->page_size - 2) / s->page_size + 1;
  if (list * s->page_size > (1ll << 30))
    return fail(DSA_ERR_INVALID_ARG, "lists of %lld pages of %d tokens: more than 2^30 tokens", list, s->page_size);
  *n_blocks = static_cast<int>(blocks);
  *max_list = static_cast<int>(list);
  return DSA_OK;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

int kv_cache_write_rope(const void *q, long long q_stride, const void *k_new, long long k_stride, const void *v_new,
                        long long v_stride, const int32_t *q_start, const int32_t *kv_len, const int32_t *page_table,
                        const dsa_paged_shape *shape, const dsa_rope_cfg *cfg, void *q_out, long long qo_stride,
                        void *k_pages, void *v_pages, uint8_t *k_scale, uint8_t *v_scale, void *stream) {
  clear_error();
  int st = check_paged_shape(shape);
  if (st) return st;
  if ((st = check_rope(cfg, shape))) return st;
  if ((st = check_cache(shape, k_pages, v_pages, k_scale, v_scale, kv_len, page_table))) return st;
  if (!aligned(q_start, 4)) return fail(DSA_ERR_ALIGNMENT, "q_start must be non-NULL and 4-byte aligned");
  if ((st = check_stride("q_stride", q_stride, shape->H_q, shape->D))) return st;
  if ((st = check_stride("k_stride", k_stride, shape->H_kv, shape->D))) return st;
  if ((st = check_stride("v_stride", v_stride, shape->H_kv, shape->D))) return st;
  if ((st = check_stride("qo_stride", qo_stride, shape->H_q, shape->D))) return st;
  if (shape->n_tok == 0) return DSA_OK;
  if (!aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(q_out, 16))
    return fail(DSA_ERR_ALIGNMENT, "q, k_new, v_new and q_out must be non-NULL and 16-byte aligned");
  const long long wq = static_cast<long long>(shape->H_q) * shape->D, wk = static_cast<long long>(shape->H_kv) * shape->D;
  const Rows out = {"q_out", q_out, qo_stride, wq};
  const Rows in[] = {{"q", q, q_stride, wq}, {"k_new", k_new, k_stride, wk}, {"v_new", v_new, v_stride, wk}};
  const bool in_place = q_out == q && qo_stride == q_stride;
  for (int i = in_place ? 1 : 0; i < 3; ++i)
    if (!rows_apart(out, in[i], shape->n_tok)) return fail(DSA_ERR_INVALID_ARG, "q_out and %s overlap", in[i].name);
  const long long wb = shape->D * (cfg->weight_f32 ? 4ll : 2ll);
  const Span outs[] = {{"k_pages", k_pages, page_bytes(shape)},
                       {"v_pages", v_pages, page_bytes(shape)},
                       {"k_scale", k_scale, scale_bytes(shape)},
                       {"v_scale", v_scale, scale_bytes(shape)}};
  const Span ins[] = {{"q", q, token_bytes(shape, q_stride, shape->H_q)},
                      {"q_out", q_out, token_bytes(shape, qo_stride, shape->H_q)},
                      {"k_new", k_new, token_bytes(shape, k_stride, shape->H_kv)},
                      {"v_new", v_new, token_bytes(shape, v_stride, shape->H_kv)},
                      {"q_start", q_start, 4ll * (shape->B + 1)},
                      {"kv_len", kv_len, 4ll * shape->B},
                      {"page_table", page_table, table_bytes(shape)},
                      {"q_weight", cfg->q_weight, wb},
                      {"k_weight", cfg->k_weight, wb},
                      {"inv_freq", cfg->rot ? cfg->inv_freq : nullptr, 4ll * cfg->rot}};
  if ((st = check_apart(outs, ins))) return st;
  const Span qo[] = {ins[1]};
  const Span rest[] = {ins[4], ins[5], ins[6], ins[7], ins[8], ins[9]};
  if ((st = check_apart(qo, rest))) return st;
  RopeWriteArgs a{};
  a.q = static_cast<const uint16_t *>(q);
  a.k_new = static_cast<const uint16_t *>(k_new);
  a.v_new = static_cast<const uint16_t *>(v_new);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.qo_stride = qo_stride;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.page_table = page_table;
  a.B = shape->B;
  a.n_tok = shape->n_tok;
  a.max_pages = shape->max_pages;
  a.n_pages = shape->n_pages;
  a.page_size = shape->page_size;
  a.H_q = shape->H_q;
  a.H_kv = shape->H_kv;
  a.D = shape->D;
  a.fp8 = shape->dtype == DSA_BF16_FP8KV;
  a.cfg = *cfg;
  a.q_out = static_cast<uint16_t *>(q_out);
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  const cudaError_t e = launch_kv_write_rope(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rotating cache write launch");
  return DSA_OK;
}

int page_digest_update(const void *k_pages, const uint8_t *k_scale, const int32_t *q_start, const int32_t *kv_len,
                       const int32_t *page_table, const dsa_paged_shape *shape, int8_t *bounds, int8_t *exp,
                       void *stream) {
  clear_error();
  int st = check_paged_shape(shape);
  if (st) return st;
  if ((st = check_cache(shape, k_pages, k_pages, k_scale, k_scale, kv_len, page_table))) return st;
  if (!aligned(q_start, 4)) return fail(DSA_ERR_ALIGNMENT, "q_start must be non-NULL and 4-byte aligned");
  if ((st = check_digest(bounds, exp))) return st;
  if (shape->n_tok == 0) return DSA_OK;
  const Span outs[] = {{"bounds", bounds, bounds_bytes(shape)}, {"exp", exp, exp_bytes(shape)}};
  const Span ins[] = {{"k_pages", k_pages, page_bytes(shape)},
                      {"k_scale", k_scale, scale_bytes(shape)},
                      {"q_start", q_start, 4ll * (shape->B + 1)},
                      {"kv_len", kv_len, 4ll * shape->B},
                      {"page_table", page_table, table_bytes(shape)}};
  if ((st = check_apart(outs, ins))) return st;
  DigestArgs a{};
  a.k_pages = k_pages;
  a.k_scale = k_scale;
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
  a.bounds = bounds;
  a.exp = exp;
  const cudaError_t e = launch_page_digest(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "page digest launch");
  return DSA_OK;
}

int page_select_sizes(const dsa_paged_shape *shape, const dsa_page_select_cfg *cfg, int *n_blocks, int *max_list) {
  clear_error();
  int st = check_paged_shape(shape);
  if (st) return st;
  if (!n_blocks || !max_list) return fail(DSA_ERR_ALIGNMENT, "n_blocks or max_list is NULL");
  return select_sizes(shape, cfg, n_blocks, max_list);
}

int page_select(const void *q, long long q_stride, const int8_t *bounds, const int8_t *exp, const int32_t *q_start,
                const int32_t *kv_len, const int32_t *page_table, const dsa_paged_shape *shape,
                const dsa_page_select_cfg *cfg, int32_t *sel_q_start, int32_t *sel_kv_len, int32_t *sel_table,
                int32_t *sel_index, void *stream) {
  clear_error();
  int st = check_paged_shape(shape);
  if (st) return st;
  PageSelectArgs a{};
  if ((st = select_sizes(shape, cfg, &a.n_blocks, &a.max_list))) return st;
  if ((st = check_digest(bounds, exp))) return st;
  if (!aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(page_table, 4))
    return fail(DSA_ERR_ALIGNMENT, "q_start, kv_len and page_table must be non-NULL and 4-byte aligned");
  if ((st = check_stride("q_stride", q_stride, shape->H_q, shape->D))) return st;
  const bool none = shape->n_tok == 0;   // (outputs that are NULL are then skipped)
  if (!none && !aligned(q, 16)) return fail(DSA_ERR_ALIGNMENT, "q must be non-NULL and 16-byte aligned");
  auto bad = [](const void *p, bool may_be_null) { return p ? !aligned(p, 4) : !may_be_null; };
  if (bad(sel_q_start, none) || bad(sel_kv_len, none) || bad(sel_table, none) || bad(sel_index, true))
    return fail(DSA_ERR_ALIGNMENT, "sel_q_start, sel_kv_len and sel_table must be non-NULL, all outputs 4-byte aligned");
  const long long lists = static_cast<long long>(a.n_blocks) * shape->H_kv * a.max_list * 4;
  const Span outs[] = {{"sel_q_start", sel_q_start, 4ll * (a.n_blocks + 1)},
                       {"sel_kv_len", sel_kv_len, 4ll * a.n_blocks},
                       {"sel_table", sel_table, lists},
                       {"sel_index", sel_index, lists}};
  const Span ins[] = {{"q", q, token_bytes(shape, q_stride, shape->H_q)},
                      {"bounds", bounds, bounds_bytes(shape)},
                      {"exp", exp, exp_bytes(shape)},
                      {"q_start", q_start, 4ll * (shape->B + 1)},
                      {"kv_len", kv_len, 4ll * shape->B},
                      {"page_table", page_table, table_bytes(shape)}};
  if ((st = check_apart(outs, ins))) return st;
  if (none) {
    // blocks without rows, keys and pages
    for (const Span &o : outs) {
      const int byte = o.p == sel_q_start || o.p == sel_kv_len ? 0 : 0xff;
      const cudaError_t e = !o.p ? cudaSuccess
                                 : cudaMemsetAsync(const_cast<void *>(o.p), byte, static_cast<size_t>(o.n),
                                                   static_cast<cudaStream_t>(stream));
      if (e != cudaSuccess) return cuda_fail(e, "page selection without tokens");
    }
    return DSA_OK;
  }
  a.q = static_cast<const uint16_t *>(q);
  a.q_stride = q_stride;
  a.bounds = bounds;
  a.exp = exp;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.page_table = page_table;
  a.B = shape->B;
  a.n_tok = shape->n_tok;
  a.max_pages = shape->max_pages;
  a.n_pages = shape->n_pages;
  a.page_size = shape->page_size;
  a.H_q = shape->H_q;
  a.H_kv = shape->H_kv;
  a.D = shape->D;
  a.cfg = *cfg;
  a.sel_q_start = sel_q_start;
  a.sel_kv_len = sel_kv_len;
  a.sel_table = sel_table;
  a.sel_index = sel_index;
  const cudaError_t e = launch_page_select(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "page selection launch");
  return DSA_OK;
}

int kv_pages_copy(const int32_t *src, const int32_t *dst, int n, const dsa_paged_shape *shape, void *k_pages,
                  void *v_pages, uint8_t *k_scale, uint8_t *v_scale, int8_t *bounds, int8_t *exp, void *stream) {
  clear_error();
  int st = check_paged_shape(shape);
  if (st) return st;
  if (n < 0 || n > kMaxCopies) return fail(DSA_ERR_INVALID_ARG, "n=%d outside [0, %d]", n, kMaxCopies);
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16))
    return fail(DSA_ERR_ALIGNMENT, "k_pages and v_pages must be non-NULL and 16-byte aligned");
  const bool fp8 = shape->dtype == DSA_BF16_FP8KV;
  if (fp8 && (!k_scale || !v_scale)) return fail(DSA_ERR_ALIGNMENT, "an FP8 cache needs k_scale and v_scale");
  if (!bounds != !exp) return fail(DSA_ERR_INVALID_ARG, "bounds and exp go together");
  if (bounds && (st = check_digest(bounds, exp))) return st;
  if (n == 0) return DSA_OK;
  if (!aligned(src, 4) || !aligned(dst, 4))
    return fail(DSA_ERR_ALIGNMENT, "src and dst must be non-NULL and 4-byte aligned");
  const Span outs[] = {{"k_pages", k_pages, page_bytes(shape)},   {"v_pages", v_pages, page_bytes(shape)},
                       {"k_scale", k_scale, scale_bytes(shape)},  {"v_scale", v_scale, scale_bytes(shape)},
                       {"bounds", bounds, bounds_bytes(shape)},   {"exp", exp, exp_bytes(shape)}};
  const Span ins[] = {{"src", src, 4ll * n}, {"dst", dst, 4ll * n}};
  if ((st = check_apart(outs, ins))) return st;
  const long long row = static_cast<long long>(shape->page_size) * shape->H_kv;
  PageCopyArgs a{};
  a.src = src;
  a.dst = dst;
  a.n = n;
  a.n_pages = shape->n_pages;
  a.big[0] = static_cast<char *>(k_pages);
  a.big[1] = static_cast<char *>(v_pages);
  a.big_bytes = row * shape->D * (fp8 ? 1 : 2);
  a.small[0] = fp8 ? reinterpret_cast<char *>(k_scale) : nullptr;
  a.small[1] = fp8 ? reinterpret_cast<char *>(v_scale) : nullptr;
  a.small[2] = reinterpret_cast<char *>(bounds);
  a.small[3] = reinterpret_cast<char *>(exp);
  a.small_bytes[0] = a.small_bytes[1] = static_cast<int>(row);
  a.small_bytes[2] = shape->H_kv * 2 * shape->D;
  a.small_bytes[3] = shape->H_kv;
  const cudaError_t e = launch_page_copy(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "page copy launch");
  return DSA_OK;
}

}  // extern "C"
