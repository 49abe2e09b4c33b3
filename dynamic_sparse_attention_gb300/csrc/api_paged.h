// Host-side checks that the entry points of the paged cache share (api_paged.cpp, api_pages.cpp).
#pragma once

#include "api_common.h"

namespace dsa {

constexpr int kMaxSeqs = 4096;   // sequences of a call: the schedule holds one sum of each in shared memory

inline int check_paged_shape(const dsa_paged_shape *s) {
  if (!s) return fail(DSA_ERR_INVALID_ARG, "shape is NULL");
  if (s->B < 1) return fail(DSA_ERR_INVALID_ARG, "B=%d < 1", s->B);
  if (s->B > kMaxSeqs) return fail(DSA_ERR_UNSUPPORTED, "B=%d > %d", s->B, kMaxSeqs);
  if (s->n_tok < 0 || s->n_tok > (1 << 30))
    return fail(DSA_ERR_INVALID_ARG, "n_tok=%d outside [0, 2^30]", s->n_tok);
  if (s->n_pages < 1 || s->max_pages < 1)
    return fail(DSA_ERR_INVALID_ARG, "n_pages=%d and max_pages=%d must be >= 1", s->n_pages, s->max_pages);
  if (s->page_size < 16 || s->page_size > 1024 || (s->page_size & (s->page_size - 1)))
    return fail(DSA_ERR_UNSUPPORTED, "page_size=%d is not a power of two in [16, 1024]", s->page_size);
  if (static_cast<long long>(s->max_pages) * s->page_size > (1ll << 30))
    return fail(DSA_ERR_INVALID_ARG, "max_pages * page_size = %lld tokens > 2^30",
                static_cast<long long>(s->max_pages) * s->page_size);
  if (s->H_q < 1 || s->H_kv < 1 || s->H_q % s->H_kv != 0)
    return fail(DSA_ERR_INVALID_ARG, "H_q=%d must be a positive multiple of H_kv=%d", s->H_q, s->H_kv);
  if (s->H_q > 128) return fail(DSA_ERR_UNSUPPORTED, "H_q=%d > 128", s->H_q);
  if (s->D != 64 && s->D != 128) return fail(DSA_ERR_UNSUPPORTED, "D=%d not in {64, 128}", s->D);
  if (s->dtype != DSA_BF16 && s->dtype != DSA_BF16_FP8KV)
    return fail(DSA_ERR_UNSUPPORTED, "dtype=%d not DSA_BF16 / DSA_BF16_FP8KV", s->dtype);
  return DSA_OK;
}

// the cache's arrays and the tables that every call reads
inline int check_cache(const dsa_paged_shape *s, const void *k_pages, const void *v_pages, const uint8_t *k_scale,
                const uint8_t *v_scale, const int32_t *kv_len, const int32_t *page_table) {
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16))
    return fail(DSA_ERR_ALIGNMENT, "k_pages and v_pages must be non-NULL and 16-byte aligned");
  if (s->dtype == DSA_BF16_FP8KV && (!k_scale || !v_scale))
    return fail(DSA_ERR_ALIGNMENT, "an FP8 cache needs k_scale and v_scale");
  if (!aligned(kv_len, 4) || !aligned(page_table, 4))
    return fail(DSA_ERR_ALIGNMENT, "kv_len and page_table must be non-NULL and 4-byte aligned");
  return DSA_OK;
}

inline int check_stride(const char *name, long long stride, int heads, int D) {
  if (stride < static_cast<long long>(heads) * D || stride % 8 != 0 || stride >= (1ll << 38))
    return fail(DSA_ERR_INVALID_ARG, "%s=%lld must be a multiple of 8 in [%d, 2^38)", name, stride, heads * D);
  return DSA_OK;
}

// a range of device memory
struct Span {
  const char *name;
  const void *p;
  long long n;
};

// each of `outs` is apart from the others and from every one of `ins`
template <int N, int M>
int check_apart(const Span (&outs)[N], const Span (&ins)[M]) {
  auto apart = [](const Span &x, const Span &y) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
    return !x.p || !y.p || x.n <= 0 || y.n <= 0 || (a < b ? static_cast<unsigned long long>(x.n) <= b - a
                                  : static_cast<unsigned long long>(y.n) <= a - b);
  };
  for (int i = 0; i < N; ++i) {
    for (int j = 0; j < i; ++j)
      if (!apart(outs[i], outs[j]))
        return fail(DSA_ERR_INVALID_ARG, "%s and %s overlap", outs[i].name, outs[j].name);
    for (int j = 0; j < M; ++j)
      if (!apart(outs[i], ins[j])) return fail(DSA_ERR_INVALID_ARG, "%s and %s overlap", outs[i].name, ins[j].name);
  }
  return DSA_OK;
}

inline long long token_bytes(const dsa_paged_shape *s, long long stride, int heads) {
  return ((s->n_tok - 1) * stride + static_cast<long long>(heads) * s->D) * 2;
}

inline long long page_bytes(const dsa_paged_shape *s) {
  return static_cast<long long>(s->n_pages) * s->page_size * s->H_kv * s->D * (s->dtype == DSA_BF16_FP8KV ? 1 : 2);
}

inline long long scale_bytes(const dsa_paged_shape *s) {   // (a bf16 cache has none, whatever the pointers)
  return s->dtype == DSA_BF16_FP8KV ? static_cast<long long>(s->n_pages) * s->page_size * s->H_kv : 0;
}

inline long long table_bytes(const dsa_paged_shape *s) { return static_cast<long long>(s->B) * s->max_pages * 4; }

}  // namespace dsa
