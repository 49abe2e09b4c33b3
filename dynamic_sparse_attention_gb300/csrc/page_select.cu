// Digests of cache pages and the choice of pages by them (page_digest_update, page_select).
//
// Mathematics.  A page's digest holds, for each KV head, every channel's smallest and largest key
// as whole numbers lo_d <= k_d 2^-e <= hi_d in [-127, 127] (rounded outwards).  For a query row
// q' 2^(e_q), q' whole in [-127, 127],
//   q' . k 2^-e <= sum_d max(q'_d lo_d, q'_d hi_d) = sum_d (min(q'_d, 0) lo_d + max(q'_d, 0) hi_d),
// a bound on the row's score with any key of the page, and two dot products of 8-bit integers.
// The sum is below 128 * 127^2 < 2^21 in size and the scales are powers of two in [2^-50, 2^50], so
// the score is exact in fp32 in whatever order it is summed, by integer or tensor-core
// arithmetic alike (products below 2^14 and sums below 2^21 are whole in fp32's 24 bits): the
// selection has one answer, the same for every kernel and every split of the work.
//
// Measured: digests of 131,071 tokens of 8 heads of 128 in bf16 47 us, 5,820 GB/s (86 % of 6,791: HBM), in
// FP8 81 us, 1,725 GB/s (25 %: 8-byte loads, and a scale byte for each row); selection of 16 tokens over up to
// 32,768 keys in pages of 64 10 us, of one token over 1,048,576 25 us (chains of latencies: the digests are
// 1.4 and 5 us of bytes), of 2,048 tokens over 131,072 in blocks of 64 85 us, of 32, 16, 8 and 4 tokens 113,
// 184, 365 and 394 (32/8 heads; 68 GFLOP in two products, 36 us of the tensor core's burst rate; every block
// gathers and widens the digests for itself, and 64 columns or fewer leave half of an MMA empty).
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "launch.h"
#include "mma_sync.cuh"
#include "profile.h"
#include "tc_ptx.cuh"

namespace dsa {

DSA_CHECK_WORD(page_select_check_word)

namespace cg = cooperative_groups;

namespace {

using namespace tc;

static __device__ int g_select_error;   // sticky error word, read by dsa_device_error
std::atomic<unsigned long long> g_wait_limit_ns{500000000ull};   // of later launches

// ------------------------------------------------------------------ digests

constexpr int kDigestThreads = 256, kDigestPairs = kDigestThreads / 64;
constexpr int kMaxWindow = 1024, kDigestHeads = 2;   // token rows and heads of a CTA

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {   // bf16 pairs; a NaN loses
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Least e in [-50, 50] with a * 2^-e <= 127 for the finite a with fp32 bits `u`: a = 1.m * 2^x
// takes x - 6 while 1.m <= 127 / 64, else x - 5; 0 for a = 0.
__device__ __forceinline__ int exponent127(uint32_t u) {
  if (u == 0u) return 0;
  const int e = static_cast<int>(u >> 23) - 133 + ((u & 0x7fffffu) > 0x7e0000u ? 1 : 0);
  return min(max(e, -50), 50);
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// A digest's exponent as the caller's array has it: outside the digests' range it is no power of two
// that keeps a score finite, and counts as the nearest one inside.
__device__ __forceinline__ float two_to_stored(int e) {
  DSA_CHECK(e >= -50 && e <= 50);
  return two_to(min(max(e, -50), 50));
}

// The 8 keys' channels of lane's 16-byte piece (bf16) or 8-byte piece (E4M3 with the row's scale
// byte, as the bf16 values that they stand for).
template <bool FP8>
__device__ __forceinline__ uint4 load_keys(const DigestArgs &a, size_t row, int D, int piece) {
  if constexpr (FP8) {
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.k_pages) + row * D) + piece);
    const uint32_t s = __ldg(a.k_scale + row);
    // 2^(s - 127), for s = 0 a subnormal of fp32; NaN for s = 255
    const float f = __uint_as_float(s == 255u ? 0x7fffffffu : s == 0u ? 0x00400000u : s << 23);
    float x[8];
    f16x2_to_f32x2(e4m3x2_to_f16x2(w.x), x[0], x[1]);
    f16x2_to_f32x2(e4m3x2_to_f16x2(w.x >> 16), x[2], x[3]);
    f16x2_to_f32x2(e4m3x2_to_f16x2(w.y), x[4], x[5]);
    f16x2_to_f32x2(e4m3x2_to_f16x2(w.y >> 16), x[6], x[7]);
    return make_uint4(pack_bf16x2(x[0] * f, x[1] * f), pack_bf16x2(x[2] * f, x[3] * f),
                      pack_bf16x2(x[4] * f, x[5] * f), pack_bf16x2(x[6] * f, x[7] * f));
  } else {
    return __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.k_pages) + row * D) + piece);
  }
}

__device__ __forceinline__ bool is_inf(uint32_t w) {
  return (w & 0x7fffu) == 0x7f80u || ((w >> 16) & 0x7fffu) == 0x7f80u;
}

// Two warps digest one page of one head: D / 8 lanes hold 8 channels of a token each, the groups of
// them take the page's tokens in turn with running bounds in registers, and the second warp
// hands its bounds to the first.
template <int D, bool FP8>
__device__ void digest_page(const DigestArgs &a, int page, int head, int keys, uint4 (*s_part)[32] /* [2] */) {
  constexpr int LPT = D / 8, TPW = 32 / LPT, U = 8;   // lanes per token, tokens per step, steps in flight
  const int lane = threadIdx.x & 31, piece = lane % LPT, t0 = lane / LPT;
  const int second = (threadIdx.x >> 5) & 1, bar = 1 + (threadIdx.x >> 6);
  const size_t row0 = (static_cast<size_t>(page) << a.lg_page) * a.H_kv + head;
  constexpr uint32_t kNan2 = 0x7fff7fffu;
  uint32_t lo[4] = {kNan2, kNan2, kNan2, kNan2}, hi[4] = {kNan2, kNan2, kNan2, kNan2};
  for (int t = t0 + second * U * TPW; t < keys; t += 2 * U * TPW) {
    uint4 u[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      u[i] = t + i * TPW < keys ? load_keys<FP8>(a, row0 + static_cast<size_t>(t + i * TPW) * a.H_kv, D, piece)
                                : make_uint4(kNan2, kNan2, kNan2, kNan2);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        lo[c] = min2(lo[c], w[c]);
        hi[c] = max2(hi[c], w[c]);
      }
    }
  }
  if (second) {
    s_part[0][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    s_part[1][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
  named_bar_sync(bar, 64);
  if (!second) {
    const uint4 l = s_part[0][lane], h = s_part[1][lane];
    const uint32_t w[4] = {l.x, l.y, l.z, l.w}, x[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      lo[c] = min2(lo[c], w[c]);
      hi[c] = max2(hi[c], x[c]);
    }
  }
  named_bar_sync(bar, 64);                    // read: the next page's may be written
  if (second) return;
#pragma unroll
  for (int o = LPT; o < 32; o <<= 1)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      lo[c] = min2(lo[c], __shfl_xor_sync(kFull, lo[c], o));
      hi[c] = max2(hi[c], __shfl_xor_sync(kFull, hi[c], o));
    }
  // the largest finite magnitude; where a bound is infinite the finite keys behind it are looked
  // for again
  uint32_t m = 0;
  bool inf = false;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    inf |= is_inf(lo[c]) || is_inf(hi[c]);
    const uint32_t x[4] = {lo[c] << 16, lo[c], hi[c] << 16, hi[c]};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = x[i] & 0x7fff0000u;
      m = max(m, v < 0x7f800000u ? v : 0u);
    }
  }
  if (__any_sync(kFull, inf)) {
    for (int t = t0; t < keys; t += TPW) {
      const uint4 u = load_keys<FP8>(a, row0 + static_cast<size_t>(t) * a.H_kv, D, piece);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t x = (w[c] << 16) & 0x7fff0000u, y = w[c] & 0x7fff0000u;
        m = max(m, max(x < 0x7f800000u ? x : 0u, y < 0x7f800000u ? y : 0u));
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
  const int e = exponent127(m);
  const float inv = two_to(-e);
  // (a NaN bound, a channel without numbers, becomes 0; the conversion saturates infinities)
  uint32_t b[4] = {0, 0, 0, 0};              // lo of channels 0-3, 4-7, then hi
#pragma unroll
  for (int c = 0; c < 4; ++c) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float x = h ? bf16_hi(lo[c]) : bf16_lo(lo[c]), y = h ? bf16_hi(hi[c]) : bf16_lo(hi[c]);
      const int v = min(max(__float2int_rd(x * inv), -127), 127), w = min(max(__float2int_ru(y * inv), -127), 127);
      b[c >> 1] |= (static_cast<uint32_t>(v) & 0xffu) << (16 * (c & 1) + 8 * h);
      b[2 + (c >> 1)] |= (static_cast<uint32_t>(w) & 0xffu) << (16 * (c & 1) + 8 * h);
    }
  }
  if (t0 == 0) {
    const size_t out = static_cast<size_t>(page) * a.H_kv + head;
    uint2 *dst = reinterpret_cast<uint2 *>(a.bounds + out * 2 * D);
    dst[piece] = make_uint2(b[0], b[1]);
    dst[LPT + piece] = make_uint2(b[2], b[3]);
    if (lane == 0) a.exp[out] = static_cast<int8_t>(e);
  }
}

// A CTA takes the pages whose first row of a chunk lies in its `window` token rows, for kDigestHeads
// heads.  (As many CTAs as fit the GPU four times, however long the chunks: with a CTA for each page
// and a warp for each of its heads 58 us for a prompt of 128K tokens, the last of four rounds nearly
// empty.)
template <int D, bool FP8>
__global__ void __launch_bounds__(kDigestThreads, 4) digest_kernel(const DigestArgs a) {
  __shared__ int s_seq[kMaxWindow];
  __shared__ int s_page[kMaxWindow], s_keys[kMaxWindow];
  __shared__ uint4 s_part[kDigestPairs][2][32];
  __shared__ int s_n;
  const int tid = threadIdx.x, lane = tid & 31;
  const int n0 = blockIdx.x * a.window, n1 = min(a.n_tok, n0 + a.window);
  const int h0 = blockIdx.y * kDigestHeads, nh = min(kDigestHeads, a.H_kv - h0);
  grid_dep_wait();
  for (int i = tid; i < a.window; i += kDigestThreads) s_seq[i] = -1;
  if (tid == 0) s_n = 0;
  __syncthreads();
  for (int b0 = tid & ~31; b0 < a.B; b0 += kDigestThreads) {
    // the rows of a warp's sequences, marked by all of its lanes
    int lo = 0, hi = 0;
    if (b0 + lane < a.B) {
      const int qs = a.q_start[b0 + lane], qe = a.q_start[b0 + lane + 1];
      DSA_CHECK(qs >= 0 && qe <= a.n_tok);
      lo = max(qs, n0);
      hi = min(qe, n1);
    }
    uint32_t some = __ballot_sync(kFull, lo < hi);
    while (some) {
      const int src = __ffs(some) - 1;
      some &= some - 1;
      const int x = __shfl_sync(kFull, lo, src), y = __shfl_sync(kFull, hi, src);
      for (int n = x + lane; n < y; n += 32) s_seq[n - n0] = b0 + src;
    }
  }
  __syncthreads();
  for (int i = tid; i < n1 - n0; i += kDigestThreads) {
    const int b = s_seq[i], n = n0 + i;
    if (b < 0) continue;
    const int qs = a.q_start[b], qe = a.q_start[b + 1], cap = a.max_pages << a.lg_page;
    const int kv = min(max(a.kv_len[b], 0), cap);
    DSA_CHECK(kv == a.kv_len[b]);
    const long long pos = kv - (static_cast<long long>(qe) - n);
    if (pos >= 0 && ((pos & (a.page_size - 1)) == 0 || n == qs)) {
      const int p = static_cast<int>(pos >> a.lg_page);
      const int page = a.page_table[static_cast<size_t>(b) * a.max_pages + p];
      DSA_CHECK(page >= 0 && page < a.n_pages);
      if (page >= 0 && page < a.n_pages) {
        const int at = atomicAdd(&s_n, 1);   // (any order: each page is its own work)
        s_page[at] = page;
        s_keys[at] = min(a.page_size, kv - (p << a.lg_page));
      }
    }
  }
  __syncthreads();
  const int work = s_n * nh, pair = tid >> 6;
  for (int i = pair; i < work; i += kDigestPairs)
    digest_page<D, FP8>(a, s_page[i / nh], h0 + i % nh, s_keys[i / nh], s_part[pair]);
}

// ------------------------------------------------------------------ selection

// A block of queries and what its lists are made of.
struct Block {
  int b, lo, n;        // sequence, first token row, tokens
  int s0, first;       // candidates: pages [s0, first) of the sequence
  int own1;            // last own page (-1: no keys)
  int picked;          // candidates listed
  int keys;            // length of a list in keys
};

__device__ __forceinline__ int clamp_row(const PageSelectArgs &a, int x) { return min(max(x, 0), a.n_tok); }

// Block j: a scan over the sequences' counts of blocks, a run of them per thread.
template <int NT>
__device__ Block find_block(const PageSelectArgs &a, int j, int *s_scan /* [NT / 32 + 1] */, int *s_found /* [5] */) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int qb = a.cfg.q_block;
  const int per = (a.B + NT - 1) / NT, b0 = tid * per, b1 = min(a.B, b0 + per);
  int sum = 0, qs = 0, qe = 0, kv = 0;        // of the run's first sequence, asked for with the rest
  if (b0 < b1) {
    kv = a.kv_len[b0];
    qs = clamp_row(a, a.q_start[b0]);
    qe = clamp_row(a, a.q_start[b0 + 1]);
    sum = (max(qe - qs, 0) + qb - 1) / qb;
    for (int b = b0 + 1; b < b1; ++b)
      sum += (max(clamp_row(a, a.q_start[b + 1]) - clamp_row(a, a.q_start[b]), 0) + qb - 1) / qb;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_scan[warp] = incl;
  if (tid == 0) s_found[0] = -1;
  __syncthreads();
  int at = incl - sum;
  for (int w = 0; w < warp; ++w) at += s_scan[w];
  if (j >= at && j < at + sum) {
    for (int b = b0; b < b1; ++b) {
      if (b > b0) {
        qs = clamp_row(a, a.q_start[b]);
        qe = clamp_row(a, a.q_start[b + 1]);
        kv = a.kv_len[b];
      }
      const int x = (max(qe - qs, 0) + qb - 1) / qb;
      if (j < at + x) {
        s_found[0] = b;
        s_found[1] = j - at;
        s_found[2] = qs;
        s_found[3] = qe;
        s_found[4] = kv;
        break;
      }
      at += x;
    }
  }
  __syncthreads();
  Block k;
  k.b = s_found[0];
  k.s0 = k.first = k.picked = k.keys = 0;
  k.own1 = -1;
  if (k.b < 0) {
    // behind the last block: no rows, no keys, and no scores that tell pages apart, so the `keep` earliest
    // of the last sequence are picked (but not those that are sinks or local)
    k.b = a.B - 1;
    k.lo = clamp_row(a, a.q_start[a.B]);
    k.n = 0;
    const int own0 = min(max(a.kv_len[k.b], 0), a.max_pages << a.lg_page) >> a.lg_page;
    k.first = max(0, own0 - min(a.cfg.n_local, own0));
    k.s0 = min(a.cfg.n_sink, k.first);
    k.picked = max(0, min(a.cfg.keep, k.first) - k.s0);
    return k;
  }
  qs = s_found[2];
  qe = s_found[3];
  k.lo = qs + s_found[1] * qb;
  k.n = min(qb, qe - k.lo);
  const int cap = a.max_pages << a.lg_page;
  DSA_CHECK(s_found[4] >= qe - qs && s_found[4] <= cap);
  kv = min(max(s_found[4], 0), cap);
  const int p0 = kv - (qe - k.lo), p1 = p0 + k.n - 1, pc = max(p0, 0);
  if (p1 < 0) return k;
  const int own0 = pc >> a.lg_page;
  k.own1 = p1 >> a.lg_page;
  k.first = max(0, own0 - min(a.cfg.n_local, own0));
  k.s0 = min(a.cfg.n_sink, k.first);
  k.picked = min(a.cfg.keep, k.first - k.s0);
  k.keys = ((k.s0 + k.picked + own0 - k.first) << a.lg_page) + (pc & (a.page_size - 1)) + p1 - pc + 1;
  return k;
}

// entry i of the list of (block j, head g)
__device__ __forceinline__ void put(const PageSelectArgs &a, int j, int g, int i, int page, int index) {
  const size_t at = (static_cast<size_t>(j) * a.H_kv + g) * a.max_list + i;
  a.sel_table[at] = page;
  if (a.sel_index) a.sel_index[at] = index;
}

// What a list holds beside its picks, by one warp.  (A block without rows: its picks, and nothing else.)
__device__ void put_fixed(const PageSelectArgs &a, int j, int g, const Block &k) {
  const int lane = threadIdx.x & 31;
  const int32_t *table = a.page_table + static_cast<size_t>(k.b) * a.max_pages;
  if (k.n == 0) {
    for (int i = lane; i < a.max_list; i += 32) {
      const int index = i < k.picked ? k.s0 + i : -1;
      put(a, j, g, i, index < 0 ? -1 : table[index], index);
    }
    if (g == 0 && lane == 0) {
      a.sel_q_start[j] = k.lo;
      a.sel_kv_len[j] = 0;
      if (j == a.n_blocks - 1) a.sel_q_start[j + 1] = k.lo;
    }
    return;
  }
  const int count = k.own1 < 0 ? 0 : k.s0 + k.picked + k.own1 + 1 - k.first;
  for (int i = lane; i < a.max_list; i += 32) {
    if (i >= k.s0 && i < k.s0 + k.picked) continue;
    const int index = i >= count ? -1 : i < k.s0 ? i : k.first + i - k.s0 - k.picked;
    put(a, j, g, i, index < 0 ? -1 : table[index], index);
  }
  if (g == 0 && lane == 0) {
    a.sel_q_start[j] = k.lo;
    a.sel_kv_len[j] = k.keys;
    if (j == a.n_blocks - 1) a.sel_q_start[j + 1] = k.lo + k.n;
  }
}

// A lane's D / 32 elements of row r of a block (bf16 words), and what they are in fp32 with the row's
// exponent.
template <int D>
__device__ __forceinline__ void load_row(const PageSelectArgs &a, const Block &k, int g, int r, uint32_t *w) {
  const int lane = threadIdx.x & 31, G = a.H_q / a.H_kv;
  const uint16_t *src = a.q + static_cast<size_t>(k.lo + r / G) * a.q_stride + static_cast<size_t>(g * G + r % G) * D;
  if constexpr (D == 128) {
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(src) + lane);
    w[0] = u.x;
    w[1] = u.y;
  } else {
    w[0] = __ldg(reinterpret_cast<const uint32_t *>(src) + lane);
  }
}
template <int D>
__device__ __forceinline__ int row_of(const uint32_t *w, float *x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    x[i] = (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    const uint32_t v = __float_as_uint(x[i]) & 0x7fffffffu;
    m = max(m, v < 0x7f800000u ? v : 0u);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
  return exponent127(m);
}
// whole number of a scaled element (a NaN: 0)
__device__ __forceinline__ int whole(float x) { return min(max(__float2int_rn(x), -127), 127); }

struct SelectShared {
  uint32_t hist[4][256];   // of each pass, read by the whole cluster
  uint32_t tot[2][256];
  uint32_t low, high;      // of the CTA's keys
  int kept[2];             // keys above the threshold, within it
  int scan[17], found[5];
  int scan2[2][17];
};

template <int NT>
__device__ __forceinline__ void clear_shared(SelectShared &sh) {
  for (int i = threadIdx.x; i < 4 * 256; i += NT) (&sh.hist[0][0])[i] = 0;
  if (threadIdx.x == 0) {
    sh.low = 0xffffffffu;
    sh.high = 0;
  }
}

// The `k.picked` best of the cluster's keys (each CTA holds nl of them, of pages p_first ..) into the
// list.  The interval of keys that holds the last pick is narrowed 256 times at a time, from the least
// and largest key on, by histograms that the CTAs read from each other, until all of its keys are
// picks or all are equal; then every CTA writes its own picks behind those of the lower ranks.
// (Digits of the whole 32 bits, four passes whose first two put nearly all keys into a bin or two:
// 1.2 us a pass.)
template <int NT>
__device__ void pick(const PageSelectArgs &a, cg::cluster_group &cluster, SelectShared &sh, const uint32_t *key, int nl,
                     int p_first, int j, int g, const Block &k) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  auto sync = [&]() {
    if (C > 1) cluster.sync();
    else __syncthreads();
  };
  {
    uint32_t low = 0xffffffffu, high = 0;
    for (int i = tid; i < nl; i += NT) {
      low = min(low, key[i]);
      high = max(high, key[i]);
    }
    low = __reduce_min_sync(kFull, low);
    high = __reduce_max_sync(kFull, high);
    if (lane == 0) {
      atomicMin(&sh.low, low);
      atomicMax(&sh.high, high);
    }
  }
  sync();
  uint32_t lo = 0xffffffffu, hi = 0;
  for (int c = 0; c < C; ++c) {
    lo = min(lo, *cluster.map_shared_rank(&sh.low, c));
    hi = max(hi, *cluster.map_shared_rank(&sh.high, c));
  }
  uint32_t left = static_cast<uint32_t>(k.picked);   // picks in [lo, hi]; every key above is one
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = max(0, 24 - __clz(hi - lo | 1u));
    for (int i = tid; i < nl; i += NT) {
      const uint32_t x = key[i] - lo;
      if (x <= hi - lo) atomicAdd(&sh.hist[pass][x >> shift], 1u);
    }
    sync();
    if (tid < 256) {
      uint32_t t = 0;
      for (int c = 0; c < C; ++c) t += *cluster.map_shared_rank(&sh.hist[pass][tid], c);
      sh.tot[pass & 1][tid] = t;
    }
    __syncthreads();
    // every warp finds the bin that holds the last pick: lane's bins from the top down
    const int top = 255 - lane * 8;
    uint32_t c[8], sum = 0;
#pragma unroll
    for (int t = 0; t < 8; ++t) sum += c[t] = sh.tot[pass & 1][top - t];
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    uint32_t run = incl - sum, bin = 0, in = 0;
    const bool mine = run < left && left <= incl;
    if (mine) {
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        if (in == 0) {
          if (run + c[t] >= left) {
            bin = static_cast<uint32_t>(top - t);
            in = c[t];
          } else {
            run += c[t];
          }
        }
      }
    }
    const int who = __ffs(__ballot_sync(kFull, mine)) - 1;   // (the histograms hold `left` keys at least)
    left -= __shfl_sync(kFull, run, who);
    lo += __shfl_sync(kFull, bin, who) << shift;
    in = __shfl_sync(kFull, in, who);
    hi = lo + min(hi - lo, (1u << shift) - 1u);   // (the bin's end may lie past 2^32)
    if (shift == 0 || in == left) break;      // (the same for every warp of the cluster)
  }
  // keys above `hi` are in, and the first `left` of those from `lo` on
  const int per = (nl + NT - 1) / NT, i0 = min(nl, tid * per), i1 = min(nl, i0 + per);
  int gt = 0, eq = 0;
  for (int i = i0; i < i1; ++i) {
    gt += key[i] > hi;
    eq += key[i] >= lo && key[i] <= hi;
  }
  int ig = gt, ie = eq;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, ig, o), w = __shfl_up_sync(kFull, ie, o);
    if (lane >= o) {
      ig += v;
      ie += w;
    }
  }
  if (lane == 31) {
    sh.scan2[0][warp] = ig;
    sh.scan2[1][warp] = ie;
  }
  __syncthreads();
  int og = ig - gt, oe = ie - eq;             // before this thread's
  int tg = 0, te = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w == warp) {
      og += tg;
      oe += te;
    }
    tg += sh.scan2[0][w];
    te += sh.scan2[1][w];
  }
  if (C > 1) {
    if (tid == 0) {
      sh.kept[0] = tg;
      sh.kept[1] = te;
    }
    cluster.sync();
    for (int c = 0; c < rank; ++c) {
      const int *o = cluster.map_shared_rank(sh.kept, c);
      og += o[0];
      oe += o[1];
    }
  }
  const int32_t *table = a.page_table + static_cast<size_t>(k.b) * a.max_pages;
  for (int i = i0; i < i1; ++i) {
    const bool is_eq = key[i] >= lo && key[i] <= hi;
    if (key[i] > hi || (is_eq && oe < static_cast<int>(left))) {
      const int at = og + min(oe, static_cast<int>(left));
      put(a, j, g, k.s0 + at, table[p_first + i], p_first + i);
    }
    og += key[i] > hi;
    oe += is_eq;
  }
  if (C > 1) cluster.sync();                  // shared memory stays until every reader is done
}

// Every candidate is listed.
template <int NT>
__device__ void pick_all(const PageSelectArgs &a, int rank, int C, int j, int g, const Block &k) {
  const int32_t *table = a.page_table + static_cast<size_t>(k.b) * a.max_pages;
  for (int i = rank * NT + threadIdx.x; i < k.picked; i += C * NT)
    put(a, j, g, k.s0 + i, table[k.s0 + i], k.s0 + i);
}

// four signed bytes -> fp16 pairs (exact): 1024 + (x + 128) has x + 128 in its low mantissa bits
__device__ __forceinline__ uint2 widen_s8(uint32_t w) {
  w ^= 0x80808080u;
  uint32_t lo, hi;
  asm("prmt.b32 %0, %1, %2, 0x4140;\n" : "=r"(lo) : "r"(w), "r"(0x64646464u));
  asm("prmt.b32 %0, %1, %2, 0x4342;\n" : "=r"(hi) : "r"(w), "r"(0x64646464u));
  asm("sub.rn.f16x2 %0, %0, %1;\n" : "+r"(lo) : "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %0, %1;\n" : "+r"(hi) : "r"(0x64806480u));
  return make_uint2(lo, hi);
}

// Few rows (a decode step's): a launch is bound by gathering the digests, 256 bytes a page and head.
// A warp takes 16 pages at a time, the lanes' 16-byte pieces covering whole sectors of their rows,
// and multiplies them from registers: the 4 bytes of a lane's word are its elements of one
// 16-element step of mma.sync, in the same order on both sides, so nothing is moved between lanes.
// (A page per thread with dp4a: 32 rows a load, each a line of its own: 38 us for a token over 1M
// keys.)
constexpr int kFewThreads = 256, kFewRows = 16;

template <int D, int NT8>                     // NT8: 8-row columns of queries
__global__ void __launch_bounds__(kFewThreads, 2) select_few_kernel(const PageSelectArgs a) {
  constexpr int P = D / 32;                   // 16-byte pieces of a row per lane (4 lanes a row)
  extern __shared__ uint32_t s_key[];         // [a.slice]
  __shared__ __align__(16) unsigned char s_q[8 * NT8][2 * D];   // whole numbers below zero, above zero
  __shared__ float s_unit[8 * NT8];
  __shared__ SelectShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, t = lane & 3;
  const int item = blockIdx.x / C, j = item / a.H_kv, g = item % a.H_kv;
  clear_shared<kFewThreads>(sh);
  grid_dep_wait();
  const Block k = find_block<kFewThreads>(a, j, sh.scan, sh.found);
  const int n = k.first - k.s0;               // candidates
  if (k.n == 0 || k.picked == n || k.picked == 0) {       // (the same for the whole cluster)
    if (rank == 0 && warp == 0) put_fixed(a, j, g, k);
    if (k.n > 0) pick_all<kFewThreads>(a, rank, C, j, g, k);
    return;
  }
  const int per = (n + C - 1) / C;
  const int p_first = k.s0 + min(n, rank * per), nl = min(k.first, p_first + per) - p_first;
  const int32_t *table = a.page_table + static_cast<size_t>(k.b) * a.max_pages + p_first;
  const int tasks = (nl + 15) / 16;
  // what put_fixed reads, on its way meanwhile
  if (rank == 0 && warp == kFewThreads / 32 - 1) {
    const int index = lane < k.s0 ? lane : k.first + lane - k.s0;
    if (index <= k.own1)
      asm volatile("prefetch.global.L1 [%0];\n" ::"l"(a.page_table + static_cast<size_t>(k.b) * a.max_pages + index));
  }
  // digests (and the exponent of the page that the lane writes the key of) of a task, requested ahead
  auto ids_of = [&](int task) -> int {
    const int i = task * 16 + (lane & 15), id = i < nl ? table[i] : -1;
    DSA_CHECK(i >= nl || (id >= 0 && id < a.n_pages));
    return id;
  };
  uint4 ra[P], rb[P];
  constexpr int kNone = 128;                  // (no exponent)
  int e_next = kNone;
  auto fetch = [&](int ids) {
    const int pa = __shfl_sync(kFull, ids, gr), pb = __shfl_sync(kFull, ids, gr + 8);
    const bool oka = pa >= 0 && pa < a.n_pages, okb = pb >= 0 && pb < a.n_pages;
    const size_t rowa = static_cast<size_t>(pa) * a.H_kv + g, rowb = static_cast<size_t>(pb) * a.H_kv + g;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      ra[i] = oka ? __ldg(reinterpret_cast<const uint4 *>(a.bounds + rowa * 2 * D) + i * 4 + t) : make_uint4(0, 0, 0, 0);
      rb[i] = okb ? __ldg(reinterpret_cast<const uint4 *>(a.bounds + rowb * 2 * D) + i * 4 + t) : make_uint4(0, 0, 0, 0);
    }
    e_next = t < 2 && (t ? okb : oka) ? a.exp[t ? rowb : rowa] : kNone;   // (looked at a task later)
  };
  const int ids0 = ids_of(warp);
  int ids = ids_of(warp + kFewThreads / 32);
  const int R = k.n * (a.H_q / a.H_kv);
  for (int r = warp; r < 8 * NT8; r += kFewThreads / 32) {   // (rows behind the last repeat the first)
    constexpr int E = D / 32;
    uint32_t w[E / 2];
    float x[E];
    load_row<D>(a, k, g, r < R ? r : 0, w);
    if (r == warp) fetch(ids0);               // behind the row's own load
    const int e = row_of<D>(w, x);
    const float inv = two_to(-e);
    uint32_t pos = 0, neg = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int v = whole(x[i] * inv);
      pos |= (static_cast<uint32_t>(max(v, 0)) & 0xffu) << (8 * i);
      neg |= (static_cast<uint32_t>(min(v, 0)) & 0xffu) << (8 * i);
    }
    if constexpr (E == 4) {
      reinterpret_cast<uint32_t *>(s_q[r])[lane] = neg;
      reinterpret_cast<uint32_t *>(s_q[r] + D)[lane] = pos;
    } else {
      reinterpret_cast<uint16_t *>(s_q[r])[lane] = static_cast<uint16_t>(neg);
      reinterpret_cast<uint16_t *>(s_q[r] + D)[lane] = static_cast<uint16_t>(pos);
    }
    if (lane == 0) s_unit[r] = two_to(e);
  }
  __syncthreads();
  uint32_t bq[NT8][P][8];                     // the queries' fragments: row gr of a column, the lane's bytes
  float u0[NT8], u1[NT8];
#pragma unroll
  for (int c = 0; c < NT8; ++c) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const uint4 v = *reinterpret_cast<const uint4 *>(s_q[8 * c + gr] + (i * 4 + t) * 16);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint2 h = widen_s8(w[x]);
        bq[c][i][2 * x] = h.x;
        bq[c][i][2 * x + 1] = h.y;
      }
    }
    u0[c] = s_unit[8 * c + 2 * t];
    u1[c] = s_unit[8 * c + 2 * t + 1];
  }
  for (int task = warp; task < tasks; task += kFewThreads / 32) {
    float acc[NT8][2][4];
#pragma unroll
    for (int c = 0; c < NT8; ++c)
#pragma unroll
      for (int x = 0; x < 8; ++x) acc[c][x >> 2][x & 3] = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const uint32_t wa[4] = {ra[i].x, ra[i].y, ra[i].z, ra[i].w}, wb[4] = {rb[i].x, rb[i].y, rb[i].z, rb[i].w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint2 va = widen_s8(wa[x]), vb = widen_s8(wb[x]);
        const uint32_t af[4] = {va.x, vb.x, va.y, vb.y};
#pragma unroll
        for (int c = 0; c < NT8; ++c) mma_16816_f16(acc[c][x & 1], af, bq[c][i][2 * x], bq[c][i][2 * x + 1]);
      }
    }
    const int e = e_next;
    const int next = ids;
    ids = ids_of(task + 2 * (kFewThreads / 32));
    fetch(next);                              // (all -1 behind the last task: nothing is read)
    float sa = -INFINITY, sb = -INFINITY;     // pages gr and gr + 8 over the lane's rows
#pragma unroll
    for (int c = 0; c < NT8; ++c) {
      float s[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) s[x] = acc[c][0][x] + acc[c][1][x];   // (whole numbers: exact)
      sa = fmaxf(sa, fmaxf(s[0] * u0[c], s[1] * u1[c]));
      sb = fmaxf(sb, fmaxf(s[2] * u0[c], s[3] * u1[c]));
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      sa = fmaxf(sa, __shfl_xor_sync(kFull, sa, o));
      sb = fmaxf(sb, __shfl_xor_sync(kFull, sb, o));
    }
    const int i = task * 16 + gr + 8 * t;
    if (t < 2 && i < nl) s_key[i] = e != kNone ? ordered_key((t ? sb : sa) * two_to_stored(e)) : 0u;   // no page: below every score
  }
  if (rank == 0 && warp == kFewThreads / 32 - 1) put_fixed(a, j, g, k);
  __syncthreads();
  pick<kFewThreads>(a, cluster, sh, s_key, nl, p_first, j, g, k);
}

// Many rows (a chunk's blocks): the products on tcgen05, the integers as fp16.  Pages lie on the
// TMEM lanes (M = 128) and the block's rows on its columns (N = 64 or 128; 256 rows as two products),
// so a thread owns a page and takes the largest score of its columns without talking to another.  The
// rows' integers stay in shared memory, those below zero against lo and those above against hi (K =
// 2 D).  Digests come in tiles of 128 pages by cp.async and go, widened to fp16, to TMEM as the A
// operand.  While one product's scores are read, the next is computed.  The same with mma.sync took 355 us
// for 2,048 tokens in blocks of 64 over 2,048 pages of 8 heads.
constexpr int kManyEpi = 8, kManyConv = 8;                       // warps: epilogue, converters, MMA issuer
constexpr int kManyThreads = (kManyEpi + kManyConv + 1) * 32;
constexpr int kTilePages = 128;

// The whole warp waits, at most `limit` clocks; the outcome is warp-uniform.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort, uint32_t limit) {
  if (__all_sync(kFull, mbar_test_wait(bar, parity))) return true;
  const uint32_t t0 = static_cast<uint32_t>(clock());
  do {
    if (__any_sync(kFull, *abort || static_cast<uint32_t>(clock()) - t0 > limit)) {
      *abort = 1;
      return false;
    }
  } while (!__all_sync(kFull, mbar_try_wait(bar, parity)));
  return true;
}

// Shared memory of a launch whose CTAs hold `rows` rows (a multiple of 64, at most 256) at a time.
struct ManyLayout {
  uint32_t oRaw, oUnit, oBar, oShared, oKey;
};
__host__ __device__ constexpr ManyLayout many_layout(int D, int rows) {
  ManyLayout m{};
  m.oRaw = static_cast<uint32_t>(rows) * 4 * D;                 // rows of 2 D fp16, in blocks of 64
  m.oUnit = m.oRaw + 2 * kTilePages * 2 * D;                    // two tiles of digests
  m.oBar = m.oUnit + rows * 4;
  m.oShared = m.oBar + 128;
  m.oKey = m.oShared + (sizeof(SelectShared) + 15) / 16 * 16;
  return m;
}

// 16 bytes to shared memory, zeros where there is nothing to read
__device__ __forceinline__ void cp_async_16_or_0(void *dst, const void *src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_addr(dst)), "l"(src), "r"(ok ? 16 : 0));
}

template <int D, int RN>                      // RN: rows held at a time, 64, 128 or 256
__global__ void __launch_bounds__(kManyThreads, 1) select_many_kernel(const PageSelectArgs a) {
  constexpr int KB = 2 * D / 64;              // 64-element blocks of K
  constexpr int A = D;                        // TMEM columns of a tile's digests (2 D fp16)
  constexpr int NH = RN > 128 ? 2 : 1, N = RN / NH;   // products per tile, rows of one: a tile's scores, or halves
  constexpr int PP = 2 * D / 16;              // 16-byte pieces of a digest row
  extern __shared__ __align__(1024) unsigned char sm[];
  constexpr ManyLayout L = many_layout(D, RN);
  SelectShared &sh = *reinterpret_cast<SelectShared *>(sm + L.oShared);
  float *s_unit = reinterpret_cast<float *>(sm + L.oUnit);
  uint64_t *a_full = reinterpret_cast<uint64_t *>(sm + L.oBar), *a_empty = a_full + 2, *d_full = a_empty + 2,
           *d_empty = d_full + 2, *drained = d_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drained + 1);
  volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
  uint32_t *s_key = reinterpret_cast<uint32_t *>(sm + L.oKey);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int item = blockIdx.x / C, j = item / a.H_kv, g = item % a.H_kv;
  clear_shared<kManyThreads>(sh);
  grid_dep_wait();
  const Block k = find_block<kManyThreads>(a, j, sh.scan, sh.found);
  const int n = k.first - k.s0;
  if (k.n == 0 || k.picked == n || k.picked == 0) {
    if (rank == 0 && warp == 0) put_fixed(a, j, g, k);
    if (k.n > 0) pick_all<kManyThreads>(a, rank, C, j, g, k);
    return;
  }
  const int per = (n + C - 1) / C;
  const int p_first = k.s0 + min(n, rank * per), nl = min(k.first, p_first + per) - p_first;
  for (int i = tid; i < nl; i += kManyThreads) s_key[i] = 0;
  const int R = k.n * (a.H_q / a.H_kv);
  const int32_t *table = a.page_table + static_cast<size_t>(k.b) * a.max_pages + p_first;
  const int tiles = (nl + kTilePages - 1) / kTilePages;
  constexpr uint32_t cols = 2 * N + 2 * A <= 256 ? 256u : 512u;   // TMEM: scores of two products, two tiles
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&a_full[s], kManyConv);
      mbar_init(&a_empty[s], 1);
      mbar_init(&d_full[s], 1);
      mbar_init(&d_empty[s], kManyEpi / 2);
    }
    mbar_init(drained, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == kManyEpi + kManyConv) {
    tmem_alloc(tmem_slot, cols);
    tmem_relinquish();
  }
  // what a role carries over from one set of rows to the next
  Ring<2> buf;                                // the digests' buffer
  uint32_t unit = 0;                          // products so far: they take the scores' buffers in turn
  bool ok = true;

  for (int r0 = 0; r0 < R; r0 += RN) {
    __syncthreads();                          // the rows before are read (and the barriers are there)
    const int rows = min(RN, R - r0);
    const int rn = RN;                        // columns (those behind the last row repeat it)
    // D / 8 lanes hold 8 elements of a row each; a warp asks for U steps of its rows at once
    constexpr int LPR = D / 8, RPW = 32 / LPR, U = 8, W = kManyThreads / 32 * RPW;
    const int G = a.H_q / a.H_kv, piece = lane % LPR;
    for (int r1 = warp * RPW + lane / LPR; r1 - lane / LPR < rn; r1 += U * W) {
      uint4 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + min(r1 + u * W, rows - 1);
        w[u] = __ldg(reinterpret_cast<const uint4 *>(a.q + static_cast<size_t>(k.lo + r / G) * a.q_stride +
                                                     static_cast<size_t>(g * G + r % G) * D) + piece);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r1 + u * W;
        if (r - lane / LPR >= rn) break;      // (the whole warp)
        const uint32_t x[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        constexpr uint32_t kAbs = 0x7fff7fffu;
        uint32_t m2 = __vmaxu2(__vmaxu2(x[0] & kAbs, x[1] & kAbs), __vmaxu2(x[2] & kAbs, x[3] & kAbs));
        uint32_t m = max(m2 & 0xffffu, m2 >> 16);
        const bool odd = __any_sync(kFull, m >= 0x7f80u);   // infinities or NaN among them: rare
        if (odd) {
          m = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t v = (x[i >> 1] >> (16 * (i & 1))) & 0x7fffu;
            m = max(m, v < 0x7f80u ? v : 0u);
          }
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
        const int e = exponent127(m << 16);
        const float inv = two_to(-e);
        uint32_t neg[4], pos[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // nearest whole number, ties to even: the sum's last place is 1 (conversions to integers and
          // back have a quarter of the rate)
          constexpr float kMagic = 12582912.f;
          float v = fmaf(bf16_lo(x[i]), inv, kMagic) - kMagic, y = fmaf(bf16_hi(x[i]), inv, kMagic) - kMagic;
          if (odd) {
            v = v == v ? v : 0.f;
            y = y == y ? y : 0.f;
          }
          neg[i] = pack_f16x2(fmaxf(fminf(v, 0.f), -127.f), fmaxf(fminf(y, 0.f), -127.f));
          pos[i] = pack_f16x2(fminf(fmaxf(v, 0.f), 127.f), fminf(fmaxf(y, 0.f), 127.f));
        }
        // 128-byte rows of 64 elements, 16-byte pieces swizzled by the row; blocks of K RN rows apart
        if (r < rn) {
          unsigned char *dst = sm + (piece >> 3) * RN * 128 + r * 128 + (((piece & 7) ^ (r & 7)) << 4);
          *reinterpret_cast<uint4 *>(dst) = make_uint4(neg[0], neg[1], neg[2], neg[3]);
          *reinterpret_cast<uint4 *>(dst + (KB / 2) * RN * 128) = make_uint4(pos[0], pos[1], pos[2], pos[3]);
          if (piece == 0) s_unit[r] = two_to(e);
        }
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);   // this warp's TMEM lanes

    if (warp < kManyEpi) {
      // ---- epilogue: page (lane) x columns; four warps read one buffer's scores while the others read the
      // other's
      const uint32_t mine = warp >> 2;
      const int row = (warp & 3) * 32 + lane;
      // this thread's page two tiles ahead and its exponent one ahead (looked at when used, so that
      // neither load is waited for)
      auto page_of = [&](int tile) -> int {
        const int i = tile * kTilePages + row, page = i < nl ? table[i] : -1;
        DSA_CHECK(i >= nl || (page >= 0 && page < a.n_pages));
        return page;
      };
      constexpr int kNone = 128;               // (no exponent)
      auto exp_of = [&](int page) -> int {
        return page >= 0 && page < a.n_pages ? a.exp[static_cast<size_t>(page) * a.H_kv + g] : kNone;
      };
      const int page0 = page_of(0);
      int page_next = page_of(1), e_next = exp_of(page0);
      for (int tile = 0; ok && tile < tiles; ++tile) {
        const int e = e_next;
        e_next = exp_of(page_next);
        page_next = page_of(tile + 2);
#pragma unroll 1
        for (int h = 0; h < NH; ++h, ++unit) {
          if ((unit & 1u) != mine) continue;
          if (!(ok = warp_wait(&d_full[mine], (unit >> 1) & 1u, abort, a.wait_clocks))) break;
          tc_fence_after();
          const float4 *u4 = reinterpret_cast<const float4 *>(s_unit + h * N);
          float b0 = -INFINITY, b1 = -INFINITY;
          for (int c = 0; c < N; c += 32) {
            uint32_t s[32];
            tmem_ld32(t_lane + mine * N + c, s);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              const float4 u = u4[(c + x) / 4];
              const float2 y = fmul2(make_float2(__uint_as_float(s[x]), __uint_as_float(s[x + 1])), make_float2(u.x, u.y));
              const float2 z = fmul2(make_float2(__uint_as_float(s[x + 2]), __uint_as_float(s[x + 3])), make_float2(u.z, u.w));
              b0 = fmax3(b0, y.x, y.y);
              b1 = fmax3(b1, z.x, z.y);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&d_empty[mine]);
          if (e != kNone) atomicMax(&s_key[tile * kTilePages + row], ordered_key(fmaxf(b0, b1) * two_to_stored(e)));
        }
      }
    } else if (warp == kManyEpi + kManyConv) {
      // ---- MMA issuer
      // (an instruction takes 71 clocks to issue whatever its N, so a product has as many rows as may be;
      // the operands are what the compiler can tell to be the same for the whole warp, see tc_ptx.cuh)
      const uint32_t leader = lane == 0 ? 1u : 0u;
      constexpr uint32_t id = idesc_f16_f32(kTilePages, N);
      const uint32_t tm = __shfl_sync(kFull, tmem, 0);
      const uint64_t db = sdesc_sw128(smem_u32(sm), 16, 1024);
#pragma unroll 1
      for (int tile = 0; ok && tile < tiles; ++tile, buf.step()) {
        const int slot = __shfl_sync(kFull, buf.slot, 0);
        if (!(ok = warp_wait(&a_full[slot], buf.phase, abort, a.wait_clocks))) break;
        const uint32_t at = tm + 2 * N + slot * A;
#pragma unroll
        for (int h = 0; h < NH; ++h, ++unit) {
          const uint32_t to = __shfl_sync(kFull, unit & 1u, 0);
          if (!ok || !(ok = warp_wait(&d_empty[to], ((unit >> 1) & 1u) ^ 1u, abort, a.wait_clocks))) break;
          tc_fence_after();
#pragma unroll
          for (int s = 0; s < 4 * KB; ++s)    // 16 elements of K: 8 columns of A, 32 bytes of B's rows
            mma_ts(leader, tm + to * N, at + 8 * s, db + ((s >> 2) * RN + h * N) * 8 + 2 * (s & 3), id, s > 0 ? 1u : 0u);
          commit_if(leader, &d_full[to]);
        }
        if (ok) commit_if(leader, &a_empty[slot]);
      }
    } else {
      // ---- converters: 16-byte pieces of the digests into a raw tile (PP threads a row), then a thread
      // per page and half of its row widens them
      const int ct = tid - kManyEpi * 32, piece = ct % PP, half = ct >> 7, row = ct & 127;
      constexpr int RPP = kManyConv * 32 / PP, NP = kTilePages / RPP;   // rows per pass, passes
      int ids[NP];
      auto ids_of = [&](int tile) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int x = tile * kTilePages + ct / PP + i * RPP;
          ids[i] = x < nl ? table[x] : -1;
        }
      };
      auto fetch = [&](int tile) {            // the tile of `ids`
        unsigned char *raw = sm + L.oRaw + (tile & 1) * kTilePages * 2 * D;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int r = ct / PP + i * RPP;
          const bool good = ids[i] >= 0 && ids[i] < a.n_pages;
          cp_async_16_or_0(raw + r * 2 * D + ((piece ^ (r & (PP - 1))) << 4),
                           a.bounds + (static_cast<size_t>(good ? ids[i] : 0) * a.H_kv + g) * 2 * D + piece * 16, good);
        }
      };
      // two tiles in flight, the third's pages known (a group of copies is closed for every tile, so
      // that they can be counted)
      for (int tile = 0; tile < 2; ++tile) {
        ids_of(tile);
        if (tile < tiles) fetch(tile);
        cp_async_commit();
      }
      ids_of(2);
      for (int tile = 0; tile < tiles; ++tile, buf.step()) {
        cp_async_wait<1>();
        named_bar_sync(1, kManyConv * 32);    // the tile is there for all (every converter comes here, ok or not)
        if (ok) ok = warp_wait(&a_empty[buf.slot], buf.phase ^ 1u, abort, a.wait_clocks);
        if (ok) {
          tc_fence_after();
          const unsigned char *raw = sm + L.oRaw + (tile & 1) * kTilePages * 2 * D + row * 2 * D;
          // half a row: PP / 2 pieces, 8 columns each
#pragma unroll
          for (int p = 0; p < PP / 2; p += 2) {
            uint32_t h[16];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint4 v = *reinterpret_cast<const uint4 *>(raw + (((half * (PP / 2) + p + q) ^ (row & (PP - 1))) << 4));
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint2 y = widen_s8(w[x]);
                h[8 * q + 2 * x] = y.x;
                h[8 * q + 2 * x + 1] = y.y;
              }
            }
            tmem_st16(t_lane + 2 * N + buf.slot * A + half * (A / 2) + 8 * p, h);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&a_full[buf.slot]);
        }
        named_bar_sync(1, kManyConv * 32);    // the raw tile is read
        if (tile + 2 < tiles) fetch(tile + 2);
        cp_async_commit();
        ids_of(tile + 3);
      }
      cp_async_wait<0>();
      // (while the last scores are computed and read)
      if (rank == 0 && warp == kManyEpi && r0 + RN >= R) put_fixed(a, j, g, k);
    }
    ok = __syncthreads_and(ok);               // (also: every score of these rows is in)
    if (!ok) break;
  }
  if (warp == kManyEpi + kManyConv) {
    // the tensor core is idle before its memory goes, also where a wait ran out
    commit_if(lane == 0, drained);
    const uint64_t t0 = global_ns();
    while (!__all_sync(kFull, mbar_try_wait(drained, 0)))
      if (__any_sync(kFull, global_ns() - t0 > 200000000ull)) break;
    tmem_dealloc(*tmem_slot, cols);
    if (lane == 0 && !ok) atomicOr(&g_select_error, 1);
  }
  if (rank == 0 && warp == 0 && !ok) put_fixed(a, j, g, k);
  __syncthreads();
  pick<kManyThreads>(a, cluster, sh, s_key, nl, p_first, j, g, k);
}

// dynamic shared memory of a launch, at most
constexpr size_t kFewBytes = kSelectMaxPages / 16 * 4, kManyBytes = 227 * 1024;
static_assert(many_layout(128, 128).oKey + kSelectMaxPages / 16 * 4 <= kManyBytes, "widest table");

// What a launch needs of the current device: the kernel's shared memory and clusters allowed there.  Set
// once per device, and to the most that any call asks for: the limit belongs to the kernel, not to the call,
// and one that each call set to its own size refused the wider call of another host thread.
template <auto kKernel>
cudaError_t prepare(size_t most, bool again = false) {
  static std::atomic<bool> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool keep = dev >= 0 && dev < 64;
  if (keep && !again && known[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && keep) known[dev].store(true, std::memory_order_release);
  return e;
}

template <auto kKernel>
cudaError_t launch_cluster(int items, int C, int threads, size_t smem, size_t most, cudaStream_t s,
                           const PageSelectArgs &a) {
  cudaError_t e = prepare<kKernel>(most);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items) * C);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  for (int turn = 0; turn < 2; ++turn) {
    ProfScope ps("page_select", s);
    e = cudaLaunchKernelEx(&cfg, kKernel, a);
    if ((e != cudaErrorInvalidValue && e != cudaErrorInvalidClusterSize) || turn) break;
    // a context that was torn down and made again has forgotten what was allowed
    cudaGetLastError();
    if ((e = prepare<kKernel>(most, true)) != cudaSuccess) break;
  }
  return e;
}

template <int D>
cudaError_t launch_select_d(PageSelectArgs a, cudaStream_t s) {
  const int items = a.n_blocks * a.H_kv, rows = a.cfg.q_block * (a.H_q / a.H_kv);
  const bool few = rows <= kFewRows;
  // CTAs of an item, while the launch does not fill the GPU with them.  Few rows: 16 tokens of 8 heads
  // over 512 pages take 10.3 us with one, 11.7 with two, 19.9 with four; over 2,048 pages 27.5, 22.1,
  // 30.0; a token over 16,384 47.0, 29.2 and 25.0 us with 4, 8 and 16.  Many rows: a block of 64
  // tokens of 8 heads over 2,048 pages 24.0, 21.2 and 40.4 us with 4, 8 and 16 (16 CTAs of a whole SM
  // find no room in a cluster's SMs at once).  The table's width stands for the sequences', which the host
  // does not know: 16 tokens over 512 pages take 12.3 us in a table of 2,048 or 16,384, one token over 64
  // pages 13.0 in place of 6.9.
  const int most = few ? 16 : 8;
  int C = 1;
  while (C < most && a.max_pages > C * kTilePages && items * C * (a.max_pages > C * 1024 && few ? 1 : 2) <= 152) C *= 2;
  a.slice = (a.max_pages + C - 1) / C;
  while (C < 16 && a.slice > kSelectMaxPages / 16) {
    C *= 2;
    a.slice = (a.max_pages + C - 1) / C;
  }
  const size_t keys = static_cast<size_t>(a.slice) * 4;
  // (16 rows by tcgen05 instead: 2,048 tokens in blocks of 4 over 2,048 pages 707 us in place of 394)
  if (rows <= 8) return launch_cluster<select_few_kernel<D, 1>>(items, C, kFewThreads, keys, kFewBytes, s, a);
  if (few) return launch_cluster<select_few_kernel<D, 2>>(items, C, kFewThreads, keys, kFewBytes, s, a);
  // about two clocks a nanosecond; at most 2^31 of them, a second
  a.wait_clocks = static_cast<uint32_t>(std::min(2ull * g_wait_limit_ns, 0x7fffffffull));
  // rows held at a time: as many as a block has, 128 where the keys of a wide table need the room
  const size_t smem = many_layout(D, rows <= 64 ? 64 : 128).oKey + keys, smem256 = many_layout(D, 256).oKey + keys;
  if (rows <= 64) return launch_cluster<select_many_kernel<D, 64>>(items, C, kManyThreads, smem, kManyBytes, s, a);
  if (rows <= 128 || smem256 > kManyBytes)
    return launch_cluster<select_many_kernel<D, 128>>(items, C, kManyThreads, smem, kManyBytes, s, a);
  return launch_cluster<select_many_kernel<D, 256>>(items, C, kManyThreads, smem256, kManyBytes, s, a);
}

}  // namespace

cudaError_t launch_page_digest(const DigestArgs &a0, cudaStream_t s) {
  DigestArgs a = a0;
  while ((1 << a.lg_page) < a.page_size) ++a.lg_page;
  // token rows per CTA: an equal share of a launch that fills the GPU's 152 SMs once with four CTAs each
  const int heads = (a.H_kv + kDigestHeads - 1) / kDigestHeads;
  const int ctas = std::max(1, 4 * 152 / heads);
  a.window = std::min(std::max((a.n_tok + ctas - 1) / ctas, 1), kMaxWindow);
  const dim3 grid((a.n_tok + a.window - 1) / a.window, heads);
  ProfScope ps("page_digest", s);
  if (a.fp8)
    return a.D == 128 ? launch_pdl(digest_kernel<128, true>, grid, dim3(kDigestThreads), 0, s, a)
                      : launch_pdl(digest_kernel<64, true>, grid, dim3(kDigestThreads), 0, s, a);
  return a.D == 128 ? launch_pdl(digest_kernel<128, false>, grid, dim3(kDigestThreads), 0, s, a)
                    : launch_pdl(digest_kernel<64, false>, grid, dim3(kDigestThreads), 0, s, a);
}

cudaError_t launch_page_select(const PageSelectArgs &a0, cudaStream_t s) {
  PageSelectArgs a = a0;
  while ((1 << a.lg_page) < a.page_size) ++a.lg_page;
  return a.D == 128 ? launch_select_d<128>(a, s) : launch_select_d<64>(a, s);
}

int page_select_device_error() {
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_select_error, sizeof(int)) != cudaSuccess) return -1;
  if (cudaMemcpyToSymbol(g_select_error, &zero, sizeof(int)) != cudaSuccess) return -1;
  return v;
}

void page_select_set_wait_limit(unsigned long long ns) { g_wait_limit_ns = std::min(ns, 1ull << 40); }

}  // namespace dsa
