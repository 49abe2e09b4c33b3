// The paged key/value cache: writing a chunk of new tokens, reading rows back.
//
// Mathematics (FP8 cache): a token's row x[0..D) of one head is held as E4M3 codes c and one
// scale byte s with e = s - 127, the value of element i being c_i * 2^e.  With a = max |x_i|
// over the finite elements, e is the smallest integer with a * 2^-e <= 448 (the largest E4M3
// value), kept in [-116, 119]; a row of zeros takes e = 0.  A power of two scales without
// rounding, so the only rounding is x * 2^-e to E4M3 (nearest, ties to even, saturating), and
// the value read back is exactly a bf16: E4M3 has four significant bits and 2^(e-9) >= 2^-125,
// 448 * 2^119 < 2^127 stay inside bf16's normal range.  A floating-point code keeps the same
// relative precision under any power of two, so a finer scale would gain nothing but the
// top of the range.  A row that holds a NaN takes the scale byte 255 (E8M0's NaN) and reads
// back as NaN throughout.
//
// Both kernels are bound by HBM: a row is read once and written once.  Measured (of 6,773 GB/s):
// writing 48,549 tokens of 8 heads of 128 to an FP8 cache (299 MB) 50 to 52 us, 5,800 GB/s (85 %);
// 10,764 tokens of 16 heads of 64 in bf16 (88 MB) 18 us; reading 131,072 tokens of 8 heads of 128
// back from FP8 (807 MB) 120 to 122 us, 6,600 GB/s (98 %); a decode step's few rows take a launch,
// 2.4 us.
#include "common.cuh"
#include "launch.h"
#include "mma_sync.cuh"
#include "profile.h"

namespace dsa {

DSA_CHECK_WORD(kv_cache_check_word)

namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ write

// two fp32 -> two E4M3 codes (lo in the low byte), nearest even, saturating; NaN stays NaN
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Scale exponent of a row whose largest finite magnitude has the bf16 bits `u` (sign clear):
// a = 1.m * 2^x takes e = x - 8 while 1.m <= 1.75 (448 = 1.75 * 2^8), else x - 7.
__device__ __forceinline__ int row_exponent(uint32_t u) {
  if (u == 0u) return 0;
  const int e = static_cast<int>(u >> 7) - 135 + ((u & 0x7fu) > 0x60u ? 1 : 0);
  return min(max(e, -116), 119);
}

// two bf16 -> two E4M3 codes of x * inv (inv a power of two in both halves: exact)
__device__ __forceinline__ uint32_t quantise2(uint32_t w, float2 inv) {
  float2 x;
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 c, a, b;\n"
      " mov.b64 {%0, %1}, c;\n}\n"
      : "=f"(x.x), "=f"(x.y)
      : "f"(bf16_lo(w)), "f"(bf16_hi(w)), "f"(inv.x), "f"(inv.y));
  return f32x2_to_e4m3x2(x.x, x.y);
}

// 8 bf16 of one 16-byte piece -> 8 codes of x * inv
__device__ __forceinline__ uint2 quantise8(const uint4 &u, float2 inv) {
  return make_uint2(quantise2(u.x, inv) | (quantise2(u.y, inv) << 16), quantise2(u.z, inv) | (quantise2(u.w, inv) << 16));
}

// largest magnitude (bf16 bits) of either half over two 16-byte pieces
__device__ __forceinline__ uint32_t max2x8(const uint4 &u, const uint4 &v) {
  constexpr uint32_t k = 0x7fff7fffu;
  return __vmaxu2(__vmaxu2(__vmaxu2(u.x & k, u.y & k), __vmaxu2(u.z & k, u.w & k)),
                  __vmaxu2(__vmaxu2(v.x & k, v.y & k), __vmaxu2(v.z & k, v.w & k)));
}

// the same over finite elements alone, one result; 0xffff if the pieces hold a NaN
__device__ __forceinline__ uint32_t finite_max(const uint4 &u, const uint4 &v) {
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll 1
  for (int i = 0; i < 16; ++i) {
    const uint32_t x = (w[i >> 1] >> (16 * (i & 1))) & 0x7fffu;
    m = max(m, x < 0x7f80u ? x : x == 0x7f80u ? 0u : 0xffffu);
  }
  return m;
}

// One CTA writes `tpc` tokens.  First every sequence whose rows meet the CTA's tokens marks
// them, then a thread per token looks up its slot (page * page_size + offset; -1: not written):
// one round of loads for all sequences and one for the tokens, whatever B is.  Then rows (token, K or
// V, head) go out D / 16 lanes each, a lane holding the 16-byte pieces l and l + D / 16 of
// the row, so that every load covers whole row segments and every store whole sectors.
template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const CacheWriteArgs a) {
  constexpr int LPR = D / 16;                 // lanes per row
  constexpr int RPP = kThreads / LPR;         // rows per pass of the CTA
  extern __shared__ long long s_slot[];       // [tpc]
  const int tid = threadIdx.x;
  const int n0 = blockIdx.x * a.tpc, n1 = min(a.n_tok, n0 + a.tpc);
  grid_dep_wait();
  for (int i = tid; i < a.tpc; i += kThreads) s_slot[i] = -1;
  __syncthreads();
  for (int b = tid; b < a.B; b += kThreads) {
    const int qs = a.q_start[b], qe = a.q_start[b + 1];
    DSA_CHECK(qs >= 0 && qe <= a.n_tok);
    for (int n = max(qs, n0); n < min(qe, n1); ++n) s_slot[n - n0] = b;
  }
  __syncthreads();
  if (tid < n1 - n0 && s_slot[tid] >= 0) {
    const int b = static_cast<int>(s_slot[tid]);
    const int qe = a.q_start[b + 1], kv = a.kv_len[b], cap = a.max_pages << a.lg_page;
    DSA_CHECK(kv >= 0 && kv <= cap);
    const long long pos = min(max(kv, 0), cap) - (static_cast<long long>(qe) - (n0 + tid));
    DSA_CHECK(pos >= 0);
    long long slot = -1;
    if (pos >= 0) {
      const int page = a.page_table[static_cast<size_t>(b) * a.max_pages + (pos >> a.lg_page)];
      DSA_CHECK(page >= 0 && page < a.n_pages);
      if (page >= 0 && page < a.n_pages)
        slot = (static_cast<long long>(page) << a.lg_page) + (pos & (a.page_size - 1));
    }
    s_slot[tid] = slot;
  }
  __syncthreads();
  const int l = tid % LPR;
  const int per_tok = 2 * a.H_kv;             // rows of a token: K heads, then V heads
  const int rows = (n1 - n0) * per_tok;
  // this thread's row of the pass: row x of token n0 + i
  int i = (tid / LPR) / per_tok, x = (tid / LPR) % per_tok;
#pragma unroll 2
  for (int base = 0; base < rows; base += RPP) {   // uniform trip count
    const bool is_k = x < a.H_kv;
    const int h = is_k ? x : x - a.H_kv;
    const long long slot = i < n1 - n0 ? s_slot[i] : -1;
    uint4 u0 = make_uint4(0, 0, 0, 0), u1 = u0;
    if (slot >= 0) {
      const uint4 *src = reinterpret_cast<const uint4 *>(
          (is_k ? a.k_new + (n0 + i) * a.k_stride : a.v_new + (n0 + i) * a.v_stride) + static_cast<size_t>(h) * D);
      u0 = __ldg(src + l);
      u1 = __ldg(src + l + LPR);
    }
    const size_t row = static_cast<size_t>(slot) * a.H_kv + h;
    if constexpr (FP8) {
      uint32_t m2 = max2x8(u0, u1);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(kFull, m2, o));
      uint32_t m = max(m2 & 0xffffu, m2 >> 16);
      if (__any_sync(kFull, m >= 0x7f80u)) {         // infinities or NaN in some row: rare
        m = finite_max(u0, u1);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
      }
      if (slot >= 0) {
        const bool nan = m == 0xffffu;
        const int e = nan ? 0 : row_exponent(m);
        const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        const float2 inv = make_float2(f, f);
        uint2 *dst = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(is_k ? a.k_pages : a.v_pages) + row * D);
        dst[l] = quantise8(u0, inv);
        dst[l + LPR] = quantise8(u1, inv);
        if (l == 0) (is_k ? a.k_scale : a.v_scale)[row] = static_cast<uint8_t>(nan ? 255 : e + 127);
      }
    } else if (slot >= 0) {
      uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(is_k ? a.k_pages : a.v_pages) + row * D);
      dst[l] = u0;
      dst[l + LPR] = u1;
    }
    i += RPP / per_tok;
    x += RPP % per_tok;
    if (x >= per_tok) {
      x -= per_tok;
      ++i;
    }
  }
}

// ------------------------------------------------------------------ read

constexpr int kReadTok = 16;   // tokens per CTA: the smallest page, so a CTA stays inside one

// A page's rows are contiguous, and so are the output's: a CTA copies (bf16) or widens (FP8)
// 16 tokens of one sequence, 8 elements (one 16-byte store) per thread and step, four steps'
// loads in flight.
template <bool FP8>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const CacheReadArgs a) {
  const int b = blockIdx.y;
  const bool is_k = blockIdx.z == 0;
  const long long t0 = static_cast<long long>(blockIdx.x) * kReadTok;
  grid_dep_wait();
  const int kv = a.kv_len[b];
  const long long held = static_cast<long long>(a.max_pages) * a.page_size;
  DSA_CHECK(kv >= 0 && kv <= held);
  const long long cap = min(held, static_cast<long long>(a.T_max));
  const long long end = min(max(static_cast<long long>(kv), 0ll), cap);
  if (t0 >= end) return;
  const int page = a.page_table[static_cast<size_t>(b) * a.max_pages + t0 / a.page_size];
  DSA_CHECK(page >= 0 && page < a.n_pages);
  if (page < 0 || page >= a.n_pages) return;
  const int nt = static_cast<int>(min(end - t0, static_cast<long long>(kReadTok)));
  const size_t row0 = (static_cast<size_t>(page) * a.page_size + t0 % a.page_size) * a.H_kv;
  const int pieces = nt * a.H_kv * (a.D / 8);          // 8 elements each
  uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(is_k ? a.k_out : a.v_out) +
                                         (static_cast<size_t>(b) * a.T_max + t0) * a.H_kv * a.D);
  const void *pages = is_k ? a.k_pages : a.v_pages;
  constexpr int U = 4;
  if constexpr (FP8) {
    const uint2 *src = reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(pages) + row0 * a.D);
    const uint8_t *sc = (is_k ? a.k_scale : a.v_scale) + row0;
    const int lg = a.D == 128 ? 4 : 3;                 // log2 of the pieces of a row
    for (int i0 = threadIdx.x; i0 < pieces; i0 += kThreads * U) {
      uint2 w[U];
      uint32_t s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kThreads;
        if (i < pieces) {
          w[u] = __ldcs(src + i);
          s[u] = __ldg(sc + (i >> lg));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kThreads;
        if (i < pieces) {
          // 2^(s - 127), for s = 0 a subnormal of fp32; NaN for s = 255
          const float f = __uint_as_float(s[u] == 255u ? 0x7fffffffu : s[u] == 0u ? 0x00400000u : s[u] << 23);
          float x[8];
          f16x2_to_f32x2(e4m3x2_to_f16x2(w[u].x), x[0], x[1]);
          f16x2_to_f32x2(e4m3x2_to_f16x2(w[u].x >> 16), x[2], x[3]);
          f16x2_to_f32x2(e4m3x2_to_f16x2(w[u].y), x[4], x[5]);
          f16x2_to_f32x2(e4m3x2_to_f16x2(w[u].y >> 16), x[6], x[7]);
          uint4 o;
          o.x = pack_bf16x2(x[0] * f, x[1] * f);
          o.y = pack_bf16x2(x[2] * f, x[3] * f);
          o.z = pack_bf16x2(x[4] * f, x[5] * f);
          o.w = pack_bf16x2(x[6] * f, x[7] * f);
          __stcs(dst + i, o);
        }
      }
    }
  } else {
    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(pages) + row0 * a.D);
    for (int i0 = threadIdx.x; i0 < pieces; i0 += kThreads * U) {
      uint4 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kThreads;
        if (i < pieces) w[u] = __ldcs(src + i);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kThreads;
        if (i < pieces) __stcs(dst + i, w[u]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv_write(const CacheWriteArgs &a0, cudaStream_t s) {
  CacheWriteArgs a = a0;
  // tokens per CTA: enough rows for one pass of the CTA's lanes, up to 16 tokens once the
  // launch still fills the GPU twice over
  const int rpp = kThreads / (a.D / 16);
  int tpc = (rpp + 2 * a.H_kv - 1) / (2 * a.H_kv);
  while (tpc < 16 && a.n_tok / (2 * tpc) >= 4 * 152) tpc *= 2;
  a.tpc = tpc;
  while ((1 << a.lg_page) < a.page_size) ++a.lg_page;
  const dim3 grid((a.n_tok + tpc - 1) / tpc);
  const size_t smem = static_cast<size_t>(tpc) * sizeof(long long);
  ProfScope ps("kv_cache_write", s);
  if (a.fp8)
    return a.D == 128 ? launch_pdl(kv_write_kernel<128, true>, grid, dim3(kThreads), smem, s, a)
                      : launch_pdl(kv_write_kernel<64, true>, grid, dim3(kThreads), smem, s, a);
  return a.D == 128 ? launch_pdl(kv_write_kernel<128, false>, grid, dim3(kThreads), smem, s, a)
                    : launch_pdl(kv_write_kernel<64, false>, grid, dim3(kThreads), smem, s, a);
}

cudaError_t launch_kv_read(const CacheReadArgs &a, cudaStream_t s) {
  const dim3 grid((a.T_max + kReadTok - 1) / kReadTok, a.B, 2);
  ProfScope ps("kv_cache_read", s);
  return a.fp8 ? launch_pdl(kv_read_kernel<true>, grid, dim3(kThreads), 0, s, a)
               : launch_pdl(kv_read_kernel<false>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace dsa
