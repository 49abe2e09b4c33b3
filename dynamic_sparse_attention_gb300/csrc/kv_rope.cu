// kv_cache_write_rope: head norms and rotation on the way into the paged cache.
//
// Mathematics: a head's row x [D] becomes y = x * rsqrt(mean(x^2) + eps) * w, and each pair of
// its first `rot` dimensions is turned by p * inv_freq[i] for the token's position p.  A turn's
// fraction is what cosine and sine see, so inv_freq / 2 pi is held as a 64-bit fraction of a turn
// and multiplied by p modulo 2^64: the top 32 bits are the angle.  It is off by p * inv_freq * 2^-52
// radians (the two roundings of inv_freq / 2 pi) and 2^-23 (the 32 bits, and their fp32) at most: 2^-21
// at position 2^30 of the fastest pair.  Rows are fp32 from load
// to store and rounded once: to bf16, or for an FP8 cache by the rule of kv_cache.cu applied to
// the fp32 values (values are bf16 already, so they come out as kv_cache_write stores them).
//
// Bound by HBM: every row is read once and written once.  Measured (of 6,791 GB/s): 34,700 tokens of 32
// query and 8 key heads of 128, bf16 (1,193 MB), 196 us, 6,070 GB/s (89 %), into an FP8 cache (1,095 MB) 207
// us, 5,280 GB/s (78 %); a decode step's 16 tokens 4.9 us, a launch's latencies.
#include "common.cuh"
#include "launch.h"
#include "mma_sync.cuh"
#include "profile.h"

namespace dsa {

DSA_CHECK_WORD(kv_rope_check_word)

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTok = 16;   // tokens per CTA at most

__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Scale exponent of a row whose largest finite magnitude has the fp32 bits `u`: a = 1.m * 2^x takes
// x - 8 while 1.m <= 1.75 (448 = 1.75 * 2^8), else x - 7.
__device__ __forceinline__ int row_exponent(uint32_t u) {
  if (u == 0u) return 0;
  const int e = static_cast<int>(u >> 23) - 135 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, -116), 119);
}

__device__ __forceinline__ uint2 quantise8(const float *y, float inv) {
  return make_uint2(f32x2_to_e4m3x2(y[0] * inv, y[1] * inv) | (f32x2_to_e4m3x2(y[2] * inv, y[3] * inv) << 16),
                    f32x2_to_e4m3x2(y[4] * inv, y[5] * inv) | (f32x2_to_e4m3x2(y[6] * inv, y[7] * inv) << 16));
}

__device__ __forceinline__ uint4 pack8(const float *y) {
  return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                    pack_bf16x2(y[6], y[7]));
}

// One CTA takes `tpc` tokens, `wpt` warps to a token.  A row is held by D / 16 lanes, two 16-byte
// pieces each, dealt out so that both halves of every rotated pair are in one lane: lane l has
// pieces l and l + rot / 16 of the rotated ones (pairs (i, i + rot / 2) are as far apart; pairs
// (2 i, 2 i + 1) lie inside a piece), the lanes behind those two neighbours of the rest.  A lane
// then turns 8 pairs by the same 8 angles in every row of the token.
template <int D, bool FP8, bool INTER>
__global__ void __launch_bounds__(kThreads, 3) kv_rope_kernel(const RopeWriteArgs a) {
  constexpr int LPR = D / 16;                 // lanes per row
  constexpr int RPW = 32 / LPR;               // rows per warp at a time
  constexpr int APL = 8 / RPW;                // angles that a lane computes (its row group's share of 8)
  __shared__ long long s_slot[kMaxTok];       // page * page_size + offset; -1: no page; -2: no chunk
  __shared__ int s_pos[kMaxTok];
  __shared__ unsigned long long s_freq[D / 2];
  __shared__ __align__(16) float s_w[2][D];
  __shared__ __align__(16) float s_turn[kWarps][2][LPR][8];   // cosine, sine of the warp's token
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n0 = blockIdx.x * a.tpc, n1 = min(a.n_tok, n0 + a.tpc);
  grid_dep_wait();
  if (tid < kMaxTok) s_slot[tid] = -2;
  if (tid < a.cfg.rot / 2) {
    double t = a.cfg.inv_freq[tid] * 0.15915494309189533577;   // 1 / 2 pi
    t -= floor(t);
    s_freq[tid] = __double2ull_rz(t * 18446744073709551616.0);
  }
  for (int i = tid; i < 2 * D; i += kThreads) {
    const void *w = i < D ? a.cfg.q_weight : a.cfg.k_weight;
    const int d = i < D ? i : i - D;
    s_w[0][i] = !w ? 1.f
                : a.cfg.weight_f32 ? static_cast<const float *>(w)[d]
                                   : bf16_to_f32(static_cast<const uint16_t *>(w)[d]);
  }
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
    s_pos[tid] = static_cast<int>(pos);       // >= -2^30
  }
  __syncthreads();

  const int l = lane % LPR, rg = lane / LPR;
  const int rp = a.cfg.rot / 16;              // lanes whose pieces are rotated
  const bool turns = l < rp;
  const int p0 = turns ? l : 2 * rp + 2 * (l - rp), p1 = turns ? l + rp : p0 + 1;
  const int rows = a.H_q + 2 * a.H_kv;
  const float inv_d = 1.f / D;
  for (int i = warp / a.wpt; i < n1 - n0; i += kWarps / a.wpt) {
    const long long slot = s_slot[i];
    if (slot == -2) continue;                 // the whole warp
    const size_t n = static_cast<size_t>(n0) + i;
    // row group r0 of the token (the lane's row of it)
    auto fetch = [&](int r0, uint4 &u0, uint4 &u1) {
      const int r = r0 + rg;
      const bool is_q = r < a.H_q, is_k = !is_q && r < a.H_q + a.H_kv;
      const int h = is_q ? r : is_k ? r - a.H_q : r - a.H_q - a.H_kv;
      u0 = u1 = make_uint4(0, 0, 0, 0);
      if (r < rows && (is_q || slot >= 0)) {
        const uint16_t *src = (is_q ? a.q + n * a.q_stride : is_k ? a.k_new + n * a.k_stride : a.v_new + n * a.v_stride) +
                              static_cast<size_t>(h) * D;
        u0 = __ldcs(reinterpret_cast<const uint4 *>(src) + p0);
        u1 = __ldcs(reinterpret_cast<const uint4 *>(src) + p1);
      }
    };
    // two groups at a time, the next two requested meanwhile (34,700 tokens: 244 us without and with
    // one ahead, 196 so); the angles wait in shared memory, whose 16 registers let a third CTA run
    const int step = a.wpt * RPW, first = (warp % a.wpt) * RPW;
    uint4 u0, u1, v0, v1;
    fetch(first, u0, u1);
    fetch(first + step, v0, v1);
    // the token's 8 angles of this lane, each computed by one row group for all
    __syncwarp();
    {
      const unsigned long long pos = static_cast<unsigned long long>(static_cast<long long>(s_pos[i]));
#pragma unroll
      for (int x = 0; x < APL; ++x) {
        const int t = rg * APL + x;           // which of the 8
        const int f = INTER ? (t < 4 ? 4 * p0 + t : 4 * p1 + t - 4) : 8 * l + t;
        if (turns) {
          const int frac = static_cast<int>((s_freq[f] * pos) >> 32);   // of a turn, times 2^32
          float c, s;
          sincospif(static_cast<float>(frac) * 0x1p-31f, &s, &c);
          s_turn[warp][0][l][t] = c * a.cfg.rope_scale;
          s_turn[warp][1][l][t] = s * a.cfg.rope_scale;
        }
      }
    }
    __syncwarp();
    auto cs = [&](int e) -> float { return s_turn[warp][0][l][e]; };
    auto sn = [&](int e) -> float { return s_turn[warp][1][l][e]; };
    auto process = [&](int r0, const uint4 &w0, const uint4 &w1) {
      const int r = r0 + rg;
      const bool is_q = r < a.H_q, is_k = !is_q && r < a.H_q + a.H_kv;
      const int h = is_q ? r : is_k ? r - a.H_q : r - a.H_q - a.H_kv;
      const bool live = r < rows && (is_q || slot >= 0);
      float y0[8], y1[8];
      unpack16(w0, y0, uint16_t());
      unpack16(w1, y1, uint16_t());
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y0[e], y0[e], fmaf(y1[e], y1[e], ss));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
      if (is_q || is_k) {
        if (is_q ? a.cfg.q_weight != nullptr : a.cfg.k_weight != nullptr) {
          const float f = rsqrtf(ss * inv_d + a.cfg.eps);
          const float *w = s_w[is_q ? 0 : 1];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y0[e] = y0[e] * f * w[8 * p0 + e];
            y1[e] = y1[e] * f * w[8 * p1 + e];
          }
        }
        if (turns) {
          if constexpr (INTER) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = y0[2 * e], z = y0[2 * e + 1], v = y1[2 * e], w = y1[2 * e + 1];
              y0[2 * e] = x * cs(e) - z * sn(e);
              y0[2 * e + 1] = z * cs(e) + x * sn(e);
              y1[2 * e] = v * cs(4 + e) - w * sn(4 + e);
              y1[2 * e + 1] = w * cs(4 + e) + v * sn(4 + e);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float x = y0[e], z = y1[e];
              y0[e] = x * cs(e) - z * sn(e);
              y1[e] = z * cs(e) + x * sn(e);
            }
          }
        }
      }
      if constexpr (FP8) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          m = max(m, max(__float_as_uint(y0[e]) & 0x7fffffffu, __float_as_uint(y1[e]) & 0x7fffffffu));
        uint32_t top = m;
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
        if (__any_sync(kFull, top >= 0x7f800000u)) {   // infinities or NaN in some row: rare
          m = 0;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint32_t x = __float_as_uint(e < 8 ? y0[e & 7] : y1[e & 7]) & 0x7fffffffu;
            m = max(m, x < 0x7f800000u ? x : x == 0x7f800000u ? 0u : 0xffffffffu);
          }
          top = m;
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(kFull, top, o));
        }
        if (live && !is_q) {
          const bool nan = top == 0xffffffffu;
          const int e = nan ? 0 : row_exponent(top);
          const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
          const size_t row = static_cast<size_t>(slot) * a.H_kv + h;
          uint2 *dst = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(is_k ? a.k_pages : a.v_pages) + row * D);
          dst[p0] = quantise8(y0, inv);
          dst[p1] = quantise8(y1, inv);
          if (l == 0) (is_k ? a.k_scale : a.v_scale)[row] = static_cast<uint8_t>(nan ? 255 : e + 127);
        }
      }
      if (live && (is_q || !FP8)) {
        uint16_t *dst = is_q ? a.q_out + n * a.qo_stride + static_cast<size_t>(h) * D
                             : static_cast<uint16_t *>(is_k ? a.k_pages : a.v_pages) +
                                   (static_cast<size_t>(slot) * a.H_kv + h) * D;
        const bool same = !is_q && !is_k;     // values pass as they are
        reinterpret_cast<uint4 *>(dst)[p0] = same ? w0 : pack8(y0);
        reinterpret_cast<uint4 *>(dst)[p1] = same ? w1 : pack8(y1);
      }
    };
    for (int r0 = first; r0 < rows; r0 += 2 * step) {
      const uint4 w0 = u0, w1 = u1, x0 = v0, x1 = v1;
      fetch(r0 + 2 * step, u0, u1);
      fetch(r0 + 3 * step, v0, v1);
      process(r0, w0, w1);
      if (r0 + step < rows) process(r0 + step, x0, x1);
    }
  }
}

template <int D, bool FP8>
cudaError_t launch_d(const RopeWriteArgs &a, dim3 grid, cudaStream_t s) {
  return a.cfg.interleaved ? launch_pdl(kv_rope_kernel<D, FP8, true>, grid, dim3(kThreads), 0, s, a)
                           : launch_pdl(kv_rope_kernel<D, FP8, false>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_kv_write_rope(const RopeWriteArgs &a0, cudaStream_t s) {
  RopeWriteArgs a = a0;
  // few tokens: one per CTA, its rows over all warps; many: a warp takes a token's rows, so that its
  // angles are computed once, and a CTA enough of them to pay for its own start
  a.tpc = 1;
  while (a.tpc < kMaxTok && a.n_tok / (2 * a.tpc) >= 4 * 152) a.tpc *= 2;
  a.wpt = a.tpc >= kWarps ? 1 : kWarps / a.tpc;
  while ((1 << a.lg_page) < a.page_size) ++a.lg_page;
  const dim3 grid((a.n_tok + a.tpc - 1) / a.tpc);
  ProfScope ps("kv_cache_write_rope", s);
  if (a.fp8) return a.D == 128 ? launch_d<128, true>(a, grid, s) : launch_d<64, true>(a, grid, s);
  return a.D == 128 ? launch_d<128, false>(a, grid, s) : launch_d<64, false>(a, grid, s);
}

}  // namespace dsa
