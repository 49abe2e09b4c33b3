// Attention of a ragged chunk of new tokens over the paged cache (tcgen05 + TMA + TMEM).
//
// Row (token n of sequence b at position p, query head h) sees the keys
//   A = { j <= p : j > p - n_stream or j < n_sink }
// and gets out = sum_A exp(s_j - lse) v_j, s_j = scale q . k_j, lse = log sum_A exp(s_j).
//
// Work.  The G = H_q / H_kv heads that share a KV head are packed with the tokens into MMA
// rows (row = token * G + head), so a K/V tile is loaded once for all of them and a single
// token already brings G rows.  An item is one KV head of up to two such 128-row tiles of
// one sequence, over the 128-key tiles that any of its rows sees (sink tiles, then window
// tiles).  The items' key tiles of the whole launch, laid end to end, are cut into equal
// shares, one per CTA (one CTA per SM): uneven lengths, one long context and many short ones
// all fill the GPU without a schedule made on the host, which knows no length.  A CTA finds
// its share from q_start and kv_len alone (one parallel pass over the sequences).  An item
// that a share boundary cuts leaves fp32 partials (O, m, l) in the workspace, and a second
// kernel merges them.
//
// One CTA, two streams of scores (i = 0, 1), each with its own TMEM buffers S_i, O_i and its
// own softmax warpgroup, so that one stream's softmax runs while the tensor core works for
// the other:
//   two-tile items: stream i is query tile i, both see every key tile (256 rows per loaded
//     K/V tile);
//   one-tile items (a few tokens): both streams hold the same query tile and take the key
//     tiles alternately; their halves are merged in TMEM at the end of the item.
// Warps: 0-3 and 4-7 softmax of stream 0 and 1 (one thread per row, 128 keys), 8 producer
// (TMA), 9 MMA issuer; FP8 caches add the converter warps 12-15, which widen the E4M3 tiles
// that TMA brings into a staging ring to bf16 operand tiles (exact: code * 2^e is a bf16).
//   S_i = Q_i K^T (M = N = 128, K = D), P over the first half of S_i, O_i += P V.
// Each stream issues P V (tile t) and right behind it Q K^T (its next tile): S_i full then
// also says that P V before it has retired, so moving the softmax reference (O rescaled in
// TMEM) needs no wait of its own.
//
// Softmax: the reference m follows the running maximum lazily, moving only when the maximum
// exceeds it by more than 2^kSlack; P <= 2^kSlack is rounded to bf16 for the tensor core
// (relative half step 2^-9 of each probability, as fine as the output's own rounding), the
// row sum l adds the unrounded fp32 values, O accumulates in fp32.
//
// Keys that no row of the item sees (behind the sequence, before the window, bad pages) have
// their value rows zeroed, so whatever the pages hold there cannot reach the sums as 0 * NaN.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "api_common.h"
#include "common.cuh"
#include "launch.h"
#include "mma_sync.cuh"
#include "profile.h"
#include "tc_ptx.cuh"

namespace dsa {

DSA_CHECK_WORD(paged_attn_check_word)

namespace {

using namespace tc;

constexpr int kRows = 128;         // query rows per tile
constexpr int kKeys = 128;         // keys per tile
constexpr int kMetaRing = 8;       // tile descriptions in flight (the rings run at most 4 ahead)
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;      // log2 units
constexpr uint64_t kWaitLimitNs = 500000000ull;

static __device__ int g_paged_error;   // sticky error word, read by dsa_device_error
static __device__ unsigned long long g_wait_limit_ns = kWaitLimitNs;

struct TileMeta {
  uint32_t seen[kKeys / 32];   // bit c: key c of the tile is in a good page and some row sees it
  int page[8];                 // page of each 16..128-key part (n_pages: none, reads as zero)
};

template <int D, bool FP8>
struct Cfg {
  static constexpr int kHalves = D / 64;                    // 128-byte column blocks of a bf16 tile
  static constexpr uint32_t kHalf = kKeys * 128;            // bytes of one of them (128 rows)
  static constexpr uint32_t kTile = kHalves * kHalf;        // a Q, K or V tile in bf16
  static constexpr uint32_t kRaw = kKeys * D;               // an FP8 tile
  static constexpr int kSlots = FP8 ? 3 : 5;                // operand ring (K and V tiles in order)
  static constexpr int kRawSlots = FP8 ? 4 : 0;             // staging ring
  static constexpr int kThreads = FP8 ? 512 : 384;
  static constexpr int kClean = FP8 ? 0 : 4;                // value tiles checked ahead of their use
  // registers a thread after the split by warpgroup (softmax x 2, warps 8-11, converters);
  // what the launch holds, threads x kRegLaunch, is what the shares add up to
  static constexpr int kRegLaunch = FP8 ? 128 : 168;
  static constexpr int kRegSoft = FP8 ? 184 : 208, kRegMisc = FP8 ? 56 : 88, kRegConv = FP8 ? 88 : 0;
  static_assert(256 * kRegSoft + 128 * kRegMisc + 128 * kRegConv == kThreads * kRegLaunch, "register split");
  static constexpr uint32_t oQ = 0;
  static constexpr uint32_t oRing = oQ + 2 * kTile;
  static constexpr uint32_t oRaw = oRing + kSlots * kTile;
  static constexpr uint32_t oMeta = oRaw + kRawSlots * kRaw;
  static constexpr uint32_t oMl = oMeta + kMetaRing * sizeof(TileMeta);
  static constexpr uint32_t oBar = oMl + kRows * 8;         // stream 1's (m, l) of one-tile items
  // q_full, q_empty, slot full/empty, raw full/empty, s_full x2, p_full x2, o_final x2,
  // ml_ready, o1_free, fin, clean
  static constexpr int kBars = 2 + 2 * kSlots + 2 * kRawSlots + 6 + 3 + kClean;
  static constexpr uint32_t oMisc = oBar + kBars * 8;
  static constexpr uint32_t kBytes = oMisc + 96 + 1024;
  static constexpr uint32_t cS = 0, cO = 2 * kKeys;         // TMEM columns: S_0, S_1 | O_0, O_1
  static_assert(cO + 2 * D <= kTmemCols, "TMEM columns");
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

struct Args {
  CUtensorMap tq, tk, tv;
  const int32_t *q_start, *kv_len, *page_table;
  const uint8_t *k_scale, *v_scale;
  uint16_t *out;
  float *lse;
  float *part;           // [2 * max_ctas][D / 4][part_rows][4]
  float *part_ml;        // [2 * max_ctas][part_rows][2]
  PagedPiece *piece;     // [max_ctas]
  int B, n_tok, max_pages, n_pages, page_size, lg_page, H_q, H_kv, G, TT;
  int part_rows, lg_min_units;
  int n_sink, n_stream;  // n_stream < 0: no window
  float sl2;
};

// ------------------------------------------------------------------ schedule

// Keys and tiles of the entry (sequence b, pair m of query tiles), the same for every KV head.
struct Entry {
  int tok0, ntok;      // first token row (global), tokens
  int p0;              // position of the first token
  int p_hi;            // position of the last one (< 0: no row sees a key)
  int ns, w0;          // tiles [0, ns), then [w0, w0 + n - ns)
  int n;               // tiles (at least 1: an entry without keys still writes its rows)
  int lw;              // log2 of a tile's schedule weight: two query tiles weigh 2, one 1
  bool keys;           // some row sees a key
};

struct Seq {
  int qs, nq, kv;
};

__device__ __forceinline__ Seq load_seq(const Args &a, int b) {
  const int qs = a.q_start[b], qe = a.q_start[b + 1], kv = a.kv_len[b];
  const int cap = a.max_pages << a.lg_page;
  DSA_CHECK(qs >= 0 && qe >= qs && qe <= a.n_tok && kv >= qe - qs && kv <= cap);
  Seq s;
  s.qs = min(max(qs, 0), a.n_tok);
  s.nq = max(min(qe, a.n_tok) - s.qs, 0);
  s.kv = min(max(kv, 0), cap);
  return s;
}

__device__ __forceinline__ int n_pairs(const Args &a, const Seq &s) {
  return (s.nq + 2 * a.TT - 1) / (2 * a.TT);
}

__device__ __forceinline__ Entry make_entry(const Args &a, const Seq &s, int m) {
  Entry e;
  e.tok0 = s.qs + m * 2 * a.TT;
  e.ntok = min(2 * a.TT, s.nq - m * 2 * a.TT);
  e.p0 = s.kv - s.nq + m * 2 * a.TT;
  e.p_hi = e.p0 + e.ntok - 1;
  e.lw = e.ntok > a.TT ? 1 : 0;
  e.ns = e.w0 = e.n = 0;
  if (e.p_hi >= 0) {
    const int last = e.p_hi / kKeys;
    if (a.n_stream < 0) {
      e.n = last + 1;
    } else {
      const int sinks = min(a.n_sink, e.p_hi + 1);
      const int s_tiles = (sinks + kKeys - 1) / kKeys;
      if (a.n_stream == 0) {
        e.ns = e.w0 = e.n = s_tiles;
      } else {
        const int lo = max(max(e.p0, 0) - a.n_stream + 1, 0);   // n_stream >= 1: no overflow
        e.w0 = lo / kKeys;
        e.ns = min(s_tiles, e.w0);
        e.n = e.ns + last - e.w0 + 1;
      }
    }
  }
  e.keys = e.n > 0;
  e.n = max(e.n, 1);
  return e;
}

// What a CTA's planning leaves for its warps: the share [u0, u1), the item it begins in (first
// unit, sequence, pair, KV head) and how the launch's units are dealt out.
struct Plan {
  long long item_u0, u0, u1, q;
  int r, P;
  int b, m, g;
  Seq s;
};
static_assert(sizeof(Plan) <= 80, "room behind the barriers");

// A CTA's walk over the items of its share [u0, u1) of schedule units.
struct Walk {
  long long u0, u1;     // the share
  long long item_u0;    // first unit of the current item
  int b, m, g;
  Seq s;
  Entry e;
  int t0, t1;           // key tiles of the current item in this share
  bool valid;
};

// first unit of share c: the units are dealt out q to each, the first r shares one more
__device__ __forceinline__ long long share_begin(long long q, int r, int c) { return q * c + min(c, r); }

// tiles [t0, t1) of an item (n tiles of 2^lw units from item_u0 on) in the share [u0, u1)
__device__ __forceinline__ void piece_of(long long u0, long long u1, long long item_u0, int n, int lw,
                                         int &t0, int &t1) {
  t0 = u0 > item_u0 ? static_cast<int>(min((u0 - item_u0) >> lw, static_cast<long long>(n))) : 0;
  t1 = u1 < item_u0 + (static_cast<long long>(n) << lw) ? static_cast<int>((u1 - item_u0) >> lw) : n;
}

// the first non-empty piece at or after the current item
__device__ __forceinline__ void walk_settle(const Args &a, Walk &w) {
  while (true) {
    w.valid = w.item_u0 < w.u1;
    if (!w.valid) return;
    piece_of(w.u0, w.u1, w.item_u0, w.e.n, w.e.lw, w.t0, w.t1);
    if (w.t1 > w.t0) return;
    w.item_u0 += static_cast<long long>(w.e.n) << w.e.lw;
    if (++w.g == a.H_kv) {
      w.g = 0;
      ++w.m;
      while (w.m >= n_pairs(a, w.s)) {
        w.m = 0;
        if (++w.b >= a.B) {
          w.valid = false;
          return;
        }
        w.s = load_seq(a, w.b);
      }
      w.e = make_entry(a, w.s, w.m);
    }
  }
}

__device__ __forceinline__ void walk_next(const Args &a, Walk &w) {
  w.u0 = max(w.u0, w.item_u0 + (static_cast<long long>(w.e.n) << w.e.lw));   // this item is done
  walk_settle(a, w);
}

// key tile `k` of an entry -> its first key
__device__ __forceinline__ int tile_base(const Entry &e, int k) {
  return (k < e.ns ? k : e.w0 + k - e.ns) * kKeys;
}

// ------------------------------------------------------------------ waits

// Bounded wait: gives up when another thread of the CTA did, or after the limit.
__device__ __forceinline__ bool slow_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  const uint64_t t0 = global_ns();
  const uint64_t limit = g_wait_limit_ns;
  const uint32_t hint = limit < 20000ull ? static_cast<uint32_t>(limit) : 20000u;
  uint32_t spins = 0;
  while (true) {
    if (mbar_try_wait_hint(bar, parity, hint)) return true;
    if (*abort) return false;
    if ((++spins & 3u) == 0u && global_ns() - t0 > limit) {
      *abort = 1;
      return false;
    }
  }
}

// the whole warp waits; the outcome is warp-uniform
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = slow_wait(bar, parity, abort) ? 1 : 0;
  ok = __shfl_sync(kFull, ok, 0);
  // every lane observes the phase itself, so that what was released by it is visible to it
  if (ok && !mbar_try_wait(bar, parity)) ok = 0;
  return __all_sync(kFull, ok) != 0;
}

__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_ns() - t0 > limit_ns) return;
}

// a ring position: slot and phase parity
template <int N>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// ------------------------------------------------------------------ FP8 -> bf16

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <uint32_t kSel>
__device__ __forceinline__ uint32_t prmt(uint32_t x) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;\n" : "=r"(r) : "r"(x), "n"(kSel));
  return r;
}

// Four E4M3 codes -> four bf16 times f (a power of two in both halves, 2^(120 + e)): a code's
// seven magnitude bits at bits 4..10 of a bf16 read as its value times 2^-120 (bias 127 against
// 7, subnormal codes as bf16 subnormals), so one exact multiply gives code * 2^e.  Bytes are
// spread over halves with their sign replicated, moved up by 4 and cut to sign and magnitude:
// three integer operations for two codes, one of which can run as a multiply on the FMA pipe
// (the ALU pipe, at half rate, is what bounds this).
__device__ __forceinline__ uint2 widen4(uint32_t c, uint32_t f) {
  const uint32_t x0 = (prmt<0x9180>(c) * 16u) & 0x87f087f0u, x1 = (prmt<0xb3a2>(c) * 16u) & 0x87f087f0u;
  return make_uint2(mul_bf16x2(x0, f), mul_bf16x2(x1, f));
}

// Lanes `mask` apart exchange: the one with `up` set gives x and takes the other's y for it.
__device__ __forceinline__ void swap4(uint4 &x, uint4 &y, int up, int mask) {
  uint4 t = up ? x : y;
  t.x = __shfl_xor_sync(kFull, t.x, mask);
  t.y = __shfl_xor_sync(kFull, t.y, mask);
  t.z = __shfl_xor_sync(kFull, t.z, mask);
  t.w = __shfl_xor_sync(kFull, t.w, mask);
  if (up) x = t;
  else y = t;
}

// ------------------------------------------------------------------ kernel

template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::kThreads, 1) paged_attn_kernel(const __grid_constant__ Args a) {
  using C = Cfg<D, FP8>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::oBar);
  uint64_t *q_full = bars, *q_empty = bars + 1;
  uint64_t *full = bars + 2, *empty = full + C::kSlots;
  uint64_t *raw_full = empty + C::kSlots, *raw_empty = raw_full + C::kRawSlots;
  uint64_t *s_full = raw_empty + C::kRawSlots, *p_full = s_full + 2, *o_final = p_full + 2;
  uint64_t *ml_ready = o_final + 2, *o1_free = ml_ready + 1, *fin = o1_free + 1, *clean = fin + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::oMisc);
  volatile int *abort = reinterpret_cast<volatile int *>(sm + C::oMisc + 4);
  Plan *plan = reinterpret_cast<Plan *>(sm + C::oMisc + 16);
  TileMeta *meta = reinterpret_cast<TileMeta *>(sm + C::oMeta);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&full[i], FP8 ? 4 : 1);
      mbar_init(&empty[i], FP8 ? 1 : 3);   // the MMAs that read it; bf16: and both cleaners
    }
    for (int i = 0; i < C::kRawSlots; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_final[i], 1);
    }
    mbar_init(ml_ready, 4);
    mbar_init(o1_free, 4);
    mbar_init(fin, 1);
    for (int i = 0; i < C::kClean; ++i) mbar_init(&clean[i], 2);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  grid_dep_wait();
  grid_dep_release();

  // ---------------------------------------------------------------- this CTA's share
  // units of every sequence (in the still unused ring), their running sum, and the item in
  // which the share begins
  {
    long long *su = reinterpret_cast<long long *>(sm);   // [B]
    for (int b0 = 0; b0 < a.B; b0 += C::kThreads) {
      const int b = b0 + tid;
      long long u = 0;
      bool many = false;
      if (b < a.B) {
        const Seq s = load_seq(a, b);
        many = s.nq > 2 * a.TT;
        if (!many && s.nq > 0) {
          const Entry e = make_entry(a, s, 0);
          u = (static_cast<long long>(e.n) << e.lw) * a.H_kv;
        }
      }
      uint32_t todo = __ballot_sync(kFull, many);
      while (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const Seq s = load_seq(a, b0 + (tid & ~31) + src);
        const int np = n_pairs(a, s);
        long long x = 0;
        for (int m = lane; m < np; m += 32) {
          const Entry e = make_entry(a, s, m);
          x += static_cast<long long>(e.n) << e.lw;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
        if (lane == src) u = x * a.H_kv;
      }
      if (b < a.B) su[b] = u;
    }
    __syncthreads();
    if (warp == 0) {
      long long run = 0;
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        long long v = b < a.B ? su[b] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(kFull, v, o);
          if (lane >= o) v += y;
        }
        if (b < a.B) su[b] = run + v;   // inclusive
        run += __shfl_sync(kFull, v, 31);
      }
      // shares: at least min_units each, so that a short launch is not cut finer than pays
      const long long total = run;
      const int P = static_cast<int>(min(static_cast<long long>(gridDim.x), max(1ll, total >> a.lg_min_units)));
      const long long q = total < (1ll << 31) ? static_cast<long long>(static_cast<uint32_t>(total) / static_cast<uint32_t>(P))
                                              : total / P;
      const int r = static_cast<int>(total - q * P);
      const int c = blockIdx.x;
      const long long u0 = c < P ? share_begin(q, r, c) : total, u1 = c < P ? share_begin(q, r, c + 1) : total;
      // the sequence that holds unit u0: the first with su[b] > u0
      int lo = 0, hi = a.B;   // su[hi] > u0 whenever u0 < total
      __syncwarp();
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (su[mid] > u0) hi = mid;
        else lo = mid + 1;
      }
      int m = 0, g = 0;
      long long base = lo > 0 ? su[lo - 1] : 0;
      Seq s = {0, 0, 0};
      if (u0 < u1 && lo < a.B) {
        s = load_seq(a, lo);
        const int np = n_pairs(a, s);
        // its pair that holds u0, 32 pairs at a time
        for (int m0 = 0; m0 < np; m0 += 32) {
          const int mm = m0 + lane;
          uint32_t item = 0;   // units of one KV head: at most 2^24
          if (mm < np) {
            const Entry e = make_entry(a, s, mm);
            item = static_cast<uint32_t>(e.n) << e.lw;
          }
          const long long own = static_cast<long long>(item) * a.H_kv;
          long long v = own;
          if (np > 1) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const long long y = __shfl_up_sync(kFull, v, o);
              if (lane >= o) v += y;
            }
          }
          const uint32_t past = __ballot_sync(kFull, item > 0 && base + v > u0);
          if (past) {
            const int l = __ffs(past) - 1;
            m = m0 + l;
            base += __shfl_sync(kFull, v - own, l);
            item = __shfl_sync(kFull, item, l);
            g = static_cast<int>(static_cast<uint32_t>(u0 - base) / item);   // below 2^31 units an entry
            base += static_cast<long long>(item) * g;
            break;
          }
          base += __shfl_sync(kFull, v, 31);
        }
      }
      if (lane == 0) {
        *plan = Plan{base, u0, u1, q, r, P, lo, m, g, s};
      }
    }
  }
  fence_proxy_async_smem();   // the planning scratch becomes ring slots that TMA fills
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk w;
  w.u0 = plan->u0;
  w.u1 = plan->u1;
  w.item_u0 = plan->item_u0;
  w.b = plan->b;
  w.m = plan->m;
  w.g = plan->g;
  w.s = plan->s;
  w.valid = false;
  if (w.u0 < w.u1 && w.b < a.B) {
    w.e = make_entry(a, w.s, w.m);
    walk_settle(a, w);
  }
  if (tid == 0) a.piece[blockIdx.x].valid = 0;   // until this share begins a cut item

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax, epilogue
    reg_inc<C::kRegSoft>();
    const int i = warp >> 2;                          // stream
    const int row = (warp & 3) * 32 + lane;           // row of the query tile
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = tl + C::cS + i * kKeys;
    const uint32_t o_col = tl + C::cO + i * D;
    float2 *ml = reinterpret_cast<float2 *>(sm + C::oMl);
    const int rtok = row / a.G, rhead = row - rtok * a.G;
    uint32_t s_phase = 0, of_phase = 0, ml_phase = 0;
    uint32_t tile = 0;                                // key tiles seen so far (meta ring)
    bool ok = true;
    for (; ok && w.valid; walk_next(a, w)) {
      const Entry &e = w.e;
      const bool single = e.lw == 0;
      const int T = w.t1 - w.t0;
      const int tok = rtok + (single ? 0 : i * a.TT); // token of the entry
      const bool row_ok = rtok < a.TT && tok < e.ntok;
      const bool warp_ok = __any_sync(kFull, row_ok);
      const int p = e.p0 + (row_ok ? tok : e.ntok - 1);
      float m_ref = -INFINITY, l = 0.f;               // base-2 units
      if (e.keys) {
        for (int k = single ? i : 0; k < T; k += single ? 2 : 1) {
          ok = warp_wait(&s_full[i], s_phase, abort);
          if (!ok) break;
          s_phase ^= 1u;
          tc_fence_after();
          if (warp_ok) {
            const int base = tile_base(e, w.t0 + k);
            const TileMeta *md = &meta[(tile + k) % kMetaRing];
            uint32_t s[kKeys];
#pragma unroll
            for (int c = 0; c < kKeys; c += 32) tmem_ld32(s_col + c, s + c);
            const uint4 seen = *reinterpret_cast<const uint4 *>(md->seen);
            const int hi = p - base;                  // keys c <= hi are not after the row
            const int lo = a.n_stream < 0 ? 0 : p - a.n_stream + 1 - base;   // c >= lo: in its window
            const int sk = a.n_sink - base;           // c < sk: a first token
            const bool trim = hi < kKeys - 1 || (lo > 0 && sk < kKeys) ||
                              (seen.x & seen.y & seen.z & seen.w) != 0xffffffffu;
            tmem_wait_ld();
            if (__any_sync(kFull, trim)) {
              const uint32_t sw[4] = {seen.x, seen.y, seen.z, seen.w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                // bits below x of the q-th 32 keys
                auto below = [&](int x) -> uint32_t {
                  const int y = x - 32 * q;
                  return y <= 0 ? 0u : (y >= 32 ? 0xffffffffu : (1u << y) - 1u);
                };
                const uint32_t v = sw[q] & below(hi + 1) & (~below(lo) | below(sk));
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  s[32 * q + c] = (v >> c) & 1u ? s[32 * q + c] : __float_as_uint(-INFINITY);
              }
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < kKeys; c += 2)
              mx[(c >> 1) & 3] = fmax3(mx[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
            const float mt = fmax3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * a.sl2;
            const bool move = mt > m_ref + kSlack;
            if (__any_sync(kFull, move)) {
              float f = 1.f;
              if (move) {
                f = m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - mt);
                l *= f;
                m_ref = mt;
              }
              if (k > (single ? i : 0)) {             // O holds earlier tiles of this piece
                const float2 f2 = make_float2(f, f);
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                  uint32_t o[16];
                  tmem_ld16(o_col + c, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int x = 0; x < 16; x += 2) {
                    const float2 y = fmul2(make_float2(__uint_as_float(o[x]), __uint_as_float(o[x + 1])), f2);
                    o[x] = __float_as_uint(y.x);
                    o[x + 1] = __float_as_uint(y.y);
                  }
                  tmem_st16(o_col + c, o);
                }
              }
            }
            const float nm = m_ref == -INFINITY ? 0.f : -m_ref;
            const float2 nm2 = make_float2(nm, nm), sl22 = make_float2(a.sl2, a.sl2);
            float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
            for (int c0 = 0; c0 < kKeys; c0 += 32) {
              uint32_t pk[16];
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                const float2 y = ffma2(make_float2(__uint_as_float(s[c0 + c]), __uint_as_float(s[c0 + c + 1])), sl22, nm2);
                const float2 x = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                if ((c >> 1) & 1) acc1 = fadd2(acc1, x);
                else acc0 = fadd2(acc0, x);
                pk[c >> 1] = pack_bf16x2(x.x, x.y);
              }
              tmem_st16(s_col + c0 / 2, pk);
            }
            const float2 as = fadd2(acc0, acc1);
            l += as.x + as.y;
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[i]);
        }
        if (!ok) break;
        tile += T;
      }
      // ---------------- end of the piece: O_i complete after the stream's last P V
      const int mine = !e.keys ? 0 : single ? (T - i + 1) / 2 : T;   // tiles of this stream
      if (mine > 0) {
        ok = warp_wait(&o_final[i], of_phase, abort);
        if (!ok) break;
        of_phase ^= 1u;
        tc_fence_after();
      }
      if (single && i == 1) {
        // hand (m, l) to stream 0, which merges the halves, and wait until it has read O_1
        ml[row] = make_float2(m_ref, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_ready);
        ok = warp_wait(o1_free, ml_phase, abort);
        ml_phase ^= 1u;
        continue;
      }
      float f0 = 1.f, f1 = 0.f, m = m_ref;
      bool two = false;
      if (single) {
        ok = warp_wait(ml_ready, ml_phase, abort);
        if (!ok) break;
        ml_phase ^= 1u;
        tc_fence_after();
        const float2 o = ml[row];
        two = e.keys && T > 1;                        // stream 1 had a tile: O_1 is defined
        m = fmaxf(m_ref, o.x);
        f0 = m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - m);
        f1 = o.x == -INFINITY ? 0.f : fast_exp2(o.x - m);
        l = l * f0 + o.y * f1;
      }
      const bool whole = w.t0 == 0 && w.t1 == e.n;
      const bool some = mine > 0;
      const float inv = whole ? (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) : 1.f;   // NaN stays NaN
      const float g0 = f0 * inv, g1 = f1 * inv;
      const int head = w.g * a.G + rhead;
      const size_t orow = static_cast<size_t>(e.tok0 + tok) * a.H_q + head;
      const int slot = 2 * blockIdx.x + (w.t0 == 0 ? 1 : 0);
      const int prow = (single ? 0 : i * kRows) + row;
      if (warp_ok) {
        long long quad_row[4];                        // output rows of the lane's quad (-1: none)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          quad_row[x] = __shfl_sync(kFull, row_ok ? static_cast<long long>(orow) : -1ll, (lane & ~3) + x);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          if (some) tmem_ld32(o_col + c, o);
          if (two) {
            uint32_t o1[32];
            tmem_ld32(o_col + D + c, o1);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x)
              o[x] = __float_as_uint((f0 == 0.f ? 0.f : __uint_as_float(o[x]) * g0) +
                                     (f1 == 0.f ? 0.f : __uint_as_float(o1[x]) * g1));
          } else {
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x)
              o[x] = !some || l == 0.f ? 0u : __float_as_uint(__uint_as_float(o[x]) * g0);
          }
          if (whole) {
            // 4 x 4 transpose of 16-byte pieces over four lanes: store j then covers 64
            // contiguous bytes of row j of the quad instead of 16 bytes of every row
            uint4 y[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              y[x].x = pack_bf16x2(__uint_as_float(o[8 * x]), __uint_as_float(o[8 * x + 1]));
              y[x].y = pack_bf16x2(__uint_as_float(o[8 * x + 2]), __uint_as_float(o[8 * x + 3]));
              y[x].z = pack_bf16x2(__uint_as_float(o[8 * x + 4]), __uint_as_float(o[8 * x + 5]));
              y[x].w = pack_bf16x2(__uint_as_float(o[8 * x + 6]), __uint_as_float(o[8 * x + 7]));
            }
            swap4(y[0], y[1], lane & 1, 1);
            swap4(y[2], y[3], lane & 1, 1);
            swap4(y[0], y[2], lane & 2, 2);
            swap4(y[1], y[3], lane & 2, 2);
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (quad_row[x] >= 0)
                *reinterpret_cast<uint4 *>(a.out + quad_row[x] * D + c + 8 * (lane & 3)) = y[x];
          } else if (row_ok) {
            float4 *dst = reinterpret_cast<float4 *>(a.part) +
                          (static_cast<size_t>(slot) * (D / 4) + c / 4) * a.part_rows + prow;
#pragma unroll
            for (int x = 0; x < 8; ++x)
              dst[static_cast<size_t>(x) * a.part_rows] =
                  make_float4(__uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1]),
                              __uint_as_float(o[4 * x + 2]), __uint_as_float(o[4 * x + 3]));
          }
        }
        if (row_ok) {
          if (whole) {
            if (a.lse) a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
          } else {
            reinterpret_cast<float2 *>(a.part_ml)[static_cast<size_t>(slot) * a.part_rows + prow] = make_float2(m, l);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (single && lane == 0) mbar_arrive(o1_free);
      // the share in which a cut item begins describes it for the merge
      if (i == 0 && row == 0 && w.t0 == 0 && !whole) {
        PagedPiece d;
        d.item_u0 = w.item_u0;
        d.q = plan->q;
        d.r = plan->r;
        d.P = plan->P;
        d.n = e.n;
        d.lw = e.lw;
        d.tok0 = e.tok0;
        d.ntok = e.ntok;
        d.g = w.g;
        d.valid = 1;
        a.piece[blockIdx.x] = d;
      }
    }
  } else if (warp == 8) {
    // ---------------------------------------------------------------- producer
    reg_dec<C::kRegMisc>();
    constexpr int NS = FP8 ? C::kRawSlots : C::kSlots;
    constexpr uint32_t kBytes = FP8 ? C::kRaw : C::kTile;
    uint64_t *rf = FP8 ? raw_full : full, *re = FP8 ? raw_empty : empty;
    unsigned char *ring = sm + (FP8 ? C::oRaw : C::oRing);
    const int R = min(a.page_size, kKeys);            // rows per box
    const int parts = kKeys / R;
    Ring<NS ? NS : 1> rp;
    uint32_t q_phase = 0;
    uint32_t tile = 0;
    bool ok = true, q_open = false;
    // one K or V tile into the next ring slot
    auto load = [&](const CUtensorMap *map, int k, int g) -> bool {
      if (!warp_wait(&re[rp.slot], rp.phase ^ 1u, abort)) return false;
      const TileMeta *md = &meta[(tile + k) % kMetaRing];
      unsigned char *dst = ring + rp.slot * kBytes;
      const int base = tile_base(w.e, w.t0 + k);
      if (lane == 0) mbar_arrive_expect_tx(&rf[rp.slot], kBytes);
      __syncwarp();
      const int boxes = FP8 ? parts : parts * C::kHalves;
      if (lane < boxes) {
        const int part = FP8 ? lane : lane / C::kHalves, hh = FP8 ? 0 : lane - part * C::kHalves;
        tma_load_4d(dst + (FP8 ? part * R * D : hh * C::kHalf + part * R * 128), map, &rf[rp.slot], 64 * hh, g,
                    base & (a.page_size - 1) & ~(R - 1), md->page[part]);
      }
      __syncwarp();
      rp.step();
      return true;
    };
    for (; ok && w.valid; walk_next(a, w)) {
      const Entry &e = w.e;
      if (!e.keys) continue;
      const bool single = e.lw == 0;
      const int T = w.t1 - w.t0;
      // the item's query tiles, once the MMAs of the one before have read theirs
      if (q_open) {
        ok = warp_wait(q_empty, q_phase, abort);
        if (!ok) break;
        q_phase ^= 1u;
      }
      q_open = true;
      if (lane == 0) {
        const int nt = single ? 1 : 2;
        mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(nt * C::kHalves * a.TT * a.G * 128));
        for (int t = 0; t < nt; ++t)
          for (int hh = 0; hh < C::kHalves; ++hh)
            tma_load_4d(sm + C::oQ + t * C::kTile + hh * C::kHalf, &a.tq, q_full, 64 * hh, w.g * a.G,
                        e.tok0 + t * a.TT, 0);
      }
      __syncwarp();
      const int32_t *table = a.page_table + static_cast<size_t>(w.b) * a.max_pages;
      // this lane's page of tile k
      auto page_of = [&](int k) -> int {
        int page = a.n_pages;
        const int pos = tile_base(e, w.t0 + k) + lane * R;
        if (k < T && lane < parts && pos <= e.p_hi) {   // p_hi < capacity: inside the table
          page = table[pos >> a.lg_page];
          DSA_CHECK(page >= 0 && page < a.n_pages);
          if (page < 0 || page >= a.n_pages) page = a.n_pages;
        }
        return page;
      };
      int page_next = page_of(0);
      // pages and visible keys of tile k; the next tile's pages are requested meanwhile
      auto describe = [&](int k) {
        TileMeta *md = &meta[(tile + k) % kMetaRing];
        const int base = tile_base(e, w.t0 + k);
        const int page = page_next;
        page_next = page_of(k + 1);
        if (lane < 8) md->page[lane] = page;
        const int lo = a.n_stream < 0 ? 0 : a.n_stream == 0 ? 0x7fffffff : max(e.p0, 0) - a.n_stream + 1;
#pragma unroll
        for (int q = 0; q < kKeys / 32; ++q) {
          const int c = 32 * q + lane, j = base + c;
          const bool good = __shfl_sync(kFull, page, c / R) != a.n_pages;
          const uint32_t v = __ballot_sync(kFull, good && j <= e.p_hi && (j >= lo || j < a.n_sink));
          if (lane == 0) md->seen[q] = v;
        }
        __syncwarp();
      };
      const int ahead = single ? 2 : 1;
      for (int k = 0; ok && k < min(ahead, T); ++k) {
        describe(k);
        ok = load(&a.tk, k, w.g);
      }
      for (int k = 0; ok && k < T; ++k) {
        ok = load(&a.tv, k, w.g);
        if (ok && k + ahead < T) {
          describe(k + ahead);
          ok = load(&a.tk, k + ahead, w.g);
        }
      }
      tile += T;
    }
    if (!ok || *abort) {
      // let this CTA's copies land before it exits
      if (lane == 0) {
        if (q_open) drain_wait(q_full, q_phase, 200000000ull);
        for (int s = 0; s < NS; ++s) {
          // slots before rp.slot were last filled in this round, the others in the one before
          // (or never: that wait returns at once)
          drain_wait(&rf[s], s < rp.slot ? rp.phase : rp.phase ^ 1u, 200000000ull);
        }
      }
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------- MMA issuer
    reg_dec<C::kRegMisc>();
    constexpr uint32_t id_qk = idesc_bf16_f32(kRows, kKeys, false, false);
    constexpr uint32_t id_pv = idesc_bf16_f32(kRows, D, false, true);
    const uint32_t sQ = smem_u32(sm + C::oQ);
    const uint32_t sR = smem_u32(sm + C::oRing);
    Ring<C::kSlots> rp;
    uint32_t q_phase = 0, p_phase[2] = {0, 0};
    uint32_t tile = 0;
    bool ok = true;
    // S_i = Q K^T with the K tile of ring slot `slot`
    auto qk = [&](int i, int qt, int slot) {
      if (lane == 0) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::kHalf + (kk & 3) * 32;
          tc_mma(tmem + C::cS + i * kKeys, sdesc_sw128(sQ + qt * C::kTile + off, 16, 1024),
                 sdesc_sw128(sR + slot * C::kTile + off, 16, 1024), id_qk, kk > 0 ? 1u : 0u);
        }
        tc_commit(&s_full[i]);
      }
    };
    auto pv = [&](int i, int slot, bool first) {
      if (lane == 0) {
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          tc_mma_ts(tmem + C::cO + i * D, tmem + C::cS + i * kKeys + kk * 8,
                    sdesc_sw128(sR + slot * C::kTile + kk * 2048, C::kHalf, 1024), id_pv,
                    (!first || kk > 0) ? 1u : 0u);
      }
    };
    // the next ring slot, once filled
    auto next = [&](int &slot) -> bool {
      if (!warp_wait(&full[rp.slot], rp.phase, abort)) return false;
      tc_fence_after();
      slot = rp.slot;
      rp.step();
      return true;
    };
    // a value tile, once filled and (bf16 caches) rid of rows that no row of the item sees
    Ring<FP8 ? 1 : C::kClean> rc;
    auto next_v = [&](int &slot) -> bool {
      if (!next(slot)) return false;
      if constexpr (!FP8) {
        if (!warp_wait(&clean[rc.slot], rc.phase, abort)) return false;
        rc.step();
      }
      return true;
    };
    auto wait_p = [&](int i) -> bool {
      if (!warp_wait(&p_full[i], p_phase[i], abort)) return false;
      p_phase[i] ^= 1u;
      tc_fence_after();
      return true;
    };
    auto release = [&](int slot) {
      if (lane == 0) tc_commit(&empty[slot]);
    };
    // the query tiles may be overwritten once the item's last Q K^T has read them
    auto q_done = [&]() {
      if (lane == 0) tc_commit(q_empty);
    };
    for (; ok && w.valid; walk_next(a, w)) {
      const Entry &e = w.e;
      if (!e.keys) continue;
      const bool single = e.lw == 0;
      const int T = w.t1 - w.t0;
      if (!(ok = warp_wait(q_full, q_phase, abort))) break;
      q_phase ^= 1u;
      tc_fence_after();
      int ks, vs;
      if (single) {
        for (int k = 0; ok && k < min(2, T); ++k)
          if ((ok = next(ks))) {
            qk(k, 0, ks);
            release(ks);
            if (k + 1 == T) q_done();
          }
        for (int k = 0; ok && k < T; ++k) {
          const int i = k & 1;
          if (!(ok = next_v(vs))) break;
          if (!(ok = wait_p(i))) break;
          pv(i, vs, k < 2);
          release(vs);
          if (k + 2 >= T) {
            if (lane == 0) tc_commit(&o_final[i]);
          } else {
            if (!(ok = next(ks))) break;
            qk(i, 0, ks);
            release(ks);
            if (k + 3 == T) q_done();
          }
        }
      } else {
        if ((ok = next(ks))) {
          qk(0, 0, ks);
          qk(1, 1, ks);
          release(ks);
          if (T == 1) q_done();
        }
        for (int k = 0; ok && k < T; ++k) {
          const bool more = k + 1 < T;
          if (!(ok = next_v(vs))) break;
          if (!(ok = wait_p(0))) break;
          pv(0, vs, k == 0);
          if (more) {
            if (!(ok = next(ks))) break;
            qk(0, 0, ks);
          } else if (lane == 0) {
            tc_commit(&o_final[0]);
          }
          if (!(ok = wait_p(1))) break;
          pv(1, vs, k == 0);
          release(vs);
          if (more) {
            qk(1, 1, ks);
            release(ks);
            if (k + 2 == T) q_done();
          } else if (lane == 0) {
            tc_commit(&o_final[1]);
          }
        }
      }
      tile += T;
    }
    if (lane == 0) tc_commit(fin);
    __syncwarp();
  } else if (FP8 && warp >= 12) {
    // ---------------------------------------------------------------- converters
    if constexpr (FP8) {
      reg_dec<C::kRegConv>();
      const int r = (warp - 12) * 32 + lane;          // the thread's row of every tile
      Ring<C::kRawSlots> rr;
      Ring<C::kSlots> rp;
      uint32_t tile = 0;
      bool ok = true;
      // tile k (already described) with this row's scale byte sb
      auto convert = [&](int k, uint32_t sb_raw) -> bool {
        if (!warp_wait(&raw_full[rr.slot], rr.phase, abort)) return false;
        const TileMeta *md = &meta[(tile + k) % kMetaRing];
        const bool seen = (md->seen[r >> 5] >> (r & 31)) & 1u;
        const int sb = seen ? static_cast<int>(sb_raw) : 127;
        // 2^e as 2^(120 + e) on the raw bits (scales above 2^7: see below); a row that is not
        // seen is multiplied by 0, one with a NaN scale (255) by NaN
        const int e1 = min(sb - 127, 7), e2 = sb - 127 - e1;
        const uint32_t f = !seen ? 0u : sb == 255 ? 0x7fff7fffu : (static_cast<uint32_t>(e1 + 247) << 7) * 0x00010001u;
        if (!warp_wait(&empty[rp.slot], rp.phase ^ 1u, abort)) return false;
        const unsigned char *src = sm + C::oRaw + rr.slot * C::kRaw + r * D;
        unsigned char *dst = sm + C::oRing + rp.slot * C::kTile + r * 128;
        // 16-byte piece p of the row of codes: 128-byte rows hold it at p ^ (r & 7), 64-byte
        // rows at p ^ ((r >> 1) & 3); piece q of the bf16 row goes to q ^ (r & 7) of its half
        auto piece = [&](int p) -> uint4 {
          return *reinterpret_cast<const uint4 *>(src + ((D == 128 ? p ^ (r & 7) : p ^ ((r >> 1) & 3)) << 4));
        };
        auto put = [&](int q, const uint4 &o) {
          *reinterpret_cast<uint4 *>(dst + (q >> 3) * C::kHalf + (((q & 7) ^ (r & 7)) << 4)) = o;
        };
#pragma unroll
        for (int p0 = 0; p0 < D / 16; p0 += 4) {
          uint4 c[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) c[p] = piece(p0 + p);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const uint2 y0 = widen4(c[p].x, f), y1 = widen4(c[p].y, f);
            const uint2 y2 = widen4(c[p].z, f), y3 = widen4(c[p].w, f);
            put(2 * (p0 + p), make_uint4(y0.x, y0.y, y1.x, y1.y));
            put(2 * (p0 + p) + 1, make_uint4(y2.x, y2.y, y3.x, y3.y));
          }
        }
        if (__any_sync(kFull, seen && e2 > 0 && sb != 255)) {
          // rare: a scale above 2^7 takes a second exact multiply
          const uint32_t f2 = (static_cast<uint32_t>(e2 + 127) << 7) * 0x00010001u;
#pragma unroll 1
          for (int q = 0; seen && e2 > 0 && sb != 255 && q < D / 8; ++q) {
            uint4 *o = reinterpret_cast<uint4 *>(dst + (q >> 3) * C::kHalf + (((q & 7) ^ (r & 7)) << 4));
            *o = make_uint4(mul_bf16x2(o->x, f2), mul_bf16x2(o->y, f2), mul_bf16x2(o->z, f2), mul_bf16x2(o->w, f2));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&raw_empty[rr.slot]);
          mbar_arrive(&full[rp.slot]);
        }
        rr.step();
        rp.step();
        return true;
      };
      for (; ok && w.valid; walk_next(a, w)) {
        if (!w.e.keys) continue;
        const int ahead = w.e.lw == 0 ? 2 : 1;
        const int T = w.t1 - w.t0;
        // the row's page two tiles ahead and its scale bytes one tile ahead of the conversion
        // of K, so that neither load's latency is waited for; a V byte waits (in `vq`, oldest
        // lowest) for its tile's turn
        const int32_t *table = a.page_table + static_cast<size_t>(w.b) * a.max_pages;
        auto page_of = [&](int k) -> int {
          const int pos = tile_base(w.e, w.t0 + k) + r;
          if (k >= T || pos > w.e.p_hi) return -1;
          const int page = table[pos >> a.lg_page];
          return page >= 0 && page < a.n_pages ? page : -1;
        };
        auto scales_of = [&](int k, int page, uint32_t &ks, uint32_t &vs) {
          ks = vs = 127;
          if (page < 0) return;
          const size_t at = (static_cast<size_t>(page) * a.page_size +
                             ((tile_base(w.e, w.t0 + k) + r) & (a.page_size - 1))) * a.H_kv + w.g;
          ks = a.k_scale[at];
          vs = a.v_scale[at];
        };
        int front = 0, nv = 0;
        uint32_t ks, vs, vq = 0;
        int page = page_of(0);
        int page_next = page_of(1);
        scales_of(0, page, ks, vs);
        auto convert_k = [&]() -> bool {
          uint32_t ks1, vs1;
          scales_of(front + 1, page_next, ks1, vs1);
          page_next = page_of(front + 2);
          if (!convert(front, ks)) return false;
          vq |= vs << (8 * nv++);
          ks = ks1;
          vs = vs1;
          ++front;
          return true;
        };
        for (int k = 0; ok && k < min(ahead, T); ++k) ok = convert_k();
        for (int k = 0; ok && k < T; ++k) {
          ok = convert(k, vq & 0xffu);
          vq >>= 8;
          --nv;
          if (ok && k + ahead < T) ok = convert_k();
        }
        tile += T;
      }
    }
  } else {
    // ---------------------------------------------------------------- warps 10, 11: cleaners
    // value rows that no row of the item sees are zeroed in their slot (the converters do it
    // for FP8 caches), 64 rows of every tile each
    reg_dec<C::kRegMisc>();
    if constexpr (!FP8) {
      Ring<C::kSlots> rp;
      Ring<C::kClean> rc;
      uint32_t tile = 0;
      bool ok = true;
      const int half = warp - 10;
      for (; ok && w.valid; walk_next(a, w)) {
        if (!w.e.keys) continue;
        const int ahead = w.e.lw == 0 ? 2 : 1;
        const int T = w.t1 - w.t0;
        // Every slot is waited for and released, K tiles too: only who holds a slot back sees
        // each of its phases.
        auto next = [&]() -> bool { return warp_wait(&full[rp.slot], rp.phase, abort); };
        auto done = [&]() {
          if (lane == 0) mbar_arrive(&empty[rp.slot]);
          rp.step();
        };
        for (int k = 0; ok && k < min(ahead, T); ++k)
          if ((ok = next())) done();
        for (int k = 0; ok && k < T; ++k) {
          if (!(ok = next())) break;
          const uint2 seen = *reinterpret_cast<const uint2 *>(&meta[(tile + k) % kMetaRing].seen[2 * half]);
          if ((seen.x & seen.y) != 0xffffffffu) {
#pragma unroll 1
            for (int r = lane >> 3; r < kKeys / 2; r += 4)   // eight lanes per 128-byte row
              if (!(((r < 32 ? seen.x : seen.y) >> (r & 31)) & 1u))
#pragma unroll
                for (int hh = 0; hh < C::kHalves; ++hh)
                  *reinterpret_cast<uint4 *>(sm + C::oRing + rp.slot * C::kTile + hh * C::kHalf +
                                             (64 * half + r) * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(&clean[rc.slot]);
          rc.step();
          done();
          if (k + ahead < T && (ok = next())) done();
        }
        tile += T;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    if (lane == 0) drain_wait(fin, 0, 1000000000ull);   // every MMA retired before TMEM is freed
    __syncwarp();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0 && *abort) atomicExch(&g_paged_error, 1);
}

// ------------------------------------------------------------------ merge

struct MergeArgs {
  const PagedPiece *piece;
  const float *part, *part_ml;
  uint16_t *out;
  float *lse;
  int part_rows, H_q, G, TT;
};

constexpr int kMergeRows = 8;   // rows per CTA; a warp holds 4 groups of 4 dims of them

// CTA (c, y) merges rows 8 y .. of the item that share c begins and a boundary cuts: the
// pieces of shares c, c + 1, ... until the item ends, weighted by exp2(m - max m).  Lanes run
// over the rows first, so partials are read in whole lines.
template <int D>
__global__ void __launch_bounds__(D * 2) paged_merge_kernel(const MergeArgs a) {
  grid_dep_wait();
  const PagedPiece pc = a.piece[blockIdx.x];
  const int x = blockIdx.y * kMergeRows + (threadIdx.x & 7);
  if (!pc.valid || static_cast<int>(blockIdx.y) * kMergeRows >= pc.ntok * a.G) return;
  const bool in = x < pc.ntok * a.G;
  const int t = (in ? x : 0) / a.G, j = (in ? x : 0) - t * a.G;
  const int qt = t >= a.TT ? 1 : 0;
  const int prow = qt * kRows + (t - qt * a.TT) * a.G + j;
  const int c4 = threadIdx.x >> 3;
  const long long end = pc.item_u0 + (static_cast<long long>(pc.n) << pc.lw);
  // the shares of the item: blockIdx.x .. last
  const int c0 = blockIdx.x;
  int last = c0;
  while (last + 1 < pc.P && share_begin(pc.q, pc.r, last + 1) < end) ++last;
  auto slot_of = [&](int c) -> int {   // < 0: an empty piece
    int t0, t1;
    piece_of(share_begin(pc.q, pc.r, c), share_begin(pc.q, pc.r, c + 1), pc.item_u0, pc.n, pc.lw, t0, t1);
    return t1 > t0 ? 2 * c + (t0 == 0 ? 1 : 0) : -1;
  };
  const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml);
  const float4 *po = reinterpret_cast<const float4 *>(a.part);
  float M = -INFINITY;
#pragma unroll 4
  for (int c = c0; c <= last; ++c) {
    const int s = slot_of(c);
    if (s >= 0) M = fmaxf(M, ml[static_cast<size_t>(s) * a.part_rows + prow].x);
  }
  float L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = c0; c <= last; ++c) {
    const int s = slot_of(c);
    if (s < 0) continue;
    const float2 v = ml[static_cast<size_t>(s) * a.part_rows + prow];
    const float4 o = po[(static_cast<size_t>(s) * (D / 4) + c4) * a.part_rows + prow];
    if (v.x == -INFINITY) continue;
    const float f = fast_exp2(v.x - M);
    L = fmaf(v.y, f, L);
    acc.x = fmaf(o.x, f, acc.x);
    acc.y = fmaf(o.y, f, acc.y);
    acc.z = fmaf(o.z, f, acc.z);
    acc.w = fmaf(o.w, f, acc.w);
  }
  if (!in) return;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const size_t orow = static_cast<size_t>(pc.tok0 + t) * a.H_q + pc.g * a.G + j;
  uint2 w;
  w.x = L == 0.f ? 0u : pack_bf16x2(acc.x * inv, acc.y * inv);
  w.y = L == 0.f ? 0u : pack_bf16x2(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2 *>(a.out + orow * D + 4 * c4) = w;
  if (c4 == 0 && a.lse) a.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

// ------------------------------------------------------------------ host side

// [n_pages, page_size, H, D] codes, box = D x 1 head x rows x 1 page
bool make_code_map(CUtensorMap *m, const void *base, int D, int H, int S, int B, int rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(S),
                        static_cast<cuuint64_t>(B)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H) * D,
                           static_cast<cuuint64_t>(S) * H * D};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(D), 1, static_cast<cuuint32_t>(rows), 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [n_tok, H_q, D] queries with a token stride, box = 64 dims x G heads x TT tokens
bool make_query_map(CUtensorMap *m, const void *base, int D, int H, long long stride, int N, int G, int TT) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(N), 1};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(stride) * 2,
                           static_cast<cuuint64_t>(stride) * 2 * N};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(TT), 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool FP8>
cudaError_t launch_d(const PagedAttnArgs &pa, cudaStream_t s) {
  using C = Cfg<D, FP8>;
  Args a;
  std::memset(&a, 0, sizeof(a));
  const int G = pa.H_q / pa.H_kv, TT = kRows / G;
  const int R = std::min(pa.page_size, kKeys);
  const bool maps =
      make_query_map(&a.tq, pa.q, D, pa.H_q, pa.q_stride, pa.n_tok, G, TT) &&
      (FP8 ? make_code_map(&a.tk, pa.k_pages, D, pa.H_kv, pa.page_size, pa.n_pages, R) &&
                 make_code_map(&a.tv, pa.v_pages, D, pa.H_kv, pa.page_size, pa.n_pages, R)
           : make_bshd_map(&a.tk, pa.k_pages, D, pa.H_kv, pa.page_size, pa.n_pages, R) &&
                 make_bshd_map(&a.tv, pa.v_pages, D, pa.H_kv, pa.page_size, pa.n_pages, R));
  if (!maps) return cudaErrorInvalidValue;
  a.q_start = pa.q_start;
  a.kv_len = pa.kv_len;
  a.page_table = pa.page_table;
  a.k_scale = pa.k_scale;
  a.v_scale = pa.v_scale;
  a.out = pa.out;
  a.lse = pa.lse;
  a.part = pa.part;
  a.part_ml = pa.part_ml;
  a.piece = pa.piece;
  a.B = pa.B;
  a.n_tok = pa.n_tok;
  a.max_pages = pa.max_pages;
  a.n_pages = pa.n_pages;
  a.page_size = pa.page_size;
  while ((1 << a.lg_page) < pa.page_size) ++a.lg_page;
  a.H_q = pa.H_q;
  a.H_kv = pa.H_kv;
  a.G = G;
  a.TT = TT;
  a.part_rows = pa.part_rows;
  a.lg_min_units = 1;
  const int cap = pa.max_pages * pa.page_size;
  a.n_sink = std::min(pa.n_sink, cap);
  a.n_stream = pa.n_stream < 0 ? -1 : std::min(pa.n_stream, cap);
  a.sl2 = pa.scale * kLog2e;
  auto kern = paged_attn_kernel<D, FP8>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kBytes);
  if (e != cudaSuccess) return e;
  // the warpgroups' register shares add up to what the launch holds; a build that holds less
  // would wait for registers that no warp gives back
  static std::atomic<bool> regs_ok{false};
  if (!regs_ok) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    if (fa.numRegs != C::kRegLaunch) return cudaErrorInvalidKernelImage;
    regs_ok = true;
  }
  int dev = 0, sms = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  // no more CTAs than the launch can have shares of min_units
  const long long pairs = pa.B + pa.n_tok / (2 * TT);
  const long long most = pairs * pa.H_kv * 2 * ((cap + kKeys - 1) / kKeys + 1) / (1 << a.lg_min_units) + 1;
  const int P = static_cast<int>(std::min(static_cast<long long>(std::min(sms, kPagedMaxCtas)), most));
  {
    ProfScope ps(FP8 ? "paged_attn_fp8" : "paged_attn", s);
    e = launch_pdl(kern, dim3(P), dim3(C::kThreads), C::kBytes, s, a);
  }
  if (e != cudaSuccess) return e;
  MergeArgs ma;
  ma.piece = pa.piece;
  ma.part = pa.part;
  ma.part_ml = pa.part_ml;
  ma.out = pa.out;
  ma.lse = pa.lse;
  ma.part_rows = pa.part_rows;
  ma.H_q = pa.H_q;
  ma.G = G;
  ma.TT = TT;
  const int rows = std::min(2 * TT, pa.n_tok) * G;
  ProfScope ps("paged_attn_merge", s);
  return launch_pdl(paged_merge_kernel<D>, dim3(P, (rows + kMergeRows - 1) / kMergeRows), dim3(D * 2), 0, s, ma);
}

}  // namespace

// Rows of a partial: both query tiles, or only the rows a launch of few tokens can have.
int paged_part_rows(int n_tok, int G) {
  const int TT = kRows / G;
  return n_tok > TT ? 2 * kRows : ((n_tok * G + 3) & ~3);
}

int paged_attn_ready() {
  if (tensor_map_encoder() == nullptr)
    return fail(DSA_ERR_UNSUPPORTED, "the driver offers no cuTensorMapEncodeTiled entry point");
  return DSA_OK;
}

cudaError_t launch_paged_attn(const PagedAttnArgs &a, cudaStream_t s) {
  if (a.fp8) return a.D == 128 ? launch_d<128, true>(a, s) : launch_d<64, true>(a, s);
  return a.D == 128 ? launch_d<128, false>(a, s) : launch_d<64, false>(a, s);
}

int paged_attn_device_error() {
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_paged_error, sizeof(int)) != cudaSuccess) return -1;
  if (cudaMemcpyToSymbol(g_paged_error, &zero, sizeof(int)) != cudaSuccess) return -1;
  return v;
}

int paged_attn_set_wait_limit(unsigned long long ns) {
  return cudaMemcpyToSymbol(g_wait_limit_ns, &ns, sizeof(ns)) == cudaSuccess ? 0 : -1;
}

}  // namespace dsa
