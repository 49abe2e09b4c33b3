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
// tiles).  The items' key tiles of the whole launch, laid end to end and weighed by what they
// and the items take (kUnitsTwo and so on), are cut into equal shares, one per CTA (one CTA per
// SM): uneven lengths, one long context and many short ones all fill the GPU without a schedule
// made on the host, which knows no length.  A CTA finds its share from q_start and kv_len alone
// (one parallel pass over the sequences).  An item that a share boundary cuts leaves fp32
// partials (O, m, l) in the workspace, and a second kernel merges them.
//
// One CTA, two streams of scores (i = 0, 1), each with its own TMEM buffers S_i, O_i and its
// own four softmax warps, so that one stream's softmax runs while the tensor core works for
// the other:
//   two-tile items: stream i is query tile i, both see every key tile (256 rows per loaded
//     K/V tile);
//   one-tile items (a few tokens): both streams hold the same query tile and take the key
//     tiles alternately; the epilogue joins their halves.
// FP8 decode steps (FEW, a kernel of their own: items of at most 32 rows) hold the query rows four
// times in the tile, once in each softmax warp's TMEM lanes: each warp takes the exponentials of
// 32 of a tile's keys (one warp would take all of them otherwise) and P goes through shared memory
// (1M-key FP8 token: 556 us without, 485 with; 16 sequences of up to 32,768 FP8
// keys: 170 and 150, with 64-wide heads 152 and 127).  Chosen by the launch, not by the item: both in
// one kernel cost the larger items a tenth (mixed FP8 step 417 us against 378).
// Warps: 0-3 and 4-7 softmax of stream 0 and 1 (one thread per row), 8 producer (schedule and
// TMA), 9 and 10 MMA issuers of stream 0 and 1 (one issuer for both spent 1,800 clocks a turn
// on waits, 16 MMAs and commits against 1,024 in the tensor core), 11 cleaner (bf16 caches),
// 12-15 epilogue (results out of TMEM while the softmax warps are at the next item); FP8 caches
// add the converter warps 16-23, which widen the E4M3 tiles that TMA brings into a staging ring
// to bf16 operand tiles (exact: code * 2^e is a bf16), four warps the K tiles and four the V
// tiles.  The producer walks the share and hands out its items through a small ring, so that no
// other role holds that state: beside 224 KB of shared memory next to no L1 is left, and a
// spilled register costs a round trip to L2.  Every role is one compact loop: instruction
// fetches bound this kernel before its pipes do (with each role's code unrolled and inlined per
// case the FP8 cases took two to three times as long; an epilogue of 64 columns at a time in
// place of 32 cost the 8K window 159 -> 188 us, and 16 made the FP8 cases 4 % faster).
//
// What bounds it (one GB300, 6,773 GB/s and 1,849 TFLOP/s measured):
//   2,048 tokens against 131,072 bf16 keys, 32/8 heads of 128: 3.0 to 3.45 ms as the card's power
//     limit has it, 3.34 as a rule: 1,307 TFLOP/s, 71 % of the tensor core's burst and 79 % of its
//     sustained rate (in FP8 3.78 ms, 62 % of burst).  Beside
//     2,048 clocks of MMAs a turn of both streams takes 3,500: softmax and the two products of a
//     stream depend on one another, and 512 TMEM columns hold no third stream.
//   16 tokens over 284,580 bf16 keys in all: 180 to 186 us, 6,290 to 6,490 GB/s (93 to 96 %): HBM;
//     64-wide heads 125 us, 4,650 GB/s (69 %); in FP8 150 and 127 us, 3,920 and 2,330 GB/s.
//   one token over 1,048,576 FP8 keys: 485 to 506 us, 4,460 GB/s (66 %): the converters' chain (a tile
//     takes each of their warps 1,700 clocks of about 2,000; sixteen such warps with fewer
//     registers are slower, 538 us, and P from TMEM in place of shared memory changes nothing).
//   16 sequences, 5 prompts in progress and 11 decoding, 160,300 FP8 keys: 376 us, 829 TFLOP/s
//     (45 %): the softmax, which reads the scores twice.
//   8,192 tokens, window 1,024 and 256 first keys, bf16: 158 us, 1,004 TFLOP/s of the attended
//     pairs (54 %): ten key tiles an item, of which three are cut by the mask, and two more that
//     pass between two items (in FP8 206 us, 41 %).
//   one token over 2,048 keys: 15 us, a chain of latencies (share, page, Q and K, two products,
//     partials, merge) with 1.2 us of bytes in it.
//
//   S_i = Q_i K^T (M = N = 128, K = D), P over S_i (each 32 columns' P in the first 16),
//   O_i += P V.
// Each stream issues P V (tile t) and right behind it Q K^T (its next tile): S_i full then
// also says that P V before it has retired, so moving the softmax reference (O rescaled in
// TMEM) needs no wait of its own.  With 64-wide heads in bf16 (kEarly) P has columns of its own:
// Q K^T of the next tile goes out as soon as the softmax holds a tile's scores, and P V of the tile
// before is waited for before its O is scaled or its P written over (5,703 tokens of two prompts,
// 16 heads of 64: 78 -> 68 us; the softmax warps are then busy for 2,700 clocks of a 2,900-clock
// turn; in FP8, without that, 98.5 us).
//
// Softmax: the reference m follows the running maximum lazily, moving only when the maximum
// exceeds it by more than 2^kSlack; P <= 2^kSlack is rounded to bf16 for the tensor core
// (relative half step 2^-8 of each probability, as fine as the output's own rounding; fp16 would keep
// three bits more, but both operands of a product have one type, and values with their scale do
// not fit fp16), the row sum l adds the unrounded fp32 values, O accumulates in fp32.  Against
// float64 the results of normal inputs are off by 0.0019 to 0.0022 relative to their size, where
// the same formulas with P in fp32 and the one rounding of the result give 0.0017.  O is not divided
// by l before the end: values times 2^kSlack, summed over the keys, have to fit fp32.
//
// Keys that no row of the item sees (behind the sequence, before the window, bad pages) have
// their value rows zeroed, so whatever the pages hold there cannot reach the sums as 0 * NaN.
// Where some rows of an item see a key and others do not (tiles at the diagonal, at a window's
// edge), infinities and NaN in its value row are taken out as well, and the epilogue adds them to
// the rows that do see the key (add_lost).  Such tiles are searched for them as they arrive.
// Where a row's weight for a key that it sees underflows to 0, an infinity there comes out as NaN.
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
// The schedule's units are tenths of the time of a key tile of a two-tile item: that, a key tile
// of a one-tile item in bf16 (bound by its bytes) and FP8, what an item costs beside its tiles
// (the pipeline runs empty between two items, results leave), and the least that a share is worth
// cutting for.  With as many tiles for every CTA, whatever their items, CTAs took 296,000 to
// 491,000 clocks (7 to 39 items, 68 tiles, 8K window): 252 us against 163.  One-tile items' tiles, with
// 2 less, as they are and with 2 more, in us: mixed FP8 step of 32/8 heads of 128 510, 376, 399; 32/4
// heads 472, 339, 349; 8/8 heads 208, 173, 195; 64-wide 467, 343, 357; the same steps in bf16 494,
// 396, 336; 465, 347, 297; 221, 191, 177; 357, 282, 241 (bf16 tiles of long one-tile items cost nearer
// 9); 64-wide prompts 74, 68, 69.  An item at 10, 20 and 30: 8K window 169, 158, 159, with
// 64-wide heads 127, 119, 122, 64-wide prompts 71, 68, 69, the mixed steps within 1 %.
constexpr int kUnitsTwo = 10, kUnitsOne = 7, kUnitsOne8 = 6, kUnitsItem = 20, kUnitsMin = 24;
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;      // log2 units
constexpr uint64_t kWaitLimitNs = 500000000ull;

static __device__ int g_paged_error;   // sticky error word, read by dsa_device_error
std::atomic<unsigned long long> g_wait_limit_ns{kWaitLimitNs};   // of later launches

struct TileMeta {
  uint32_t seen[kKeys / 32];   // bit c: key c of the tile is in a good page and some row sees it
};

// A piece of the CTA's share: key tiles [t0, t0 + T) of one item (kinds: see Walk).
struct alignas(16) Item {
  int ns, w0;          // the entry's tiles: [0, ns), then from w0 on
  int t0, T;
  int tok0, ntok;      // first token row (global), tokens
  int p0, p_hi;        // positions of the first and the last token
  int b, g;            // sequence, KV head
  int flags;           // kSingle ...
};
constexpr int kItems = 4;      // pieces handed out ahead
constexpr int kLostRing = 2 * kItems;   // (an entry is cleared when its item before has left the epilogue)
constexpr int kSingle = 1;     // one query tile: both streams take turns over the key tiles
constexpr int kHasKeys = 2;    // some row sees a key
constexpr int kWhole = 4;      // every tile of the item: the result is final
constexpr int kStart = 8;      // the item's first tile
constexpr int kEnd = 16;       // no piece: the share is done
constexpr int kFewRows = 32;   // rows at most of a launch whose softmax warps share them (FEW)
constexpr uint32_t kFewTile = kFewRows * 128;   // bytes of them over 64 dims, or of their P over 64 keys

template <int D, bool FP8, bool FEW>
struct Cfg {
  static constexpr int kHalves = D / 64;                    // 128-byte column blocks of a bf16 tile
  static constexpr uint32_t kHalf = kKeys * 128;            // bytes of one of them (128 rows)
  static constexpr uint32_t kTile = kHalves * kHalf;        // a Q, K or V tile in bf16
  static constexpr uint32_t kRaw = kKeys * D;               // an FP8 tile
  // 64-wide heads leave TMEM columns for P beside S (bf16: each row's scores are in registers
  // then), so that Q K^T of a stream's next tile is issued before P V of the last.
  static constexpr bool kEarly = !FP8 && D == 64;
  static constexpr int kSlots = FP8 ? 3 : kEarly ? 8 : 5;   // operand ring (K and V tiles in order)
  // K tiles before the first V: items of one query tile, of two
  static constexpr int kAhead1 = kEarly ? 4 : 2, kAhead2 = kEarly ? 2 : 1;
  static constexpr int kRawSlots = FP8 ? 4 : 0;             // staging ring
  static constexpr int kClean = FP8 ? 0 : kEarly ? 8 : 4;   // value tiles cleaned ahead of their use
  static constexpr int kMetaRing = kEarly ? 16 : 8;         // tile descriptions: the rings run 8 or 5 ahead at most
  static constexpr int kSoft = 8;                           // softmax warps
  static constexpr int kEpi = kSoft + 4, kConv = kEpi + 4;  // first epilogue and converter warps
  static constexpr int kThreads = (kEpi + 4 + (FP8 ? 8 : 0)) * 32;
  // registers a thread after the split by warpgroup (softmax x 2, warps 8-11, epilogue,
  // converters x 2); what the launch holds, threads x kRegLaunch, is what the shares add up to
  static constexpr int kRegLaunch = FP8 ? 80 : 128;
  static constexpr int kRegSoft = FEW ? 80 : FP8 ? 104 : 176, kRegMisc = FP8 ? 64 : 72, kRegEpi = FP8 ? 64 : 88,
                       kRegConv = FEW ? 96 : FP8 ? 72 : 0;
  static_assert(256 * kRegSoft + 128 * kRegMisc + 128 * kRegEpi + 256 * kRegConv == kThreads * kRegLaunch,
                "register split");
  // Scores a thread holds at a time.  bf16: the whole row of the tile.  FP8: 32, read from TMEM
  // once for the maximum and again for P: the unrolled body beside the converters' did not
  // fit the instruction cache (3.3 of 10 stall cycles were instruction fetches; 64 at a time,
  // with the registers for it: mixed FP8 step 377 -> 391 us).
  static constexpr int kPart = FP8 ? 32 : 128;
  static constexpr uint32_t oQ = 0;
  static constexpr uint32_t oRing = oQ + 2 * kTile;
  static constexpr uint32_t oRaw = oRing + kSlots * kTile;
  static constexpr uint32_t oMeta = oRaw + kRawSlots * kRaw;
  static constexpr uint32_t oMl = oMeta + kMetaRing * sizeof(TileMeta);   // [2 streams][128 rows] (m, l)
  static constexpr uint32_t oItem = oMl + 2 * kRows * 8;
  static constexpr uint32_t oBar = oItem + kItems * sizeof(Item);
  // q_full, q_empty, slot full/empty, raw full/empty, then for both streams s_full, p_full,
  // o_final, ml_full, drained, turn; fin, clean, item full/empty, maxed, s_free, o_done
  static constexpr int kBars = 2 + 2 * kSlots + 2 * kRawSlots + 12 + 1 + kClean + 2 * kItems + 6;
  static constexpr int kReaders = kSoft + 2 + 4 + (FP8 ? 8 : 1);   // warps that read each item (not the producer)
  static constexpr uint32_t oMisc = oBar + kBars * 8;
  // FEW, in the space of the second query tile: P of both streams (rows of 64 keys,
  // [stream][half]); and the warps' maxima [stream][2][4 warps][32 rows]
  static constexpr uint32_t oP = oQ + kTile;
  static constexpr uint32_t oLost = oMisc + 16;             // by item: something was taken out of its values
  static constexpr uint32_t oMax = D == 128 ? oP + 4 * kFewTile : oLost + 4 * kLostRing;
  static constexpr uint32_t kBytes = oLost + 4 * kLostRing + (FEW && D != 128 ? 2048 : 0);
  static constexpr uint32_t cS = 0, cO = 2 * kKeys, cP = cO + 2 * D;   // TMEM columns: S_0, S_1 | O_0, O_1 | kEarly: P_0, P_1
  static_assert(cP + (kEarly ? kKeys : 0) <= kTmemCols, "TMEM columns");
  static_assert(kBytes <= 227 * 1024, "shared memory");
  static_assert(kSlots * kTile >= 4096 * 8, "planning scratch");
  static_assert(kRawSlots <= 2 * kSlots, "converters tell a slot's last two uses apart by parity");
};

struct Args {
  CUtensorMap tq, tk, tv;
  const void *v_pages;   // for add_lost
  const int32_t *q_start, *kv_len, *page_table;
  const uint8_t *k_scale, *v_scale;
  uint16_t *out;
  float *lse;
  float *part;           // [2 * max_ctas][D / 4][part_rows][4]
  float *part_ml;        // [2 * max_ctas][part_rows][2]
  PagedPiece *piece;     // [max_ctas]
  int B, n_tok, max_pages, n_pages, page_size, lg_page, H_q, H_kv, G, TT;
  int TE;                // tokens of an entry: two query tiles' (FEW: one's)
  int part_rows;
  int n_sink, n_stream;  // n_stream < 0: no window
  float sl2;
  uint32_t wait_clocks;  // limit of a wait
};

// ------------------------------------------------------------------ schedule

// Keys and tiles of the entry (sequence b, pair m of query tiles), the same for every KV head.
struct Entry {
  int tok0, ntok;      // first token row (global), tokens
  int p0;              // position of the first token
  int p_hi;            // position of the last one (< 0: no row sees a key)
  int ns, w0;          // tiles [0, ns), then [w0, w0 + n - ns)
  int n;               // tiles (at least 1: an entry without keys still writes its rows)
  int u;               // schedule units of a tile
  bool one;            // one query tile
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
  return (s.nq + a.TE - 1) / a.TE;
}

__device__ __forceinline__ Entry make_entry(const Args &a, const Seq &s, int m) {
  Entry e;
  e.tok0 = s.qs + m * a.TE;
  e.ntok = min(a.TE, s.nq - m * a.TE);
  e.p0 = s.kv - s.nq + m * a.TE;
  e.p_hi = e.p0 + e.ntok - 1;
  e.one = e.ntok <= a.TT;
  e.u = !e.one ? kUnitsTwo : a.k_scale ? kUnitsOne8 : kUnitsOne;
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

// What a CTA's planning leaves for its producer: the share [u0, u1), the item it begins in (first
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

// Schedule units of an item of n tiles of u units: what it costs beside its tiles, then those.
__device__ __forceinline__ long long units_of(int n, int u) { return kUnitsItem + static_cast<long long>(n) * u; }

// tiles [t0, t1) of an item (its units from item_u0 on) in the share [u0, u1)
__device__ __forceinline__ void piece_of(long long u0, long long u1, long long item_u0, int n, int u, int &t0,
                                         int &t1) {
  auto tile = [&](long long x) -> int {   // at most 2^23 tiles of 10 units: 32 bits
    x = min(max(x - item_u0 - kUnitsItem, 0ll), static_cast<long long>(n) * u);
    return static_cast<int>(static_cast<uint32_t>(x) / static_cast<uint32_t>(u));
  };
  t0 = tile(u0);
  t1 = tile(u1);
}

// the first non-empty piece at or after the current item
__device__ __forceinline__ void walk_settle(const Args &a, Walk &w) {
  while (true) {
    w.valid = w.item_u0 < w.u1;
    if (!w.valid) return;
    piece_of(w.u0, w.u1, w.item_u0, w.e.n, w.e.u, w.t0, w.t1);
    if (w.t1 > w.t0) return;
    w.item_u0 += units_of(w.e.n, w.e.u);
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
  w.u0 = max(w.u0, w.item_u0 + units_of(w.e.n, w.e.u));   // this item is done
  walk_settle(a, w);
}

// first key of tile k of a piece
__device__ __forceinline__ int tile_base(const Item &it, int k) {
  const int t = it.t0 + k;
  return (t < it.ns ? t : it.w0 + t - it.ns) * kKeys;
}

// ------------------------------------------------------------------ waits

// What bounds the waits of a CTA: a word set once one gave up, and the limit in clocks.
struct WaitCtl {
  volatile int *abort;
  uint32_t limit, soon;   // the word is looked at after `soon` clocks
};
__device__ __forceinline__ uint32_t clock_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%clock;\n" : "=r"(t));
  return t;
}

__device__ __forceinline__ bool mbar_test_wait(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// The whole warp waits; the outcome is warp-uniform.  Every lane asks, without a time hint: the
// hardware then holds the warp until the phase completes (or a limit of its own passes).  One
// lane polling, or hints, cost the other roles issue slots and woke late: 128K chunk 3.57 ->
// 3.89 ms, and up to 5.5 with long hints.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const WaitCtl &w) {
  if (__all_sync(kFull, mbar_test_wait(bar, parity))) return true;
  const uint32_t t0 = clock_lo();
  do {
    const uint32_t t = clock_lo() - t0;
    if (__any_sync(kFull, t > w.soon) && __any_sync(kFull, t > w.limit || *w.abort)) {
      *w.abort = 1;
      return false;
    }
  } while (!__all_sync(kFull, mbar_try_wait(bar, parity)));
  return true;
}

// The same for what takes a whole piece of T key tiles: T limits more.
__device__ __forceinline__ bool warp_wait_piece(uint64_t *bar, uint32_t parity, const WaitCtl &w, int T) {
  uint32_t t0 = clock_lo();
  while (!__all_sync(kFull, mbar_try_wait(bar, parity))) {
    const uint32_t t = clock_lo() - t0;
    if (!__any_sync(kFull, t > w.soon)) continue;
    const bool over = __any_sync(kFull, t > w.limit);
    if ((over && T-- <= 0) || __any_sync(kFull, *w.abort)) {
      *w.abort = 1;
      return false;
    }
    if (over) t0 = clock_lo();
  }
  return true;
}

__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_ns() - t0 > limit_ns) return;
}

// The tensor-core instructions of the MMA warp, executed by the whole warp with the leader's
// predicate inside: the warp stays converged, so descriptors and addresses live in uniform
// registers.  (In a branch that only lane 0 takes, every operand is moved there first, about
// 125 clocks an instruction against the 64 that the tensor core needs for it.)
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
// arrive on `bar` when every tensor-core instruction issued so far has completed
__device__ __forceinline__ void commit_if(uint32_t pred, uint64_t *bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"(pred)
      : "memory");
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
// three integer operations for two codes, one of which can run as a multiply on the FMA pipe (the
// ALU pipe, at half rate, is the busiest one of the FP8 launches, at 48 %; what bounds the long token
// is the chain of waits around this).
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

// ------------------------------------------------------------------ infinities and NaN

// Every row of the item sees every key of the tile that begins at `base` (bad pages aside).
__device__ __forceinline__ bool seen_by_all(const Args &a, const Item &it, int base) {
  return base + kKeys - 1 <= it.p0 &&
         (a.n_stream < 0 || base > it.p_hi - a.n_stream || base + kKeys <= a.n_sink);
}

// 16-bit halves of `w` that are infinite or NaN in bf16 as masks
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return __vcmpgeu2(w & 0x7fff7fffu, 0x7f807f80u); }

// What was taken out of a value tile (see the cleaner and the converters) goes to those of the
// warp's n_rows rows, from row `first` of stream i's query tile on, that see it, as with a positive
// weight: an infinity stays one of its sign, and opposite ones or a NaN make a NaN.
// add(row - first, token, column, value) adds to a row's result or partial; a column's lane is
// the same for every key.
template <int D, bool FP8, class Add>
__device__ __forceinline__ void add_lost(const Args &a, const Item &it, int first, int n_rows, int i, Add add) {
  const int lane = threadIdx.x & 31;
  const int32_t *table = a.page_table + static_cast<size_t>(it.b) * a.max_pages;
  const int col = (lane % (D / 4)) * 4;
#pragma unroll 1
  for (int k = 0; k < it.T; ++k) {
    const int base = tile_base(it, k);
    if (seen_by_all(a, it, base)) continue;
#pragma unroll 1
    for (int j = base; j < min(base + kKeys, it.p_hi + 1); ++j) {
      const int page = table[j >> a.lg_page];
      if (page < 0 || page >= a.n_pages) continue;
      const size_t r = ((static_cast<size_t>(page) << a.lg_page) + (j & (a.page_size - 1))) * a.H_kv + it.g;
      uint2 v;
      if constexpr (FP8) {
        const uint32_t sb = a.v_scale[r];
        v.x = v.y = sb == 255u ? 0x7fff7fffu : 0u;
        if (sb > 246u && sb != 255u) {                // larger codes are infinite in bf16: 2^7 first, then the rest
          const uint32_t f2 = ((sb - 7u) << 7) * 0x00010001u;
          v = widen4(*reinterpret_cast<const uint32_t *>(static_cast<const uint8_t *>(a.v_pages) + r * D + col), 0x7f007f00u);
          v.x = mul_bf16x2(v.x, f2);
          v.y = mul_bf16x2(v.y, f2);
        }
      } else v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.v_pages) + r * D + col);
      if (!__any_sync(kFull, not_finite(v.x) | not_finite(v.y))) continue;
#pragma unroll 1
      for (int row = 0; row < n_rows; ++row) {
        const int tok = (first + row) / a.G + i * a.TT, p = it.p0 + tok;
        if ((first + row) / a.G >= a.TT || tok >= it.ntok) continue;
        if (j > p || !(a.n_stream < 0 || j > p - a.n_stream || j < a.n_sink)) continue;
        if (lane >= D / 4) continue;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          const uint32_t x = (q < 2 ? v.x : v.y) >> (16 * (q & 1));
          if (not_finite(x) & 0xffffu) add(row, tok, col + q, bf16_lo(x));
        }
      }
    }
  }
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
// a share below, at or above what the launch holds
template <int N, int kLaunch>
__device__ __forceinline__ void reg_set() {
  if constexpr (N > kLaunch) reg_inc<N>();
  else if constexpr (N < kLaunch) reg_dec<N>();
}

template <int D, bool FP8, bool FEW>
__global__ void __launch_bounds__(Cfg<D, FP8, FEW>::kThreads, 1) paged_attn_kernel(const __grid_constant__ Args a) {
  using C = Cfg<D, FP8, FEW>;
  extern __shared__ __align__(1024) unsigned char sm[];
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + C::oBar);
  uint64_t *q_full = bars, *q_empty = bars + 1;
  uint64_t *full = bars + 2, *empty = full + C::kSlots;
  uint64_t *raw_full = empty + C::kSlots, *raw_empty = raw_full + C::kRawSlots;
  uint64_t *s_full = raw_empty + C::kRawSlots, *p_full = s_full + 2, *o_final = p_full + 2;
  uint64_t *ml_full = o_final + 2, *drained = ml_full + 2, *turn = drained + 2, *fin = turn + 2;
  uint64_t *clean = fin + 1, *item_full = clean + C::kClean, *item_empty = item_full + kItems;
  uint64_t *maxed = item_empty + kItems, *s_free = maxed + 2, *o_done = s_free + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::oMisc);
  const WaitCtl abort{reinterpret_cast<volatile int *>(sm + C::oMisc + 4), a.wait_clocks, min(a.wait_clocks, 100000u)};
  Plan *plan = reinterpret_cast<Plan *>(sm + C::oMl);   // read before the first piece is handed out
  TileMeta *meta = reinterpret_cast<TileMeta *>(sm + C::oMeta);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(sm) & 1023u) {   // the swizzled tiles need 1024-byte atoms
    if (tid == 0) atomicExch(&g_paged_error, 1);
    return;
  }

  if (tid == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&full[i], FP8 ? 4 : 1);
      mbar_init(&empty[i], FP8 ? 2 : 3);   // both MMA issuers; bf16: and the cleaner
    }
    for (int i = 0; i < C::kRawSlots; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_final[i], 1);
      mbar_init(&ml_full[i], 4);
      mbar_init(&drained[i], 4);
      mbar_init(&turn[i], 1);
      mbar_init(&maxed[i], 4);
      mbar_init(&s_free[i], 4);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(fin, 2);
    for (int i = 0; i < C::kClean; ++i) mbar_init(&clean[i], 1);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], C::kReaders);
    }
    *abort.abort = 0;
    fence_mbar_init();
  }
  if (warp == C::kSoft + 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  grid_dep_wait();
  grid_dep_release();

  // ---------------------------------------------------------------- this CTA's share
  // units of every sequence (in the still unused ring), their running sum, and the item in
  // which the share begins
  {
    long long *su = reinterpret_cast<long long *>(sm + C::oRing);   // [B]
    for (int b0 = 0; b0 < a.B; b0 += C::kThreads) {
      const int b = b0 + tid;
      long long u = 0;
      bool many = false;
      if (b < a.B) {
        const Seq s = load_seq(a, b);
        many = s.nq > a.TE;
        if (!many && s.nq > 0) {
          const Entry e = make_entry(a, s, 0);
          u = units_of(e.n, e.u) * a.H_kv;
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
          x += units_of(e.n, e.u);
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
      // shares: at least kUnitsMin each, so that a short launch is not cut finer than pays
      const long long total = run;
      const int P = static_cast<int>(min(static_cast<long long>(gridDim.x), max(1ll, total / kUnitsMin)));
      // total / P digit by digit (total < 2^47: 4096 sequences of 2^23 tiles, 10 units, 128 heads
      // at most, and P < 2^16)
      const uint32_t up = static_cast<uint32_t>(P), high = static_cast<uint32_t>(total >> 16);
      const uint32_t mid = ((high % up) << 16) | static_cast<uint32_t>(total & 0xffff);
      const long long q = (static_cast<long long>(high / up) << 16) + mid / up;
      const int r = static_cast<int>(mid % up);
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
          uint32_t item = 0;   // units of one KV head: below 2^27
          if (mm < np) {
            const Entry e = make_entry(a, s, mm);
            item = static_cast<uint32_t>(units_of(e.n, e.u));
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
            for (int x = 64; x > 0; x >>= 1)            // (u0 - base) / item, below H_kv <= 128
              if (static_cast<long long>(item) * (g + x) <= u0 - base) g += x;
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
  Item *items = reinterpret_cast<Item *>(sm + C::oItem);
  volatile int *lost = reinterpret_cast<volatile int *>(sm + C::oLost);
  // Readers of the item ring: the next piece into `it` (a copy), false at the end
  Ring<kItems> ri;
  int lost_at = 0;                                    // the piece's entry of `lost`
  auto next_item = [&](Item &it) -> bool {
    if (!warp_wait(&item_full[ri.slot], ri.phase, abort)) return false;
    it = items[ri.slot];
    lost_at = ri.slot + (ri.phase ? kItems : 0);
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[ri.slot]);
    ri.step();
    return !(it.flags & kEnd);
  };

  if (warp < C::kSoft) {
    // ---------------------------------------------------------------- softmax
    reg_set<C::kRegSoft, C::kRegLaunch>();
    const int i = warp >> 2;                          // stream
    const int row = (warp & 3) * 32 + lane;           // row of the query tile
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_col = tl + C::cS + i * kKeys;
    const uint32_t o_col = tl + C::cO + i * D;
    float2 *ml = reinterpret_cast<float2 *>(sm + C::oMl) + i * kRows + row;
    uint32_t s_phase = 0, d_phase = 1, x_buf = 0;
    const uint32_t p_col = C::kEarly ? tl + C::cP + i * (kKeys / 2) : s_col;
    uint32_t tile = 0;                                // key tiles seen so far (meta ring)
    bool ok = true;
    // The piece is read from its ring entry as it is needed and given back at the end.
    for (;; ri.step()) {
      if (!ok || !(ok = warp_wait(&item_full[ri.slot], ri.phase, abort))) break;
      const Item &it = items[ri.slot];
      if (it.flags & kEnd) break;
      const bool single = FEW || (it.flags & kSingle), keys = it.flags & kHasKeys;
      // FEW: the rows lie in every warp's lanes (see the producer), and each warp takes 32 of
      // the keys.
      const int rtok = (FEW ? lane : row) / a.G;
      const int tok = rtok + (single ? 0 : i * a.TT); // token of the piece's entry
      const bool row_ok = rtok < a.TT && tok < it.ntok;
      const bool warp_ok = __any_sync(kFull, row_ok);
      const int p = it.p0 + (row_ok ? tok : it.ntok - 1);
      float m_ref = -INFINITY, l = 0.f;               // base-2 units
      if (keys) {
        const int first = single ? i : 0, step = single ? 2 : 1;
#pragma unroll 1
        for (int k = first; k < it.T; k += step) {   // (T and the tile's place: one broadcast load)
          ok = warp_wait(&s_full[i], s_phase, abort);
          if (!ok) break;
          s_phase ^= 1u;
          tc_fence_after();
          if (warp_ok) {
            const int base = tile_base(it, k);
            const uint4 seen = *reinterpret_cast<const uint4 *>(meta[(tile + k) % C::kMetaRing].seen);
            const int hi = p - base;                  // keys c <= hi are not after the row
            const int lo = a.n_stream < 0 ? 0 : p - a.n_stream + 1 - base;   // c >= lo: in its window
            const int sk = a.n_sink - base;           // c < sk: a first token
            const bool trim = __any_sync(kFull, hi < kKeys - 1 || (lo > 0 && sk < kKeys) ||
                                                    (seen.x & seen.y & seen.z & seen.w) != 0xffffffffu);
            // scores of part `part`, minus infinity where the row does not see the key
            uint32_t s[C::kPart];
            auto scores = [&](int part) {
#pragma unroll
              for (int c = 0; c < C::kPart; c += 32) tmem_ld32(s_col + C::kPart * part + c, s + c);
              tmem_wait_ld();
              if (trim) {
#pragma unroll
                for (int c = 0; c < C::kPart; c += 32) {
                  const int q = C::kPart / 32 * part + c / 32;   // which 32 keys of the tile
                  auto below = [&](int x) -> uint32_t {          // bits below x of them
                    const int y = x - 32 * q;
                    return y <= 0 ? 0u : (y >= 32 ? 0xffffffffu : (1u << y) - 1u);
                  };
                  const uint32_t sw = q == 0 ? seen.x : q == 1 ? seen.y : q == 2 ? seen.z : seen.w;
                  const uint32_t v = sw & below(hi + 1) & (~below(lo) | below(sk));
#pragma unroll
                  for (int x = 0; x < 32; ++x) s[c + x] = (v >> x) & 1u ? s[c + x] : __float_as_uint(-INFINITY);
                }
              }
            };
            constexpr int kParts = kKeys / C::kPart;
            const int part0 = FEW ? warp & 3 : 0, part1 = FEW ? part0 : kParts - 1;
            float mt = -INFINITY;
#pragma unroll 1
            for (int part = part0; part <= part1; ++part) {
              scores(part);
              float mx[4] = {mt, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int c = 0; c < C::kPart; c += 2)
                mx[(c >> 1) & 3] = fmax3(mx[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
              mt = fmax3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
            }
            if (FEW) {                                // the maximum over all four warps' keys
              float *x = reinterpret_cast<float *>(sm + C::oMax) + (2 * i + x_buf) * kRows;
              x[row] = mt;
              __syncwarp();
              if (lane == 0) mbar_arrive(&maxed[i]);
              if (!(ok = warp_wait(&maxed[i], x_buf, abort))) break;
              x_buf ^= 1u;                            // buffer and phase alike: the one before is read
              mt = fmax3(x[lane], x[lane + 32], fmaxf(x[lane + 64], x[lane + 96]));
            }
            if (C::kEarly) {
              // the scores are here: S may be filled again; and P V of the tile before, which may
              // still run, is waited for before its O is scaled or its P written over
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&s_free[i]);
              if (!(ok = warp_wait(&o_done[i], s_phase, abort))) break;
              tc_fence_after();
            }
            mt *= a.sl2;
            const bool move = mt > m_ref + kSlack;
            if (__any_sync(kFull, move)) {
              float f = 1.f;
              if (move) {
                f = m_ref == -INFINITY ? 0.f : fast_exp2(m_ref - mt);
                l *= f;
                m_ref = mt;
              }
              if (k > first && (!FEW || (warp & 3) == 0)) {   // O holds earlier tiles of this piece
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
#pragma unroll 1
            for (int part = part1; part >= part0; --part) {   // the last part is still here
              if (kParts > 1 && part < part1) scores(part);
#pragma unroll
              for (int c0 = 0; c0 < C::kPart; c0 += 32) {
                uint32_t pk[16];
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                  const float2 y = ffma2(make_float2(__uint_as_float(s[c0 + c]), __uint_as_float(s[c0 + c + 1])), sl22, nm2);
                  const float2 x = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                  if ((c >> 1) & 1) acc1 = fadd2(acc1, x);
                  else acc0 = fadd2(acc0, x);
                  pk[c >> 1] = pack_bf16x2(x.x, x.y);
                }
                if (FEW) {                            // 64 bytes of the row's 128 for these 64 keys
                  unsigned char *dst = sm + C::oP + (2 * i + (part >> 1)) * kFewTile + lane * 128;
#pragma unroll
                  for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<uint4 *>(dst + ((((part & 1) * 4 + q) ^ (lane & 7)) << 4)) =
                        make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
                  fence_proxy_async_smem();
                } else {
                  tmem_st16(C::kEarly ? p_col + c0 / 2 : s_col + C::kPart * part + c0, pk);
                }
              }
            }
            const float2 as = fadd2(acc0, acc1);
            l += as.x + as.y;
            tmem_wait_st();
          } else if (C::kEarly) {
            // (warps without rows keep step: they would be counted for two tiles of one phase)
            if (lane == 0) mbar_arrive(&s_free[i]);
            if (!(ok = warp_wait(&o_done[i], s_phase, abort))) break;
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[i]);
        }
        if (!ok) break;
        tile += it.T;
      }
      // (m, l) to the epilogue, once it has drained the piece before
      if (!(ok = warp_wait(&drained[i], d_phase, abort))) break;
      d_phase ^= 1u;
      *ml = make_float2(m_ref, l);
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ml_full[i]);
        mbar_arrive(&item_empty[ri.slot]);
      }
    }
  } else if (warp == C::kSoft) {
    // ---------------------------------------------------------------- producer
    reg_set<C::kRegMisc, C::kRegLaunch>();
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
    Item it;
    Walk w;
    w.u0 = plan->u0;
    w.u1 = plan->u1;
    w.item_u0 = plan->item_u0;
    w.b = plan->b;
    w.m = plan->m;
    w.g = plan->g;
    w.s = plan->s;
    w.valid = false;
    const long long plan_q = plan->q;
    const int plan_r = plan->r, plan_P = plan->P;
    if (lane == 0) a.piece[blockIdx.x].valid = 0;     // until this share begins a cut item
    if (w.u0 < w.u1 && w.b < a.B) {
      w.e = make_entry(a, w.s, w.m);
      walk_settle(a, w);
    }
    // the next piece of the share to every role (and into `it`); false at the end
    auto hand_out = [&]() -> bool {
      if (!(ok = warp_wait(&item_empty[ri.slot], ri.phase ^ 1u, abort))) return false;
      const bool start = w.t0 == 0, whole = start && w.t1 == w.e.n;
      it.tok0 = w.e.tok0;
      it.ntok = w.e.ntok;
      it.p0 = w.e.p0;
      it.p_hi = w.e.p_hi;
      it.ns = w.e.ns;
      it.w0 = w.e.w0;
      it.t0 = w.t0;
      it.T = w.t1 - w.t0;
      it.b = w.b;
      it.g = w.g;
      it.flags = !w.valid ? kEnd : (w.e.one ? kSingle : 0) | (w.e.keys ? kHasKeys : 0) | (whole ? kWhole : 0) |
                                       (start ? kStart : 0);
      if (lane == 0) {
        items[ri.slot] = it;
        lost[ri.slot + (ri.phase ? kItems : 0)] = 0;
        mbar_arrive(&item_full[ri.slot]);
        if (w.valid && start && !whole) {             // a cut item, described for the merge where it begins
          PagedPiece d;
          d.item_u0 = w.item_u0;
          d.q = plan_q;
          d.r = plan_r;
          d.P = plan_P;
          d.n = w.e.n;
          d.u = w.e.u;
          d.tok0 = w.e.tok0;
          d.ntok = w.e.ntok;
          d.g = w.g;
          d.valid = 1;
          a.piece[blockIdx.x] = d;
        }
      }
      __syncwarp();
      ri.step();
      return w.valid;
    };
    // lane x of `boxes` brings box x of a tile, of the part that lies in one page
    const int boxes = FP8 ? parts : parts * C::kHalves;
    const int part = FP8 ? lane : lane / C::kHalves, hh = FP8 ? 0 : lane - part * C::kHalves;
    for (; ok && hand_out(); walk_next(a, w)) {
      if (!(it.flags & kHasKeys)) continue;
      const bool single = FEW || (it.flags & kSingle);
      const int T = it.T;
      // the item's query tiles, once the MMAs of the one before have read theirs
      if (q_open) {
        ok = warp_wait(q_empty, q_phase, abort);
        if (!ok) break;
        q_phase ^= 1u;
      }
      q_open = true;
      if (lane == 0) {
        // two tiles, one, or a few rows into each softmax warp's lanes
        const int nt = FEW ? 4 : single ? 1 : 2;
        constexpr uint32_t kPitch = FEW ? kFewTile : C::kTile;
        mbar_arrive_expect_tx(q_full, static_cast<uint32_t>(nt * C::kHalves * a.TT * a.G * 128));
        for (int t = 0; t < nt; ++t)
          for (int hh = 0; hh < C::kHalves; ++hh)
            tma_load_4d(sm + C::oQ + t * kPitch + hh * C::kHalf, &a.tq, q_full, 64 * hh, it.g * a.G,
                        it.tok0 + (FEW ? 0 : t * a.TT), 0);
      }
      __syncwarp();
      const int32_t *table = a.page_table + static_cast<size_t>(it.b) * a.max_pages;
      // the page of this lane's part of tile k (n_pages: none, reads as zero)
      auto page_of = [&](int k) -> int {
        int page = a.n_pages;
        const int pos = tile_base(it, k) + part * R;
        if (k < T && part < parts && pos <= it.p_hi) {   // p_hi < capacity: inside the table
          page = table[pos >> a.lg_page];
          DSA_CHECK(page >= 0 && page < a.n_pages);
          if (page < 0 || page >= a.n_pages) page = a.n_pages;
        }
        return page;
      };
      int pg0 = a.n_pages, pg1 = pg0, pg2 = pg0, pg3 = pg0;   // pages of the last K tiles
      int page_next = page_of(0);
      const int ahead = single ? C::kAhead1 : C::kAhead2;   // K tiles in flight before the first V
      const int lo = a.n_stream < 0 ? 0 : a.n_stream == 0 ? 0x7fffffff : max(it.p0, 0) - a.n_stream + 1;
#pragma unroll 1
      for (int x = 0; ok && x < 2 * (T + ahead); ++x) {
        const bool value = !(x & 1);                  // V of tile x / 2 - ahead, then K of tile x / 2
        const int k = value ? (x >> 1) - ahead : x >> 1;
        if (k < 0 || k >= T) continue;
        const int base = tile_base(it, k);
        const int back = min((x >> 1) - 1, T - 1) - k;   // V: K tiles loaded since its own
        int page = back == 0 ? pg0 : !C::kEarly || back == 1 ? pg1 : back == 2 ? pg2 : pg3;
        if (!value) {
          page = page_next;
          page_next = page_of(k + 1);                 // requested meanwhile
          if (C::kEarly) {
            pg3 = pg2;
            pg2 = pg1;
          }
          pg1 = pg0;
          pg0 = page;
          // the tile's visible keys
          uint32_t *seen = meta[(tile + k) % C::kMetaRing].seen;
#pragma unroll
          for (int q = 0; q < kKeys / 32; ++q) {
            const int c = 32 * q + lane, j = base + c;
            const bool good = __shfl_sync(kFull, page, (c / R) * (FP8 ? 1 : C::kHalves)) != a.n_pages;
            const uint32_t v = __ballot_sync(kFull, good && j <= it.p_hi && (j >= lo || j < a.n_sink));
            if (lane == 0) seen[q] = v;
          }
        }
        if (!(ok = warp_wait(&re[rp.slot], rp.phase ^ 1u, abort))) break;
        unsigned char *dst = ring + rp.slot * kBytes;
        if (lane == 0) mbar_arrive_expect_tx(&rf[rp.slot], kBytes);
        __syncwarp();
        if (lane < boxes)
          tma_load_4d(dst + (FP8 ? part * R * D : hh * C::kHalf + part * R * 128), value ? &a.tv : &a.tk, &rf[rp.slot],
                      64 * hh, it.g, base & (a.page_size - 1) & ~(R - 1), page);
        __syncwarp();
        rp.step();
      }
      tile += T;
    }
    // every copy has landed before the CTA can exit, also when another role gave up
    if (lane == 0) {
      if (q_open) drain_wait(q_full, q_phase, 200000000ull);
      for (int s = 0; s < NS; ++s)
        // slots before rp.slot were last filled in this round, the others in the one before (or
        // never: that wait returns at once)
        drain_wait(&rf[s], s < rp.slot ? rp.phase : rp.phase ^ 1u, 200000000ull);
    }
    __syncwarp();
  } else if (warp <= C::kSoft + 2) {
    // ---------------------------------------------------------------- MMA issuers
    reg_set<C::kRegMisc, C::kRegLaunch>();
    constexpr uint32_t id_qk = idesc_bf16_f32(kRows, kKeys, false, false);
    constexpr uint32_t id_pv = idesc_bf16_f32(kRows, D, false, true);
    const int i = __shfl_sync(kFull, warp - C::kSoft - 1, 0);   // stream
    const uint32_t tm = __shfl_sync(kFull, tmem, 0);
    const uint32_t s_tm = tm + C::cS + i * kKeys, o_tm = tm + C::cO + i * D, p_tm = tm + C::cP + i * (kKeys / 2);
    // descriptors of the first tiles; the address field counts 16 bytes
    const uint64_t dq = sdesc_sw128(smem_u32(sm + C::oQ), 16, 1024);
    const uint64_t dk = sdesc_sw128(smem_u32(sm + C::oRing), 16, 1024);
    const uint64_t dv = sdesc_sw128(smem_u32(sm + C::oRing), C::kHalf, 1024);
    const uint64_t dp = sdesc_sw128(smem_u32(sm + C::oP + 2 * i * kFewTile), 16, 1024);
    const uint32_t leader = lane == 0 ? 1u : 0u;
    Ring<C::kSlots> rp;
    Ring<FP8 ? 1 : C::kClean> rc;
    uint32_t q_phase = 0, p_phase = 0, d_phase = 0, f_phase = 1, t_phase = i ^ 1;
    bool ok = true;
    // The streams take turns: P V and the Q K^T behind it of one, then of the other.  Left to
    // themselves they fall into step, and then share the tensor core during one half of the
    // time and the exponential unit during the other.
    auto take_turn = [&]() -> bool {
      if (!warp_wait(&turn[i], t_phase, abort)) return false;
      t_phase ^= 1u;
      return true;
    };
    auto pass_turn = [&]() {
      if (lane == 0) mbar_arrive(&turn[i ^ 1]);
      __syncwarp();
    };
    Item it;
    while (ok && next_item(it)) {
      // O_i of the piece before has been read (every piece is waited for, so that no phase is
      // missed)
      d_phase ^= 1u;
      const bool single = FEW || (it.flags & kSingle);
      const int T = it.T, ahead = single ? C::kAhead1 : C::kAhead2;
      if (!(it.flags & kHasKeys)) {
        ok = warp_wait(&drained[i], d_phase, abort);
        continue;
      }
      if (!(ok = warp_wait(q_full, q_phase, abort))) break;
      q_phase ^= 1u;
      const int last = single ? T - 1 - ((T - 1 - i) & 1) : T - 1;   // the stream's last key tile
      if (last < 0) {                                 // it has none: one key tile, stream 1
        ok = warp_wait(&drained[i], d_phase, abort);
        if (lane == 0) mbar_arrive(q_empty);
      }
      const uint64_t ad = dq + (single ? 0u : static_cast<uint32_t>(i)) * (C::kTile >> 4);
      // the slots in ring order (the producer's): P V of tile k, then Q K^T of the stream's next
#pragma unroll 1
      for (int x = 0; ok && x < 2 * (T + ahead); ++x) {
        const bool value = !(x & 1);
        const int k = value ? (x >> 1) - ahead : x >> 1;
        if (k < 0 || k >= T) continue;
        const int slot = __shfl_sync(kFull, rp.slot, 0);
        // a V tile is ready once filled and (bf16 caches) rid of rows that no row sees
        if (!FP8 && value) {
          ok = warp_wait(&clean[rc.slot], rc.phase, abort);
          rc.step();
        } else {
          ok = warp_wait(&full[slot], rp.phase, abort);
        }
        if (!ok) break;
        rp.step();
        if (single && ((k ^ i) & 1)) {                // the other stream's: only seen and given back
          if (lane == 0) mbar_arrive(&empty[slot]);
          __syncwarp();
          continue;
        }
        if (value) {
          const bool first = single ? k == i : k == 0;
          if (!(ok = warp_wait(&p_full[i], p_phase, abort))) break;
          p_phase ^= 1u;
          if (first && !(ok = warp_wait(&drained[i], d_phase, abort))) break;
          if (!C::kEarly && !(ok = take_turn())) break;
          tc_fence_after();
          const uint64_t bd = dv + static_cast<uint32_t>(slot) * (C::kTile >> 4);
          const uint32_t acc = first ? 0u : 1u;
          if (FEW) {
            // P in shared memory; the tile's rows behind kFewRows are whatever lies there, their
            // O is not read
#pragma unroll 2
            for (uint32_t kk = 0; kk < kKeys / 16; ++kk)
              mma_ss(leader, o_tm, dp + (kk >> 2) * (kFewTile >> 4) + (kk & 3) * 2, bd + kk * 128, id_pv,
                     kk > 0 ? 1u : acc);
          } else {
#pragma unroll
            for (uint32_t kk = 0; kk < kKeys / 16; ++kk)
              mma_ts(leader, o_tm, C::kEarly ? p_tm + kk * 8 : s_tm + (kk >> 1) * 32 + (kk & 1) * 8, bd + kk * 128, id_pv,
                     kk > 0 ? 1u : acc);
          }
          commit_if(leader, &empty[slot]);
          if (k == last) {
            if (FEW) commit_if(leader, q_empty);      // P lies in the second query tile's space
            commit_if(leader, &o_final[i]);
            if (!C::kEarly) pass_turn();
          }
          if (C::kEarly) commit_if(leader, &o_done[i]);
        } else {
          if (C::kEarly) {                            // the scores of the stream's tile before are read
            if (!(ok = warp_wait(&s_free[i], f_phase, abort))) break;
            f_phase ^= 1u;
          }
          tc_fence_after();
          const uint64_t bd = dk + static_cast<uint32_t>(slot) * (C::kTile >> 4);
#pragma unroll
          for (uint32_t kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * (C::kHalf >> 4) + (kk & 3) * 2;
            mma_ss(leader, s_tm, ad + off, bd + off, id_qk, kk > 0 ? 1u : 0u);
            // (the turn reaches the other issuer while the last ones run)
            if (!C::kEarly && kk == D / 16 - 2 && k >= ahead) pass_turn();
          }
          commit_if(leader, &s_full[i]);
          commit_if(leader, &empty[slot]);
          if (k == last && !FEW) commit_if(leader, q_empty);
        }
      }
      if (!C::kEarly && ok && single && i == 1 && (T & 1)) {        // stream 0 had one tile more
        ok = take_turn();
        pass_turn();
      }
    }
    commit_if(leader, fin);
    __syncwarp();
  } else if (warp >= C::kEpi && warp < C::kEpi + 4) {
    // ---------------------------------------------------------------- epilogue
    // O out of TMEM, normalised into out (or, of a cut item, as it is into the workspace)
    reg_set<C::kRegEpi, C::kRegLaunch>();
    const int row = (warp & 3) * 32 + lane;           // row of the query tile
    const uint32_t o_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + C::cO;
    const float2 *ml = reinterpret_cast<const float2 *>(sm + C::oMl) + row;
    const int rtok = row / a.G, rhead = row - rtok * a.G;
    uint32_t ml_phase = 0, of_phase[2] = {0, 0};
    bool ok = true;
    Item it;
    while (ok && next_item(it)) {
      const bool single = FEW || (it.flags & kSingle), keys = it.flags & kHasKeys, whole = it.flags & kWhole;
      const int slot = 2 * blockIdx.x + (it.flags & kStart ? 1 : 0);
      // (m, l) of stream i, and O_i complete; false: gave up
      auto wait_o = [&](int i, bool any) -> bool {
        if (!warp_wait_piece(&ml_full[i], ml_phase, abort, it.T)) return false;
        if (any) {
          if (!warp_wait(&o_final[i], of_phase[i], abort)) return false;
          of_phase[i] ^= 1u;
        }
        tc_fence_after();
        return true;
      };
#pragma unroll 1
      for (int i = 0; i < (single ? 1 : 2); ++i) {
        const int tok = rtok + i * a.TT;              // token of the piece's entry
        const bool row_ok = rtok < a.TT && tok < it.ntok;
        if (!(ok = wait_o(i, keys))) break;
        auto sum = [&](int s) -> float {              // (FEW: a sum per softmax warp, one reference)
          const float2 *x = ml + s * kRows;
          return FEW && warp == C::kEpi ? (x[0].y + x[32].y) + (x[64].y + x[96].y) : x[0].y;
        };
        float m = ml[i * kRows].x, l = sum(i), f0 = 1.f, f1 = 0.f;
        bool two = false;
        if (single) {                                 // the other half of the key tiles
          two = keys && it.T > 1;
          if (!(ok = wait_o(1, two))) break;
          const float2 o = make_float2(ml[kRows].x, sum(1));
          const float mm = fmaxf(m, o.x);
          f0 = m == -INFINITY ? 0.f : fast_exp2(m - mm);
          f1 = o.x == -INFINITY ? 0.f : fast_exp2(o.x - mm);
          l = l * f0 + o.y * f1;
          m = mm;
        }
        const float inv = whole ? (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) : 1.f;   // NaN stays NaN
        const float g0 = f0 * inv, g1 = f1 * inv;
        // A row of this piece is empty if its sum is 0: m cannot tell, fmax3 passes over NaN, and a
        // factor of 0 must reach O, where 0 * infinity or NaN is NaN (seen ones are never lost).
        const bool none = !keys || l == 0.f;
        const size_t orow = static_cast<size_t>(it.tok0 + tok) * a.H_q + it.g * a.G + rhead;
        const int prow = i * kRows + row;
        auto release = [&]() {                        // TMEM and (m, l) are read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&drained[i]);
            if (single) mbar_arrive(&drained[1]);
          }
        };
        if (!__any_sync(kFull, row_ok)) {
          release();
        } else {
          const uint32_t o_col = o_base + i * D;
          // 16 columns of O (the streams' halves merged, normalised if the result is final)
          auto columns = [&](int c, float *x) {
            uint32_t o[16];
            if (keys) tmem_ld16(o_col + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 16; q += 2) {
              const float2 y = fmul2(make_float2(__uint_as_float(o[q]), __uint_as_float(o[q + 1])), make_float2(g0, g0));
              x[q] = none ? 0.f : y.x;
              x[q + 1] = none ? 0.f : y.y;
            }
            if (two) {
              tmem_ld16(o_col + D + c, o);
              tmem_wait_ld();
              if (l != 0.f) {
#pragma unroll
                for (int q = 0; q < 16; ++q) x[q] = fmaf(__uint_as_float(o[q]), g1, x[q]);
              }
            }
          };
          const long long mine_row = row_ok ? static_cast<long long>(orow) : -1ll;
          const long long to0 = __shfl_sync(kFull, mine_row, lane & ~1), to1 = __shfl_sync(kFull, mine_row, lane | 1);
          float4 *dst = reinterpret_cast<float4 *>(a.part) + static_cast<size_t>(slot) * (D / 4) * a.part_rows + prow;
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float x[16];
            columns(c, x);
            if (c + 16 == D) release();               // the next item's P V need not wait for the stores
            if (whole) {
              uint4 y0 = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                    pack_bf16x2(x[6], x[7]));
              uint4 y1 = make_uint4(pack_bf16x2(x[8], x[9]), pack_bf16x2(x[10], x[11]), pack_bf16x2(x[12], x[13]),
                                    pack_bf16x2(x[14], x[15]));
              // two lanes exchange halves: each store then covers whole sectors of a row (-1: none)
              swap4(y0, y1, lane & 1, 1);
              if (to0 >= 0) *reinterpret_cast<uint4 *>(a.out + to0 * D + c + 8 * (lane & 1)) = y0;
              if (to1 >= 0) *reinterpret_cast<uint4 *>(a.out + to1 * D + c + 8 * (lane & 1)) = y1;
            } else if (row_ok) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                dst[static_cast<size_t>(c / 4 + q) * a.part_rows] =
                    make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
            }
          }
          if (keys && lost[lost_at]) {                // rare
            __syncwarp();                             // the stores above come first
            const int first = (warp & 3) * 32;
            const uint32_t empty = __ballot_sync(kFull, l == 0.f);   // (every score minus infinity)
            add_lost<D, FP8>(a, it, first, 32, i, [&](int r, int tok, int c, float v) {
              if (whole) {
                if ((empty >> r) & 1u) return;
                uint16_t *o = a.out + (static_cast<size_t>(it.tok0 + tok) * a.H_q + it.g * a.G + (first + r) % a.G) * D + c;
                *o = static_cast<uint16_t>(pack_bf16x2(bf16_lo(*o) + v, 0.f));
              } else {
                a.part[((static_cast<size_t>(slot) * (D / 4) + c / 4) * a.part_rows + i * kRows + first + r) * 4 + (c & 3)] += v;
              }
            });
          }
          if (row_ok) {
            if (!whole)
              reinterpret_cast<float2 *>(a.part_ml)[static_cast<size_t>(slot) * a.part_rows + prow] = make_float2(m, l);
            else if (a.lse)
              a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
          }
        }
      }
      ml_phase ^= 1u;
    }
  } else if (FP8 && warp >= C::kConv) {
    // ---------------------------------------------------------------- converters
    if constexpr (FP8) {
      reg_set<C::kRegConv, C::kRegLaunch>();
      Item it;
      const int r = (warp & 3) * 32 + lane;           // the thread's row of every tile
      const bool values = warp >= C::kConv + 4;       // V tiles, or K tiles
      Ring<C::kRawSlots> rr;
      Ring<C::kSlots> rp;
      uint32_t tile = 0;
      bool ok = true;
      auto skip = [&]() -> bool {
        if (!warp_wait(&raw_full[rr.slot], rr.phase, abort)) return false;
        if (lane == 0) mbar_arrive(&raw_empty[rr.slot]);
        rr.step();
        rp.step();
        return true;
      };
      // tile k (already described) with this row's scale byte sb
      auto convert = [&](int k, uint32_t sb_raw) -> bool {
        // (The tile's description came with its K tile, which a V converter has seen go by.  K
        // rows that no row sees need no zeroes: their scores are masked.)
        const bool seen = !values || ((meta[(tile + k) % C::kMetaRing].seen[r >> 5] >> (r & 31)) & 1u);
        const int sb = seen ? static_cast<int>(sb_raw) : 127;
        // 2^e as 2^(120 + e) on the raw bits (scales above 2^7: see below); a row that is not
        // seen is multiplied by 0, one with a NaN scale (255) by NaN
        const int e1 = min(sb - 127, 7), e2 = sb - 127 - e1;
        const uint32_t f = !seen ? 0u : sb == 255 ? 0x7fff7fffu : (static_cast<uint32_t>(e1 + 247) << 7) * 0x00010001u;
        // The tile has come; the operand slot's tile before, another warps' perhaps, has been filled
        // and given back.  Its filling is asked for as well, and in this order: every converter is
        // past the tile four back, or this one's staging slot would not be full, so the slot's use
        // two back has been filled, and a parity tells its last use from that one; once that is
        // filled the use two back has been given back, and the same holds for the release.
        uint64_t *w0 = &raw_full[rr.slot], *w1 = &full[rp.slot], *w2 = &empty[rp.slot];
        const uint32_t before = rp.phase ^ 1u;
        bool ready = mbar_test_wait(w0, rr.phase);
        ready &= mbar_test_wait(w1, before);
        ready &= mbar_test_wait(w2, before);
        if (!__all_sync(kFull, ready) && !(warp_wait(w0, rr.phase, abort) && warp_wait(w1, before, abort) &&
                                           warp_wait(w2, before, abort)))
          return false;
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
        constexpr int kAtOnce = FEW ? D / 16 : 2;     // loads in flight, as registers allow
#pragma unroll
        for (int p0 = 0; p0 < D / 16; p0 += kAtOnce) {
          uint4 c[kAtOnce];
#pragma unroll
          for (int p = 0; p < kAtOnce; ++p) c[p] = piece(p0 + p);
#pragma unroll
          for (int p = 0; p < kAtOnce; ++p) {
            const uint2 y0 = widen4(c[p].x, f), y1 = widen4(c[p].y, f);
            const uint2 y2 = widen4(c[p].z, f), y3 = widen4(c[p].w, f);
            put(2 * (p0 + p), make_uint4(y0.x, y0.y, y1.x, y1.y));
            put(2 * (p0 + p) + 1, make_uint4(y2.x, y2.y, y3.x, y3.y));
          }
        }
        if (__any_sync(kFull, seen && e2 > 0)) {
          // rare: a scale above 2^7 takes a second multiply, and values that are NaN then (255) or
          // infinite (above 246) and that not every row of the item sees are taken out (see add_lost)
          const uint32_t f2 = (static_cast<uint32_t>(e2 + 127) << 7) * 0x00010001u;
          const bool out = values && sb > 246 && !seen_by_all(a, it, tile_base(it, k));
#pragma unroll 1
          for (int q = 0; seen && e2 > 0 && q < D / 8; ++q) {
            uint4 *o = reinterpret_cast<uint4 *>(dst + (q >> 3) * C::kHalf + (((q & 7) ^ (r & 7)) << 4));
            uint4 u = make_uint4(mul_bf16x2(o->x, f2), mul_bf16x2(o->y, f2), mul_bf16x2(o->z, f2), mul_bf16x2(o->w, f2));
            if (out) {
              const uint4 n = make_uint4(not_finite(u.x), not_finite(u.y), not_finite(u.z), not_finite(u.w));
              if (n.x | n.y | n.z | n.w) lost[lost_at] = 1;
              u = make_uint4(u.x & ~n.x, u.y & ~n.y, u.z & ~n.z, u.w & ~n.w);
            }
            *o = u;
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
      while (ok && next_item(it)) {
        if (!(it.flags & kHasKeys)) continue;
        const int ahead = FEW || (it.flags & kSingle) ? C::kAhead1 : C::kAhead2;
        const int T = it.T;
        // the row's page two tiles ahead and its scale byte one tile ahead of the conversion,
        // so that neither load's latency is waited for
        const int32_t *table = a.page_table + static_cast<size_t>(it.b) * a.max_pages;
        const uint8_t *scales = values ? a.v_scale : a.k_scale;
        auto page_of = [&](int k) -> int {
          const int pos = tile_base(it, k) + r;
          return k < T && pos <= it.p_hi ? table[pos >> a.lg_page] : -1;   // checked when used
        };
        auto scale_of = [&](int k, int page) -> uint32_t {
          if (page < 0 || page >= a.n_pages) return 127;
          return scales[(static_cast<size_t>(page) * a.page_size + ((tile_base(it, k) + r) & (a.page_size - 1))) * a.H_kv +
                        it.g];
        };
        int page = page_of(0);
        int page_next = page_of(1);
        uint32_t sb = scale_of(0, page);
        int mine = 0;                                 // tiles of this warp's kind so far
        // one operand tile in ring order: this warp's kind is converted, the other kind's slots
        // are only seen and given back (see the cleaner)
        auto step = [&](bool value) -> bool {
          if (value != values) return skip();
          const uint32_t sb1 = scale_of(mine + 1, page_next);
          page_next = page_of(mine + 2);
          if (!convert(mine, sb)) return false;
          sb = sb1;
          ++mine;
          return true;
        };
#pragma unroll 1
        for (int x = 0; ok && x < 2 * (T + ahead); ++x) {   // the producer's order
          const int k = x & 1 ? x >> 1 : (x >> 1) - ahead;
          if (k >= 0 && k < T) ok = step(!(x & 1));
        }
        tile += T;
      }
    }
  } else {
    // ---------------------------------------------------------------- cleaner
    // value rows that no row of the item sees are zeroed in their slot, infinities and NaN of tiles
    // that the mask cuts taken out (the converters do both for FP8 caches)
    reg_set<C::kRegMisc, C::kRegLaunch>();
    if constexpr (!FP8) {
      Ring<C::kSlots> rp;
      Ring<C::kClean> rc;
      uint32_t tile = 0;
      bool ok = true;
      Item it;
      while (ok && next_item(it)) {
        if (!(it.flags & kHasKeys)) continue;
        const int ahead = FEW || (it.flags & kSingle) ? C::kAhead1 : C::kAhead2;
        // Every slot is waited for and released, K tiles too: only who holds a slot back sees
        // each of its phases.
#pragma unroll 1
        for (int x = 0; x < 2 * (it.T + ahead); ++x) {   // the producer's order
          const bool value = !(x & 1);
          const int k = value ? (x >> 1) - ahead : x >> 1;
          if (k < 0 || k >= it.T) continue;
          if (!(ok = warp_wait(&full[rp.slot], rp.phase, abort))) break;
          if (value) {
            unsigned char *v = sm + C::oRing + rp.slot * C::kTile;
            const uint4 s4 = *reinterpret_cast<const uint4 *>(meta[(tile + k) % C::kMetaRing].seen);
            if ((s4.x & s4.y & s4.z & s4.w) != 0xffffffffu) {
              const int at = lane >> 3;               // eight lanes per 128-byte row
#pragma unroll 1
              for (int r0 = 0; r0 < kKeys; r0 += 32) {
                const uint32_t sw = r0 == 0 ? s4.x : r0 == 32 ? s4.y : r0 == 64 ? s4.z : s4.w;
                if (sw == 0xffffffffu) continue;
#pragma unroll 1
                for (int r = 0; r < 32; r += 4)
                  if (!((sw >> (r + at)) & 1u))
#pragma unroll
                    for (int hh = 0; hh < C::kHalves; ++hh)
                      *reinterpret_cast<uint4 *>(v + hh * C::kHalf + (r0 + r + at) * 128 + (lane & 7) * 16) =
                          make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
            if (!seen_by_all(a, it, tile_base(it, k))) {
              uint4 *w = reinterpret_cast<uint4 *>(v);
              constexpr uint32_t kMag = 0x7fff7fffu;
              uint32_t m = 0;                         // largest magnitudes of both halves
#pragma unroll 4
              for (uint32_t x = lane; x < C::kTile / 16; x += 32) {
                const uint4 u = w[x];
                m = __vmaxu2(m, __vmaxu2(__vmaxu2(u.x & kMag, u.y & kMag), __vmaxu2(u.z & kMag, u.w & kMag)));
              }
              if (__any_sync(kFull, not_finite(m))) {   // rare
#pragma unroll 1
                for (uint32_t x = lane; x < C::kTile / 16; x += 32) {
                  const uint4 u = w[x];
                  w[x] = make_uint4(u.x & ~not_finite(u.x), u.y & ~not_finite(u.y), u.z & ~not_finite(u.z),
                                    u.w & ~not_finite(u.w));
                }
                lost[lost_at] = 1;
                fence_proxy_async_smem();
                __syncwarp();
              }
            }
            if (lane == 0) mbar_arrive(&clean[rc.slot]);
            rc.step();
          }
          if (lane == 0) mbar_arrive(&empty[rp.slot]);
          rp.step();
        }
        tile += it.T;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kSoft + 1) {
    tc_fence_after();
    if (lane == 0) drain_wait(fin, 0, 1000000000ull);   // every MMA retired before TMEM is freed
    __syncwarp();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0 && *abort.abort) atomicExch(&g_paged_error, 1);
}

// ------------------------------------------------------------------ merge

struct MergeArgs {
  const PagedPiece *piece;
  const float *part, *part_ml;
  uint16_t *out;
  float *lse;
  int part_rows, H_q, G, TT;
};

constexpr int kMergeWarps = 8;

// CTA (c, y) merges rows of the item that share c begins and a boundary cuts, a row per warp at
// a time: the pieces of shares c, c + 1, ... until the item ends, weighted by exp2(m - max m).
// Each lane fetches one piece's (m, l), so that all weights of a row cost one round of loads;
// then D / 4 lanes add up the pieces' O (with D = 64 the half-warps take alternate pieces).
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) paged_merge_kernel(const MergeArgs a) {
  const int lane = threadIdx.x & 31;
  grid_dep_wait();
  const PagedPiece pc = a.piece[blockIdx.x];
  if (!pc.valid) return;
  const long long end = pc.item_u0 + units_of(pc.n, pc.u);
  const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml);
  const float4 *po = reinterpret_cast<const float4 *>(a.part);
  constexpr int kStep = 128 / D;                      // pieces added per step
  const int c4 = lane % (D / 4), odd = lane / (D / 4);
  for (int x = blockIdx.y * kMergeWarps + (threadIdx.x >> 5); x < pc.ntok * a.G; x += gridDim.y * kMergeWarps) {
    const int t = x / a.G, j = x - t * a.G;
    const int qt = t >= a.TT ? 1 : 0;
    const int prow = qt * kRows + (t - qt * a.TT) * a.G + j;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int c0 = blockIdx.x; c0 < pc.P; c0 += 32) {   // 32 shares at a time
      const int c = c0 + lane;
      int slot = -1;                                  // this lane's share has no piece
      if (c < pc.P && share_begin(pc.q, pc.r, c) < end) {
        int t0, t1;
        piece_of(share_begin(pc.q, pc.r, c), share_begin(pc.q, pc.r, c + 1), pc.item_u0, pc.n, pc.u, t0, t1);
        if (t1 > t0) slot = 2 * c + (t0 == 0 ? 1 : 0);
      }
      const uint32_t have = __ballot_sync(kFull, slot >= 0);
      if (!have) break;
      const float2 v = slot >= 0 ? ml[static_cast<size_t>(slot) * a.part_rows + prow] : make_float2(-INFINITY, 0.f);
      const float m = fmaxf(M, warp_max(v.x));
      const float old = M == -INFINITY ? 0.f : fast_exp2(M - m);
      const float w = v.x == -INFINITY ? 0.f : fast_exp2(v.x - m);   // 0 for a piece without keys
      L = L * old + warp_sum(v.y * w);
      acc.x *= old;
      acc.y *= old;
      acc.z *= old;
      acc.w *= old;
      M = m;
      const int n = 32 - __clz(have);                 // shares of an item lie side by side
#pragma unroll 4
      for (int p = 0; p < n; p += kStep) {
        const int src = (p + odd) & 31;
        const float f = __shfl_sync(kFull, w, src);
        const int s = __shfl_sync(kFull, slot, src);
        if (p + odd < n && s >= 0) {                  // (f may be 0: infinities and NaN still count)
          const float4 o = po[(static_cast<size_t>(s) * (D / 4) + c4) * a.part_rows + prow];
          acc.x = fmaf(o.x, f, acc.x);
          acc.y = fmaf(o.y, f, acc.y);
          acc.z = fmaf(o.z, f, acc.z);
          acc.w = fmaf(o.w, f, acc.w);
        }
      }
    }
    if (D == 64) {
      acc.x += __shfl_xor_sync(kFull, acc.x, 16);
      acc.y += __shfl_xor_sync(kFull, acc.y, 16);
      acc.z += __shfl_xor_sync(kFull, acc.z, 16);
      acc.w += __shfl_xor_sync(kFull, acc.w, 16);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const size_t orow = static_cast<size_t>(pc.tok0 + t) * a.H_q + pc.g * a.G + j;
    if (odd == 0) {
      uint2 w;
      w.x = L == 0.f ? 0u : pack_bf16x2(acc.x * inv, acc.y * inv);
      w.y = L == 0.f ? 0u : pack_bf16x2(acc.z * inv, acc.w * inv);
      *reinterpret_cast<uint2 *>(a.out + orow * D + 4 * c4) = w;
    }
    if (lane == 0 && a.lse) a.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
  }
}

// The same for launches whose items have more rows than one tile: those have few pieces each
// and many rows, so a warp takes 32 rows (a lane each) and 16 dims, reads whole lines of the
// partials and writes whole sectors.  Reading them a row per warp took 22 us of a 240 us launch
// (8K tokens, window 1024).
template <int D>
__global__ void __launch_bounds__(D * 2) paged_merge_rows_kernel(const MergeArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  const PagedPiece pc = a.piece[blockIdx.x];
  if (!pc.valid) return;
  const int prow = blockIdx.y * 32 + lane;
  const int qt = prow / kRows, r = prow - qt * kRows;
  const int t = qt * a.TT + r / a.G, j = r % a.G;
  const bool in = r < a.TT * a.G && t < pc.ntok;
  if (!__any_sync(kFull, in)) return;
  const long long end = pc.item_u0 + units_of(pc.n, pc.u);
  const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml) + prow;
  const float4 *po = reinterpret_cast<const float4 *>(a.part) + static_cast<size_t>(4 * warp) * a.part_rows + prow;
  float M = -INFINITY, L = 0.f;
  float4 acc[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int c = blockIdx.x; c < pc.P; ++c) {
    const long long u0 = share_begin(pc.q, pc.r, c);
    if (u0 >= end) break;
    int t0, t1;
    piece_of(u0, share_begin(pc.q, pc.r, c + 1), pc.item_u0, pc.n, pc.u, t0, t1);
    if (t1 <= t0 || !in) continue;
    const int slot = 2 * c + (t0 == 0 ? 1 : 0);
    const float2 v = ml[static_cast<size_t>(slot) * a.part_rows];
    float4 o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = po[(static_cast<size_t>(slot) * (D / 4) + q) * a.part_rows];
    if (v.x == -INFINITY && v.y == 0.f) continue;     // no keys for this row in the piece
    const float m = fmaxf(M, v.x);                    // (-inf with a sum of NaN: only scores of NaN)
    const float old = M == -INFINITY ? 0.f : fast_exp2(M - m), w = v.x == -INFINITY ? 0.f : fast_exp2(v.x - m);
    M = m;
    L = L * old + v.y * w;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      acc[q].x = acc[q].x * old + o[q].x * w;
      acc[q].y = acc[q].y * old + o[q].y * w;
      acc[q].z = acc[q].z * old + o[q].z * w;
      acc[q].w = acc[q].w * old + o[q].w * w;
    }
  }
  if (!in) return;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const size_t orow = static_cast<size_t>(pc.tok0 + t) * a.H_q + pc.g * a.G + j;
  uint4 *dst = reinterpret_cast<uint4 *>(a.out + orow * D + 16 * warp);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float4 x = acc[2 * q], y = acc[2 * q + 1];
    dst[q] = L == 0.f ? make_uint4(0u, 0u, 0u, 0u)
                      : make_uint4(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv),
                                   pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
  }
  if (warp == 0 && a.lse) a.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
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

// What a launch needs of the current device: its SMs, the kernel's shared memory allowed there
// and its registers as the warpgroups' shares expect them (they add up to what the launch holds;
// a build that holds less would wait for registers that no warp gives back).  Asked once per
// device: the three calls took 1.2 us of each launch.
template <int D, bool FP8, bool FEW, class Kern>
cudaError_t prepare(Kern kern, int &sms, bool again = false) {
  using C = Cfg<D, FP8, FEW>;
  static std::atomic<int> known[64];                  // SMs by device, 0: not asked yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool keep = dev >= 0 && dev < 64;
  if (keep && !again && (sms = known[dev].load(std::memory_order_acquire)) > 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kBytes);
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa;
  if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
  if (fa.numRegs != C::kRegLaunch) return cudaErrorInvalidKernelImage;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  if (keep) known[dev].store(sms, std::memory_order_release);
  return cudaSuccess;
}

template <int D, bool FP8, bool FEW>
cudaError_t launch_d(const PagedAttnArgs &pa, cudaStream_t s) {
  using C = Cfg<D, FP8, FEW>;
  Args a;
  std::memset(&a, 0, sizeof(a));
  const int G = pa.H_q / pa.H_kv, TT = (FEW ? kFewRows : kRows) / G;
  const int R = std::min(pa.page_size, kKeys);
  const bool maps =
      make_query_map(&a.tq, pa.q, D, pa.H_q, pa.q_stride, pa.n_tok, G, TT) &&
      (FP8 ? make_code_map(&a.tk, pa.k_pages, D, pa.H_kv, pa.page_size, pa.n_pages, R) &&
                 make_code_map(&a.tv, pa.v_pages, D, pa.H_kv, pa.page_size, pa.n_pages, R)
           : make_bshd_map(&a.tk, pa.k_pages, D, pa.H_kv, pa.page_size, pa.n_pages, R) &&
                 make_bshd_map(&a.tv, pa.v_pages, D, pa.H_kv, pa.page_size, pa.n_pages, R));
  if (!maps) return cudaErrorInvalidValue;
  a.v_pages = pa.v_pages;
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
  a.TE = FEW ? TT : 2 * TT;
  a.part_rows = pa.part_rows;
  const int cap = pa.max_pages * pa.page_size;
  a.n_sink = std::min(pa.n_sink, cap);
  a.n_stream = pa.n_stream < 0 ? -1 : std::min(pa.n_stream, cap);
  a.sl2 = pa.scale * kLog2e;
  // about two clocks a nanosecond; at most 2^31 of them, a second
  a.wait_clocks = static_cast<uint32_t>(std::min(2ull * g_wait_limit_ns, 0x7fffffffull));
  auto kern = paged_attn_kernel<D, FP8, FEW>;
  int sms = 0;
  cudaError_t e = prepare<D, FP8, FEW>(kern, sms);
  if (e != cudaSuccess) return e;
  // no more CTAs than the launch can have shares of kUnitsMin
  const long long pairs = pa.B + pa.n_tok / a.TE;
  const long long most = pairs * pa.H_kv * (kUnitsTwo * ((cap + kKeys - 1) / kKeys + 1) + kUnitsItem) / kUnitsMin + 1;
  const int P = static_cast<int>(std::min(static_cast<long long>(std::min(sms, kPagedMaxCtas)), most));
  for (int turn = 0; turn < 2; ++turn) {
    ProfScope ps(FP8 ? "paged_attn_fp8" : "paged_attn", s);
    e = launch_pdl(kern, dim3(P), dim3(C::kThreads), C::kBytes, s, a);
    if (e != cudaErrorInvalidValue || turn) break;
    // a context that was torn down and made again has forgotten the shared memory's limit
    cudaGetLastError();
    if ((e = prepare<D, FP8, FEW>(kern, sms, true)) != cudaSuccess) break;
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
  ma.TT = kRows / G;
  const int rows = std::min(a.TE, pa.n_tok) * G;
  ProfScope ps("paged_attn_merge", s);
  if (!FEW && pa.part_rows > kRows)
    return launch_pdl(paged_merge_rows_kernel<D>, dim3(P, pa.part_rows / 32), dim3(D * 2), 0, s, ma);
  const int y = (rows + kMergeWarps - 1) / kMergeWarps;
  return launch_pdl(paged_merge_kernel<D>, dim3(P, y), dim3(kMergeWarps * 32), 0, s, ma);
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
  // FEW holds 32 rows of a sequence at a time: launches that cannot have more, and those with no
  // more tokens than sequences, which are decode steps.  (Should such a launch put many tokens in
  // one sequence all the same, that one's keys are read once for each 32 rows.)
  const int few = kFewRows / (a.H_q / a.H_kv);
  if (a.fp8 && few > 0 && a.n_tok <= std::max(few, a.B))
    return a.D == 128 ? launch_d<128, true, true>(a, s) : launch_d<64, true, true>(a, s);
  if (a.fp8) return a.D == 128 ? launch_d<128, true, false>(a, s) : launch_d<64, true, false>(a, s);
  return a.D == 128 ? launch_d<128, false, false>(a, s) : launch_d<64, false, false>(a, s);
}

int paged_attn_device_error() {
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_paged_error, sizeof(int)) != cudaSuccess) return -1;
  if (cudaMemcpyToSymbol(g_paged_error, &zero, sizeof(int)) != cudaSuccess) return -1;
  return v;
}

int paged_attn_set_wait_limit(unsigned long long ns) {
  g_wait_limit_ns = std::min(ns, 1ull << 40);
  return 0;
}

}  // namespace dsa
