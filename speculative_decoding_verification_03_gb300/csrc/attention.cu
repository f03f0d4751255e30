// Attention of a chunk of new tokens over the paged key-value cache.
//
// out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(c s_ij - m_i),  s = q k^T,
// c = scale log2 e, m_i a running maximum: one pass over a sequence's slots.
//
// Rows.  The query heads that share a key head are rows of one matrix: row r
// of (sequence, key head) is token r / G, head r % G of the group, so that a
// verification step of 6 tokens with G = 4 is 24 rows that read the cache
// once.  A tile is 128 slots of the cache.  Three shapes of items:
//   narrow  e4m3 and at most 32 rows (decoding, verification, small trees): the
//           products are turned round, S^T = K Q^T and O^T = V^T P^T, with the tile's
//           128 slots (then the 128 dimensions) as M and 32 rows as N.  One thread
//           takes one slot of all rows, so all 128 share what e4m3 weights cost
//           (256 x 6 tokens 402 us, as wide items 717; in bf16 wide items do as well
//           or better: 64 x 5 tokens over 300 32 us and narrow ones 39, over 500 to
//           8000 201 and 199, 256 x 1 over 400 90 and 91, 1 over 1021 15 and 16)
//   wide    up to 128 rows: S = Q K^T, O = P V by half tiles of 64 slots, one thread
//           a row; P takes its scores' place in tensor memory
//   pair    more: 256 rows an item, two wide halves that share every K and V tile,
//           since so many rows are bound by the products and shared memory's feed
//
// One persistent CTA an SM holds two pipelines ("groups"), each of
//   4 softmax warps  TMEM columns for scores and for an accumulator
//   a products warp  issues the products.  An issue blocks while the tensor core
//                    is busy, so what a warp does between its products is hidden
//                    only behind the other group's
//   a copy warp      tiled TMA copies of K and V pages into a ring of slots
//   an items warp    walks the group's items and loads their queries
//   a scales warp    (e4m3) the tokens' scales, tiles ahead
// so that one group's exponentials, and what an item's end takes, run under the
// other's products and copies.  Scores have two buffers: the next ones are made
// while these become weights.  The groups are independent (own items, own half
// of the ring) but for pairs, where one half of the ring holds K, one V.  A CTA
// works on pairs only or on the others only; the CTAs are shared out by the work.
//
// Work split.  The tile steps of all items of a kind, and a few before each
// item's for its start and end, form one line that is cut into equal pieces, one a
// group (single) or CTA (pair): single tokens over a long cache are split along it,
// a batch along sequences and heads, whichever it is, without a plan from the host
// (lengths are on the device).  An item cut
// between pieces leaves each part's (m, l, O) in the workspace; who brings the
// last part joins them, in the parts' order, so results do not depend on timing.
//
// The maximum follows lazily: O is rescaled only when a row's maximum rises
// by more than a number (in log2) that its weights' type has room for, which keeps O's rescaling off the usual path.
//
// e4m3 caches stay e4m3 into the tensor core, and each operand against them is
// given as a sum of 8-bit numbers: a bf16 query as an e4m3 and an e5m2 number,
// exact down to 2^-14 of its row's largest, a weight as three e5m2 numbers, which are
// the upper bytes of a half-precision number and of what those leave, and so hold
// eight bits of small weights too.  (One slot may take most of a row's weight and
// thousands share the rest: with two e4m3 codes weights below 2^-15 of the
// largest were lost.)  That is a fourth of the shared memory that widening K and V
// would take.  A key's scale multiplies its scores; a value's scale, relative to the
// largest of late, its weight.
//
// Waits are by an mbarrier's phase parity, which tells the phase waited for only
// from the one before it.  So whoever waits on a barrier waits for each of its
// phases in turn, and no phase passes without all who wait on it.  The items warp
// watches the clock for its group: its waits (for an item to be done) are limited
// in time, all others end when it gives up.
//
// Sixteen warps run seven programs at once, so their loops share the SM's
// instruction cache, and what does not fit costs more than its instructions
// (measured: 40 % of fetches missed, each warp stalled on them a third of its
// time).  Hence loops are rolled where registers allow, each step has one site,
// and a wait is a few instructions.
//
// Measured (one GB300; copy 6779 GB/s, bf16 products 1928 TFLOP/s; in a graph), the
// bytes or operations that the method cannot do without over the time.  (These are the
// kernel's as it is.  Figures beside a choice compare what was tried with it; those
// for forms that are gone are from when they were tried.)
//   64 sequences, 5 tokens each over 500 to 8000, 32 heads of 8, bf16   202 us  5.92 TB/s
//   2 sequences, 1 token each over 130,000, 64 heads of 8, bf16         174 us  6.14 TB/s
//     (memory: 87 and 90 % of a copy's rate)
//   256 sequences, 6 tokens each over 700 to 6000, e4m3                 402 us  4.50 TB/s
//     (the softmax warps' instructions: twice the slots a byte of bf16's)
//   256 trees of 16 tokens over 100 to 2000, 28 heads of 4, bf16        144 us  4.11 TB/s
//     (an item's start and end beside eight tiles, and the way from a half's
//     weights over its products to the scores after it)
//   3 prompts of 1500 to 2048 tokens over 3000 to 16000, bf16           690 us  1228 TFLOP/s
//     (the same way, and shared memory's feed of the scores' products: with half
//     of those 623 us; 712 us over seconds, when the power limit lowers the clock)
//   the trees and the prompts over e4m3                                 272 and 1439 us
//     (wide items: five products for two, three codes a weight, a maximum that may
//     rise by one)
//   1 token over 1021, 32 heads of 8, bf16                               16 us
//     (latency: lengths, items, queries, one tile, eight parts joined)
#include <cmath>
#include <cstddef>
#include <cstring>

#include "kv_common.cuh"
#include "sv_tensor.cuh"

namespace sv {
namespace {

constexpr int kMaxDim = 128;
constexpr int kTile = 128;                 // rows and slots of a tile
constexpr int kHalfTile = kTile / 2;
constexpr int kThreads = 16 * 32;
constexpr int kMaxSms = 160;
constexpr int kMaxPart = 4;                // K / V tiles that a group's half of the ring holds
constexpr int kItems = 3;                  // a group's items handed over and not yet done
constexpr int kScaleStages = 2;            // (a wide item uses one)
constexpr int kScaleAhead = 8;             // tiles whose scale bytes are under way
// What an item's start and end take, in tile steps: by the kind of item, as short
// tiles leave them more.  Measured, us: bf16 single items with 2 / 3 / 4, trees of 16
// nodes 144 / 146 / 147, 64 x 5 tokens 202 / 202 / 203; e4m3 with 4 / 6 / 8 / 10, 256 x 6
// tokens 427 / 410 / 402 / 407; pairs with 5 / 6 / 8, prompts 690 / 691 / 700.
constexpr int kItemUnits = 2, kItemUnitsF8 = 8, kItemUnitsPair = 5;
constexpr int kNarrow = 32;                // rows of a narrow tile
constexpr uint32_t kHalfBytes = kTile * 128;  // 128 rows of 128 bytes: one swizzled half of a tile
constexpr size_t kSmemLimit = 232448;         // 227 KB a CTA
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kNoRow = 0x7fffffff;         // a thread without a row masks nothing
constexpr int kWideLazyF8 = 4, kNarrowLazyF8 = 6;  // log2 of the largest weights over e4m3,
constexpr int kTopF8 = 15;                         // and of what they are in their codes
constexpr int kScaleDrop = 4, kScaleFall = 60;     // log2: see scales()
constexpr float kNone = -1e30f;            // a narrow row's maximum before its first slot

// Workspace: status word, arrival counters [CTA][group] (back to zero after
// every call), then the parts of cut items: two a group (the one it continues,
// the one it begins), each m [128], l [128], O [128][128].
constexpr size_t kCounterOff = 256;
constexpr size_t kPartFloats = 2 * kTile + (size_t)kTile * kMaxDim;
constexpr size_t kPartOff = 4096;
constexpr size_t kAttWsBytes = kPartOff + (size_t)kMaxSms * 2 * 2 * kPartFloats * sizeof(float);
static_assert(kCounterOff + kMaxSms * 2 * 4 <= kPartOff && kAttWsBytes % 256 == 0, "workspace layout");

struct AttParams {
  int B, T, Hq, Hkv, G, D, table_stride, tree_nodes, page_size, num_pages;
  int box_rows;    // slots a TMA copy takes: gcd(page_size, 64)
  int halves;      // 128-byte halves of a K / V row
  int part;        // tiles that a half of the ring holds
  int q_box;       // tokens that a wide item's query copy takes (0: rows are copied one by one)
  const uint16_t *q;
  uint16_t *out;
  int64_t q_ts, q_hs, o_ts, o_hs;
  const int32_t *q_start, *kv_len, *table, *parents;
  const uint8_t *k_exp, *v_exp;
  float c;         // |scale| log2 e
  uint32_t q_sign; // 0x80008000 for a negative scale: the queries change sign
  float *lse;
  uint8_t *ws;
  uint64_t wait_ns;
  int withhold;
};

// A group's piece of an item: tiles [tile0, tile0 + n).
struct Item {
  int b, h, q0, base, cap;  // sequence, key head, first packed token, cached tokens, slots the table has
  int row0, rows, seen;     // the group's rows (in a pair perhaps none), slots that the item's last row sees
  int tile0, n;             // n == 0: no more items
  int first, parts;         // the first part's place, parts
  int narrow;               // an e4m3 cache and at most kNarrow rows: products turned round
  int steps;                // tiles, or wide half tiles (the last tile's second half only if seen)
};

struct alignas(16) ScaleStage {  // one tile's scales
  float a[kTile];    // a score's factor: c times the key's scale
  float w[kTile];    // a weight's factor: the value's scale over 2^(R - 127 + lazy - kTopF8), R the largest of late
  float shift;       // 2^(R of the previous tile - R)
  float unit;        // 2^(R - 127 + lazy - kTopF8): what O is in units of
};
struct F8Group {
  ScaleStage sc[kScaleStages];
  float q_scale[kTile];
  uint32_t bytes[kScaleAhead][2][kTile / 4];  // scale bytes of K and V as they arrive
};
// What all threads of a softmax group know of its rows.
struct alignas(16) Rows {
  float minus[kNarrow];     // minus the maximum (log2)
  float scale[kNarrow];     // e4m3: the query's scale
  float factor[kNarrow];    // what a raised maximum leaves of the sums,
  float o_factor[kNarrow];  // and of O
  float top[4][kNarrow];    // the warps' maxima
  float m[kTile], inv[kTile];  // where parts are joined: maximum, 1 / sum
  int lim[kNarrow];         // a row sees the slots below,
  uint64_t above[kNarrow];  // and these nodes of a tree
  int64_t out[kNarrow];     // where its output goes
  int vote[2][4];
};
// A group's share of the dynamic shared memory, before the ring: queries (two
// halves of a wide tile, or one of a narrow one and then P's first and last codes),
// narrow P's middle codes, rows, scales.
constexpr uint32_t kPOff = kHalfBytes, kMidOff = 2 * kHalfBytes, kRowsOff = kMidOff + kHalfBytes / 2, kF8Off = kRowsOff + 3072,
                   kGroupBytes = 3 * kHalfBytes;
static_assert(sizeof(Rows) <= 3072 && kF8Off + sizeof(F8Group) <= kGroupBytes, "a group's share");

struct Group {
  // Its half of the ring holds tiles (of narrow items and pairs) or half tiles (of
  // single wide items), each with their barriers.
  uint64_t full[kMaxPart], empty[kMaxPart], half_full[2 * kMaxPart], half_empty[2 * kMaxPart];
  uint64_t s_full[4];                            // scores there, wide ones and narrow ones in either buffer
  uint64_t p_ready[2], pv_done[2];               // P there, O += P V done
  uint64_t q_ready[2], q_free[2], o_free;         // narrow queries have two places
  uint64_t join, vote;                           // the softmax warps among themselves
  uint64_t finished;                             // they are through with all items
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t sc_full, sc_empty[kScaleStages];      // a wide tile's scales there (a narrow one's: see s_full), read
  uint64_t q_in;                                 // a wide item's query copy there
  Item items[kItems];
  int last;
  int b0;            // the sequence in which its piece begins,
  long long u_b0;    // where that sequence begins,
  long long u0, u1;  // and the piece
};

// Arrivals that complete a phase of each barrier, in Group's order, for bf16 and
// e4m3 caches (two on a slot's `empty` in pairs, where both products warps read it).
constexpr int kBarriers = 50;
__constant__ const uint8_t kCounts[2][kBarriers] = {
    {1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 4, 4, 1, 1, 1, 1, 1, 1, 4, 4, 4, 4, 1, 1, 1, 6, 6, 6, 1, 4, 4, 1},
    {1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, 2, 2, 4, 4, 1, 1, 1, 1, 5, 5, 4, 4, 4, 4, 1, 1, 1, 7, 7, 7, 1, 4, 4, 1}};
static_assert(kMaxPart == 4 && kItems == 3 && kScaleStages == 2 && offsetof(Group, items) == 8 * kBarriers &&
                  offsetof(Group, q_free) == 8 * 34 && offsetof(Group, item_empty) == 8 * 43,
              "kCounts follows Group");

struct Shared {
  Group group[2];
  uint32_t tmem;
  int abort;
  int pair;          // the kind of this CTA's items
  int cta0;          // the first CTA of its kind
  long long per;     // units of a piece
};

constexpr size_t kStaticBytes = 2048;  // Shared, up to the 1024-byte boundary where the tiles begin
static_assert(sizeof(Shared) <= kStaticBytes, "two halves of 64 KB fit beside it");

// ---- the line of work ---------------------------------------------------------------
// sum over i < n of floor((a i + b) / m), all >= 0, m > 0 (the Euclid-like
// reduction of a sum of floors)
__device__ __noinline__ long long floor_sum(long long n, long long m, long long a, long long b) {
  long long s = 0;
  while (n > 0) {
    s += n * (n - 1) / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const long long y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const long long t = m;
    m = a;
    a = t;
  }
  return s;
}

struct Seq {
  int q0, n, base, cap;  // first packed token, chunk, cached tokens, slots the table has
  int rows, np;          // rows of a key head, items
  bool flat;             // every item sees all slots (a tree, or a length cut by the table)
  bool bad;
  __device__ bool pair() const { return rows > kTile; }
  __device__ int seen(const AttParams &P, int p) const {  // slots that item p's last row sees
    if (flat) return (int)min((long long)base + n, (long long)cap);
    const int x = min((p + 1) * 2 * kTile, rows);
    return base + (x + P.G - 1) / P.G;
  }
  __device__ int tiles(const AttParams &P, int p) const { return (seen(P, p) + kTile - 1) / kTile; }
  __device__ int own(const AttParams &P) const { return pair() ? kItemUnitsPair : (P.k_exp ? kItemUnitsF8 : kItemUnits); }
  // units (tile steps and the items' own, a pair's twice) of items 0 .. p - 1:
  // with nested ceilings,
  // ceil((base + ceil(x / G)) / 128) = floor((base G + x + 128 G - 1) / (128 G))
  __device__ long long before(const AttParams &P, int p) const {
    if (p == 0) return 0;
    if (flat) return 2ll * p * (tiles(P, 0) + own(P));
    const long long m = (long long)kTile * P.G;
    return 2 * (floor_sum(p, m, 2 * kTile, (long long)base * P.G + 2 * kTile + m - 1) + (long long)p * own(P));
  }
  __device__ long long units(const AttParams &P) const {
    return np == 0 ? 0 : before(P, np - 1) + (pair() ? 2ll : 1ll) * (tiles(P, np - 1) + own(P));
  }
  // Where there are few items, parts that are too short for what it takes to join
  // them would not pay: of n tiles in p parts, n / p tiles and p parts' rows come one
  // after the other, and sqrt(n rows / 128) tiles a part measured best (us with none /
  // half / once / twice that: 1 x 32 tokens over 4000 79 / 54 / 48 / 59, 1 x 16 over
  // 8000 50 / 50 / 41 / 46, 1 x 100 over 10,000 88 / 88 / 77 / 83).  At least a whole
  // step of a pair.
  __device__ int least_piece(const AttParams &P) const {
    float n;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(n) : "f"((float)tiles(P, np - 1) * min(rows, kTile) * (1.f / kTile)));
    return max((int)n, 1) * (pair() ? 2 : 1);
  }
};
// (64-bit divisions are slow, and their operands nearly always small)
__device__ __noinline__ long long divide64(long long a, long long b) { return a / b; }
__device__ __forceinline__ long long divide(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : divide64(a, b);
}

__device__ __forceinline__ Seq read_seq(const AttParams &P, int b) {
  Seq s;
  s.q0 = __ldg(P.q_start + b);
  const int end = min(__ldg(P.q_start + b + 1), P.T);
  s.n = s.q0 < 0 ? 0 : max(end - s.q0, 0);
  s.base = __ldg(P.kv_len + b);
  s.bad = s.base < 0;
  s.base = max(s.base, 0);
  s.cap = (int)min((long long)P.table_stride * P.page_size, 0x7fffff00ll);
  const bool cut = (long long)s.base + s.n > s.cap;
  s.bad = (s.bad || cut) && s.n > 0;
  s.flat = cut || P.parents;
  s.rows = s.n * P.G;
  s.np = (s.rows + 2 * kTile - 1) / (2 * kTile);
  return s;
}

// A group's steps, item by item.
struct Walk {
  const AttParams &P;
  const Shared &sh;
  const int g;
  long long us;
  int b, h, p;
  Seq s;

  __device__ Walk(const AttParams &P_, const Shared &sh_, int g_) : P(P_), sh(sh_), g(g_) {
    const Group &gr = sh.group[g];
    b = gr.b0;
    us = h = p = 0;
    if (b >= P.B) return;
    s = read_seq(P, b);
    const long long all = s.units(P);
    long long at = gr.u0 - gr.u_b0;
    h = (int)divide(at, all);
    at -= h * all;
    int hi = s.np;  // the last item with before(p) <= at
    while (hi - p > 1) {
      const int mid = (p + hi) >> 1;
      if (s.before(P, mid) <= at) p = mid;
      else hi = mid;
    }
    us = gr.u_b0 + h * all + s.before(P, p);
  }
  __device__ bool fits(const Seq &x) const { return x.np != 0 && x.pair() == (sh.pair != 0); }
  // On to the first sequence from `from` on that has items of the CTA's kind.  Nearly
  // always that is `from`; others are looked at 32 at a time, a lane each (one
  // token beside 2000 sequences without 288 us one by one, 300 tokens beside 2000
  // single ones 526).
  __device__ __forceinline__ void seek(int from) {
    b = from;
    if (b < P.B) s = read_seq(P, b);
    if (b >= P.B || fits(s)) return;
    for (++b; b < P.B; b += 32) {
      const int at = b + (threadIdx.x & 31);
      const uint32_t found = __ballot_sync(0xffffffffu, at < P.B && fits(read_seq(P, min(at, P.B - 1))));
      if (found) {
        b += __ffs(found) - 1;
        s = read_seq(P, b);
        return;
      }
    }
  }
  __device__ bool next(Item &it) {
    const long long u0 = sh.group[g].u0, u1 = sh.group[g].u1;
    while (b < P.B && us < u1) {
      const int nt = s.tiles(P, p), w = sh.pair ? 2 : 1;
      const long long first_step = us + w * s.own(P);  // (the item's own units come before its steps)
      const int s0 = first_step >= u0 ? 0 : (int)((u0 - first_step + w - 1) >> (w - 1));
      const int s1 = u1 <= first_step ? 0 : (int)min((long long)nt, (u1 - first_step + w - 1) >> (w - 1));
      if (s0 < s1) {
        it.b = b;
        it.h = h;
        it.q0 = s.q0;
        it.base = s.base;
        it.cap = s.cap;
        it.row0 = p * 2 * kTile + (sh.pair ? g * kTile : 0);
        it.rows = max(0, min(kTile, s.rows - it.row0));
        it.seen = s.seen(P, p);
        it.tile0 = s0;
        it.n = s1 - s0;
        const int first = (int)divide(first_step, sh.per), last = (int)divide(first_step + (long long)w * (nt - 1), sh.per);
        it.first = sh.pair ? 2 * (sh.cta0 + first) + g : first;
        it.parts = last - first + 1;
        it.narrow = P.k_exp && !sh.pair && it.rows <= kNarrow;
        it.steps = it.narrow ? it.n : 2 * it.n - (it.seen - (s1 - 1) * kTile <= kTile / 2);
      }
      us += (long long)w * (nt + s.own(P));
      if (++p == s.np) {
        p = 0;
        if (++h == P.Hkv) {
          h = 0;
          if (us < u1) seek(b + 1);  // (else the piece is at its end)
        }
      }
      if (s0 < s1) return true;
    }
    return false;
  }
};

// A role's place in a ring of `size` entries: entry, and phase in the top bit.
struct Cursor {
  uint32_t v = 0;
  __device__ __forceinline__ uint32_t at() const { return v & 0xffffu; }
  __device__ __forceinline__ uint32_t phase() const { return v >> 31; }
  __device__ __forceinline__ void step(uint32_t by, uint32_t size) {  // by <= size
    v += by;
    if (at() >= size) v = (v - size) ^ 0x80000000u;
  }
  __device__ __forceinline__ void skip(uint32_t by, uint32_t size) {
    v ^= (by / size & 1) << 31;
    step(by % size, size);
  }
};

// What every role needs: waits, and its group's items in order.
struct Role {
  const AttParams &P;
  Shared &sh;
  Group &gr;
  int g, lane;
  Cursor item;
  __device__ Role(const AttParams &P_, Shared &sh_, int g_)
      : P(P_), sh(sh_), gr(sh_.group[g_]), g(g_), lane(threadIdx.x & 31) {}
  __device__ __forceinline__ uint32_t *status() const { return reinterpret_cast<uint32_t *>(P.ws); }
  // until the phase is complete, or the items warp has given up
  __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) const {
    while (!mbar_try_wait_sleep(bar, parity & 1, 20000u))
      if (*(volatile int *)&sh.abort) return false;
    return true;
  }
  // at most wait_ns (the items warp's)
  __device__ __forceinline__ bool wait_limited(uint64_t *bar, uint32_t parity) const {
    return mbar_wait_bounded(bar, parity & 1, &sh.abort, status(), P.wait_ns);
  }
  // one arrival of a warp whose lanes are all done with what came before
  __device__ __forceinline__ void arrive(uint64_t *bar) const {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  }
  __device__ __forceinline__ const Item *next() const {
    if (!wait(&gr.item_full[item.at()], item.phase())) return nullptr;
    const Item *it = &gr.items[item.at()];
    return it->n ? it : nullptr;
  }
  __device__ __forceinline__ void done() {
    arrive(&gr.item_empty[item.at()]);
    item.step(1, kItems);
  }
};

// For an e4m3 product: the power of two 2^(byte - 127) that brings a row's
// largest magnitude (as bits) to at most 448; an infinity would saturate, so
// its row becomes NaN, as its products would.
__device__ __forceinline__ float q_scale(uint32_t top_bits, float &inv) {
  int byte = (int)(top_bits >> 23) - 8 + ((top_bits & 0x7fffffu) > 0x600000u);
  byte = byte < 1 ? 1 : (byte > 253 ? 253 : byte);
  inv = top_bits < 0x7f800000u ? scale_of_byte(254 - byte) : __uint_as_float(0x7fc00000u);
  return scale_of_byte(byte);
}
// Four values as e4m3 codes and the e5m2 codes of what those leave.  An e4m3 code
// leaves at most 8 units of a bf16 value's last place, which e5m2's three bits hold
// exactly, whatever their size; e4m3 would hold them down to 2^-9 only.
__device__ __forceinline__ void split_queries(float a, float b, float c, float d, uint32_t &hi, uint32_t &lo) {
  const uint32_t h0 = e4m3x2_from_f32(a, b), h1 = e4m3x2_from_f32(c, d);
  const float2 d0 = f32x2_from_f16x2(f16x2_from_e4m3x2((uint16_t)h0));
  const float2 d1 = f32x2_from_f16x2(f16x2_from_e4m3x2((uint16_t)h1));
  hi = h0 | h1 << 16;
  lo = e5m2x2_from_f32(a - d0.x, b - d0.y) | e5m2x2_from_f32(c - d1.x, d - d1.y) << 16;
}
// Four weights as three e5m2 codes each.  e5m2 is half precision's upper byte, so
// the codes are the upper bytes of the weight in half precision, of what that leaves,
// and of what that leaves, each remainder held kGain times larger than the one
// before.  Each code keeps three bits at least, so what is cut off is less than 2^-8
// of a weight, 0.0003 of it on average (rounding would take two instructions more a
// pair and code).  The last code's least bit stands for 2^-16 / kGain^2.
template <int kGain>
__device__ __forceinline__ void split_weights(float2 a, float2 b, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
  auto half2 = [](float2 v) {
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(v.y), "f"(v.x));
    return h;
  };
  auto left = [](uint32_t x) {  // what the code leaves: exact
    uint32_t d;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(x & 0xff00ff00u));
    if (kGain == 8) asm("mul.f16x2 %0, %1, %2;" : "=r"(d) : "r"(d), "r"(0x48004800u));
    return d;
  };
  static_assert(kGain == 1 || kGain == 8, "half-precision 8 is 0x4800");
  uint32_t h0 = half2(a), h1 = half2(b);
  hi = __byte_perm(h0, h1, 0x7531);
  h0 = left(h0);
  h1 = left(h1);
  mid = __byte_perm(h0, h1, 0x7531);
  lo = __byte_perm(left(h0), left(h1), 0x7531);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// ---- softmax warps ---------------------------------------------------------------------
template <bool kF8>
struct Softmax : Role {
  // A raised maximum m is set kHead over the largest score, and raised again when
  // a score is kLazy over it.  bf16 weights have fp32's range.  Over e4m3, a weight of
  // 2^kLazy is 2^kTopF8 in its codes, half precision's largest power of two.  Wide
  // weights sit as high as they can, since their three codes add to one accumulator
  // and the last may not fall below e5m2's least step, 2^-16: eight bits are kept of
  // weights down to 2^-22 of the largest.  Narrow remainders have columns of their own
  // and are held kGain and kGain^2 larger, so there is room to let scores rise by eight
  // before a maximum is raised, with eight bits down to 2^-21 of the largest weight (256
  // x 6 tokens, us by how far they may rise: 7 413, 8 402, 9 393, each a bit of that range).
  static constexpr float kWideLazy = kF8 ? kWideLazyF8 : 16, kNarrowLazy = kNarrowLazyF8;
  static constexpr float kWideHead = kF8 ? -3.f : 0.f, kNarrowHead = 2.f;
  static constexpr int kGain = 8;
  static constexpr int kJoinRows = kF8 ? 1 : 2;
  // A wide P's columns: 32 slots are 16 of bf16 pairs, or 8 of first codes and 8 of
  // the others 16 and 32 columns on
  static constexpr int kColumns = kF8 ? 8 : 16, kNext = kF8 ? 16 : 8;
  F8Group &f8;
  Rows &rows;
  uint8_t *p_smem;
  uint32_t s_at, o_at;  // this warp's lanes of the group's columns
  int row, warp;        // thread and warp of the group
  // phases, as bits: s_full and pv_done (of either buffer), joins, votes, queries
  enum : uint32_t { kS0 = 1, kPv0 = 16, kJoin = 64, kVote = 128, kQ0 = 256, kSc = 1024 };
  uint32_t phases = 0;
  int q_place = 0;      // the next narrow item's

  __device__ Softmax(const AttParams &P_, Shared &sh_, int g_, F8Group &f8_, Rows &rows_, uint8_t *p, uint32_t tm)
      : Role(P_, sh_, g_), f8(f8_), rows(rows_), p_smem(p), row(threadIdx.x & 127), warp((threadIdx.x >> 5) & 3) {
    s_at = tm + ((uint32_t)(warp * 32) << 16) + g * 2 * kTile;
    o_at = s_at + kTile;
  }

  // The next phase of a barrier that is waited for in turn.
  __device__ __forceinline__ bool next_phase(uint64_t *bar, uint32_t bit) {
    const uint32_t now = (phases & bit) != 0;
    phases ^= bit;
    return wait(bar, now);
  }
  // pv_done's bit counts the products asked for: the newest is the phase before.
  __device__ __forceinline__ bool products_done(int buf) { return wait(&gr.pv_done[buf], !(phases & kPv0 << buf)); }
  __device__ __forceinline__ bool join() {
    arrive(&gr.join);
    return next_phase(&gr.join, kJoin);
  }

  // the i-th of an item's parts, whose first has place `first`
  __device__ __forceinline__ float *part(int first, int i) const {
    const int place = first + (sh.pair ? 2 * i : i);
    return reinterpret_cast<float *>(P.ws + kPartOff) + ((size_t)place * 2 + (i == 0)) * kPartFloats;
  }
  __device__ __forceinline__ float *my_part(const Item &it) const {
    if (it.parts == 1) return nullptr;
    const int place = 2 * blockIdx.x + g;  // (single items' CTAs are the first ones)
    return part(it.first, (place - it.first) >> (sh.pair ? 1 : 0));
  }

  // Hand over this part; who brings the last joins them: first the rows' maxima
  // and sums, a row a thread, then each warp adds up rows, four columns a lane;
  // both with eight parts' loads under way, of two rows with bf16 caches (1 x 32
  // tokens over 4000 55 -> 48 us; with e4m3 the registers are missed in the loops
  // over tiles: 256 x 6 tokens 402 -> 564 us).
  __device__ __forceinline__ bool join_parts(const Item &it) {
    __threadfence();
    if (!join()) return false;
    if (row == 0) {
      uint32_t *cnt = reinterpret_cast<uint32_t *>(P.ws + kCounterOff) + it.first;
      const bool last = atomicAdd(cnt, 1u) == (uint32_t)it.parts - 1;
      if (last) *cnt = 0;
      __threadfence();
      gr.last = last;
    }
    if (!join()) return false;
    if (gr.last) {
      const int rows_n = it.rows;
      float m = -INFINITY, l = 0.f;  // of this thread's row
#pragma unroll 1
      for (int i0 = 0; i0 < it.parts; i0 += 8) {
        float mi[8], li[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float *src = part(it.first, min(i0 + k, it.parts - 1)) + min(row, rows_n - 1);
          mi[k] = __ldcg(src);
          li[k] = i0 + k < it.parts ? __ldcg(src + kTile) : 0.f;
        }
        float up = m;
#pragma unroll
        for (int k = 0; k < 8; ++k) up = fmaxf(up, mi[k]);
        l *= m == -INFINITY ? 0.f : ex2_approx(m - up);
#pragma unroll
        for (int k = 0; k < 8; ++k) l += mi[k] == -INFINITY ? 0.f : ex2_approx(mi[k] - up) * li[k];
        m = up;
      }
      if (row < rows_n) {
        rows.m[row] = m;
        rows.inv[row] = l == 0.f ? 0.f : 1.f / l;
        if (P.lse) {
          const int at = it.row0 + row, tok = at / P.G;
          P.lse[(int64_t)(it.q0 + tok) * P.Hq + it.h * P.G + at - tok * P.G] = l == 0.f ? -INFINITY : kLn2 * m + logf(l);
        }
      }
      if (!join()) return false;
#pragma unroll 1
      for (int r0 = warp; r0 < rows_n; r0 += 4 * kJoinRows) {
        float4 o[kJoinRows];
#pragma unroll
        for (int j = 0; j < kJoinRows; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int i0 = 0; i0 < it.parts; i0 += 8) {
          float4 x[kJoinRows][8];
          float mi[kJoinRows][8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float *src = part(it.first, min(i0 + k, it.parts - 1));
#pragma unroll
            for (int j = 0; j < kJoinRows; ++j) {
              const int r = min(r0 + 4 * j, rows_n - 1);
              mi[j][k] = __ldcg(src + r);
              if (4 * lane < P.D)
                x[j][k] = __ldcg(reinterpret_cast<const float4 *>(src + 2 * kTile + (size_t)r * kMaxDim) + lane);
            }
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
#pragma unroll
            for (int j = 0; j < kJoinRows; ++j) {
              if (i0 + k < it.parts && mi[j][k] != -INFINITY) {
                const float e = ex2_approx(mi[j][k] - rows.m[min(r0 + 4 * j, rows_n - 1)]);
                o[j].x += e * x[j][k].x;
                o[j].y += e * x[j][k].y;
                o[j].z += e * x[j][k].z;
                o[j].w += e * x[j][k].w;
              }
            }
          }
        }
#pragma unroll
        for (int j = 0; j < kJoinRows; ++j) {
          const int r = r0 + 4 * j;
          if (r < rows_n && 4 * lane < P.D) {
            const float inv = rows.inv[r];
            const int at = it.row0 + r, tok = at / P.G, head = it.h * P.G + at - tok * P.G;
            *reinterpret_cast<uint2 *>(P.out + (int64_t)(it.q0 + tok) * P.o_ts + (int64_t)head * P.o_hs + 4 * lane) =
                make_uint2(bf16x2_from_f32(o[j].x * inv, o[j].y * inv), bf16x2_from_f32(o[j].z * inv, o[j].w * inv));
          }
        }
      }
    }
    return join();  // `last` and the rows are read
  }

  // what row r sees of a tree: the nodes above it, as bits
  __device__ __forceinline__ uint64_t nodes_above(const Item &it, int tok) const {
    uint64_t above = 1ull;
    bool bad = false;
    const int32_t *par = P.parents + (size_t)it.b * P.tree_nodes;
    for (int x = tok; x > 0; x = tree_parent(par, P.tree_nodes, x, bad))
      if (x < 64) above |= 1ull << x;
    if (bad) atomicOr(status(), SV_FLAG_BAD_LEN);
    return above;
  }
  __device__ __forceinline__ int limit(const Item &it, int tok) const {
    return (int)min((long long)it.base + (P.parents ? 0 : tok + 1), (long long)it.cap);
  }

  // ---- wide: one thread a row
  // O of this warp's rows times f
  __device__ __forceinline__ void rescale(float f) {
#pragma unroll 1
    for (int c = 0; c < P.D; c += 32) {
      uint32_t o[32];
      tmem_ld32(o_at + c, o);
      tmem_wait_ld();
      pin32(o);
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
      tmem_st32(o_at + c, o);
    }
  }
  // what the row sees of 32 slots from j on, as bits
  __device__ __forceinline__ uint32_t sees(const Item &it, int j, int lim, uint64_t above) const {
    const int left = lim - j;
    uint32_t see = left >= 32 ? 0xffffffffu : (left <= 0 ? 0u : (1u << left) - 1u);
    if (P.parents && lim != kNoRow) {
      const int node = j - it.base;  // the node at bit 0
      if (node >= 0) see |= node < 64 ? (uint32_t)(above >> node) : 0u;
      else if (node > -32) see |= (uint32_t)above << -node;
      if (it.row0 + kTile > 64 * P.G) {  // a token past 64 nodes sees itself
        const int tok = (it.row0 + row) / P.G, self = tok - node;
        if (tok >= 64 && self >= 0 && self < 32) see |= 1u << self;
      }
      const int room = it.cap - j;
      if (room < 32) see &= room <= 0 ? 0u : (1u << room) - 1u;
    }
    return see;
  }

  // A half tile's scores in TMEM to weights.  m is the row's maximum so far, which
  // l and O are relative to.
  __device__ __forceinline__ bool wide_step(const Item &it, int u, int lim, uint64_t above, float qs,
                                            const ScaleStage *stage, float &m, float &l) {
    const int buf = u & 1, slot0 = (u & 1) * 64;
    const uint32_t s_buf = s_at + buf * 64;
    uint32_t x[2][32];
    tmem_ld32(s_buf, x[0]);
    tmem_ld32(s_buf + 32, x[1]);
    tmem_wait_ld();
    pin32(x[0]);
    pin32(x[1]);
    if (kF8) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 a = *reinterpret_cast<const float4 *>(&stage->a[slot0 + 32 * i + e]);
          const float2 y =
              __fmul2_rn(make_float2(__uint_as_float(x[i][e]), __uint_as_float(x[i][e + 1])), make_float2(a.x, a.y));
          const float2 z =
              __fmul2_rn(make_float2(__uint_as_float(x[i][e + 2]), __uint_as_float(x[i][e + 3])), make_float2(a.z, a.w));
          x[i][e] = __float_as_uint(y.x);
          x[i][e + 1] = __float_as_uint(y.y);
          x[i][e + 2] = __float_as_uint(z.x);
          x[i][e + 3] = __float_as_uint(z.y);
        }
    }
    const int j0 = it.tile0 * kTile + u * 64;
    if (__any_sync(0xffffffffu, j0 + 64 > lim)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t see = sees(it, j0 + 32 * i, lim, above);
#pragma unroll
        for (int e = 0; e < 32; ++e) x[i][e] = (see >> e) & 1 ? x[i][e] : 0xff800000u;
      }
    }
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // four chains
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 32; e += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mx[k] = max3(mx[k], __uint_as_float(x[i][e + 2 * k]), __uint_as_float(x[i][e + 2 * k + 1]));
    const float factor = kF8 ? qs : P.c;
    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * factor;

    // O is brought to a maximum that rose by more than kLazy in some row
    const float shift = kF8 && u > 0 && buf == 0 ? stage->shift : 1.f;
    if (__any_sync(0xffffffffu, (top > m + kWideLazy && lim != kNoRow) || shift != 1.f)) {
      const float up = fmaxf(m, top + kWideHead);
      const float f = m == -INFINITY ? 0.f : ex2_approx(m - up);
      l *= f;
      m = up;
      if (u > 0) {
        if (!products_done(buf ^ 1)) return false;  // the half tile's before
        tc_fence_after();
        rescale(f * shift);
      }
    }

    const float minus = m == -INFINITY ? 0.f : -m;
    const float2 fac2 = make_float2(factor, factor), min2 = make_float2(minus, minus);
    float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t hi[8], mid[8], lo[8];  // P: bf16 pairs in the first two, or the three codes
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        float2 a =
            __ffma2_rn(make_float2(__uint_as_float(x[i][2 * e]), __uint_as_float(x[i][2 * e + 1])), fac2, min2);
        float2 b =
            __ffma2_rn(make_float2(__uint_as_float(x[i][2 * e + 2]), __uint_as_float(x[i][2 * e + 3])), fac2, min2);
        a.x = ex2_approx(a.x);
        a.y = ex2_approx(a.y);
        b.x = ex2_approx(b.x);
        b.y = ex2_approx(b.y);
        sum0 = __fadd2_rn(sum0, a);
        sum1 = __fadd2_rn(sum1, b);
        if (!kF8) {
          (e < 8 ? hi : mid)[e % 8] = bf16x2_from_f32(a.x, a.y);
          (e < 8 ? hi : mid)[e % 8 + 1] = bf16x2_from_f32(b.x, b.y);
        } else {
          const float4 w = *reinterpret_cast<const float4 *>(&stage->w[slot0 + 32 * i + 2 * e]);
          split_weights<1>(__fmul2_rn(a, make_float2(w.x, w.y)), __fmul2_rn(b, make_float2(w.z, w.w)), hi[e / 2],
                           mid[e / 2], lo[e / 2]);
        }
      }
      tmem_st8(s_buf + kColumns * i, hi);
      tmem_st8(s_buf + kColumns * i + kNext, mid);
      if (kF8) tmem_st8(s_buf + kColumns * i + 2 * kNext, lo);
    }
    l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
    tmem_wait_st();
    return true;
  }

  __device__ __forceinline__ bool wide(const Item &it) {
    float qs = 1.f;
    if (kF8) {
      if (!next_phase(&gr.q_ready[0], kQ0)) return false;
      if (row < it.rows) qs = f8.q_scale[row];
      arrive(&gr.q_free[0]);
    }
    int lim = kNoRow;
    uint64_t above = 0;
    if (row < it.rows) {
      const int tok = (it.row0 + row) / P.G;
      lim = limit(it, tok);
      if (P.parents) above = nodes_above(it, tok);
    }
    float m = -INFINITY, l = 0.f, unit = 1.f;  // m in log2
    const bool active = warp * 32 < it.rows;
#pragma unroll 1
    for (int u = 0; u < it.steps; ++u) {
      const int buf = u & 1;
      if (!next_phase(&gr.s_full[buf], kS0 << buf)) return false;
      tc_fence_after();
      if (kF8 && buf == 0 && !next_phase(&gr.sc_full, kSc)) return false;
      const ScaleStage *stage = &f8.sc[0];
      if (kF8) unit = stage->unit;
      if (active && !wide_step(it, u, lim, above, qs, stage, m, l)) return false;
      phases ^= kPv0 << buf;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&gr.p_ready[buf]);
        if (kF8 && (buf == 1 || u + 1 == it.steps)) mbar_arrive(&gr.sc_empty[0]);
      }
    }

    const bool mine = row < it.rows;
    const int at = it.row0 + (mine ? row : 0);
    const int tok = at / P.G, head = it.h * P.G + at - tok * P.G;
    float *to_part = my_part(it);
    uint16_t *o_row = P.out + (int64_t)(it.q0 + tok) * P.o_ts + (int64_t)head * P.o_hs;
    const float fin = unit * (to_part ? 1.f : (l == 0.f ? 0.f : 1.f / l));
    if (!products_done(0) || !products_done(1)) return false;
    tc_fence_after();
#pragma unroll 1
    for (int c = 0; active && c < P.D; c += 32) {
      uint32_t o[32];
      float y[32];
      const int cols = P.D - c;  // 16 or at least 32
      tmem_ld32(o_at + c, o);
      tmem_wait_ld();
      pin32(o);
#pragma unroll
      for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(o[e]) * fin;
      if (mine && to_part) {
        float4 *dst = reinterpret_cast<float4 *>(to_part + 2 * kTile + (size_t)row * kMaxDim + c);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e < 4 || cols > 16) __stcg(dst + e, make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]));
      } else if (mine) {
        uint4 *dst = reinterpret_cast<uint4 *>(o_row + c);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < 2 || cols > 16) dst[e] = make_uint4(bf16x2_from_f32(y[8 * e], y[8 * e + 1]), bf16x2_from_f32(y[8 * e + 2], y[8 * e + 3]),
                              bf16x2_from_f32(y[8 * e + 4], y[8 * e + 5]), bf16x2_from_f32(y[8 * e + 6], y[8 * e + 7]));
      }
    }
    tc_fence_before();  // O is read
    arrive(&gr.o_free);
    if (mine && to_part) {
      __stcg(to_part + row, m);
      __stcg(to_part + kTile + row, l);
    } else if (mine && P.lse) {
      P.lse[(int64_t)(it.q0 + tok) * P.Hq + head] = l == 0.f ? -INFINITY : kLn2 * m + logf(l);
    }
    return !to_part || join_parts(it);
  }

  // ---- narrow (e4m3): one thread a slot of the tile, 32 rows
  // The scores of a slot, scaled: y = x - m (log2), or (again) x itself; returns
  // their largest.  `seen` has a bit for every row that sees the slot.  (Rows past
  // the item's are zeros and stay in: leaving blocks of them out measured slower.)
  __device__ __forceinline__ float narrow_scores(uint32_t s_buf, float a, uint32_t seen, bool again,
                                                 float (&y)[kNarrow]) const {
    uint32_t h[32];
    tmem_ld32(s_buf, h);
    tmem_wait_ld();
    pin32(h);
    const bool all_seen = __all_sync(0xffffffffu, seen == ~0u);
    float top = -INFINITY, top2 = -INFINITY;
#pragma unroll
    for (int r0 = 0; r0 < kNarrow; r0 += 8) {
#pragma unroll
      for (int e = r0; e < r0 + 8; e += 4) {
        float4 mi = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!again) mi = *reinterpret_cast<const float4 *>(&rows.minus[e]);
        float2 u = make_float2(__uint_as_float(h[e]), __uint_as_float(h[e + 1]));
        float2 z = make_float2(__uint_as_float(h[e + 2]), __uint_as_float(h[e + 3]));
        const float4 qs = *reinterpret_cast<const float4 *>(&rows.scale[e]);
        u = __ffma2_rn(__fmul2_rn(u, make_float2(a, a)), make_float2(qs.x, qs.y), make_float2(mi.x, mi.y));
        z = __ffma2_rn(__fmul2_rn(z, make_float2(a, a)), make_float2(qs.z, qs.w), make_float2(mi.z, mi.w));
        y[e] = u.x;
        y[e + 1] = u.y;
        y[e + 2] = z.x;
        y[e + 3] = z.y;
      }
      if (!all_seen) {
#pragma unroll
        for (int r = r0; r < r0 + 8; ++r)
          if (!(seen >> r & 1)) y[r] = -INFINITY;
      }
#pragma unroll
      for (int r = r0; r < r0 + 8; r += 4) {
        top = max3(top, y[r], y[r + 1]);
        top2 = max3(top2, y[r + 2], y[r + 3]);
      }
    }
    return fmaxf(top, top2);
  }

  // The four warps must agree on the rows' maxima: each votes whether some y is
  // above kNarrowLazy, and takes the exponentials while the votes come in; only if one
  // is are the scores read again for new maxima.
  __device__ __forceinline__ bool narrow(const Item &it) {
    if (!next_phase(&gr.q_ready[q_place], kQ0 << q_place)) return false;
    if (row < kNarrow) {
      const bool mine = row < it.rows;
      const int at = it.row0 + (mine ? row : 0), tok = at / P.G, head = it.h * P.G + at - tok * P.G;
      rows.minus[row] = -kNone;
      rows.lim[row] = limit(it, tok);
      if (P.parents) rows.above[row] = nodes_above(it, tok);
      rows.out[row] = (int64_t)(it.q0 + tok) * P.o_ts + (int64_t)head * P.o_hs;
      rows.scale[row] = f8.q_scale[q_place * kNarrow + row];
    }
    arrive(&gr.q_free[q_place]);
    q_place ^= 1;
    if (!join()) return false;

    float l[kNarrow];
#pragma unroll
    for (int r = 0; r < kNarrow; ++r) l[r] = 0.f;
    float unit = 1.f;
#pragma unroll 1
    for (int t = 0; t < it.n; ++t) {
      const int buf = t & 1;  // of scores and of weights
      // (with it the products of tile t - 2 are done, issued before these scores:
      // P's buffer is free; and the tile's scales are there)
      if (!next_phase(&gr.s_full[2 + buf], kS0 << (2 + buf))) return false;
      tc_fence_after();
      const ScaleStage &stage = f8.sc[buf];
      const float a = stage.a[row], w = stage.w[row], shift = t > 0 ? stage.shift : 1.f;
      unit = stage.unit;
      arrive(&gr.sc_empty[buf]);
      uint32_t seen = ~0u;
      if ((it.tile0 + t + 1) * kTile > rows.lim[0]) {  // (row 0 sees least)
        const int j = (it.tile0 + t) * kTile + row, node = j - it.base;
        seen = 0;
#pragma unroll 1
        for (int r = 0; r < kNarrow; ++r) {
          bool see = j < rows.lim[r];
          if (P.parents && !see && j < it.cap && node >= 0)  // (a tree has at most 64 nodes, an item at most 32 tokens)
            see = node < 64 && (rows.above[r] >> node & 1);
          seen |= (uint32_t)see << r;
        }
      }
      const uint32_t s_buf = s_at + buf * 64;
      float y[kNarrow];
      bool again = t == 0;  // whether some y is too large: the rows' maxima rise
#pragma unroll 1
      for (;;) {
        const float top = narrow_scores(s_buf, a, seen, again, y);
        if (again) break;
        const bool raise = __any_sync(0xffffffffu, top > kNarrowLazy || shift != 1.f);
        if (lane == 0) rows.vote[buf][warp] = raise;
        arrive(&gr.vote);
#pragma unroll
        for (int r = 0; r < kNarrow; ++r) y[r] = ex2_approx(y[r]);
        if (!next_phase(&gr.vote, kVote)) return false;
        const int4 votes = *reinterpret_cast<const int4 *>(rows.vote[buf]);
        again = (votes.x | votes.y | votes.z | votes.w) != 0;
        if (!again) break;
      }
      if (again) {
        float tops = -INFINITY;  // of row `lane`
#pragma unroll
        for (int r = 0; r < kNarrow; ++r) {
          const float top = warp_max(y[r]);
          if (lane == r) tops = top;
        }
        rows.top[warp][lane] = tops;
        if (!join()) return false;
        if (row < kNarrow) {
          const float old = -rows.minus[row];
          const float top =
              fmaxf(fmaxf(rows.top[0][row], rows.top[1][row]), fmaxf(rows.top[2][row], rows.top[3][row]));
          const float up = fmaxf(old, top + kNarrowHead);
          const float factor = old == kNone ? 0.f : ex2_approx(old - up);
          rows.factor[row] = factor;
          rows.o_factor[row] = factor * shift;
          rows.minus[row] = -up;
        }
        if (!join()) return false;
#pragma unroll
        for (int r = 0; r < kNarrow; r += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(&rows.factor[r]);
          const float4 mi = *reinterpret_cast<const float4 *>(&rows.minus[r]);
          const float2 l0 = __fmul2_rn(make_float2(l[r], l[r + 1]), make_float2(f.x, f.y));
          const float2 l1 = __fmul2_rn(make_float2(l[r + 2], l[r + 3]), make_float2(f.z, f.w));
          const float2 y0 = __fadd2_rn(make_float2(y[r], y[r + 1]), make_float2(mi.x, mi.y));
          const float2 y1 = __fadd2_rn(make_float2(y[r + 2], y[r + 3]), make_float2(mi.z, mi.w));
          l[r] = l0.x;
          l[r + 1] = l0.y;
          l[r + 2] = l1.x;
          l[r + 3] = l1.y;
          y[r] = ex2_approx(y0.x);
          y[r + 1] = ex2_approx(y0.y);
          y[r + 2] = ex2_approx(y1.x);
          y[r + 3] = ex2_approx(y1.y);
        }
        if (t > 0) {
          if (!products_done(buf ^ 1)) return false;  // tile t - 1's
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 3 * kNarrow; c += 16) {
            uint32_t o[16];
            tmem_ld16(o_at + c, o);
            tmem_wait_ld();
            pin16(o);
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 f = *reinterpret_cast<const float4 *>(&rows.o_factor[(c & (kNarrow - 1)) + e]);
              const float2 a = __fmul2_rn(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), make_float2(f.x, f.y));
              const float2 b = __fmul2_rn(make_float2(__uint_as_float(o[e + 2]), __uint_as_float(o[e + 3])), make_float2(f.z, f.w));
              o[e] = __float_as_uint(a.x);
              o[e + 1] = __float_as_uint(a.y);
              o[e + 2] = __float_as_uint(b.x);
              o[e + 3] = __float_as_uint(b.y);
            }
            tmem_st8(o_at + c, o);
            tmem_st8(o_at + c + 8, o + 8);
          }
          tmem_wait_st();
        }
      }
      tc_fence_before();
      // P^T: a slot's 32 weights side by side (first codes, then last ones) in half of a
      // row of 128 bytes, swizzled as the tensor core reads it; the middle codes in a
      // fourth of a row, those of slots 64 on beside those before
      uint8_t *dst = p_smem + row * 128, *mid_dst = p_smem + (kMidOff - kPOff) + (row & 63) * 128;
      const int sw = (row & 7) ^ (buf * 4), mid_sw = (row & 7) ^ (buf * 4 + (row >> 6) * 2);
      constexpr int kBlock = 16;  // rows of 16 bytes
#pragma unroll
      for (int r0 = 0; r0 < kNarrow; r0 += kBlock) {
#pragma unroll
        for (int r = r0; r < r0 + kBlock; r += 2) {
          const float2 sum = __fadd2_rn(make_float2(l[r], l[r + 1]), make_float2(y[r], y[r + 1]));
          l[r] = sum.x;
          l[r + 1] = sum.y;
        }
        uint32_t hi[4], mid[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + 4 * e;
          split_weights<kGain>(__fmul2_rn(make_float2(y[r], y[r + 1]), make_float2(w, w)),
                               __fmul2_rn(make_float2(y[r + 2], y[r + 3]), make_float2(w, w)), hi[e], mid[e], lo[e]);
        }
        *reinterpret_cast<uint4 *>(mid_dst + ((r0 / kBlock ^ mid_sw) << 4)) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
        *reinterpret_cast<uint4 *>(dst + (((kNarrow + r0) / kBlock ^ sw) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4 *>(dst + ((r0 / kBlock ^ sw) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      }
      fence_async_smem();
      phases ^= kPv0 << buf;
      arrive(&gr.p_ready[buf]);
    }

    // ---- the item's end: the slots' sums added up, through P's space
    if (!products_done(0) || !products_done(1)) return false;
    tc_fence_after();
    float *to_part = my_part(it);
    float *x = reinterpret_cast<float *>(p_smem);
#pragma unroll
    for (int r = 0; r < kNarrow; ++r) x[r * kTile + row] = l[r];
    if (!join()) return false;
#pragma unroll 1
    for (int r = warp; r < it.rows; r += 4) {
      const float4 v = *reinterpret_cast<const float4 *>(x + r * kTile + 4 * lane);
      const float sum = warp_sum((v.x + v.y) + (v.z + v.w));
      if (lane == 0) {
        rows.factor[r] = sum;
        rows.inv[r] = unit * (to_part ? 1.f : (sum == 0.f ? 0.f : 1.f / sum));
      }
    }
    if (!join()) return false;
#pragma unroll 1
    for (int c = 0; c < it.rows; c += 16) {  // O^T: a dimension a thread, so that a row is written side by side
      uint32_t h[16], lo[16], mid[16];
      tmem_ld16(o_at + c, h);
      tmem_ld16(o_at + kNarrow + c, lo);
      tmem_ld16(o_at + 2 * kNarrow + c, mid);
      tmem_wait_ld();
      pin16(h);
      pin16(lo);
      pin16(mid);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float m = fmaf(__uint_as_float(lo[e]), 1.f / kGain, __uint_as_float(mid[e]));
        const float o = fmaf(m, 1.f / kGain, __uint_as_float(h[e])) * rows.inv[c + e];
        if (c + e < it.rows && row < P.D) {
          if (to_part) __stcg(to_part + 2 * kTile + (size_t)(c + e) * kMaxDim + row, o);
          else P.out[rows.out[c + e] + row] = (uint16_t)bf16x2_from_f32(o, 0.f);
        }
      }
    }
    tc_fence_before();  // O is read
    arrive(&gr.o_free);
    if (row < it.rows) {
      const float sum = rows.factor[row], m = sum == 0.f ? -INFINITY : -rows.minus[row];
      if (to_part) {
        __stcg(to_part + row, m);
        __stcg(to_part + kTile + row, sum);
      } else if (P.lse) {
        const int at = it.row0 + row, tok = at / P.G;
        P.lse[(int64_t)(it.q0 + tok) * P.Hq + it.h * P.G + at - tok * P.G] = sum == 0.f ? -INFINITY : kLn2 * m + logf(sum);
      }
    }
    return to_part ? join_parts(it) : join();  // the rows are read
  }

  __device__ void run() {
    while (const Item *it = next()) {
      bool ok;
      if (kF8 && it->narrow) ok = narrow(*it);
      else ok = wide(*it);
      if (!ok) return;
      done();
    }
    arrive(&gr.finished);
  }
};

// ---- the products ----------------------------------------------------------------------
// kFull: heads of kMaxDim values, whose products' steps over them need no test (256 x 6
// tokens 402 us with it, 413 without; prompts 690 and 698).
template <bool kF8, bool kFull>
struct Products : Role {
  static constexpr int kSteps = kF8 ? 4 : 8;  // of 32 or 16 slots in a tile
  static constexpr uint32_t kStepDesc = kTile / kSteps * 128 >> 4;
  uint8_t *ring_smem;
  int ksteps;  // 32 bytes of K each
  uint32_t slot_bytes, s_at, o_at;
  // the descriptors' low words; the high ones are the same for all of them
  uint32_t q_desc, p_desc, mid_desc, k_desc, v_desc, v_half;
  // phases, as bits: p_ready (of either buffer), q_ready (of either place)
  enum : uint32_t { kP0 = 1, kQ0 = 4 };
  uint32_t phases = 0;
  bool ok = true;

  __device__ Products(const AttParams &P_, Shared &sh_, int g_, uint8_t *smem, uint8_t *ring, uint32_t tmem)
      : Role(P_, sh_, g_), ring_smem(ring) {
    ksteps = kF8 ? (P.D + 31) / 32 : P.D / 16;
    slot_bytes = P.halves * kHalfBytes;
    s_at = __shfl_sync(0xffffffffu, tmem + g * 2 * kTile, 0);  // (the same in all lanes, and known to be: see elect_one)
    o_at = s_at + kTile;
    q_desc = (uint32_t)smem_desc(smem_addr(smem) + g * kGroupBytes, 16, 1024);
    p_desc = q_desc + (kPOff >> 4);
    mid_desc = q_desc + (kMidOff >> 4);
    k_desc = (uint32_t)smem_desc(smem_addr(ring), 16, 1024);
    // (V's 128-byte columns lie a half apart)
    v_desc = (uint32_t)smem_desc(smem_addr(ring), kF8 || P.halves == 1 ? 0 : kHalfBytes, 1024);
    v_half = (uint32_t)smem_desc(smem_addr(ring), kF8 || P.halves == 1 ? 0 : kHalfBytes / 2, 1024);
  }
  // Until the phase is complete or the items warp has given up.  Then this lane issues
  // no more (see `ok`), and run() ends before the next item; an answer on which all
  // lanes had to agree at every wait cost prompts 4 %, and sleeping while it waits
  // another 2 %.
  __device__ __forceinline__ void wait_for(uint64_t *bar, uint32_t parity) {
    while (!mbar_try_wait(bar, parity & 1)) {
      if (*(volatile int *)&sh.abort) {
        ok = false;
        return;
      }
    }
  }
  __device__ __forceinline__ void next_phase(uint64_t *bar, uint32_t bit) {
    const uint32_t now = (phases & bit) != 0;
    phases ^= bit;
    wait_for(bar, now);
  }

  // In both kinds of items the scores of step u + 2 follow the values of step u: their
  // buffer's last scores have been read when the weights made of them were there.

  // S^T = K Q^T and O^T += V^T P^T (e4m3), a step a tile
  __device__ __forceinline__ void narrow_item(const Item &it, int n, int place, Cursor kc, Cursor vc, uint32_t n_items) {
    constexpr uint32_t id_s = mma_idesc(kE4m3, kE4m3, kTile, kNarrow, false, false);
    constexpr uint32_t id_low = mma_idesc(kE4m3, kE5m2, kTile, kNarrow, false, false);
    // the weights' first and last codes, and their middle ones, in columns of their own
    constexpr uint32_t id_o = mma_idesc(kE4m3, kE5m2, kTile, 2 * kNarrow, true, true);
    constexpr uint32_t id_mid = mma_idesc(kE4m3, kE5m2, kTile, kNarrow, true, true);
    constexpr uint32_t q_half = kNarrow * 128 >> 4;
    const uint32_t q_at = q_desc + place * (kHalfBytes / 2 >> 4);
#pragma unroll 1
    for (int u = -2; u < n; ++u) {
      const int buf = u & 1;
      if (u >= 0) {
        wait_for(&gr.full[vc.at()], vc.phase());
        if (u + 1 == n) clear_tail(it.seen - (it.tile0 + u) * kTile, kTile, (g * P.part + vc.at()) * slot_bytes);
        // the accumulator's earlier item has been written out
        if (u == 0) wait_for(&gr.o_free, n_items ^ 1);
        next_phase(&gr.p_ready[buf], kP0 << buf);
        tc_fence_after();
        if (elect_one() && ok) {
          const uint32_t v = v_desc + (g * P.part + vc.at()) * (slot_bytes >> 4), p = p_desc + buf * (64 >> 4),
                         mid = mid_desc + buf * (64 >> 4);
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            mma_ss<true>(o_at, v + i * kStepDesc, p + i * kStepDesc, id_o, u > 0 || i > 0);
            mma_ss<true>(o_at + 2 * kNarrow, v + i * kStepDesc, mid + (i & 1) * kStepDesc + (i >> 1) * (kNarrow >> 4), id_mid,
                         u > 0 || i > 0);
          }
          tc_commit(&gr.empty[vc.at()]);
          tc_commit(&gr.pv_done[buf]);  // last: the CTA may end soon after it
        }
        __syncwarp();
        vc.step(u + 2 >= n ? 1 : 2, P.part);
      }
      if (u + 2 >= n) continue;
      wait_for(&gr.full[kc.at()], kc.phase());
      if (elect_one() && ok) {
        const uint32_t k = k_desc + (g * P.part + kc.at()) * (slot_bytes >> 4), s_to = s_at + buf * 64;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!kFull && i >= ksteps) break;
          mma_ss<true>(s_to, k + i * 2, q_at + i * 2, id_s, i > 0);
          mma_ss<true>(s_to, k + i * 2, q_at + q_half + i * 2, id_low, true);
        }
        tc_commit(&gr.s_full[2 + buf]);
        tc_commit(&gr.empty[kc.at()]);
        if (u + 3 == n) tc_commit(&gr.q_free[place]);
      }
      __syncwarp();
      kc.step(u == -2 ? 1 : 2, P.part);
    }
  }

  // S = Q K^T and O += P V, a step half a tile.  K and V come by tiles for pairs,
  // which have loads enough under way, and by half tiles for single items, whose
  // half of the ring would hold one tile of each (trees of 16 nodes 165 us by tiles,
  // 152 us by halves; prompts 715 and 737 us).
  __device__ __forceinline__ void wide_item(const Item &it, Cursor kc, Cursor vc, bool pair, uint32_t n_items) {
    constexpr uint32_t id_s = mma_idesc(kF8 ? kE4m3 : kBf16, kF8 ? kE4m3 : kBf16, kTile, kTile / 2, false, false);
    constexpr uint32_t id_low = mma_idesc(kE5m2, kE4m3, kTile, kTile / 2, false, false);
    const uint32_t id_o = mma_idesc(kF8 ? kE5m2 : kBf16, kF8 ? kE4m3 : kBf16, kTile, (uint32_t)P.D, false, true);
    constexpr uint32_t kHalf = kHalfBytes >> 4;
    const int steps = __shfl_sync(0xffffffffu, it.steps, 0), by = pair ? 1 : 2;
    const uint32_t size = pair ? P.part : 2 * P.part, unit = pair ? slot_bytes : slot_bytes / 2;
    const uint32_t k_base = pair ? 0 : g * size, v_base = pair ? size : g * size;
    const uint32_t halves_k = pair ? kHalf : kHalf / 2;          // between the halves of K's rows
    const uint32_t later = pair ? kHalf / 2 : 0;                 // to a tile's second half
    const uint32_t v_first = pair ? v_desc : v_half;
    Group &kg = sh.group[pair ? 0 : g], &vg = sh.group[pair ? 1 : g];
    uint64_t *const k_full = pair ? kg.full : kg.half_full, *const v_full = pair ? vg.full : vg.half_full;
    uint64_t *const k_empty = pair ? kg.empty : kg.half_empty, *const v_empty = pair ? vg.empty : vg.half_empty;
#pragma unroll 1
    for (int u = -2; u < steps; ++u) {
      const int half = u & 1;
      const bool first = !pair || half == 0;  // step of its unit
      if (u >= 0) {
        const bool last = !pair || half == 1 || u + 1 == steps;
        if (first) {
          wait_for(&v_full[vc.at()], vc.phase());
          const int rows = pair ? kTile : kHalfTile;
          if (steps - u <= (pair ? 2 : 1))
            clear_tail(it.seen - it.tile0 * kTile - u * kHalfTile, rows, (v_base + vc.at()) * unit);
          // the accumulator's earlier item has been written out
          if (u == 0) wait_for(&gr.o_free, n_items ^ 1);
        }
        const uint32_t v = v_first + (v_base + vc.at()) * (unit >> 4) + half * later, p = s_at + half * 64;
        next_phase(&gr.p_ready[half], kP0 << half);
        tc_fence_after();
        if (elect_one() && ok) {
#pragma unroll
          for (int i = 0; i < kSteps / 2; ++i) {
            mma_ts<kF8>(o_at, p + i * 8, v + i * kStepDesc, id_o, u > 0 || i > 0);
            if (kF8) {
              mma_ts<kF8>(o_at, p + 16 + i * 8, v + i * kStepDesc, id_o, true);
              mma_ts<kF8>(o_at, p + 32 + i * 8, v + i * kStepDesc, id_o, true);
            }
          }
          if (last) tc_commit(&v_empty[vc.at()]);
          tc_commit(&gr.pv_done[half]);  // last: the CTA may end soon after it
        }
        __syncwarp();
        if (last) vc.step(u + 2 >= steps ? 1 : by, size);
      }
      if (u + 2 >= steps) continue;
      const bool last = !pair || half == 1 || u + 3 == steps;
      if (first) wait_for(&k_full[kc.at()], kc.phase());
      if (elect_one() && ok) {
        const uint32_t k = k_desc + (k_base + kc.at()) * (unit >> 4) + half * later, s_to = s_at + half * 64;
#pragma unroll
        for (int i = 0; i < (kF8 ? 4 : 8); ++i) {
          if (!kFull && i >= ksteps) break;
          const uint32_t oq = kF8 ? i * 2 : (i >> 2) * kHalf + (i & 3) * 2;
          const uint32_t ok = kF8 ? i * 2 : (i >> 2) * halves_k + (i & 3) * 2;
          mma_ss<kF8>(s_to, q_desc + oq, k + ok, id_s, i > 0);
          if (kF8) mma_ss<kF8>(s_to, q_desc + kHalf + oq, k + ok, id_low, true);
        }
        tc_commit(&gr.s_full[half]);
        if (last) tc_commit(&k_empty[kc.at()]);
        if (u + 3 == steps) tc_commit(&gr.q_free[0]);
      }
      __syncwarp();
      if (last) kc.step(u == -2 ? 1 : by, size);
    }
  }

  __device__ void run() {
    const bool pair = __shfl_sync(0xffffffffu, sh.pair, 0);
    // K and V come in turn through the group's half of the ring, a tile or (single
    // wide items) half of one at a time, in the order of their use: K0 K1 V0 K2 V1 ..
    // K(n-1) V(n-2) V(n-1); or a pair's K through the first group's half and V
    // through the second's
    Cursor tiles, halves, pair_v;  // the item's first load (a pair's V, beside its K)
    uint32_t n_items = 0;
    int q_place = 0;  // the next narrow item's

    for (;;) {
      const Item *item_at = next();
      if (!__all_sync(0xffffffffu, item_at != nullptr)) break;
      const Item &it = *item_at;
      const int n = __shfl_sync(0xffffffffu, it.n, 0), narrow = __shfl_sync(0xffffffffu, it.narrow, 0);
      Cursor kc = tiles, vc = tiles;
      if (pair) {
        vc = pair_v;
        tiles.skip(n, P.part);
        pair_v.skip(n, P.part);
      } else if (narrow) {
        vc.step(n > 1 ? 2 : 1, P.part);
        tiles.skip(2 * n, P.part);
      } else {
        const int steps = __shfl_sync(0xffffffffu, it.steps, 0);
        kc = vc = halves;
        vc.step(steps > 1 ? 2 : 1, 2 * P.part);
        halves.skip(2 * steps, 2 * P.part);
      }
      const int place = narrow ? q_place : 0;
      if (narrow) q_place ^= 1;
      next_phase(&gr.q_ready[place], kQ0 << place);
      if (kF8 && narrow) narrow_item(it, n, place, kc, vc, n_items);
      else wide_item(it, kc, vc, pair, n_items);
      ++n_items;
      done();
    }
    if (sh.abort) fail();
  }
  // Slots past the last seen one hold whatever the cache or the ring holds
  // there: zeros in V, so that 0 times it stays 0.  (A pair's two warps write
  // the same zeros.)
  __device__ __forceinline__ void clear_tail(int seen, int rows, uint32_t v) {
    if (seen >= rows) return;
    for (int hf = 0; hf < P.halves; ++hf)
      for (uint32_t i = lane * 16; i < (uint32_t)(rows - seen) * 128; i += 512)
        *reinterpret_cast<uint4 *>(ring_smem + v + (hf * rows + seen) * 128 + i) = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    __syncwarp();
  }
  // Tensor and shared memory go only once the products under way are done, and a
  // copy of queries that another group's time-out left under way; on the usual path the
  // softmax warps, and who waits for the queries, have seen to that.
  __device__ void fail() {
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 1000000ull) __nanosleep(1000);
  }
};

// ---- K and V pages ---------------------------------------------------------------------
template <bool kF8>
__device__ void copy_pages(const AttParams &P, Shared &sh, int g, uint8_t *ring_smem, const CUtensorMap *k_map,
                           const CUtensorMap *v_map) {
  Role R(P, sh, g);
  if (P.withhold) return;
  Group &gr = R.gr;
  const bool pair = sh.pair;  // then one group's warp copies K, the other's V
  const int lane = R.lane, box = P.box_rows, chunks = kTile / box;
  const int chunk = lane / P.halves, half = lane - chunk * P.halves;  // this lane's copy of a tile
  const uint32_t slot_bytes = P.halves * kHalfBytes, ring = smem_addr(ring_smem) + g * P.part * slot_bytes;
  Cursor cursors[2];             // by half tiles, by tiles
  uint32_t used[2] = {0, 0};     // slots that have had a load
  int before = -1;               // how the item before came
  bool ok = true;
  while (const Item *item_at = R.next()) {
    const Item &it = *item_at;
    const int whole = pair || it.narrow, n = whole ? it.n : it.steps;
    const uint32_t size = whole ? P.part : 2 * P.part, unit = whole ? slot_bytes : slot_bytes / 2;
    const int rows = whole ? kTile : kHalfTile;
    uint64_t *const full = whole ? gr.full : gr.half_full, *const empty = whole ? gr.empty : gr.half_empty;
    Cursor c = whole ? cursors[1] : cursors[0];
    uint32_t most = whole ? used[1] : used[0];
    // the ring's slots change their places: all that is in it must have been used
    if (before >= 0 && before != whole) {
      Cursor other = whole ? cursors[0] : cursors[1];
      const uint32_t others = whole ? 2 * P.part : P.part;
#pragma unroll 1
      for (uint32_t i = 0; ok && i < others; ++i, other.step(1, others))
        ok = R.wait(whole ? &gr.half_empty[other.at()] : &gr.empty[other.at()], other.phase() ^ 1);
      if (!ok) break;
    }
    before = whole;
    const int32_t *tab = P.table + (size_t)it.b * P.table_stride;
    // A page is looked up a tile before its first copy; K runs a unit ahead of V,
    // in a pair each warp copies one of the two.
    const int last_k = pair && g ? 0 : n, last_v = pair && !g ? 0 : n;
    int page_now = -1, place_now = 0, page_v = -1, place_v = 0, page_next = -1, place_next = 0;
    auto look_up = [&](int t) {
      const int j = (it.tile0 + t) * kTile + chunk * box, at = j / P.page_size;
      page_next = -1;  // nothing to copy
      if (chunk >= chunks || t >= it.n || j >= it.seen) return;
      place_next = j - at * P.page_size;
      page_next = __ldg(tab + at);
      if (page_next < 0 || page_next >= P.num_pages) {
        atomicOr(R.status(), SV_FLAG_PAGE_RANGE);
        page_next = P.num_pages;  // outside the map: zeros
      }
    };
    int looked = -1;  // the tile that page_now is of
    look_up(0);
    int tk = last_k ? 0 : n, tv = last_v ? 0 : n;
#pragma unroll 1
    while (ok && (tk < n || tv < n)) {
      const bool value = tk >= n || (tv < n && tk > tv + 1);
      const int u = value ? tv : tk, t = whole ? u : u >> 1;
      if (t > looked) {  // on to the next tile's page
        page_v = page_now;
        place_v = place_now;
        page_now = page_next;
        place_now = place_next;
        looked = t;
        look_up(t + 1);
      }
      const int page = t < looked ? page_v : page_now, place = t < looked ? place_v : place_now;
      ok = R.wait(&empty[c.at()], c.phase() ^ 1);
      if (!ok) break;
      const int count = min(rows / box, (it.seen - it.tile0 * kTile - u * rows + box - 1) / box);
      if (lane == 0) mbar_arrive_expect_tx(&full[c.at()], (uint32_t)(count * P.halves * box * 128));
      __syncwarp();
      const int row = chunk * box - (whole ? 0 : (u & 1) * kHalfTile);  // of the unit
      if (page >= 0 && row >= 0 && row < rows)
        tma_load4(ring + c.at() * unit + (half * rows + row) * 128, value ? v_map : k_map, half * (kF8 ? 128 : 64), it.h,
                  place, page, &full[c.at()]);
      most = max(most, c.at() + 1);
      c.step(1, size);
      if (value) ++tv;
      else ++tk;
    }
    if (whole) {
      cursors[1] = c;
      used[1] = most;
    } else {
      cursors[0] = c;
      used[0] = most;
    }
    if (!ok) break;
    R.done();
  }
  if (!sh.abort) return;
  // a wait gave up: let the copies in flight land (each slot's newest)
  auto land = [&](uint64_t *full, const Cursor &c, uint32_t most) {
    for (uint32_t i = 0; i < most; ++i) {
      const uint32_t phase = i < c.at() ? c.phase() : c.phase() ^ 1;
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(&full[i], phase) && global_ns() - t0 < 1000000ull) {
      }
    }
  };
  land(gr.half_full, cursors[0], used[0]);
  land(gr.full, cursors[1], used[1]);
}

// ---- the tokens' scales (e4m3) -----------------------------------------------------------
// A tile's scale bytes come from memory kScaleAhead tiles early (its latency
// under load is that of several tiles), across items.
__device__ void scales(const AttParams &P, Shared &sh, int g, F8Group &f8) {
  Role R(P, sh, g);
  Group &gr = R.gr;
  const int lane = R.lane;
  uint32_t empty = 3;  // phases of sc_empty
  // the fetching side: the item and tile to fetch next, and how many are
  // fetched and not yet used
  Cursor f_item, f_at, u_at;
  int f_t = 0, under_way = 0;
  bool f_open = false, f_end = false;
  auto fetch = [&]() {  // one tile, if its item is known; a copy group in any case
    if (!f_open && !f_end && under_way < kScaleAhead &&
        __all_sync(0xffffffffu, mbar_try_wait(&gr.item_full[f_item.at()], f_item.phase()))) {
      f_open = gr.items[f_item.at()].n != 0;
      f_end = !f_open;
      f_t = 0;
    }
    if (f_open && under_way < kScaleAhead) {
      const Item &it = gr.items[f_item.at()];
      const int j = (it.tile0 + f_t) * kTile + 4 * lane;  // four tokens a lane, in one page
      uint32_t *dst = &f8.bytes[f_at.at()][0][lane];
      int page = -1;
      int64_t at = 0;
      if (j < it.seen) {
        const int pg = j / P.page_size;
        page = __ldg(P.table + (size_t)it.b * P.table_stride + pg);
        at = ((int64_t)page * P.Hkv + it.h) * P.page_size + (j - pg * P.page_size);
      }
      if (page >= 0 && page < P.num_pages) {
        copy4_async(dst, P.k_exp + at);
        copy4_async(dst + kTile / 4, P.v_exp + at);
      } else {
        dst[0] = dst[kTile / 4] = 0x01010101u;
      }
      f_at.step(1, kScaleAhead);
      ++under_way;
      if (++f_t == it.n) {
        f_open = false;
        f_item.step(1, kItems);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  while (const Item *item_at = R.next()) {
    const Item &it = *item_at;
    const int n = it.n;
    const int lazy = it.narrow ? kNarrowLazyF8 : kWideLazyF8;
    int run = 0, most = 0;  // R, the largest value exponent of late, and of all the item's
    for (int t = 0; t < n; ++t) {
#pragma unroll 1
      for (int tries = under_way ? 1 : kScaleAhead; tries > 0; --tries) fetch();
      // each fetched tile has a group of its own: all but the newest
      // under_way - 1 groups hold the oldest one's copies
      wait_copies(under_way - 1);
      uint32_t ke = f8.bytes[u_at.at()][0][lane], ve = f8.bytes[u_at.at()][1][lane];
      u_at.step(1, kScaleAhead);
      --under_way;
      const int left = min(it.seen - (it.tile0 + t) * kTile - 4 * lane, 4);  // bytes past the last slot mean nothing
      if (left < 4) {
        ke = left <= 0 ? 0 : ke & ((1u << 8 * left) - 1u);
        ve = left <= 0 ? 0 : ve & ((1u << 8 * left) - 1u);
      }
      int top = 1;
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, (int)(ve >> 8 * e & 0xff));
      // R rises at once, and falls when a tile's largest is more than kScaleDrop below
      // it, so that one large value costs the weights of its own tile's slots at most.  (O
      // is below 2^56 when it comes in, and grows as R falls: kScaleFall leaves it in range.)
      const int old = run;
      run = __reduce_max_sync(0xffffffffu, top);
      most = max(most, run);
      if (run < old) run = run < old - kScaleDrop ? max(run, most - kScaleFall) : old;
      // a narrow tile's scales go by its scores' buffer and are announced with them
      const int stage = it.narrow ? t & 1 : 0;
      ScaleStage &st = f8.sc[stage];
      if (!R.wait(&gr.sc_empty[stage], empty >> stage)) return;
      empty ^= 1u << stage;
      float a[4], w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int kb = ke >> 8 * e & 0xff, vb = ve >> 8 * e & 0xff;
        a[e] = kb ? scale_of_byte(kb) * P.c : 1.f;  // (a masked -inf stays one)
        const int x = vb - run + 127 + kTopF8 - lazy;  // weights up to 2^lazy are up to 2^kTopF8 in their codes
        w[e] = vb && x > 0 ? scale_of_byte(x) : 0.f;
      }
      *reinterpret_cast<float4 *>(&st.a[4 * lane]) = make_float4(a[0], a[1], a[2], a[3]);
      *reinterpret_cast<float4 *>(&st.w[4 * lane]) = make_float4(w[0], w[1], w[2], w[3]);
      if (lane == 0) {
        const int d = old - run + 127;
        st.shift = old == 0 ? 1.f : (d > 0 ? scale_of_byte(d) : 0.f);
        st.unit = ldexpf(1.f, run - 127 + lazy - kTopF8);
      }
      R.arrive(it.narrow ? &gr.s_full[2 + stage] : &gr.sc_full);
    }
    R.done();
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---- the items and their queries -----------------------------------------------------------
// Query rows lie in two halves of 128 bytes: kHalfBytes apart for a wide item, 32
// rows for a narrow one, whose rows past the last are zeros.  With e4m3 caches the
// high codes and then the low ones take the halves' place.
//
// A wide item's come with one TMA copy a half where its first row is a token's
// first and the copy's whole tokens have all its rows (with G = 5 they have 125, and
// a pair's half has 128): rows of other tokens that come along are never looked at.  (Row by row a
// wide item's took 5 to 9 us, for which its products waited.)  Otherwise all rows'
// copies are under way together.
__device__ __forceinline__ void copy_queries(const AttParams &P, const Item &it, int lane, uint8_t *tile) {
  const int per = P.D > 64 ? 16 : 8, v = lane % per, step = 32 / per;  // 16-byte pieces a row, rows at a time
  const bool in = 8 * v < P.D;
  const int rows = it.rows;
  const uint32_t half = it.narrow ? kNarrow * 128 : kHalfBytes;
  // the row's address advances by additions alone: by `on` a step, and by `wrap`
  // where the step passes the group's last head
  const int at = it.row0 + lane / per, tok = at / P.G, step_tok = step / P.G, step_gh = step - step_tok * P.G;
  int gh = at - tok * P.G;
  const int64_t on = step_tok * P.q_ts + step_gh * P.q_hs, wrap = P.q_ts - P.G * P.q_hs;
  const uint16_t *src = P.q + (int64_t)(it.q0 + tok) * P.q_ts + (int64_t)(it.h * P.G + gh) * P.q_hs + 8 * v;
  auto place = [&](int r) { return tile + r * 128 + (v >> 3) * half + (((v & 7) ^ (r & 7)) << 4); };
#pragma unroll 1
  for (int r = lane / per; r < rows; r += step) {
    if (in) copy16_async(place(r), src);
    gh += step_gh;
    src += on + (gh >= P.G ? wrap : 0);
    gh -= gh >= P.G ? P.G : 0;
  }
  for (int r = rows + lane / per; it.narrow && r < kNarrow; r += step) *reinterpret_cast<uint4 *>(place(r)) = make_uint4(0, 0, 0, 0);
  asm volatile("cp.async.wait_all;" ::: "memory");
}
// What the products need of them: a negative scale's sign, or the two codes.
template <bool kF8>
__device__ __forceinline__ void make_queries(const AttParams &P, const Item &it, int lane, float *scales, uint8_t *tile) {
  const uint32_t half = it.narrow ? kNarrow * 128 : kHalfBytes;
  const int rows = it.rows;
  __syncwarp();
  if (!kF8) {
    if (P.q_sign) {
      for (int i = lane; i < rows * 16; i += 32) {
        uint4 *at = reinterpret_cast<uint4 *>(tile + (i & 8 ? half : 0) + (i >> 4) * 128 + (i & 7) * 16);
        uint4 x = *at;
        x.x ^= P.q_sign;
        x.y ^= P.q_sign;
        x.z ^= P.q_sign;
        x.w ^= P.q_sign;
        *at = x;
      }
    }
  } else {
    // lane: values 4 lane .. of a row; they lie in 16-byte piece lane / 2
    const int pc = lane >> 1;
    const uint32_t from = (pc >> 3) * half + (lane & 1) * 8;
    const int all = it.narrow ? kNarrow : rows;
#pragma unroll 1  // (by fours, its code in the way of the others' cost 256 x 6 tokens 8 %)
    for (int r = 0; r < all; ++r) {
      uint2 x = make_uint2(0, 0);
      if (4 * lane < P.D) x = *reinterpret_cast<const uint2 *>(tile + r * 128 + from + (((pc & 7) ^ (r & 7)) << 4));
      x.x ^= P.q_sign;
      x.y ^= P.q_sign;
      uint32_t top = max(max(x.x & 0x7fffu, x.x >> 16 & 0x7fffu), max(x.y & 0x7fffu, x.y >> 16 & 0x7fffu));
      top = __reduce_max_sync(0xffffffffu, top);  // (and every lane has read the row)
      float inv;
      const float s = q_scale(top << 16, inv);
      uint32_t hi, lo;
      split_queries(bf16lo(x.x) * inv, bf16hi(x.x) * inv, bf16lo(x.y) * inv, bf16hi(x.y) * inv, hi, lo);
      uint8_t *dst = tile + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4;
      *reinterpret_cast<uint32_t *>(dst) = hi;
      *reinterpret_cast<uint32_t *>(dst + half) = lo;
      if (lane == 0) scales[r] = s;
    }
  }
  fence_async_smem();
}
// The next item's query rows on their way to L2 while the tile is still in use.
__device__ __forceinline__ void prefetch_queries(const AttParams &P, const Item &it, int lane) {
  const uint16_t *base = P.q + (int64_t)it.q0 * P.q_ts + (int64_t)it.h * P.G * P.q_hs;
  for (int r = lane; r < it.rows; r += 32) {
    const int at = it.row0 + r, tok = at / P.G;
    const uint16_t *src = base + tok * P.q_ts + (at - tok * P.G) * P.q_hs;
    for (int d = 0; d < P.D; d += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + d));
  }
}

template <bool kF8>
__device__ void hand_out(const AttParams &P, Shared &sh, int g, F8Group &f8, uint8_t *q_tile, const CUtensorMap *q_map) {
  Role R(P, sh, g);
  Group &gr = R.gr;
  Walk W(P, sh, g);
  Cursor c;
  // Narrow queries alternate between two places, each with its barriers, so that
  // the next item's are there when this one's scores end; wide ones take both
  // places and P's, with the first place's barriers.
  uint32_t uses[2] = {0, 0}, q_phase = 0;
  int q_place = 0, before = -1;  // the item before: 1 narrow, 0 wide; its entry
  Cursor last;
  for (;;) {
    const Item &it = gr.items[c.at()];
    bool more;
    {
      Item made;
      made.n = 0;
      more = W.next(made);
      if (!R.wait_limited(&gr.item_empty[c.at()], c.phase() ^ 1)) return;
      if (R.lane == 0) gr.items[c.at()] = made;
    }
    R.arrive(&gr.item_full[c.at()]);
    if (!more) break;
    prefetch_queries(P, it, R.lane);
    const int place = it.narrow ? q_place : 0;
    const bool both = !it.narrow || before == 0;
    if (!R.wait_limited(&gr.q_free[place], uses[place] ^ 1)) return;
    if (both && !R.wait_limited(&gr.q_free[place ^ 1], uses[place ^ 1] ^ 1)) return;
    // (P's space: the item before is done with)
    if (!it.narrow && before == 1 && !R.wait_limited(&gr.item_empty[last.at()], last.phase())) return;
    uint8_t *tile = q_tile + place * (kHalfBytes / 2);
    const int tok = it.row0 / P.G;
    if (!it.narrow && tok * P.G == it.row0 && it.rows <= P.q_box * P.G) {
      if (R.lane == 0) {
        fence_async_smem();  // (others wrote to the places before)
        const int halves = P.D > 64 ? 2 : 1;
        mbar_arrive_expect_tx(&gr.q_in, (uint32_t)(halves * P.q_box * P.G * 128));
        for (int hf = 0; hf < halves; ++hf)
          tma_load4(smem_addr(tile) + hf * kHalfBytes, q_map, 64 * hf, it.h * P.G, it.q0 + tok, 0, &gr.q_in);
      }
      if (!R.wait_limited(&gr.q_in, q_phase)) return;
      q_phase ^= 1;
    } else {
      copy_queries(P, it, R.lane, tile);
    }
    make_queries<kF8>(P, it, R.lane, f8.q_scale + place * kNarrow, tile);
    R.arrive(&gr.q_ready[place]);
    ++uses[place];
    if (it.narrow) q_place ^= 1;
    before = it.narrow;
    last = c;
    c.step(1, kItems);
  }
  R.wait_limited(&gr.finished, 0);
}

// ---- the kernel -----------------------------------------------------------------------
// Two values' sums over the CTA's threads before this one, and over all; and the
// largest of two more.
__device__ __forceinline__ void scan_before(const long long (&v)[2], const int (&w)[2], long long *smem,
                                            long long (&before)[2], long long (&all)[2], int (&most)[2]) {
  constexpr int kWarps = kThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int *most_smem = reinterpret_cast<int *>(smem + 2 * kWarps);
  auto scan = [&](long long x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    before[k] = scan(v[k]);
    most[k] = __reduce_max_sync(0xffffffffu, w[k]);
    if (lane == 31) {
      smem[k * kWarps + warp] = before[k];
      most_smem[k * kWarps + warp] = most[k];
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const long long warps = scan(lane < kWarps ? smem[k * kWarps + lane] : 0);
    const long long mine = __shfl_sync(0xffffffffu, warps, warp ? warp - 1 : 0);
    before[k] += (warp ? mine : 0) - v[k];
    all[k] = __shfl_sync(0xffffffffu, warps, 31);
    most[k] = __reduce_max_sync(0xffffffffu, most_smem[k * kWarps + (lane & (kWarps - 1))]);
  }
}

template <bool kF8, bool kFull>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const AttParams P, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                     const __grid_constant__ CUtensorMap q_map) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5;
  uint8_t *ring_smem = smem + 2 * kGroupBytes;

  if (tid == 0) {
    sh.abort = 0;
    sh.group[0].b0 = sh.group[1].b0 = P.B;
    prefetch_map(&k_map);
    prefetch_map(&v_map);
  }
  if (warp == 8) tmem_alloc_all(&sh.tmem);

  // The lines of work: every sequence's units, summed by kind and cut (each CTA
  // for itself: a few hundred lengths from L2, and no second launch).
  {
    long long *scan = reinterpret_cast<long long *>(smem);
    const int per = (P.B + kThreads - 1) / kThreads;
    const int b_lo = min(tid * per, P.B), b_hi = min(b_lo + per, P.B);
    long long sum[2] = {0, 0}, pre[2], all[2];
    int least[2] = {0, 0}, piece_least[2];
    for (int b = b_lo; b < b_hi; ++b) {
      const Seq s = read_seq(P, b);
      sum[s.pair()] += s.units(P) * P.Hkv;
      if (s.np) least[s.pair()] = max(least[s.pair()], s.least_piece(P));
      if (s.bad && blockIdx.x == 0) atomicOr(reinterpret_cast<uint32_t *>(P.ws), SV_FLAG_BAD_LEN);
    }
    scan_before(sum, least, scan, pre, all, piece_least);
    // CTAs for single items, then CTAs for pairs, so that the longer of the two
    // shares is as short as can be
    const int grid = gridDim.x;
    int singles = all[1] == 0 ? grid : (int)((float)all[0] / ((float)all[0] + (float)all[1]) * grid);
    if (all[0] && all[1]) {
      singles = max(1, min(singles, grid - 1));
      const float a = (float)all[0], b = (float)all[1];
      if (singles + 1 < grid && fmaxf(a / (singles + 1), b / (grid - singles - 1)) < fmaxf(a / singles, b / (grid - singles)))
        ++singles;
    }
    const int pair = (int)blockIdx.x >= singles;
    const int pieces = pair ? grid - singles : 2 * singles, cta0 = pair ? singles : 0;
    const long long piece = max(divide(all[pair] + pieces - 1, pieces), (long long)piece_least[pair]);
    for (int g = 0; g < 2; ++g) {
      const long long u0 = (pair ? (int)blockIdx.x - cta0 : 2 * (int)blockIdx.x + g) * piece;
      if (u0 >= pre[pair] && u0 < pre[pair] + sum[pair]) {
        long long at = pre[pair];
        for (int b = b_lo; b < b_hi; ++b) {
          const Seq s = read_seq(P, b);
          const long long x = s.pair() == (pair != 0) ? s.units(P) * P.Hkv : 0;
          if (u0 < at + x) {
            Group &gr = sh.group[g];
            gr.b0 = b;
            gr.u_b0 = at;
            gr.u0 = u0;
            gr.u1 = min(u0 + piece, all[pair]);
            break;
          }
          at += x;
        }
      }
    }
    if (tid == 0) {
      sh.pair = pair;
      sh.cta0 = cta0;
      sh.per = piece;
    }
    // the barriers, one a thread
    if ((tid & 63) < kBarriers && tid < 128) {
      const int i = tid & 63;
      int count = kF8 ? kCounts[1][i] : kCounts[0][i];
      if (i >= kMaxPart && i < 2 * kMaxPart && pair) count = 2;
      mbar_init(reinterpret_cast<uint64_t *>(&sh.group[tid >> 6]) + i, count);
      fence_barrier_init();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  // 128 registers a thread at launch (65,536 over 512 threads), shared out
  // again by warpgroup: 2 x 168 + 2 x 88 = 2 x 184 + 2 x 72 = 4 x 128.  Measured with
  // 168 / 176 / 184 for the softmax warps, us: 256 x 6 e4m3 tokens 402 / 412 / 417, bf16
  // trees of 16 nodes 148 / 144 / 144, 64 x 5 bf16 tokens 204 / 202 / 202.
  if (warp < 8) {
    const int g = warp >> 2;
    uint8_t *mine = smem + g * kGroupBytes;
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kF8 ? 168 : 184));
    Softmax<kF8>(P, sh, g, *reinterpret_cast<F8Group *>(mine + kF8Off), *reinterpret_cast<Rows *>(mine + kRowsOff),
                 mine + kPOff, sh.tmem)
        .run();
  } else {
    const int g = warp & 1;
    uint8_t *mine = smem + g * kGroupBytes;
    F8Group &f8 = *reinterpret_cast<F8Group *>(mine + kF8Off);
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kF8 ? 88 : 72));
    if (warp < 10) Products<kF8, kFull>(P, sh, g, smem, ring_smem, sh.tmem).run();
    else if (warp < 12) copy_pages<kF8>(P, sh, g, ring_smem, &k_map, &v_map);
    else if (warp < 14) hand_out<kF8>(P, sh, g, f8, mine, &q_map);
    else if (kF8) scales(P, sh, g, f8);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_free_all(sh.tmem);
  }
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once through the runtime (the
// library does not link the driver library).
EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// A tensor of 4 dimensions, innermost first, strides in bytes from the second
// on; a copy takes 128 bytes x box, swizzled.  L2 fetches 256 bytes where a row has
// them: fetching beyond a 128-byte row, into another head's, read a third more of an
// e4m3 cache from memory than the heads' own rows.
bool make_map(CUtensorMap *map, const void *base, bool f8, const cuuint64_t (&dims)[4], const cuuint64_t (&strides)[3],
              const cuuint32_t (&rest)[3]) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t box[4] = {f8 ? 128u : 64u, rest[0], rest[1], rest[2]}, ones[4] = {1, 1, 1, 1};
  return fn(map, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims,
            strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            dims[0] * (f8 ? 1 : 2) >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// K or V, [pages][page_size][heads][dim]: a copy takes `rows` slots of one head and page
bool cache_map(CUtensorMap *map, const void *base, const sv_kv_cache_t &c, int rows) {
  const bool f8 = c.dtype == SV_E4M3;
  const cuuint64_t esz = f8 ? 1 : 2;
  return make_map(map, base, f8, {(cuuint64_t)c.dim, (cuuint64_t)c.heads, (cuuint64_t)c.page_size, (cuuint64_t)c.num_pages},
                  {c.head_stride * esz, c.token_stride * esz, c.page_stride * esz}, {1, (cuuint32_t)rows, 1});
}
// queries, [tokens][heads][dim]: a copy takes a group's heads of q_box tokens
bool query_map(CUtensorMap *map, const AttParams &P) {
  if (P.q_hs == 0 || (P.q_ts == 0 && P.T > 1)) return false;  // (rows that are one another's: no map has them)
  const cuuint64_t ts = 2 * (P.T > 1 ? P.q_ts : P.Hq * P.q_hs);
  return make_map(map, P.q, false, {(cuuint64_t)P.D, (cuuint64_t)P.Hq, (cuuint64_t)P.T, 1},
                  {(cuuint64_t)P.q_hs * 2, ts, ts * P.T}, {(cuuint32_t)P.G, (cuuint32_t)P.q_box, 1});
}

template <bool kF8, bool kFull>
cudaError_t launch(const AttParams &P, const CUtensorMap (&maps)[3], int grid, size_t smem, cudaStream_t st) {
  const cudaError_t e =
      cudaFuncSetAttribute(attention_kernel<kF8, kFull>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  attention_kernel<kF8, kFull><<<grid, kThreads, smem, st>>>(P, maps[0], maps[1], maps[2]);
  return cudaGetLastError();
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

size_t sv_attention_workspace_bytes(void) { return kAttWsBytes; }

sv_status_t sv_attention_reset(void *workspace, size_t workspace_bytes, void *stream) {
  if (!workspace || !host_aligned(workspace, 256) || workspace_bytes < kAttWsBytes) return SV_ERR_WORKSPACE;
  return host_cuda_status(cudaMemsetAsync(workspace, 0, kPartOff, static_cast<cudaStream_t>(stream)));
}

sv_status_t sv_paged_attention(int B, int T, int q_heads, const sv_kv_cache_t *cache, sv_dtype_t dtype, const void *q,
                               int64_t q_token_stride, int64_t q_head_stride, const int32_t *q_start,
                               const int32_t *kv_len, const int32_t *block_table, int table_stride,
                               const int32_t *parents, int tree_nodes, float scale, void *out,
                               int64_t out_token_stride, int64_t out_head_stride, float *lse, void *workspace,
                               size_t workspace_bytes, void *stream) {
  if (B < 0 || B > (1 << 20) || T < 0 || q_heads < 1 || dtype != SV_BF16) return SV_ERR_INVALID;
  const sv_status_t cs = host_check_cache(cache);
  if (cs != SV_OK) return cs;
  if (cache->dim > kMaxDim || q_heads % cache->heads || q_heads / cache->heads > 128) return SV_ERR_INVALID;
  if (table_stride < 1 || !(scale == scale) || std::fabs(scale) > 1e30f) return SV_ERR_INVALID;
  if (parents && (tree_nodes < 1 || tree_nodes > SV_TREE_MAX_CHUNK)) return SV_ERR_INVALID;
  if (!workspace || !host_aligned(workspace, 256) || workspace_bytes < kAttWsBytes) return SV_ERR_WORKSPACE;
  if (B == 0 || T == 0) return SV_OK;
  if (!q || !out || q == out || !q_start || !kv_len || !block_table) return SV_ERR_INVALID;
  if (!host_aligned(q, 16) || !host_aligned(out, 16) || q_token_stride % 8 || q_head_stride % 8 ||
      out_token_stride % 8 || out_head_stride % 8 || q_token_stride < 0 || q_head_stride < 0 ||
      (T > 1 && out_token_stride < cache->dim) || (q_heads > 1 && out_head_stride < cache->dim))
    return SV_ERR_INVALID;
  const void *words[] = {q_start, kv_len, block_table, parents, lse};
  for (const void *p : words)
    if (!host_aligned(p, 4)) return SV_ERR_INVALID;
  if (cache->dtype == SV_E4M3 && (!host_aligned(cache->k_exp, 4) || !host_aligned(cache->v_exp, 4))) return SV_ERR_INVALID;
  const int G = q_heads / cache->heads;
  if ((int64_t)T * G > (1 << 30)) return SV_ERR_INVALID;
  int sms = 0;
  const sv_status_t ds = host_device_info(&sms);
  if (ds != SV_OK) return ds;
  if (sms > kMaxSms) return SV_ERR_UNSUPPORTED;

  const bool f8 = cache->dtype == SV_E4M3;
  AttParams P{};
  P.B = B;
  P.T = T;
  P.Hq = q_heads;
  P.Hkv = cache->heads;
  P.G = G;
  P.D = cache->dim;
  P.table_stride = table_stride;
  P.tree_nodes = tree_nodes;
  P.page_size = cache->page_size;
  P.num_pages = cache->num_pages;
  P.box_rows = gcd(cache->page_size, kHalfTile);
  P.halves = f8 || cache->dim <= 64 ? 1 : 2;
  const size_t fixed = 2 * kGroupBytes;
  const size_t fit = (kSmemLimit - kStaticBytes - fixed) / (P.halves * kHalfBytes);
  P.part = (int)(fit / 2 < kMaxPart ? fit / 2 : kMaxPart);
  P.q = static_cast<const uint16_t *>(q);
  P.out = static_cast<uint16_t *>(out);
  P.q_ts = q_token_stride;
  P.q_hs = q_head_stride;
  P.o_ts = out_token_stride;
  P.o_hs = out_head_stride;
  P.q_start = q_start;
  P.kv_len = kv_len;
  P.table = block_table;
  P.parents = parents;
  P.k_exp = f8 ? cache->k_exp : nullptr;
  P.v_exp = f8 ? cache->v_exp : nullptr;
  // (a factor of 0 would turn a masked -inf into NaN: as good as 0 is 2^-100)
  P.c = std::fmax(std::fabs(scale) * kLog2e, 7.9e-31f);
  P.q_sign = scale < 0.f ? 0x80008000u : 0u;
  P.lse = lse;
  P.ws = static_cast<uint8_t *>(workspace);
  unsigned long long limit = 0;
  host_wait_test(&limit, &P.withhold);
  P.wait_ns = limit ? limit : kWaitNs;

  CUtensorMap maps[3];  // of keys, values, and (if some item may be wide) queries
  if (!cache_map(&maps[0], cache->k, *cache, P.box_rows) || !cache_map(&maps[1], cache->v, *cache, P.box_rows))
    return SV_ERR_CUDA;
  maps[2] = maps[0];
  P.q_box = !f8 || (int64_t)T * G > kNarrow ? kTile / G : 0;
  if (P.q_box && !query_map(&maps[2], P)) P.q_box = 0;
  const size_t smem = fixed + (size_t)2 * P.part * P.halves * kHalfBytes;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const auto start = cache->dim == kMaxDim ? (f8 ? launch<true, true> : launch<false, true>)
                                           : (f8 ? launch<true, false> : launch<false, false>);
  return host_cuda_status(start(P, maps, sms, smem, st));
}

}  // extern "C"
