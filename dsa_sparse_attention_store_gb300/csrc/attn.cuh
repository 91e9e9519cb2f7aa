// Attention over the paged K/V cache: for a tree of drafted tokens (every
// committed key and the drafted ancestors) and over the indexer's selection.
//
// Mathematics, for a query row (one head of one token) and its visible keys:
//   s_j = scale q.k_j,  o = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m),
//   x_j = s_j log2 e,   lse = (m + log2 sum_j 2^(x_j - m)) / log2 e,
// in one pass over key tiles with a running m and sum. Statistics and the
// accumulator are fp32; the weights enter the second product as bf16 (its
// operands share a type, and a weight's relative error of 2^-8 is that of
// the output's own rounding); their sum is of the unrounded weights. ex2 is
// the hardware's, within 2^-22.
//
// Layout. A unit is one kv head of one sequence and up to 32, 128 or 256 of its
// rows (tokens x the G query heads that share the kv head), or, over a
// selection, one kv head of one token (G rows). The units' key tiles are laid
// end to end and cut into equal ranges, one per CTA, so ragged batches balance
// whatever their lengths. A unit that a cut divides leaves partial sums in the
// workspace and the join kernel adds them in a fixed order.
//
// Forms. Rows up to 128 (small trees, large groups) are bound by reading the
// cache: two CTAs per SM, so that one's softmax runs under the other's products,
// and the queries stay in TMEM as the A operand of the first product, which
// leaves shared memory to the tiles. Rows beyond that (kWide: large trees, chunks
// of a prefill) are bound by the tensor cores and by what L2 delivers: one CTA
// per SM with two groups of four softmax warps that share every tile between 256
// rows; queries in shared memory, which leaves TMEM for two score buffers, so
// that the next tile's scores are there when a tile's softmax ends. Up to 32 rows
// (kTreeFew, kSparseFew: a decode step, selections of usual groups) take one
// softmax warp and 8 KB of queries in shared memory, so two CTAs per SM have two
// score buffers as well.
//
// A CTA: one or two groups of softmax warps (4, or 1 for few rows; a row per
// thread and TMEM lane) and 4 loader warps. One thread issues a group's products:
// of the group's first warp where scores and softmax take turns anyway (a barrier
// of the four warps is cheaper than a hop to another warp), of a warp of its own
// with two score buffers, because issuing waits for the tensor cores' queue. TMEM columns
// of a group: accumulator [0, D), then one or two score buffers of 64 with the
// bf16 weights over them, then the queries where they are in TMEM. Keys and
// values pass through a ring of 64-key tiles in the 128-byte swizzle: K is
// read K-major, V MN-major.
//
// Loaders: a pair of warps brings keys, a pair values. In bf16, tiles that
// every row sees whole come by TMA boxes and selections by TMA gathers of four
// rows; tiles where visibility ends by 16-byte asynchronous copies straight
// into the swizzle. fp8 and fp4 codes come by asynchronous copies into a ring
// private to each thread, two or three tiles ahead, from where the thread
// widens them into the operand tile. Rows of no visible key are zeros there,
// never what the page holds: a weight of zero times a stale NaN would be NaN.
// In tiles that only some rows see, values that are not finite are replaced by
// zeros too and added afterwards to the rows that do see them (fix_nonfinite).
//
// What bounds it, and what it measures (device time of a call, join included,
// against a copy rate of 6.79 TB/s and 1909 bf16 TFLOP/s):
//  - one token of 64 sequences of 2048 to 16384, 8 kv heads, G 8, D 128, bf16:
//    HBM. 361 to 368 us, 6.6 TB/s. In fp8 350 us, fp4 335: the loaders' work on
//    a tile.
//  - 2048 tokens behind 8192, the same heads: the softmax of 64 keys takes about
//    2000 cycles of a group beside the products' 1330 (two groups; tensor pipe
//    52 %, issue slots 47 % busy). 508 us, 1220 TFLOP/s. In fp8 and fp4 675:
//    widening joins the chain.
//  - 8 tokens of 8 sequences of 131072, 4 kv heads, G 16, fp8: the chain of a
//    tile (scores, softmax, values: 276 us with a bf16 cache out of L2) and the
//    loaders, which share the issue slots with it (58 % busy; 300 us without the
//    widening's arithmetic). 347 us, 3.2 TB/s, 790 TFLOP/s.
//  - 2048 queries over 512 keys each, 8 kv heads, G 8, bf16: the loaders' time
//    to issue gathers (75 cycles each) and the start of a unit every 8 tiles;
//    nothing is saturated (issue slots 42 %, tensor pipe 39 % for 128 rows of
//    which 8 are real, L2 31 %). 575 us, 7.4 TB/s out of L2. In fp8 880, fp4 810:
//    widening 64 keys and values for 8 rows.
//  - listed units (spans): 2048 tokens behind 8192 with scores capped by a tanh,
//    bf16: the softmax of 64 keys takes 2670 cycles, 700 of them the cap's
//    polynomial (fp32 pipe 36 %, issue slots 46 %, tensor pipe 38 % busy). 688 us;
//    514 without a cap, 636 with a bias. A token of 64 sequences, capped: HBM, 372 us.
#pragma once
#include <type_traits>

#include "kv_format.cuh"
#include "ptx.cuh"

namespace dsa {
namespace at {

constexpr int kTile = kvf::kPage;  // keys of a tile: a page's, or 64 selected ones
// Entries of the per-tile and per-segment rings. A wait looks at one bit of an
// entry's round, so it may come neither a round early nor a round late. Not
// late: a tile's values are released only after the group's weights, for which
// it has read the tile's mask, loaders run at most 10 tiles past a value that
// is not released, and a group that has no rows in a unit releases its tiles
// only after it has read its last unit's segment entry (u_done). Not early:
// the second group of the wide form skips units of at most 128 rows without
// waiting for their tiles, so it may be any number of tiles ahead of the
// loaders; it looks at the entry of a unit's first tile only when it has that
// tile's scores, which exist after the loaders announced it, and from there on
// it goes tile by tile.
constexpr int kRing = 16;
enum Form { kTree = 0, kSparse = 1, kWide = 2, kTreeFew = 3, kSparseFew = 4, kForms = 5 };
constexpr int kFewRows = 32;
// Span form: a row's maximum moves when it is passed by 2^16, not the others'
// 2^8. With scores of a standard deviation of 4 that saves a sixth of the time
// of units of 9 tiles; the accumulator has room for values that add up to less
// than 2^111.
constexpr float kSpanStep = 16.f;

struct AttnArgs {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;
  long long qt, qh, ot, oh;  // strides, in elements
  const uint8_t* cache;
  const int32_t *page_table, *seq_lens, *cu_q, *sel;
  const uint32_t* mask;
  unsigned int* status;
  int4* meta;     // [2 x grid]
  float2* ml;     // [2 x grid][rows of a unit]
  float* part;    // [2 x grid][rows of a unit][D]
  float scale2;   // scale * log2 e
  int B, Tq, max_pages, num_pages, kv_heads, G, k, mask_words, slots;
};

// Units of the span form come from a list that its plan kernel writes (attn_span.cu):
// up to 32, 128 or 256 rows of neighbouring tokens and the tiles that one of them sees.
struct Unit {
  int b, q0, nd, len;     // row of the page table; first query, queries and keys of the rows' sequence (or group)
  int r0, t0, t1, base;   // first row among those queries' rows; tiles; whether the rows have keys in a shared prefix too
  int lo, full;           // every row sees the places from lo to before full
  int group_q0, group_at; // base: the group's first query, and the place of its first unit in the groups' list
};

// What a token sees: the places [lo, hi) of its sequence, and where it lies
// itself. ctx: places from there on are the new tokens, which a mask may hide.
struct Token {
  int lo, hi, place, ctx;
};

struct Cap {
  float cap2, to_cap;  // cap log2 e, 2 log2 e scale / cap; 0: no cap
  // Capped score log2 e / x in powers of x^2, and where that holds. x = q.k; in
  // kWideCap x = scale q.k / cap, a multiplication more, for there the powers of
  // scale / cap may leave fp32's range.
  float poly[5], poly_most;
  float to_ratio;  // scale / cap
};

struct SpanArgs : AttnArgs, Cap {
  const int4* units;   // [slots][3], the words of a Unit; without one t0 = t1 = 0
  const int* tiles;    // [slots] tiles of a unit, 0 where there is none
  const int4* tokens;  // [Tq]
  const float* slopes; // [heads] or null
  float fixed;               // what every row is weighed under where capped scores allow it, else -inf
  int units_n;
  int raw_mode;        // whole units' sums go to `raw`, for rows_join_kernel: 1 all, 2 those with Unit::base
  float2* raw_ml;      // [Tq][heads] maximum and sum of weights
  float* raw;          // [Tq][heads][D]
  int2* ends;          // [slots][kv_heads] the CTAs that have a unit's first and last tile, if raw_mode
};

// One stretch of a unit's key tiles.
struct Seg {
  int b, h;
  int r0, rows;       // first row of the unit among its sequence's rows, and how many
  int q0, nd, len;    // the sequence's first query, its queries, its keys (a selection: the query itself, ...)
  int t0, t1, nt;     // tiles [t0, t1) of the unit's, which end before nt
  int full;           // keys before this position are visible to every row
};
struct SpanSeg : Seg {
  int tb, lo, base;   // the unit's first tile; `full` holds from this position on; Unit::base
  int place;          // of the unit in the list
};

struct Start {
  int b, h, r, tile;
};

// What a kernel does to the scores. Not listed: the tree and the selection
// forms. The listed units' kernels are apart, because one with all of their code
// spilled (a chunk of 2048 tokens without a cap took 611 us in it, 568 alone):
// scores as they are; capped ones, all weighed under one exponent; biased ones,
// capped or not; and caps too wide for one exponent, biased or not, whose small
// scores need more care (the chunk with a bias and a cap of 20 took 1418 us by
// that kernel, 1298 by the biased one's).
enum Scores { kUnlisted = 0, kAsTheyAre = 1, kCapped = 2, kBiased = 3, kWideCap = 4, kScores = 5 };

template <int FMT, int D, int FORM, int SCORES = kUnlisted>
struct Cfg {
  static constexpr bool SPAN = SCORES != kUnlisted;
  // A segment's tiles from the last to the first: a bias makes the nearest keys'
  // weights the largest, so the maximum is known after the first tile and does
  // not move in every one (2048 tokens behind 8192 1176 -> 634 us). Without a
  // bias the first tile would be the one in which rows see the fewest keys
  // (packed documents 394 -> 429).
  static constexpr bool BACKWARDS = SCORES == kBiased || SCORES == kWideCap;
  // Results over the sum of the weights as the product has them, rounded to bf16:
  // without a running maximum even the weight of a row's only key is not 1, and
  // its rounding would come on top of the result's. In tiles that some row does
  // not see whole; rows of fewer than 64 keys have no others. (In all tiles, and
  // without a cap too, it cost 3 % of a decode step and 9 to 11 % of a chunk.)
  static constexpr bool ROUND = SCORES == kCapped;
  using Args = std::conditional_t<SPAN, SpanArgs, AttnArgs>;
  using Segment = std::conditional_t<SPAN, SpanSeg, Seg>;
  static constexpr bool SPARSE = FORM == kSparse || FORM == kSparseFew;
  static constexpr bool FEW = FORM == kTreeFew || FORM == kSparseFew;
  static constexpr bool TWO = FORM == kWide || FEW;    // two score buffers, queries in shared memory, warps that issue the products
  static constexpr int WG = FORM == kWide ? 2 : 1;     // groups of softmax warps
  static constexpr int SW = FEW ? 1 : 4;               // softmax warps of a group
  static constexpr int QROWS = 32 * SW;                // rows of a group
  static constexpr int ROWS = QROWS * WG;              // rows of a unit
  static constexpr int SBUF = TWO ? 2 : 1;             // score buffers
  static constexpr int THREADS = ROWS + 128 + (TWO ? 32 * WG : 0);
  static constexpr int CTAS = FORM == kWide ? 1 : 2;   // per SM
  static constexpr int NBLK = D / 64;
  static constexpr int SLOT = kTile * D * 2;
  // chunks of 16 code bytes: of a row's 64 dimensions, and a loader thread's per tile
  static constexpr int CPB = FMT == DSA_FMT_BF16 ? 8 : FMT == DSA_FMT_FP8 ? 4 : 2;
  static constexpr int NCH = NBLK * CPB;
  static constexpr bool RAW = FMT != DSA_FMT_BF16;
  static constexpr int RAW_SLOT = RAW ? NCH * 64 * 16 + 64 * 4 + (D == 64 ? 64 * 4 : 0) : 0;  // codes, a scale word a row, flags
  // ring depths that fill the shared memory (113 KB or 227 KB a CTA): operand tiles, and tiles of codes
  // on their way of each loader pair
  static constexpr int P = !RAW ? 3 : FMT == DSA_FMT_FP8 || (FEW && D == 128) ? 2 : 3;
  static constexpr int NS = D == 64 ? (FORM == kWide || !RAW ? 12 : 10)
                            : FORM == kWide ? (!RAW ? 10 : FMT == DSA_FMT_FP8 ? 7 : 8)
                                            : (!RAW ? 6 : FMT == DSA_FMT_FP8 ? 4 : 5);
  static constexpr int QBYTES = TWO ? ROWS * D * 2 : 0;
  // TMEM columns of a group, and of the CTA (two CTAs share the SM's 512)
  static constexpr uint32_t O = 0, S = D, Q = D + 64 * SBUF, STRIDE = 256, TMEM = 256 * WG;
};

struct Shared {
  uint64_t full[12], empty[12];
  uint64_t mfull[kRing], vdone[kRing];
  // by group and score buffer (a barrier per buffer: no phase can complete twice
  // before a wait for it): scores there, weights there, their product done; by
  // group: queries there, a unit's segment entry read, the end
  uint64_t s_full[2][2], o_full[2][2], p_ready[2][2], q_ready[2], u_done[2], fin[2];
  unsigned long long vmask[kRing];  // visible keys of a tile, as far as the loader knows
  int bad[kRing];                      // segment number + 1 where a loader replaced a value
  int info[4][4];                      // a loader warp's tiles on their way
  long long scan[16];
  Start start;
  uint32_t tmem;
  int abort;
};

template <class C>
constexpr int smem_bytes() {
  return C::NS * C::SLOT + C::QBYTES + 2 * C::P * C::RAW_SLOT + static_cast<int>(sizeof(Shared));
}

// Key tiles of the row tile that starts at row r0 (at least one, so that
// rows without a key are written too).
template <class C>
__device__ __forceinline__ int tiles_of(const AttnArgs& a, int nd, int len, int r) {
  int end = len;
  // Rows are below 2^31, so the tile's last one has 32 bits. In 64 the plan's
  // divisions, one a row tile in one thread, and those of every unit's start
  // took 23 of 440 us of a chunk of 4096 tokens (8 kv heads, G 8), 114 of 828
  // with one kv head of 64 query heads.
  if (!a.mask) {
    const uint32_t seen = (static_cast<uint32_t>(r + 1) * C::ROWS - 1) / static_cast<uint32_t>(a.G) + 1;
    end = len - nd + static_cast<int>(min(static_cast<uint32_t>(nd), seen));
  }
  return max(1, (end + kTile - 1) / kTile);
}

// 64-key tiles of a query's selection and, after them, the drafted tokens
__device__ __forceinline__ int selection_tiles(const AttnArgs& a) {
  return (a.k + kTile - 1) / kTile + (a.mask ? (a.mask_words + 1) / 2 : 0);
}

__device__ __forceinline__ bool read_seq(const AttnArgs& a, int b, int& q0, int& nd, int& len) {
  q0 = a.cu_q[b];
  const int q1 = a.cu_q[b + 1];
  len = a.seq_lens[b];
  nd = q1 - q0;
  return q0 >= 0 && q1 >= q0 && q1 <= a.Tq && len >= nd && static_cast<long long>(len) <= 64LL * a.max_pages;
}

template <class C>
struct Iter {
  const typename C::Args& a;
  long long left;
  int b, h, r, tile;  // span form: b is the unit's place in the list
  int q0, nd, len, nrt;
  bool ok;
  __device__ Iter(const typename C::Args& a_, const Start& s, long long n) : a(a_), left(n), b(s.b), h(s.h), r(s.r), tile(s.tile) {
    if constexpr (!C::SPAN) start();
  }
  __device__ void start() {
    ok = read_seq(a, b, q0, nd, len);
    nrt = static_cast<int>((static_cast<long long>(nd) * a.G + C::ROWS - 1) / C::ROWS);
  }
  // the next stretch; a selection's r is its query
  __device__ bool next(typename C::Segment& s) {
    if (left <= 0) return false;
    if constexpr (C::SPAN) {
      int4 x, y, z;
      while (true) {
        x = a.units[3 * b];
        y = a.units[3 * b + 1];
        z = a.units[3 * b + 2];
        if (y.y < y.z) break;  // a gap of the list has no tiles
        advance();
      }
      s.b = x.x;
      s.q0 = x.y;
      s.nd = x.z;
      s.len = x.w;
      s.r0 = y.x;
      s.tb = y.y;
      s.nt = y.z;
      s.base = y.w;
      s.lo = z.x;
      s.full = z.y;
      s.place = b;
      s.rows = static_cast<int>(min(static_cast<long long>(C::ROWS), static_cast<long long>(s.nd) * a.G - s.r0));
      s.h = h;
      s.t0 = s.tb + tile;
      const long long room = s.nt - s.t0;
      s.t1 = left < room ? s.t0 + static_cast<int>(left) : s.nt;
      left -= s.t1 - s.t0;
      tile = 0;
      advance();
      return true;
    }
    if constexpr (C::SPARSE) {
      while (b + 1 < a.B && a.cu_q[b + 1] <= r) {
        ++b;
        ok = read_seq(a, b, q0, nd, len);
      }
      s.nt = selection_tiles(a);
      s.r0 = 0;
      s.rows = a.G;
      s.q0 = r;
      const bool mine = ok && r >= q0 && r < q0 + nd;  // not so only for inconsistent lengths
      s.nd = mine ? nd : 0;
      s.len = mine ? len : 0;
      s.full = 0;
    } else {
      while (!ok || nrt == 0) {
        if (++b >= a.B) return false;
        ok = read_seq(a, b, q0, nd, len);
        nrt = static_cast<int>((static_cast<long long>(nd) * a.G + C::ROWS - 1) / C::ROWS);
        h = r = tile = 0;
      }
      s.nt = tiles_of<C>(a, nd, len, r);
      s.r0 = r * C::ROWS;
      s.rows = min(C::ROWS, nd * a.G - s.r0);
      s.q0 = q0;
      s.nd = nd;
      s.len = len;
      s.full = len - nd + (a.mask ? 0 : s.r0 / a.G + 1);
    }
    s.b = b;
    s.h = h;
    s.t0 = tile;
    const long long room = s.nt - tile;
    s.t1 = left < room ? tile + static_cast<int>(left) : s.nt;
    left -= s.t1 - s.t0;
    tile = 0;
    if constexpr (C::SPARSE) {
      if (++h == a.kv_heads) {
        h = 0;
        ++r;
      }
    } else {
      if (++r == nrt) {
        r = 0;
        if (++h == a.kv_heads) {
          h = 0;
          nrt = 0;  // on to the next sequence
        }
      }
    }
    return true;
  }
  // span form: the next place of the list, then the next kv head's turn at it
  __device__ void advance() {
    if constexpr (C::SPAN)
      if (++b == a.units_n) {
        b = 0;
        ++h;
      }
  }
};

// Where CTA c's share of total tiles begins, of n CTAs.
__device__ __forceinline__ long long share(long long total, int c, int n) {
  if (total < 0x7FFFFFFFLL) {  // by divisions of 32 bits
    const uint32_t t = static_cast<uint32_t>(total), q = t / n;
    return static_cast<long long>(q) * c + (t - q * n) * static_cast<uint32_t>(c) / n;
  }
  return total / n * c + total % n * c / n;
}

// The launch's tiles, and where this CTA's range begins. Every thread of
// the block calls it; the result is in sh.
template <class C>
__device__ __forceinline__ void make_plan(const typename C::Args& a, Shared& sh, int cta, int grid, long long& begin, long long& count) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long total;
  constexpr int kThreads = C::THREADS;
  if constexpr (C::SPARSE) {
    const int nt = selection_tiles(a);
    total = static_cast<long long>(a.Tq) * a.kv_heads * nt;
    const long long n = total < grid ? total : grid;
    begin = cta < n ? total * cta / n : total;
    count = cta < n ? total * (cta + 1) / n - begin : 0;
    if (tid == 0) {
      const long long u = begin / nt;
      sh.start = Start{0, static_cast<int>(u % a.kv_heads), static_cast<int>(u / a.kv_heads), static_cast<int>(begin % nt)};
    }
    __syncthreads();
    // the sequence of the first query
    const int t = sh.start.r;
    for (int b = tid; b < a.B; b += kThreads) {
      int q0, nd, len;
      const bool ok = read_seq(a, b, q0, nd, len);
      if (!ok && cta == 0) atomicOr(a.status, DSA_DEV_BOUNDS);
      if (ok && q0 <= t && t < q0 + nd) sh.start.b = b;
    }
    __syncthreads();
    return;
  }
  // each thread adds up a run of sequences (or of the list); a scan over the threads places them
  int N = a.B;
  if constexpr (C::SPAN) N = a.units_n;
  const int per = (N + kThreads - 1) / kThreads;
  const int b0 = min(N, tid * per), b1 = min(N, b0 + per);
  auto weigh = [&](int b) -> long long {
    if constexpr (C::SPAN) return a.tiles[b];
    int q0, nd, len;
    if (!read_seq(a, b, q0, nd, len)) {
      if (cta == 0) atomicOr(a.status, DSA_DEV_BOUNDS);
      return 0;
    }
    const int nrt = static_cast<int>((static_cast<long long>(nd) * a.G + C::ROWS - 1) / C::ROWS);
    long long n = 0;
    if (a.mask)
      n = static_cast<long long>(nrt) * tiles_of<C>(a, nd, len, 0);
    else
      for (int r = 0; r < nrt; ++r) n += tiles_of<C>(a, nd, len, r);
    return n * a.kv_heads;
  };
  long long sum = 0, last = 0;
  for (int b = b0; b < b1; ++b) sum += last = weigh(b);
  long long inc = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) sh.scan[warp] = inc;
  __syncthreads();
  long long before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sh.scan[w];
    total += sh.scan[w];
  }
  const long long ex = before + inc - sum;
  [[maybe_unused]] const long long head = total;  // span form: the list's tiles, which every kv head has
  if constexpr (C::SPAN) total *= a.kv_heads;
  const long long n = total < grid ? total : grid;
  if constexpr (C::SPAN) {
    begin = cta < n ? share(total, cta, static_cast<int>(n)) : total;
    count = cta < n ? share(total, cta + 1, static_cast<int>(n)) - begin : 0;
    if (count > 0) {
      const long long h = total < 0x7FFFFFFFLL ? static_cast<uint32_t>(begin) / static_cast<uint32_t>(head) : begin / head;
      long long x = begin - h * head - ex;
      if (0 <= x && x < sum) {
        int b = b0;
        for (long long w; x >= (w = weigh(b)); ++b) x -= w;
        sh.start = Start{b, static_cast<int>(h), 0, static_cast<int>(x)};
      }
    }
    __syncthreads();
    return;
  }
  begin = cta < n ? total * cta / n : total;
  count = cta < n ? total * (cta + 1) / n - begin : 0;
  if (count > 0 && ex <= begin && begin < ex + sum) {
    long long x = begin - ex;
    int b = b0;
    while (b + 1 < b1) {  // a single sequence needs no second look
      const long long w = weigh(b);
      if (x < w) break;
      x -= w;
      ++b;
    }
    int q0, nd, len;
    read_seq(a, b, q0, nd, len);
    const long long w = b1 - b0 == 1 ? last : weigh(b);
    const long long ph = w / a.kv_heads;
    const int h = static_cast<int>(x / ph);
    x -= h * ph;
    int r = 0;
    while (true) {
      const int nt = tiles_of<C>(a, nd, len, r);
      if (x < nt) break;
      x -= nt;
      ++r;
    }
    sh.start = Start{b, h, r, static_cast<int>(x)};
  }
  __syncthreads();
}

// The low n bits, n clamped to 0 .. 64.
__device__ __forceinline__ unsigned long long low_bits(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// Of the 64 keys from position p0 on, those that token `token`, which sees `y`, may see.
__device__ __forceinline__ unsigned long long span_mask(const AttnArgs& a, long long token, const Token& y, int p0) {
  unsigned long long m = low_bits(y.hi - p0) & ~low_bits(y.lo - p0);
  if (a.mask && p0 + 64 > y.ctx) {
    const uint32_t* w = a.mask + token * a.mask_words;
    auto word = [&](int j) -> uint32_t { return j < a.mask_words ? w[j] : 0u; };
    const int n = y.ctx - p0;  // committed keys of the tile, if positive
    if (n > 0) {
      m &= low_bits(n) | ((word(0) | (static_cast<unsigned long long>(word(1)) << 32)) << n);
    } else {
      const int j = -n >> 5, sh = -n & 31;
      const uint32_t w0 = word(j), w1 = word(j + 1), w2 = word(j + 2);
      m &= __funnelshift_r(w0, w1, sh) | (static_cast<unsigned long long>(__funnelshift_r(w1, w2, sh)) << 32);
    }
  }
  return m;
}

// Of the 64 keys from position p0 on, those that a row of query i may see (tree form).
__device__ __forceinline__ unsigned long long row_mask(const AttnArgs& a, const Seg& s, int i, int p0) {
  const int ctx = s.len - s.nd;
  if (!a.mask) return low_bits(ctx + i + 1 - p0);
  const uint32_t* w = a.mask + static_cast<long long>(s.q0 + i) * a.mask_words;
  auto word = [&](int j) -> uint32_t { return j < a.mask_words ? w[j] : 0u; };
  const int o = p0 - ctx;
  if (o >= 0) {
    const int j = o >> 5, sh = o & 31;
    const uint32_t w0 = word(j), w1 = word(j + 1), w2 = word(j + 2);
    return __funnelshift_r(w0, w1, sh) | (static_cast<unsigned long long>(__funnelshift_r(w1, w2, sh)) << 32);
  }
  const int n = -o;  // committed keys of the tile
  if (n >= 64) return ~0ull;
  return low_bits(n) | ((word(0) | (static_cast<unsigned long long>(word(1)) << 32)) << n);
}

__device__ __forceinline__ Token token_at(const SpanArgs& a, long long t) {
  const int4 y = a.tokens[t];
  return Token{y.x, y.y, y.z, y.w};
}

// The place a token measures its keys' distance from: its own, or the nearest
// that it sees. Softmax takes no notice of the difference; exponents stay small
// for the keys that matter where all of them are far away. away(): how far that
// place is, for lse.
__device__ __forceinline__ int nearest(const Token& y) { return max(y.lo, min(y.place, y.hi - 1)); }
__device__ __forceinline__ float away(const Token& y) { return fabsf(static_cast<float>(y.place - nearest(y))); }

// One step of turning four lanes' four 16-byte runs around: lanes that differ in
// bit N exchange the runs that differ in it.
template <int N>
__device__ __forceinline__ void swap_runs(uint32_t (&w)[4][4], bool upper) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i & N) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? w[i][e] : w[i | N][e], N);
      if (upper)
        w[i][e] = got;
      else
        w[i | N][e] = got;
    }
  }
}

// 64 bytes of each lane's row to `to`, null for none
__device__ __forceinline__ void store_runs(uint32_t (&w)[4][4], void* to) {
  const int lane = threadIdx.x & 31;
  swap_runs<1>(w, lane & 1);
  swap_runs<2>(w, lane & 2);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned long long p = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), (lane & 28) + i);
    if (p) reinterpret_cast<uint4*>(p)[lane & 3] = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
  }
}

// cap tanh(y), y = scale q.k / cap, times log2 e. Where all |y| are at most
// kCapPoly y P(y^2) with a minimax polynomial on the fp32 pipe, within 2^-20 of
// itself however small y is. Else 1 - 2 / (1 + e^2y), for infinities too, by two
// operations of the special-function unit. Its error of 2^-22 is one of 1, for
// the difference cancels where y is small, and so one of cap in the score: enough
// for caps of up to 62 (2^-16).
constexpr int kCapTerms = 5;
constexpr double kCapPoly = 0.625;
constexpr float kCapOne = 90.f;  // cap log2 e up to which the rows can be weighed under one exponent

// Cap::poly at two x^2
__device__ __forceinline__ unsigned long long cap_factor(const Cap& a, unsigned long long u) {
  unsigned long long y = pack2(a.poly[kCapTerms - 1], a.poly[kCapTerms - 1]);
#pragma unroll
  for (int k = kCapTerms - 2; k >= 0; --k) y = fma2(y, u, pack2(a.poly[k], a.poly[k]));
  return y;
}

// In TMEM, where a tile's scores stay capped: in registers the 64 chains spill.
__device__ __forceinline__ void cap_any(const SpanArgs& a, uint32_t taddr) {
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t x[32];
    tmem_ld32(taddr + 32 * c, x);
    tmem_ld_wait32(x);
#pragma unroll
    for (int i = 0; i < 32; ++i)
      x[i] = __float_as_uint(fmaf(-2.f * a.cap2, rcp(1.f + ex2(__uint_as_float(x[i]) * a.to_cap)), a.cap2));
    tmem_st32(taddr + 32 * c, x);
  }
  tmem_st_wait();
}

// The same for wide caps: scores that are small enough take the polynomial beside
// others that are not (a key at -cap has no weight, and those that have some may
// have small scores). Not inlined: the code that few tiles reach cost the others
// more registers (2048 tokens behind 8192 with a cap of 63 992 us, so 927).
inline __device__ __noinline__ void cap_each(const Cap a, uint32_t taddr) {
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t x[32];
    tmem_ld32(taddr + 32 * c, x);
    tmem_ld_wait32(x);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float x0 = __uint_as_float(x[i]), x1 = __uint_as_float(x[i + 1]);
      const unsigned long long y = mul2(pack2(x0, x1), pack2(a.to_ratio, a.to_ratio)), u = mul2(y, y);
      float u0, u1, y0, y1;
      unpack2(u, u0, u1);
      unpack2(mul2(cap_factor(a, u), y), y0, y1);
      // twice the largest caps is no fp32 number
      const float z0 = fmaf(-2.f * rcp(1.f + ex2(x0 * a.to_cap)), a.cap2, a.cap2);
      const float z1 = fmaf(-2.f * rcp(1.f + ex2(x1 * a.to_cap)), a.cap2, a.cap2);
      x[i] = __float_as_uint(u0 <= a.poly_most ? y0 : z0);
      x[i + 1] = __float_as_uint(u1 <= a.poly_most ? y1 : z1);
    }
    tmem_st32(taddr + 32 * c, x);
  }
  tmem_st_wait();
}

// 64 scores capped by the polynomial, in place; whether all of a row's were
// small enough for it.
template <bool RATIO>
__device__ __forceinline__ bool cap_near(const SpanArgs& a, uint32_t (&x)[2][32]) {
  float most = 0.f;
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      unsigned long long s = pack2(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1]));
      if constexpr (RATIO) s = mul2(s, pack2(a.to_ratio, a.to_ratio));
      const unsigned long long u = mul2(s, s);
      float u0, u1, y0, y1;
      unpack2(u, u0, u1);
      unpack2(mul2(cap_factor(a, u), s), y0, y1);
      most = fmaxf(most, fmaxf(u0, u1));
      x[c][2 * i] = __float_as_uint(y0);
      x[c][2 * i + 1] = __float_as_uint(y1);
    }
  return most <= a.poly_most;
}

// Takes slope |from - j| off 64 exponents of 2; `from` counts from the first
// key. Where no key lies past it in any of the warp's rows the bias is slope (j -
// from), of which slope from is left to the caller: one operation a score.
__device__ __forceinline__ float bias_scores(uint32_t (&x)[2][32], float slope2, float from, bool edge) {
  asm volatile("" : "+f"(slope2), "+f"(from));  // or the 64 products move out of the loop around, into registers there are not
  if (!edge) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < 32; ++i) x[c][i] = __float_as_uint(fmaf(slope2, static_cast<float>(32 * c + i), __uint_as_float(x[c][i])));
    return -slope2 * from;
  }
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < 32; ++i)
      x[c][i] = __float_as_uint(fmaf(-slope2, fabsf(from - static_cast<float>(32 * c + i)), __uint_as_float(x[c][i])));
  return 0.f;
}

// The weights 2^(x - sub) of a row's 64 keys, as bf16 pairs, their sum, and the
// largest exponent x. x = mul score; or, CAP, the score capped by the
// polynomial, and instead of the largest exponent, which nobody asks for, the
// largest (q.k)^2.
struct Weighed {
  float most, sum, rounded;  // ROUNDED: the sum of the weights as they go into the product, too (else the same sum)
};

template <bool CAP, bool ROUNDED = false>
__device__ __forceinline__ Weighed weigh(const SpanArgs& a, const uint32_t (&x)[2][32], uint32_t (&p)[32], float mul, float sub) {
  const unsigned long long sc = pack2(mul, mul), sb = pack2(-sub, -sub);
  unsigned long long sum[2] = {0ull, 0ull};  // pairs of fp32 zeros
  constexpr float kLeast = CAP ? 0.f : -INFINITY;
  float mx[4] = {kLeast, kLeast, kLeast, kLeast}, rounded[2] = {0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const unsigned long long s = pack2(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1]));
      const unsigned long long u = CAP ? mul2(s, s) : s;
      float e0, e1;
      unpack2(u, e0, e1);
      mx[i & 3] = fmaxf(mx[i & 3], fmaxf(e0, e1));
      unpack2(CAP ? fma2(s, cap_factor(a, u), sb) : fma2(s, sc, sb), e0, e1);
      e0 = ex2(e0);
      e1 = ex2(e1);
      sum[i & 1] = add2(sum[i & 1], pack2(e0, e1));
      const __nv_bfloat162 w = __floats2bfloat162_rn(e0, e1);
      memcpy(&p[16 * c + i], &w, 4);
      if constexpr (ROUNDED) {
        rounded[0] = add_bf16(rounded[0], __bfloat16_as_ushort(w.x));
        rounded[1] = add_bf16(rounded[1], __bfloat16_as_ushort(w.y));
      }
    }
  float l0, l1;
  unpack2(add2(sum[0], sum[1]), l0, l1);
  const float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
  return Weighed{CAP ? most : most * mul, l0 + l1, ROUNDED ? rounded[0] + rounded[1] : l0 + l1};
}

__device__ __forceinline__ float widen_one(uint32_t bits) { return __uint_as_float(bits << 16); }

// Adds the values that are not finite, of the pages [t0, t1) that hold keys
// only some rows see, to the rows that see them. Only reached where a loader
// found one.
template <int FMT, int D, class Segment>
__device__ __noinline__ void fix_nonfinite(const AttnArgs& a, const Segment& s, int t0, int t1, int i, bool valid, uint32_t o_taddr,
                                           const Token tok = Token{}) {
  using L = kvf::Layout<FMT, D>;
  for (int d = 0; d < D; ++d) {
    float add = 0.f;
    for (int t = t0; t < t1; ++t) {
      if (t * kTile >= s.len) break;
      constexpr bool SPAN = std::is_same_v<Segment, SpanSeg>;
      if constexpr (SPAN) {
        if (t * kTile >= s.lo && (t + 1) * kTile <= s.full) continue;  // tiles that every row sees kept theirs
      }
      const int page = a.page_table[static_cast<long long>(s.b) * a.max_pages + t];
      if (page < 0 || page >= a.num_pages) continue;
      const uint8_t* blk = a.cache + (static_cast<long long>(page) * a.kv_heads + s.h) * L::HEAD_BYTES;
      unsigned long long m = !valid ? 0ull : SPAN ? span_mask(a, s.q0 + i, tok, t * kTile) : row_mask(a, s, i, t * kTile);
      m &= low_bits(s.len - t * kTile);
      while (m) {
        const int j = __ffsll(static_cast<long long>(m)) - 1;
        m &= m - 1;
        float v = 0.f;
        if constexpr (FMT == DSA_FMT_BF16)
          v = widen_one(reinterpret_cast<const uint16_t*>(blk + L::V_CODES)[j * D + d]);
        else
          v = blk[L::V_SCALES + j * L::SB + d / kvf::kBlock] == 255 ? __uint_as_float(0x7FFFFFFFu) : 0.f;
        if ((__float_as_uint(v) & 0x7F800000u) == 0x7F800000u) add += v;
      }
    }
    __syncwarp();  // the lanes' keys differ; the load takes them together
    const float o = __uint_as_float(tmem_ld1(o_taddr + d));
    __syncwarp();
    tmem_st1(o_taddr + d, __float_as_uint(o + add));
  }
}

template <int FMT, int D, int FORM, int SCORES>
__global__ void __launch_bounds__(Cfg<FMT, D, FORM, SCORES>::THREADS, Cfg<FMT, D, FORM, SCORES>::CTAS)
    attn_kernel(const __grid_constant__ CUtensorMap tm, const typename Cfg<FMT, D, FORM, SCORES>::Args a) {
  using C = Cfg<FMT, D, FORM, SCORES>;
  using Segment = typename C::Segment;
  using L = kvf::Layout<FMT, D>;
  constexpr int NSW = C::SW * C::WG;  // softmax warps
  extern __shared__ __align__(1024) uint8_t smem[];
  // Queries first: the first product reads 128 rows of them whatever a group
  // has, in the few-row forms the ring's bytes beyond 32. What comes of those
  // stays in accumulator lanes that nothing reads.
  uint8_t* const qsm = smem;
  uint8_t* const tiles = smem + C::QBYTES;
  uint8_t* const raw = tiles + C::NS * C::SLOT;
  static_assert(C::QBYTES + C::NS * C::SLOT >= 128 * D * 2, "queries that the first product reads");
  Shared& sh = *reinterpret_cast<Shared*>(raw + 2 * C::P * C::RAW_SLOT);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, grid = gridDim.x;

  if (tid == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&sh.full[i], 2);  // a pair of loader warps
      mbar_init(&sh.empty[i], C::WG);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sh.mfull[i], 1);
      mbar_init(&sh.vdone[i], 2);
      sh.bad[i] = 0;
    }
    mbar_init(&sh.fin[0], 1);
    mbar_init(&sh.fin[1], 1);
    for (int i = 0; i < C::WG; ++i) {
      mbar_init(&sh.s_full[i][0], 1);
      mbar_init(&sh.s_full[i][1], 1);
      mbar_init(&sh.p_ready[i][0], C::SW);
      mbar_init(&sh.p_ready[i][1], C::SW);
      mbar_init(&sh.q_ready[i], C::SW);
      mbar_init(&sh.u_done[i], C::SW);
      mbar_init(&sh.o_full[i][0], 1);
      mbar_init(&sh.o_full[i][1], 1);
    }
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&sh.tmem, C::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  long long begin, count;
  make_plan<C>(a, sh, cta, grid, begin, count);
  volatile int* abort_flag = &sh.abort;
  // a wait that runs out is recorded once and stops every role (the others'
  // next waits run out too)
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_wait(bar, parity)) return true;
    if (!*abort_flag) atomicOr(a.status, DSA_DEV_TIMEOUT);
    *abort_flag = 1;
    return false;
  };
  // the same by a whole warp, with one answer for all its lanes
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, wait(bar, parity));
  };
  int slot = 0, round = 0;  // of the operand ring, for every role
  auto advance = [&]() {
    if (++slot == C::NS) {
      slot = 0;
      round ^= 1;
    }
  };

  constexpr uint32_t kIdescQk = idesc_f16(128, kTile, true);
  constexpr uint32_t kIdescPv = idesc_f16(128, D, true) | kIdescBMn;
  const uint64_t kdesc = sw128_desc(smem_u32(tiles)), vdesc = sw128_mn_desc(smem_u32(tiles), kTile * 128);
  const uint64_t qdesc0 = sw128_desc(smem_u32(qsm));
  // The products. One thread issues them (elect_one: the compiler then keeps
  // the operands in uniform registers; issuing a tile's took 1100 cycles
  // without, most of it moving operands).
  auto issue_scores = [&](uint32_t tb, uint64_t q, uint64_t k, int at, int wg, int buf) {
    const uint32_t d = tb + C::S + buf * 64;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const uint64_t b = k + (((i / 4) * (kTile * 128) + (i % 4) * 32) >> 4);
      if constexpr (C::TWO)
        tc_mma_f16(d, q + (((i / 4) * (C::QROWS * 128) + (i % 4) * 32) >> 4), b, kIdescQk, i > 0);
      else
        tc_mma_f16_ta(d, tb + C::Q + 8 * i, b, kIdescQk, i > 0);
    }
    tc_commit(&sh.empty[at]);
    tc_commit(&sh.s_full[wg][buf]);
  };
  auto issue_values = [&](uint32_t tb, uint64_t v, int at, int wg, int buf, bool first) {
#pragma unroll
    for (int i = 0; i < kTile / 16; ++i)
      tc_mma_f16_ta(tb + C::O, tb + C::S + buf * 64 + 8 * i, v + ((i * 2048) >> 4), kIdescPv, !first || i > 0);
    tc_commit(&sh.empty[at]);
    tc_commit(&sh.o_full[wg][buf]);
  };
  auto scores = [&](int wg, int at, int buf) {
    if (elect_one()) issue_scores(sh.tmem + wg * C::STRIDE, qdesc0 + wg * ((C::QROWS * D * 2) >> 4), kdesc + at * (C::SLOT >> 4), at, wg, buf);
    __syncwarp();
  };
  auto values = [&](int wg, int at, int buf, bool first) {
    if (elect_one()) issue_values(sh.tmem + wg * C::STRIDE, vdesc + at * (C::SLOT >> 4), at, wg, buf, first);
    __syncwarp();
  };
  // products in flight end before their TMEM goes back, after an abort too
  auto settle_products = [&](int i) {
    __syncwarp();
    if (elect_one()) {
      tc_commit(&sh.fin[i]);
      mbar_wait(&sh.fin[i], 0);
    }
    __syncwarp();
  };
  auto has_rows = [&](int wg, const Segment& g) { return wg * C::QROWS < g.rows; };

  if (count <= 0) {
    if (tid == 0) a.meta[2 * cta] = make_int4(0, 0, 0, 0);
  } else if (warp < NSW) {
    // ------------------------------------------------------------ softmax
    const int wg = warp / C::SW, gw = warp % C::SW;  // group, and warp of the group
    const uint32_t tb = sh.tmem + wg * C::STRIDE;
    const uint32_t lanes = static_cast<uint32_t>(gw * 32) << 16;
    const uint32_t tO = tb + C::O + lanes;
    const bool issues = !C::TWO && gw == 0;  // this warp issues the products
    Iter<C> it(a, sh.start, count);
    Segment s;
    bool more = it.next(s), run = true;
    int seg = 0, n = 0;   // segments, tiles
    int ns = 0;           // tiles this group has worked on: score buffers and accumulator phases
    // what the join has to know of this CTA, see join_kernel
    int* const meta = reinterpret_cast<int*>(a.meta + 2 * cta);
    if (tid == 0) a.meta[2 * cta] = make_int4(0, 0, 0, 0);
    const int row = tid;  // of the unit
    // a row's query (in its sequence; 0 of a selection, whose rows are one token's) and head of the group
    struct Row {
      int q, g;
    };
    auto row_at = [&](const Segment& g) -> Row {
      if (C::SPARSE) return Row{0, row};
      const int r = g.r0 + row, q = r / a.G;
      return Row{q, r - q * a.G};
    };
    auto query = [&](const Segment& g, Row r) {
      return a.q + static_cast<long long>(g.q0 + r.q) * a.qt + static_cast<long long>(g.h * a.G + r.g) * a.qh;
    };
    // the next unit's queries on their way to L1
    auto warm = [&](const Segment& g) {
      if (row < g.rows) {
        const __nv_bfloat16* q = query(g, row_at(g));
#pragma unroll
        for (int i = 0; i < C::NBLK; ++i) touch(q + 64 * i);
      }
    };
    Row at_row = {0, 0};
    // the unit's queries, then its first tiles' scores
    auto start_unit = [&](const Segment& g) {
      const bool valid = row < g.rows;
      at_row = row_at(g);
      [[maybe_unused]] const uint4* src = reinterpret_cast<const uint4*>(valid ? query(g, at_row) : a.q);
      if constexpr (C::TWO && C::SPAN) {
        // the warp that issues the products brings them
      } else if constexpr (C::TWO) {
        uint8_t* dst = qsm + wg * (C::QROWS * D * 2) + row % C::QROWS * 128;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint4 v = valid ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(dst + (i / 8) * (C::QROWS * 128) + (((i & 7) ^ (row & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
      } else {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 v = valid ? __ldg(src + c * 8 + i) : make_uint4(0, 0, 0, 0);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
          }
          __syncwarp();  // loads only where the row is real
          tmem_st32(tb + C::Q + lanes + 32 * c, w);
        }
        tmem_st_wait();
        tc_fence_before();
      }
      if constexpr (C::TWO) {
        __syncwarp();
        if (!C::SPAN && lane == 0) mbar_arrive(&sh.q_ready[wg]);
      } else {
        if (gw == 0) run = run && wait_warp(&sh.full[slot], round);
        run = named_bar_all(1, 128, run);  // the group's warps go on, or stop, together
        if (gw == 0 && run) {
          tc_fence_after();
          scores(0, slot, 0);
          __syncwarp();
        }
        advance();
      }
    };
    // the second product of the last tile has completed
    auto tile_at = [&](int t) { return C::BACKWARDS ? s.t0 + s.t1 - 1 - t : t; };
    auto wait_product = [&]() { return wait_warp(&sh.o_full[wg][(ns - 1) & (C::SBUF - 1)], ((ns - 1) / C::SBUF) & 1); };
    if (more && has_rows(wg, s)) start_unit(s);
    while (more && run) {
      if (!has_rows(wg, s)) {  // a unit of at most 128 rows: nothing for the second group
        n += s.t1 - s.t0;
        ++seg;
        more = it.next(s);
        if (more && has_rows(wg, s)) start_unit(s);
        continue;
      }
      if constexpr (!C::TWO || !C::SPAN) {
        Iter<C> peek = it;
        Segment nx;
        if (peek.next(nx) && has_rows(wg, nx)) warm(nx);
      }
      const bool active = row - lane < s.rows;  // some row of this warp is real
      const bool valid = row < s.rows;
      const Row mine = at_row;
      const int qi = mine.q;                   // the row's query in its sequence
      float m = -INFINITY, l = 0.f;
      [[maybe_unused]] float lr = 0.f;  // the sum of the rounded weights, see Cfg::ROUND
      // the place that a row measures distance from, and its head's slope
      [[maybe_unused]] int near = 0;
      [[maybe_unused]] float slope2 = 0.f;
      if constexpr (C::SPAN) {
        if constexpr (SCORES == kCapped) m = a.fixed;
        if (SCORES >= kBiased && a.slopes && valid) {
          near = nearest(token_at(a, s.q0 + qi));
          slope2 = a.slopes[s.h * a.G + mine.g] * 1.4426950408889634f;
        }
      }
      for (int t = s.t0; t < s.t1; ++t, ++n, ++ns) {
        const int buf = ns & (C::SBUF - 1);
        auto wait_scores = [&]() { run = run && wait_warp(&sh.s_full[wg][buf], (ns / C::SBUF) & 1); };
        // A unit's first tile after skipped ones: once its scores are there the
        // loaders have announced it, so the wait for its mask cannot end a round
        // early (see kRing). The mask's way to a register is hidden behind the
        // scores otherwise (a chunk of 2048 tokens takes 505 us so and 516 with
        // the scores first on every tile).
        if (C::WG > 1 && t == s.t0) wait_scores();
        run = run && wait_warp(&sh.mfull[n % kRing], (n / kRing) & 1);
        unsigned long long see = sh.vmask[n % kRing];
        wait_scores();
        tc_fence_after();
        const uint32_t tS = tb + C::S + 64 * buf + lanes;
        if (active && run) {
          const int p0 = tile_at(t) * kTile;
          if (!C::SPAN && !C::SPARSE && valid && p0 + kTile > s.full) see &= row_mask(a, s, qi, p0);
          uint32_t p[32];
          if constexpr (!C::SPAN) {
            const bool some = !__all_sync(0xffffffffu, see == ~0ull);  // a key that some row does not see
            const unsigned long long sc = pack2(a.scale2, a.scale2);
            // The weights are taken under the running maximum while the tile's
            // own is found. Only if that is more than 2^8 above it (a unit's
            // first tile, rarely later) does the maximum move, are the sums
            // rescaled and the tile's weights taken again; the weights stay
            // below 2^8 otherwise.
            while (true) {
              uint32_t x[2][32];
              tmem_ld32(tS, x[0]);
              tmem_ld32(tS + 32, x[1]);
              const float sub = m == -INFINITY ? 0.f : m;
              unsigned long long sum[2] = {0ull, 0ull};  // pairs of fp32 zeros
              float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
              tmem_ld_wait32(x[0]);
              tmem_ld_wait32(x[1]);
              const unsigned long long sb = pack2(-sub, -sub);
              if (some) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  const uint32_t bits = static_cast<uint32_t>(see >> (32 * c));
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    if (!((bits >> i) & 1)) x[c][i] = 0xFF800000u;
                }
              }
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float s0 = __uint_as_float(x[c][2 * i]), s1 = __uint_as_float(x[c][2 * i + 1]);
                  mx[i & 3] = fmaxf(mx[i & 3], fmaxf(s0, s1));
                  float e0, e1;
                  unpack2(fma2(pack2(s0, s1), sc, sb), e0, e1);
                  e0 = ex2(e0);
                  e1 = ex2(e1);
                  sum[i & 1] = add2(sum[i & 1], pack2(e0, e1));
                  const __nv_bfloat162 w = __floats2bfloat162_rn(e0, e1);
                  memcpy(&p[16 * c + i], &w, 4);
                }
              const float mnew = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale2;
              const bool grow = mnew > m + 8.f || (m == -INFINITY && mnew > m);
              if (!__any_sync(0xffffffffu, grow)) {
                float l0, l1;
                unpack2(add2(sum[0], sum[1]), l0, l1);
                l += l0 + l1;
                break;
              }
              // weights of up to 2^8 stand before this factor: flushed to zero below
              // 2^-126 it would lose weights of 2^-118, which fp32 holds
              const float alpha = grow ? ex2_denorm(m - mnew) : 1.f;
              if (t > s.t0) {  // after the last tile's second product
                run = run && wait_product();
                tc_fence_after();
                l *= alpha;
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) tmem_scale16(tO + 16 * c, alpha);
                tmem_st_wait();
              }
              if (grow) m = mnew;
            }
          } else {
            if (valid && (p0 + kTile > s.full || p0 < s.lo)) see &= span_mask(a, s.q0 + qi, token_at(a, s.q0 + qi), p0);
            [[maybe_unused]] const float from = static_cast<float>(near - p0);
            const bool some = !__all_sync(0xffffffffu, see == ~0ull);  // a key that some row does not see
            constexpr bool CAP = SCORES == kCapped, WIDE_CAP = SCORES == kWideCap, BIAS = SCORES == kBiased || WIDE_CAP;
            [[maybe_unused]] bool capped = !CAP && !(BIAS && (WIDE_CAP || a.cap2 != 0.f));  // in TMEM, or not to be
            if constexpr (CAP) {
              if (some) {  // masks come after the cap, and few tiles have one
                cap_any(a, tS);
                capped = true;
              }
            }
            while (true) {
              uint32_t x[2][32];
              tmem_ld32(tS, x[0]);
              tmem_ld32(tS + 32, x[1]);
              tmem_ld_wait32(x[0]);
              tmem_ld_wait32(x[1]);
              Weighed w;
              if (CAP && !capped) {
                w = weigh<true>(a, x, p, 1.f, m);
                if (__all_sync(0xffffffffu, w.most <= a.poly_most)) {
                  l += w.sum;
                  lr += w.rounded;
                  break;
                }
                cap_any(a, tS);
                capped = true;
                continue;
              }
              float shift = 0.f;  // of all of the tile's exponents
              if constexpr (BIAS) {
                if (!capped && !__all_sync(0xffffffffu, cap_near<WIDE_CAP>(a, x))) {
                  if constexpr (WIDE_CAP)
                    cap_each(a, tS);
                  else
                    cap_any(a, tS);
                  capped = true;
                  continue;
                }
                if (!WIDE_CAP && a.cap2 == 0.f) {
#pragma unroll
                  for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[c][i] = __float_as_uint(__uint_as_float(x[c][i]) * a.scale2);
                }
                shift = bias_scores(x, slope2, from, !__all_sync(0xffffffffu, from >= 63.f || !valid));
              }
              if (some) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  const uint32_t bits = static_cast<uint32_t>(see >> (32 * c));
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    if (!((bits >> i) & 1)) x[c][i] = 0xFF800000u;
                }
              }
              w = weigh<false, C::ROUND>(a, x, p, CAP || BIAS ? 1.f : a.scale2, (m == -INFINITY ? 0.f : m) - shift);
              w.most += shift;
              const bool grow = !CAP && (w.most > m + kSpanStep || (m == -INFINITY && w.most > m));
              if (!__any_sync(0xffffffffu, grow)) {
                l += w.sum;
                lr += w.rounded;
                break;
              }
              const float mnew = w.most;
              const float alpha = grow ? ex2_denorm(m - mnew) : 1.f;
              if (t > s.t0) {  // after the last tile's second product
                run = run && wait_product();
                tc_fence_after();
                l *= alpha;
                lr *= alpha;
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) tmem_scale16(tO + 16 * c, alpha);
                tmem_st_wait();
              }
              if (grow) m = mnew;
            }
          }
          tmem_st32(tS, p);  // over scores that are not needed any more
        }
        if constexpr (C::TWO) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (!run) break;
          if (lane == 0) mbar_arrive(&sh.p_ready[wg][buf]);
        } else {
          const bool more_scores = t + 1 < s.t1;
          const int vslot = slot, vround = round;
          advance();
          const bool there = issues && mbar_test(smem_u32(&sh.full[vslot]), vround);
          tmem_st_wait();
          tc_fence_before();
          run = named_bar_all(1, 128, run);  // the four warps go on, or stop, together
          if (!run) break;
          if (issues) {
            tc_fence_after();
            if (elect_one()) {
              run = there || wait(&sh.full[vslot], vround);
              if (run) issue_values(tb, vdesc + vslot * (C::SLOT >> 4), vslot, 0, 0, t == s.t0);
              if (run && more_scores) {
                run = wait(&sh.full[slot], round);
                if (run) issue_scores(tb, 0, kdesc + slot * (C::SLOT >> 4), slot, 0, 0);
              }
            }
            run = __all_sync(0xffffffffu, run);  // seen by the other warps at the next barrier
          }
          if (more_scores) advance();
        }
      }
      // the next unit's queries go up before this one's sums come down: every
      // product with the old ones has completed (s_full of the last tile)
      const Segment done = s;
      more = it.next(s);
      if (more && has_rows(wg, s)) start_unit(s);
      run = run && wait_product();
      bool fix = false;  // a loader replaced a value of this segment
      if (!C::SPARSE) {
        run = run && wait_warp(&sh.vdone[seg % kRing], (seg / kRing) & 1);
        fix = *static_cast<volatile int*>(&sh.bad[seg % kRing]) == seg + 1;
        if constexpr (C::WG > 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.u_done[wg]);
        }
      }
      tc_fence_after();
      int unit = 0;  // the unit's first tile
      if constexpr (C::SPAN) unit = done.tb;
      const bool first = done.t0 == unit, last = done.t1 == done.nt;
      if constexpr (C::SPAN) {
        if (tid == 0 && a.raw_mode) {
          int2* const ends = a.ends + static_cast<long long>(done.place) * a.kv_heads + done.h;
          if (first) ends->x = cta;
          if (last) ends->y = cta;
        }
      }
      if (tid == 0 && !first) {
        meta[1] = 1;
        meta[2] = last;
      } else if (tid == 0 && !last) {
        meta[0] = 1;
        meta[3] = done.rows;
        a.meta[2 * cta + 1] = make_int4(done.r0, done.q0, done.h, 0);
      }
      if (active && run) {
        if (fix) {
          if constexpr (C::SPAN)
            fix_nonfinite<FMT, D>(a, done, done.t0, done.t1, qi, valid, tO, token_at(a, min(done.q0 + qi, a.Tq - 1)));
          else
            fix_nonfinite<FMT, D>(a, done, max(done.t0, done.full / kTile), done.t1, qi, valid, tO);
        }
        const long long tok = done.q0 + mine.q;
        const int head = done.h * a.G + mine.g;
        const int piece = 2 * cta + (first ? 1 : 0);
        __nv_bfloat16* dst = a.out + tok * a.ot + head * a.oh;
        float* part = a.part + (static_cast<long long>(piece) * C::ROWS + row) * D;
        bool whole = first && last;
        if constexpr (C::SPAN) {
          if (whole && (a.raw_mode == 1 || (a.raw_mode == 2 && done.base))) {
            whole = false;
            part = a.raw + (tok * a.kv_heads * a.G + head) * D;
          }
        }
        float inv = l > 0.f ? 1.f / l : 0.f;
        // lse is of the exact weights; sums for a join are brought to them by the
        // two sums' ratio
        [[maybe_unused]] float ratio = 1.f;
        if constexpr (C::ROUND) {
          inv = lr > 0.f ? 1.f / lr : 0.f;
          if (lr > 0.f) ratio = l * inv;
        }
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          __syncwarp();
          tmem_ld32(tO + 32 * c, o);
          tmem_ld_wait32(o);
          if constexpr (C::SPAN) {
            // Four lanes exchange their rows' 16-byte runs, so that a store's lanes
            // have 64 bytes of a row each four; by rows it takes the L1 32 steps.
            uint32_t w[4][4];
            if (whole) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float u = __uint_as_float(o[8 * i + 2 * e]) * inv, v = __uint_as_float(o[8 * i + 2 * e + 1]) * inv;
                  const __nv_bfloat162 p = l == 0.f ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(u, v);
                  memcpy(&w[i][e], &p, 4);
                }
              store_runs(w, valid ? dst + 32 * c : nullptr);
            } else {
#pragma unroll
              for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i / 4][i % 4] = C::ROUND ? __float_as_uint(__uint_as_float(o[16 * half + i]) * ratio) : o[16 * half + i];
                store_runs(w, valid ? part + 32 * c + 16 * half : nullptr);
              }
            }
            continue;
          }
          if (!valid) {
          } else if (whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float u = __uint_as_float(o[8 * i + 2 * e]) * inv, v = __uint_as_float(o[8 * i + 2 * e + 1]) * inv;
                const __nv_bfloat162 p = l == 0.f ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(u, v);
                memcpy(&w[e], &p, 4);
              }
              *reinterpret_cast<uint4*>(dst + 32 * c + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(part + 32 * c + 4 * i) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        if (valid) {
          if (whole) {
            float top = m;
            if constexpr (C::SPAN) {
              if (a.slopes) top -= a.slopes[head] * 1.4426950408889634f * away(token_at(a, tok));
            }
            if (a.lse) a.lse[tok * a.kv_heads * a.G + head] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
          } else if (C::SPAN && first && last) {
            if constexpr (C::SPAN) a.raw_ml[tok * a.kv_heads * a.G + head] = make_float2(m, l);
          } else {
            a.ml[static_cast<long long>(piece) * C::ROWS + row] = make_float2(m, l);
          }
        }
        tc_fence_before();
      }
      ++seg;
    }
    if (issues) settle_products(gw);
  } else if (C::TWO && warp >= NSW + 4) {
    // ------------------------------------------------------------ products
    const int wg = warp - NSW - 4;
    Iter<C> it(a, sh.start, count);
    Segment s;
    bool run = true;
    int ns = 0, units = 0, passed = 0;  // tiles, units, and units known to be read out
    // Span form: this warp brings the queries too, the next unit's as soon as the
    // last scores of this one are there, while softmax has one or two tiles to
    // go. By the softmax warps, between two units, it took 5300 cycles of each.
    [[maybe_unused]] bool asked = false;
    [[maybe_unused]] auto ask_queries = [&](const Segment& g) {
      // a row's 16-byte runs by neighbouring lanes, two or four rows a step
      constexpr int RUNS = D / 8, AT_ONCE = 32 / RUNS;
      uint8_t* const to = qsm + wg * (C::QROWS * D * 2);
      const int at = lane % RUNS;
#pragma unroll 1
      for (int k = 0; k < C::QROWS / 32; ++k) {
        const int row = wg * C::QROWS + 32 * k + lane, r = g.r0 + row, q = r / a.G;
        const __nv_bfloat16* src = a.q + static_cast<long long>(g.q0 + q) * a.qt + static_cast<long long>(g.h * a.G + r - q * a.G) * a.qh;
        const unsigned long long from = row < g.rows ? reinterpret_cast<unsigned long long>(src) : 0ull;
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
          const int x = i * AT_ONCE + lane / RUNS;
          const unsigned long long p = __shfl_sync(0xffffffffu, from, x);
          cp_async16(smem_u32(to + (at / 8) * (C::QROWS * 128) + (32 * k + x) * 128 + (((at & 7) ^ (x & 7)) << 4)),
                     p ? reinterpret_cast<const uint4*>(p) + at : reinterpret_cast<const uint4*>(a.q), p != 0);
        }
      }
      cp_async_commit();
    };
    [[maybe_unused]] Segment nx;
    bool more = it.next(s);
    while (run && more) {
      [[maybe_unused]] bool more_next = false;
      auto on = [&]() {  // to the next segment
        if constexpr (C::SPAN) {
          s = nx;
          more = more_next;
        } else {
          more = it.next(s);
        }
      };
      if (!has_rows(wg, s)) {
        // Nothing for this group: it only passes the tiles on, once its softmax
        // has read the last unit's segment entry (see kRing). Of the units before
        // that one it has: their successor's weights came after.
        if constexpr (C::SPAN) more_next = it.next(nx);
        if (units > passed) run = wait_warp(&sh.u_done[wg], (units - 1) & 1);
        passed = units;
        for (int i = 2 * (s.t1 - s.t0); run && i > 0; --i) {
          run = wait_warp(&sh.full[slot], round);
          if (run && lane == 0) mbar_arrive(&sh.empty[slot]);
          advance();
        }
        on();
        continue;
      }
      auto next_scores = [&](int buf) {
        run = run && wait_warp(&sh.full[slot], round);
        if (!run) return;
        tc_fence_after();
        scores(wg, slot, buf);
        __syncwarp();
        advance();
      };
      if constexpr (C::SPAN) {
        if (!asked) ask_queries(s);
        asked = false;
        cp_async_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
      } else {
        run = wait_warp(&sh.q_ready[wg], units & 1);
      }
      ++units;
      for (int i = 0; i < 2 && s.t0 + i < s.t1; ++i) next_scores((ns + i) & 1);
      if constexpr (C::SPAN) more_next = it.next(nx);
      for (int t = s.t0; run && t < s.t1; ++t, ++ns) {
        const int buf = ns & 1;
        run = wait_warp(&sh.full[slot], round) && wait_warp(&sh.p_ready[wg][buf], (ns >> 1) & 1);
        if (!run) break;
        tc_fence_after();
        values(wg, slot, buf, t == s.t0);
        __syncwarp();
        advance();
        if (t + 2 < s.t1) next_scores(buf);
        if constexpr (C::SPAN) {
          if (run && !asked && t + 3 >= s.t1 && more_next && has_rows(wg, nx)) {
            const int e = ns + s.t1 - 1 - t;  // the last tile, whose scores have been asked for
            run = wait_warp(&sh.s_full[wg][e & 1], (e >> 1) & 1);
            if (run) ask_queries(nx);
            asked = run;
          }
        }
      }
      on();
    }
    if constexpr (C::SPAN) cp_async_wait<0>();
    settle_products(wg);
  } else if (warp < NSW + 4) {
    // ------------------------------------------------------------ loaders
    // A pair of warps brings the keys, another the values. A thread moves NCH
    // 16-byte chunks of a tile.
    constexpr int CPB = C::CPB, NCH = C::NCH;
    constexpr int RL = 8 / CPB;              // rows that 8 lanes cover: their stores hit all 32 banks
    constexpr int RSTEP = RL * 8 / C::NBLK;  // this thread's rows are so far apart
    const int lw = warp - NSW;
    const bool v = lw >= 2;
    const int ti = (lw & 1) * 32 + lane;
    const int chunk = ti % CPB, blk = (ti / 8) % C::NBLK;
    const int row0 = (ti / (8 * C::NBLK)) * RL + (ti / CPB) % RL;
    const int code_off = (blk * CPB + chunk) * 16;
    const int scale_off = (blk * 64 + chunk * (64 / CPB)) / kvf::kBlock;
    // A warp's chunks are those of 32 rows. A lane brings the scales of one of
    // them, so that a thread's NCH rows are neighbours in shared memory.
    const int scale_row = (lw & 1) * (32 / NCH) + lane / NCH + lane % NCH * RSTEP;
    const int scale_word = (lw & 1) * 32 + row0 % (32 / NCH) * NCH;  // of this thread's first row
    uint8_t* const ring = raw + v * (C::P * C::RAW_SLOT);
    const uint32_t page_step = static_cast<uint32_t>(a.kv_heads) * L::HEAD_BYTES;
    const int32_t code_at = v ? L::V_CODES : L::K_CODES, scale_at = v ? L::V_SCALES : L::K_SCALES;
    // where unit u (16 bytes) of row i of this thread lies in an operand tile
    auto place = [&](uint8_t* tile, int i, int u) -> uint8_t* {
      const int r = row0 + i * RSTEP;
      return tile + blk * (kTile * 128) + r * 128 + ((u ^ (r & 7)) << 4);
    };

    Iter<C> it(a, sh.start, count);
    Segment s;
    int n = 0, parts = 0;             // tiles; operand tiles of both kinds before this segment
    int issued = 0, sent = 0;         // tiles asked for by copies, and handed over
    int mine = -1, mine_round = 0;    // the last operand tile asked for, and its round
    bool run = true;

    // A tile has landed: hand it to the products. info: bits 0-3 the slot, 4
    // replace what is not finite, 5 a segment's last, 6 the slot's round, 8..
    // the segment
    auto hand_over = [&](int info) {
      const int at = info & 15, seg = info >> 8;
      uint8_t* const tile = tiles + at * C::SLOT;
      bool found = false;
      if constexpr (C::RAW) {
        const uint8_t* src = ring + (sent % C::P) * C::RAW_SLOT;
        const uint32_t* const scales = reinterpret_cast<const uint32_t*>(src + NCH * 64 * 16);
        __syncwarp();  // the other lanes' copies: the scales
        [[maybe_unused]] uint32_t odd = 0;
        if constexpr (D == 64) odd = scales[64 + ti];
        constexpr int BATCH = NCH < 4 ? NCH : FMT == DSA_FMT_FP8 ? 4 : 2;  // chunks at a time: enough to overlap their latencies
        // not unrolled: fewer instructions to fetch (2048 selections of 512 keys in
        // fp8 941 -> 864 us, trees the same)
#pragma unroll 1
        for (int i0 = 0; i0 < NCH; i0 += BATCH) {
          uint32_t w[BATCH][32 / CPB];
          using F = kvf::Factor<C::RAW ? FMT : DSA_FMT_FP8>;
          uint32_t byte[BATCH], sw[BATCH];
          bool two = false;
          static_assert(BATCH == 4 || BATCH == 2, "scale words of a batch are one load");
          if constexpr (BATCH == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(scales + scale_word + i0);
            sw[0] = x.x;
            sw[1] = x.y;
            sw[2] = x.z;
            sw[3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(scales + scale_word + i0);
            sw[0] = x.x;
            sw[1] = x.y;
          }
#pragma unroll
          for (int b = 0; b < BATCH; ++b) {
            const int i = i0 + b;
            const uint4 c4 = reinterpret_cast<const uint4*>(src)[i * 64 + ti];
            const uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w};
            byte[b] = (sw[b] >> (8 * (scale_off + (D == 64 ? 2 * ((odd >> i) & 1) : 0)))) & 0xFFu;
            F f;
            f.set(byte[b]);
            kvf::widen(c, f, w[b]);
            two |= F::two(byte[b]);
          }
          if (two) {
#pragma unroll
            for (int b = 0; b < BATCH; ++b) F::rest(byte[b], w[b]);
          }
          if (info & 16) {
#pragma unroll
            for (int b = 0; b < BATCH; ++b) found |= kvf::zero_nonfinite(w[b]);
          }
#pragma unroll
          for (int b = 0; b < BATCH; ++b)
#pragma unroll
            for (int j = 0; j < 8 / CPB; ++j)
              *reinterpret_cast<uint4*>(place(tile, i0 + b, chunk * (8 / CPB) + j)) =
                  make_uint4(w[b][4 * j], w[b][4 * j + 1], w[b][4 * j + 2], w[b][4 * j + 3]);
        }
      } else if (info & 16) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          uint4* p = reinterpret_cast<uint4*>(place(tile, i, chunk));
          const uint4 c = *p;
          uint32_t w[4] = {c.x, c.y, c.z, c.w};
          if (kvf::zero_nonfinite(w)) {
            found = true;
            *p = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (found) *static_cast<volatile int*>(&sh.bad[seg % kRing]) = seg + 1;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.full[at]);
        if (info & 32) mbar_arrive(&sh.vdone[seg % kRing]);
      }
      ++sent;
    };
    auto hand_over_all = [&]() {
      cp_async_wait<0>();
      while (sent < issued) hand_over(sh.info[lw][sent & 3]);
    };
    // hand over the oldest tile of codes; `left` younger ones may stay in flight
    auto settle = [&](auto left) -> bool {
      cp_async_wait<decltype(left)::value>();
      const int info = sh.info[lw][sent & 3];
      // codes are widened into a slot that has to be free; copies into the
      // slot itself waited for that before they were issued
      if (C::RAW && !wait_warp(&sh.empty[info & 15], ((info >> 6) & 1) ^ 1)) return false;
      hand_over(info);
      return true;
    };
    // An operand tile that copies or TMA will fill; what has landed goes out
    // before this warp waits for one. The wait looks at one bit of the slot's
    // round, so it must not come two rounds early: a pair fills every one of
    // its tiles, in order and at most three places apart, and to fill the last
    // one it waited until the tile NS places before that was released, with
    // all tiles before it; so the tile two rounds back in this slot has been.
    auto acquire = [&](int at, int rnd) -> bool {
      if (__all_sync(0xffffffffu, mbar_test(smem_u32(&sh.empty[at]), rnd ^ 1))) return true;
      hand_over_all();
      return wait_warp(&sh.empty[at], rnd ^ 1);
    };
    // ask for a tile: src(r, half, ok, off) gives where the head's part of row
    // r's page begins, whether the row is there, and its place in the page (half
    // of the tile r lies in; 2: not known in the code). whole: that beginning
    // for all rows of a page of 64 keys, else null.
    auto ask = [&](auto src, const uint8_t* whole, int at, int rnd, bool clean, bool last, int seg) -> bool {
      if (!C::RAW && !acquire(at, rnd)) return false;
      uint8_t* const to = ring + (issued % C::P) * C::RAW_SLOT;
      auto dst = [&](int i) { return C::RAW ? smem_u32(to) + ti * 16 + i * 1024 : smem_u32(place(tiles + at * C::SLOT, i, chunk)); };
      [[maybe_unused]] const uint32_t scale_dst = smem_u32(to) + NCH * 64 * 16 + (ti << 2);
      [[maybe_unused]] uint32_t odd = 0;
      if (whole) {
        const uint8_t* const code = whole + (code_at + row0 * L::CB + code_off);
#pragma unroll
        for (int i = 0; i < NCH; ++i) cp_async16(dst(i), code + i * RSTEP * L::CB, true);
        if constexpr (C::RAW) {
          cp_async4(scale_dst, whole + (scale_at + ((scale_row * L::SB) & ~3)), true);
          if (D == 64) odd = row0 & 1 ? ~0u : 0u;
        }
      } else {
        bool ok;
        int off;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          const uint8_t* head = src(row0 + i * RSTEP, i * RSTEP >= 32, ok, off);  // row0 < RSTEP
          cp_async16(dst(i), head + code_at + off * L::CB + code_off, ok);
          if (C::RAW && D == 64) odd |= (off & 1) << i;
        }
        if constexpr (C::RAW) {
          const uint8_t* head = src(scale_row, 2, ok, off);
          cp_async4(scale_dst, head + scale_at + ((off * L::SB) & ~3), ok);
        }
      }
      if constexpr (C::RAW && D == 64) reinterpret_cast<uint32_t*>(to + NCH * 64 * 16)[64 + ti] = odd;
      cp_async_commit();
      if (lane == 0) sh.info[lw][issued & 3] = at | (clean ? 16 : 0) | (last ? 32 : 0) | (rnd << 6) | (seg << 8);
      __syncwarp();
      ++issued;
      if (issued - sent == C::P) return settle(std::integral_constant<int, C::P - 1>());
      return true;
    };

    for (int seg = 0; run && it.next(s); ++seg) {
      const int32_t* table = a.page_table + static_cast<long long>(s.b) * a.max_pages;
      const uint8_t* const heads = a.cache + static_cast<long long>(s.h) * L::HEAD_BYTES;
      const int npg = (s.len + kTile - 1) / kTile, nt = s.t1 - s.t0;
      // A selection's keys go through three steps, a tile apart, so that no
      // load is waited for: the entry, its page, its row in the cache. This
      // lane has keys `lane` and `lane + 32` of a tile.
      int e0 = -1, e1 = -1, g0 = -1, g1 = -1, u0 = -1, u1 = -1;  // entries; those whose pages are on their way; pages
      const int ksel = (a.k + kTile - 1) / kTile;                // tiles of the selection; drafted tokens follow
      const int32_t* const sel = C::SPARSE ? a.sel + static_cast<long long>(s.q0) * a.k : nullptr;
      auto entry = [&](int t, int j) -> int {  // a position (or cache slot) or negative
        int x = t * kTile + j;
        if (t >= s.t1) return -1;
        if (t < ksel) return x < a.k ? sel[x] : -1;
        x -= ksel * kTile;
        if (x >= s.nd || (x >> 5) >= a.mask_words) return -1;
        return (a.mask[static_cast<long long>(s.q0) * a.mask_words + (x >> 5)] >> (x & 31)) & 1 ? s.len - s.nd + x : -1;
      };
      // the page of tile t's entry e, as the table (or the slot) has it; e becomes negative where there is none
      auto page_of = [&](int& e, int t) -> int {
        const bool slot = a.slots && t < ksel;  // drafted tokens are positions
        const int limit = s.len == 0 ? 0 : slot ? a.num_pages * kTile : s.len;
        if (e >= limit) {
          if (limit > 0) atomicOr(a.status, DSA_DEV_BOUNDS);
          e = -1;
        }
        return e < 0 ? -1 : slot ? e >> 6 : table[e >> 6];
      };
      // the row: in bf16 its number in the cache as rows of D elements, -1
      // where there is no key; else where the page's part of this head begins,
      // which leaves room for the row's place in it, 0 where there is none
      constexpr bool GATHER = C::SPARSE && FMT == DSA_FMT_BF16;
      using RowId = std::conditional_t<GATHER, int, unsigned long long>;
      constexpr RowId NONE = GATHER ? static_cast<RowId>(-1) : static_cast<RowId>(0);
      auto row_of = [&](int e, int page) -> RowId {
        if (e < 0) return NONE;
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.num_pages)) {
          atomicOr(a.status, DSA_DEV_BOUNDS);
          return NONE;
        }
        if constexpr (GATHER)
          return ((page * a.kv_heads + s.h) * 2 + v) * kTile + (e & 63);
        else
          return reinterpret_cast<unsigned long long>(heads + static_cast<uint64_t>(page) * page_step) | (e & 63);
      };
      int pg = -1;  // page ids of 32 tiles
      if (C::SPARSE) {
        g0 = entry(s.t0, lane);
        g1 = entry(s.t0, lane + 32);
        e0 = entry(s.t0 + 1, lane);
        e1 = entry(s.t0 + 1, lane + 32);
        u0 = page_of(g0, s.t0);
        u1 = page_of(g1, s.t0);
      }
      for (int x = 0; run && x < nt; ++x, ++n) {
        const int t = C::BACKWARDS ? s.t1 - 1 - x : s.t0 + x;
        // the tile's place in the order the products take keys and values:
        // K0 V0 K1 V1 .., or K0 K1 V0 K2 V1 .. with two score buffers
        const int order = parts + (C::SBUF == 1 ? 2 * x + v : !v ? (x ? 2 * x - 1 : 0) : x + 1 < nt ? 2 * x + 2 : 2 * nt - 1);
        const int at = order % C::NS, rnd = (order / C::NS) & 1;
        const bool last = v && x + 1 == nt;
        unsigned long long vm;
        int page = -1;
        RowId k0 = NONE, k1 = NONE;
        if constexpr (C::SPARSE) {
          k0 = row_of(g0, u0);
          k1 = row_of(g1, u1);
          g0 = e0;
          g1 = e1;
          u0 = page_of(g0, t + 1);
          u1 = page_of(g1, t + 1);
          e0 = entry(t + 2, lane);
          e1 = entry(t + 2, lane + 32);
          vm = __ballot_sync(0xffffffffu, k0 != NONE) | (static_cast<unsigned long long>(__ballot_sync(0xffffffffu, k1 != NONE)) << 32);
        } else {
          if ((x & 31) == 0) {
            const int mine_at = C::BACKWARDS ? t - lane : t + lane;
            pg = mine_at < min(s.t1, npg) && (!C::BACKWARDS || mine_at >= s.t0) ? table[mine_at] : -1;
          }
          page = __shfl_sync(0xffffffffu, pg, x & 31);
          const bool ok = page >= 0 && page < a.num_pages;
          if (!ok && t < npg && lw == 0 && lane == 0) atomicOr(a.status, DSA_DEV_BOUNDS);
          vm = ok ? low_bits(s.len - t * kTile) : 0ull;
        }
        if (lw == 0 && lane == 0) {
          sh.vmask[n % kRing] = vm;
          mbar_arrive(&sh.mfull[n % kRing]);
        }
        mine = at;
        mine_round = rnd;
        if constexpr (GATHER) {
          // by TMA, four rows of 64 dimensions an instruction. A key that is not
          // there is a row outside the cache. A warp's lanes issue theirs one
          // after another (75 cycles each), so both warps of the pair do: half
          // of the dimensions each, or half of the rows.
          constexpr int LANES = 8 * C::NBLK;  // a warp's instructions
          const int q = C::NBLK == 2 ? lane & 15 : (lw & 1) * 8 + (lane & 7);  // four rows
          const int c = C::NBLK == 2 ? lw & 1 : 0;                             // 64 dimensions
          int y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = 4 * q + j;
            const int p0 = __shfl_sync(0xffffffffu, k0, r & 31), p1 = __shfl_sync(0xffffffffu, k1, r & 31);
            y[j] = r < 32 ? p0 : p1;
          }
          run = acquire(at, rnd);
          if (run && lane == 0) mbar_arrive_expect_tx(&sh.full[at], C::SLOT / 2);
          __syncwarp();
          if (run && lane < LANES)
            tma_gather4(tiles + at * C::SLOT + c * (kTile * 128) + q * 512, &tm, c * 64, y[0], y[1], y[2], y[3], &sh.full[at]);
          if (run && last && lane == 0) mbar_arrive(&sh.vdone[seg % kRing]);
          __syncwarp();
        } else if constexpr (C::SPARSE) {
          run = ask(
              [&](int r, int half, bool& ok, int& off) {
                RowId k = __shfl_sync(0xffffffffu, half == 1 ? k1 : k0, r & 31);
                if (half == 2) {
                  const RowId kk = __shfl_sync(0xffffffffu, k1, r & 31);
                  if (r >= 32) k = kk;
                }
                ok = k != 0;
                off = static_cast<int>(k & 63);
                return ok ? reinterpret_cast<const uint8_t*>(k - off) : a.cache;
              },
              nullptr, at, rnd, false, last, seg);
        } else {
          bool all = (t + 1) * kTile <= s.full;
          if constexpr (C::SPAN) all = all && t * kTile >= s.lo;
          const bool whole = vm == ~0ull && all;  // every row sees every key
          const uint8_t* const head = heads + static_cast<uint64_t>(vm ? static_cast<uint32_t>(page) : 0u) * page_step;
          if (FMT == DSA_FMT_BF16 && whole) {
            // by TMA: 64 keys of 64 dimensions a box
            run = acquire(at, rnd);
            if (run && lane == 0) {
              if (lw & 1) {
                mbar_arrive(&sh.full[at]);
              } else {
                mbar_arrive_expect_tx(&sh.full[at], C::SLOT);
                const int y = ((page * a.kv_heads + s.h) * 2 + v) * kTile;
#pragma unroll
                for (int c = 0; c < C::NBLK; ++c)
                  tma_load_2d(tiles + at * C::SLOT + c * (kTile * 128), &tm, c * 64, y, &sh.full[at]);
              }
              if (last) mbar_arrive(&sh.vdone[seg % kRing]);
            }
            __syncwarp();
            if (run && sent < issued) hand_over_all();  // copies asked for before go out too
          } else {
            run = ask(
                [&](int r, int, bool& ok, int& off) {
                  off = r;
                  ok = (vm >> r) & 1;
                  return head;
                },
                vm == ~0ull ? head : nullptr, at, rnd, v && !all, last, seg);
          }
        }
      }
      parts += 2 * nt;
    }
    if constexpr (C::RAW) {
      while (run && sent < issued) run = settle(std::integral_constant<int, 0>());
    } else if (run) {
      hand_over_all();
    }
    cp_async_wait<0>();
    // after a wait that ran out, TMA copies in flight land before the CTA exits
    // (the last into each slot; `mine` is the last this warp asked for)
    if (*abort_flag && FMT == DSA_FMT_BF16 && (lw & 1) == 0 && lane == 0 && mine >= 0)
      for (int i = 0; i < C::NS; ++i) {
        const int rnd = i <= mine ? mine_round : mine_round ^ 1;
        mbar_wait(&sh.full[i], rnd, 20000000LL);
      }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(sh.tmem, C::TMEM);
  }
}

template <int FMT, int D, int FORM, int SCORES, class Args>
dsa_status run_one(dsa_ctx* ctx, const CUtensorMap& tm, const Args& a, int grid, cudaStream_t stream) {
  using C = Cfg<FMT, D, FORM, SCORES>;
  auto kern = attn_kernel<FMT, D, FORM, SCORES>;
  constexpr int bytes = smem_bytes<C>();
  static_assert(bytes * C::CTAS <= 233472 - 1024 * C::CTAS, "shared memory of an SM");
  constexpr int at = ((SCORES * 3 + FMT) * 2 + (D == 128)) * kForms + FORM;  // once a context and kernel
  static_assert(at < 64 * static_cast<int>(sizeof(ctx->attn_ready) / sizeof(uint64_t)), "a bit for each kernel");
  if (!(ctx->attn_ready[at / 64] >> (at % 64) & 1)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return DSA_ERR_CUDA;
    ctx->attn_ready[at / 64] |= 1ull << (at % 64);
  }
  LaunchScope scope(ctx, DSA_K_ATTN, stream);
  return launch_pdl(kern, dim3(grid), dim3(C::THREADS), bytes, stream, tm, a) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

template <int FMT, int D, int SCORES, class Args>
dsa_status run_dim(dsa_ctx* ctx, int form, const CUtensorMap& tm, const Args& a, int grid, cudaStream_t stream) {
  if constexpr (SCORES == kUnlisted) {
    if (form == kSparse) return run_one<FMT, D, kSparse, SCORES>(ctx, tm, a, grid, stream);
    if (form == kSparseFew) return run_one<FMT, D, kSparseFew, SCORES>(ctx, tm, a, grid, stream);
  }
  switch (form) {
    case kTree: return run_one<FMT, D, kTree, SCORES>(ctx, tm, a, grid, stream);
    case kTreeFew: return run_one<FMT, D, kTreeFew, SCORES>(ctx, tm, a, grid, stream);
    default: return run_one<FMT, D, kWide, SCORES>(ctx, tm, a, grid, stream);
  }
}

template <int FMT, int SCORES = kUnlisted, class Args>
dsa_status run_fmt(dsa_ctx* ctx, int form, int D, const CUtensorMap& tm, const Args& a, int grid, cudaStream_t stream) {
  if (D == 128) return run_dim<FMT, 128, SCORES>(ctx, form, tm, a, grid, stream);
  return run_dim<FMT, 64, SCORES>(ctx, form, tm, a, grid, stream);
}

// Where the parts of the workspace begin: two pieces a CTA, 256 rows on each SM
// whatever the form.
struct Workspace {
  size_t ml, part, bytes;
};
Workspace layout(const dsa_ctx* ctx, int D);

// What a call's arguments and workspace say, and a bf16 cache as rows of D
// elements (a page's K or V of one head is 64 of them). In attn.cu.
void fill_args(const dsa_ctx* ctx, const dsa_attn_args& p, AttnArgs& a);
bool cache_map(const dsa_ctx* ctx, const dsa_attn_args& p, int box_rows, CUtensorMap& tm);

// One cache format's kernels: attn.cu (bf16), attn_fp8.cu, attn_fp4.cu.
dsa_status run_bf16(dsa_ctx* ctx, int form, int D, const CUtensorMap& tm, const AttnArgs& a, int grid, cudaStream_t stream);
dsa_status run_fp8(dsa_ctx* ctx, int form, int D, const CUtensorMap& tm, const AttnArgs& a, int grid, cudaStream_t stream);
dsa_status run_fp4(dsa_ctx* ctx, int form, int D, const CUtensorMap& tm, const AttnArgs& a, int grid, cudaStream_t stream);

// Listed units' kernels of one cache format and treatment of the scores:
// span_*.cu, span_cap_*.cu, span_bias_*.cu, span_wide_*.cu, so that they compile in parallel.
using RunSpan = dsa_status(dsa_ctx* ctx, int form, int D, const CUtensorMap& tm, const SpanArgs& a, int grid, cudaStream_t stream);
RunSpan run_span_bf16, run_span_fp8, run_span_fp4, run_span_cap_bf16, run_span_cap_fp8, run_span_cap_fp4, run_span_bias_bf16,
    run_span_bias_fp8, run_span_bias_fp4, run_span_wide_bf16, run_span_wide_fp8, run_span_wide_fp4;

}  // namespace at
}  // namespace dsa
