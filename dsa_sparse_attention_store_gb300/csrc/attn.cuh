// Attention over the paged K/V cache: for a tree of drafted tokens (every
// committed key and the drafted ancestors) and over the indexer's selection.
//
// Mathematics, for a query row (one head of one token) and its visible keys:
//   s_j = scale q.k_j,  o = sum_j 2^(x_j - m) v_j / sum_j 2^(x_j - m),
//   x_j = s_j log2 e,   lse = (m + log2 sum_j 2^(x_j - m)) / log2 e,
// in one pass over key tiles with a running m and sum. Statistics and the
// accumulator are fp32; the weights enter the second product as bf16 (its
// operands share a type, and a weight's relative error of 2^-9 is that of
// the output's own rounding); their sum is of the unrounded weights.
//
// Layout. A unit is one kv head of one sequence and up to 128 of its rows
// (tokens x the G query heads that share the kv head), or, over a selection,
// one kv head of one token (G rows). The units' 64-key tiles (a page each, or
// 64 selected keys) are laid end to end and cut into equal ranges, one per
// CTA, so ragged batches balance whatever their lengths. A unit that a cut
// divides leaves partial sums in the workspace and the join kernel adds them
// in a fixed order.
//
// A CTA: 4 softmax warps (a row per thread and TMEM lane; one thread of them
// issues the products) and 4 loader warps; two CTAs per SM, so that one's softmax runs under the other's
// products. TMEM columns: accumulator [0, D), scores [D, D + 64) with the
// bf16 weights over them, queries [D + 64, D + 64 + D/2): both products take
// their A operand from TMEM, and shared memory holds only a ring of 64-key K
// and V tiles in the 128-byte swizzle (K is read K-major, V MN-major, from
// the same layout).
//
// Loaders: in bf16, tiles that every row sees whole come by TMA; all others
// (fp8 and fp4 codes, selections, the tiles where visibility ends) are read
// into registers one tile ahead, widened, and stored swizzled. Rows of no
// visible key are zeros there, never what the page holds: a weight of zero
// times a stale NaN would be NaN. In tiles that only some rows see, values
// that are not finite are replaced by zeros too and added afterwards to the
// rows that do see them (fix_nonfinite).
#pragma once
#include "kv_format.cuh"
#include "ptx.cuh"

namespace dsa {
namespace at {

constexpr int kTile = 64;
constexpr int kRows = 128;
constexpr int kThreads = 256;
constexpr int kRing = 8;  // entries of the per-tile and per-segment rings; loaders run at most 5 tiles ahead

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
  float2* ml;     // [2 x grid][128]
  float* part;    // [2 x grid][128][D]
  float scale2;   // scale * log2 e
  int B, Tq, max_pages, num_pages, kv_heads, G, k, mask_words, slots;
};

// One stretch of a unit's key tiles.
struct Seg {
  int b, h;
  int r0, rows;       // first row of the unit among its sequence's rows, and how many
  int q0, nd, len;    // the sequence's first query, its queries, its keys (a selection: the query itself, ...)
  int t0, t1, nt;     // tiles [t0, t1) of nt
  int full;           // keys before this position are visible to every row
};

struct Start {
  int b, h, r, tile;
};

template <int D>
struct Cfg {
  static constexpr int NBLK = D / 64;
  static constexpr int SLOT = kTile * D * 2;
  static constexpr int NS = D == 128 ? 6 : 10;
  static constexpr int TMEM = 256;  // a power of two; two CTAs share the SM's 512
  static constexpr uint32_t O = 0, S = D, Q = D + 64;
};

struct Shared {
  uint64_t full[10], empty[10];
  uint64_t mfull[kRing], vdone[kRing];
  uint64_t s_full, o_full, fin;
  unsigned long long vmask[kRing];  // visible keys of a tile, as far as the loader knows
  int bad[kRing];                   // segment number + 1 where a loader replaced a value
  long long scan[16];
  Start start;
  long long total;
  uint32_t tmem;
  int abort;
};

template <int D>
constexpr int smem_bytes() { return Cfg<D>::NS * Cfg<D>::SLOT + static_cast<int>(sizeof(Shared)); }

// Key tiles of the row tile that starts at row r0 (at least one, so that
// rows without a key are written too).
__device__ __forceinline__ int tiles_of(const AttnArgs& a, int nd, int len, int r) {
  int end = len;
  if (!a.mask) end = len - nd + min(nd, static_cast<int>((static_cast<long long>(r + 1) * kRows - 1) / a.G) + 1);
  return max(1, (end + kTile - 1) / kTile);
}

__device__ __forceinline__ bool read_seq(const AttnArgs& a, int b, int& q0, int& nd, int& len) {
  q0 = a.cu_q[b];
  const int q1 = a.cu_q[b + 1];
  len = a.seq_lens[b];
  nd = q1 - q0;
  return q0 >= 0 && q1 >= q0 && q1 <= a.Tq && len >= nd && static_cast<long long>(len) <= 64LL * a.max_pages;
}

template <bool SPARSE>
struct Iter {
  const AttnArgs& a;
  long long left;
  int b, h, r, tile;
  int q0, nd, len, nrt;
  bool ok;
  __device__ Iter(const AttnArgs& a_, const Start& s, long long n) : a(a_), left(n), b(s.b), h(s.h), r(s.r), tile(s.tile) {
    ok = read_seq(a, b, q0, nd, len);
    nrt = static_cast<int>((static_cast<long long>(nd) * a.G + kRows - 1) / kRows);
  }
  // the next stretch; a selection's r is its query
  __device__ bool next(Seg& s) {
    if (left <= 0) return false;
    if constexpr (SPARSE) {
      while (b + 1 < a.B && a.cu_q[b + 1] <= r) {
        ++b;
        ok = read_seq(a, b, q0, nd, len);
      }
      s.nt = max(1, (a.k + kTile - 1) / kTile + (a.mask ? (a.mask_words + 1) / 2 : 0));
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
        nrt = static_cast<int>((static_cast<long long>(nd) * a.G + kRows - 1) / kRows);
        h = r = tile = 0;
      }
      s.nt = tiles_of(a, nd, len, r);
      s.r0 = r * kRows;
      s.rows = min(kRows, nd * a.G - s.r0);
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
    if constexpr (SPARSE) {
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
};

// The launch's tiles, and where this CTA's range begins. Every thread of
// the block calls it; the result is in sh.
template <bool SPARSE>
__device__ __forceinline__ void make_plan(const AttnArgs& a, Shared& sh, int cta, int grid, long long& begin, long long& count) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long total;
  if constexpr (SPARSE) {
    const int nt = max(1, (a.k + kTile - 1) / kTile + (a.mask ? (a.mask_words + 1) / 2 : 0));
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
  // each thread adds up a run of sequences; a scan over the threads places them
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  auto weigh = [&](int b) -> long long {
    int q0, nd, len;
    if (!read_seq(a, b, q0, nd, len)) {
      if (cta == 0) atomicOr(a.status, DSA_DEV_BOUNDS);
      return 0;
    }
    const int nrt = static_cast<int>((static_cast<long long>(nd) * a.G + kRows - 1) / kRows);
    long long n = 0;
    if (a.mask)
      n = static_cast<long long>(nrt) * tiles_of(a, nd, len, 0);
    else
      for (int r = 0; r < nrt; ++r) n += tiles_of(a, nd, len, r);
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
  const long long n = total < grid ? total : grid;
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
      const int nt = tiles_of(a, nd, len, r);
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

// Keys of the tile at position p0 that a row of query i may see (tree form).
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

__device__ __forceinline__ float widen_one(uint32_t bits) { return __uint_as_float(bits << 16); }

// Adds the values that are not finite, of the partially visible tiles
// [t0, t1), to the rows that see their keys. Only reached where a loader
// found one.
template <int FMT, int D>
__device__ __noinline__ void fix_nonfinite(const AttnArgs& a, const Seg& s, int t0, int t1, int i, bool valid, uint32_t o_taddr) {
  using L = kvf::Layout<FMT, D>;
  for (int d = 0; d < D; ++d) {
    float add = 0.f;
    for (int t = t0; t < t1; ++t) {
      if (t * kTile >= s.len) break;
      const int page = a.page_table[static_cast<long long>(s.b) * a.max_pages + t];
      if (page < 0 || page >= a.num_pages) continue;
      const uint8_t* blk = a.cache + (static_cast<long long>(page) * a.kv_heads + s.h) * L::HEAD_BYTES;
      unsigned long long m = valid ? row_mask(a, s, i, t * kTile) & low_bits(s.len - t * kTile) : 0ull;
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
    const float o = __uint_as_float(tmem_ld1(o_taddr + d));
    __syncwarp();
    tmem_st1(o_taddr + d, __float_as_uint(o + add));
  }
}

template <int FMT, int D, bool SPARSE>
__global__ void __launch_bounds__(kThreads, 2) attn_kernel(const __grid_constant__ CUtensorMap tm, const AttnArgs a) {
  using C = Cfg<D>;
  using L = kvf::Layout<FMT, D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem + C::NS * C::SLOT);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, grid = gridDim.x;

  if (tid == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&sh.full[i], 4);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sh.mfull[i], 1);
      mbar_init(&sh.vdone[i], 4);
      sh.bad[i] = 0;
    }
    mbar_init(&sh.s_full, 1);
    mbar_init(&sh.o_full, 1);
    mbar_init(&sh.fin, 1);
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
  const uint32_t tb = sh.tmem;
  pdl_wait();
  pdl_trigger();
  long long begin, count;
  make_plan<SPARSE>(a, sh, cta, grid, begin, count);
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

  if (count <= 0) {
    if (tid == 0) a.meta[2 * cta] = make_int4(0, 0, 0, 0);
  } else if (warp < 4) {
    // ------------------------------------------------------------ softmax
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tO = tb + C::O + lanes, tS = tb + C::S + lanes, tQ = tb + C::Q + lanes;
    Iter<SPARSE> it(a, sh.start, count);
    Seg s;
    bool more = it.next(s), run = true;
    int seg = 0, n = 0;
    int4 m0 = make_int4(0, 0, 0, 0), m1 = m0;
    // the ring slot the next product reads, and the products themselves: one
    // thread of warp 0 issues them, after a barrier of the four warps
    int slot = 0, round = 0;
    auto advance = [&]() {
      if (++slot == C::NS) {
        slot = 0;
        round ^= 1;
      }
    };
    constexpr uint32_t kIdescQk = idesc_f16(128, kTile, true);
    constexpr uint32_t kIdescPv = idesc_f16(128, D, true) | kIdescBMn;
    const uint64_t kdesc = sw128_desc(smem_u32(smem)), vdesc = sw128_mn_desc(smem_u32(smem), kTile * 128);
    // Called by the whole warp; the operands come from lane 0, so that the
    // compiler keeps them in uniform registers (issue took 1100 cycles a tile
    // without, most of it moving operands)
    auto scores = [&](int at) {
      const uint64_t k = kdesc + __shfl_sync(0xffffffffu, at, 0) * (C::SLOT >> 4);
      if (!elect_one()) return;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        tc_mma_f16_ta(tb + C::S, tb + C::Q + 8 * i, k + (((i / 4) * (kTile * 128) + (i % 4) * 32) >> 4), kIdescQk, i > 0);
      tc_commit(&sh.empty[at]);
      tc_commit(&sh.s_full);
    };
    auto values = [&](int at, bool first, bool last) {
      const uint64_t v = vdesc + __shfl_sync(0xffffffffu, at, 0) * (C::SLOT >> 4);
      if (!elect_one()) return;
#pragma unroll
      for (int i = 0; i < kTile / 16; ++i)
        tc_mma_f16_ta(tb + C::O, tb + C::S + 8 * i, v + ((i * 2048) >> 4), kIdescPv, !first || i > 0);
      tc_commit(&sh.empty[at]);
      if (last) tc_commit(&sh.o_full);
    };
    auto load_q = [&](const Seg& g) {
      const bool valid = tid < g.rows;
      const int r = g.r0 + tid;
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (valid ? static_cast<long long>(g.q0 + r / a.G) * a.qt + static_cast<long long>(g.h * a.G + r % a.G) * a.qh : 0));
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
        tmem_st32(tQ + 32 * c, w);
      }
      tmem_st_wait();
      tc_fence_before();
      if (warp == 0) run = run && wait_warp(&sh.full[slot], round);
      run = named_bar_all(1, 128, run);  // the four warps go on, or stop, together
      if (warp == 0 && run) {
        tc_fence_after();
        scores(slot);
        __syncwarp();
      }
      advance();
    };
    if (more) load_q(s);
    while (more) {
      const bool active = warp * 32 < s.rows;  // some row of this warp is real
      const bool valid = tid < s.rows;
      const int qi = (s.r0 + tid) / a.G;       // the row's query in its sequence
      float m = -INFINITY, l = 0.f;
      for (int t = s.t0; t < s.t1; ++t, ++n) {
        run = run && wait_warp(&sh.mfull[n % kRing], (n / kRing) & 1);
        const unsigned long long vm = sh.vmask[n % kRing];
        // V of this tile and K of the next, usually long there: looked at
        // while the scores are on their way
        const bool more_tiles = t + 1 < s.t1;
        const int vslot = slot, vround = round;
        advance();
        bool there = true;
        if (warp == 0)
          there = __all_sync(0xffffffffu, mbar_try_wait(smem_u32(&sh.full[vslot]), vround) &&
                                              (!more_tiles || mbar_try_wait(smem_u32(&sh.full[slot]), round)));
        run = run && wait_warp(&sh.s_full, n & 1);
        tc_fence_after();
        if (active && run) {
          uint32_t x0[32], x1[32];
          tmem_ld32(tS, x0);
          tmem_ld_wait32(x0);
          tmem_ld32(tS + 32, x1);
          const int p0 = t * kTile;
          unsigned long long see = vm;
          if (!SPARSE && valid && p0 + kTile > s.full) see &= row_mask(a, s, qi, p0);
          const bool some = __any_sync(0xffffffffu, see != ~0ull);  // a key that some row does not see
          if (some) {
            const uint32_t lo = static_cast<uint32_t>(see);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((lo >> i) & 1)) x0[i] = 0xFF800000u;
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            mx[(i >> 1) & 3] = fmaxf(mx[(i >> 1) & 3], fmaxf(__uint_as_float(x0[i]), __uint_as_float(x0[i + 1])));
          tmem_ld_wait32(x1);
          if (some) {
            const uint32_t hi = static_cast<uint32_t>(see >> 32);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((hi >> i) & 1)) x1[i] = 0xFF800000u;
          }
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            mx[(i >> 1) & 3] = fmaxf(mx[(i >> 1) & 3], fmaxf(__uint_as_float(x1[i]), __uint_as_float(x1[i + 1])));
          const float mnew = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale2;
          // the running maximum moves only when it grows by more than 2^8:
          // the weights stay below 2^8 and the accumulator is rarely rescaled
          const bool grow = mnew > m + 8.f || (m == -INFINITY && mnew > m);
          if (__any_sync(0xffffffffu, grow)) {
            const float to = grow ? mnew : m;
            const float alpha = grow ? ex2(m - mnew) : 1.f;
            if (t > s.t0) {  // s_full of this tile follows the last tile's second product
              l *= alpha;
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) tmem_scale16(tO + 16 * c, alpha);
              tmem_st_wait();
            }
            m = to;
          }
          const float sub = m == -INFINITY ? 0.f : m;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          auto weigh = [&](const uint32_t (&x)[32], uint32_t at) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float e0 = ex2(fmaf(__uint_as_float(x[2 * i]), a.scale2, -sub));
              const float e1 = ex2(fmaf(__uint_as_float(x[2 * i + 1]), a.scale2, -sub));
              sum[(2 * i) & 3] += e0;
              sum[(2 * i + 1) & 3] += e1;
              const __nv_bfloat162 w = __floats2bfloat162_rn(e0, e1);
              memcpy(&p[i], &w, 4);
            }
            tmem_st16(at, p);
          };
          weigh(x0, tS);  // over scores that are in registers by now
          weigh(x1, tS + 16);
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        if (warp == 0 && run && !there) {
          run = wait_warp(&sh.full[vslot], vround);
          if (run && more_tiles) run = wait_warp(&sh.full[slot], round);
        }
        tmem_st_wait();
        tc_fence_before();
        run = named_bar_all(1, 128, run);
        if (warp == 0 && run) {
          tc_fence_after();
          values(vslot, t == s.t0, !more_tiles);
          __syncwarp();
          if (more_tiles) scores(slot);
          __syncwarp();
        }
        if (more_tiles) advance();
        if (!run) break;
      }
      if (!run) break;
      // the next unit's queries go up before this one's sums come down: every
      // product with the old ones has completed (s_full of the last tile)
      const Seg done = s;
      more = it.next(s);
      if (more) load_q(s);
      run = run && wait_warp(&sh.o_full, seg & 1);
      if (!SPARSE) run = run && wait_warp(&sh.vdone[seg % kRing], (seg / kRing) & 1);
      tc_fence_after();
      const bool first = done.t0 == 0, last = done.t1 == done.nt;
      if (!first) {
        m0.y = 1;
        m0.z = last;
      } else if (!last) {
        m0.x = 1;
        m0.w = done.rows;
        m1 = make_int4(done.r0, done.q0, done.h, 0);
      }
      if (active && run) {
        if (!SPARSE && *static_cast<volatile int*>(&sh.bad[seg % kRing]) == seg + 1)
          fix_nonfinite<FMT, D>(a, done, max(done.t0, done.full / kTile), done.t1, qi, valid, tO);
        const int r = done.r0 + tid;
        const long long tok = done.q0 + r / a.G;
        const int head = done.h * a.G + r % a.G;
        const int slot = 2 * cta + (first ? 1 : 0);
        const float inv = l > 0.f ? 1.f / l : 0.f;
        __nv_bfloat16* dst = a.out + tok * a.ot + head * a.oh;
        float* part = a.part + (static_cast<long long>(slot) * kRows + tid) * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + 32 * c, o);
          tmem_ld_wait32(o);
          if (!valid) {
          } else if (first && last) {
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
          __syncwarp();
        }
        if (valid) {
          if (first && last) {
            if (a.lse) a.lse[tok * a.kv_heads * a.G + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
          } else {
            a.ml[static_cast<long long>(slot) * kRows + tid] = make_float2(m, l);
          }
        }
        tc_fence_before();
      }
      ++seg;
    }
    if (tid == 0) {
      a.meta[2 * cta] = m0;
      a.meta[2 * cta + 1] = m1;
      // products in flight end before their TMEM goes back, after an abort too
      tc_commit(&sh.fin);
      mbar_wait(&sh.fin, 0);
    }
  } else {
    // ------------------------------------------------------------ loaders
    constexpr int CPB = FMT == DSA_FMT_BF16 ? 8 : FMT == DSA_FMT_FP8 ? 4 : 2;  // 16-byte chunks of a row's 64 dimensions
    constexpr int RL = 8 / CPB;            // rows that 8 lanes cover: their stores hit all 32 banks
    constexpr int NCH = C::NBLK * CPB / 2; // chunks a thread moves per tile
    constexpr int RSTEP = RL * 16 / C::NBLK;
    const int lt = tid - 128, lw = warp - 4;
    const int chunk = lt % CPB, blk = (lt / 8) % C::NBLK;
    const int row0 = (lt / (8 * C::NBLK)) * RL + (lt / CPB) % RL;
    const int code_off = (blk * CPB + chunk) * 16;
    const int scale_off = (blk * 64 + chunk * (64 / CPB)) / kvf::kBlock;
    struct Tile {
      uint4 raw[NCH];
      uint32_t sc[FMT == DSA_FMT_BF16 ? 1 : NCH];
    };
    int slot = 0, round = 0, issued = 0;  // the next ring slot
    auto advance = [&]() {
      ++issued;
      if (++slot == C::NS) {
        slot = 0;
        round ^= 1;
      }
    };
    // where each of this thread's rows lies: a page and an offset, or none
    auto fetch = [&](Tile& t, const int (&at)[NCH], int h, bool v) {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        t.raw[i] = make_uint4(0, 0, 0, 0);
        if (FMT != DSA_FMT_BF16) t.sc[FMT == DSA_FMT_BF16 ? 0 : i] = 0;
        if (at[i] >= 0) {
          const uint8_t* b = a.cache + (static_cast<long long>(at[i] >> 6) * a.kv_heads + h) * L::HEAD_BYTES;
          const int off = at[i] & 63;
          t.raw[i] = __ldg(reinterpret_cast<const uint4*>(b + (v ? L::V_CODES : L::K_CODES) + off * L::CB + code_off));
          if (FMT != DSA_FMT_BF16)
            t.sc[FMT == DSA_FMT_BF16 ? 0 : i] = __ldg(b + (v ? L::V_SCALES : L::K_SCALES) + off * L::SB + scale_off);
        }
      }
    };
    // widened, into the ring; `clean` replaces what is not finite and reports it
    auto commit = [&](const Tile& t, bool clean, int seg) -> bool {
      if (!wait_warp(&sh.empty[slot], round ^ 1)) return false;
      uint8_t* base = smem + slot * C::SLOT + blk * (kTile * 128);
      bool found = false;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int row = row0 + i * RSTEP;
        uint32_t w[32 / CPB];
        if constexpr (FMT == DSA_FMT_BF16) {
          w[0] = t.raw[i].x;
          w[1] = t.raw[i].y;
          w[2] = t.raw[i].z;
          w[3] = t.raw[i].w;
        } else if constexpr (FMT == DSA_FMT_FP8) {
          const kvf::Factor<FMT> f(t.sc[i]);
          const uint32_t c[4] = {t.raw[i].x, t.raw[i].y, t.raw[i].z, t.raw[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t o[2];
            kvf::widen_e4m3(c[j], f, o);
            w[2 * j] = o[0];
            w[2 * j + 1] = o[1];
          }
        } else {
          const kvf::Factor<FMT> f(t.sc[i]);
          const uint32_t c[4] = {t.raw[i].x, t.raw[i].y, t.raw[i].z, t.raw[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t o[4];
            kvf::widen_e2m1(c[j], f, o);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[4 * j + e] = o[e];
          }
        }
        if (clean) {
#pragma unroll
          for (int j = 0; j < 32 / CPB; ++j) {
            if ((w[j] & 0x7F800000u) == 0x7F800000u) {
              w[j] &= 0x0000FFFFu;
              found = true;
            }
            if ((w[j] & 0x7F80u) == 0x7F80u) {
              w[j] &= 0xFFFF0000u;
              found = true;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 8 / CPB; ++j) {
          const int unit = (chunk * (8 / CPB) + j) ^ (row & 7);
          *reinterpret_cast<uint4*>(base + row * 128 + unit * 16) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        }
      }
      if (found) *static_cast<volatile int*>(&sh.bad[seg % kRing]) = seg + 1;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.full[slot]);
      advance();
      return true;
    };

    Iter<SPARSE> it(a, sh.start, count);
    Seg s;
    int seg = 0, n = 0;
    bool run = true;
    Tile hold;                                   // a V tile on its way from memory
    bool pending = false, hold_clean = false;
    int hold_seg = 0, hold_last = 0;
    auto flush = [&]() -> bool {                 // it goes into the ring
      if (!pending) return true;
      pending = false;
      if (!commit(hold, hold_clean, hold_seg)) return false;
      if (hold_last) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.vdone[hold_seg % kRing]);
      }
      return true;
    };
    while (run && it.next(s)) {
      const int32_t* pt = a.page_table + static_cast<long long>(s.b) * a.max_pages;
      int pg = -1;
      const int npg = (s.len + kTile - 1) / kTile;
      // a selection: this lane's two keys of a tile, as cache slots
      auto slot_of = [&](int t, int j) -> int {
        int x = t * kTile + j, pos;
        const int ksel = (a.k + kTile - 1) / kTile * kTile;
        if (x < a.k) {
          pos = a.sel[static_cast<long long>(s.q0) * a.k + x];
          if (pos < 0 || s.len == 0) return -1;
          if (a.slots) {
            if (pos < a.num_pages * 64) return pos;
            atomicOr(a.status, DSA_DEV_BOUNDS);
            return -1;
          }
          if (pos >= s.len) {
            atomicOr(a.status, DSA_DEV_BOUNDS);
            return -1;
          }
        } else {
          x -= ksel;
          if (x < 0 || !a.mask || x >= s.nd || (x >> 5) >= a.mask_words) return -1;
          if (!((a.mask[static_cast<long long>(s.q0) * a.mask_words + (x >> 5)] >> (x & 31)) & 1)) return -1;
          pos = s.len - s.nd + x;
        }
        const int page = pt[pos >> 6];
        if (page < 0 || page >= a.num_pages) {
          atomicOr(a.status, DSA_DEV_BOUNDS);
          return -1;
        }
        return page * 64 + (pos & 63);
      };
      int k0 = -1, k1 = -1;
      if (SPARSE) {
        k0 = slot_of(s.t0, lane);
        k1 = slot_of(s.t0, lane + 32);
      }
      for (int t = s.t0; t < s.t1; ++t, ++n) {
        int at[NCH];
        unsigned long long vm;
        bool tma = false, clean = false;
        int page = -1;
        if constexpr (SPARSE) {
          vm = __ballot_sync(0xffffffffu, k0 >= 0) |
               (static_cast<unsigned long long>(__ballot_sync(0xffffffffu, k1 >= 0)) << 32);
#pragma unroll
          for (int i = 0; i < NCH; ++i) {
            const int row = row0 + i * RSTEP;
            const int u = __shfl_sync(0xffffffffu, k0, row & 31), v = __shfl_sync(0xffffffffu, k1, row & 31);
            at[i] = row < 32 ? u : v;
          }
          if (t + 1 < s.t1) {
            k0 = slot_of(t + 1, lane);
            k1 = slot_of(t + 1, lane + 32);
          }
        } else {
          const int rel = (t - s.t0) & 31;
          if (rel == 0) pg = t + lane < min(s.t1, npg) ? pt[t + lane] : -1;
          page = __shfl_sync(0xffffffffu, pg, rel);
          const bool ok = page >= 0 && page < a.num_pages;
          if (!ok && t < npg && lw == 0 && lane == 0) atomicOr(a.status, DSA_DEV_BOUNDS);
          vm = ok ? low_bits(s.len - t * kTile) : 0ull;
          tma = FMT == DSA_FMT_BF16 && ok && (t + 1) * kTile <= s.full;
          clean = (t + 1) * kTile > s.full;
#pragma unroll
          for (int i = 0; i < NCH; ++i) {
            const int row = row0 + i * RSTEP;
            at[i] = (vm >> row) & 1 ? page * 64 + row : -1;
          }
        }
        Tile kt;
        if (!tma) fetch(kt, at, s.h, false);
        if (!flush()) {
          run = false;
          break;
        }
        if (lw == 0 && lane == 0) {
          sh.vmask[n % kRing] = vm;
          mbar_arrive(&sh.mfull[n % kRing]);
        }
        if (tma) {
          // K, then V: a page's 64 rows, 64 dimensions a box
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            if (!wait_warp(&sh.empty[slot], round ^ 1)) {
              run = false;
              break;
            }
            if (lane == 0) {
              if (lw == 0) {
                mbar_arrive_expect_tx(&sh.full[slot], C::SLOT);
                const int y = ((page * a.kv_heads + s.h) * 2 + v) * kTile;
#pragma unroll
                for (int c = 0; c < C::NBLK; ++c)
                  tma_load_2d(smem + slot * C::SLOT + c * (kTile * 128), &tm, c * 64, y, &sh.full[slot]);
              } else {
                mbar_arrive(&sh.full[slot]);
              }
            }
            advance();
          }
          if (!run) break;
          if (t + 1 == s.t1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.vdone[seg % kRing]);
          }
        } else {
          fetch(hold, at, s.h, true);
          if (!commit(kt, false, seg)) {
            run = false;
            break;
          }
          pending = true;
          hold_clean = clean;
          hold_seg = seg;
          hold_last = t + 1 == s.t1;
        }
      }
      ++seg;
    }
    if (run) run = flush();
    // after a wait that ran out, copies in flight land before the CTA exits
    if (*abort_flag && FMT == DSA_FMT_BF16 && lw == 0 && lane == 0) {
      for (int i = 1; i <= C::NS && issued - i >= 0; ++i) {
        const int x = issued - i;
        mbar_wait(&sh.full[x % C::NS], (x / C::NS) & 1, 20000000LL);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tb, C::TMEM);
  }
}

typedef dsa_status (*RunFn)(dsa_ctx*, bool, int, const CUtensorMap&, const AttnArgs&, int, cudaStream_t);

template <int FMT, int D, bool SPARSE>
dsa_status run_one(dsa_ctx* ctx, const CUtensorMap& tm, const AttnArgs& a, int grid, cudaStream_t stream) {
  auto kern = attn_kernel<FMT, D, SPARSE>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<D>()) != cudaSuccess)
    return DSA_ERR_CUDA;
  LaunchScope scope(ctx, DSA_K_ATTN, stream);
  return launch_pdl(kern, dim3(grid), dim3(kThreads), smem_bytes<D>(), stream, tm, a) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

template <int FMT>
dsa_status run_fmt(dsa_ctx* ctx, bool sparse, int D, const CUtensorMap& tm, const AttnArgs& a, int grid, cudaStream_t stream) {
  if (D == 128)
    return sparse ? run_one<FMT, 128, true>(ctx, tm, a, grid, stream) : run_one<FMT, 128, false>(ctx, tm, a, grid, stream);
  return sparse ? run_one<FMT, 64, true>(ctx, tm, a, grid, stream) : run_one<FMT, 64, false>(ctx, tm, a, grid, stream);
}

// One cache format's kernels: attn.cu (bf16), attn_fp8.cu, attn_fp4.cu.
dsa_status run_bf16(dsa_ctx* ctx, bool sparse, int D, const CUtensorMap& tm, const AttnArgs& a, int grid, cudaStream_t stream);
dsa_status run_fp8(dsa_ctx* ctx, bool sparse, int D, const CUtensorMap& tm, const AttnArgs& a, int grid, cudaStream_t stream);
dsa_status run_fp4(dsa_ctx* ctx, bool sparse, int D, const CUtensorMap& tm, const AttnArgs& a, int grid, cudaStream_t stream);

}  // namespace at
}  // namespace dsa
