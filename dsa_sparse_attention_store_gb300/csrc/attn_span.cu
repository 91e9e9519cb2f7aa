// Attention of spans and behind shared prefixes: the plan of the units and the
// launches. The attention itself is attn.cuh's span form.
//
// The plan lists units of up to 32, 128 or 256 rows (tokens x the G query heads
// of a kv head; one list for all kv heads) with the 64-key tiles that one of
// their tokens sees. It says of each token which places it sees, and of each
// unit which places all of its tokens see, where no masks are needed. A unit of
// sequence b that begins at its row r0 = r rows has the place
//   floor(cu_q[b] G / rows) + b + r
// in the list: different for all units, in order, and with at most one gap a
// sequence, so no scan over the sequences comes first. In the list of groups the
// places of rows that share nothing are gaps too; the attention's warps pass gaps
// one by one, where they come to the end of the list for a kv head (64 decode steps
// behind a prefix beside a prefill of 8192 tokens 1432 us, apart 1241 and 91).
//
// Behind shared prefixes there are two lists. The first takes a group's
// sequences for one, with all of their tokens, and the whole pages that they
// share. The second takes each sequence alone and the keys behind those pages.
// The sums of both go to the workspace, 32 bits each, and are joined row by row.
#include <algorithm>
#include <cmath>

#include "attn_join.cuh"

namespace dsa {
namespace at {

struct SpanPlan {
  const int32_t *first, *last;
  const int32_t *cu_groups, *shared;  // or null
  int4* tokens;
  int4 *units, *group_units;    // of sequences, of groups
  int *tiles, *group_tiles;
  int n, group_n, rows, group_rows, groups, window;
};

// The last i < N with before(i) <= u, before not decreasing (0 if there is
// none). A warp's lanes look at 32 places at a time.
template <class F>
__device__ __forceinline__ int last_at(int N, long long u, F before) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = N;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step;
    const int c = __popc(__ballot_sync(0xffffffffu, i < hi && before(i) <= u));
    lo += c * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// the last i of [lo, hi) with x[i] <= u, by one thread
__device__ __forceinline__ int last_of(const int32_t* x, int lo, int hi, int u) {
  while (hi - lo > 1) {
    const int i = lo + (hi - lo) / 2;
    if (x[i] <= u)
      lo = i;
    else
      hi = i;
  }
  return lo;
}

__device__ __forceinline__ bool read_group(const AttnArgs& a, const SpanPlan& p, int g, int& b0, int& b1) {
  b0 = p.cu_groups[g];
  b1 = p.cu_groups[g + 1];
  return b0 >= 0 && b0 <= b1 && b1 <= a.B;
}

// Whole pages that group g's sequences read from the first one's row; one
// sequence alone has none to share. Nor has a group whose queries do not lie
// between those of q: it has no units, and its good sequences read all their keys
// themselves.
__device__ __forceinline__ int shared_pages(const AttnArgs& a, const SpanPlan& p, int g) {
  int b0, b1, q0, nd, len;
  if (!read_group(a, p, g, b0, b1) || b1 - b0 < 2 || !read_seq(a, b0, q0, nd, len)) return 0;
  const int q1 = a.cu_q[b1];
  if (q1 < q0 || q1 > a.Tq) return 0;
  return max(0, min(p.shared[g], len)) / kTile;
}

// What token i of sequence b sees.
__device__ __forceinline__ Token token_of(const AttnArgs& a, const SpanPlan& p, int q0, int nd, int len, int i) {
  Token y;
  y.ctx = len - nd;
  y.place = y.ctx + i;
  y.lo = p.first ? p.first[q0 + i] : 0;
  if (p.window) y.lo = max(y.lo, y.place - p.window + 1);
  y.lo = max(y.lo, 0);
  y.hi = min(len, p.last ? p.last[q0 + i] : a.mask ? len : y.place + 1);
  if (y.hi <= y.lo) y.lo = y.hi = 0;
  return y;
}

// A warp a place of the lists.
__global__ void __launch_bounds__(256) span_plan_kernel(const AttnArgs a, const SpanPlan p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long at = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) >> 5, self = at * 32 + lane;
  int q0, nd, len;
  if (self < a.B && !read_seq(a, static_cast<int>(self), q0, nd, len)) atomicOr(a.status, DSA_DEV_BOUNDS);
  if (self < p.groups) {
    int b0, b1;
    if (!read_group(a, p, static_cast<int>(self), b0, b1) || p.shared[self] < 0) atomicOr(a.status, DSA_DEV_BOUNDS);
  }
  if (at >= static_cast<long long>(p.n) + p.group_n) return;
  const bool group = at >= p.n;
  const int u = static_cast<int>(group ? at - p.n : at), rows = group ? p.group_rows : p.rows;
  int* const tiles = (group ? p.group_tiles : p.tiles) + u;
  // the sequences' first row of the page table, queries and keys; t0, t1: tiles they may have
  int b, b1, r, t0, t1;
  bool ok;
  if (!group) {
    auto before = [&](int i) -> long long { return static_cast<long long>(a.cu_q[i]) * a.G / rows + i; };
    b = last_at(a.B, u, before);
    b1 = b + 1;
    ok = read_seq(a, b, q0, nd, len);
    const long long from = u - before(b);
    r = static_cast<int>(from);
    ok = ok && from >= 0;
    t0 = 0;
    t1 = 0x7FFFFFFF;
    if (p.groups) {
      const int g = last_of(p.cu_groups, 0, p.groups, b);
      int g0, g1;
      if (read_group(a, p, g, g0, g1) && g0 <= b && b < g1) t0 = shared_pages(a, p, g);
    }
  } else {
    auto before = [&](int i) -> long long {
      return static_cast<long long>(a.cu_q[min(max(p.cu_groups[i], 0), a.B)]) * a.G / rows + i;
    };
    const int g = last_at(p.groups, u, before);
    ok = read_group(a, p, g, b, b1);
    t0 = 0;
    t1 = ok ? shared_pages(a, p, g) : 0;
    ok = ok && t1 > 0;
    q0 = ok ? a.cu_q[b] : 0;
    const int q1 = ok ? a.cu_q[b1] : 0;
    nd = q1 - q0;
    len = t1 * kTile;
    ok = ok && q0 >= 0 && q1 >= q0 && q1 <= a.Tq;
    const long long from = u - before(g);
    r = static_cast<int>(from);
    ok = ok && from >= 0;
  }
  if (!ok || static_cast<long long>(r) * rows >= static_cast<long long>(nd) * a.G) {
    if (lane == 0) {
      *tiles = 0;
      (group ? p.group_units : p.units)[3LL * u + 1] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  const int r0 = r * rows;
  const int i0 = r0 / a.G, i1 = static_cast<int>((min(static_cast<long long>(r0) + rows, static_cast<long long>(nd) * a.G) - 1) / a.G);
  int min_lo = 0x7FFFFFFF, max_lo = 0, min_hi = len, max_hi = 0;
  for (int i = i0 + lane; i <= i1; i += 32) {
    Token y;
    if (!group) {
      y = token_of(a, p, q0, nd, len, i);
    } else {
      int s0, sn, sl;
      const int t = q0 + i, s = last_of(a.cu_q, b, b1, t);
      y = Token{0, 0, 0, 0};
      if (read_seq(a, s, s0, sn, sl) && s0 <= t && t < s0 + sn) y = token_of(a, p, s0, sn, sl, t - s0);
    }
    p.tokens[q0 + i] = make_int4(y.lo, y.hi, y.place, y.ctx);  // the same from every warp that has the token
    if (y.hi > 0) min_lo = min(min_lo, y.lo);
    max_lo = max(max_lo, y.lo);
    max_hi = max(max_hi, y.hi);
    min_hi = min(min_hi, a.mask ? min(y.hi, y.ctx) : y.hi);
  }
  min_lo = __reduce_min_sync(0xffffffffu, min_lo);
  max_lo = __reduce_max_sync(0xffffffffu, max_lo);
  min_hi = __reduce_min_sync(0xffffffffu, min_hi);
  max_hi = __reduce_max_sync(0xffffffffu, max_hi);
  if (lane == 0) {
    const int base = !group && t0 > 0;
    int group_q0 = 0, group_at = 0;
    if (base) {
      const int g = last_of(p.cu_groups, 0, p.groups, b);
      group_q0 = a.cu_q[p.cu_groups[g]];
      group_at = static_cast<int>(static_cast<long long>(group_q0) * a.G / p.group_rows + g);
    }
    int e0 = max(t0, min_lo / kTile), e1 = min(t1, (max_hi + kTile - 1) / kTile);
    if (e1 <= e0) {  // nothing to see: one tile, so that the rows are written
      e0 = t0;
      e1 = t0 + 1;
    }
    int4* const x = (group ? p.group_units : p.units) + 3LL * u;
    x[0] = make_int4(b, q0, nd, len);
    x[1] = make_int4(r0, e0, e1, base);
    x[2] = make_int4(max_lo, min_hi, group_q0, group_at);
    *tiles = e1 - e0;
  }
}

// The join behind shared prefixes: of each row's sums over the prefix and over
// its sequence's own keys, each whole or in the pieces of the CTAs that the cuts
// gave a part to. A row a warp; in the order of the keys, so the result does not
// depend on timing.
struct RowsJoin {
  SpanArgs group, own;  // the two passes
  int group_rows, own_rows, group_grid, own_grid;
};

// Whether a pass left a unit's ends: not after a wait that ran out.
__device__ __forceinline__ bool ends_there(int2 e, int grid) { return e.x >= 0 && e.x <= e.y && e.y < grid; }

template <int D>
__global__ void __launch_bounds__(256) rows_join_kernel(const RowsJoin j) {
  constexpr int E = D / 32;  // dimensions a lane holds
  pdl_wait();
  pdl_trigger();
  const SpanArgs &a = j.own, &b = j.group;
  const int u = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.z * 8 + warp;  // of the unit
  if (a.tiles[u] == 0) return;
  const int4 x = a.units[3 * u], y = a.units[3 * u + 1], z = a.units[3 * u + 2];
  if (y.x + static_cast<long long>(row) >= static_cast<long long>(x.z) * a.G) return;
  const bool base = y.w;
  const int i = (y.x + row) / a.G, g = y.x + row - i * a.G;
  const long long tok = x.y + i, r = base ? (tok - z.z) * a.G + g : 0;  // and the row of the group
  const int place = z.w + static_cast<int>(r / j.group_rows);
  for (int h = blockIdx.y; h < a.kv_heads; h += gridDim.y) {
    const int2 own = a.ends[static_cast<long long>(u) * a.kv_heads + h];
    if (!ends_there(own, j.own_grid) || (!base && own.x == own.y)) continue;  // nothing there, or written as it is
    int2 all = make_int2(0, -1);
    if (base) {
      // a group's queries that do not hang together (reported by the plan) may have no units
      if (r < 0 || place < 0 || place >= b.units_n || b.tiles[place] == 0) continue;
      all = b.ends[static_cast<long long>(place) * a.kv_heads + h];
      if (!ends_there(all, j.group_grid)) continue;
    }
    const int head = h * a.G + g, before = all.y - all.x + 1, n = before + own.y - own.x + 1;
    const long long at = tok * a.kv_heads * a.G + head;
    // where piece p is, the prefix's first: maximum and sum, and sums
    auto piece = [&](int p, const float2*& ml, const float*& o) {
      const bool of_group = p < before;
      const SpanArgs& q = of_group ? b : a;
      const int2 e = of_group ? all : own;
      const int rows = of_group ? j.group_rows : j.own_rows, k = of_group ? p : p - before;
      const long long slot = (2LL * (e.x + k) + (k == 0)) * rows + (of_group ? static_cast<int>(r % j.group_rows) : row);
      ml = e.x == e.y ? q.raw_ml + at : q.ml + slot;
      o = e.x == e.y ? q.raw + at * D : q.part + slot * D;
    };
    float m = -INFINITY, l = 0.f, o[E] = {};
    for (int p0 = 0; p0 < n; p0 += 32) {  // a lane a piece: the maxima
      const float2* ml;
      const float* src = a.raw;
      float2 v = make_float2(-INFINITY, 0.f);
      if (p0 + lane < n) {
        piece(p0 + lane, ml, src);
        v = __ldcg(ml);
      }
      float top = v.x;
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      top = fmaxf(top, m);
      // sums hold weights of more than 1: denormal factors count
      const float old = m == top ? 1.f : ex2_denorm(m - top), now = v.x == top ? 1.f : ex2_denorm(v.x - top);
      l *= old;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= old;
      m = top;
#pragma unroll 8
      for (int p = 0; p < min(32, n - p0); ++p) {
        const float w = __shfl_sync(0xffffffffu, now, p);
        const float* at_p = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), p));
        l = fmaf(__shfl_sync(0xffffffffu, v.y, p), w, l);
        if constexpr (E == 4) {
          const float4 f = __ldcg(reinterpret_cast<const float4*>(at_p) + lane);
          o[0] = fmaf(f.x, w, o[0]);
          o[1] = fmaf(f.y, w, o[1]);
          o[2] = fmaf(f.z, w, o[2]);
          o[3] = fmaf(f.w, w, o[3]);
        } else {
          const float2 f = __ldcg(reinterpret_cast<const float2*>(at_p) + lane);
          o[0] = fmaf(f.x, w, o[0]);
          o[1] = fmaf(f.y, w, o[1]);
        }
      }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      const __nv_bfloat162 v = l == 0.f ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(o[2 * e] * inv, o[2 * e + 1] * inv);
      memcpy(&w[e], &v, 4);
    }
    __nv_bfloat16* dst = a.out + tok * a.ot + head * a.oh + lane * E;
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(dst) = w[0];
    if (a.lse && lane == 0) {
      if (a.slopes) m -= a.slopes[head] * 1.4426950408889634f * away(token_at(a, tok));
      a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
  }
}

// The form for n sequences (or groups) with these rows in all; the rule is launch_attn's.
struct Shape {
  int form, rows, grid, places;  // rows of a unit, CTAs, places of the list
};

Shape shape_of(const dsa_ctx* ctx, long long rows, int n) {
  Shape f;
  f.form = rows > 128LL * n ? kWide : rows <= static_cast<long long>(kFewRows) * n ? kTreeFew : kTree;
  f.rows = f.form == kWide ? 256 : f.form == kTreeFew ? kFewRows : 128;
  f.grid = f.form == kWide ? ctx->num_sms : 2 * ctx->num_sms;
  f.places = static_cast<int>(rows / f.rows) + n + 1;
  return f;
}

// The cap as the kernels have it. tanh(y) / y in powers of y^2, for |y| up to
// 0.625: minimax in tanh's absolute error (2^-25; evaluated in fp32, 2^-23.5), by
// least squares with weights raised where the error was largest until it was
// level. y = scale q.k / cap.
void cap_args(double scale, double cap, SpanArgs& a) {
  constexpr double kTanh[kCapTerms] = {0.999999463558197, -0.33330482244491577, 0.13291031122207642, -0.05136286839842796,
                                       0.014530066400766373};
  const double log2e = 1.4426950408889634, k = scale / cap;
  a.cap2 = static_cast<float>(cap * log2e);
  a.to_cap = static_cast<float>(2 * log2e * k);
  a.to_ratio = static_cast<float>(k);
  const double range = cap * log2e;
  if (range > kCapOne) {
    for (int i = 0; i < kCapTerms; ++i) a.poly[i] = static_cast<float>(kTanh[i] * range);
    a.poly_most = static_cast<float>(kCapPoly * kCapPoly);
    return;
  }
  double power = k * range;
  bool fits = true;
  for (int i = 0; i < kCapTerms; ++i, power *= k * k) {
    a.poly[i] = static_cast<float>(kTanh[i] * power);
    fits = fits && std::isfinite(a.poly[i]) && std::fabs(a.poly[i]) >= 1.17549435e-38f;
  }
  a.poly_most = static_cast<float>(kCapPoly / k * (kCapPoly / k));
  // a scale far from the usual ones (for a cap of 50, below 0.003): never by the polynomial
  if (!fits || !std::isfinite(a.poly_most)) a.poly_most = -1.f;
  // Capped scores lie within cap of zero, so all rows can be weighed under the
  // same exponent and no maximum is looked for: the largest possible weight is 2^H.
  // H is 8, or as much as keeps the smallest one at 2^-72 or, from a cap of 50 on,
  // as far below 1 as 2^H is above: a row whose keys all score near -cap has no
  // other weights, and its values are to keep their bits in fp32 sums just as the
  // ones of a row near cap are to keep them finite.
  const double room = std::fmax(8.0, std::fmin(2 * range - 72, range));
  if (!a.slopes) a.fixed = static_cast<float>(range - room);
}

// What follows the attention's own workspace.
struct SpanWorkspace {
  size_t tokens, units, tiles, group_units, group_tiles, ends, group_ends, group_ml, group_part, raw_ml, raw, group_raw_ml,
      group_raw, bytes;
};

SpanWorkspace span_layout(const dsa_ctx* ctx, long long Tq, int B, int groups, long long heads, long long kv_heads, int D) {
  const long long G = heads / kv_heads;
  size_t at = layout(ctx, D).bytes;
  auto take = [&](size_t bytes) {
    const size_t here = (at + 255) / 256 * 256;
    at = here + bytes;
    return here;
  };
  SpanWorkspace w = {};
  const size_t places = shape_of(ctx, Tq * G, B).places;
  w.tokens = take(Tq * sizeof(int4));
  w.units = take(places * 3 * sizeof(int4));
  w.tiles = take(places * sizeof(int));
  if (groups) {
    const size_t more = shape_of(ctx, Tq * G, groups).places;
    w.group_units = take(more * 3 * sizeof(int4));
    w.group_tiles = take(more * sizeof(int));
    w.ends = take(places * kv_heads * sizeof(int2));
    w.group_ends = take(more * kv_heads * sizeof(int2));
    // the first pass's pieces; the second's are where dsa_tree_attn has them
    const Workspace pieces = layout(ctx, D);
    w.group_ml = take(pieces.part - pieces.ml);
    w.group_part = take(pieces.bytes - pieces.part);
    const size_t rows = static_cast<size_t>(Tq) * heads;
    w.raw_ml = take(rows * sizeof(float2));
    w.raw = take(rows * D * sizeof(float));
    w.group_raw_ml = take(rows * sizeof(float2));
    w.group_raw = take(rows * D * sizeof(float));
  }
  w.bytes = at;
  return w;
}

}  // namespace at

size_t span_workspace(const dsa_ctx* ctx, int32_t Tq, int32_t B, int32_t groups, int32_t heads, int32_t kv_heads, int32_t head_dim) {
  return at::span_layout(ctx, Tq, B, groups, heads, kv_heads, head_dim).bytes;
}

dsa_status launch_span(dsa_ctx* ctx, const dsa_attn_args& p, const dsa_span& span, const int32_t* cu_groups,
                       const int32_t* shared, int32_t groups, cudaStream_t stream) {
  using namespace at;
  const SpanWorkspace w = span_layout(ctx, p.Tq, p.B, groups, p.heads, p.kv_heads, p.head_dim);
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  SpanArgs a = {};
  fill_args(ctx, p, a);
  a.slopes = span.slopes;
  a.fixed = -INFINITY;
  if (span.cap != 0.0) cap_args(p.scale, span.cap, a);
  a.tokens = reinterpret_cast<int4*>(ws + w.tokens);
  CUtensorMap tm = {};
  if (!cache_map(ctx, p, kTile, tm)) return DSA_ERR_CUDA;

  const long long rows = static_cast<long long>(p.Tq) * a.G;
  const Shape own = shape_of(ctx, rows, p.B), all = groups ? shape_of(ctx, rows, groups) : Shape{};
  SpanPlan plan = {};
  plan.first = span.first;
  plan.last = span.last;
  plan.window = span.window;
  plan.cu_groups = cu_groups;
  plan.shared = shared;
  plan.groups = groups;
  plan.tokens = reinterpret_cast<int4*>(ws + w.tokens);
  plan.units = reinterpret_cast<int4*>(ws + w.units);
  plan.tiles = reinterpret_cast<int*>(ws + w.tiles);
  plan.group_units = reinterpret_cast<int4*>(ws + w.group_units);
  plan.group_tiles = reinterpret_cast<int*>(ws + w.group_tiles);
  plan.n = own.places;
  plan.rows = own.rows;
  plan.group_n = all.places;
  plan.group_rows = all.rows;
  {
    LaunchScope scope(ctx, DSA_K_SPAN_PLAN, stream);
    const long long warps = static_cast<long long>(plan.n) + plan.group_n;
    if (launch_pdl(span_plan_kernel, dim3(static_cast<unsigned>((warps + 7) / 8)), dim3(256), 0, stream,
                   static_cast<const AttnArgs&>(a), plan) != cudaSuccess)
      return DSA_ERR_CUDA;
  }
  static constexpr RunSpan* kRun[4][3] = {{run_span_bf16, run_span_fp8, run_span_fp4},
                                          {run_span_cap_bf16, run_span_cap_fp8, run_span_cap_fp4},
                                          {run_span_bias_bf16, run_span_bias_fp8, run_span_bias_fp4},
                                          {run_span_wide_bf16, run_span_wide_fp8, run_span_wide_fp4}};
  const bool wide_cap = span.cap * 1.4426950408889634 > kCapOne;
  RunSpan* const run = kRun[wide_cap ? 3 : a.slopes ? 2 : a.cap2 != 0.f ? 1 : 0][p.fmt];
  a.units = plan.units;
  a.tiles = plan.tiles;
  a.units_n = plan.n;
  if (!groups) {
    const dsa_status st = run(ctx, own.form, p.head_dim, tm, a, own.grid, stream);
    if (st != DSA_OK) return st;
    LaunchScope scope(ctx, DSA_K_ATTN_JOIN, stream);
    // a row a warp, or, with so few units that they may have dozens of pieces, a
    // few a block (64 decode steps 363 us with 4 rows of blocks and 372 with 8; one
    // of 131072 keys and one kv head 43 and 32)
    const bool many = static_cast<long long>(own.places) * p.kv_heads * 16 < own.grid;
    const cudaError_t e = launch_pdl(p.head_dim == 128 ? join_kernel<128, SpanArgs> : join_kernel<64, SpanArgs>,
                                     dim3(own.grid, many ? 8 : own.rows / 8), dim3(256), 0, stream, a, own.grid, own.rows);
    return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
  }
  a.raw_mode = 2;
  a.ends = reinterpret_cast<int2*>(ws + w.ends);
  a.raw_ml = reinterpret_cast<float2*>(ws + w.raw_ml);
  a.raw = reinterpret_cast<float*>(ws + w.raw);
  SpanArgs b = a;
  b.raw_mode = 1;
  b.units = plan.group_units;
  b.tiles = plan.group_tiles;
  b.units_n = plan.group_n;
  b.ends = reinterpret_cast<int2*>(ws + w.group_ends);
  b.ml = reinterpret_cast<float2*>(ws + w.group_ml);
  b.part = reinterpret_cast<float*>(ws + w.group_part);
  b.raw_ml = reinterpret_cast<float2*>(ws + w.group_raw_ml);
  b.raw = reinterpret_cast<float*>(ws + w.group_raw);
  dsa_status st = run(ctx, all.form, p.head_dim, tm, b, all.grid, stream);
  if (st == DSA_OK) st = run(ctx, own.form, p.head_dim, tm, a, own.grid, stream);
  if (st != DSA_OK) return st;
  LaunchScope scope(ctx, DSA_K_ATTN_JOIN, stream);
  const RowsJoin join = {b, a, all.rows, own.rows, all.grid, own.grid};
  const cudaError_t e = launch_pdl(p.head_dim == 128 ? rows_join_kernel<128> : rows_join_kernel<64>,
                                   dim3(own.places, std::min(p.kv_heads, 32768), own.rows / 8), dim3(256), 0, stream, join);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
