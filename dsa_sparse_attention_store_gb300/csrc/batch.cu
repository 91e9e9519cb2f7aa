// Page tables and slot maps of a step, from the lengths of its requests.
//
// Every block adds up all sequences' tokens, new pages and returned pages (a
// run of sequences a thread, then a scan over the threads), so that one launch
// does and no block waits for another; then the blocks divide the tokens and
// the returned pages. The pool is never moved: the i-th page that is taken is
// entry count + returned - 1 - i of the free pages followed by the returned
// ones, and the returned ones are found through the same sums. No entry that is
// read is written: pages are read from the free stack only where all returned
// ones are taken too, and then none is written to it; a row that is read for
// its returned pages gets no new ones.
//
// What bounds it: one launch and the chain lengths -> sums -> token for small
// steps, 12 bytes a token for large ones.
#include "internal.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 1024;
constexpr int kPage = 64;

struct Request {
  int old, n, pages, fresh, ended, keep;  // tokens there and to come; pages there, to take, to return; first page to return
  bool ends, ok;
};

__device__ __forceinline__ Request request(const BatchPlanArgs& a, int b) {
  Request x = {};
  const int o = a.old_lens[b], n = a.new_lens[b], keep = a.own_from ? a.own_from[b] : 0;
  const long long most = static_cast<long long>(a.max_pages) * kPage;
  x.ok = o >= 0 && keep >= 0 && static_cast<long long>(o) + max(n, 0) <= most;
  x.ends = n < 0;
  if (!x.ok) return x;
  x.old = o;
  x.pages = (o + kPage - 1) / kPage;
  x.keep = keep;
  if (x.ends) {
    x.ended = max(0, x.pages - keep);
  } else {
    x.n = n;
    x.fresh = static_cast<int>((static_cast<long long>(o) + n + kPage - 1) / kPage) - x.pages;
  }
  return x;
}

struct Sums {
  long long tokens, fresh, ended;
};

__global__ void __launch_bounds__(kThreads) batch_plan_kernel(const BatchPlanArgs a) {
  __shared__ Sums s_before[kThreads + 1];  // of a thread's run of sequences: what came before it
  __shared__ Sums s_warp[32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, grid = gridDim.x, cta = blockIdx.x;
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  Sums sum = {0, 0, 0};
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const Request x = request(a, b);
    sum.tokens += x.n;
    sum.fresh += x.fresh;
    sum.ended += x.ended;
    bad |= !x.ok;
  }
  Sums inc = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, inc.tokens, d), f = __shfl_up_sync(0xffffffffu, inc.fresh, d),
                    e = __shfl_up_sync(0xffffffffu, inc.ended, d);
    if (lane >= d) {
      inc.tokens += t;
      inc.fresh += f;
      inc.ended += e;
    }
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  Sums before = {0, 0, 0};
  for (int w = 0; w < warp; ++w) {
    before.tokens += s_warp[w].tokens;
    before.fresh += s_warp[w].fresh;
    before.ended += s_warp[w].ended;
  }
  before.tokens += inc.tokens - sum.tokens;
  before.fresh += inc.fresh - sum.fresh;
  before.ended += inc.ended - sum.ended;
  s_before[tid] = before;
  if (tid == kThreads - 1) s_before[kThreads] = Sums{before.tokens + sum.tokens, before.fresh + sum.fresh, before.ended + sum.ended};
  __syncthreads();
  const Sums all = s_before[kThreads];
  const int given = *a.free_count, count = min(max(given, 0), a.cap);
  const long long pool = count + all.ended, left = pool - all.fresh;

  // lengths, by this block's share of the threads' runs
  if (tid % grid == cta) {
    long long t = before.tokens;
    for (int b = b0; b < b1; ++b) {
      const Request x = request(a, b);
      a.cu_q[b] = static_cast<int>(min(t, 0x7FFFFFFFLL));
      a.lens[b] = x.ok && !x.ends ? x.old + x.n : 0;
      t += x.n;
    }
  }
  if (cta == 0 && tid == 0) {
    a.cu_q[a.B] = static_cast<int>(min(all.tokens, 0x7FFFFFFFLL));
    *a.left = static_cast<int>(min(max(left, 0LL), static_cast<long long>(a.cap)));
    bad |= given != count || left < 0 || left > a.cap || all.tokens > a.T;
  }

  // the run of sequences in which sum `f` of those before passes i
  auto run_of = [&](auto f, long long i) {
    int lo = 0, hi = kThreads;
    while (hi - lo > 1) {
      const int m = (lo + hi) / 2;
      if (f(s_before[m]) <= i)
        lo = m;
      else
        hi = m;
    }
    return lo;
  };
  // returned page j
  auto returned = [&](long long j) -> int {
    const int run = run_of([](const Sums& s) { return s.ended; }, j);
    j -= s_before[run].ended;
    for (int b = run * per; b < min(a.B, run * per + per); ++b) {
      const Request x = request(a, b);
      if (j < x.ended) return a.table[static_cast<long long>(b) * a.max_pages + x.keep + j];
      j -= x.ended;
    }
    return -1;
  };
  // the i-th page that is taken
  auto taken = [&](long long i) -> int {
    const long long v = pool - 1 - i;
    return v < 0 ? -1 : v < count ? a.stack[v] : returned(v - count);
  };
  const long long step = static_cast<long long>(grid) * kThreads;
  for (long long t = static_cast<long long>(cta) * kThreads + tid; t < max(all.tokens, static_cast<long long>(a.T)); t += step) {
    int seq = -1, pos = -1, slot = -1;
    if (t < all.tokens) {
      const int run = run_of([](const Sums& s) { return s.tokens; }, t);
      Sums s = s_before[run];
      seq = run * per;
      Request x = request(a, seq);
      while (t >= s.tokens + x.n) {
        s.tokens += x.n;
        s.fresh += x.fresh;
        x = request(a, ++seq);
      }
      pos = x.old + static_cast<int>(t - s.tokens);
      const int p = pos / kPage;
      int32_t* const entry = a.table + static_cast<long long>(seq) * a.max_pages + p;
      const int page = p < x.pages ? *entry : taken(s.fresh + p - x.pages);
      const bool there = page >= 0 && page < a.num_pages;
      if (p >= x.pages && pos % kPage == 0) *entry = page;  // a new page's first token
      bad |= !there;
      if (there) slot = page * kPage + pos % kPage;
    }
    if (t < a.T) {
      a.seq[t] = seq;
      a.pos[t] = pos;
      if (a.slots) a.slots[t] = slot;
    }
  }
  // pages that came back and were not taken again
  for (long long j = static_cast<long long>(cta) * kThreads + tid; j < min(left, static_cast<long long>(a.cap)) - count; j += step)
    a.stack[count + j] = returned(j);
  if (bad) atomicOr(a.status, DSA_DEV_BOUNDS);
}

}  // namespace

dsa_status launch_batch_plan(dsa_ctx* ctx, const BatchPlanArgs& a, cudaStream_t stream) {
  LaunchScope scope(ctx, DSA_K_BATCH_PLAN, stream);
  const int most = (max(a.T, a.B) + 2 * kThreads - 1) / (2 * kThreads);
  const int grid = max(1, min(most, ctx->num_sms));
  return launch_pdl(batch_plan_kernel, dim3(grid), dim3(kThreads), 0, stream, a) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
