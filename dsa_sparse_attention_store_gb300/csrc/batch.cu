// Page tables and slot maps of a step, from the lengths of its requests.
//
// Every block adds up all sequences' tokens, new pages and returned pages into
// shared memory, so that one launch does and no block waits for another; then
// the blocks divide the tokens, the new pages and the returned ones, and find
// each one's sequence by bisection there. The pool is never moved: the i-th page
// that is taken is entry count + returned - 1 - i of the free pages followed by
// the returned ones, and a returned one is found through the same sums. No entry
// that is read is written: pages are read from the free stack only where all
// returned ones are taken too, and then none is written to it; a row that is
// read for its returned pages gets no new ones.
//
// What bounds it: a step of 64 tokens one launch and the chain of loads lengths
// -> page -> slot, 3.2 us. 16384 sequences with a million tokens, of which a ninth
// end, 25.8 us (12.6 MB, 1.9 us at the copy rate): the sums over all sequences,
// which every block makes for itself (about 9), the bisections and dependent
// loads of a thread's tokens (8), and of the pages that come back (5). With a walk
// along 16 sequences for each token it took 57; with sums divided between the
// four blocks of a cluster 28, for a cluster's launch and barriers take as long.
#include <algorithm>

#include "internal.cuh"

namespace dsa {
namespace {

struct BatchPlanArgs : dsa_batch_args {
  unsigned int* status;
};

constexpr int kPage = 64;
constexpr int kMost = 0x7FFFFFFF;
// Sums that shared memory has room for: of a sequence each up to 16384, of a run
// of neighbours beyond.
constexpr int kSums = 16384;

struct Request {
  int old, n, pages, fresh, ended, keep;  // tokens there and to come; pages there, to take, to return; first page to return
  bool ends, ok;
};

__device__ __forceinline__ Request request(const BatchPlanArgs& a, int b) {
  Request x = {};
  // 64 max_pages and so all that is not refused is below 2^31
  const uint32_t o = a.old_lens[b], keep = a.own_from ? a.own_from[b] : 0, most = a.max_pages * kPage;
  const int n = a.new_lens[b];
  x.ends = n < 0;
  const uint32_t len = o + max(n, 0), pages = (o + kPage - 1) / kPage;
  x.ok = o <= most && len <= most && keep < 0x80000000u;
  if (!x.ok) return x;
  x.old = o;
  x.pages = pages;
  x.keep = keep;
  if (x.ends) {
    x.ended = max(0, x.pages - x.keep);
  } else {
    x.n = n;
    x.fresh = (len + kPage - 1) / kPage - pages;
  }
  return x;
}

struct Sums {
  long long tokens, fresh, ended;
  __device__ __forceinline__ void add(const Sums& x) {
    tokens += x.tokens;
    fresh += x.fresh;
    ended += x.ended;
  }
};

// over a warp's lanes, the own one included
__device__ __forceinline__ Sums scan(Sums x) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums y = {__shfl_up_sync(0xffffffffu, x.tokens, d), __shfl_up_sync(0xffffffffu, x.fresh, d),
                    __shfl_up_sync(0xffffffffu, x.ended, d)};
    if (static_cast<int>(threadIdx.x & 31) >= d) x.add(y);
  }
  return x;
}

__device__ __forceinline__ Sums shfl(const Sums& x, int from) {
  return {__shfl_sync(0xffffffffu, x.tokens, from), __shfl_sync(0xffffffffu, x.fresh, from), __shfl_sync(0xffffffffu, x.ended, from)};
}

__device__ __forceinline__ int clamp_sum(long long x) { return static_cast<int>(min(x, static_cast<long long>(kMost))); }

// per: sequences of a run; runs of them; own: neighbouring runs a thread adds
// up, an odd number, so that a warp's accesses fall into different banks. A
// thread has EACH neighbouring tokens: four look up their sequence and page once
// where they are the same.
template <int THREADS, int EACH>
__global__ void __launch_bounds__(THREADS) batch_plan_kernel(const BatchPlanArgs a, int per, int runs, int own) {
  extern __shared__ int s_sums[];  // of each run, then before it: tokens, new pages, returned pages
  __shared__ Sums s_warp[THREADS / 32];
  __shared__ int s_bad;
  int *const s_tokens = s_sums, *const s_fresh = s_sums + runs, *const s_ended = s_sums + 2 * runs;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, grid = gridDim.x, cta = blockIdx.x;
  if (tid == 0) s_bad = 0;
  pdl_wait();
  pdl_trigger();
  bool bad = false;
  if (per == 1) {
#pragma unroll 4
    for (int r = tid; r < runs; r += THREADS) {
      const Request x = request(a, r);
      s_tokens[r] = x.n;
      s_fresh[r] = x.fresh;
      s_ended[r] = x.ended;
      bad |= !x.ok;
    }
  } else {
    for (int r = tid; r < runs; r += THREADS) {
      long long t = 0, f = 0, e = 0;
      for (int b = r * per; b < min(a.B, r * per + per); ++b) {
        const Request x = request(a, b);
        t += x.n;
        f += x.fresh;
        e += x.ended;
        bad |= !x.ok;
      }
      s_tokens[r] = clamp_sum(t);
      s_fresh[r] = clamp_sum(f);
      s_ended[r] = clamp_sum(e);
    }
  }
  const int given = *a.free_count, count = min(max(given, 0), a.free_cap);
  __syncthreads();
  const int r0 = min(runs, tid * own), r1 = min(runs, r0 + own);
  // pages, below 2^25 of a sequence: in up to 17 runs of up to 4 sequences, or 33 of one
  long long sum_tokens = 0;
  uint32_t sum_fresh = 0, sum_ended = 0;
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    sum_tokens += s_tokens[r];
    sum_fresh += s_fresh[r];
    sum_ended += s_ended[r];
  }
  const Sums sum = {sum_tokens, sum_fresh, sum_ended}, inc = scan(sum);
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  Sums all = {0, 0, 0}, before = {inc.tokens - sum.tokens, inc.fresh - sum.fresh, inc.ended - sum.ended};
  if constexpr (THREADS == 1024) {  // a warp's sums a lane: one after another they take a microsecond more
    const Sums warps = scan(s_warp[lane]), x = shfl(warps, max(warp, 1) - 1);
    if (warp) before.add(x);
    all = shfl(warps, 31);
  } else {
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      const Sums x = s_warp[w];
      if (w < warp) before.add(x);
      all.add(x);
    }
  }
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    const int t = s_tokens[r], f = s_fresh[r], e = s_ended[r];
    s_tokens[r] = clamp_sum(before.tokens);
    s_fresh[r] = clamp_sum(before.fresh);
    s_ended[r] = clamp_sum(before.ended);
    before.tokens += t;
    before.fresh += f;
    before.ended += e;
  }
  __syncthreads();
  const long long pool = count + all.ended, left = pool - all.fresh;
  const int step = grid * THREADS, first = cta * THREADS + tid;

  for (int r = first; r < runs; r += step) {  // lengths
    long long t = s_tokens[r];
    for (int b = r * per; b < min(a.B, r * per + per); ++b) {
      const Request x = request(a, b);
      a.cu_q[b] = clamp_sum(t);
      a.seq_lens[b] = x.ok && !x.ends ? x.old + x.n : 0;
      t += x.n;
    }
  }
  if (first == 0) {
    a.cu_q[a.B] = clamp_sum(all.tokens);
    *a.free_left = static_cast<int>(min(max(left, 0LL), static_cast<long long>(a.free_cap)));
    bad |= given != count || left < 0 || left > a.free_cap || all.tokens > a.T;
  }

  // the last run with sums[run] <= i
  auto run_of = [&](const int* sums, int i) {
    int lo = 0, n = runs;
    while (n > 1) {
      const int half = n / 2;
      if (sums[lo + half] <= i) lo += half;
      n -= half;
    }
    return lo;
  };
  // returned page j
  auto returned = [&](int j) -> int {
    const int run = run_of(s_ended, j);
    j -= s_ended[run];
    for (int b = run * per; b < min(a.B, run * per + per); ++b) {
      const Request x = request(a, b);
      if (j < x.ended) return a.page_table[static_cast<long long>(b) * a.max_pages + x.keep + j];
      j -= x.ended;
    }
    return -1;
  };
  // the i-th page that is taken
  auto taken = [&](long long i) -> int {
    const long long v = pool - 1 - i;
    return v < 0 ? -1 : v < count ? a.free_pages[v] : returned(clamp_sum(v - count));
  };
  const long long tokens = min(all.tokens, static_cast<long long>(a.T));
  const bool wide = EACH == 4 && !((reinterpret_cast<uintptr_t>(a.seq_id) | reinterpret_cast<uintptr_t>(a.cache_pos) |
                                     reinterpret_cast<uintptr_t>(a.slots)) & 15);
  for (long long t0 = static_cast<long long>(first) * EACH; t0 < a.T; t0 += static_cast<long long>(step) * EACH) {
    int seq[EACH], pos[EACH], slot[EACH];
    Request x = {};
    long long at = 0, end = -1, fresh = 0;  // the sequence's first token and one past its last, new pages before it
    int b = 0, p = -1, page = -1;           // the sequence, the last token's place in its row, its page
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      const long long t = t0 + k;
      seq[k] = pos[k] = slot[k] = -1;
      if (t >= tokens) continue;
      if (t >= end) {
        const int run = run_of(s_tokens, static_cast<int>(t));
        at = s_tokens[run];
        fresh = s_fresh[run];
        b = run * per;
        x = request(a, b);
        while (t >= at + x.n) {
          at += x.n;
          fresh += x.fresh;
          x = request(a, ++b);
        }
        end = at + x.n;
        p = -1;
      }
      seq[k] = b;
      pos[k] = x.old + static_cast<int>(t - at);
      if (pos[k] / kPage != p) {
        p = pos[k] / kPage;
        page = p < x.pages ? a.page_table[static_cast<long long>(b) * a.max_pages + p] : taken(fresh + p - x.pages);
      }
      const bool there = page >= 0 && page < a.num_pages;
      bad |= !there;
      if (there) slot[k] = page * kPage + pos[k] % kPage;
    }
    if (wide && t0 + EACH <= a.T) {
      if constexpr (EACH == 4) {
        *reinterpret_cast<int4*>(a.seq_id + t0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
        *reinterpret_cast<int4*>(a.cache_pos + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        if (a.slots) *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < EACH; ++k)
        if (t0 + k < a.T) {
          a.seq_id[t0 + k] = seq[k];
          a.cache_pos[t0 + k] = pos[k];
          if (a.slots) a.slots[t0 + k] = slot[k];
        }
    }
  }
  const long long fresh_pages = min(all.fresh, static_cast<long long>(kMost));
  for (long long i = first; i < fresh_pages; i += step) {
    const int run = run_of(s_fresh, static_cast<int>(i));
    long long at = s_fresh[run];
    int seq = run * per;
    Request x = request(a, seq);
    while (i >= at + x.fresh) {
      at += x.fresh;
      x = request(a, ++seq);
    }
    a.page_table[static_cast<long long>(seq) * a.max_pages + x.pages + (i - at)] = taken(i);
  }
  // pages that came back and were not taken again
  for (long long j = first; j < min(left, static_cast<long long>(a.free_cap)) - count; j += step)
    a.free_pages[count + j] = returned(static_cast<int>(j));
  if (bad) s_bad = 1;
  __syncthreads();
  if (tid == 0 && s_bad) atomicOr(a.status, DSA_DEV_BOUNDS);
}

constexpr int kSmallThreads = 128, kMidThreads = 256, kThreads = 1024;

template <int THREADS, int EACH>
cudaError_t launch(const BatchPlanArgs& a, int grid, cudaStream_t stream) {
  const int per = (a.B + kSums - 1) / kSums, runs = (a.B + per - 1) / per, own = ((runs + THREADS - 1) / THREADS) | 1;
  return launch_pdl(batch_plan_kernel<THREADS, EACH>, dim3(grid), dim3(THREADS), 12 * static_cast<size_t>(runs), stream, a, per,
                    runs, own);
}

}  // namespace

dsa_status launch_batch_plan(dsa_ctx* ctx, const dsa_batch_args& args, cudaStream_t stream) {
  BatchPlanArgs a = {args, ctx->status};
  if (!ctx->batch_ready) {
    for (auto kern : {batch_plan_kernel<kMidThreads, 1>, batch_plan_kernel<kThreads, 1>, batch_plan_kernel<kThreads, 4>})
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 12 * kSums) != cudaSuccess) return DSA_ERR_CUDA;
    ctx->batch_ready = 1;
  }
  LaunchScope scope(ctx, DSA_K_BATCH_PLAN, stream);
  const int most = std::max(a.T, a.B);
  // One small block for a decode step: fewer warps to meet. Blocks of 256 while
  // they have few sums and tokens a thread (1000 sequences of a token each 6.5 us,
  // in blocks of 1024 7.5; 100 of 1000 tokens 6.0 and 9.2; but 4000 of 64 tokens
  // 15.9 and 14.0, 16384 of one 15.7 and 14.4). Beyond, four tokens a thread
  // where sequences have as many (in the smaller blocks that takes 1 to 3 us more).
  // A block on each SM, or as many as have two sequences or tokens a thread, or
  // eight pages that may come back.
  const long long pages = static_cast<long long>(a.B) * a.max_pages;
  auto blocks = [&](int threads) {
    return static_cast<int>(std::min(std::max({1LL, (most + 2LL * threads - 1) / (2 * threads), pages / (8 * threads)}),
                                     static_cast<long long>(ctx->num_sms)));
  };
  const bool mid = a.T <= 131072 && a.B <= 8192, four = a.T / 8 >= a.B && a.T >= 16384;
  const cudaError_t e = most <= 2 * kSmallThreads ? launch<kSmallThreads, 1>(a, blocks(kSmallThreads), stream)
                        : mid                     ? launch<kMidThreads, 1>(a, blocks(kMidThreads), stream)
                        : four                    ? launch<kThreads, 4>(a, blocks(kThreads), stream)
                                                  : launch<kThreads, 1>(a, blocks(kThreads), stream);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
