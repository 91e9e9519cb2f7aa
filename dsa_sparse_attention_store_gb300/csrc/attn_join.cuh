// The join of units that the cuts between CTAs divided (attn.cuh).
#pragma once
#include "attn.cuh"

namespace dsa {
namespace at {

// Joins the pieces of a unit that the cuts divided: the CTA whose range the
// unit starts in holds the first piece (its tail), the CTAs after it the
// others (their heads) up to the one that marks the unit's end. Each block
// takes the unit that starts in CTA blockIdx.x, if any, and every
// gridDim.y-th row of it. Pieces are added in CTA order, so the result does
// not depend on timing.
//
// Few pieces (the usual case): a warp per row. Many (a long context and few
// rows): the block's warps share a row's pieces.
// 20 pieces of 256 rows (32 sequences behind 131072 tokens) took 83 us by the
// block and 15 by warps.
template <class Args>
constexpr int kFew = std::is_same_v<Args, SpanArgs> ? 64 : 16;

template <int D, class Args>
__global__ void __launch_bounds__(256) join_kernel(const Args a, int grid, int rows) {
  constexpr int E = D / 32;  // dimensions a lane holds
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int4 m0 = a.meta[2 * c];
  if (!m0.x) return;
  const int4 m1 = a.meta[2 * c + 1];
  __shared__ int s_end;
  __shared__ float s_o[8][D];
  __shared__ float s_l[8];
  if (tid == 0) s_end = grid - 1;
  __syncthreads();
  for (int i = c + 1 + tid; i < grid; i += 256) {
    if (a.meta[2 * i].z) {
      atomicMin(&s_end, i);
      break;
    }
  }
  __syncthreads();
  const int n = s_end - c + 1;  // pieces
  auto slot = [&](int p) -> long long { return p == 0 ? 2 * c + 1 : 2 * (c + p); };
  auto finish = [&](int row, float m, float l, const float (&o)[E]) {
    const int r = m1.x + row;
    const long long tok = m1.y + r / a.G;
    const int head = m1.z * a.G + r % a.G;
    float top = m;  // for lse
    if constexpr (std::is_same_v<Args, SpanArgs>) {
      if (a.slopes && a.lse && lane == 0) top -= a.slopes[head] * 1.4426950408889634f * away(token_at(a, tok));
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const __nv_bfloat162 v =
          l == 0.f ? __floats2bfloat162_rn(0.f, 0.f) : __floats2bfloat162_rn(o[2 * i] * inv, o[2 * i + 1] * inv);
      memcpy(&w[i], &v, 4);
    }
    __nv_bfloat16* dst = a.out + tok * a.ot + head * a.oh + lane * E;
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(dst) = w[0];
    if (a.lse && lane == 0)
      a.lse[tok * a.kv_heads * a.G + head] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
  };
  auto add = [&](int p, int row, float w, float (&o)[E]) {
    const float* src = a.part + (slot(p) * rows + row) * D + lane * E;
    if constexpr (E == 4) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
      o[0] = fmaf(v.x, w, o[0]);
      o[1] = fmaf(v.y, w, o[1]);
      o[2] = fmaf(v.z, w, o[2]);
      o[3] = fmaf(v.w, w, o[3]);
    } else {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
      o[0] = fmaf(v.x, w, o[0]);
      o[1] = fmaf(v.y, w, o[1]);
    }
  };
  // the largest maximum over the pieces; a piece without a visible key has -inf and a weight of 0
  auto top = [&](int row) {
    float m = -INFINITY;
    for (int p = lane; p < n; p += 32) m = fmaxf(m, __ldcg(a.ml + slot(p) * rows + row).x);
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    return m;
  };
  // a piece's sums hold weights of up to 2^8: denormal factors count
  auto weight = [&](float2 v, float m) { return v.x == -INFINITY ? 0.f : v.x == m ? 1.f : ex2_denorm(v.x - m); };
  if (n <= kFew<Args>) {
    for (int row = blockIdx.y * 8 + warp; row < m0.w; row += gridDim.y * 8) {
      const float m = top(row);
      float o[E] = {}, l = 0.f;
#pragma unroll 4
      for (int p = 0; p < n; ++p) {
        const float2 v = __ldcg(a.ml + slot(p) * rows + row);
        const float w = weight(v, m);
        l = fmaf(v.y, w, l);
        add(p, row, w, o);
      }
      finish(row, m, l, o);
    }
  } else {
    for (int row = blockIdx.y; row < m0.w; row += gridDim.y) {
      const float m = top(row);
      float o[E] = {}, l = 0.f;
#pragma unroll 4
      for (int p = warp; p < n; p += 8) {
        const float2 v = __ldcg(a.ml + slot(p) * rows + row);
        const float w = weight(v, m);
        l = fmaf(v.y, w, l);
        add(p, row, w, o);
      }
#pragma unroll
      for (int i = 0; i < E; ++i) s_o[warp][lane * E + i] = o[i];
      if (lane == 0) s_l[warp] = l;
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int w = 1; w < 8; ++w) {
          l += s_l[w];
#pragma unroll
          for (int i = 0; i < E; ++i) o[i] += s_o[w][lane * E + i];
        }
        finish(row, m, l, o);
      }
      __syncthreads();
    }
  }
}

}  // namespace at
}  // namespace dsa
