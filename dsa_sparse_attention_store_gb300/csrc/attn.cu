// Attention: the bf16 kernels, the join of divided units, and the launch.
// The kernel is in attn.cuh.
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
constexpr int kFew = 16;

template <int D>
__global__ void __launch_bounds__(256) join_kernel(const AttnArgs a, int grid, int rows) {
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
      a.lse[tok * a.kv_heads * a.G + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
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
  if (n <= kFew) {
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

dsa_status run_bf16(dsa_ctx* ctx, int form, int D, const CUtensorMap& tm, const AttnArgs& a, int grid, cudaStream_t stream) {
  return run_fmt<DSA_FMT_BF16>(ctx, form, D, tm, a, grid, stream);
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Two pieces a CTA, 256 rows on each SM whatever the form.
struct Workspace {
  size_t ml, part, bytes;
};

Workspace layout(const dsa_ctx* ctx, int D) {
  const size_t rows = 2 * 256 * static_cast<size_t>(ctx->num_sms);
  Workspace w;
  w.ml = (4 * static_cast<size_t>(ctx->num_sms) * sizeof(int4) + 255) / 256 * 256;
  w.part = w.ml + rows * sizeof(float2);
  w.bytes = w.part + rows * D * sizeof(float);
  return w;
}

}  // namespace at

size_t attn_workspace(const dsa_ctx* ctx, int32_t head_dim) { return at::layout(ctx, head_dim).bytes; }

dsa_status launch_attn(dsa_ctx* ctx, const dsa_attn_args& p, const int32_t* sel, int32_t k, cudaStream_t stream) {
  using namespace at;
  const Workspace w = layout(ctx, p.head_dim);
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
  AttnArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(p.q);
  a.out = static_cast<__nv_bfloat16*>(p.out);
  a.lse = p.lse;
  a.qt = p.q_stride_t;
  a.qh = p.q_stride_h;
  a.ot = p.out_stride_t;
  a.oh = p.out_stride_h;
  a.cache = static_cast<const uint8_t*>(p.cache);
  a.page_table = p.page_table;
  a.seq_lens = p.seq_lens;
  a.cu_q = p.cu_q;
  a.sel = sel;
  a.mask = p.mask;
  a.status = ctx->status;
  a.meta = reinterpret_cast<int4*>(ws);
  a.ml = reinterpret_cast<float2*>(ws + w.ml);
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.scale2 = static_cast<float>(p.scale * 1.4426950408889634);
  a.B = p.B;
  a.Tq = p.Tq;
  a.max_pages = p.max_pages;
  a.num_pages = p.num_pages;
  a.kv_heads = p.kv_heads;
  a.G = p.heads / p.kv_heads;
  a.k = k;
  a.mask_words = p.mask ? p.mask_words : 0;
  a.slots = ctx->slot_output;
  CUtensorMap tm = {};
  if (p.fmt == DSA_FMT_BF16) {  // the cache as rows of D elements; a page's K or V of one head is 64 of them
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.head_dim),
                                static_cast<cuuint64_t>(p.num_pages) * p.kv_heads * 2 * kTile};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.head_dim) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(sel ? 1 : kTile)};  // a selection gathers rows
    const cuuint32_t estr[2] = {1, 1};
    if (reinterpret_cast<EncodeFn>(ctx->encode_tiled)(
            &tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p.cache), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return DSA_ERR_CUDA;
  }
  // the wide form where the sequences' rows fill more than one 128-row unit on
  // average: 16 sequences of 4509 to 10498 tokens, 8 kv heads, bf16 (fp8), take
  // with 128 rows 113.7 (135.5) us in the wide form and 113.6 (108.7) in the
  // other, with 160 rows 130.2 (154.1) and 168.5 (177.6), with 512 250.2 (299.7)
  // and 318.9 (347.0)
  const bool wide = static_cast<long long>(p.Tq) * a.G > 128LL * p.B;
  // the few-row forms up to 32 rows: 64 sequences of 2048 to 16384 tokens, 8 kv
  // heads, bf16 (fp8), take with 8 rows 368 (350) us in them and 385 (356) in
  // the 128-row form, with 32 rows 375 (355) and 389 (363), and with 64 rows,
  // which read the cache twice there, 729 (682) and 399 (395). Selections, 8 kv
  // heads, G 8, D 128: 2048 of 512 keys in bf16 575 and 616; 512 of 2048 keys in
  // fp8 (fp4) 804 (738) and 824 (741), 8192 of 128 keys 1051 (949) and 1177
  // (1099), but 2048 of 512 keys 874 (809) and 863 (772), 3495 of 300 keys 1047
  // (967) and 979 (882). In fp8 and fp4 the 128-row form is ahead for units of 5
  // to 8 tiles alone (and not for D 64 in fp4): the rule does not follow that dip
  const bool few = sel ? a.G <= kFewRows : static_cast<long long>(p.Tq) * a.G <= static_cast<long long>(kFewRows) * p.B;
  const int form = sel ? (few ? kSparseFew : kSparse) : wide ? kWide : few ? kTreeFew : kTree;
  const int grid = form == kWide ? ctx->num_sms : 2 * ctx->num_sms, rows = form == kWide ? 256 : few ? kFewRows : 128;
  const auto run = p.fmt == DSA_FMT_BF16 ? run_bf16 : p.fmt == DSA_FMT_FP8 ? run_fp8 : run_fp4;
  const dsa_status st = run(ctx, form, p.head_dim, tm, a, grid, stream);
  if (st != DSA_OK) return st;
  LaunchScope scope(ctx, DSA_K_ATTN_JOIN, stream);
  const cudaError_t e = launch_pdl(p.head_dim == 128 ? join_kernel<128> : join_kernel<64>, dim3(grid, 8), dim3(256), 0,
                                   stream, a, grid, rows);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
