// Attention: the bf16 kernels and the launch. The kernel is in attn.cuh, the
// join of divided units in attn_join.cuh.
#include "attn_join.cuh"

namespace dsa {
namespace at {

dsa_status run_bf16(dsa_ctx* ctx, int form, int D, const CUtensorMap& tm, const AttnArgs& a, int grid, cudaStream_t stream) {
  return run_fmt<DSA_FMT_BF16>(ctx, form, D, tm, a, grid, stream);
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Workspace layout(const dsa_ctx* ctx, int D) {
  const size_t rows = 2 * 256 * static_cast<size_t>(ctx->num_sms);
  Workspace w;
  w.ml = (4 * static_cast<size_t>(ctx->num_sms) * sizeof(int4) + 255) / 256 * 256;
  w.part = w.ml + rows * sizeof(float2);
  w.bytes = w.part + rows * D * sizeof(float);
  return w;
}

bool cache_map(const dsa_ctx* ctx, const dsa_attn_args& p, int box_rows, CUtensorMap& tm) {
  if (p.fmt != DSA_FMT_BF16) return true;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.head_dim),
                              static_cast<cuuint64_t>(p.num_pages) * p.kv_heads * 2 * kTile};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.head_dim) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return reinterpret_cast<EncodeFn>(ctx->encode_tiled)(
             &tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p.cache), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

void fill_args(const dsa_ctx* ctx, const dsa_attn_args& p, AttnArgs& a) {
  const Workspace w = layout(ctx, p.head_dim);
  uint8_t* ws = static_cast<uint8_t*>(p.workspace);
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
  a.mask_words = p.mask ? p.mask_words : 0;
}

}  // namespace at

size_t attn_workspace(const dsa_ctx* ctx, int32_t head_dim) { return at::layout(ctx, head_dim).bytes; }

dsa_status launch_attn(dsa_ctx* ctx, const dsa_attn_args& p, const int32_t* sel, int32_t k, cudaStream_t stream) {
  using namespace at;
  AttnArgs a = {};
  fill_args(ctx, p, a);
  a.sel = sel;
  a.k = k;
  a.slots = ctx->slot_output;
  CUtensorMap tm = {};
  if (!cache_map(ctx, p, sel ? 1 : kTile, tm)) return DSA_ERR_CUDA;  // a selection gathers rows
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
  const cudaError_t e = launch_pdl(p.head_dim == 128 ? join_kernel<128, AttnArgs> : join_kernel<64, AttnArgs>, dim3(grid, 8), dim3(256), 0,
                                   stream, a, grid, rows);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
