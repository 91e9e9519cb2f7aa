// Attention of listed units over fp4 caches, caps too wide for one exponent: the kernel of attn.cuh, in
// a translation unit of its own so that they compile in parallel.
#include "attn.cuh"

namespace dsa {
namespace at {

dsa_status run_span_wide_fp4(dsa_ctx* ctx, int form, int D, const CUtensorMap& tm, const SpanArgs& a, int grid, cudaStream_t stream) {
  return run_fmt<DSA_FMT_FP4, kWideCap>(ctx, form, D, tm, a, grid, stream);
}

}  // namespace at
}  // namespace dsa
