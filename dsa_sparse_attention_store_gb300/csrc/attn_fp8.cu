// Attention over fp8 caches: the kernel of attn.cuh, in a translation unit of
// its own so that the formats compile in parallel.
#include "attn.cuh"

namespace dsa {
namespace at {

dsa_status run_fp8(dsa_ctx* ctx, int form, int D, const CUtensorMap& tm, const AttnArgs& a, int grid, cudaStream_t stream) {
  return run_fmt<DSA_FMT_FP8>(ctx, form, D, tm, a, grid, stream);
}

}  // namespace at
}  // namespace dsa
