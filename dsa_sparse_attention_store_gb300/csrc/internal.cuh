// Internal declarations shared by the library's translation units.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

#include "../../include/dsaidx.h"

// device status word bits
#define DSA_DEV_BOUNDS 1u
#define DSA_DEV_TIMEOUT 2u

struct dsa_prof_rec {
  int kind;
  cudaEvent_t ev0, ev1;
};

struct dsa_ctx {
  int device;
  int num_sms;
  float theta;
  float eps;
  int max_pos;
  // RoPE (cos, sin) in fp32, [max_pos][32] float4, lane-interleaved: float4
  // 8v + j of a row holds pairs 8j + 2v and 8j + 2v + 1 (j < 8, v < 4)
  float4* rope;
  int hadamard;          // store keys rotated by the 128-point Walsh-Hadamard transform
  int slot_output;       // top-k returns cache slots instead of positions
  float* gamma;          // [128]
  unsigned int* status;  // device status word
  void* encode_tiled;    // cuTensorMapEncodeTiled entry point
  uint64_t attn_ready;   // attention kernels whose shared memory limit is raised
  // kernel timing (dsa_profile_*)
  int prof_on;
  int prof_n;                    // records in use
  dsa_prof_rec* prof;            // kProfCap records, events created on enable
  long long launches[DSA_K_ALL];
};

namespace dsa {
constexpr int kProfCap = 8192;

// Every call that enqueues work first checks that the calling thread's
// current device is the context's: the kernels launch on the current device
// but read the context's device memory (table, gamma, status word), so a
// call made with another device current is rejected before anything is
// enqueued. Returns DSA_ERR_CUDA when no device can be queried.
inline dsa_status check_device(const dsa_ctx* ctx) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return DSA_ERR_CUDA;
  return dev == ctx->device ? DSA_OK : DSA_ERR_INVALID_ARG;
}
// Record the start/end of one kernel launch of kind `kind` on `stream`.
struct LaunchScope {
  dsa_ctx* ctx;
  int kind;
  dsa_prof_rec* rec;
  cudaStream_t stream;
  LaunchScope(dsa_ctx* c, int k, cudaStream_t s) : ctx(c), kind(k), rec(nullptr), stream(s) {
    ctx->launches[kind] += 1;
    if (ctx->prof_on && ctx->prof_n < kProfCap) {
      rec = &ctx->prof[ctx->prof_n++];
      rec->kind = kind;
      cudaEventRecord(rec->ev0, stream);
    }
  }
  ~LaunchScope() {
    if (rec) cudaEventRecord(rec->ev1, stream);
  }
};

// Launch with programmatic dependent launch allowed: the kernel may start
// while the previous kernel on the stream is still running, so every kernel
// launched this way executes griddepcontrol.wait before it reads global
// memory that a predecessor may write.
template <typename... Kargs, typename... Args>
cudaError_t launch_pdl(void (*kern)(Kargs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
}  // namespace dsa

namespace dsa {

dsa_status launch_store(dsa_ctx* ctx, const void* k_raw, const int32_t* pos, const int32_t* seq,
                        const int32_t* page_table, int32_t T, int32_t B, int32_t max_pages,
                        void* cache, int32_t num_pages, dsa_fmt fmt, cudaStream_t stream);

size_t topk_workspace(const dsa_ctx* ctx, int32_t Tq, int32_t B, int32_t k, dsa_fmt fmt);
int max_sequences();  // largest B dsa_index_topk accepts

dsa_status launch_topk(dsa_ctx* ctx, const void* q, const float* head_w, const void* cache,
                       int32_t num_pages, dsa_fmt fmt, const int32_t* page_table,
                       int32_t max_pages, const int32_t* seq_lens, const int32_t* cu_q,
                       int32_t B, int32_t Tq, int32_t causal, int32_t k, int32_t* out_idx,
                       float* out_score, void* workspace, size_t ws_bytes, cudaStream_t stream);

dsa_status rope_create(dsa_ctx* ctx, dsa_rope** out, const dsa_rope_desc& desc);

dsa_status launch_rope(dsa_ctx* ctx, const dsa_rope* rope, const void* x, void* y, dsa_dtype dtype,
                       const int32_t* pos, int32_t T, int32_t H, int32_t D, int32_t start, long long xt,
                       long long xh, long long yt, long long yh, int32_t inverse, cudaStream_t stream);

size_t kv_page_bytes(int32_t kv_heads, int32_t head_dim, dsa_fmt fmt);

dsa_status launch_kv_store(dsa_ctx* ctx, const void* k, const void* v, long long kt, long long kh, long long vt,
                           long long vh, const int32_t* cache_pos, const int32_t* seq_id,
                           const int32_t* page_table, int32_t T, int32_t B, int32_t max_pages, int32_t kv_heads,
                           int32_t head_dim, void* cache, int32_t num_pages, dsa_fmt fmt, const dsa_rope* rope,
                           const int32_t* rope_pos, int32_t start, cudaStream_t stream);

dsa_status launch_kv_load(dsa_ctx* ctx, const void* cache, int32_t num_pages, dsa_fmt fmt, int32_t kv_heads,
                          int32_t head_dim, const int32_t* cache_pos, const int32_t* seq_id,
                          const int32_t* page_table, int32_t T, int32_t B, int32_t max_pages, void* k, void* v,
                          long long kt, long long kh, long long vt, long long vh, cudaStream_t stream);

size_t attn_workspace(const dsa_ctx* ctx, int32_t head_dim);

// sel NULL: the tree form
dsa_status launch_attn(dsa_ctx* ctx, const dsa_attn_args& args, const int32_t* sel, int32_t k, cudaStream_t stream);

}  // namespace dsa
