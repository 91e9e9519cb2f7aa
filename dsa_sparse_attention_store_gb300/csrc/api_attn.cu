// C ABI of the operators that follow the indexer (rotary positions, K/V
// cache, attention): argument validation and dispatch to their launchers.
#include <cmath>

#include "internal.cuh"
#include "rope.cuh"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

cudaStream_t as_stream(dsa_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

bool known(dsa_fmt f) { return f == DSA_FMT_BF16 || f == DSA_FMT_FP8 || f == DSA_FMT_FP4; }

bool positive(double v) { return v > 0.0 && std::isfinite(v); }

// Whether two of the n0 x n1 rows at element strides s0 and s1 share one of
// their `width` elements: then the kernel's threads would write it in any
// order. For outputs; inputs may be expanded.
bool rows_meet(long long n0, int64_t s0, long long n1, int64_t s1, long long width) {
  using Wide = __int128;  // products of sizes and strides
  const Wide t0 = s0 < 0 ? -static_cast<Wide>(s0) : s0, t1 = s1 < 0 ? -static_cast<Wide>(s1) : s1;
  if ((n0 > 1 && t0 < width) || (n1 > 1 && t1 < width)) return true;
  if (n0 <= 1 || n1 <= 1) return false;
  const Wide a = t0 < t1 ? t0 : t1, b = t0 < t1 ? t1 : t0;  // the closer rows and the farther ones
  const Wide na = t0 < t1 ? n0 : n1, nb = t0 < t1 ? n1 : n0;
  const Wide reach = (na - 1) * a + width;  // b at least that: none can meet, all usual layouts
  for (Wide d = 1; d < nb && d * b < reach; ++d) {
    const Wide e = d * b / a, off = d * b - e * a;  // the closest rows below and above
    if ((e < na && off < width) || (e + 1 < na && a - off < width) || (e >= na && d * b - (na - 1) * a < width)) return true;
  }
  return false;
}

// what the two directions of the cache share
dsa_status check_kv(const void* cache, int32_t num_pages, dsa_fmt fmt, int32_t kv_heads, int32_t head_dim, int32_t T,
                    int32_t B, int32_t max_pages, const void* k, const void* v, const int64_t (&strides)[4],
                    const int32_t* cache_pos, const int32_t* seq_id, const int32_t* page_table) {
  if (!known(fmt) || (head_dim != 64 && head_dim != 128)) return DSA_ERR_UNSUPPORTED;
  if (T < 0 || B <= 0 || max_pages <= 0 || num_pages <= 0 || kv_heads <= 0) return DSA_ERR_INVALID_ARG;
  if (T == 0) return DSA_OK;
  if (!k || !v || !cache || !cache_pos || !seq_id || !page_table) return DSA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cache, 256) || !aligned(cache_pos, 4) || !aligned(seq_id, 4) ||
      !aligned(page_table, 4))
    return DSA_ERR_INVALID_ARG;
  for (int64_t s : strides)
    if (s % 8) return DSA_ERR_INVALID_ARG;
  return DSA_OK;
}

dsa_status check_attn(const dsa_attn_args& p) {
  if (!known(p.fmt) || (p.head_dim != 64 && p.head_dim != 128)) return DSA_ERR_UNSUPPORTED;
  if (p.Tq < 0 || p.B <= 0 || p.max_pages <= 0 || p.num_pages <= 0 || p.heads <= 0 || p.kv_heads <= 0 ||
      p.heads % p.kv_heads || !positive(p.scale) || !(static_cast<float>(p.scale * 1.4426950408889634) > 0.f) ||
      !std::isfinite(static_cast<float>(p.scale * 1.4426950408889634)) || (p.mask && p.mask_words <= 0))
    return DSA_ERR_INVALID_ARG;
  if (static_cast<long long>(p.num_pages) * 64 > 0x7FFFFFFFLL || p.kv_heads > 65536 ||
      static_cast<long long>(p.Tq) * p.heads > 0x7FFFFFFFLL || p.B == 0x7FFFFFFF)
    return DSA_ERR_UNSUPPORTED;
  // a bf16 cache is addressed by rows of one head's key or value
  if (p.fmt == DSA_FMT_BF16 && static_cast<long long>(p.num_pages) * p.kv_heads * 128 > 0x7FFFFFFFLL)
    return DSA_ERR_UNSUPPORTED;
  if (p.Tq == 0) return DSA_OK;
  if (!p.q || !p.out || !p.cache || !p.page_table || !p.seq_lens || !p.cu_q || !p.workspace) return DSA_ERR_INVALID_ARG;
  if (!aligned(p.q, 16) || !aligned(p.out, 16) || !aligned(p.cache, 256) || !aligned(p.workspace, 256) ||
      !aligned(p.lse, 4) || !aligned(p.mask, 4) || !aligned(p.page_table, 4) || !aligned(p.seq_lens, 4) ||
      !aligned(p.cu_q, 4) || p.q_stride_t % 8 || p.q_stride_h % 8 || p.out_stride_t % 8 || p.out_stride_h % 8 ||
      rows_meet(p.Tq, p.out_stride_t, p.heads, p.out_stride_h, p.head_dim))
    return DSA_ERR_INVALID_ARG;
  return DSA_OK;
}

}  // namespace

extern "C" {

dsa_status dsa_rope_create(dsa_ctx* ctx, dsa_rope** out, const dsa_rope_desc* d) {
  if (!ctx || !out || !d) return DSA_ERR_INVALID_ARG;
  *out = nullptr;
  if (d->rot_dim < 2 || d->rot_dim > 1024 || d->rot_dim % 2) return DSA_ERR_UNSUPPORTED;
  if (d->layout != DSA_ROPE_HALF && d->layout != DSA_ROPE_INTERLEAVED) return DSA_ERR_UNSUPPORTED;
  if (d->scaling < DSA_ROPE_PLAIN || d->scaling > DSA_ROPE_BY_PARTS) return DSA_ERR_UNSUPPORTED;
  if (!positive(d->theta) || d->max_pos <= 0 || !positive(d->mscale)) return DSA_ERR_INVALID_ARG;
  if (d->scaling != DSA_ROPE_PLAIN && !positive(d->factor)) return DSA_ERR_INVALID_ARG;
  if (d->scaling == DSA_ROPE_BY_PARTS &&
      (!positive(d->orig_max_pos) || !std::isfinite(d->beta_slow) || !std::isfinite(d->beta_fast) ||
       !(d->beta_slow < d->beta_fast)))
    return DSA_ERR_INVALID_ARG;
  if (const dsa_status s = dsa::check_device(ctx)) return s;
  return dsa::rope_create(ctx, out, *d);
}

dsa_status dsa_rope_destroy(dsa_rope* rope) {
  if (!rope) return DSA_ERR_INVALID_ARG;
  int cur = -1;
  const bool have_cur = cudaGetDevice(&cur) == cudaSuccess;
  if (have_cur && cur != rope->device) cudaSetDevice(rope->device);
  cudaDeviceSynchronize();
  cudaFree(rope->table);
  delete rope;
  if (have_cur && cur >= 0) cudaSetDevice(cur);
  return DSA_OK;
}

dsa_status dsa_rope_apply(dsa_ctx* ctx, const dsa_rope* rope, const void* x, void* y, dsa_dtype dtype,
                          const int32_t* pos, int32_t T, int32_t H, int32_t D, int32_t rot_start,
                          int64_t x_stride_t, int64_t x_stride_h, int64_t y_stride_t, int64_t y_stride_h,
                          int32_t inverse, dsa_stream_t stream) {
  if (!ctx || !rope) return DSA_ERR_INVALID_ARG;
  if (dtype != DSA_BF16 && dtype != DSA_F16 && dtype != DSA_F32) return DSA_ERR_UNSUPPORTED;
  if (T < 0 || H <= 0 || D <= 0 || rot_start < 0) return DSA_ERR_INVALID_ARG;
  if (T == 0) return DSA_OK;
  if (!x || !y || !pos) return DSA_ERR_INVALID_ARG;
  const uintptr_t es = dtype == DSA_F32 ? 4 : 2;
  if (!aligned(x, es) || !aligned(y, es) || !aligned(pos, 4)) return DSA_ERR_INVALID_ARG;
  if (x == y && (x_stride_t != y_stride_t || x_stride_h != y_stride_h)) return DSA_ERR_INVALID_ARG;
  if (y != x && rows_meet(T, y_stride_t, H, y_stride_h, D)) return DSA_ERR_INVALID_ARG;
  if (const dsa_status s = dsa::check_device(ctx)) return s;
  if (rope->device != ctx->device || static_cast<long long>(rot_start) + rope->rot_dim > D) return DSA_ERR_INVALID_ARG;
  // in place only the rotated part is written
  if (y == x && rows_meet(T, y_stride_t, H, y_stride_h, rope->rot_dim)) return DSA_ERR_INVALID_ARG;
  return dsa::launch_rope(ctx, rope, x, y, dtype, pos, T, H, D, rot_start, x_stride_t, x_stride_h, y_stride_t,
                          y_stride_h, inverse ? 1 : 0, as_stream(stream));
}

size_t dsa_kv_page_bytes(int32_t kv_heads, int32_t head_dim, dsa_fmt fmt) {
  if (kv_heads <= 0 || (head_dim != 64 && head_dim != 128) || !known(fmt)) return 0;
  return dsa::kv_page_bytes(kv_heads, head_dim, fmt);
}

dsa_status dsa_kv_store(dsa_ctx* ctx, const void* k, const void* v, int64_t k_stride_t, int64_t k_stride_h,
                        int64_t v_stride_t, int64_t v_stride_h, const int32_t* cache_pos, const int32_t* seq_id,
                        const int32_t* page_table, int32_t T, int32_t B, int32_t max_pages, int32_t kv_heads,
                        int32_t head_dim, void* cache, int32_t num_pages, dsa_fmt fmt, const dsa_rope* rope,
                        const int32_t* rope_pos, int32_t rot_start, dsa_stream_t stream) {
  if (!ctx) return DSA_ERR_INVALID_ARG;
  const int64_t strides[4] = {k_stride_t, k_stride_h, v_stride_t, v_stride_h};
  if (const dsa_status s = check_kv(cache, num_pages, fmt, kv_heads, head_dim, T, B, max_pages, k, v, strides,
                                    cache_pos, seq_id, page_table))
    return s;
  if (rot_start < 0 || !aligned(rope_pos, 4)) return DSA_ERR_INVALID_ARG;
  if (T == 0) return DSA_OK;
  if (const dsa_status s = dsa::check_device(ctx)) return s;
  if (rope && (rope->device != ctx->device || static_cast<long long>(rot_start) + rope->rot_dim > head_dim))
    return DSA_ERR_INVALID_ARG;
  return dsa::launch_kv_store(ctx, k, v, k_stride_t, k_stride_h, v_stride_t, v_stride_h, cache_pos, seq_id, page_table,
                              T, B, max_pages, kv_heads, head_dim, cache, num_pages, fmt, rope, rope_pos, rot_start,
                              as_stream(stream));
}

dsa_status dsa_kv_load(dsa_ctx* ctx, const void* cache, int32_t num_pages, dsa_fmt fmt, int32_t kv_heads,
                       int32_t head_dim, const int32_t* cache_pos, const int32_t* seq_id, const int32_t* page_table,
                       int32_t T, int32_t B, int32_t max_pages, void* k, void* v, int64_t k_stride_t,
                       int64_t k_stride_h, int64_t v_stride_t, int64_t v_stride_h, dsa_stream_t stream) {
  if (!ctx) return DSA_ERR_INVALID_ARG;
  const int64_t strides[4] = {k_stride_t, k_stride_h, v_stride_t, v_stride_h};
  if (const dsa_status s = check_kv(cache, num_pages, fmt, kv_heads, head_dim, T, B, max_pages, k, v, strides,
                                    cache_pos, seq_id, page_table))
    return s;
  if (T == 0) return DSA_OK;
  if (rows_meet(T, k_stride_t, kv_heads, k_stride_h, head_dim) || rows_meet(T, v_stride_t, kv_heads, v_stride_h, head_dim))
    return DSA_ERR_INVALID_ARG;
  if (const dsa_status s = dsa::check_device(ctx)) return s;
  return dsa::launch_kv_load(ctx, cache, num_pages, fmt, kv_heads, head_dim, cache_pos, seq_id, page_table, T, B,
                             max_pages, k, v, k_stride_t, k_stride_h, v_stride_t, v_stride_h, as_stream(stream));
}

size_t dsa_attn_workspace_size(const dsa_ctx* ctx, int32_t head_dim) {
  if (!ctx || (head_dim != 64 && head_dim != 128)) return 0;
  return dsa::attn_workspace(ctx, head_dim);
}

dsa_status dsa_tree_attn(dsa_ctx* ctx, const dsa_attn_args* args, dsa_stream_t stream) {
  if (!ctx || !args) return DSA_ERR_INVALID_ARG;
  if (const dsa_status s = check_attn(*args)) return s;
  if (args->Tq == 0) return DSA_OK;
  if (const dsa_status s = dsa::check_device(ctx)) return s;
  if (args->ws_bytes < dsa::attn_workspace(ctx, args->head_dim)) return DSA_ERR_WORKSPACE;
  return dsa::launch_attn(ctx, *args, nullptr, 0, as_stream(stream));
}

dsa_status dsa_sparse_attn(dsa_ctx* ctx, const dsa_attn_args* args, const int32_t* sel, int32_t k,
                           dsa_stream_t stream) {
  if (!ctx || !args) return DSA_ERR_INVALID_ARG;
  if (const dsa_status s = check_attn(*args)) return s;
  if (k < 1 || k > 65536 || args->heads / args->kv_heads > 128) return DSA_ERR_UNSUPPORTED;
  if (args->Tq == 0) return DSA_OK;
  if (!sel || !aligned(sel, 4)) return DSA_ERR_INVALID_ARG;
  if (const dsa_status s = dsa::check_device(ctx)) return s;
  if (args->ws_bytes < dsa::attn_workspace(ctx, args->head_dim)) return DSA_ERR_WORKSPACE;
  return dsa::launch_attn(ctx, *args, sel, k, as_stream(stream));
}

}  // extern "C"
