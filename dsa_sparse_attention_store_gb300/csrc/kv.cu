// K/V cache: write (rotate keys, quantise, scatter into pages) and read back.
//
// One row is one token's key or value of one kv head: D / 8 lanes with 8
// dimensions each. A key's rotation needs the partner dimensions, which the
// lane loads itself (the row is in L1 by then), so a row's lanes share
// nothing but the maximum of a 32-dimension block (4 lanes, two shuffles).
// The rotation is fp32 with every product and sum rounded separately and the
// rotated value is rounded once, to the cache's format.
//
// Bound: HBM for long batches (each value read once, its code written once),
// the two dependent loads position -> page id -> row for short ones.
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "kv_format.cuh"
#include "rope.cuh"

namespace dsa {
namespace {

using namespace kvf;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}

struct KvArgs {
  const __nv_bfloat16 *k, *v;   // store: sources
  __nv_bfloat16 *ko, *vo;       // load: destinations
  long long kt, kh, vt, vh;     // strides, in elements
  const int32_t *cache_pos, *seq_id, *page_table, *rope_pos;
  const float2* table;          // rotary table, or NULL
  uint8_t* cache;
  unsigned int* status;
  int T, B, max_pages, num_pages, kv_heads;
  int R, start, rope_max, half_layout, wide;  // wide: a lane's 8 dimensions pair with 8 others, or among themselves
};

// the token's page, or -1 (reported by the row's first lane)
__device__ __forceinline__ int find_page(const KvArgs& a, int t, int& off, bool report) {
  const int pos = a.cache_pos[t], s = a.seq_id[t];
  int page = -1;
  if (s >= 0 && s < a.B && pos >= 0 && (pos >> 6) < a.max_pages) {
    page = a.page_table[static_cast<long long>(s) * a.max_pages + (pos >> 6)];
    if (page >= a.num_pages) page = -1;
  }
  if (page < 0) page = -1;
  if (page < 0 && report) atomicOr(a.status, DSA_DEV_BOUNDS);
  off = pos & (kPage - 1);
  return page;
}

template <int FMT, int D>
__global__ void __launch_bounds__(128) kv_store_kernel(KvArgs a) {
  using L = Layout<FMT, D>;
  constexpr int LANES = D / 8;
  pdl_wait();
  pdl_trigger();
  const long long row = static_cast<long long>(blockIdx.x) * (128 / LANES) + threadIdx.x / LANES;
  const int l = threadIdx.x % LANES, d0 = 8 * l;
  const bool live = row < static_cast<long long>(a.T) * a.kv_heads;
  const int t = live ? static_cast<int>(row / a.kv_heads) : 0;
  const int h = live ? static_cast<int>(row % a.kv_heads) : 0;
  const bool is_v = blockIdx.y == 1;
  const __nv_bfloat16* src = is_v ? a.v + t * a.vt + h * a.vh : a.k + t * a.kt + h * a.kh;
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  int off = 0, page = -1;
  if (live) {
    const uint4 raw = __ldg(reinterpret_cast<const uint4*>(src + d0));
    page = find_page(a, t, off, l == 0 && h == 0);
    unpack8(raw, x);
  }
  int rp = 0;
  if (a.table && live) {  // a token whose rotary position is out of range is not written
    rp = a.rope_pos[t];
    if (rp < 0 || rp >= a.rope_max) {
      page = -1;
      rp = 0;
      if (l == 0 && h == 0) atomicOr(a.status, DSA_DEV_BOUNDS);
    }
  }
  if (a.table && !is_v && live && d0 < a.start + a.R && d0 + 8 > a.start) {
    const float2* tab = a.table + static_cast<long long>(rp) * (a.R >> 1);
    const int half = a.R >> 1, p0 = d0 - a.start;
    if (a.wide) {
      float c[8], s[8], o[8];
      if (a.half_layout) {
        const bool upper = p0 >= half;
        const int i0 = upper ? p0 - half : p0;
        const uint4 raw = __ldg(reinterpret_cast<const uint4*>(src + (upper ? d0 - half : d0 + half)));
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float4 w = __ldg(reinterpret_cast<const float4*>(tab + i0 + i));
          c[i] = w.x;
          s[i] = upper ? w.y : -w.y;
          c[i + 1] = w.z;
          s[i + 1] = upper ? w.w : -w.w;
        }
        unpack8(raw, o);
      } else {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 w = __ldg(reinterpret_cast<const float4*>(tab + ((p0 + i) >> 1)));
          c[i] = c[i + 1] = w.x;
          c[i + 2] = c[i + 3] = w.z;
          s[i] = -w.y;
          s[i + 1] = w.y;
          s[i + 2] = -w.w;
          s[i + 3] = w.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = x[i ^ 1];
      }
      // own * c -+ partner * s: x - y and x + (-y) round alike
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(__fmul_rn(x[i], c[i]), __fmul_rn(o[i], s[i]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int p = p0 + i;
        if (p < 0 || p >= a.R) continue;
        const bool upper = a.half_layout ? p >= half : p & 1;
        const int pair = a.half_layout ? (upper ? p - half : p) : p >> 1;
        const int other = a.half_layout ? (upper ? p - half : p + half) : p ^ 1;
        const float2 w = __ldg(tab + pair);
        const float y = __bfloat162float(src[a.start + other]);
        x[i] = __fadd_rn(__fmul_rn(x[i], w.x), __fmul_rn(y, upper ? w.y : -w.y));
      }
    }
  }
  uint8_t* blk = a.cache + (static_cast<long long>(page < 0 ? 0 : page) * a.kv_heads + h) * L::HEAD_BYTES;
  uint8_t* dst = blk + (is_v ? L::V_CODES : L::K_CODES) + off * L::CB;
  if constexpr (FMT == DSA_FMT_BF16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      memcpy(&w[i], &p, 4);
    }
    if (page >= 0) *reinterpret_cast<uint4*>(dst + 16 * l) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    uint32_t amax = 0;  // as bits: above any finite value where a NaN or infinity is among them
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const bool bad = amax >= 0x7F800000u;
    const int e = Scale<FMT>::exponent(amax);
    const float inv = bad ? 0.f : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = bad ? 0.f : __fmul_rn(x[i], inv);
    if constexpr (FMT == DSA_FMT_FP8) {
      uint32_t w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
      }
      if (page >= 0) *reinterpret_cast<uint2*>(dst + 8 * l) = make_uint2(w[0], w[1]);
    } else {
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w |= static_cast<uint32_t>(
                 __nv_cvt_float2_to_fp4x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_E2M1, cudaRoundNearest))
             << (8 * i);
      if (page >= 0) *reinterpret_cast<uint32_t*>(dst + 4 * l) = w;
    }
    if (page >= 0 && (l & 3) == 0)
      blk[(is_v ? L::V_SCALES : L::K_SCALES) + off * L::SB + (l >> 2)] = bad ? 255 : static_cast<uint8_t>(e + 127);
  }
}

template <int FMT, int D>
__global__ void __launch_bounds__(128) kv_load_kernel(KvArgs a) {
  using L = Layout<FMT, D>;
  constexpr int LANES = D / 8;
  pdl_wait();
  pdl_trigger();
  const long long row = static_cast<long long>(blockIdx.x) * (128 / LANES) + threadIdx.x / LANES;
  const int l = threadIdx.x % LANES;
  if (row >= static_cast<long long>(a.T) * a.kv_heads) return;
  const int t = static_cast<int>(row / a.kv_heads), h = static_cast<int>(row % a.kv_heads);
  const bool is_v = blockIdx.y == 1;
  __nv_bfloat16* out = (is_v ? a.vo + t * a.vt + h * a.vh : a.ko + t * a.kt + h * a.kh) + 8 * l;
  int off;
  const int page = find_page(a, t, off, l == 0 && h == 0);
  uint4 w = make_uint4(0, 0, 0, 0);  // a row that has no page reads as zeros
  if (page >= 0) {
    const uint8_t* blk = a.cache + (static_cast<long long>(page) * a.kv_heads + h) * L::HEAD_BYTES;
    const uint8_t* src = blk + (is_v ? L::V_CODES : L::K_CODES) + off * L::CB;
    if constexpr (FMT == DSA_FMT_BF16) {
      w = *reinterpret_cast<const uint4*>(src + 16 * l);
    } else {
      Factor<FMT> f;
      f.set(blk[(is_v ? L::V_SCALES : L::K_SCALES) + off * L::SB + (l >> 2)]);
      if constexpr (FMT == DSA_FMT_FP8) {
        const uint2 v = *reinterpret_cast<const uint2*>(src + 8 * l);
        const uint32_t c[2] = {v.x, v.y};
        uint32_t o[4];
        widen(c, f, o);
        f.rest(o);
        w = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        const uint32_t c[1] = {*reinterpret_cast<const uint32_t*>(src + 4 * l)};
        uint32_t o[4];
        widen(c, f, o);
        f.rest(o);
        w = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
  *reinterpret_cast<uint4*>(out) = w;
}

template <int D>
auto store_of(dsa_fmt fmt) {
  return fmt == DSA_FMT_BF16 ? kv_store_kernel<DSA_FMT_BF16, D>
         : fmt == DSA_FMT_FP8 ? kv_store_kernel<DSA_FMT_FP8, D> : kv_store_kernel<DSA_FMT_FP4, D>;
}
template <int D>
auto load_of(dsa_fmt fmt) {
  return fmt == DSA_FMT_BF16 ? kv_load_kernel<DSA_FMT_BF16, D>
         : fmt == DSA_FMT_FP8 ? kv_load_kernel<DSA_FMT_FP8, D> : kv_load_kernel<DSA_FMT_FP4, D>;
}

dsa_status launch(dsa_ctx* ctx, int kind, void (*kern)(KvArgs), int D, KvArgs& a, cudaStream_t stream) {
  a.status = ctx->status;
  const long long rows = static_cast<long long>(a.T) * a.kv_heads;
  const long long blocks = (rows * (D / 8) + 127) / 128;
  if (blocks > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
  LaunchScope scope(ctx, kind, stream);
  const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>(blocks), 2), dim3(128), 0, stream, a);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace

size_t kv_page_bytes(int32_t kv_heads, int32_t head_dim, dsa_fmt fmt) {
  const size_t row = fmt == DSA_FMT_BF16 ? 2 * head_dim
                     : fmt == DSA_FMT_FP8 ? head_dim + head_dim / kBlock : head_dim / 2 + head_dim / kBlock;
  return static_cast<size_t>(kv_heads) * 2 * kPage * row;
}

dsa_status launch_kv_store(dsa_ctx* ctx, const void* k, const void* v, long long kt, long long kh, long long vt,
                           long long vh, const int32_t* cache_pos, const int32_t* seq_id,
                           const int32_t* page_table, int32_t T, int32_t B, int32_t max_pages, int32_t kv_heads,
                           int32_t head_dim, void* cache, int32_t num_pages, dsa_fmt fmt, const dsa_rope* rope,
                           const int32_t* rope_pos, int32_t start, cudaStream_t stream) {
  KvArgs a = {};
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.kt = kt;
  a.kh = kh;
  a.vt = vt;
  a.vh = vh;
  a.cache_pos = cache_pos;
  a.seq_id = seq_id;
  a.page_table = page_table;
  a.rope_pos = rope_pos ? rope_pos : cache_pos;
  a.cache = static_cast<uint8_t*>(cache);
  a.T = T;
  a.B = B;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.kv_heads = kv_heads;
  if (rope) {
    a.table = rope->table;
    a.R = rope->rot_dim;
    a.start = start;
    a.rope_max = rope->max_pos;
    a.half_layout = rope->layout == DSA_ROPE_HALF;
    a.wide = start % 8 == 0 && (a.half_layout ? (a.R / 2) % 8 == 0 : a.R % 8 == 0);
  }
  return launch(ctx, DSA_K_KV_STORE, head_dim == 128 ? store_of<128>(fmt) : store_of<64>(fmt), head_dim, a, stream);
}

dsa_status launch_kv_load(dsa_ctx* ctx, const void* cache, int32_t num_pages, dsa_fmt fmt, int32_t kv_heads,
                          int32_t head_dim, const int32_t* cache_pos, const int32_t* seq_id,
                          const int32_t* page_table, int32_t T, int32_t B, int32_t max_pages, void* k, void* v,
                          long long kt, long long kh, long long vt, long long vh, cudaStream_t stream) {
  KvArgs a = {};
  a.ko = static_cast<__nv_bfloat16*>(k);
  a.vo = static_cast<__nv_bfloat16*>(v);
  a.kt = kt;
  a.kh = kh;
  a.vt = vt;
  a.vh = vh;
  a.cache_pos = cache_pos;
  a.seq_id = seq_id;
  a.page_table = page_table;
  a.cache = const_cast<uint8_t*>(static_cast<const uint8_t*>(cache));
  a.T = T;
  a.B = B;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.kv_heads = kv_heads;
  return launch(ctx, DSA_K_KV_LOAD, head_dim == 128 ? load_of<128>(fmt) : load_of<64>(fmt), head_dim, a, stream);
}

}  // namespace dsa
