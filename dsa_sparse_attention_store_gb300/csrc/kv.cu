// K/V cache: write (rotate keys, quantise, scatter into pages) and read back.
//
// A row is one token's key or value of one kv head: D / 8 lanes with 8
// dimensions each. A thread has its lane's part of the key and the value of
// up to HPT heads of one token, so that position -> page id -> row, the
// dependent loads, are walked once for 2 HPT rows and their data loads are in
// flight together, and the cos/sin of the rotation serve all keys. A row's
// lanes share the maximum of a 32-dimension block (4 lanes, two shuffles) and,
// in the half layout, the partner dimensions (a shuffle). The rotation is
// fp32 with every product and sum rounded separately and the rotated value is
// rounded once, to the cache's format.
//
// Bound: for long batches HBM in bf16; writing fp8 or fp4, the quantising
// instructions and the loads they wait for (fp4: issue slots 57 % busy, integer
// pipe 46 %, DRAM 36 %); the dependent loads for short ones. 22528 tokens x 8
// heads x 128: written and read back in 63 us bf16 (floor 54), 60 us fp8 (41),
// 56 us fp4 (34; store 38 to 44, load 22 with launch overhead); 64 tokens 3.9 us.
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
  int groups;                   // a token's heads are split among so many threads of a lane
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

// the larger one; NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// 8 fp32 values of a row -> the cache (codes at dst for this lane, the block's
// scale); every lane of the warp calls it, `ok` says whether the row is written
template <int FMT>
__device__ __forceinline__ void put_row(const float (&v)[8], bool ok, uint8_t* codes, uint8_t* scale, int l) {
  if constexpr (FMT == DSA_FMT_BF16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      memcpy(&w[i], &p, 4);
    }
    if (ok) *reinterpret_cast<uint4*>(codes + 16 * l) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float top = fabsf(v[0]);  // a NaN stays one
#pragma unroll
    for (int i = 1; i < 8; ++i) top = max_nan(top, fabsf(v[i]));
    uint32_t amax = __float_as_uint(top) & 0x7FFFFFFFu;  // as bits: above any finite value for NaN and infinity
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const bool bad = amax >= 0x7F800000u;
    const int e = Scale<FMT>::exponent(amax);
    const float inv = bad ? 0.f : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(v[i], inv);
    if (bad) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
    }
    if constexpr (FMT == DSA_FMT_FP8) {
      uint32_t w[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
      }
      if (ok) *reinterpret_cast<uint2*>(codes + 8 * l) = make_uint2(w[0], w[1]);
    } else {
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w |= static_cast<uint32_t>(
                 __nv_cvt_float2_to_fp4x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_E2M1, cudaRoundNearest))
             << (8 * i);
      if (ok) *reinterpret_cast<uint32_t*>(codes + 4 * l) = w;
    }
    if (ok && (l & 3) == 0) scale[l >> 2] = bad ? 255 : static_cast<uint8_t>(e + 127);
  }
}

// the thread's place: lane of a row, token and first head (heads h, h +
// groups, ...); a warp's threads are consecutive
struct Place {
  int l, t, h;
  bool live;
};
template <int D>
__device__ __forceinline__ Place place_of(const KvArgs& a) {
  const long long x = static_cast<long long>(blockIdx.x) * 128 + threadIdx.x;
  const long long row = x / (D / 8);
  Place p;
  p.l = static_cast<int>(x % (D / 8));
  p.live = row < static_cast<long long>(a.T) * a.groups;
  p.t = p.live ? static_cast<int>(row / a.groups) : 0;
  p.h = p.live ? static_cast<int>(row % a.groups) : 0;
  return p;
}

template <int FMT, int D, int HPT>
__global__ void __launch_bounds__(128) kv_store_kernel(KvArgs a) {
  using L = Layout<FMT, D>;
  pdl_wait();
  pdl_trigger();
  const Place p = place_of<D>(a);
  const int l = p.l, t = p.t, d0 = 8 * l;
  uint4 rk[HPT], rv[HPT];
  int rp = 0;
#pragma unroll
  for (int j = 0; j < HPT; ++j) {
    const int h = p.h + j * a.groups;
    const bool in = p.live && h < a.kv_heads;
    rk[j] = in ? __ldg(reinterpret_cast<const uint4*>(a.k + t * a.kt + h * a.kh + d0)) : make_uint4(0, 0, 0, 0);
    rv[j] = in ? __ldg(reinterpret_cast<const uint4*>(a.v + t * a.vt + h * a.vh + d0)) : make_uint4(0, 0, 0, 0);
  }
  int off = 0, page = -1;
  if (p.live) {
    if (a.table) rp = a.rope_pos[t];
    page = find_page(a, t, off, l == 0 && p.h == 0);
    if (a.table && (rp < 0 || rp >= a.rope_max)) {  // a token whose rotary position is out of range is not written
      page = -1;
      rp = 0;
      if (l == 0 && p.h == 0) atomicOr(a.status, DSA_DEV_BOUNDS);
    }
  }
  const bool turns = a.table && d0 < a.start + a.R && d0 + 8 > a.start;  // some of this lane's dimensions do
  const int half = a.R >> 1, p0 = d0 - a.start;
  const bool upper = p0 >= half;
  const float2* tab = a.table + static_cast<long long>(rp) * half;
  float c[8], s[8];  // own * c + partner * s
  if (turns && a.wide) {
    if (a.half_layout) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(tab + (upper ? p0 - half : p0) + i));
        c[i] = w.x;
        s[i] = upper ? w.y : -w.y;
        c[i + 1] = w.z;
        s[i + 1] = upper ? w.w : -w.w;
      }
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
    }
  }
  // the lane of the row that holds the partners (half layout)
  const int lane = threadIdx.x & 31;
  const int mate = turns && a.wide && a.half_layout ? (lane & ~(D / 8 - 1)) | (upper ? l - (half >> 3) : l + (half >> 3)) : lane;
  uint8_t* const blk = a.cache + static_cast<long long>(page < 0 ? 0 : page) * a.kv_heads * L::HEAD_BYTES;
#pragma unroll
  for (int j = 0; j < HPT; ++j) {
    const int h = p.h + j * a.groups;
    const bool ok = page >= 0 && h < a.kv_heads;
    float x[8];
    unpack8(rk[j], x);
    if (a.table) {  // uniform
      if (a.wide) {
        float o[8];
        if (a.half_layout) {
          uint4 m;
          m.x = __shfl_sync(0xffffffffu, rk[j].x, mate);
          m.y = __shfl_sync(0xffffffffu, rk[j].y, mate);
          m.z = __shfl_sync(0xffffffffu, rk[j].z, mate);
          m.w = __shfl_sync(0xffffffffu, rk[j].w, mate);
          unpack8(m, o);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = x[i ^ 1];
        }
        if (turns) {
          // x - y and x + (-y) round alike
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(__fmul_rn(x[i], c[i]), __fmul_rn(o[i], s[i]));
        }
      } else if (turns && p.live && h < a.kv_heads) {
        const __nv_bfloat16* src = a.k + t * a.kt + h * a.kh;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int d = p0 + i;
          if (d < 0 || d >= a.R) continue;
          const bool up = a.half_layout ? d >= half : d & 1;
          const int pair = a.half_layout ? (up ? d - half : d) : d >> 1;
          const int other = a.half_layout ? (up ? d - half : d + half) : d ^ 1;
          const float2 w = __ldg(tab + pair);
          const float y = __bfloat162float(src[a.start + other]);
          x[i] = __fadd_rn(__fmul_rn(x[i], w.x), __fmul_rn(y, up ? w.y : -w.y));
        }
      }
    }
    uint8_t* const b = blk + static_cast<long long>(ok ? h : 0) * L::HEAD_BYTES;
    put_row<FMT>(x, ok, b + L::K_CODES + off * L::CB, b + L::K_SCALES + off * L::SB, l);
    unpack8(rv[j], x);
    put_row<FMT>(x, ok, b + L::V_CODES + off * L::CB, b + L::V_SCALES + off * L::SB, l);
  }
}

template <int FMT, int D, int HPT>
__global__ void __launch_bounds__(128) kv_load_kernel(KvArgs a) {
  using L = Layout<FMT, D>;
  constexpr int W = FMT == DSA_FMT_BF16 ? 4 : FMT == DSA_FMT_FP8 ? 2 : 1;  // words of codes a lane has
  pdl_wait();
  pdl_trigger();
  const Place p = place_of<D>(a);
  if (!p.live) return;
  const int l = p.l, t = p.t;
  int off;
  const int page = find_page(a, t, off, l == 0 && p.h == 0);
  const uint8_t* const blk = a.cache + static_cast<long long>(page < 0 ? 0 : page) * a.kv_heads * L::HEAD_BYTES;
  uint32_t c[2 * HPT][W], sc[2 * HPT];
#pragma unroll
  for (int j = 0; j < 2 * HPT; ++j) {
    const int h = p.h + (j >> 1) * a.groups;
    const uint8_t* b = blk + static_cast<long long>(h) * L::HEAD_BYTES;
    const uint8_t* src = b + (j & 1 ? L::V_CODES : L::K_CODES) + off * L::CB + 4 * W * l;
    sc[j] = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) c[j][i] = 0;
    if (page >= 0 && h < a.kv_heads) {
      if constexpr (W == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(src);
        c[j][0] = v.x;
        c[j][1] = v.y;
        c[j][2] = v.z;
        c[j][3] = v.w;
      } else if constexpr (W == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(src);
        c[j][0] = v.x;
        c[j][1] = v.y;
      } else {
        c[j][0] = *reinterpret_cast<const uint32_t*>(src);
      }
      if constexpr (W != 4) sc[j] = b[(j & 1 ? L::V_SCALES : L::K_SCALES) + off * L::SB + (l >> 2)];
    }
  }
#pragma unroll
  for (int j = 0; j < 2 * HPT; ++j) {
    const int h = p.h + (j >> 1) * a.groups;
    if (h >= a.kv_heads) continue;
    uint32_t w[4];
    if constexpr (W == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = c[j][i];
    } else {
      Factor<FMT> f;
      f.set(sc[j]);
      widen(c[j], f, w);
      f.rest(sc[j], w);
    }
    __nv_bfloat16* out = (j & 1 ? a.vo + t * a.vt + h * a.vh : a.ko + t * a.kt + h * a.kh) + 8 * l;
    // a token that has no page reads as zeros
    *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

typedef void (*Kern)(KvArgs);
template <int D, int HPT>
Kern store_of(dsa_fmt fmt) {
  return fmt == DSA_FMT_BF16 ? kv_store_kernel<DSA_FMT_BF16, D, HPT>
         : fmt == DSA_FMT_FP8 ? kv_store_kernel<DSA_FMT_FP8, D, HPT> : kv_store_kernel<DSA_FMT_FP4, D, HPT>;
}
template <int D, int HPT>
Kern load_of(dsa_fmt fmt) {
  return fmt == DSA_FMT_BF16 ? kv_load_kernel<DSA_FMT_BF16, D, HPT>
         : fmt == DSA_FMT_FP8 ? kv_load_kernel<DSA_FMT_FP8, D, HPT> : kv_load_kernel<DSA_FMT_FP4, D, HPT>;
}

dsa_status launch(dsa_ctx* ctx, bool store, int D, dsa_fmt fmt, KvArgs& a, cudaStream_t stream) {
  a.status = ctx->status;
  // four heads a thread once there are many: 8 heads of 512 tokens, fp8, written
  // and read back 5.6 against 4.9 us, of 1024 6.4 against 7.3, of 4509 12.8 against 15.6
  const long long threads = static_cast<long long>(a.T) * a.kv_heads * (D / 8);
  const bool many = a.kv_heads >= 4 && threads >= 768LL * ctx->num_sms;
  a.groups = many ? (a.kv_heads + 3) / 4 : a.kv_heads;
  const long long blocks = (static_cast<long long>(a.T) * a.groups * (D / 8) + 127) / 128;
  if (blocks > 0x7FFFFFFFLL) return DSA_ERR_UNSUPPORTED;
  const Kern kern = store ? (D == 128 ? (many ? store_of<128, 4>(fmt) : store_of<128, 1>(fmt))
                                      : (many ? store_of<64, 4>(fmt) : store_of<64, 1>(fmt)))
                          : (D == 128 ? (many ? load_of<128, 4>(fmt) : load_of<128, 1>(fmt))
                                      : (many ? load_of<64, 4>(fmt) : load_of<64, 1>(fmt)));
  LaunchScope scope(ctx, store ? DSA_K_KV_STORE : DSA_K_KV_LOAD, stream);
  const cudaError_t e = launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(128), 0, stream, a);
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
  return launch(ctx, true, head_dim, fmt, a, stream);
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
  return launch(ctx, false, head_dim, fmt, a, stream);
}

}  // namespace dsa
