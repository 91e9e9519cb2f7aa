// Rotary positions: the table of a plan, and the rotation of [T][H][D] rows.
//
// Mathematics: pair i of the rotated part (a, b) turns by the angle
// pos * f_i:  a' = a c - b s,  b' = b c + a s  with c = m cos, s = m sin.
// The inverse (also the gradient of the forward rotation) takes s with the
// other sign. Frequencies f_i = theta^(-2i/R); "linear" divides them by the
// factor; "by parts" (YaRN, arXiv 2309.00071, section 3.2) divides those that
// turn fewer than beta_slow times over the original context, keeps those
// that turn more than beta_fast times and blends linearly between.
//
// Angles are products in double (a float loses the angle of far positions:
// at position 131072 the fastest pair's angle has an ulp of 2^-7 rad), and
// cos and sin are rounded once to fp32, when the plan is made. The rotation
// is fp32 with every product and sum rounded separately (the index store's
// rule) and one rounding to the tensor's type.
//
// Bound: HBM (each element read and written once; the table row of a token
// is shared by its heads through L1/L2). 22528 tokens x 64 heads x 128 bf16:
// 107 us, 6.9 TB/s, what a copy takes. 64 tokens: 1.9 us, a launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <new>

#include "rope.cuh"

namespace dsa {
namespace {

__global__ void __launch_bounds__(256) rope_table_kernel(const double* __restrict__ freq, int half, int max_pos,
                                                         double mscale, float2* __restrict__ table) {
  const long long n = static_cast<long long>(max_pos) * half;
  for (long long x = blockIdx.x * 256LL + threadIdx.x; x < n; x += gridDim.x * 256LL) {
    const int p = static_cast<int>(x / half), i = static_cast<int>(x % half);
    double s, c;
    sincos(static_cast<double>(p) * freq[i], &s, &c);
    table[x] = make_float2(static_cast<float>(mscale * c), static_cast<float>(mscale * s));
  }
}

// element types: to fp32 and back, singly and two to a word (one conversion
// instruction for two values: with one for each, bf16 ran at half the speed)
struct Bf16 {
  using type = __nv_bfloat16;
  static constexpr int PER_WORD = 2;
  static __device__ __forceinline__ float up(type v) { return __bfloat162float(v); }
  static __device__ __forceinline__ type down(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ void up2(uint32_t w, float& a, float& b) {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
  }
  static __device__ __forceinline__ uint32_t down2(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    uint32_t w;
    memcpy(&w, &p, 4);
    return w;
  }
};
struct F16 {
  using type = __half;
  static constexpr int PER_WORD = 2;
  static __device__ __forceinline__ float up(type v) { return __half2float(v); }
  static __device__ __forceinline__ type down(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ void up2(uint32_t w, float& a, float& b) {
    __half2 p;
    memcpy(&p, &w, 4);
    const float2 f = __half22float2(p);
    a = f.x;
    b = f.y;
  }
  static __device__ __forceinline__ uint32_t down2(float a, float b) {
    const __half2 p = __floats2half2_rn(a, b);
    uint32_t w;
    memcpy(&w, &p, 4);
    return w;
  }
};
struct F32 {
  using type = float;
  static constexpr int PER_WORD = 1;
  static __device__ __forceinline__ float up(type v) { return v; }
  static __device__ __forceinline__ type down(float v) { return v; }
};

// a run of V elements as it lies in memory: one element, or 16 bytes
template <typename E, int V>
struct Run {
  uint4 w;
  __device__ __forceinline__ void load(const typename E::type* p) { w = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void store(typename E::type* p) const { __stcs(reinterpret_cast<uint4*>(p), w); }
  __device__ __forceinline__ void get(float (&f)[V]) const {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (E::PER_WORD == 2)
        E::up2(v[i], f[2 * i], f[2 * i + 1]);
      else
        f[i] = __uint_as_float(v[i]);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[V]) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (E::PER_WORD == 2)
        v[i] = E::down2(f[2 * i], f[2 * i + 1]);
      else
        v[i] = __float_as_uint(f[i]);
    }
    w = make_uint4(v[0], v[1], v[2], v[3]);
  }
};
template <typename E>
struct Run<E, 1> {
  typename E::type w;
  __device__ __forceinline__ void load(const typename E::type* p) { w = *p; }
  __device__ __forceinline__ void store(typename E::type* p) const { *p = w; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = E::up(w); }
  __device__ __forceinline__ void set(const float (&f)[1]) { w = E::down(f[0]); }
};

struct RopeArgs {
  const void* x;
  void* y;
  const int32_t* pos;
  const float2* table;
  unsigned int* status;
  long long xt, xh, yt, yh;  // strides, in elements
  int T, H, D, R, start, max_pos, inverse;
  int npair;   // items of a head that rotate V pairs
  int ncopy;   // items that copy 2 V untouched elements (0 in place)
  int groups;  // threads share a token's heads: each takes heads g, g + groups, ...
  int tpb;     // tokens per block (>= 1)
};

// One thread: two runs of V elements of up to HPT heads of one token, so that
// the cos/sin it loads serve all of them and 2 HPT loads are in flight. The
// runs are V consecutive elements of the rotated part and those half the part
// further on (the partners in the half layout; pairs of their own in the
// interleaved one), or of the untouched part and those half of it further on:
// neighbouring threads read neighbouring runs either way. V is 16 bytes' worth
// of elements where sizes, offsets and addresses allow; otherwise a run is one
// pair's element (V = 1).
template <typename E, int V, int HPT, bool INTERLEAVED>
__global__ void __launch_bounds__(256) rope_kernel(RopeArgs a) {
  pdl_wait();
  pdl_trigger();
  using El = typename E::type;
  const int items = a.npair + a.ncopy;
  const int per = items * a.groups;
  const int q = threadIdx.x / per;                    // 0 when per > 256
  const int r = (threadIdx.x - q * per) + blockIdx.y * 256;
  const long long t = static_cast<long long>(blockIdx.x) * a.tpb + q;
  if (q >= a.tpb || r >= per || t >= a.T) return;
  const int item = r % items, g = r / items;
  const int pos = a.pos[t];
  if (pos < 0 || pos >= a.max_pos) {  // reported, and the row stays as it was
    if (r == 0) atomicOr(a.status, DSA_DEV_BOUNDS);
    return;
  }
  const El* x = static_cast<const El*>(a.x) + t * a.xt;
  El* y = static_cast<El*>(a.y) + t * a.yt;
  int e0, e1;  // where the runs begin
  float c[V], s[V];
  const bool rot = item < a.npair;
  if (rot) {
    const float2* tab = a.table + static_cast<long long>(pos) * (a.R >> 1);
    if constexpr (V >= 2) {
      // interleaved: V / 2 pairs of the first run, then V / 2 of the second
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const int pair = INTERLEAVED ? (i < V / 2 ? 0 : (a.R >> 2) - V / 2) + item * (V / 2) + i : item * V + i;
        const float4 w = __ldg(reinterpret_cast<const float4*>(tab + pair));
        c[i] = w.x;
        s[i] = w.y;
        c[i + 1] = w.z;
        s[i + 1] = w.w;
      }
    } else {
      const float2 w = __ldg(tab + item);
      c[0] = w.x;
      s[0] = w.y;
    }
    if (a.inverse) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = -s[i];
    }
    e0 = a.start + (INTERLEAVED && V == 1 ? 2 * item : item * V);
    e1 = INTERLEAVED && V == 1 ? e0 + 1 : e0 + (a.R >> 1);
  } else {
    e0 = (item - a.npair) * V;
    e1 = e0 + a.ncopy * V;
    if (e0 >= a.start) e0 += a.R;
    if (e1 >= a.start) e1 += a.R;
  }
  for (int h0 = g; h0 < a.H; h0 += a.groups * HPT) {
    Run<E, V> r0[HPT], r1[HPT];
#pragma unroll
    for (int j = 0; j < HPT; ++j) {
      const int h = h0 + j * a.groups;
      if (h < a.H) {
        r0[j].load(x + h * a.xh + e0);
        if (e1 < a.D) r1[j].load(x + h * a.xh + e1);
      }
    }
#pragma unroll
    for (int j = 0; j < HPT; ++j) {
      const int h = h0 + j * a.groups;
      if (h >= a.H) continue;
      if (rot) {
        float f0[V], f1[V];
        r0[j].get(f0);
        r1[j].get(f1);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          // pair i: element i of both runs, or two neighbours of one
          float& ea = INTERLEAVED && V > 1 ? (2 * i < V ? f0 : f1)[(2 * i) % V] : f0[i];
          float& eb = INTERLEAVED && V > 1 ? (2 * i < V ? f0 : f1)[(2 * i + 1) % V] : f1[i];
          const float u = ea, w = eb;
          ea = __fsub_rn(__fmul_rn(u, c[i]), __fmul_rn(w, s[i]));
          eb = __fadd_rn(__fmul_rn(w, c[i]), __fmul_rn(u, s[i]));
        }
        r0[j].set(f0);
        r1[j].set(f1);
      }
      r0[j].store(y + h * a.yh + e0);
      if (e1 < a.D) r1[j].store(y + h * a.yh + e1);
    }
  }
}

template <typename E, int V>
cudaError_t launch(const RopeArgs& a, bool interleaved, bool many, dim3 grid, cudaStream_t stream) {
  auto kern = interleaved ? (many ? rope_kernel<E, V, 4, true> : rope_kernel<E, V, 1, true>)
                          : (many ? rope_kernel<E, V, 4, false> : rope_kernel<E, V, 1, false>);
  return launch_pdl(kern, grid, dim3(256), 0, stream, a);
}

}  // namespace

dsa_status rope_create(dsa_ctx* ctx, dsa_rope** out, const dsa_rope_desc& d) {
  const int half = d.rot_dim / 2;
  double f[512];  // rot_dim is at most 1024
  for (int i = 0; i < half; ++i) {
    const double base = std::pow(d.theta, -(2.0 * i) / d.rot_dim);
    double v = base;
    if (d.scaling == DSA_ROPE_LINEAR) v = base / d.factor;
    if (d.scaling == DSA_ROPE_BY_PARTS) {
      const double turns = d.orig_max_pos * base / (2.0 * 3.14159265358979323846);
      double keep = (turns - d.beta_slow) / (d.beta_fast - d.beta_slow);
      keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
      v = base / d.factor * (1.0 - keep) + base * keep;
    }
    f[i] = v;
  }
  dsa_rope* r = new (std::nothrow) dsa_rope();
  if (!r) return DSA_ERR_CUDA;
  r->device = ctx->device;
  r->rot_dim = d.rot_dim;
  r->layout = d.layout;
  r->max_pos = d.max_pos;
  double* df = nullptr;
  const size_t n = static_cast<size_t>(d.max_pos) * half;
  bool ok = cudaMalloc(&r->table, n * sizeof(float2)) == cudaSuccess &&
            cudaMalloc(&df, half * sizeof(double)) == cudaSuccess &&
            cudaMemcpy(df, f, half * sizeof(double), cudaMemcpyHostToDevice) == cudaSuccess;
  if (ok) {
    const size_t blocks = (n + 255) / 256;
    rope_table_kernel<<<static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 256>>>(df, half, d.max_pos, d.mscale,
                                                                                    r->table);
    ok = cudaGetLastError() == cudaSuccess && cudaDeviceSynchronize() == cudaSuccess;
  }
  cudaFree(df);
  if (!ok) {
    cudaFree(r->table);
    cudaGetLastError();  // a table that does not fit leaves no error behind
    delete r;
    return DSA_ERR_CUDA;
  }
  *out = r;
  return DSA_OK;
}

dsa_status launch_rope(dsa_ctx* ctx, const dsa_rope* rope, const void* x, void* y, dsa_dtype dtype,
                       const int32_t* pos, int32_t T, int32_t H, int32_t D, int32_t start, long long xt,
                       long long xh, long long yt, long long yh, int32_t inverse, cudaStream_t stream) {
  RopeArgs a = {};
  a.x = x;
  a.y = y;
  a.pos = pos;
  a.table = rope->table;
  a.status = ctx->status;
  a.xt = xt;
  a.xh = xh;
  a.yt = yt;
  a.yh = yh;
  a.T = T;
  a.H = H;
  a.D = D;
  a.R = rope->rot_dim;
  a.start = start;
  a.max_pos = rope->max_pos;
  a.inverse = inverse;
  // 16-byte runs where every run starts on a 16-byte boundary and the table
  // row on one too; single pairs otherwise
  const int es = dtype == DSA_F32 ? 4 : 2, v = 16 / es;
  const uintptr_t at = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y);
  const bool wide = at % 16 == 0 && xt % v == 0 && xh % v == 0 && yt % v == 0 && yh % v == 0 && start % v == 0 &&
                    D % v == 0 && (a.R / 2) % v == 0;
  const int V = wide ? v : 1;
  a.npair = a.R / 2 / V;
  a.ncopy = x == y ? 0 : (D - a.R + 2 * V - 1) / (2 * V);
  const int items = a.npair + a.ncopy;
  // four heads a thread once there are many: 64 heads of 128 tokens 2.9 against
  // 2.7 us, of 256 2.8 against 3.5, of 2048 10.0 against 16.1
  const long long threads = static_cast<long long>(T) * H * items;
  const bool many = threads >= 768LL * ctx->num_sms && H >= 4;
  a.groups = many ? (H + 3) / 4 : H;
  const long long per = static_cast<long long>(items) * a.groups;
  if (per > 0x7FFFFFFFLL - 256) return DSA_ERR_UNSUPPORTED;
  a.tpb = per >= 256 ? 1 : static_cast<int>(256 / per);
  const long long by = per <= 256 ? 1 : (per + 255) / 256;
  const long long bx = (static_cast<long long>(T) + a.tpb - 1) / a.tpb;
  if (by > 65535) return DSA_ERR_UNSUPPORTED;
  LaunchScope scope(ctx, DSA_K_ROPE, stream);
  const bool il = rope->layout == DSA_ROPE_INTERLEAVED;
  const dim3 grid(static_cast<unsigned>(bx), static_cast<unsigned>(by));
  cudaError_t e;
  if (dtype == DSA_F32)
    e = wide ? launch<F32, 4>(a, il, many, grid, stream) : launch<F32, 1>(a, il, many, grid, stream);
  else if (dtype == DSA_F16)
    e = wide ? launch<F16, 8>(a, il, many, grid, stream) : launch<F16, 1>(a, il, many, grid, stream);
  else
    e = wide ? launch<Bf16, 8>(a, il, many, grid, stream) : launch<Bf16, 1>(a, il, many, grid, stream);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
