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
// is shared by its heads through L1/L2).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <new>
#include <vector>

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

// element types: 16-byte (or single-element) loads to fp32 and back
struct Bf16 {
  using type = __nv_bfloat16;
  static __device__ __forceinline__ float up(type v) { return __bfloat162float(v); }
  static __device__ __forceinline__ type down(float v) { return __float2bfloat16_rn(v); }
};
struct F16 {
  using type = __half;
  static __device__ __forceinline__ float up(type v) { return __half2float(v); }
  static __device__ __forceinline__ type down(float v) { return __float2half_rn(v); }
};
struct F32 {
  using type = float;
  static __device__ __forceinline__ float up(type v) { return v; }
  static __device__ __forceinline__ type down(float v) { return v; }
};

template <typename E, int V>
struct alignas(sizeof(typename E::type) * V) Pack {
  typename E::type v[V];
};

struct RopeArgs {
  const void* x;
  void* y;
  const int32_t* pos;
  const float2* table;
  unsigned int* status;
  long long xt, xh, yt, yh;  // strides, in elements
  int T, H, D, R, start, max_pos, inverse;
  int npair;   // items that rotate V pairs of a head
  int ncopy;   // items that copy 2 V untouched elements of a head (0 in place)
  int groups;  // threads share a token's heads: each takes heads g, g + groups, ...
  int tpb;     // tokens per block (>= 1)
};

// One thread: V pairs (or 2 V untouched elements) of up to HPT heads of one
// token, so that the cos/sin it loads serve all of them and 2 HPT loads are
// in flight. V is 16 bytes' worth of elements where sizes, offsets and
// addresses allow, else 1.
template <typename E, int V, int HPT, bool INTERLEAVED>
__global__ void __launch_bounds__(256) rope_kernel(RopeArgs a) {
  pdl_wait();
  pdl_trigger();
  using P = Pack<E, V>;
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
  int e0, e1;  // the item's two runs of V elements
  float c[V], s[V];
  const bool rot = item < a.npair;
  if (rot) {
    const float2* tab = a.table + static_cast<long long>(pos) * (a.R >> 1) + item * V;
    if constexpr (V >= 2) {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(tab + i));
        c[i] = w.x;
        s[i] = w.y;
        c[i + 1] = w.z;
        s[i + 1] = w.w;
      }
    } else {
      const float2 w = __ldg(tab);
      c[0] = w.x;
      s[0] = w.y;
    }
    if (a.inverse) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = -s[i];
    }
    e0 = a.start + (INTERLEAVED ? 2 : 1) * item * V;
    e1 = INTERLEAVED ? e0 + V : e0 + (a.R >> 1);
  } else {
    e0 = (item - a.npair) * 2 * V;
    e1 = e0 + V;
    if (e0 >= a.start) e0 += a.R;
    if (e1 >= a.start) e1 += a.R;
  }
  for (int h0 = g; h0 < a.H; h0 += a.groups * HPT) {
    P p0[HPT], p1[HPT];
#pragma unroll
    for (int j = 0; j < HPT; ++j) {
      const int h = h0 + j * a.groups;
      if (h < a.H) {
        if (e0 < a.D) p0[j] = *reinterpret_cast<const P*>(x + h * a.xh + e0);
        if (e1 < a.D) p1[j] = *reinterpret_cast<const P*>(x + h * a.xh + e1);
      }
    }
#pragma unroll
    for (int j = 0; j < HPT; ++j) {
      const int h = h0 + j * a.groups;
      if (h >= a.H) continue;
      if (rot) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          // interleaved: the two runs hold 2 V consecutive elements, pair i at 2 i
          El& ea = INTERLEAVED ? (2 * i < V ? p0[j] : p1[j]).v[(2 * i) % V] : p0[j].v[i];
          El& eb = INTERLEAVED ? (2 * i + 1 < V ? p0[j] : p1[j]).v[(2 * i + 1) % V] : p1[j].v[i];
          const float u = E::up(ea), w = E::up(eb);
          ea = E::down(__fsub_rn(__fmul_rn(u, c[i]), __fmul_rn(w, s[i])));
          eb = E::down(__fadd_rn(__fmul_rn(w, c[i]), __fmul_rn(u, s[i])));
        }
      }
      if (e0 < a.D) *reinterpret_cast<P*>(y + h * a.yh + e0) = p0[j];
      if (e1 < a.D) *reinterpret_cast<P*>(y + h * a.yh + e1) = p1[j];
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
  std::vector<double> f(half);
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
            cudaMemcpy(df, f.data(), half * sizeof(double), cudaMemcpyHostToDevice) == cudaSuccess;
  if (ok) {
    const size_t blocks = (n + 255) / 256;
    rope_table_kernel<<<static_cast<unsigned>(blocks < 4096 ? blocks : 4096), 256>>>(df, half, d.max_pos, d.mscale,
                                                                                    r->table);
    ok = cudaGetLastError() == cudaSuccess && cudaDeviceSynchronize() == cudaSuccess;
  }
  cudaFree(df);
  if (!ok) {
    cudaFree(r->table);
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
  // four heads a thread once that still leaves two waves of threads
  const long long threads = static_cast<long long>(T) * H * items;
  const bool many = threads / 4 >= 2LL * ctx->num_sms * 2048 && H >= 4;
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
