// The K/V cache's page layout and its fp8 / fp4 codes.
//
// A page holds 64 tokens. It is one block per kv head, and a head's block is
//   K codes [64][CB]  V codes [64][CB]  K scales [64][D/32]  V scales [64][D/32]
// (no scales in bf16), so one head's keys of a page are one contiguous tile.
// In fp8 (e4m3) and fp4 (e2m1) 32 dimensions share a power-of-two scale, a
// byte holding its exponent + 127: the OCP microscaling formats MXFP8 and
// MXFP4, with the exponent rounded up so that no value saturates below the
// largest scale (448 * 2^119, 6 * 2^125). A stored value is then a bf16 number
// exactly: a code has at most 4 significant bits and the scale moves only the
// exponent. Reading back loses nothing, and the attention's bf16 tensor-core
// operands are the stored values themselves.
#pragma once
#include <cuda_bf16.h>

#include "internal.cuh"

namespace dsa {
namespace kvf {

constexpr int kPage = 64;
constexpr int kBlock = 32;  // dimensions that share a scale

template <int FMT, int D>
struct Layout {
  static constexpr int CB = FMT == DSA_FMT_BF16 ? 2 * D : FMT == DSA_FMT_FP8 ? D : D / 2;  // code bytes a row
  static constexpr int SB = FMT == DSA_FMT_BF16 ? 0 : D / kBlock;                          // scale bytes a row
  static constexpr int K_CODES = 0;
  static constexpr int V_CODES = kPage * CB;
  static constexpr int K_SCALES = 2 * kPage * CB;
  static constexpr int V_SCALES = 2 * kPage * CB + kPage * SB;
  static constexpr int HEAD_BYTES = 2 * kPage * (CB + SB);
};

// Exponent limits: the smallest keeps every code's value a normal bf16
// number, the largest keeps the largest code finite in bf16.
template <int FMT>
struct Scale {
  static constexpr int LO = FMT == DSA_FMT_FP8 ? -117 : -125;
  static constexpr int HI = FMT == DSA_FMT_FP8 ? 119 : 125;
  // smallest e with amax <= MAX 2^e, MAX = 448 = 1.75 2^8 or 6 = 1.5 2^2,
  // from amax's bits (finite): its exponent, one more if the mantissa is above MAX's
  static __device__ __forceinline__ int exponent(uint32_t amax) {
    const int e = static_cast<int>(amax >> 23) - 127 - (FMT == DSA_FMT_FP8 ? 8 : 2) +
                  ((amax & 0x7FFFFFu) > (FMT == DSA_FMT_FP8 ? 0x600000u : 0x400000u) ? 1 : 0);
    return min(max(e, LO), HI);
  }
};

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  __nv_bfloat162 x, y;
  memcpy(&x, &a, 4);
  memcpy(&y, &b, 4);
  const __nv_bfloat162 r = __hmul2_rn(x, y);
  uint32_t o;
  memcpy(&o, &r, 4);
  return o;
}

// The factors that turn a code placed in a bf16's bits into its value. The
// code's sign, exponent and mantissa are moved to where bf16 has them; read
// as bf16 that is value * 2^-BIAS (the subnormal codes too, as bf16
// subnormals), so one multiplication by 2^(BIAS + e) gives the value,
// exactly. Above 2^127 it takes two. Scale byte 255 stands for NaN.
template <int FMT>
struct Factor {
  static constexpr int BIAS = FMT == DSA_FMT_FP8 ? 120 : 126;
  static constexpr uint32_t ONE = 254 - BIAS;  // the largest scale byte one factor covers
  uint32_t f;  // bf16x2 factor
  __device__ __forceinline__ void set(uint32_t byte) { f = (min(byte, ONE) + BIAS) * 0x00800080u; }
  // scales above 2^7 (fp8) or 2 (fp4), and NaN, take a second factor: rare
  static __device__ __forceinline__ bool two(uint32_t byte) { return byte > ONE; }
  template <int N>
  static __device__ __forceinline__ void rest(uint32_t byte, uint32_t (&r)[N]) {
    if (two(byte)) {
      const uint32_t g = byte == 255u ? 0x7FFF7FFFu : (byte + 127 - ONE) * 0x00800080u;
#pragma unroll
      for (int i = 0; i < N; ++i) r[i] = mul_bf16x2(r[i], g);
    }
  }
};

// two bytes of a and b (0-3 and 4-7), each sign-extended to 16 bits: selectors
// 8 | i stand for eight copies of byte i's sign
__device__ __forceinline__ uint32_t sext2(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// N words of four e4m3 codes -> bf16 pairs, up to the second factor. A code
// sign-extended to 16 bits and shifted by 4 has its sign, exponent and
// mantissa where bf16 has them; the bits between are cleared.
template <int N>
__device__ __forceinline__ void widen(const uint32_t (&w)[N], const Factor<DSA_FMT_FP8>& s, uint32_t (&o)[2 * N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    o[2 * i] = mul_bf16x2((sext2(w[i], w[i], 0x9180) << 4) & 0x87F087F0u, s.f);
    o[2 * i + 1] = mul_bf16x2((sext2(w[i], w[i], 0xB3A2) << 4) & 0x87F087F0u, s.f);
  }
}

// N words of eight e2m1 codes (the even dimension in the low nibble) -> bf16
// pairs, up to the second factor. Likewise, with a code in a byte's high
// nibble: the odd ones as they are, the even ones in the word shifted by 4.
template <int N>
__device__ __forceinline__ void widen(const uint32_t (&w)[N], const Factor<DSA_FMT_FP4>& s, uint32_t (&o)[4 * N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t even = w[i] << 4;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[4 * i + j] = mul_bf16x2((sext2(even, w[i], 0xC480 + 0x1111 * j) << 2) & 0x81C081C0u, s.f);
  }
}

// bf16 pairs: what is not finite becomes zero; whether anything did
template <int N>
__device__ __forceinline__ bool zero_nonfinite(uint32_t (&w)[N]) {
  bool found = false;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if ((w[j] & 0x7F800000u) == 0x7F800000u) {
      w[j] &= 0x0000FFFFu;
      found = true;
    }
    if ((w[j] & 0x7F80u) == 0x7F80u) {
      w[j] &= 0xFFFF0000u;
      found = true;
    }
  }
  return found;
}

}  // namespace kvf
}  // namespace dsa
