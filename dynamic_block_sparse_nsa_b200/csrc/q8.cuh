// The 8-bit paged KV cache: its device view, e4m3 conversions, power-of-two
// block scales and the checks every kernel makes of a sequence.
//
// Cache: k_pages, v_pages [P, Hkv, page, d] e4m3 codes (one head's page is
// page * d contiguous bytes), k_scale, v_scale [P, Hkv] fp32: a component is
// code * scale. Token x of sequence b is slot x % page of page
// table[b, x / page].
#pragma once

#include <cuda_fp16.h>

#include "device_common.cuh"
#include "internal.h"

namespace nsa {
namespace q8 {

// Two e4m3 codes (low byte first) as halves; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return h;
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t c) {
  const uint32_t h = e4m3x2_to_half2(c);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Two fp32 values as e4m3 codes (lo in the low byte), to nearest with ties to
// even; NaN becomes the NaN code. Callers keep |x| <= 448.
__device__ __forceinline__ uint16_t float2_to_e4m3x2(float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}

// Exponent e of the smallest power of two 2^e >= 2^-126 with a <= 448 * 2^e
// (a >= 0 finite). 448 = 1.75 * 2^8, so with a = f * 2^x, 1 <= f < 2, that is
// x - 8, and one more when f > 1.75.
__device__ __forceinline__ int scale_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  const int x = (int)(u >> 23) - 127;  // a subnormal a gives -127, clamped below
  const int e = x - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <typename T>
struct Vec8;  // 8 elements, 16-byte accesses; Raw: as they are in memory
template <>
struct Vec8<__nv_bfloat16> {
  using Raw = uint4;
  static __device__ __forceinline__ Raw load_raw(const __nv_bfloat16* p) {
    return __ldg(reinterpret_cast<const uint4*>(p));
  }
  static __device__ __forceinline__ void unpack(const Raw& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* x) {
    unpack(load_raw(p), x);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec8<float> {
  struct Raw {
    float4 a, b;
  };
  static __device__ __forceinline__ Raw load_raw(const float* p) {
    const float4* q = reinterpret_cast<const float4*>(p);
    return Raw{__ldg(q), __ldg(q + 1)};
  }
  static __device__ __forceinline__ void unpack(const Raw& v, float* x) {
    *reinterpret_cast<float4*>(x) = v.a;
    *reinterpret_cast<float4*>(x + 4) = v.b;
  }
  static __device__ __forceinline__ void load(const float* p, float* x) {
    *reinterpret_cast<float4*>(x) = __ldg(reinterpret_cast<const float4*>(p));
    *reinterpret_cast<float4*>(x + 4) = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  static __device__ __forceinline__ void store(float* p, const float* x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// One sequence of a call: its tokens cu[b] .. cu[b + 1] - 1 of N (one token
// each, row b, when cu is null). False when the offsets are out of order.
__device__ __forceinline__ bool token_range(const int32_t* cu, int b, int N, int& first, int& n) {
  first = b;
  n = 1;
  if (!cu) return true;
  first = cu[b];
  const int end = cu[b + 1];
  n = 0;
  if (first < 0 || end < first || end > N) return false;
  n = end - first;
  return true;
}

}  // namespace q8
}  // namespace nsa
