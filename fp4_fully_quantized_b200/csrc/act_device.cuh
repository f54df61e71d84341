// act_device.cuh -- activations with their derivatives, and the 8-bit block
// format of activation checkpoints (sm_100a).
//
// The 8-bit format: 32 consecutive values of a row share the power of two 2^e
// with the least e (>= -127) that gives max <= 448 * 2^e, stored as E8M0
// (byte e + 127); each value is E4M3 (4 significant bits, largest 448) of
// value * 2^-e, rounded to nearest even, so no finite value saturates and a
// value within 2^-13 of the block maximum keeps a relative error of at most 2^-4.
// (The power-of-two rule of the MX formats, floor(log2 max) - 8, would clip
// block maxima above 448 * 2^e by up to 1/8.)  A block that holds Inf or NaN
// gets scale byte 255, E8M0's NaN: it decodes to NaN as a whole, never to
// plausible values.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp4.h"
#include "fp4_device.cuh"

namespace fp4dev {

constexpr uint32_t kCkptNanScale = 255u;

// Scale byte from the block's max |v| given as binary32 bits without the sign
// (an integer compare orders them and keeps NaN on top).
__device__ __forceinline__ uint32_t ckpt_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return kCkptNanScale;
  const int e = (int)(amax_bits >> 23) - 135 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return amax_bits == 0u ? 0u : (uint32_t)(max(e, -127) + 127);
}

// 2^-e for a scale byte e + 127 in [0, 254] (exact; NaN for byte 255).
__device__ __forceinline__ float ckpt_inv_scale(uint32_t byte) {
  return byte == kCkptNanScale ? __uint_as_float(0x7FC00000u) : __uint_as_float((254u - byte) << 23);
}

// 2^e (exact, subnormal for byte 0; NaN for byte 255).
__device__ __forceinline__ float ckpt_scale(uint32_t byte) {
  if (byte == 0u) return __uint_as_float(1u << 22);
  return byte == kCkptNanScale ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte << 23);
}

// Four floats -> four E4M3 codes, element k in byte k.
__device__ __forceinline__ uint32_t e4m3x4_rn(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Four E4M3 codes -> four floats (exact: E4M3 widens to FP16 without loss).
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float* v) {
  uint32_t h0, h1;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"((uint16_t)(w & 0xFFFFu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"((uint16_t)(w >> 16)));
  const float2 f0 = __half22float2(*reinterpret_cast<__half2*>(&h0));
  const float2 f1 = __half22float2(*reinterpret_cast<__half2*>(&h1));
  v[0] = f0.x; v[1] = f0.y; v[2] = f1.x; v[3] = f1.y;
}

// max(m, |a|, |b|) for m >= 0, NaN if one of them is.
__device__ __forceinline__ float max_abs3(float m, float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// ---------------------------------------------------------------------------
// Activations.  silu(z) = z p, p = 1 / (1 + exp(-z)); gelu(z) = z Phi(z) with
// the normal CDF Phi; gelu_tanh(z) = z (1 + tanh u) / 2 = z p(2u),
// u = sqrt(2/pi) (z + 0.044715 z^3).  The exponential and the quotient are the
// fast forms (relative error about 2^-21 over the range where p matters,
// against 2^-9 of the BF16 result).  z^2 is capped in gelu_tanh where p is
// 0 or 1 in binary32 anyway, so that a large z does not meet Inf * 0.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float logistic(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

// The normal CDF and e = exp(-z^2/2), by the rational approximation of erfc of
// Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26: for x >= 0
// erfc(x) = (a1 t + ... + a5 t^5) exp(-x^2), t = 1 / (1 + 0.3275911 x), to
// 1.5e-7, with x = |z| / sqrt(2) (so the exponential is the density's too, and
// the lower tail is not a difference).  An absolute error of 0.75e-7 is one
// and a quarter units of FP32's last place at 1.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float t = __fdividef(1.0f, 1.0f + 0.23164190f * fabsf(z));   // 0.3275911 / sqrt(2)
  e = __expf(-0.5f * z * z);
  float q = 1.061405429f;
  q = q * t - 1.453152027f;
  q = q * t + 1.421413741f;
  q = q * t - 0.284496736f;
  q = q * t + 0.254829592f;
  const float tail = 0.5f * (q * t) * e;
  return z < 0.0f ? tail : 1.0f - tail;
}

constexpr float kTwoC = 1.5957691216057308f;          // 2 sqrt(2/pi)

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == FQT_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
  if constexpr (ACT == FQT_ACT_SILU) return z * logistic(z);
  if constexpr (ACT == FQT_ACT_GELU) {
    float e;
    return z * normal_cdf(z, e);
  }
  if constexpr (ACT == FQT_ACT_GELU_TANH)
    return z * logistic(kTwoC * z * (1.0f + 0.044715f * fminf(z * z, 1e4f)));
  return z;
}

// The value and the derivative at z.
template <int ACT>
__device__ __forceinline__ void act_both(float z, float& f, float& df) {
  if constexpr (ACT == FQT_ACT_NONE) { f = z; df = 1.0f; }
  if constexpr (ACT == FQT_ACT_RELU) {
    f = z > 0.0f ? z : (z != z ? z : 0.0f);
    df = z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  }
  if constexpr (ACT == FQT_ACT_SILU) {
    const float p = logistic(z);
    f = z * p;
    df = p + f * (1.0f - p);
  }
  if constexpr (ACT == FQT_ACT_GELU) {
    float e;
    const float cdf = normal_cdf(z, e);
    f = z * cdf;
    df = cdf + z * (0.3989422804014327f * e);
  }
  if constexpr (ACT == FQT_ACT_GELU_TANH) {
    const float z2 = fminf(z * z, 1e4f);
    const float p = logistic(kTwoC * z * (1.0f + 0.044715f * z2));
    f = z * p;
    df = p + f * (1.0f - p) * (kTwoC * (1.0f + 0.134145f * z2));
  }
}

// ---------------------------------------------------------------------------
// Eight consecutive values of a row <-> memory (16-byte aligned).
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}
__device__ __forceinline__ uint2 ld_stream2(const void* p) {
  uint2 r;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
               : "=r"(r.x), "=r"(r.y) : "l"(p) : "memory");
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Rounds v to BF16, in place, and returns the packed words.
__device__ __forceinline__ uint4 pack_bf16x8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// max |v| of eight packed BF16 values, as binary32 bits.
__device__ __forceinline__ uint32_t amax_bits_bf16x8(const uint4& u) {
  const uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu),
                              __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
  return max(m >> 16, m & 0xFFFFu) << 16;
}

// Eight consecutive values at element i of a BF16 or FP32 array (16-byte aligned).
__device__ __forceinline__ void load8(const void* base, int64_t i, bool f32, float* v) {
  if (f32) {
    const float4 a = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i)[0];
    const float4 b = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    bf16x8_to_f32(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + i), v);
  }
}

__device__ __forceinline__ void store8(void* base, int64_t i, bool f32, const float* v) {
  if (f32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + i) = pack_bf16x8(v);
  }
}

// A thread's eight values of a 32-column block (four neighbouring lanes hold it;
// every lane of the warp calls this) to E4M3; false for a block with Inf or NaN.
__device__ __forceinline__ bool encode8(const float* v, uint8_t* codes, uint8_t* scale, bool valid) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  const uint32_t byte = ckpt_scale_byte(m);
  const float inv = ckpt_inv_scale(byte);
  if (valid) {
    *reinterpret_cast<uint2*>(codes) =
        make_uint2(e4m3x4_rn(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                   e4m3x4_rn(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
    if ((threadIdx.x & 3) == 0) *scale = (uint8_t)byte;
  }
  return byte != kCkptNanScale;
}

}  // namespace fp4dev
