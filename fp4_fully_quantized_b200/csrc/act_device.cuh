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
// Eight consecutive FP32 values as four pairs: one instruction multiplies or adds
// two of them (fma.rn.f32x2), each rounded as the scalar form rounds it.  The
// kernels that use this are bound by instruction issue where they are not bound
// by HBM.
// ---------------------------------------------------------------------------
typedef unsigned long long f32x2;
struct F8 { f32x2 p[4]; };

__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// ---------------------------------------------------------------------------
// Activations, two values at a time.  silu(z) = z p, p = 1 / (1 + exp(-z));
// gelu(z) = z Phi(z) with the normal CDF Phi; gelu_tanh(z) = z (1 + tanh u) / 2 =
// z p(2u), u = sqrt(2/pi) (z + 0.044715 z^3).  Exponential and reciprocal are the
// hardware's approximations (2 and 1 units in the last place, subnormals
// flushed).  With the roundings of the arguments a value is within (|t| + 4) 2^-20
// of itself (t = z or 2u), GELU within 2^-20 |z| and, left of zero, 2^-10 of
// itself: a quarter of a BF16 half-step or less, but some 16 (|t| + 4) half-steps
// of FP32, which the GEMM's epilogue may store.  z^2 is capped in gelu_tanh where
// p is 0 or 1 in binary32 anyway, so that a large z does not meet Inf * 0.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ f32x2 both(float v) { return pair(v, v); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTwoC = 1.5957691216057308f;          // 2 sqrt(2/pi)

// 1 / (1 + 2^t)
__device__ __forceinline__ f32x2 logistic2(f32x2 t) {
  const float2 x = unpair(t);
  const float2 d = unpair(add2(pair(ex2_approx(x.x), ex2_approx(x.y)), both(1.0f)));
  return pair(rcp_approx(d.x), rcp_approx(d.y));
}

// 1 for v >= 0, else 0, in one instruction.
__device__ __forceinline__ float step(float v) {
  float r;
  asm("set.ge.f32.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
  return r;
}

// Minus the upper normal tail, -Q(a) = Phi(a) - 1, and e = exp(-a^2/2) at
// a = min(|z|, 14): Q(a) = p(t) e with t = 1 / (1 + 0.33 a), the form that
// Hastings gave such approximations (Abramowitz and Stegun, 7.1.26, is one), and p
// of degree five with a constant term.  Its coefficients are a weighted minimax
// fit of exp(a^2/2) Q(a) on [0, 14] (a linear program): within 0.98e-7 of Q, 1.6
// units of FP32's last place at 1, and within 2^-10 of Q relative to
// it, where 7.1.26 itself (0.75e-7) is off by 0.16 % at a = 5, 1 % at 8 and 4 %
// at 14.  In FP32 arithmetic 2.4e-7.  e is the density's exponential too.
__device__ __forceinline__ void normal_tail2(float2 z, f32x2& a, f32x2& nq, f32x2& e) {
  a = pair(min_nan(fabsf(z.x), 14.0f), min_nan(fabsf(z.y), 14.0f));
  const float2 d = unpair(fma2(a, both(0.33f), both(1.0f)));
  const f32x2 t = pair(rcp_approx(d.x), rcp_approx(d.y));
  const float2 x = unpair(mul2(mul2(a, both(-0.5f * kLog2e)), a));
  e = pair(ex2_approx(x.x), ex2_approx(x.y));
  f32x2 q = fma2(t, both(0.115314774f), both(-0.398171842f));
  q = fma2(q, t, both(0.126772538f));
  q = fma2(q, t, both(-0.230730325f));
  q = fma2(q, t, both(-0.111643821f));
  q = fma2(q, t, both(-0.00154125539f));
  nq = mul2(q, e);
}

// act(z)
template <int ACT>
__device__ __forceinline__ f32x2 act_value2(f32x2 z) {
  if constexpr (ACT == FQT_ACT_NONE) return z;
  const float2 v = unpair(z);
  if constexpr (ACT == FQT_ACT_RELU) return pair(max_nan(v.x, 0.0f), max_nan(v.y, 0.0f));
  if constexpr (ACT == FQT_ACT_SILU) return mul2(z, logistic2(mul2(z, both(-kLog2e))));
  if constexpr (ACT == FQT_ACT_GELU) {
    // z Phi(z) = max(z, 0) - |z| Q(|z|)
    f32x2 a, nq, e;
    normal_tail2(v, a, nq, e);
    return fma2(a, nq, pair(fmaxf(v.x, 0.0f), fmaxf(v.y, 0.0f)));
  }
  if constexpr (ACT == FQT_ACT_GELU_TANH) {
    const float2 s = unpair(mul2(z, z));
    const f32x2 z2 = pair(fminf(s.x, 1e4f), fminf(s.y, 1e4f));
    return mul2(z, logistic2(mul2(z, fma2(z2, both(-kTwoC * kLog2e * 0.044715f), both(-kTwoC * kLog2e)))));
  }
}

// act(z) and act'(z)
template <int ACT>
__device__ __forceinline__ void act_both2(f32x2 z, f32x2& f, f32x2& df) {
  const float2 v = unpair(z);
  if constexpr (ACT == FQT_ACT_NONE) { f = z; df = both(1.0f); }
  if constexpr (ACT == FQT_ACT_RELU) {
    f = act_value2<ACT>(z);
    df = pair(v.x > 0.0f ? 1.0f : (v.x != v.x ? v.x : 0.0f), v.y > 0.0f ? 1.0f : (v.y != v.y ? v.y : 0.0f));
  }
  if constexpr (ACT == FQT_ACT_SILU) {
    const f32x2 p = logistic2(mul2(z, both(-kLog2e)));
    f = mul2(z, p);
    df = fma2(f, fma2(p, both(-1.0f), both(1.0f)), p);
  }
  if constexpr (ACT == FQT_ACT_GELU) {
    // Phi + z phi: 1 + (|z| phi - Q) right of zero, -(|z| phi - Q) left of it;
    // beyond |z| = 14 both are below 2^-126
    f32x2 a, nq, e;
    normal_tail2(v, a, nq, e);
    f = fma2(a, nq, pair(fmaxf(v.x, 0.0f), fmaxf(v.y, 0.0f)));
    const f32x2 right = pair(step(v.x), step(v.y));
    df = fma2(fma2(mul2(a, both(0.3989422804014327f)), e, nq), fma2(right, both(2.0f), both(-1.0f)), right);
  }
  if constexpr (ACT == FQT_ACT_GELU_TANH) {
    const float2 s = unpair(mul2(z, z));
    const f32x2 z2 = pair(fminf(s.x, 1e4f), fminf(s.y, 1e4f));
    const f32x2 p =
        logistic2(mul2(z, fma2(z2, both(-kTwoC * kLog2e * 0.044715f), both(-kTwoC * kLog2e))));
    f = mul2(z, p);
    const f32x2 slope = fma2(z2, both(kTwoC * 0.134145f), both(kTwoC));
    df = fma2(mul2(f, fma2(p, both(-1.0f), both(1.0f))), slope, p);
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

// Eight values rounded to BF16, packed.
__device__ __forceinline__ uint4 pack_bf16x8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// A running max |v| over packed BF16 values, two lanes; NaN stays.
struct AmaxBf16 {
  __nv_bfloat162 m = __nv_bfloat162(__float2bfloat16(0.0f), __float2bfloat16(0.0f));
  __device__ __forceinline__ void add(const uint4& u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
  }
  // into *dst (if not NULL), as binary32 bits: they order by magnitude, NaN on top
  __device__ __forceinline__ void to(float* dst) const {
    if (dst == nullptr) return;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&m);
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, max(w >> 16, w & 0xFFFFu) << 16);
    if ((threadIdx.x & 31) == 0) atomicMax(reinterpret_cast<unsigned int*>(dst), top);
  }
};

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

__device__ __forceinline__ F8 zero8() { return F8{{0ull, 0ull, 0ull, 0ull}}; }
__device__ __forceinline__ F8 scaled8(const F8& v, float k) {
  const f32x2 kk = pair(k, k);
  return F8{{mul2(v.p[0], kk), mul2(v.p[1], kk), mul2(v.p[2], kk), mul2(v.p[3], kk)}};
}

__device__ __forceinline__ F8 bf16x8(const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.p[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  return r;
}
__device__ __forceinline__ F8 e4m3x8(const uint2& q) {
  F8 r;
  float v[4];
  e4m3x4_to_f32(q.x, v);
  r.p[0] = pair(v[0], v[1]);
  r.p[1] = pair(v[2], v[3]);
  e4m3x4_to_f32(q.y, v);
  r.p[2] = pair(v[0], v[1]);
  r.p[3] = pair(v[2], v[3]);
  return r;
}
template <bool F32>
__device__ __forceinline__ F8 get8(const void* base, int64_t i) {
  if constexpr (F32) {
    const ulonglong2* p = reinterpret_cast<const ulonglong2*>(static_cast<const float*>(base) + i);
    const ulonglong2 a = p[0], b = p[1];
    return F8{{a.x, a.y, b.x, b.y}};
  } else {
    return bf16x8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + i));
  }
}
__device__ __forceinline__ uint4 pack_bf16x8(const F8& v) {
  uint4 u;
  float2 f = unpair(v.p[0]);
  u.x = pack_bf16x2(f.x, f.y);
  f = unpair(v.p[1]);
  u.y = pack_bf16x2(f.x, f.y);
  f = unpair(v.p[2]);
  u.z = pack_bf16x2(f.x, f.y);
  f = unpair(v.p[3]);
  u.w = pack_bf16x2(f.x, f.y);
  return u;
}
template <bool F32>
__device__ __forceinline__ void put8(void* base, int64_t i, const F8& v) {
  if constexpr (F32) {
    ulonglong2* p = reinterpret_cast<ulonglong2*>(static_cast<float*>(base) + i);
    p[0] = make_ulonglong2(v.p[0], v.p[1]);
    p[1] = make_ulonglong2(v.p[2], v.p[3]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + i) = pack_bf16x8(v);
  }
}

// A thread's eight values of a 32-column block (four neighbouring lanes hold it
// and call this together) to E4M3; false for a block with Inf or NaN.
__device__ __forceinline__ bool encode8(const F8& x, uint8_t* codes, uint8_t* scale, bool valid) {
  const float2 a = unpair(x.p[0]), b = unpair(x.p[1]), c = unpair(x.p[2]), d = unpair(x.p[3]);
  uint32_t m = abs_bits(max_abs3(max_abs3(max_abs3(max_abs3(0.0f, a.x, a.y), b.x, b.y), c.x, c.y), d.x, d.y));
  const uint32_t quad = 0xFu << (threadIdx.x & 28);
  m = max(m, __shfl_xor_sync(quad, m, 1));
  m = max(m, __shfl_xor_sync(quad, m, 2));
  const uint32_t byte = ckpt_scale_byte(m);
  if (valid) {
    const F8 v = scaled8(x, ckpt_inv_scale(byte));
    const float2 e = unpair(v.p[0]), f = unpair(v.p[1]), g = unpair(v.p[2]), h = unpair(v.p[3]);
    *reinterpret_cast<uint2*>(codes) = make_uint2(e4m3x4_rn(e.x, e.y, f.x, f.y), e4m3x4_rn(g.x, g.y, h.x, h.y));
    if ((threadIdx.x & 3) == 0) *scale = (uint8_t)byte;
  }
  return byte != kCkptNanScale;
}

}  // namespace fp4dev
