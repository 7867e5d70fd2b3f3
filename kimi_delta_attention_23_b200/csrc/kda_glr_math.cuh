// kda_glr_math.cuh -- the gate of the gated linear recurrence in packed two-lane fp32 arithmetic.
//
// The forward pass at HBM speed has about 13 issue slots per element and SM sub-core, so the gate is
// evaluated two channels at a time (fma.rn.f32x2 and friends), with two MUFU operations per element:
// e = 2^(-|z| log2 e) and a = 2^(g log2 e).  softplus(z) = max(z, 0) + log1p(e) takes log1p as e times a
// degree-7 polynomial: a logarithm of the rounded 1 + e would lose the gates of slow channels
// (softplus << 1), whose decays multiply up over thousands of tokens; decays near 1 come from a
// polynomial for the same reason.
//
// Both polynomials are weighted least-squares fits on Chebyshev nodes made for this file, with the
// largest relative error of their fp32 Horner evaluation beside them.
#pragma once

#include "kda_common.cuh"

namespace kda {
namespace glr {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kTiny = 1.17549435e-38f;  // the smallest normal fp32

__device__ __forceinline__ uint64_t as_u64(float2 x) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x.x), "f"(x.y));
  return r;
}
__device__ __forceinline__ float2 as_f2(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
  return as_f2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(r);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rsq(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// log2(1 + e) / e for e in [0, 1] (relative error 3.2e-7, about that of the hardware exponential)
__device__ __forceinline__ float2 log2_1p_ratio(float2 e) {
  float2 p = both(-0.0123193823f);
  p = fma2(p, e, both(0.0636075735f));
  p = fma2(p, e, both(-0.15535143f));
  p = fma2(p, e, both(0.25600943f));
  p = fma2(p, e, both(-0.353394717f));
  p = fma2(p, e, both(0.480063677f));
  p = fma2(p, e, both(-0.721310079f));
  return fma2(p, e, both(1.44269478f));
}

// (exp(y) - 1) / y for y in [-1/2, 0] (relative error 1.5e-7)
__device__ __forceinline__ float2 expm1_ratio(float2 y) {
  float2 p = both(0.00677103736f);
  p = fma2(p, y, both(0.0410012789f));
  p = fma2(p, y, both(0.166548148f));
  p = fma2(p, y, both(0.49999249f));
  return fma2(p, y, both(0.99999994f));
}

// What one head's gate needs besides the pre-activation: -exp(a_log), and the safe gate's bound times
// log2 e (-inf when there is none).
struct HeadGate {
  float c, lb2;
};
__device__ __forceinline__ HeadGate head_gate(float a_log, bool safe, float lb) {
  return {-expf(a_log), safe ? lb * kLog2e : -INFINITY};
}

// The gate is kept in units of log2: z2 = z log2 e from the raw value and the bias times log2 e, then
// e = exp(-|z|), then g log2 e = -exp(a_log) (max(z2, 0) + log2(1 + e)) before any clamp.
__device__ __forceinline__ float2 pre_log2(float2 raw, float2 bias2) { return fma2(raw, both(kLog2e), bias2); }
__device__ __forceinline__ float2 exp_neg_abs(float2 z2) { return make_float2(ex2(-fabsf(z2.x)), ex2(-fabsf(z2.y))); }
__device__ __forceinline__ float2 gate_log2(float2 z2, float2 e, float c) {
  return mul2(both(c), fma2(e, log2_1p_ratio(e), make_float2(fmaxf(z2.x, 0.f), fmaxf(z2.y, 0.f))));
}
// (a gate that is not a number stays one)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 clamp2(float2 g2, float lb2) {
  return make_float2(max_nan(g2.x, lb2), max_nan(g2.y, lb2));
}

// The decay a = 2^g2 and what it leaves, 1 - a.  Slow channels (a >= e^(-1/2)) take both from the
// polynomial: the hardware exponential is off by up to 2^-22, of a kind with the tokens' 1 - a there,
// and thousands of such decays multiply up.
struct Decay {
  float2 a, rest;
};
__device__ __forceinline__ Decay decay_of(float2 g2) {
  const float2 y = mul2(g2, both(kLn2)), m = mul2(y, expm1_ratio(y)), far = make_float2(ex2(g2.x), ex2(g2.y));
  const bool near_x = y.x > -0.5f, near_y = y.y > -0.5f;
  return {make_float2(near_x ? 1.f + m.x : far.x, near_y ? 1.f + m.y : far.y),
          make_float2(near_x ? -m.x : 1.f - far.x, near_y ? -m.y : 1.f - far.y)};
}
// 1 - a^2, at least the smallest normal number: a channel that is wide open (a = 1) so lets in 1e-19 of
// its input, which is nothing, and needs no case of its own.
__device__ __forceinline__ float2 one_minus_sq(const Decay& d) {
  const float2 u = fma2(d.rest, d.a, d.rest);
  return make_float2(fmaxf(u.x, kTiny), fmaxf(u.y, kTiny));
}
__device__ __forceinline__ float2 rsq2(float2 u) { return make_float2(rsq(u.x), rsq(u.y)); }

// sigmoid(x), or x itself where it is a probability already
__device__ __forceinline__ float beta_fast(float x, bool prob) { return prob ? x : rcp(1.f + ex2(-x * kLog2e)); }

// four consecutive channels of an input row in shared or global memory
__device__ __forceinline__ void unpack4(const __nv_bfloat16* p, float2& lo, float2& hi) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  lo = make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
  hi = make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void unpack4(const float* p, float2& lo, float2& hi) {
  const float4 w = *reinterpret_cast<const float4*>(p);
  lo = make_float2(w.x, w.y);
  hi = make_float2(w.z, w.w);
}
__device__ __forceinline__ uint32_t pack_bf16(float2 x) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x.y), "f"(x.x));
  return r;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float2 lo, float2 hi) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(lo), pack_bf16(hi));
}
__device__ __forceinline__ void store4(float* p, float2 lo, float2 hi) {
  *reinterpret_cast<float4*>(p) = make_float4(lo.x, lo.y, hi.x, hi.y);
}
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f32(float* p, float x) { *p = x; }

}  // namespace glr
}  // namespace kda
