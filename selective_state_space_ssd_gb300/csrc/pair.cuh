// Two fp32 numbers in one register pair, and operations on both at once.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace ssd {

struct P {
  float2 v;
};
__device__ __forceinline__ P pair(float x, float y) { return P{make_float2(x, y)}; }
__device__ __forceinline__ P both(float x) { return pair(x, x); }
__device__ __forceinline__ void split(P p, float& x, float& y) { x = p.v.x, y = p.v.y; }
__device__ __forceinline__ float low(P p) { return p.v.x; }
__device__ __forceinline__ P fma(P a, P b, P c) { return P{__ffma2_rn(a.v, b.v, c.v)}; }
__device__ __forceinline__ P operator*(P a, P b) { return P{__fmul2_rn(a.v, b.v)}; }
__device__ __forceinline__ P operator+(P a, P b) { return P{__fadd2_rn(a.v, b.v)}; }
__device__ __forceinline__ P less(P a, P b) { return fma(b, both(-1.f), a); }  // a - b
template <typename F>
__device__ __forceinline__ P each(P p, const F& f) {
  float x, y;
  split(p, x, y);
  return pair(f(x), f(y));
}

__device__ __forceinline__ float exp2_f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float inv_f(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sqrt_f(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rsqrt_f(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The smaller one, the greater one; NaN if one is.
__device__ __forceinline__ float min_nan(float x, float y) {
  float z;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ float max_nan(float x, float y) {
  float z;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ P exp_neg(P z) {  // e^-z (infinity from about -88 on, where s is 0)
  return each(z * both(-kLog2e), [](float x) { return exp2_f(x); });
}
__device__ __forceinline__ P inv_one_more(P x) {
  return each(x + both(1.f), [](float v) { return inv_f(v); });
}
__device__ __forceinline__ P sigmoid(P z) { return inv_one_more(exp_neg(z)); }
__device__ __forceinline__ P one_less(P x) { return fma(x, both(-1.f), both(1.f)); }
__device__ __forceinline__ P one_more(P x) { return x + both(1.f); }

}  // namespace ssd
